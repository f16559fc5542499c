"""What is timed of the 8-bit latent cache: writing it, reading it back, and decoding over it.

An 8-bit cache is a pool of blocks of 128 tokens, 74240 bytes each: per token 576 e4m3 values (the latent
c^KV, 512, and the rotated RoPE key k^R, 64) and one fp32 scale, a power of two.  Byte of column c of row r:

    c <  512: (c / 128) * 16384 + r * 128 + (((c % 128) / 16) ^ (r % 8)) * 16 + c % 16
    c >= 512: 65536 + r * 64 + (((c - 512) / 16) ^ (r / 2 % 4)) * 16 + c % 16

and the scale of row r is the float at byte 73728 + 4 r.  A block table gives each sequence its blocks.

``append``: T new tokens are rotated, quantised and written.  ``read``: whole sequences are brought back
into a bf16 pool.  ``decode``: absorbed attention of n_q new tokens a sequence over the 8-bit cache, then
W^UV.
"""

import random

import torch

own = False

D_C, D_R, D_H, ROW = 512, 64, 128, 576
TOK = 128                   # tokens of a block
BLOCK8, CODES8 = 74240, 73728
BLOCK = 147456              # bytes of a bf16 block
SCALE = 192 ** -0.5
LEAST, MOST = 2.0 ** -40, 448.0


def listed():
    return [
        # one sequence's new token, one layer: the smallest write, all latency
        {"name": "append_1", "op": "append", "T": 1, "B": 1, "n_q": 1, "pos_hi": 4096},
        # a decode step of 128 sequences with two tokens each
        {"name": "append_step", "op": "append", "T": 256, "B": 128, "n_q": 2, "pos_hi": 32768},
        # a long prompt (an odd number of tokens) written at once
        {"name": "append_prompt", "op": "append", "T": 32749, "B": 1, "n_q": 0, "pos_hi": 0},
        # one sequence's prefix brought back before its next prefill chunk
        {"name": "read_prefix", "op": "read", "B": 1, "lo": 8192, "hi": 8192, "lens": 1},
        # a ragged batch moved to a bf16 pool
        {"name": "read_ragged", "op": "read", "B": 33, "lo": 1, "hi": 32768, "lens": 2},
        # one short sequence, 16 heads: latency
        {"name": "decode_tiny", "op": "decode", "B": 1, "H": 16, "n_q": 1, "lo": 256, "hi": 256, "lens": 1},
        # 16 heads, a full serving batch
        {"name": "decode_v2lite", "op": "decode", "B": 64, "H": 16, "n_q": 1, "lo": 4096, "hi": 4096, "lens": 1},
        # 128 heads, a serving batch at 8K
        {"name": "decode_v2", "op": "decode", "B": 32, "H": 128, "n_q": 1, "lo": 8192, "hi": 8192, "lens": 1},
        # few long sequences: the split over the long axis carries it
        {"name": "decode_128k", "op": "decode", "B": 4, "H": 128, "n_q": 1, "lo": 131072, "hi": 131072, "lens": 1},
        # a ragged serving batch with one speculated token each: the largest
        {"name": "decode_ragged", "op": "decode", "B": 128, "H": 128, "n_q": 2, "lo": 1, "hi": 32768, "lens": 3},
        # a prompt's chunk against its prefix, few heads, odd sizes
        {"name": "decode_chunk", "op": "decode", "B": 2, "H": 20, "n_q": 101, "lo": 5000, "hi": 7001, "lens": 4},
        # short ragged sequences, an odd number of heads
        {"name": "decode_short", "op": "decode", "B": 37, "H": 11, "n_q": 3, "lo": 1, "hi": 700, "lens": 5},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "decode", "decode"])
    if op == "append":
        if rng.random() < 0.5:      # a step: n_q tokens of each of B sequences
            B, n_q = _log(rng, 1, 256), rng.choice([1, 1, 2, 3, 5])
            return {"op": op, "T": B * n_q, "B": B, "n_q": n_q, "pos_hi": _log(rng, 16, 131072)}
        return {"op": op, "T": _log(rng, 2, 32749), "B": 1, "n_q": 0, "pos_hi": 0}
    if op == "read":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, min(131072, 500000 // B))
        return {"op": op, "B": B, "lo": rng.randint(1, hi), "hi": hi, "lens": rng.randrange(1 << 20)}
    while True:
        B, n_q = _log(rng, 1, 160), rng.choice([1, 1, 1, 2, 3, _log(rng, 4, 256)])
        H = rng.choice([1, 8, 16, 32, 64, 128, 128, rng.randint(1, 128)])
        hi = _log(rng, n_q, 131072)
        if B * hi <= 1500000 and B * hi * n_q * H <= 400000000:
            return {"op": op, "B": B, "H": H, "n_q": n_q, "lo": rng.randint(1, hi), "hi": hi,
                    "lens": rng.randrange(1 << 20)}


def _lengths(case):
    r = random.Random(case["lens"])
    least = case.get("n_q", 1)
    return [max(least, r.randint(case["lo"], case["hi"])) for _ in range(case["B"])]


def work(case):
    if case["op"] == "append":
        T = case["T"]
        return {"bytes": T * (2 * ROW + 8 + 4 * D_R + ROW + 4), "flops": T * (3 * ROW + 6 * D_R // 2)}
    n = sum(_lengths(case))
    if case["op"] == "read":
        return {"bytes": n * (ROW + 4 + 2 * ROW), "flops": n * ROW}
    H, rows = case["H"], case["n_q"] * case["H"]
    R = case["B"] * rows
    return {"bytes": n * (ROW + 4) + R * (2 * ROW + 2 * D_H + 4) + 2 * H * D_H * D_C,
            "flops": 2 * n * rows * (ROW + D_C) + 2 * R * D_C * D_H}


# ------------------------------------------------------------------ layout

def _map8(dev):
    """[128, 576] byte offset of (row, column) in a block of the 8-bit pool."""
    r, c = torch.arange(TOK, device=dev)[:, None], torch.arange(ROW, device=dev)[None, :]
    lat = (c // 128) * 16384 + r * 128 + (((c % 128) // 16) ^ (r % 8)) * 16 + c % 16
    rope = 65536 + r * 64 + ((((c - D_C) // 16) % 4) ^ ((r // 2) % 4)) * 16 + c % 16
    return torch.where(c < D_C, lat, rope)


def _map16(dev):
    """[128, 576] element offset of (row, column) in a block of the bf16 pool."""
    r, c = torch.arange(TOK, device=dev)[:, None], torch.arange(ROW, device=dev)[None, :]
    return ((c // 64) * 16384 + r * 128 + (((c % 64) // 8) ^ (r % 8)) * 16 + (c % 8) * 2) // 2


def _table(lengths, g, dev):
    """Blocks of one pool handed out in random order: int32 [B, max_blocks] (unused entries -1), pool size."""
    n = [-(-x // TOK) for x in lengths]
    perm = torch.randperm(sum(n) + len(n), generator=g, device=dev).to(torch.int32)
    tab = torch.full((len(n), max(n)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(n):
        tab[b, :k] = perm[at:at + k]
        at += k
    return tab, sum(n) + len(n)


def _quantise(x):
    """Rows of fp32 x -> (e4m3 codes, power-of-two scales)."""
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    m, e = torch.frexp(top / MOST)              # top / 448 = m 2^e, 0.5 <= m < 1
    s = torch.ldexp(torch.ones_like(top), torch.where(m == 0.5, e - 1, e))
    s = torch.where(top > 0, s.clamp_min(LEAST), 1.0)
    y = torch.where(torch.isfinite(x), x / s[..., None], float("nan"))
    return y.to(torch.float8_e4m3fn), s


def _views(pool):
    """The e4m3 values and the scales that an 8-bit pool holds."""
    return pool[:, :CODES8].view(torch.float8_e4m3fn), pool[:, CODES8:].view(torch.float32)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed * 1000003 + 17)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": case}
    if case["op"] == "append":
        T, B = case["T"], case["B"]
        if case["n_q"]:         # n_q tokens at the end of every sequence
            r = random.Random(seed)
            first = [r.randint(0, case["pos_hi"] - 1) for _ in range(B)]
            seq = [b for b in range(B) for _ in range(case["n_q"])]
            pos = [first[b] + j for b in range(B) for j in range(case["n_q"])]
            top, cap = case["pos_hi"] + case["n_q"], 2 * B + 1
        else:                   # a whole prompt
            seq, pos = [0] * T, list(range(T))
            top, cap = T, -(-T // TOK) + 1
        # the pool holds the blocks that are written; a table row's other entries are not read
        used = sorted({(b, p // TOK) for b, p in zip(seq, pos)})
        s["table"] = torch.full((B, -(-top // TOK)), -1, dtype=torch.int32)
        order = random.Random(seed + 1).sample(range(cap), len(used))
        for (b, k), blk in zip(used, order):
            s["table"][b, k] = blk
        s["table"] = s["table"].to(dev)
        s["seq"] = torch.tensor(seq, dtype=torch.int32, device=dev)
        s["pos"] = torch.tensor(pos, dtype=torch.int32, device=dev)
        s["c_kv"] = (rand(T, D_C) * torch.exp(0.3 * rand(T, 1))).bfloat16()
        s["k_rope"] = rand(T, D_R).bfloat16()
        ang = torch.arange(top, device=dev, dtype=torch.float64)[:, None] * \
            10000.0 ** (-2.0 * torch.arange(D_R // 2, device=dev, dtype=torch.float64) / D_R)
        s["rope"] = torch.stack([ang.cos(), ang.sin()], -1).reshape(top, D_R).float().contiguous()
        s["pool"] = torch.zeros(cap, BLOCK8, dtype=torch.uint8, device=dev)
        return s
    lengths = _lengths(case)
    s["lengths"] = lengths
    s["kv_len"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    s["table"], cap = _table(lengths, g, dev)
    pool = torch.zeros(cap, BLOCK8, dtype=torch.uint8, device=dev)
    at = _map8(dev).reshape(-1)
    for i in range(0, cap, 512):
        n = min(512, cap - i)
        amp = torch.exp(0.3 * rand(n * TOK, 1))
        codes, scales = _quantise((rand(n * TOK, ROW) * amp).bfloat16().float())
        part = torch.zeros(n, CODES8, dtype=torch.uint8, device=dev)
        part[:, at] = codes.view(torch.uint8).reshape(n, -1)
        pool[i:i + n, :CODES8] = part
        pool[i:i + n, CODES8:] = scales.reshape(n, TOK).contiguous().view(torch.uint8)
    s["pool"] = pool
    if case["op"] == "read":
        s["table16"], cap16 = _table(lengths, g, dev)
        s["pool16"] = torch.zeros(cap16, BLOCK, dtype=torch.uint8, device=dev)
        return s
    B, H, n_q = case["B"], case["H"], case["n_q"]
    q = rand(B * n_q, H, ROW)
    q[..., :D_C] *= 0.5             # (W^UK_h)^T q^C: 128 terms of variance 1/512
    s["q"] = q.bfloat16()
    s["W_UV"] = (rand(H, D_H, D_C) * D_C ** -0.5).bfloat16()
    s["out"] = torch.empty(B * n_q, H, D_H, dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.empty(B * n_q, H, dtype=torch.float32, device=dev)
    if own:
        import mla_latent_kv_34_b200 as mla
        s["workspace"] = torch.empty(mla.decode8_workspace_bytes(B, n_q, H), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if own:
        return _own(s)
    return {"append": _append, "read": _read, "decode": _decode}[case["op"]](s)


def _own(s):
    import mla_latent_kv_34_b200 as mla
    case = s["case"]
    if case["op"] == "append":
        mla.append_cache8(s["pool"], s["table"], s["seq"], s["pos"], s["c_kv"], s["k_rope"], s["rope"])
        return _views(s["pool"])
    if case["op"] == "read":
        mla.read_cache8(s["pool"], s["table"], s["kv_len"], s["pool16"], s["table16"])
        return s["pool16"].view(torch.bfloat16)
    mla.decode8(s["q"], s["pool"], s["table"], s["kv_len"], s["W_UV"], case["n_q"], SCALE,
                workspace=s["workspace"], out=s["out"], lse_out=s["lse"])
    return s["out"], s["lse"]


def _append(s):
    cs = s["rope"][s["pos"].long()].reshape(-1, D_R // 2, 2)
    x = s["k_rope"].float().reshape(-1, D_R // 2, 2)
    y0 = x[..., 0] * cs[..., 0] - x[..., 1] * cs[..., 1]
    y1 = x[..., 0] * cs[..., 1] + x[..., 1] * cs[..., 0]
    k = torch.stack([y0, y1], -1).reshape(-1, D_R).bfloat16()
    codes, scales = _quantise(torch.cat([s["c_kv"], k], -1).float())
    blk = s["table"][s["seq"].long(), (s["pos"] // TOK).long()].long()
    row = (s["pos"] % TOK).long()
    pool = s["pool"]
    pool[blk[:, None], _map8(pool.device)[row]] = codes.view(torch.uint8)
    _views(pool)[1][blk, row] = scales
    return _views(pool)


def _rows(s, b, dtype=torch.float32):
    """The cached rows of sequence b."""
    L = s["lengths"][b]
    blk = s["table"][b, :-(-L // TOK)].long()
    codes, scales = _views(s["pool"][blk])
    x = codes.contiguous().view(torch.uint8)[:, _map8(blk.device).reshape(-1)].view(torch.float8_e4m3fn)
    return (x.to(dtype).reshape(-1, ROW) * scales.reshape(-1, 1).to(dtype))[:L]


def _read(s):
    pool16 = s["pool16"].view(torch.bfloat16)
    at = _map16(pool16.device)
    for b, L in enumerate(s["lengths"]):
        t = torch.arange(L, device=pool16.device)
        blk = s["table16"][b].long()[t // TOK]
        pool16[blk[:, None], at[t % TOK]] = _rows(s, b).bfloat16()
    return pool16


def _decode(s):
    case = s["case"]
    H, n_q = case["H"], case["n_q"]
    W = s["W_UV"].float()
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    for b, L in enumerate(s["lengths"]):
        x = _rows(s, b)
        t = torch.arange(L, device=x.device)
        for j0 in range(0, n_q, 32):
            j1 = min(n_q, j0 + 32)
            q = s["q"][b * n_q + j0:b * n_q + j1].float()
            sc = (q.reshape(-1, ROW) @ x.T).reshape(j1 - j0, H, L) * SCALE
            last = L - n_q + torch.arange(j0, j1, device=x.device)
            sc = sc.masked_fill(t[None, None, :] > last[:, None, None], float("-inf"))
            top = sc.amax(-1, keepdim=True)
            p = torch.exp(sc - top)
            z = p.sum(-1, keepdim=True)
            o = (p.reshape(-1, L) @ x[:, :D_C]).reshape(j1 - j0, H, D_C) / z
            rows = slice(b * n_q + j0, b * n_q + j1)
            out[rows] = torch.einsum("jhc,hdc->jhd", o, W).bfloat16()
            lse[rows] = (top + torch.log(z)).squeeze(-1)
    return out, lse


# ------------------------------------------------------------------ in 64 bits

def _e4m3_table(dev):
    """The 256 values of e4m3 codes (bit 7 sign, four exponent bits of bias 7, three fraction bits; 0x7f NaN)."""
    v = []
    for i in range(256):
        e, f = (i >> 3) & 15, i & 7
        a = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v.append((float("nan") if i & 127 == 127 else a) * (-1 if i >> 7 else 1))
    return torch.tensor(v, dtype=torch.float64, device=dev)


def _values64(pool):
    """[blocks, 128, 576] in 64 bits, by taking the units of 16 bytes apart."""
    n = pool.shape[0]
    v = _e4m3_table(pool.device)
    r = torch.arange(TOK, device=pool.device)
    lat = pool[:, :65536].reshape(n, 4, TOK, 8, 16)
    rope = pool[:, 65536:CODES8].reshape(n, TOK, 4, 16)
    u8 = (torch.arange(8, device=pool.device)[None, :] ^ (r[:, None] & 7))
    u4 = (torch.arange(4, device=pool.device)[None, :] ^ ((r[:, None] >> 1) & 3))
    lat = torch.gather(lat, 3, u8[None, None, :, :, None].expand(n, 4, TOK, 8, 16))
    rope = torch.gather(rope, 2, u4[None, :, :, None].expand(n, TOK, 4, 16))
    rows = torch.cat([lat.permute(0, 2, 1, 3, 4).reshape(n, TOK, D_C), rope.reshape(n, TOK, D_R)], -1)
    scale = pool[:, CODES8:].contiguous().view(torch.float32).double()
    return v[rows.long()] * scale[:, :, None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _append64(s)
    dev = s["pool"].device
    if case["op"] == "read":
        out = torch.zeros(s["pool16"].shape[0], BLOCK // 2, dtype=torch.float64, device=dev)
        units = torch.arange(8, device=dev)[None, :] ^ (torch.arange(TOK, device=dev)[:, None] & 7)
        for b, L in enumerate(s["lengths"]):
            for k in range(-(-L // TOK)):
                x = _values64(s["pool"][s["table"][b, k].long()][None])[0]
                x[max(0, L - k * TOK):] = 0.0
                x = x.reshape(TOK, 9, 8, 8).permute(1, 0, 2, 3)
                x = torch.gather(x, 2, units[None, :, :, None].expand(9, TOK, 8, 8))
                out[s["table16"][b, k].long()] = x.reshape(-1)
        return out
    H, n_q = case["H"], case["n_q"]
    W = s["W_UV"].double()
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=dev)
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=dev)
    for b, L in enumerate(s["lengths"]):
        blocks = s["table"][b, :-(-L // TOK)].long()
        x = torch.cat([_values64(s["pool"][blocks[i:i + 64]]).reshape(-1, ROW) for i in range(0, len(blocks), 64)])[:L]
        for j in range(n_q):
            n = L - n_q + j + 1         # keys that query j sees
            a = s["q"][b * n_q + j].double() @ x[:n].T / 192.0 ** 0.5
            lse[b * n_q + j] = torch.logsumexp(a, -1)
            o = torch.exp(a - lse[b * n_q + j][:, None]) @ x[:n, :D_C]
            out[b * n_q + j] = (W @ o[:, :, None]).squeeze(-1)
    return out, lse


def _nearest(x, bits, least):
    """x in 64 bits rounded to `bits` significant bits, ties to even, in steps of at least 2^least."""
    step = torch.ldexp(torch.ones_like(x), (torch.frexp(x)[1] - bits).clamp_min(least))
    return torch.round(x / step) * step


def _append64(s):
    dev = s["pool"].device
    x = s["k_rope"].double()
    c, w = s["rope"].double()[s["pos"].long()].reshape(-1, D_R // 2, 2).unbind(-1)
    k = torch.empty_like(x)
    k[:, 0::2] = x[:, 0::2] * c - x[:, 1::2] * w
    k[:, 1::2] = x[:, 1::2] * c + x[:, 0::2] * w
    rows = torch.cat([s["c_kv"].double(), _nearest(k, 8, -133)], -1)
    f, e = torch.frexp(rows.abs().amax(-1))     # 448 = 0.875 * 2^9
    scale = torch.ldexp(torch.ones_like(f), torch.where(f <= 0.875, e - 9, e - 8).clamp_min(-40))
    rows = _nearest(rows / scale[:, None], 4, -9)
    n = s["pool"].shape[0]
    lat = torch.zeros(n, 4, TOK, 8, 16, dtype=torch.float64, device=dev)
    rope = torch.zeros(n, TOK, 4, 16, dtype=torch.float64, device=dev)
    scales = torch.zeros(n, TOK, dtype=torch.float64, device=dev)
    blk = s["table"][s["seq"].long(), (s["pos"] // TOK).long()].long()
    r = (s["pos"] % TOK).long()
    for u in range(32):
        lat[blk, u // 8, r, (u % 8) ^ (r & 7)] = rows[:, 16 * u:16 * u + 16]
    for u in range(4):
        rope[blk, r, u ^ ((r >> 1) & 3)] = rows[:, D_C + 16 * u:D_C + 16 * u + 16]
    scales[blk, r] = scale
    return torch.cat([lat.reshape(n, -1), rope.reshape(n, -1)], 1), scales
