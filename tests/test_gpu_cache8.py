"""The 8-bit latent cache on the GPU: quantised append and read-back bit for bit, decode against 64 bits.

Tolerances of decode8, from its roundings (u = 2^-8, half a bf16 step).  P is rounded to 8 significant bits (within u)
or, in the one-SM kernel's 32-row form, to 9 with a dither (within u as well), and held by two terms; far below the
reference their steps are absolute, and dithered over the tokens, so that the sum of a long tail keeps within another u
of the whole: 2 u in all.  With A = sum_t P_t |c_t| and d the error of
a score (576 products summed in fp32: d <= 577 * 2^-23 * max_t sum |q_i c_ti| * scale), o_lat is off by at most
(2 u + 2 d + 2^-14) A (it is held by two bf16 terms, within 2^-16), and out is rounded to bf16:
    |out - ref| <= |W^UV| (2 u + 2 d + 2^-14) A + u |ref| (1 + 2^-7) + 2^-20,
2^-14 for the fp32 sums and exponentials and for those 2^-16.  In the 2-norm: P's roundings change o_lat by
sum_t e_t P_t c_t with |e_t| <= u, at most u of it where one token carries the row (its one error then scales every column
alike; many tokens' errors are independent and come to less); the rounding of out is independent over the columns, uniform
within u, so of rms u / sqrt(3).  Together at most u sqrt(1 + 1/3) = u sqrt(4/3).  lse is off by
d + 2^-13 (sums of a tile, then of tiles, in fp32).
"""

import numpy as np
import pytest
import torch

import mla_latent_kv_34_b200 as mla
from gpu_harness import BLOCK_MAP, block_tables, rel_l2, to_dev_bf16
from oracle import cache8 as o8
from oracle.append import rope_table_f32

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
SCALE = 192 ** -0.5


def f32_to_bf16_bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().view(torch.int16).numpy().view(np.uint16)


def bf16_to_f64(bits):
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def rotate_bits(k_bits, pos, rope):
    """R_pos k^R with separately rounded fp32 products and sums, rounded to bf16."""
    x = (k_bits.astype(np.uint32) << 16).view(np.float32)
    c, s = rope[pos][:, 0::2], rope[pos][:, 1::2]
    y = np.empty_like(x)
    y[:, 0::2] = (x[:, 0::2] * c) - (x[:, 1::2] * s)
    y[:, 1::2] = (x[:, 0::2] * s) + (x[:, 1::2] * c)
    return f32_to_bf16_bits(y)


def rope_host(n):
    c, s = rope_table_f32(list(range(n)))
    t = np.empty((n, 64), dtype=np.float32)
    t[:, 0::2], t[:, 1::2] = c, s
    return t


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Problem8:
    """An 8-bit paged cache built on the host, with NaN codes and NaN scales wherever no token is."""

    def __init__(self, lengths, H, n_q, seed=0, amp=0.3, rows=None, q=None, extra_cols=1, q_amp=0.5):
        rng = np.random.default_rng(seed)
        self.lengths, self.H, self.n_q, self.B = np.asarray(lengths), H, n_q, len(lengths)
        self.tables, cap, self.unowned = block_tables(np.maximum(self.lengths, 1), shuffle_seed=seed + 1,
                                                      extra_cols=extra_cols)
        self.pool = np.full((cap, o8.BLOCK8_BYTES), 0x7F, dtype=np.uint8)
        self.pool[:, o8.SCALES_AT:] = np.frombuffer(np.full(128, np.nan, np.float32).tobytes(), np.uint8)
        self.rows = []
        for b, L in enumerate(self.lengths):
            x = rng.standard_normal((L, 576)) * np.exp(amp * rng.standard_normal((L, 1)))
            x = bf16_to_f64(f32_to_bf16_bits(x)) if rows is None else rows(b, x)
            codes, s = o8.quantise(x)
            t = np.arange(L)
            o8.pack(self.pool, self.tables[b, t // 128], t % 128, codes, s)
            self.rows.append(o8.VALUES[codes] * s[:, None])
        T = self.B * n_q
        qv = rng.standard_normal((T, H, 576))
        qv[..., :512] *= q_amp
        self.q_bits = f32_to_bf16_bits(qv if q is None else q(qv))
        self.W_bits = f32_to_bf16_bits(rng.standard_normal((H, 128, 512)) / np.sqrt(512))
        self.cache8 = torch.from_numpy(self.pool).cuda()
        self.table, self.kv_len = i32(self.tables), i32(self.lengths)
        self.q, self.W = to_dev_bf16(self.q_bits, "cuda"), to_dev_bf16(self.W_bits, "cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def decode(self, **kw):
        lse = torch.full((self.B * self.n_q, self.H), 77.0, device="cuda")
        out = mla.decode8(self.q, self.cache8, self.table, self.kv_len, self.W, self.n_q, SCALE, lse_out=lse,
                          dev_status=self.status, **kw)
        return out, lse

    def check(self, out, lse, seqs=None, l2=True):
        out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        W = bf16_to_f64(self.W_bits)
        got, want = [], []
        for b in (range(self.B) if seqs is None else seqs):
            rows = slice(b * self.n_q, (b + 1) * self.n_q)
            ref, ref_lse, _, A, reach = o8.attend(self.rows[b], bf16_to_f64(self.q_bits[rows]), W, self.n_q, SCALE)
            d = 577 * 2.0 ** -23 * reach
            err = (2 * U + 2 * d[..., None] + 2.0 ** -14) * A
            tol = np.einsum("jhc,hdc->jhd", err, np.abs(W)) + U * np.abs(ref) * (1 + 2.0 ** -7) + 2.0 ** -20
            assert np.isfinite(out[rows]).all() and np.isfinite(lse[rows]).all(), b
            excess = (np.abs(out[rows] - ref) - tol).max()
            assert excess <= 0, (b, excess, np.abs(out[rows] - ref).max())
            assert (np.abs(lse[rows] - ref_lse) <= d + 2.0 ** -13).all(), (b, np.abs(lse[rows] - ref_lse).max())
            got.append(out[rows].reshape(-1))
            want.append(ref.reshape(-1))
        if l2:
            e = rel_l2(np.concatenate(got), np.concatenate(want))
            assert e <= U * np.sqrt(4 / 3), e


# ------------------------------------------------------------------ append

def special_rows(n, rng):
    x = rng.standard_normal((n, 512)) * np.exp(2.0 * rng.standard_normal((n, 1)))
    k = rng.standard_normal((n, 64))
    special = [np.zeros(512), np.full(512, 448.0), np.full(512, 450.0), np.full(512, 1e-30), np.full(512, -3.5),
               np.linspace(-448, 448, 512), 2.0 ** -np.arange(512).clip(0, 60), np.full(512, 3e38)]
    for i, s in enumerate(special[:n]):
        x[i] = s
        if i in (0, 3):
            k[i] = 0.0
    if n > 12:
        x[8, 5], x[9, 6], x[10, 7], x[11, :] = np.inf, -np.inf, np.nan, np.nan
        k[12, 3] = np.nan
        k[11] = 0.0
    return f32_to_bf16_bits(x), f32_to_bf16_bits(k)


@pytest.mark.parametrize("T", [1, 2, 7, 129, 700, 9601])
def test_append8_bit_exact(T):
    rng = np.random.default_rng(T)
    c, k = special_rows(T, rng)
    mb, nseq = (7, 4) if T <= 700 else (25, 4)
    cap = nseq * mb + 2
    tables = rng.permutation(cap)[:nseq * mb].reshape(nseq, mb).astype(np.int32)
    place = rng.permutation(nseq * mb * 128)[:T]
    seq, pos = (place // (mb * 128)).astype(np.int32), (place % (mb * 128)).astype(np.int32)
    rope = rope_host(mb * 128)
    before = rng.integers(0, 256, (cap, o8.BLOCK8_BYTES)).astype(np.uint8)
    cache = torch.from_numpy(before.copy()).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.append_cache8(cache, i32(tables), i32(seq), i32(pos), to_dev_bf16(c, "cuda"), to_dev_bf16(k, "cuda"),
                      torch.from_numpy(rope).cuda(), status)
    got = cache.cpu().numpy()
    x = bf16_to_f64(np.concatenate([c, rotate_bits(k, pos, rope)], 1))
    codes, scales = o8.quantise(x)
    want = before.copy()
    o8.pack(want, tables[seq, pos // 128], pos % 128, codes, scales)
    nan = (want & 127 == 127) & (got & 127 == 127)  # NaN of either sign
    nan[:, o8.SCALES_AT:] = False
    assert ((got == want) | nan).all()
    assert status.item() == 0


def test_append8_matches_the_bf16_row():
    """The row that is quantised is the one that append_cache stores."""
    rng = np.random.default_rng(5)
    T = 300
    c, k = f32_to_bf16_bits(rng.standard_normal((T, 512))), f32_to_bf16_bits(rng.standard_normal((T, 64)))
    tab, seq, pos = i32([[2, 0, 1]]), i32(np.zeros(T)), i32(np.arange(T))
    rope = mla.rope_table(T)
    c16 = torch.zeros(3, mla.BLOCK_BYTES, dtype=torch.uint8, device="cuda")
    c8 = torch.zeros(3, mla.BLOCK8_BYTES, dtype=torch.uint8, device="cuda")
    mla.append_cache(c16, tab, seq, pos, to_dev_bf16(c, "cuda"), to_dev_bf16(k, "cuda"), rope)
    mla.append_cache8(c8, tab, seq, pos, to_dev_bf16(c, "cuda"), to_dev_bf16(k, "cuda"), rope)
    t = np.arange(T)
    blocks = np.array([2, 0, 1])[t // 128]
    bits = c16.cpu().numpy().view(np.uint16).reshape(3, -1)[blocks[:, None], BLOCK_MAP[t % 128]]
    codes, scales = o8.quantise(bf16_to_f64(bits))
    got = o8.unpack(c8.cpu().numpy(), blocks, t % 128)
    np.testing.assert_array_equal(got[0], codes)
    np.testing.assert_array_equal(got[1], scales)


def test_append8_skips_and_reports():
    T = 8
    seq = np.array([0, 2, -1, 0, 0, 1, 0, 0])          # 1: past the table, 2: negative
    pos = np.array([0, 0, 0, -3, 256, 3, 200, 255])    # 3: negative, 4: past the row, 6, 7: past the RoPE table
    tab = i32([[0, 1], [9, 9]])                        # sequence 1: entry outside the pool
    c = torch.ones(T, 512, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(T, 64, dtype=torch.bfloat16, device="cuda")
    cache = torch.full((2, mla.BLOCK8_BYTES), 0xA5, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.append_cache8(cache, tab, i32(seq), i32(pos), c, k, mla.rope_table(200), status)
    assert status.item() == 1 | 2
    want = np.full((2, mla.BLOCK8_BYTES), 0xA5, dtype=np.uint8)
    rope = rope_host(1)
    x = np.concatenate([np.ones((1, 512)), bf16_to_f64(rotate_bits(f32_to_bf16_bits(np.ones((1, 64))), [0], rope))], 1)
    o8.pack(want, [0], [0], *o8.quantise(x))
    np.testing.assert_array_equal(cache.cpu().numpy(), want)
    mla.append_cache8(cache, tab, i32([]), i32([]), c[:0], k[:0], mla.rope_table(200), status)
    np.testing.assert_array_equal(cache.cpu().numpy(), want)


# ------------------------------------------------------------------ read back

@pytest.mark.parametrize("lengths", [[1], [127, 128, 129], [0, 5, 0, 300, 31, 32, 33, 0], [1000] * 3 + [2, 640], [0, 0]])
def test_read8_bit_exact(lengths):
    p = Problem8(lengths, 1, 1, seed=len(lengths))
    tables16, cap16, _ = block_tables(np.maximum(lengths, 1), shuffle_seed=99, extra_cols=2)
    before = np.random.default_rng(1).integers(0, 1 << 16, (cap16, mla.BLOCK_BYTES // 2)).astype(np.uint16)
    cache = torch.from_numpy(before.view(np.uint8).copy()).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.read_cache8(p.cache8, p.table, p.kv_len, cache, i32(tables16), status)
    want = before.copy()
    for b, L in enumerate(lengths):
        t = np.arange(L)
        want[tables16[b, t // 128][:, None], BLOCK_MAP[t % 128]] = f32_to_bf16_bits(p.rows[b])
    np.testing.assert_array_equal(cache.cpu().numpy().view(np.uint16), want)
    assert status.item() == 0


def test_read8_special_values():
    """NaN codes come back as NaN, the smallest and largest scales exactly."""
    x = np.zeros((4, 576))
    x[0, :3] = np.nan, 1.0, -0.0
    x[1, :2] = 2.0 ** -42, 2.0 ** -49
    x[2, :2] = 1.5 * 2.0 ** 127, 2.0 ** 115
    p = Problem8([4], 1, 1, rows=lambda b, _: x)
    cache = torch.zeros(1, mla.BLOCK_BYTES, dtype=torch.uint8, device="cuda")
    mla.read_cache8(p.cache8, p.table, p.kv_len, cache, i32([[0]]))
    got = bf16_to_f64(cache.cpu().numpy().view(np.uint16)[0, BLOCK_MAP[:4]])
    np.testing.assert_array_equal(got, x)


def test_read8_skips_and_reports():
    p = Problem8([200, 300, 100, 256], 1, 1)
    kv = i32([200, -1, 5000, 256])
    t8 = p.tables.copy()
    t8[0, 1] = p.pool.shape[0]
    cache = torch.zeros(6, mla.BLOCK_BYTES, dtype=torch.uint8, device="cuda")
    t16 = i32([[0, 1, 4, 4], [4, 4, 4, 4], [4, 4, 4, 4], [2, -1, 4, 4]])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.read_cache8(p.cache8, i32(t8), kv, cache, t16, status)
    assert status.item() == 1 | 4
    got = cache.cpu().numpy().view(np.uint16)
    want = np.zeros_like(got)
    want[0][BLOCK_MAP] = f32_to_bf16_bits(p.rows[0][:128])
    want[2][BLOCK_MAP] = f32_to_bf16_bits(p.rows[3][:128])
    np.testing.assert_array_equal(got, want)


# ------------------------------------------------------------------ decode

@pytest.mark.parametrize("lengths,H,n_q", [
    ([1], 1, 1), ([1], 128, 1), ([2], 16, 2), ([127], 16, 1), ([128], 128, 1), ([129], 5, 1),
    ([256], 16, 1), ([5, 3, 4], 20, 3), ([3, 700, 130, 33], 11, 3), ([640, 1, 2, 129], 32, 1), ([300, 40], 33, 1),
    ([513, 200], 64, 1), ([900, 1, 250], 128, 1), ([200, 1025], 128, 2), ([77, 400], 100, 3), ([1500], 128, 3),
    ([300], 20, 101), ([256], 1, 256), ([4000, 3], 16, 2), ([3000], 128, 1)])
def test_decode8_against_64_bits(lengths, H, n_q):
    p = Problem8(lengths, H, n_q, seed=H + n_q)
    out, lse = p.decode()
    assert p.status.item() == 0
    p.check(out, lse, l2=min(lengths) > 100)


@pytest.mark.parametrize("lengths,H,n_q", [
    ([1 + 7 * i % 300 for i in range(70)], 128, 1), ([3 + 11 * i % 170 for i in range(30)], 128, 3),
    ([40 + 29 * i % 200 for i in range(9)], 5, 40), ([130, 7], 100, 1), ([1500, 700, 40], 40, 1),
    ([1400, 9, 513], 24, 1), ([700, 900], 16, 3), ([300, 257], 128, 256)])
def test_decode8_many_rows_heads_and_pieces(lengths, H, n_q):
    """Blocks of query rows of several sequences, several blocks a head, rows that straddle the
    groups of 128, and one to three sequences a work unit."""
    p = Problem8(lengths, H, n_q, seed=H)
    out, lse = p.decode()
    assert p.status.item() == 0
    p.check(out, lse, l2=False)
    p.check(*p.decode(num_splits=3), l2=False)


def test_decode8_empty_sequences_between_others():
    p = Problem8([1 + 5 * i % 130 for i in range(70)], 128, 1, seed=31)
    gone = [0, 8, 9, 63, 64, 69]
    kv = p.lengths.copy()
    kv[gone] = 0
    lse = torch.full((70, 128), 77.0, device="cuda")
    out = mla.decode8(p.q, p.cache8, p.table, i32(kv), p.W, 1, SCALE, lse_out=lse, dev_status=p.status)
    assert p.status.item() == 4
    p.check(out, lse, seqs=[b for b in range(70) if b not in gone], l2=False)
    assert (out[gone] == 0).all() and torch.isneginf(lse[gone]).all()


def test_decode8_workspace_of_any_alignment_and_two_calls_at_once():
    """Workspaces that start 16 bytes past a multiple of 32; calls on two streams that run at the same time."""
    ps = [Problem8([500, 90], 128, 1, seed=40), Problem8([900, 64, 200], 16, 1, seed=41)]
    ws = []
    for p in ps:
        n = mla.decode8_workspace_bytes(p.B, 1, p.H)
        w = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        at = 16 + (-w.data_ptr()) % 32
        ws.append((w, at, w[at:at + n]))
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    res = []
    for _ in range(3):
        for p, (_w, _at, v), s in zip(ps, ws, streams):
            lse = torch.empty(p.B, p.H, device="cuda")
            with torch.cuda.stream(s):
                out = mla.decode8(p.q, p.cache8, p.table, p.kv_len, p.W, 1, SCALE, workspace=v, lse_out=lse)
            res.append((p, out, lse))
    torch.cuda.synchronize()
    for p, out, lse in res:
        p.check(out, lse)
    for (w, at, v) in ws:
        assert (w[:at] == 0xFF).all() and (w[at + v.numel():] == 0xFF).all()


def test_decode8_wide_range_of_scales():
    """Rows whose magnitudes differ by 2^20 within a tile: the large ones carry the output where they are."""
    p = Problem8([700, 300], 24, 1, seed=3, amp=4.0, q_amp=0.02, q=lambda q: 0.05 * q)
    p.check(*p.decode(), l2=False)
    p = Problem8([700, 300], 128, 1, seed=3, amp=4.0, q=lambda q: 0.05 * q)
    p.check(*p.decode(), l2=False)


@pytest.mark.parametrize("H", [16, 40, 128])
@pytest.mark.parametrize("gap", [8.0, 12.0, 30.0])
def test_decode8_sink_token(H, gap):
    """One token far above thousands of others, whose small P have to keep their sum: the first, and one in the middle."""
    for at in (0, 1500):
        def rows(b, x, at=at):
            x = 0.05 * x
            x[:, 575] = 0.0
            x[at, 575] = gap
            return bf16_to_f64(f32_to_bf16_bits(x))

        def q(v):
            v = 0.1 * v
            v[..., 575] = np.sqrt(192.0)
            return v
        p = Problem8([3000], H, 1, seed=7, rows=rows, q=q)
        p.check(*p.decode(num_splits=1), l2=False)
        p.check(*p.decode(), l2=False)


def test_decode8_rising_and_falling_scores():
    """Tile maxima that move by 2^20 up and down from tile to tile."""
    for H in (16, 128):
        def rows(b, x):
            x[:, 575] = np.repeat(np.random.default_rng(2).uniform(-14, 14, 16), 128)[:len(x)]
            return bf16_to_f64(f32_to_bf16_bits(x))

        def q(v):
            v[..., 575] = np.sqrt(192.0)
            return v
        p = Problem8([2000], H, 1, seed=9, rows=rows, q=q)
        p.check(*p.decode(num_splits=1), l2=False)


def test_decode8_large_and_small_queries():
    for k in (2.0 ** -60, 2.0 ** 40):
        p = Problem8([300], 20, 1, seed=4, rows=lambda b, x: bf16_to_f64(f32_to_bf16_bits(x / k * 0.5)) if k > 1 else
                     bf16_to_f64(f32_to_bf16_bits(x * 64)), q=lambda v: v * k)
        if k > 1:  # rows of 2^-40: W^UV's output is far below the absolute term, so compare scaled up
            assert np.isfinite(p.decode()[0].float().cpu().numpy()).all()
        p.check(*p.decode(), l2=False)


def test_decode8_short_long_and_bad_sequences():
    p = Problem8([300, 200, 400], 16, 2, seed=8)
    kv = i32([300, 1, 5000])
    lse = torch.full((6, 16), 77.0, device="cuda")
    out = mla.decode8(p.q, p.cache8, p.table, kv, p.W, 2, SCALE, lse_out=lse, dev_status=p.status)
    assert p.status.item() == 1 | 4
    p.check(out, lse, seqs=[0])
    assert (out[2:] == 0).all() and torch.isneginf(lse[2:]).all()
    p.status.zero_()
    tab = p.table.clone()
    tab[1, 0] = p.pool.shape[0]
    out = mla.decode8(p.q, p.cache8, tab, p.kv_len, p.W, 2, SCALE, lse_out=lse, dev_status=p.status)
    assert p.status.item() == 1
    p.check(out, lse, seqs=[0, 2])
    out = mla.decode8(p.q[:0], p.cache8, p.table[:0], p.kv_len[:0], p.W, 2, SCALE)
    assert out.shape == (0, 16, 128)


@pytest.mark.parametrize("H,n_q", [(16, 1), (128, 2)])
def test_decode8_splits_agree(H, n_q):
    p = Problem8([1000, 70, 513], H, n_q, seed=6)
    for s in (1, 2, 7, 256):
        p.check(*p.decode(num_splits=s))


@pytest.mark.parametrize("H", [16, 128])
def test_decode8_nan_and_inf_in_a_row(H):
    """A visible NaN makes its sequence's rows NaN (as in a bf16 cache), and no other's."""
    def rows(b, x):
        if b == 1:
            x[7, 3] = np.inf
        return x
    p = Problem8([200, 150, 130], H, 1, rows=lambda b, x: rows(b, bf16_to_f64(f32_to_bf16_bits(x))))
    out, lse = p.decode()
    assert torch.isnan(out[1]).any() and torch.isnan(lse[1]).all()
    p.check(out, lse, seqs=[0, 2])


def test_decode8_same_block_in_two_sequences_and_twice():
    """A shared prefix block, and a block that one sequence names twice, are read like any other."""
    p = Problem8([256, 256], 128, 1, seed=12)
    p.tables[1, 0] = p.tables[0, 0]
    p.tables[1, 1] = p.tables[0, 0]
    p.table = i32(p.tables)
    p.rows[1] = np.concatenate([p.rows[0][:128]] * 2)
    p.check(*p.decode())


def test_decode8_repeats_bit_for_bit_and_leaves_its_inputs():
    for H, n_q in ((16, 1), (128, 1)):
        p = Problem8([1000, 300], H, n_q, seed=2)
        out, lse = p.decode()
        for _ in range(3):
            o2, l2 = p.decode()
            assert torch.equal(out, o2) and torch.equal(lse, l2)
        np.testing.assert_array_equal(p.cache8.cpu().numpy(), p.pool)


def test_decode8_on_a_stream_and_in_graphs():
    """Another stream than the current one; two captured graphs with workspaces of their own, replayed in turn and on
    changed inputs."""
    p = Problem8([500, 90], 128, 1, seed=21)
    a = Problem8([400, 64, 200], 16, 1, seed=22)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lse = torch.empty(2, 128, device="cuda")
    out = mla.decode8(p.q, p.cache8, p.table, p.kv_len, p.W, 1, SCALE, lse_out=lse, stream=s)
    s.synchronize()
    p.check(out, lse)
    graphs = []
    for x in (p, a):
        ws = torch.empty(mla.decode8_workspace_bytes(x.B, 1, x.H), dtype=torch.uint8, device="cuda")
        o, l = torch.empty(x.B, x.H, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(x.B, x.H, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mla.decode8(x.q, x.cache8, x.table, x.kv_len, x.W, 1, SCALE, workspace=ws, out=o, lse_out=l)
        graphs.append((x, g, o, l, ws))
    for _ in range(2):
        for x, g, o, l, _ws in graphs:
            o.fill_(float("nan"))
            g.replay()
        torch.cuda.synchronize()
        for x, g, o, l, _ws in graphs:
            x.check(o, l)
        # the next replay sees new lengths and queries
        for x, *_ in graphs:
            x.lengths = np.maximum(x.lengths - 37, 1)
            x.kv_len.copy_(i32(x.lengths))
            x.rows = [r[:n] for r, n in zip(x.rows, x.lengths)]
            x.q_bits = x.q_bits[::-1].copy()
            x.q.copy_(to_dev_bf16(x.q_bits, "cuda"))


def test_cache8_pool_past_32_bits():
    """Blocks whose byte offsets pass 2^32, in all three operators."""
    cap = (1 << 32) // mla.BLOCK8_BYTES + 40
    p = Problem8([300, 129], 16, 1, seed=30)
    pool = torch.empty(cap, mla.BLOCK8_BYTES, dtype=torch.uint8, device="cuda")
    base = cap - p.pool.shape[0]
    pool[base:] = p.cache8
    p.cache8, p.table = pool, p.table + base
    p.check(*p.decode())
    c = to_dev_bf16(f32_to_bf16_bits(np.ones((1, 512))), "cuda")
    k = torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")
    mla.append_cache8(pool, p.table, i32([0]), i32([130]), c, k, mla.rope_table(256))
    p.rows[0][130] = np.concatenate([np.ones(512), np.zeros(64)])
    p.check(*p.decode())
    cap16 = (1 << 32) // mla.BLOCK_BYTES + 40
    pool16 = torch.zeros(cap16, mla.BLOCK_BYTES, dtype=torch.uint8, device="cuda")
    t16 = np.array([[cap16 - 1, cap16 - 3, cap16 - 5], [cap16 - 2, cap16 - 9, 0]])
    mla.read_cache8(pool, p.table, p.kv_len, pool16, i32(t16))
    got = pool16[cap16 - 1].cpu().numpy().view(np.uint16)[BLOCK_MAP]
    np.testing.assert_array_equal(got, f32_to_bf16_bits(p.rows[0][:128]))
    assert not pool16[0].any()


# ------------------------------------------------------------------ together

def test_steps_over_a_growing_8bit_cache():
    """A prompt written at once, then steps that append a token each and decode, as a serving loop makes them."""
    rng = np.random.default_rng(11)
    lengths, H = np.array([200, 126]), 16
    top = lengths + 4
    tables, cap, _ = block_tables(top, shuffle_seed=4)
    tab, rope = i32(tables), rope_host(256)
    rope_dev = torch.from_numpy(rope).cuda()
    cache = torch.full((cap, mla.BLOCK8_BYTES), 0x7F, dtype=torch.uint8, device="cuda")
    c = [f32_to_bf16_bits(rng.standard_normal((n, 512))) for n in top]
    k = [f32_to_bf16_bits(rng.standard_normal((n, 64))) for n in top]
    seq = np.repeat([0, 1], lengths)
    pos = np.concatenate([np.arange(n) for n in lengths])
    mla.append_cache8(cache, tab, i32(seq), i32(pos), to_dev_bf16(np.concatenate([c[0][:200], c[1][:126]]), "cuda"),
                      to_dev_bf16(np.concatenate([k[0][:200], k[1][:126]]), "cuda"), rope_dev)
    p = Problem8([1, 1], H, 1)
    rows = []
    for b in range(2):
        codes, s = o8.quantise(bf16_to_f64(np.concatenate([c[b], rotate_bits(k[b], np.arange(top[b]), rope)], 1)))
        rows.append(o8.VALUES[codes] * s[:, None])
    for step in range(4):
        at = lengths + step
        mla.append_cache8(cache, tab, i32([0, 1]), i32(at),
                          to_dev_bf16(np.stack([c[b][at[b]] for b in range(2)]), "cuda"),
                          to_dev_bf16(np.stack([k[b][at[b]] for b in range(2)]), "cuda"), rope_dev)
        p.cache8, p.table, p.kv_len = cache, tab, i32(at + 1)
        p.rows = [rows[b][:at[b] + 1] for b in range(2)]
        p.check(*p.decode())


def test_prefill_chunk_behind_an_8bit_prefix():
    """The prefix is read back into a bf16 pool and the naive prefill runs over it; the same queries decoded over the
    8-bit cache give the same result, within both forms' roundings."""
    H, L, n = 4, 500, 60
    rng = np.random.default_rng(13)
    p = Problem8([L], H, n, seed=13)
    Wk = f32_to_bf16_bits(rng.standard_normal((H, 128, 512)) / np.sqrt(512))
    qn, qr = f32_to_bf16_bits(rng.standard_normal((n, H, 128))), f32_to_bf16_bits(rng.standard_normal((n, H, 64)))
    pool16, rope = mla.new_cache(6), mla.rope_table(L)
    t16 = i32([[4, 0, 5, 1]])
    mla.read_cache8(p.cache8, p.table, p.kv_len, pool16, t16)
    a = mla.prefill_naive(to_dev_bf16(qn, "cuda"), to_dev_bf16(qr, "cuda"), rope, pool16, t16[0], L,
                          to_dev_bf16(Wk, "cuda"), p.W, SCALE)
    q = mla.absorb_q(to_dev_bf16(qn, "cuda"), to_dev_bf16(qr, "cuda"), i32(L - n + np.arange(n)), to_dev_bf16(Wk, "cuda"), rope)
    p.q, p.q_bits = q, q.cpu().view(torch.int16).numpy().view(np.uint16)
    out, lse = p.decode()
    p.check(out, lse)
    a, b = a.float().cpu().numpy(), out.float().cpu().numpy()
    # each form has at most five bf16 roundings between the same inputs and its output (q_abs or k^C, v^C, P, o, out)
    assert rel_l2(a, b) <= 2 * np.sqrt(5) * U
