"""The 8-bit latent cache on the CPU: the oracle's own pins, and the host-side refusals of its entry points."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import cache8 as o8


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_34_b200 as m
    return m


def test_e4m3_values():
    v = o8.VALUES
    assert v[0x7E] == 448.0 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0x38] == 1.0
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF]) and v[0xFE] == -448.0
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(v, t)


def test_e4m3_encode_rounds_to_nearest_even():
    x = np.concatenate([np.linspace(-448, 448, 20001), 2.0 ** np.arange(-12, 9), [17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    got = o8.VALUES[o8.e4m3_encode(x)]
    np.testing.assert_array_equal(got, torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy())
    assert list(o8.VALUES[o8.e4m3_encode(np.array([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10]))]) == [16, 20, 0, 2.0 ** -8]


def test_quantise_scale_is_least_power_of_two():
    x = np.zeros((6, 576))
    x[0, 3], x[1, 3], x[2, 3] = 448.0, 450.0, -3.5
    x[3, 0], x[3, 1], x[3, 2] = np.nan, np.inf, 1.0
    x[4, 5] = 2.0 ** -80
    codes, s = o8.quantise(x)
    assert list(s) == [1.0, 2.0, 2.0 ** -7, 2.0 ** -8, 2.0 ** -40, 1.0]
    assert codes[3, 0] == 0x7F and codes[3, 1] == 0x7F and codes[4, 5] == 0 and not codes[5].any()
    assert o8.VALUES[codes[2, 3]] * s[2] == -3.5


def test_layout_is_a_permutation():
    assert np.array_equal(np.sort(o8.OFFSETS.reshape(-1)), np.arange(128 * 576))


def test_append8_refusals(mla):
    L, f, odd = mla.lib, ctypes.c_void_p(4096), ctypes.c_void_p(4098)

    def app(cache=f, cap=10, tab=f, nseq=2, mb=4, seq=f, pos=f, c=f, k=f, rope=f, rl=5, T=3):
        return L.mla_append_cache8(cache, cap, tab, nseq, mb, seq, pos, c, k, rope, rl, T, None, None)
    assert L.mla_append_cache8(None, 0, None, 0, 0, None, None, None, None, None, 0, 0, None, None) == 0
    for bad in (dict(cache=None), dict(cache=odd), dict(cap=-1), dict(cap=1 << 31), dict(tab=None), dict(nseq=0),
                dict(mb=0), dict(mb=-1), dict(seq=None), dict(pos=None), dict(c=None), dict(c=odd), dict(k=None),
                dict(k=odd), dict(rope=None), dict(rope=odd), dict(rl=-1), dict(T=-1)):
        assert app(**bad) == 1, bad


def test_read8_refusals(mla):
    L, f, odd = mla.lib, ctypes.c_void_p(4096), ctypes.c_void_p(4098)

    def read(c8=f, cap8=10, t8=f, mb8=4, kv=f, B=2, c=f, cap=10, t=f, mb=4):
        return L.mla_read_cache8(c8, cap8, t8, mb8, kv, B, c, cap, t, mb, None, None)
    assert L.mla_read_cache8(None, 0, None, 0, None, 0, None, 0, None, 0, None, None) == 0
    for bad in (dict(c8=None), dict(c8=odd), dict(cap8=0), dict(cap8=-1), dict(cap8=1 << 31), dict(t8=None),
                dict(mb8=0), dict(mb8=1 << 25), dict(kv=None), dict(B=-1), dict(c=None), dict(c=odd), dict(cap=0),
                dict(cap=1 << 31), dict(t=None), dict(mb=0), dict(mb=1 << 25)):
        assert read(**bad) == 1, bad


def test_decode8_refusals(mla):
    L, f, odd = mla.lib, ctypes.c_void_p(4096), ctypes.c_void_p(4098)

    def dec(q=f, c=f, cap=10, tab=f, mb=4, kv=f, W=f, B=1, n_q=1, H=16, scale=0.07, splits=0, ws=f, nb=1 << 32, out=f):
        return L.mla_decode8(q, c, cap, tab, mb, kv, W, B, n_q, H, scale, splits, ws, nb, out, None, None, None)
    assert L.mla_decode8(None, None, 0, None, 0, None, None, 0, 1, 16, 0.07, 0, None, 0, None, None, None, None) == 0
    for bad in (dict(q=None), dict(q=odd), dict(c=None), dict(c=odd), dict(cap=0), dict(cap=-1), dict(tab=None),
                dict(mb=0), dict(kv=None), dict(W=None), dict(W=odd), dict(B=-1), dict(scale=0.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(ws=None), dict(ws=odd), dict(out=None),
                dict(out=odd)):
        assert dec(**bad) == 1, bad
    for bad in (dict(n_q=0), dict(n_q=257), dict(H=0), dict(H=129), dict(splits=-1), dict(splits=257),
                dict(B=1 << 20, n_q=256)):
        assert dec(**bad) == 2, bad
    need = L.mla_decode8_workspace_bytes(4, 2, 128, 3)
    assert need > 0 and dec(B=4, n_q=2, H=128, splits=3, nb=need - 1) == 4
    assert L.mla_decode8_workspace_bytes(-1, 1, 16, 0) == 0


def test_decode8_workspace_holds_every_piece(mla):
    """Four and 512 fp32 for each row of a slot, a slot for each sequence and work unit."""
    for B, n_q, H in ((1, 1, 16), (3, 2, 16), (64, 3, 16), (1, 1, 49), (7, 2, 128), (2, 256, 128), (500, 1, 1)):
        R = n_q * H
        groups, units, rows = ((1, 148, 32 if R <= 32 else 64) if R <= 48 else
                               (-(-R // 128), max(1, 74 // -(-R // 128)), 128))
        n = groups * (B + units) * rows
        got = mla.decode8_workspace_bytes(B, n_q, H)
        assert n * 2064 <= got <= n * 2064 + 1040, (B, n_q, H)
    assert mla.decode8_workspace_bytes(0, 1, 16) == 0


def test_binding_refuses_wrong_tensors(mla):
    """Shapes, types and devices are refused before the library is called (CPU tensors here)."""
    i32 = dict(dtype=torch.int32)
    pool = torch.zeros(2, mla.BLOCK8_BYTES, dtype=torch.uint8)
    tab, one = torch.zeros(1, 2, **i32), torch.ones(1, **i32)
    q, W = torch.zeros(1, 16, 576, dtype=torch.bfloat16), torch.zeros(16, 128, 512, dtype=torch.bfloat16)
    with pytest.raises(mla.MLAError):
        mla.decode8(q, pool, tab, one, W, 1, 0.07, workspace=pool, out=torch.zeros(1, 16, 128, dtype=torch.bfloat16))
    with pytest.raises(mla.MLAError):
        mla.decode8(q, pool, tab, one, W, 2, 0.07)
    with pytest.raises(mla.MLAError):
        mla.read_cache8(pool[:, :100], tab, one, pool, tab)
    with pytest.raises(mla.MLAError):
        mla.append_cache8(pool, tab, one, one, torch.zeros(1, 512, dtype=torch.bfloat16),
                          torch.zeros(1, 64, dtype=torch.bfloat16), torch.zeros(4, 64))


@pytest.mark.parametrize("mass", [0.05, 0.2, 0.5])
def test_peaked_cases_show_a_lost_tail(mass):
    """The cases of test_gpu_cache8_peaked.py fail where the tail's probabilities are dropped from o but not from its sum."""
    from cache8_cases import L2, peaked_queries, peaked_rows
    x = peaked_rows(8000, mass)
    codes, s = o8.quantise(x)
    rows, q = o8.VALUES[codes] * s[:, None], peaked_queries((1, 2))
    W = np.random.default_rng(1).standard_normal((2, 128, 512)) / np.sqrt(512)
    out, _, o, A, _ = o8.attend(rows, q, W, 1, 192 ** -0.5)
    a = q[0] @ rows.T / np.sqrt(192.0)
    p = np.exp(a - a.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    # (the peak's score, below 16, is rounded by 2^-4 of itself at most, the scores' other columns add less than 0.1)
    assert np.abs(np.log(p[:, 1:].sum(1) / mass)).max() < 1.1
    lost = np.einsum("hc,hdc->hd", p[:, :1] * rows[0, :512], W)
    assert np.linalg.norm(lost - out[0]) > 1.5 * L2 * np.linalg.norm(out)


@pytest.mark.parametrize("name", ["mla_decode8_workspace_bytes", "mla_decode_workspace_bytes",
                                  "mla_decode_cudacore_workspace_bytes"])
def test_workspace_sizes_of_refused_shapes(mla, name):
    """Shapes that the calls refuse have size 0: no overflow, no division by zero (n_q * H = 2^32, B = 0 of an automatic
    split), which ended the process."""
    size = getattr(mla.lib, name)
    top = (1 << 31) - 1
    for B, n_q, H, splits in ((1, 1 << 16, 1 << 16, 0), (1, 257, 16, 0), (1, 1, 129, 0), (1, 0, 16, 0), (1, 1, 0, 0),
                              (-1, 1, 16, 0), (1, 1, 16, -1), (1, 1, 16, 257), (top, 256, 128, 0), (top, top, top, 3),
                              (1 << 24, 1, 1, 0), (1 << 16, 1 << 15, 1, 0)):
        assert size(B, n_q, H, splits) == 0, (B, n_q, H, splits)
    assert size(0, 1, 16, 0) == 0 or name == "mla_decode_workspace_bytes"
    assert size(0, 1, 16, 2) == 0 or name == "mla_decode_workspace_bytes"
    for B, n_q, H in ((1, 1, 1), (1, 256, 128), (65535, 256, 1), (4096, 2, 128)):
        assert size(B, n_q, H, 0) >= B * n_q * H * 2048, (B, n_q, H)


def test_static_decode_refuses_shapes_before_the_device(mla):
    f = ctypes.c_void_p(4096)
    for B, n_q, H, splits in ((1, 1, 129, 0), (1, 257, 16, 0), (1, 1, 16, 257), (1 << 24, 1, 1, 0)):
        assert mla.lib.mla_decode_static(f, f, 10, f, 4, f, f, B, n_q, H, 0.07, splits, f, None, None, None) == 2
