"""64-bit emulation of the 8-bit latent cache: codes, scales, block layout, and attention over its values.

A row's scale is the least power of two s >= 2^-40 with max |x_i| <= 448 s over the finite x_i (1 if none is
nonzero); its codes are e4m3(x_i / s), rounded to nearest with ties to even, NaN for what is not finite
(mla_append_cache8 in include/mla.h).  e4m3: sign, four exponent bits of bias 7, three fraction bits, no
infinities, 0x7f the NaN.
"""

from __future__ import annotations

import numpy as np

BLOCK8_BYTES, SCALES_AT = 74240, 73728


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes."""
    v = np.empty(256)
    for i in range(256):
        e, f = (i >> 3) & 15, i & 7
        a = f / 512.0 if e == 0 else (1.0 + f / 8.0) * 2.0 ** (e - 7)
        v[i] = (np.nan if (i & 127) == 127 else a) * (-1.0 if i & 128 else 1.0)
    return v


VALUES = e4m3_values()


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Nearest code of finite |x| <= 448, ties to the even code; 0x7f for NaN."""
    pos = VALUES[:127]                       # increasing, 0 .. 448
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def quantise(x: np.ndarray):
    """Rows [n, 576] in 64 bits -> (codes uint8 [n, 576], scales [n])."""
    finite = np.isfinite(x)
    top = np.where(finite, np.abs(x), 0.0).max(axis=1)
    s = np.ones(len(x))
    for i, t in enumerate(top):
        if t == 0.0:
            continue
        k = -40
        while t > 448.0 * 2.0 ** k:
            k += 1
        s[i] = 2.0 ** k
    return e4m3_encode(np.where(finite, x, np.nan) / s[:, None]), s


def offsets() -> np.ndarray:
    """[128, 576] byte of (row, column) in a block."""
    o = np.empty((128, 576), dtype=np.int64)
    for r in range(128):
        for c in range(576):
            if c < 512:
                o[r, c] = (c // 128) * 16384 + r * 128 + (((c % 128) // 16) ^ (r % 8)) * 16 + c % 16
            else:
                o[r, c] = 65536 + r * 64 + (((c - 512) // 16) ^ (r // 2 % 4)) * 16 + c % 16
    return o


OFFSETS = offsets()


def pack(pool: np.ndarray, blocks, rows, codes, scales) -> None:
    """Write rows into a pool uint8 [cap, BLOCK8_BYTES] in place."""
    blocks, rows = np.asarray(blocks), np.asarray(rows)
    pool[blocks[:, None], OFFSETS[rows]] = codes
    f = pool[:, SCALES_AT:].copy().view(np.float32)
    f[blocks, rows] = scales
    pool[:, SCALES_AT:] = f.view(np.uint8)


def unpack(pool: np.ndarray, blocks, rows):
    """(codes, scales) of rows of a pool."""
    blocks, rows = np.asarray(blocks), np.asarray(rows)
    return (pool[blocks[:, None], OFFSETS[rows]],
            np.ascontiguousarray(pool[:, SCALES_AT:]).view(np.float32)[blocks, rows].astype(np.float64))


def attend(rows: np.ndarray, q: np.ndarray, W_UV: np.ndarray, n_q: int, scale: float):
    """One sequence: rows [L, 576] (the values the cache stands for), absorbed queries q [n_q, H, 576], W_UV [H, 128, 512].

    Returns out [n_q, H, 128], lse [n_q, H], and for the error bounds o_lat and A = sum_t P_t |c_t| [n_q, H, 512]
    and reach = max_t sum_i |q_i c_ti| * scale [n_q, H].
    """
    L = len(rows)
    n, H = q.shape[:2]
    out, lse = np.empty((n, H, 128)), np.empty((n, H))
    o, A, reach = np.empty((n, H, 512)), np.empty((n, H, 512)), np.empty((n, H))
    for j in range(n):
        x = rows[:L - n_q + j + 1]
        s = q[j] @ x.T * scale
        m = s.max(axis=1)
        p = np.exp(s - m[:, None])
        z = p.sum(axis=1)
        p /= z[:, None]
        lse[j] = m + np.log(z)
        o[j] = p @ x[:, :512]
        A[j] = p @ np.abs(x[:, :512])
        reach[j] = (np.abs(q[j]) @ np.abs(x).T).max(axis=1) * scale
        out[j] = np.einsum("hc,hdc->hd", o[j], W_UV)
    return out, lse, o, A, reach
