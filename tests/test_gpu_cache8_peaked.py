"""decode8 where the softmax is peaked or the rows' scales differ, against 64 bits.

The tolerances are those of test_gpu_cache8.py, elementwise and in the 2-norm.  Its derivation takes every probability as
held within u of itself, or, far below the row's largest, in absolute steps whose sum over the tail keeps within u of the
whole.  The cases here are the ones in which that is hard: a tail of thousands of tokens far below one, and with a mean, so
that its sum shows in the output.
"""

import numpy as np
import pytest

from cache8_cases import bf16_values, peaked_queries, peaked_rows
from test_gpu_cache8 import Problem8

pytestmark = pytest.mark.gpu


def check(p, **kw):
    out, lse = p.decode(**kw)
    assert p.status.item() == 0
    p.check(out, lse)


def peaked(n, H, n_q=1, lengths=None, **kw):
    lengths = [n] if lengths is None else lengths
    return Problem8(lengths, H, n_q, rows=lambda b, x: peaked_rows(len(x), seed=b, **kw),
                    q=lambda v: peaked_queries(v.shape[:-1]))


@pytest.mark.parametrize("H", [16, 24, 40, 128])
@pytest.mark.parametrize("mass", [0.05, 0.5])
@pytest.mark.parametrize("at", [0, 1500])
@pytest.mark.parametrize("ratio", [1.0, 8.0])
def test_decode8_tail_behind_a_peak(H, mass, at, ratio):
    """8 K tokens in one piece; the peak first, and in the middle, where it moves what came before."""
    check(peaked(8000, H, mass=mass, at=at, ratio=ratio), num_splits=1)


@pytest.mark.parametrize("H", [16, 40, 128])
@pytest.mark.parametrize("mass,mean", [(0.05, 0.5), (0.2, 0.5), (0.8, 0.0)])
def test_decode8_long_tail_in_one_piece(H, mass, mean):
    check(peaked(32768, H, mass=mass, mean=mean), num_splits=1)


def test_decode8_equal_tail():
    """Tails of equal probabilities, 2^11 to 2^27 below the first token's: their rounding has to keep the sum."""
    for H in (16, 40, 128):
        for gap in range(8, 20, 2):
            def rows(b, x):
                y = peaked_rows(len(x), mass=0.5, spread=0.0)
                y[:, 575] = 0.0
                y[0, 575] = gap / 8.0
                return y
            check(Problem8([8192], H, 1, rows=rows, q=lambda v: peaked_queries(v.shape[:-1])), num_splits=1)


@pytest.mark.parametrize("H,n_q", [(16, 2), (128, 2), (20, 40)])
def test_decode8_tail_behind_a_peak_several_tokens(H, n_q):
    """A step of several tokens and a prompt's chunk, and a batch of as many sequences as work units."""
    check(peaked(4000, H, n_q, mass=0.3, at=7), num_splits=1)
    check(peaked(0, H, n_q, lengths=[1500, 700, 2100], mass=0.3, at=7), num_splits=3)


@pytest.mark.parametrize("H", [16, 40, 128])
def test_decode8_peaks_one_after_another(H):
    """Scores that rise and fall by 2^6 to 2^20 over several tiles, and a wide normal spread, latents with a mean."""
    for kind in range(3):
        def rows(b, x):
            n = len(x)
            y = peaked_rows(n, mass=0.5, spread=0.3, seed=kind)
            t = np.arange(n)
            s = {0: 6.0 * np.sin(t / 200.0), 1: np.where(t % 1000 < 3, 9.0, -3.0 * (t // 1500 % 2)),
                 2: 3.0 * np.random.default_rng(3).standard_normal(n)}[kind]
            y[:, 575] = s / 8.0
            return y
        check(Problem8([6000], H, 1, rows=lambda b, x: bf16_values(rows(b, x)), q=lambda v: peaked_queries(v.shape[:-1])),
              num_splits=1)
