"""Rows of an 8-bit cache whose softmax is peaked: one token above a long tail that has a share of the sum."""

import numpy as np

U = 2.0 ** -8
# The 2-norm of decode8's error (derived in test_gpu_cache8.py's docstring): probabilities within U each, out rounded.
L2 = U * np.sqrt(4 / 3)
SCORE = 8.0     # the query's column 575 is SCORE sqrt(192), and a row's column 575 its score / SCORE


def bf16_values(x):
    """fp64 rounded to bf16 (eight significant bits, ties to even), as fp64."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(m * 256) / 256, e)


def peaked_rows(n, mass, at=0, ratio=1.0, mean=0.5, spread=0.5, seed=0):
    """[n, 576] values: token `at` has the share 1 - mass of the softmax, the others `mass` together, log-normal with `spread`.

    Latents have a common mean of `mean` standard deviations, so that a tail that is lost, or has the wrong sum, shows in
    the output.  The peak's column 574 (RoPE, not asked for by the query) is `ratio` times what its latents reach, and
    so is its scale.
    """
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, 576))
    x[:, :512] = np.sqrt(1 - mean ** 2) * x[:, :512] + mean * rng.standard_normal(512)
    s = spread * rng.standard_normal(n)
    s[at] = np.log(np.exp(np.delete(s, at)).sum() * (1 - mass) / mass)
    x[:, 512:] = 0.0
    x[:, 575] = s / SCORE
    if ratio > 1:
        x[at, 574] = ratio * np.abs(x[at, :512]).max()
    return bf16_values(x)


def peaked_queries(shape, seed=0):
    """Queries [.., 576] that read the scores of peaked_rows, and a little of everything else but column 574."""
    q = 0.01 * np.random.default_rng(seed).standard_normal((*shape, 576))
    q[..., 574] = 0.0
    q[..., 575] = SCORE * np.sqrt(192.0)
    return bf16_values(q)
