"""A bound on the 2-norm of an output row's error in the latent attention tests.

The bounds per element are worst cases: every rounding in the same direction, sum_n
p_n |v_n|, which for a long context is some 30 times the output itself, so that a lost
tile of keys stays below them. Errors of single keys do not add up like that. A row's
error is, with u half a bf16 step,
  * sum_n d_n p_n v_n, each weight off by |d_n| <= u. The part that the d_n have in
    common (equal weights round alike) is at most u |o|. What is left varies from key
    to key with at most u / sqrt(3) root mean square (a uniform error): its square
    adds up key by key, to u / sqrt(3) sqrt(sum_n p_n^2 |v_n|^2) expected;
  * the scores' errors, e_n in absolute terms, as relative errors of the weights, the
    same two ways;
  * E4M3 cells: weights cut at 2^-24 of the largest p_n s_n, on codes v_n / s_n;
  * u |o| of the output's own rounding.
The parts that vary are taken four times: over 128 dims and more a norm is within a
few tenths of its expectation, so four times is not met by chance."""
import numpy as np

from tests import latent_reference as ref

TIMES = 4.0


def bound(p, v, want, score_error, scales=None):
    """Bound for rows p [..][N] (weights), v [N][D] and want [..][D] = p v;
    score_error [..] absolute, of the rows' scores."""
    u = ref.BF16_HALF
    size2 = (v ** 2).sum(-1)
    spread = np.sqrt(p ** 2 @ size2)
    norm = np.linalg.norm(want, axis=-1)
    tol = 2 * u * norm + TIMES / np.sqrt(3) * u * spread
    tol = tol + score_error * (norm + TIMES * spread)
    if scales is not None:
        cut = 2.0 ** -24 * (p * scales).max(-1)
        seen = (p > 0).astype(np.float64)
        tol = tol + TIMES / np.sqrt(3) * cut * np.sqrt(seen @ (size2 / scales ** 2))
    return tol


def absorbed_bound(q, c, kr, p, want, scale, scales=None):
    """q [Tq][H][L + 64], c [N][L], kr [N][64]; the scores' error as in the tests by
    element: 2^-20 of scale sum |q||k|, and on E4M3 cells 2^-17 of the row's largest
    query element on the latent part."""
    k = np.concatenate((c, kr), -1)
    e = 2.0 ** -20 * scale * (np.abs(q) @ np.abs(k).T).max(-1)
    if scales is not None:
        e = e + scale * 2.0 ** -17 * np.abs(q[..., :c.shape[-1]]).max(-1) * np.abs(c).sum(-1).max()
    return bound(p, c, want, e, scales)
