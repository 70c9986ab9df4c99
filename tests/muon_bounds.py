"""How far results of full precision may be off.  TEST INFRASTRUCTURE.

Twice what the documented roundings cost on the matrix at hand
(oracle.muon.rounded; the kernels' are another draw of the same size), and
the fp32 arithmetic around them: a sum over k elements is 3 k / 32 matrix
instructions, each off by at most half a step (2^-24) of the sum so far, which
as random draws come to 2^-24 sqrt(3 k / 32); an epilogue and the statistics
round some four times more; and the polynomial's slope is at most 3.4 on the
way, taken as four.  For matrices without directions far below the others,
where errors grow from step to step, and for the norm of the difference over
the result's."""

import numpy as np

from oracle import muon as OM


def rel(x, y):
    n = np.linalg.norm(y)
    d = np.linalg.norm(np.asarray(x, np.float64) - y)
    return d / n if n else d


def arithmetic(shape):
    return 4 * 2.0 ** -24 * (np.sqrt(3 * max(shape) / 32) + 4)


def full_bound(U, exact, steps=5, coef=OM.COEF, eps=1e-7):
    model = max(rel(OM.rounded(U, steps, coef, eps, True, p), exact)
                for p in (False, True))
    return 2 * model + arithmetic(U.shape)
