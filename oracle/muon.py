"""Newton-Schulz orthogonalisation and the Muon step in float64 (numpy).

TEST INFRASTRUCTURE: see oracle/__init__.py.  Written from the formulas:

  X = U / (|U|_F + eps);   A = X X^T,  X <- a X + (b A + c A A) X  per step
  (X^T X and X (b A + c A A) for more rows than columns)

  g = mean of the W slices;  M = mu M + g;  U = g + mu M or M
  master = master (1 - lr wd) - lr s orth(U);  param = bf16(master)

`rounded` is the same iteration with fp16 roundings at the places the
library documents for its precision: what they cost on given inputs is the
measure its results are held to.
"""

from __future__ import annotations

import numpy as np

COEF = (3.4445, -4.7750, 2.0315)


def rows_of(coef, steps):
    return [tuple(coef)] * steps if np.ndim(coef[0]) == 0 else list(coef)


def start(U, eps):
    U = np.asarray(U, np.float64)
    n = np.sqrt(np.sum(U * U))
    return U / (n + np.float64(np.float32(eps)))


def orthogonalize(U, steps=5, coef=COEF, eps=1e-7):
    """One matrix, float64."""
    U = np.asarray(U, np.float64)
    if U.shape[0] > U.shape[1]:
        return orthogonalize(U.T, steps, coef, eps).T
    X = start(U, eps)
    for a, b, c in rows_of(coef, steps):
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return X


def _f16(x):
    """Round to fp16 at the library's scale of 2^10."""
    with np.errstate(over="ignore"):
        return (x * 1024).astype(np.float16).astype(np.float64) / 1024


def chain_of(steps, pairs, full=False):
    """Steps taken together: in full precision twos, an odd count's single one
    second; else the first two."""
    if not pairs or steps < 2:
        return [1] * steps
    if full:
        out = [2] * (steps // 2)
        if steps % 2:
            out.insert(1, 1)
        return out
    return [2] + [1] * (steps - 2)


def exponent(U, eps):
    """The library holds a matrix whose norm is below eps as 2^e X, with
    2^e |X| in [1/2, 1)."""
    n = np.sqrt(np.sum(np.asarray(U, np.float64) ** 2))
    t = n / (n + np.float64(np.float32(eps)))
    return max(0, -int(np.frexp(t)[1])) if t > 0 else 0


def shift_of(a, b, c):
    """Bits a step takes from e: it multiplies s <= 1/4 by at most 2^t."""
    return max(0, int(np.ceil(np.log2(abs(a) + abs(b) / 16 + abs(c) / 256))))


def rounded(U, steps=5, coef=COEF, eps=1e-7, full=False, pairs=False,
            drop=None):
    """One matrix, with the library's fp16 roundings and exact sums; `pairs`:
    two steps taken together on the smaller side, as the library does where
    that is less work.  `drop`: a mistake, for tests of tolerances: which
    product ("gram", "poly", "prod" or "update") of full precision lacks its
    high x low ("hl") or low x high ("lh") part."""
    U = np.asarray(U, np.float64)
    if U.shape[0] > U.shape[1]:
        return rounded(U.T, steps, coef, eps, full, pairs, drop).T

    def pair(x):
        hi = _f16(x)
        return hi, _f16(x - hi)

    def times(p, q, what):
        s = p[0] @ q[0]
        if full and drop != (what, "hl"):
            s = s + p[0] @ q[1]
        if full and drop != (what, "lh"):
            s = s + p[1] @ q[0]
        return s

    def square(M):
        """fp16 without the diagonal (a pair if full), and the diagonal; one
        triangle counts for both."""
        M = np.tril(M) + np.tril(M, -1).T
        d = M.diagonal().copy()
        h, l = pair(M - np.diag(d))
        return (h, l if full else np.zeros_like(l)), d

    def whole(M):
        return M[0][0] + M[0][1] + np.diag(M[1])

    def product(M, N, what="prod"):
        (R, d), (S, f) = M, N
        return (times(R, S, what) + d[:, None] * (S[0] + S[1]) +
                (R[0] + R[1]) * f[None] + np.diag(d * f))

    e = exponent(U, eps)
    X = start(U, eps) * 2.0 ** e
    rows = rows_of(coef, steps)
    k = 0
    for many in chain_of(steps, pairs, full):
        x = pair(X)
        A = square(times(x, (x[0].T, x[1].T), "gram"))
        E = None
        for q in range(many):
            a, b, c = rows[k]
            e1 = max(e - shift_of(a, b, c), 0)
            a, b, c = (a * 2.0 ** (e1 - e), b * 2.0 ** (e1 - 3 * e),
                       c * 2.0 ** (e1 - 5 * e))
            e = e1
            k += 1
            M = b * whole(A) + c * product(A, A, "poly")
            C = square(M + a * np.eye(len(M)))
            E = C if E is None else square(product(C, E))
            if q + 1 < many:
                A = square(product(square(product(C, A)), C))
        X = E[1][:, None] * (x[0] + x[1]) + times(E[0], x, "update")
    return X * 2.0 ** -e


def scale(mode, rows, cols):
    return {"none": 1.0, "shape": max(1.0, rows / cols) ** 0.5,
            "rms": 0.2 * max(rows, cols) ** 0.5}[mode]


def momentum(g, m, mu, nesterov):
    """fp32, one rounding per operation: (M, U) from g and the old M."""
    f = np.float32
    m = f(mu) * m + g
    return m, (g + f(mu) * m if nesterov else m)


def apply(master, O, lr, wd, s):
    """float64: the stepped weights, from fp32 ones and O."""
    lr, wd = np.float64(np.float32(lr)), np.float64(np.float32(wd))
    return master.astype(np.float64) * (1 - lr * wd) - lr * s * O
