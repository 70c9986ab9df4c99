"""zs_orthogonalize and zs_muon_step on the GPU: calls that the header allows
and whose sizes, strides, types or places differ from the ordinary ones, in
both precisions, by the kernels of small matrices and by the others.

Tolerances as in test_muon_products_gpu.py: twice what the documented
roundings cost by the oracle's model, plus fp32 arithmetic, plus half a step
of a bf16 output (2^-8)."""

import numpy as np
import pytest
import torch

import zero_sharded_optimizer_shard_amd as zs
from muon_bounds import arithmetic, full_bound, rel
from oracle import muon as OM

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
PRECISIONS = ["fast", "full"]


def gen(seed):
    return np.random.default_rng(seed)


def bound(U, e, precision, out=F32, steps=5, coef=OM.COEF, eps=1e-7):
    t = full_bound(U, e, steps, coef, eps) if precision == "full" else \
        2 * max(rel(OM.rounded(U, steps, coef, eps, pairs=p), e)
                for p in (False, True)) + 2.0 ** -18
    return t + (2.0 ** -8 if out == BF16 else 0)


def run(xs, outs, precision, **kw):
    ws = torch.empty(zs.zs_orthogonalize_workspace(xs, precision),
                     dtype=torch.uint8, device="cuda").fill_(255)
    zs.zs_orthogonalize(xs, outs, workspace=ws, precision=precision, **kw)
    return outs


def check(U, o, precision, steps=5, coef=OM.COEF, eps=1e-7):
    """U: numpy, as the call saw it."""
    e = OM.orthogonalize(U, steps, coef, eps)
    t = bound(U, e, precision, o.dtype, steps, coef, eps)
    got = o.float().cpu().numpy()
    assert np.all(np.isfinite(got))
    assert rel(got, e) <= t, (rel(got, e), t)


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("shape", [(40, 60), (200, 60), (100, 120), (70, 300),
                                   (300, 150), (450, 60)],
                         ids=lambda s: "%dx%d" % s)
def test_norms_below_eps(shape, precision):
    """X starts at |U| / (|U| + eps): a stack of matrices from far above eps
    to far below, and back."""
    rng = gen(sum(shape))
    sizes = [1.0, 1e-7, 3e-8, 1e-9, 1e-12, 1e-20, 1e-30, 1e-3]
    U = rng.standard_normal((len(sizes),) + shape)
    U = np.stack([u * s / np.linalg.norm(u) for u, s in zip(U, sizes)])
    U = U.astype(np.float32)
    for steps in (1, 5, 10):
        x = torch.from_numpy(U).cuda()
        o = run([x], [torch.empty_like(x)], precision, steps=steps)[0]
        for u, v in zip(U, o):
            check(u, v, precision, steps)
    x = torch.from_numpy(U).cuda()
    o = run([x], [torch.empty_like(x)], precision, eps=1e3)[0]
    for u, v in zip(U[:5], o):
        check(u, v, precision, eps=1e3)
    # coefficients that grow slowly, and fast
    for coef in ((1.5, -0.5, 0.0), (0.25, 0.0, 0.0), (4.5, -9.0, 6.0)):
        o = run([x], [torch.empty_like(x)], precision, steps=2, coef=coef)[0]
        for u, v in zip(U, o):
            check(u, v, precision, 2, coef)


@pytest.mark.parametrize("precision", PRECISIONS)
def test_norms_below_eps_in_twos(precision):
    rng = gen(1)
    U = rng.standard_normal((256, 1500)).astype(np.float32)
    U /= np.linalg.norm(U)
    sizes = np.float32(10.0) ** -np.arange(24, dtype=np.float32)
    x = (torch.from_numpy(U).cuda() *
         torch.from_numpy(sizes).cuda()[:, None, None])
    o = run([x], [torch.empty_like(x)], precision)[0]
    for k in (0, 5, 6, 7, 8, 12, 23):
        check(x[k].cpu().numpy(), o[k], precision)


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("shape", [(48, 64), (140, 200)],
                         ids=lambda s: "%dx%d" % s)
def test_step_of_a_momentum_below_eps(shape, precision):
    """An expert without tokens: no gradient, and a momentum that has decayed
    to nearly nothing."""
    n = shape[0] * shape[1]
    lay = zs.zs_layout_build_tensors([n], 1, 0)
    nt = lay.sizes()[2]
    m = gen(2).standard_normal(n).astype(np.float32) * np.float32(1e-15)
    state = torch.zeros(nt, 3, zs.ZS_TILE, device="cuda")
    rows = torch.zeros(nt * zs.ZS_TILE, device="cuda")
    rows[:n] = torch.from_numpy(m).cuda()
    state[:, 1] = rows.view(nt, zs.ZS_TILE)
    g = torch.zeros(lay.sizes()[1], dtype=BF16, device="cuda")
    p = torch.zeros(lay.sizes()[1], dtype=BF16, device="cuda")
    t = [(0,) + shape]
    ws = torch.empty(zs.zs_muon_workspace(lay, t, precision),
                     dtype=torch.uint8, device="cuda")
    zs.zs_muon_step(lay, t, [g], state, p, grad_stride=g.numel(), lr=1.0,
                    momentum=0.5, weight_decay=0.0, nesterov=False,
                    scale="none", precision=precision, workspace=ws)
    got = -state[:, 0].reshape(-1)[:n].view(shape)
    check((m * np.float32(0.5)).reshape(shape), got, precision)


def directions(rng, m, n, k, f):
    """k directions f times the strongest of the noise below them."""
    q = lambda a, b: np.linalg.qr(rng.standard_normal((a, b)))[0]  # noqa
    w = rng.standard_normal((m, n))
    return w / np.linalg.norm(w, 2) + f * q(m, k) @ q(n, k).T


def decay(rng, m, n, p):
    """Singular values k^-p."""
    q = lambda a, b: np.linalg.qr(rng.standard_normal((a, b)))[0]  # noqa
    return (q(m, m) * np.arange(1., m + 1) ** -p) @ q(n, m).T


def lowrank(rng, m, n, k):
    return rng.standard_normal((m, k)) @ rng.standard_normal((k, n))


def entry(rng, m, n, size):
    U = rng.standard_normal((m, n))
    U[3, 5] = size
    return U


# kind, and the header's figures for five steps: fast, full
SPECTRA = {
    "noise": (lambda r: r.standard_normal((256, 1024)), 1e-3, 2e-6),
    "noise 64": (lambda r: r.standard_normal((64, 128)), 1e-3, 2e-6),
    "long tails": (lambda r: r.standard_t(2, (300, 70)), 2e-3, 2e-6),
    "8 x 30": (lambda r: directions(r, 256, 1024, 8, 30), 1e-3, 2e-6),
    "8 x 100": (lambda r: directions(r, 256, 3000, 8, 100), 2e-3, 2e-5),
    "8 x 100, 64": (lambda r: directions(r, 64, 300, 8, 100), 2e-3, 2e-5),
    "1/k": (lambda r: decay(r, 256, 3000, 1), 2e-3, 2e-5),
    "1/k^2": (lambda r: decay(r, 64, 300, 2), 2e-3, 2e-5),
    "8 x 100, 32": (lambda r: directions(r, 32, 1200, 8, 100), 3e-3, 1e-5),
    "1 x 100, 2": (lambda r: directions(r, 2, 1200, 1, 100), 5e-3, 1e-5),
    "8 x 1000, 32": (lambda r: directions(r, 32, 1200, 8, 1000), 7e-3, 5e-5),
    "8 x 1000, 64": (lambda r: directions(r, 64, 1200, 8, 1000), 7e-3, 5e-5),
    "mean": (lambda r: 1000 + r.standard_normal((256, 2048)), 7e-3, 5e-5),
    "rank 8": (lambda r: lowrank(r, 64, 256, 8), 7e-3, 5e-5),
    "rank 8, tall": (lambda r: lowrank(r, 1024, 256, 8), 7e-3, 5e-5),
    "1 x 1000, 2": (lambda r: directions(r, 2, 1200, 1, 1000), 4e-2, 5e-5),
    "entry 1e6": (lambda r: entry(r, 256, 1024, 1e6), 2e-3, 1e-5),
    "entry 1e8": (lambda r: entry(r, 256, 1024, 1e8), 2e-3, 1e-5),
}


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("kind", SPECTRA)
def test_accuracy_by_kind_of_matrix(kind, precision):
    """The header's figures at five steps.  At 5 to 10: twice the oracle's
    model, and in full precision fp32 arithmetic of which the first step's
    grows by a in each of the others where the matrix has nothing."""
    make, fast, full = SPECTRA[kind]
    U = make(gen(50)).astype(np.float32)
    x = torch.from_numpy(U).cuda().expand(8, *U.shape)
    for steps in (5, 6, 8, 10):
        o = run([x], [torch.empty(x.shape, device="cuda")], precision,
                steps=steps)[0]
        e = OM.orthogonalize(U, steps)
        t = bound(U, e, precision, F32, steps)
        if precision == "full":
            t += arithmetic(U.shape) * OM.COEF[0] ** (steps - 1) / \
                np.linalg.norm(e)
        got = rel(o[0].cpu().numpy(), e)
        assert got <= t, (steps, got, t)
        if steps == 5:
            assert got <= (full if precision == "full" else fast), got
        assert torch.equal(o[7], o[0])
