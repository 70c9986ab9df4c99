"""Every kernel of the Newton-Schulz products on the GPU (muon_plan.COVER: by
the library's own plan every product, tile, precision, orientation and way
of storing), against the formulas in 64 bits.

Tolerances.  Fast precision: twice what the documented roundings cost in the
oracle's model, plus 2^-18 for fp32 sums.  Full precision:
muon_bounds.full_bound, which a product without one of its parts misses by
more than twice.  Half a step of a bf16 output besides (2^-8).  For matrices
above 1000 rows the model runs on one of the same proportions and a quarter
of the sides, whose errors are the larger ones."""

import numpy as np
import pytest
import torch

import muon_plan as P
import zero_sharded_optimizer_shard_amd as zs
from muon_bounds import full_bound, rel
from oracle import muon as OM
from oracle import step as OS
from test_muon_gpu import Case

pytestmark = pytest.mark.gpu

CASES = [(precision, last, s) for (precision, last), stacks in P.COVER.items()
         for s in stacks]


def ids(c):
    return "%s-%s-%dx%dx%d" % (c[0], {P.OUT_BF16: "bf16", P.OUT_F32: "f32",
                                      P.STEP: "step"}[c[1]], *c[2])


def exact(U, steps=5, eps=1e-7):
    """The formulas in 64 bits on the GPU, of one matrix there."""
    U = U.double()
    if U.shape[0] > U.shape[1]:
        return exact(U.t().contiguous(), steps, eps).t()
    X = U / (U.norm() + np.float64(np.float32(eps)))
    a, b, c = OM.COEF
    for _ in range(steps):
        A = X @ X.t().contiguous()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X


def bound(U, precision, steps=5):
    """U numpy, one member of the stack (or less of it)."""
    if min(U.shape) > 1000:
        U = U[:U.shape[0] // 4, :U.shape[1] // 4]
    e = OM.orthogonalize(U, steps)
    if precision == "full":
        return full_bound(U, e, steps)
    return 2 * max(rel(OM.rounded(U, steps, pairs=p), e)
                   for p in (False, True)) + 2.0 ** -18


def members(batch):
    return sorted({0, batch // 2, batch - 1})


@pytest.mark.parametrize("case", [c for c in CASES if c[1] != P.STEP], ids=ids)
def test_orthogonalize(case):
    precision, last, shape = case
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    x = torch.randn(shape, generator=g, device="cuda")
    o = torch.full(shape, 7.0, device="cuda", dtype=torch.bfloat16
                   if last == P.OUT_BF16 else torch.float32)
    ws = torch.empty(zs.zs_orthogonalize_workspace([x], precision),
                     dtype=torch.uint8, device="cuda").fill_(255)
    zs.zs_orthogonalize([x], [o], workspace=ws, precision=precision)
    t = bound(x[0].cpu().numpy(), precision)
    if last == P.OUT_BF16:
        t += 2.0 ** -8
    for k in members(shape[0]):
        e = exact(x[k])
        r = ((o[k].double() - e).norm() / e.norm()).item()
        assert r <= t, (k, r, t)


@pytest.mark.parametrize("case", [c for c in CASES if c[1] == P.STEP], ids=ids)
def test_step(case):
    """With a learning rate at which the update is the larger part of the new
    weights: its error is not lost in their rounding."""
    precision, _, shape = case
    B, R, C = shape
    layout = "tiled" if R > C else "slices"
    c = Case([shape], 2, layout, seed=sum(shape), vectors=())
    d = c.device()
    lr, wd, mu = 0.5, 0.1, 0.95
    ts = c.tensors()
    ws = torch.empty(zs.zs_muon_workspace(c.lay, ts, precision),
                     dtype=torch.uint8, device="cuda").fill_(255)
    zs.zs_muon_step(c.lay, ts, [c.grads(d, 0)], d.state, d.shard, d.flat,
                    grad_layout=layout, grad_stride=c.n, lr=lr, momentum=mu,
                    weight_decay=wd, scale="rms", precision=precision,
                    workspace=ws)
    master, mom, v = c.rows(d)
    b = c.buckets[0]
    at = slice(b.shard_off, b.shard_off + B * R * C)
    M, U = OM.momentum(OS.reduce_mean(c.G)[at], c.mom[at], mu, True)
    assert np.array_equal(mom[at].view(np.int32), M.view(np.int32))
    assert np.array_equal(v, c.v)
    bits = OS.bf16_round(master[at])
    assert np.array_equal(d.shard.cpu().numpy().view(np.uint16)[at], bits)
    flat = d.flat.cpu().numpy().view(np.uint16)
    assert np.array_equal(flat[b.flat_off:b.flat_off + B * R * C], bits)
    live = np.zeros(c.n, bool)
    live[at] = True
    assert np.array_equal(master[~live], c.master[~live])
    U = U.reshape(shape)
    t = bound(U[0], precision)
    s = OM.scale("rms", R, C)
    old, new = (a[at].reshape(shape) for a in (c.master, master))
    for k in members(B):
        O = exact(torch.from_numpy(U[k]).cuda()).cpu().numpy()
        want = OM.apply(old[k], O, lr, wd, s)
        tol = t * lr * s * np.linalg.norm(O) + \
            3 * 2.0 ** -24 * np.linalg.norm(want)
        assert np.linalg.norm(new[k] - want) <= tol
