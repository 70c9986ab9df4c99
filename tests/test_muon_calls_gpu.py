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
from test_muon_gpu import Case
from test_muon_products_gpu import exact

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


# small matrices (one launch) and others, wide and tall, columns a multiple of
# four and not
SHAPES = [(60, 72), (250, 33), (66, 200), (200, 72), (140, 150), (70, 333)]


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("xt,ot", [(BF16, BF16), (BF16, F32), (F32, BF16)],
                         ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
def test_types(shape, xt, ot, precision):
    x = torch.from_numpy(gen(3).standard_normal(shape)).cuda().to(xt)
    o = run([x], [torch.empty(shape, dtype=ot, device="cuda")], precision)[0]
    check(x.double().cpu().numpy(), o, precision)


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("gap", [24, 23])
@pytest.mark.parametrize("pitch,off", [(0, 0), (5, 0), (8, 0), (3, 1), (8, 1),
                                       (64, 4)])
def test_strides_and_alignment(pitch, off, gap, dtype, precision):
    """Stacks in wider buffers: every base, pitch and distance of the members
    that decides between loads by fours and one by one, in and out apart."""
    b = 2
    for r, c in SHAPES[1:]:
        U = gen(r).standard_normal((b, r, c))

        def place(fill, pitch, off):
            step = r * (c + pitch) + gap
            buf = torch.full((off + b * step,), fill, dtype=dtype,
                             device="cuda")
            return buf, torch.as_strided(buf, (b, r, c),
                                         (step, c + pitch, 1), off)

        plain = place(0.0, 0, 0)[1] if gap % 4 == 0 else \
            torch.empty(b, r, c, dtype=dtype, device="cuda")
        for xs, os in ((True, False), (False, True), (True, True)):
            xb, x = place(3.0, pitch, off)
            ob, o = place(5.0, pitch, off)
            if not xs:
                x = torch.empty(b, r, c, dtype=dtype, device="cuda")
            x.copy_(torch.from_numpy(U))
            if not os:
                o = plain
            keep, kx = ob.clone(), x.clone()
            run([x], [o], precision)
            assert torch.equal(x, kx)
            if xs and not os:           # the first of the three
                for k in range(b):
                    check(x[k].double().cpu().numpy(), o[k], precision)
                want = o.clone()
            assert torch.equal(o, want)
            if os:
                torch.as_strided(keep, o.shape, o.stride(), off).copy_(o)
                assert torch.equal(ob, keep)    # nothing else was written


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("shape", [(70, 300), (300, 150), (2050, 2056)],
                         ids=lambda s: "%dx%d" % s)
@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e15, 1e30])
def test_any_magnitude(size, shape, precision):
    """The norm is taken in 64 bits by the kernels of large matrices too."""
    U = gen(4).standard_normal(shape).astype(np.float32) * np.float32(size)
    eps = 1e-7 if size > 1 else size * 1e-3
    x = torch.from_numpy(U).cuda()
    o = run([x], [torch.empty_like(x)], precision, eps=eps)[0]
    if shape[0] < 1000:
        check(U, o, precision, eps=eps)
        return
    # the formulas in 64 bits on the GPU; the bound from a quarter of the
    # sides, whose errors are the larger ones
    V = U[:shape[0] // 4, :shape[1] // 4]
    t = bound(V, OM.orthogonalize(V, eps=eps), precision, eps=eps)
    e = exact(x, eps=eps)
    assert ((o.double() - e).norm() / e.norm()).item() <= t


def test_norm_of_many_parts():
    """More partial sums than a workgroup adds on its way, at sizes whose
    squares fp32 does not hold."""
    x = torch.randn(4104, 4100, device="cuda",
                    generator=torch.Generator("cuda").manual_seed(5))
    want = run([x], [torch.empty_like(x)], "fast", steps=1, coef=(1., 0., 0.))
    e = x.double() / (x.double().norm() + 1e-7)
    t = 2.0 ** -21
    assert (want[0].double() - e).norm() <= t * e.norm()
    y = x * 2.0 ** 100
    got = run([y], [torch.empty_like(y)], "fast", steps=1, coef=(1., 0., 0.))
    assert (got[0].double() - e).norm() <= t * e.norm()


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("shape", [(3, 60, 72), (3, 130, 300), (3, 400, 70),
                                   (24, 256, 1500)],
                         ids=lambda s: "%dx%dx%d" % s)
def test_in_place(shape, dtype, precision):
    x = torch.from_numpy(gen(6).standard_normal(shape)).cuda().to(dtype)
    want = run([x], [torch.empty_like(x)], precision)[0]
    run([x], [x], precision)
    assert torch.equal(x, want)


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("shape", [(60, 72), (150, 200), (24, 256, 1500)],
                         ids=str)
def test_captured_calls(shape, precision):
    """Replays on new inputs and a spoilt workspace, eager work between."""
    rng = gen(7)
    xs = [torch.from_numpy(rng.standard_normal(shape)).cuda().float()
          for _ in range(4)]
    want = [run([x], [torch.empty_like(x)], precision)[0] for x in xs]
    x, o = xs[0].clone(), torch.empty_like(xs[0])
    ws = torch.empty(zs.zs_orthogonalize_workspace([x], precision),
                     dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        zs.zs_orthogonalize([x], [o], workspace=ws, precision=precision)
    for k in (0, 1, 2, 3, 0):
        x.copy_(xs[k])
        ws.fill_(255)
        o.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[k])
        assert torch.equal(run([x], [torch.empty_like(x)], precision)[0], o)


@pytest.mark.parametrize("shape", [(60, 72), (900, 1100), (24, 256, 1500)],
                         ids=str)
def test_two_calls_at_once(shape):
    """Two streams, a workspace each, one call in each precision."""
    xs = [torch.from_numpy(gen(8 + k).standard_normal(shape)).cuda().float()
          for k in range(2)]
    want = [run([x], [torch.empty_like(x)], p)[0]
            for x, p in zip(xs, PRECISIONS)]
    ws = [torch.empty(zs.zs_orthogonalize_workspace([x], p),
                      dtype=torch.uint8, device="cuda")
          for x, p in zip(xs, PRECISIONS)]
    outs = [torch.empty_like(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(4):
        for x, o, w, st, p in zip(xs, outs, ws, streams, PRECISIONS):
            zs.zs_orthogonalize([x], [o], workspace=w, stream=st, precision=p)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("shape", [(256, 64), (512, 700), (24, 256, 1500)],
                         ids=str)
def test_same_bits_every_time(shape, precision):
    x = torch.from_numpy(gen(9).standard_normal(shape)).cuda().float()
    a = run([x], [torch.empty_like(x)], precision)[0]
    for _ in range(3):
        assert torch.equal(run([x], [torch.empty_like(x)], precision)[0], a)


@pytest.mark.parametrize("layout", ["slices", "tiled"])
@pytest.mark.parametrize("W", [1, 3, 8])
def test_step_in_full_precision(W, layout):
    """Five steps of small matrices and others together."""
    c = Case([(130, 70), (70, 340), (3, 40, 36), (1, 515), (513, 1),
              (2, 90, 91)], W, layout, seed=60 + W)
    d = c.device()
    c.step(d, "full", nesterov=W != 3)
    c.check(d, "full", nesterov=W != 3)


@pytest.mark.parametrize("precision", PRECISIONS)
def test_steps_at_once(precision):
    """Two owners' steps on two streams, a workspace each."""
    cs = [Case([(130, 270), (3, 40, 36), (200, 150)], 2, "tiled",
               seed=70 + k) for k in range(2)]
    want, ds = [], []
    for c in cs:
        d = c.device()
        for _ in range(3):
            c.step(d, precision)
        want.append(d)
        ds.append(c.device())
    ws = [torch.empty(zs.zs_muon_workspace(c.lay, c.tensors(), precision),
                      dtype=torch.uint8, device="cuda") for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, d, w, st in zip(cs, ds, ws, streams):
            c.step(d, precision, ws=w, stream=st)
    torch.cuda.synchronize()
    for a, b in zip(want, ds):
        assert torch.equal(a.state, b.state)
        assert torch.equal(a.shard, b.shard) and torch.equal(a.flat, b.flat)


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("shape", [(48, 72), (70, 300)],
                         ids=lambda s: "%dx%d" % s)
@pytest.mark.parametrize("far", ["members", "rows"])
def test_offsets_past_32_bits(far, shape, precision):
    """Members, and rows, more than 2^32 elements from the first."""
    r, c = shape
    U = gen(10).standard_normal((2, r, c)).astype(np.float32)
    step, row = ((1 << 32) + 4, c) if far == "members" else \
        ((1 << 20), (1 << 32) // (r - 1) + 4)

    def place(dtype):
        span = step + (r - 1) * row + c
        return torch.as_strided(torch.empty(span, dtype=dtype, device="cuda"),
                                (2, r, c), (step, row, 1))
    x = place(BF16)
    x.copy_(torch.from_numpy(U))
    o = run([x], [place(BF16)], precision)[0]
    for k in range(2):
        check(x[k].double().cpu().numpy(), o[k], precision)


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("shape", [(1, 1 << 22), (3, 1 << 22), (1 << 22, 2)],
                         ids=lambda s: "%dx%d" % s)
def test_longest_matrices(shape, precision):
    """2^-18 is for sums of a few thousand; these have 2^17 additions of a
    chain of 32 products, 2^-24 sqrt(2^17) = 2e-5 of the sum each as random
    draws, which muon_bounds.arithmetic counts (1.5e-4)."""
    U = gen(11).standard_normal(shape).astype(np.float32)
    x = torch.from_numpy(U).cuda()
    o = run([x], [torch.empty_like(x)], precision)[0]
    e = OM.orthogonalize(U)
    t = bound(U, e, precision) + arithmetic(U.shape)
    assert rel(o.cpu().numpy(), e) <= t


@pytest.mark.parametrize("precision", PRECISIONS)
def test_largest_matrix(precision):
    """The longest smaller side, one step: its products have sums as long as
    any, so the bound of one row of such a matrix holds for it."""
    n = 32768
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(n, n, generator=g, device="cuda").bfloat16()
    o = run([x], [torch.empty_like(x)], precision, steps=1)[0]
    # b A + c A A of X, row by row of the result: a few of them, in 64 bits
    X = x.double()
    X /= X.norm() + np.float64(np.float32(1e-7))
    a, b, c = OM.COEF
    for i in (0, 1, 191, 192, 20000, n - 1):
        row = X[i:i + 1]
        A = (X @ row.t().contiguous()).t().contiguous()     # row i of A
        AA = (X @ (A @ X).t().contiguous()).t()
        e = a * row + (b * A + c * AA) @ X
        got = o[i:i + 1].double()
        # one step rounds its update by 2^-11 of C's off-diagonal part, whose
        # size beside a is below 1/100 here, and the result to bf16
        t = 2.0 ** -8 + 2.0 ** -16
        assert ((got - e).norm() / e.norm()).item() <= t


@pytest.mark.parametrize("layout", ["slices", "tiled"])
def test_step_behind_a_tensor_of_2_to_the_32(layout):
    """A matrix whose state, gradients and outputs lie past 32 bits."""
    r, c = 130, 72
    n, W = r * c, 2
    big = (1 << 32) + 1000
    lay = zs.zs_layout_build_tensors([big, big, n, n], W, 0)
    flat_numel, shard, tiles, _, buckets = lay.sizes()
    b = buckets[1]
    assert b.slice_numel < 2 * n and b.shard_off > 1 << 32
    rng = gen(13)
    G = rng.standard_normal((W, n))
    P0, M0 = (rng.standard_normal(n).astype(np.float32) for _ in range(2))
    nt = tiles - b.tile_off
    state = torch.empty(tiles, 3, zs.ZS_TILE, device="cuda")
    rows = torch.zeros(3, nt * zs.ZS_TILE)
    rows[0, :n], rows[1, :n] = torch.from_numpy(P0), torch.from_numpy(M0)
    state[b.tile_off:] = rows.view(3, nt, zs.ZS_TILE).transpose(0, 1).cuda()
    g = torch.from_numpy(G).to(BF16)
    if layout == "tiled":
        grads = torch.zeros(nt, W, zs.ZS_TILE, dtype=BF16)
        for s in range(W):
            row = torch.zeros(nt * zs.ZS_TILE, dtype=BF16)
            row[:n] = g[s]
            grads[:, s] = row.view(nt, zs.ZS_TILE)
        grads, stride = grads.cuda(), 0
    else:                               # rows of whole-shard gradients
        stride = shard
        whole = torch.empty(W * shard, dtype=BF16, device="cuda")
        grads = whole[b.shard_off:]
        for s in range(W):
            grads[s * stride:s * stride + n] = g[s].cuda()
    p = torch.empty(shard, dtype=BF16, device="cuda")
    flat = torch.empty(flat_numel, dtype=BF16, device="cuda")
    t = [(1, r, c)]
    ws = torch.empty(zs.zs_muon_workspace(lay, t, "full"), dtype=torch.uint8,
                     device="cuda")
    zs.zs_muon_step(lay, t, [grads], state, p, flat, grad_layout=layout,
                    grad_stride=stride, lr=0.5, momentum=0.9,
                    weight_decay=0.1, precision="full", workspace=ws)
    mean = (g[0].float().numpy() + g[1].float().numpy()) / np.float32(2)
    M, U = OM.momentum(mean, M0, 0.9, True)
    got = state[b.tile_off:].transpose(0, 1).reshape(3, -1)[:, :n].cpu()
    assert np.array_equal(got[1].numpy(), M)
    U = U.reshape(r, c)
    O = OM.orthogonalize(U)
    s = OM.scale("rms", r, c)
    want = OM.apply(P0, O.ravel(), 0.5, 0.1, s)
    tol = full_bound(U, O) * 0.5 * s * np.linalg.norm(O) + \
        3 * 2.0 ** -24 * np.linalg.norm(want)
    assert np.linalg.norm(got[0].numpy() - want) <= tol
    for out, off in ((p, b.shard_off), (flat, b.flat_off)):
        assert torch.equal(out[off:off + n].cpu(), got[0].to(BF16))
