"""zs_orthogonalize and zs_muon_step on the GPU against the float64 oracle.

Tolerances.  What the documented fp16 roundings cost on a test's own inputs
is computed on the CPU (oracle.muon.rounded: float64 with those roundings,
steps one by one and in twos: which of them a call takes goes by the sizes of
all its matrices).
The kernels make the same roundings of values that differ in their last
bits, so their error is another draw of the same size: they are held to
twice the oracle's, plus 2^-18 for fp32 sums and the statistics of small
matrices, where few roundings are drawn (in the 2-norm over the result's
norm), plus half a step of the output's type.  Full precision rounds to
2^-22, below the fp32 arithmetic around it: its products and epilogues round
each value of a step a few times to 2^-24, the polynomial multiplies that by
at most 4 a step in the directions that are still growing (its slope at zero
is 3.4), so 2^-24 * 8 * 4^5 / sqrt(3) would be the worst of one direction
and 2^-13 bounds all.
"""

import numpy as np
import pytest
import torch

import zero_sharded_optimizer_shard_amd as zs
from oracle import muon as OM
from oracle import step as OS
from oracle.layout import build_tensor_layout

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def gen(seed):
    return np.random.default_rng(seed)


def matrix(rng, r, c, kind="noise"):
    if kind == "noise":
        x = rng.standard_normal((r, c))
    elif kind == "lowrank":                 # no noise at all: null directions
        k = max(1, min(r, c) // 32)
        x = rng.standard_normal((r, k)) @ rng.standard_normal((k, c))
    elif kind == "zero":
        x = np.zeros((r, c))
    else:                                   # strong directions over a floor
        k = max(1, min(r, c) // 32)
        x = rng.standard_normal((r, k)) @ rng.standard_normal((k, c))
        x += 0.3 * rng.standard_normal((r, c))
    return (x * 1e-3).astype(np.float32)


def run(mats, outs, precision="fast", poison=True, **kw):
    n = zs.zs_orthogonalize_workspace(mats, precision)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    if poison:                              # NaN in every type
        ws.fill_(255)
    zs.zs_orthogonalize(mats, outs, workspace=ws, precision=precision, **kw)
    return outs


def rel(x, y):
    n = np.linalg.norm(y)
    d = np.linalg.norm(np.asarray(x, np.float64) - y)
    return d / n if n else d


def bound(U, exact, precision, out, steps=5, coef=OM.COEF, eps=1e-7):
    if precision == "full":
        t = 2.0 ** -13
    else:
        t = 2 * max(rel(OM.rounded(U, steps, coef, eps, pairs=p), exact)
                    for p in (False, True)) + 2.0 ** -18
    return t + (2.0 ** -8 if out == torch.bfloat16 else 0)


def check(U, O, precision="fast", steps=5, coef=OM.COEF, eps=1e-7):
    """U numpy [r, c] as the call saw it, O the output tensor."""
    exact = OM.orthogonalize(U, steps, coef, eps)
    got = O.float().cpu().numpy()
    assert np.all(np.isfinite(got))
    t = bound(U, exact, precision, O.dtype, steps, coef, eps)
    assert rel(got, exact) <= t, (rel(got, exact), t)


SHAPES = [(1, 1), (1, 7), (7, 1), (3, 5), (64, 64), (63, 65), (65, 63),
          (64, 128), (127, 129), (128, 128), (129, 257), (257, 129),
          (192, 448), (300, 1000), (1000, 300), (1, 4099), (4099, 1),
          (515, 513), (768, 320), (50, 500), (500, 50), (100, 128),
          (128, 97), (33, 250), (250, 33)]


@pytest.mark.parametrize("precision", ["fast", "full"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
def test_shapes(shape, precision):
    rng = gen(sum(shape))
    U = matrix(rng, *shape)
    x = torch.from_numpy(U).cuda()
    o = torch.full_like(x, 7.0)
    run([x], [o], precision)
    check(U, o, precision)
    assert torch.equal(x.cpu(), torch.from_numpy(U))


@pytest.mark.parametrize("kind", ["lowrank", "strong"])
@pytest.mark.parametrize("shape", [(128, 128), (96, 640), (640, 96)],
                         ids=lambda s: "%dx%d" % s)
@pytest.mark.parametrize("precision", ["fast", "full"])
def test_spectra(kind, shape, precision):
    U = matrix(gen(3), *shape, kind)
    x = torch.from_numpy(U).cuda()
    o = run([x], [torch.empty_like(x)], precision)[0]
    check(U, o, precision)


@pytest.mark.parametrize("xt,ot", [(torch.bfloat16, torch.bfloat16),
                                   (torch.bfloat16, torch.float32),
                                   (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("shape", [(67, 130), (130, 68)],
                         ids=lambda s: "%dx%d" % s)
def test_types(xt, ot, shape):
    x = torch.from_numpy(matrix(gen(4), *shape)).cuda().to(xt)
    o = run([x], [torch.empty(shape, dtype=ot, device="cuda")])[0]
    check(x.float().cpu().numpy(), o)


@pytest.mark.parametrize("steps,coef", [
    (1, OM.COEF), (2, OM.COEF), (8, OM.COEF), (3, (1.5, -0.5, 0.0)),
    (3, [(4.0, -6.0, 2.9), (3.4445, -4.775, 2.0315), (2.0, -1.5, 0.5)])])
def test_steps_and_coefficients(steps, coef):
    U = matrix(gen(5), 100, 140)
    x = torch.from_numpy(U).cuda()
    for precision in ("fast", "full"):
        o = run([x], [torch.empty_like(x)], precision, steps=steps,
                coef=coef)[0]
        check(U, o, precision, steps, coef)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pitch,off", [(0, 0), (5, 0), (8, 0), (3, 1),
                                       (64, 4)])
def test_strides_and_alignment(dtype, pitch, off):
    """A stack in a wider buffer, read and written in place of nothing else."""
    b, r, c = 3, 66, 72
    rng = gen(6)
    U = np.stack([matrix(rng, r, c) for _ in range(b)])

    def place(fill):
        buf = torch.full((off + b * (r * (c + pitch) + 24),), fill,
                         dtype=dtype, device="cuda")
        return buf, torch.as_strided(
            buf, (b, r, c), (r * (c + pitch) + 24, c + pitch, 1), off)

    xb, x = place(3.0)
    x.copy_(torch.from_numpy(U))
    ob, o = place(5.0)
    keep = ob.clone()
    run([x], [o])
    for k in range(b):
        check(x[k].float().cpu().numpy(), o[k])
    torch.as_strided(keep, o.shape, o.stride(), off).copy_(o)
    assert torch.equal(ob, keep)            # nothing else was written


@pytest.mark.parametrize("precision", ["fast", "full"])
@pytest.mark.parametrize("shape", [(2, 1984, 2050), (5, 900, 2304),
                                   (3, 2304, 1100), (36, 700, 330),
                                   (1, 256, 20000)],
                         ids=lambda s: "%dx%dx%d" % s)
def test_large_tiles(shape, precision):
    """Sizes at which the larger tiles carry the products, one matrix of the
    stack against float64 on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    x = torch.randn(shape, generator=g, device="cuda")
    o = run([x], [torch.empty_like(x)], precision)[0]
    for k in (0, shape[0] - 1):
        U = x[k].double()
        U = (U.t() if shape[1] > shape[2] else U).contiguous()
        X = U / (U.norm() + np.float64(np.float32(1e-7)))
        a, b, c = OM.COEF
        for _ in range(5):
            A = X @ X.t().contiguous()
            X = a * X + (b * A + c * (A @ A)) @ X
        got = (o[k].t() if shape[1] > shape[2] else o[k]).double()
        r = ((got - X).norm() / X.norm()).item()
        # roundings drawn by the million: those of a smaller matrix of the
        # same proportions, whose errors are the larger ones
        small = [max(8, s // 8) for s in U.shape]
        V = matrix(gen(1), *small)
        t = bound(V, OM.orthogonalize(V), precision, torch.float32)
        assert r <= t, (r, t)


@pytest.mark.parametrize("shape", [(4, 66, 72), (3, 150, 70), (3, 40, 31)],
                         ids=lambda s: "%dx%dx%d" % s)
def test_outputs_side_by_side(shape):
    """Heads of one matrix: the stack's members share its rows, in place too."""
    h, r, c = shape
    rng = gen(14)
    U = np.stack([matrix(rng, r, c) for _ in range(h)])
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.full((r, h * c + 5), 3.0, device="cuda", dtype=dtype)
        o = buf[:, :h * c].view(r, h, c).transpose(0, 1)
        x = torch.from_numpy(U).cuda().to(dtype)
        run([x], [o])
        for k in range(h):
            check(x[k].float().cpu().numpy(), o[k])
        assert torch.all(buf[:, h * c:] == 3)
        want = o.clone()
        o.copy_(x)
        run([o], [o])
        assert torch.equal(o, want)


def test_in_place_and_broadcast_input():
    U = matrix(gen(7), 130, 70)
    x = torch.from_numpy(U).cuda()
    run([x], [x])
    check(U, x)
    one = torch.from_numpy(U).cuda()
    o = torch.empty(4, 130, 70, device="cuda")
    run([one.expand(4, 130, 70)], [o])
    for k in range(4):
        assert torch.equal(o[k], x)


def test_group_of_shapes_equals_single_calls():
    rng = gen(8)
    shapes = [(64, 64), (5, 130, 33), (1, 1), (200, 72), (0, 8, 8), (2, 0, 5),
              (2, 128, 256), (513, 40)]
    xs = [torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()
          for s in shapes]
    for precision in ("fast", "full"):
        a = run(xs, [torch.empty_like(x) for x in xs], precision)
        for x, o in zip(xs, a):
            if x.numel():
                s = run([x], [torch.empty_like(x)], precision)[0]
                ref = s.cpu().numpy()
                # steps in twos or one by one, by all sizes of the call
                assert rel(o.cpu().numpy(), ref.astype(np.float64)) < 2.0 ** -7
                m = x if x.dim() == 2 else x[-1]
                check(m.cpu().numpy(), o if x.dim() == 2 else o[-1],
                      precision)
    assert run(xs[4:6], [torch.empty_like(x) for x in xs[4:6]]) is not None


@pytest.mark.parametrize("steps", [2, 3, 4, 6, 8])
def test_steps_of_a_stack(steps):
    """A dozen directions some twenty times as strong as the others, in a
    stack that takes steps in twos."""
    rng = gen(13)
    U = (rng.standard_normal((384, 12)) @ rng.standard_normal((12, 1500)) +
         rng.standard_normal((384, 1500))).astype(np.float32)
    x = torch.from_numpy(U).cuda().expand(24, 384, 1500)
    o = torch.empty(24, 384, 1500, device="cuda")
    run([x], [o], steps=steps)
    check(U, o[0], steps=steps)
    assert torch.equal(o[23], o[0])


@pytest.mark.parametrize("kind,steps", [("8", 5), ("8", 6), ("k", 5)])
def test_stack_of_strong_directions(kind, steps):
    """Eight directions a hundred times the others, or singular values 1/k,
    in a stack that takes steps in twos: as exact as one by one."""
    rng = gen(15)
    q = lambda a, b: np.linalg.qr(rng.standard_normal((a, b)))[0]  # noqa
    if kind == "k":
        U = (q(256, 256) / np.arange(1, 257)) @ q(3000, 256).T
    else:
        U = rng.standard_normal((256, 3000))
        U = U / np.linalg.norm(U, 2) + 100 * q(256, 8) @ q(3000, 8).T
    U = U.astype(np.float32)
    x = torch.from_numpy(U).cuda().expand(24, 256, 3000)
    o = torch.empty(24, 256, 3000, device="cuda")
    run([x], [o], steps=steps)
    exact = OM.orthogonalize(U, steps)
    t = 2 * rel(OM.rounded(U, steps, pairs=False), exact) + 2.0 ** -18
    got = rel(o[0].cpu().numpy(), exact)
    assert got <= t, (got, t)
    assert torch.equal(o[23], o[0])


def test_stack_of_64_rows():
    """One direction thirty times the others: as exact as one by one, where
    twos are 2.7 times as far off."""
    rng = gen(16)
    u, v = rng.standard_normal((64, 1)), rng.standard_normal((1, 1200))
    U = rng.standard_normal((64, 1200))
    U = (U / np.linalg.norm(U, 2) + 30 * (u / np.linalg.norm(u)) @
         (v / np.linalg.norm(v))).astype(np.float32)
    x = torch.from_numpy(U).cuda().expand(24, 64, 1200)
    o = torch.empty(24, 64, 1200, device="cuda")
    run([x], [o])
    check_singly(U, o[0])
    assert torch.equal(o[23], o[0])


def strong(rng, r, c):
    """One direction six times as strong as the others."""
    u, v = rng.standard_normal((r, 1)), rng.standard_normal((1, c))
    w = rng.standard_normal((r, c)) / max(r, c) ** 0.5
    return (6 * (u / np.linalg.norm(u)) @ (v / np.linalg.norm(v)) + w).astype(
        np.float32)


def check_singly(U, O):
    """As exact as steps one by one: of few rows, twos are ten times less."""
    exact = OM.orthogonalize(U)
    t = 2 * rel(OM.rounded(U, pairs=False), exact) + 2.0 ** -18
    got = rel(O.cpu().numpy(), exact)
    assert got <= t, (got, t)


THIN = [(8, 6000), (6000, 3), (16, 9000), (2, 7001)]


@pytest.mark.parametrize("shape", THIN, ids=lambda s: "%dx%d" % s)
def test_few_rows(shape):
    U = strong(gen(sum(shape)), *shape)
    x = torch.from_numpy(U).cuda()
    check_singly(U, run([x], [torch.empty_like(x)])[0])


def test_few_rows_beside_others():
    rng = gen(12)
    us = [strong(rng, *s) for s in THIN[:2] + [(256, 8000), (1, 9000)]]
    xs = [torch.from_numpy(u).cuda() for u in us]
    a = run(xs, [torch.empty_like(x) for x in xs])
    for u, o in zip(us[:2], a):
        check_singly(u, o)
    for u, o in zip(us, a):
        check(u, o)


@pytest.mark.parametrize("shape", [(48, 80), (140, 150)],
                         ids=lambda s: "%dx%d" % s)
@pytest.mark.parametrize("precision", ["fast", "full"])
def test_zero_nan_and_infinity(precision, shape):
    rng = gen(9)
    U = np.stack([matrix(rng, *shape) for _ in range(5)])
    U[1] = 0
    U[2, 3, 4] = np.nan
    U[3, 0, 0] = np.inf
    x = torch.from_numpy(U).cuda()
    o = run([x], [torch.empty_like(x)], precision)[0]
    assert torch.all(o[1] == 0)
    assert torch.isnan(o[2]).all() and torch.isnan(o[3]).all()
    for k in (0, 4):
        check(U[k], o[k], precision)


@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e15, 1e30])
def test_any_magnitude(size):
    """The norm is taken in 64 bits; eps counts where the norm is small."""
    U = (matrix(gen(10), 70, 90, "strong") * np.float32(1e3)).astype(
        np.float32) * np.float32(size)
    eps = 1e-7 if size > 1 else size * 1e-3
    x = torch.from_numpy(U).cuda()
    o = run([x], [torch.empty_like(x)], eps=eps)[0]
    check(U, o, eps=eps)


def test_same_bits_every_time():
    x = torch.from_numpy(matrix(gen(11), 700, 900, "strong")).cuda()
    a = run([x], [torch.empty_like(x)], poison=False)[0]
    for k in range(3):
        assert torch.equal(run([x], [torch.empty_like(x)])[0], a)


def test_two_calls_at_once():
    """Two streams, a workspace each: the results of one after the other."""
    xs = [torch.from_numpy(matrix(gen(40 + k), 900, 1100)).cuda()
          for k in range(2)]
    want = [run([x], [torch.empty_like(x)])[0] for x in xs]
    ws = [torch.empty(zs.zs_orthogonalize_workspace([x]), dtype=torch.uint8,
                      device="cuda") for x in xs]
    outs = [torch.empty_like(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(4):
        for x, o, w, st in zip(xs, outs, ws, streams):
            zs.zs_orthogonalize([x], [o], workspace=w, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_stack_of_many_small_matrices():
    """More workgroups than the chip holds, of every small kind."""
    for shape in ((700, 40, 60), (400, 64, 256), (300, 300, 64),
                  (300, 128, 120)):
        x = torch.randn(shape, device="cuda",
                        generator=torch.Generator("cuda").manual_seed(1))
        o = run([x], [torch.empty_like(x)])[0]
        for k in (0, 1, shape[0] // 2, shape[0] - 1):
            check(x[k].cpu().numpy(), o[k])
        one = run([x[5]], [torch.empty_like(x[5])])[0]
        assert torch.equal(one, o[5])


def test_another_stream_and_a_captured_graph():
    U = [matrix(gen(20 + k), 150, 200) for k in range(4)]
    x = torch.from_numpy(U[0]).cuda()
    o = torch.empty_like(x)
    ws = torch.empty(zs.zs_orthogonalize_workspace([x]), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    zs.zs_orthogonalize([x], [o], workspace=ws, stream=side)
    side.synchronize()
    check(U[0], o)
    want = o.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        zs.zs_orthogonalize([x], [o], workspace=ws)
    for k in range(4):
        x.copy_(torch.from_numpy(U[k]))
        ws.fill_(255)
        o.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        check(U[k], o)
        if k == 0:
            assert torch.equal(o, want)


# ---- the step ---------------------------------------------------------------

LR, MU, WD = 3e-4, 0.95, 0.1
TILE = zs.ZS_TILE


class Case:
    """Rank 0 of W with matrices and two vectors, every rank owning one copy
    of each tensor."""

    def __init__(self, shapes, W, layout, seed=0, vectors=(300, 77)):
        rng = gen(seed)
        self.shapes, self.W, self.layout = shapes, W, layout
        sizes = [int(np.prod(s)) for s in shapes] + list(vectors)
        numels = [n for n in sizes for _ in range(W)]
        self.lay = zs.zs_layout_build_tensors(numels, W, 0)
        self.lay_o = build_tensor_layout(numels, W, 0)
        self.flat_numel, self.n = self.lay.sizes()[:2]
        self.buckets = self.lay.sizes()[4]
        chunks = zs.zs_layout_chunks(self.lay)
        self.bucket_of = {}
        for i, ch in enumerate(chunks):
            self.bucket_of[sizes.index(ch.numel)] = i
        assert len(set(sizes)) == len(sizes) == len(self.buckets)
        self.sizes = sizes
        n = self.n
        self.G = OS.bf16_round(
            (rng.standard_normal((W, n)) * 1e-3).astype(np.float32).ravel()
        ).reshape(W, n)
        self.master = (rng.standard_normal(n) * 0.02).astype(np.float32)
        self.mom = (rng.standard_normal(n) * 5e-3).astype(np.float32)
        self.v = np.abs(rng.standard_normal(n) * 1e-6).astype(np.float32)
        self.live = np.zeros(n, bool)       # not padding
        for k, b in self.bucket_of.items():
            o = self.buckets[b].shard_off
            self.live[o:o + sizes[k]] = True
        for a in (self.master, self.mom, self.v):
            a[~self.live] = 0
        self.G[:, ~self.live] = 0

    def device(self):
        d = type("D", (), {})()
        f = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        nt = self.lay.sizes()[2]
        d.state = torch.empty(nt, 3, TILE, device="cuda")
        zs.zs_state_pack(self.lay, f(self.master), f(self.mom), f(self.v),
                         d.state)
        g = f(self.G.view(np.int16))
        d.slices = g
        if self.layout == "tiled":
            d.tiled = torch.empty(nt, self.W, TILE, dtype=torch.int16,
                                  device="cuda")
            zs.zs_grads_tile(self.lay, -1, g, self.n, d.tiled)
        d.shard = torch.full((self.n,), 111, dtype=torch.int16,
                             device="cuda")
        d.flat = torch.full((self.flat_numel,), 222, dtype=torch.int16,
                            device="cuda")
        return d

    def grads(self, d, k):
        b = self.buckets[self.bucket_of[k]]
        if self.layout == "tiled":
            return d.tiled[b.tile_off:b.tile_off +
                           -(-b.slice_numel // TILE)]
        return d.slices.view(-1)[b.shard_off:]

    def tensors(self, which=None):
        ks = range(len(self.shapes)) if which is None else which
        return [(self.bucket_of[k],) + tuple(self.shapes[k]) for k in ks]

    def step(self, d, precision="fast", out="both", which=None, ws=None,
             **kw):
        ts = self.tensors(which)
        ks = range(len(self.shapes)) if which is None else which
        if ws is None:
            ws = torch.empty(zs.zs_muon_workspace(self.lay, ts, precision),
                             dtype=torch.uint8, device="cuda")
            ws.fill_(255)
        args = dict(lr=LR, momentum=MU, weight_decay=WD, **kw)
        zs.zs_muon_step(self.lay, ts, [self.grads(d, k) for k in ks],
                        d.state, d.shard if out != "flat" else None,
                        d.flat if out != "shard" else None,
                        grad_layout=self.layout, grad_stride=self.n,
                        precision=precision, workspace=ws, **args)

    def rows(self, d):
        out = [torch.empty(self.n, device="cuda") for _ in range(3)]
        zs.zs_state_unpack(self.lay, d.state, *out)
        return [o.cpu().numpy() for o in out]

    def check(self, d, precision="fast", out="both", nesterov=True,
              scale="rms", steps=5, which=None):
        master, mom, v = self.rows(d)
        assert np.array_equal(v, self.v)    # row 2 is not the step's
        shard = d.shard.cpu().numpy().view(np.uint16)
        flat = d.flat.cpu().numpy().view(np.uint16)
        touched = np.zeros(self.n, bool)
        tflat = np.zeros(self.flat_numel, bool)
        g = OS.reduce_mean(self.G)
        ks = range(len(self.shapes)) if which is None else which
        for k in ks:
            s = self.shapes[k]
            B, R, C = s if len(s) == 3 else (1,) + tuple(s)
            b = self.buckets[self.bucket_of[k]]
            at = slice(b.shard_off, b.shard_off + self.sizes[k])
            touched[at] = True
            M, U = OM.momentum(g[at], self.mom[at], MU, nesterov)
            assert np.array_equal(mom[at].view(np.int32), M.view(np.int32))
            U = U.reshape(B, R, C)
            O = np.stack([OM.orthogonalize(u, steps) for u in U])
            want = OM.apply(self.master[at], O.ravel(), LR, WD,
                            OM.scale(scale, R, C))
            upd = LR * OM.scale(scale, R, C) * np.linalg.norm(O)
            t = max(bound(u, o, precision, torch.float32, steps)
                    for u, o in zip(U, O)) if precision == "fast" \
                else 2.0 ** -13
            # three fp32 roundings of the result beside the error of O
            tol = t * upd + 3 * 2.0 ** -24 * np.linalg.norm(want)
            assert np.linalg.norm(master[at] - want) <= tol
            bits = OS.bf16_round(master[at])
            if out != "flat":
                assert np.array_equal(shard[at], bits)
            if out != "shard":
                f = slice(b.flat_off, b.flat_off + self.sizes[k])
                tflat[f] = True
                assert np.array_equal(flat[f], bits)
        if out == "flat":
            assert np.all(shard == 111)
        else:
            assert np.all(shard[~touched] == 111)
        if out == "shard":
            assert np.all(flat == 222)
        else:
            assert np.all(flat[~tflat] == 222)
        assert np.array_equal(master[~touched], self.master[~touched])
        assert np.array_equal(mom[~touched], self.mom[~touched])


SETS = [[(64, 64)], [(130, 70), (70, 140), (3, 40, 36), (1, 515), (513, 1)],
        [(5, 31, 63), (257, 100)], [(2, 90, 91), (120, 333)]]


@pytest.mark.parametrize("layout", ["slices", "tiled"])
@pytest.mark.parametrize("W", [1, 2, 3, 8, 17])
@pytest.mark.parametrize("shapes", SETS, ids=str)
def test_step(shapes, W, layout):
    c = Case(shapes, W, layout, seed=W)
    d = c.device()
    nesterov = W != 2
    scale = {1: "none", 2: "shape"}.get(W, "rms")
    c.step(d, nesterov=nesterov, scale=scale)
    c.check(d, nesterov=nesterov, scale=scale)


@pytest.mark.parametrize("shapes", [[(2111, 2052)], [(1501, 1503)],
                                    [(9, 640, 700), (64, 64)]], ids=str)
def test_step_of_large_matrices(shapes):
    """Large tiles, and more partial sums of squares than a workgroup adds on
    its way."""
    c = Case(shapes, 2, "tiled", seed=35)
    d = c.device()
    c.step(d, steps=2)
    c.check(d, steps=2)


def test_step_of_few_rows_beside_others():
    c = Case([(5, 6000), (256, 8000), (9001, 2)], 2, "tiled", seed=36)
    d = c.device()
    c.step(d)
    c.check(d)


@pytest.mark.parametrize("precision", ["fast", "full"])
@pytest.mark.parametrize("out", ["shard", "flat"])
def test_step_outputs_and_precision(precision, out):
    c = Case(SETS[1], 4, "tiled", seed=31)
    d = c.device()
    c.step(d, precision, out, steps=3)
    c.check(d, precision, out, steps=3)


def test_step_of_some_tensors_leaves_the_others():
    c = Case(SETS[1], 2, "slices", seed=32)
    d = c.device()
    c.step(d, which=[3, 1])
    c.check(d, which=[3, 1])


def test_step_captured_in_a_graph():
    c = Case(SETS[2], 2, "tiled", seed=33)
    d, e = c.device(), c.device()
    ws = torch.empty(zs.zs_muon_workspace(c.lay, c.tensors()),
                     dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.step(d, ws=ws)
    for k in range(3):
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        c.step(e)
        torch.cuda.synchronize()
        assert torch.equal(d.state, e.state)
        assert torch.equal(d.shard, e.shard) and torch.equal(d.flat, e.flat)
        if k == 0:
            c.check(d)


def test_muon_and_adamw_on_one_state(tmp_path):
    """The set as it is used: matrices by Muon, the rest by AdamW, on one
    tiled state, over three steps with a checkpoint between."""
    c = Case(SETS[1], 2, "tiled", seed=34)
    d = c.device()
    hp = dict(lr=LR, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=WD)
    nm = len(c.shapes)
    vec = [c.bucket_of[nm], c.bucket_of[nm + 1]]
    mw, mm, mv = c.master.copy(), c.mom.copy(), c.v.copy()
    bits = np.zeros(c.n, np.uint16)
    for t in (1, 2, 3):
        c.master, c.mom, c.v = (a.copy() for a in (mw, mm, mv))
        d.shard.fill_(111)
        d.flat.fill_(222)
        c.step(d)
        c.check(d)
        zs.zs_buckets_step(c.lay, vec, [c.grads(d, nm), c.grads(d, nm + 1)],
                           d.state, d.shard, d.flat, grad_layout="tiled",
                           step=t, **hp)
        for k, b in ((nm, vec[0]), (nm + 1, vec[1])):
            o = c.buckets[b].shard_off
            at = slice(o, o + c.sizes[k])
            OS.step(np.ascontiguousarray(c.G[:, at]), mw[at], mm[at], mv[at],
                    OS.AdamW(**hp), t)
            bits[at] = OS.bf16_round(mw[at])
        got = c.rows(d)
        for k, b in ((nm, vec[0]), (nm + 1, vec[1])):
            o = c.buckets[b].shard_off
            at = slice(o, o + c.sizes[k])
            for x, y in zip(got, (mw, mm, mv)):
                assert np.array_equal(x[at], y[at])
        # the matrices' rows, as the kernels left them, for the next step
        for a, x in ((mw, got[0]), (mm, got[1]), (mv, got[2])):
            a[:] = x
        if t == 2:
            path = str(tmp_path / "ck")
            zs.zs_checkpoint_save(c.lay, path, d.state, t)
            d.state.fill_(float("nan"))
            assert zs.zs_checkpoint_load(c.lay, path, d.state) == t
