"""The list operators on the GPU against oracle/tensors.py: the AdamW step
with states in 32 bits (bit for bit) and in 8 (codes and scales bit for bit,
weights to a bound by arithmetic), the sum of squares, the conversions; every
kind of weights and gradients, sizes and addresses where a piece, a block or
four elements end, and what lies between the arrays left as it was."""

import math

import numpy as np
import pytest
import torch

import zero_sharded_optimizer_shard_amd as zs
from oracle import tensors as OT

pytestmark = pytest.mark.gpu

HP = (3e-4, 0.9, 0.95, 1e-8, 0.1)
HP2 = (1e-3, 0.8, 0.999, 1e-6, 0.0)
SIZES = [1, 2, 3, 4, 5, 63, 64, 65, 255, 256, 257, 511, 513, 1023, 1024,
         1025, 1279, 2047, 2048, 2050, 0, 4099, 10007]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def bits(x):
    """A numpy array's or a tensor's bytes."""
    if isinstance(x, torch.Tensor):
        return x.contiguous().view(torch.uint8).cpu().numpy()
    return np.ascontiguousarray(x).view(np.uint8)


def same(got, want, where=""):
    g, w = bits(got), bits(want)
    assert g.shape == w.shape, where
    if not np.array_equal(g, w):
        bad = np.flatnonzero(g != w)
        raise AssertionError(f"{where}: {len(bad)} bytes differ, first at "
                             f"{bad[0]} of {len(g)}")


class Arena:
    """Arrays with guards around them; `check` compares every guard."""

    def __init__(self):
        self.all = []

    def put(self, x, shift=0):
        """A device tensor of numpy array x (uint16: bf16), `shift` elements
        past a 256-byte boundary."""
        whole = torch.full((x.nbytes + 1024 + shift * x.itemsize,), 0x5a,
                           dtype=torch.uint8, device="cuda")
        at = -whole.data_ptr() % 256 + 256 + shift * x.itemsize
        view = whole[at:at + x.nbytes]
        view.copy_(torch.from_numpy(bits(x).reshape(-1)))
        self.all.append((whole, at, x.nbytes, whole.clone()))
        return view.view({np.dtype(np.uint16): torch.bfloat16,
                          np.dtype(np.float32): torch.float32,
                          np.dtype(np.int8): torch.int8,
                          np.dtype(np.uint8): torch.uint8}[x.dtype])

    def check(self):
        for whole, at, n, was in self.all:
            assert torch.equal(whole[:at], was[:at])
            assert torch.equal(whole[at + n:], was[at + n:])


def normal(rng, n, sigma):
    return (rng.standard_normal(n) * sigma).astype(np.float32)


class Case:
    """A list with its host copy."""

    def __init__(self, sizes, bits=32, weights="master", grad="bf16",
                 world=1, shift=0, seed=0, groups=None, edit=None,
                 apart=0):
        """shift: elements past an aligned address; apart: as many more with
        every array."""
        rng = np.random.default_rng(seed)
        self.arena, self.sizes, self.world = Arena(), sizes, world
        self.bits, self.weights, self.grad = bits, weights, grad
        self.groups = groups or [0] * len(sizes)
        self.host, self.dev = [], []
        for n in sizes:
            h = {}
            spread = np.exp(rng.standard_normal(n)).astype(np.float32)
            G = normal(rng, (world, n), 1e-3) * spread
            h["grad"] = OT.to_bf16(G).reshape(world, n) if grad == "bf16" \
                else G
            w = normal(rng, n, 0.02)
            if weights == "master":
                h["master"], h["param"] = w, OT.to_bf16(w + 1)
            else:
                h["param"] = OT.to_bf16(w) if weights == "bf16" else w
            m = normal(rng, n, 3e-4) * spread
            v = np.square(normal(rng, n, 1e-3) * spread)
            if bits == 32:
                h["m"], h["v"] = m, v
            else:
                q = OT.hold(m, v)
                h["m"], h["m_scale"] = q[0].astype(np.int8), q[1]
                h["v"], h["v_scale"] = q[2].astype(np.uint8), q[3]
            if edit:
                edit(h)
            self.host.append(h)
            d = {k: self.arena.put(
                x, 0 if bits == 8 and k in ("m", "v") else shift + apart * i)
                for i, (k, x) in enumerate(h.items()) if k != "grad"}
            stride = n + 5 + shift if world > 1 else n
            rows = np.zeros((world, stride), h["grad"].dtype)
            rows[:, :n] = h["grad"]
            g = self.arena.put(rows.reshape(-1), shift)
            d["grad"] = g.view(world, stride)[:, :n] if world > 1 else g
            self.dev.append(d)
        self.list = self.make()

    def column(self, name):
        return [d[name] for d in self.dev] if all(name in d for d in
                                                  self.dev) else None

    def make(self, **kw):
        lst = zs.zs_tensors_create(
            params=self.column("param"), grads=self.column("grad"),
            master=self.column("master"), m=self.column("m"),
            v=self.column("v"), m_scale=self.column("m_scale"),
            v_scale=self.column("v_scale"), world=self.world,
            groups=self.groups, **kw)
        upload(lst)
        return lst

    def step(self, hps=(HP,), t=3, **kw):
        zs.zs_tensors_step(self.list, [zs.zs_adamw(*h) for h in hps], step=t,
                           **kw)

    def means(self):
        return [OT.mean(OT.bf16(h["grad"]) if self.grad == "bf16"
                        else h["grad"]) for h in self.host]

    def expect(self, hps=(HP,), t=3, c=None):
        """The oracle's step on the host copies, and what the weights may be
        off by."""
        for h, g, k in zip(self.host, self.means(), self.groups):
            hp = hps[k]
            if c is not None:
                with np.errstate(all="ignore"):
                    g = g * c
            if self.bits == 8:
                m, v = OT.stands_for(h["m"], h["m_scale"], h["v"],
                                     h["v_scale"])
            else:
                m, v = h["m"], h["v"]
            m, v, root = OT.moments(g, m, v, hp, t)
            w = h["master"] if "master" in h else h["param"]
            if w.dtype == np.uint16:
                w = OT.bf16(w)
            if self.bits == 32:
                w1 = OT.weights(w, m, root, hp, t)
                h["m"], h["v"] = m, v
                h["off"] = 0.0
            else:
                q = OT.encode(m, 127) + OT.encode(root, 255)
                h["m"], h["m_scale"] = q[0].astype(np.int8), q[1]
                h["v"], h["v_scale"] = q[2].astype(np.uint8), q[3]
                kept, update = OT.weights64(w, m, root, hp, t)
                w1 = kept - update
                # in the update: the constant of sqrt(1-b2^t) rounded on
                # either side and the sum with eps (3 half steps of 2^-24),
                # a reciprocal to one step (2) and its product (1), 6 in
                # all; w*dec and the difference rounded once each
                with np.errstate(all="ignore"):
                    h["off"] = 2.0 ** -24 * (8 * np.abs(update) +
                                             np.abs(kept) + np.abs(w1)) \
                        + 1e-44
            h["w"] = w1

    def check(self, where=""):
        for i, (h, d) in enumerate(zip(self.host, self.dev)):
            at = f"{where} tensor {i} of {self.sizes[i]}"
            for k in ("m", "v"):
                same(d[k], h[k], f"{at}: {k}")
            for k in ("m_scale", "v_scale"):
                if k in h:
                    a, b = d[k].cpu().numpy(), h[k]
                    assert np.array_equal(np.isnan(a), np.isnan(b)), at
                    same(np.nan_to_num(a), np.nan_to_num(b), f"{at}: {k}")
            got = d["master" if "master" in h else "param"]
            got32 = got.float().cpu().numpy()
            if self.bits == 32:
                want = OT.to_bf16(h["w"]) if got.dtype == torch.bfloat16 \
                    else h["w"]
                same(got, want, f"{at}: weights")
            else:
                off = h["off"] + (2.0 ** -8 * np.abs(h["w"])
                                  if got.dtype == torch.bfloat16 else 0)
                far = np.abs(got32.astype(np.float64) - h["w"])
                nan = np.isnan(h["w"])
                assert np.array_equal(nan, np.isnan(got32)), at
                assert np.all(far[~nan] <= off[~nan]), \
                    f"{at}: weights {np.max(far[~nan] / off[~nan])} bounds"
            if "master" in h:
                # the parameter is the rounded master
                same(d["param"], OT.to_bf16(got32), f"{at}: param")
                h["master"] = got32
                h["param"] = OT.to_bf16(got32)
            else:
                h["param"] = got.view(torch.int16).cpu().numpy().view(
                    np.uint16) if got.dtype == torch.bfloat16 else got32
        self.arena.check()


def upload(lst):
    zs.zs_tensors_upload(lst, torch.empty(zs.zs_tensors_table_bytes(lst),
                                          dtype=torch.uint8, device="cuda"))


def sumsq_of(lst):
    out = torch.full((1,), -1.0, dtype=torch.float64, device="cuda")
    ws = torch.empty(zs.zs_tensors_sumsq_workspace(lst), dtype=torch.uint8,
                     device="cuda")
    zs.zs_tensors_sumsq(lst, out, workspace=ws)
    return out


# ---- the step --------------------------------------------------------------------

@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("weights", ["master", "bf16", "f32"])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("world", [1, 2, 3, 6])
@pytest.mark.parametrize("shift", [0, 1])
def test_step_kinds(bits, weights, grad, world, shift):
    c = Case(SIZES, bits, weights, grad, world, shift, seed=world)
    for t in (1, 2):
        c.step(t=t)
        c.expect(t=t)
        c.check(f"step {t}")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("world", [4, 5, 8, 9, 16, 33])
def test_step_many_ranks(bits, world):
    c = Case([1, 700, 1024, 3001], bits, world=world, seed=world)
    c.step()
    c.expect()
    c.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("weights", ["master", "f32"])
@pytest.mark.parametrize("shift,apart", [
    (2, 0), (3, 0), (4, 0), (8, 0), (31, 0), (33, 0), (37, 0), (60, 0),
    (63, 0), (0, 1), (0, 4), (0, 32), (3, 16), (1, 64)])
def test_step_other_addresses(bits, weights, shift, apart):
    """Arrays that share their distance from a line, or four elements, or
    nothing; tensors that end before the first line."""
    c = Case([1, 3, 5, 40, 64, 255, 256, 300, 1024, 2051], bits, weights,
             "bf16", 2, shift, apart=apart)
    c.step()
    c.expect()
    c.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_step_tiny_gradients_and_eps(bits):
    """Moments near fp32's least normal number over an eps of their size: the
    update is of the usual size, and as exact."""
    def edit(h):
        h["grad"] *= np.float32(1e-33)
        if bits == 32:
            h["m"] *= np.float32(1e-33)
            h["v"][:] = 0
        else:
            h["m_scale"] *= np.float32(1e-33)
            h["v"][:], h["v_scale"][:] = 0, 0
    c = Case([1500], bits, "f32", "f32", edit=edit)
    hp = (1e-3, 0.9, 0.95, 1e-36, 0.1)
    c.step([hp])
    c.expect([hp])
    c.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_step_groups(bits):
    c = Case([3000, 5, 1024, 300], bits, groups=[0, 1, 15, 1])
    hps = [HP, HP2] + [HP] * 13 + [(1e-2, 0.0, 0.0, 1e-3, 0.5)]
    c.step(hps, t=1000)
    c.expect(hps, t=1000)
    c.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("max_norm", [1e-3, 0.05, 1e3, math.inf])
def test_step_clipped(bits, max_norm):
    c = Case(SIZES, bits, world=3, seed=4)
    s = sumsq_of(c.list)
    c.step(sumsq=s, max_norm=max_norm)
    coef = OT.coefficient(s.item(), max_norm)
    assert (coef < 1) == (max_norm < 0.1)
    c.expect(c=coef)
    c.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sum_", [math.inf, math.nan, -math.inf, -1.0])
def test_step_writes_nothing_on_a_sum_that_is_none(bits, sum_):
    c = Case(SIZES, bits, world=2)
    was = [{k: x.clone() for k, x in d.items()} for d in c.dev]
    s = torch.full((1,), sum_, dtype=torch.float64, device="cuda")
    c.step(sumsq=s, max_norm=1.0)
    for a, b in zip(was, c.dev):
        for k in a:
            same(a[k].contiguous(), b[k].contiguous(), k)
    c.arena.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_step_zero_sum(bits):
    def edit(h):
        h["grad"][:] = 0
    c = Case([700, 1500], bits, edit=edit)
    s = sumsq_of(c.list)
    assert s.item() == 0.0
    c.step(sumsq=s, max_norm=1.0)
    c.expect(c=np.float32(1))
    c.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_step_without_sumsq_passes_inf_and_nan_on(bits, bad):
    """In 32 bits element by element, in 8 by the block."""
    def edit(h):
        n = h["grad"].shape[1]
        if n > 300:
            h["grad"][0, 299] = bad
    c = Case([300, 1024, 1500, 200], bits, "f32", "f32", edit=edit)
    c.step()
    c.expect()
    for h, d in zip(c.host, c.dev):
        got = d["param"].cpu().numpy()
        assert np.isnan(got).sum() == np.isnan(h["w"]).sum() <= 1
        if bits == 8:
            same(d["m"], h["m"])
            same(d["v"], h["v"])
            for k in ("m_scale", "v_scale"):
                assert np.array_equal(np.isnan(d[k].cpu().numpy()),
                                      np.isnan(h[k]))
                assert np.isnan(h[k]).sum() == (h["m"].size > 300)
    c.arena.check()


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-20, 1e-12, 1e10, 1e18])
@pytest.mark.parametrize("bits", [32, 8])
def test_step_magnitudes(bits, scale):
    """Gradients and moments of any size, subnormal ones among them."""
    def edit(h):
        f = np.float32(scale * 1e3)
        h["grad"] *= f
        with np.errstate(all="ignore"):
            if bits == 32:
                h["m"] *= f
                h["v"] *= f
                h["v"] *= f
            else:
                h["m_scale"] *= f
                h["v_scale"] *= f
    c = Case([257, 1500], bits, "f32", "f32", edit=edit)
    c.step()
    c.expect()
    c.check()


def test_step8_fresh_states():
    """Codes and scales of zeros, as a new optimizer has them."""
    def edit(h):
        for k in ("m", "m_scale", "v", "v_scale"):
            h[k][:] = 0
    c = Case([1, 300, 4099], 8, edit=edit)
    for t in (1, 2, 3):
        c.step(t=t)
        c.expect(t=t)
        c.check(f"step {t}")


def test_step8_blocks_of_zeros_and_far_apart_values():
    def edit(h):
        n = h["grad"].shape[1]
        for k in ("m", "m_scale", "v", "v_scale"):
            h[k][:] = 0
        h["grad"][:] = 0                                # first block: zeros
        h["grad"][:, 256:512] = np.exp2(
            -np.arange(256) / 2).astype(np.float32)     # second: 128 octaves
        h["grad"][:, n - 1] = 2.0 ** -120               # last: below 2^-100
    c = Case([1025], 8, "f32", "f32", edit=edit)
    c.step(t=1)
    c.expect(t=1)
    h = c.host[0]
    assert h["m_scale"][0] == 0 and h["m_scale"][4] == 0
    # no root that is not 0 has a code of 0 (2^-145 times 1-b2 is in fp32)
    assert np.all(h["v"][256:256 + 145] >= 1)
    c.check()


def test_step_equals_zs_step():
    """The tensors of a whole-tensor layout, stepped by zs_step on its tiled
    state and by a list on plain arrays: the same bits."""
    numels, W = [4096, 1000, 128 * 77, 3], 2
    lay = zs.zs_layout_build_tensors(numels, W, 0)
    _, n, tiles, _, buckets = lay.sizes()
    rng = np.random.default_rng(1)
    G = torch.from_numpy(normal(rng, (W, n), 1e-3)).bfloat16().cuda()
    w, m = (torch.from_numpy(normal(rng, n, s)).cuda()
            for s in (0.02, 1e-3))
    v = m.square()
    state = torch.zeros(tiles * 3 * zs.ZS_TILE, device="cuda")
    zs.zs_state_pack(lay, w, m, v, state)
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros_like(p)
    zs.zs_step(lay, G, state, p, grad_stride=n, step=5,
               **dict(zip(("lr", "beta1", "beta2", "eps", "weight_decay"),
                          HP)))

    def cut(x):
        return [x[..., b.shard_off:b.shard_off + b.slice_numel]
                for b in buckets]
    lst = zs.zs_tensors_create(params=cut(q), grads=cut(G), master=cut(w),
                               m=cut(m), v=cut(v), world=W)
    upload(lst)
    zs.zs_tensors_step(lst, zs.zs_adamw(*HP), step=5)
    a, b, c = (torch.zeros(n, device="cuda") for _ in range(3))
    zs.zs_state_unpack(lay, state, a, b, c)
    for x, y in ((p, q), (a, w), (b, m), (c, v)):
        same(x, y)


def test_step_flat_buckets_in_eight_bits():
    """A rank's slices of a flat layout as a list: gradients from its [W][n]
    slices, parameters straight into the all-gather buffer; the norm over all
    ranks clips every rank's step; other ranks' positions stay."""
    numels, W, clip = [5000, 300, 12345], 4, 0.02
    rng = np.random.default_rng(2)
    full, total = None, 0.0
    ranks = []
    for r in range(W):
        lay = zs.zs_layout_build(numels, W, r, 1 << 14)
        F, n, _, _, buckets = lay.sizes()
        if full is None:
            full = torch.full((F,), 7.0, dtype=torch.bfloat16,
                              device="cuda")
        st = {k: torch.zeros(n, dtype=d, device="cuda") for k, d in (
            ("m", torch.int8), ("v", torch.uint8))}
        # a block never spans two tensors of the list
        nb = [-(-b.slice_numel // 256) for b in buckets]
        sc = torch.zeros(2, sum(nb), device="cuda")
        G = torch.from_numpy(normal(rng, (W, n), 1e-3)).bfloat16().cuda()
        w = torch.from_numpy(normal(rng, n, 0.02)).cuda()
        w0 = w.clone()

        def cut(x):
            return [x[..., b.shard_off:b.shard_off + b.slice_numel]
                    for b in buckets]
        offs = np.cumsum([0] + nb)
        lst = zs.zs_tensors_create(
            params=[full[b.flat_off + r * b.slice_numel:][:b.slice_numel]
                    for b in buckets],
            grads=cut(G), master=cut(w), m=cut(st["m"]), v=cut(st["v"]),
            m_scale=[sc[0, a:b] for a, b in zip(offs, offs[1:])],
            v_scale=[sc[1, a:b] for a, b in zip(offs, offs[1:])], world=W)
        upload(lst)
        s = sumsq_of(lst)
        total = total + s
        ranks.append((lst, G, w, w0, st, sc, buckets))
    coef = OT.coefficient(total.item(), clip)
    assert coef < 1
    for lst, *_ in ranks:
        zs.zs_tensors_step(lst, zs.zs_adamw(*HP), step=1, sumsq=total,
                           max_norm=clip)
    for r, (lst, G, w, w0, st, sc, buckets) in enumerate(ranks):
        g = OT.mean(G.float().cpu().numpy()) * coef
        zero = np.zeros_like(g)
        m, v, root = OT.moments(g, zero, zero, HP, 1)
        kept, update = OT.weights64(w0.cpu().numpy(), m, root, HP, 1)
        got = w.cpu().numpy()
        assert np.all(np.abs(got - (kept - update)) <= 2.0 ** -24 * (
            8 * np.abs(update) + 2 * np.abs(kept) + np.abs(update)) + 1e-44)
        for b in buckets:
            sl = slice(b.shard_off, b.shard_off + b.slice_numel)
            at = b.flat_off + r * b.slice_numel
            same(full[at:at + b.slice_numel], OT.to_bf16(got[sl]))
            same(st["m"][sl], OT.encode(m[sl], 127)[0].astype(np.int8))
            same(st["v"][sl], OT.encode(root[sl], 255)[0].astype(np.uint8))


def test_many_tensors():
    sizes = [1 + (7 * k) % 300 for k in range(1500)] + [1024 * 3]
    for bits in (32, 8):
        c = Case(sizes, bits, groups=[k % 2 for k in range(len(sizes))])
        s = sumsq_of(c.list)
        c.step([HP, HP2], sumsq=s, max_norm=0.05)
        c.expect([HP, HP2], c=OT.coefficient(s.item(), 0.05))
        c.check()


def test_empty_list():
    lst = zs.zs_tensors_create(params=[], grads=[], m=[], v=[])
    upload(lst)
    zs.zs_tensors_step(lst, zs.zs_adamw(*HP), step=1)
    assert sumsq_of(lst).item() == 0.0
    z = torch.zeros(0, device="cuda")
    lst = zs.zs_tensors_create(params=[z], grads=[z], m=[z], v=[z])
    upload(lst)
    zs.zs_tensors_step(lst, zs.zs_adamw(*HP), step=1)
    assert sumsq_of(lst).item() == 0.0


# ---- the sum of squares ------------------------------------------------------------

@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("world", [1, 2, 3, 8])
@pytest.mark.parametrize("shift", [0, 1, 37])
@pytest.mark.parametrize("sizes", [[1], [768], SIZES, [33000, 5, 70001]])
def test_sumsq(grad, world, shift, sizes):
    c = Case(sizes, 32, "f32", grad, world, shift, seed=9)
    got = sumsq_of(c.list).item()
    want = OT.sumsq(c.means())
    # squares are exact to 2^-53 and n sums of positive numbers add at most
    # n * 2^-53 on either side
    assert abs(got - want) <= 2 * (sum(sizes) + 1) * 2.0 ** -53 * want
    assert sumsq_of(c.list).item() == got
    c.arena.check()


def test_sumsq_of_values_whose_squares_fp32_has_not():
    for x in (1e-30, 1e30, 3e38):
        g = torch.full((5000,), x, device="cuda")
        lst = zs.zs_tensors_create(grads=[g])
        upload(lst)
        want = 5000 * float(np.float32(x)) ** 2
        assert abs(sumsq_of(lst).item() / want - 1) < 1e-12


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("n", [10, 100000])
def test_sumsq_passes_inf_and_nan_on(bad, n):
    g = torch.zeros(n, device="cuda")
    g[n // 3] = bad
    lst = zs.zs_tensors_create(grads=[g])
    upload(lst)
    got = sumsq_of(lst).item()
    assert math.isnan(got) if math.isnan(bad) else got == math.inf


def test_sumsq_large():
    """Every workgroup with many pieces, and the last not full."""
    n = (1 << 26) + 12345
    g = torch.randn(n, device="cuda").bfloat16()
    lst = zs.zs_tensors_create(grads=[g[:100], g[100:5000], g[5000:]])
    upload(lst)
    want = g.double().square().sum().item()
    assert abs(sumsq_of(lst).item() - want) <= 2 * n * 2.0 ** -53 * want


# ---- conversions --------------------------------------------------------------------

class States:
    def __init__(self, sizes, shift=0, m=None, v=None):
        self.arena, self.sizes = Arena(), sizes
        put = self.arena.put
        rng = np.random.default_rng(11)
        self.m = m or [normal(rng, n, 1e-3) for n in sizes]
        self.v = v or [np.square(normal(rng, n, 1e-3)) for n in sizes]
        self.d = {"m": [put(x, shift) for x in self.m],
                  "v": [put(x, shift) for x in self.v]}
        blocks = [-(-n // 256) for n in sizes]
        self.q = {"m": [put(np.full(n, 99, np.int8)) for n in sizes],
                  "v": [put(np.full(n, 99, np.uint8)) for n in sizes],
                  "m_scale": [put(np.full(n, 9, np.float32), shift)
                              for n in blocks],
                  "v_scale": [put(np.full(n, 9, np.float32), shift)
                              for n in blocks]}
        self.o = {k: [put(np.full(n, 9, np.float32), shift) for n in sizes]
                  for k in ("m", "v")}
        self.lists = [zs.zs_tensors_create(**d)
                      for d in (self.d, self.q, self.o)]
        for lst in self.lists:
            upload(lst)

    def check(self):
        a, b, c = self.lists
        zs.zs_tensors_convert(a, b)
        zs.zs_tensors_convert(b, c)
        for i, (m, v) in enumerate(zip(self.m, self.v)):
            mq, ms, vq, vs = OT.hold(m, v)
            at = f"tensor {i} of {self.sizes[i]}"
            same(self.q["m"][i], mq.astype(np.int8), at)
            same(self.q["v"][i], vq.astype(np.uint8), at)
            for k, S in (("m_scale", ms), ("v_scale", vs)):
                got = self.q[k][i].cpu().numpy()
                assert np.array_equal(np.isnan(got), np.isnan(S)), at
                same(np.nan_to_num(got), np.nan_to_num(S), at)
            for k, want in zip(("m", "v"), OT.stands_for(mq, ms, vq, vs)):
                got = self.o[k][i].cpu().numpy()
                assert np.array_equal(np.isnan(got), np.isnan(want)), at
                same(np.nan_to_num(got), np.nan_to_num(want), at)
            same(self.d["m"][i], m)
            same(self.d["v"][i], v)
        self.arena.check()


@pytest.mark.parametrize("shift", [0, 1, 2])
def test_convert(shift):
    s = States(SIZES, shift)
    s.check()
    # codes come back the same from the values that they stand for
    was = [x.clone() for x in s.q["m"] + s.q["v"]]
    zs.zs_tensors_convert(s.lists[2], s.lists[1])
    for a, b in zip(was, s.q["m"] + s.q["v"]):
        same(a, b)


@pytest.mark.parametrize("shift", [0, 1, 37])
def test_convert_of_step_lists(shift):
    """A step's fp32 list, whose units start at a line, to 8 bits and back
    while both step on."""
    sizes = [1, 300, 1024, 5003]
    a = Case(sizes, 32, "bf16", shift=shift, seed=3)
    b = Case(sizes, 8, "bf16", shift=shift, seed=4)
    a.step()
    a.expect()
    a.check()
    zs.zs_tensors_convert(a.list, b.list)
    for x, y, d in zip(a.host, b.host, b.dev):
        q = OT.hold(x["m"], x["v"])
        y.update(m=q[0].astype(np.int8), m_scale=q[1],
                 v=q[2].astype(np.uint8), v_scale=q[3])
        for k in ("m", "m_scale", "v", "v_scale"):
            same(d[k], y[k])
    b.step()
    b.expect()
    b.check()
    zs.zs_tensors_convert(b.list, a.list)
    for x, y in zip(a.host, b.host):
        x["m"], x["v"] = OT.stands_for(y["m"], y["m_scale"], y["v"],
                                       y["v_scale"])
    a.step(t=9)
    a.expect(t=9)
    a.check()


def test_convert_at_every_border():
    """Values next to the borders between codes, in blocks whose A is
    top^2."""
    for top in (127, 255):
        k = np.arange(top)
        b = ((k + 0.5) ** 2).astype(np.float32)
        x = np.concatenate([np.nextafter(b, np.float32(0)), b,
                            np.nextafter(b, np.float32(1e9))])
        pad = -len(x) % 255
        x = np.append(x, np.zeros(pad, np.float32)).reshape(-1, 255)
        x = np.concatenate([x, np.full((len(x), 1), top ** 2, np.float32)],
                           1).reshape(-1)
        if top == 127:
            States([x.size], m=[x * np.where(np.arange(x.size) % 2, -1, 1)
                                .astype(np.float32)], v=[x]).check()
        else:
            # squares whose roots are next to the borders
            v = np.square(x.astype(np.float64)).astype(np.float32)
            States([x.size], m=[x], v=[v]).check()


def test_convert_all_sizes_of_values():
    rng = np.random.default_rng(8)
    n = 256 * 300
    u = rng.integers(0, 1 << 32, n, dtype=np.uint64).astype(np.uint32)
    m = u.view(np.float32).copy()
    m[~np.isfinite(m)] = 1.0
    # one block of an exponent each, and all of them mixed
    e = np.repeat(np.arange(256) % 255, 256).astype(np.uint32)
    m2 = ((rng.integers(0, 1 << 23, e.size).astype(np.uint32)) |
          (e << 23)).view(np.float32)
    States([n, m2.size], m=[m, m2], v=[np.abs(m), m2]).check()


def test_convert_special_blocks():
    m = np.ones(2048, np.float32)
    v = np.ones(2048, np.float32)
    m[10], m[300], m[600] = np.nan, np.inf, -np.inf
    m[768:1024] = 0
    m[1024:1280] = 2.0 ** -101
    v[1300], v[1600], v[1900] = np.nan, np.inf, -1.0
    v[512:768] = 0
    v[768:1024] = 2.0 ** -149
    v[0] = -0.0
    m[1] = -0.0
    States([2048], m=[m], v=[v]).check()


# ---- calls ------------------------------------------------------------------------

def test_captured_and_replayed():
    """Norm, clipped step and conversion in one graph, replayed with eager
    work between."""
    g = Case([5000, 33, 70000], 8, world=2, seed=6)
    e = Case([5000, 33, 70000], 8, world=2, seed=6)
    graph = torch.cuda.CUDAGraph()
    s = torch.zeros(1, dtype=torch.float64, device="cuda")
    ws = torch.empty(zs.zs_tensors_sumsq_workspace(g.list),
                     dtype=torch.uint8, device="cuda")
    vals = [[torch.zeros(n, device="cuda") for n in g.sizes]
            for _ in range(2)]
    to = zs.zs_tensors_create(m=vals[0], v=vals[1])
    upload(to)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        zs.zs_tensors_sumsq(g.list, s, workspace=ws)
        g.step(sumsq=s, max_norm=0.05, t=4)
        zs.zs_tensors_convert(g.list, to)
    for r in range(4):
        for c in (g, e):
            for d in c.dev:
                d["grad"].mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        e.step(sumsq=sumsq_of(e.list), max_norm=0.05, t=4)
        want = sumsq_of(e.list)
        assert s.item() == want.item()
        for i, (a, b) in enumerate(zip(g.dev, e.dev)):
            for k in a:
                same(a[k].contiguous(), b[k].contiguous(),
                     f"replay {r} tensor {i} {k}")
            m, v = OT.stands_for(*(b[k].cpu().numpy() for k in (
                "m", "m_scale", "v", "v_scale")))
            same(vals[0][i], m)
            same(vals[1][i], v)
    g.arena.check()


def test_upload_under_capture_is_refused():
    c = Case([100])
    lst = zs.zs_tensors_create(grads=c.column("grad"))
    table = torch.empty(zs.zs_tensors_table_bytes(lst), dtype=torch.uint8,
                        device="cuda")
    keep = torch.zeros(8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        keep.add_(1)
        with pytest.raises(zs.ZsError) as ei:
            zs.zs_tensors_upload(lst, table)
    assert ei.value.code == -1
    graph.replay()
    with pytest.raises(zs.ZsError) as ei:
        sumsq_of(lst)                           # still without a table
    assert ei.value.code == -1
    assert keep[0].item() == 1


def test_two_streams():
    """Two lists at once, each on its own stream with its own workspace."""
    cases = [Case([20000, 77, 300000], 8, seed=k) for k in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    sums = []
    for c, st in zip(cases, streams):
        with torch.cuda.stream(st):
            s = sumsq_of(c.list)
            zs.zs_tensors_step(c.list, zs.zs_adamw(*HP), step=3, sumsq=s,
                               max_norm=0.1)
            sums.append(s)
    torch.cuda.synchronize()
    for c, s in zip(cases, sums):
        want = OT.sumsq(c.means())
        assert abs(s.item() / want - 1) < 1e-9
        c.expect(c=OT.coefficient(s.item(), 0.1))
        c.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_without_residency_cap(bits):
    was = zs.zs_set_residency_cap(False)
    try:
        c = Case([70000, 5], bits, world=8)
        c.step()
        c.expect()
        c.check()
        s = States([70000])
        s.check()
    finally:
        zs.zs_set_residency_cap(bool(was))


def test_explicit_stream():
    c = Case([3000], 32)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    zs.zs_tensors_step(c.list, zs.zs_adamw(*HP), step=3, stream=st)
    st.synchronize()
    c.expect()
    c.check()


def test_second_table_is_refused():
    """Captured calls and calls on their way may read the first."""
    c = Case([3000, 5], 32)
    with pytest.raises(zs.ZsError) as ei:
        upload(c.list)
    assert ei.value.code == -1
    c.step()
    c.expect()
    c.check()


def test_offsets_past_32_bits():
    """A tensor of more than 2^32 bytes and one of more than 2^32 elements'
    worth of codes: the last pieces are the formula's."""
    n = (1 << 32) + 1000
    last = 3000
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(n, dtype=torch.int8, device="cuda")
    v = torch.zeros(n, dtype=torch.uint8, device="cuda")
    S = [torch.zeros(-(-n // 256), device="cuda") for _ in range(2)]
    rng = np.random.default_rng(3)
    G, w = normal(rng, last, 1e-3), normal(rng, last, 0.02)
    g[-last:] = torch.from_numpy(G).cuda()
    p[-last:] = torch.from_numpy(w).cuda()
    lst = zs.zs_tensors_create(params=[p], grads=[g], m=[m], v=[v],
                               m_scale=[S[0]], v_scale=[S[1]])
    upload(lst)
    G, w = OT.bf16(OT.to_bf16(G)), OT.bf16(OT.to_bf16(w))
    want = OT.sumsq([G])
    assert abs(sumsq_of(lst).item() / want - 1) < 1e-12
    zs.zs_tensors_step(lst, zs.zs_adamw(*HP), step=1)
    # from a block's start on
    lead = n - last - (n - last) % 256
    skip = n - last - lead
    G = np.concatenate([np.zeros(skip, np.float32), G])
    w = np.concatenate([np.zeros(skip, np.float32), w])
    m1, _, root = OT.moments(G, 0 * G, 0 * G, HP, 1)
    same(m[lead:], OT.encode(m1, 127)[0].astype(np.int8))
    same(v[lead:], OT.encode(root, 255)[0].astype(np.uint8))
    same(S[0][lead // 256:], OT.encode(m1, 127)[1])
    same(S[1][lead // 256:], OT.encode(root, 255)[1])
    kept, update = OT.weights64(w, m1, root, HP, 1)
    got = p[lead:].float().cpu().numpy()
    assert np.all(np.abs(got - (kept - update)) <=
                  (2.0 ** -8 + 2.0 ** -20) * np.abs(kept - update) +
                  2.0 ** -20 * np.abs(update))
    assert not m[:lead].any() and not p[:lead].any()


def test_more_pieces_than_a_launch_takes():
    """More than 2^34 elements go in two launches; what is at the ends of both
    is stepped once, and counted."""
    n, first = (1 << 34) + 5000, ((1 << 24) - 1) * 1024
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(n, dtype=torch.int8, device="cuda")
    v = torch.zeros(n, dtype=torch.uint8, device="cuda")
    S = [torch.zeros(-(-n // 256), device="cuda") for _ in range(2)]
    at = torch.tensor([0, first - 1, first, n - 1], device="cuda")
    p[at], g[at] = 1.0, 0.5
    lst = zs.zs_tensors_create(params=[p], grads=[g], m=[m], v=[v],
                               m_scale=[S[0]], v_scale=[S[1]])
    upload(lst)
    assert sumsq_of(lst).item() == 1.0
    # a step of lr 0.1 moves a weight by 0.1: to 0.8984 in bf16
    zs.zs_tensors_step(lst, zs.zs_adamw(0.1, 0.9, 0.95, 1e-8, 0.0), step=1)
    assert p[at].tolist() == [0.8984375] * 4
    assert m[at].tolist() == [127] * 4 and v[at].tolist() == [255] * 4
    for x in (p, m, v):
        x[at] = 0
        assert not x[:1 << 33].any() and not x[1 << 33:].any()


# ---- the binding's refusals ----------------------------------------------------------

def test_binding_refusals():
    f = torch.zeros(600, device="cuda")
    b = f.bfloat16()
    q, u = f.to(torch.int8), f.to(torch.uint8)
    s = torch.zeros(3, device="cuda")
    new = zs.zs_tensors_create
    with pytest.raises(TypeError):
        new(grads=[f, b])
    with pytest.raises(TypeError):
        new(grads=[f.double()])
    with pytest.raises(TypeError):
        new(params=[f.half()])
    with pytest.raises(TypeError):
        new(m=[f], v=[b])
    with pytest.raises(TypeError):
        new(m=[q], v=[f])
    with pytest.raises(TypeError):
        new(m=[f, q], v=[f, u])
    with pytest.raises(TypeError):
        new(params=[b], grads=[b], master=[b], m=[f], v=[f])
    with pytest.raises(TypeError):
        new(m=[q], v=[u], m_scale=[b[:3]], v_scale=[s])
    with pytest.raises(ValueError):
        new(m=[q], v=[u], m_scale=[s[:2]], v_scale=[s])
    with pytest.raises(ValueError):
        new(params=[f], m=[f[:599]], v=[f])
    with pytest.raises(ValueError):
        new(params=[f], grads=[f[:599]])
    with pytest.raises(ValueError):
        new(params=[f], grads=[f, f])
    with pytest.raises(ValueError):
        new(params=[f.view(20, 30).t()])
    with pytest.raises(ValueError):
        new(grads=[f.view(20, 30).t()])
    with pytest.raises(ValueError):
        new(params=[f[:300]], grads=[f.view(2, 300)], world=3)
    with pytest.raises(ValueError):
        new(params=[f[:20]], grads=[f.view(300, 2).t()[:, :20]], world=2)
    with pytest.raises(ValueError):
        new(grads=[f.cpu()])
    with pytest.raises(zs.ZsError):                 # no scales
        new(m=[q], v=[u])
    with pytest.raises(zs.ZsError):                 # twice
        new(params=[f, f], grads=[b, b])
    lst = new(grads=[f])
    with pytest.raises(zs.ZsError):
        zs.zs_tensors_upload(lst, torch.empty(8, dtype=torch.uint8,
                                              device="cuda"))
    upload(lst)
    with pytest.raises(zs.ZsError):
        zs.zs_tensors_step(lst, zs.zs_adamw(*HP), step=1)
    with pytest.raises(TypeError):
        zs.zs_tensors_sumsq(lst, f, workspace=u)
    big = torch.zeros(1 << 20, device="cuda")
    lst = new(grads=[big])
    upload(lst)
    out = torch.zeros(1, dtype=torch.float64, device="cuda")
    with pytest.raises(zs.ZsError):
        zs.zs_tensors_sumsq(lst, out, workspace=u[:8])
