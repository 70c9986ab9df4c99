"""Every kernel of the step over lists of tensors, on every way it accesses
memory: four and eight ranks have kernels of their own beside one and any other
number, each kind of weights, gradients and states too, and each of them takes
parts whose gradients lie at lines of 128 bytes, at four elements or anywhere,
and the ends of tensors.  Rows of gradients lie at the strides that lead there;
`ways` says from the addresses which of them a list takes.

Codes, scales and fp32 states are compared bit for bit with oracle/tensors.py,
bf16 parameters with the two that the bounds of the weight round to."""

import numpy as np
import pytest
import torch

import zero_sharded_optimizer_shard_amd as zs
from oracle import tensors as OT
from test_tensors_gpu import HP, Arena, normal, same, upload

pytestmark = pytest.mark.gpu

UNIT = {32: 256, 8: 512}        # elements of a part
LINE = 128


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def row_stride(n, rows, size):
    """Elements from one rank's row to the next."""
    line = LINE // size
    if rows == "lines":
        return -(-n // line) * line + line
    if rows == "fours":
        at = -(-n // 4) * 4
        return at + 4 if at % line == 0 else at
    at = n + 3
    return at if at % 4 else at + 1


class Rows:
    """One list with its host copy; rows of gradients at a kind of stride."""

    def __init__(self, sizes, state, weights, grad, world, rows="lines",
                 shift=0, apart=0, seed=0, edit=None):
        """shift: elements past an aligned address; apart: as many more with
        every array."""
        rng = np.random.default_rng(seed)
        self.state, self.world, self.sizes = state, world, sizes
        self.arena, self.host, self.dev = Arena(), [], []
        for n in sizes:
            spread = np.exp(rng.standard_normal(n)).astype(np.float32)
            G = normal(rng, (world, n), 1e-3) * spread
            w, m = normal(rng, n, 0.02), normal(rng, n, 3e-4) * spread
            v = np.square(normal(rng, n, 1e-3) * spread)
            h = {"grad": OT.to_bf16(G).reshape(world, n) if grad == "bf16"
                 else G}
            if weights == "master":
                h["master"], h["param"] = w, OT.to_bf16(w + 1)
            else:
                h["param"] = OT.to_bf16(w) if weights == "bf16" else w
            if state == 8:
                q = OT.hold(m, v)
                h.update(m=q[0].astype(np.int8), m_scale=q[1],
                         v=q[2].astype(np.uint8), v_scale=q[3])
            else:
                h.update(m=m, v=v)
            if edit:
                edit(h)
            d = {}
            for i, (k, x) in enumerate(h.items()):
                if k == "grad":
                    stride = row_stride(n, rows, x.itemsize)
                    # what lies between rows is not to be read
                    g = np.full((world, stride), 0x7fc0 if grad == "bf16"
                                else np.nan, x.dtype)
                    g[:, :n] = x
                    g = self.arena.put(g.reshape(-1), shift)
                    d[k] = g.view(world, stride)[:, :n] if world > 1 \
                        else g[:n]
                else:
                    codes = state == 8 and k in ("m", "v")
                    d[k] = self.arena.put(x, 0 if codes else
                                          shift + apart * i)
            self.host.append(h)
            self.dev.append(d)
        d = {k: [x[k] for x in self.dev] for k in self.dev[0]}
        self.list = zs.zs_tensors_create(
            params=d["param"], grads=d["grad"], world=world,
            **{k: d[k] for k in ("master", "m", "v", "m_scale", "v_scale")
               if k in d})
        upload(self.list)

    def ways(self):
        """Which ways the parts of the list are accessed."""
        out = set()
        for n, d in zip(self.sizes, self.dev):
            step = d["grad"].stride(0) if self.world > 1 else 0
            written = [x for k, x in d.items()
                       if k != "grad" and not k.endswith("scale")]

            def at(x, lead, to):
                return (x.data_ptr() + lead * x.element_size()) % to == 0

            def fours(lead):
                return step % 4 == 0 and all(
                    at(x, lead, 4 * x.element_size())
                    for x in written + [d["grad"]])

            def lines(lead):
                return fours(lead) and all(at(x, lead, LINE)
                                           for x in written)
            lead = 0
            if self.state == 32:
                lead = next((k for k in range(64) if lines(k)), None)
                if lead is None:
                    lead = next((k for k in (3, 2, 1) if fours(k)), 0)
            whole = (n - lead) // UNIT[self.state]
            if lead or n - lead > whole * UNIT[self.state]:
                out.add("edge")
            if whole <= 0:
                continue
            size = d["grad"].element_size()
            if not fours(lead):
                out.add("whole")
            elif (self.world > 1 and at(d["grad"], lead, LINE) and
                  step * size % LINE == 0):
                out.add("lines")
            else:
                out.add("aligned")
        return out

    def step(self, t=3, c=None, **kw):
        """A step of the list, and of the host copy with what its weights may
        be off by."""
        zs.zs_tensors_step(self.list, zs.zs_adamw(*HP), step=t, **kw)
        for h in self.host:
            G = h["grad"]
            g = OT.mean(OT.bf16(G) if G.dtype == np.uint16 else G)
            if c is not None:
                with np.errstate(all="ignore"):
                    g = g * c
            m, v = (h["m"], h["v"]) if self.state == 32 else OT.stands_for(
                h["m"], h["m_scale"], h["v"], h["v_scale"])
            m, v, root = OT.moments(g, m, v, HP, t)
            w = h.get("master", h["param"])
            w = OT.bf16(w) if w.dtype == np.uint16 else w
            if self.state == 32:
                h.update(m=m, v=v, w=OT.weights(w, m, root, HP, t), off=0.0)
                continue
            q = OT.encode(m, 127) + OT.encode(root, 255)
            kept, update = OT.weights64(w, m, root, HP, t)
            with np.errstate(all="ignore"):
                # as in test_tensors_gpu.py: eight half steps of 2^-24 in the
                # update, w*dec and the difference rounded once each
                off = 2.0 ** -24 * (8 * np.abs(update) + np.abs(kept) +
                                    np.abs(kept - update)) + 1e-44
                h.update(m=q[0].astype(np.int8), m_scale=q[1],
                         v=q[2].astype(np.uint8), v_scale=q[3],
                         w=kept - update, off=off)

    def check(self):
        for i, (h, d) in enumerate(zip(self.host, self.dev)):
            where = f"tensor {i} of {self.sizes[i]}"
            for k in ("m", "v"):
                if h[k].dtype == np.float32:
                    same_float(d[k], h[k], f"{where}: {k}")
                else:
                    same(d[k], h[k], f"{where}: {k}")
            for k in ("m_scale", "v_scale"):
                if k in h:
                    same_float(d[k], h[k], f"{where}: {k}")
            x = d.get("master", d["param"])
            if self.state == 32:
                w = h["w"] if x.dtype == torch.float32 \
                    else OT.bf16(OT.to_bf16(h["w"]))
                same_float(x.float(), w, f"{where}: weights")
            else:
                between(x, h["w"], h["off"], f"{where}: weights")
            if "master" in d:
                p = OT.to_bf16(x.cpu().numpy())
                same_float(d["param"].float(), OT.bf16(p), f"{where}: param")
            same(d["grad"].reshape(-1), h["grad"].reshape(-1),
                 f"{where}: grad")
        self.arena.check()


def same_float(got, want, where):
    """The same bits; any NaN for a NaN."""
    a, b = got.cpu().numpy(), want
    nan = np.isnan(b)
    assert np.array_equal(np.isnan(a), nan), where
    same(np.where(nan, np.float32(0), a), np.where(nan, np.float32(0), b),
         where)


def between(x, w, off, where):
    """x within `off` of w, or in bf16 one of those that such values round
    to."""
    got = x.float().cpu().numpy().astype(np.float64)
    nan = np.isnan(w)
    assert np.array_equal(np.isnan(got), nan), where
    got, w, off = got[~nan], w[~nan], off[~nan]
    with np.errstate(all="ignore"):
        lo, hi = w - off, w + off
        if x.dtype == torch.bfloat16:
            # fp32 values on the outer side of each bound
            a, b = lo.astype(np.float32), hi.astype(np.float32)
            a = np.where(a > lo, np.nextafter(a, np.float32(-np.inf)), a)
            b = np.where(b < hi, np.nextafter(b, np.float32(np.inf)), b)
            lo, hi = OT.bf16(OT.to_bf16(a)), OT.bf16(OT.to_bf16(b))
    inf = np.isinf(w)
    assert np.array_equal(got[inf], w[inf]), where
    assert np.all((lo <= got) & (got <= hi) | inf), where


# a few whole parts, what is left of one, and tensors that have no whole one
SIZES = [1, 300, 4 * 512 + 7, 4 * 1024]
WAYS = {"lines": "lines", "fours": "aligned", "odd": "whole"}


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("weights", ["master", "bf16", "f32"])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("world", [2, 3, 4, 5, 8])
@pytest.mark.parametrize("rows", ["lines", "fours", "odd"])
def test_rows_of_ranks(state, weights, grad, world, rows):
    c = Rows(SIZES, state, weights, grad, world, rows, seed=world)
    assert c.ways() == {WAYS[rows], "edge"}
    c.step()
    c.check()


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("weights", ["master", "bf16", "f32"])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("shift,apart", [(0, 0), (1, 1)])
def test_one_rank(state, weights, grad, shift, apart):
    c = Rows(SIZES, state, weights, grad, 1, shift=shift, apart=apart, seed=7)
    assert c.ways() == {"whole" if shift else "aligned", "edge"}
    c.step()
    c.check()


@pytest.mark.parametrize("weights", ["master", "bf16", "f32"])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("world", [4, 8])
def test_rows_at_lines_behind_a_lead(weights, grad, world):
    """All arrays and rows share their distance from a line, as a flat
    buffer's views do: units start at that line."""
    c = Rows(SIZES, 32, weights, grad, world, "lines", shift=37, seed=3)
    assert c.ways() == {"lines", "edge"}
    c.step()
    c.check()


@pytest.mark.parametrize("weights", ["master", "bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 37, 60])
def test_tensors_that_need_one_piece_more(weights, shift):
    """Units that start late in tensors of whole pieces, or nearly: their last
    elements are in pieces behind all others, one behind the other."""
    sizes = [1024, 2048, 5, 4095, 1, 5120, 1000, 300, 1023, 2049]
    c = Rows(sizes, 32, weights, "bf16", 1, shift=shift, seed=17)
    for t in (1, 2):
        c.step(t=t)
        c.check()
        for h, d in zip(c.host, c.dev):
            x = d["master" if "master" in d else "param"]
            h["master" if "master" in h else "param"] = \
                x.cpu().numpy() if x.dtype == torch.float32 else \
                OT.to_bf16(x.float().cpu().numpy())


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("weights", ["master", "bf16", "f32"])
@pytest.mark.parametrize("world,rows", [(1, "lines"), (4, "fours"),
                                        (8, "lines"), (3, "odd")])
def test_more_parts_than_a_round_of_runs(state, weights, world, rows):
    """With 8-bit states and fp32 weights XCDs take runs of 32 parts, 256 in
    all: two rounds of runs and a rest, over two tensors."""
    c = Rows([300 * 512 + 5, 250 * 512 + 9], state, weights, "bf16", world,
             rows, seed=5)
    c.step()
    c.check()


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("weights", ["master", "bf16", "f32"])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("world", [1, 4, 5])
def test_inf_and_nan_reach_every_kind_of_weights(state, weights, bad, world):
    """One gradient's: its weight is NaN, and with 8-bit states its block's
    states; nothing else changes by it."""
    def edit(h):
        if h["grad"].shape[1] > 300:
            h["grad"][world - 1, 299] = bad
    c = Rows([300, 1500], state, weights, "f32", world, edit=edit)
    c.step()
    assert [int(np.isnan(h["w"]).sum()) for h in c.host] == [0, 1]
    c.check()
    if state == 8:
        for h in c.host:
            assert np.flatnonzero(np.isnan(h["m_scale"])).tolist() == \
                np.flatnonzero(np.isnan(h["v_scale"])).tolist() == \
                [1] * (h["m"].size > 300)


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("world", [4, 8])
@pytest.mark.parametrize("rows", ["lines", "fours"])
def test_clipped_rows(state, world, rows):
    c = Rows(SIZES, state, "master", "bf16", world, rows, seed=11)
    s = torch.full((1,), 9.0, dtype=torch.float64, device="cuda")
    c.step(c=OT.coefficient(9.0, 0.75), sumsq=s, max_norm=0.75)
    c.check()


@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("world", [2, 4, 8])
@pytest.mark.parametrize("rows", ["lines", "fours", "odd"])
def test_sum_over_rows(grad, world, rows):
    c = Rows(SIZES + [70001], 32, "f32", grad, world, rows, seed=13)
    out = torch.zeros(1, dtype=torch.float64, device="cuda")
    ws = torch.empty(zs.zs_tensors_sumsq_workspace(c.list),
                     dtype=torch.uint8, device="cuda")
    zs.zs_tensors_sumsq(c.list, out, workspace=ws)
    want = OT.sumsq([OT.mean(OT.bf16(h["grad"]) if grad == "bf16"
                             else h["grad"]) for h in c.host])
    # exact squares to 2^-53, n sums of positive numbers on either side
    assert abs(out.item() - want) <= \
        2 * (sum(c.sizes) + 1) * 2.0 ** -53 * want
    c.arena.check()
