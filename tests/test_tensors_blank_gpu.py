"""Steps with 8-bit states of elements that have no gradient: what they hold of
m fades, as it does in fp32, so that their weights come to rest.  Against
oracle/tensors.py, and against a list with fp32 states over many steps."""

import numpy as np
import pytest
import torch

import zero_sharded_optimizer_shard_amd as zs
from oracle import tensors as OT
from test_tensors_gpu import HP, upload
from test_tensors_paths_gpu import Rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


# ---- one step after the other, bit for bit

def blanks(rng, n, i):
    """Which elements of a tensor have no gradient."""
    b = rng.random(n) < 0.4
    b[256:512] = True                   # a whole block: codes stay, A fades
    b[512:768] = True                   # all but one
    b[600:601] = False
    if i % 2:
        b[-1:] = False                  # the last block's only one
        b[-(n % 256):-1] = True
    return b


def value(G, blank, rng):
    """Gradients with zeros of both signs at `blank`; elsewhere some that are
    zero on all ranks but one, and some whose mean is zero."""
    W, n = G.shape
    neg = rng.random((W, n)) < 0.5
    zero = np.where(neg, -0.0, 0.0).astype(np.float32)
    if W > 1:
        one = rng.random(n) < 0.2
        keep = rng.integers(0, W, n)
        G = np.where(one & (np.arange(W)[:, None] != keep), zero, G)
        pair = ~one & (rng.random(n) < 0.2)
        G[:, pair] = 0
        G[0, pair], G[W - 1, pair] = 0.5, -0.5
    return np.where(blank, zero, G).astype(np.float32)


@pytest.mark.parametrize("weights", ["master", "bf16", "f32"])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("world,rows", [
    (1, "lines"), (2, "odd"), (3, "fours"), (4, "lines"), (4, "odd"),
    (5, "lines"), (8, "fours"), (8, "odd"), (11, "lines")])
@pytest.mark.parametrize("max_norm", [None, 0.75])
def test_blank_elements(weights, grad, world, rows, max_norm):
    rng = np.random.default_rng(world)
    where = []

    def edit(h):
        n = h["grad"].shape[1]
        where.append(blanks(rng, n, len(where)))
        G = h["grad"] if grad == "f32" else OT.bf16(h["grad"])
        G = value(G, where[-1], rng)
        h["grad"] = OT.to_bf16(G).reshape(G.shape) if grad == "bf16" else G
        # codes of every size, small ones above all
        h["m"] = rng.integers(-20, 21, n).astype(np.int8)
        h["m"][::7] = rng.integers(-127, 128, len(h["m"][::7]))
        h["m"][256:257] = 127
    c = Rows([1, 300, 700, 1024, 4 * 512 + 7], 8, weights, grad, world, rows,
             seed=world, edit=edit)
    kw, coef = {}, None
    if max_norm:
        kw = {"sumsq": torch.full((1,), 4.0, dtype=torch.float64,
                                  device="cuda"), "max_norm": max_norm}
        coef = OT.coefficient(4.0, max_norm)
    faded = 0
    for t in (3, 4, 5):
        states = [OT.stands_for(h["m"], h["m_scale"], h["v"], h["v_scale"])[0]
                  for h in c.host]
        was = [h["m"].astype(int) for h in c.host]
        c.step(t=t, c=coef, **kw)
        for h, m, b in zip(c.host, states, where):
            G = OT.bf16(h["grad"]) if grad == "bf16" else h["grad"]
            assert np.array_equal((G == 0).all(0), b)
            g = OT.mean(G) * np.float32(coef if max_norm else 1)
            m = OT.moments(g, m, 0 * m, HP, t)[0]
            q = OT.faded(h["m"].astype(int), m, b)
            faded += int((q != h["m"]).sum())
            h["m"] = q.astype(np.int8)
        c.check()
        for h, q, b in zip(c.host, was, where):
            # in the whole block without gradients only scales fade
            if h["m"].size >= 512 and b[256:512].all():
                assert np.array_equal(h["m"][256:512], q[256:512])
        for h, d in zip(c.host, c.dev):
            w = (d["master"] if "master" in d else d["param"])
            if "master" in h:
                h["master"] = w.cpu().numpy()
            else:
                h["param"] = w.cpu().numpy() if weights == "f32" else \
                    OT.to_bf16(w.float().cpu().numpy())
    assert faded > 100


def test_a_block_with_nan_or_without_scale():
    """One element's NaN makes the block's states NaN, blank ones too; a block
    whose largest is below 2^-100 is held as zeros."""
    def edit(h):
        h["grad"][0, ::3] = 0
        h["grad"][0, 255] = np.nan
        h["grad"][0, 256:512] *= np.float32(2.0 ** -110)
        h["m_scale"][1] = 2.0 ** -125
    c = Rows([512], 8, "f32", "f32", 1, edit=edit)
    c.step()
    assert np.isnan(c.host[0]["m_scale"][0]) and c.host[0]["m_scale"][1] == 0
    c.check()


# ---- beside fp32 states

def lists(n):
    """(list with 8-bit states, its weights), and the same with fp32 states,
    over one gradient."""
    g = torch.zeros(n, device="cuda")
    out = []
    for state in (8, 32):
        p = torch.zeros(n, device="cuda")
        if state == 8:
            kw = {"m": torch.zeros(n, dtype=torch.int8, device="cuda"),
                  "v": torch.zeros(n, dtype=torch.uint8, device="cuda"),
                  "m_scale": torch.zeros(n // 256, device="cuda"),
                  "v_scale": torch.zeros(n // 256, device="cuda")}
        else:
            kw = {k: torch.zeros(n, device="cuda") for k in ("m", "v")}
        lst = zs.zs_tensors_create(params=[p], grads=[g],
                                   **{k: [x] for k, x in kw.items()})
        upload(lst)
        out.append((lst, p, kw["m"]))
    return g, out


@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("beta1,beta2", [(0.9, 0.95), (0.95, 0.95),
                                         (0.9, 0.999)])
def test_weights_without_gradients_come_to_rest(spread, beta1, beta2):
    """An eighth of the elements of every block has no gradient after step
    300: in units of lr they move by what is left in m, a few, and then no
    more (they moved by hundreds more in 1500 steps where codes of m stayed)."""
    n = 64 * 256
    gen = torch.Generator(device="cuda").manual_seed(5)

    def randn():
        return torch.randn(n, generator=gen, device="cuda")
    sigma = 1e-3 * torch.exp(spread * randn())
    dead = torch.arange(n, device="cuda") % 8 == 0
    g, ((a, p8, m8), (b, p32, _)) = lists(n)
    at = {}
    for t in range(1, 1801):
        g.copy_((randn() + 0.1) * sigma)
        if t > 300:
            g[dead] = 0
        for lst in (a, b):
            zs.zs_tensors_step(lst, zs.zs_adamw(1.0, beta1, beta2, 1e-8, 0.0),
                               step=t)
        if t in (300, 900, 1800):
            at[t] = p8[dead].double(), p32[dead].double()

    def moved(x, t, u):
        return (at[u][x] - at[t][x]).square().mean().sqrt().item()
    # sum of what is left of m over its root: below 1 / (1 - beta1) lr
    left = moved(1, 300, 1800)
    assert 0.5 < left < 1 / (1 - beta1)
    assert moved(0, 300, 1800) < 1 / (1 - beta1)
    assert moved(0, 900, 1800) == 0 and not m8[dead].any()
