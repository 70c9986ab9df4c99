"""What is measured of the operators over lists of tensors: the AdamW step
with states in 32 bits or in 8 (zs_tensors_step), the sum of squares of the
gradients that clipping by the global norm takes (zs_tensors_sumsq), and the
conversion of states between 8 and 32 bits (zs_tensors_convert).

Each case is run either in its plain form (torch operations in 32 bits) or,
with `own` true, by the library's calls.  The plain form states the
operators; every fp32 operation is rounded once:

  mean      g = (G_0 + ... + G_{W-1}) / W, summed in rank order
  sumsq     s = sum of g^2 over all tensors, in 64 bits
  clip      g <- g c,  c = MAX_NORM / sqrt(s) where sqrt(s) > MAX_NORM, else 1
  AdamW     m <- b1 m + (1-b1) g,  v <- b2 v + (1-b2) g^2
            P <- P (1 - lr wd) - lr/(1-b1^t) m / (sqrt(v)/sqrt(1-b2^t) + eps)
  8 bits    of each block of 256 elements, A the largest: x = q^2 A / top^2,
            q the whole number nearest to top sqrt(x / A); top = 127 for |m|,
            which keeps its sign, and 255 for the root of v, where q is at
            least 1 unless the root is 0

The tensors of a case lie in flat buffers, each from a multiple of 256
elements on; what is held in 8 bits is returned as the values it stands for.
"""

import struct
from functools import reduce

import torch

own = False

BLOCK = 256
VECTOR = 8192        # tensors up to this size (norms, biases) do not decay


def _f32(x):
    return struct.unpack("f", struct.pack("f", x))[0]


LR, B1, B2, EPS, WD = (_f32(x) for x in (3e-4, 0.9, 0.95, 1e-8, 0.1))
STEP = 100
MAX_NORM = 1.0
MASTER_SIGMA, GRAD_SIGMA = 0.02, 1e-3
STEP_SIZE = LR / (1 - B1 ** STEP)
ROOT_BC2 = (1 - B2 ** STEP) ** 0.5
TINY = 2.0 ** -100   # a block whose largest is below is held as zeros


# ---- cases -------------------------------------------------------------------

def _case(name, op, tensors, world=1, grad="bf16", weights="master",
          clip=False, shift=0):
    """`tensors`: sizes as "N" or "N*count", in order.  weights: "master"
    (bf16 with an fp32 master), "bf16" or "f32" (updated in place).  shift:
    elements that gradients and weights start past an aligned address."""
    return dict(name=name, op=op, tensors=tensors, world=world, grad=grad,
                weights=weights, clip=clip, shift=shift)


def _gpt2(d=768, vocab=50257, ctx=1024, layers=12):
    block = [d, d, 3 * d * d, 3 * d, d * d, d, d, d, 4 * d * d, 4 * d,
             4 * d * d, d]
    return ",".join(map(str, [vocab * d, ctx * d] + layers * block + [d, d]))


_TINY = "262144,524288,262144,512*4,65536"
_LAYER = "4096,16777216,4194304*2,16777216,4096,58720256*3"
_RAGGED = ("1,3,17,255,256,257,1023,1025,4099,50257,1010477*3,128255,"
           "2050049,31*40,7000001")


def listed():
    return [
        # one norm vector by itself: a call's latency
        _case("adamw one vector", "adamw", "768", grad="f32", weights="f32"),
        # every tensor of a 12-layer 768-wide model, clipped
        _case("adamw gpt2 list", "adamw", _gpt2(), clip=True),
        # odd sizes at odd addresses, three ranks, no master
        _case("adamw ragged W=3", "adamw", _RAGGED, world=3, weights="bf16",
              shift=1),
        # one layer of an 8B-shaped model, eight ranks' slices
        _case("adamw 8B layer W=8", "adamw", _LAYER, world=8),
        # the smallest parameter list of the repository
        _case("adamw8 tiny list W=4", "adamw8", _TINY, world=4),
        # as above, with the states in 8 bits
        _case("adamw8 gpt2 list", "adamw8", _gpt2(), clip=True),
        # odd sizes at odd addresses, all in fp32
        _case("adamw8 ragged f32", "adamw8", _RAGGED, grad="f32",
              weights="f32", shift=1),
        # the least memory: bf16 weights and 8-bit states
        _case("adamw8 8B layer bf16", "adamw8", _LAYER, weights="bf16"),
        # the norm before the tiny list's step, and before a layer's
        _case("sumsq tiny list W=4", "sumsq", _TINY, world=4),
        _case("sumsq 8B layer", "sumsq", _LAYER),
        # a checkpoint in 32 bits from states in 8
        _case("unpack gpt2 list", "unpack", _gpt2()),
        # training in 8 bits begun from 32: there, and back for a look
        _case("pack+unpack 8B layer", "repack", _LAYER),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    """1 to 200 tensors of 1 to 40 M elements, spread by their logarithm, odd
    ones among them, 100 M elements at most."""
    op = rng.choice(["adamw", "adamw", "adamw8", "adamw8", "sumsq", "unpack",
                     "repack"])
    top = _log(rng, 1000, 40_000_000)
    sizes, left = [], 100_000_000
    for _ in range(_log(rng, 1, 200)):
        n = _log(rng, 1, top)
        if rng.random() < 0.5:           # sizes as models have them
            n = max(64, n // 64 * 64)
        if n <= left:
            sizes.append(n)
            left -= n
    d = _case("", op, ",".join(map(str, sizes)))
    if op in ("adamw", "adamw8", "sumsq"):
        d.update(world=rng.choice([1, 1, 2, 3, 4, 8]),
                 grad=rng.choice(["bf16", "bf16", "f32"]),
                 shift=rng.choice([0, 0, 0, 1]))
    if op in ("adamw", "adamw8"):
        d.update(weights=rng.choice(["master", "master", "bf16", "f32"]),
                 clip=rng.random() < 0.5)
    del d["name"]
    return d


def _sizes(case):
    out = []
    for t in case["tensors"].split(","):
        n, _, count = t.partition("*")
        out += [int(n)] * int(count or 1)
    return out


def work(case):
    """Bytes: inputs and outputs once, the states in 8 bits as they are held
    and the values that they stand for where those are returned.  Operations:
    about 20 an element of a step, four of a conversion."""
    n, W = sum(_sizes(case)), case["world"]
    grads = W * (2 if case["grad"] == "bf16" else 4)
    weights = {"master": 10, "bf16": 4, "f32": 8}[case["weights"]]
    held = 2 + 8 / BLOCK
    b, f = {"adamw": (grads + weights + 16, W + 20),
            "adamw8": (grads + weights + 2 * held + 8, W + 30),
            "sumsq": (grads, W + 2),
            "unpack": (held + 8, 4),
            "repack": (8 + held + 8, 14)}[case["op"]]
    return {"bytes": n * b, "flops": n * f}


# ---- inputs -------------------------------------------------------------------

def _places(sizes):
    out, off = [], 0
    for n in sizes:
        out.append(off)
        off += -(-n // BLOCK) * BLOCK
    return out, off


def _buffer(n, dtype, shift, rows=None):
    """Zeros, [n] or [rows, n], from `shift` elements past an aligned address
    on (rows a multiple of 16 bytes apart)."""
    b = torch.zeros((rows or 1) * (n + 8), dtype=dtype, device="cuda")
    b = b.view(rows or 1, n + 8)[:, shift:shift + n]
    return b if rows else b[0]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    sizes = _sizes(case)
    offs, N = _places(sizes)
    nb, W, op = N // BLOCK, case["world"], case["op"]
    lens = torch.tensor(sizes, device="cuda")
    starts = torch.tensor(offs, device="cuda")
    # which tensor a block is of; the padding behind a tensor holds zeros
    tensor = torch.repeat_interleave((lens + BLOCK - 1) // BLOCK,
                                     output_size=nb)
    inside = (torch.arange(N, device="cuda").view(nb, BLOCK)
              < (starts + lens)[tensor][:, None]).view(N)

    def randn():
        return torch.randn(N, generator=g, device="cuda").mul_(inside)

    # blocks (rows of a matrix) differ in size, as gradients do
    size = GRAD_SIGMA * torch.exp(0.7 * torch.randn(nb, 1, generator=g,
                                                    device="cuda"))
    size = size.expand(nb, BLOCK).reshape(N)
    f32, bf16 = torch.float32, torch.bfloat16
    shift = case["shift"]
    if op in ("adamw", "adamw8", "sumsq"):
        st["grads"] = _buffer(N, bf16 if case["grad"] == "bf16" else f32,
                              shift, W)
        signal = 0.5 * randn()
        for s in range(W):
            st["grads"][s] = (signal + randn()) * size
    m = 0.3 * randn() * size
    v = ((0.2 + randn().abs()) * size * inside).square_()
    if op != "sumsq":
        if op in ("adamw", "repack"):
            st["m"], st["v"] = (_buffer(N, f32, shift) for _ in range(2))
            st["m"].copy_(m)
            st["v"].copy_(v)
        if op in ("adamw8", "unpack"):
            st.update(zip(("m", "m_scale", "v", "v_scale"),
                          _encode(m, 127, True) + _encode(v.sqrt(), 255,
                                                          False)))
        if op == "repack":
            st.update(zip(("m8", "m_scale", "v8", "v_scale"),
                          _encode(m * 0, 127, True) + _encode(v * 0, 255,
                                                              False)))
    del m, v
    if op in ("adamw", "adamw8"):
        w = MASTER_SIGMA * randn()
        if case["weights"] == "master":
            st["master"] = _buffer(N, f32, shift)
            st["master"].copy_(w)
        st["params"] = _buffer(N, f32 if case["weights"] == "f32" else bf16,
                               shift)
        st["params"].copy_(w)
        st["decay"] = torch.tensor(
            [1.0 if n <= VECTOR else 1 - LR * WD for n in sizes],
            dtype=f32, device="cuda")
        st["tensor"] = tensor
        if case["clip"]:
            st["sumsq"] = torch.full((1,), 3.7 + seed % 7 / 8,
                                     dtype=torch.float64, device="cuda")
    if own:
        _plan(st, sizes, offs, N)
    return st


def _plan(st, sizes, offs, N):
    """The handle, tables and buffers that a program makes once."""
    import zero_sharded_optimizer_shard_amd as zs

    def views(t, per=1):
        return None if t is None else [
            t[..., o // per:o // per + -(-n // per)]
            for o, n in zip(offs, sizes)]

    def tensors(**kw):
        lst = zs.zs_tensors_create(**kw)
        zs.zs_tensors_upload(lst, torch.empty(
            zs.zs_tensors_table_bytes(lst), dtype=torch.uint8,
            device="cuda"))
        return lst

    op = st["op"]
    if op == "sumsq":
        st["list"] = tensors(grads=views(st["grads"]), world=st["world"])
        st["out"] = torch.empty(1, dtype=torch.float64, device="cuda")
        st["workspace"] = torch.empty(
            zs.zs_tensors_sumsq_workspace(st["list"]), dtype=torch.uint8,
            device="cuda")
        return
    scales = {k: views(st[k], BLOCK) for k in ("m_scale", "v_scale")
              if k in st}
    if op in ("adamw", "adamw8"):
        st["list"] = tensors(
            grads=views(st["grads"]), world=st["world"],
            params=views(st["params"]), master=views(st.get("master")),
            m=views(st["m"]), v=views(st["v"]),
            groups=[int(n <= VECTOR) for n in sizes], **scales)
        st["hp"] = [zs.zs_adamw(LR, B1, B2, EPS, wd) for wd in (WD, 0.0)]
    elif op == "unpack":
        st["list"] = tensors(m=views(st["m"]), v=views(st["v"]), **scales)
    else:
        st["from"] = tensors(m=views(st["m"]), v=views(st["v"]))
        st["list"] = tensors(m=views(st["m8"]), v=views(st["v8"]), **scales)
    if op != "adamw":
        st["values"] = torch.zeros(2, N, device="cuda")
        st["to"] = tensors(m=views(st["values"][0]),
                           v=views(st["values"][1]))


# ---- the plain form ------------------------------------------------------------

def _over(x, by):
    """x / by, divided (a product with 1 / by is rounded twice)."""
    return x / torch.full((1,), by, dtype=x.dtype, device=x.device)


def _mean(st):
    return _over(reduce(torch.add, st["grads"].float().unbind(0)),
                 float(st["world"]))


def _encode(x, top, signed):
    """(codes, scales) of the blocks of x.  The root is taken in 64 bits, as
    it decides between neighbours next to a border."""
    x = x.view(-1, BLOCK)
    most = x.abs().amax(-1, keepdim=True)
    some = most >= TINY
    scale = torch.where(some, most * _f32(1 / top ** 2), 0.0)
    inv = torch.where(some, torch.full_like(most, top ** 2) / most, 0.0)
    q = torch.floor((x.abs() * inv).double().sqrt() + 0.5)
    if signed:
        q = (q * x.sign()).to(torch.int8)
    else:
        q = torch.where(some & (x > 0), q.clamp(min=1), 0).to(torch.uint8)
    return q.view(-1), scale.view(-1)


def _decode(q, scale):
    q = q.float().view(-1, BLOCK)
    return (q * q.abs() * scale.view(-1, 1)).view(-1)


def _values(m, m_scale, v, v_scale):
    root = _decode(v, v_scale)
    return _decode(m, m_scale), root * root


def _clipped(st, g):
    if not st["clip"]:
        return g
    norm = st["sumsq"].sqrt()
    return g * torch.where(norm > MAX_NORM, torch.full_like(norm, MAX_NORM)
                           / norm, 1.0).float()


def _plain_step(st):
    g = _clipped(st, _mean(st))
    if st["op"] == "adamw8":
        m, v = _values(st["m"], st["m_scale"], st["v"], st["v_scale"])
    else:
        m, v = st["m"], st["v"]
    m = B1 * m + (1 - B1) * g
    v = B2 * v + (1 - B2) * (g * g)
    root = v.sqrt()
    P = st["master"] if "master" in st else st["params"].float()
    P = (P.view(-1, BLOCK) * st["decay"][st["tensor"]][:, None]).view(-1)
    P = P - STEP_SIZE * (m / (_over(root, ROOT_BC2) + EPS))
    if "master" in st:
        st["master"].copy_(P)
    st["params"].copy_(P)
    if st["op"] == "adamw":
        st["m"].copy_(m)
        st["v"].copy_(v)
        return m, v
    st["m"], st["m_scale"] = _encode(m, 127, True)
    st["v"], st["v_scale"] = _encode(root, 255, False)
    return _values(st["m"], st["m_scale"], st["v"], st["v_scale"])


def _weights(st):
    return {k: st[k] for k in ("params", "master") if k in st}


def run(st):
    if own:
        return _own(st)
    op = st["op"]
    if op == "sumsq":
        return _mean(st).double().square_().sum().view(1)
    if op == "unpack":
        m, v = _values(st["m"], st["m_scale"], st["v"], st["v_scale"])
    elif op == "repack":
        m, v = _values(*_encode(st["m"], 127, True),
                       *_encode(st["v"].sqrt(), 255, False))
    else:
        m, v = _plain_step(st)
    return {"m": m, "v": v, **_weights(st)}


def _own(st):
    import zero_sharded_optimizer_shard_amd as zs
    op = st["op"]
    if op == "sumsq":
        zs.zs_tensors_sumsq(st["list"], st["out"],
                            workspace=st["workspace"])
        return st["out"]
    if op == "repack":
        zs.zs_tensors_convert(st["from"], st["list"])
    elif op != "unpack":
        zs.zs_tensors_step(st["list"], st["hp"], step=STEP,
                           sumsq=st.get("sumsq"), max_norm=MAX_NORM)
    if op == "adamw":
        return {"m": st["m"], "v": st["v"], **_weights(st)}
    zs.zs_tensors_convert(st["list"], st["to"])
    return {"m": st["values"][0], "v": st["values"][1], **_weights(st)}


# ---- 64 bits --------------------------------------------------------------------

def _round(x):
    """The fp32 value next to a 64-bit one, in 64 bits."""
    return x.float().double()


def _held(x, top):
    """What blocks of fp32 values (given in 64 bits) are held as: the codes
    by their borders, which are whole numbers and a quarter."""
    b = x.view(-1, BLOCK)
    most = b.abs().amax(-1, keepdim=True).clamp(min=1e-300)
    y = _round(b.abs() * _round(top ** 2 / most))
    borders = (torch.arange(top, dtype=torch.float64, device=x.device)
               + 0.5) ** 2
    q = torch.bucketize(y, borders, right=True).double()
    if top == 255:
        q = torch.maximum(q, (b > 0).double())
    out = b.sign() * q * q * _round(most * _f32(1 / top ** 2))
    return torch.where(most < TINY, 0.0, out).reshape(-1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "adamw":
        g = st["grads"].double().mean(0)
    elif op in ("adamw8", "sumsq"):
        # the codes and the sum are of the mean that fp32 has
        g = _round(reduce(lambda a, b: _round(a + b),
                          st["grads"].double().unbind(0)) / case["world"])
    if op == "sumsq":
        return (g * g).sum().view(1)
    if op in ("adamw8", "unpack"):
        m, root = (q.double().view(-1, BLOCK) for q in (st["m"], st["v"]))
        m = (m.sign() * m ** 2 * st["m_scale"].double()[:, None]).view(-1)
        root = (root ** 2 * st["v_scale"].double()[:, None]).view(-1)
        if op == "unpack":
            return {"m": m, "v": root ** 2}
        # the next codes are of the fp32 values that the step has
        m, v = _round(m), _round(_round(root) ** 2)
        if case["clip"]:
            c = min(1.0, MAX_NORM / st["sumsq"].item() ** 0.5)
            g = _round(g * _f32(c))
        m = _round(_round(B1 * m) + _round(_f32(1 - B1) * g))
        v = _round(_round(B2 * v) + _round(_f32(1 - B2) * _round(g * g)))
        held_m = _held(m, 127)
        held_v = _held(_round(v.sqrt()), 255).square_()
    elif op == "repack":
        return {"m": _held(st["m"].double(), 127),
                "v": _held(_round(st["v"].double().sqrt()), 255).square_()}
    else:
        if case["clip"]:
            g = g * min(1.0, MAX_NORM / st["sumsq"].item() ** 0.5)
        m = st["m"].double() + (1 - B1) * (g - st["m"])
        v = st["v"].double() + (1 - B2) * (g.square() - st["v"])
        held_m, held_v = m, v
    P = st["master" if "master" in st else "params"].double()
    wd = torch.where(st["decay"] < 1, WD, 0.0).double()[st["tensor"], None]
    update = m / (1 - B1 ** STEP) / ((v / (1 - B2 ** STEP)).sqrt() + EPS)
    P = P - LR * ((wd * P.view(-1, BLOCK)).view(-1) + update)
    out = {"params": P, "m": held_m, "v": held_v}
    if "master" in st:
        out["master"] = P
    return out
