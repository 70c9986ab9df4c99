"""What is measured of the Muon operators: orthogonalisation by Newton-Schulz
products (zs_orthogonalize) and the whole-tensor Muon step (zs_muon_step).

Each case is run either in its plain form (torch products in 32 bits, rounded
once at the end) or, with `own` true, by the library's calls.  The plain form
states the operators:

  orthogonalise   X_0 = U / (|U|_F + eps), and per step with (a, b, c)
                  A = X X^T,  X <- a X + (b A + c A A) X
                  (for a matrix with more rows than columns X^T X on the right)
  Muon step       g = (G_0 + ... + G_{W-1}) / W,   M <- mu M + g
                  U = g + mu M (Nesterov) or M,    O = orthogonalise(U)
                  P <- P (1 - lr wd) - lr s O,     s by the matrix's shape
                  p = bf16(P)
"""

from functools import reduce

import torch

own = False

TILE = 8192          # elements of one state tile (ZS_TILE)
ALIGN = 128          # elements a tensor's place in the shard is padded to
A, B, C = 3.4445, -4.7750, 2.0315
EPS = 1e-7
LR, MU, WD = 3e-4, 0.95, 0.1
MASTER_SIGMA, GRAD_SIGMA = 0.02, 1e-3


# ---- cases -------------------------------------------------------------------

def _orth(name, shape, dtype, precision, batch=1, pitch=0, steps=5):
    """`pitch`: elements between the rows beyond the columns (a view into a
    wider matrix)."""
    return dict(name=name, op="orthogonalize", rows=shape[0], cols=shape[1],
                batch=batch, dtype=dtype, precision=precision, pitch=pitch,
                steps=steps)


def _muon(name, tensors, world, layout, precision="fast", nesterov=True,
          scale="rms", steps=5):
    """`tensors`: the matrices this rank owns, as "RxC" or "BxRxC" (a stack of
    B matrices in one tensor, each stepped by itself)."""
    return dict(name=name, op="muon_step", tensors=tensors, world=world,
                layout=layout, precision=precision, nesterov=nesterov,
                scale=scale, steps=steps)


def listed():
    return [
        # one small matrix by itself: a call's latency
        _orth("orth 64x64 bf16", (64, 64), "bf16", "fast"),
        # a tensor of the smallest parameter list, in full precision
        _orth("orth 512x1024 f32", (512, 1024), "f32", "full"),
        # the attention output projections of a 12-layer 768-wide model
        _orth("orth 12x768x768 bf16", (768, 768), "bf16", "fast", batch=12),
        # odd sides, rows of a wider matrix, more rows than columns
        _orth("orth 3x1001x333 f32 pitch", (1001, 333), "f32", "full",
              batch=3, pitch=7),
        # a key projection of an 8B-shaped layer in full precision
        _orth("orth 1024x4096 f32", (1024, 4096), "f32", "full"),
        # a query projection of the same layer
        _orth("orth 4096x4096 bf16", (4096, 4096), "bf16", "fast"),
        # the matrices of the smallest parameter list, owned whole
        _muon("muon tiny W=4", "512x512,512x1024,1024x256,1024x64", 4,
              "tiled"),
        # one block of the 12-layer model, rows as the parameter list has them
        _muon("muon gpt2 block W=8", "768x2304,768x768", 8, "slices",
              scale="shape"),
        # ragged: odd sides, a single row, a single column, three ranks
        _muon("muon ragged W=3", "777x1301,129x65,1x4099,515x1,5x31x63", 3,
              "slices", nesterov=False, scale="none", precision="full"),
        # a stack of experts in one tensor
        _muon("muon experts W=2", "16x1408x512", 2, "tiled"),
        # an owner's part of an 8B-shaped model: one tensor of each shape
        _muon("muon 8B-shaped W=8",
              "4096x4096,1024x4096,14336x4096,4096x14336", 8, "tiled"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _flops(m, n):
    m, n = min(m, n), max(m, n)
    return 3 * m * m * n + m ** 3


def draw(rng):
    """Sides spread over 1..6000 by their logarithm, odd ones among them, and
    no more work than one 4096 x 8192 matrix."""
    most = _flops(4096, 8192)

    def shape():
        while True:
            r, c = _log(rng, 1, 6000), _log(rng, 1, 6000)
            if rng.random() < 0.4:       # sides as models have them
                r, c = max(64, r // 64 * 64), max(64, c // 64 * 64)
            if _flops(r, c) <= most / 4:
                return r, c

    precision = rng.choice(["fast", "fast", "full"])
    steps = rng.choice([5, 5, 5, 1, 6])
    if rng.random() < 0.5:
        r, c = shape()
        batch = min(rng.choice([1, 1, 2, 5, 24]),
                    max(1, most // _flops(r, c)))
        dtype = "f32" if precision == "full" else "bf16"
        d = _orth("", (r, c), dtype, precision, batch,
                  rng.choice([0, 0, 3, 64]), steps)
    else:
        d = _muon("", ",".join("%dx%d" % shape()
                               for _ in range(rng.randint(1, 4))),
                  rng.choice([1, 2, 3, 4, 8]),
                  rng.choice(["tiled", "slices"]), precision,
                  rng.random() < 0.7, rng.choice(["rms", "none"]), steps)
    del d["name"]
    return d


def _shapes(case):
    """[(batch, rows, cols)] of a case's tensors."""
    if case["op"] == "orthogonalize":
        return [(case["batch"], case["rows"], case["cols"])]
    s = [tuple(int(v) for v in t.split("x"))
         for t in case["tensors"].split(",")]
    return [t if len(t) == 3 else (1,) + t for t in s]


def work(case):
    """Bytes: inputs and outputs once.  Operations: per step the products of
    X X^T and A A for one triangle each (both are symmetric) and B X."""
    shapes = _shapes(case)
    n = sum(b * r * c for b, r, c in shapes)
    flops = case["steps"] * sum(b * _flops(r, c) for b, r, c in shapes)
    if case["op"] == "orthogonalize":
        return {"bytes": n * (4 if case["dtype"] == "bf16" else 8),
                "flops": flops}
    # W gradients, master and momentum read and written, the parameter out
    return {"bytes": n * (2 * case["world"] + 18), "flops": flops}


# ---- inputs -------------------------------------------------------------------

def _matrix(g, b, r, c, sigma, noise=0.5):
    """A few strong directions over a floor of noise, as gradients have."""
    k = max(1, min(r, c) // 32)
    u = torch.randn(b, r, k, generator=g, device="cuda")
    v = torch.randn(b, k, c, generator=g, device="cuda")
    s = torch.linspace(1.0, 0.2, k, device="cuda") / k ** 0.5
    x = torch.bmm(u * s, v)
    x += noise * torch.randn(b, r, c, generator=g, device="cuda")
    return x.mul_(sigma)


def _places(shapes):
    """Per tensor (elements, first shard element, first tile, tiles)."""
    out, off, tile = [], 0, 0
    for b, r, c in shapes:
        n = b * r * c
        pad = -(-n // ALIGN) * ALIGN
        t = -(-pad // TILE)
        out.append((n, off, tile, t))
        off, tile = off + pad, tile + t
    return out, off, tile


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    shapes = _shapes(case)
    if case["op"] == "orthogonalize":
        (b, r, c), = shapes
        t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        wide = torch.zeros(b, r, c + case["pitch"], dtype=t, device="cuda")
        wide[..., :c] = _matrix(g, b, r, c, GRAD_SIGMA).to(t)
        st["x"] = wide[..., :c]
        if own:
            import zero_sharded_optimizer_shard_amd as zs
            st["o"] = torch.empty_like(wide)[..., :c]
            st["workspace"] = torch.empty(
                zs.zs_orthogonalize_workspace([st["x"]], case["precision"]),
                dtype=torch.uint8, device="cuda")
        return st
    W = case["world"]
    places, n, tiles = _places(shapes)
    state = torch.zeros(tiles, 3, TILE, device="cuda")
    grads = []
    st["stride"] = n
    flat = torch.zeros(W, n, dtype=torch.bfloat16, device="cuda")
    tiled = torch.zeros(tiles, W, TILE, dtype=torch.bfloat16, device="cuda")
    for (b, r, c), (e, off, tile, t) in zip(shapes, places):
        rows = torch.zeros(2, t * TILE, device="cuda")
        rows[0, :e] = MASTER_SIGMA * torch.randn(e, generator=g,
                                                 device="cuda")
        signal = _matrix(g, b, r, c, GRAD_SIGMA).view(-1)
        # a momentum of several steps: the signal summed, the noise less so
        rows[1, :e] = 6 * signal + 2 * GRAD_SIGMA * torch.randn(
            e, generator=g, device="cuda")
        state[tile:tile + t, :2] = rows.view(2, t, TILE).transpose(0, 1)
        for s in range(W):
            x = signal + GRAD_SIGMA * torch.randn(e, generator=g,
                                                  device="cuda")
            flat[s, off:off + e] = x.bfloat16()
            row = torch.zeros(t * TILE, dtype=torch.bfloat16, device="cuda")
            row[:e] = flat[s, off:off + e]
            tiled[tile:tile + t, s] = row.view(t, TILE)
        if case["layout"] == "tiled":
            grads.append(tiled[tile:tile + t])
        else:
            grads.append(flat[:, off:])
    st.update(state=state, grads=grads, params=torch.zeros(
        n, dtype=torch.bfloat16, device="cuda"))
    if own:
        import zero_sharded_optimizer_shard_amd as zs
        # every rank owns one tensor of each shape; this is the first rank
        st["plan"] = zs.zs_layout_build_tensors(
            [e for e, _, _, _ in places for _ in range(W)], W, 0)
        st["tensors"] = [(i,) + s for i, s in enumerate(shapes)]
        # slices: the rows of the shard's [W][stride] buffer from the
        # tensor's first element on
        st["grads"] = [x if case["layout"] == "tiled" else
                       flat.view(-1)[off:]
                       for x, (_, off, _, _) in zip(grads, places)]
        st["workspace"] = torch.empty(
            zs.zs_muon_workspace(st["plan"], st["tensors"],
                                 case["precision"]),
            dtype=torch.uint8, device="cuda")
    return st


# ---- the plain form ------------------------------------------------------------

def _step(X):
    """One step in 32 bits, on the side with fewer rows."""
    if X.shape[-2] > X.shape[-1]:
        return _step(X.mT.contiguous()).mT
    M = X @ X.mT.contiguous()
    return A * X + (B * M + C * (M @ M)) @ X


def _orthogonalised(U, steps):
    U = U.float()
    norm = U.double().square().sum((-2, -1), keepdim=True).sqrt() + EPS
    return reduce(lambda X, _: _step(X), range(steps), U * (1 / norm).float())


def _scale(mode, r, c):
    return {"none": 1.0, "shape": max(1.0, r / c) ** 0.5,
            "rms": 0.2 * max(r, c) ** 0.5}[mode]


def _muon_plain(st, shape, place, grads):
    (b, r, c), (e, off, tile, t) = shape, place
    rows = st["state"][tile:tile + t]
    if st["layout"] == "tiled":
        G = grads.transpose(0, 1).reshape(st["world"], -1)[:, :e]
    else:
        G = grads[:, :e]
    g = G.float().sum(0) / st["world"]
    P = rows[:, 0].reshape(-1)[:e]
    M = MU * rows[:, 1].reshape(-1)[:e] + g
    U = g + MU * M if st["nesterov"] else M
    O = _orthogonalised(U.view(b, r, c), st["steps"]).reshape(-1)
    P = P * (1 - LR * WD) - LR * _scale(st["scale"], r, c) * O
    both = torch.nn.functional.pad(torch.stack([P, M]), (0, t * TILE - e))
    rows[:, :2] = both.view(2, t, TILE).transpose(0, 1)
    st["params"][off:off + e] = P.bfloat16()


def run(st):
    if own:
        import zero_sharded_optimizer_shard_amd as zs
    if st["op"] == "orthogonalize":
        if own:
            zs.zs_orthogonalize([st["x"]], [st["o"]], steps=st["steps"],
                                coef=(A, B, C), eps=EPS,
                                precision=st["precision"],
                                workspace=st["workspace"])
            return st["o"]
        return _orthogonalised(st["x"], st["steps"]).to(st["x"].dtype)
    if own:
        zs.zs_muon_step(st["plan"], st["tensors"], st["grads"], st["state"],
                        st["params"], grad_layout=st["layout"],
                        grad_stride=st["stride"], lr=LR, momentum=MU,
                        weight_decay=WD, nesterov=st["nesterov"],
                        scale=st["scale"], steps=st["steps"],
                        coef=(A, B, C), eps=EPS, precision=st["precision"],
                        workspace=st["workspace"])
    else:
        shapes = _shapes(st)
        list(map(lambda s, p, x: _muon_plain(st, s, p, x), shapes,
                 _places(shapes)[0], st["grads"]))
    return {"master": st["state"][:, 0], "momentum": st["state"][:, 1],
            "params": st["params"]}


# ---- 64 bits --------------------------------------------------------------------

def _polynomial(U, steps):
    """The same map through the Gram matrix: X_k = Q_k(G) X_0 with
    G = X_0 X_0^T, all in 64 bits."""
    U = U.double()
    if U.shape[-2] > U.shape[-1]:
        return _polynomial(U.transpose(-2, -1).contiguous(),
                           steps).transpose(-2, -1)
    X = U / (torch.linalg.vector_norm(U, dim=(-2, -1), keepdim=True) + EPS)
    G = torch.matmul(X, X.transpose(-2, -1).contiguous())
    eye = torch.eye(G.shape[-1], dtype=G.dtype, device=G.device)
    Q = eye.expand_as(G)
    for _ in range(steps):
        L = torch.matmul(torch.matmul(Q, G), Q)      # Q commutes with G
        Q = torch.matmul(A * eye + torch.matmul(B * eye + C * L, L), Q)
    return torch.matmul(Q, X)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "orthogonalize":
        return _polynomial(st["x"], case["steps"])
    shapes = _shapes(case)
    places, n, tiles = _places(shapes)
    state = st["state"].double()
    params = torch.zeros(n, dtype=torch.float64, device="cuda")
    for (b, r, c), (e, off, tile, t), x in zip(shapes, places, st["grads"]):
        P, M = (state[tile:tile + t, k].reshape(-1)[:e].clone()
                for k in (0, 1))
        if case["layout"] == "tiled":
            G = torch.stack([x[:, s].reshape(-1)[:e]
                             for s in range(case["world"])])
        else:
            G = x[:, :e]
        g = G.double().mean(0)
        M = M * MU + g
        U = M * MU + g if case["nesterov"] else M
        O = _polynomial(U.reshape(b, r, c), case["steps"]).reshape(-1)
        P = P - LR * (WD * P + _scale(case["scale"], r, c) * O)
        for k, v in ((0, P), (1, M)):
            row = torch.zeros(t * TILE, dtype=torch.float64, device="cuda")
            row[:e] = v
            state[tile:tile + t, k] = row.view(t, TILE)
        params[off:off + e] = P
    return {"master": state[:, 0], "momentum": state[:, 1], "params": params}
