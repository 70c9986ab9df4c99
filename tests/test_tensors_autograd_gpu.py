"""A list's step as a torch training loop has it: autograd adds into the list's
gradient buffers, and the list steps the parameters in place."""

import numpy as np
import pytest
import torch

import zero_sharded_optimizer_shard_amd as zs
from oracle import tensors as OT
from test_tensors_gpu import HP, same, sumsq_of, upload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_in_kept_buffers(dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gen = torch.Generator(device="cuda").manual_seed(1)
    params = [torch.nn.Parameter((0.1 * torch.randn(
        s, generator=gen, device="cuda")).to(dtype))
        for s in ((33, 70), (33,), (5, 33), (1,))]
    for p in params:
        p.grad = torch.zeros_like(p)
    m = [torch.zeros(p.numel(), device="cuda") for p in params]
    v = [torch.zeros(p.numel(), device="cuda") for p in params]
    lst = zs.zs_tensors_create(params=params, grads=[p.grad for p in params],
                               m=m, v=v)
    upload(lst)
    host = [[x.detach().float().cpu().numpy().reshape(-1).copy()
             for x in (p, a, b)] for p, a, b in zip(params, m, v)]
    at = [p.grad.data_ptr() for p in params]
    for t in (1, 2, 3):
        x = torch.randn(16, 70, generator=gen, device="cuda").to(dtype)
        w, b, u, c = params
        y = torch.tanh(x @ w.t() + b) @ u.t() + c
        y.float().square().mean().backward()
        g = [p.grad.detach().float().cpu().numpy().reshape(-1).copy()
             for p in params]
        assert all(x.any() for x in g)
        s = sumsq_of(lst)
        zs.zs_tensors_step(lst, zs.zs_adamw(*HP), step=t, sumsq=s,
                           max_norm=0.01)
        coef = OT.coefficient(s.item(), 0.01)
        for h, G, p, a, b in zip(host, g, params, m, v):
            h[1], h[2], root = OT.moments(G * coef, h[1], h[2], HP, t)
            h[0] = OT.weights(h[0], h[1], root, HP, t)
            if dtype == torch.bfloat16:
                h[0] = OT.bf16(OT.to_bf16(h[0]))
            same(p.detach().float().reshape(-1), h[0])
            same(a, h[1])
            same(b, h[2])
        for p, k in zip(params, at):
            p.grad.zero_()       # zero_grad(set_to_none=False)
            assert p.grad.data_ptr() == k
