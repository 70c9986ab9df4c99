"""The sum of squares is a function of the gradients' values and of the list's
sizes alone: replicas that hold the same gradients at other addresses, beside
other arrays, get the same bits, and so clip and step alike."""

import numpy as np
import pytest
import torch

import zero_sharded_optimizer_shard_amd as zs
from oracle import tensors as OT
from test_tensors_gpu import normal, sumsq_of, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def at(x, shift):
    """A copy of device tensor x, `shift` elements past a 256-byte
    boundary."""
    b = torch.zeros(x.numel() + 512, dtype=x.dtype, device="cuda")
    lead = -b.data_ptr() % 256 // x.element_size() + shift
    b = b[lead:lead + x.numel()].view(x.shape)
    b.copy_(x)
    return b


def sum_of(G, sizes, kind, shift, grad_shift=None):
    """The sum over a list of tensors of `sizes` whose arrays start `shift`
    elements past a line, and the gradients `grad_shift`."""
    grad_shift = shift if grad_shift is None else grad_shift
    kw = {"grads": [at(g, grad_shift) for g in G], "world": G[0].shape[0]}
    if kind != "none":
        kw["params"] = [at(torch.zeros(n, device="cuda"), shift)
                        for n in sizes]
        if kind == "32":
            for k in ("m", "v"):
                kw[k] = [at(torch.zeros(n, device="cuda"), shift)
                         for n in sizes]
    if kw["world"] == 1:
        kw["grads"] = [g[0] for g in kw["grads"]]
    lst = zs.zs_tensors_create(**kw)
    upload(lst)
    return sumsq_of(lst).item()


# 4088 and 5120 need one piece more where they start late in one;
# the last sizes are past one workgroup
@pytest.mark.parametrize("sizes", [[1024], [1, 4088, 5120, 700],
                                   [5000, 1024 * 40, 33, 250000]])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("world", [1, 2, 4])
def test_addresses_do_not_matter(sizes, grad, world):
    rng = np.random.default_rng(world)
    G = [torch.from_numpy(normal(rng, (world, n), 1e-3)).cuda().to(grad)
         for n in sizes]
    want = sum_of(G, sizes, "none", 0)
    plain = OT.sumsq([OT.mean(g.float().cpu().numpy()) for g in G])
    # exact squares to 2^-53, n sums of positive numbers on either side
    assert abs(want - plain) <= 2 * (sum(sizes) + 1) * 2.0 ** -53 * plain
    for kind in ("none", "params", "32"):
        for shift, other in ((0, None), (4, None), (8, None), (37, None),
                             (1, None), (63, None), (37, 0), (2, 5)):
            got = sum_of(G, sizes, kind, shift, other)
            assert got == want, (kind, shift, other)
