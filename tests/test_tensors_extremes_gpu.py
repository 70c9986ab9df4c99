"""The step over lists of tensors at the ends of what its hyper-parameters may
be, against oracle/tensors.py."""

import numpy as np
import pytest
import torch

import zero_sharded_optimizer_shard_amd as zs
from oracle import tensors as OT
from test_tensors_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [2.0 ** 100, 2.0 ** 124,
                                 2.0 ** 124 * (1 + 2.0 ** -23), 2.0 ** 126,
                                 1.5 * 2.0 ** 126, 2.0 ** 127,
                                 float(np.finfo(np.float32).max)])
@pytest.mark.parametrize("weights", ["master", "bf16", "f32"])
def test_eps_to_the_end_of_fp32(bits, eps, weights):
    """Moments near the largest number over an eps of their size: the update
    is of the usual size, though its denominator has no normal reciprocal."""
    def edit(h):
        if bits == 32:
            h["m"] *= np.float32(1e39 / 16)
        else:
            h["m_scale"] *= np.float32(1e39 / 16)
    c = Case([1500, 3], bits, weights, "f32", edit=edit)
    assert np.abs(c.host[0]["m"]).max() > 0
    hp = (0.5, 0.5, 0.95, eps, 0.1)
    c.step([hp], t=2)
    c.expect([hp], t=2)
    h = c.host[0]
    kept = (OT.bf16(h["param"]) if weights == "bf16" else
            h["master" if weights == "master" else "param"]) * np.float32(0.95)
    assert np.abs(h["w"] - kept).max() * eps > 1e34      # it moved
    c.check()
