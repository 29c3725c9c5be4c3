"""What the training step's calls promise besides their formulas: small second
moments, what autograd is told, which tensors an optimizer takes and keeps, and
what it refuses. Sizes are small; the formulas' own tests are in
test_gpu_adamw.py, test_gpu_residual_norm.py and test_gpu_embedding.py."""
import copy
import pickle

import numpy as np
import pytest

import nf4_quantize_amd as nq
from gpu_util import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


# ------------------------------------------------------------------ small moments

@pytest.mark.parametrize("eps", [0.0, 1e-24, 1e-8])
def test_root_of_small_second_moments(dev, eps):
    """Second moments among fp32's subnormals (below 2^-126) and around them: the
    step is lr m / (sqrt(v) + eps), not lr m / eps. The moments before the step are
    given, the gradient is zero, so v' = beta2 v up to one rounding: U of itself and
    2^-149, that is 2^-150 / v of the root; the bias corrections at step 100000
    are 1 in fp32 for the first and 1 - 3.5e-44 for the second. Then 24 U as in the
    other tests of the step, and 2 U of the weight."""
    import torch

    n = 300
    exps = np.linspace(-143, -110, n)
    v0 = np.exp2(exps).astype(np.float32)
    v1 = v0.astype(np.float64) * 0.999
    m0 = (np.sqrt(v0.astype(np.float64)) * np.where(np.arange(n) % 2, 1.0, -0.5)).astype(np.float32)
    p = torch.full((n,), 0.25, device=dev)
    opt = nq.NF4AdamW([p], lr=1e-2, weight_decay=0.0, eps=eps, state_bits=32)
    opt.bind_state([torch.from_numpy(m0).to(dev)], [torch.from_numpy(v0).to(dev)])
    opt.step([torch.zeros(n, device=dev)], step=100000)
    step = 1e-2 * 0.9 * m0.astype(np.float64) / (np.sqrt(v1) + float(np.float32(eps)))
    tol = 2 * U * 0.26 + np.abs(step) * (24 * U + 2.0 ** -149 / v1)
    got = p.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - (0.25 - step)) <= tol), float(np.max(np.abs(got - (0.25 - step)) / tol))
