"""The powers of two that bring a row's t into the tensor cores' operands: taken from
t behind the cap's slope, for gradients of every size.  References in 64 bits and
tolerances as for the backward pass.
"""
import numpy as np
import pytest

from test_gpu_backward import _dense, _reference, _weights, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    return torch


@pytest.mark.parametrize("fmt", ["q5_k", "q4_k"])
@pytest.mark.parametrize("b", [1, 12, 20])
@pytest.mark.parametrize("saturated", [20.0, 20.0 * (1 - 2.0 ** -22)])
def test_backward_beside_saturated_logits(torch_cuda, fmt, b, saturated):
    """The row's largest gradients meet a cap whose slope is 0 or nearly so: what is left is 2^-26 of them."""
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    n, k = 600, 512
    rng = np.random.default_rng(b)
    wq = _weights(n, k, fmt, 61)
    logits = rng.uniform(-8, 8, (b, n)).astype(np.float32)
    gl = (rng.standard_normal((b, n)) * 2.0 ** -26).astype(np.float32)
    for r in range(b):
        at = rng.choice(n, 3, replace=False)
        logits[r, at] = np.float32(saturated) * rng.choice([-1, 1], 3)
        gl[r, at] = [1.0, -0.7, 3.0]
    with mlh.LMHead(n, k, max_batch=b, device=0, fmt=fmt) as head:
        gh, _ = head.backward(torch.from_numpy(gl).cuda(), torch.from_numpy(wq).cuda(), logits=torch.from_numpy(logits).cuda(), scale=1.0)
        torch.cuda.synchronize()
    want, tol, _, _ = _reference(gl, logits, None, None, _dense(wq, n, k, fmt), 1.0, 20.0)
    _within("grad_hidden", gh.cpu().numpy(), want, tol)
