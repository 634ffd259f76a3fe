"""Block factors at the ends of what the tensor cores take, and past them.

A block with |d| or |dmin| of 4 or more makes the whole call sum in f32 from the
blocks; below, every factor goes through the operands: powers of two held at
2^-20, subnormal f16 values, scales that end subnormal, factors of 2 to 4 that are
not split.  References in 64 bits and tolerances as for the backward pass.
"""
import numpy as np
import pytest

from test_gpu_backward import _dense, _grads, _reference, _within

pytestmark = pytest.mark.gpu

BELOW = [0.0, -0.0, 6e-8, -1.2e-7, 9e-7, 1e-6, 1e-5, 0.03, 1.0, -1.0, 1.999, 2.0, -2.5, 3.998, -3.998]


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    return torch


def _blocks(rng, n, k, fmt, factors):
    size = 176 if fmt == "q5_k" else 144
    wq = rng.integers(0, 256, (n, k // 256, size), dtype=np.uint8)
    d = rng.choice(np.array(factors, dtype=np.float16), (n, k // 256, 2))
    wq[:, :, :4] = d.view(np.uint8).reshape(n, k // 256, 4)
    wq[5] = 0
    wq[6, :, 4:] = 255
    return wq


def _run(torch, wq, gl, fmt):
    import q5_lm_head_gb300 as mlh
    n, k = wq.shape[0], 256 * wq.shape[1]
    with mlh.LMHead(n, k, max_batch=gl.shape[0], device=0, fmt=fmt) as head:
        gh, _ = head.backward(torch.from_numpy(gl).cuda(), torch.from_numpy(wq.reshape(-1)).cuda(), scale=1.0, cap=0.0)
        torch.cuda.synchronize()
        assert head.device_status() == 0
    want, tol, _, _ = _reference(gl, None, None, None, _dense(wq, n, k, fmt), 1.0, 0.0)
    _within("grad_hidden", gh.cpu().numpy(), want, tol)
    return gh


@pytest.mark.parametrize("fmt", ["q5_k", "q4_k"])
@pytest.mark.parametrize("b", [1, 8, 11, 32])
@pytest.mark.parametrize("factors", [BELOW, BELOW[:6], BELOW[2:5], BELOW[10:]])
def test_factors_below_four(torch_cuda, fmt, b, factors):
    rng = np.random.default_rng(b + len(factors))
    n = 403
    wq = _blocks(rng, n, 1024, fmt, factors)
    _run(torch_cuda, wq, _grads(rng, b, n), fmt)
    _run(torch_cuda, wq, rng.standard_normal((b, n)).astype(np.float32), fmt)


@pytest.mark.parametrize("fmt", ["q5_k", "q4_k"])
@pytest.mark.parametrize("b", [1, 11, 32])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("value", [4.0, -4.0, 60000.0])
def test_one_block_of_four_and_more(torch_cuda, fmt, b, which, value):
    """Large in d or dmin, in a corner: its own column is right, and so are all others."""
    rng = np.random.default_rng(b + which)
    n, k = 301, 768
    for row, col in ((0, 0), (300, 2), (97, 1)):
        wq = _blocks(rng, n, k, fmt, BELOW)
        half = np.array([value], dtype=np.float16).view(np.uint8)
        wq[row, col, 2 * which:2 * which + 2] = half
        _run(torch_cuda, wq, _grads(rng, b, n), fmt)
