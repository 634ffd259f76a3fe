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


@pytest.mark.parametrize("fmt", ["q5_k", "q4_k"])
@pytest.mark.parametrize("b", [1, 12, 20])
@pytest.mark.parametrize("scale", [0.196116, -1.9990234375])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_backward_of_gradients_times_powers_of_two(torch_cuda, fmt, b, scale, cap):
    """A power of two goes through every rounding: the same bits at the other end, up to f32's largest
    values and down to where a gradient's last bits would leave its normal range."""
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    n, k = 640, 512
    gen = torch.Generator(device="cuda").manual_seed(b)
    w = torch.from_numpy(np.ascontiguousarray(_weights(n, k, fmt, 62))).cuda()
    g = (torch.rand((b, n), generator=gen, device="cuda") + 1) * 0.5
    g *= torch.where(torch.rand((b, n), generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    logits = torch.rand((b, n), generator=gen, device="cuda") * 20 - 10
    with mlh.LMHead(n, k, max_batch=b, device=0, fmt=fmt) as head:
        want = head.backward(g, w, logits=logits, scale=scale, cap=cap)[0].clone()
        assert bool(want.isfinite().all()) and float(want.abs().max()) < 2 ** 8
        for power in (-113, -60, 60, 114, 116, 118, 120):         # 2^8 2^120 is still f32's
            got = head.backward(g * 2.0 ** power, w, logits=logits, scale=scale, cap=cap)[0]
            torch.cuda.synchronize()
            back = got.double() * 2.0 ** -power
            tiny = 2.0 ** -149 * 2.0 ** -power if power < 0 else 0.0      # results below the normal range are rounded once more
            assert bool(((back - want.double()).abs() <= tiny).all()), power
        # the largest gradients there are, on weights that keep their sums in range
        big = g * 2.0 ** 127 * 1.99
        assert bool(big.isfinite().all())
        small = w.view(n, -1, 176 if fmt == "q5_k" else 144).clone()
        small[:, :, :4] = torch.tensor([[[2.0 ** -20, 2.0 ** -20]]], dtype=torch.float16, device="cuda").view(torch.uint8)
        got = head.backward(big, small.view(-1), logits=logits, scale=scale, cap=cap)[0]
        base = head.backward(big * 2.0 ** -100, small.view(-1), logits=logits, scale=scale, cap=cap)[0]
        assert bool(got.isfinite().all()) and torch.equal(got, base * 2.0 ** 100)
