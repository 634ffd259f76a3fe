"""Entropies of rows that are nearly sure of a few values, which come late in the row.

H = ln 2 (log2 S - U / S) with U = sum 2^a a of exponents a against a reference that
lies at most 16 (in log2's units) below the thread's maximum.  u = 2^-24: a peak's
exponent is at most 16, its product with 2^a is off by 16u, so is the sum that the
move onto the row's maximum takes off again; 2^a and the move's factor are off by
4u each, as the logarithm sees 6u; joins of warps and CTAs move once more each,
with exponents of 0 for the peaks: 12u each.  In all 68u of an entropy in
log2's units, 48u of one in natural ones, and 4u of its value; the other values,
30 below, add less than 1u.
"""
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    return torch


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("n,v", [(1, 202048), (16, 202048), (77, 50257), (200, 50257), (400, 20011)])
@pytest.mark.parametrize("peaks", [1, 2, 5])
@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_entropy_of_peaked_rows(torch_cuda, dtype, n, v, peaks, temperature):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    temperature = float(torch.tensor(temperature))
    g = torch.Generator(device="cuda").manual_seed(n + v + peaks)
    x = torch.randn((n, v), generator=g, device="cuda").clamp(-2, 2).to(getattr(torch, dtype))
    at = v // 3 + torch.randint(0, v // 8, (n, peaks), generator=g, device="cuda") + torch.arange(peaks, device="cuda") * (v // 8)
    height = 32 + 8 * torch.rand((n, 1), generator=g, device="cuda")
    near = torch.rand((n, peaks), generator=g, device="cuda") * (peaks > 1)
    x.scatter_(1, at, (height + near).to(x.dtype))
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        got = head.score(x, temperature=temperature).entropy.double()
        torch.cuda.synchronize()
    q = torch.log_softmax(x.double() / temperature, dim=1)
    want = -(q.exp() * q).sum(dim=1)
    assert bool((got >= 0).all()), f"{float(got.min()):.3g}"
    err = (got - want).abs()
    assert bool((err <= 48 * U + 4 * U * want).all()), f"off by {float(err.max()):.3g}"
