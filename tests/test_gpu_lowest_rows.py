"""Rows in which nothing but masks of the type's lowest value is left: a softmax is
uniform over them, and its logarithms are differences of values of 3.4e38 in size,
which have to be taken before the normaliser is added.

Tolerance (u = 2^-24): all addends of a sum are 1, so the sum is exact up to 2^24
of them, its logarithm and the result are off by 4u of their size, and
what the teacher's entries add by 45u (1 + the largest logarithm).
"""
import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = ("float32", "float16", "bfloat16")


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    return torch


def _row(torch, v, dtype, masked, left):
    """`left` values of the type's lowest, the rest -infinity (or all of the lowest)."""
    x = torch.full((1, v), -math.inf)
    x[0, torch.randperm(v, generator=torch.Generator().manual_seed(v))[:left if masked else v]] = torch.finfo(getattr(torch, dtype)).min
    return x.to(getattr(torch, dtype)).cuda(), left if masked else v


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("temperature", [1.0, 0.5, 3.0])
@pytest.mark.parametrize("v", [70, 50257, 2000003])
def test_distill_rows_of_the_lowest_value(torch_cuda, dtype, masked, tail, temperature, v):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    x, left = _row(torch, v, dtype, masked, 40)
    ids = (x[0] > -math.inf).nonzero()[:, 0][torch.tensor([1, 5, 30], device="cuda")].to(torch.int32)[None]
    p = [0.4, 0.3, 0.1] if tail else [0.5, 0.375, 0.125]
    lp = torch.tensor([p], device="cuda").log()
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        loss, grad = head.distill(x, ids, lp, None, temperature, tail)
        torch.cuda.synchronize()
    want = sum(q * (math.log(q) + math.log(left)) for q in p)
    if tail:
        want += 0.2 * (math.log(0.2) - math.log((left - 3) / left))
    assert abs(float(loss[0]) - want) <= 45 * U * (1 + math.log(v)) + 200 * U
    assert bool(grad.isfinite().all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("temperature", [1.0, 0.5, 3.0])
@pytest.mark.parametrize("v", [70, 50257, 202048])
def test_score_rows_of_the_lowest_value(torch_cuda, dtype, masked, temperature, v):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    x, left = _row(torch, v, dtype, masked, 40)
    at = (x[0] > -math.inf).nonzero()[:, 0].to(torch.int32)
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        out = head.score(x, at[7:8], 8, temperature)
        torch.cuda.synchronize()
    tol = 4 * U * math.log(left) + 2 * U
    assert abs(float(out.logprob[0]) + math.log(left)) <= tol
    assert abs(float(out.entropy[0]) - math.log(left)) <= tol
    assert float((out.top_logprobs + math.log(left)).abs().max()) <= tol
    assert torch.equal(out.top_ids[0], at[:8]) and int(out.rank[0]) == 7
