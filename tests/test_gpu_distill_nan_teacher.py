"""A teacher whose row was not a number: score gives NaN log probabilities there, and a
distillation from them has no loss, rather than one of 0.  Other rows are not touched."""
import math

import pytest

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


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("v", [300, 50257, 2000003])
def test_distill_from_a_teacher_that_is_not_a_number(torch_cuda, dtype, tail, v):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    g = torch.Generator(device="cuda").manual_seed(v)
    x = torch.randn((5, v), generator=g, device="cuda").to(getattr(torch, dtype))
    teacher = torch.randn((5, v), generator=g, device="cuda")
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        clean = head.score(teacher, n_top=6)
        bad = teacher.clone()
        bad[1, v // 2] = math.nan
        scores = head.score(bad, n_top=6)
        lp, ids = scores.top_logprobs.clone(), clean.top_ids.clone()
        assert bool(lp[1].isnan().all()) and bool(lp[[0, 2, 3, 4]].isfinite().all())
        lp[2, 3] = math.nan                     # one entry alone
        lp[3, 2], ids[3, 2] = math.nan, -1      # one that is left out
        w = torch.tensor([1.0, 1.0, 1.0, 1.0, 0.0], device="cuda")
        lp[4] = math.nan                        # a row of weight 0
        loss, grad = head.distill(x, ids, lp, w, tail=tail)
        alone, _ = head.distill(x, ids, lp, w, tail=tail, want_grad=False)
        want, wgrad = head.distill(x, clean.top_ids, clean.top_logprobs, w, tail=tail)
        torch.cuda.synchronize()
    assert bool(loss[[1, 2]].isnan().all()) and bool(grad[[1, 2]].isnan().any(dim=1).all())
    assert float(loss[0]) == float(want[0]) and torch.equal(grad[0], wgrad[0])
    assert bool(loss[3].isfinite()) and bool(grad[3].isfinite().all()) and float(loss[4]) == 0 and not bool(grad[4].any())
    assert torch.equal(alone.nan_to_num(nan=7.0), loss.nan_to_num(nan=7.0))
