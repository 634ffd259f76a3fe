"""A renormalised teacher is the same for any shift of its values: teacher logits, at low
teacher temperatures hundreds or thousands in size, serve as well as logarithms.
The entries here are multiples of 1/64 and the shifts whole numbers, so shifted
entries are exact and the results have to be the same bits."""
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


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("v,top", [(300, 5), (50257, 64), (2000003, 20)])
def test_a_teachers_shift(torch_cuda, dtype, v, top):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    g = torch.Generator(device="cuda").manual_seed(v)
    x = (torch.randn((3, v), generator=g, device="cuda") * 3).to(getattr(torch, dtype))
    ids = torch.rand((3, v), generator=g, device="cuda").topk(top, dim=1).indices.to(torch.int32)
    entries = (torch.randn((3, top), generator=g, device="cuda") * 3 * 64).round() / 64
    entries[1, 2] = -float("inf")
    p = torch.softmax(entries.double(), dim=1)
    logq = torch.log_softmax(x.double(), dim=1).gather(1, ids.long())
    logp = torch.log_softmax(entries.double(), dim=1)
    want = torch.where(p > 0, p * (logp - logq), torch.zeros_like(p)).sum(dim=1)
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        loss, grad = (t.clone() for t in head.distill(x, ids, entries))
        for shift in (-20.0, 28.0, 400.0, -5000.0, 100000.0):
            moved = entries + shift
            assert torch.equal((moved - shift).nan_to_num(neginf=-1e9), entries.nan_to_num(neginf=-1e9))
            got = head.distill(x, ids, moved)
            assert torch.equal(got[0], loss) and torch.equal(got[1], grad), shift
    tol = (v / 256 + 80 + 200) * 2.0 ** -24 * 2 + 45 * 2.0 ** -24 * 30      # as for the losses, logarithms below 30
    assert bool(((loss.double() - want).abs() <= tol).all())
