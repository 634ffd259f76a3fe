"""embed_backward's workspace wherever a caller may have it (GPU): on every multiple of 16
bytes, as one cut from a pool lies.  Whole numbers whose sums f32 holds exactly, so the
result has to be right to the bit; nothing beside the workspace is written."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("off", [0, 16, 32, 48, 112, 240])
@pytest.mark.parametrize("n,k", [(4, 256), (301, 1024), (4099, 256), (2000, 6656)])
def test_workspace_on_any_16_bytes(off, n, k):
    import q5_lm_head_gb300 as q
    v, side = 50, 256
    gen = torch.Generator(device="cuda").manual_seed(n + off)
    tokens = torch.randint(0, 4, (n,), generator=gen, device="cuda").to(torch.int32) * 9     # long runs over many chunks
    tokens[n // 2] = -1
    grad = torch.randint(-8, 9, (n, k), generator=gen, device="cuda")
    ok = tokens >= 0
    want = torch.zeros((v, k), dtype=torch.int64, device="cuda").index_add_(0, tokens.long().clamp(min=0), grad * ok.unsqueeze(1))
    grad = grad.float()
    out = torch.empty((v, k), device="cuda")
    with q.LMHead(v, k, 1) as head:
        need = q.muse_lmhead_embed_backward_workspace(head.handle, n)
        pool = torch.full((side + off + need + side,), 77, dtype=torch.uint8, device="cuda")
        assert pool.data_ptr() % 256 == 0
        work = pool.data_ptr() + side + off
        for acc in (0, 1):
            st = q.muse_lmhead_embed_backward(head.handle, grad.data_ptr(), q.MUSE_DTYPE_F32, k, tokens.data_ptr(), n, 1.0,
                                              out.data_ptr(), q.MUSE_DTYPE_F32, k, acc, work, need, torch.cuda.current_stream().cuda_stream)
            assert st == 0
            assert torch.equal(out.to(torch.int64), want * (acc + 1))
    assert bool((pool[:side + off] == 77).all()) and bool((pool[side + off + need:] == 77).all())
