"""Runs of one token that many warps of all SMs hold parts of, joined by whichever comes
last, over and over (GPU): no warp may add up a part before it is there.  Whole numbers
whose sums f32 holds exactly, other ones in every call, in one workspace that still
holds the parts of the call before."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,k,ids", [(301, 256, 3), (3600, 256, 1), (3600, 256, 40), (16384, 1024, 2), (5000, 6656, 5)])
def test_parts_are_there_when_they_are_added(n, k, ids):
    import q5_lm_head_gb300 as q
    gen = torch.Generator(device="cuda").manual_seed(n)
    v, calls = 64, 100
    out, sums = torch.empty((v, k), device="cuda"), []
    with q.LMHead(v, k, 1) as head:
        need = q.muse_lmhead_embed_backward_workspace(head.handle, n)
        work = torch.empty((need,), dtype=torch.uint8, device="cuda")
        tokens = torch.randint(0, ids, (n,), generator=gen, device="cuda").to(torch.int32)
        base = torch.randint(-8, 9, (n, k), generator=gen, device="cuda").float()
        want = torch.zeros((v, k), device="cuda").index_add_(0, tokens.long(), base)
        assert float(want.abs().max()) * calls < 2 ** 24
        grads = [base * float(i) for i in range(8)]
        for i in range(calls):
            st = q.muse_lmhead_embed_backward(head.handle, grads[i % 8].data_ptr(), q.MUSE_DTYPE_F32, k, tokens.data_ptr(), n, 1.0,
                                              out.data_ptr(), q.MUSE_DTYPE_F32, k, 0, work.data_ptr(), need,
                                              torch.cuda.current_stream().cuda_stream)
            assert st == 0
            sums.append((out != want * float(i % 8)).sum())
    assert int(torch.stack(sums).sum()) == 0
