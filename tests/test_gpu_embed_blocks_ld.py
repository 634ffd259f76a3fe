"""A table of blocks has no row distance: whatever muse_lmhead_embed is given as table_ld changes nothing (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ld", [-1, 1, 2 ** 62, 2 ** 63 - 1, -2 ** 63])
def test_blocks_ignore_the_distance(ld):
    import q5_lm_head_gb300 as q
    v, k, n = 40, 512, 9
    gen = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randint(0, 60, (v * (k // 256) * 176,), generator=gen, device="cuda", dtype=torch.uint8)
    tokens = torch.randint(0, v, (n,), generator=gen, device="cuda").to(torch.int32)
    out = torch.empty((n, k), device="cuda")
    with q.LMHead(v, k, 1) as head:
        want = head.embed(tokens, table)
        st = q.muse_lmhead_embed(head.handle, table.data_ptr(), q.MUSE_DTYPE_BLOCKS, ld, tokens.data_ptr(), n, 1.0, out.data_ptr(),
                                 q.MUSE_DTYPE_F32, k, torch.cuda.current_stream().cuda_stream)
        assert st == 0
    assert torch.equal(out.view(torch.int32), want.view(torch.int32))
