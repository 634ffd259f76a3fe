"""Gradient by a token table where one token stands at very many positions (GPU).

The sorted positions are summed in chunks, a long run's chunks in groups.  The
gradients here are small whole numbers whose sums f32 holds exactly, so every sum,
whichever way it is split, has to be right to the bit; the runs begin and end on
both sides of a chunk's and a group's borders."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def check(lengths, v, k, seed):
    """Runs of these lengths for tokens 0, 2, 4 .. at shuffled positions, against sums in 64-bit integers."""
    import q5_lm_head_gb300 as q
    gen = torch.Generator(device="cuda").manual_seed(seed)
    tokens = torch.repeat_interleave(torch.arange(len(lengths), device="cuda") * 2, torch.tensor(lengths, device="cuda"))
    assert int(tokens.max()) < v
    n = tokens.numel()
    tokens = tokens[torch.randperm(n, generator=gen, device="cuda")].to(torch.int32)
    grad = torch.randint(-8, 9, (n, k), generator=gen, device="cuda")
    want = torch.zeros((v, k), dtype=torch.int64, device="cuda").index_add_(0, tokens.long(), grad)
    assert int(want.abs().max()) < 2 ** 24
    with q.LMHead(v, k, 1) as head:
        got = head.embed_backward(grad.to(torch.float32), tokens, scale=2.0)
        assert torch.equal(got.to(torch.int64), 2 * want) and torch.equal(got, got.round())
        again = head.embed_backward(grad.to(torch.bfloat16), tokens, scale=4.0, grad_table=got, accumulate=True)
        assert torch.equal(again.to(torch.int64), 6 * want)


@pytest.mark.parametrize("chunks", [31, 32, 33, 63, 64, 65, 66, 95, 96, 97, 128, 129])
@pytest.mark.parametrize("before", [0, 1, 4, 8, 30 * 8, 31 * 8 - 1, 31 * 8, 31 * 8 + 1, 32 * 8])
def test_one_long_run(chunks, before):
    """Runs that span about `chunks` chunks of 4 or 8 positions, behind a shorter one and before another."""
    for each in (4, 8):
        first = before * each // 8
        for more in (-1, 0, 1):
            length = chunks * each + more
            rest = 40 if each == 4 else 4100 - length - first     # 4,100 positions have chunks of eight
            check([first, length, max(rest, 5)], 9, 256, chunks)


@pytest.mark.parametrize("lengths", [
    [16384], [1] + [16383], [16383, 1], [8192, 8192], [8200, 8184], [1024] * 16, [1040] * 15 + [784],
    [511, 513, 1023, 1025, 2047, 2049, 4095, 4097, 1024], [3] * 100 + [9000] + [1] * 700 + [6000],
])
@pytest.mark.parametrize("k", [256, 6656])
def test_long_runs_side_by_side(lengths, k):
    """Several long runs that end and begin in one chunk, up to all positions of one token."""
    check(lengths, 2 * len(lengths) + 3, k, len(lengths))


def test_padded_batch_of_one_token():
    """65,536 positions, most of them of one token, others padded."""
    check([60000, 5, 5531], 64, 512, 3)


@pytest.mark.parametrize("k", [256, 1024, 6656])
def test_workspace_serves_fewer_positions(k):
    """The workspace of n positions is no smaller than that of fewer, and a call with fewer runs in it."""
    import q5_lm_head_gb300 as q
    v, most = 40, 5000
    with q.LMHead(v, k, 1) as head:
        bytes_of = [q.muse_lmhead_embed_backward_workspace(head.handle, n) for n in range(0, 40000, 7)]
        assert bytes_of == sorted(bytes_of)
        large = [q.muse_lmhead_embed_backward_workspace(head.handle, n) for n in range(10 ** 6, 2 * 10 ** 9, 10 ** 7)]
        assert large == sorted(large) and bytes_of[-1] <= large[0]
        work = torch.empty((q.muse_lmhead_embed_backward_workspace(head.handle, most),), dtype=torch.uint8, device="cuda")
        out = torch.empty((v, k), device="cuda")
        for n in (most, 4999, 3700, 1001, 37, 3, 1, 0):
            tokens = (torch.arange(n, device="cuda") % 2 * 7).to(torch.int32)
            grad = torch.randint(-8, 9, (n, k), device="cuda")
            want = torch.zeros((v, k), dtype=torch.int64, device="cuda").index_add_(0, tokens.long(), grad)
            grad = grad.to(torch.float32)
            st = q.muse_lmhead_embed_backward(head.handle, grad.data_ptr(), q.MUSE_DTYPE_F32, k, tokens.data_ptr(), n, 1.0,
                                              out.data_ptr(), q.MUSE_DTYPE_F32, k, 0, work.data_ptr(), work.numel(),
                                              torch.cuda.current_stream().cuda_stream)
            assert st == 0
            assert torch.equal(out.to(torch.int64), want)
