"""Runs of one token that end and begin on the borders where the joining of their parts
changes (GPU): chunks that make up a group, parts from which groups are joined first, a
run's first and last chunk at a group's ends.  The lengths follow from the chunk in use,
restated here.  Whole numbers whose sums f32 holds exactly: right to the bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

GROUP, MANY = 32, 64            # chunks of a group; parts behind the first from which groups are joined
LEAST, MOST = 3, 128            # positions of a chunk
SPANS = (1, 2, 31, 32, 33, 62, 63, 64, 65, 66, 95, 96, 97, 127, 128, 129)


def chunk_of(n, tiles, sms):
    return min(max(-(-n * tiles // (24 * sms)), LEAST), MOST)


def positions_for(chunk, tiles, sms):
    """As many as have chunks of that size."""
    n = chunk * 24 * sms // tiles
    assert chunk_of(n, tiles, sms) == chunk
    return n


@pytest.mark.parametrize("start", [0, 1, 2, 30, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("chunk,k", [(3, 256), (4, 256), (7, 512), (3, 6656), (5, 6656)])
def test_run_over_borders(chunk, k, start):
    """One run from chunk `start` on over each span, from the first and the last position of its first chunk to those of its last."""
    import q5_lm_head_gb300 as q
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # narrow matrices have room for every span in one chunk size; of wide ones, whose chunks are few, the spans that fit
    n = positions_for(chunk, k // 256, sms)
    v = 9
    gen = torch.Generator(device="cuda").manual_seed(start)
    grad = torch.randint(-8, 9, (n, k), generator=gen, device="cuda")
    shuffle = torch.randperm(n, generator=gen, device="cuda")
    seen, wrong = [], []
    with q.LMHead(v, k, 1) as head:
        out = torch.empty((v, k), device="cuda")
        values = grad.float()
        for span in SPANS:
            for head_at in {0, chunk - 1}:
                for tail_at in {0, chunk - 1}:
                    first, end = start * chunk + head_at, (start + span) * chunk + tail_at + 1
                    if end > n:
                        continue
                    assert first // chunk == start and (end - 1) // chunk - first // chunk == span
                    tokens = torch.full((n,), 8, dtype=torch.int32, device="cuda")      # the rest lies behind, of one token too
                    tokens[:first] = 1
                    tokens[first:end] = 4
                    at = torch.empty_like(tokens)
                    at[shuffle] = tokens
                    want = torch.zeros((v, k), dtype=torch.int64, device="cuda").index_add_(0, at.long(), grad)
                    head.embed_backward(values, at, grad_table=out)
                    wrong.append((out.to(torch.int64) != want).any())
                    seen.append(span)
    assert not bool(torch.stack(wrong).any())
    room = n // chunk - start - 1
    assert set(seen) == {s for s in SPANS if s <= room}
    if k <= 512:
        assert set(seen) == set(SPANS)
    else:
        assert {63, 64, 65} <= set(seen)


@pytest.mark.parametrize("chunk", [3, 4])
def test_runs_share_their_chunks_and_counters(chunk):
    """Long runs one after another: each ends in the chunk where the next begins, at every distance to a group's border."""
    import q5_lm_head_gb300 as q
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n, k = positions_for(chunk, 1, sms), 256
    gen = torch.Generator(device="cuda").manual_seed(chunk)
    grad = torch.randint(-8, 9, (n, k), generator=gen, device="cuda")
    values, wrong = grad.float(), []
    for each in (chunk + 1, 32 * chunk - 1, 32 * chunk + 1, 64 * chunk - 1, 64 * chunk + 1, 65 * chunk + 1, 97 * chunk + 2, 128 * chunk + 1):
        v = -(-n // each)
        tokens = torch.arange(n, device="cuda") // each
        at = torch.empty_like(tokens)
        at[torch.randperm(n, generator=gen, device="cuda")] = tokens
        want = torch.zeros((v, k), dtype=torch.int64, device="cuda").index_add_(0, at, grad)
        with q.LMHead(v, k, 1) as head:
            got = head.embed_backward(values, at.to(torch.int32))
        wrong.append((got.to(torch.int64) != want).any())
    assert not bool(torch.stack(wrong).any())
