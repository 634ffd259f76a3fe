"""muse_lmhead_sample with more rows than the SMs take at once, whose last rows run in a grid of their own (GPU).

A row's token and log probability depend on nothing but the row, so rows that are
given in pieces small enough for one grid have to get the same bits.  The pieces
themselves are checked against 64 bits in the other tests of this operator."""
import pytest
import torch

pytestmark = pytest.mark.gpu

V = 33001


@pytest.fixture(scope="module")
def head():
    import q5_lm_head_gb300 as q
    with q.LMHead(V, 256, 1) as h:
        yield h


def settings(n, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pick = torch.randint(0, 5, (n,), generator=gen, device="cuda")
    one = torch.ones(n, device="cuda")
    return dict(temperature=torch.where(pick == 4, 0.0 * one, 0.5 + torch.rand(n, generator=gen, device="cuda")),
                top_k=torch.where(pick == 1, 50, 0).to(torch.int32), top_p=torch.where(pick == 2, 0.9 * one, one),
                min_p=torch.where(pick == 3, 0.05 * one, 0.0 * one))


def part(how, a, b):
    return {k: s[a:b].contiguous() if isinstance(s, torch.Tensor) else s for k, s in how.items()}


def in_pieces(head, x, u, how, size=100):
    got = [head.sample(x[a:a + size], u[a:a + size].contiguous(), **part(how, a, min(a + size, x.shape[0])))
           for a in range(0, x.shape[0], size)]
    return torch.cat([t for t, _ in got]), torch.cat([p for _, p in got])


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n", [300, 303, 304, 305, 306, 330, 456, 457, 607, 608, 609, 700, 1216, 1217, 1300, 1600])
def test_rows_in_two_grids(head, n, dtype):
    """Counts on both sides of whole fillings of the SMs; every row with settings of its own, one row masked."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    x = (torch.randn(n, V, generator=gen, device="cuda") * 2.5).to(dtype)
    x[n - 1, :] = float("-inf")
    x[n // 2, 7] = float("nan")
    u = torch.rand(n, generator=gen, device="cuda")
    how = settings(n, n)
    tokens, logprobs = head.sample(x, u, **how)
    want, want_p = in_pieces(head, x, u, how)
    assert torch.equal(tokens, want)
    assert torch.equal(logprobs.view(torch.int32), want_p.view(torch.int32))
    assert int(tokens[n - 1]) == -1 and int(tokens[n // 2]) == -1


def test_padded_rows_and_no_logprobs(head):
    """Rows at a distance and at no alignment; the entry point without logprobs; rows behind the last one as they were."""
    import q5_lm_head_gb300 as q
    n = 400
    wide = torch.full((n + 3, V + 5), float("nan"), device="cuda", dtype=torch.bfloat16)
    x = wide[:n, 3:3 + V]
    x.copy_(torch.randn(n, V, device="cuda") * 2)
    u = torch.rand(n, device="cuda")
    tokens = torch.full((n + 2,), 77, device="cuda", dtype=torch.int32)
    how = q.MuseSampling(1.0, 0, 0.9, 0.0)
    st = q.muse_lmhead_sample(head.handle, x.data_ptr(), q.MUSE_DTYPE_BF16, n, V + 5, how, u.data_ptr(), tokens.data_ptr(), None,
                              torch.cuda.current_stream().cuda_stream)
    assert st == 0
    want, _ = in_pieces(head, x, u, dict(top_p=0.9))
    assert torch.equal(tokens[:n], want) and tokens[n:].tolist() == [77, 77]


@pytest.mark.parametrize("captured", [False, True])
def test_what_comes_before_and_after(head, captured):
    """Logits written right before the call and over right after it, tokens looked up right after it, again and again."""
    n = 420
    gen = torch.Generator(device="cuda").manual_seed(5)
    xs = [torch.randn(n, V, generator=gen, device="cuda") * 2.5 for _ in range(3)]
    us = [torch.rand(n, generator=gen, device="cuda") for _ in range(3)]
    table = torch.randn(V, 256, generator=gen, device="cuda")
    want = [in_pieces(head, x, u, dict(top_p=0.9)) for x, u in zip(xs, us)]
    x, u = torch.empty_like(xs[0]), torch.empty_like(us[0])

    def step():
        outs = []
        for i in range(6):
            x.copy_(xs[i % 3])
            u.copy_(us[i % 3])
            tokens, logprobs = head.sample(x, u, top_p=0.9)
            outs.append((tokens, logprobs, head.embed(tokens, table)))
        x.zero_()
        return outs

    if captured:
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        for _ in range(3):
            for o in outs:
                for t in o:
                    t.zero_()
            graph.replay()
            torch.cuda.synchronize()
    else:
        outs = step()
    for i, (tokens, logprobs, rows) in enumerate(outs):
        assert torch.equal(tokens, want[i % 3][0]) and torch.equal(logprobs, want[i % 3][1])
        assert torch.equal(rows, table[tokens.long()])


def test_two_calls_at_once(head):
    """Two streams with calls of two grids each."""
    n = 350
    streams = [torch.cuda.Stream() for _ in range(2)]
    x = [torch.randn(n, V, device="cuda") * 2.5 for _ in range(2)]
    u = [torch.rand(n, device="cuda") for _ in range(2)]
    want = [in_pieces(head, x[i], u[i], dict(top_p=0.95, min_p=0.01)) for i in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for i, s in enumerate(streams):
            got.append((i, head.sample(x[i], u[i], top_p=0.95, min_p=0.01, stream=s)))
    torch.cuda.synchronize()
    for i, (tokens, logprobs) in got:
        assert torch.equal(tokens, want[i][0]) and torch.equal(logprobs, want[i][1])
