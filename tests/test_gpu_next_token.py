"""The operators around the next token as they are used together: a decode loop
(forward, draw, look up) eager and captured, and a training step through lookup,
head, distillation and back into the table."""
import numpy as np
import pytest

import q5k_synth as synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    wl = synth.WORKLOADS["tiny"]
    hidden, gamma, wq = synth.inputs_for(wl)
    dev = lambda t: torch.from_numpy(np.ascontiguousarray(t)).cuda()                      # noqa: E731
    return torch, mlh, wl, dev(hidden), dev(gamma), dev(wq)


@pytest.mark.parametrize("batch", [1, 4])
def test_forward_sample_is_forward_then_sample(env, batch):
    torch, mlh, wl, hidden, gamma, w = env
    h = torch.cat([hidden * s for s in (1.0, 0.5, -1.0, 2.0)])[:batch].contiguous()
    u = torch.rand((batch,), device="cuda")
    t = torch.tensor([0.7, 0.0, 1.0, 1.5], device="cuda")[:batch].contiguous()
    with mlh.LMHead(wl.n_rows, wl.k, max_batch=4, device=0) as head:
        logits, argmax = head.forward(h, w, gamma)
        for settings in (dict(), dict(temperature=0.0), dict(temperature=t, top_k=20, top_p=0.9, min_p=0.01)):
            want = head.sample(logits, u, **settings)
            got = head.forward_sample(h, w, u, gamma, **settings)
            assert torch.equal(got[0], logits) and torch.equal(got[1], want[0]) and torch.equal(got[2], want[1])
        assert torch.equal(head.forward_sample(h, w, u, gamma, temperature=0.0)[1], argmax)
        # the log probability is that of the whole distribution where nothing is filtered
        tokens, logprobs = head.sample(logits, u)
        assert bool(((logprobs - head.score(logits, tokens).logprob).abs() <= 1e-4).all())


def test_decode_loop(env):
    """Each step's token, looked up in the head's own matrix, is the next step's input; the
    captured loop gives the eager one's tokens."""
    torch, mlh, wl, hidden, gamma, w = env
    steps, n = 6, 3
    u = torch.rand((steps, n), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    with mlh.LMHead(wl.n_rows, wl.k, max_batch=n, device=0) as head:
        first = torch.arange(n, dtype=torch.int32, device="cuda") * 100

        def run():
            tokens, out = first, []
            for s in range(steps):
                x = head.embed(tokens, w, scale=wl.k ** 0.5)
                _, tokens, _ = head.forward_sample(x, w, u[s], gamma, temperature=0.9, top_k=100, top_p=0.95)
                out.append(tokens)
            return torch.stack(out)

        want = run()
        torch.cuda.synchronize()
        assert bool(((want >= 0) & (want < wl.n_rows)).all())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        for _ in range(3):
            got.fill_(-9)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want)
        first.add_(1)
        again = run()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, again)
        assert head.device_status() == 0


def test_training_step(env):
    """Table -> head -> distillation -> head's gradient -> table's gradient, against the same chain whose
    last step is done in 64 bits from the same gradient by the rows."""
    torch, mlh, wl, hidden, gamma, w = env
    n = 24
    gen = torch.Generator(device="cuda").manual_seed(8)
    table = torch.randn((wl.n_rows, wl.k), generator=gen, device="cuda").to(torch.bfloat16)
    tokens = torch.randint(-1, 9, (n,), generator=gen, device="cuda", dtype=torch.int32)
    with mlh.LMHead(wl.n_rows, wl.k, max_batch=32, device=0) as head:
        x = head.embed(tokens, table, dtype=torch.float32)
        logits = head.forward(x, w, gamma, want_argmax=False)
        teacher = head.score(torch.roll(logits, 1, 0), n_top=16)
        weight = (tokens >= 0).float() / n
        _, grad = head.distill(logits, teacher.top_ids, teacher.top_logprobs, row_weight=weight, tail=True)
        by_x, _ = head.backward(grad, w, logits=logits, hidden=x, gamma=gamma)
        got = head.embed_backward(by_x, tokens, dtype=torch.float32)
        more = head.embed_backward(by_x, tokens, grad_table=got.clone(), accumulate=True)
    want, size = (torch.zeros((wl.n_rows, wl.k), dtype=torch.float64, device="cuda") for _ in range(2))
    ok = tokens >= 0
    want.index_add_(0, tokens[ok].long(), by_x[ok].double())
    size.index_add_(0, tokens[ok].long(), by_x[ok].double().abs())
    assert bool(((got.double() - want).abs() <= n * U * size).all()) and float(want.abs().max()) > 0
    assert bool(((more.double() - 2 * want).abs() <= (2 * n + 3) * U * size).all())


def test_every_device_tensor_on_a_side_stream(env):
    torch, mlh, wl, hidden, gamma, w = env
    u = torch.rand((1,), device="cuda")
    tokens = torch.tensor([5, 7, 5], dtype=torch.int32, device="cuda")
    with mlh.LMHead(wl.n_rows, wl.k, max_batch=4, device=0) as head:
        logits = head.forward(hidden, w, gamma, want_argmax=False)
        rows = head.embed(tokens, w)
        want = (head.sample(logits, u, top_k=9)[0], head.forward_sample(hidden, w, u, gamma)[1], rows, head.embed_backward(rows, tokens))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            torch.cuda._sleep(5_000_000)
        got = (head.sample(logits.clone(), u, top_k=9, stream=side)[0], head.forward_sample(hidden, w, u, gamma, stream=side)[1],
               head.embed(tokens, w, stream=side), head.embed_backward(rows, tokens, stream=side))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
