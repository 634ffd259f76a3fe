"""Calls on another stream than the current one: memory that torch hands out again
while one of the two streams is still using it.  A stream is kept busy by torch's
timed sleep of some milliseconds, so that what is queued behind it runs late."""
import numpy as np
import pytest

import q5k_synth as synth

pytestmark = pytest.mark.gpu

SLEEP = 20_000_000          # cycles: about 10 ms


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
    head = mlh.LMHead(wl.n_rows, wl.k, max_batch=4, device=0)
    h = dev(np.concatenate([hidden * s for s in (1.0, 0.5, -1.0, 2.0)]))
    w, g = dev(wq), dev(gamma)
    logits = head.forward(h, w, g, want_argmax=False)
    scores = head.score(logits, n_top=8)
    grad = head.distill(logits, scores.top_ids, scores.top_logprobs.roll(1, 0), tail=True)[1]
    head.backward(grad, w, logits=logits, hidden=h, gamma=g)
    torch.cuda.synchronize()
    tokens = torch.arange(4, dtype=torch.int32, device="cuda")

    def calls(logits, grad, h):
        return {
            "forward": lambda s: head.forward(h, w, g, stream=s),
            "forward_logprobs": lambda s: head.forward_logprobs(h, w, g, stream=s),
            "forward_group": lambda s: head.forward_group(h[0], [(w, wl.n_rows, 1.0, 0.0, None)], g, stream=s),
            "score": lambda s: head.score(logits, tokens, n_top=8, stream=s),
            "forward_score": lambda s: (lambda o: (o[0], *o[1]))(head.forward_score(h, w, g, tokens=tokens, n_top=8, stream=s)),
            "distill": lambda s: head.distill(logits, scores.top_ids, scores.top_logprobs, tail=True, stream=s),
            "backward": lambda s: head.backward(grad, w, logits=logits, hidden=h, gamma=g, stream=s),
        }

    yield torch, head, calls, (logits, grad, h)
    head.close()


CALLS = ("forward", "forward_logprobs", "forward_group", "score", "forward_score", "distill", "backward")


@pytest.mark.parametrize("name", CALLS)
def test_results_do_not_take_memory_that_the_current_stream_still_reads(env, name):
    torch, head, calls, inputs = env
    call = calls(*inputs)[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    held = [torch.full_like(t, 3) for t in want]
    kept = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    for a, b in zip(kept, held):
        a.copy_(b)                            # queued behind the sleep
    del held, a, b                            # and its sources let go
    got = call(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    torch.cuda.synchronize()
    assert all(bool((t == 3).all()) for t in kept)


@pytest.mark.parametrize("name", CALLS)
def test_results_let_go_before_the_current_stream_has_read_them(env, name):
    torch, head, calls, inputs = env
    call = calls(*inputs)[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    kept = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SLEEP)
    for a, b in zip(kept, got):
        a.copy_(b)
    sizes = [(t.shape, t.dtype) for t in got]
    del got, a, b
    with torch.cuda.stream(side):             # what the side stream makes next
        other = [torch.full(shape, 9, dtype=dtype, device="cuda") for shape, dtype in sizes]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(kept, want)) and len(other) == len(kept)


@pytest.mark.parametrize("name", CALLS)
def test_inputs_let_go_before_the_call_has_run(env, name):
    torch, head, calls, inputs = env
    want = [t.clone() for t in calls(*inputs)[name](None)]
    mine = [t.clone() for t in inputs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    table = calls(*mine)
    got = table[name](side)
    del table
    sizes = [t.shape for t in mine]
    del mine
    other = [torch.full(shape, 9.0, device="cuda") for shape in sizes]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and len(other) == 3


def test_a_stream_by_its_handle(env):
    torch, head, calls, inputs = env

    class Handle:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    side = torch.cuda.Stream()
    want = head.score(inputs[0], n_top=3)
    got = head.score(inputs[0], n_top=3, stream=Handle(side))
    torch.cuda.synchronize()
    assert torch.equal(got.top_ids, want.top_ids) and torch.equal(got.lse, want.lse)
