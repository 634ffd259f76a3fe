"""Drawing, lookup and the table's gradient on another stream than the current one:
memory that torch hands out again while one of the two streams is still using it
(as test_gpu_streams does for the other calls)."""
import numpy as np
import pytest

import q5k_synth as synth

pytestmark = pytest.mark.gpu

SLEEP = 20_000_000          # cycles: about 10 ms
CALLS = ("sample", "sample_settings", "forward_sample", "embed", "embed_dense", "embed_backward")


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
    w, g = dev(wq), dev(gamma)
    h = dev(np.concatenate([hidden * s for s in (1.0, 0.5, -1.0, 2.0)]))
    logits = head.forward(h, w, g, want_argmax=False)
    table = torch.randn((wl.n_rows, wl.k), device="cuda").to(torch.bfloat16)
    inputs = (logits, h, torch.rand((4,), device="cuda"), torch.full((4,), 0.75, device="cuda"), table)
    tokens = torch.tensor([3, 9, 3, 2000], dtype=torch.int32, device="cuda")

    def calls(logits, h, u, t, table):
        return {
            "sample": lambda s: head.sample(logits, u, top_p=0.9, stream=s),
            "sample_settings": lambda s: head.sample(logits, u, temperature=t, top_k=5, stream=s),
            "forward_sample": lambda s: head.forward_sample(h, w, u, g, temperature=t, stream=s),
            "embed": lambda s: (head.embed(tokens, w, stream=s),),
            "embed_dense": lambda s: (head.embed(tokens, table, scale=2.0, stream=s),),
            "embed_backward": lambda s: (head.embed_backward(h, tokens, stream=s),),
        }

    yield torch, calls, inputs
    head.close()


@pytest.mark.parametrize("name", CALLS)
def test_results_do_not_take_memory_that_the_current_stream_still_reads(env, name):
    torch, calls, inputs = env
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
def test_inputs_let_go_before_the_call_has_run(env, name):
    torch, calls, inputs = env
    want = [t.clone() for t in calls(*inputs)[name](None)]
    mine = [t.clone() for t in inputs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    table = calls(*mine)
    got = table[name](side)
    del table
    sizes = [(t.shape, t.dtype) for t in mine]
    del mine
    other = [torch.full(shape, 9, dtype=dtype, device="cuda") for shape, dtype in sizes]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and len(other) == len(sizes)


@pytest.mark.parametrize("name", CALLS)
def test_calls_one_behind_another_and_on_two_streams(env, name):
    """The same call queued many times, on one stream and on two: no state of one reaches another."""
    torch, calls, inputs = env
    call = calls(*inputs)[name]
    want = [t.clone() for t in call(None)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [call(None) for _ in range(20)] + [call(streams[i % 2]) for i in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for out in got for p, q in zip(out, want))
