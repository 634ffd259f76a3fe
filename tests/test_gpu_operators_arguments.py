"""Forms of arguments that the forwards take and the calls beside them have to take too."""
import numpy as np
import pytest

import q5k_synth as synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    n, k = 700, 512
    w = torch.from_numpy(np.ascontiguousarray(synth.q5k_matrix(n, k, synth.stream_key(71, "W:args")))).cuda()
    with mlh.LMHead(n, k, max_batch=2, device=0) as head:
        yield torch, head, w, torch.randn(k, device="cuda"), 1 + 0.1 * torch.randn(k, device="cuda")


def test_one_row_without_a_batch_dimension(env):
    """hidden [k] goes into the forward as it is; it goes into the backward pass as it is, too."""
    torch, head, w, hidden, gamma = env
    logits = head.forward(hidden, w, gamma, want_argmax=False)
    grad = torch.randn_like(logits)
    want = head.backward(grad, w, logits=logits, hidden=hidden[None], gamma=gamma)
    for g in (grad, grad[0]):
        for x in (logits, logits[0]):
            for h in (hidden[None], hidden):
                got = head.backward(g, w, logits=x, hidden=h, gamma=gamma)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ValueError):
        head.backward(torch.cat([grad, grad]), w, logits=logits[0], hidden=hidden, gamma=gamma)


def test_numbers_of_other_types(env):
    """Scale, cap, eps and temperature as numpy scalars or tensors of one value, as the forwards take them."""
    torch, head, w, hidden, gamma = env
    logits = head.forward(hidden, w, gamma, scale=0.5, cap=8.0, want_argmax=False)
    scores = head.score(logits, n_top=4, temperature=0.5)
    loss, grad = head.distill(logits, scores.top_ids, scores.top_logprobs, temperature=2.0)
    back = head.backward(grad, w, logits=logits, hidden=hidden, gamma=gamma, eps=0.25, scale=0.5, cap=8.0)
    for make in (np.float32, np.float64, torch.tensor):
        a = make(0.5), make(8.0)
        assert torch.equal(head.forward(hidden, w, gamma, scale=a[0], cap=a[1], want_argmax=False), logits)
        assert torch.equal(head.score(logits, n_top=4, temperature=a[0]).top_logprobs, scores.top_logprobs)
        assert torch.equal(head.distill(logits, scores.top_ids, scores.top_logprobs, temperature=make(2.0))[1], grad)
        got = head.backward(grad, w, logits=logits, hidden=hidden, gamma=gamma, eps=make(0.25), scale=a[0], cap=a[1])
        assert torch.equal(got[0], back[0]) and torch.equal(got[1], back[1])
