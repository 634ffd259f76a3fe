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
