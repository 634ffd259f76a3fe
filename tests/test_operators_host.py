"""Refusals of the scoring, distillation and backward calls, without a GPU:
every rejection below comes before any CUDA call, from a host-side stand-in of
a handle's checks (a NULL handle) or from the binding's own checks on tensors."""
import pytest


@pytest.fixture(scope="module")
def mlh():
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    return mlh


def test_null_handles(mlh):
    assert mlh.muse_lmhead_score(None, 16, 0, 1, 8, 16, 1.0, 1, 16, 16, 16, 16, 16, 16, None) == -1
    assert mlh.muse_lmhead_forward_score(None, 16, 1, None, 1e-5, 16, 1.0, 0.0, 16, 16, 1.0, 1, 16, 16, 16, 16, 16, 16, None) == -1
    assert mlh.muse_lmhead_distill(None, 16, 0, 1, 8, 16, 16, 4, 0, None, 1.0, 16, None, 0, None) == -1
    assert mlh.muse_lmhead_backward(None, 16, 16, 16, 1, None, 1e-5, 16, 1.0, 0.0, 16, None, None) == -1


def _head(mlh, n_rows=8, k=256):
    """An LMHead without a handle: the binding's checks come before the library's."""
    h = mlh.LMHead.__new__(mlh.LMHead)
    h.device, h.n_rows, h.k, h.max_batch, h.fmt, h.block_bytes, h.handle = 0, n_rows, k, 1, "q5_k", 176, None
    return h


def test_binding_refuses_wrong_tensors(mlh):
    import torch
    h = _head(mlh)
    cpu = torch.zeros((2, 8))
    for call in (lambda: h.score(cpu), lambda: h.distill(cpu, torch.zeros((2, 3), dtype=torch.int32), torch.zeros((2, 3))),
                 lambda: h.backward(cpu, torch.zeros(8 * 176, dtype=torch.uint8)),
                 lambda: h.forward_score(torch.zeros((1, 256)), torch.zeros(8 * 176, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call()


def test_scores_are_named(mlh):
    assert mlh.TokenScores._fields == ("logprob", "rank", "lse", "entropy", "top_ids", "top_logprobs")
