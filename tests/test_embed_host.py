"""Refusals of the token table's calls without a GPU: each comes before any CUDA
call, from a NULL handle or from the binding's own checks on tensors."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def mlh():
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    return mlh


def test_null_handles(mlh):
    assert mlh.muse_lmhead_embed(None, 16, 0, 256, 16, 1, 1.0, 16, 0, 256, None) == -1
    assert mlh.muse_lmhead_embed_backward(None, 16, 0, 256, 16, 1, 1.0, 16, 0, 256, 0, 16, 1 << 20, None) == -1
    assert mlh.load_library().muse_lmhead_embed_backward_workspace(None, 1, ctypes.byref(ctypes.c_int64())) == -1
    with pytest.raises(mlh.MuseError):
        mlh.muse_lmhead_embed_backward_workspace(None, 1)


def test_binding_refuses_wrong_tensors(mlh):
    import torch
    h = mlh.LMHead.__new__(mlh.LMHead)
    h.device, h.n_rows, h.k, h.max_batch, h.fmt, h.block_bytes, h.handle = 0, 8, 256, 1, "q5_k", 176, None
    tokens, table = torch.zeros((3,), dtype=torch.int32), torch.zeros((8, 256))
    for call in (lambda: h.embed(tokens, table), lambda: h.embed(tokens.long(), table), lambda: h.embed_backward(torch.zeros((3, 256)), tokens),
                 lambda: h.embed_backward(torch.zeros((3, 256)), tokens, accumulate=True)):
        with pytest.raises(ValueError):
            call()
