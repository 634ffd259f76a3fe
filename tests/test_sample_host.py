"""Refusals of the sampling calls without a GPU: each comes before any CUDA call,
from a NULL handle or from the binding's own checks on tensors."""
import pytest


@pytest.fixture(scope="module")
def mlh():
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    return mlh


def test_null_handles(mlh):
    how = mlh.MuseSampling(1.0, 0, 1.0, 0.0)
    assert mlh.muse_lmhead_sample(None, 16, 0, 1, 8, how, 16, 16, 16, None) == -1
    assert mlh.muse_lmhead_forward_sample(None, 16, 1, None, 1e-5, 16, 1.0, 0.0, 16, how, 16, 16, 16, None) == -1


def test_struct_layout(mlh):
    s = mlh.MuseSampling
    assert [getattr(s, f).offset for f, _ in s._fields_] == [0, 4, 8, 12, 16, 24, 32, 40]


def test_binding_refuses_wrong_tensors(mlh):
    import torch
    h = mlh.LMHead.__new__(mlh.LMHead)
    h.device, h.n_rows, h.k, h.max_batch, h.fmt, h.block_bytes, h.handle = 0, 8, 256, 1, "q5_k", 176, None
    for call in (lambda: h.sample(torch.zeros((2, 8)), torch.zeros(2)),
                 lambda: h._sampling(2, torch.zeros(2), 0, 1.0, 0.0), lambda: h._sampling(2, 1.0, torch.zeros(2), 1.0, 0.0),
                 lambda: h.forward_sample(torch.zeros((1, 256)), torch.zeros(8 * 176, dtype=torch.uint8), torch.zeros(1))):
        with pytest.raises(ValueError):
            call()


def test_settings_of_numbers(mlh):
    h = mlh.LMHead.__new__(mlh.LMHead)
    h.device, h.n_rows, h.handle = 0, 1000, None
    how = h._sampling(3, 0.5, 10 ** 12, 0.875, 0.25)
    assert (how.temperature, how.top_k, how.top_p, how.min_p) == (0.5, 1000, 0.875, 0.25)
    assert not (how.temperatures or how.top_ks or how.top_ps or how.min_ps)
    assert h._sampling(3, 1.0, -10 ** 12, 1.0, 0.0).top_k == 0
