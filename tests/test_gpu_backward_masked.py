"""Masked logits on their way back: a logit outside -cap..cap (-infinity, or a type's
lowest value) did not come through the cap, so nothing goes back through it,
whatever its gradient holds.  References in 64 bits and tolerances as for the
backward pass, with t = 0 at the masked places.
"""
import math

import numpy as np
import pytest

from test_gpu_backward import _dense, _grads, _reference, _weights, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    return torch


@pytest.mark.parametrize("mask", [-math.inf, float(np.finfo(np.float32).min), -3e4])
@pytest.mark.parametrize("given", ["zero", "some", "inf", "nan"])
@pytest.mark.parametrize("fmt", ["q5_k", "q4_k"])
@pytest.mark.parametrize("b", [1, 6, 12, 32])
def test_backward_of_masked_logits(torch_cuda, mask, given, fmt, b):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    n, k, cap = 1501, 768, 20.0
    rng = np.random.default_rng(b)
    wq = _weights(n, k, fmt, 41)
    logits = (cap * np.tanh(rng.standard_normal((b, n)))).astype(np.float32)
    masked = rng.random((b, n)) < 0.6
    masked[0] = True                                # a row of nothing else
    masked[-1, -1] = True
    gl = _grads(rng, b, n)
    clean = np.where(masked, 0, gl).astype(np.float32)
    gl = {"zero": clean, "some": gl, "inf": np.where(masked, np.float32(math.inf), gl),
          "nan": np.where(masked, np.float32(math.nan), gl)}[given]
    seen = np.where(masked, np.float32(mask), logits)
    hidden = rng.standard_normal((b, k)).astype(np.float32)
    gamma = (1 + 0.1 * rng.standard_normal(k)).astype(np.float32)
    dev = lambda t: torch.from_numpy(np.ascontiguousarray(t)).cuda()                      # noqa: E731
    with mlh.LMHead(n, k, max_batch=b, device=0, fmt=fmt) as head:
        gh, gg = head.backward(dev(gl), dev(wq), logits=dev(seen), hidden=dev(hidden), gamma=dev(gamma), scale=0.7, cap=cap)
        torch.cuda.synchronize()
        assert head.device_status() == 0
    want, tol, wg, tg = _reference(clean, logits, hidden, gamma, _dense(wq, n, k, fmt), float(np.float32(0.7)), cap)
    _within("grad_hidden", gh.cpu().numpy(), want, tol)
    _within("grad_gamma", gg.cpu().numpy(), wg, tg)
    assert not gh[0].any()


def test_backward_of_masked_logits_beside_a_large_block(torch_cuda):
    """A block factor of 4 and more: the sums in f32 from the blocks themselves."""
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    n, k, b = 301, 512, 3
    rng = np.random.default_rng(3)
    wq = _weights(n, k, "q5_k", 42).reshape(n, k // 256, 176).copy()
    wq[17, 1, :2] = np.array([5.0], dtype=np.float16).view(np.uint8)
    logits = (20 * np.tanh(rng.standard_normal((b, n)))).astype(np.float32)
    masked = rng.random((b, n)) < 0.5
    gl = _grads(rng, b, n)
    dev = lambda t: torch.from_numpy(np.ascontiguousarray(t)).cuda()                      # noqa: E731
    with mlh.LMHead(n, k, max_batch=b, device=0) as head:
        gh, _ = head.backward(dev(gl), dev(wq.reshape(-1)), logits=dev(np.where(masked, np.float32(-math.inf), logits)), scale=1.0)
        torch.cuda.synchronize()
    want, tol, _, _ = _reference(np.where(masked, 0, gl).astype(np.float32), logits, None, None, _dense(wq, n, k, "q5_k"), 1.0, 20.0)
    _within("grad_hidden", gh.cpu().numpy(), want, tol)


def test_backward_keeps_a_logit_that_is_not_a_number(torch_cuda):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    n, k = 700, 256
    wq = torch.from_numpy(np.ascontiguousarray(_weights(n, k, "q5_k", 43))).cuda()
    g, x = torch.randn((2, n), device="cuda"), torch.zeros((2, n), device="cuda")
    x[1, 9] = math.nan
    with mlh.LMHead(n, k, max_batch=2, device=0) as head:
        gh, _ = head.backward(g, wq, logits=x, scale=1.0)
        torch.cuda.synchronize()
    assert bool(gh[0].isfinite().all()) and bool(gh[1].isnan().all())


@pytest.mark.parametrize("mask", [-math.inf, float(np.finfo(np.float32).min)])
@pytest.mark.parametrize("tail", [False, True])
def test_a_masked_step(torch_cuda, mask, tail):
    """forward -> mask -> score (the teacher's) -> distill -> backward."""
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    b, n, k, top = 5, 2003, 512, 8
    rng = np.random.default_rng(51)
    wq = _weights(n, k, "q5_k", 44)
    w = torch.from_numpy(wq).cuda()
    gamma = (1 + 0.1 * rng.standard_normal(k)).astype(np.float32)
    teach, hidden = (rng.standard_normal((b, k)).astype(np.float32) for _ in range(2))
    allowed = torch.from_numpy(rng.random((b, n)) < 0.3).cuda()
    g, h = torch.from_numpy(gamma).cuda(), torch.from_numpy(hidden).cuda()
    with mlh.LMHead(n, k, max_batch=b, device=0) as head:
        seen = head.forward(torch.from_numpy(teach).cuda(), w, g)[0].masked_fill_(~allowed, mask)
        scores = head.score(seen, n_top=top)
        plain = head.forward(h, w, g)[0]
        logits = plain.masked_fill(~allowed, mask)
        loss, grad = head.distill(logits, scores.top_ids, scores.top_logprobs, tail=tail)
        gh, gg = head.backward(grad, w, logits=logits, hidden=h, gamma=g)
        torch.cuda.synchronize()
        assert head.device_status() == 0
    assert bool(allowed.gather(1, scores.top_ids.long()).all())
    assert bool(loss.isfinite().all()) and not bool(grad[~allowed].any())
    want, tol, wg, tg = _reference(grad.cpu().numpy(), plain.cpu().numpy(), hidden, gamma, _dense(wq, n, k, "q5_k"),
                                   float(np.float32(0.196116)), 20.0)
    _within("grad_hidden", gh.cpu().numpy(), want, tol)
    _within("grad_gamma", gg.cpu().numpy(), wg, tg)
