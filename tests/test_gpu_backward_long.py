"""The backward pass over many stages a CTA: every build of its kernel (8, 16 and
32 batch slots, Q5_K and Q4_K) refills its rings and opens new sets of sums many
times, as the full head does, and the error is held against the norm of the
result, where a lost half of an operand or sums left too long on the tensor cores
would show.

Tolerance by the norm (u = 2^-24, gradients of random sign): the tensor cores cut
a sum off towards zero, u of it a step on the average and 2u at most; a set of
sums takes at most 288 rows, 18 steps of 16 rows, twice where both halves of an
operand go to the same sums: 36 steps, over which the sum grows, so 2/3 of 36u =
24u of a set's sum.  The sets' signs are independent, so of the whole 24u as well
(in the norm), for each kind of products (quants, scales, mins).  Halves good to
4u, t's six roundings and the f32 sums of the sets (a random walk of V/256
roundings of u/2 each: below 15u for these sizes) come to less than that:
50u (|sum t d sc (q - c0)| + |sum t c0 d sc| + |sum t dmin m|) = 3e-6 of these norms.
Left out, the sets would be chains of a share's 2,300 steps, 1,500u; the lower
halves, 2^-12 / sqrt(3) = 2,300u.
"""
import numpy as np
import pytest

import q5k_synth as synth
from test_gpu_backward import U, _grads, _reference, _weights, _dense, _within

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


def _products(wq, n, kb, fmt):
    """Block column kb as its three kinds of products in 64 bits: d sc (q - c0), c0 d sc and -dmin m."""
    size, qs0, c0 = (176, 48, 16) if fmt == "q5_k" else (144, 16, 8)
    b = np.ascontiguousarray(wq).reshape(n, -1, size)[:, kb]
    half = b[:, :4].copy().view(np.float16).astype(np.float64)
    out = np.empty((3, n, 8, 32))
    for s in range(8):
        w0, w1, w2 = (b[:, 4 + 4 * i + s % 4].astype(np.int64) for i in range(3))
        sc, mn = (w0 & 63, w1 & 63) if s < 4 else ((w2 & 15) | (w0 >> 6 << 4), (w2 >> 4) | (w1 >> 6 << 4))
        q = (b[:, qs0 + 32 * (s // 2):qs0 + 32 * (s // 2) + 32].astype(np.int64) >> (4 * (s % 2))) & 15
        if fmt == "q5_k":
            q = q | (((b[:, 16:48].astype(np.int64) >> s) & 1) << 4)
        out[0, :, s] = (half[:, 0] * sc)[:, None] * (q - c0)
        out[1, :, s] = (half[:, 0] * sc * c0)[:, None]
        out[2, :, s] = (-half[:, 1] * mn)[:, None]
    return out.reshape(3, n, 256)


def _norm_check(name, got, gl, parts):
    sums = [gl.astype(np.float64) @ p for p in parts]
    want = sums[0] + sums[1] + sums[2]
    err = np.linalg.norm(got.astype(np.float64) - want, axis=1)
    tol = 50 * U * sum(np.linalg.norm(s, axis=1) for s in sums)
    assert (err <= tol).all(), f"{name}: norm of the error {err / tol} of what is allowed"


N, K, COLUMNS = 29003, 6656, (0, 13, 25)      # 11 shares of 27 stages of 96 rows, or 41 of 64, and a rest in the last


@pytest.fixture(scope="module")
def matrices(torch_cuda):
    out = {}
    for fmt in ("q5_k", "q4_k"):
        wq = _weights(N, K, fmt, 31)
        out[fmt] = wq, torch_cuda.from_numpy(np.ascontiguousarray(wq)).cuda(), {kb: _products(wq, N, kb, fmt) for kb in COLUMNS}
    return out


@pytest.mark.parametrize("fmt", ["q5_k", "q4_k"])
@pytest.mark.parametrize("b", [1, 8, 9, 16, 17, 32])
def test_backward_over_many_stages(torch_cuda, matrices, fmt, b):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    wq, w, products = matrices[fmt]
    rng = np.random.default_rng(b)
    random = rng.standard_normal((b, N)).astype(np.float32)
    steep = _grads(rng, b, N)
    raw = np.ascontiguousarray(wq).reshape(N, K // 256, -1)
    with mlh.LMHead(N, K, max_batch=b, device=0, fmt=fmt) as head:
        for gl in (random, steep):
            g = torch.from_numpy(gl).cuda()
            first, _ = head.backward(g, w, scale=1.0, cap=0.0)
            first = first.clone()
            again = [head.backward(g, w, scale=1.0, cap=0.0)[0] for _ in range(20)]
            torch.cuda.synchronize()
            assert head.device_status() == 0
            assert all(torch.equal(t, first) for t in again)
            for kb in COLUMNS:
                got = first[:, 256 * kb:256 * kb + 256].cpu().numpy()
                want, tol, _, _ = _reference(gl, None, None, None, _dense(raw[:, kb], N, 256, fmt), 1.0, 0.0)
                _within(f"block column {kb}", got, want, tol)
                if gl is random:
                    _norm_check(f"block column {kb}", got, gl, products[kb])


@pytest.mark.parametrize("b", [3, 12, 32])
def test_backward_full_head_by_the_norm(torch_cuda, b):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    n, k = 202048, 6656
    wq = synth.inputs_for(synth.WORKLOADS["lmhead_b1"])[2]
    gl = np.random.default_rng(b).standard_normal((b, n)).astype(np.float32)
    with mlh.LMHead(n, k, max_batch=b, device=0) as head:
        gh, _ = head.backward(torch.from_numpy(gl).cuda(), torch.from_numpy(wq).cuda(), scale=1.0, cap=0.0)
        torch.cuda.synchronize()
        assert head.device_status() == 0
    for kb in (0, 25):
        _norm_check(f"block column {kb}", gh[:, 256 * kb:256 * kb + 256].cpu().numpy(), gl, _products(wq, n, kb, "q5_k"))
