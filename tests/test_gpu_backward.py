"""GPU parity of muse_lmhead_backward: the gradient by the logits back through
soft cap, scale, the Q5_K or Q4_K matrix and the final norm, against the
formulas in 64 bits over the oracle's dequantised weights, against differences
of the f64 oracle's forward, and in a run forward -> score -> distill ->
backward as a training step makes it.

Tolerances (u = 2^-24): t_v carries six roundings; a weight or an operand split
in two 16-bit halves is good to 2^-22 = 4u; a sum of V products in any order,
kept in f32, is off by at most V u, and no kernel adds more than V/8 + 64 in a
chain.  The products are those of a weight's parts, W = d sc (q - c0) + c0 d sc -
dmin m with c0 the quants' middle: each part t_v P is rounded on its own scale,
and where the parts of a W cancel (q = 0: -c0 d sc + c0 d sc) the rounding of
each stays.  So |gx - exact| <= c sum_v |t_v| (|d sc (q - c0)| + |c0 d sc| + |dmin m|)
with c = (V/8 + 96) u: a bound by sum |t_v W_vk| alone would hold for a kernel
that adds rounded weights, and needs W's parts to be added before t, which no
order of exact products does.  The norm's backward passes that error on linearly
and adds at most 40u of its terms.
"""
import numpy as np
import pytest

import oracle
import q5k_synth as synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = synth.RMS_EPS


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    return torch


def _weights(n, k, fmt, seed):
    return synth.q5k_matrix(n, k, synth.stream_key(seed, f"W:bwd{n}:{k}"), fmt=fmt)


def _dense(wq, n, k, fmt):
    """The matrix in 64 bits and the sizes of its weights' parts, from the block layout (numpy, no code of the package)."""
    size, qs0 = (176, 48) if fmt == "q5_k" else (144, 16)
    b = np.ascontiguousarray(wq).reshape(n, k // 256, size)
    half = b[:, :, :4].copy().view(np.float16).astype(np.float64)
    out, size_of, c0 = np.empty((n, k // 256, 8, 32)), np.empty((n, k // 256, 8, 32)), 16 if fmt == "q5_k" else 8
    for s in range(8):
        w0, w1, w2 = (b[:, :, 4 + 4 * i + s % 4].astype(np.int64) for i in range(3))
        sc, mn = (w0 & 63, w1 & 63) if s < 4 else ((w2 & 15) | (w0 >> 6 << 4), (w2 >> 4) | (w1 >> 6 << 4))
        q = (b[:, :, qs0 + 32 * (s // 2):qs0 + 32 * (s // 2) + 32].astype(np.int64) >> (4 * (s % 2))) & 15
        if fmt == "q5_k":
            q = q | (((b[:, :, 16:48].astype(np.int64) >> s) & 1) << 4)
        ds, dm = (half[:, :, 0] * sc)[..., None], (half[:, :, 1] * mn)[..., None]
        out[:, :, s] = ds * q - dm
        size_of[:, :, s] = np.abs(ds) * (np.abs(q - c0) + c0) + np.abs(dm)
    return out.reshape(n, k), size_of.reshape(n, k)


def _reference(gl, logits, hidden, gamma, w, scale, cap):
    gl = gl.astype(np.float64)
    t = gl * scale
    if cap > 0:
        ld = logits.astype(np.float64)
        t = t * (cap - ld) * (cap + ld) / cap ** 2
    w, parts = w
    gx, ax = t @ w, np.abs(t) @ parts
    tol = (w.shape[0] / 8 + 96) * U * ax
    if gamma is None:
        return gx, tol, None, None
    h, g = hidden.astype(np.float64), gamma.astype(np.float64)
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + float(np.float32(EPS)))
    u = gx * g
    gh = r * (u - h * r ** 2 * (u * h).mean(1, keepdims=True))
    mean = (np.abs(u) * np.abs(h)).mean(1, keepdims=True)
    tol_h = r * (tol * np.abs(g) + np.abs(h) * r ** 2 * (tol * np.abs(g) * np.abs(h)).mean(1, keepdims=True))
    tol_h = tol_h + 40 * U * r * (np.abs(u) + np.abs(h) * r ** 2 * mean)
    gg = (gx * h * r).sum(0)
    tol_g = (tol * np.abs(h) * r).sum(0) + 40 * U * (np.abs(gx) * np.abs(h) * r).sum(0)
    return gh, tol_h, gg, tol_g


def _within(name, got, want, tol):
    err = np.abs(got.astype(np.float64) - want)
    assert np.isfinite(got).all(), name
    over = err - tol - 1e-37
    at = np.unravel_index(over.argmax(), over.shape)
    assert over.max() <= 0, f"{name}: off by {err[at]:.3g} at {at}, allowed {tol[at]:.3g}"


def _grads(rng, b, n):
    x = rng.standard_normal((b, n)) * 2
    g = np.exp(x - x.max(1, keepdims=True))
    g /= g.sum(1, keepdims=True)
    g[np.arange(b), rng.integers(0, n, b)] -= 1
    return (g / b).astype(np.float32)


SHAPES = [(1, 1, 256), (1, 3, 512), (2, 16, 256), (1, 2048, 6656), (5, 2048, 6656), (8, 129, 1024), (9, 1000, 768),
          (16, 4096, 512), (17, 333, 4096), (32, 777, 2560), (31, 20000, 256), (3, 40000, 512), (2, 257, 6656),
          (32, 1537, 6656), (4, 64, 13312)]


@pytest.mark.parametrize("fmt", ["q5_k", "q4_k"])
@pytest.mark.parametrize("norm,cap", [(True, 20.0), (False, 0.0)])
@pytest.mark.parametrize("b,n,k", SHAPES)
def test_backward_shapes(torch_cuda, fmt, norm, cap, b, n, k):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    rng = np.random.default_rng(b * 1000 + n + k)
    wq = _weights(n, k, fmt, 11)
    gl = _grads(rng, b, n)
    logits = (20 * np.tanh(rng.standard_normal((b, n)))).astype(np.float32)
    logits[0, 0] = 20.0                             # saturated: no gradient through it
    hidden = (rng.standard_normal((b, k)) * rng.uniform(0.5, 4, (b, 1))).astype(np.float32)
    gamma = (1 + 0.1 * rng.standard_normal(k)).astype(np.float32) if norm else None
    dev = [None if t is None else torch.from_numpy(np.ascontiguousarray(t)).cuda() for t in (gl, wq, logits, hidden, gamma)]
    with mlh.LMHead(n, k, max_batch=b, device=0, fmt=fmt) as head:
        gh, gg = head.backward(dev[0], dev[1], logits=dev[2] if cap > 0 else None, hidden=dev[3] if norm else None,
                               gamma=dev[4], scale=synth.LOGIT_SCALE, cap=cap)
        again, _ = head.backward(dev[0], dev[1], logits=dev[2], hidden=dev[3], gamma=dev[4], scale=synth.LOGIT_SCALE, cap=cap)
        torch.cuda.synchronize()
        assert head.device_status() == 0
    assert torch.equal(gh, again)                   # a fixed order of the sums
    want, tol, wg, tg = _reference(gl, logits, hidden, gamma, _dense(wq, n, k, fmt), float(np.float32(synth.LOGIT_SCALE)), cap)
    _within("grad_hidden", gh.cpu().numpy(), want, tol)
    if norm:
        _within("grad_gamma", gg.cpu().numpy(), wg, tg)
    else:
        assert gg is None


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1.0, 1e12])
def test_backward_sizes_of_gradients(torch_cuda, size):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    b, n, k = 4, 3001, 512
    rng = np.random.default_rng(5)
    wq = _weights(n, k, "q5_k", 12)
    gl = (_grads(rng, b, n) * size).astype(np.float32)
    gl[1] = 0.0                                     # a padded row
    gl[2] *= 1e-6                                   # rows of very different sizes
    gl[3, 100:] = 0.0
    with mlh.LMHead(n, k, max_batch=b, device=0) as head:
        gh, _ = head.backward(torch.from_numpy(gl).cuda(), torch.from_numpy(wq).cuda(), scale=1.0, cap=0.0)
        torch.cuda.synchronize()
    want, tol, _, _ = _reference(gl, None, None, None, _dense(wq, n, k, "q5_k"), 1.0, 0.0)
    _within("grad_hidden", gh.cpu().numpy(), want, tol)
    assert not gh[1].any()


def test_backward_extreme_blocks(torch_cuda):
    """Largest scales, mins, quants and block factors, and blocks of nothing."""
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    rng = np.random.default_rng(9)
    for fmt, size in (("q5_k", 176), ("q4_k", 144)):
        n, k, b = 300, 1024, 3
        wq = rng.integers(0, 256, (n, k // 256, size), dtype=np.uint8)
        d = rng.choice(np.array([0.0, 6e-8, 1e-5, 0.03, 1.0, -1.0, 60000.0], dtype=np.float16), (n, k // 256, 2))
        wq[:, :, :4] = d.view(np.uint8).reshape(n, k // 256, 4)
        wq[5] = 0
        wq[6, :, 4:] = 255
        gl = _grads(rng, b, n)
        with mlh.LMHead(n, k, max_batch=b, device=0, fmt=fmt) as head:
            gh, _ = head.backward(torch.from_numpy(gl).cuda(), torch.from_numpy(wq.reshape(-1)).cuda(), scale=1.0, cap=0.0)
            torch.cuda.synchronize()
        want, tol, _, _ = _reference(gl, None, None, None, _dense(wq, n, k, fmt), 1.0, 0.0)
        _within("grad_hidden", gh.cpu().numpy(), want, tol)


def test_backward_against_differences_of_the_oracle(torch_cuda):
    """d(sum c * logits)/d(hidden, gamma) against central differences of the f64 oracle's forward."""
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    b, n, k = 2, 96, 256
    rng = np.random.default_rng(3)
    wq = _weights(n, k, "q5_k", 13)
    hidden = rng.standard_normal((b, k)).astype(np.float32)
    gamma = (1 + 0.1 * rng.standard_normal(k)).astype(np.float32)
    c = rng.standard_normal((b, n)).astype(np.float32)
    dev = lambda t: torch.from_numpy(np.ascontiguousarray(t)).cuda()                      # noqa: E731
    with mlh.LMHead(n, k, max_batch=b, device=0) as head:
        logits, _ = head.forward(dev(hidden), dev(wq), dev(gamma))
        gh, gg = head.backward(dev(c), dev(wq), logits=logits, hidden=dev(hidden), gamma=dev(gamma))
        torch.cuda.synchronize()
    gh, gg = gh.cpu().numpy(), gg.cpu().numpy()
    f = lambda h, g: float((oracle.lmhead(h, g, wq, synth.LOGIT_SCALE, synth.SOFTCAP, EPS) * c).sum())   # noqa: E731
    step = np.float32(2.0 ** -7)
    for j in range(0, k, 37):
        for at in ((0, j), (1, j)):
            up, dn = hidden.copy(), hidden.copy()
            up[at] += step
            dn[at] -= step
            d = (f(up, gamma) - f(dn, gamma)) / (float(up[at]) - float(dn[at]))
            assert abs(d - gh[at]) <= 2e-3 * max(1.0, np.abs(gh).max())   # h^2/6 of third derivatives, h = 2^-7
        up, dn = gamma.copy(), gamma.copy()
        up[j] += step
        dn[j] -= step
        d = (f(hidden, up) - f(hidden, dn)) / (float(up[j]) - float(dn[j]))
        assert abs(d - gg[j]) <= 2e-3 * max(1.0, np.abs(gg).max())


def test_a_distillation_step(torch_cuda):
    """Teacher scores -> student forward -> distill -> backward, eager and as a
    replayed graph, against the chain in 64 bits."""
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    b, n, k, top = 6, 3001, 512, 12
    rng = np.random.default_rng(21)
    wq = _weights(n, k, "q5_k", 14)
    w64 = _dense(wq, n, k, "q5_k")
    gamma = (1 + 0.1 * rng.standard_normal(k)).astype(np.float32)
    teach = rng.standard_normal((b, k)).astype(np.float32)
    w = torch.from_numpy(wq).cuda()
    g = torch.from_numpy(gamma).cuda()
    weight = torch.full((b,), 1.0 / b, device="cuda")
    hidden = torch.empty((b, k), device="cuda")
    with mlh.LMHead(n, k, max_batch=b, device=0) as head:
        _, scores = head.forward_score(torch.from_numpy(teach).cuda(), w, g, n_top=top)

        def step():
            logits, _ = head.forward(hidden, w, g)
            loss, grad = head.distill(logits, scores.top_ids, scores.top_logprobs, weight, tail=True)
            return (logits, loss, grad, *head.backward(grad, w, logits=logits, hidden=hidden, gamma=g))

        s = torch.cuda.Stream()
        runs = [(teach + d * rng.standard_normal((b, k))).astype(np.float32) for d in (0.3, 1.0)]
        hidden.copy_(torch.from_numpy(runs[0]))
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                got = step()
        torch.cuda.synchronize()
        for h in runs:
            hidden.copy_(torch.from_numpy(h))
            eager = [t.clone() for t in step()]
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(eager, got))
            logits, loss, grad, gh, gg = (t.cpu().numpy() for t in got)
            ids, lp = scores.top_ids.cpu().numpy(), scores.top_logprobs.cpu().numpy().astype(np.float64)
            x = logits.astype(np.float64)
            q = np.exp(x - x.max(1, keepdims=True))
            q /= q.sum(1, keepdims=True)
            p = np.exp(lp)
            out = np.ones_like(q)
            np.put_along_axis(out, ids.astype(np.int64), 0.0, axis=1)
            qt, pt = (q * out).sum(1), 1 - p.sum(1)
            want = ((p * (lp - np.log(np.take_along_axis(q, ids.astype(np.int64), 1)))).sum(1) + pt * np.log(pt / qt)) / b
            assert np.abs(loss - want).max() <= 2e-6
            full = q * (1 - out * (pt / qt)[:, None])
            for r in range(b):
                full[r, ids[r]] -= p[r]
            assert np.abs(grad - full / b).max() <= 2e-7
            ref, tol, rg, tg = _reference(grad, logits, h, gamma, w64, float(np.float32(synth.LOGIT_SCALE)), 20.0)
            _within("grad_hidden", gh, ref, tol)
            _within("grad_gamma", gg, rg, tg)
        assert head.device_status() == 0


def test_backward_full_head(torch_cuda):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    n, k, b = 202048, 6656, 3
    rng = np.random.default_rng(2)
    wq = synth.inputs_for(synth.WORKLOADS["lmhead_b1"])[2]
    gl = _grads(rng, b, n)
    with mlh.LMHead(n, k, max_batch=b, device=0) as head:
        gh, _ = head.backward(torch.from_numpy(gl).cuda(), torch.from_numpy(wq).cuda(), scale=1.0, cap=0.0)
        torch.cuda.synchronize()
        assert head.device_status() == 0
    cols = np.asarray([0, 255, 3333 // 256 * 256, 6655])     # a few block columns, every row
    raw = np.ascontiguousarray(wq).reshape(n, k // 256, 176)
    for kb in sorted({int(c) // 256 for c in cols}):
        w = _dense(raw[:, kb], n, 256, "q5_k")
        want, tol, _, _ = _reference(gl, None, None, None, w, 1.0, 0.0)
        _within("grad_hidden", gh[:, kb * 256:kb * 256 + 256].cpu().numpy(), want, tol)


@pytest.mark.parametrize("b,n,k,fmt", [(1, 6007, 6656, "q5_k"), (5, 2048, 6656, "q4_k"), (12, 3001, 1024, "q5_k"), (32, 1501, 2560, "q4_k")])
def test_backward_back_to_back_with_other_gradients(torch_cuda, b, n, k, fmt):
    """Calls one behind another on one handle: each kernel starts early and has to see its own call's values."""
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    rng = np.random.default_rng(b)
    wq = torch.from_numpy(np.ascontiguousarray(_weights(n, k, fmt, 15))).cuda()
    grads = [torch.from_numpy((_grads(rng, b, n) * s).astype(np.float32)).cuda() for s in (1.0, 1e-5, 300.0)]
    hidden = torch.from_numpy(rng.standard_normal((b, k)).astype(np.float32)).cuda()
    gamma = torch.from_numpy((1 + 0.1 * rng.standard_normal(k)).astype(np.float32)).cuda()
    with mlh.LMHead(n, k, max_batch=b, device=0, fmt=fmt) as head:
        call = lambda g: head.backward(g, wq, hidden=hidden, gamma=gamma, scale=0.7, cap=0.0)       # noqa: E731
        want = []
        for g in grads:
            out = call(g)
            torch.cuda.synchronize()
            want.append([t.clone() for t in out])
        got = [(i % 3, call(grads[i % 3])) for i in range(300)]
        torch.cuda.synchronize()
        assert head.device_status() == 0
    for i, out in got:
        assert all(torch.equal(p, q) for p, q in zip(out, want[i]))


def test_backward_nan_and_infinity_stay_in_their_row(torch_cuda):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    b, n, k = 4, 1001, 512
    rng = np.random.default_rng(8)
    w = torch.from_numpy(np.ascontiguousarray(_weights(n, k, "q5_k", 16))).cuda()
    g = torch.from_numpy(_grads(rng, b, n)).cuda()
    bad = g.clone()
    bad[1, 77], bad[2, 500] = float("nan"), float("inf")
    with mlh.LMHead(n, k, max_batch=b, device=0) as head:
        want, _ = head.backward(g, w, scale=1.0, cap=0.0)
        got, _ = head.backward(bad, w, scale=1.0, cap=0.0)
        torch.cuda.synchronize()
        assert head.device_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])
    assert not bool(got[1].isfinite().any()) and not bool(got[2].isfinite().any())


def test_backward_refuses_its_first_call_in_a_capture(torch_cuda):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    n, k = 512, 256
    w = torch.zeros(n * 176, dtype=torch.uint8, device="cuda")
    g = torch.zeros((1, n), device="cuda")
    s = torch.cuda.Stream()
    with mlh.LMHead(n, k, max_batch=1, device=0) as head:
        with torch.cuda.stream(s):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                with pytest.raises(mlh.MuseError) as err:
                    head.backward(g, w, cap=0.0)
                g.add_(0.0)                          # the capture goes on
            assert err.value.status == -8
            head.backward(g, w, cap=0.0)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                out, _ = head.backward(g, w, cap=0.0)
            graph.replay()
        torch.cuda.synchronize()
    assert not out.any()


def test_backward_first_call_beside_another_streams_capture(torch_cuda):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    n, k = 512, 256
    w = torch.zeros(n * 176, dtype=torch.uint8, device="cuda")
    g = torch.zeros((1, n), device="cuda")
    out = torch.ones((1, k), device="cuda")
    x = torch.ones(8, device="cuda")
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with mlh.LMHead(n, k, max_batch=1, device=0) as head:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            x.add_(1.0)
            head.backward(g, w, cap=0.0, grad_hidden=out, stream=other)   # allocates; runs at once on its stream
        torch.cuda.synchronize()
        assert not bool(out.any())
        graph.replay()
        torch.cuda.synchronize()
        assert bool((x == 2.0).all())


def test_backward_with_a_cap_whose_square_overflows(torch_cuda):
    """The slope is 1 to 4 roundings there: against the call without a cap."""
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    b, n, k = 3, 700, 512
    rng = np.random.default_rng(5)
    wq, g = _weights(n, k, "q5_k", 5), _grads(rng, b, n)
    w, gl = torch.from_numpy(wq).cuda(), torch.from_numpy(g).cuda()
    logits = torch.randn((b, n), device="cuda")
    want, tol, _, _ = _reference(g, None, None, None, _dense(wq, n, k, "q5_k"), 1.0, 0.0)
    with mlh.LMHead(n, k, max_batch=b, device=0) as head:
        for cap in (1e20, 1e30, 3e38):
            got, _ = head.backward(gl, w, logits=logits, scale=1.0, cap=cap)
            _within(f"cap {cap}", got.cpu().numpy(), want, tol)


def test_backward_small_gradients_beside_a_large_one_without_weights(torch_cuda):
    """The f16 pair of a gradient ends at 2^-24 where the row's largest lies at 2^11 or above: what it
    drops is at most 2^-35 of the largest, times each weight's parts."""
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    n, k = 600, 512
    rng = np.random.default_rng(6)
    wq = _weights(n, k, "q5_k", 6).reshape(n, -1).copy()
    wq[7] = 0
    g = (rng.standard_normal((1, n)) * 2.0 ** -22).astype(np.float32)
    g[0, 7] = 3.0
    dense = _dense(wq, n, k, "q5_k")
    want, tol, _, _ = _reference(g, None, None, None, dense, 1.0, 0.0)
    tol = tol + 2.0 ** -34 * 3.0 * dense[1].sum(0)[None]       # once in the pair, once in its product with a block's factor
    with mlh.LMHead(n, k, max_batch=1, device=0) as head:
        got, _ = head.backward(torch.from_numpy(g).cuda(), torch.from_numpy(wq.reshape(-1)).cuda(), scale=1.0, cap=0.0)
        _within("grad_hidden", got.cpu().numpy(), want, tol)


@pytest.mark.parametrize("fmt", ["q5_k", "q4_k"])
def test_backward_batches_of_every_size_on_one_handle_eager_and_replayed(torch_cuda, fmt):
    """The workspace is laid out for max_batch: every batch size gives the bits of a handle of its own."""
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    n, k = 1100, 768
    rng = np.random.default_rng(11)
    w = torch.from_numpy(_weights(n, k, fmt, 11)).cuda()
    gamma = torch.randn(k, device="cuda")
    stream = torch.cuda.Stream()
    with mlh.LMHead(n, k, max_batch=32, device=0, fmt=fmt) as head:
        calls = []
        for b in (3, 32, 1, 17, 8, 9, 16, 2):
            g, lo = torch.from_numpy(_grads(rng, b, n)).cuda(), torch.randn((b, n), device="cuda") * 5
            h = torch.randn((b, k), device="cuda")
            with mlh.LMHead(n, k, max_batch=b, device=0, fmt=fmt) as own:
                want = own.backward(g, w, logits=lo, hidden=h, gamma=gamma, cap=20.0)
                torch.cuda.synchronize()
            calls.append((g, lo, h, want))
            got = head.backward(g, w, logits=lo, hidden=h, gamma=gamma, cap=20.0)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                outs = [head.backward(g, w, logits=lo, hidden=h, gamma=gamma, cap=20.0) for g, lo, h, _ in calls]
            for _ in range(3):
                for a, c in outs:
                    a.fill_(7.0)
                    c.fill_(7.0)
                graph.replay()
        torch.cuda.synchronize()
        for (a, c), (_, _, _, want) in zip(outs, calls):
            assert torch.equal(a, want[0]) and torch.equal(c, want[1])
        assert head.device_status() == 0


def test_backward_of_two_handles_on_two_streams(torch_cuda):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    rng = np.random.default_rng(13)
    cases, streams = [(5, 9000, 1024, "q5_k"), (20, 4000, 2560, "q4_k")], [torch.cuda.Stream(), torch.cuda.Stream()]
    heads, args, want = [], [], []
    for b, n, k, fmt in cases:
        heads.append(mlh.LMHead(n, k, max_batch=b, device=0, fmt=fmt))
        g, lo = torch.from_numpy(_grads(rng, b, n)).cuda(), torch.randn((b, n), device="cuda") * 5
        args.append((g, torch.from_numpy(_weights(n, k, fmt, 13)).cuda(), lo, torch.randn((b, k), device="cuda"),
                     torch.randn(k, device="cuda")))
    try:
        for head, a in zip(heads, args):
            want.append(head.backward(*a, cap=20.0))
        torch.cuda.synchronize()
        got = [[], []]
        for _ in range(20):
            for i in (0, 1):
                out = torch.empty_like(want[i][0])
                with torch.cuda.stream(streams[i]):
                    got[i].append(heads[i].backward(*args[i], cap=20.0, grad_hidden=out))
        torch.cuda.synchronize()
        for i in (0, 1):
            assert all(torch.equal(x, want[i][0]) and torch.equal(y, want[i][1]) for x, y in got[i])
            assert heads[i].device_status() == 0
    finally:
        for head in heads:
            head.close()
