"""GPU parity of muse_lmhead_distill: loss and gradient of a distillation from a
teacher's top alternatives, against the formulas in 64 bits and the gradient
against differences of the loss.

Tolerances (u = 2^-24): a sum of the row's exponentials is off by at most
t = (V/256 + 80) u relative, as for the scores; so is q, and log q by t plus
2u (|z| + |log q|).  A loss is a sum of p-weighted differences of logarithms:
off by w (2t + 8u (1 + largest |log|)) with p's own rounding 40u p |log| under
the same bound.  A gradient element w/T (F q - p - ...): w/T (2t + 40u)(F q + p + pt q/qt),
then one rounding to the logits' type, half a step (eps/2 relative, or half the
smallest subnormal).
"""
import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = ("float32", "float16", "bfloat16")


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    return torch


def _reference(torch, x, ids, lp, weight, temperature, tail):
    """Row by row in 64 bits on the CPU; also the sizes that the tolerances need."""
    n, v = x.shape
    loss, grad = torch.zeros(n, dtype=torch.float64), torch.zeros((n, v), dtype=torch.float64)
    size, big = torch.zeros((n, v), dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    for r in range(n):
        w = 1.0 if weight is None else float(weight[r])
        if w == 0.0 or float(x[r].max()) == -math.inf:
            continue
        z = x[r] / temperature
        logq = z - torch.logsumexp(z, dim=0)
        q = logq.exp()
        ent = [(int(i), float(l)) for i, l in zip(ids[r].tolist(), lp[r].tolist()) if 0 <= i < v]
        raw = torch.tensor([l for _, l in ent], dtype=torch.float64)
        p = raw.exp() if tail else torch.softmax(raw, dim=0) if len(ent) and float(raw.max()) > -math.inf else raw * 0
        p = torch.nan_to_num(p, nan=0.0)
        total = float(p.sum())
        pt = max(0.0, 1.0 - total) if tail else 0.0
        g = (total + pt) * q
        sz = (total + pt) * q
        out = torch.ones(v, dtype=torch.float64)
        for (i, _), pj in zip(ent, p.tolist()):
            g[i] -= pj
            sz[i] += pj
            out[i] = 0.0
            if pj > 0:
                loss[r] += pj * (math.log(pj) - float(logq[i]))
                big[r] = max(big[r], abs(math.log(pj)), abs(float(logq[i])) if math.isfinite(logq[i]) else 0.0)
        if pt > 0:
            qt = float((q * out).sum())
            big[r] = max(big[r], abs(math.log(pt)), abs(math.log(qt)) if qt > 0 else 0.0)
            loss[r] += pt * (math.log(pt) - (math.log(qt) if qt > 0 else -math.inf))
            if qt > 0:
                g -= out * q * (pt / qt)
                sz += out * q * (pt / qt)
        zabs = z[z.isfinite()].abs().max()
        big[r] = big[r] + zabs
        loss[r] *= w
        grad[r] = g * (w / temperature)
        size[r] = sz * (abs(w) / temperature)
    return loss, grad, size, big


def _check(torch, head, x, ids, lp, weight=None, temperature=1.0, tail=False, in_place=False):
    ref_loss, ref_grad, size, big = _reference(torch, x.double().cpu(), ids.cpu(), lp.double().cpu(),
                                               None if weight is None else weight.cpu(), temperature, tail)
    alone, none = head.distill(x, ids, lp, weight, temperature, tail, want_grad=False)
    assert none is None
    loss, grad = head.distill(x, ids, lp, weight, temperature, tail, grad=x if in_place else None)
    torch.cuda.synchronize()
    assert grad.dtype == x.dtype
    v = x.shape[1]
    t = (v / 256 + 80) * U
    # an exp's argument (x - m)/T carries 3u |dz|, dz up to the row's spread
    spread = 3 * U * 2 * big
    w = torch.ones_like(ref_loss) if weight is None else weight.double().abs().cpu()
    fin = ref_loss.isfinite()
    tol = w * (2 * t + 8 * U * (1 + big)) + 45 * U * w * (1 + big)
    for got in (alone.cpu().double(), loss.cpu().double()):
        assert bool((got[~fin] == ref_loss[~fin]).all())
        err = (got - ref_loss).abs()[fin]
        assert bool((err <= tol[fin]).all()), f"loss off by {float(err.max()):.3g}, allowed {float(tol[fin][err.argmax()]):.3g}"
    info = torch.finfo(x.dtype)
    tol = (2 * t + 40 * U + spread[:, None]) * size + info.eps / 2 * ref_grad.abs() * (1 + 1e-3) + info.smallest_normal * info.eps
    err = (grad.double().cpu() - ref_grad).abs()
    over = err - tol
    assert bool((over <= 0).all()), f"gradient off by {float(err.flatten()[over.argmax()]):.3g} at {int(over.argmax())}, allowed {float(tol.flatten()[over.argmax()]):.3g}"


def _case(torch, n, v, top, dtype, pad=0, offset=0, seed=0, dup=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 31 * n + v)
    dev = "cuda"
    flat = torch.randn((offset + n * (v + pad),), generator=g, device=dev) * 3
    x = torch.as_strided((20 * torch.tanh(flat / 20)).to(dtype), (n, v), (v + pad, 1), offset)
    ids = torch.rand((n, max(v, top)), generator=g, device=dev).argsort(dim=1)[:, :top]    # beyond v: left out
    if dup:
        ids[:, 1::2] = ids[:, 0:1]
    lp = torch.log_softmax(torch.randn((n, top), generator=g, device=dev) * 2, dim=1) + math.log(0.85)
    w = torch.rand((n,), generator=g, device=dev) + 0.5
    return x, ids.to(torch.int32).contiguous(), lp.contiguous(), w


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("n,v,top,pad,offset,temperature", [
    (1, 2, 1, 0, 0, 1.0), (3, 5, 4, 1, 1, 0.5), (2, 7, 64, 0, 0, 1.0), (4, 257, 3, 2, 3, 1.0), (33, 1000, 20, 0, 0, 2.0),
    (5, 2048, 64, 0, 0, 1.0), (7, 4099, 16, 1, 1, 1.0), (3, 32003, 16, 0, 0, 1.0), (2, 50257, 33, 3, 2, 2.0),
    (170, 6007, 5, 0, 0, 1.0), (2, 202048, 32, 0, 0, 1.0), (1, 202048, 64, 0, 0, 2.0), (1, 260003, 8, 0, 0, 1.0),
    (2, 500001, 20, 1, 1, 1.0), (2, 2000003, 20, 0, 0, 1.0)])
def test_distill_shapes(torch_cuda, dtype, tail, n, v, top, pad, offset, temperature):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    x, ids, lp, w = _case(torch, n, v, top, getattr(torch, dtype), pad, offset)
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        _check(torch, head, x, ids, lp, None, temperature, tail)
        _check(torch, head, x, ids, lp, w, temperature, tail, in_place=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("v", [70, 3001, 100003])
def test_distill_padding_masks_and_duplicates(torch_cuda, dtype, tail, v):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    dt = getattr(torch, dtype)
    x, ids, lp, w = _case(torch, 9, v, 8, dt)
    ids[0, 3:] = -1                                # a shorter teacher
    ids[1, :] = -5                                 # none at all
    ids[2, 2] = v                                  # out of range
    lp[3, 4:] = -math.inf                          # given, with no probability
    lp[4, :] = -math.inf
    w[5] = 0.0
    x[5, 1] = math.nan                             # a row of weight 0 may hold anything
    x[6] = -math.inf                               # a row without a distribution
    x[7] = torch.finfo(dt).min                     # a mask of the lowest value on everything: uniform
    keep = x[8, ids[8].long()].clone()
    x[8] = -math.inf                               # everything but the teacher's ids masked
    x[8, ids[8].long()] = keep
    lp[8] = torch.log_softmax(lp[8], dim=0) + 0.0
    if tail:
        lp[8] += 1e-3                              # its mass is over 1: no tail is left
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        _check(torch, head, x, ids, lp, w, 1.0, tail)
        x2, ids2, lp2, w2 = _case(torch, 4, v, 8, dt, dup=True)
        lp2 = lp2 - math.log(2.0)
        _check(torch, head, x2, ids2, lp2, w2, 1.5, tail)
        xm = x2.clone()
        xm[0, int(ids2[0, 0])] = -math.inf         # the teacher expects a masked token
        loss, grad = head.distill(xm, ids2, lp2, w2, 1.5, tail)
        assert float(loss[0]) == math.inf and bool(grad.isfinite().all()) and bool(loss[1:].isfinite().all())
        _check(torch, head, xm, ids2, lp2, w2, 1.5, tail)


def test_distill_nan_and_infinity_stay_in_their_row(torch_cuda):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    v = 20011
    x, ids, lp, w = _case(torch, 4, v, 8, torch.float32)
    bad = x.clone()
    bad[1, 7], bad[2, 9] = math.nan, math.inf
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        loss, grad = head.distill(bad, ids, lp, w)
        want, wgrad = head.distill(x, ids, lp, w)
    assert bool(loss[1:3].isnan().all()) and bool(grad[1:3].isnan().any(dim=1).all())
    for r in (0, 3):
        assert torch.equal(loss[r], want[r]) and torch.equal(grad[r], wgrad[r])


@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_against_differences(torch_cuda, tail):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    v, h = 24, 2.0 ** -6
    x, ids, lp, w = _case(torch, 2, v, 5, torch.float32)
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        _, grad = head.distill(x, ids, lp, w, 1.3, tail)
        for i in range(v):
            a, b = x.clone(), x.clone()
            a[:, i] += h
            b[:, i] -= h
            d = (head.distill(a, ids, lp, w, 1.3, tail, want_grad=False)[0].double()
                 - head.distill(b, ids, lp, w, 1.3, tail, want_grad=False)[0].double()) / ((a - b)[:, i].double())
            # second-order term: |third derivative| <= w/T^3, h^2/6 of it; each loss is off by 200u w at most
            tol = w.double() * (h * h / 6 / 1.3 ** 3 + 200 * U / h)
            assert bool(((d - grad[:, i].double()).abs() <= tol).all())


def test_distill_leaves_what_is_beside_the_rows(torch_cuda):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    n, v, ld = 5, 3001, 3011
    x, ids, lp, w = _case(torch, n, v, 8, torch.bfloat16)
    out = torch.full((n + 1, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        _, grad = head.distill(x, ids, lp, w)
        head.distill(x, ids, lp, w, grad=out[:n, 3:3 + v])
        assert head.distill(x[:0], ids[:0], lp[:0])[0].shape == (0,)
    assert torch.equal(out[:n, 3:3 + v], grad)
    assert bool((out[n] == 7).all()) and bool((out[:, :3] == 7).all()) and bool((out[:, 3 + v:] == 7).all())


def test_distill_offsets_past_32_bits(torch_cuda):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    v, n = 202048, 10700                           # 2.16e9 elements
    x = torch.zeros((n, v), dtype=torch.float16, device="cuda")
    few, ids4, lp4, w4 = _case(torch, 3, v, 4, torch.float16)
    rows = [0, n - 2, n - 1]
    x[rows] = few
    ids = torch.zeros((n, 4), dtype=torch.int32, device="cuda")
    lp = torch.full((n, 4), -2.0, device="cuda")
    ids[rows], lp[rows] = ids4, lp4
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        want, wgrad = head.distill(few, ids4, lp4, tail=True)
        loss, grad = head.distill(x, ids, lp, tail=True, grad=x)
        torch.cuda.synchronize()
    assert float((loss[rows] - want).abs().max()) <= (v / 256 + 80) * U * 4 + 200 * U
    assert float((grad[rows].float() - wgrad.float()).abs().max()) <= 2.0 ** -11


def test_distill_in_a_graph_and_on_two_streams(torch_cuda):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    n, v = 3, 50257
    sets = [_case(torch, n, v, 9, torch.bfloat16, seed=s) for s in (1, 2)]
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        want = [[t.clone() for t in head.distill(*c, tail=True)] for c in sets]
        hold = [t.clone() for t in sets[0]]
        s, other = torch.cuda.Stream(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            head.distill(*hold, tail=True)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                got = head.distill(*hold, tail=True)
        torch.cuda.synchronize()
        for k in (0, 1, 0):
            for a, b in zip(hold, sets[k]):
                a.copy_(b)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want[k]))
        res = []
        for _ in range(10):
            with torch.cuda.stream(s):
                res.append((head.distill(*sets[0], tail=True), want[0]))
            with torch.cuda.stream(other):
                res.append((head.distill(*sets[1], tail=True), want[1]))
        torch.cuda.synchronize()
        for r, ref in res:
            assert all(torch.equal(p, q) for p, q in zip(r, ref))


def test_distill_back_to_back_behind_a_forward(torch_cuda):
    """Forward and distillation one behind another: each loss has to come from its own forward's logits."""
    import numpy as np
    import q5_lm_head_gb300 as mlh
    import q5k_synth as synth
    torch = torch_cuda
    wl = synth.WORKLOADS["tiny"]
    hidden, gamma, wq = synth.inputs_for(wl)
    w, g = torch.from_numpy(np.ascontiguousarray(wq)).cuda(), torch.from_numpy(gamma).cuda()
    rows = [torch.from_numpy((hidden * s).astype(np.float32)).cuda() for s in (1.0, 0.3, -2.0)]
    for r in rows[1:]:
        r += torch.arange(wl.k, device="cuda") % 3
    _, ids, lp, _ = _case(torch, 1, wl.n_rows, 12, torch.float32)
    with mlh.LMHead(wl.n_rows, wl.k, max_batch=1, device=0) as head:
        logits = torch.empty((1, wl.n_rows), device="cuda")

        def call(h):
            head.forward(h, w, g, logits=logits)
            return head.distill(logits, ids, lp, tail=True)

        want = []
        for h in rows:
            out = call(h)
            torch.cuda.synchronize()
            want.append([t.clone() for t in out])
        got = [(i % 3, call(rows[i % 3])) for i in range(300)]
        torch.cuda.synchronize()
    for i, out in got:
        assert all(torch.equal(p, q) for p, q in zip(out, want[i]))


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("v", [5000, 300000, 2000003])
def test_distill_masks_of_the_lowest_value_at_low_temperature(torch_cuda, tail, v):
    """Exponents of lowest values overflow f32 at temperature 0.5; the loss of a row whose teacher
    expects none of them is the one with -infinity in their place, and the gradient everywhere."""
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    x, ids, lp, w = _case(torch, 3, v, 16, torch.float32)
    mask = torch.rand(x.shape, generator=torch.Generator(device="cuda").manual_seed(v), device="cuda") < 0.5
    mask.scatter_(1, ids.long().clamp(0, v - 1), False)
    low = x.masked_fill(mask, torch.finfo(torch.float32).min)
    inf = x.masked_fill(mask, -math.inf)
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        _check(torch, head, inf, ids, lp, w, 0.5, tail)
        want = head.distill(inf, ids, lp, w, 0.5, tail)
        got = head.distill(low, ids, lp, w, 0.5, tail)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # and one that the teacher does expect: a finite loss, as large as its logit
        low[1, int(ids[1, 0])] = torch.finfo(torch.float32).min
        lp = torch.full_like(lp, math.log(0.05))
        loss, grad = head.distill(low, ids, lp, None, 2.0, tail)
        torch.cuda.synchronize()
        p = 0.05 if tail else 1 / 16
        assert abs(float(loss[1]) / (p * torch.finfo(torch.float32).max / 2.0) - 1) < 1e-5
        assert bool(grad.isfinite().all())
