"""Masks of large finite values, and logits of any size: -1e9, -1e10, -1e20 and their like,
f16's -65504 at temperatures of 1e-5, rows of values about 7e5 or 1e8 that differ by
a few.  A share of a row may hold nothing but masks.  References in 64 bits, by
differences from the row's maximum.

Tolerance (u = 2^-24): as for scores and distillation: a sum is off by
t = (V/256 + 80) u and by 3u of the exponents of the values that carry it, which
are below 32: 100u more; 2u of the size of a value or normaliser; a loss by
2t + 200u + 45u (1 + its largest logarithm), a gradient by 2t + 200u + 6u of its
exponent, of the sizes of its terms, and half a step of its type.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    return torch


def _check(torch, x, temperature, top=5):
    import q5_lm_head_gb300 as mlh
    n, v = x.shape
    temperature = float(torch.tensor(temperature, dtype=torch.float32))
    k = min(top, v)
    t = (v / 256 + 80) * U + 100 * U
    order = torch.sort(x.float() + 0.0, dim=1, descending=True, stable=True).indices
    tokens = order[:, min(2, v - 1)].to(torch.int32).contiguous()
    d = x.double() - x.double().max(dim=1, keepdim=True).values
    dz = d / temperature
    logs = dz.exp().sum(dim=1, keepdim=True).log()
    logp = dz - logs
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(dim=1)
    lse = x.double().max(dim=1).values / temperature + logs[:, 0]
    size = lambda w: torch.where(w.isfinite(), w.abs(), torch.zeros_like(w))               # noqa: E731
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        out = head.score(x, tokens, k, temperature)
        # the teacher's entries: the row's first values, and nearly all of the probability
        ids = order[:, :k].to(torch.int32).contiguous()
        teacher = torch.log_softmax(torch.randn((n, k), generator=torch.Generator().manual_seed(v)), dim=1).cuda() + math.log(0.9)
        results = {tail: head.distill(x, ids, teacher, None, temperature, tail) for tail in (False, True)}
        torch.cuda.synchronize()

    def close(name, got, want, tol):
        got = got.double()
        want = torch.where(want < -3.4028236e38, torch.full_like(want, -math.inf), want)
        fin = want.isfinite()
        assert bool((got[~fin] == want[~fin]).all()), name
        err = (got - want)[fin].abs()
        assert bool((err <= tol[fin]).all()), f"{name}: {got[fin][(err - tol[fin]).argmax()]:.9g}, should be {want[fin][(err - tol[fin]).argmax()]:.9g}"

    close("lse", out.lse, lse, t + 2 * U * size(lse))
    close("entropy", out.entropy, entropy, t * (4 + math.log(v)) + 0 * entropy)
    lp = logp.gather(1, tokens.long()[:, None])[:, 0]
    close("logprob", out.logprob, lp, t + 2 * U * size(lp))
    top_lp = logp.gather(1, order[:, :k])
    close("top", out.top_logprobs, top_lp, t + 2 * U * size(top_lp))
    assert torch.equal(out.top_ids.long(), order[:, :k]) and bool((out.rank == min(2, v - 1)).all())

    info = torch.finfo(x.dtype)
    rest = torch.ones((n, v), dtype=torch.bool, device="cuda")
    rest.scatter_(1, order[:, :k], False)
    for tail, (loss, grad) in results.items():
        lt = teacher.double() if tail else torch.log_softmax(teacher.double(), dim=1)
        pt = lt.exp()
        left = (1 - pt.sum(dim=1)) * (1.0 if tail else 0.0)
        want = (pt * (lt - top_lp)).sum(dim=1)
        big = torch.maximum(lt.abs().amax(dim=1), size(top_lp).amax(dim=1))
        total = (pt.sum(dim=1) + left)[:, None]
        g, s = total * p, total * p
        g, s = g.scatter_add(1, order[:, :k], -pt), s.scatter_add(1, order[:, :k], pt)
        far = size(d)
        if tail and v > k:
            o = d.masked_fill(~rest, -math.inf)
            most = o.max(dim=1, keepdim=True).values
            e = ((o - most) / temperature).exp()
            r = e.sum(dim=1, keepdim=True)
            logq = most / temperature + r.log() - logs
            want = want + left * (left.log() - logq[:, 0])
            big = torch.maximum(big, size(logq[:, 0]))
            g, s = g - left[:, None] * e / r, s + left[:, None] * e / r
            far = torch.where(rest, size(o - most), far)
        elif tail:
            continue                              # nothing but the teacher's entries: no class for the rest
        far = (far / temperature).clamp(max=100.0)
        close(f"loss {tail}", loss, want, 2 * t + 200 * U + 45 * U * (1 + big))
        tol = (2 * t + 200 * U + 6 * U * far) * s + info.eps / 2 * (g.abs() + 1e-30) * 1.001 + info.smallest_normal * info.eps * temperature
        if 1 / temperature < 1000:                # below, 16 bits do not hold the gradient
            close(f"grad {tail}", (grad.double() * temperature).flatten(), g.flatten(), (tol + 2.0 ** -125).flatten())
        else:
            assert not bool(grad.isnan().any())


def _rows(torch, v, dtype, mask):
    """Masks on nearly everything, on one value in two, on one block, on everything but the last."""
    g = torch.Generator(device="cuda").manual_seed(v)
    x = torch.randn((5, v), generator=g, device="cuda") * 3
    u = torch.rand((5, v), generator=g, device="cuda")
    at = torch.arange(v, device="cuda")
    x[0].masked_fill_(u[0] < 0.999, mask)
    x[1].masked_fill_(u[1] < 0.5, mask)
    x[2].masked_fill_((at < v // 3) | (at > v // 2), mask)
    x[3].masked_fill_(at < v - 6, mask)
    x[4] = mask
    x[:, v // 2] = 1.0
    x[4, v // 2] = mask
    return x.to(getattr(torch, dtype))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("mask", [-1e4, -1e8, -1e9, -1e10, -1.3e11, -1e15, -1e20, -7.7e25, -9e29, -1e30, -1e31, -1e38])
@pytest.mark.parametrize("v", [700, 50257])
def test_masks_of_large_finite_values(torch_cuda, dtype, mask, v):
    torch = torch_cuda
    for temperature in (1.0, 0.3):
        _check(torch, _rows(torch, v, dtype, mask), temperature)


@pytest.mark.parametrize("v", [80, 4099, 202048])
@pytest.mark.parametrize("temperature", [2.0 ** -20, 5e-6, 1e-5, 1e-3])
def test_lowest_f16_at_low_temperature(torch_cuda, v, temperature):
    torch = torch_cuda
    _check(torch, _rows(torch, v, "float16", -65504.0), temperature)
    _check(torch, _rows(torch, v, "float16", -600.0), temperature)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("about,spread", [(726817.4, 20.0), (7.3e5, 3.0), (93032639.0, 40.0), (9.3e7, 200.0), (1e8, 64.0), (1e9, 300.0),
                                          (1e12, 3e5), (6.9e29, 1e23)])
@pytest.mark.parametrize("v", [300, 50257])
def test_rows_of_large_values_that_differ_by_little(torch_cuda, sign, about, spread, v):
    """Both sides of where a reference's product with log2(e) is used rounded (2^20 and 2^27 among them)."""
    torch = torch_cuda
    g = torch.Generator(device="cuda").manual_seed(v)
    x = (sign * about + spread * torch.randn((3, v), generator=g, device="cuda", dtype=torch.float64)).float()
    x[1, : v // 2] = sign * about
    x[2, v // 4:] = -1e20
    _check(torch, x, 1.0)
    _check(torch, x, 4.0)


def test_rows_of_large_values_read_by_one_cta(torch_cuda):
    torch = torch_cuda
    for mask in (-1e10, -1e20):
        _check(torch, _rows(torch, 2000003, "float32", mask), 1.0)
