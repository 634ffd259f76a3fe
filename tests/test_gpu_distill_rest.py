"""The class for all tokens that the teacher does not name, where the student puts
nearly nothing on it: its probability underflows in 32 bits against the row's
maximum, its logarithm and its shares do not.

The reference works on logarithms in 64 bits: log q_t = lse(z outside) - lse(z),
the gradient outside the ids F q_i - p_t softmax(z outside)_i.

Tolerances (u = 2^-24): a sum of exponentials against its own maximum is off by
t = (V/256 + 80) u relative, as for the scores, and where its values carry weight
their exponents are below 32 in size and off by 3u of it: 100u more.  p_t = 1 - sum p of
64 entries at most, each good to 6u relative: 6u absolute, 60u of the p_t >= 0.1
here.  A loss is then off by w (2t + 200u) and 45u w (1 + the largest logarithm)
for the roundings of p and of the result; an element of the gradient by
2t + 200u + 6u |its exponent| of the sizes of its terms, by half a step of its
type and by what the exponentials flush (2^-126 of w/T).
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
    """loss, grad, its terms' size, its exponents' size, the largest logarithm; rows in 64 bits."""
    n, v = x.shape
    z = x.double() / temperature
    lse = torch.logsumexp(z, dim=1)
    loss, big = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    grad, size, far = (torch.zeros((n, v), dtype=torch.float64) for _ in range(3))
    for r in range(n):
        at, l = ids[r].long(), lp[r].double()
        p = l.exp() if tail else torch.softmax(l, dim=0)
        out = torch.ones(v, dtype=torch.bool)
        out[at] = False
        logq = z[r] - lse[r]
        q = logq.exp()
        pt = max(0.0, 1.0 - float(p.sum())) if tail else 0.0
        f = float(p.sum()) + pt
        g, s = f * q, f * q
        g.index_add_(0, at, -p)
        s.index_add_(0, at, p)
        logs = [p.log(), logq[at]]
        loss[r] = (p * (p.log() - logq[at])).sum()
        rest = torch.logsumexp(z[r][out], dim=0)
        if pt > 0:
            share = torch.where(out, (z[r] - rest).exp(), torch.zeros_like(q))
            g, s = g - pt * share, s + pt * share
            loss[r] += pt * (math.log(pt) - float(rest - lse[r]))
            logs.append((rest - lse[r])[None])
        big[r] = max(float(t.abs().max()) for t in logs)
        top = torch.where(out, z[r][out].max(), z[r].max())
        far[r] = torch.where(z[r].isfinite(), (z[r] - top).abs(), torch.zeros_like(q))
        w = 1.0 if weight is None else float(weight[r])
        loss[r], grad[r], size[r] = loss[r] * w, g * (w / temperature), s * (abs(w) / temperature)
    return loss, grad, size, far, big


def _check(torch, x, ids, lp, weight, temperature, tail=True):
    import q5_lm_head_gb300 as mlh
    n, v = x.shape
    want, grad, size, far, big = _reference(torch, x.cpu(), ids.cpu(), lp.cpu(), None if weight is None else weight.cpu(), temperature, tail)
    assert bool(want.isfinite().all())
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        alone, _ = head.distill(x, ids, lp, weight, temperature, tail, want_grad=False)
        loss, got = head.distill(x, ids, lp, weight, temperature, tail)
        torch.cuda.synchronize()
    t = (v / 256 + 80) * U
    w = torch.ones(n, dtype=torch.float64) if weight is None else weight.cpu().double().abs()
    tol = w * (2 * t + 200 * U + 45 * U * (1 + big))
    for one in (alone, loss):
        err = (one.cpu().double() - want).abs()
        assert bool((err <= tol).all()), f"loss {one.tolist()}, should be {want.tolist()}"
    info = torch.finfo(x.dtype)
    tol = (2 * t + 200 * U + 6 * U * far) * size + info.eps / 2 * grad.abs() * (1 + 1e-3) + info.smallest_normal * info.eps
    tol = tol + (w / temperature * 2.0 ** -125)[:, None]
    got = got.cpu().double()
    assert bool(got.isfinite().all()), "gradient not finite"
    over = (got - grad).abs() - tol
    at = int(over.argmax())
    assert bool((over <= 0).all()), f"gradient {float(got.flatten()[at]):.6g} at {at}, should be {float(grad.flatten()[at]):.6g}"


def _rows(torch, v, dtype, high, low, places, masked, seed=0):
    """Rows of values around `low` (at most as much above as below), of which some are masked, with
    `high` (a value an entry) at `places`; teacher entries on these with 0.9 of the probability."""
    g = torch.Generator().manual_seed(v + seed)
    n, k = len(places), len(high)
    x = low + torch.randn((n, v), generator=g).clamp(-3, 3)
    if masked:
        x[torch.rand((n, v), generator=g) < 0.4] = -math.inf
        x[:, v // 2] = low
    ids = torch.tensor([[p % v for p in row] for row in places])
    for r in range(n):
        x[r, ids[r]] = torch.tensor(high, dtype=torch.float32)
    lp = torch.log_softmax(torch.randn((n, k), generator=g), dim=1) + math.log(0.9)
    return x.to(getattr(torch, dtype)).cuda(), ids.to(torch.int32).cuda(), lp.cuda()


# places of the ids: together, in one warp, far apart, in the first and last values
PLACES = [(0, 1, 2), (3, 40, 9), (5, 1000, 60000), (7, 199999, 100001), (202047, 202046, 0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("temperature", [0.05, 0.1, 0.2, 0.25])
@pytest.mark.parametrize("v", [70, 3001, 202048])
def test_rest_of_capped_logits_at_low_temperature(torch_cuda, dtype, masked, temperature, v):
    """19 against about -5, and two middling ids between them: a few hundred binary orders."""
    torch = torch_cuda
    temperature = float(torch.tensor(temperature, dtype=torch.float32))
    x, ids, lp = _rows(torch, v, dtype, (19.0, 9.5, 2.0), -5.0, PLACES, masked)
    keep = [r for r in range(len(PLACES)) if len(set(ids[r].tolist())) == 3]
    w = torch.tensor([1.0, 0.5, 2.0, 0.03, 1.0], device="cuda")
    _check(torch, x[keep], ids[keep], lp[keep], w[keep], temperature)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gap", [20, 60, 80, 86, 87, 88, 89, 95, 100, 103, 104, 130, 300, 600])
@pytest.mark.parametrize("v", [257, 50257])
def test_rest_far_below_the_ids_without_a_cap(torch_cuda, dtype, gap, v):
    torch = torch_cuda
    for masked in (False, True):
        for high in ((gap / 2, gap / 2 - 40.0, 0.0), (gap / 2, gap / 4, -gap / 4), (gap / 2,) * 3):
            x, ids, lp = _rows(torch, v, dtype, high, -gap / 2, PLACES[:4], masked, seed=gap)
            keep = [r for r in range(4) if len(set(ids[r].tolist())) == 3]
            _check(torch, x[keep], ids[keep], lp[keep], None, 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gap", [60, 90, 104, 300])
def test_rest_of_rows_read_by_one_cta(torch_cuda, dtype, gap):
    """More values than a cluster holds."""
    torch = torch_cuda
    x, ids, lp = _rows(torch, 2000003, dtype, (gap / 2, 0.0, -gap / 4), -gap / 2, [(5, 1000, 60000), (7, 1999999, 100001)], gap != 90)
    _check(torch, x, ids, lp, None, 1.0)
    _check(torch, x, ids, lp, None, 0.25)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rest_above_the_ids(torch_cuda, dtype, tail):
    """The other way round: the ids lie hundreds of binary orders below the rest."""
    torch = torch_cuda
    for v in (3001, 202048, 2000003):
        x, ids, lp = _rows(torch, v, dtype, (-100.0, -130.0, -7.0), 8.0, PLACES[1:3], True)
        _check(torch, x, ids, lp, None, 1.0, tail)
        _check(torch, x, ids, lp, None, 0.25, tail)
