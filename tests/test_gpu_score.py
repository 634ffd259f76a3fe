"""GPU parity of muse_lmhead_score and muse_lmhead_forward_score: token
logprobs, ranks, normaliser, entropy and top alternatives of rows of logits,
against the formulas in 64 bits ("Chapter 20 — Final norm, LM head, and the
soft cap", §20.7: softmax and logprobs over the capped logits).

Tolerances, derived from the arithmetic: u = 2^-24 is half a step of f32 at 1.
dz = (x - m)/T carries three roundings (3u |dz|) and its exp two units in the
last place more (4u), and e^dz |dz| <= 1/e, so an addend is off by at most 6u of
the sum's largest; a running sum of L addends is off by at most L u, and no
kernel adds more than V/256 + 64 in a chain.  So S is off by at most
t = (V/256 + 80) u relative, log S by t absolute, lse and logprobs by t plus two
roundings of the values (2u |value|) and of m/T (2u |m/T|); U/S (at most
log V + 1 in size, 14 at these sizes) by 2 t 14.  Ranks and ids are exact.
"""
import math

import numpy as np
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


def _reference(torch, x, tokens, n_top, temperature):
    """x: [n, v] float64 on the CPU."""
    n, v = x.shape
    z = x / temperature
    m = z.max(dim=1).values
    empty = m == -math.inf
    dz = torch.where(empty[:, None], torch.zeros_like(z), z - m[:, None])
    e = torch.where(empty[:, None], torch.zeros_like(z), dz.exp())
    s = e.sum(dim=1)
    logs = torch.where(empty, torch.zeros_like(s), s.log())
    lse = torch.where(empty, m, m + logs)
    us = torch.where(e > 0, e * dz, torch.zeros_like(e)).sum(dim=1) / torch.where(empty, torch.ones_like(s), s)
    ent = logs - us
    lp = torch.where(empty[:, None], torch.full_like(z, -math.inf), z - torch.where(empty, torch.zeros_like(m), lse)[:, None])
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    place = torch.empty_like(order)
    place.scatter_(1, order, torch.arange(v).expand(n, v).contiguous())
    k = min(n_top, v)
    ids = torch.full((n, n_top), -1, dtype=torch.int64)
    top = torch.full((n, n_top), -math.inf, dtype=torch.float64)
    ids[:, :k] = order[:, :k]
    top[:, :k] = lp.gather(1, order[:, :k])
    out = {"lse": lse, "entropy": ent, "ids": ids, "top": top, "m": m}
    if tokens is not None:
        t = tokens.long()
        ok = (t >= 0) & (t < v)
        c = t.clamp(0, v - 1)[:, None]
        out["logprob"] = torch.where(ok, lp.gather(1, c)[:, 0], torch.zeros_like(lse))
        out["rank"] = torch.where(ok, place.gather(1, c)[:, 0], torch.full((n,), -1))
    return out


def _close(name, got, want, tol):
    got, want = got.double(), want.double()
    most = (2.0 - 2.0 ** -24) * 2.0 ** 127      # from here on f32's nearest value is an infinity (max - lowest is there)
    want = want.masked_fill(want >= most, math.inf).masked_fill(want <= -most, -math.inf)
    fin = want.isfinite()
    assert bool((got[~fin] == want[~fin]).all()), name
    err = (got[fin] - want[fin]).abs()
    bad = err > tol.expand_as(want)[fin]
    assert not bool(bad.any()), f"{name}: off by {float(err.max()):.3g}, allowed {float(tol.expand_as(want)[fin][err.argmax()]):.3g}"


def _check(torch, out, x, tokens, n_top, temperature):
    ref = _reference(torch, x.double().cpu(), None if tokens is None else tokens.cpu(), n_top, temperature)
    t = (x.shape[1] / 256 + 80) * U
    zm = torch.where(ref["m"].isfinite(), ref["m"].abs(), torch.zeros_like(ref["m"]))

    def tol(want):
        size = torch.where(want.isfinite(), want.abs(), torch.zeros_like(want))
        return t + 2 * U * size + 2 * U * (zm if want.dim() == 1 else zm[:, None])

    _close("lse", out.lse.cpu(), ref["lse"], tol(ref["lse"]))
    _close("entropy", out.entropy.cpu(), ref["entropy"], torch.full_like(ref["entropy"], t * 30))
    if tokens is not None:
        _close("logprob", out.logprob.cpu(), ref["logprob"], tol(ref["logprob"]))
        assert torch.equal(out.rank.cpu().long(), ref["rank"])
    if n_top:
        assert torch.equal(out.top_ids.cpu().long(), ref["ids"])
        _close("top_logprobs", out.top_logprobs.cpu(), ref["top"], tol(ref["top"]))


def _rows(torch, n, v, dtype, pad=0, offset=0, seed=0, scale=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 7919 * n + v)
    flat = torch.randn((offset + n * (v + pad),), generator=g, device="cuda") * scale
    flat = (20 * torch.tanh(flat / 20)).to(dtype)
    return torch.as_strided(flat, (n, v), (v + pad, 1), offset)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,v,pad,offset,n_top,temperature", [
    (1, 1, 0, 0, 1, 1.0), (3, 1, 2, 1, 5, 1.0), (2, 2, 0, 0, 64, 0.7), (5, 7, 1, 3, 3, 2.0), (4, 33, 0, 1, 33, 1.0),
    (3, 64, 0, 0, 64, 1.0), (7, 511, 1, 0, 20, 1.0), (77, 1000, 3, 5, 5, 0.7), (1, 2048, 0, 0, 64, 1.0),
    (2, 4097, 0, 1, 8, 2.0), (1, 32003, 0, 0, 20, 1.0), (9, 50257, 4, 3, 64, 1.0), (330, 2048, 0, 0, 4, 1.0),
    (1, 202048, 0, 0, 20, 1.0), (3, 202048, 1, 1, 0, 1.0), (40, 65536, 0, 0, 1, 1.0), (160, 10007, 0, 0, 17, 1.5)])
def test_score_shapes(torch_cuda, dtype, n, v, pad, offset, n_top, temperature):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    x = _rows(torch, n, v, getattr(torch, dtype), pad, offset)
    g = torch.Generator(device="cuda")
    g.manual_seed(v)
    tokens = torch.randint(0, v, (n,), generator=g, device="cuda").to(torch.int32)
    tokens[0] = int(x[0].float().argmax())
    if n > 2:
        tokens[1], tokens[2] = -1, v            # padded rows
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        _check(torch, head.score(x, tokens, n_top, temperature), x, tokens, n_top, temperature)


def _special(torch, v, dtype):
    """Rows where masks, ties and orders can go wrong, by name."""
    dt = getattr(torch, dtype)
    low, high = torch.finfo(dt).min, torch.finfo(dt).max
    g = torch.Generator()
    g.manual_seed(v)
    base = torch.randn((v,), generator=g) * 3
    at = torch.randperm(v, generator=g)
    rows = {
        "all masked": torch.full((v,), -math.inf),
        "all lowest": torch.full((v,), low),
        "all equal": torch.full((v,), 1.5),
        "one left, the last": torch.where(torch.arange(v) == v - 1, base, torch.tensor(-math.inf)),
        "ten left": base.clone().index_fill_(0, at[10:], -math.inf),
        "ten over the lowest": base.clone().index_fill_(0, at[10:], low),
        "ascending": torch.arange(v).float() / v,
        "descending": -torch.arange(v).float() / v,
        "a few values": (base * 0.7).round(),
        "two values": (base > 0).float(),
        "zeros of both signs": torch.where(base > 0, torch.tensor(0.0), torch.tensor(-0.0)),
        "far apart": torch.where(at < 3, torch.tensor(high), torch.where(at < v // 2, torch.tensor(low), base)),
        "top at the end": torch.where(torch.arange(v) >= v - 70, base + 30, base),
        "masked but the end": torch.where(torch.arange(v) < v - 3, torch.tensor(-math.inf), base),
        "one peak": torch.where(torch.arange(v) == v // 2, torch.tensor(60.0), base),
    }
    return list(rows), torch.stack(list(rows.values())).to(dt)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("v", [3, 65, 1000, 5003, 40000, 202048])
@pytest.mark.parametrize("n_top", [1, 20, 64])
def test_score_masks_ties_and_orders(torch_cuda, dtype, v, n_top):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    names, x = _special(torch, v, dtype)
    x = x.cuda()
    tokens = torch.tensor([(i * 7919) % v for i in range(len(names))], dtype=torch.int32, device="cuda")
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        _check(torch, head.score(x, tokens, n_top), x, tokens, n_top, 1.0)
        for i in range(len(names)):               # one row at a time: the split of a row differs with the row count
            one = head.score(x[i], tokens[i:i + 1], n_top)
            _check(torch, one, x[i:i + 1], tokens[i:i + 1], n_top, 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("v", [9, 5000, 202048])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_score_rows_with_nan_or_infinity_stay_to_themselves(torch_cuda, dtype, v, bad):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    x = _rows(torch, 4, v, getattr(torch, dtype))
    clean = x.clone()
    x[1, v // 2] = float(bad)
    x[3, :] = float(bad)
    tokens = torch.tensor([0, v // 2, 1, 2], dtype=torch.int32, device="cuda")
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        out = head.score(x, tokens, 5)
        ref = head.score(clean, tokens, 5)
    for r in (1, 3):
        assert math.isnan(float(out.lse[r])) and math.isnan(float(out.logprob[r])) and math.isnan(float(out.entropy[r]))
    assert int(out.top_ids.min()) >= -1 and int(out.top_ids.max()) < v
    for a, b in zip(out, ref):
        for r in (0, 2):
            assert torch.equal(a[r], b[r])


def test_score_outputs_one_by_one(torch_cuda):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    v, n = 5003, 6
    x = _rows(torch, n, v, torch.float32)
    tokens = torch.arange(n, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.full(s, 7.0, device="cuda")                                       # noqa: E731
    i = lambda *s: torch.full(s, 7, device="cuda", dtype=torch.int32)                      # noqa: E731
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        full = head.score(x, tokens, 3)
        s = torch.cuda.current_stream().cuda_stream
        for keep in range(5):
            outs = [f(n), i(n), f(n), f(n), i(n, 3), f(n, 3)]
            names = [{0}, {1}, {2}, {3}, {4, 5}][keep]
            at = [t.data_ptr() if j in names else None for j, t in enumerate(outs)]
            st = mlh.muse_lmhead_score(head.handle, x.data_ptr(), 0, n, v, tokens.data_ptr(), 1.0,
                                       3 if keep == 4 else 0, *at, s)
            assert st == 0
            for j, t in enumerate(outs):
                want = full[j] if j in names else torch.full_like(t, 7)
                assert torch.equal(t, want)
        empty = head.score(x[:0], tokens[:0], 3)                                            # no rows: nothing to do
        assert empty.lse.shape == (0,) and empty.top_ids.shape == (0, 3)


def test_score_offsets_past_32_bits(torch_cuda):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    v, n = 202048, 10700                           # 2.16e9 elements: past 2^31
    x = torch.full((n, v), -3.0, dtype=torch.float16, device="cuda")
    rows = [0, 5000, n - 2, n - 1]
    x[rows] = _rows(torch, len(rows), v, torch.float16)
    tokens = torch.full((n,), v - 1, dtype=torch.int32, device="cuda")
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        out = head.score(x, tokens, 4)
    pick = type(out)(*(t[rows] for t in out))
    _check(torch, pick, x[rows], tokens[rows], 4, 1.0)
    assert abs(float(out.lse[7]) - (math.log(v) - 3)) < 1e-4 and out.top_ids[7].tolist() == [0, 1, 2, 3]


def test_score_in_a_graph_and_on_two_streams(torch_cuda):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    v, n = 50257, 3
    a, b = _rows(torch, n, v, torch.bfloat16, seed=1), _rows(torch, n, v, torch.bfloat16, seed=2)
    tokens = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        want = [[t.clone() for t in head.score(t, tokens, 9)] for t in (a, b)]
        x = a.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            head.score(x, tokens, 9)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                got = head.score(x, tokens, 9)
        torch.cuda.synchronize()
        for src, ref in ((a, want[0]), (b, want[1]), (a, want[0])):
            x.copy_(src)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, ref))
        other = torch.cuda.Stream()
        res = []
        for _ in range(20):                        # one handle, two streams at once: score shares nothing
            with torch.cuda.stream(s):
                res.append((head.score(a, tokens, 9), want[0]))
            with torch.cuda.stream(other):
                res.append((head.score(b, tokens, 9), want[1]))
        torch.cuda.synchronize()
        for r, ref in res:
            assert all(torch.equal(p, q) for p, q in zip(r, ref))


@pytest.mark.parametrize("b", [1, 5])
def test_forward_score_is_forward_then_score(torch_cuda, b):
    import q5_lm_head_gb300 as mlh
    import q5k_synth as synth
    torch = torch_cuda
    wl = synth.WORKLOADS["tiny"]
    hidden, gamma, wq = synth.inputs_for(wl)
    hidden = np.concatenate([hidden * (1 + 0.3 * i) for i in range(b)])
    h, g, w = (torch.from_numpy(np.ascontiguousarray(t)).cuda() for t in (hidden, gamma, wq))
    tokens = torch.arange(b, dtype=torch.int32, device="cuda") * 17
    with mlh.LMHead(wl.n_rows, wl.k, max_batch=b, device=0) as head:
        logits, out = head.forward_score(h, w, g, tokens=tokens, n_top=6)
        again, argmax = head.forward(h, w, g)
        ref = head.score(again, tokens, 6)
        lp, lse = head.forward_logprobs(h, w, g, want_argmax=False)
        torch.cuda.synchronize()
        assert head.device_status() == 0
    assert torch.equal(logits, again)
    assert all(torch.equal(p, q) for p, q in zip(out, ref))
    assert torch.equal(out.top_ids[:, 0], argmax)
    _check(torch, out, logits, tokens, 6, 1.0)
    assert float((lse - out.lse).abs().max()) <= 2e-5     # both within (V/256 + 80) u + 4u |lse| of the same value


@pytest.mark.parametrize("b", [1, 5])
def test_forward_score_back_to_back_with_other_rows(torch_cuda, b):
    """The scores' kernel starts while the forward still runs: it has to see that forward's logits."""
    import q5_lm_head_gb300 as mlh
    import q5k_synth as synth
    torch = torch_cuda
    wl = synth.WORKLOADS["tiny"]
    hidden, gamma, wq = synth.inputs_for(wl)
    w, g = torch.from_numpy(np.ascontiguousarray(wq)).cuda(), torch.from_numpy(gamma).cuda()
    rng = np.random.default_rng(b)
    rows = [torch.from_numpy((hidden * (1 + i) + rng.standard_normal((b, wl.k))).astype(np.float32)).cuda() for i in range(3)]
    tokens = torch.arange(b, dtype=torch.int32, device="cuda") * 31
    with mlh.LMHead(wl.n_rows, wl.k, max_batch=b, device=0) as head:
        want = []
        for h in rows:
            logits, out = head.forward_score(h, w, g, tokens=tokens, n_top=9)
            torch.cuda.synchronize()
            want.append([t.clone() for t in (logits, *out)])
        logits = torch.empty((b, wl.n_rows), device="cuda")
        got = [(i % 3, head.forward_score(rows[i % 3], w, g, tokens=tokens, n_top=9, logits=logits)[1]) for i in range(300)]
        torch.cuda.synchronize()
        assert head.device_status() == 0
    for i, out in got:
        assert all(torch.equal(p, q) for p, q in zip(out, want[i][1:]))


@pytest.mark.parametrize("temperature", [2.0 ** -20, 0.01, 100.0, 2.0 ** 20])
def test_score_temperatures(torch_cuda, temperature):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    x = _rows(torch, 3, 5003, torch.float32)
    tokens = torch.tensor([int(x[0].argmax()), 5, 6], dtype=torch.int32, device="cuda")
    with mlh.LMHead(5003, 256, max_batch=1, device=0) as head:
        _check(torch, head.score(x, tokens, 7, temperature), x, tokens, 7, temperature)


@pytest.mark.parametrize("n,v", [(3, 2500), (5, 9000), (9, 60000), (20, 20000), (40, 30000), (77, 40000), (100, 33000),
                                 (140, 9001), (153, 9001), (200, 2000), (228, 9000), (229, 5000), (304, 5000), (305, 5000)])
def test_score_rows_by_every_number_of_ctas(torch_cuda, n, v):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    x = _rows(torch, n, v, torch.bfloat16, pad=3, offset=1)
    tokens = torch.arange(n, dtype=torch.int32, device="cuda") * 37 % v
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        out = head.score(x, tokens, n_top=64)
        torch.cuda.synchronize()
    _check(torch, out, x, tokens, 64, 1.0)


@pytest.mark.parametrize("n,v", [(1, 40), (2, 9000), (80, 6000), (400, 3000)])
@pytest.mark.parametrize("largest", [False, True])
def test_score_zeros_of_both_signs_are_one_value(torch_cuda, n, v, largest):
    import q5_lm_head_gb300 as mlh
    torch = torch_cuda
    g = torch.Generator(device="cuda")
    g.manual_seed(v)
    x = torch.where(torch.rand((n, v), generator=g, device="cuda") < 0.5, 0.0, -0.0)
    if not largest:
        x[:, ::7] = 1.0
        x[:, 3::5] = -1.0
    tokens = torch.arange(n, dtype=torch.int32, device="cuda") * 13 % v
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        out = head.score(x, tokens, n_top=32)
        torch.cuda.synchronize()
    order = torch.sort(x + 0.0, dim=1, descending=True, stable=True).indices
    assert torch.equal(out.top_ids.long(), order[:, :32])
    place = torch.empty_like(order)
    place.scatter_(1, order, torch.arange(v, device="cuda").expand(n, v).contiguous())
    assert torch.equal(out.rank.long(), place.gather(1, tokens.long()[:, None])[:, 0])
