"""muse_lmhead_sample against its definition in 64 bits.

A drawn token is right when the number u * (kept mass) lies within its share of the
kept mass.  The kernel's weights are whole numbers of 2^-38 of the largest one's
power of two, off by half a step and by at most 2^-32 of themselves, and those below 2^-42 of the
largest are 0: with s = 2^-32 of the kept mass + V 2^-38 of the largest weight, the sums up to a
border and the number that is compared with it are off by s at most each: 2 s on either side of
a token's share.  The border of top-p moves by the same: a draw is right with the
kept set of p - d or of p + d, d = 2 s of the mass.  Log probabilities: sums as above,
the logit's difference exact in 64 bits, one rounding to f32: half a step of f32 of
the result and 2^-30 + V 2^-37 of the largest weight's share.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = ("float32", "float16", "bfloat16")


@pytest.fixture(scope="module")
def env():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    return torch, mlh


def _kept(x, t, k, p, mp, move):
    """Mask of what the filters keep; `move` shifts top-p's border by that share of the mass."""
    order = np.argsort(-x, kind="stable")
    w = np.exp((x - x.max()) / t)
    keep = np.zeros(x.size, dtype=bool)
    first = order[:k] if 0 < k < x.size else order
    if p < 1:
        upto = np.cumsum(w[first])
        before = np.concatenate([[0.0], upto[:-1]])
        first = first[(before < (p + move) * upto[-1]) | (np.arange(first.size) == 0)]
    keep[first] = True
    if mp > 0:
        keep &= x >= x.max() + t * math.log(min(mp, 1.0))
    return keep


def _check_row(x, u, t, k, p, mp, token, logprob):
    x, u, t, p, mp, k = x.astype(np.float64), float(u), float(t), float(p), float(mp), int(k)
    v = x.size
    if t == 0:
        assert token == int(np.argmax(x)) and logprob == 0.0
        return
    if p <= 0:
        k, p = 1, 1.0
    w = np.exp((x - x.max()) / t)
    slack = lambda mass: 2 * (2.0 ** -32 * mass + v * 2.0 ** -38)                        # noqa: E731
    d = slack(w.sum()) / w.sum()
    u = min(max(u, 0.0) if u == u else 0.0, 1.0)
    seen = []
    for move in (0.0, d, -d):
        keep = _kept(x, t, k, p, mp, move)
        kw = np.where(keep, w, 0.0)
        upto = np.cumsum(kw)
        total = upto[-1]
        lo, hi, s = upto[token] - kw[token], upto[token], slack(total)
        right = bool(keep[token]) and lo - s <= u * total <= hi + s
        want = (x[token] - x.max()) / t - math.log(total)
        near = abs(logprob - want) <= abs(want) * U * 1.01 + 2.0 ** -30 + v * 2.0 ** -37 / total
        seen.append((right, near, lo, u * total, hi, want))
        if right and near:
            return
    raise AssertionError((token, logprob, seen))


def _run(env, x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    torch, mlh = env
    n, v = x.shape
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        tokens, logprobs = head.sample(x, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
        again = head.sample(x, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    torch.cuda.synchronize()
    assert tokens.dtype == torch.int32 and logprobs.dtype == torch.float32
    assert torch.equal(tokens, again[0]) and torch.equal(logprobs.nan_to_num(nan=9.0), again[1].nan_to_num(nan=9.0))
    return tokens.cpu().numpy(), logprobs.cpu().numpy()


def _check(env, x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    torch, _ = env
    n = x.shape[0]
    tokens, logprobs = _run(env, x, u, temperature, top_k, top_p, min_p)
    rows, us = x.float().cpu().numpy(), u.cpu().numpy()
    column = lambda s: s.cpu().numpy() if isinstance(s, torch.Tensor) else np.full(n, s, dtype=np.float32)     # noqa: E731
    t, k, p, mp = (column(s) for s in (temperature, top_k, top_p, min_p))
    for r in range(n):
        _check_row(rows[r], us[r], t[r], k[r], p[r], mp[r], int(tokens[r]), float(logprobs[r]))
    return tokens, logprobs


def _rows(torch, n, v, seed, scale=3.0, dtype="float32", pad=0, off=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, v + pad + off), generator=gen, device="cuda") * scale
    u = torch.rand((n,), generator=gen, device="cuda")
    return x.to(getattr(torch, dtype))[:, off:off + v], u


SETTINGS = [dict(), dict(temperature=0.5), dict(top_k=1), dict(top_k=7), dict(top_k=50, top_p=0.9), dict(top_p=0.5), dict(top_p=0.95),
            dict(top_p=0.999), dict(min_p=0.1), dict(top_k=40, min_p=0.02), dict(top_p=0.8, min_p=0.3), dict(top_k=300, top_p=0.97, min_p=0.001, temperature=1.5),
            dict(temperature=0.0), dict(top_p=0.0), dict(top_p=1e-30), dict(min_p=1.0), dict(min_p=5.0), dict(temperature=4.0, top_p=0.9)]


@pytest.mark.parametrize("settings", SETTINGS, ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()) or "plain")
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v", [(1, 1), (3, 2), (5, 33), (40, 1000), (6, 32003), (2, 202048)])
def test_draws(env, settings, dtype, n, v):
    x, u = _rows(env[0], n, v, v + n, dtype=dtype)
    _check(env, x, u, **settings)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,off", [(1, 0), (7, 0), (0, 1), (3, 5), (9, 2)])
@pytest.mark.parametrize("v", [1, 9, 517, 50257])
def test_rows_at_any_distance_and_alignment(env, dtype, pad, off, v):
    x, u = _rows(env[0], 5, v, v, dtype=dtype, pad=pad, off=off)
    _check(env, x, u, top_p=0.9)
    _check(env, x, u)


@pytest.mark.parametrize("n", [1, 2, 30, 77, 153, 400, 1100])
def test_many_rows(env, n):
    x, u = _rows(env[0], n, 3001, n)
    _check(env, x, u, top_k=20, top_p=0.9)
    _check(env, x, u)


def test_a_setting_for_each_row(env):
    torch, _ = env
    n, v = 64, 5003
    x, u = _rows(torch, n, v, 11)
    pick = lambda values, dtype: torch.tensor([values[i % len(values)] for i in range(n)], dtype=dtype, device="cuda")     # noqa: E731
    _check(env, x, u, pick([0.0, 1.0, 0.7, 2.0, 0.25], torch.float32), pick([0, 1, 50, -3, 5003, 9999, 200], torch.int32),
           pick([1.0, 0.9, 0.3, 2.0, 0.99, -1.0], torch.float32), pick([0.0, 0.05, -1.0, 0.5], torch.float32))


def test_equal_logits_share_alike(env):
    """Rows of equal values: whole numbers of equal weights, so u draws token floor(u * n) exactly."""
    torch, _ = env
    for v, value in [(1, 0.0), (2, -7.25), (3, 19.9), (8, 1e-30), (1000, -3.4e38), (4096, 3.0e38), (50257, 0.1)]:
        us = np.array([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 0.3, 1 / 3, 1e-9, 1e-40, 1.0, 7.0, -1.0, np.nan], dtype=np.float32)
        x = torch.full((us.size, v), value, device="cuda")
        tokens, logprobs = _run(env, x, torch.from_numpy(us).cuda())
        for u, tok, lp in zip(us, tokens, logprobs):
            f = float(u) if u == u else 0.0
            want = v - 1 if f >= 1 else 0 if f <= 0 else int(math.floor(float(np.float64(u) * v)))
            assert tok == want, (v, value, u, tok, want)
            assert abs(lp + math.log(v)) <= U * math.log(v) * 1.01
        # the first k of the equal ones
        k = min(v, 5)
        tokens, _ = _run(env, x, torch.from_numpy(us).cuda(), top_k=k)
        for u, tok in zip(us, tokens):
            f = float(u) if u == u else 0.0
            assert tok == (k - 1 if f >= 1 else 0 if f <= 0 else int(math.floor(f * k)))
        # half of the mass: the entries before which less than half lies
        half = -(-v // 2)
        tokens, _ = _run(env, x, torch.from_numpy(us).cuda(), top_p=0.5)
        for u, tok in zip(us, tokens):
            f = float(u) if u == u else 0.0
            assert tok == (half - 1 if f >= 1 else 0 if f <= 0 else int(math.floor(f * half)))


@pytest.mark.parametrize("settings", [dict(), dict(top_k=3), dict(top_p=0.9), dict(min_p=0.5), dict(top_k=100, top_p=0.99)], ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_few_different_values(env, settings, dtype):
    """Borders that fall among many equal logits: the first of them by index."""
    torch, _ = env
    gen = torch.Generator(device="cuda").manual_seed(5)
    n, v = 24, 20011
    x = torch.randint(0, 5, (n, v), generator=gen, device="cuda").to(getattr(torch, dtype))
    x[:, ::2] *= -0.0                                        # zeros of both signs are one value
    _check(env, x, torch.rand((n,), generator=gen, device="cuda"), **settings)


def test_masks(env):
    """-infinity is never drawn, lowest values only where nothing else is left."""
    torch, mlh = env
    gen = torch.Generator(device="cuda").manual_seed(6)
    n, v = 12, 7001
    for dtype in TYPES:
        t = getattr(torch, dtype)
        for mask in (-math.inf, float(torch.finfo(t).min)):
            x = (torch.randn((n, v), generator=gen, device="cuda") * 3).to(t)
            keep = torch.rand((n, v), generator=gen, device="cuda") < 0.01
            keep[0] = False
            keep[0, v - 1] = True
            keep[1] = False
            keep[1, 0] = True
            x[~keep] = mask
            u = torch.rand((n,), generator=gen, device="cuda")
            u[2:4] = torch.tensor([0.0, 1.0])
            for settings in (dict(), dict(top_k=100), dict(top_p=0.9), dict(top_k=5000, top_p=0.999)):
                tokens, _ = _run(env, x, u, **settings)
                assert bool(keep.cpu()[torch.arange(n), torch.from_numpy(tokens).long()].all())
                if mask == -math.inf:
                    _check(env, torch.where(keep, x, torch.full_like(x, -1e4)), u, **settings)     # weights 0 either way
                assert tokens[0] == v - 1 and tokens[1] == 0


def test_rows_without_a_distribution(env):
    torch, _ = env
    v = 3000
    x, u = _rows(torch, 8, v, 2)
    x[1] = -math.inf
    x[2, 5] = math.nan
    x[3, 7] = math.inf
    x[4] = math.nan
    x[5, v - 1] = math.nan
    x[6, 1:] = -math.inf
    for settings in (dict(), dict(top_k=4), dict(top_p=0.8), dict(min_p=0.2), dict(temperature=0.0)):
        tokens, logprobs = _run(env, x, u, **settings)
        assert list(tokens[1:7]) == [-1, -1, -1, -1, -1, 0] and logprobs[1] == -math.inf and np.isnan(logprobs[2:6]).all() and logprobs[6] == 0
        for r in (0, 7):
            f = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, **{}) | settings
            _check_row(x[r].cpu().numpy(), u[r].item(), f["temperature"], f["top_k"], f["top_p"], f["min_p"], int(tokens[r]), float(logprobs[r]))
    bad = torch.tensor([1.0, -1.0, math.nan, math.inf, 2.0 ** -30, 2.0 ** 21, 1.0, 1.0], device="cuda")
    y, _ = _rows(torch, 8, v, 3)
    tokens, logprobs = _run(env, y, u, temperature=bad)
    assert list(tokens[1:6]) == [-1] * 5 and np.isnan(logprobs[1:6]).all() and tokens[0] >= 0 and tokens[7] >= 0
    nan = torch.full((8,), math.nan, device="cuda")
    for settings in (dict(top_p=nan), dict(min_p=nan)):
        tokens, logprobs = _run(env, y, u, **settings)
        assert (tokens == -1).all() and np.isnan(logprobs).all()


@pytest.mark.parametrize("temperature", [2.0 ** -20, 1e-4, 0.01, 0.03, 50.0, 1e4, 2.0 ** 20])
@pytest.mark.parametrize("scale,shift", [(3.0, 0.0), (1.0, 1000.0), (100.0, -3e4), (1e5, 0.0), (1e-3, 0.0), (1e30, 0.0)])
def test_temperatures_and_large_logits(env, temperature, scale, shift):
    torch, _ = env
    x, u = _rows(torch, 6, 9001, 8, scale=scale)
    _check(env, x + shift, u, temperature=temperature)
    _check(env, x + shift, u, temperature=temperature, top_p=0.7, top_k=500)


@pytest.mark.parametrize("settings", [dict(), dict(top_k=30, top_p=0.9), dict(top_p=0.99), dict(min_p=0.01)], ids=str)
@pytest.mark.parametrize("dtype,v", [("float32", 1_000_003), ("bfloat16", 1_600_001), ("float16", 3_000_017), ("float32", 20_000_003)])
def test_long_rows(env, settings, dtype, v):
    """Rows that a cluster cannot hold, and those whose weights have to be shortened."""
    torch, _ = env
    x, u = _rows(torch, 2, v, 4, dtype=dtype)
    _check(env, x, u, **settings)


def test_offsets_past_32_bits(env):
    torch, _ = env
    n, v, ld = 3, 1000, 1 << 31
    whole = torch.zeros((n * ld,), dtype=torch.bfloat16, device="cuda")
    x = whole.as_strided((n, v), (ld, 1))
    x.copy_(torch.randn((n, v), device="cuda") * 3)
    _check(env, x, torch.rand((n,), device="cuda"), top_p=0.9)
    del whole, x
    torch.cuda.empty_cache()


def test_shares_of_many_draws(env):
    """65,536 evenly spaced numbers draw each token its share of the times, to one for each border."""
    torch, mlh = env
    n, v = 65536, 40
    one = (torch.randn((1, v), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 2)
    u = (torch.arange(n, device="cuda", dtype=torch.float32) + 0.5) / n
    for settings, keep in ((dict(), None), (dict(top_k=9, top_p=0.9), (9, 0.9))):
        with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
            tokens, _ = head.sample(one.expand(n, v).contiguous(), u, **settings)
        got = torch.bincount(tokens.long(), minlength=v).cpu().numpy()
        x = one[0].cpu().numpy().astype(np.float64)
        w = np.where(_kept(x, 1.0, *(keep or (0, 1.0)), 0.0, 0.0), np.exp(x), 0.0)
        assert np.abs(got - n * w / w.sum()).max() <= 1.001
        assert bool((tokens[1:] >= tokens[:-1]).all())


def test_captured_and_on_two_streams(env):
    torch, mlh = env
    n, v = 16, 50257
    x, u = _rows(torch, n, v, 3)
    y, _ = _rows(torch, n, v, 4)
    with mlh.LMHead(v, 256, max_batch=1, device=0) as head:
        want = [head.sample(t, u, temperature=0.8, top_k=40, top_p=0.95) for t in (x, y)]
        torch.cuda.synchronize()
        graphs, outs = [], []
        for t in (x, y):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs.append(head.sample(t, u, temperature=0.8, top_k=40, top_p=0.95))
            graphs.append(graph)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(10):
            for o in outs:
                o[0].fill_(-5)
            torch.cuda.synchronize()
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
            torch.cuda.synchronize()
            for o, w in zip(outs, want):
                assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
        assert head.sample(x[:0], u[:0])[0].shape == (0,)
