"""muse_lmhead_embed_backward: the gradient by a token table against sums in 64 bits.

Tolerance (u = 2^-24): a sum of m values in f32, in any order, is off by at most
(m - 1) u of the sum of their sizes, the product with the scale (and with
accumulate the addition to the old value) by u each of what it gives, the result
by half a step of its type and of the type's smallest step.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = ("float32", "float16", "bfloat16")
SMALL = {"float32": 2.0 ** -150, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}


@pytest.fixture(scope="module")
def env():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    return torch, mlh


def _reference(torch, grad, tokens, v, scale, old=None):
    """(sums, the limit of what f32 adds to their rounding), on the CPU in 64 bits."""
    g, tok = grad.double().cpu(), tokens.long().cpu()
    ok = (tok >= 0) & (tok < v)
    s = float(np.float32(scale))
    total, size = torch.zeros((v, g.shape[1]), dtype=torch.float64), torch.zeros((v, g.shape[1]), dtype=torch.float64)
    count = torch.zeros((v, 1), dtype=torch.float64)
    total.index_add_(0, tok[ok], g[ok])
    size.index_add_(0, tok[ok], g[ok].abs())
    count.index_add_(0, tok[ok], torch.ones((int(ok.sum()), 1), dtype=torch.float64))
    want, limit = total * s, count * U * size * abs(s)
    if old is not None:
        want = want + old.double().cpu()
        limit = limit + U * (want.abs() + size * abs(s))
    return want, limit * (1 + 1e-3)


def _check(torch, got, want, limit, dtype):
    limit = limit + want.abs() * (torch.finfo(got.dtype).eps / 2 + U) + SMALL[dtype]
    off = (got.double().cpu() - want).abs()
    assert bool((off <= limit).all()), float((off / limit).max())


def _tokens(torch, kind, n, v, gen):
    if kind == "one":
        return torch.full((n,), v // 2, dtype=torch.int32, device="cuda")
    if kind == "different":
        return torch.randperm(max(n, v), generator=gen, device="cuda")[:n].to(torch.int32) % v
    if kind == "few":
        return (torch.randint(0, 3, (n,), generator=gen, device="cuda") * (v // 3)).to(torch.int32)
    if kind == "padded":
        t = torch.randint(-v, 2 * v, (n,), generator=gen, device="cuda").to(torch.int32)
        return t
    if kind == "none":
        return torch.full((n,), -1, dtype=torch.int32, device="cuda")
    rank = torch.exp(torch.rand((n,), generator=gen, device="cuda") * float(np.log(v + 1))).long().clamp(1, v) - 1
    return rank.to(torch.int32)


@pytest.mark.parametrize("kind", ["one", "different", "few", "padded", "none", "text"])
@pytest.mark.parametrize("n,v,k", [(1, 7, 256), (2, 1, 256), (33, 300, 512), (513, 1999, 256), (2100, 37, 768), (20000, 5000, 256)])
def test_sums(env, kind, n, v, k):
    torch, mlh = env
    gen = torch.Generator(device="cuda").manual_seed(n + v)
    grad = torch.randn((n, k), generator=gen, device="cuda")
    tokens = _tokens(torch, kind, n, v, gen)
    grad[(tokens < 0) | (tokens >= v)] = float("nan")         # left out, and not read
    want, limit = _reference(torch, torch.nan_to_num(grad), tokens, v, 1.3)
    with mlh.LMHead(v, k, max_batch=1, device=0) as head:
        got = head.embed_backward(grad, tokens, scale=1.3)
        _check(torch, got, want, limit, "float32")
        assert torch.equal(got, head.embed_backward(grad, tokens, scale=1.3))      # the same bits


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_types(env, dtype, out, accumulate):
    torch, mlh = env
    n, v, k = 700, 400, 512
    gen = torch.Generator(device="cuda").manual_seed(3)
    grad = torch.randn((n, k), generator=gen, device="cuda").to(getattr(torch, dtype))
    tokens = _tokens(torch, "text", n, v, gen)
    old = torch.randn((v, k), generator=gen, device="cuda").to(getattr(torch, out))
    want, limit = _reference(torch, grad, tokens, v, 0.75, old if accumulate else None)
    table = old.clone()
    with mlh.LMHead(v, k, max_batch=1, device=0) as head:
        got = head.embed_backward(grad, tokens, scale=0.75, grad_table=table, accumulate=accumulate)
    assert got is table
    _check(torch, got, want, limit, out)
    if accumulate:
        used = torch.zeros((v,), dtype=torch.bool, device="cuda")
        used[tokens.long()] = True
        assert torch.equal(got[~used], old[~used])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,off", [(1, 0), (8, 0), (0, 1), (3, 3), (4, 4)])
def test_rows_at_any_distance_and_alignment(env, dtype, pad, off):
    torch, mlh = env
    n, v, k = 90, 50, 256
    t = getattr(torch, dtype)
    grad = torch.randn((n, k + pad + off), device="cuda").to(t)[:, off:off + k]
    whole = torch.full((v, k + pad + off), 7.0, device="cuda").to(t)
    tokens = torch.randint(0, v - 9, (n,), device="cuda", dtype=torch.int32)
    want, limit = _reference(torch, grad, tokens, v, 1.0)
    with mlh.LMHead(v, k, max_batch=1, device=0) as head:
        got = head.embed_backward(grad, tokens, grad_table=whole[:, off:off + k])
    _check(torch, got, want, limit, dtype)
    assert bool((whole[:, :off] == 7).all()) and bool((whole[:, off + k:] == 7).all())


def test_special_values_stay_in_their_rows(env):
    torch, mlh = env
    n, v, k = 40, 8, 256
    grad = torch.ones((n, k), device="cuda")
    tokens = (torch.arange(n, device="cuda") % 4).to(torch.int32)
    grad[1] = float("nan")
    grad[2] = float("inf")
    with mlh.LMHead(v, k, max_batch=1, device=0) as head:
        got = head.embed_backward(grad, tokens)
    assert bool((got[0] == 10).all()) and bool(got[1].isnan().all()) and bool((got[2] == float("inf")).all())
    assert bool((got[3] == 10).all()) and bool((got[4:] == 0).all())


def test_no_positions(env):
    torch, mlh = env
    v, k = 33, 256
    none, grad = torch.zeros((0,), dtype=torch.int32, device="cuda"), torch.zeros((0, k), device="cuda")
    with mlh.LMHead(v, k, max_batch=1, device=0) as head:
        assert bool((head.embed_backward(grad, none) == 0).all())
        table = torch.full((v, k), 3.0, device="cuda")
        assert bool((head.embed_backward(grad, none, grad_table=table, accumulate=True) == 3).all())
        assert bool((head.embed_backward(grad, none, grad_table=table) == 0).all())


def test_gradient_is_that_of_the_lookup(env):
    """Differences of sum(embed(table) * weight) by elements of the table."""
    torch, mlh = env
    n, v, k = 31, 12, 256
    gen = torch.Generator(device="cuda").manual_seed(9)
    table = torch.randn((v, k), generator=gen, device="cuda")
    weight = torch.randn((n, k), generator=gen, device="cuda")
    tokens = torch.randint(-1, v, (n,), generator=gen, device="cuda", dtype=torch.int32)
    with mlh.LMHead(v, k, max_batch=1, device=0) as head:
        got = head.embed_backward(weight, tokens, scale=3.0).cpu()
        value = lambda t: float((head.embed(tokens, t, scale=3.0).double() * weight.double()).sum())     # noqa: E731
        for at in [(0, 0), (3, 17), (11, 255), (7, 128)]:
            up, down = table.clone(), table.clone()
            up[at] += 0.5
            down[at] -= 0.5
            step = float(up[at].double() - down[at].double())
            # embed's products are off by u of up to 6 * 3 each, a row's worth of them changing: n of these, over the step
            assert abs((value(up) - value(down)) / step - float(got[at])) <= 2 * n * 18 * U * 6 + 1e-5 * abs(float(got[at]))


def test_many_positions_of_a_captured_call_and_two_at_once(env):
    """Two graphs with a workspace each, replayed on two streams, against eager calls."""
    torch, mlh = env
    n, v, k = 9000, 700, 512
    gen = torch.Generator(device="cuda").manual_seed(4)
    grads = [torch.randn((n, k), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    tokens = [_tokens(torch, kind, n, v, gen) for kind in ("text", "different")]
    with mlh.LMHead(v, k, max_batch=1, device=0) as head:
        want = [head.embed_backward(g, t).clone() for g, t in zip(grads, tokens)]
        torch.cuda.synchronize()
        graphs, outs = [], []
        for g, t in zip(grads, tokens):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs.append(head.embed_backward(g, t))
            graphs.append(graph)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(5):
            for o in outs:
                o.fill_(5)
            torch.cuda.synchronize()
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_offsets_past_32_bits(env):
    torch, mlh = env
    v, k, n = 700_000, 6656, 5
    grad = torch.randn((n, k), device="cuda").half()
    tokens = torch.tensor([v - 1, 0, v - 2, v - 1, 350_000], dtype=torch.int32, device="cuda")
    with mlh.LMHead(v, k, max_batch=1, device=0) as head:
        got = head.embed_backward(grad, tokens)
        assert torch.equal(got[v - 2], grad[2]) and torch.equal(got[0], grad[1]) and torch.equal(got[350_000], grad[4])
        assert torch.equal(got[v - 1], (grad[0].float() + grad[3].float()).half())
        assert int(got.count_nonzero()) == int(got[[0, 350_000, v - 2, v - 1]].count_nonzero())
    del got
    torch.cuda.empty_cache()
