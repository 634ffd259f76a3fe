"""muse_lmhead_embed: rows of a token table against the blocks' values in 64 bits.

Tolerance (u_t = half a step of the output's type relative to a value): a block's
value is rounded once to f32 (its products are exact there), its product with the
scale once more, and the result once to the output's type: 2 * 2^-24 + u_t of the
value, and half of the type's smallest step.
"""
import numpy as np
import pytest

import oracle
import q5k_synth as synth

pytestmark = pytest.mark.gpu

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


def _blocks(v, k, fmt):
    """(bytes of a [v, k] table, its values in 64 bits)"""
    key = synth.stream_key(5, f"table{v}x{k}{fmt}")
    raw = np.ascontiguousarray(synth.q5k_rows(v, k, key, fmt=fmt)).reshape(-1)
    size = 176 if fmt == "q5_k" else 144
    one = oracle.q5k_dequant_block if fmt == "q5_k" else oracle.q4k_dequant_block
    values = np.stack([one(b) for b in raw.reshape(-1, size)]).reshape(v, k)
    return raw, values.astype(np.float64)


def _check(torch, got, want, dtype):
    assert got.dtype == getattr(torch, dtype)
    limit = want.abs() * (2 * 2.0 ** -24 + torch.finfo(got.dtype).eps / 2) + SMALL[dtype]
    off = (got.double().cpu() - want).abs()
    assert bool((off <= limit).all()), float((off / limit).max())


@pytest.mark.parametrize("fmt", ["q5_k", "q4_k"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k", [256, 768, 1792])
def test_blocks(env, fmt, dtype, k):
    torch, mlh = env
    v = 37
    raw, values = _blocks(v, k, fmt)
    tokens = torch.tensor([0, v - 1, 5, 5, -1, v, 17, 2 ** 31 - 1, -2 ** 31, 1], dtype=torch.int32, device="cuda")
    ok = (tokens >= 0) & (tokens < v)
    want = torch.from_numpy(values)[torch.where(ok, tokens, 0).long().cpu()] * float(np.float32(1.7)) * ok.cpu().unsqueeze(1)
    with mlh.LMHead(v, k, max_batch=1, device=0, fmt=fmt) as head:
        got = head.embed(tokens, torch.from_numpy(raw).cuda(), scale=1.7, dtype=getattr(torch, dtype))
        torch.cuda.synchronize()
        _check(torch, got, want, dtype)
        assert head.embed(tokens, torch.from_numpy(raw).cuda()).dtype == torch.float32


@pytest.mark.parametrize("table", TYPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 7, 300])
def test_dense(env, table, dtype, n):
    torch, mlh = env
    v, k = 211, 512
    gen = torch.Generator(device="cuda").manual_seed(n)
    rows = torch.randn((v, k), generator=gen, device="cuda").to(getattr(torch, table))
    tokens = torch.randint(-2, v + 2, (n,), generator=gen, device="cuda", dtype=torch.int32)
    ok = (tokens >= 0) & (tokens < v)
    want = (rows[torch.where(ok, tokens, 0).long()].double() * float(np.float32(22.6)) * ok.unsqueeze(1)).cpu()
    with mlh.LMHead(v, k, max_batch=1, device=0) as head:
        _check(torch, head.embed(tokens, rows, scale=22.6, dtype=getattr(torch, dtype)), want, dtype)
        plain = head.embed(tokens, rows)
        assert plain.dtype == rows.dtype and torch.equal(plain, torch.where(ok.unsqueeze(1), rows[torch.where(ok, tokens, 0).long()], 0))


@pytest.mark.parametrize("table", TYPES)
@pytest.mark.parametrize("pad,off", [(1, 0), (8, 0), (0, 1), (3, 3), (4, 4)])
def test_rows_at_any_distance_and_alignment(env, table, pad, off):
    """Strided tables and outputs; what lies beside the rows stays."""
    torch, mlh = env
    v, k, n = 50, 256, 13
    t = getattr(torch, table)
    whole = torch.randn((v, k + pad + off), device="cuda").to(t)
    rows = whole[:, off:off + k]
    tokens = torch.arange(n, dtype=torch.int32, device="cuda") * 3
    tokens[4] = -1
    out = torch.full((n, k + pad + off), 7.0, device="cuda").to(t)
    with mlh.LMHead(v, k, max_batch=1, device=0) as head:
        got = head.embed(tokens, rows, out=out[:, off:off + k])
        torch.cuda.synchronize()
    want = rows[tokens.clamp(min=0).long()].clone()
    want[4] = 0
    assert torch.equal(got, want) and got.data_ptr() == out[:, off:].data_ptr()
    assert bool((out[:, :off] == 7).all()) and bool((out[:, off + k:] == 7).all())


def test_special_values_stay_in_their_rows(env):
    torch, mlh = env
    v, k = 5, 256
    rows = torch.ones((v, k), device="cuda")
    rows[1], rows[2], rows[3, 7] = float("nan"), float("inf"), -float("inf")
    with mlh.LMHead(v, k, max_batch=1, device=0) as head:
        got = head.embed(torch.arange(-1, v, dtype=torch.int32, device="cuda"), rows, scale=2.0)
    assert bool((got[0] == 0).all()) and torch.equal(got[1:], rows * 2) is False   # NaN rows compare unequal
    assert torch.equal(torch.nan_to_num(got[1:], nan=9.0), torch.nan_to_num(rows * 2, nan=9.0))


def test_no_tokens_and_a_captured_call(env):
    torch, mlh = env
    v, k, n = 64, 512, 9
    rows = torch.randn((v, k), device="cuda", dtype=torch.bfloat16)
    with mlh.LMHead(v, k, max_batch=1, device=0) as head:
        assert head.embed(torch.zeros((0,), dtype=torch.int32, device="cuda"), rows).shape == (0, k)
        tokens = torch.zeros((n,), dtype=torch.int32, device="cuda")
        out = torch.empty((n, k), dtype=torch.bfloat16, device="cuda")
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            head.embed(tokens, rows, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            head.embed(tokens, rows, out=out)
        for i in range(3):
            tokens.copy_(torch.randint(0, v, (n,), device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, rows[tokens.long()])


def test_offsets_past_32_bits(env):
    """A table of more than 2^32 bytes and elements, read at its end."""
    torch, mlh = env
    v, k = 700_000, 6656
    rows = torch.zeros((v, k), dtype=torch.float16, device="cuda")       # 9.3 GB, 4.7e9 elements
    mark = torch.randn((3, k), device="cuda").half()
    rows[-3:] = mark
    tokens = torch.tensor([v - 1, v - 3, v - 2, 0], dtype=torch.int32, device="cuda")
    with mlh.LMHead(v, k, max_batch=1, device=0) as head:
        got = head.embed(tokens, rows)
        assert torch.equal(got[:3], mark[[2, 0, 1]]) and bool((got[3] == 0).all())
    del rows, got
    torch.cuda.empty_cache()
