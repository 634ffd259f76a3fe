"""Cases of the operators around the next token, with their plain forms.

Three operators, each in the form a user calls and in elementary torch operations:

* sample          the next token of each row of logits, drawn with temperature,
                  top-k, top-p and min-p from a given uniform number, and the log
                  probability that it was drawn with
* embed           rows of a token table, quantised like the head's matrix or
                  dense, times a scale
* embed_backward  the gradient by such a table from the gradient by the rows that
                  were looked up, the rows of one token added up in their order

`run` computes the plain form, or calls the package where `own` is true.
"""
import math

import torch

own = False

VOCAB, WIDTH = 202048, 6656          # the LM head of the package's default workload
CAP = 20.0
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK_BYTES = {"q5_k": 176, "q4_k": 144}


def listed():
    return [
        # one decoded token of a chat
        {"name": "sample_token", "op": "sample", "rows": 1, "vocab": VOCAB, "pad": 0, "type": "f32", "how": "chat", "masked": False},
        # the 16 positions of a verify step, from the whole distribution
        {"name": "sample_verify", "op": "sample", "rows": 16, "vocab": VOCAB, "pad": 0, "type": "f32", "how": "plain", "masked": False},
        # a full batch of the head, every row with its own request's settings
        {"name": "sample_batch", "op": "sample", "rows": 32, "vocab": VOCAB, "pad": 0, "type": "f32", "how": "mixed", "masked": False},
        # a grammar's mask over an odd vocabulary, rows at no alignment
        {"name": "sample_masked", "op": "sample", "rows": 77, "vocab": 50257, "pad": 4, "type": "bf16", "how": "nucleus", "masked": True},
        # a step of many rollouts at once
        {"name": "sample_rollouts", "op": "sample", "rows": 1024, "vocab": VOCAB, "pad": 0, "type": "bf16", "how": "nucleus", "masked": False},
        # the token that was drawn, on its way back into the model
        {"name": "embed_token", "op": "embed", "rows": 1, "vocab": VOCAB, "width": WIDTH, "table": "q4_k", "out": "f32", "scale": 1.0},
        # a long prompt
        {"name": "embed_prompt", "op": "embed", "rows": 16384, "vocab": VOCAB, "width": WIDTH, "table": "q5_k", "out": "bf16", "scale": 1.0},
        # a training batch of odd length from a dense table, scaled by the root of the width
        {"name": "embed_train", "op": "embed", "rows": 4099, "vocab": VOCAB, "width": WIDTH, "table": "bf16", "out": "bf16", "scale": WIDTH ** 0.5},
        # a short batch and a small table in 32 bits
        {"name": "embed_backward_small", "op": "embed_backward", "rows": 301, "vocab": 2048, "width": WIDTH, "grad": "f32", "out": "f32", "scale": 1.0},
        # many tokens of a small vocabulary: long runs of one token
        {"name": "embed_backward_runs", "op": "embed_backward", "rows": 16384, "vocab": 32003, "width": 1024, "grad": "f16", "out": "f32", "scale": 32.0},
        # a packed sequence against the whole table
        {"name": "embed_backward_sequence", "op": "embed_backward", "rows": 16384, "vocab": VOCAB, "width": WIDTH, "grad": "bf16", "out": "bf16", "scale": WIDTH ** 0.5},
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["sample", "embed", "embed_backward"])
    vocab = _spread(rng, 1000, VOCAB)
    if op == "sample":
        kind = rng.choice(["f32", "f32", "bf16", "f16"])
        return {"op": op, "rows": _spread(rng, 1, 512 if kind == "f32" else 1024), "vocab": vocab, "pad": rng.choice([0, 0, 0, 1, 4, 6]), "type": kind,
                "how": rng.choice(["plain", "chat", "nucleus", "floor", "mixed"]), "masked": rng.random() < 0.3}
    width = 256 * rng.choice([4, 7, 10, 16, 20, 26])
    scale = rng.choice([1.0, width ** 0.5])
    if op == "embed":
        return {"op": op, "rows": _spread(rng, 1, 16384), "vocab": vocab, "width": width, "table": rng.choice(["q5_k", "q4_k", "f32", "bf16", "f16"]),
                "out": rng.choice(["f32", "bf16", "f16"]), "scale": scale}
    grad, out = rng.choice(["f32", "bf16", "f16"]), rng.choice(["f32", "bf16", "f16"])
    return {"op": op, "rows": _spread(rng, 1, 8192 if grad == "f32" else 16384), "vocab": min(vocab, VOCAB // 2 - 4000) if out == "f32" else vocab,
            "width": width, "grad": grad, "out": out, "scale": scale}


# ---------------------------------------------------------------- inputs
def _settings(how, n, gen, dev):
    """Temperature, top-k, top-p and min-p: numbers for all rows, or a tensor each."""
    if how == "plain":
        return {"temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0}
    if how == "chat":
        return {"temperature": 0.75, "top_k": 50, "top_p": 0.9375, "min_p": 0.0}
    if how == "nucleus":
        return {"temperature": 1.0, "top_k": 0, "top_p": 0.9375, "min_p": 0.0}
    if how == "floor":
        return {"temperature": 1.25, "top_k": 0, "top_p": 1.0, "min_p": 0.0625}
    pick = lambda values, dtype: torch.tensor(values, dtype=dtype, device=dev)[torch.randint(0, len(values), (n,), generator=gen, device=dev)]     # noqa: E731
    return {"temperature": pick([0.0, 0.625, 0.75, 1.0, 1.25], torch.float32), "top_k": pick([0, 0, 20, 50, 200], torch.int32),
            "top_p": pick([1.0, 1.0, 0.875, 0.9375], torch.float32), "min_p": pick([0.0, 0.0, 0.03125, 0.125], torch.float32)}


def _tokens(n, v, gen, dev):
    """Tokens as a text has them: the r-th most frequent one with a share of about 1 / r."""
    rank = torch.exp(torch.rand((n,), generator=gen, device=dev, dtype=torch.float64) * math.log(v + 1)).long().clamp(1, v) - 1
    step = int(0.618 * v) | 1
    while math.gcd(step, v) != 1:
        step += 2
    at = torch.randint(0, v, (1,), generator=gen, device=dev)
    tok = (rank * step + at) % v
    if n > 4:
        tok[3] = -1                                           # a padded position
    return tok.to(torch.int32)


def _table(v, k, kind, gen, dev):
    if kind not in BLOCK_BYTES:
        return torch.randn((v, k), generator=gen, device=dev, dtype=TYPES[kind])
    nb, size = k // 256, BLOCK_BYTES[kind]
    w = torch.randint(0, 256, (v, nb, size), generator=gen, device=dev, dtype=torch.uint8)
    d = (torch.rand((v, nb), generator=gen, device=dev) * 8e-4 + 2e-4).half()
    mid = 15.5 if kind == "q5_k" else 7.5                     # the mins take off the quants' middle
    dmin = (d.float() * mid * (torch.rand((v, nb), generator=gen, device=dev) * 0.4 + 0.8)).half()
    w[:, :, 0:2] = d.unsqueeze(-1).view(torch.uint8)
    w[:, :, 2:4] = dmin.unsqueeze(-1).view(torch.uint8)
    w[:, :, 8:12] = w[:, :, 4:8]                              # a sub-block's min goes with its scale
    low = w[:, :, 12:16] & 15
    w[:, :, 12:16] = low | (low << 4)
    return w.reshape(-1)


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 29)
    n, v = case["rows"], case["vocab"]
    s = dict(case)
    if case["op"] == "sample":
        x = torch.randn((n, v + case["pad"]), generator=gen, device=dev) * 2.5
        likely = torch.randint(0, v, (n, 48), generator=gen, device=dev)
        x.scatter_add_(1, likely, torch.rand((n, 48), generator=gen, device=dev) * 9.0 + 4.0)   # what the model thinks comes next
        x = CAP * torch.tanh(x * (1.0 / CAP))
        x = x.to(TYPES[case["type"]])[:, :v]
        if case["masked"]:
            keep = torch.rand((n, v), generator=gen, device=dev) < 0.1
            keep[:, :16] = True
            x.masked_fill_(~keep, -math.inf)
        s["x"] = x
        s["uniforms"] = torch.rand((n,), generator=gen, device=dev)
        s["settings"] = _settings(case["how"], n, gen, dev)
    else:
        k = case["width"]
        s["tokens"] = _tokens(n, v, gen, dev)
        if case["op"] == "embed":
            s["rows_of"] = _table(v, k, case["table"], gen, dev)
        else:
            s["gradient"] = torch.randn((n, k), generator=gen, device=dev, dtype=TYPES[case["grad"]])
    if own:
        import q5_lm_head_gb300 as lm
        s["head"] = lm.LMHead(v, case.get("width", WIDTH), max_batch=1, device=0, fmt=case["table"] if case.get("table") in BLOCK_BYTES else "q5_k")
    return s


# ---------------------------------------------------------------- plain forms
def _column(value, n, dev):
    """A setting as a column: 32 bits as the caller gives it, 64 to count with."""
    if not torch.is_tensor(value):
        value = torch.full((n,), value, device=dev, dtype=torch.float32)
    return value.double().unsqueeze(1)


def _sample(x, uniforms, temperature, top_k, top_p, min_p):
    """Sums of a row's probabilities in 64 bits: the number drawn lies next to a border."""
    tokens, logprobs = [], []
    for lo in range(0, x.shape[0], 64):
        xs = x[lo:lo + 64].float()
        n, v = xs.shape
        part = lambda s: _column(s[lo:lo + 64] if torch.is_tensor(s) else s, n, x.device)      # noqa: E731
        t, k, p, mp, u = part(temperature), part(top_k), part(top_p), part(min_p), part(uniforms)
        greedy = t == 0
        t = torch.where(greedy, torch.ones_like(t), t)
        k = torch.where(greedy, torch.ones_like(k), k)
        m = xs.max(dim=1, keepdim=True).values.double()
        w = ((xs.double() - m) / t).exp()
        if torch.is_tensor(top_k) or top_k > 0 or top_p < 1:
            order = xs.sort(dim=1, descending=True, stable=True).indices
            place = torch.arange(v, device=x.device)
            ws = torch.where((k <= 0) | (place < k), w.gather(1, order), torch.zeros_like(w))
            upto = ws.cumsum(dim=1)
            before = torch.cat([torch.zeros_like(m), upto[:, :-1]], dim=1)
            keep = (ws > 0) & ((p >= 1) | (before < p * upto[:, -1:]) | (place == 0))
            keep = torch.zeros_like(keep).scatter(1, order, keep)
        else:
            keep = w > 0
        if torch.is_tensor(min_p) or min_p > 0:
            keep = keep & ((mp <= 0) | (xs.double() >= m + t * mp.log()))
        w = torch.where(keep, w, torch.zeros_like(w))
        upto = w.cumsum(dim=1)
        total = upto[:, -1:]
        token = (upto > u * total).to(torch.uint8).argmax(dim=1, keepdim=True)
        tokens.append(token.squeeze(1).to(torch.int32))
        logprobs.append((w.gather(1, token) / total).log().squeeze(1).float())
    return torch.cat(tokens), torch.cat(logprobs)


def _dequantise(b, fmt):
    """Blocks [n, blocks, bytes] to values."""
    n, nb, _ = b.shape
    dd = b[:, :, 0:4].contiguous().view(torch.float16).float()
    lo6, lo4 = b[:, :, 4:12] & 63, b[:, :, 12:16]
    high = b[:, :, 4:12] >> 6
    sc = torch.cat([lo6[:, :, :4], (lo4 & 15) | (high[:, :, :4] << 4)], dim=2)
    mn = torch.cat([lo6[:, :, 4:], (lo4 >> 4) | (high[:, :, 4:] << 4)], dim=2)
    qs = b[:, :, (48 if fmt == "q5_k" else 16):].reshape(n, nb, 4, 32)
    q = torch.stack([qs & 15, qs >> 4], dim=3).reshape(n, nb, 8, 32)
    if fmt == "q5_k":
        shift = torch.arange(8, dtype=torch.uint8, device=b.device).reshape(1, 1, 8, 1)
        q = q | (((b[:, :, 16:48].unsqueeze(2) >> shift) & 1) << 4)
    w = (dd[:, :, :1] * sc.float()).unsqueeze(3) * q.float() - (dd[:, :, 1:] * mn.float()).unsqueeze(3)
    return w.reshape(n, nb * 256)


def _embed(table, tokens, fmt, v, k, scale, out):
    ok = (tokens >= 0) & (tokens < v)
    at = torch.where(ok, tokens, torch.zeros_like(tokens)).long()
    rows = _dequantise(table.reshape(v, k // 256, BLOCK_BYTES[fmt])[at], fmt) if fmt in BLOCK_BYTES else table[at].float()
    return torch.where(ok.unsqueeze(1), rows * scale, torch.zeros_like(rows)).to(out)


def _embed_backward(grad, tokens, v, scale, out):
    ok = (tokens >= 0) & (tokens < v)
    sums = torch.zeros((v, grad.shape[1]), dtype=torch.float32, device=grad.device)
    sums.index_add_(0, torch.where(ok, tokens, torch.zeros_like(tokens)).long(), torch.where(ok.unsqueeze(1), grad.float(), 0.0))
    return (sums * scale).to(out)


def run(state):
    s = state
    if s["op"] == "sample":
        if own:
            return s["head"].sample(s["x"], s["uniforms"], **s["settings"])
        return _sample(s["x"], s["uniforms"], **s["settings"])
    if s["op"] == "embed":
        if own:
            return s["head"].embed(s["tokens"], s["rows_of"], scale=s["scale"], dtype=TYPES[s["out"]])
        return _embed(s["rows_of"], s["tokens"], s["table"], s["vocab"], s["width"], s["scale"], TYPES[s["out"]])
    if own:
        return s["head"].embed_backward(s["gradient"], s["tokens"], scale=s["scale"], dtype=TYPES[s["out"]])
    return _embed_backward(s["gradient"], s["tokens"], s["vocab"], s["scale"], TYPES[s["out"]])


def work(case):
    n, v = case["rows"], case["vocab"]
    if case["op"] == "sample":
        return {"bytes": n * (v * (4 if case["type"] == "f32" else 2) + 12 + (16 if case["how"] == "mixed" else 0)), "flops": 4 * n * v}
    k = case["width"]
    size = lambda kind: k // 256 * BLOCK_BYTES[kind] if kind in BLOCK_BYTES else k * (4 if kind == "f32" else 2)     # noqa: E731
    if case["op"] == "embed":
        rows = min(n, _different(n, v))                       # a table's row is read once, however often its token comes
        return {"bytes": rows * size(case["table"]) + n * (size(case["out"]) + 4), "flops": 2 * n * k}
    return {"bytes": n * (size(case["grad"]) + 4) + v * size(case["out"]), "flops": n * k}


def _different(n, v):
    """Different tokens that n draws with shares of 1 / r have, on average: the sum of 1 - exp(-n / (r ln v))."""
    total, lo = 0.0, 1
    while lo <= v:                                            # ranks in steps of an eighth
        hi = min(v, max(lo, lo + lo // 8))
        total += (hi - lo + 1) * (1 - math.exp(-n / (0.5 * (lo + hi) * math.log(v + 1))))
        lo = hi + 1
    return max(1, int(total))


# ---------------------------------------------------------------- 64 bits, from the definitions
def exact(case, seed):
    plan = prepare(case, seed)
    n, v = case["rows"], case["vocab"]
    if case["op"] == "sample":
        return _exact_sample(plan, n)
    k = case["width"]
    tok = plan["tokens"].long()
    used = (tok >= 0).nonzero().squeeze(1)
    if case["op"] == "embed":
        out = torch.zeros((n, k), dtype=torch.float64, device=tok.device)
        for lo in range(0, used.numel(), 2048):
            at = used[lo:lo + 2048]
            out[at] = _exact_rows(plan["rows_of"], tok[at], case["table"], v, k) * case["scale"]
        return out
    out = torch.zeros((v, k), dtype=torch.float64, device=tok.device)
    order = tok[used].argsort(stable=True)
    at, tok = used[order], tok[used][order]
    ids, counts = torch.unique_consecutive(tok, return_counts=True)
    ends = counts.cumsum(0)
    start, few = ends - counts, counts <= 8
    long_runs = [(i, int(start[i]), int(ends[i])) for i in (~few).nonzero().squeeze(1).tolist()]
    for lo in range(0, k, 512):
        g = plan["gradient"][at, lo:lo + 512].double() * case["scale"]
        part = torch.zeros((ids.numel(), g.shape[1]), dtype=torch.float64, device=g.device)
        for j in range(8):
            has = few & (counts > j)
            part[has] += g[start[has] + j]
        for i, first, end in long_runs:
            part[i] = g[first:end].sum(dim=0)
        out[ids, lo:lo + 512] = part
    return out


def _exact_sample(plan, n):
    tokens, logprobs = [], []
    value = lambda name, r: float(plan["settings"][name][r]) if torch.is_tensor(plan["settings"][name]) else float(plan["settings"][name])     # noqa: E731
    for r in range(n):
        x = plan["x"][r].double()
        t, k, p, mp = (value(name, r) for name in ("temperature", "top_k", "top_p", "min_p"))
        if t == 0:                                            # the first of the largest
            tokens.append((x == x.max()).nonzero()[0, 0])
            logprobs.append(torch.zeros((), dtype=torch.float64, device=x.device))
            continue
        logq = torch.log_softmax(x / t, dim=0)
        kept = torch.argsort(x, descending=True, stable=True)
        if k > 0:
            kept = kept[:int(k)]
        if p < 1:
            share = torch.softmax(logq[kept], dim=0)
            full = (torch.cumsum(share, 0) >= p).nonzero()    # the first prefix that holds p
            if full.numel():
                kept = kept[:int(full[0, 0]) + 1]
        if mp > 0:
            kept = kept[logq[kept] >= logq.max() + math.log(mp)]
        kept = kept[logq[kept] > -math.inf].sort().values
        norm = torch.logsumexp(logq[kept], dim=0)
        upto = torch.cumsum((logq[kept] - norm).exp(), 0)
        at = torch.searchsorted(upto, plan["uniforms"][r].double() * upto[-1], right=True).clamp(max=kept.numel() - 1)
        tokens.append(kept[at])
        logprobs.append(logq[kept[at]] - norm)
    return torch.stack(tokens).to(torch.int32), torch.stack(logprobs)


def _exact_rows(table, tok, fmt, v, k):
    if fmt not in BLOCK_BYTES:
        return table[tok].double()
    raw = table.reshape(v, k // 256, BLOCK_BYTES[fmt])[tok]
    half = raw[:, :, :4].contiguous().view(torch.float16).double()
    b = raw.to(torch.int32)
    out = torch.empty((tok.numel(), k // 256, 8, 32), dtype=torch.float64, device=tok.device)
    for j in range(8):                                        # sub-block j: 6 bits of scale and of min, its nibbles and high bits
        if j < 4:
            sc, mn = b[:, :, 4 + j] % 64, b[:, :, 8 + j] % 64
        else:
            sc = b[:, :, 8 + j] % 16 + 16 * (b[:, :, j] // 64)
            mn = b[:, :, 8 + j] // 16 + 16 * (b[:, :, 4 + j] // 64)
        first = (48 if fmt == "q5_k" else 16) + 32 * (j // 2)
        q = (b[:, :, first:first + 32] // (16 if j % 2 else 1)) % 16
        if fmt == "q5_k":
            q = q + 16 * ((b[:, :, 16:48] // (1 << j)) % 2)
        out[:, :, j, :] = (half[:, :, 0] * sc).unsqueeze(2) * q - (half[:, :, 1] * mn).unsqueeze(2)
    return out.reshape(tok.numel(), k)
