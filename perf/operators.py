"""Cases of the output stage's scoring and training operators, with their plain forms.

Three operators, each in the form a user calls and in elementary torch operations:

* score     log probabilities of given tokens over the capped logits, with the
            normaliser, the entropy, the token's rank and the top alternatives
* distill   distillation from a teacher's top alternatives: the loss of each row
            and its gradient by the student's logits
* backward  the output stage's backward pass: the gradient by the logits back
            through cap, scale, the quantised matrix and the final norm

`run` computes the plain form, or calls the package where `own` is true.
"""
import math

import torch

own = False

VOCAB, WIDTH = 202048, 6656          # the LM head of the package's default workload
SCALE, CAP, EPS = 0.196116, 20.0, 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK_BYTES = {"q5_k": 176, "q4_k": 144}


def listed():
    return [
        # one decoded token with the alternatives an API returns
        {"name": "score_token", "op": "score", "rows": 1, "vocab": VOCAB, "pad": 0, "type": "f32", "top": 20, "temperature": 1.0, "masked": False},
        # the 16 positions of a verify step
        {"name": "score_verify", "op": "score", "rows": 16, "vocab": VOCAB, "pad": 0, "type": "f32", "top": 8, "temperature": 0.7, "masked": False},
        # a grammar's mask over an odd vocabulary, rows at no alignment
        {"name": "score_masked", "op": "score", "rows": 77, "vocab": 50257, "pad": 4, "type": "bf16", "top": 64, "temperature": 1.0, "masked": True},
        # a scored document: one row for each of its positions
        {"name": "score_document", "op": "score", "rows": 1024, "vocab": VOCAB, "pad": 0, "type": "f32", "top": 5, "temperature": 1.0, "masked": False},
        # one full batch of the head as a training step, the tail as one more class
        {"name": "distill_batch", "op": "distill", "rows": 32, "vocab": VOCAB, "pad": 0, "type": "f32", "top": 32, "temperature": 1.0, "tail": True, "grad": True},
        # a packed sequence of 1,024 positions in 16 bits
        {"name": "distill_sequence", "op": "distill", "rows": 1024, "vocab": VOCAB, "pad": 0, "type": "bf16", "top": 64, "temperature": 2.0, "tail": False, "grad": True},
        # a validation pass: the loss alone, odd sizes
        {"name": "distill_validate", "op": "distill", "rows": 301, "vocab": 32003, "pad": 0, "type": "f16", "top": 16, "temperature": 1.0, "tail": True, "grad": False},
        # the head's backward pass: one position, a full batch, the 4-bit head, a small matrix without a cap
        {"name": "backward_one", "op": "backward", "rows": 1, "vocab": VOCAB, "width": WIDTH, "format": "q5_k", "cap": CAP, "norm": True},
        {"name": "backward_batch", "op": "backward", "rows": 32, "vocab": VOCAB, "width": WIDTH, "format": "q5_k", "cap": CAP, "norm": True},
        {"name": "backward_q4k", "op": "backward", "rows": 8, "vocab": VOCAB, "width": WIDTH, "format": "q4_k", "cap": CAP, "norm": True},
        {"name": "backward_small", "op": "backward", "rows": 5, "vocab": 2048, "width": WIDTH, "format": "q5_k", "cap": 0.0, "norm": False},
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["score", "distill", "backward"])
    if op == "backward":
        width = 256 * rng.choice([4, 7, 10, 16, 20, 26])
        return {"op": op, "rows": _spread(rng, 1, 32), "vocab": _spread(rng, 1000, VOCAB), "width": width, "format": rng.choice(["q5_k", "q4_k"]),
                "cap": rng.choice([CAP, 0.0]), "norm": rng.random() < 0.7}
    vocab = _spread(rng, 1000, VOCAB)
    rows = _spread(rng, 1, 1024)
    case = {"op": op, "rows": rows, "vocab": vocab, "pad": rng.choice([0, 0, 0, 1, 4, 6]), "type": rng.choice(["f32", "f32", "bf16", "f16"]),
            "top": rng.choice([1, 3, 5, 8, 20, 33, 64]), "temperature": rng.choice([1.0, 0.7, 2.0])}
    if case["type"] == "f32" and op == "distill":    # no more bytes than the largest listed one
        case["rows"] = max(1, rows // 2)
    if op == "score":
        case["masked"] = rng.random() < 0.3
    else:
        case["tail"], case["grad"] = rng.random() < 0.5, rng.random() < 0.8
    return case


# ---------------------------------------------------------------- inputs
def _logits(n, v, pad, dtype, gen, dev):
    x = torch.randn((n, v + pad), generator=gen, device=dev) * 3.0
    x = CAP * torch.tanh(x * (1.0 / CAP))
    return x.to(dtype)[:, :v]


def _weights(n, k, fmt, gen, dev):
    """Blocks whose weights lie around zero, as a checkpoint's do: the mins take off the quants' middle."""
    nb, size = k // 256, BLOCK_BYTES[fmt]
    w = torch.randint(0, 256, (n, nb, size), generator=gen, device=dev, dtype=torch.uint8)
    d = (torch.rand((n, nb), generator=gen, device=dev) * 8e-4 + 2e-4).half()
    mid = 15.5 if fmt == "q5_k" else 7.5
    dmin = (d.float() * mid * (torch.rand((n, nb), generator=gen, device=dev) * 0.4 + 0.8)).half()
    w[:, :, 0:2] = d.unsqueeze(-1).view(torch.uint8)
    w[:, :, 2:4] = dmin.unsqueeze(-1).view(torch.uint8)
    w[:, :, 8:12] = w[:, :, 4:8]                              # a sub-block's min goes with its scale
    low = w[:, :, 12:16] & 15
    w[:, :, 12:16] = low | (low << 4)
    return w


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 17)
    n, v = case["rows"], case["vocab"]
    s = dict(case)
    if case["op"] == "backward":
        k = case["width"]
        s["weights"] = _weights(n=v, k=k, fmt=case["format"], gen=gen, dev=dev).reshape(-1)
        s["hidden"] = torch.randn((n, k), generator=gen, device=dev) * (torch.rand((n, 1), generator=gen, device=dev) * 3.5 + 0.5)
        s["gamma"] = 1.0 + 0.1 * torch.randn((k,), generator=gen, device=dev) if case["norm"] else None
        s["logits"] = _logits(n, v, 0, torch.float32, gen, dev).contiguous()
        g = torch.softmax(s["logits"], dim=1)
        at = torch.randint(0, v, (n, 32), generator=gen, device=dev)
        g = g.scatter_add(1, at, -torch.softmax(torch.randn((n, 32), generator=gen, device=dev) * 2, dim=1))
        s["grad_logits"] = (g / n).contiguous()
    else:
        top = case["top"]
        x = _logits(n, v, case["pad"], TYPES[case["type"]], gen, dev)
        if case["op"] == "score":
            if case["masked"]:
                keep = torch.rand((n, v), generator=gen, device=dev) < 0.1
                keep[:, : 2 * top] = True
                x.masked_fill_(~keep, -math.inf)
            tok = torch.randint(0, v, (n,), generator=gen, device=dev)
            best = x.float().argmax(dim=1)
            tok = torch.where(torch.rand((n,), generator=gen, device=dev) < 0.6, best, tok)
            if n > 4:
                tok[3] = -1                                   # a padded row
            s["tokens"] = tok.to(torch.int32)
        else:
            start = torch.randint(0, v, (n, 1), generator=gen, device=dev)
            step = torch.randint(1, max(2, v // (top + 1)), (n, 1), generator=gen, device=dev)
            ids = (start + step * torch.arange(top, device=dev)) % v
            u = torch.randn((n, top), generator=gen, device=dev) * 2
            x.scatter_add_(1, ids, (u + 4.0).to(x.dtype))      # the student knows some of it
            u = (u + 0.5 * torch.randn((n, top), generator=gen, device=dev)).sort(dim=1, descending=True).values
            lp = torch.log_softmax(u, dim=1) + math.log(0.9)
            if n > 4 and top > 2:
                ids[1, top - 1] = -1                          # a teacher with fewer alternatives
            w = torch.rand((n,), generator=gen, device=dev) * 0.5 + 0.75
            if n > 4:
                w[2] = 0.0                                    # a row of the prompt
            s["ids"], s["lp"], s["weight"] = ids.to(torch.int32), lp.contiguous(), w / n
        s["x"] = x
    if own:
        import q5_lm_head_gb300 as lm
        s["head"] = lm.LMHead(v, case.get("width", WIDTH), max_batch=min(n, 32), device=0, fmt=case.get("format", "q5_k"))
    return s


# ---------------------------------------------------------------- plain forms, 32 bits
def _keys(x):
    """A whole number for each value that orders as (value, lower index first)."""
    bits = (x + 0.0).view(torch.int32)
    order = bits ^ ((bits >> 31) & 0x7FFFFFFF)
    return order.long() * 4294967296 + (x.shape[1] - 1 - torch.arange(x.shape[1], device=x.device))


def _score(x, tokens, top, temperature):
    x = x.float()
    z = x / temperature
    m = z.max(dim=1, keepdim=True).values
    lse = m + (z - m).exp().sum(dim=1, keepdim=True).log()
    lp = z - lse
    p = lp.exp()
    entropy = -(torch.where(p > 0, lp, torch.zeros_like(lp)) * p).sum(dim=1)
    has = tokens >= 0
    at = tokens.clamp(min=0).long().unsqueeze(1)
    got = x.gather(1, at)
    before = torch.arange(x.shape[1], device=x.device) < at
    rank = ((x > got) | ((x == got) & before)).sum(dim=1)
    logprob = torch.where(has, lp.gather(1, at).squeeze(1), torch.zeros_like(entropy))
    rank = torch.where(has, rank, torch.full_like(rank, -1)).to(torch.int32)
    ids = _keys(x).topk(top, dim=1).indices
    return logprob, rank, lse.squeeze(1), entropy, ids.to(torch.int32), lp.gather(1, ids)


def _distill(x, ids, lp, weight, temperature, tail, want_grad):
    n, v = x.shape
    z = x.float() / temperature
    m = z.max(dim=1, keepdim=True).values
    e = (z - m).exp()
    total = e.sum(dim=1, keepdim=True)
    logq = z - m - total.log()
    ok = (ids >= 0) & (ids < v)
    at = torch.where(ok, ids, torch.zeros_like(ids)).long()
    lp = torch.where(ok, lp, torch.full_like(lp, -math.inf))
    if tail:
        p = lp.exp()
    else:
        p = (lp - lp.max(dim=1, keepdim=True).values).exp()
        p = p / p.sum(dim=1, keepdim=True)
    loss = torch.where(p > 0, p * (p.log() - logq.gather(1, at)), torch.zeros_like(p)).sum(dim=1)
    mass = p.sum(dim=1, keepdim=True)
    factor = mass
    if tail:
        out = torch.zeros((n, v + 1), dtype=torch.bool, device=x.device)
        out = ~out.scatter(1, torch.where(ok, at, torch.full_like(at, v)), True)[:, :v]
        rest = (e * out).sum(dim=1, keepdim=True) / total
        pt = (1.0 - mass).clamp(min=0.0)
        loss = loss + torch.where(pt > 0, pt * (pt.log() - rest.log()), torch.zeros_like(pt)).squeeze(1)
        factor = (mass + pt) - out * (pt / rest)
    loss = loss * weight
    if not want_grad:
        return loss, None
    grad = (e / total * factor).scatter_add(1, at, -p) * (weight.unsqueeze(1) / temperature)
    return loss, grad.to(x.dtype)


def _dequantise(raw, n, k, fmt):
    b = raw.reshape(n, k // 256, BLOCK_BYTES[fmt])
    dd = b[:, :, 0:4].contiguous().view(torch.float16).float()
    lo6, lo4 = b[:, :, 4:12] & 63, b[:, :, 12:16]
    high = b[:, :, 4:12] >> 6
    sc = torch.cat([lo6[:, :, :4], (lo4 & 15) | (high[:, :, :4] << 4)], dim=2)
    mn = torch.cat([lo6[:, :, 4:], (lo4 >> 4) | (high[:, :, 4:] << 4)], dim=2)
    qs = b[:, :, (48 if fmt == "q5_k" else 16):].reshape(n, k // 256, 4, 32)
    q = torch.stack([qs & 15, qs >> 4], dim=3).reshape(n, k // 256, 8, 32)
    if fmt == "q5_k":
        shift = torch.arange(8, dtype=torch.uint8, device=raw.device).reshape(1, 1, 8, 1)
        q = q | (((b[:, :, 16:48].unsqueeze(2) >> shift) & 1) << 4)
    w = (dd[:, :, :1] * sc.float()).unsqueeze(3) * q.float() - (dd[:, :, 1:] * mn.float()).unsqueeze(3)
    return w.reshape(n, k)


def _backward(s):
    g = s["grad_logits"]
    if s["cap"] > 0:
        g = g * ((s["cap"] - s["logits"]) * (s["cap"] + s["logits"]) / (s["cap"] * s["cap"]))
    g = g * SCALE
    gx = g @ _dequantise(s["weights"], s["vocab"], s["width"], s["format"])
    if s["gamma"] is None:
        return gx, None
    h = s["hidden"]
    r = 1.0 / ((h * h).mean(dim=1, keepdim=True) + EPS).sqrt()
    hat, gg = h * r, gx * s["gamma"]
    return r * (gg - hat * (gg * hat).mean(dim=1, keepdim=True)), (gx * hat).sum(dim=0)


def run(state):
    s = state
    if s["op"] == "score":
        if own:
            return tuple(s["head"].score(s["x"], tokens=s["tokens"], n_top=s["top"], temperature=s["temperature"]))
        return _score(s["x"], s["tokens"], s["top"], s["temperature"])
    if s["op"] == "distill":
        if own:
            return s["head"].distill(s["x"], s["ids"], s["lp"], row_weight=s["weight"], temperature=s["temperature"], tail=s["tail"], want_grad=s["grad"])
        return _distill(s["x"], s["ids"], s["lp"], s["weight"], s["temperature"], s["tail"], s["grad"])
    if own:
        return s["head"].backward(s["grad_logits"], s["weights"], logits=s["logits"] if s["cap"] > 0 else None, hidden=s["hidden"] if s["norm"] else None,
                                  gamma=s["gamma"], eps=EPS, scale=SCALE, cap=s["cap"])
    return _backward(s)


def work(case):
    n, v = case["rows"], case["vocab"]
    if case["op"] == "backward":
        k = case["width"]
        acts = 4 * n * v * (2 if case["cap"] > 0 else 1) + 4 * n * k * (2 if case["norm"] else 1) + (8 * k if case["norm"] else 0)
        return {"bytes": v * (k // 256) * BLOCK_BYTES[case["format"]] + acts, "flops": 2 * n * v * k}
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "score":
        return {"bytes": n * (v * size + 4 + 16 + 8 * case["top"]), "flops": 5 * n * v}
    return {"bytes": n * (v * size * (2 if case["grad"] else 1) + 8 * case["top"] + 8), "flops": (6 if case["grad"] else 3) * n * v}


# ---------------------------------------------------------------- 64 bits, from the definitions
def exact(case, seed):
    plan = prepare(case, seed)
    n, v = case["rows"], case["vocab"]
    if case["op"] == "backward":
        return _exact_backward(plan, n, v, case["width"])
    outs = []
    for lo in range(0, n, 128):                               # 128 rows at a time: 64 bits of a large vocabulary are much
        x = plan["x"][lo:lo + 128].double()
        logq = torch.log_softmax(x / case["temperature"], dim=1)
        if case["op"] == "score":
            tok = plan["tokens"][lo:lo + 128].long()
            order = torch.sort(x, dim=1, descending=True, stable=True).indices
            place = torch.argsort(order, dim=1)
            row = torch.arange(x.shape[0], device=x.device)
            q = logq.exp()
            ent = -torch.nan_to_num(q * logq, nan=0.0).sum(dim=1)
            lse = torch.logsumexp(x / case["temperature"], dim=1)
            none = tok < 0
            lp, rank = logq[row, tok], place[row, tok].to(torch.int32)
            lp[none], rank[none] = 0.0, -1
            ids = order[:, :case["top"]]
            outs.append((lp, rank, lse, ent, ids.to(torch.int32), torch.stack([logq[row, ids[:, j]] for j in range(case["top"])], dim=1)))
            continue
        ids, lp = plan["ids"][lo:lo + 128].long(), plan["lp"][lo:lo + 128].double()
        w = plan["weight"][lo:lo + 128].double()
        q = logq.exp()
        loss, grad = torch.zeros_like(w), torch.zeros_like(q)
        p = torch.where(ids >= 0, lp.exp(), 0.0)
        if not case["tail"]:
            p /= p.sum(dim=1, keepdim=True)
        row = torch.arange(x.shape[0], device=x.device)
        named = torch.zeros_like(q)
        for j in range(case["top"]):                          # d/dz of p (log p - log q_i) is p (q - one at i)
            i, pj = ids[:, j].clamp(min=0), p[:, j]
            loss += torch.where(pj > 0, pj * (pj.clamp(min=1e-300).log() - logq[row, i]), 0.0)
            grad += pj.unsqueeze(1) * q
            grad[row, i] -= pj
            named[row, i] = torch.where(ids[:, j] >= 0, 1.0, named[row, i])
        if case["tail"]:                                      # the rest is one class: d/dz of -pt log qt is pt (q - q / qt where it is in the rest)
            rest = q * (1.0 - named)
            qt, pt = rest.sum(dim=1), 1.0 - p.sum(dim=1)
            loss += pt * (pt.log() - qt.log())
            grad += pt.unsqueeze(1) * (q - rest / qt.unsqueeze(1))
        outs.append((loss * w, grad * (w / case["temperature"]).unsqueeze(1)) if case["grad"] else (loss * w,))
    got = [torch.cat(o) for o in zip(*outs)]
    return tuple(got) if case["op"] == "score" or case["grad"] else (got[0], None)


def _exact_backward(plan, n, v, k):
    nb, size, q5 = k // 256, BLOCK_BYTES[plan["format"]], plan["format"] == "q5_k"
    raw = plan["weights"].reshape(v, nb, size)
    g = plan["grad_logits"].double() * SCALE
    if plan["cap"] > 0:
        g = g * (1.0 - (plan["logits"].double() / plan["cap"]) ** 2)
    gx = torch.zeros((n, nb, 8, 32), dtype=torch.float64, device=g.device)
    for lo in range(0, v, 16384):
        b, gg = raw[lo:lo + 16384].to(torch.int32), g[:, lo:lo + 16384]
        half = raw[lo:lo + 16384, :, :4].contiguous().view(torch.float16).double()
        d, dmin = half[:, :, 0], half[:, :, 1]
        for j in range(8):
            if j < 4:
                sc, mn = b[:, :, 4 + j] % 64, b[:, :, 8 + j] % 64
            else:
                sc = b[:, :, 8 + j] % 16 + 16 * (b[:, :, j] // 64)
                mn = b[:, :, 8 + j] // 16 + 16 * (b[:, :, 4 + j] // 64)
            first = (48 if q5 else 16) + 32 * (j // 2)
            q = (b[:, :, first:first + 32] // (16 if j % 2 else 1)) % 16
            if q5:
                q = q + 16 * ((b[:, :, 16:48] // (1 << j)) % 2)
            w = (d * sc).unsqueeze(2) * q - (dmin * mn).unsqueeze(2)
            gx[:, :, j, :] += (gg @ w.reshape(w.shape[0], -1)).reshape(n, nb, 32)
    gx = gx.reshape(n, k)
    if plan["gamma"] is None:
        return gx, None
    h, gamma = plan["hidden"].double(), plan["gamma"].double()
    rms = (h.square().mean(dim=1, keepdim=True) + EPS).sqrt()
    by_x = gx * gamma
    return by_x / rms - h * (by_x * h).sum(dim=1, keepdim=True) / (k * rms ** 3), (gx * h / rms).sum(dim=0)
