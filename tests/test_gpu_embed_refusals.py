"""Refusals of muse_lmhead_embed and _embed_backward on a real handle: a negative
status and nothing launched (the outputs keep what they held)."""
import math

import pytest

pytestmark = pytest.mark.gpu

NULL, SHAPE, ALIGN, VALUE, NOMEM = -1, -2, -4, -5, -8
V, K, N = 40, 256, 3


@pytest.fixture(scope="module")
def env():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    t = {"table": torch.full((V, K), 7.0, device="cuda"), "rows": torch.full((N, K), 7.0, device="cuda"),
         "tok": torch.full((N,), 7, dtype=torch.int32, device="cuda"), "work": torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda")}
    head = mlh.LMHead(V, K, max_batch=1, device=0)
    yield torch, mlh, head, t
    head.close()


def _embed(mlh, head, t, **o):
    p = {k: v.data_ptr() for k, v in t.items()}
    a = {"table": p["table"], "type": 0, "tld": K, "tok": p["tok"], "n": N, "scale": 1.0, "out": p["rows"], "otype": 0, "old": K, **o}
    return mlh.muse_lmhead_embed(head.handle, a["table"], a["type"], a["tld"], a["tok"], a["n"], a["scale"], a["out"], a["otype"], a["old"], None)


def _backward(mlh, head, t, **o):
    p = {k: v.data_ptr() for k, v in t.items()}
    a = {"grad": p["rows"], "type": 0, "gld": K, "tok": p["tok"], "n": N, "scale": 1.0, "table": p["table"], "ttype": 0, "tld": K, "acc": 0,
         "work": p["work"], "bytes": 1 << 20, **o}
    return mlh.muse_lmhead_embed_backward(head.handle, a["grad"], a["type"], a["gld"], a["tok"], a["n"], a["scale"], a["table"], a["ttype"],
                                          a["tld"], a["acc"], a["work"], a["bytes"], None)


def _unchanged(torch, t):
    torch.cuda.synchronize()
    return all(bool((v == 7).all()) for v in t.values())


def test_embed_refusals(env):
    torch, mlh, head, t = env
    p = {k: v.data_ptr() for k, v in t.items()}
    for want, o in [(NULL, {"table": None}), (NULL, {"tok": None}), (NULL, {"out": None}), (SHAPE, {"n": -1}), (SHAPE, {"n": 1 << 31}),
                    (SHAPE, {"tld": K - 1}), (SHAPE, {"old": K - 1}), (SHAPE, {"old": 1 << 61}), (VALUE, {"type": 4}), (VALUE, {"type": -1}),
                    (VALUE, {"otype": 3}), (VALUE, {"scale": math.nan}), (VALUE, {"scale": math.inf}), (ALIGN, {"table": p["table"] + 2}),
                    (ALIGN, {"table": p["table"] + 8, "type": 3}), (ALIGN, {"out": p["rows"] + 1, "otype": 1}), (ALIGN, {"tok": p["tok"] + 2})]:
        assert _embed(mlh, head, t, **o) == want, o
    assert _embed(mlh, head, t, n=0, tok=None) == 0
    assert _unchanged(torch, t)
    for call in (lambda: head.embed(t["tok"].long(), t["table"]), lambda: head.embed(t["tok"].view(1, N), t["table"]),
                 lambda: head.embed(t["tok"], t["table"][:-1]), lambda: head.embed(t["tok"], t["table"].double()),
                 lambda: head.embed(t["tok"], t["work"]), lambda: head.embed(t["tok"], t["table"], out=t["rows"][:-1]),
                 lambda: head.embed(t["tok"], t["table"], dtype=torch.float16, out=t["rows"]), lambda: head.embed(t["tok"], t["table"].t()),
                 lambda: head.embed(t["tok"], t["table"], dtype=torch.float64)):
        with pytest.raises(ValueError):
            call()


def test_embed_backward_refusals(env):
    torch, mlh, head, t = env
    p = {k: v.data_ptr() for k, v in t.items()}
    need = mlh.muse_lmhead_embed_backward_workspace(head.handle, N)
    for want, o in [(NULL, {"grad": None}), (NULL, {"tok": None}), (NULL, {"table": None}), (NULL, {"work": None}), (SHAPE, {"n": -1}),
                    (SHAPE, {"n": 1 << 31}), (SHAPE, {"gld": K - 1}), (SHAPE, {"tld": K - 1}), (VALUE, {"type": 3}), (VALUE, {"ttype": 3}),
                    (VALUE, {"scale": -math.inf}), (VALUE, {"acc": 2}), (ALIGN, {"grad": p["rows"] + 2}), (ALIGN, {"table": p["table"] + 1, "ttype": 2}),
                    (ALIGN, {"tok": p["tok"] + 1}), (ALIGN, {"work": p["work"] + 8}), (NOMEM, {"bytes": need - 1})]:
        assert _backward(mlh, head, t, **o) == want, o
    assert _backward(mlh, head, t, n=0, acc=1, tok=None, grad=None) == 0
    assert _unchanged(torch, t)
    for call in (lambda: head.embed_backward(t["rows"], t["tok"][:-1]), lambda: head.embed_backward(t["rows"], t["tok"].long()),
                 lambda: head.embed_backward(t["rows"], t["tok"], accumulate=True), lambda: head.embed_backward(t["rows"][:, :-1], t["tok"]),
                 lambda: head.embed_backward(t["rows"], t["tok"], grad_table=t["table"][:-1]),
                 lambda: head.embed_backward(t["rows"], t["tok"], dtype=torch.float16, grad_table=t["table"])):
        with pytest.raises(ValueError):
            call()
