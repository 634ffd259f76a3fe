"""Refusals of muse_lmhead_score, _forward_score, _distill and _backward on a
real handle: a negative status and nothing launched (the outputs keep what they
held)."""
import math

import pytest

pytestmark = pytest.mark.gpu

NULL, SHAPE, BATCH, ALIGN, VALUE = -1, -2, -3, -4, -5
V, K, N = 512, 256, 2


@pytest.fixture(scope="module")
def env():
    import torch
    import q5_lm_head_gb300 as mlh
    from q5_lm_head_gb300 import _build
    _build.build()
    mlh.load_library()
    torch.cuda.set_device(0)
    f = lambda *s: torch.full(s, 7.0, device="cuda")                                       # noqa: E731
    i = lambda *s: torch.full(s, 7, device="cuda", dtype=torch.int32)                      # noqa: E731
    t = {"x": f(N, V), "tok": i(N), "lp": f(N), "rank": i(N), "lse": f(N), "ent": f(N), "ids": i(N, 4), "top": f(N, 4),
         "hid": f(N, K), "w": torch.zeros(V * 176, dtype=torch.uint8, device="cuda"), "gamma": f(K), "loss": f(N),
         "grad": f(N, V), "gh": f(N, K), "gg": f(K)}
    head = mlh.LMHead(V, K, max_batch=N, device=0)
    yield torch, mlh, head, t
    head.close()


def _score(mlh, h, t, **o):
    p = {k: v.data_ptr() for k, v in t.items()}
    a = {"x": p["x"], "dtype": 0, "n": N, "ld": V, "tok": p["tok"], "T": 1.0, "k": 4, "lp": p["lp"], "rank": p["rank"],
         "lse": p["lse"], "ent": p["ent"], "ids": p["ids"], "top": p["top"], **o}
    return mlh.muse_lmhead_score(h, a["x"], a["dtype"], a["n"], a["ld"], a["tok"], a["T"], a["k"], a["lp"], a["rank"],
                                 a["lse"], a["ent"], a["ids"], a["top"], None)


def _distill(mlh, h, t, **o):
    p = {k: v.data_ptr() for k, v in t.items()}
    a = {"x": p["x"], "dtype": 0, "n": N, "ld": V, "ids": p["ids"], "top": p["top"], "k": 4, "tail": 1, "w": None, "T": 1.0,
         "loss": p["loss"], "grad": p["grad"], "gld": V, **o}
    return mlh.muse_lmhead_distill(h, a["x"], a["dtype"], a["n"], a["ld"], a["ids"], a["top"], a["k"], a["tail"], a["w"], a["T"],
                                   a["loss"], a["grad"], a["gld"], None)


def _backward(mlh, h, t, **o):
    p = {k: v.data_ptr() for k, v in t.items()}
    a = {"gl": p["grad"], "x": p["x"], "hid": p["hid"], "b": N, "gamma": p["gamma"], "eps": 1e-5, "w": p["w"], "scale": 1.0,
         "cap": 20.0, "gh": p["gh"], "gg": p["gg"], **o}
    return mlh.muse_lmhead_backward(h, a["gl"], a["x"], a["hid"], a["b"], a["gamma"], a["eps"], a["w"], a["scale"], a["cap"],
                                    a["gh"], a["gg"], None)


def _unchanged(torch, t):
    torch.cuda.synchronize()
    return all(bool((v == 7).all()) for k, v in t.items() if k != "w")


def test_score_refusals(env):
    torch, mlh, head, t = env
    x = t["x"].data_ptr()
    for want, o in [(NULL, {"x": None}), (VALUE, {"dtype": 3}), (VALUE, {"dtype": -1}), (SHAPE, {"n": -1}), (SHAPE, {"n": 1 << 31}),
                    (SHAPE, {"ld": V - 1}), (SHAPE, {"ld": 1 << 61}), (NULL, {"tok": None}), (VALUE, {"T": 0.0}), (VALUE, {"T": -1.0}),
                    (VALUE, {"T": math.nan}), (VALUE, {"T": math.inf}), (SHAPE, {"k": -1}), (SHAPE, {"k": 65}), (NULL, {"ids": None}),
                    (NULL, {"top": None}), (ALIGN, {"x": x + 2}), (ALIGN, {"x": x + 1, "dtype": 2}), (ALIGN, {"lse": t["lse"].data_ptr() + 1}),
                    (NULL, {"lp": None, "rank": None, "lse": None, "ent": None, "ids": None, "top": None, "k": 0})]:
        assert _score(mlh, head.handle, t, **o) == want, o
    assert _score(mlh, head.handle, t, n=0, x=None) == 0
    assert _unchanged(torch, t)
    for bad in (t["x"].double(), t["x"][:, ::2], t["x"].t(), t["x"][:, 1:], t["x"].expand(2, V).as_strided((2, V), (1, 1))):
        with pytest.raises(ValueError):
            head.score(bad)
    with pytest.raises(ValueError):
        head.score(t["x"], tokens=t["tok"].long())
    with pytest.raises(ValueError):
        head.score(t["x"], n_top=65)


def test_forward_score_refusals(env):
    torch, mlh, head, t = env
    p = {k: v.data_ptr() for k, v in t.items()}

    def call(b=N, top=4, temp=1.0, logits=p["x"], tok=p["tok"]):
        return mlh.muse_lmhead_forward_score(head.handle, p["hid"], b, None, 1e-5, p["w"], 1.0, 0.0, logits, tok, temp, top, p["lp"],
                                             p["rank"], p["lse"], p["ent"], p["ids"], p["top"], None)

    assert call(b=0) == BATCH and call(b=N + 1) == BATCH and call(top=65) == SHAPE and call(temp=0.0) == VALUE
    assert call(logits=None) == NULL and call(logits=p["x"] + 4) == ALIGN and call(tok=None) == NULL
    assert _unchanged(torch, t)


def test_distill_refusals(env):
    torch, mlh, head, t = env
    x, g = t["x"].data_ptr(), t["grad"].data_ptr()
    for want, o in [(NULL, {"x": None}), (NULL, {"ids": None}), (NULL, {"top": None}), (NULL, {"loss": None, "grad": None}),
                    (SHAPE, {"k": 0}), (SHAPE, {"k": 65}), (SHAPE, {"ld": V - 1}), (SHAPE, {"gld": V - 1}), (SHAPE, {"n": -1}),
                    (VALUE, {"dtype": 3}), (VALUE, {"tail": 2}), (VALUE, {"T": 0.0}), (VALUE, {"T": math.nan}),
                    (ALIGN, {"x": x + 2}), (ALIGN, {"grad": g + 2}), (ALIGN, {"w": t["loss"].data_ptr() + 2}),
                    (SHAPE, {"grad": x, "gld": V + 4})]:
        assert _distill(mlh, head.handle, t, **o) == want, o
    assert _distill(mlh, head.handle, t, n=0) == 0
    assert _unchanged(torch, t)
    with pytest.raises(ValueError):
        head.distill(t["x"], t["ids"], t["top"], grad=t["grad"].half())
    with pytest.raises(ValueError):
        head.distill(t["x"], t["ids"].long(), t["top"])
    with pytest.raises(ValueError):
        head.distill(t["x"], t["ids"], t["top"][:, :3])
    with pytest.raises(ValueError):
        head.distill(t["x"], t["ids"][:1], t["top"][:1])


def test_backward_refusals(env):
    torch, mlh, head, t = env
    p = {k: v.data_ptr() for k, v in t.items()}
    for want, o in [(NULL, {"gl": None}), (NULL, {"x": None}), (NULL, {"hid": None}), (NULL, {"gamma": None}), (NULL, {"w": None}),
                    (NULL, {"gh": None}), (BATCH, {"b": 0}), (BATCH, {"b": N + 1}), (VALUE, {"eps": -1.0}), (VALUE, {"scale": math.nan}),
                    (VALUE, {"cap": math.inf}), (ALIGN, {"gl": p["grad"] + 4}), (ALIGN, {"w": p["w"] + 8}), (ALIGN, {"gh": p["gh"] + 4}),
                    (ALIGN, {"gg": p["gg"] + 4}), (ALIGN, {"hid": p["hid"] + 4}), (ALIGN, {"x": p["x"] + 4})]:
        assert _backward(mlh, head.handle, t, **o) == want, o
    assert _unchanged(torch, t)
    with pytest.raises(ValueError):
        head.backward(t["grad"], t["w"], logits=t["x"], gamma=t["gamma"])
    with pytest.raises(mlh.MuseError):
        head.backward(t["grad"], t["w"], cap=20.0)
