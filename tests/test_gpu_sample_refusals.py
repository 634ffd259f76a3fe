"""Refusals of muse_lmhead_sample and _forward_sample on a real handle: a negative
status and nothing launched (the outputs keep what they held)."""
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
    t = {"x": f(N, V), "u": f(N), "tok": i(N), "lp": f(N), "set": f(N), "kset": i(N), "hid": f(N, K),
         "w": torch.zeros(V * 176, dtype=torch.uint8, device="cuda")}
    head = mlh.LMHead(V, K, max_batch=N, device=0)
    yield torch, mlh, head, t
    head.close()


def _unchanged(torch, t):
    torch.cuda.synchronize()
    return all(bool((v == 7).all()) for k, v in t.items() if k != "w")


def test_sample_refusals(env):
    torch, mlh, head, t = env
    p = {k: v.data_ptr() for k, v in t.items()}

    def call(how=(1.0, 0, 1.0, 0.0), **o):
        a = {"x": p["x"], "dtype": 0, "n": N, "ld": V, "u": p["u"], "tok": p["tok"], "lp": p["lp"], **o}
        return mlh.muse_lmhead_sample(head.handle, a["x"], a["dtype"], a["n"], a["ld"], None if how is None else mlh.MuseSampling(*how),
                                      a["u"], a["tok"], a["lp"], None)

    for want, o in [(NULL, {"x": None}), (NULL, {"u": None}), (NULL, {"tok": None}), (NULL, {"how": None}), (VALUE, {"dtype": 3}),
                    (SHAPE, {"n": -1}), (SHAPE, {"n": 1 << 31}), (SHAPE, {"ld": V - 1}), (SHAPE, {"ld": 1 << 61}),
                    (VALUE, {"how": (-1.0, 0, 1.0, 0.0)}), (VALUE, {"how": (math.nan, 0, 1.0, 0.0)}), (VALUE, {"how": (math.inf, 0, 1.0, 0.0)}),
                    (VALUE, {"how": (2.0 ** -21, 0, 1.0, 0.0)}), (VALUE, {"how": (2.0 ** 21, 0, 1.0, 0.0)}),
                    (VALUE, {"how": (1.0, 0, math.nan, 0.0)}), (VALUE, {"how": (1.0, 0, 1.0, math.nan)}),
                    (ALIGN, {"x": p["x"] + 2}), (ALIGN, {"x": p["x"] + 1, "dtype": 2}), (ALIGN, {"u": p["u"] + 2}), (ALIGN, {"tok": p["tok"] + 1}),
                    (ALIGN, {"lp": p["lp"] + 3}), (ALIGN, {"how": (1.0, 0, 1.0, 0.0, p["set"] + 1)}), (ALIGN, {"how": (1.0, 0, 1.0, 0.0, None, p["kset"] + 2)}),
                    (ALIGN, {"how": (1.0, 0, 1.0, 0.0, None, None, p["set"] + 2)}), (ALIGN, {"how": (1.0, 0, 1.0, 0.0, None, None, None, p["set"] + 2)})]:
        assert call(**o) == want, o
    assert call(n=0, x=None, u=None, tok=None) == 0
    assert _unchanged(torch, t)
    with pytest.raises(mlh.MuseError):
        head.sample(t["x"], t["u"], temperature=-1.0)
    for bad in (dict(uniforms=t["u"][:1]), dict(uniforms=t["u"].double()), dict(logits=t["x"][:, ::2]), dict(top_k=t["set"]),
                dict(temperature=t["set"].half()), dict(top_p=t["set"][:1]), dict(min_p=t["set"].cpu())):
        with pytest.raises(ValueError):
            head.sample(**({"logits": t["x"], "uniforms": t["u"]} | bad))
    assert _unchanged(torch, t)
    # without logprobs
    assert mlh.muse_lmhead_sample(head.handle, p["x"], 0, N, V, mlh.MuseSampling(0.0, 0, 1.0, 0.0), p["u"], p["tok"], None, None) == 0
    torch.cuda.synchronize()
    assert t["tok"].tolist() == [0, 0]
    t["tok"].fill_(7)


def test_forward_sample_refusals(env):
    torch, mlh, head, t = env
    p = {k: v.data_ptr() for k, v in t.items()}
    one = mlh.MuseSampling(1.0, 0, 1.0, 0.0)

    def call(b=N, how=one, logits=p["x"], u=p["u"], tok=p["tok"], hid=p["hid"]):
        return mlh.muse_lmhead_forward_sample(head.handle, hid, b, None, 1e-5, p["w"], 1.0, 0.0, logits, how, u, tok, p["lp"], None)

    assert call(b=0) == BATCH and call(b=N + 1) == BATCH and call(how=None) == NULL and call(how=mlh.MuseSampling(-2.0, 0, 1.0, 0.0)) == VALUE
    assert call(logits=None) == NULL and call(logits=p["x"] + 4) == ALIGN and call(u=None) == NULL and call(tok=None) == NULL
    assert call(hid=None) == NULL and call(hid=p["hid"] + 4) == ALIGN and call(u=p["u"] + 2) == ALIGN
    assert _unchanged(torch, t)
