"""Rows on which top-p's border is hard to come by: flat and steep ones, sorted ones,
rows whose likely tokens lie where a sample does not look, crowds of equals, shares
next to 0 and 1; and the launch shapes of many long rows.  Checked as in
test_gpu_sample, whose tolerances hold for any row."""
import math

import pytest

from test_gpu_sample import TYPES, _check, _rows, env  # noqa: F401

pytestmark = pytest.mark.gpu


def _shapes(torch, v, gen):
    """Rows by name."""
    noise = lambda s: torch.randn((v,), generator=gen, device="cuda") * s                 # noqa: E731
    up = torch.linspace(-12, 12, v, device="cuda")
    every = torch.arange(v, device="cuda")
    steps = torch.floor(up)                                      # 25 crowds of equals
    lone = noise(1.0)
    lone[v // 3] += 30.0
    pair = torch.full((v,), -3.0, device="cuda")
    pair[5], pair[v - 2] = 1.0, 1.0
    return {
        "flat": noise(0.01), "low": noise(0.5), "wide": noise(4.0), "rising": up.clone(), "falling": -up, "steps": steps, "lone": lone, "pair": pair,
        "unsampled": torch.where(every % 8 == 3, 4.0, 0.0) + noise(0.5), "first_of_vectors": torch.where(every % 8 == 0, 4.0, 0.0) + noise(0.5),
        "first_of_steps": torch.where(every % 1024 < 8, 6.0, 0.0) + noise(0.5), "half": torch.where(every < v // 2, -math.inf, 0.0) + noise(1.0),
        "tail_of_crowd": torch.where(every % 50 == 7, 2.0, -8.0), "two_levels": torch.where(every % 3 == 0, 0.0, -0.69314718),
    }


SHARES = (1e-6, 0.1, 0.5, 0.9, 0.99, 0.99999, 1 - 2.0 ** -24)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [700, 20011, 202048])
def test_shapes_of_rows(env, dtype, v):                                                  # noqa: F811
    torch, _ = env
    gen = torch.Generator(device="cuda").manual_seed(v)
    shapes = _shapes(torch, v, gen)
    x = torch.stack(list(shapes.values())).to(getattr(torch, dtype))
    u = torch.rand((x.shape[0],), generator=gen, device="cuda")
    for p in SHARES:
        _check(env, x, u, top_p=p)
    _check(env, x, u, top_p=0.9, min_p=0.2)
    _check(env, x, u, top_p=0.9, min_p=0.9, temperature=0.7)
    _check(env, x, u, top_p=0.8, top_k=700)
    _check(env, x, u, top_k=300, top_p=0.99)
    _check(env, x, u, temperature=3.0, top_p=0.95)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("off", [0, 3])
@pytest.mark.parametrize("n,v", [(20, 60013), (40, 60013), (80, 60013), (160, 60013), (240, 60013)])
def test_launch_shapes_of_long_rows(env, dtype, off, n, v):                              # noqa: F811
    x, u = _rows(env[0], n, v, n, scale=2.0, dtype=dtype, off=off)
    _check(env, x, u, top_p=0.93)
    _check(env, x, u)
    _check(env, x, u, top_k=40)


def test_flat_rows_need_the_exact_mass(env):                                             # noqa: F811
    """Kept tokens of a few millionths each: the estimate's bounds hold two borders in one row of twenty or so."""
    for scale in (0.05, 0.4):
        x, u = _rows(env[0], 150, 50021, 7, scale=scale)
        for p in (0.3, 0.9):
            _check(env, x, u, top_p=p)


def test_settings_mixed_over_launch_shapes(env):                                         # noqa: F811
    torch, _ = env
    for n, v in ((24, 40009), (230, 40009)):
        x, u = _rows(torch, n, v, n)
        pick = lambda values, dtype: torch.tensor([values[i % len(values)] for i in range(n)], dtype=dtype, device="cuda")     # noqa: E731
        _check(env, x, u, pick([1.0, 0.0, 0.5, 1e-3, 2.0], torch.float32), pick([0, 0, 40, 600], torch.int32), pick([0.9, 1.0, 0.5], torch.float32),
               pick([0.0, 0.02], torch.float32))
