"""muse_lmhead_sample with top-p where its border falls on hundreds or thousands of equal logits (GPU).

Logits of 16 bits far from 0 lie on few values, each of which a large vocabulary
holds thousands of times.  Checked against the definition in 64 bits, as in
test_gpu_sample, whose tolerance this uses."""
import pytest

from test_gpu_sample import TYPES, _check, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v", [(1, 202048), (5, 50257), (20, 9001), (160, 20011)])
@pytest.mark.parametrize("top_p", [0.3, 0.9, 0.99])
def test_logits_far_from_zero(env, dtype, n, v, top_p):
    """Steps of 2^-5 and 2^-4 in bf16."""
    torch, _ = env
    gen = torch.Generator(device="cuda").manual_seed(v + n)
    x = (torch.randn((n, v), generator=gen, device="cuda") * 2 + 9).to(getattr(torch, dtype))
    _check(env, x, torch.rand((n,), generator=gen, device="cuda"), top_p=top_p)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("values", [[1.0], [0.0, 1.0], [-1.0, 0.0, 2.5], [0.0, 0.5, 1.0, 1.5, 2.0, 2.5, 3.0], [-60.0, 4.0, 4.5]])
@pytest.mark.parametrize("top_p", [0.01, 0.5, 0.87, 0.999])
def test_few_different_logits(env, dtype, values, top_p):
    """Shares of a row that hold one value each, spread over all CTAs."""
    torch, _ = env
    gen = torch.Generator(device="cuda").manual_seed(len(values))
    for n, v in ((3, 40009), (12, 3001)):
        pick = torch.randint(0, len(values), (n, v), generator=gen, device="cuda")
        x = torch.tensor(values, device="cuda")[pick].to(getattr(torch, dtype))
        _check(env, x, torch.rand((n,), generator=gen, device="cuda"), top_p=top_p)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("spread", [1, 600, 30000])
def test_a_crowd_among_others(env, dtype, spread):
    """One value many times, in one stretch of the row or all over it, among others that differ."""
    torch, _ = env
    n, v = 6, 60013
    gen = torch.Generator(device="cuda").manual_seed(spread)
    x = torch.randn((n, v), generator=gen, device="cuda")
    at = (torch.arange(3000, device="cuda") * (spread if spread == 1 else v // 3000) + (0 if spread != 600 else 7)) % v
    x[:, at] = 1.25
    x[0, at[::2]] = -0.0
    x[0, at[1::2]] = 0.0
    for top_p in (0.2, 0.5, 0.52, 0.55, 0.6, 0.9):
        _check(env, x.to(getattr(torch, dtype)), torch.rand((n,), generator=gen, device="cuda"), top_p=top_p)


@pytest.mark.parametrize("dtype", TYPES)
def test_signs_of_zero(env, dtype):
    """Zeros of both signs are equal, and thousands of them are kept by index."""
    torch, _ = env
    n, v = 4, 30011
    x = torch.full((n, v), -3.0, device="cuda")
    x[:, ::3] = 0.0
    x[:, 1::6] = -0.0
    u = torch.tensor([0.0, 0.3, 0.7, 1.0], device="cuda")
    tokens, _ = _check(env, x.to(getattr(torch, dtype)), u, top_p=0.5)
    assert tokens[0] == 0


@pytest.mark.parametrize("masked", [0.0, 0.5, 0.999])
def test_crowds_with_masks_settings_and_min_p(env, masked):
    torch, _ = env
    n, v = 24, 50257
    gen = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn((n, v), generator=gen, device="cuda") * 2 + 9
    x[torch.rand((n, v), generator=gen, device="cuda") < masked] = float("-inf")
    x[:, 5] = 1.0
    u = torch.rand((n,), generator=gen, device="cuda")
    t = 0.5 + torch.rand((n,), generator=gen, device="cuda")
    p = torch.rand((n,), generator=gen, device="cuda") * 0.9 + 0.05
    mp = torch.where(torch.arange(n, device="cuda") % 3 == 0, 0.01, 0.0)
    k = torch.where(torch.arange(n, device="cuda") % 4 == 1, 2000, 0).to(torch.int32)
    _check(env, x.to(torch.bfloat16), u, temperature=t, top_k=k, top_p=p, min_p=mp)
