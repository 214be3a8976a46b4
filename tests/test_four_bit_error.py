"""What the 4-bit cache's documentation promises of an element's error, over groups of every size.

For a group with largest magnitude a, factor f and g = a / (6 f), the scale G is g rounded to e4m3
and the codes 0, 0.5, 1, 1.5, 2, 3, 4, 6 times G f.
  G > 0, an element of at most 6 G f: off by half a step of the codes.  Half a step is G f from 5 G f
    on, G f / 2 from 2.5 G f on, G f / 4 below: of an element's own size a fifth at most in the first two
    cases, and a is not less; in the third a >= 3 G f (G is at most 2 g) makes it a twelfth of a.
  G < g, an element beyond 6 G f: cut to 6 G f, off by up to a (1 - G / g).  2^-9, the smallest G, takes
    g up to 1.5 x 2^-9: off by up to a third, where a is below 9 x 2^-9 f = 0.0176 f.  The next one takes
    g up to 2.5 x 2^-9: off by a fifth; larger ones are nearer together for their size.
  G = 0: g up to 2^-10, a up to 0.00586 f; an element is off by itself.
  a above 6 x 448 f = 2688 f: what lies above is cut to 2688 f.
Rounding: y = x (1 / (G f)) is off by 2^-23 of itself, at most 6 x 2^-23 steps of G f, and the value that
is read, code (G f), by as much; against an error of at least G f / 4 (where a bound is reached) both are
less than 2^-17 of it."""
import os

import pytest
import torch

from paged_kv_cache_90_gb300 import binding
from paged_kv_cache_90_gb300 import build as pkv_build
from test_four_bit_cache import caches, dequantise, quantise

gpu = pytest.mark.gpu
HEADER = os.path.join(os.path.dirname(pkv_build.HERE), "include", "pkv.h")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    binding.load_library()


def groups(f):
    """[rows, 1, 128] float32: groups of every size from 2^-10 f to 2^13 f, their largest next to the
    borders of the scale among them, with elements at and beside the borders of the codes."""
    g = torch.Generator().manual_seed(7)
    tops = [2.0 ** (i / 16) for i in range(-160, 208)]
    for k in [0.5 + i for i in range(16)]:   # (ties of subnormal scales and of the first normal ones)
        tops += [6 * k * 2.0 ** -9 * (1 + e) for e in (-2.0 ** -10, 0.0, 2.0 ** -10)]
    tops += [0.01757, 0.0176, 2688.0, 2689.0, 2900.0]
    top = torch.tensor(tops, dtype=torch.float32) * f
    x = torch.rand(len(tops), 8, 16, generator=g) * 2 - 1
    x[:, 1] = torch.linspace(-1, 1, 16)
    # the middle of two codes (and beside it), for the scale that the group gets
    s = (top / (6 * f)).clamp(max=448.0).to(torch.float8_e4m3fn).float() * f
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.5])
    for j, e in enumerate((-2.0 ** -18, 0.0, 2.0 ** -18)):
        y = mid * (1 + e) * s[:, None]
        x[:, 2 + j, :8] = torch.where(y <= top[:, None], y, top[:, None]) / top[:, None]
    x = x * top[:, None, None]
    x[:, :, 11] = top[:, None]
    x[:, 5, 11] = -top
    return x.flatten(1)[:, None], top.double()


def check_promise(x, back, f):
    a = x.double().unflatten(-1, (-1, 16)).abs().amax(-1) / f
    err = (back.double() - x.double()).unflatten(-1, (-1, 16)).abs().amax(-1) / f
    slack = 1 + 2.0 ** -17
    assert (err <= a * slack).all()                                  # (a group that vanishes: itself)
    assert (back.unflatten(-1, (-1, 16)).abs().amax(-1)[a < 0.0058] == 0).all()
    assert (back.unflatten(-1, (-1, 16)).abs().amax(-1)[a >= 0.0059] > 0).all()
    small, whole, cut = (a >= 0.0059) & (a < 0.0176), (a >= 0.0176) & (a <= 2688), a > 2688
    assert (err[small] <= a[small] / 3 * slack).all()
    assert (err[whole] <= a[whole] / 5 * slack).all()
    assert (err[cut] <= torch.maximum(a[cut] / 5, a[cut] - 2688)[...] * slack).all()
    assert small.any() and whole.any() and cut.any()
    return float((err / a)[small].max()), float((err / a)[whole].max())


FACTORS = [1.0, 0.37, 2.0 ** -20, 3e5]


@pytest.mark.parametrize("f", FACTORS)
def test_promise_of_the_definition(f):
    """The bounds hold and are reached; a fifth alone, whatever the size, does not hold."""
    x, _ = groups(f)
    third, fifth = check_promise(x, dequantise(*quantise(x, f), f), f)
    assert 0.32 < third and 0.195 < fifth
    with open(HEADER) as h:
        said = " ".join(h.read().replace("\n *", " ").split())
    assert ("An element is off by at most a / 5 where a is 0.0176 f to 2688 f, and by at most a / 3 below that, "
            "down to 0.0059 f; groups below 0.0058 f vanish (G = 0), and values beyond 2688 f are cut off there.") in said


@gpu
@pytest.mark.parametrize("f", FACTORS)
def test_promise_of_the_kernels(f):
    x, _ = groups(f)
    T = x.shape[0]
    kc, vc, ks, vs = caches(-(-T // 16), 1, 16, 128)
    slots = torch.arange(T).cuda()
    binding.quantize_and_cache(x.cuda(), -x.cuda(), kc, vc, ks, vs, slots, k_scale=f, v_scale=f)
    k, v = torch.empty(T, 1, 128, device="cuda"), torch.empty(T, 1, 128, device="cuda")
    binding.read_cache(k, v, kc, vc, slots, k_scale=f, v_scale=f, k_token_scales=ks, v_token_scales=vs)
    assert check_promise(x, k.cpu(), f)[0] > 0.32 and check_promise(x, -v.cpu(), f)[0] > 0.32
    assert binding.read_device_errors() == 0
