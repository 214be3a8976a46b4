"""Rotary positions far out, against the angle in exact arithmetic: the frequency as the double
that it is, 2 pi to 100 digits.  The tolerance is that of test_token_ops.py."""
import math
from fractions import Fraction

import pytest
import torch
from test_token_ops import check_near

from paged_kv_cache_90_gb300 import binding
from paged_kv_cache_90_gb300 import build as pkv_build

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    binding.load_library()


def two_pi():
    """2 pi to 110 digits (Machin: pi / 4 = 4 arctan(1/5) - arctan(1/239))."""
    one = 10 ** 120

    def arctan(n):
        term = total = one // n
        k, sign = 1, -1
        while term:
            term //= n * n
            k += 2
            total += sign * (term // k)
            sign = -sign
        return total

    return Fraction(8 * (4 * arctan(5) - arctan(239)), one)


def rotate_exact(x, pos, rot):
    y, size = x.double().clone(), x.double().abs()
    rd, tau = rot.rotary_dim, two_pi()
    for i in range(rd // 2):
        lo, hi = (2 * i, 2 * i + 1) if rot.interleaved else (i, i + rd // 2)
        for t, p in enumerate(pos.tolist()):
            turn = p * Fraction(rot.frequency[i]) / tau % 1
            a = 2 * math.pi * float(turn - 1 if turn > Fraction(1, 2) else turn)
            c, s = math.cos(a) * rot.magnitude, math.sin(a) * rot.magnitude
            u, v = x[t, :, lo].double(), x[t, :, hi].double()
            y[t, :, lo], y[t, :, hi] = u * c - v * s, v * c + u * s
            size[t, :, lo] = size[t, :, hi] = rot.magnitude * (u.abs() + v.abs())
    return y, size


@gpu
@pytest.mark.parametrize("kw", [dict(rotary_dim=128), dict(rotary_dim=128, interleaved=True), dict(rotary_dim=50),
                                dict(rotary_dim=8, frequencies=[-1.0, 1e-300, -1e-9, 3e5]),
                                dict(rotary_dim=8, frequencies=[1e15, -7e18, 0.0, 2 * math.pi])])
def test_positions_of_any_size(kw):
    pos = torch.tensor([0, 3, 2 ** 31 - 1, -2 ** 31, 2 ** 33 + 1, 2 ** 36 + 12345, -2 ** 40 - 77, 2 ** 47 + 3, 2 ** 53 + 1,
                        2 ** 62 + 987654321, -2 ** 63, 2 ** 63 - 1])
    rot = binding.rotary(**kw)
    g = torch.Generator().manual_seed(2)
    T, bs = pos.numel(), 16
    q, k, v = (torch.randn(T, h, 128, generator=g) for h in (3, 2, 2))
    kc = torch.zeros(2, 2, bs, 128).cuda()
    vc, slots = kc.clone(), torch.arange(T)
    out = torch.empty_like(q).cuda()
    binding.rotary_and_cache(out, q.cuda(), k.cuda(), v.cuda(), pos.cuda(), kc, vc, slots.cuda(), rot)
    check_near(out.cpu(), *rotate_exact(q, pos, rot), torch.float32)
    check_near(kc.cpu()[slots // bs, :, slots % bs], *rotate_exact(k, pos, rot), torch.float32)
    assert binding.read_device_errors() == 0


def test_frequencies_past_the_range_are_refused():
    z = torch.zeros
    binding.set_option("dry_run", 1)
    try:
        for f, fine in ((2.0 ** 64, True), (-2.0 ** 64, True), (2.0 ** 65, False), (-1e300, False), (math.nan, False)):
            try:
                binding.rotary_and_cache(z(1, 1, 64), z(1, 1, 64), z(1, 1, 64), z(1, 1, 64), z(1, dtype=torch.int64),
                                         z(1, 1, 16, 64), z(1, 1, 16, 64), z(1, dtype=torch.int64),
                                         binding.rotary(2, frequencies=[f]))
                assert fine, f
            except binding.PkvError as e:
                assert e.status == 1 and not fine, f
    finally:
        binding.set_option("dry_run", 0)


def test_magnitudes_past_binary32_are_refused():
    """The factor is used in binary32, where a larger double would be infinite."""
    z = torch.zeros
    binding.set_option("dry_run", 1)
    try:
        for m, fine in ((3.4e38, True), (-3.4e38, True), (0.0, True), (3.5e38, False), (-1e300, False), (math.inf, False)):
            try:
                binding.rotary_and_cache(z(1, 1, 64), z(1, 1, 64), z(1, 1, 64), z(1, 1, 64), z(1, dtype=torch.int64),
                                         z(1, 1, 16, 64), z(1, 1, 16, 64), z(1, dtype=torch.int64),
                                         binding.rotary(64, magnitude=m))
                assert fine, m
            except binding.PkvError as e:
                assert e.status == 1 and not fine, m
    finally:
        binding.set_option("dry_run", 0)


def test_two_pi():
    assert float(two_pi()) == 2 * math.pi
    assert str(two_pi().numerator * 10 ** 60 // two_pi().denominator) == \
        "6283185307179586476925286766559005768394338798750211641949889"
