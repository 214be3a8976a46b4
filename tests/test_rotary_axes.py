"""Rotary positions with several axes and the cache write: against the definition in 64 bits
(the tolerance of test_token_ops, whose rotation it is), against the call with one axis bit for
bit, and refusals."""
import math

import pytest
import torch

from paged_kv_cache_90_gb300 import binding
from paged_kv_cache_90_gb300 import build as pkv_build
from test_token_ops import check_near, inputs

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    binding.load_library()


@pytest.fixture
def dry():
    binding.set_option("dry_run", 1)
    yield
    binding.set_option("dry_run", 0)


def rotate64(x, pos, rot, axes):
    """(rotated, |x| + |y|) of [T, H, D] in 64 bits, pair by pair."""
    y, size = x.double().clone(), x.double().abs()
    half = rot.rotary_dim // 2
    for i in range(half):
        a = torch.remainder(pos[axes[i]].double() * (rot.frequency[i] / (2 * math.pi)), 1.0) * 2 * math.pi
        c, s = torch.cos(a)[:, None] * rot.magnitude, torch.sin(a)[:, None] * rot.magnitude
        lo, hi = (2 * i, 2 * i + 1) if rot.interleaved else (i, i + half)
        u, v = x.double()[..., lo], x.double()[..., hi]
        y[..., lo], y[..., hi] = u * c - v * s, v * c + u * s
        size[..., lo] = size[..., hi] = rot.magnitude * (u.abs() + v.abs())
    return y, size


CASES = [dict(d=128, rotary_dim=128, sections=(24, 20, 20)), dict(d=128, rotary_dim=128, sections=(24, 20, 20), cyclic=True),
         dict(d=128, rotary_dim=128, sections=(16, 48), interleaved=True), dict(d=64, rotary_dim=48, sections=(12, 12)),
         dict(d=64, rotary_dim=64, sections=(7, 9, 11, 5), cyclic=True, interleaved=True),
         dict(d=128, rotary_dim=50, sections=(10, 10, 5)), dict(d=64, rotary_dim=6, sections=(1, 1, 1)),
         dict(d=128, rotary_dim=128, sections=(64,)), dict(d=128, rotary_dim=96, sections=(0, 0, 48), scaling="ramp", factor=4.0,
                                                          original_max_position=4096)]


@gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kw", CASES)
def test_rotary_axes_and_cache(kw, dt):
    kw = dict(kw)
    d, sections, cyclic = kw.pop("d"), kw.pop("sections"), kw.pop("cyclic", False)
    axes = binding.rotary_axes(sections, cyclic)
    assert [axes.count(a) for a in range(len(sections))] == list(sections)
    rot = binding.rotary(**kw, axes=axes)
    for T, hq, hk, bs, wide in ((1, 8, 2, 16, False), (37, 3, 3, 8, True), (500, 5, 1, 2, False)):
        q, k, v, _, slots, nb = inputs(T, T, hq, hk, d, bs, dt, pad=(0,) if T > 1 else ())
        g = torch.Generator().manual_seed(T)
        n = len(sections) + 1 if wide else len(sections)   # (more rows than axes: the others are not read)
        pos = torch.randint(-5, 1 << 20, (n, T), generator=g)
        kc = torch.full((nb, hk, bs, d), 9.0, dtype=dt).cuda()
        vc = kc.clone()
        p = pos.int() if T == 1 else pos
        if wide:  # a view of a longer array
            p = torch.cat([p, torch.zeros(n, 11, dtype=p.dtype)], 1).cuda()[:, :T]
        out = torch.empty_like(q).cuda()
        assert binding.rotary_and_cache(out, q.cuda(), k.cuda(), v.cuda(), p.cuda(), kc, vc, slots.cuda(), rot) is out
        ref, size = rotate64(q, pos, rot, axes)
        check_near(out.cpu(), ref, size, dt)
        ok = slots >= 0
        at = (slots[ok] // bs, slice(None), slots[ok] % bs)
        ref, size = rotate64(k, pos, rot, axes)
        check_near(kc.cpu()[at], ref[ok], size[ok], dt)
        assert torch.equal(vc.cpu()[at], v[ok])
        assert torch.equal(out.cpu()[..., rot.rotary_dim:], q[..., rot.rotary_dim:])
    assert binding.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("cache", ["same", "e4m3", "int8", "e2m1"])
@pytest.mark.parametrize("kw", [dict(rotary_dim=128), dict(rotary_dim=128, interleaved=True), dict(rotary_dim=50)])
def test_text_tokens_are_turned_as_with_one_axis(kw, cache):
    """The same number on every axis: the bits of the call with one position a token."""
    q, k, v, pos, slots, nb = inputs(4, 200, 4, 2, 128, 16, torch.bfloat16)
    pos[:3] = torch.tensor([-7, 2 ** 40, 0])
    axes = binding.rotary_axes((kw["rotary_dim"] // 2 - 12, 7, 5), True)
    got = []
    for p, rot in ((pos.cuda(), binding.rotary(**kw)), (pos.cuda().expand(3, -1), binding.rotary(**kw, axes=axes)),
                   (pos.cuda().repeat(3, 1), binding.rotary(**kw, axes=axes))):
        dt = {"same": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8, "e2m1": torch.uint8}[cache]
        kc = torch.zeros(nb, 2, 16, 64 if cache == "e2m1" else 128, device="cuda").to(dt)
        vc = torch.zeros(nb, 2, 16, 64 if cache == "e2m1" else 128, device="cuda").to(dt)
        extra = {}
        if cache == "int8":
            extra = dict(k_token_scales=torch.zeros(nb, 2, 16, device="cuda"), v_token_scales=torch.zeros(nb, 2, 16, device="cuda"))
        if cache == "e2m1":
            extra = {n: torch.zeros(nb, 2, 16, 8, device="cuda").to(torch.float8_e4m3fn) for n in ("k_token_scales", "v_token_scales")}
        out = torch.empty_like(q).cuda()
        binding.rotary_and_cache(out, q.cuda(), k.cuda(), v.cuda(), p, kc, vc, slots.cuda(), rot, **extra)
        got.append([out, kc, vc] + list(extra.values()))
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@gpu
def test_in_place_on_a_side_stream_from_a_graph():
    rot = binding.rotary(128, axes=binding.rotary_axes((24, 20, 20)))
    q, k, v, _, slots, nb = inputs(8, 64, 4, 2, 128, 16, torch.bfloat16)
    pos = torch.randint(0, 4000, (3, 64))
    x, p, k, v, slots = q.cuda(), pos.cuda(), k.cuda(), v.cuda(), slots.cuda()
    kc = torch.zeros(nb, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    want = binding.rotary_and_cache(torch.empty_like(x), x, k, v, p, kc, vc, slots, rot).clone()
    first = kc.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    kc.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            binding.rotary_and_cache(x, x, k, v, p, kc, vc, slots, rot)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, want) and torch.equal(kc, first)
    p.add_(17)  # the graph reads the positions anew
    x.copy_(q)
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(x, want)
    assert binding.read_device_errors() == 0


def test_axes_of_pairs():
    assert binding.rotary_axes((2, 1, 3)) == [0, 0, 1, 2, 2, 2]
    assert binding.rotary_axes((2, 1, 3), cyclic=True) == [0, 1, 2, 0, 2, 2]
    for bad in ((), (1, 1, 1, 1, 1), (3, -1)):
        with pytest.raises(ValueError):
            binding.rotary_axes(bad)
    for bad in ([0] * 3, [0, 1, 2, 4], [0, 0, 0, -1]):
        with pytest.raises(ValueError):
            binding.rotary(8, axes=bad)
    assert binding.rotary(8).axes is None and binding.rotary(8, axes=[0, 1, 2, 1]).axes.num_axes == 3


def test_refusals(dry):
    rot = binding.rotary(64, axes=binding.rotary_axes((16, 8, 8)))
    x = torch.zeros(5, 2, 128)
    c = torch.zeros(4, 2, 16, 128)

    def status(pos, r=rot):
        try:
            binding.rotary_and_cache(x, x.clone(), x.clone(), x.clone(), pos, c, c.clone(), torch.zeros(5, dtype=torch.int64), r)
            return 0
        except binding.PkvError as e:
            assert e.message
            return e.status
    pos = torch.zeros(3, 5, dtype=torch.int64)
    assert status(pos) == 0 and status(pos.int()) == 0
    assert status(pos[:2]) == 1                                    # fewer rows than axes
    assert status(pos[:, :4]) == 1 and status(pos[0]) == 1 and status(pos.T.contiguous().T) == 1
    assert status(pos.float()) == 2
    bad = binding.rotary(64, axes=[0] * 32)
    bad.axes.axis[3] = 1
    assert status(pos, bad) == 1
    for n in (0, 5, -1):
        bad = binding.rotary(64, axes=[0] * 32)
        bad.axes.num_axes = n
        assert status(pos, bad) == 1
