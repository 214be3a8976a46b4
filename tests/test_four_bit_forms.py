"""Rotary writes with axes whose positions differ into every kind of cache that rounds, at both head
sizes, with factors of a tensor and of a head.

What a cache holds is checked in two steps.  The keys as they are rotated, through a cache of binary32
(bf16 activations as the same numbers in binary32): against the definition in 64 bits, within the
tolerance of test_token_ops (8 units of 2^-24 of |x| + |y|).  Then the codes and scales: those of these
keys, bit for bit, since the rotation is one whatever the cache."""
import pytest
import torch

from paged_kv_cache_90_gb300 import binding
from paged_kv_cache_90_gb300 import build as pkv_build
from test_four_bit_cache import check_write
from test_rotary_axes import rotate64
from test_token_ops import check_near, inputs, quantise

pytestmark = pytest.mark.gpu

# the three layouts of a row's columns over its lanes, all columns turned or not
ROTATIONS = [dict(rotary_dim=64, sections=(12, 10, 10)), dict(rotary_dim=64, sections=(12, 10, 10), cyclic=True),
             dict(rotary_dim=48, sections=(8, 8, 8), cyclic=True), dict(rotary_dim=40, sections=(9, 11)),
             dict(rotary_dim=64, sections=(8, 8, 9, 7), cyclic=True, interleaved=True),
             dict(rotary_dim=50, sections=(10, 10, 5)), dict(rotary_dim=20, sections=(0, 5, 5), interleaved=True)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    binding.load_library()


class Write:
    """A rotary write whose keys, rotated, are known in binary32 (`kr`)."""

    def __init__(self, T, hq, hk, d, bs, kw, dt):
        kw = dict(kw)
        axes = binding.rotary_axes(kw.pop("sections"), kw.pop("cyclic", False))
        self.rot = binding.rotary(**kw, axes=axes)
        pad = (2,) if T > 2 else ()
        self.q, self.k, self.v, _, self.slots, self.nb = inputs(T + d, T, hq, hk, d, bs, dt, pad=pad)
        self.hk, self.d, self.bs = hk, d, bs
        g = torch.Generator().manual_seed(T)
        self.pos = torch.randint(-40, 1 << 20, (self.rot.axes.num_axes, T), generator=g)
        kc = torch.zeros(self.nb, hk, bs, d, device="cuda")
        qf, kf, vf = (x.float().cuda() for x in (self.q, self.k, self.v))
        binding.rotary_and_cache(torch.empty_like(qf), qf, kf, vf, self.pos.cuda(), kc, torch.zeros_like(kc),
                                 self.slots.cuda(), self.rot)
        self.ok = self.slots >= 0
        self.at = (self.slots[self.ok] // bs, slice(None), self.slots[self.ok] % bs)
        self.kr = self.k.float().clone()   # (rows without a slot: any)
        self.kr[self.ok] = kc.cpu()[self.at]
        ref, size = rotate64(self.k, self.pos, self.rot, axes)
        check_near(self.kr[self.ok], ref[self.ok], size[self.ok], torch.float32)
        self.q_ref = rotate64(self.q, self.pos, self.rot, axes)

    def run(self, kc, vc, **kw):
        out = torch.empty_like(self.q).cuda()
        binding.rotary_and_cache(out, self.q.cuda(), self.k.cuda(), self.v.cuda(), self.pos.cuda(), kc, vc,
                                 self.slots.cuda(), self.rot, **kw)
        check_near(out.cpu(), *self.q_ref, self.q.dtype)


def scales(hk, form):
    """(a number or a list of one for each head, the arguments that say so)."""
    if form == "tensor":
        return 0.37, 1.7, dict(k_scale=0.37, v_scale=1.7)
    k, v = [0.25 + 0.3 * h for h in range(hk)], [2.0 ** (h - 2) for h in range(hk)]
    return k, v, dict(k_head_scales=torch.tensor(k).cuda(), v_head_scales=torch.tensor(v).cuda())


CALLS = [(1, 8, 2, 16), (37, 3, 3, 8), (260, 5, 1, 2)]


@pytest.mark.parametrize("form", ["tensor", "heads"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", ROTATIONS)
def test_four_bit_cache(kw, d, dt, form):
    for T, hq, hk, bs in CALLS:
        w = Write(T, hq, hk, d, bs, kw, dt)
        kf, vf, args = scales(hk, form)
        check_write(w.kr, w.v.float(), w.slots, w.nb, bs, kf, vf,
                    lambda kc, vc, ks, vs: w.run(kc, vc, k_token_scales=ks, v_token_scales=vs, **args))


@pytest.mark.parametrize("cache", ["int8", "e4m3", "e4m3 heads"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kw", ROTATIONS)
def test_eight_bit_caches(kw, dt, cache):
    for (T, hq, hk, bs), d in zip(CALLS, (64, 128, 64)):
        w = Write(T, hq, hk, d, bs, kw, dt)
        if cache == "int8":
            kc = torch.full((w.nb, hk, bs, d), 9, dtype=torch.int8).cuda()
            vc, ks = kc.clone(), torch.full((w.nb, hk, bs), 5.0).cuda()
            vs = ks.clone()
            w.run(kc, vc, k_token_scales=ks, v_token_scales=vs)
            for x, c, s in ((w.kr, kc, ks), (w.v.float(), vc, vs)):
                code, scale = quantise(x)
                assert torch.equal(c.cpu()[w.at], code[w.ok]) and torch.equal(s.cpu()[w.at], scale[w.ok])
        else:
            kf, vf, args = scales(hk, "heads" if cache == "e4m3 heads" else "tensor")
            kc = torch.zeros(w.nb, hk, bs, d).to(torch.float8_e4m3fn).cuda()
            vc = kc.clone()
            w.run(kc, vc, **args)
            for x, c, f in ((w.kr, kc, kf), (w.v.float(), vc, vf)):
                f = torch.as_tensor(f, dtype=torch.float32).expand(hk)[None, :, None]
                code = (x / f).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                assert torch.equal(c.view(torch.uint8).cpu()[w.at], code[w.ok])
    assert binding.read_device_errors() == 0
