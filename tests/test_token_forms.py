"""Forms of the token calls and of the attention over token-scaled caches beside the usual ones: rotary
writes into 8-bit caches in every layout of a row, decode with f32 queries and with scales of zero
and below (the CUDA-core kernel, with and without a window), windows with more than 16 heads a KV
head.  Tolerances as in test_token_ops.py and test_tree_attention.py."""
import pytest
import torch
from test_token_ops import check_near, inputs, quantise, rotate64
from test_tree_attention import Case

from paged_kv_cache_90_gb300 import binding
from paged_kv_cache_90_gb300 import build as pkv_build

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    binding.load_library()


FORMS = [dict(rotary_dim=64), dict(rotary_dim=64, interleaved=True), dict(rotary_dim=24), dict(rotary_dim=20),
         dict(rotary_dim=20, interleaved=True), dict(rotary_dim=0)]


@gpu
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", FORMS)
def test_rotary_writes_into_8bit_caches(kw, d, dt, cache):
    """The key's stored value is half a step from the rotated key, the rotation's error aside; values
    are those of the plain write; free slots stay."""
    rot = binding.rotary(**kw)
    hq, hk, bs = 5, 3, 8
    q, k, v, pos, slots, nb = inputs(d, 61, hq, hk, d, bs, dt, pad=(3, 60))
    ok = slots >= 0
    at = (slots[ok] // bs, slice(None), slots[ok] % bs)
    ref, size = rotate64(k, pos, rot)
    fp = 8 * 2.0 ** -24 * size
    dev = [t.cuda() for t in (q, k, v, pos)]
    out = torch.empty_like(dev[0])
    if cache == "int8":
        kc = torch.full((nb, hk, bs, d), 77, dtype=torch.int8).cuda()
        vc, ks = kc.clone(), torch.full((nb, hk, bs), 5.0).cuda()
        vs = ks.clone()
        binding.rotary_and_cache(out, *dev, kc, vc, slots.cuda(), rot, k_token_scales=ks, v_token_scales=vs)
        cv, sv = quantise(v.float())
        assert torch.equal(vc.cpu()[at], cv[ok]) and torch.equal(vs.cpu()[at], sv[ok])
        s = ks.cpu()[at].double()[..., None]
        top = ref[ok].abs().amax(-1, keepdim=True)
        assert float(((s - top / 127).abs() - (fp[ok].amax(-1, keepdim=True) / 127 + 2.0 ** -23 * s)).max()) <= 0
        err = (kc.cpu()[at].double() * s - ref[ok]).abs()
        assert float((err - (0.5 * s * (1 + 2.0 ** -16) + fp[ok])).max()) <= 0
        free = torch.ones(nb, bs, dtype=torch.bool)
        free[slots[ok] // bs, slots[ok] % bs] = False
        assert (kc.cpu().permute(0, 2, 1, 3)[free] == 77).all() and (ks.cpu().permute(0, 2, 1)[free] == 5).all()
    else:
        kc = torch.zeros(nb, hk, bs, d).to(torch.float8_e4m3fn).cuda()
        vc, kc2, vc2 = kc.clone(), kc.clone(), kc.clone()
        binding.rotary_and_cache(out, *dev, kc, vc, slots.cuda(), rot, k_scale=0.03, v_scale=0.02)
        binding.reshape_and_cache(dev[1], dev[2], kc2, vc2, slots.cuda(), k_scale=0.03, v_scale=0.02)
        assert torch.equal(vc.view(torch.uint8), vc2.view(torch.uint8))
        s = float(torch.tensor(0.03))
        err = (kc.cpu().float()[at].double() * s - ref[ok]).abs() - fp[ok]
        step = torch.maximum(2.0 ** -4 * ref[ok].abs() * (1 + 2.0 ** -20), torch.full_like(ref[ok], 2.0 ** -10 * s))
        assert float((err - step).max()) <= 0
    check_near(out.cpu(), *rotate64(q, pos, rot), dt)
    assert binding.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("window", [0, 1, 60, 128])
@pytest.mark.parametrize("hk,group,d,bs", [(2, 4, 128, 16), (1, 20, 64, 2), (2, 1, 128, 32)])
def test_decode_quantized_f32_queries(hk, group, d, bs, window):
    Case(window, [1, 0, 59, 61, 300, 129], None, hk, group, d, bs, cache="int8", qdtype=torch.float32, decode=True,
         window=window).check()


@gpu
@pytest.mark.parametrize("scale", [0.0, -0.1])
@pytest.mark.parametrize("decode,cache", [(False, "bf16"), (False, "int8"), (True, "int8")])
def test_scales_of_zero_and_below(scale, decode, cache):
    """(one rounding less than the bound allows: the weights stay in binary32 here)"""
    c = Case(4, [100, 17], [5, 17], 2, 4, 128, 16, cache=cache, decode=decode, window=30 if decode else 0)
    c.scale = scale
    ref, wabs, dz = c.reference()
    out = c.call(c.device())
    over = (out.double().cpu() - ref).abs() - c.bound(ref, wabs, dz.abs())
    assert float(over.max()) <= 0 and binding.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("window", [1, 100, 128, 1000])
@pytest.mark.parametrize("hk,group,d,bs", [(1, 17, 128, 16), (2, 32, 64, 2), (1, 128, 128, 32)])
def test_decode_quantized_windows_of_many_heads(hk, group, d, bs, window):
    c = Case(window, [1, 99, 100, 101, 600, 0, 2000], None, hk, group, d, bs, cache="int8", decode=True, window=window)
    real = c.tables.clone()
    for s, L in enumerate(c.lens):      # blocks that have left the window may be gone
        c.tables[s, :max(0, L - window) // bs] = -1
    x = c.device()
    c.tables = real
    out = c.call(x)
    torch.cuda.synchronize()
    assert binding.read_device_errors() == 0
    c.check(out)
