"""Rotary positions with the cache write, the token-scaled 8-bit cache's write and read
back: against the definitions in 64 bits (rotation) and in IEEE binary32 (codes and scales,
bit for bit), refusals, and a whole speculative step through the library.

Tolerance of a rotated element: an angle's cosine and sine are off by at most 4 2^-24 (two
units of sincospif, the angle's own rounding to binary32, pi 2^-25, and 2^-32 of a turn), the
two products, their scaling by the magnitude and the sum add four roundings more, all relative
to magnitude * (|x| + |y|): 8 2^-24 of it, then half a step of what is stored."""
import math

import pytest
import torch

from paged_kv_cache_90_gb300 import binding
from paged_kv_cache_90_gb300 import build as pkv_build

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


def quantise(x):
    top = x.abs().amax(-1)
    s = top / torch.full_like(top, 127.0)
    bad = ~torch.isfinite(x).all(-1)
    s = torch.where(bad, math.nan, torch.where(s >= 2.0 ** -126, s, 0.0))
    q = torch.round(x / torch.where(s > 0, s, torch.ones_like(s))[..., None]).clamp(-127, 127)
    return torch.where((s > 0)[..., None], q, 0.0).to(torch.int8), s


def rotate64(x, pos, rot):
    """(rotated, magnitude * (|x| + |y|)) of [T, H, D] in 64 bits."""
    y, size = x.double().clone(), x.double().abs()
    rd = rot.rotary_dim
    f = torch.tensor(list(rot.frequency)[:rd // 2], dtype=torch.float64)
    a = torch.remainder(pos.double()[:, None] * (f / (2 * math.pi)), 1.0) * 2 * math.pi
    c, s = (torch.cos(a) * rot.magnitude)[:, None], (torch.sin(a) * rot.magnitude)[:, None]
    i = torch.arange(rd // 2)
    lo, hi = (2 * i, 2 * i + 1) if rot.interleaved else (i, i + rd // 2)
    u, v = x.double()[..., lo], x.double()[..., hi]
    y[..., lo], y[..., hi] = u * c - v * s, v * c + u * s
    size[..., lo] = size[..., hi] = rot.magnitude * (u.abs() + v.abs())
    return y, size


def inputs(seed, T, hq, hk, d, bs, dt, far=1 << 20, pad=()):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(T, h, d, generator=g).to(dt) for h in (hq, hk, hk))
    nb = -(-T // bs) + 4
    slots = torch.randperm(nb * bs, generator=g)[:T]
    for i in pad:
        slots[i] = -1
    pos = torch.randint(0, far, (T,), generator=g)
    return q, k, v, pos, slots, nb


def check_near(got, ref, size, dt):
    step = torch.finfo(dt).eps / 2
    fp = 8 * 2.0 ** -24 * size
    over = (got.double() - ref).abs() - (fp + step * (ref.abs() + fp) + 1e-40)
    assert float(over.max()) <= 0, float(over.max())


ROTATIONS = [dict(rotary_dim=128), dict(rotary_dim=128, interleaved=True), dict(rotary_dim=32, scaling="linear", factor=4.0),
             dict(rotary_dim=96, interleaved=True, scaling="base", factor=8.0),
             dict(rotary_dim=2), dict(rotary_dim=0), dict(rotary_dim=50), dict(rotary_dim=50, interleaved=True),
             dict(rotary_dim=128, base=500000.0, scaling="bands", factor=8.0, original_max_position=8192),
             dict(rotary_dim=128, scaling="ramp", factor=16.0, original_max_position=4096)]


@gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kw", ROTATIONS)
def test_rotary_and_cache(kw, dt):
    rot = binding.rotary(**kw)
    for T, hq, hk, bs, pad in ((1, 8, 2, 16, ()), (37, 3, 3, 8, (0, 20)), (700, 5, 1, 2, (699,))):
        q, k, v, pos, slots, nb = inputs(T, T, hq, hk, 128, bs, dt, pad=pad)
        kc = torch.full((nb, hk, bs, 128), 9.0, dtype=dt).cuda()
        vc = kc.clone()
        out = torch.empty_like(q).cuda()
        got = binding.rotary_and_cache(out, q.cuda(), k.cuda(), v.cuda(), pos.cuda(), kc, vc, slots.cuda(), rot)
        assert got is out
        ref, size = rotate64(q, pos, rot)
        check_near(out.cpu(), ref, size, dt)
        kc, vc = kc.cpu(), vc.cpu()
        ok = slots >= 0
        at = (slots[ok] // bs, slice(None), slots[ok] % bs)
        ref, size = rotate64(k, pos, rot)
        check_near(kc[at], ref[ok], size[ok], dt)
        assert torch.equal(vc[at], v[ok])
        free = torch.ones(nb, bs, dtype=torch.bool)
        free[slots[ok] // bs, slots[ok] % bs] = False
        assert (kc.permute(0, 2, 1, 3)[free] == 9).all() and (vc.permute(0, 2, 1, 3)[free] == 9).all()
        # columns that are not rotated are copied
        assert torch.equal(out.cpu()[..., rot.rotary_dim:], q[..., rot.rotary_dim:])
    assert binding.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_rotary_far_and_negative_positions_in_place(d):
    """Positions to 2^31 and below zero, int32 and int64; the queries rotated in place,
    strided; rotating back gives the start."""
    rot = binding.rotary(d, interleaved=False)
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 7, 2 ** 31 - 1, -2 ** 31, 123456789])
    q, k, v, _, slots, nb = inputs(3, 7, 4, 2, d, 16, torch.float32)
    ref, size = rotate64(q, pos, rot)
    for p in (pos, pos.int()):
        wide = torch.zeros(7, 6, d + 8).cuda()
        wide[:, 1:5, :d] = q.cuda()
        x = wide[:, 1:5, :d]
        kc = torch.zeros(nb, 2, 16, d).cuda()
        vc = torch.zeros_like(kc)
        binding.rotary_and_cache(x, x, k.cuda(), v.cuda(), p.cuda(), kc, vc, slots.cuda(), rot)
        check_near(x.cpu(), ref, size, torch.float32)
        assert (wide[:, 0] == 0).all() and (wide[:, 5] == 0).all() and (wide[:, :, d:] == 0).all()
        binding.rotary_and_cache(x, x, k.cuda(), v.cuda(), (-p.cuda() if p.dtype == torch.int64 else -p.cuda().long()),
                                 kc, vc, slots.cuda(), rot)
        back = (x.cpu().double() - q.double()).abs()
        assert float((back - 32 * 2.0 ** -24 * size).max()) <= 0  # (two rotations, sizes up to twice the first's)


@gpu
@pytest.mark.parametrize("cache", ["e4m3", "e4m3_heads", "int8"])
def test_rotary_into_8bit_caches(cache):
    """What is stored is the nearest code to the rotated key, give or take the rotation's own
    error where that lies on a border (one code at most); values match the plain writes bit
    for bit."""
    rot = binding.rotary(128)
    q, k, v, pos, slots, nb = inputs(5, 90, 4, 2, 128, 16, torch.bfloat16, pad=(3,))
    ok = slots >= 0
    at = (slots[ok] // 16, slice(None), slots[ok] % 16)
    ref, size = rotate64(k, pos, rot)
    fp = 8 * 2.0 ** -24 * size
    dev = [t.cuda() for t in (q, k, v, pos)]
    out = torch.empty_like(dev[0])
    if cache == "int8":
        kc = torch.zeros(nb, 2, 16, 128, dtype=torch.int8).cuda()
        vc, ks = torch.zeros_like(kc), torch.full((nb, 2, 16), 5.0).cuda()
        vs = ks.clone()
        binding.rotary_and_cache(out, *dev, kc, vc, slots.cuda(), rot, k_token_scales=ks, v_token_scales=vs)
        cv, sv = quantise(v.float())
        assert torch.equal(vc.cpu()[at], cv[ok]) and torch.equal(vs.cpu()[at], sv[ok])
        s = ks.cpu()[at].double()[..., None]
        top = ref[ok].abs().amax(-1, keepdim=True)
        assert float(((s - top / 127).abs() - (fp[ok].amax(-1, keepdim=True) / 127 + 2.0 ** -23 * s)).max()) <= 0
        # the stored value: half a step from the rotated key, its error aside
        err = (kc.cpu()[at].double() * s - ref[ok]).abs()
        assert float((err - (0.5 * s * (1 + 2.0 ** -16) + fp[ok])).max()) <= 0
    else:
        hs = torch.tensor([0.02, 0.05])
        kw = dict(k_head_scales=hs.cuda(), v_head_scales=hs.cuda()) if cache == "e4m3_heads" else dict(k_scale=0.03, v_scale=0.03)
        kc = torch.zeros(nb, 2, 16, 128).to(torch.float8_e4m3fn).cuda()
        vc, kc2, vc2 = kc.clone(), kc.clone(), kc.clone()
        binding.rotary_and_cache(out, *dev, kc, vc, slots.cuda(), rot, **kw)
        binding.reshape_and_cache(dev[1], dev[2], kc2, vc2, slots.cuda(), **kw)
        assert torch.equal(vc.view(torch.uint8), vc2.view(torch.uint8))
        s = (hs if cache == "e4m3_heads" else torch.tensor([0.03, 0.03])).double().view(1, 2, 1)
        got = kc.cpu().float()[at].double() * s
        # half a step of e4m3: 2^-4 relative, 2^-10 at least (below its smallest normal number)
        err = (got - ref[ok]).abs() - fp[ok] - torch.maximum(2.0 ** -4 * ref[ok].abs() * (1 + 2.0 ** -20), 2.0 ** -10 * s)
        assert float(err.max()) <= 0
    check_near(out.cpu(), *rotate64(q, pos, rot), torch.bfloat16)
    assert binding.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,hk,d,bs", [(1, 1, 64, 2), (1, 8, 128, 16), (63, 3, 128, 8), (1000, 8, 64, 32), (3000, 2, 128, 16)])
def test_quantize_and_read_back(T, hk, d, bs, dt):
    g = torch.Generator().manual_seed(T)
    _, k, v, _, slots, nb = inputs(T, T, 1, hk, d, bs, dt, pad=(T // 2,) if T > 1 else ())
    k[..., 3] *= 20
    v = (v.float() * torch.exp(3 * torch.randn(T, hk, 1, generator=g))).to(dt)
    if T > 40:
        k[5] = 0.0
        v[6, 0] = 1e-38
        k[7, 0, 9] = math.inf
        v[8, 0, 0] = math.nan
        k[9] = torch.full((hk, d), 2.0)
        v[10] = (torch.randint(-127, 128, (hk, d), generator=g) * 0.5).to(dt)    # quotients on borders
        v[10, :, 0] = 127.0
        if dt == torch.float32:
            k[11] *= 1e30
            k[12] *= 1e-30
            k[13] *= 3e-39
    kc = torch.full((nb, hk, bs, d), 77, dtype=torch.int8).cuda()
    vc, ks = kc.clone(), torch.full((nb, hk, bs), 3.0).cuda()
    vs = ks.clone()
    binding.quantize_and_cache(k.cuda(), v.cuda(), kc, vc, ks, vs, slots.cuda())
    ok = slots >= 0
    at = (slots[ok] // bs, slice(None), slots[ok] % bs)
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        code, scale = quantise(x.float())
        assert torch.equal(c.cpu()[at], code[ok])
        got = s.cpu()[at]
        assert torch.equal(got.view(torch.int32)[~torch.isnan(got)], scale[ok].view(torch.int32)[~torch.isnan(got)])
        assert torch.equal(torch.isnan(got), torch.isnan(scale[ok]))
        assert int((c.cpu() == 77).all(-1).sum()) >= (nb * bs - int(ok.sum())) * hk
    for rd in (torch.float32, torch.bfloat16):
        bk = torch.full((T, hk, d), 4.0, dtype=rd).cuda()
        bv = bk.clone()
        binding.read_cache(bk, bv, kc, vc, slots.cuda(), k_token_scales=ks, v_token_scales=vs)
        for x, b in ((k, bk), (v, bv)):
            code, scale = quantise(x.float())
            want = (code.float() * scale[..., None]).to(rd)
            want[~ok] = 4.0
            assert torch.equal(b.cpu()[~torch.isnan(want)], want[~torch.isnan(want)])
            assert torch.equal(torch.isnan(b.cpu()), torch.isnan(want))
    assert binding.read_device_errors() == 0
    # written again from what was read: the same codes, scales within a unit in the last place
    bk = torch.zeros(T, hk, d).cuda()
    bv = torch.zeros_like(bk)
    binding.read_cache(bk, bv, kc, vc, slots.cuda(), k_token_scales=ks, v_token_scales=vs)
    kc2, vc2, ks2, vs2 = kc.clone(), vc.clone(), ks.clone(), vs.clone()
    binding.quantize_and_cache(bk, bv, kc2, vc2, ks2, vs2, slots.cuda())
    fine = torch.isfinite(ks) & torch.isfinite(vs)
    assert torch.equal(kc2[fine], kc[fine]) and torch.equal(vc2[fine], vc[fine])
    assert int((ks2.view(torch.int32) - ks.view(torch.int32))[fine].abs().max()) <= 1


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_codes_next_to_the_borders(d):
    """Quotients at the middle of two codes and one binary32 number beside it, at scales that
    are and are not powers of two, huge and tiny: the codes of the binary32 quotient, ties to
    even, bit for bit."""
    tops = [127.0, 1.0, 3.7e-3, 3.402823466e38, 1.3e38, 2.0e-36, 1.6e-36, 127.0 * 2.0 ** -60, 5.5]
    rows = []
    for top in tops:
        s = torch.tensor(top) / torch.tensor(127.0)
        h = (torch.arange(-127, 127).double() + 0.5) * s.double()
        mid = h.float()
        near = torch.cat([mid, torch.nextafter(mid, torch.tensor(math.inf)), torch.nextafter(mid, torch.tensor(-math.inf))])
        near = near[near.abs() < top]
        near = torch.cat([near, near[: -near.numel() % (d - 1)]]).view(-1, d - 1)
        rows.append(torch.cat([torch.full((near.shape[0], 1), top), near], 1))
    x = torch.cat(rows)
    T, bs = x.shape[0], 16
    nb = -(-T // bs)
    k, v = x[:, None].clone(), -x[:, None].flip(0)
    kc = torch.zeros(nb, 1, bs, d, dtype=torch.int8).cuda()
    vc, ks, vs = kc.clone(), torch.zeros(nb, 1, bs).cuda(), torch.zeros(nb, 1, bs).cuda()
    slots = torch.arange(T)
    binding.quantize_and_cache(k.cuda(), v.cuda(), kc, vc, ks, vs, slots.cuda())
    for y, c, sc in ((k, kc, ks), (v, vc, vs)):
        code, scale = quantise(y)
        assert torch.equal(sc.cpu()[slots // bs, :, slots % bs], scale)
        assert torch.equal(c.cpu()[slots // bs, :, slots % bs], code)
    assert binding.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("kw", [dict(rotary_dim=64), dict(rotary_dim=24), dict(rotary_dim=20), dict(rotary_dim=6),
                                dict(rotary_dim=20, interleaved=True), dict(rotary_dim=64, interleaved=True)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rotary_of_one_projection(kw, dt):
    """Query, key and value as views of one tensor, as a joint projection gives them, more
    heads than a warp's slice holds, rotated in place."""
    T, hq, hk, d, bs = 21, 71, 1, 64, 4
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, hq + 2 * hk, d, generator=g).to(dt)
    rot = binding.rotary(**kw)
    pos = torch.randint(-50, 5000, (T,), generator=g).int()
    slots = torch.randperm(40, generator=g)[:T]
    kc = torch.zeros(10, hk, bs, d, dtype=dt).cuda()
    vc = kc.clone()
    y = x.cuda()
    q, k, v = y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:]
    binding.rotary_and_cache(q, q, k, v, pos.cuda(), kc, vc, slots.cuda(), rot)
    check_near(y.cpu()[:, :hq], *rotate64(x[:, :hq], pos, rot), dt)
    check_near(kc.cpu()[slots // bs, :, slots % bs], *rotate64(x[:, hq:hq + hk], pos, rot), dt)
    assert torch.equal(vc.cpu()[slots // bs, :, slots % bs], x[:, hq + hk:])
    assert torch.equal(y.cpu()[:, hq:], x[:, hq:])
    assert binding.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("cache", [torch.float32, torch.bfloat16, torch.float8_e4m3fn])
def test_read_cache_of_the_other_types(cache):
    T, hk, d, bs, nb = 50, 2, 128, 16, 6
    g = torch.Generator().manual_seed(1)
    pool = torch.randn(2, nb, hk, bs, d, generator=g).to(cache)
    kc, vc = pool.cuda()[0], pool.cuda()[1]
    slots = torch.randint(0, nb * bs, (T,), generator=g)       # repeated slots are fine
    s = 0.25 if cache == torch.float8_e4m3fn else 1.0
    for rd in (torch.float32, torch.bfloat16):
        bk = torch.zeros(T, hk, d, dtype=rd).cuda()
        bv = torch.zeros_like(bk)
        binding.read_cache(bk, bv, kc, vc, slots.cuda(), k_scale=s, v_scale=2 * s)
        f = pool.float()
        assert torch.equal(bk.cpu(), (f[0][slots // bs, :, slots % bs] * s).to(rd))
        assert torch.equal(bv.cpu(), (f[1][slots // bs, :, slots % bs] * (2 * s if s != 1 else 1)).to(rd))


@gpu
def test_slots_past_the_cache_are_reported():
    k = torch.ones(3, 2, 64).cuda()
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.int8).cuda()
    vc, ks = kc.clone(), torch.zeros(4, 2, 16).cuda()
    vs = ks.clone()
    slots = torch.tensor([64, 1, 1 << 40]).cuda()
    binding.quantize_and_cache(k, k, kc, vc, ks, vs, slots)
    assert binding.read_device_errors() == binding.DEVERR["slot"]
    assert int((ks != 0).sum()) == 2
    out = torch.full((3, 2, 64), 5.0).cuda()
    binding.read_cache(out, out.clone(), kc, vc, slots, k_token_scales=ks, v_token_scales=vs)
    assert binding.read_device_errors() == binding.DEVERR["slot"]
    assert (out[0] == 5).all() and (out[2] == 5).all() and (out[1] == 1).all()


# ---- a speculative step, as an engine makes it ----------------------------------------------


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_speculative_steps_equal_decoding_token_by_token(cache):
    """Prompts written with rotated keys; then trees of drafts are written (positions by
    depth), attended, and the accepted branch is moved to the positions that follow, which
    then decodes like a sequence that never saw the other branches."""
    hq, hk, d, bs, S = 8, 2, 128, 16, 3
    g = torch.Generator().manual_seed(8)
    rot = binding.rotary(d, base=500000.0)
    lens, n = [21, 5, 130], 6
    depth, parents = [0, 1, 1, 2, 2, 3], [-1, 0, 0, 1, 2, 3]
    path = [0, 1, 3, 5]                                        # the accepted branch
    mask = []
    for i in range(n):
        mask.append((mask[parents[i]] if parents[i] >= 0 else 0) | (1 << i))
    mb = 10
    tables = torch.randperm(S * mb, generator=g).int().view(S, mb).cuda()
    dtc = torch.int8 if cache == "int8" else torch.bfloat16
    kc = torch.zeros(S * mb, hk, bs, d, dtype=dtc).cuda()
    vc = torch.zeros_like(kc)
    sc = {}
    if cache == "int8":
        sc = dict(k_token_scales=torch.zeros(S * mb, hk, bs).cuda(), v_token_scales=torch.zeros(S * mb, hk, bs).cuda())

    def slots(s, j):
        return tables[s].long()[torch.as_tensor(j).cuda() // bs] * bs + torch.as_tensor(j).cuda() % bs

    def rand(t, h):
        return torch.randn(t, h, d, generator=g).bfloat16().cuda()

    for s, L in enumerate(lens):                               # the prompts
        q = rand(L, hq)
        binding.rotary_and_cache(q, q, rand(L, hk), rand(L, hk), torch.arange(L).cuda(), kc, vc,
                                 slots(s, torch.arange(L)), rot, **sc)
    # the drafts, every sequence's tree in one batch
    q, k, v = rand(S * n, hq), rand(S * n, hk), rand(S * n, hk)
    pos = torch.cat([torch.tensor(depth) + L for L in lens]).cuda()
    sm = torch.cat([slots(s, torch.arange(n) + L) for s, L in enumerate(lens)])
    tq = torch.empty_like(q)
    binding.rotary_and_cache(tq, q, k, v, pos, kc, vc, sm, rot, **sc)
    out = torch.empty_like(q)
    starts = torch.arange(0, S * n + 1, n).int().cuda()
    m = torch.tensor(mask * S)[:, None].cuda()
    binding.paged_attention_tree(out, tq, kc, vc, tables, (torch.tensor(lens) + n).int().cuda(), starts, m, hk, d ** -0.5,
                                 bs, mb, **sc)
    # the same tokens one at a time on copies of the prompts: a branch is a sequence
    kc1, vc1 = kc.clone(), vc.clone()
    sc1 = {name: t.clone() for name, t in sc.items()}
    for step, node in enumerate(path):
        rows = torch.arange(S).cuda() * n + node
        at = torch.cat([slots(s, torch.tensor([L + step])) for s, L in enumerate(lens)])
        q1 = torch.empty_like(q[rows])
        binding.rotary_and_cache(q1, q[rows].contiguous(), k[rows].contiguous(), v[rows].contiguous(), pos[rows], kc1, vc1,
                                 at, rot, **sc1)
        o1 = torch.empty_like(q1)
        cl = (torch.tensor(lens) + step + 1).int().cuda()
        if cache == "int8":
            binding.paged_attention_decode_quantized(o1, q1, kc1, vc1, sc1["k_token_scales"], sc1["v_token_scales"], tables,
                                                     cl, hk, d ** -0.5, bs, mb)
        else:
            binding.paged_attention_decode(o1, q1, kc1, vc1, tables, cl, hk, d ** -0.5, bs, mb)
        # both round the result to bf16, and the weights to 16 bits: at most a step apart
        # plus twice the weights' half step of sum p |V| (|V| < 6 here, by its type's largest)
        diff = (o1.float() - out[rows].float()).abs()
        assert float((diff - (2.0 ** -7 * o1.float().abs() + 2.0 ** -7 * float(v.abs().max()))).max()) <= 0
    # the accepted branch takes its place: read its tokens, write them where they belong
    src = torch.cat([slots(s, torch.tensor(path) + L) for s, L in enumerate(lens)])
    dst = torch.cat([slots(s, torch.arange(len(path)) + L) for s, L in enumerate(lens)])
    dt = torch.float32 if cache == "int8" else torch.bfloat16
    tk = torch.empty(S * len(path), hk, d, dtype=dt).cuda()
    tv = torch.empty_like(tk)
    binding.read_cache(tk, tv, kc, vc, src, **sc)
    if cache == "int8":
        binding.quantize_and_cache(tk, tv, kc, vc, sc["k_token_scales"], sc["v_token_scales"], dst)
    else:
        binding.reshape_and_cache(tk, tv, kc, vc, dst)
    at = (dst // bs, slice(None), dst % bs)
    assert torch.equal(kc[at], kc1[at]) and torch.equal(vc[at], vc1[at])
    assert binding.read_device_errors() == 0


# ---- on the host ----------------------------------------------------------------------------


def test_rotary_frequencies():
    def f(**kw):
        r = binding.rotary(**kw)
        return list(r.frequency)[:r.rotary_dim // 2], r.magnitude
    plain, one = f(rotary_dim=64)
    assert one == 1.0 and all(math.isclose(x, 10000.0 ** (-2 * i / 64), rel_tol=1e-14) for i, x in enumerate(plain))
    assert all(math.isclose(8 * a, b) for a, b in zip(f(rotary_dim=64, scaling="linear", factor=8.0)[0], plain))
    got = f(rotary_dim=64, scaling="base", factor=8.0)[0]
    assert got[0] == 1.0 and math.isclose(8 * got[-1], plain[-1], rel_tol=1e-12)   # the slowest pair is stretched whole
    got = f(rotary_dim=64, scaling="bands", factor=8.0, original_max_position=8192)[0]
    for a, b in zip(got, plain):
        turns = 8192 * b / (2 * math.pi)
        assert a == b if turns >= 4 else math.isclose(8 * a, b) if turns <= 1 else b / 8 < a < b
    got, m = f(rotary_dim=64, scaling="ramp", factor=8.0, original_max_position=8192)
    assert math.isclose(m, 0.1 * math.log(8.0) + 1)
    turns = [8192 * b / (2 * math.pi) for b in plain]
    assert all(a == b for a, b, t in zip(got, plain, turns) if t > 64)
    assert all(math.isclose(8 * a, b) for a, b, t in zip(got, plain, turns) if t < 0.5)
    ratio = [a / b for a, b in zip(got, plain)]
    assert ratio == sorted(ratio, reverse=True)
    r = binding.rotary(8, frequencies=[1.0, 0.5, 0.25, 0.0], magnitude=2.0)
    assert list(r.frequency)[:4] == [1.0, 0.5, 0.25, 0.0] and r.magnitude == 2.0


@pytest.mark.parametrize("kw", [dict(rotary_dim=3), dict(rotary_dim=130), dict(rotary_dim=-2), dict(rotary_dim=8, base=1.0),
                                dict(rotary_dim=8, base=math.nan), dict(rotary_dim=8, scaling="linear", factor=0.5),
                                dict(rotary_dim=8, scaling="bands", factor=2.0), dict(rotary_dim=8, scaling="ramp", factor=2.0)])
def test_rotary_refusals(kw):
    with pytest.raises(binding.PkvError) as e:
        binding.rotary(**kw)
    assert e.value.status == 1


def test_rotary_binding_refusals():
    with pytest.raises(ValueError):
        binding.rotary(8, scaling="unknown")
    with pytest.raises(ValueError):
        binding.rotary(8, frequencies=[1.0])


def _token_args(**over):
    z = torch.zeros
    a = dict(query_out=z(4, 8, 128, dtype=torch.bfloat16), query=z(4, 8, 128, dtype=torch.bfloat16),
             key=z(4, 2, 128, dtype=torch.bfloat16), value=z(4, 2, 128, dtype=torch.bfloat16),
             positions=z(4, dtype=torch.int64), key_cache=z(10, 2, 16, 128, dtype=torch.bfloat16),
             value_cache=z(10, 2, 16, 128, dtype=torch.bfloat16), slot_mapping=torch.arange(4),
             rotary=binding.rotary(128))
    a.update(over)
    return a


def _status(fn, **kw):
    try:
        fn(**kw)
        return 0
    except binding.PkvError as e:
        assert e.message
        return e.status


def _i8(**over):
    c, s = torch.zeros(10, 2, 16, 128, dtype=torch.int8), torch.zeros(10, 2, 16)
    return {**dict(key_cache=c, value_cache=c.clone(), k_token_scales=s, v_token_scales=s.clone()), **over}


def test_rotary_and_cache_refusals(dry):
    f, z = binding.rotary_and_cache, torch.zeros
    assert _status(f, **_token_args()) == 0
    assert _status(f, **_token_args(**_i8())) == 0
    assert _status(f, **_token_args(positions=z(4, dtype=torch.int32))) == 0
    f8 = z(10, 2, 16, 128).to(torch.float8_e4m3fn)
    assert _status(f, **_token_args(key_cache=f8, value_cache=f8)) == 0
    bad = binding.rotary(128)
    bad.frequency[5] = math.nan
    odd = binding.rotary(128)
    odd.rotary_dim = 7
    wide = z(4, 8, 136, dtype=torch.bfloat16)
    for over, want in [
        (dict(query=z(4, 8, 128)), 1), (dict(query=z(3, 8, 128, dtype=torch.bfloat16)), 1),
        (dict(query_out=z(4, 7, 128, dtype=torch.bfloat16)), 1),
        (dict(positions=z(3, dtype=torch.int64)), 1), (dict(positions=z(4)), 2),
        (dict(positions=z(8, dtype=torch.int64)[::2]), 1),
        (dict(key=z(4, 3, 128, dtype=torch.bfloat16), value=z(4, 3, 128, dtype=torch.bfloat16)), 1),
        (dict(value=z(4, 2, 128)), 1),
        (dict(slot_mapping=torch.arange(4, dtype=torch.int32)), 2), (dict(slot_mapping=torch.arange(8)[::2]), 1),
        (dict(key_cache=z(10, 2, 16, 128), value_cache=z(10, 2, 16, 128)), 2),      # bf16 tokens, f32 cache
        (dict(rotary=bad), 1), (dict(rotary=odd), 1),
        (dict(query=wide[..., 4:132], query_out=wide[..., 4:132]), 1),              # off a 16-byte boundary
        (dict(query=wide[..., :128], query_out=wide.view(-1)[:4 * 8 * 128].view(4, 8, 128)), 1),  # in place, other strides
        (_i8(v_token_scales=None), 1), (_i8(k_token_scales=z(10, 2, 15)), 1),
        (dict(k_token_scales=z(10, 2, 16), v_token_scales=z(10, 2, 16)), 1),
    ]:
        assert _status(f, **_token_args(**over)) == want, list(over)
    r = binding.rotary(128)
    d64 = dict(query=z(4, 8, 64, dtype=torch.bfloat16), query_out=z(4, 8, 64, dtype=torch.bfloat16),
               key=z(4, 2, 64, dtype=torch.bfloat16), value=z(4, 2, 64, dtype=torch.bfloat16),
               key_cache=z(10, 2, 16, 64, dtype=torch.bfloat16), value_cache=z(10, 2, 16, 64, dtype=torch.bfloat16))
    assert _status(f, **_token_args(**d64, rotary=r)) == 1                          # wider than the head
    assert _status(f, **_token_args(**d64, rotary=binding.rotary(64))) == 0


def test_quantize_and_read_refusals(dry):
    def args(**over):
        a = {k: v for k, v in _token_args(**_i8()).items() if k in ("key", "value", "slot_mapping")}
        return {**a, **_i8(), **over}
    bf = torch.zeros(10, 2, 16, 128, dtype=torch.bfloat16)
    for f in (binding.quantize_and_cache, binding.read_cache):
        assert _status(f, **args()) == 0
        assert _status(f, **args(key=torch.zeros(4, 2, 128, dtype=torch.int8),
                                 value=torch.zeros(4, 2, 128, dtype=torch.int8))) == 2
        assert _status(f, **args(slot_mapping=torch.arange(3))) == 1
        assert _status(f, **args(key_cache=bf, value_cache=bf)) == 1                # scales without an i8 cache
        assert _status(f, **args(key_cache=torch.zeros(10, 2, 3, 128, dtype=torch.int8),
                                 value_cache=torch.zeros(10, 2, 3, 128, dtype=torch.int8))) == 2
    assert _status(binding.read_cache, **args(k_token_scales=None, v_token_scales=None)) == 1
    assert _status(binding.read_cache, **args(key_cache=bf, value_cache=bf, k_token_scales=None, v_token_scales=None)) == 0
