"""The 4-bit cache (e2m1 codes, an e4m3 scale for every 16 columns): write and read back bit
for bit against the definition in IEEE binary32, decode and tree attention against the
definition in 64 bits, refusals.

Tolerance of the attention: that of test_tree_attention.Case (the result's rounding, scores,
sums), with weights rounded to f16: half a step, 2^-11 of each, and for those that are subnormal
in f16 2^-31 of the row's largest, which is at most 1, so L 2^-31 max |V| for a row of L
positions.  Keys and values are exact: a code times its scale has six significant bits."""
import math

import pytest
import torch

from paged_kv_cache_90_gb300 import binding
from paged_kv_cache_90_gb300 import build as pkv_build
from test_tree_attention import LAYOUTS, Case

gpu = pytest.mark.gpu
VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    binding.load_library()


@pytest.fixture
def dry():
    binding.set_option("dry_run", 1)
    yield
    binding.set_option("dry_run", 0)


def factors(f, heads):
    """[heads, 1] binary32 factors of a number or a list of one for each head."""
    f = torch.as_tensor(f, dtype=torch.float32)
    return f.expand(heads)[:, None] if f.dim() == 0 else f[:, None]


def quantise(x, f):
    """Rows [..., heads, D] of float32 -> bytes of two codes, scales as bytes (CPU, binary32)."""
    y = x.unflatten(-1, (-1, 16))
    f = factors(f, x.shape[-2])
    top = y.abs().amax(-1)
    bad = ~torch.isfinite(y).all(-1)
    g = (top / (6.0 * f)).clamp(max=448.0)
    s = torch.where(bad, 0.0, g).to(torch.float8_e4m3fn)
    step = s.float() * f
    number = (step >= 2.0 ** -126) & (step <= 2.0 ** 126) & ~bad
    s = torch.where(number, s.view(torch.uint8), torch.zeros_like(s.view(torch.uint8)))
    q = torch.where(number[..., None], y, torch.zeros_like(y)) * torch.where(number, 1.0 / step, 1.0)[..., None]
    a = q.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() +
            (a >= 3.5).int() + (a > 5.0).int())
    code = (code + 8 * torch.signbit(q).int()) * number[..., None]
    code = code.flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.where(bad, 0x7f, s.int()).to(torch.uint8)


def dequantise(b, s, f, dtype=torch.float32):
    """Bytes and scales' bytes [..., heads, *] -> values; in binary32 as the read back gives them."""
    n = torch.stack([b & 15, b >> 4], -1).flatten(-2).long()
    v = torch.where(n >= 8, -VALUES[n & 7], VALUES[n & 7]).to(dtype)
    g = s.view(torch.float8_e4m3fn).float().to(dtype) * factors(f, b.shape[-2]).to(dtype)
    return v * g.repeat_interleave(16, -1)


class FourBit(Case):
    """test_tree_attention's case over a 4-bit cache."""

    def __init__(self, seed, lens, nodes, hk, group, d, bs, k_factor=1.0, v_factor=1.0, **kw):
        poison = kw.pop("poison", True)
        super().__init__(seed, lens, nodes, hk, group, d, bs, cache="f32", poison=False, **kw)
        self.k_factor, self.v_factor = k_factor, v_factor
        out = []
        for x, f in ((self.kc, k_factor), (self.vc, v_factor)):
            b, s = quantise((x * factors(f, hk)[:, :, None]).transpose(1, 2), f)
            b, s = b.transpose(1, 2).contiguous(), s.transpose(1, 2).contiguous()
            if poison:
                s = s.masked_fill(~self.used[:, None, :, None], 0x7f)
            out += [b, s]
        self.kc, self.k_scales, self.vc, self.v_scales = out
        self.cache = "e2m1"
        self.refresh()

    def refresh(self):
        def wide(b, s, f):
            return dequantise(b.transpose(1, 2), s.transpose(1, 2), f, torch.float64).transpose(1, 2)
        self.K64, self.V64 = wide(self.kc, self.k_scales, self.k_factor), wide(self.vc, self.v_scales, self.v_factor)

    def bound(self, ref, wabs, dz):
        u = 2.0 ** -24
        L = max(self.lens + [1])
        half = self.q.dtype == torch.bfloat16
        # a score is off by at most (d + 8) u |scale| sum |q| |K|, whatever the scale's sign (dz has it)
        rel = (2.0 ** -11 if half else 0.0) + 2 * ((self.d + 8) * u * dz.abs() + 2.0 ** -22) + L * u
        V = torch.where(torch.isfinite(self.V64), self.V64.abs(), 0.0).amax((0, 2, 3))  # [hk]
        floor = L * 2.0 ** -31 * V.repeat_interleave(self.group)[None, :, None] if half else 0.0
        fp = rel * wabs + floor
        return torch.finfo(self.q.dtype).eps / 2 * (ref.abs() + fp) + fp + 1e-30

    def device(self):
        x = super().device()
        x["ks"], x["vs"] = x["ks"].view(torch.float8_e4m3fn), x["vs"].view(torch.float8_e4m3fn)
        return x

    def call(self, x, stream=None):
        kw = {}
        for n, f in (("k", self.k_factor), ("v", self.v_factor)):
            if isinstance(f, list):
                self.keep_alive = getattr(self, "keep_alive", {})
                self.keep_alive.setdefault(n, torch.tensor(f, device="cuda"))
                kw[n + "_head_scales"] = self.keep_alive[n]
            else:
                kw[n + "_scale"] = f
        if self.decode:
            return binding.paged_attention_decode_quantized(
                x["out"], x["q"], x["kc"], x["vc"], x["ks"], x["vs"], x["tables"], x["lens"], self.hk, self.scale,
                self.bs, self.mb, sliding_window=self.window, stream=stream, **kw)
        return binding.paged_attention_tree(
            x["out"], x["q"], x["kc"], x["vc"], x["tables"], x["lens"], x["starts"], x["mask"], self.hk, self.scale,
            self.bs, self.mb, k_token_scales=x["ks"], v_token_scales=x["vs"], stream=stream, **kw)


# ---- write and read back ------------------------------------------------------------------


def caches(nb, hk, bs, d, fill=0xa5):
    b = torch.full((nb, hk, bs, d // 2), fill, dtype=torch.uint8, device="cuda")
    s = torch.full((nb, hk, bs, d // 16), fill, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    return b, b.clone(), s, s.view(torch.uint8).clone().view(torch.float8_e4m3fn)


def tokens(seed, T, hk, d, dt, size=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, hk, d, generator=g) * torch.exp(1.5 * torch.randn(T, hk, 1, generator=g)) * size
    x[..., 5] *= 8.0
    return x.to(dt)


def check_write(k, v, slots, nb, bs, kf, vf, write):
    """`write(caches)` stores k and v: codes and scales bit for bit, nothing elsewhere; then the
    read back, into both types."""
    T, hk, d = k.shape
    kc, vc, ks, vs = caches(nb, hk, bs, d)
    write(kc, vc, ks, vs)
    ok = slots >= 0
    blk, off = slots[ok] // bs, slots[ok] % bs
    free = torch.ones(nb, bs, dtype=torch.bool)
    free[blk, off] = False
    for x, c, s, f in ((k, kc, ks, kf), (v, vc, vs, vf)):
        b, g = quantise(x.float(), f)
        c, s = c.cpu(), s.view(torch.uint8).cpu()
        assert torch.equal(s[blk, :, off], g[ok])
        assert torch.equal(c[blk, :, off], b[ok])
        assert (c.transpose(1, 2)[free] == 0xa5).all() and (s.transpose(1, 2)[free] == 0xa5).all()
    kw = {n: torch.tensor(f, device="cuda") if isinstance(f, list) else f
          for n, f in (("k_head_scales" if isinstance(kf, list) else "k_scale", kf),
                       ("v_head_scales" if isinstance(vf, list) else "v_scale", vf))}
    for dt in (torch.float32, torch.bfloat16):
        kb, vb = torch.full((T, hk, d), 7.0, dtype=dt, device="cuda"), torch.full((T, hk, d), 7.0, dtype=dt, device="cuda")
        binding.read_cache(kb, vb, kc, vc, slots.cuda(), k_token_scales=ks, v_token_scales=vs, **kw)
        for x, back, f in ((k, kb, kf), (v, vb, vf)):
            ref = dequantise(*quantise(x.float(), f), f).to(dt)
            back = back.cpu()
            assert torch.equal(back[ok].nan_to_num(123.0), ref[ok].nan_to_num(123.0))
            assert (back[~ok] == 7).all()
    assert binding.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,hk,d,bs", [(1, 1, 64, 2), (1, 8, 128, 16), (63, 3, 128, 8), (700, 8, 64, 32), (900, 5, 128, 4)])
def test_write_and_read_back(T, hk, d, bs, dt):
    nb = -(-T // bs) + 3
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(T))[:T]
    if T > 5:
        slots[3] = -1
    for kf, vf in ((1.0, 1.0), (0.37, 5.0), ([0.1 * (i + 1) for i in range(hk)], [2.0 ** i for i in range(hk)])):
        k, v = tokens(T, T, hk, d, dt), tokens(T + 1, T, hk, d, dt, 3.0)
        kw = {n: torch.tensor(f, device="cuda") if isinstance(f, list) else f
              for n, f in (("k_head_scales" if isinstance(kf, list) else "k_scale", kf),
                           ("v_head_scales" if isinstance(vf, list) else "v_scale", vf))}
        check_write(k, v, slots, nb, bs, kf, vf, lambda kc, vc, ks, vs: binding.quantize_and_cache(
            k.cuda(), v.cuda(), kc, vc, ks, vs, slots.cuda(), **kw))


@gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_groups_of_every_size(dt):
    """Zeros, values from the smallest to the largest numbers, single large elements, infinities
    and NaN (of one group alone), signs of zero; a group's largest at every e4m3 step and border."""
    g = torch.Generator().manual_seed(4)
    rows = [torch.zeros(16), -torch.zeros(16), torch.full((16,), 448.0 * 6), torch.full((16,), 1e30), torch.full((16,), 1e-30)]
    rows += [torch.randn(16, generator=g) * 2.0 ** e for e in range(-148, 127, 3)]
    for m in list(range(-9, 9)):  # ties of the scale and around them
        for k in (1.0, 1.0625, 1.125, 1.1875, 1.9375, 1.96875):
            x = torch.rand(16, generator=g) * 2.0 ** m
            x[3] = 6.0 * k * 2.0 ** m
            rows += [x, -x]
    for bad in (math.inf, -math.inf, math.nan):
        x = torch.randn(16, generator=g)
        x[9] = bad
        rows.append(x)
    # every border between two codes, at a scale of one, and the numbers next to them
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 5.5, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    rows += [ties, -ties, torch.nextafter(ties, torch.tensor(0.0)), torch.nextafter(ties, torch.tensor(9.0)).clamp(max=6.0)]
    n = -(-len(rows) // 8)
    x = torch.cat(rows + [torch.zeros(16)] * (8 * n - len(rows))).view(n, 1, 128).to(dt)
    x = torch.cat([x, x.roll(1, -1)], 1)
    slots = torch.arange(n) + 5
    for f in (1.0, 2.0 ** -100, 2.0 ** 100, 0.3):
        check_write(x, x.flip(0), slots, n, 16, f, f, lambda kc, vc, ks, vs: binding.quantize_and_cache(
            x.cuda(), x.flip(0).cuda(), kc, vc, ks, vs, slots.cuda(), k_scale=f, v_scale=f))


@gpu
def test_error_of_what_is_written():
    """Normal draws, to what the format promises: at most a fifth of a group's largest."""
    x = torch.randn(300, 4, 128, generator=torch.Generator().manual_seed(1))
    kc, vc, ks, vs = caches(20, 4, 16, 128)
    slots = torch.arange(300).cuda()
    binding.quantize_and_cache(x.cuda(), x.cuda(), kc, vc, ks, vs, slots)
    k, v = torch.empty(300, 4, 128, device="cuda"), torch.empty(300, 4, 128, device="cuda")
    binding.read_cache(k, v, kc, vc, slots, k_token_scales=ks, v_token_scales=vs)
    err = (k.cpu() - x).abs().unflatten(-1, (-1, 16)).amax(-1)
    assert (err <= x.abs().unflatten(-1, (-1, 16)).amax(-1) / 5).all()


ROTATIONS = [dict(rotary_dim=128), dict(rotary_dim=128, interleaved=True), dict(rotary_dim=48), dict(rotary_dim=40),
             dict(rotary_dim=50), dict(rotary_dim=6, interleaved=True), dict(rotary_dim=0)]


@gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kw", ROTATIONS)
def test_rotary_write(kw, dt):
    """The rotated keys of the f32 cache, quantised by the definition, are what the 4-bit cache
    holds, and the queries are the same: one rotation, whatever the cache."""
    rot = binding.rotary(**kw)
    for T, hq, hk, bs in ((1, 8, 2, 16), (37, 3, 3, 8), (300, 5, 1, 4)):
        g = torch.Generator().manual_seed(T)
        q, k, v = (torch.randn(T, h, 128, generator=g).to(dt) for h in (hq, hk, hk))
        nb = -(-T // bs) + 2
        slots = torch.randperm(nb * bs, generator=g)[:T]
        pos = torch.randint(0, 1 << 20, (T,), generator=g).cuda()
        kr = torch.empty_like(k).float()
        # binary32 keys as they are rotated: through a cache that holds them (bf16 activations: the
        # same numbers as f32 ones, rotated by the same operations)
        kc, vc = torch.zeros(nb, hk, bs, 128, device="cuda"), torch.zeros(nb, hk, bs, 128, device="cuda")
        qf = q.float().cuda()
        binding.rotary_and_cache(torch.empty_like(qf), qf, k.float().cuda(), v.float().cuda(), pos, kc, vc, slots.cuda(), rot)
        kr = kc.cpu()[slots // bs, :, slots % bs]
        want = torch.empty_like(q).cuda()
        kc2, vc2 = torch.zeros(nb, hk, bs, 128, device="cuda").to(dt), torch.zeros(nb, hk, bs, 128, device="cuda").to(dt)
        binding.rotary_and_cache(want, q.cuda(), k.cuda(), v.cuda(), pos, kc2, vc2, slots.cuda(), rot)

        def write(kc, vc, ks, vs):
            out = torch.empty_like(q).cuda()
            binding.rotary_and_cache(out, q.cuda(), k.cuda(), v.cuda(), pos, kc, vc, slots.cuda(), rot, k_scale=0.5,
                                     k_token_scales=ks, v_token_scales=vs)
            assert torch.equal(out, want)
        check_write(kr, v.float(), slots, nb, bs, 0.5, 1.0, write)


# ---- attention -----------------------------------------------------------------------------


@gpu
@pytest.mark.parametrize("hk,group,d", LAYOUTS)
def test_decode_head_layouts(hk, group, d):
    FourBit(hk + group, [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 400, 0, 1025], None, hk, group, d, 16,
            decode=True).check()


@gpu
@pytest.mark.parametrize("bs,d", [(2, 64), (2, 128), (4, 128), (4, 64), (8, 64), (8, 128), (32, 128)])
@pytest.mark.parametrize("window", [0, 1, 100, 128, 1000])
def test_decode_windows_and_block_sizes(window, bs, d):
    c = FourBit(20 + window, [1, 99, 100, 101, 600, 2000], None, 2, 4, d, bs, decode=True, window=window)
    real = c.tables.clone()
    if window:  # blocks that have left the window may be gone
        for s, L in enumerate(c.lens):
            c.tables[s, :max(0, L - window) // bs] = -1
    x = c.device()
    c.tables = real
    out = c.call(x)
    torch.cuda.synchronize()
    assert binding.read_device_errors() == 0
    c.check(out)


@gpu
@pytest.mark.parametrize("group", [4, 12, 20])
def test_decode_many_and_long(group):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(1, 700, (150,), generator=g).tolist() + [8000]
    FourBit(21, lens, None, 2, group, 128, 16, decode=True).check()


@gpu
@pytest.mark.parametrize("qdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("decode", [True, False])
def test_factors_of_tensors_and_heads(decode, qdtype):
    lens, nodes = [300, 33, 1, 700], [9, 3, 1, 20]
    for kf, vf in ((0.05, 7.0), ([0.5, 3.0], [100.0, 0.01]), (2.0 ** -30, 2.0 ** 40)):
        c = FourBit(5, lens, nodes, 2, 4, 128, 16, k_factor=kf, v_factor=vf, decode=decode, qdtype=qdtype)
        if kf == 2.0 ** -30:
            c.scale = c.scale * 2.0 ** 30
        c.check()


@gpu
@pytest.mark.parametrize("hk,group,d", LAYOUTS)
def test_tree_head_layouts(hk, group, d):
    FourBit(hk * 100 + group, [40, 300, 1, 129, 17], [7, 12, 1, 4, 17], hk, group, d, 16).check()


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [2, 4, 8, 16, 32])
def test_tree_block_sizes(bs, d):
    FourBit(bs, [33, 130, 5, 64], [5, 9, 5, 3], 2, 4, d, bs).check()


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("decode", [True, False])
def test_f32_queries(d, decode):
    FourBit(d, [70, 9], [6, 9], 2, 2, d, 16, qdtype=torch.float32, decode=decode).check()


@gpu
@pytest.mark.parametrize("L,n", [(1, 1), (2, 2), (63, 63), (64, 1), (65, 64), (127, 3), (128, 128), (129, 1), (129, 129),
                                 (200, 130), (256, 64), (257, 33), (511, 65), (1000, 256)])
def test_tree_lengths_around_tiles(L, n):
    FourBit(L * 1000 + n, [L, 20], [n, 3], 2, 4, 128, 16, words=-(-n // 64) + (L % 2)).check()


@gpu
@pytest.mark.parametrize("masks", ["chain", "bits", "none"])
def test_tree_masks(masks):
    FourBit(5, [50, 8, 150, 64], [8, 8, 20, 64], 2, 4, 128, 16, masks=masks).check()


@gpu
def test_rows_that_attend_to_nothing_are_zero():
    c = FourBit(6, [6, 12], [6, 12], 2, 4, 128, 16, masks="none")
    out = c.call(c.device())
    assert torch.equal(out, torch.zeros_like(out))


@gpu
def test_tree_many_sequences_and_long_ones():
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(1, 90, (200,), generator=g).tolist() + [9000, 513]
    nodes = [min(L, int(n)) for L, n in zip(lens, torch.randint(0, 9, (202,), generator=g).tolist())]
    lens[7], nodes[7], nodes[-2] = 0, 0, 64
    FourBit(10, lens, nodes, 2, 4, 64, 16).check()


@gpu
@pytest.mark.parametrize("decode", [True, False])
def test_scores_far_apart(decode):
    """Scores of hundreds: the running maximum moves from tile to tile, and most weights vanish."""
    FourBit(14, [700, 300], [10, 3], 2, 4, 128, 16, q_scale=60.0, decode=decode).check()


@gpu
@pytest.mark.parametrize("decode", [True, False])
def test_queries_of_any_size(decode):
    for e in (-120, -60, 0, 60):
        c = FourBit(15, [300, 40], [10, 3], 2, 4, 128, 16, q_scale=2.0 ** e, decode=decode)
        c.scale = 128 ** -0.5 * 2.0 ** -e
        c.check()


@gpu
@pytest.mark.parametrize("decode", [True, False])
def test_values_far_apart(decode):
    """Values over the whole range of the scales."""
    FourBit(16, [700, 90], [10, 3], 2, 4, 128, 16, spread=3.0, decode=decode).check()


@gpu
@pytest.mark.parametrize("group,n,L", [(4, 5, 40), (4, 64, 300), (4, 70, 70), (1, 3, 200), (20, 6, 140)])
def test_nan_groups_of_hidden_nodes_stay_there(group, n, L):
    """Scales that are NaN, of single groups of V and of K: columns of rows that see the node are
    NaN, nothing else."""
    c = FourBit(12, [L], [n], 2, group, 128, 16, words=-(-n // 64))
    for node, grp, head, what in ((1, 5, 0, "v"), (2, 0, 1, "v"), (n - 1, 7, 0, "v"), (0, 3, 1, "k")):
        j = L - n + node
        (c.v_scales if what == "v" else c.k_scales)[int(c.tables[0, j // 16]), head, j % 16, grp] = 0xff if node == 2 else 0x7f
    c.refresh()
    c.check()
    assert not torch.isnan(c.reference()[0]).all()


@gpu
@pytest.mark.parametrize("decode", [True, False])
def test_nan_groups_of_the_context_show(decode):
    c = FourBit(13, [300, 60], [9, 2], 2, 4, 128, 16, decode=decode)
    for s, j, grp, what in ((0, 17, 4, "v"), (1, 40, 2, "k")):
        (c.v_scales if what == "v" else c.k_scales)[int(c.tables[s, j // 16]), 1, j % 16, grp] = 0x7f
    c.refresh()
    c.check()


@gpu
@pytest.mark.parametrize("decode", [True, False])
def test_strided_views_and_a_side_stream(decode):
    """K and V as views of one tensor with the heads outermost, scales too, queries and outputs
    as slices of wider rows, tables with a row stride, on a stream of its own."""
    c = FourBit(30, [90, 200], [7, 20], 2, 4, 128, 16, decode=decode)
    x = c.device()
    both = torch.stack([x["kc"].transpose(0, 1), x["vc"].transpose(0, 1)])
    x["kc"], x["vc"] = both[0].transpose(0, 1), both[1].transpose(0, 1)
    sc = torch.stack([x[n].view(torch.uint8).transpose(0, 1) for n in ("ks", "vs")]).view(torch.float8_e4m3fn)
    x["ks"], x["vs"] = sc[0].transpose(0, 1), sc[1].transpose(0, 1)
    wide_q = torch.zeros(c.T, 10, 136, dtype=torch.bfloat16, device="cuda")
    wide_q[:, 1:9, :128] = x["q"]
    x["q"] = wide_q[:, 1:9, :128]
    wide_o = torch.full((c.T, 9, 144), 7.0, dtype=torch.bfloat16, device="cuda")
    x["out"] = wide_o[:, :8, 8:136]
    wide_t = torch.full((2, c.mb + 5), -1, dtype=torch.int32, device="cuda")
    wide_t[:, :c.mb] = x["tables"]
    x["tables"] = wide_t[:, :c.mb]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c.call(x, stream=st)
    torch.cuda.synchronize()
    assert binding.read_device_errors() == 0
    c.check(x["out"])
    assert (wide_o[:, 8] == 7).all() and (wide_o[:, :, :8] == 7).all() and (wide_o[:, :, 136:] == 7).all()


@gpu
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("shift", [1, 3])
def test_rows_and_scales_of_any_alignment(shift, decode):
    """Query and output rows off a 16-byte boundary, scale arrays off it by a token's."""
    c = FourBit(31, [90, 20, 300], [7, 2, 1], 2, 2, 128, 16, decode=decode)
    x = c.device()
    odd = torch.zeros(c.T * 4 * 128 + shift, dtype=torch.bfloat16, device="cuda")
    odd[shift:] = x["q"].reshape(-1)
    x["q"] = odd[shift:].view(c.T, 4, 128)
    o = torch.zeros(c.T * 4 * 128 + shift, dtype=torch.bfloat16, device="cuda")
    x["out"] = o[shift:].view(c.T, 4, 128)
    c.check(c.call(x))
    x = c.device()
    for n in ("ks", "vs"):
        raw = torch.zeros(x[n].numel() + 8, dtype=torch.uint8, device="cuda")
        raw[8:] = x[n].view(torch.uint8).reshape(-1)
        x[n] = raw[8:].view(torch.float8_e4m3fn).view(x[n].shape)
    c.check(c.call(x))


@gpu
def test_rows_behind_the_batch_and_bad_sequences_stay():
    c = FourBit(32, [60, 40, 70], [5, 4, 6], 2, 4, 128, 16)
    x = c.device()
    pad = torch.zeros(6, 8, 128, dtype=torch.bfloat16, device="cuda")
    x["q"] = torch.cat([x["q"], pad])
    x["out"] = torch.full_like(x["q"], 7.0)
    x["mask"] = torch.cat([x["mask"], torch.ones(6, 1, dtype=torch.int64, device="cuda")])
    c.call(x)
    torch.cuda.synchronize()
    assert binding.read_device_errors() == 0
    c.check(x["out"][:c.T])
    assert (x["out"][c.T:] == 7).all()
    for bad in (-1, 3, c.mb * 16 + 1):  # negative, shorter than its nodes, past the table
        x["lens"][1] = bad
        x["out"].fill_(7.0)
        c.call(x)
        assert binding.read_device_errors() == binding.DEVERR["context_len"]
        assert (x["out"][5:9] == 7).all() and (x["out"][c.T:] == 7).all()


@gpu
@pytest.mark.parametrize("decode", [True, False])
def test_bad_table_entries_are_reported(decode):
    c = FourBit(33, [60, 40], [5, 4], 2, 4, 128, 16, decode=decode)
    x = c.device()
    for bad in (c.kc.shape[0], -1):
        x["tables"][0, 1] = bad
        c.call(x)
        assert binding.read_device_errors() == binding.DEVERR["table_entry"]


@gpu
@pytest.mark.parametrize("decode", [True, False])
def test_same_bits_every_time_and_from_a_graph(decode):
    a = FourBit(34, [5000, 300], [30, 5], 2, 4, 128, 16, decode=decode)
    b = FourBit(35, [800], [64], 2, 4, 128, 16, decode=decode)
    xa, xb = a.device(), b.device()
    ea, eb = a.call(xa).clone(), b.call(xb).clone()
    for _ in range(3):
        assert torch.equal(a.call(xa), ea) and torch.equal(b.call(xb), eb)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call(xa)
        b.call(xb)
    xa["out"].zero_(), xb["out"].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(xa["out"], ea) and torch.equal(xb["out"], eb)
    xa["q"].mul_(0.5)
    g.replay()
    got = xa["out"].clone()
    assert torch.equal(got, a.call(xa))
    assert binding.read_device_errors() == 0


@gpu
def test_copy_blocks_of_a_four_bit_cache():
    kc, vc, ks, vs = caches(9, 3, 4, 64)
    g = torch.Generator().manual_seed(0)
    for x in (kc, ks):
        raw = x.view(torch.uint8)
        raw.copy_(torch.randint(0, 256, raw.shape, generator=g, dtype=torch.uint8))
        want = raw.clone()
        want[[7, 2]] = want[[0, 5]]
        binding.copy_blocks(x, torch.tensor([[0, 7], [5, 2]]).cuda())
        assert torch.equal(raw, want)
    assert binding.read_device_errors() == 0


# ---- refusals ------------------------------------------------------------------------------


def _four(nb=20, hk=2, bs=16, d=128):
    c = torch.zeros(nb, hk, bs, d // 2, dtype=torch.uint8)
    s = torch.zeros(nb, hk, bs, d // 16).to(torch.float8_e4m3fn)
    return dict(key_cache=c, value_cache=c.clone(), k_token_scales=s, v_token_scales=s.clone())


def _status(fn, **kw):
    try:
        fn(**kw)
        return 0
    except binding.PkvError as e:
        assert e.message
        return e.status


def _bad_scales(a):
    """Argument sets with scales that do not fit the cache, and the status of each."""
    s = a["k_token_scales"]
    yield dict(k_token_scales=None, v_token_scales=None), 1
    yield dict(k_token_scales=torch.ones(20, 2, 16), v_token_scales=torch.ones(20, 2, 16)), 1
    yield dict(k_token_scales=torch.zeros(20, 2, 16, 8), v_token_scales=torch.zeros(20, 2, 16, 8)), 2
    yield dict(k_token_scales=s[:, :, :, :4], v_token_scales=s[:, :, :, :4]), 1
    yield dict(k_token_scales=s[:19], v_token_scales=s[:19]), 1
    raw = torch.zeros(s.numel() + 4, dtype=torch.uint8)
    odd = raw[4:].view(torch.float8_e4m3fn).view(s.shape)
    yield dict(k_token_scales=odd, v_token_scales=s), 1
    yield dict(v_token_scales=torch.zeros(20, 4, 16, 8).to(torch.float8_e4m3fn)[:, ::2]), 1  # other strides than K's
    yield dict(key_cache=torch.zeros(20, 2, 16, 32, dtype=torch.uint8)), 1
    yield dict(key_cache=torch.zeros(20, 2, 16, 16, dtype=torch.uint8), value_cache=torch.zeros(20, 2, 16, 16, dtype=torch.uint8)), 2
    yield dict(k_scale=0.0), 1
    yield dict(v_scale=-1.0), 1
    yield dict(v_scale=math.inf), 1


def _quantize_args(**over):
    a = dict(key=torch.zeros(5, 2, 128), value=torch.zeros(5, 2, 128), slot_mapping=torch.zeros(5, dtype=torch.int64), **_four())
    a.update(over)
    return a


def test_write_and_read_refusals(dry):
    f = binding.quantize_and_cache
    a = _quantize_args()
    assert _status(f, **a) == 0
    for over, status in _bad_scales(a):
        if over.get("k_token_scales", 1) is None:
            continue  # (not optional here)
        assert _status(f, **{**a, **over}) == status, over.keys()
        assert _status(binding.read_cache, **{**a, **over}) == status, over.keys()
    assert _status(binding.read_cache, **{**a, "k_token_scales": None, "v_token_scales": None}) == 1
    assert _status(f, **_quantize_args(key=torch.zeros(5, 2, 64), value=torch.zeros(5, 2, 64))) == 1
    assert _status(f, **_quantize_args(key=torch.zeros(5, 3, 128), value=torch.zeros(5, 3, 128))) == 1
    # calls without scale arrays do not take these caches
    w = {k: v for k, v in a.items() if "token" not in k}
    assert _status(binding.reshape_and_cache, **w) == 2


def test_attention_refusals(dry):
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    a = dict(out=q.clone(), query=q, block_tables=torch.zeros(3, 4, dtype=torch.int32),
             context_lens=torch.ones(3, dtype=torch.int32), num_kv_heads=2, scale=0.1, block_size=16, max_blocks_per_seq=4,
             **_four())
    assert _status(binding.paged_attention_decode_quantized, **a) == 0
    t = dict(a, query_start_loc=torch.zeros(4, dtype=torch.int32), tree_mask=torch.zeros(3, 1, dtype=torch.int64))
    assert _status(binding.paged_attention_tree, **t) == 0
    for over, status in _bad_scales(a):
        assert _status(binding.paged_attention_tree, **{**t, **over}) == status, over.keys()
        if over.get("k_token_scales", 1) is not None:
            assert _status(binding.paged_attention_decode_quantized, **{**a, **over}) == status, over.keys()
    d = {k: v for k, v in a.items() if "token" not in k}
    assert _status(binding.paged_attention_decode, **d) == 2
    assert _status(binding.paged_attention_prefill, **d, query_start_loc=torch.zeros(4, dtype=torch.int32)) == 2
    # head scales go with the cache's device and type
    with pytest.raises(ValueError):
        binding.paged_attention_decode_quantized(**a, k_head_scales=torch.ones(2, dtype=torch.float64))
