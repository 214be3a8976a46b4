"""The token calls and the tree attention at the limits of what they take: caches past 2^31 elements,
1024 drafted nodes, 128 heads a KV head and more, scales for each head, no query heads, no tokens;
and a step of all of them captured into a graph.  Tolerances as in test_tree_attention.py."""
import math

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


def far_pool(t, shape, first):
    """A pool of `shape` whose blocks from `first` on are t's (the rest is not initialised)."""
    big = torch.empty(shape, dtype=t.dtype, device="cuda")
    big[first:first + t.shape[0]] = t
    return big


@gpu
@pytest.mark.parametrize("cache,decode", [("bf16", False), ("int8", False), ("int8", True), ("e4m3", False)])
def test_attention_past_2_to_31_elements(cache, decode):
    """The blocks of a case at the far end of a large pool: the bits of the small one."""
    c = Case(60, [300, 45], [9, 5], 8, 4, 128, 32, cache=cache, decode=decode, poison=False)
    x = c.device()
    near = c.call(x).clone()
    first = 2 ** 31 // (8 * 32 * 128) + 5
    nb = first + c.kc.shape[0]
    x["kc"], x["vc"] = (far_pool(x[k], (nb, 8, 32, 128), first) for k in ("kc", "vc"))
    if cache == "int8":
        x["ks"], x["vs"] = (far_pool(x[k], (nb, 8, 32), first) for k in ("ks", "vs"))
    x["tables"] = torch.where(x["tables"] >= 0, x["tables"] + first, x["tables"])
    assert torch.equal(c.call(x).view(torch.int16), near.view(torch.int16))
    assert binding.read_device_errors() == 0


@gpu
def test_token_passes_past_2_to_31_elements():
    T, hk, d, bs = 70, 8, 128, 32
    q, k, v, pos, slots, nb = inputs(61, T, 4, hk, d, bs, torch.bfloat16)
    first = 2 ** 31 // (hk * bs * d) + 5
    rot = binding.rotary(d)
    dev = [t.cuda() for t in (q, k, v, pos)]
    small, large = [], []
    for out, at, blocks in ((small, 0, nb), (large, first, first + nb)):
        kc, vc = (torch.empty(blocks, hk, bs, d, dtype=torch.int8, device="cuda") for _ in range(2))
        ks, vs = (torch.empty(blocks, hk, bs, device="cuda") for _ in range(2))
        kb, vb = (torch.empty(blocks, hk, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        s = slots.cuda() + at * bs
        y = torch.empty_like(dev[0])
        binding.rotary_and_cache(y, *dev, kc, vc, s, rot, k_token_scales=ks, v_token_scales=vs)
        binding.rotary_and_cache(y, *dev, kb, vb, s, rot)
        pairs = torch.stack([s // bs, s // bs + 1], 1)[:1].contiguous()
        rk, rv, rk2, rv2 = (torch.empty(T, hk, d, device="cuda") for _ in range(4))
        binding.read_cache(rk, rv, kc, vc, s, k_token_scales=ks, v_token_scales=vs)
        binding.read_cache(rk2, rv2, kb, vb, s)
        binding.quantize_and_cache(rk2, rv2, kc, vc, ks, vs, s)
        b, o = s // bs, s % bs
        out += [y, rk, rv, rk2, rv2, kc[b, :, o], vc[b, :, o], ks[b, :, o], vs[b, :, o]]
        src = int(pairs[0, 0])
        want = kc[src].clone(), ks[src].clone()
        pairs[0, 1] = at + nb - 1 if src != at + nb - 1 else at
        binding.copy_blocks(kc, pairs)
        binding.copy_blocks(ks, pairs)
        dst = int(pairs[0, 1])
        assert torch.equal(kc[dst], want[0]) and torch.equal(ks[dst].view(torch.int32), want[1].view(torch.int32))
        del kc, vc, ks, vs, kb, vb
    for a, b in zip(small, large):
        assert torch.equal(a, b)
    assert binding.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("L,group,d,masks", [(1500, 1, 64, "tree"), (1024, 4, 64, "bits"), (1100, 3, 128, "chain")])
def test_trees_of_1024_nodes(L, group, d, masks, cache):
    c = Case(62, [L, 30], [1024, 3], 1, group, d, 16, cache=cache, words=16, masks=masks)
    if cache == "bf16":
        for node, val in ((0, math.nan), (500, math.inf), (1023, -math.inf), (640, math.nan)):
            j = L - 1024 + node
            c.vc[int(c.tables[0, j // 16]), 0, j % 16, 7] = val
        c.K64, c.V64 = c.kc.double(), c.vc.double()
    c.check()


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("group,d", [(127, 64), (128, 128), (129, 64), (64, 128), (65, 64)])
def test_many_heads_a_kv_head(group, d, cache):
    Case(group, [200, 33, 5], [3, 7, 1], 1, group, d, 16, cache=cache).check()
    if cache == "int8":
        Case(group, [200, 33, 500, 0], None, 1, group, d, 16, cache=cache, decode=True).check()


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_contexts_that_fill_their_tables(cache):
    c = Case(63, [256, 128, 64], [8, 128, 64], 2, 2, 64, 16, cache=cache, words=2)
    c.mb = 16
    c.tables = c.tables[:, :16].contiguous()
    c.check()


@gpu
@pytest.mark.parametrize("hk,group", [(3, 2), (2, 9)])
def test_e4m3_trees_and_read_back_with_scales_for_each_head(hk, group):
    c = Case(64, [90, 20], [7, 5], hk, group, 128, 16, cache="e4m3")
    x = c.device()
    ks, vs = torch.rand(hk) * 0.02 + 0.005, torch.rand(hk) * 0.03 + 0.01
    c.K64, c.V64 = (t.float().double() * s.double().view(1, hk, 1, 1) for t, s in ((c.kc, ks), (c.vc, vs)))
    out = binding.paged_attention_tree(
        x["out"], x["q"], x["kc"], x["vc"], x["tables"], x["lens"], x["starts"], x["mask"], hk, c.scale, 16, c.mb,
        k_head_scales=ks.cuda(), v_head_scales=vs.cuda())
    c.check(out)
    slots = torch.arange(40)
    k, v = (torch.empty(40, hk, 128).cuda() for _ in range(2))
    binding.read_cache(k, v, x["kc"], x["vc"], slots.cuda(), k_head_scales=ks.cuda(), v_head_scales=vs.cuda())
    for got, t, s in ((k, c.kc, ks), (v, c.vc, vs)):
        want = t.float()[slots // 16, :, slots % 16] * s.view(1, hk, 1)
        there = ~torch.isnan(want)                             # (values past e4m3's range are NaN codes)
        assert torch.equal(torch.isnan(got.cpu()), ~there) and torch.equal(got.cpu()[there], want[there])
    assert binding.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("rd", [0, 128, 50])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rotary_without_query_heads_and_without_tokens(rd, dt):
    rot = binding.rotary(rd)
    q, k, v, pos, slots, nb = inputs(65, 33, 1, 2, 128, 16, dt)
    none = torch.empty(33, 0, 128, dtype=dt).cuda()
    kc = torch.zeros(nb, 2, 16, 128, dtype=dt).cuda()
    vc = torch.zeros_like(kc)
    binding.rotary_and_cache(none, none, k.cuda(), v.cuda(), pos.cuda(), kc, vc, slots.cuda(), rot)
    at = (slots // 16, slice(None), slots % 16)
    check_near(kc.cpu()[at], *rotate64(k, pos, rot), dt)
    assert torch.equal(vc.cpu()[at], v)
    c8 = torch.zeros(nb, 2, 16, 128, dtype=torch.int8).cuda()
    v8, ks = torch.zeros_like(c8), torch.zeros(nb, 2, 16).cuda()
    vs = torch.zeros_like(ks)
    binding.rotary_and_cache(none, none, k.cuda(), v.cuda(), pos.cuda(), c8, v8, slots.cuda(), rot, k_token_scales=ks,
                             v_token_scales=vs)
    code, scale = quantise(v.float())
    assert torch.equal(v8.cpu()[at], code) and torch.equal(vs.cpu()[at], scale)
    n0 = binding.launch_count()
    e = torch.empty
    binding.rotary_and_cache(e(0, 4, 128, dtype=dt).cuda(), e(0, 4, 128, dtype=dt).cuda(), k[:0].cuda(), v[:0].cuda(),
                             pos[:0].cuda(), kc, vc, slots[:0].cuda(), rot)
    binding.quantize_and_cache(k[:0].cuda(), v[:0].cuda(), c8, v8, ks, vs, slots[:0].cuda())
    binding.read_cache(k[:0].cuda(), v[:0].cuda(), kc, vc, slots[:0].cuda())
    assert binding.launch_count() == n0 and binding.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_a_captured_step_gives_the_eager_steps_bits(cache):
    """Rotation and write, block copy, tree attention, read back and write in another place: captured
    once and replayed on other inputs, against the same calls made eagerly on copies."""
    hq, hk, d, bs, S, n, mb = 8, 2, 128, 16, 3, 5, 6
    g = torch.Generator().manual_seed(66)
    rot = binding.rotary(d, scaling="bands", factor=8.0, original_max_position=8192)
    dt = torch.int8 if cache == "int8" else torch.bfloat16
    T, nb = S * n, S * mb + 2

    def fresh():
        x = dict(kc=torch.zeros(nb, hk, bs, d, dtype=dt).cuda(), vc=torch.zeros(nb, hk, bs, d, dtype=dt).cuda())
        if cache == "int8":
            x.update(ks=torch.zeros(nb, hk, bs).cuda(), vs=torch.zeros(nb, hk, bs).cuda())
        x.update(q=torch.empty(T, hq, d, dtype=torch.bfloat16).cuda(), out=torch.zeros(T, hq, d, dtype=torch.bfloat16).cuda(),
                 k=torch.empty(T, hk, d, dtype=torch.bfloat16).cuda(), v=torch.empty(T, hk, d, dtype=torch.bfloat16).cuda(),
                 rk=torch.zeros(T, hk, d).cuda(), rv=torch.zeros(T, hk, d).cuda(), pos=torch.zeros(T, dtype=torch.int64).cuda(),
                 slots=torch.zeros(T, dtype=torch.int64).cuda(), lens=torch.zeros(S, dtype=torch.int32).cuda(),
                 tables=torch.arange(S * mb).int().view(S, mb).cuda(), starts=torch.arange(0, T + 1, n).int().cuda(),
                 mask=torch.tensor([[(2 << i) - 1] for i in range(n)] * S).cuda(),
                 pairs=torch.tensor([[0, nb - 1], [mb, nb - 2]]).cuda())
        return x

    def step(x):
        sc = dict(k_token_scales=x["ks"], v_token_scales=x["vs"]) if cache == "int8" else {}
        binding.rotary_and_cache(x["q"], x["q"], x["k"], x["v"], x["pos"], x["kc"], x["vc"], x["slots"], rot, **sc)
        for name in ("kc", "vc") + (("ks", "vs") if cache == "int8" else ()):
            binding.copy_blocks(x[name], x["pairs"])
        binding.paged_attention_tree(x["out"], x["q"], x["kc"], x["vc"], x["tables"], x["lens"], x["starts"], x["mask"],
                                     hk, d ** -0.5, bs, mb, **sc)
        binding.read_cache(x["rk"], x["rv"], x["kc"], x["vc"], x["slots"], **sc)
        if cache == "int8":
            binding.quantize_and_cache(x["rk"], x["rv"], x["kc"], x["vc"], x["ks"], x["vs"], x["slots"])

    def load(x, i, q, k, v):
        base = 20 * i
        x["q"].copy_(q), x["k"].copy_(k), x["v"].copy_(v)
        j = torch.arange(n).repeat(S) + base
        x["pos"].copy_(j + 100)
        x["slots"].copy_(torch.arange(S).repeat_interleave(n) * mb * bs + j)
        x["lens"].fill_(base + n)

    a, b = fresh(), fresh()
    load(b, 0, torch.zeros(T, hq, d), torch.zeros(T, hk, d), torch.zeros(T, hk, d))
    step(b)                                                    # (the workspace has its size)
    torch.cuda.synchronize()
    b = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for i in range(4):
        new = [torch.randn(T, h, d, generator=g) for h in (hq, hk, hk)]
        load(a, i, *new), load(b, i, *new)
        step(a)
        graph.replay()
        torch.cuda.synchronize()
        for name in a:
            x, y = a[name], b[name]
            same = x.view(torch.int16) if x.dtype == torch.bfloat16 else x
            assert torch.equal(same, y.view(torch.int16) if y.dtype == torch.bfloat16 else y), (i, name)
        assert bool((a["out"] != 0).any())
    assert binding.read_device_errors() == 0
