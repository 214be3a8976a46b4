"""The 4-bit cache, position axes and the calls over many caches at the limits of what they take:
pools past 2^32 bytes, block strides past 2^32, 1024 drafted nodes, 64 to 129 heads a KV head, scales
of the scores of any sign, queries that are no numbers, workspaces, caches without heads; and a step
of all of them captured into a graph.  Tolerances as in test_four_bit_cache.py."""
import math

import pytest
import torch
from test_four_bit_cache import FourBit, caches
from test_pages import Draft, noise
from test_token_limits import far_pool

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


def bits(t):
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32)


def far_bytes(t, shape, first):
    return far_pool(t.view(torch.uint8), shape, first).view(t.dtype)


@gpu
@pytest.mark.parametrize("decode,qdtype", [(True, torch.bfloat16), (False, torch.bfloat16), (False, torch.float32)])
def test_attention_past_2_to_32_bytes(decode, qdtype):
    """The blocks of a case at the far end of a large pool: the bits of the small one."""
    c = FourBit(60, [300, 45], [9, 5], 8, 4, 128, 32, decode=decode, qdtype=qdtype, poison=False)
    x = c.device()
    near = c.call(x).clone()
    first = 2 ** 32 // (8 * 32 * 64) + 5
    nb = first + c.kc.shape[0]
    x["kc"], x["vc"] = (far_bytes(x[k], (nb, 8, 32, 64), first) for k in ("kc", "vc"))
    x["ks"], x["vs"] = (far_bytes(x[k], (nb, 8, 32, 8), first) for k in ("ks", "vs"))
    x["tables"] = torch.where(x["tables"] >= 0, x["tables"] + first, x["tables"])
    assert torch.equal(bits(c.call(x)), bits(near))
    assert binding.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("decode", [True, False])
def test_blocks_more_than_2_to_32_bytes_apart(decode):
    c = FourBit(62, [50, 20], [9, 5], 1, 4, 64, 32, decode=decode, poison=False)
    x = c.device()
    for n in ("kc", "vc"):
        shape = x[n].shape
        apart = torch.empty((shape[0] - 1) * (2 ** 32 + 64) + shape[1:].numel(), dtype=torch.uint8, device="cuda")
        view = apart.as_strided(shape, (2 ** 32 + 64, shape[2] * shape[3], shape[3], 1))
        view.copy_(x[n])
        x[n] = view
    c.check(c.call(x))


@gpu
def test_passes_past_2_to_32_bytes():
    """Writes, read back, copies and kept tokens at the far end of a pool: the bytes of the small one."""
    T, hk, d, bs, nb = 70, 8, 128, 32, 6
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(T, hk, d, generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn(T, 4, d, generator=g).bfloat16().cuda()
    slots = torch.randperm(nb * bs, generator=g)[:T]
    positions = torch.randint(0, 2 ** 20, (3, T), generator=g).cuda()
    rot = binding.rotary(d, axes=binding.rotary_axes([16, 24, 24]))
    first = 2 ** 32 // (hk * bs * d // 2) + 5
    small, large = [], []
    for out, at in ((small, 0), (large, first)):
        kc, vc = (torch.empty(at + nb, hk, bs, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.empty(at + nb, hk, bs, d // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
        for t in (kc, vc, ks, vs):
            t[at:] = 0x11
        ks, vs = ks.view(torch.float8_e4m3fn), vs.view(torch.float8_e4m3fn)
        scales = dict(k_token_scales=ks, v_token_scales=vs)
        s = slots.cuda() + at * bs
        binding.quantize_and_cache(k, v, kc, vc, ks, vs, s)
        back = [torch.empty_like(k), torch.empty_like(v)]
        binding.read_cache(*back, kc, vc, s, **scales)
        out += [t.clone() for t in back]
        y = torch.empty_like(q)
        binding.rotary_and_cache(y, q, k, v, positions, kc, vc, s, rot, **scales)
        cl = binding.cache_list([kc, vc, ks, vs])
        binding.copy_cache_blocks(cl, torch.tensor([[at, at + 5], [at + 1, at + 4]], device="cuda"))
        i32 = dict(dtype=torch.int32, device="cuda")
        binding.keep_tokens(cl, torch.tensor([[at + 2, at + 3]], **i32), torch.tensor([60], **i32),
                            torch.tensor([0, 40], **i32), torch.arange(1, 80, 2, **i32), torch.tensor([20], **i32), bs, 2)
        out += [y] + [t[at:].view(torch.uint8).clone() for t in (kc, vc, ks, vs)]
        assert binding.read_device_errors() == 0
    for a, b in zip(small, large):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@gpu
@pytest.mark.parametrize("L,n", [(1024, 1024), (1500, 1024), (1100, 1000)])
def test_trees_of_up_to_1024_nodes(L, n):
    """Nodes that touch up to nine tiles, with a NaN scale hidden from most of them."""
    c = FourBit(n + L, [L, 3], [n, 3], 1, 2, 64, 16, words=16)
    j = L - n + n // 2
    c.v_scales[int(c.tables[0, j // 16]), 0, j % 16, 1] = 0x7f
    c.refresh()
    c.check()


@gpu
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("group", [17, 33, 64, 65, 127, 128, 129])
def test_many_heads_of_a_kv_head(group, decode):
    FourBit(group, [200, 17, 129], [5, 2, 1], 1, group, 64, 16, decode=decode).check()


@gpu
@pytest.mark.parametrize("group,bs", [(4, 16), (4, 4), (20, 16)])
@pytest.mark.parametrize("factor", [0.0, -1.0, -60.0])
def test_score_scales_of_any_sign(factor, group, bs):
    for decode in (True, False):
        c = FourBit(70, [300, 40, 1], [10, 3, 1], 2, group, 128, bs, decode=decode)
        c.scale *= factor
        c.check()


@gpu
@pytest.mark.parametrize("decode", [True, False])
def test_queries_that_are_no_numbers_spoil_their_own_rows_alone(decode):
    c = FourBit(71, [300, 40, 260], [10, 3, 9], 2, 8, 128, 16, decode=decode)
    x = c.device()
    good = c.call(x).clone()
    for row, head, value in ((0, 3, math.nan), (1, 8, math.inf), (2, 15, -math.inf)):
        x["q"][row, head, 7] = value
    out = c.call(x)
    spoilt = torch.zeros(c.T, 16, dtype=torch.bool, device="cuda")
    spoilt[0, 3] = spoilt[1, 8] = spoilt[2, 15] = True
    assert torch.isnan(out[spoilt]).all()
    assert torch.equal(bits(out)[~spoilt], bits(good)[~spoilt])


@gpu
def test_tables_that_are_full_and_one_block_pools():
    for decode in (True, False):
        c = FourBit(72, [64, 32, 17], [4, 1, 2], 2, 4, 128, 16, decode=decode, poison=False)
        x = c.device()
        x["tables"], c.mb = x["tables"][:, :4].contiguous(), 4  # no entry behind the longest context
        c.check(c.call(x))
    c = FourBit(73, [7], [3], 1, 4, 64, 8, poison=False)
    x = c.device()
    b = int(c.tables[0, 0])
    for n in ("kc", "vc", "ks", "vs"):
        x[n] = x[n].view(torch.uint8)[b:b + 1].clone().view(x[n].dtype)
    x["tables"] = torch.zeros_like(x["tables"])
    c.check(c.call(x))


@gpu
def test_empty_batches_and_no_heads():
    kc, vc, ks, vs = caches(3, 2, 16, 128)
    before = [t.view(torch.uint8).clone() for t in (kc, vc, ks, vs)]
    scales = dict(k_token_scales=ks, v_token_scales=vs)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    k = torch.empty(0, 2, 128, device="cuda")
    rot = binding.rotary(128, axes=[0] * 64)
    binding.quantize_and_cache(k, k, kc, vc, ks, vs, none)
    binding.rotary_and_cache(k, k, k, k, none[None], kc, vc, none, rot, **scales)
    # no query heads: keys and values are written all the same
    k = torch.randn(2, 2, 128, device="cuda")
    q = torch.empty(2, 0, 128, device="cuda")
    for t, b in zip((kc, vc, ks, vs), before):
        assert torch.equal(t.view(torch.uint8), b)
    binding.rotary_and_cache(q, q, k, k, torch.zeros(1, 2, dtype=torch.int64, device="cuda"), kc, vc,
                             torch.tensor([3, 20], device="cuda"), rot, **scales)
    assert torch.equal(kc, vc) and torch.equal(ks.view(torch.uint8), vs.view(torch.uint8))  # (position 0)
    assert not torch.equal(kc, before[0]) and binding.read_device_errors() == 0


@gpu
def test_kept_lengths_of_caches_without_heads():
    d = Draft(8, [40, 9], [12, 3], [5, 0], 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    empty = torch.empty(d.nb, 0, 16, 64, dtype=torch.bfloat16, device="cuda")
    full = noise((d.nb, 2, 16, 64), torch.bfloat16, torch.Generator().manual_seed(1))
    for cs in ([empty], [empty] * 2 + [full]):
        new = torch.zeros(2, **i32)
        d.call(cs, new)
        assert new.tolist() == [33, 6] and binding.read_device_errors() == 0
    binding.copy_cache_blocks([empty], torch.tensor([[0, 1]], device="cuda"))
    assert binding.read_device_errors() == 0


def test_new_lengths_share_no_memory_with_inputs(dry):
    """Every block of the launch reads the inputs, so a length that is written there is refused."""
    c = torch.zeros(6, 2, 16, 128)
    pool = torch.zeros(64, dtype=torch.int32)
    a = dict(caches=[c], block_tables=pool[0:12].view(3, 4), context_lens=pool[12:15], query_start_loc=pool[15:19],
             keep=pool[19:28], keep_counts=pool[28:31], block_size=16, max_blocks_per_seq=4)
    binding.keep_tokens(**a, new_lens=pool[31:34])
    for at in (0, 9, 11, 12, 13, 14, 18, 27, 28, 30):
        with pytest.raises(binding.PkvError) as e:
            binding.keep_tokens(**a, new_lens=pool[at:at + 3])
        assert e.value.status == 1


def test_workspace_of_a_four_bit_step():
    """What pkv_tree_workspace_bytes names is enough for decode and trees of every head layout."""
    f = binding.tree_workspace_bytes
    for group in (1, 4, 8, 9, 16, 17, 128):
        for T in (1, 7, 200, 5000):
            need = f(T, T, 2 * group, 2, 128)
            assert need > 0 and f(1, 1, 2 * group, 2, 128) <= need


@gpu
def test_a_step_in_a_graph_with_the_workspace_reserved():
    """Write with axes, tree, kept tokens, decode of the next token and a copied block: captured
    after the workspace is reserved, replayed on new inputs, against the same calls one by one."""
    hk, group, d, bs, nb, n = 2, 4, 128, 16, 12, 9
    g = torch.Generator().manual_seed(9)
    i32 = dict(dtype=torch.int32, device="cuda")
    binding.reserve_workspace(binding.tree_workspace_bytes(2, 2 * n, hk * group, hk, d))
    tables = torch.tensor([[3, 7, 1, 9], [0, 5, 11, 2]], **i32)
    lens, starts = torch.tensor([40, 60], **i32), torch.tensor([0, n, 2 * n], **i32)
    slots = torch.cat([tables[s].long()[p // bs] * bs + p % bs for s, L in enumerate((40, 60))
                       for p in [torch.arange(L - n, L, device="cuda")]])
    mask = torch.tensor([(1 << (i % n + 1)) - 1 for i in range(2 * n)], device="cuda")[:, None]
    positions = torch.stack([torch.arange(2 * n), torch.arange(2 * n) // 3, torch.arange(2 * n) % 3]).cuda()
    rot = binding.rotary(d, axes=binding.rotary_axes([16, 24, 24], cyclic=True))
    kc, vc, ks, vs = caches(nb, hk, bs, d, fill=0x21)
    cl = binding.cache_list([kc, vc, ks, vs])
    keep, counts, new = torch.tensor(list(range(0, n)) * 2, **i32), torch.tensor([4, 2], **i32), torch.zeros(2, **i32)
    pairs = torch.tensor([[3, 4], [11, 6]], device="cuda")
    q, q2 = (torch.empty(2 * n, hk * group, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.empty(2 * n, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out, out1 = torch.empty_like(q), torch.empty(2, hk * group, d, dtype=torch.bfloat16, device="cuda")

    def step():
        binding.rotary_and_cache(q2, q, k, v, positions, kc, vc, slots, rot, k_token_scales=ks, v_token_scales=vs)
        binding.paged_attention_tree(out, q2, kc, vc, tables, lens, starts, mask, hk, d ** -0.5, bs, 4,
                                     k_token_scales=ks, v_token_scales=vs)
        binding.keep_tokens(cl, tables, lens, starts, keep, counts, bs, 4, new_lens=new)
        binding.paged_attention_decode_quantized(out1, q2[:2], kc, vc, ks, vs, tables, new, hk, d ** -0.5, bs, 4)
        binding.copy_cache_blocks(cl, pairs)

    def fill(seed):
        g.manual_seed(seed)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g))
        keep[:4] = torch.tensor(sorted(torch.randperm(n, generator=g)[:4].tolist()), **i32)
        keep[n:n + 2] = torch.tensor(sorted(torch.randperm(n, generator=g)[:2].tolist()), **i32)

    def state():
        return [bits(out).clone(), bits(out1).clone(), bits(q2).clone(), new.clone()] + \
            [t.view(torch.uint8).clone() for t in (kc, vc, ks, vs)]

    start = [t.view(torch.uint8).clone() for t in (kc, vc, ks, vs)]
    fill(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (2, 3):
        fill(seed)
        got = []
        for run in (graph.replay, step):
            for t, s in zip((kc, vc, ks, vs), start):
                t.view(torch.uint8).copy_(s)
            run()
            torch.cuda.synchronize()
            got.append(state())
        assert all(torch.equal(a, b) for a, b in zip(*got))
        assert got[0][3].tolist() == [35, 53]
    assert binding.read_device_errors() == 0
