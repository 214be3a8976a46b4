"""Pages of many caches: blocks copied in all of them at once, accepted drafted tokens moved
together (byte for byte against indexing), the block manager's forks, cuts and packing, and a
whole step of a server over a 4-bit cache."""
import random

import pytest
import torch

from paged_kv_cache_90_gb300 import binding
from paged_kv_cache_90_gb300 import build as pkv_build
from paged_kv_cache_90_gb300.block_manager import BlockAllocator, BlockManager, PoolExhausted, PrefixCache, validate_cow_pairs

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


def noise(shape, dt, g):
    n = torch.zeros(shape, dtype=dt).element_size() if dt.is_floating_point else torch.iinfo(dt).bits // 8
    b = torch.randint(0, 256, (*shape[:-1], shape[-1] * n), generator=g, dtype=torch.uint8)
    return b.cuda().view(dt)


def some_caches(seed, nb, bs, layers=2):
    """Caches and scale arrays of every type, some with strides of their own."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for i in range(layers):
        hk, d = (3, 128) if i % 2 == 0 else (1, 64)
        for dt, w in ((torch.bfloat16, d), (torch.float32, d), (torch.float8_e4m3fn, d), (torch.int8, d), (torch.uint8, d // 2),
                      (torch.float8_e4m3fn, d // 16)):
            out.append(noise((nb, hk, bs, w), dt, g))
        out.append(torch.rand(nb, hk, bs, generator=g).cuda())
    # heads outermost; K and V of one tensor; wider scale rows
    out.append(noise((2, nb, bs, 128), torch.bfloat16, g).transpose(0, 1))
    both = noise((nb, 2, 3, bs, 128), torch.int8, g)
    out += [both[:, 0], both[:, 1]]
    out.append(torch.rand(nb, 5, bs, generator=g).cuda()[:, 1:4])
    return out


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---- copies --------------------------------------------------------------------------------


@gpu
@pytest.mark.parametrize("bs", [2, 8, 16, 32])
@pytest.mark.parametrize("n", [1, 3, 17])
def test_copy_cache_blocks(n, bs):
    nb = 40
    cs = some_caches(n, nb, bs)
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(n))
    src = perm[n:][torch.arange(n) % 5]   # sources may repeat
    pairs = torch.stack([src, perm[:n]], 1).cuda()
    want = []
    for c in cs:
        w = c.contiguous().view(torch.uint8).clone()
        w[perm[:n].cuda()] = w[src.cuda()]
        want.append(w)
    binding.copy_cache_blocks(binding.cache_list(cs), pairs)
    torch.cuda.synchronize()
    assert binding.read_device_errors() == 0
    for c, w in zip(cs, want):
        assert torch.equal(c.contiguous().view(torch.uint8), w)


@gpu
def test_copy_of_more_caches_than_a_launch_takes():
    """230 caches (three launches), passed as they are; what lies between the views stays."""
    g = torch.Generator().manual_seed(2)
    pool = noise((230, 6, 2, 8, 64), torch.bfloat16, g)
    want = pool.clone()
    want[:, 4] = want[:, 1]
    n0 = binding.launch_count()
    binding.copy_cache_blocks([pool[i] for i in range(230)], torch.tensor([[1, 4]]).cuda())
    assert same(pool, want) and binding.launch_count() - n0 == 3


@gpu
def test_copy_of_large_blocks_and_no_pairs():
    g = torch.Generator().manual_seed(3)
    c = noise((5, 64, 32, 128), torch.float32, g)   # 1 MB a block: many chunks
    want = c.clone()
    want[3] = want[0]
    binding.copy_cache_blocks([c], torch.tensor([[0, 3]]).cuda())
    assert same(c, want)
    binding.copy_cache_blocks([c], torch.empty(0, 2, dtype=torch.int64).cuda())
    assert same(c, want)


@gpu
def test_pairs_outside_the_pool_are_skipped_and_reported():
    g = torch.Generator().manual_seed(4)
    cs = [noise((6, 2, 16, 64), torch.bfloat16, g), torch.rand(6, 2, 16, generator=g).cuda()]
    want = [c.clone() for c in cs]
    for w in want:
        w[2] = w[5]
    binding.copy_cache_blocks(cs, torch.tensor([[0, 6], [5, 2], [-1, 3], [1 << 40, 1]]).cuda())
    assert binding.read_device_errors() == binding.DEVERR["copy_pair"]
    assert all(same(c, w) for c, w in zip(cs, want))
    binding.set_option("debug_sync", 1)
    try:
        for bad in ([[0, 1], [2, 1]], [[0, 1], [1, 2]]):
            with pytest.raises(binding.PkvError) as e:
                binding.copy_cache_blocks(cs, torch.tensor(bad).cuda())
            assert e.value.status == 4
        binding.copy_cache_blocks(cs, torch.tensor([[0, 1], [0, 2]]).cuda())
    finally:
        binding.set_option("debug_sync", 0)


# ---- accepted tokens -----------------------------------------------------------------------


class Draft:
    """Sequences with drafted nodes and the ascending ones that stay."""

    def __init__(self, seed, lens, nodes, kept, bs, pad=0):
        rng = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        self.lens, self.nodes, self.kept, self.bs = lens, nodes, kept, bs
        counts = [-(-n // bs) for n in lens]
        self.mb = max(counts + [1]) + 1
        self.nb = sum(counts) + 2
        perm = torch.randperm(self.nb, generator=g)
        self.tables = torch.full((len(lens), self.mb), -1, dtype=torch.int32)
        at = 0
        for s, c in enumerate(counts):
            self.tables[s, :c] = perm[at:at + c].int()
            at += c
        self.starts = torch.tensor([0] + nodes).cumsum(0).int()
        self.keep = torch.full((sum(nodes) + pad,), -9, dtype=torch.int32)
        for s, (n, k) in enumerate(zip(nodes, kept)):
            a = int(self.starts[s])
            self.keep[a:a + k] = torch.tensor(sorted(rng.sample(range(n), k)), dtype=torch.int32)
        self.skip = set()

    def slots(self, s, pos):
        return int(self.tables[s, pos // self.bs]) * self.bs + pos % self.bs

    def want(self, caches):
        """The caches afterwards, as bytes with the slots first."""
        of = torch.arange(self.nb * self.bs)
        for s, (L, n, k) in enumerate(zip(self.lens, self.nodes, self.kept)):
            if s in self.skip:
                continue
            for i in range(k):
                a = int(self.keep[int(self.starts[s]) + i])
                of[self.slots(s, L - n + i)] = self.slots(s, L - n + a)
        return [self.flat(c)[of.cuda()] for c in caches]

    def flat(self, c):
        n = c.shape[0] * c.shape[2]
        return c.transpose(1, 2).reshape(-1).view(torch.uint8).reshape(n, -1)

    def call(self, caches, new_lens=None, **over):
        x = dict(block_tables=self.tables.cuda(), context_lens=torch.tensor(self.lens, dtype=torch.int32).cuda(),
                 query_start_loc=self.starts.cuda(), keep=self.keep.cuda(),
                 keep_counts=torch.tensor(self.kept, dtype=torch.int32).cuda())
        x.update(over)
        return binding.keep_tokens(caches, **x, block_size=self.bs, max_blocks_per_seq=self.mb, new_lens=new_lens)

    def check(self, caches):
        want = self.want(caches)
        new = torch.full((len(self.lens),), 77, dtype=torch.int32, device="cuda")
        assert self.call(caches, new) is new
        torch.cuda.synchronize()
        assert binding.read_device_errors() == 0
        for c, w in zip(caches, want):
            assert torch.equal(self.flat(c), w)
        assert new.tolist() == [L - n + k for L, n, k in zip(self.lens, self.nodes, self.kept)]


@gpu
@pytest.mark.parametrize("bs", [2, 4, 8, 16, 32])
def test_keep_tokens(bs):
    """Every overlap: paths whose places are others' sources, all kept, none, one, prefixes,
    sequences without nodes or tokens, nodes that are the whole context."""
    d = Draft(bs, [40, 1, 33, 64, 9, 0, 130, 17, 20], [12, 1, 33, 5, 0, 0, 100, 17, 8], [5, 1, 20, 0, 0, 0, 71, 17, 1], bs)
    d.check(some_caches(bs, d.nb, bs))


@gpu
@pytest.mark.parametrize("n,k", [(64, 63), (65, 64), (200, 129), (300, 299), (1024, 400)])
def test_keep_of_many_nodes(n, k):
    """More kept tokens than are placed at a time."""
    d = Draft(n, [n + 13, n], [n, n], [k, 2], 16, pad=5)
    d.check([c for c in some_caches(n, d.nb, 16, layers=1)][:5])


@gpu
def test_keep_without_lengths_and_for_many_caches():
    d = Draft(3, [50, 60], [20, 30], [7, 11], 16)
    g = torch.Generator().manual_seed(1)
    pool = noise((150, d.nb, 2, 16, 64), torch.bfloat16, g)
    cs = [pool[i] for i in range(150)]
    want = d.want(cs)
    assert d.call(binding.cache_list(cs)) is None
    assert binding.read_device_errors() == 0
    for c, w in zip(cs, want):
        assert torch.equal(d.flat(c), w)
    d = Draft(4, [50, 60], [20, 30], [7, 11], 16)
    d.check([noise((d.nb, 2, 16, 64), torch.bfloat16, g) for _ in range(100)])


@gpu
def test_bad_sequences_stay_as_they_are():
    cases = []   # (what is changed, the error)
    for k, v in (([4, 2, 8], "keep"), ([-1, 3, 4], "keep"), ([2, 2, 5], "keep"), ([3, 4, 7], "keep")):
        cases.append((dict(keep=k), v))
    cases += [(dict(count=9), "keep"), (dict(count=-1), "keep"), (dict(len=7), "context_len"), (dict(len=-3), "context_len"),
              (dict(len=10 ** 6), "context_len"), (dict(entry=-1), "table_entry"), (dict(entry=10 ** 6), "table_entry")]
    for change, err in cases:
        d = Draft(5, [40, 50, 30], [8, 8, 8], [3, 3, 3], 8)
        a = int(d.starts[1])
        d.keep[a:a + 3] = torch.tensor(change.get("keep", [1, 3, 7]), dtype=torch.int32)
        if change.get("keep") == [3, 4, 7]:
            d.keep[a:a + 3] = torch.tensor([3, 4, 2 ** 31 - 1], dtype=torch.int32)
        counts = torch.tensor(d.kept, dtype=torch.int32)
        lens = torch.tensor(d.lens, dtype=torch.int32)
        tables = d.tables.clone()
        counts[1] = change.get("count", 3)
        lens[1] = change.get("len", 50)
        if "entry" in change:
            tables[1, 5] = change["entry"]   # positions 40..47: places 42.. of the path
        d.skip = {1}
        cs = some_caches(1, d.nb, 8, layers=1)
        want = d.want(cs)
        new = torch.full((3,), 77, dtype=torch.int32, device="cuda")
        d.call(cs, new, context_lens=lens.cuda(), keep_counts=counts.cuda(), block_tables=tables.cuda())
        assert binding.read_device_errors() == binding.DEVERR[err], change
        for c, w in zip(cs, want):
            assert torch.equal(d.flat(c), w), change
        assert new.tolist() == [35, 77, 25]


@gpu
def test_rows_outside_the_batch_are_reported():
    d = Draft(6, [40, 50], [8, 8], [3, 3], 8)
    cs = [noise((d.nb, 1, 8, 64), torch.bfloat16, torch.Generator().manual_seed(1))]
    before = cs[0].clone()
    for starts in ([0, 8, 17], [-1, 8, 7], [0, -2 ** 31, 2 ** 31 - 1], [16, 2 ** 31 - 1, 0]):
        d.call(cs, query_start_loc=torch.tensor(starts, dtype=torch.int32).cuda(),
               keep_counts=torch.zeros(2, dtype=torch.int32).cuda())
        assert binding.read_device_errors() == binding.DEVERR["context_len"], starts
    assert same(cs[0], before)


@gpu
def test_calls_from_graphs_and_on_a_side_stream():
    """A captured copy and a captured keep, replayed on other pairs and paths."""
    d = Draft(7, [60, 90], [20, 40], [9, 13], 16)
    g = torch.Generator().manual_seed(1)
    cs = [noise((d.nb + 4, 2, 16, 64), torch.bfloat16, g) for _ in range(3)]
    cl = binding.cache_list(cs)
    pairs = torch.tensor([[0, d.nb], [1, d.nb + 1]]).cuda()
    keep, counts, new = d.keep.cuda(), torch.tensor(d.kept, dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    tables, lens, starts = d.tables.cuda(), torch.tensor(d.lens, dtype=torch.int32).cuda(), d.starts.cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        binding.copy_cache_blocks(cl, pairs)
        binding.keep_tokens(cl, tables, lens, starts, keep, counts, 16, d.mb, new_lens=new)
    for seed in (8, 9):
        e = Draft(7, d.lens, d.nodes, d.kept, 16)
        other = Draft(seed, d.lens, d.nodes, d.kept, 16)
        e.keep, e.nb = other.keep, d.nb + 4
        keep.copy_(other.keep)
        p = torch.tensor([[seed % 3, d.nb + 2], [3, d.nb + 3]])
        pairs.copy_(p)
        want = []
        for c in cs:
            w = c.clone()
            w[p[:, 1].cuda()] = w[p[:, 0].cuda()]
            want.append(w)
        want = e.want(want)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(e.flat(c), w) for c, w in zip(cs, want))
        assert new.tolist() == [49, 63]
    assert binding.read_device_errors() == 0


# ---- refusals ------------------------------------------------------------------------------


def _status(fn, *a, **kw):
    try:
        fn(*a, **kw)
        return 0
    except binding.PkvError as e:
        assert e.message
        return e.status


def test_copy_refusals(dry):
    f = binding.copy_cache_blocks
    pairs = torch.zeros(3, 2, dtype=torch.int64)
    c, s = torch.zeros(6, 2, 16, 128), torch.zeros(6, 2, 16)
    assert _status(f, [c, s, c.bfloat16(), c.to(torch.int8)], pairs) == 0
    with pytest.raises(ValueError):
        f([], pairs)
    assert _status(f, [c, c[:5]], pairs) == 1                          # another pool
    assert _status(f, [c, torch.zeros(6, 2, 8, 128)], pairs) == 1      # another block size
    assert _status(f, [c, torch.zeros(6, 2, 16, 96)], pairs) == 2
    assert _status(f, [torch.zeros(6, 2, 3, 128)], pairs) == 2
    assert _status(f, [c, torch.zeros(6, 2, 16, 128, dtype=torch.int32)], pairs) == 2
    assert _status(f, [c, torch.zeros(6, 2, 16, dtype=torch.bfloat16)], pairs) == 2
    assert _status(f, [c], pairs.int()) == 2
    assert _status(f, [c], torch.zeros(3, 3, dtype=torch.int64)) == 1
    assert _status(f, [c], torch.zeros(6, 2, dtype=torch.int64)[::2]) == 1
    assert _status(f, [c.transpose(2, 3)], pairs) == 1
    assert _status(f, [c[:, :, :8]], pairs) == 0                       # (tiles of eight tokens, apart)
    assert _status(f, [c] * 1025, pairs) == 1
    lib = binding.load_library()
    assert lib.pkv_copy_cache_blocks(None, 1, binding._ref(pairs), None) == 1
    array = (type(binding.CacheList([c])._array[0]) * 1)()             # a null descriptor
    assert lib.pkv_copy_cache_blocks(array, 1, binding._ref(pairs), None) == 1


def test_keep_refusals(dry):
    c = torch.zeros(6, 2, 16, 128)
    a = dict(caches=[c, torch.zeros(6, 2, 16)], block_tables=torch.zeros(3, 4, dtype=torch.int32),
             context_lens=torch.zeros(3, dtype=torch.int32), query_start_loc=torch.zeros(4, dtype=torch.int32),
             keep=torch.zeros(9, dtype=torch.int32), keep_counts=torch.zeros(3, dtype=torch.int32), block_size=16,
             max_blocks_per_seq=4, new_lens=torch.zeros(3, dtype=torch.int32))
    f = binding.keep_tokens
    assert _status(f, **a) == 0 and _status(f, **{**a, "new_lens": None}) == 0
    for over in (dict(caches=[c, c]), dict(caches=[c, c[:5]]), dict(block_size=8), dict(max_blocks_per_seq=3),
                 dict(context_lens=torch.zeros(2, dtype=torch.int32)), dict(query_start_loc=torch.zeros(3, dtype=torch.int32)),
                 dict(keep_counts=torch.zeros(4, dtype=torch.int32)), dict(new_lens=torch.zeros(2, dtype=torch.int32)),
                 dict(new_lens=a["context_lens"]), dict(keep=torch.zeros(18, dtype=torch.int32)[::2]),
                 dict(keep=torch.zeros(3, 3, dtype=torch.int32))):
        assert _status(f, **{**a, **over}) == 1, over.keys()
    for over in (dict(keep=torch.zeros(9, dtype=torch.int64)), dict(context_lens=torch.zeros(3)),
                 dict(block_tables=torch.zeros(3, 4, dtype=torch.int64)), dict(keep_counts=torch.zeros(3, dtype=torch.int64))):
        assert _status(f, **{**a, **over}) == 2, over.keys()


# ---- the block manager ---------------------------------------------------------------------


def test_fork_copy_gives_the_child_its_own_partial_block():
    m = BlockManager(BlockAllocator(10, 4))
    m.add_sequence("a", 10)
    assert m.fork_copy("a", "b") == (2, 3)
    assert m.seqs["a"].blocks == [0, 1, 2] and m.seqs["b"].blocks == [0, 1, 3]
    assert m.append_token("a")[1] is None and m.append_token("b")[1] is None   # no copy is due
    m.add_sequence("c", 8)
    assert m.fork_copy("c", "d") is None and m.seqs["d"].blocks == m.seqs["c"].blocks
    m.check_structure()
    with pytest.raises(ValueError):
        m.fork_copy("a", "b")
    m.check_structure()
    full = BlockManager(BlockAllocator(3, 4))
    full.add_sequence("a", 10)
    with pytest.raises(PoolExhausted):
        full.fork_copy("a", "b")
    full.check_structure()
    assert "b" not in full.seqs


def test_truncate_gives_blocks_back():
    m = BlockManager(BlockAllocator(10, 4))
    m.add_sequence("a", 14)
    assert m.truncate("a", 9) == [3] and m.truncate("a", 9) == [] and m.seqs["a"].length == 9
    m.fork("a", "b")
    assert m.truncate("b", 4) == [1, 2] and m.alloc.refcount[1] == 1
    m.check_structure()
    for bad in (10, -1):
        with pytest.raises(ValueError):
            m.truncate("a", bad)
    m.release_outside_window("a", 3)
    with pytest.raises(ValueError):
        m.truncate("a", 4)   # its last token's block is gone
    assert m.truncate("b", 0) == [0]
    m.check_structure()


@pytest.mark.parametrize("seed", range(6))
def test_compact_packs_the_pool(seed):
    """Sequences that share, forks, windows and cached prefixes: afterwards the blocks in use are
    the first ones, every token is where its table says, and the moves are a parallel copy."""
    rng = random.Random(seed)
    order = list(range(60))
    rng.shuffle(order)
    m = BlockManager(BlockAllocator(60, 4, order))
    pc = PrefixCache(m)
    for i in range(8):
        pc.add_prompt(i, [7] * 8 + [rng.randint(0, 3) for _ in range(rng.randint(1, 12))])
    m.fork_copy(2, "fork")
    m.release_outside_window(5, 3)
    for i in (0, 3, 6):
        m.free_sequence(i)
    # what each block holds: the physical pool as a list
    pool = [object() for _ in range(60)]
    view = {k: [None if b < 0 else pool[b] for b in s.blocks] for k, s in m.seqs.items()}
    held = {h: pool[b] for h, b in pc.by_hash.items()}
    used = sum(c > 0 for c in m.alloc.refcount)
    with pytest.raises(ValueError):
        m.compact()   # the prefix cache's blocks would be lost
    moves = m.compact([pc])
    validate_cow_pairs(moves, 60)
    old = list(pool)
    for src, dst in moves:
        pool[dst] = old[src]
    assert all(b < used for s in m.seqs.values() for b in s.blocks)
    assert all(c > 0 for c in m.alloc.refcount[:used]) and not any(m.alloc.refcount[used:])
    assert view == {k: [None if b < 0 else pool[b] for b in s.blocks] for k, s in m.seqs.items()}
    assert held == {h: pool[b] for h, b in pc.by_hash.items()}
    m.check_structure(pc.held())
    assert m.compact([pc]) == [] and m.alloc.allocate() == used


# ---- a run of them together ----------------------------------------------------------------


@gpu
def test_a_servers_steps_over_a_four_bit_cache():
    """Two layers: a prompt with image tokens written through the rotation with three axes, a
    fork, a drafted tree verified, its accepted path kept, the pool packed, and the next token
    decoded: the decode equals that over a cache that was filled in order with the same tokens."""
    hk, group, d, bs, nb, L0 = 2, 4, 128, 8, 40, 37
    g = torch.Generator().manual_seed(11)
    rot = binding.rotary(d, 500000.0, axes=binding.rotary_axes((24, 20, 20), cyclic=True))
    scale = d ** -0.5

    def layer(n):
        b = torch.zeros(n, hk, bs, d // 2, dtype=torch.uint8, device="cuda")
        s = torch.zeros(n, hk, bs, d // 16, device="cuda").to(torch.float8_e4m3fn)
        return [b, b.clone(), s, s.view(torch.uint8).clone().view(torch.float8_e4m3fn)]
    layers = [layer(nb), layer(nb)]
    caches = binding.cache_list([c for x in layers for c in x])
    order = list(range(nb))
    random.Random(3).shuffle(order)
    m = BlockManager(BlockAllocator(nb, bs, order))
    text = torch.randn(2, 80, 3, hk * group, d, generator=g).to(torch.bfloat16).cuda()   # [layer, token, q/k/v, head]
    grid = torch.stack([torch.arange(80), torch.arange(80) // 6, torch.arange(80) % 6])
    grid[:, 30:] = torch.arange(30, 80)
    grid = grid.cuda()

    def write(into, li, toks, pos, slots):
        x = text[li, toks]
        q, k, v = x[:, 0].contiguous(), x[:, 1, :hk].contiguous(), x[:, 2, :hk].contiguous()
        binding.rotary_and_cache(q, q, k, v, grid[:, pos].contiguous(), into[0], into[1], torch.tensor(slots).cuda(), rot,
                                 k_token_scales=into[2], v_token_scales=into[3])
        return q

    m.add_sequence("old", 30)     # holes to pack away later
    slots = m.add_sequence("a", L0)
    for li in range(2):
        write(layers[li], li, list(range(L0)), list(range(L0)), slots)
    pair = m.fork_copy("a", "b")
    binding.copy_cache_blocks(caches, torch.tensor([pair]).cuda())
    m.free_sequence("a")
    m.free_sequence("old")
    # nine drafted nodes of "b": a tree whose path 0, 2, 5, 8 is accepted
    parents = [-1, 0, 0, 1, 2, 2, 3, 4, 5]
    depth, masks = [], []
    for i, p in enumerate(parents):
        depth.append(0 if p < 0 else depth[p] + 1)
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
    toks = [40 + i for i in range(9)]
    slots = []
    for _ in toks:
        slot, cow = m.append_token("b")
        assert cow is None
        slots.append(slot)
    path = [0, 2, 5, 8]

    def table():
        row = m.block_table_rows(["b"], 10)
        return torch.tensor(row, dtype=torch.int32).cuda()
    lens = torch.tensor([L0 + 9], dtype=torch.int32).cuda()
    outs = []
    for li in range(2):
        q = write(layers[li], li, toks, [L0 + x for x in depth], slots)
        out = torch.empty_like(q)
        binding.paged_attention_tree(out, q, layers[li][0], layers[li][1], table(), lens,
                                     torch.tensor([0, 9], dtype=torch.int32).cuda(),
                                     torch.tensor(masks, dtype=torch.int64)[:, None].cuda(), hk, scale, bs, 10,
                                     k_token_scales=layers[li][2], v_token_scales=layers[li][3])
        outs.append(out)
    new = torch.zeros(1, dtype=torch.int32).cuda()
    binding.keep_tokens(caches, table(), lens, torch.tensor([0, 9], dtype=torch.int32).cuda(),
                        torch.tensor(path + [-1] * 5, dtype=torch.int32).cuda(), torch.tensor([4], dtype=torch.int32).cuda(),
                        bs, 10, new_lens=new)
    assert new.tolist() == [L0 + 4]
    m.truncate("b", L0 + 4)
    moves = m.compact()
    assert moves
    binding.copy_cache_blocks(caches, torch.tensor(moves).cuda())
    m.check_structure()
    slot, cow = m.append_token("b")
    assert cow is None
    # the same tokens, written in order into fresh caches
    seq = list(range(L0)) + [toks[i] for i in path] + [60]
    for li in range(2):
        q = write(layers[li], li, [60], [L0 + 4], [slot])
        out, ref = torch.empty_like(q), torch.empty_like(q)
        lens2 = torch.tensor([L0 + 5], dtype=torch.int32).cuda()
        binding.paged_attention_decode_quantized(out, q, *layers[li][:2], *layers[li][2:], table(), lens2, hk, scale, bs, 10)
        plain = layer(10)
        allq = write(plain, li, seq, list(range(L0 + 5)), list(range(L0 + 5)))
        assert torch.equal(allq[-1:], q)
        t2 = torch.arange(10, dtype=torch.int32)[None].cuda()
        binding.paged_attention_decode_quantized(ref, q, *plain[:2], *plain[2:], t2, lens2, hk, scale, bs, 10)
        assert torch.equal(out, ref)
        # and the tree's accepted rows are the decodes of their prefixes, up to the two kernels'
        # roundings: weights to f16 (2^-11 each), the output to bf16 (2^-8)
        for j, node in enumerate(path):
            one = torch.empty_like(q)
            binding.paged_attention_decode_quantized(one, allq[L0 + j:L0 + j + 1], *plain[:2], *plain[2:], t2,
                                                     torch.tensor([L0 + j + 1], dtype=torch.int32).cuda(), hk, scale, bs, 10)
            vmax = float(text[li, :, 2].abs().max()) * 1.2   # (an element's error is at most a fifth)
            assert float((one[0].float() - outs[li][node].float()).abs().max()) <= (2 * 2.0 ** -11 + 2 * 2.0 ** -8) * vmax
    assert binding.read_device_errors() == 0
