"""Attention of drafted token trees and decode over a token-scaled cache, against the
definition in 64 bits (torch, CPU): head layouts, cache types, lengths and trees around
tile and block edges, rows that attend to nothing, poison in hidden and unused places,
strides, refusals, capture.

Tolerance of an output element, from the arithmetic: the rounding of the result (half a
step of its type), the rounding of the softmax weights to 16 bits (half a step relative to
sum_j p_j |V_j|; bf16 for a bf16 cache, f16 for an int8 one, none where they stay in binary32),
and what binary32 sums leave: a score is off by at most (D + 8) 2^-24 of sum_d |q_d k_d| scale
(products and their sum, the scaling, the exponent's 2^-22 relative), a weight by that times
itself twice (numerator and denominator), and a sum over L positions by L 2^-24 at most; all
of them times sum_j p_j |V_j|.

With an int8 cache a weight times its value scale is an f16 number relative to the row's
largest weight so far and to a power of two at most twice the largest value scale: below
2^-14 of them it is subnormal and rounded by up to 2^-25 of them, whatever its own size.  The
row's weights sum to at least 1 in those units, so L positions are off by at most
L 2^-25 * 2 max scale * 127 = L 2^-24 max |V| together."""
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


# ---- inputs and the definition -------------------------------------------------------------


def quantise(x):
    """Codes and scales of float32 rows, in IEEE binary32 (CPU)."""
    top = x.abs().amax(-1)
    s = top / torch.full_like(top, 127.0)
    s = torch.where(s >= 2.0 ** -126, s, torch.zeros_like(s))
    q = torch.round(x / torch.where(s > 0, s, torch.ones_like(s))[..., None]).clamp(-127, 127)
    return (q * (s > 0)[..., None]).to(torch.int8), s


def chain_masks(n, words):
    return [[((1 << (i + 1)) - 1) >> (64 * w) & (2 ** 64 - 1) for w in range(words)] for i in range(n)]


def random_tree(n, words, g):
    full = []
    for i in range(n):
        parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
        full.append((full[parent] if parent >= 0 else 0) | (1 << i))
    return [[m >> (64 * w) & (2 ** 64 - 1) for w in range(words)] for m in full]


def random_bits(n, words, g):
    return [[int(torch.randint(-2 ** 63, 2 ** 63 - 1, (1,), generator=g)) & (2 ** 64 - 1) for _ in range(words)]
            for _ in range(n)]


def signed(m):
    return m - 2 ** 64 if m >= 2 ** 63 else m


class Case:
    def __init__(self, seed, lens, nodes, hk, group, d, bs, cache="bf16", qdtype=torch.bfloat16, masks="tree", words=1,
                 poison=True, q_scale=1.5, decode=False, window=0, spread=0.5):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.nodes, self.hk, self.group, self.d, self.bs = lens, nodes, hk, group, d, bs
        self.cache, self.decode, self.window, self.words = cache, decode, window, words
        S = len(lens)
        counts = [-(-n // bs) for n in lens]
        self.mb = max(counts + [1]) + 1
        nb = sum(counts) + 3
        perm = torch.randperm(nb, generator=g)
        self.tables = torch.full((S, self.mb), -1, dtype=torch.int32)   # entries past the context: never read
        at = 0
        used = torch.zeros(nb, bs, dtype=torch.bool)
        for s, c in enumerate(counts):
            self.tables[s, :c] = perm[at:at + c].int()
            for j in range(lens[s]):
                used[int(perm[at + j // bs]), j % bs] = True
            at += c
        self.used = used
        k = torch.randn(nb, hk, bs, d, generator=g)
        v = torch.randn(nb, hk, bs, d, generator=g) * torch.exp(spread * torch.randn(nb, hk, bs, 1, generator=g))
        self.k_scales = self.v_scales = None
        self.k_scale = self.v_scale = 1.0
        hole = ~used[:, None, :].expand(nb, hk, bs)
        if cache == "int8":
            self.kc, self.k_scales = quantise(k)
            self.vc, self.v_scales = quantise(v)
            if poison:
                self.k_scales = self.k_scales.masked_fill(hole, math.nan)
                self.v_scales = self.v_scales.masked_fill(hole, math.nan)
            self.K64, self.V64 = (self.kc.double() * self.k_scales.double()[..., None],
                                  self.vc.double() * self.v_scales.double()[..., None])
        elif cache == "e4m3":
            self.k_scale, self.v_scale = 0.01, 0.02
            self.kc, self.vc = (k / 0.01).to(torch.float8_e4m3fn), (v / 0.02).to(torch.float8_e4m3fn)
            self.K64, self.V64 = self.kc.double() * 0.01, self.vc.double() * 0.02
            self.K64, self.V64 = self.kc.float().double() * float(torch.tensor(0.01)), \
                self.vc.float().double() * float(torch.tensor(0.02))
        else:
            dt = torch.bfloat16 if cache == "bf16" else torch.float32
            self.kc, self.vc = k.to(dt), v.to(dt)
            if poison:
                self.kc = self.kc.masked_fill(hole[..., None], math.nan)
                self.vc = self.vc.masked_fill(hole[..., None], math.nan)
            self.K64, self.V64 = self.kc.double(), self.vc.double()
        if decode:
            self.nodes = nodes = [1] * S
        T = sum(nodes)
        self.T = T
        self.q = (torch.randn(T, hk * group, d, generator=g) * q_scale).to(qdtype)
        self.scale = d ** -0.5
        self.starts = torch.tensor([0] + nodes).cumsum(0).int()
        rows = []
        for n in nodes:
            rows += {"tree": random_tree, "bits": random_bits}[masks](n, words, g) if masks in ("tree", "bits") else \
                chain_masks(n, words) if masks == "chain" else [[0] * words] * n
        self.rows = rows
        self.mask = torch.tensor([[signed(w) for w in r] for r in rows], dtype=torch.int64).reshape(T, words)

    def keep(self, s):
        """[n, L] whether node i attends to position j."""
        L, n = self.lens[s], self.nodes[s]
        keep = torch.ones(n, L, dtype=torch.bool)
        if self.decode:
            if self.window:
                keep[:, :max(0, L - self.window)] = False
            return keep
        a = int(self.starts[s])
        for i in range(n):
            for c in range(n):
                keep[i, L - n + c] = bool(self.rows[a + i][c // 64] >> (c % 64) & 1)
        return keep

    def reference(self):
        """(outputs, sum_j p_j |V_j|, score error bound per unit roundoff), 64 bits."""
        out = torch.zeros(self.T, self.hk * self.group, self.d, dtype=torch.float64)
        self.floor = torch.zeros(self.T, self.hk * self.group, 1, dtype=torch.float64)
        wabs, dz = torch.zeros_like(out), torch.zeros(self.T, self.hk * self.group, 1, dtype=torch.float64)
        for s, L in enumerate(self.lens):
            n, a = self.nodes[s], int(self.starts[s])
            if n == 0 or L == 0:
                continue
            j = torch.arange(L)
            blk = self.tables[s].long()[j // self.bs]
            K, V = self.K64[blk, :, j % self.bs], self.V64[blk, :, j % self.bs]    # [L, hk, d]
            q = self.q[a:a + n].double().view(n, self.hk, self.group, self.d)
            keep = self.keep(s)[:, None, None]
            z = torch.einsum("nhgd,lhd->nhgl", q, K) * self.scale
            z = z.masked_fill(~keep, -math.inf)
            top = z.amax(-1, keepdim=True)
            p = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
            p = torch.where(keep, p, torch.zeros_like(p))
            den = p.sum(-1, keepdim=True)
            p = p / torch.where(den > 0, den, torch.ones_like(den))
            # a position that no weight falls on has no part, whatever it holds
            def pv(V):
                bad = ~torch.isfinite(V)
                o = torch.einsum("nhgl,lhd->nhgd", p, V.masked_fill(bad, 0.0))
                for l, h, c in bad.nonzero().tolist():
                    o[:, h, :, c] += torch.where(keep[:, 0, :, l], p[:, h, :, l] * V[l, h, c], 0.0)
                return o
            out[a:a + n] = pv(V).reshape(n, -1, self.d)
            if self.cache == "int8" and self.q.dtype == torch.bfloat16:
                top = torch.where(torch.isfinite(V), V.abs(), 0.0).amax((0, 2))              # [hk]
                self.floor[a:a + n] = (L * 2.0 ** -24 * top).repeat_interleave(self.group)[None, :, None]
            wabs[a:a + n] = pv(V.abs()).reshape(n, -1, self.d)
            za = torch.einsum("nhgd,lhd->nhgl", q.abs(), K.abs()).masked_fill(~keep, 0.0).amax(-1) * self.scale
            dz[a:a + n] = za.reshape(n, -1, 1)
        return out, wabs, dz

    def bound(self, ref, wabs, dz):
        u = 2.0 ** -24
        p16 = 0.0 if self.q.dtype == torch.float32 or self.cache in ("f32", "e4m3") else \
            2.0 ** -11 if self.cache == "int8" else 2.0 ** -8
        L = max(self.lens + [1])
        rel = p16 + 2 * ((self.d + 8) * u * dz + 2.0 ** -22) + L * u
        step = torch.finfo(self.q.dtype).eps / 2
        fp = rel * wabs + self.floor
        return step * (ref.abs() + fp) + fp + 1e-30

    def device(self):
        def mv(t):
            return None if t is None else t.cuda()
        out = torch.full_like(self.q, 7.0).cuda()
        return dict(out=out, q=mv(self.q), kc=mv(self.kc), vc=mv(self.vc), ks=mv(self.k_scales), vs=mv(self.v_scales),
                    tables=mv(self.tables), lens=torch.tensor(self.lens, dtype=torch.int32).cuda(), starts=mv(self.starts),
                    mask=mv(self.mask))

    def call(self, x, stream=None):
        if self.decode:
            return binding.paged_attention_decode_quantized(
                x["out"], x["q"], x["kc"], x["vc"], x["ks"], x["vs"], x["tables"], x["lens"], self.hk, self.scale,
                self.bs, self.mb, sliding_window=self.window, stream=stream)
        return binding.paged_attention_tree(
            x["out"], x["q"], x["kc"], x["vc"], x["tables"], x["lens"], x["starts"], x["mask"], self.hk, self.scale,
            self.bs, self.mb, k_scale=self.k_scale, v_scale=self.v_scale, k_token_scales=x["ks"],
            v_token_scales=x["vs"], stream=stream)

    def check(self, out=None):
        if out is None:
            out = self.call(self.device())
            torch.cuda.synchronize()
            assert binding.read_device_errors() == 0
        ref, wabs, dz = self.reference()
        got = out.double().cpu()
        fine = torch.isfinite(ref)
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)])
        over = ((got - ref).abs() - self.bound(ref, wabs, dz))[fine]
        assert over.numel() == 0 or float(over.max()) <= 0, f"over the bound by {float(over.max())}"


# ---- values --------------------------------------------------------------------------------

LAYOUTS = [(8, 4, 128), (2, 1, 128), (1, 8, 64), (2, 3, 128), (1, 5, 64), (4, 2, 64), (1, 16, 128), (1, 7, 128),
           (1, 71, 128)]


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("hk,group,d", LAYOUTS)
def test_tree_head_layouts(hk, group, d, cache):
    Case(hk * 100 + group, [40, 300, 1, 129, 17], [7, 12, 1, 4, 17], hk, group, d, 16, cache=cache).check()


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8", "f32", "e4m3"])
@pytest.mark.parametrize("bs", [2, 4, 8, 16, 32])
def test_tree_block_sizes_and_cache_types(bs, cache):
    Case(bs, [33, 130, 5, 64], [5, 9, 5, 3], 2, 4, 128, bs, cache=cache,
         qdtype=torch.float32 if cache == "f32" else torch.bfloat16).check()


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_f32_queries(d, cache):
    Case(d, [70, 9], [6, 9], 2, 2, d, 16, cache=cache, qdtype=torch.float32).check()


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("L,n", [(1, 1), (2, 2), (63, 63), (64, 1), (65, 64), (127, 3), (128, 128), (129, 1), (129, 129),
                                 (200, 130), (256, 64), (257, 33), (511, 65), (1000, 256)])
def test_tree_lengths_around_tiles(L, n, cache):
    """One sequence at lengths around the key tiles, trees of one to several mask words (rows
    past one and two tiles of 128), a second short one behind it."""
    Case(L * 1000 + n, [L, 20], [n, 3], 2, 4, 128, 16, cache=cache, words=-(-n // 64) + (L % 2)).check()


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("masks", ["chain", "bits", "none"])
def test_tree_masks(masks, cache):
    """Chains (causal), arbitrary bits (nodes that see later nodes, not themselves), none."""
    Case(5, [50, 8, 150, 64], [8, 8, 20, 64], 2, 4, 128, 16, cache=cache, masks=masks).check()


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8", "f32"])
def test_rows_that_attend_to_nothing_are_zero(cache):
    c = Case(6, [6, 12], [6, 12], 2, 4, 128, 16, cache=cache, masks="none",
             qdtype=torch.float32 if cache == "f32" else torch.bfloat16)
    out = c.call(c.device())
    assert torch.equal(out, torch.zeros_like(out))


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_tree_many_sequences_and_empty_ones(cache):
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(1, 90, (300,), generator=g).tolist()
    nodes = [min(L, int(n)) for L, n in zip(lens, torch.randint(0, 9, (300,), generator=g).tolist())]
    lens[7], nodes[7] = 0, 0
    Case(10, lens, nodes, 2, 4, 64, 16, cache=cache).check()


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_tree_long_contexts_split_over_the_gpu(cache):
    Case(11, [9000, 513, 4097], [64, 3, 20], 2, 4, 128, 32, cache=cache).check()


@gpu
@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("n,L", [(5, 40), (64, 300), (70, 70)])
def test_poison_in_hidden_nodes_stays_there(n, L, cache):
    """Infinities and NaN in K and V of some nodes: rows that do not attend to them are
    untouched, rows that do show them."""
    c = Case(12, [L], [n], 1, 4, 128, 16, cache=cache, words=-(-n // 64),
             qdtype=torch.float32 if cache == "f32" else torch.bfloat16)
    for node, col, val, what in ((1, 5, math.nan, "v"), (2, 0, math.inf, "v"), (3, 127, -math.inf, "v"),
                                 (n - 1, 64, math.inf, "v"), (4, 9, math.nan, "k")):
        j = L - n + node
        at = (int(c.tables[0, j // 16]), 0, j % 16, col)
        (c.vc if what == "v" else c.kc)[at] = val
    c.K64, c.V64 = c.kc.double(), c.vc.double()
    c.check()
    keep = c.keep(0)
    assert not keep[:, L - n + 1].all() and keep[:, L - n + 1].any()


@gpu
@pytest.mark.parametrize("what", ["k", "v"])
def test_nan_scale_of_a_hidden_node_stays_there(what):
    c = Case(13, [60], [9], 2, 4, 128, 16, cache="int8")
    j = 60 - 9 + 2
    (c.k_scales if what == "k" else c.v_scales)[int(c.tables[0, j // 16]), :, j % 16] = math.nan
    c.K64, c.V64 = (c.kc.double() * c.k_scales.double()[..., None], c.vc.double() * c.v_scales.double()[..., None])
    c.check()


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_scores_far_apart(cache):
    """Scores of hundreds: the running maximum moves from tile to tile, and most weights vanish."""
    Case(14, [700, 300], [10, 3], 2, 4, 128, 16, cache=cache, q_scale=60.0).check()


@gpu
def test_token_magnitudes_far_apart():
    """Value scales over many powers of two in one row's sum."""
    Case(15, [400, 90], [10, 3], 2, 4, 128, 16, cache="int8", spread=4.0).check()


@gpu
@pytest.mark.parametrize("hk,group,d", LAYOUTS)
def test_decode_quantized_head_layouts(hk, group, d):
    Case(hk + group, [1, 2, 15, 16, 17, 127, 128, 129, 400, 0, 1025], None, hk, group, d, 16, cache="int8",
         decode=True).check()


@gpu
@pytest.mark.parametrize("bs", [2, 8, 32])
@pytest.mark.parametrize("window", [0, 1, 100, 128, 1000])
def test_decode_quantized_windows(window, bs):
    c = Case(20 + window, [1, 99, 100, 101, 600, 2000], None, 2, 4, 128, bs, cache="int8", decode=True, window=window)
    if window:   # blocks that have left the window may be gone
        for s, L in enumerate(c.lens):
            c_first = max(0, L - window) // bs
            c.tables_real = c.tables.clone() if s == 0 else c.tables_real
            c.tables[s, :c_first] = -1
        x = c.device()
        c.tables = c.tables_real
        out = c.call(x)
        torch.cuda.synchronize()
        assert binding.read_device_errors() == 0
        c.check(out)
    else:
        c.check()


@gpu
def test_decode_quantized_many_and_long():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(1, 700, (200,), generator=g).tolist() + [8000]
    Case(21, lens, None, 2, 4, 64, 16, cache="int8", decode=True).check()


# ---- strides, streams, batches -------------------------------------------------------------


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_strided_views_and_a_side_stream(cache):
    """K and V as views of one tensor with the heads outermost, queries and outputs as
    slices of wider rows, tables and masks with a row stride, on a stream of its own."""
    c = Case(30, [90, 200], [7, 20], 2, 4, 128, 16, cache=cache)
    x = c.device()
    both = torch.stack([x["kc"].transpose(0, 1), x["vc"].transpose(0, 1)])     # [2, hk, nb, bs, d]
    x["kc"], x["vc"] = both[0].transpose(0, 1), both[1].transpose(0, 1)
    if cache == "int8":
        sc = torch.stack([x["ks"].transpose(0, 1), x["vs"].transpose(0, 1)])
        x["ks"], x["vs"] = sc[0].transpose(0, 1), sc[1].transpose(0, 1)
    wide_q = torch.zeros(c.T, 10, 136, dtype=torch.bfloat16, device="cuda")
    wide_q[:, 1:9, :128] = x["q"]
    x["q"] = wide_q[:, 1:9, :128]
    wide_o = torch.full((c.T, 9, 144), 7.0, dtype=torch.bfloat16, device="cuda")
    x["out"] = wide_o[:, :8, 8:136]
    wide_t = torch.full((2, c.mb + 5), -1, dtype=torch.int32, device="cuda")
    wide_t[:, :c.mb] = x["tables"]
    x["tables"] = wide_t[:, :c.mb]
    wide_m = torch.zeros(c.T, 3, dtype=torch.int64, device="cuda")
    wide_m[:, :1] = x["mask"]
    x["mask"] = wide_m[:, :1]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c.call(x, stream=st)
    torch.cuda.synchronize()
    assert binding.read_device_errors() == 0
    c.check(x["out"])
    assert (wide_o[:, 8] == 7).all() and (wide_o[:, :, :8] == 7).all() and (wide_o[:, :, 136:] == 7).all()


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_unaligned_query_rows(cache):
    """Query and output rows off a 16-byte boundary."""
    c = Case(31, [90, 20], [7, 2], 2, 2, 128, 16, cache=cache)
    x = c.device()
    odd = torch.zeros(c.T * 4 * 128 + 3, dtype=torch.bfloat16, device="cuda")
    odd[3:] = x["q"].reshape(-1)
    x["q"] = odd[3:].view(c.T, 4, 128)
    o = torch.zeros(c.T * 4 * 128 + 1, dtype=torch.bfloat16, device="cuda")
    x["out"] = o[1:].view(c.T, 4, 128)
    c.check(c.call(x))


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_rows_behind_the_batch_and_bad_sequences_stay(cache):
    """A padded batch: rows behind the last sequence's keep what they held; so do those of a
    sequence whose length does not fit, which sets the error bit."""
    c = Case(32, [60, 40, 70], [5, 4, 6], 2, 4, 128, 16, cache=cache)
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
    for bad in (-1, 3, c.mb * 16 + 1):      # negative, shorter than its nodes, past the table
        x["lens"][1] = bad
        x["out"].fill_(7.0)
        c.call(x)
        assert binding.read_device_errors() == binding.DEVERR["context_len"]
        assert (x["out"][5:9] == 7).all() and (x["out"][c.T:] == 7).all()
        x["lens"][1] = 40
        got = x["out"][:c.T].clone()
        got[5:9] = c.call(x)[5:9]
        c.check(got)


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_bad_table_entries_are_reported(cache):
    c = Case(33, [60, 40], [5, 4], 2, 4, 128, 16, cache=cache)
    x = c.device()
    x["tables"][0, 1] = c.kc.shape[0]
    c.call(x)
    assert binding.read_device_errors() == binding.DEVERR["table_entry"]


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_same_bits_every_time_and_from_a_graph(cache):
    """A long and a short call; captured together, replayed on new inputs, they give the
    eager calls' bits, as do repeated eager calls."""
    a = Case(34, [5000, 300], [30, 5], 2, 4, 128, 16, cache=cache)
    b = Case(35, [800], [64], 2, 4, 128, 16, cache=cache)
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


# ---- refusals ------------------------------------------------------------------------------


def _args(**over):
    a = dict(out=torch.empty(9, 8, 128, dtype=torch.bfloat16), query=torch.zeros(9, 8, 128, dtype=torch.bfloat16),
             key_cache=torch.zeros(20, 2, 16, 128, dtype=torch.bfloat16),
             value_cache=torch.zeros(20, 2, 16, 128, dtype=torch.bfloat16),
             block_tables=torch.zeros(3, 4, dtype=torch.int32), context_lens=torch.ones(3, dtype=torch.int32),
             query_start_loc=torch.zeros(4, dtype=torch.int32), tree_mask=torch.zeros(9, 1, dtype=torch.int64),
             num_kv_heads=2, scale=0.1, block_size=16, max_blocks_per_seq=4)
    a.update(over)
    return a


def _status(fn, **kw):
    try:
        fn(**kw)
        return 0
    except binding.PkvError as e:
        assert e.message
        return e.status


def _i8(n=1):
    c = torch.zeros(20, 2, 16, 128, dtype=torch.int8)
    s = torch.ones(20, 2, 16)
    return dict(key_cache=c, value_cache=c.clone(), k_token_scales=s, v_token_scales=s.clone())


def test_tree_refusals(dry):
    f = binding.paged_attention_tree
    assert _status(f, **_args()) == 0
    assert _status(f, **_args(**_i8())) == 0
    for over, want in [
        (dict(out=torch.empty(9, 8, 128)), 1),
        (dict(query=torch.zeros(9, 8, 128, dtype=torch.int32)), 2),
        (dict(query=torch.zeros(9, 8, 64, dtype=torch.bfloat16), out=torch.empty(9, 8, 64, dtype=torch.bfloat16)), 1),
        (dict(tree_mask=torch.zeros(8, 1, dtype=torch.int64)), 1),
        (dict(tree_mask=torch.zeros(9, 17, dtype=torch.int64)), 1),
        (dict(tree_mask=torch.zeros(9, 0, dtype=torch.int64)), 1),
        (dict(tree_mask=torch.zeros(9, 1, dtype=torch.int32)), 2),
        (dict(query_start_loc=torch.zeros(3, dtype=torch.int32)), 1),
        (dict(query_start_loc=torch.zeros(4, dtype=torch.int64)), 2),
        (dict(context_lens=torch.ones(2, dtype=torch.int32)), 1),
        (dict(context_lens=torch.ones(6, dtype=torch.int32)[::2]), 1),
        (dict(num_kv_heads=3), 1),
        (dict(block_size=8), 1),
        (dict(max_blocks_per_seq=5), 1),
        (dict(scale=math.inf), 1),
        (dict(key_cache=torch.zeros(20, 2, 16, 128, dtype=torch.int8),
              value_cache=torch.zeros(20, 2, 16, 128, dtype=torch.int8)), 1),                 # no scales
        (dict(k_token_scales=torch.ones(20, 2, 16), v_token_scales=torch.ones(20, 2, 16)), 1),  # not an i8 cache
        ({**_i8(), "v_token_scales": torch.ones(20, 2, 8)}, 1),
        ({**_i8(), "v_token_scales": torch.ones(20, 2, 16, dtype=torch.int32)}, 2),
        ({**_i8(), "v_token_scales": torch.ones(2, 20, 16).transpose(0, 1)}, 1),              # strides differ
    ]:
        assert _status(f, **_args(**over)) == want, over.keys()


def test_decode_quantized_refusals(dry):
    f = binding.paged_attention_decode_quantized
    def args(**over):
        a = _args(**_i8())
        for k in ("query_start_loc", "tree_mask"):
            a.pop(k)
        a.update(query=torch.zeros(3, 8, 128, dtype=torch.bfloat16), out=torch.empty(3, 8, 128, dtype=torch.bfloat16))
        a.update(over)
        return a
    assert _status(f, **args()) == 0
    assert _status(f, **args(sliding_window=-1)) == 1
    assert _status(f, **args(query=torch.zeros(4, 8, 128, dtype=torch.bfloat16),
                             out=torch.empty(4, 8, 128, dtype=torch.bfloat16))) == 1
    bf = torch.zeros(20, 2, 16, 128, dtype=torch.bfloat16)
    assert _status(f, **args(key_cache=bf, value_cache=bf)) == 1
    # the other calls do not take an i8 cache
    a = args()
    for k in ("k_token_scales", "v_token_scales"):
        a.pop(k)
    assert _status(binding.paged_attention_decode, **a) == 2


def test_tree_workspace_bytes():
    f = binding.tree_workspace_bytes
    assert f(0, 1, 8, 2, 128) == 0 and f(1, 0, 8, 2, 128) == 0 and f(1, 1, 7, 2, 128) == 0
    assert f(4, 64, 8, 2, 128) >= f(4, 4, 8, 2, 128) >= 0


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_batch_of_several_tiles_an_item(cache):
    """More items than SMs, each of several key tiles, one and two row tiles mixed; then the
    same batch of single-tile contexts."""
    g = torch.Generator().manual_seed(40)
    lens = torch.randint(200, 900, (44,), generator=g).tolist()
    nodes = torch.randint(1, 40, (44,), generator=g).tolist()
    Case(41, lens, nodes, 4, 4, 64, 16, cache=cache).check()
    lens = torch.randint(40, 128, (130,), generator=g).tolist()
    nodes = torch.randint(1, 9, (130,), generator=g).tolist()
    Case(42, lens, nodes, 4, 4, 64, 16, cache=cache).check()


@gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
def test_ragged_batch_from_cold_memory(cache):
    """Many items to a block whose tiles come late: with nothing of the cache in L2 a product
    may wait for its V tile long after its weights are there, and the item's output must wait
    for the last one.  Against 64 bits, and the same bits in every run."""
    g = torch.Generator().manual_seed(43)
    lens = torch.randint(160, 2049, (64,), generator=g).tolist()
    nodes = torch.randint(5, 25, (64,), generator=g).tolist()
    case = Case(44, lens, nodes, 8, 4, 128, 16, cache=cache)
    x = case.device()
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    outs = []
    for i in range(8):
        flush.fill_(i)
        outs.append(case.call(x).clone())
    torch.cuda.synchronize()
    assert binding.read_device_errors() == 0
    case.check(outs[0])
    assert all(torch.equal(o, outs[0]) for o in outs)


@gpu
@pytest.mark.parametrize("hk,group,d", [(2, 4, 128), (1, 12, 64), (1, 16, 128), (1, 40, 128)])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_decode_quantized_output_rows_of_any_alignment(hk, group, d, shift):
    """Output rows off 16 and 8 bytes, in a wider tensor whose other columns stay."""
    c = Case(45, [3, 700, 130, 1], None, hk, group, d, 16, cache="int8", decode=True)
    x = c.device()
    wide = torch.full((c.T, hk * group, d + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    x["out"] = wide[:, :, shift:shift + d]
    c.call(x)
    torch.cuda.synchronize()
    c.check(x["out"])
    assert (wide[:, :, :shift] == 7).all() and (wide[:, :, shift + d:] == 7).all()


@gpu
@pytest.mark.parametrize("hk,group", [(8, 4), (1, 16), (1, 30)])
def test_decode_quantized_from_a_graph(hk, group):
    """Captured once, replayed as the contexts grow and change: each time the eager call's
    bits; scales of 0 and of a type's largest and smallest numbers among them."""
    lens = [900, 33, 0, 4000, 128, 1]
    c = Case(46, lens, None, hk, group, 128, 16, cache="int8", decode=True)
    c.k_scales[0, :, 3] = 0.0
    c.v_scales[1, :, 2] = 3e38
    c.v_scales[2, :, 2] = 1e-38
    x = c.device()
    eager = c.call(x).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(x)
    for k in range(4):
        x["lens"][0] = 900 - 37 * k
        x["lens"][3] = 4000 - 1001 * k
        x["q"].mul_(0.75)
        x["out"].fill_(7.0)
        g.replay()
        got = x["out"].clone()
        assert torch.equal(got.view(torch.int16), c.call(x).view(torch.int16))
        assert not torch.equal(got, eager)
    assert binding.read_device_errors() == 0


@gpu
def test_decode_quantized_scales_with_strides_of_their_own():
    """Scales as a slice of a wider tensor, off 16 bytes; blocks of two tokens."""
    for bs in (2, 16):
        c = Case(47, [250, 31], None, 2, 4, 64, bs, cache="int8", decode=True)
        x = c.device()
        nb = x["ks"].shape[0]
        wide = torch.zeros(2, nb, 3, bs + 3, device="cuda")
        wide[0, :, 1:, 1:bs + 1], wide[1, :, 1:, 1:bs + 1] = x["ks"], x["vs"]
        x["ks"], x["vs"] = wide[0, :, 1:, 1:bs + 1], wide[1, :, 1:, 1:bs + 1]
        c.check(c.call(x))
        assert binding.read_device_errors() == 0
