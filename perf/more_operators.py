"""Measured cases of the 4-bit cache, several position axes and pages of many caches.

Five operators that stand beside the cache writes and the paged attention:

  axes      rotary positions with several axes (time, height, width) for queries and keys,
            keys and values written to the paged cache (``binding.rotary_and_cache`` with a
            grid of positions);
  quantize  a token's K and V written as 4-bit floats (e2m1) with an e4m3 scale for every
            16 columns, and read back (``binding.quantize_and_cache``, ``binding.read_cache``);
  decode    single-token decode attention over that cache
            (``binding.paged_attention_decode_quantized``);
  tree      attention of drafted trees over it (``binding.paged_attention_tree``);
  pages     blocks copied in the caches of all layers in one call, and drafted tokens that were
            accepted moved together (``binding.copy_cache_blocks``, ``binding.keep_tokens``).

``run`` computes them in elementary torch operations, or, with ``own``, through the
package's entry points; ``exact`` computes them from their definition in 64 bits.
"""
import math

import torch

own = False

_TWO_PI = 2.0 * math.pi
_PHI = 0.6180339887498949
_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # of an e2m1 code without its sign


def listed():
    return [
        # the patches of one small image, float32 activations, pairs side by side, two axes
        {"name": "axes_image_f32", "op": "axes", "tokens": 49, "heads": 12, "kv_heads": 4, "dim": 64, "rotary": 48,
         "interleaved": True, "sections": "12,12", "cyclic": False, "dtype": "f32", "bs": 8},
        # a prefill step of video and text tokens, three axes in turn over the pairs
        {"name": "axes_video", "op": "axes", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "sections": "24,20,20", "cyclic": True, "dtype": "bf16", "bs": 16},
        # a decode batch's new tokens into the 4-bit cache, and back
        {"name": "quantize_decode_batch", "op": "quantize", "tokens": 64, "kv_heads": 8, "dim": 128, "scale": 1.0,
         "dtype": "bf16", "bs": 16},
        # a prefill step's tokens
        {"name": "quantize_prefill", "op": "quantize", "tokens": 16384, "kv_heads": 8, "dim": 128, "scale": 1.0,
         "dtype": "bf16", "bs": 16},
        # one sequence of odd length, the smallest decode call
        {"name": "decode_one_seq", "op": "decode", "seqs": 1, "lo": 777, "hi": 777, "heads": 32, "kv_heads": 8,
         "dim": 128, "bs": 16, "window": 0},
        # the benchmark's decode batch (64 sequences, contexts spread over 128..2048)
        {"name": "decode_batch", "op": "decode", "seqs": 64, "lo": 129, "hi": 2048, "heads": 32, "kv_heads": 8,
         "dim": 128, "bs": 16, "window": 0},
        # the benchmark's long contexts
        {"name": "decode_long", "op": "decode", "seqs": 8, "lo": 32768, "hi": 32768, "heads": 32, "kv_heads": 8,
         "dim": 128, "bs": 32, "window": 0},
        # one sequence, a small tree: the lowest-latency form of speculative decoding
        {"name": "tree_one_seq", "op": "tree", "seqs": 1, "lo": 341, "hi": 341, "nodes_lo": 9, "nodes_hi": 9,
         "heads": 32, "kv_heads": 8, "dim": 128, "bs": 16},
        # ragged trees of a batch over middling contexts
        {"name": "tree_batch", "op": "tree", "seqs": 32, "lo": 1000, "hi": 8192, "nodes_lo": 8, "nodes_hi": 32,
         "heads": 32, "kv_heads": 8, "dim": 128, "bs": 16},
        # a fork: each of three children gets its own copy of a partial block, in a few layers
        {"name": "pages_fork", "op": "copy", "layers": 4, "kv_heads": 8, "dim": 128, "bs": 16, "cache": "bf16",
         "blocks": 40, "pairs": 3},
        # a fragmented pool packed: blocks of every layer move to the front
        {"name": "pages_compact", "op": "copy", "layers": 16, "kv_heads": 8, "dim": 128, "bs": 16, "cache": "bf16",
         "blocks": 320, "pairs": 150},
        # the batch's accepted drafted tokens, in every layer of an int8 cache and its scales
        {"name": "pages_accept", "op": "keep", "layers": 12, "kv_heads": 8, "dim": 128, "bs": 16, "cache": "int8",
         "seqs": 48, "lo": 40, "hi": 160, "nodes_lo": 8, "nodes_hi": 24},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "quantize", "decode", "decode", "tree", "tree", "copy", "keep"])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 20])
    bs = rng.choice([8, 16, 32])
    if op == "axes":
        pairs = rng.randint(3, dim // 2) if rng.random() < 0.5 else dim // 2
        axes = rng.randint(2, 4) if pairs >= 4 else 2
        cuts = sorted(rng.sample(range(1, pairs), axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
        return {"op": op, "tokens": _log(rng, 1, 11000), "heads": kv * min(group, 4), "kv_heads": kv, "dim": dim,
                "rotary": 2 * pairs, "interleaved": rng.random() < 0.5, "sections": ",".join(map(str, sections)),
                "cyclic": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "f32"]), "bs": bs}
    if op == "quantize":
        return {"op": op, "tokens": _log(rng, 1, 16000), "kv_heads": kv, "dim": dim,
                "scale": rng.choice([1.0, 1.0, 0.0625, 0.37, 5.0]), "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "bs": bs}
    if op in ("copy", "keep"):
        layers, cache = _log(rng, 1, 12), rng.choice(["bf16", "f32", "int8"])
        size = {"bf16": 2, "f32": 4, "int8": 1}[cache] * 2 * layers * kv * bs * dim  # bytes of a block in all caches
        most = max(8, min(400, 300_000_000 // size))  # blocks that the pool may hold
        if op == "copy":
            blocks = _log(rng, 4, most)
            return {"op": op, "layers": layers, "kv_heads": kv, "dim": dim, "bs": bs, "cache": cache, "blocks": blocks,
                    "pairs": rng.randint(1, blocks // 2)}
        n_hi = rng.randint(2, 40)
        hi = n_hi + _log(rng, 1, 200)
        n_lo, seqs = max(2, n_hi // rng.choice([1, 2, 4])), max(1, min(_log(rng, 1, 64), most * bs // (hi + bs)))
        return {"op": op, "layers": layers, "kv_heads": kv, "dim": dim, "bs": bs, "cache": cache, "seqs": seqs,
                "lo": rng.randint(n_hi, hi), "hi": hi, "nodes_lo": n_lo, "nodes_hi": n_hi}
    # contexts and batch so that no draw reads more than the largest listed case
    hi = _log(rng, 1, 32768)
    lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
    if op == "decode":
        seqs = min(_log(rng, 1, 128), max(1, 200000 // hi))
        return {"op": op, "seqs": seqs, "lo": lo, "hi": hi, "heads": kv * group, "kv_heads": kv, "dim": dim, "bs": bs,
                "window": rng.choice([0, 0, 0, rng.randint(1, hi)])}
    seqs = min(_log(rng, 1, 64), max(1, 130000 // hi))
    n_hi = max(1, min(_log(rng, 1, 64), hi, 256 // group))
    return {"op": op, "seqs": seqs, "lo": max(lo, n_hi), "hi": hi, "nodes_lo": max(1, n_hi // rng.choice([1, 2, 4])),
            "nodes_hi": n_hi, "heads": kv * group, "kv_heads": kv, "dim": dim, "bs": bs}


# ---- inputs ----------------------------------------------------------------------------


def _lens(case):
    """The sequences' context lengths: spread over lo..hi, a function of the case alone."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    return [lo + int((((i + 1) * _PHI) % 1.0) * (hi - lo + 1)) for i in range(n)]


def _nodes(case):
    """The sequences' drafted tokens (the last of each context)."""
    n, lo, hi = case["seqs"], case["nodes_lo"], case["nodes_hi"]
    return [lo + int((((i + 3) * _PHI) % 1.0) * (hi - lo + 1)) for i in range(n)]


def _kept(case):
    """How many of them were accepted: 1 to half (a path through the tree is far shorter than it)."""
    return [1 + int((((i + 5) * _PHI) % 1.0) * (n // 2)) for i, n in enumerate(_nodes(case))]


def _sections(case):
    return [int(s) for s in case["sections"].split(",")]


def _pair_axes(case):
    """The axis of each rotated pair: runs of them, or in turn until each axis has its number."""
    left = _sections(case)
    if not case["cyclic"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


def _dtype(case):
    return torch.float32 if case.get("dtype", case.get("cache")) == "f32" else torch.bfloat16


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _outliers(x):
    """A few channels of a head an order of magnitude above the rest, as keys have them."""
    x = x.float()
    x[..., 3] *= 6.0
    x[..., x.shape[-1] // 2 + 1] *= 10.0
    return x


def _tables(case, lens, g):
    """Block tables over a permuted pool with spare blocks."""
    bs = case["bs"]
    counts = [-(-n // bs) for n in lens]
    used, width = sum(counts), max(counts)
    nb = used + used // 10 + 2
    perm = torch.randperm(nb, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    ends = torch.tensor(counts, device="cuda").cumsum(0)
    first = (ends - torch.tensor(counts, device="cuda"))[:, None]
    cols = torch.arange(width, device="cuda")[None, :]
    index = (first + cols).clamp(max=nb - 1)
    return perm[index].contiguous(), nb, width


def _tree_masks(nodes, seed):
    """Ancestor masks of random trees: node i hangs below an earlier node or starts a branch."""
    rng = torch.Generator().manual_seed(seed)
    masks = []
    for n in nodes:
        pick = torch.rand(n, generator=rng).tolist()
        row = []
        for i in range(n):
            parent = i - 1 - int(pick[i] * pick[i] * 6.0)
            row.append((row[parent] if 0 <= parent < i else 0) | (1 << i))
        masks += row
    masks = [m - (1 << 64) if m >= 1 << 63 else m for m in masks]
    return torch.tensor(masks, dtype=torch.int64, device="cuda")[:, None].contiguous()


def _grid_positions(case, g):
    """Positions [axes, tokens]: runs of text tokens (all axes alike) and of frames' patches."""
    t, axes = case["tokens"], len(_sections(case))
    token = torch.arange(t, device="cuda")
    side = int(torch.randint(5, 28, (1,), generator=g, device="cuda"))
    frame, patch = token // (side * side), token % (side * side)
    grid = [frame, patch // side, patch % side, frame // 2][:axes]
    start = int(torch.randint(0, 20000, (1,), generator=g, device="cuda"))
    text = (token // 97) % 5 == 0
    return torch.stack([torch.where(text, start + token, start + x) for x in grid]).contiguous()


def _caches(case, nb, g):
    """K and V of every layer, and for an int8 cache their scale arrays."""
    hk, bs, d = case["kv_heads"], case["bs"], case["dim"]
    out = []
    for _ in range(2 * case["layers"]):
        if case["cache"] == "int8":
            out.append(torch.randint(-127, 128, (nb, hk, bs, d), generator=g, device="cuda", dtype=torch.int8))
        else:
            out.append(_randn((nb, hk, bs, d), g, _dtype(case)))
    if case["cache"] == "int8":
        out += [torch.rand(nb, hk, bs, generator=g, device="cuda") * 0.05 for _ in range(2 * case["layers"])]
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, hk, bs, op = case["dim"], case["kv_heads"], case["bs"], case["op"]
    st = {"case": case}
    if op in ("axes", "quantize"):
        t, dt = case["tokens"], _dtype(case)
        nb = -(-t // bs) + 3
        size = case.get("scale", 1.0)  # the factor of the 4-bit cache follows its tensors' size
        st["key"] = (_outliers(_randn((t, hk, d), g)) * size).to(dt)
        st["value"] = (_randn((t, hk, d), g) * torch.exp(0.5 * _randn((t, hk, 1), g)) * size).to(dt)
        # runs of tokens in scattered blocks, as an engine's block tables give them
        perm = torch.randperm(nb, generator=g, device="cuda")
        token = torch.arange(t, device="cuda")
        st["slots"] = (perm[token // bs] * bs + token % bs).contiguous()
        if op == "quantize":
            st["key_cache"] = torch.zeros(nb, hk, bs, d // 2, dtype=torch.uint8, device="cuda")
            st["value_cache"] = torch.zeros_like(st["key_cache"])
            st["k_scales"] = torch.zeros(nb, hk, bs, d // 16, device="cuda").to(torch.float8_e4m3fn)
            st["v_scales"] = st["k_scales"].clone()
            st["key_back"] = torch.empty(t, hk, d, device="cuda")
            st["value_back"] = torch.empty_like(st["key_back"])
            return st
        st["query"] = _randn((t, case["heads"], d), g, dt)
        st["query_out"] = torch.empty_like(st["query"])
        st["positions"] = _grid_positions(case, g)
        st["key_cache"] = torch.zeros(nb, hk, bs, d, dtype=dt, device="cuda")
        st["value_cache"] = torch.zeros_like(st["key_cache"])
        axes = _pair_axes(case)
        rd = case["rotary"]
        st["freqs"] = torch.tensor([10000.0 ** (-2.0 * i / rd) for i in range(rd // 2)], dtype=torch.float64, device="cuda")
        st["axes"] = torch.tensor(axes, device="cuda")
        if own:  # the handle that a program makes once, at its start
            from paged_kv_cache_90_gb300 import binding
            st["rotary"] = binding.rotary(rd, 10000.0, interleaved=case["interleaved"], axes=axes)
        return st
    if op == "copy":
        nb, n = case["blocks"], case["pairs"]
        perm = torch.randperm(nb, generator=g, device="cuda")
        src = perm[n:][torch.randint(0, nb - n, (n,), generator=g, device="cuda")]  # (children may share a source)
        st["pairs"] = torch.stack([src, perm[:n]], 1).contiguous()
        st["caches"] = _caches(case, nb, g)
        if own:
            from paged_kv_cache_90_gb300 import binding
            st["list"] = binding.cache_list(st["caches"])
        return st
    lens = _lens(case)
    tables, nb, width = _tables(case, lens, g)
    st["tables"], st["width"] = tables, width
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if op in ("tree", "keep"):
        nodes = _nodes(case)
        st["starts"] = torch.tensor([0] + nodes, device="cuda").cumsum(0).to(torch.int32)
    if op == "keep":
        # the accepted path: the first node, say, and some behind the places that the path will take
        rng = torch.Generator().manual_seed(seed)
        kept = _kept(case)
        rows = torch.full((sum(nodes),), -1, dtype=torch.int32)
        at = 0
        for n, k in zip(nodes, kept):
            path = (k + torch.randperm(n - k, generator=rng)[:k]).sort().values if n - k >= k else torch.arange(k)
            if k and torch.rand(1, generator=rng).item() < 0.5:
                path[0] = 0
            rows[at:at + k] = path.to(torch.int32)
            at += n
        st["keep"], st["counts"] = rows.cuda(), torch.tensor(kept, dtype=torch.int32, device="cuda")
        st["new_lens"] = torch.zeros_like(st["lens"])
        st["caches"] = _caches(case, nb, g)
        if own:
            from paged_kv_cache_90_gb300 import binding
            st["list"] = binding.cache_list(st["caches"])
        return st
    rows = case["seqs"]
    if op == "tree":
        rows = sum(nodes)
        st["mask"] = _tree_masks(nodes, seed)
        st["most"] = max(nodes)
    st["query"] = _randn((rows, case["heads"], d), g).mul_(1.5).to(torch.bfloat16)
    st["out"] = torch.empty_like(st["query"])
    st["key_cache"], st["k_scales"] = _quantise(_outliers(_randn((nb, hk, bs, d), g)), 1.0)
    vc = _randn((nb, hk, bs, d), g).mul_(torch.exp(0.5 * _randn((nb, hk, bs, 1), g)))
    st["value_cache"], st["v_scales"] = _quantise(vc, 1.0)
    return st


# ---- one pass --------------------------------------------------------------------------


def _quantise(x, factor):
    """Rows of float32 as bytes of two codes and e4m3 group scales: the operator's definition."""
    y = x.reshape(*x.shape[:-1], -1, 16)
    f = torch.tensor(factor, dtype=torch.float32, device=x.device)
    top = y.abs().amax(-1)
    # (divisions by tensors: one by a Python number multiplies by its reciprocal)
    scales = (top / (6.0 * f).expand_as(top)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = (scales.float() * f)[..., None]
    q = y * torch.where(step > 0, torch.ones_like(step) / step, torch.zeros_like(step))
    a = q.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(q)).reshape(x.shape).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def _dequantise(cache, scales, factor):
    codes = torch.stack([cache & 15, cache >> 4], -1).reshape(*cache.shape[:-1], -1).long()
    table = torch.tensor(_VALUES + tuple(-v for v in _VALUES), device=cache.device)
    step = scales.float() * torch.tensor(factor, dtype=torch.float32, device=cache.device)
    return table[codes] * step.repeat_interleave(16, -1)


def _scale(case):
    return case["dim"] ** -0.5


def _write(cache, slots, rows):
    bs = cache.shape[2]
    cache[slots // bs, :, slots % bs] = rows


def _rotate(x, cos, sin, rd, interleaved):
    """x in float32 [T, H, D]; cos and sin [T, 1, rd / 2]."""
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y[..., 0:rd:2] = a * cos - b * sin
        y[..., 1:rd:2] = b * cos + a * sin
    else:
        a, b = x[..., : rd // 2], x[..., rd // 2: rd]
        y[..., : rd // 2] = a * cos - b * sin
        y[..., rd // 2: rd] = b * cos + a * sin
    return y


def _axes(st):
    case = st["case"]
    angle = st["positions"].double()[st["axes"]].T * st["freqs"]  # far positions need the bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    rd, inter, dt = case["rotary"], case["interleaved"], st["query"].dtype
    st["query_out"].copy_(_rotate(st["query"].float(), cos, sin, rd, inter).to(dt))
    _write(st["key_cache"], st["slots"], _rotate(st["key"].float(), cos, sin, rd, inter).to(dt))
    _write(st["value_cache"], st["slots"], st["value"])
    return {"query": st["query_out"], "key_cache": st["key_cache"], "value_cache": st["value_cache"]}


def _quantize(st):
    bs, slots, factor = st["case"]["bs"], st["slots"], st["case"]["scale"]
    for name, cache, scales, back in (("key", "key_cache", "k_scales", "key_back"),
                                      ("value", "value_cache", "v_scales", "value_back")):
        q, s = _quantise(st[name].float(), factor)
        _write(st[cache], slots, q)
        _write(st[scales].view(torch.uint8), slots, s.view(torch.uint8))
        block, offset = slots // bs, slots % bs
        st[back].copy_(_dequantise(st[cache][block, :, offset],
                                   st[scales].view(torch.uint8)[block, :, offset].view(torch.float8_e4m3fn), factor))
    return {"key": st["key_back"], "value": st["value_back"]}


def _gather(st, cache, scales):
    """Every sequence's K or V as [S, Hk, width * bs, D] float32."""
    at = st["tables"].long()
    x = _dequantise(st[cache][at], st[scales].view(torch.uint8)[at].view(torch.float8_e4m3fn), 1.0)
    s, w, hk, bs, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(s, hk, w * bs, d)


def _softmax_pv(z, keep, v):
    z = z.masked_fill(~keep, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total > 0, total, torch.ones_like(total))


def _decode(st):
    k, v = _gather(st, "key_cache", "k_scales"), _gather(st, "value_cache", "v_scales")
    s, hk, length, d = k.shape
    window = st["case"]["window"]
    at, lens = torch.arange(length, device="cuda")[None, :], st["lens"][:, None]
    inside = at < lens
    if window:
        inside = inside & (at >= lens - window)
    v = v * inside[:, None, :, None]
    q = st["query"].float().view(s, hk, -1, d)
    z = (q @ k.transpose(-1, -2)) * _scale(st["case"])
    st["out"].copy_(_softmax_pv(z, inside[:, None, None, :], v).reshape(s, -1, d).to(st["out"].dtype))
    return st["out"]


def _tree(st):
    k, v = _gather(st, "key_cache", "k_scales"), _gather(st, "value_cache", "v_scales")
    s, hk, length, d = k.shape
    most, rows, hq = st["most"], st["query"].shape[0], st["query"].shape[1]
    starts, lens = st["starts"].long(), st["lens"].long()
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(starts[1:], row, right=True)
    node = row - starts[seq]
    q = torch.zeros(s, most, hq, d, device="cuda")
    q[seq, node] = st["query"].float()
    bits = torch.zeros(s, most, dtype=torch.int64, device="cuda")
    bits[seq, node] = st["mask"][:, 0]
    # position j is drafted node j - (L - n); earlier positions are seen by every node
    past = lens - (starts[1:] - starts[:-1])
    j = torch.arange(length, device="cuda")[None, :] - past[:, None]
    seen = (bits[:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
    inside = torch.arange(length, device="cuda")[None, :] < lens[:, None]
    keep = ((j < 0)[:, None, :] | (seen == 1)) & inside[:, None, :]
    v = v * inside[:, None, :, None]
    g = hq // hk
    q = q.view(s, most, hk, g, d).permute(0, 2, 3, 1, 4).reshape(s, hk, g * most, d)
    z = (q @ k.transpose(-1, -2)) * _scale(st["case"])
    z = z.view(s, hk, g, most, length)
    o = _softmax_pv(z, keep[:, None, None], v[:, :, None])
    st["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(s, most, hq, d)[seq, node].to(st["out"].dtype))
    return st["out"]


def _copy(st):
    src, dst = st["pairs"][:, 0], st["pairs"][:, 1]
    for c in st["caches"]:
        c[dst] = c[src]
    return st["caches"]


def _keep(st):
    bs = st["case"]["bs"]
    starts, lens, counts = st["starts"].long(), st["lens"].long(), st["counts"].long()
    nodes = starts[1:] - starts[:-1]
    row = torch.arange(st["keep"].shape[0], device="cuda")
    seq = torch.searchsorted(starts[1:], row, right=True)
    i = row - starts[seq]
    seq, i, frm = (x[i < counts[seq]] for x in (seq, i, st["keep"].long()))
    past = (lens - nodes)[seq]
    frm, to = past + frm, past + i
    fb, tb = st["tables"].long()[seq, frm // bs], st["tables"].long()[seq, to // bs]
    for c in st["caches"]:
        c[tb, :, to % bs] = c[fb, :, frm % bs]
    st["new_lens"].copy_(lens - nodes + counts)
    return {"caches": st["caches"], "lens": st["new_lens"]}


def _own(st):
    from paged_kv_cache_90_gb300 import binding
    case = st["case"]
    op = case["op"]
    if op == "axes":
        binding.rotary_and_cache(st["query_out"], st["query"], st["key"], st["value"], st["positions"], st["key_cache"],
                                 st["value_cache"], st["slots"], st["rotary"])
        return {"query": st["query_out"], "key_cache": st["key_cache"], "value_cache": st["value_cache"]}
    if op == "quantize":
        s = case["scale"]
        binding.quantize_and_cache(st["key"], st["value"], st["key_cache"], st["value_cache"], st["k_scales"],
                                   st["v_scales"], st["slots"], k_scale=s, v_scale=s)
        binding.read_cache(st["key_back"], st["value_back"], st["key_cache"], st["value_cache"], st["slots"],
                           k_scale=s, v_scale=s, k_token_scales=st["k_scales"], v_token_scales=st["v_scales"])
        return {"key": st["key_back"], "value": st["value_back"]}
    if op == "copy":
        binding.copy_cache_blocks(st["list"], st["pairs"])
        return st["caches"]
    if op == "keep":
        binding.keep_tokens(st["list"], st["tables"], st["lens"], st["starts"], st["keep"], st["counts"], case["bs"],
                            st["width"], new_lens=st["new_lens"])
        return {"caches": st["caches"], "lens": st["new_lens"]}
    if op == "decode":
        return binding.paged_attention_decode_quantized(
            st["out"], st["query"], st["key_cache"], st["value_cache"], st["k_scales"], st["v_scales"], st["tables"],
            st["lens"], case["kv_heads"], _scale(case), case["bs"], st["width"], sliding_window=case["window"])
    return binding.paged_attention_tree(
        st["out"], st["query"], st["key_cache"], st["value_cache"], st["tables"], st["lens"], st["starts"], st["mask"],
        case["kv_heads"], _scale(case), case["bs"], st["width"], k_token_scales=st["k_scales"],
        v_token_scales=st["v_scales"])


def run(state):
    if own:
        return _own(state)
    return {"axes": _axes, "quantize": _quantize, "decode": _decode, "tree": _tree, "copy": _copy,
            "keep": _keep}[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------------


def _row_bytes(case):
    """Bytes of a (token, KV head) row in the caches of all layers."""
    d = case["dim"]
    return 2 * case["layers"] * {"bf16": 2 * d, "f32": 4 * d, "int8": d + 4}[case["cache"]]


def work(case):
    hk, d, bs, op = case["kv_heads"], case["dim"], case["bs"], case["op"]
    if op == "axes":
        t, size = case["tokens"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * t * (case["heads"] + 2 * hk) * d * size + 8 * t * (1 + len(_sections(case))),
                "flops": 3 * t * (case["heads"] + hk) * case["rotary"]}
    if op == "quantize":
        n = 2 * case["tokens"] * hk  # rows of K and V: written as codes and scales, read back as float32
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": n * (size * d + 2 * (d // 2 + d // 16) + 4 * d) + 16 * case["tokens"], "flops": 3 * n * d}
    if op == "copy":
        return {"bytes": 2 * case["pairs"] * hk * bs * _row_bytes(case) + 16 * case["pairs"], "flops": 0}
    lens = _lens(case)
    if op == "keep":
        kept = sum(_kept(case))
        return {"bytes": 2 * kept * hk * _row_bytes(case) + 4 * kept + 16 * case["seqs"], "flops": 0}
    nodes = _nodes(case) if op == "tree" else [1] * case["seqs"]
    if op == "decode" and case["window"]:
        lens = [min(n, case["window"]) for n in lens]
    row = d // 2 + d // 16
    read = 2 * sum(lens) * hk * row + 4 * sum(-(-n // bs) for n in lens) + 4 * case["seqs"]
    if op == "tree":
        read += 8 * sum(nodes) + 4 * (case["seqs"] + 1)
    return {"bytes": read + 4 * sum(nodes) * case["heads"] * d,
            "flops": 4 * sum(a * b for a, b in zip(lens, nodes)) * case["heads"] * d}


# ---- the definitions in 64 bits ---------------------------------------------------------


def _exact_axes(st):
    case = st["case"]
    rd, bs = case["rotary"], case["bs"]
    pairs = torch.arange(rd // 2, device="cuda")
    lo = 2 * pairs if case["interleaved"] else pairs
    hi = lo + 1 if case["interleaved"] else lo + rd // 2
    turn = torch.empty(case["tokens"], rd // 2, dtype=torch.float64, device="cuda")
    for i, a in enumerate(_pair_axes(case)):
        turn[:, i] = torch.remainder(st["positions"][a].double() * (st["freqs"][i] / _TWO_PI), 1.0) * _TWO_PI
    unit = torch.polar(torch.ones_like(turn), turn)[:, None]

    def turned(x):
        y = x.double()
        z = torch.complex(y[..., lo], y[..., hi]) * unit
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    block, offset = st["slots"] // bs, st["slots"] % bs
    kc, vc = st["key_cache"].double(), st["value_cache"].double()
    kc.permute(0, 2, 1, 3)[block, offset] = turned(st["key"])
    vc.permute(0, 2, 1, 3)[block, offset] = st["value"].double()
    return {"query": turned(st["query"]), "key_cache": kc, "value_cache": vc}


def _exact_quantize(st):
    # the definition fixes the scale, its reciprocal and the product in IEEE binary32; what is
    # stored is a code and an 8-bit scale, and what they stand for is the product, here in 64 bits
    f, out = torch.tensor(st["case"]["scale"], dtype=torch.float32), {}
    grid = torch.tensor(_VALUES, dtype=torch.float64)
    even = torch.tensor([1, 0] * 4, dtype=torch.bool)  # the codes that a tie goes to
    for name in ("key", "value"):
        x = st[name].cpu().float()
        y = x.unflatten(-1, (-1, 16))
        g = torch.div(y.abs().max(dim=-1).values, torch.tensor(6.0) * f).clamp_max(448.0).to(torch.float8_e4m3fn).float() * f
        q = torch.where(g > 0, torch.reciprocal(g), torch.zeros_like(g))[..., None] * y
        a = q.abs().double().clamp_max(6.0)
        up = torch.searchsorted(grid, a).clamp(1, 7)  # grid[up - 1] <= a <= grid[up], but a tie's side
        below, above = a - grid[up - 1], grid[up] - a
        pick = torch.where((above < below) | ((above == below) & even[up]), up, up - 1)
        out[name] = (torch.copysign(grid[pick], q.double()) * g.double()[..., None]).reshape(x.shape)
    return out


def _exact_rows(cache, scales, block, offset):
    """Rows [n, Hk, D] of a 4-bit cache in 64 bits."""
    b, s = cache[block, :, offset].long(), scales.float()[block, :, offset].double()
    x = torch.empty(*b.shape[:-1], 2 * b.shape[-1], dtype=torch.float64, device=b.device)
    for half in (0, 1):
        n = (b >> (4 * half)) & 15
        e, m = (n >> 1) & 3, n & 1
        size = torch.where(e > 0, (2 + m).double() * torch.exp2((e - 2).double()), 0.5 * m.double())
        x[..., half::2] = torch.where(n >= 8, -size, size)
    return (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _exact_attention(st):
    case = st["case"]
    hk, d, bs = case["kv_heads"], case["dim"], case["bs"]
    g = case["heads"] // hk
    out = torch.zeros(st["query"].shape, dtype=torch.float64, device="cuda")
    lens = st["lens"].tolist()
    starts = st["starts"].tolist() if case["op"] == "tree" else list(range(case["seqs"] + 1))
    for s, length in enumerate(lens):
        first = max(0, length - case["window"]) if case.get("window") else 0
        slots = torch.arange(first, length, device="cuda")
        block, offset = st["tables"][s].long()[slots // bs], slots % bs
        k = _exact_rows(st["key_cache"], st["k_scales"], block, offset)
        v = _exact_rows(st["value_cache"], st["v_scales"], block, offset)
        a, b = starts[s], starts[s + 1]
        n = b - a
        q = st["query"][a:b].double().view(n, hk, g, d)
        z = torch.einsum("nhgd,lhd->nhgl", q, k) * _scale(case)
        if case["op"] == "tree":
            bits = st["mask"][a:b, 0, None] >> torch.arange(n, device="cuda")[None, :]
            hidden = torch.zeros(n, length, dtype=torch.bool, device="cuda")
            hidden[:, length - n:] = (bits & 1) == 0
            z.masked_fill_(hidden[:, None, None, :], -math.inf)
        out[a:b] = torch.einsum("nhgl,lhd->nhgd", torch.softmax(z, -1), v).reshape(n, -1, d)
    return out


def _wide(x):
    return x.double() if x.is_floating_point() else x


def _exact_copy(st):
    of = torch.arange(st["case"]["blocks"], device="cuda")
    for src, dst in st["pairs"].tolist():
        of[dst] = src
    return [_wide(c.index_select(0, of)) for c in st["caches"]]


def _exact_keep(st):
    bs, nb = st["case"]["bs"], st["caches"][0].shape[0]
    tables, starts, lens = st["tables"].tolist(), st["starts"].tolist(), st["lens"].tolist()
    keep, counts, new = st["keep"].tolist(), st["counts"].tolist(), []
    of = list(range(nb * bs))  # the slot whose token each slot holds in the end
    for s, length in enumerate(lens):
        past = length - (starts[s + 1] - starts[s])
        slot = [tables[s][p // bs] * bs + p % bs for p in range(past, length)]
        for i in range(counts[s]):
            of[slot[i]] = slot[keep[starts[s] + i]]
        new.append(past + counts[s])
    of = torch.tensor(of, device="cuda")
    out = []
    for c in st["caches"]:
        flat = c.transpose(1, 2).flatten(0, 1)[of]
        out.append(_wide(flat.unflatten(0, (nb, bs)).transpose(1, 2).contiguous()))
    return {"caches": out, "lens": torch.tensor(new, dtype=torch.int32, device="cuda")}


def exact(case, seed):
    st = prepare(case, seed)
    return {"axes": _exact_axes, "quantize": _exact_quantize, "copy": _exact_copy, "keep": _exact_keep,
            "decode": _exact_attention, "tree": _exact_attention}[case["op"]](st)
