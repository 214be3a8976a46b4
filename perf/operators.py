"""Measured cases of the speculative-decoding and quantised-cache operators.

Four operators that stand beside the cache write and the paged attention:

  rotary      rotary positions for queries and keys, the keys and values written to the
              paged cache in the same pass (``binding.rotary_and_cache``);
  quantize    a token's K and V quantised to 8-bit integers as they are written, one
              scale per token and KV head found on the way, and read back
              (``binding.quantize_and_cache``, ``binding.read_cache``);
  decode8     single-token decode attention over that cache
              (``binding.paged_attention_decode_quantized``);
  tree        attention of a tree of drafted tokens over a bf16 or a quantised cache
              (``binding.paged_attention_tree``).

``run`` computes them in elementary torch operations, or, with ``own``, through the
package's entry points; ``exact`` computes them from their definition in 64 bits.
"""
import math

import torch

own = False

_TWO_PI = 2.0 * math.pi
_PHI = 0.6180339887498949


def listed():
    return [
        # one sequence's next token: launch latency is all there is
        {"name": "rotary_one_token", "op": "rotary", "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "scaling": "none", "far": 4096, "dtype": "bf16", "bs": 16},
        # a decode batch of float32 activations, pairs interleaved, half of each head rotated
        {"name": "rotary_partial_f32", "op": "rotary", "tokens": 250, "heads": 12, "kv_heads": 4, "dim": 64, "rotary": 32,
         "interleaved": True, "scaling": "linear", "far": 32768, "dtype": "f32", "bs": 8},
        # the packed prompts of a prefill step, positions up to a million, wavelengths stretched by bands
        {"name": "rotary_prefill", "op": "rotary", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "scaling": "bands", "far": 1 << 20, "dtype": "bf16", "bs": 16},
        # a decode batch's new tokens into the quantised cache, and back
        {"name": "quantize_decode_batch", "op": "quantize", "tokens": 64, "kv_heads": 8, "dim": 128, "bs": 16},
        # a prefill step's tokens
        {"name": "quantize_prefill", "op": "quantize", "tokens": 16384, "kv_heads": 8, "dim": 128, "bs": 16},
        # one sequence of odd length, the smallest decode call
        {"name": "decode8_one_seq", "op": "decode8", "seqs": 1, "lo": 777, "hi": 777, "heads": 32, "kv_heads": 8,
         "dim": 128, "bs": 16},
        # the benchmark's decode batch (64 sequences, contexts spread over 128..2048)
        {"name": "decode8_batch", "op": "decode8", "seqs": 64, "lo": 129, "hi": 2048, "heads": 32, "kv_heads": 8,
         "dim": 128, "bs": 16},
        # the benchmark's long contexts
        {"name": "decode8_long", "op": "decode8", "seqs": 8, "lo": 32768, "hi": 32768, "heads": 32, "kv_heads": 8,
         "dim": 128, "bs": 32},
        # one sequence, a small tree: the lowest-latency form of speculative decoding
        {"name": "tree_one_seq", "op": "tree", "seqs": 1, "lo": 341, "hi": 341, "nodes_lo": 9, "nodes_hi": 9, "heads": 32,
         "kv_heads": 8, "dim": 128, "bs": 16, "cache": "bf16"},
        # the decode batch with ragged trees of 5 to 24 nodes
        {"name": "tree_batch", "op": "tree", "seqs": 64, "lo": 160, "hi": 2048, "nodes_lo": 5, "nodes_hi": 24,
         "heads": 32, "kv_heads": 8, "dim": 128, "bs": 16, "cache": "bf16"},
        # full 64-node trees over long contexts: 256 query rows for each KV head
        {"name": "tree_long_wide", "op": "tree", "seqs": 8, "lo": 30001, "hi": 32768, "nodes_lo": 64, "nodes_hi": 64,
         "heads": 32, "kv_heads": 8, "dim": 128, "bs": 16, "cache": "bf16"},
        # trees over the quantised cache
        {"name": "tree_quantized", "op": "tree", "seqs": 32, "lo": 1000, "hi": 8192, "nodes_lo": 8, "nodes_hi": 32,
         "heads": 32, "kv_heads": 8, "dim": 128, "bs": 16, "cache": "int8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "quantize", "decode8", "tree", "tree"])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    bs = rng.choice([8, 16, 32])
    if op == "rotary":
        return {"op": op, "tokens": _log(rng, 1, 12000), "heads": kv * min(group, 4), "kv_heads": kv, "dim": dim,
                "rotary": 2 * rng.randint(1, dim // 2) if rng.random() < 0.5 else dim, "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "base", "bands", "ramp"]), "far": _log(rng, 1000, 1 << 20),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "bs": bs}
    if op == "quantize":
        return {"op": op, "tokens": _log(rng, 1, 16000), "kv_heads": kv, "dim": dim, "bs": bs}
    # contexts and batch so that no draw reads more than the largest listed case
    hi = _log(rng, 1, 32768)
    lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
    seqs = min(_log(rng, 1, 128), max(1, 262144 // hi))
    if op == "decode8":
        return {"op": op, "seqs": seqs, "lo": lo, "hi": hi, "heads": kv * group, "kv_heads": kv, "dim": dim, "bs": bs}
    n_hi = min(_log(rng, 1, 64), hi)
    if n_hi * group > 256:
        n_hi = 256 // group
    return {"op": op, "seqs": seqs, "lo": max(lo, n_hi), "hi": hi, "nodes_lo": max(1, n_hi // rng.choice([1, 2, 4])),
            "nodes_hi": n_hi, "heads": kv * group, "kv_heads": kv, "dim": dim, "bs": bs,
            "cache": rng.choice(["bf16", "bf16", "int8"])}


# ---- inputs ----------------------------------------------------------------------------


def _lens(case):
    """The sequences' context lengths: spread over lo..hi, a function of the case alone."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    return [lo + int((((i + 1) * _PHI) % 1.0) * (hi - lo + 1)) for i in range(n)]


def _nodes(case):
    """The sequences' drafted tokens (the last of each context)."""
    n, lo, hi = case["seqs"], case["nodes_lo"], case["nodes_hi"]
    return [lo + int((((i + 3) * _PHI) % 1.0) * (hi - lo + 1)) for i in range(n)]


def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _frequencies(case):
    """Radians per position of each rotated pair, and the factor on cosine and sine."""
    rd, kind = case["rotary"], case["scaling"]
    base, factor, original, low, high = 10000.0, 8.0, 8192.0, 1.0, 4.0
    if kind == "base" and rd > 2:
        base = base * factor ** (rd / (rd - 2.0))
    freqs = []
    for i in range(rd // 2):
        f = base ** (-2.0 * i / rd)
        turns = original * f / _TWO_PI  # over the original context
        if kind == "linear":
            f /= factor
        elif kind == "bands":
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            f = f * keep + f / factor * (1.0 - keep)
        elif kind == "ramp":
            first = rd * math.log(original / (32.0 * _TWO_PI)) / (2.0 * math.log(base))
            last = rd * math.log(original / (1.0 * _TWO_PI)) / (2.0 * math.log(base))
            first, last = max(math.floor(first), 0), min(math.ceil(last), rd - 1)
            slow = min(1.0, max(0.0, (i - first) / max(last - first, 1e-3)))
            f = f * (1.0 - slow) + f / factor * slow
        freqs.append(f)
    return freqs, (0.1 * math.log(factor) + 1.0 if kind == "ramp" else 1.0)


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _outliers(x):
    """A few channels of a head an order of magnitude above the rest, as keys have them."""
    x = x.float()
    x[..., 3] *= 6.0
    x[..., x.shape[-1] // 2 + 1] *= 10.0
    return x


def _quantise(x):
    """Codes and scales of rows of float32: the operator's definition."""
    top = x.abs().amax(-1)
    s = top / torch.full_like(top, 127.0)  # (a division by a Python number multiplies by its reciprocal)
    q = torch.round(x / torch.where(s > 0, s, torch.ones_like(s))[..., None]).clamp(-127, 127)
    return q.to(torch.int8), s


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


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, hk, bs = case["dim"], case["kv_heads"], case["bs"]
    st = {"case": case}
    if case["op"] in ("rotary", "quantize"):
        t, dt = case["tokens"], _dtype(case)
        nb = -(-t // bs) + 3
        st["key"] = _outliers(_randn((t, hk, d), g)).to(dt)
        st["value"] = (_randn((t, hk, d), g) * torch.exp(0.5 * _randn((t, hk, 1), g))).to(dt)
        # runs of tokens in scattered blocks, as an engine's block tables give them
        perm = torch.randperm(nb, generator=g, device="cuda")
        token = torch.arange(t, device="cuda")
        st["slots"] = (perm[token // bs] * bs + token % bs).contiguous()
        if case["op"] == "quantize":
            st["key_cache"] = torch.zeros(nb, hk, bs, d, dtype=torch.int8, device="cuda")
            st["value_cache"] = torch.zeros_like(st["key_cache"])
            st["k_scales"] = torch.zeros(nb, hk, bs, device="cuda")
            st["v_scales"] = torch.zeros_like(st["k_scales"])
            st["key_back"] = torch.empty(t, hk, d, device="cuda")
            st["value_back"] = torch.empty_like(st["key_back"])
            return st
        st["query"] = _randn((t, case["heads"], d), g, dt)
        st["query_out"] = torch.empty_like(st["query"])
        st["positions"] = torch.randint(0, case["far"], (t,), generator=g, device="cuda")
        st["key_cache"] = torch.zeros(nb, hk, bs, d, dtype=dt, device="cuda")
        st["value_cache"] = torch.zeros_like(st["key_cache"])
        freqs, st["magnitude"] = _frequencies(case)
        st["freqs"] = torch.tensor(freqs, dtype=torch.float64, device="cuda")
        if own:  # the handle that a program makes once, at its start
            from paged_kv_cache_90_gb300 import binding
            st["rotary"] = binding.rotary(case["rotary"], 10000.0, interleaved=case["interleaved"],
                                          scaling=case["scaling"], factor=8.0, original_max_position=8192)
        return st
    lens = _lens(case)
    tables, nb, width = _tables(case, lens, g)
    st["tables"], st["width"] = tables, width
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    rows = case["seqs"]
    if case["op"] == "tree":
        nodes = _nodes(case)
        rows = sum(nodes)
        st["starts"] = torch.tensor([0] + nodes, device="cuda").cumsum(0).to(torch.int32)
        st["mask"] = _tree_masks(nodes, seed)
        st["most"] = max(nodes)
    st["query"] = _randn((rows, case["heads"], d), g).mul_(1.5).to(torch.bfloat16)
    st["out"] = torch.empty_like(st["query"])
    kc = _randn((nb, hk, bs, d), g)
    vc = _randn((nb, hk, bs, d), g) * torch.exp(0.5 * _randn((nb, hk, bs, 1), g))
    if case["op"] == "decode8" or case["cache"] == "int8":
        st["key_cache"], st["k_scales"] = _quantise(kc)
        st["value_cache"], st["v_scales"] = _quantise(vc)
    else:
        st["key_cache"], st["value_cache"] = kc.to(torch.bfloat16), vc.to(torch.bfloat16)
    return st


# ---- one pass --------------------------------------------------------------------------


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


def _rotary(st):
    case = st["case"]
    angle = st["positions"].double()[:, None] * st["freqs"][None, :]  # far positions need the bits
    cos = (torch.cos(angle) * st["magnitude"]).float()[:, None]
    sin = (torch.sin(angle) * st["magnitude"]).float()[:, None]
    rd, inter, dt = case["rotary"], case["interleaved"], st["query"].dtype
    st["query_out"].copy_(_rotate(st["query"].float(), cos, sin, rd, inter).to(dt))
    _write(st["key_cache"], st["slots"], _rotate(st["key"].float(), cos, sin, rd, inter).to(dt))
    _write(st["value_cache"], st["slots"], st["value"])
    return {"query": st["query_out"], "key_cache": st["key_cache"], "value_cache": st["value_cache"]}


def _quantize(st):
    bs, slots = st["case"]["bs"], st["slots"]
    for name, cache, scales, back in (("key", "key_cache", "k_scales", "key_back"),
                                      ("value", "value_cache", "v_scales", "value_back")):
        q, s = _quantise(st[name].float())
        _write(st[cache], slots, q)
        _write(st[scales], slots, s)
        st[back].copy_(st[cache][slots // bs, :, slots % bs].float() * st[scales][slots // bs, :, slots % bs][..., None])
    return {"key": st["key_back"], "value": st["value_back"], "k_scales": st["k_scales"], "v_scales": st["v_scales"]}


def _gather(st, cache, scales):
    """Every sequence's K or V as [S, Hk, width * bs, D] float32."""
    x = st[cache][st["tables"].long()].float()
    if scales in st:
        x = x * st[scales][st["tables"].long()][..., None]
    s, w, hk, bs, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(s, hk, w * bs, d)


def _softmax_pv(z, keep, v):
    z = z.masked_fill(~keep, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total > 0, total, torch.ones_like(total))


def _decode8(st):
    k, v = _gather(st, "key_cache", "k_scales"), _gather(st, "value_cache", "v_scales")
    s, hk, length, d = k.shape
    inside = torch.arange(length, device="cuda")[None, :] < st["lens"][:, None]
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


def _own(st):
    from paged_kv_cache_90_gb300 import binding
    case = st["case"]
    if case["op"] == "rotary":
        binding.rotary_and_cache(st["query_out"], st["query"], st["key"], st["value"], st["positions"], st["key_cache"],
                                 st["value_cache"], st["slots"], st["rotary"])
        return {"query": st["query_out"], "key_cache": st["key_cache"], "value_cache": st["value_cache"]}
    if case["op"] == "quantize":
        binding.quantize_and_cache(st["key"], st["value"], st["key_cache"], st["value_cache"], st["k_scales"],
                                   st["v_scales"], st["slots"])
        binding.read_cache(st["key_back"], st["value_back"], st["key_cache"], st["value_cache"], st["slots"],
                           k_token_scales=st["k_scales"], v_token_scales=st["v_scales"])
        return {"key": st["key_back"], "value": st["value_back"], "k_scales": st["k_scales"], "v_scales": st["v_scales"]}
    if case["op"] == "decode8":
        return binding.paged_attention_decode_quantized(
            st["out"], st["query"], st["key_cache"], st["value_cache"], st["k_scales"], st["v_scales"], st["tables"],
            st["lens"], case["kv_heads"], _scale(case), case["bs"], st["width"])
    return binding.paged_attention_tree(
        st["out"], st["query"], st["key_cache"], st["value_cache"], st["tables"], st["lens"], st["starts"], st["mask"],
        case["kv_heads"], _scale(case), case["bs"], st["width"], k_token_scales=st.get("k_scales"),
        v_token_scales=st.get("v_scales"))


def run(state):
    if own:
        return _own(state)
    return {"rotary": _rotary, "quantize": _quantize, "decode8": _decode8, "tree": _tree}[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------------


def work(case):
    hk, d, bs = case["kv_heads"], case["dim"], case["bs"]
    if case["op"] == "rotary":
        t, size = case["tokens"], 4 if case["dtype"] == "f32" else 2
        heads = case["heads"] + 2 * hk
        return {"bytes": 2 * t * heads * d * size + 16 * t, "flops": 3 * t * (case["heads"] + hk) * case["rotary"]}
    if case["op"] == "quantize":
        n = 2 * case["tokens"] * hk  # rows of K and V: written as codes and a scale, read back as float32
        return {"bytes": n * (2 * d + 2 * (d + 4) + 4 * d) + 16 * case["tokens"], "flops": 4 * n * d}
    lens = _lens(case)
    nodes = _nodes(case) if case["op"] == "tree" else [1] * case["seqs"]
    row = d + 4 if case["op"] == "decode8" or case["cache"] == "int8" else 2 * d
    entries = sum(-(-n // bs) for n in lens)
    read = 2 * sum(lens) * hk * row + 4 * entries + 4 * case["seqs"]
    if case["op"] == "tree":
        read += 8 * sum(nodes) + 4 * (case["seqs"] + 1)
    return {"bytes": read + 4 * sum(nodes) * case["heads"] * d,
            "flops": 4 * sum(a * b for a, b in zip(lens, nodes)) * case["heads"] * d}


# ---- the definitions in 64 bits ---------------------------------------------------------


def _exact_rotary(st):
    case = st["case"]
    t, rd, bs = case["tokens"], case["rotary"], case["bs"]
    pairs = torch.arange(rd // 2, device="cuda")
    lo = 2 * pairs if case["interleaved"] else pairs
    hi = lo + 1 if case["interleaved"] else lo + rd // 2
    turn = torch.remainder(st["positions"].double()[:, None] * (st["freqs"] / _TWO_PI), 1.0) * _TWO_PI
    unit = torch.polar(torch.full_like(turn, st["magnitude"]), turn)[:, None]

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
    # the definition fixes the scale and the quotient in IEEE binary32; what is stored is
    # whole, and what it stands for is the product, here in 64 bits
    bs, out = st["case"]["bs"], {}
    for name, scales in (("key", "k_scales"), ("value", "v_scales")):
        x = st[name].cpu().float()
        s = torch.div(x.abs().max(dim=-1).values, torch.tensor(127.0))
        code = torch.div(x, s.clamp_min(2.0 ** -126)[..., None]).round().clamp(-127, 127)
        full = st[scales].double().cpu()
        slots = st["slots"].cpu()
        full.permute(0, 2, 1)[slots // bs, slots % bs] = s.double()
        out[name], out[scales] = code.double() * s.double()[..., None], full
    return {k: out[k] for k in ("key", "value", "k_scales", "v_scales")}


def _exact_attention(st):
    case = st["case"]
    hk, d, bs = case["kv_heads"], case["dim"], case["bs"]
    g = case["heads"] // hk
    out = torch.zeros(st["query"].shape, dtype=torch.float64, device="cuda")
    lens = st["lens"].tolist()
    starts = st["starts"].tolist() if case["op"] == "tree" else list(range(case["seqs"] + 1))
    for s, length in enumerate(lens):
        slots = torch.arange(length, device="cuda")
        block, offset = st["tables"][s].long()[slots // bs], slots % bs
        k, v = st["key_cache"][block, :, offset].double(), st["value_cache"][block, :, offset].double()
        if "k_scales" in st:
            k = k * st["k_scales"][block, :, offset].double()[..., None]
            v = v * st["v_scales"][block, :, offset].double()[..., None]
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


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(st)
    return _exact_quantize(st) if case["op"] == "quantize" else _exact_attention(st)
