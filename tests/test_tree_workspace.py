"""pkv_tree_workspace_bytes against what the calls ask for.

A call that is captured before any workspace is reserved is refused, and its refusal names the bytes
that it needs: in a process of its own, which has reserved none, every head layout, cache and number of
tokens says what it needs, none more than the size that is named for it and the largest as much."""
import os
import subprocess
import sys
import textwrap

import pytest

REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = textwrap.dedent(r"""
    import re
    import torch
    from paged_kv_cache_90_gb300 import binding

    hk, nb, most = 2, 4, 200
    i32 = dict(dtype=torch.int32, device="cuda")
    q_all, out_all = (torch.zeros(most * hk * 128 * 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tables, lens = torch.zeros(most, 2, **i32), torch.ones(most, **i32)
    starts = {T: torch.tensor([0, T], **i32) for T in (1, 2, 7, 8, most)}
    mask = torch.zeros(most, 4, dtype=torch.int64, device="cuda")
    caches = {}
    for d in (64, 128):
        for bs in (4, 16):
            for kind, dt, n in (("e2m1", torch.uint8, d // 2), ("int8", torch.int8, d), ("bf16", torch.bfloat16, d)):
                c = torch.zeros(nb, hk, bs, n, dtype=dt, device="cuda")
                s = {"e2m1": torch.zeros(nb, hk, bs, d // 16, device="cuda").to(torch.float8_e4m3fn),
                     "int8": torch.zeros(nb, hk, bs, device="cuda"), "bf16": None}[kind]
                caches[kind, d, bs] = c, c.clone(), s, None if s is None else s.clone()
    assert binding.read_device_errors() == 0

    def need(call):
        try:
            call()
        except binding.PkvError as e:
            return int(re.search(r"needs (\d+) workspace bytes but only 0 are reserved", e.message).group(1))
        return None

    wrong = []

    def ask():
        for d in (64, 128):
            for group in (1, 3, 8, 9, 16, 17, 64, 100, 128):
                for T, one in starts.items():
                    q, out = (x[:T * hk * group * d].view(T, hk * group, d) for x in (q_all, out_all))
                    asked = {}
                    for kind in ("e2m1", "int8", "bf16"):
                        for bs in (4, 16):
                            kc, vc, ks, vs = caches[kind, d, bs]
                            if kind != "bf16":
                                asked[kind, bs, "decode"] = need(lambda: binding.paged_attention_decode_quantized(
                                    out, q, kc, vc, ks, vs, tables[:T], lens[:T], hk, 0.1, bs, 2))
                            asked[kind, bs, "tree"] = need(lambda: binding.paged_attention_tree(
                                out, q, kc, vc, tables[:1], lens[:1], one, mask[:T], hk, 0.1, bs, 2,
                                k_token_scales=ks, v_token_scales=vs))
                    named = binding.tree_workspace_bytes(T, T, hk * group, hk, d)
                    without = [k for k, v in asked.items() if v is None and k[0] == "e2m1"]
                    if without or max(v or 0 for v in asked.values()) != named:
                        wrong.append((d, group, T, named, asked))

    graph, x = torch.cuda.CUDAGraph(), torch.zeros(1, device="cuda")
    with torch.cuda.graph(graph):   # (never replayed)
        x.add_(1)
        ask()
    assert not wrong, wrong
    assert binding.read_device_errors() == 0
    print("sizes checked")
""")


@pytest.mark.gpu
def test_named_sizes_are_what_the_largest_call_asks_for():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=REPO, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and "sizes checked" in r.stdout, r.stdout + r.stderr
