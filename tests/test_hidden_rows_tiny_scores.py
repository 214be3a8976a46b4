"""Trees over a token-scaled cache whose scores are all but zero: hidden nodes stay hidden; the
tolerance is that of test_tree_attention.py."""
import pytest
import torch
from test_tree_attention import Case

from paged_kv_cache_90_gb300 import binding
from paged_kv_cache_90_gb300 import build as pkv_build

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    binding.load_library()


@gpu
@pytest.mark.parametrize("q,scale", [(1e-30, 1e-18), (1e-38, 1e-30), (1.0, 1e-38), (1e-36, 1.0)])
@pytest.mark.parametrize("masks", ["tree", "none"])
def test_hidden_nodes_of_tiny_queries_and_scales(q, scale, masks):
    c = Case(3, [90, 7], [9, 7], 2, 4, 128, 16, cache="int8", masks=masks)
    c.q = (c.q.float() * q).to(torch.bfloat16)
    c.scale = scale
    c.check()
