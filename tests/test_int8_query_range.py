"""Attention over a token-scaled int8 cache with queries near the ends of their type's range,
where the scores are ordinary numbers; the tolerance is that of test_tree_attention.py."""
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
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("hk,group,d", [(2, 4, 128), (1, 12, 64), (1, 30, 128)])
@pytest.mark.parametrize("power", [-110, -100, 100, 115, 116, 127])
def test_queries_of_any_magnitude(power, hk, group, d, decode):
    """Queries of about 2^power; the scale brings the scores back."""
    c = Case(power + 200, [200, 40], [6, 5], hk, group, d, 16, cache="int8", decode=decode)
    c.q = (c.q.float().clamp(-3, 3) * 0.5 * 2.0 ** power).to(torch.bfloat16)
    assert torch.isfinite(c.q).all()
    c.scale = 2.0 ** min(-3 - power, 120)
    c.check()


@gpu
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("hk,group,d", [(2, 4, 128), (1, 12, 64), (1, 30, 128)])
@pytest.mark.parametrize("key,query", [(110, 0), (120, -60), (-115, 0), (-115, 100), (100, 20), (-60, -60)])
def test_keys_of_any_magnitude(key, query, hk, group, d, decode):
    """Keys of about 2^key under queries of about 2^query; the scale brings the scores back (as far
    as it can)."""
    c = Case(key + 300, [200, 40], [6, 5], hk, group, d, 16, cache="int8", decode=decode)
    c.k_scales = c.k_scales * 2.0 ** key
    c.K64 = c.kc.double() * c.k_scales.double()[..., None]
    c.q = (c.q.float() * 2.0 ** query).to(torch.bfloat16)
    c.scale = 2.0 ** (-3 - key - query)
    c.check()
