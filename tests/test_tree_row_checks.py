"""Sequences whose rows lie outside the batch are reported by every kernel of the tree attention,
and the others' rows are right."""
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
@pytest.mark.parametrize("cache", ["bf16", "int8", "f32", "e4m3"])
@pytest.mark.parametrize("starts", [[0, 5, 9, 15], [0, 5, 9, 9, 12, 40]])
def test_rows_outside_the_batch_are_reported(starts, cache):
    c = Case(50, [60, 40], [5, 4], 2, 4, 128, 16, cache=cache,
             qdtype=torch.float32 if cache == "f32" else torch.bfloat16)
    x = c.device()
    more = len(starts) - 3
    x["starts"] = torch.tensor(starts, dtype=torch.int32).cuda()
    x["lens"] = torch.cat([x["lens"], torch.full((more,), 50, dtype=torch.int32).cuda()])
    x["tables"] = torch.cat([x["tables"], torch.zeros(more, c.mb, dtype=torch.int32).cuda()])
    out = c.call(x)
    assert binding.read_device_errors() == binding.DEVERR["context_len"]
    c.check(out)
