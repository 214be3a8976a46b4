"""Blocks and tokens of every cache type moved bit for bit: the read back, and the block copy of
token-scaled caches with their scales."""
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


@gpu
@pytest.mark.parametrize("dt,bits", [(torch.bfloat16, torch.int16), (torch.float32, torch.int32)])
@pytest.mark.parametrize("d", [64, 128])
def test_tokens_of_any_bits_are_moved_as_they_are(d, dt, bits):
    """Every pattern of 16 bits (NaN of every payload among them), read and written elsewhere."""
    g = torch.Generator().manual_seed(4)
    hk, bs, nb = 2, 16, 2 ** 16 // (2 * 16 * d)
    nb = max(nb, 4)
    info = torch.iinfo(bits)
    raw = torch.randint(info.min, info.max, (2, nb, hk, bs, d), generator=g, dtype=bits)
    if bits == torch.int16:
        raw.view(-1)[:2 ** 16] = torch.arange(-2 ** 15, 2 ** 15).to(torch.int16)
    kc, vc = raw[0].view(dt).cuda(), raw[1].view(dt).cuda()
    T = nb * bs
    k = torch.zeros(T, hk, d, dtype=dt).cuda()
    v = torch.zeros_like(k)
    slots = torch.randperm(T, generator=g).cuda()
    binding.read_cache(k, v, kc, vc, slots)
    assert torch.equal(k.view(bits), kc.view(bits)[slots // bs, :, slots % bs])
    assert torch.equal(v.view(bits), vc.view(bits)[slots // bs, :, slots % bs])
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    binding.reshape_and_cache(k, v, kc2, vc2, slots)
    assert torch.equal(kc2.view(bits), kc.view(bits)) and torch.equal(vc2.view(bits), vc.view(bits))
