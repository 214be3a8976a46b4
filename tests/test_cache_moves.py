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


# ---- copy-on-write of token-scaled blocks ------------------------------------------------------


@gpu
@pytest.mark.parametrize("bs,hk,d", [(2, 1, 64), (4, 3, 128), (16, 2, 128), (32, 8, 64)])
@pytest.mark.parametrize("shift", [0, 1])
def test_blocks_of_a_token_scaled_cache_are_copied_with_their_scales(bs, hk, d, shift):
    """Codes and scales bit for bit (NaN among them), the other blocks as they were; scales as a
    slice of a wider tensor too."""
    g = torch.Generator().manual_seed(bs)
    nb = 40
    codes = torch.randint(-128, 128, (nb, hk, bs, d), generator=g, dtype=torch.int8)
    scales = torch.randint(-2 ** 31, 2 ** 31 - 1, (nb, hk, bs), generator=g, dtype=torch.int32).view(torch.float32)
    perm = torch.randperm(nb, generator=g)
    pairs = torch.stack([perm[:12], perm[12:24]], 1).contiguous()
    pairs[3, 0] = pairs[4, 0]                                  # one source twice
    wide = torch.zeros(nb, hk + shift, bs + 3 * shift).cuda()
    sc = wide[:, shift:, shift:shift + bs]
    wide.view(torch.int32)[:, shift:, shift:shift + bs] = scales.view(torch.int32).cuda()
    c = codes.cuda()
    binding.copy_blocks(c, pairs.cuda())
    binding.copy_blocks(sc, pairs.cuda())
    want_c, want_s = codes.clone(), scales.clone().view(torch.int32)
    want_c[pairs[:, 1]] = codes[pairs[:, 0]]
    want_s[pairs[:, 1]] = scales.view(torch.int32)[pairs[:, 0]]
    assert torch.equal(c.cpu(), want_c)
    assert torch.equal(sc.cpu().contiguous().view(torch.int32), want_s)
    if shift:
        assert (wide[:, :1] == 0).all() and (wide[:, :, :1] == 0).all() and (wide[:, :, bs + 1:] == 0).all()
    binding.copy_blocks(sc, torch.tensor([[0, nb]]).cuda())
    assert binding.read_device_errors() == binding.DEVERR["copy_pair"]


@gpu
def test_shared_blocks_of_a_token_scaled_cache_part_on_a_write():
    """Two sequences share a prompt's blocks; one copies the last block before it writes into it, and
    both decode as sequences that never shared."""
    hq, hk, d, bs, L = 8, 2, 128, 16, 41
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(L + 2, hk, d, generator=g).bfloat16().cuda() for _ in range(2))
    kc = torch.zeros(8, hk, bs, d, dtype=torch.int8).cuda()
    vc, ks = torch.zeros_like(kc), torch.zeros(8, hk, bs).cuda()
    vs = ks.clone()
    binding.quantize_and_cache(k[:L], v[:L], kc, vc, ks, vs, torch.arange(L).cuda())
    for t in (kc, vc, ks, vs):
        binding.copy_blocks(t, torch.tensor([[L // bs, 5]]).cuda())
    tables = torch.tensor([[0, 1, 2], [0, 1, 5]], dtype=torch.int32).cuda()
    at = torch.tensor([L, 5 * bs + L % bs]).cuda()
    binding.quantize_and_cache(k[L:], v[L:], kc, vc, ks, vs, at)
    q = torch.randn(2, hq, d, generator=g).bfloat16().cuda()
    lens = torch.tensor([L + 1, L + 1], dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    binding.paged_attention_decode_quantized(out, q, kc, vc, ks, vs, tables, lens, hk, d ** -0.5, bs, 3)
    for s in range(2):
        kc1, vc1, ks1, vs1 = (torch.zeros_like(t) for t in (kc, vc, ks, vs))
        rows = torch.tensor(list(range(L)) + [L + s]).cuda()
        binding.quantize_and_cache(k[rows], v[rows], kc1, vc1, ks1, vs1, torch.arange(L + 1).cuda())
        alone = torch.empty_like(q[:1])
        binding.paged_attention_decode_quantized(alone, q[s:s + 1], kc1, vc1, ks1, vs1, tables[:1], lens[:1], hk, d ** -0.5,
                                                 bs, 3)
        assert float((alone[0].float() - out[s].float()).abs().max()) <= 2.0 ** -7 * float(v.abs().max())
    assert binding.read_device_errors() == 0


def test_block_copy_of_token_scaled_caches_refusals(dry):
    def status(cache):
        try:
            binding.copy_blocks(cache, torch.zeros(3, 2, dtype=torch.int64))
            return 0
        except binding.PkvError as e:
            assert e.message
            return e.status
    z = torch.zeros
    assert status(z(10, 2, 16, 128, dtype=torch.int8)) == 0
    assert status(z(10, 2, 16)) == 0 and status(z(10, 2, 19)[:, :, 1:17]) == 0
    assert status(z(10, 2, 3)) == 2 and status(z(10, 2, 3, 128, dtype=torch.int8)) == 2
    assert status(z(10, 2, 16, dtype=torch.int8)) == 2 and status(z(10, 2, 16, dtype=torch.bfloat16)) == 2
    assert status(z(10, 16, 2).transpose(1, 2)) == 1           # a block's scales side by side
    assert status(z(10, 2)) == 1
