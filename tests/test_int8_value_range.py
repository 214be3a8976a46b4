"""Attention over a token-scaled int8 cache when value scales lie far apart: tokens that a
row does not see, or hardly weighs, take nothing from the others, whatever their scale.

Tolerance: that of test_tree_attention.py with another last term.  A product of a weight and
its value scale is rounded to f16 relative to the largest product of the row (at least 2^6 in
those units); from 2^-14 on by half a step, 2^-11 of it, which is the weights' term; a smaller
one is subnormal and off by at most 2^-25, 2^-31 of the row's largest.  With codes of at most 127
that is L 2^-31 * 127 * max_j p_j max(s_j, 2^-80) together (a smaller scale counts as 2^-80)."""
import math

import pytest
import torch
from test_tree_attention import Case, signed

from paged_kv_cache_90_gb300 import binding
from paged_kv_cache_90_gb300 import build as pkv_build

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    binding.load_library()


class Ranged(Case):
    def reference(self):
        self.K64, self.V64 = (self.kc.double() * self.k_scales.double()[..., None],
                              self.vc.double() * self.v_scales.double()[..., None])
        ref = super().reference()
        self.floor = torch.zeros(self.T, self.hk * self.group, 1, dtype=torch.float64)
        for s, L in enumerate(self.lens):
            n, a = self.nodes[s], int(self.starts[s])
            if n == 0 or L == 0:
                continue
            j = torch.arange(L)
            blk = self.tables[s].long()[j // self.bs]
            K, sv = self.K64[blk, :, j % self.bs], self.v_scales[blk, :, j % self.bs].double().abs()   # [L, hk]
            q = self.q[a:a + n].double().view(n, self.hk, self.group, self.d)
            z = (torch.einsum("nhgd,lhd->nhgl", q, K) * self.scale).masked_fill(~self.keep(s)[:, None, None], -math.inf)
            top = z.amax(-1, keepdim=True)
            p = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
            p = p / p.sum(-1, keepdim=True).clamp(min=1.0)
            most = (p * sv.clamp(min=2.0 ** -80).t()[None, :, None]).amax(-1)
            self.floor[a:a + n] = (L * 2.0 ** -31 * 127 * most).reshape(n, -1, 1)
        return ref

    def slot(self, s, j):
        return int(self.tables[s, j // self.bs]), slice(None), j % self.bs

    def hide(self, s, node, alone=False):
        """No row sees sequence s's node (`alone`: only its own row)."""
        a = int(self.starts[s])
        for i in range(self.nodes[s]):
            row = self.rows[a + i]
            row[node // 64] &= ~(1 << (node % 64))
            if alone and i == node:
                row[node // 64] |= 1 << (node % 64)
            self.mask[a + i] = torch.tensor([signed(w) for w in row])

    def same_queries(self):
        """Every row and head of a sequence asks the same, so that a key can be aimed."""
        for s in range(len(self.lens)):
            a, b = int(self.starts[s]), int(self.starts[s + 1])
            if b > a:
                self.q[a:b] = self.q[a, 0].clone()

    def aim(self, s, j, nats, others=False):
        """Sequence s's position j gets a key whose score is `nats` for all its rows (its
        other keys zero)."""
        q = self.q[int(self.starts[s]), 0].double()
        if others:
            for i in range(self.lens[s]):
                self.kc[self.slot(s, i)] = 0
        k = (q * (nats / (self.scale * float(q @ q)))).float()
        top = float(k.abs().max()) / 127
        self.kc[self.slot(s, j)] = torch.round(k / top).to(torch.int8)
        self.k_scales[self.slot(s, j)] = top


GROUPS = [(2, 4, 128), (1, 16, 64), (1, 40, 128)]  # (a warp's, two tiles of heads', the other kernel's)


@gpu
@pytest.mark.parametrize("hk,group,d", [(2, 4, 128), (1, 16, 64)])
@pytest.mark.parametrize("L,n", [(40, 9), (900, 9), (5000, 9), (300, 40)])
def test_scales_of_hidden_nodes_reach_nothing(L, n, hk, group, d):
    """A node that no row sees and one that only its own row sees, their value scales 2^20 to 2^60
    times the others' and a type's largest: the other rows have the bits that they have with scales
    of zero there, and all are right."""
    c = Ranged(L + n, [L, 70], [n, 5], hk, group, d, 16, cache="int8")
    c.hide(0, 2)
    c.hide(0, 5, alone=True)
    two, five = c.slot(0, L - n + 2), c.slot(0, L - n + 5)
    ones = c.v_scales[two].clone(), c.v_scales[five].clone()
    c.v_scales[two], c.v_scales[five] = 0.0, 0.0
    plain = c.call(c.device()).cpu()
    others = [i for i in range(c.T) if i != 5]
    for f, g in ((2.0 ** 20, 2.0 ** 20), (2.0 ** 60, 2.0 ** 40), (2.0 ** 100, 2.0 ** 60)):
        c.v_scales[two], c.v_scales[five] = ones[0] * f, ones[1] * g
        out = c.call(c.device())
        assert torch.equal(out.cpu()[others].view(torch.int16), plain[others].view(torch.int16)), (f, g)
        c.check(out)
    c.v_scales[two] = 3.4e38
    out = c.call(c.device()).cpu()
    assert torch.equal(out[others].view(torch.int16), plain[others].view(torch.int16))
    assert binding.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("hk,group,d", GROUPS)
@pytest.mark.parametrize("power", [10, 22, 40])
def test_a_token_of_little_weight_takes_no_bits(power, hk, group, d, decode):
    """Tokens with weights of 2^-60 and less and values 2^10 to 2^40 times the others', among the first
    and the last and in between."""
    c = Ranged(power, [300, 1100, 33], [4, 3, 5], hk, group, d, 16, cache="int8", decode=decode)
    c.same_queries()
    for s, L in enumerate(c.lens):
        for j in (0, 17, L // 2, L - (7 if decode else 12)):
            c.aim(s, j, -45.0 - power)
            c.v_scales[c.slot(s, j)] = 0.03 * 2.0 ** power
    c.check()


@gpu
@pytest.mark.parametrize("hk,group,d", GROUPS)
def test_equal_weights_beside_a_large_value(hk, group, d):
    """A hundred tokens of equal weight with values near 5e-4, and one of 3e4 at 2^-60 of it."""
    c = Ranged(7, [101], None, hk, group, d, 16, cache="int8", decode=True)
    c.same_queries()
    c.aim(0, 50, -60 * math.log(2.0), others=True)
    for j in range(101):
        c.v_scales[c.slot(0, j)] = 5e-4 / 127
    c.v_scales[c.slot(0, 50)] = 3e4 / 127
    c.vc.fill_(127)
    out = c.call(c.device())
    c.check(out)
    assert float((out.float() - 5e-4).abs().max()) <= 2.0 ** -8 * 5e-4


@gpu
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("hk,group,d", GROUPS)
def test_values_of_little_size_at_a_large_weight(hk, group, d, decode):
    """A token of nearly all the weight whose value is zero or 2^-40 of the others'; a sequence of
    zero values; sequences of values around 2^-60 and 2^60."""
    c = Ranged(8, [400, 130, 50, 260, 260], [5, 6, 7, 3, 3], hk, group, d, 16, cache="int8", decode=decode)
    c.same_queries()
    c.aim(0, 0, 25.0)
    c.v_scales[c.slot(0, 0)] = 0.0
    c.aim(1, 100, 25.0)
    c.v_scales[c.slot(1, 100)] *= 2.0 ** -40
    for j in range(50):
        c.v_scales[c.slot(2, j)] = 0.0
    for j in range(260):
        c.v_scales[c.slot(3, j)] *= 2.0 ** -60
        c.v_scales[c.slot(4, j)] *= 2.0 ** 60
    out = c.call(c.device())
    c.check(out)
    a, b = int(c.starts[2]), int(c.starts[3])
    assert (out[a:b] == 0).all()


@gpu
@pytest.mark.parametrize("hk,group,d", GROUPS)
def test_value_scales_over_many_powers(hk, group, d):
    Ranged(15, [400, 90], [10, 3], hk, group, d, 16, cache="int8", spread=4.0).check()
    Ranged(16, [400, 90, 3000, 1], None, hk, group, d, 16, cache="int8", decode=True, spread=4.0).check()
    Ranged(17, [700, 1500], None, hk, group, d, 32, cache="int8", decode=True, spread=6.0, window=333).check()
