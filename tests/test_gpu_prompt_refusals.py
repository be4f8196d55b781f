"""Calls of the prompt side that are refused on the host: the outputs stay as they were."""
import math

import pytest
import torch

import prompt_util as pu
from rope_aware_key_tri_b200 import tri

pytestmark = pytest.mark.gpu


class Case:
    """One attention and one append call of 8 tokens of two sequences, made with what is changed."""

    def __init__(self, L=1):
        g = torch.Generator().manual_seed(100)
        self.ctx = pu.context(2, 2, 2, 64)
        self.pool = pu.Paged(g, L, 2, 64, 16, [40, 40])
        self.q = pu.bf16(g, (L, 8, 4, 64))
        self.cu = torch.tensor([0, 4, 8], dtype=torch.int32).cuda()
        self.lens = torch.tensor([20, 30], dtype=torch.int32).cuda()
        self.pos = torch.arange(8, dtype=torch.int32).cuda()
        self.out = torch.full((L, 8, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        self.before = [x.clone() for x in self._all()]

    def _all(self):
        p = self.pool
        return p.K, p.V, p.P, self.q, self.lens, self.out

    def attend(self, **kw):
        a = dict(q=self.q, cu_q=self.cu, out=self.out, block_table=self.pool.table, check=False)
        a.update(kw)
        return self.ctx.chunk_attention(self.pool.K, self.pool.V, self.lens, **a)

    def append(self, **kw):
        a = dict(K_new=self.q[:, :, :2], V_new=self.q[:, :, 2:], cu_new=self.cu, pos_new=self.pos, block_table=self.pool.table,
                 check=False)
        a.update(kw)
        return self.ctx.append_chunk(self.pool.K, self.pool.V, self.pool.P, self.lens, **a)

    def unchanged(self):
        torch.cuda.synchronize()
        assert self.ctx.get_error()[0] == tri.TRI_OK
        assert all(torch.equal(a, b) for a, b in zip(self.before, self._all()))
        self.ctx.close()


def test_scales_that_fp32_does_not_hold():
    c = Case()
    for scale in (1e-300, 1e-46, 2.0 ** -128, 1e39, 1e300, 5e-324):
        assert c.attend(scale=scale) == tri.TRI_EINVAL, scale
    c.unchanged()


def test_the_smallest_scale():
    """All weights equal: the mean of the values that each query sees (bf16: half a step of the result, and fp32 sums)."""
    c = Case()
    assert c.attend(scale=2.0 ** -126) == tri.TRI_OK
    for b, m in enumerate((20, 30)):
        v = c.pool.rows(c.pool.V, b, m)[0].double()
        for i in range(4):
            want = v[:, :m - 3 + i].mean(1)
            got = c.out[0, 4 * b + i].double().view(2, 2, 64)
            assert ((got - want[:, None]).abs() <= 2.0 ** -8 * want.abs()[:, None] + 2.0 ** -18 * v.abs().max()).all()
    c.ctx.close()


def test_layers_past_the_statistics():
    """Also where the sum of the first layer and their number does not fit an int."""
    c = Case()
    p = c.pool
    for first in (2, 3, 2**31 - 1):
        assert c.attend(layer_begin=first) == tri.TRI_EINVAL
        assert c.append(layer_begin=first) == tri.TRI_EINVAL
        t = torch.full((2,), 99, dtype=torch.int32, device="cuda")
        kw = dict(block_table=p.table, layer_begin=first, check=False)
        assert c.ctx.prune(p.K, p.V, p.P, c.lens, t, 8, **kw) == tri.TRI_EINVAL
        assert c.ctx.prune_noalloc(p.K, p.V, p.P, c.lens, t, 8, **kw) == tri.TRI_EINVAL
        assert c.ctx.score(p.K, c.lens, t, **kw) == tri.TRI_EINVAL
        assert c.ctx.decode_attention(p.K, p.V, c.lens, c.q[:, :2].contiguous(), **kw) == tri.TRI_EINVAL
        assert c.ctx.append(p.K, p.V, p.P, c.lens, p.table, c.q[:, :2, :2].contiguous(), c.q[:, :2, 2:].contiguous(),
                            c.pos[:2].contiguous(), layer_begin=first, check=False) == tri.TRI_EINVAL
    c.unchanged()


def test_outputs_that_lie_on_their_inputs():
    """Interleaved with them, or in place where a call allows it, they are taken."""
    c = Case(L=2)
    q, hit = c.q, tri.TRI_EINVAL
    assert c.attend(out=q) == hit
    wide = torch.zeros((2, 16, 12, 64), dtype=torch.bfloat16, device="cuda")
    wide[:, :8, :4] = q
    x = wide[:, :8, :4]
    for other in (wide[:, :8, 1:5], wide[:, 1:9, :4], wide[:, 7:15, 3:7], wide[:, :8, 3:7]):  # on some of its rows
        assert c.attend(q=x, out=other) == hit
        assert c.attend(q=other, out=x) == hit
        assert c.ctx.rope(x, c.pos, out=other, check=False) == hit
        assert c.append(q=x, q_out=other) == hit
    flat = wide.view(-1)
    shifted = flat[8:8 + q.numel()].view(2, 8, 4, 64)
    assert c.attend(q=flat[:q.numel()].view(2, 8, 4, 64), out=shifted) == hit  # off by eight elements
    assert c.ctx.rope(flat[:4096].view(2, 8, 4, 64), c.pos, out=flat[:4096].view(2, 4, 8, 64).transpose(1, 2), check=False) == hit
    c.unchanged()
    # rows beside one another in one buffer
    c = Case(L=2)
    wide = torch.zeros((2, 16, 12, 64), dtype=torch.bfloat16, device="cuda")
    wide[:, :8, :4] = c.q
    x = wide[:, :8, :4]
    want = c.out.clone()
    assert c.attend(out=want) == tri.TRI_OK
    for other in (wide[:, :8, 4:8], wide[:, :8, 8:12], wide[:, 8:, :4], wide[:, 8:, 2:6]):
        assert c.attend(q=x, out=other) == tri.TRI_OK
        assert torch.equal(other, want) and torch.equal(x, c.q)
    turned = c.ctx.rope(c.q, c.pos)
    assert c.ctx.rope(x, c.pos, out=wide[:, 8:, 8:12], check=False) == tri.TRI_OK
    assert torch.equal(wide[:, 8:, 8:12], turned)
    assert c.ctx.rope(x, c.pos, out=x, check=False) == tri.TRI_OK and torch.equal(x, turned)
    c.ctx.close()


def test_rotary_tables_that_the_arithmetic_does_not_hold():
    """Magnitudes that are nothing or infinite in fp32, either way round, and frequencies whose angle is: refused, and the table
    before them stays."""
    c = Case()
    omega, _ = tri.rope_frequencies(64, 1e4)
    c.ctx.rope_load(omega, pu.HALF, 2.0 ** 126)
    c.ctx.rope_load(omega, pu.HALF, 2.0 ** -126)
    c.ctx.rope_load(omega, pu.HALF, 2.0)
    for magnitude in (1e-300, 2.0 ** -127, 2.0 ** 127, 1e300, math.inf, math.nan, 0.0, -1.0):
        with pytest.raises(tri.TriError) as e:
            c.ctx.rope_load(omega, pu.HALF, magnitude)
        assert e.value.status == tri.TRI_EINVAL
    for w in (1e300, -1e308, math.inf):
        with pytest.raises(tri.TriError):
            c.ctx.rope_load(omega + w, pu.HALF)
    # position 0: the magnitude alone
    assert torch.equal(c.ctx.rope(c.q, torch.zeros_like(c.pos)), c.q * 2)
    assert torch.equal(c.ctx.rope(c.q, torch.zeros_like(c.pos), inverse=True), c.q / 2)
    c.unchanged()
