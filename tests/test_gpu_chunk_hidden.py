"""What a query does not see, whatever it holds, takes no part in its attention: special values among the keys and values of later
tokens, at both head widths, against the 64-bit form over what the query does see."""
import math

import numpy as np
import pytest
import torch

import prompt_util as pu
from rope_aware_key_tri_b200 import tri

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _attend(ctx, pool, new, lens, q, causal=True):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    lse = torch.empty(q.shape[:3], device="cuda")
    out = ctx.chunk_attention(pool.K, pool.V, torch.tensor(lens, dtype=torch.int32).cuda(), q, cu, lse=lse, causal=causal,
                              block_table=pool.table)
    assert ctx.get_error()[0] == tri.TRI_OK
    return out, lse


def _check_rows(out, lse, q, k, v, first, scale):
    """Rows out [n][H][d] of queries q [n][H][d] that see the keys [0, first + i) of k, v."""
    qq = q.transpose(0, 1)
    want, wlse = pu.attention(qq, k, v, first, scale)
    ta, tl = pu.attention_bounds(qq, k, v, scale)
    assert ((out.transpose(0, 1).double() - want).abs() <= ta + 2.0 ** -8 * want.abs()).all()
    none = torch.isinf(wlse)  # queries in front of the first row
    assert torch.equal(lse.T.double()[none], wlse[none])
    assert ((lse.T.double() - wlse)[~none].abs() <= tl).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("big", [3e38, -3e38])
def test_a_large_value_of_a_later_token(d, big):
    """At every place among 16 keys: the queries before it do not feel it."""
    g = _gen(70)
    ctx = pu.context(1, 1, 4, d)
    n, m = 40, 100
    q = pu.bf16(g, (1, n, 4, d), 2.0)
    for at in range(72, 90):
        pool = pu.Paged(g, 1, 1, d, 64, [m])
        u, o = pool.places(0, m)
        pool.V[:, u[at], :, o[at]] = big
        out, lse = _attend(ctx, pool, [n], [m], q)
        b = at - (m - n)  # queries before it
        k, v = pool.rows(pool.K, 0, m)[0, 0], pool.rows(pool.V, 0, m)[0, 0]
        _check_rows(out[0, :b], lse[0, :b], q[0, :b], k[:at], v[:at], m - n + 1, d ** -0.5)
    ctx.close()


@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("d", [64, 128])
def test_a_visible_value_that_is_not_finite_costs_no_other_row(d, what):
    """A value row that every query of a prompt sees is not finite in one dim: that dim shows it in every row, every other
    dim and the other sequence are as ever, and no wait runs out meanwhile."""
    g = _gen(71)
    hkv, group = 8, 4
    ctx = pu.context(1, hkv, group, d)
    new, lens = [2048, 5], [2048, 77]
    pool = pu.Paged(g, 1, hkv, d, 64, lens)
    u, o = pool.places(0, 1)
    T = sum(new)
    q = pu.bf16(g, (1, T, hkv * group, d), 2.0)
    clean, clse = _attend(ctx, pool, new, lens, q)
    before = pool.V[:, u, :, o].clone()
    pool.V[:, u, :, o] = torch.cat([before[..., :3], torch.full_like(before[..., 3:4], what), before[..., 4:]], -1)
    out, lse = _attend(ctx, pool, new, lens, q)
    assert torch.equal(lse, clse)
    assert torch.equal(out[:, 2048:], clean[:, 2048:])
    other = torch.arange(d, device="cuda") != 3
    assert torch.equal(out[..., other], clean[..., other])
    hit = out[:, :2048, :, 3]
    # (the weight of slot 0 may round to zero, and zero times infinity is a NaN)
    assert torch.isnan(hit).all() if math.isnan(what) else (~torch.isfinite(hit)).all()
    ctx.close()


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens,group", [([40], [20000], 4), ([300] * 6, [5000] * 6, 8), ([300, 1, 70], [300, 900, 200], 1),
                                            ([20, 3], [8, 500], 2)])
def test_a_value_of_a_later_token_that_is_not_finite(d, what, new, lens, group):
    """In the middle of the first sequence's new tokens, some dims of a value: the tokens before it are as if it were
    not there, in long caches whose blocks are split, with several items a CTA and with more queries than rows."""
    g = _gen(72)
    hkv = 2
    ctx = pu.context(1, hkv, group, d)
    pool = pu.Paged(g, 1, hkv, d, 16, lens)
    n, m = new[0], lens[0]
    T = sum(new)
    q = pu.bf16(g, (1, T, hkv * group, d), 2.0)
    clean, clse = _attend(ctx, pool, new, lens, q)
    at = m - n + n // 2 if m > n else m // 2
    u, o = pool.places(0, m)
    dims = torch.tensor([0, 5, 31, 32, d - 1])
    for x in dims.tolist():
        pool.V[:, u[at], :, o[at], x] = what
    out, lse = _attend(ctx, pool, new, lens, q)
    assert torch.equal(lse, clse)
    first = at - (m - n)  # the first query that sees it
    k, v = pool.rows(pool.K, 0, m)[0], pool.rows(pool.V, 0, m)[0]
    for h in range(hkv):
        s = slice(h * group, h * group + group)
        _check_rows(out[0, :first, s], lse[0, :first, s], q[0, :first, s], k[h, :at], v[h, :at], m - n + 1, d ** -0.5)
    # dims that it does not touch, tokens that see it and other sequences: bit for bit what they were
    keep = torch.ones(d, dtype=torch.bool)
    keep[dims] = False
    keep = keep.cuda()
    assert torch.equal(out[..., keep], clean[..., keep]) and torch.equal(out[:, n:], clean[:, n:])
    seen = out[:, first:n][..., ~keep]
    assert (~torch.isfinite(seen)).all()
    ctx.close()


@pytest.mark.parametrize("split", [False, True])
def test_a_key_and_values_of_later_tokens_at_head_128(split):
    """An infinite value, a NaN key and a NaN value in the middle of the chunk: the queries before them as if they were not
    there, those that see the infinity alone infinite, those that see a NaN all NaN."""
    n, m = (40, 3000) if split else (40, 100)
    new, lens = ([n], [m]) if split else ([n, 7], [m, 9])
    pool = pu.Paged(_gen(73), 1, 1, 128, 64, lens)
    u, o = pool.places(0, m)
    at = m - n + 20
    ctx = pu.context(1, 1, 4, 128)
    q = pu.bf16(_gen(74), (1, sum(new), 4, 128), 0.05)  # even weights: none of them rounds to zero
    pool.V[:, u[at], :, o[at]] = math.inf
    pool.K[:, u[at + 5], :, o[at + 5]] = math.nan
    pool.V[:, u[at + 7], :, o[at + 7]] = math.nan
    out, lse = _attend(ctx, pool, new, lens, q)
    k, v = pool.rows(pool.K, 0, m)[0, 0], pool.rows(pool.V, 0, m)[0, 0]
    _check_rows(out[0, :20], lse[0, :20], q[0, :20], k[:at], v[:at], m - n + 1, 128 ** -0.5)
    assert torch.isinf(out[0, 20:25]).all() and torch.isnan(out[0, 25:n]).all()
    if not split:
        assert torch.isfinite(out[0, n:]).all()
    ctx.close()


@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_a_key_that_is_not_finite_shows_at_head_128(what):
    """Whatever its place among the keys (the exponential is evaluated in two ways there): NaN results."""
    ctx = pu.context(1, 1, 4, 128)
    n, m = 3, 400
    q = torch.full((1, n, 4, 128), 1.0, dtype=torch.bfloat16, device="cuda")
    for at in list(range(0, 18)) + [63, 64, 127, 128, 200, 301, 396]:
        pool = pu.Paged(_gen(75), 1, 1, 128, 64, [m])
        u, o = pool.places(0, m)
        pool.K[:, u[at], :, o[at]] = what
        out, lse = _attend(ctx, pool, [n], [m], q)
        assert torch.isnan(out).all() and torch.isnan(lse).all(), at
    ctx.close()
