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
    assert ((lse.T.double() - wlse).abs() <= tl).all()


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
