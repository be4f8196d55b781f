"""Chunk attention row by row at the tolerance of attention_check, which a value tile or a 16-row piece in the wrong place does not pass:
long caches whose blocks are split and joined, pairs of warpgroups on one query tile, every page size, both head widths."""
import numpy as np
import pytest
import torch

import attention_check as ac
import prompt_util as pu
from rope_aware_key_tri_b200 import tri

pytestmark = pytest.mark.gpu


def _run(seed, L, hkv, group, d, page, new, lens, causal=True, aim=False):
    g = torch.Generator().manual_seed(seed)
    ctx = pu.context(L, hkv, group, d)
    pool = pu.Paged(g, L, hkv, d, page, lens)
    T, hq = sum(new), hkv * group
    q = pu.bf16(g, (L, T, hq, d), 2.0)
    c = np.concatenate([[0], np.cumsum(new)])
    if aim:  # the rows of a KV head aim at the keys in turn
        for b, (n, m) in enumerate(zip(new, lens)):
            k = pool.rows(pool.K, b, m)
            all_see = m - n + 1 if causal else m
            for l in range(L):
                for h in range(hkv):
                    at = torch.arange(n * group, device="cuda") * (all_see // 2 + 1 if n * group < 64 else 1) % all_see
                    q[l, c[b]:c[b + 1], h * group:h * group + group] = ac.aimed(k[l, h], at).view(n, group, d)
    cu = torch.tensor(c, dtype=torch.int32).cuda()
    out = ctx.chunk_attention(pool.K, pool.V, torch.tensor(lens, dtype=torch.int32).cuda(), q, cu, causal=causal,
                              block_table=pool.table)
    assert ctx.get_error()[0] == tri.TRI_OK
    scale = d ** -0.5
    for b, (n, m) in enumerate(zip(new, lens)):
        k, v = pool.rows(pool.K, b, m), pool.rows(pool.V, b, m)
        for l in range(L):
            for h in range(hq):
                rows, kv = q[l, c[b]:c[b + 1], h], h // group
                p = ac.weights(rows, k[l, kv], m - n + 1 if causal else None, scale)
                assert ac.excess(out[l, c[b]:c[b + 1], h], p, rows, k[l, kv], v[l, kv], scale) <= 1.0, (b, l, h)
    ctx.close()


@pytest.mark.parametrize("aim", [False, True], ids=["spread", "aimed"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,page,new,lens", [
    (8, 64, [1], [9000]), (4, 0, [1], [9000]),             # one token: parts joined, two warpgroups on a tile
    (8, 16, [17, 1], [5000, 8191]), (1, 48, [300], [7777]),  # few rows, odd lengths
    (4, 0, [1] * 16, [2176] * 16),                         # single tokens of a batch
    (4, 64, [5] * 8, [3200, 3100, 2053, 2900, 3199, 2176, 2500, 2048]),
    (8, 16, [300], [2600]), (2, 128, [700, 1, 64], [3000, 4000, 64])])
def test_values(group, page, new, lens, d, aim):
    _run(90 + d + group, 1, 2, group, d, page, new, lens, aim=aim)


@pytest.mark.parametrize("d", [64, 128])
def test_values_of_layers_without_a_mask(d):
    _run(91, 3, 2, 2, d, 32, [40, 3, 129], [1000, 2500, 600], causal=False, aim=True)
    _run(92, 2, 8, 1, d, 80, [256], [4096], causal=False)
