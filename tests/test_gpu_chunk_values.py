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


def test_sequences_that_share_pages():
    """A common prefix held once: the same page ids in several rows of the block table, one of them twice in a row."""
    g = torch.Generator().manual_seed(95)
    d, group, page, lens = 128, 4, 16, [500, 330, 64]
    ctx = pu.context(1, 2, group, d)
    pool = pu.Paged(g, 1, 2, d, page, lens)
    t = pool.table_host
    t[1, :12] = t[0, :12]
    t[2, :4] = [t[0, 3], t[0, 3], t[1, 20], t[0, 0]]
    pool.table = torch.from_numpy(t).cuda()
    new = [30, 1, 64]
    q = pu.bf16(g, (1, sum(new), 2 * group, d), 2.0)
    c = np.concatenate([[0], np.cumsum(new)])
    out = ctx.chunk_attention(pool.K, pool.V, torch.tensor(lens, dtype=torch.int32).cuda(), q,
                              torch.tensor(c, dtype=torch.int32).cuda(), block_table=pool.table)
    assert ctx.get_error()[0] == tri.TRI_OK
    for b, (n, m) in enumerate(zip(new, lens)):
        k, v = pool.rows(pool.K, b, m)[0], pool.rows(pool.V, b, m)[0]
        for h in range(2 * group):
            rows = q[0, c[b]:c[b + 1], h]
            p = ac.weights(rows, k[h // group], m - n + 1, d ** -0.5)
            assert ac.excess(out[0, c[b]:c[b + 1], h], p, rows, k[h // group], v[h // group], d ** -0.5) <= 1.0
    ctx.close()


def test_rows_past_32_bits():
    """Pages whose elements lie beyond the 2^31st (4.3 GB each of keys and values): appended, attended, and a value that is not
    finite hidden from some queries, which are then computed row by row."""
    g = torch.Generator().manual_seed(96)
    d, group, page, n, m = 64, 4, 64, 40, 200
    pages = (1 << 31) // (page * d) + 8
    ctx = pu.context(1, 1, group, d)
    K = torch.empty((1, pages, 1, page, d), dtype=torch.bfloat16, device="cuda")
    V = torch.empty_like(K)
    P = torch.empty((1, pages, 1, page), dtype=torch.int32, device="cuda")
    ids = torch.tensor([pages - 1, 3, pages - 5, pages - 2], dtype=torch.int32)
    table, at = ids[None].cuda(), ids.long().cuda()
    k, v = pu.bf16(g, (1, m, 1, d), 0.6), pu.bf16(g, (1, m, 1, d))
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx.append_chunk(K, V, P, lens, k, v, torch.tensor([0, m], dtype=torch.int32).cuda(), torch.arange(m, dtype=torch.int32).cuda(),
                     block_table=table, rotate=False)
    assert ctx.get_error()[0] == tri.TRI_OK and lens.item() == m
    assert torch.equal(K[0, at, 0].reshape(-1, d)[:m], k[0, :, 0]) and torch.equal(V[0, at, 0].reshape(-1, d)[:m], v[0, :, 0])
    assert torch.equal(P[0, at, 0].reshape(-1)[:m], torch.arange(m, dtype=torch.int32, device="cuda"))
    q = pu.bf16(g, (1, n, group, d), 2.0)
    hidden = m - n + 25
    V[0, at[hidden // page], 0, hidden % page] = float("inf")
    out = ctx.chunk_attention(K, V, lens, q, torch.tensor([0, n], dtype=torch.int32).cuda(), block_table=table)
    assert ctx.get_error()[0] == tri.TRI_OK
    for h in range(group):
        rows = q[0, :25, h]
        p = ac.weights(rows, k[0, :hidden, 0], m - n + 1, d ** -0.5)
        assert ac.excess(out[0, :25, h], p, rows, k[0, :hidden, 0], v[0, :hidden, 0], d ** -0.5) <= 1.0
    assert (~torch.isfinite(out[0, 25:])).all()
    ctx.close()
