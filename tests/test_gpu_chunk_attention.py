"""Attention of chunks of new tokens over the cache on the GPU, through the C ABI, against the 64-bit form, with tolerances
derived in prompt_util.attention_bounds."""
import math

import numpy as np
import pytest
import torch

import prompt_util as pu
import tri_synth as ts
import gpu_util as gu
from rope_aware_key_tri_b200 import tri

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _check(pool, q, new, lens, out, lse, causal, scale, group, skip=()):
    c = np.concatenate([[0], np.cumsum(new)])
    worst = 0.0
    for b, (n, m) in enumerate(zip(new, lens)):
        if n == 0 or b in skip:
            continue
        t = slice(int(c[b]), int(c[b + 1]))
        k, v = pool.rows(pool.K, b, m), pool.rows(pool.V, b, m)
        for l in range(pool.L):
            for g in range(pool.hkv):
                h = slice(g * group, g * group + group)
                qq = q[l, t, h].transpose(0, 1)
                want, wlse = pu.attention(qq, k[l, g], v[l, g], m - n + 1 if causal else None, scale)
                ta, tl = pu.attention_bounds(qq, k[l, g], v[l, g], scale)
                got, glse = out[l, t, h].transpose(0, 1).double(), lse[l, t, h].transpose(0, 1).double()
                err = (got - want).abs()
                tol = ta + 2.0 ** -8 * want.abs()
                assert (err <= tol).all(), (b, l, g, n, m, float(err.max()), ta)
                none = torch.isinf(wlse)
                assert torch.equal(torch.isinf(glse) & (glse < 0), none) and (got[none] == 0).all()
                assert ((glse - wlse)[~none].abs() <= tl).all(), (b, l, g, float((glse - wlse)[~none].abs().max()), tl)
                worst = max(worst, float((err / tol.clamp_min(1e-30)).max()))
    return worst


def _run(seed, L, hkv, group, d, page, new, lens, causal=True, scale=None, T_extra=0, ctx=None, pool=None, spare=2, q=None):
    g = _gen(seed)
    own = ctx is None
    ctx = ctx or pu.context(L, hkv, group, d)
    pool = pool or pu.Paged(g, L, hkv, d, page, lens, spare=spare)
    T, hq = sum(new) + T_extra, hkv * group
    q = pu.bf16(g, (L, T, hq, d), 2.0) if q is None else q
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    lens_dev = torch.tensor(lens, dtype=torch.int32).cuda()
    out = torch.full((L, T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((L, T, hq), 7.0, device="cuda")
    ctx.chunk_attention(pool.K, pool.V, lens_dev, q, cu, out=out, lse=lse, scale=scale, causal=causal, block_table=pool.table)
    st = ctx.get_error()
    assert st[0] == tri.TRI_OK, st
    if T_extra:
        assert (out[:, -T_extra:] == 7.0).all() and (lse[:, -T_extra:] == 7.0).all()
    worst = _check(pool, q, new, lens, out, lse, causal, d ** -0.5 if scale is None else scale, group)
    if own:
        ctx.close()
    return worst, out, lse, pool, q


def test_one_tile():
    _run(30, 1, 1, 1, 128, 0, [128], [128], causal=False)
    _run(31, 1, 1, 1, 64, 0, [128], [128], causal=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("causal", [True, False])
def test_shapes(d, group, causal):
    _run(32 + d + group, 2, 2, group, d, 64, [1, 0, 5, 130, 64, 300, 33], [1, 9, 5, 130, 700, 333, 1000], causal, T_extra=5)


@pytest.mark.parametrize("page", [0, 16, 32, 48, 64, 128, 80])
def test_pages(page):
    _run(33 + page, 1, 2, 4, 64, page, [3, 70, 1, 128], [257, 70, 129, 900])
    _run(34 + page, 1, 1, 2, 128, page, [3, 70, 1, 128], [257, 70, 129, 900])


def test_lengths_around_a_tile():
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 384, 385]
    _run(35, 1, 1, 4, 128, 64, [1] * len(lens), lens)
    _run(36, 1, 1, 4, 64, 16, lens, lens)
    _run(37, 1, 1, 8, 128, 16, lens, [n + 100 for n in lens], causal=False)


def test_empty_rows():
    """Sequences without rows, and queries in front of the first row (a cache pruned shorter than the chunk)."""
    _run(38, 1, 2, 2, 64, 64, [3, 40, 300, 200, 0], [0, 8, 1, 130, 5])
    _run(39, 1, 2, 2, 128, 0, [3, 40, 300, 200, 0], [0, 8, 1, 130, 5])
    _run(40, 1, 2, 2, 128, 0, [3, 40], [0, 8], causal=False)


@pytest.mark.parametrize("d", [64, 128])
def test_split_over_the_keys(d):
    """Few rows and long caches: the items are split and their parts merged."""
    _run(41, 1, 1, 4, d, 64, [1], [9000])
    _run(42, 1, 1, 8, d, 64, [17, 1], [5000, 8191])
    _run(43, 1, 2, 1, d, 0, [300], [7777])
    _run(44, 2, 1, 4, d, 16, [100], [6000], causal=False)


def test_many_sequences():
    rng = np.random.default_rng(3)
    new = rng.integers(0, 4, 600).tolist()
    lens = [int(n + x) for n, x in zip(new, rng.integers(0, 40, 600))]
    _run(45, 1, 1, 2, 64, 16, new, lens)


def test_mixed_lengths_and_scale():
    _run(46, 1, 2, 4, 128, 64, [1, 1, 513, 1, 40], [3000, 1, 513, 77, 2000], scale=0.3)
    _run(47, 1, 2, 4, 128, 64, [1, 1, 513, 1, 40], [3000, 1, 513, 77, 2000], scale=1e-4)


def test_growing_logits():
    """Logits that grow along the keys by far more than a tile's rescale threshold, and fall again."""
    g = _gen(48)
    for d, sign in ((128, 1), (64, 1), (128, -1)):
        pool = pu.Paged(g, 1, 1, d, 64, [1500])
        ramp = torch.linspace(-1, 1, 1500) * sign
        u, o = pool.places(0, 1500)
        k = (ramp[:, None] * torch.ones(d)).to(torch.bfloat16).cuda()
        pool.K[:, u.cuda(), :, o.cuda()] = k[:, None, None]
        q = torch.full((1, 200, 2, d), 6.0, dtype=torch.bfloat16, device="cuda")
        _run(49, 1, 1, 2, d, 64, [200], [1500], pool=pool, q=q)


@pytest.mark.parametrize("page", [0, 64])
def test_what_is_not_seen_may_be_nan(page):
    """Rows past the length (in the last page, or in a dense cache) hold NaN and infinities."""
    new, lens = [5, 60, 1], [100, 60, 513]
    pool = pu.Paged(_gen(50), 1, 2, 128, page, lens)
    keep = torch.zeros(pool.K.shape[:4], dtype=torch.bool, device="cuda")
    for b, m in enumerate(lens):
        u, o = pool.places(b, m)
        keep[:, u.cuda(), :, o.cuda()] = True
    for x, bad in ((pool.K, math.nan), (pool.V, math.nan)):
        x[~keep] = bad
    _run(51, 1, 2, 4, 128, page, new, lens, pool=pool)
    pool.V[~keep] = math.inf
    pool.K[~keep] = -math.inf
    _run(52, 1, 2, 4, 128, page, new, lens, pool=pool)


@pytest.mark.parametrize("split", [False, True])
def test_values_that_later_queries_see_are_nan(split):
    """A NaN or infinite value row in the middle of the chunk: the queries before it are as if it were not there."""
    n, m = (40, 3000) if split else (40, 100)
    new, lens = ([n], [m]) if split else ([n, 7], [m, 9])
    pool = pu.Paged(_gen(53), 1, 1, 64, 64, lens)
    u, o = pool.places(0, m)
    at = m - n + 20
    pool.V[:, u[at], :, o[at]] = math.inf
    pool.K[:, u[at + 5], :, o[at + 5]] = math.nan
    pool.V[:, u[at + 7], :, o[at + 7]] = math.nan
    ctx = pu.context(1, 1, 4, 64)
    T = sum(new)
    q = pu.bf16(_gen(54), (1, T, 4, 64), 2.0)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    lse = torch.empty((1, T, 4), device="cuda")
    out = ctx.chunk_attention(pool.K, pool.V, torch.tensor(lens, dtype=torch.int32).cuda(), q, cu, lse=lse,
                              block_table=pool.table)
    assert ctx.get_error()[0] == tri.TRI_OK
    k, v = pool.rows(pool.K, 0, m)[0, 0], pool.rows(pool.V, 0, m)[0, 0]
    want, wlse = pu.attention(q[0, :20].transpose(0, 1), k[:at], v[:at], m - n + 1, 0.125)
    ta, tl = pu.attention_bounds(q[0, :20].transpose(0, 1), k[:at], v[:at], 0.125)
    got = out[0, :20].transpose(0, 1).double()
    assert ((got - want).abs() <= ta + 2.0 ** -8 * want.abs()).all()
    assert ((lse[0, :20].T.double() - wlse).abs() <= tl).all()
    assert torch.isinf(out[0, 20:25]).all()      # they see the infinity
    assert torch.isnan(out[0, 25:n]).all()       # and then the NaN key
    if not split:
        assert torch.isfinite(out[0, n:]).all()
    ctx.close()


def test_strided_rows_and_no_lse():
    g = _gen(55)
    ctx = pu.context(2, 2, 4, 64)
    pool = pu.Paged(g, 2, 2, 64, 16, [50, 80])
    wide = pu.bf16(g, (2, 60, 12, 64), 2.0)
    q = wide[:, :, 2:10]
    cu = torch.tensor([0, 20, 60], dtype=torch.int32).cuda()
    lens = torch.tensor([50, 80], dtype=torch.int32).cuda()
    buf = torch.full((8, 60, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")  # heads outermost
    out = buf.permute(2, 1, 0, 3)
    ctx.chunk_attention(pool.K, pool.V, lens, q, cu, out=out, block_table=pool.table)
    plain = torch.empty((2, 60, 8, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((2, 60, 8), device="cuda")
    ctx.chunk_attention(pool.K, pool.V, lens, q.contiguous(), cu, out=plain, lse=lse, block_table=pool.table)
    assert ctx.get_error()[0] == tri.TRI_OK
    assert torch.equal(out, plain)
    _check(pool, q, [20, 40], [50, 80], out, lse, True, 0.125, 4)
    ctx.close()


def test_single_tokens_agree_with_decode_attention():
    """The same attention as tri_decode_attention, rounded to bf16."""
    spec = ts.CacheSpec(name="one", head_dim=128, group=4, n_kv_heads=2, n_layers=2, batch=5, rope_base=1e6, budget=64,
                        offsets=(1,), positions="from_zero", lens=(1, 17, 500, 64, 129), key_sigma=(0.1, 0.6), cap=512)
    cache = ts.make_cache(spec, 56).to("cuda")
    ctx = gu.context_for(cache)
    q = pu.bf16(_gen(57), (2, 5, 8, 128), 2.0)
    a = ctx.decode_attention(cache.K, cache.V, cache.lens, q)
    b = ctx.chunk_attention(cache.K, cache.V, cache.lens, q, torch.arange(6, dtype=torch.int32).cuda())
    assert ctx.get_error()[0] == tri.TRI_OK
    vmax = float(cache.V.float().abs().nan_to_num(0.0).max())  # rows past the lengths are NaN
    # weights rounded to bf16, the result once more; both kernels' fp32 errors are far below
    assert ((a - b.float()).abs() <= (2.0 ** -8 + 2.0 ** -12) * vmax + 2.0 ** -8 * a.abs()).all()
    ctx.close()


def test_results_do_not_depend_on_the_order_of_parts():
    _, a, la, pool, q = _run(58, 1, 2, 4, 128, 64, [3, 200], [20000, 5000])
    for _ in range(5):
        _, b, lb, _, _ = _run(58, 1, 2, 4, 128, 64, [3, 200], [20000, 5000], pool=pool, q=q)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_refused_sequences_are_not_written():
    g = _gen(59)
    ctx = pu.context(1, 1, 2, 64)
    new, lens = [4, 5, 6], [40, 50, 60]
    pool = pu.Paged(g, 1, 1, 64, 16, lens)
    pool.table[1, 2] = pool.n_pages
    q = pu.bf16(g, (1, 15, 2, 64))
    cu = torch.tensor([0, 4, 9, 15], dtype=torch.int32).cuda()
    lens_dev = torch.tensor(lens, dtype=torch.int32).cuda()
    out = torch.full((1, 15, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, 15, 2), 7.0, device="cuda")
    ctx.chunk_attention(pool.K, pool.V, lens_dev, q, cu, out=out, lse=lse, block_table=pool.table)
    st, code, unit = ctx.get_error()
    assert (st, code, unit) == (tri.TRI_EDEVICE, tri.TRI_DEV_BAD_PAGE, 1)
    assert (out[:, 4:9] == 7.0).all() and (lse[:, 4:9] == 7.0).all()
    _check(pool, q, new, lens, out, lse, True, 0.125, 2, skip=(1,))
    lens_dev[2] = pool.table.shape[1] * 16 + 1
    ctx.chunk_attention(pool.K, pool.V, lens_dev, q, cu, out=out, lse=lse, block_table=pool.table)
    st, code, unit = ctx.get_error()
    assert (st, code) == (tri.TRI_EDEVICE, tri.TRI_DEV_BAD_PAGE) or (st, code, unit) == (
        tri.TRI_EDEVICE, tri.TRI_DEV_LEN_GT_CAP, 2)  # the first of two problems
    lens_dev[2] = 60
    pool.table[1, 2] = int(pool.table_host[1, 2])
    for bad in ([0, 9, 4, 15], [0, 4, 9, 16], [-1, 4, 9, 15]):
        out.fill_(7.0)
        ctx.chunk_attention(pool.K, pool.V, lens_dev, q, torch.tensor(bad, dtype=torch.int32).cuda(), out=out, lse=lse,
                            block_table=pool.table)
        st, code, _ = ctx.get_error()
        assert st == tri.TRI_EDEVICE and code == tri.TRI_DEV_BAD_RANGE
        assert (out == 7.0).all()
    ctx.close()


def test_a_wait_that_runs_out_ends_the_call():
    """A key tile that is armed but never loaded (test hook): the waits run out, the status says so, and the next call works."""
    g = _gen(60)
    ctx = pu.context(1, 2, 2, 64)
    pool = pu.Paged(g, 1, 2, 64, 16, [300, 40])
    q = pu.bf16(g, (1, 30, 4, 64), 2.0)
    cu = torch.tensor([0, 20, 30], dtype=torch.int32).cuda()
    lens = torch.tensor([300, 40], dtype=torch.int32).cuda()
    ctx.set_test_fault(unit=1, wait_tries=20)
    ctx.chunk_attention(pool.K, pool.V, lens, q, cu, block_table=pool.table)
    st, code, unit = ctx.get_error()
    assert (st, code) == (tri.TRI_EDEVICE, tri.TRI_DEV_TIMEOUT) and unit == 1
    ctx.set_test_fault()
    _run(60, 1, 2, 2, 64, 16, [20, 10], [300, 40], ctx=ctx, pool=pool)
    ctx.close()


def test_prompt_decode_prune_together():
    """A serving step as it is used: prompts appended with the rotation and attended, the cache pruned, drafted tokens
    appended at positions past the pruned length and attended over what was kept; the second half captured in a CUDA graph
    and replayed."""
    L, hkv, G, d, page = 2, 2, 4, 64, 16
    g = _gen(61)
    ctx = pu.context(L, hkv, G, d, pu.HALF, 1e4)
    prompts, budget, drafted = [150, 77, 300], 64, [4, 1, 7]
    pool = pu.Paged(g, L, hkv, d, page, [p + 16 for p in prompts])
    omega = 1e4 ** (-2.0 * np.arange(d // 2) / d)
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")

    def tokens(counts, first):
        T = sum(counts)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
        pos = torch.cat([torch.arange(n) + f for n, f in zip(counts, first)]).int().cuda()
        return cu, pos, pu.bf16(g, (L, T, hkv * G + 2 * hkv, d))

    def parts(qkv):
        return qkv[:, :, :hkv * G], qkv[:, :, hkv * G:hkv * G + hkv], qkv[:, :, hkv * G + hkv:]

    cu, pos, qkv = tokens(prompts, [0, 0, 0])
    q, k, v = parts(qkv)
    qr = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    ctx.append_chunk(pool.K, pool.V, pool.P, lens, k, v, cu, pos, block_table=pool.table, q=q, q_out=qr)
    lse = torch.empty((L, sum(prompts), hkv * G), device="cuda")
    out = ctx.chunk_attention(pool.K, pool.V, lens, qr, cu, lse=lse, block_table=pool.table)
    assert ctx.get_error()[0] == tri.TRI_OK and lens.tolist() == prompts
    want = pu.rotate(q.double(), pos, omega, pu.HALF)
    assert ((qr.double() - want).abs() <= pu.rope_error_bound(q.double(), want, d, pu.HALF)).all()
    _check(pool, qr, prompts, prompts, out, lse, True, 0.125, G)
    # statistics for the prune (those of the context are zero): any will do
    rng = np.random.default_rng(4)
    ctx.calibrate_load(L, hkv, G, d, 1e4, pu.HALF, rng.normal(size=(L, hkv * G, d)),
                       np.full((L, hkv * G, d // 2), 2.0), np.full((L, hkv * G, d // 2), 0.5), [1, 2, 4])
    ctx.prune(pool.K, pool.V, pool.P, lens, torch.tensor(prompts, dtype=torch.int32).cuda(), budget, block_table=pool.table)
    assert ctx.get_error()[0] == tri.TRI_OK and lens.tolist() == [budget] * 3
    kept = lens.clone()
    cu, pos, qkv = tokens(drafted, prompts)
    q, k, v = parts(qkv)
    qr, out = (torch.empty((L, sum(drafted), hkv * G, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.empty((L, sum(drafted), hkv * G), device="cuda")
    after = torch.empty_like(lens)

    def step():
        ctx.append_chunk(pool.K, pool.V, pool.P, kept, k, v, cu, pos, block_table=pool.table, lens_out=after, q=q, q_out=qr)
        ctx.chunk_attention(pool.K, pool.V, after, qr, cu, out=out, lse=lse, block_table=pool.table)

    step()
    assert ctx.get_error()[0] == tri.TRI_OK
    first = [x.clone() for x in (qr, out, lse, after, pool.K, pool.P)]
    _check(pool, qr, drafted, [budget + n for n in drafted], out, lse, True, 0.125, G)
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        step()
    # an eager call of a larger shape in between makes the workspace grow: the graph keeps its own
    big = [200] * 40
    _run(62, 1, hkv, G, d, page, big, [300] * 40, ctx=ctx)
    for x in (qr, out, lse, after):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert ctx.get_error()[0] == tri.TRI_OK
    assert all(torch.equal(a, b) for a, b in zip(first, (qr, out, lse, after, pool.K, pool.P)))
    # other drafted tokens in the same buffers
    qkv.copy_(pu.bf16(g, tuple(qkv.shape)))
    graph.replay()
    assert ctx.get_error()[0] == tri.TRI_OK
    _check(pool, qr, drafted, [budget + n for n in drafted], out, lse, True, 0.125, G)
    del graph
    ctx.close()


def test_arguments_are_refused():
    """Every refusal is decided on the host: nothing is launched (the outputs stay)."""
    g = _gen(63)
    ctx = pu.context(2, 2, 2, 64)
    pool = pu.Paged(g, 1, 2, 64, 16, [40, 40])
    q = pu.bf16(g, (1, 8, 4, 64))
    cu = torch.tensor([0, 4, 8], dtype=torch.int32).cuda()
    lens = torch.tensor([40, 40], dtype=torch.int32).cuda()
    out = torch.full((1, 8, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(8, dtype=torch.int32).cuda()

    def att(code, **kw):
        a = dict(q=q, cu_q=cu, out=out, block_table=pool.table)
        a.update(kw)
        assert ctx.chunk_attention(pool.K, pool.V, lens, check=False, **a) == code, kw

    for scale in (0.0, -1.0, math.inf, math.nan):
        att(tri.TRI_EINVAL, scale=scale)
    att(tri.TRI_EINVAL, layer_begin=2)
    att(tri.TRI_EINVAL, q=q[:, :, :1].expand(1, 8, 4, 64))                  # q rows overlap
    att(tri.TRI_EINVAL, out=out[:, :, :1].expand(1, 8, 4, 64))
    att(tri.TRI_EINVAL, q=pu.bf16(g, (1, 8, 4 * 66))[..., :256 + 8].as_strided((1, 8, 4, 64), (2112, 264, 66, 1)))
    off = torch.zeros(8 * 4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    att(tri.TRI_EINVAL, q=off[1:1 + 8 * 4 * 64].view(1, 8, 4, 64))           # base not aligned
    for bad in (dict(q=q[..., :32]), dict(cu_q=cu[:2]), dict(cu_q=cu.long()), dict(out=out.float()), dict(q=q.cpu()),
                dict(lse=torch.zeros(3, device="cuda")), dict(q=pu.bf16(g, (1, 8, 2, 64)), out=out[:, :, :2])):
        with pytest.raises(ValueError):
            att(None, **bad)

    def app(code, **kw):
        a = dict(K_new=q[:, :, :2], V_new=q[:, :, 2:], cu_new=cu, pos_new=pos, block_table=pool.table)
        a.update(kw)
        assert ctx.append_chunk(pool.K, pool.V, pool.P, lens, check=False, **a) == code, kw

    before = [x.clone() for x in (pool.K, pool.V, pool.P, lens)]
    app(tri.TRI_EINVAL, rotate=False, q=q)                                   # queries without a rotation
    app(tri.TRI_EINVAL, q=q, q_out=out[:, :, :1].expand(1, 8, 4, 64))
    app(tri.TRI_EINVAL, lens_out=None)
    app(tri.TRI_EINVAL, layer_begin=2)
    for bad in (dict(K_new=q), dict(pos_new=pos[:3]), dict(cu_new=cu[:1]), dict(V_new=q[:, :4, 2:])):
        with pytest.raises(ValueError):
            app(None, **bad)
    omega, _ = tri.rope_frequencies(128, 1e4)
    ctx.rope_load(omega, pu.HALF)
    app(tri.TRI_EINVAL)                                                      # 128 rotated dims in a head of 64
    assert ctx.rope(q, pos, check=False) == tri.TRI_EINVAL
    with pytest.raises(tri.TriError):
        ctx.rope_load(omega, 2)
    with pytest.raises(tri.TriError):
        ctx.rope_load(omega * math.nan, 0)
    with pytest.raises(tri.TriError):
        ctx.rope_load(omega, 0, 0.0)
    fresh = tri.TriContext(0)
    assert fresh.rope(q, pos, check=False) == tri.TRI_ESTATE
    assert fresh.chunk_attention(pool.K, pool.V, lens, q, cu, block_table=pool.table, check=False) == tri.TRI_ESTATE
    fresh.close()
    torch.cuda.synchronize()
    assert (out == 7.0).all() and all(torch.equal(a, b) for a, b in zip(before, (pool.K, pool.V, pool.P, lens)))
    assert ctx.get_error()[0] == tri.TRI_OK
    ctx.close()


@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_a_key_that_is_not_finite_shows_in_every_row_that_sees_it(what):
    """Whatever its place among the keys: NaN results, not a weight lost on the way."""
    g = _gen(64)
    ctx = pu.context(1, 1, 4, 64)
    n, m = 3, 400
    q = torch.full((1, n, 4, 64), 1.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    lens = torch.tensor([m], dtype=torch.int32).cuda()
    for at in list(range(0, 16)) + [63, 64, 127, 128, 200, 301, 396]:
        pool = pu.Paged(g, 1, 1, 64, 16, [m])
        u, o = pool.places(0, m)
        pool.K[:, u[at], :, o[at]] = what
        lse = torch.empty((1, n, 4), device="cuda")
        out = ctx.chunk_attention(pool.K, pool.V, lens, q, cu, lse=lse, block_table=pool.table)
        assert torch.isnan(out).all() and torch.isnan(lse).all(), at
    ctx.close()


def test_plans_beyond_shared_memory():
    """More blocks than the plan keeps in shared memory, and a block table too long for one CTA to check."""
    _run(65, 1, 1, 1, 64, 16, [1] * 2100, [1 + i % 37 for i in range(2100)])
    pool = pu.Paged(_gen(66), 1, 2, 64, 16, [300, 40, 900], extra_pages=4000)
    _run(66, 1, 2, 2, 64, 16, [20, 1, 600], [300, 40, 900], pool=pool)
    pool.table[1, 1] = -1
    ctx = pu.context(1, 2, 2, 64)
    q = pu.bf16(_gen(67), (1, 3, 4, 64))
    ctx.chunk_attention(pool.K, pool.V, torch.tensor([300, 40, 900], dtype=torch.int32).cuda(), q,
                        torch.arange(4, dtype=torch.int32).cuda(), block_table=pool.table)
    assert ctx.get_error() == (tri.TRI_EDEVICE, tri.TRI_DEV_BAD_PAGE, 2)
    ctx.close()


def test_calls_on_other_streams():
    """Each call on its own stream, one after another by events: inputs made on one, used on another."""
    g = _gen(68)
    ctx = pu.context(1, 1, 4, 128)
    pool = pu.Paged(g, 1, 1, 128, 64, [600])
    q = pu.bf16(g, (1, 40, 4, 128), 2.0)
    cu, lens = torch.tensor([0, 40], dtype=torch.int32).cuda(), torch.tensor([600], dtype=torch.int32).cuda()
    pos = torch.arange(40, dtype=torch.int32).cuda()
    want = ctx.chunk_attention(pool.K, pool.V, lens, ctx.rope(q, pos), cu, block_table=pool.table)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    r, out = torch.empty_like(q), torch.empty_like(q)
    for _ in range(3):
        r.zero_(), out.zero_()
        a.wait_stream(torch.cuda.current_stream())
        ctx.rope(q, pos, out=r, stream=a)
        b.wait_stream(a)
        with torch.cuda.stream(b):
            ctx.chunk_attention(pool.K, pool.V, lens, r, cu, out=out, block_table=pool.table)
        torch.cuda.current_stream().wait_stream(b)
        assert torch.equal(out, want)
    assert ctx.get_error()[0] == tri.TRI_OK
    ctx.close()
