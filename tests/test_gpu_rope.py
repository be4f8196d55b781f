"""Rotary positions and chunk appends on the GPU, through the C ABI, against 64-bit forms."""
import numpy as np
import pytest
import torch

import prompt_util as pu
from rope_aware_key_tri_b200 import tri

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _check_rope(got, x, pos, omega, layout, mag=1.0, inverse=False):
    want = pu.rotate(x.double(), pos, omega, layout, mag, inverse)
    m = 1 / mag if inverse else mag
    tol = pu.rope_error_bound(x.double(), want, 2 * len(omega), layout, m)
    err = (got.double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert torch.equal(got[..., 2 * len(omega):].view(torch.int16), x[..., 2 * len(omega):].view(torch.int16))


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", [pu.HALF, pu.INTERLEAVED])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (128, 96)])
def test_rope_shapes(d, rot, layout, inverse):
    omega, mag = tri.rope_frequencies(rot, 1e6, "yarn", 4.0, 4096)
    ctx = tri.TriContext(0)
    ctx.rope_load(omega, layout, mag)
    for L, T, H, seed in ((1, 1, 1, 0), (2, 7, 5, 1), (1, 700, 3, 2), (3, 33, 40, 3), (1, 5000, 1, 4)):
        g = _gen(100 + seed)
        x = pu.bf16(g, (L, T, H, d), 2.0)
        pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32).cuda()
        got = ctx.rope(x, pos, inverse=inverse)
        _check_rope(got, x, pos, omega, layout, mag, inverse)
    ctx.close()


def test_rope_any_position():
    """The whole int32 range, where an fp32 angle would be meaningless."""
    omega, _ = tri.rope_frequencies(128, 1e4)
    ctx = tri.TriContext(0)
    ctx.rope_load(omega, pu.HALF)
    pos = torch.tensor([0, 1, -1, 1 << 24, (1 << 24) + 1, 2**31 - 1, -2**31, 2**30 + 7], dtype=torch.int32).cuda()
    x = pu.bf16(_gen(5), (8, 2, 128))
    _check_rope(ctx.rope(x, pos), x, pos, omega, pu.HALF)
    ctx.close()


def test_rope_strides_in_place_and_broadcast():
    omega, _ = tri.rope_frequencies(64, 1e4)
    ctx = tri.TriContext(0)
    ctx.rope_load(omega, pu.INTERLEAVED)
    g = _gen(6)
    qkv = pu.bf16(g, (2, 50, 12, 64))
    pos = torch.randint(0, 9999, (50,), generator=g, dtype=torch.int32).cuda()
    # heads 3..7 of a wider projection, in place: the rest stays
    before = qkv.clone()
    view = qkv[:, :, 3:8]
    assert ctx.rope(view, pos, out=view) is view
    _check_rope(view.contiguous(), before[:, :, 3:8].contiguous(), pos, omega, pu.INTERLEAVED)
    assert torch.equal(qkv[:, :, :3], before[:, :, :3]) and torch.equal(qkv[:, :, 8:], before[:, :, 8:])
    # heads outermost
    hm = pu.bf16(g, (5, 50, 64)).transpose(0, 1)
    _check_rope(ctx.rope(hm, pos, out=torch.empty((50, 5, 64), dtype=torch.bfloat16, device="cuda")), hm, pos, omega,
                pu.INTERLEAVED)
    # one row for every head
    one = pu.bf16(g, (50, 1, 64)).expand(50, 6, 64)
    _check_rope(ctx.rope(one, pos, out=torch.empty((50, 6, 64), dtype=torch.bfloat16, device="cuda")), one, pos, omega,
                pu.INTERLEAVED)
    # layers repeated, no tokens
    empty = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert ctx.rope(empty, torch.empty(0, dtype=torch.int32, device="cuda")).shape == (0, 4, 64)
    ctx.close()


def test_rope_inverse_is_the_gradient_and_undoes():
    """For magnitude 1 the inverse is the transpose: <rotate(x), y> = <x, inverse(y)>; and it undoes the rotation.
    Both up to the bf16 roundings (2^-8 each, of values up to sqrt(2) max)."""
    omega, _ = tri.rope_frequencies(128, 1e6)
    ctx = tri.TriContext(0)
    ctx.rope_load(omega, pu.HALF)
    g = _gen(7)
    x, y = pu.bf16(g, (64, 4, 128)), pu.bf16(g, (64, 4, 128))
    pos = torch.randint(0, 100000, (64,), generator=g, dtype=torch.int32).cuda()
    rx, iy = ctx.rope(x, pos), ctx.rope(y, pos, inverse=True)
    a, b = (rx.double() * y.double()).sum(-1), (x.double() * iy.double()).sum(-1)
    tol = (2.0 ** -8 + 2.0 ** -18) * ((rx.double() * y.double()).abs().sum(-1) + (x.double() * iy.double()).abs().sum(-1))
    assert ((a - b).abs() <= tol).all()
    back = ctx.rope(rx, pos, inverse=True)
    size = pu.rope_error_bound(x.double(), x.double(), 128, pu.HALF)
    part = (size - 2.0 ** -8 * x.double().abs()) * 2.0 ** 20   # |x_a| + |x_b| of the band
    # rx is off by 2^-8 |rx| in both components, |rx| <= |x_a| + |x_b|; then one more rounding of the result
    assert ((back.double() - x.double()).abs() <= 2.0 ** -8 * (2.1 * part + x.double().abs())).all()
    # differences: the rotation is linear, so its derivative along y is rotate(x + y) - rotate(x)
    s = (x.float() + y.float()).to(torch.bfloat16)
    diff = ctx.rope(s, pos).double() - rx.double()
    want = pu.rotate((s.double() - x.double()), pos, omega, pu.HALF)
    tol = 2.0 ** -8 * (ctx.rope(s, pos).double().abs() + rx.double().abs()) + 2.0 ** -18 * (part + 4)
    assert ((diff - want).abs() <= 1.01 * tol).all()
    ctx.close()


def test_rope_default_table_is_the_statistics():
    ctx = pu.context(1, 2, 4, 64, pu.INTERLEAVED, 1e4)
    g = _gen(8)
    x = pu.bf16(g, (9, 8, 64))
    pos = torch.arange(9, dtype=torch.int32).cuda() * 77
    omega = 1e4 ** (-2.0 * np.arange(32) / 64)
    _check_rope(ctx.rope(x, pos), x, pos, omega, pu.INTERLEAVED)
    ctx.close()


# ---- appending runs ----------------------------------------------------------------------------

def _append_case(seed, L, hkv, group, d, page, new, lens, layout, rot, with_q=True, T_extra=0, rotate=True, alias=True,
                 refuse=(), extra_pages=0):
    g = _gen(seed)
    ctx = pu.context(L, hkv, group, d, layout)
    omega, mag = tri.rope_frequencies(rot, 1e6, "yarn", 4.0, 4096)
    ctx.rope_load(omega, layout, mag)
    pool = pu.Paged(g, L, hkv, d, page, [a + b for a, b in zip(new, lens)], extra_pages=extra_pages)
    T, B, hq = sum(new) + T_extra, len(new), hkv * group
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    qkv = pu.bf16(g, (L, T, hq + 2 * hkv, d))
    q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
    pos = torch.randint(0, 1 << 17, (T,), generator=g, dtype=torch.int32).cuda()
    lens_dev = torch.tensor(lens, dtype=torch.int32).cuda()
    for b in refuse:
        if page:
            pool.table[b, (lens[b] + new[b] - 1) // page] = pool.n_pages
        else:
            lens_dev[b] = pool.K.shape[3] - new[b] + 1
    lens_out = lens_dev if alias else torch.full((B,), -5, dtype=torch.int32, device="cuda")
    start = lens_dev.clone()
    before = [x.clone() for x in (pool.K, pool.V, pool.P)]
    q_out = torch.full((L, T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda") if with_q else None
    ctx.append_chunk(pool.K, pool.V, pool.P, lens_dev, k, v, cu, pos, block_table=pool.table, lens_out=lens_out,
                     rotate=rotate, q=q if with_q else None, q_out=q_out)
    st = ctx.get_error()
    want = [x.double().clone() for x in before[:2]] + [before[2].clone()]
    size = torch.zeros_like(want[0])
    kr = pu.rotate(k.double(), pos, omega, layout, mag) if rotate else k.double()
    kt = pu.rope_error_bound(k.double(), kr, rot, layout, mag) if rotate else torch.zeros_like(kr)
    qr = pu.rotate(q.double(), pos, omega, layout, mag)
    qt = pu.rope_error_bound(q.double(), qr, rot, layout, mag)
    written = torch.zeros(T, dtype=torch.bool)
    c = np.concatenate([[0], np.cumsum(new)])
    for b in range(B):
        if b in refuse or new[b] == 0:
            continue
        u, o = pool.places(b, lens[b] + new[b])
        u, o = u[lens[b]:].cuda(), o[lens[b]:].cuda()
        t = slice(int(c[b]), int(c[b + 1]))
        written[t] = True
        want[0][:, u, :, o] = kr[:, t].transpose(0, 1)
        size[:, u, :, o] = kt[:, t].transpose(0, 1)
        want[1][:, u, :, o] = v[:, t].double().transpose(0, 1)
        want[2][:, u, :, o] = pos[t][:, None, None].expand(-1, L, hkv)
    assert ((pool.K.double() - want[0]).abs() <= size).all()
    assert torch.equal(pool.V.double(), want[1]) and torch.equal(pool.P, want[2])
    expect = [int(start[b]) + (0 if b in refuse else new[b]) for b in range(B)]
    assert lens_out.tolist() == expect
    if not alias:
        assert torch.equal(lens_dev, start)
    if with_q:
        w = written.cuda()
        assert ((q_out[:, w].double() - qr[:, w]).abs() <= qt[:, w]).all()
        assert (q_out[:, ~w] == 7.0).all()
    ctx.close()
    return st


@pytest.mark.parametrize("layout,d,rot", [(0, 128, 128), (1, 128, 64), (0, 64, 32), (1, 64, 64)])
@pytest.mark.parametrize("page", [0, 16, 48, 64])
def test_append_chunk_ragged(page, layout, d, rot):
    st = _append_case(20 + page + d + rot, 2, 2, 4, d, page, [1, 0, 130, 5, 64, 17], [3, 10, 0, 63, 64, 200], layout, rot,
                      T_extra=3)
    assert st[0] == tri.TRI_OK


@pytest.mark.parametrize("group,hkv", [(1, 1), (8, 1), (2, 8)])
def test_append_chunk_single_tokens(group, hkv):
    new = [1] * 40  # more sequences than one warp looks at in one step
    lens = list(range(40))
    assert _append_case(21, 3, hkv, group, 64, 16, new, lens, 0, 64)[0] == tri.TRI_OK


def test_append_chunk_long_run_and_no_rotation():
    assert _append_case(22, 1, 1, 1, 128, 16, [3000, 1], [40, 7], 0, 128, alias=False)[0] == tri.TRI_OK
    assert _append_case(23, 1, 2, 2, 64, 64, [100, 9], [40, 64], 1, 64, with_q=False, rotate=False)[0] == tri.TRI_OK
    assert _append_case(24, 1, 2, 2, 64, 64, [0, 0], [40, 64], 1, 64)[0] == tri.TRI_OK  # nothing to append


@pytest.mark.parametrize("page", [0, 16])
def test_append_chunk_refuses_a_whole_sequence(page):
    st, code, unit = _append_case(25, 2, 2, 2, 64, page, [40, 50, 0, 33], [8, 20, 5, 16], 0, 64, refuse=(1,))
    assert st == tri.TRI_EDEVICE and unit == 1 * 2
    assert code == (tri.TRI_DEV_BAD_PAGE if page else tri.TRI_DEV_LEN_GT_CAP)


def test_append_chunk_bad_ranges_refuse_everything():
    ctx = pu.context(1, 1, 1, 64)
    pool = pu.Paged(_gen(26), 1, 1, 64, 16, [32, 32, 32])
    lens = torch.tensor([3, 4, 5], dtype=torch.int32).cuda()
    k = pu.bf16(_gen(27), (1, 20, 1, 64))
    pos = torch.arange(20, dtype=torch.int32).cuda()
    before = [x.clone() for x in (pool.K, pool.V, pool.P, lens)]
    for cu in ([0, 8, 4, 12], [0, 4, 8, 21], [-1, 4, 8, 12], [0, 4, 30, 12]):
        ctx.append_chunk(pool.K, pool.V, pool.P, lens, k, k, torch.tensor(cu, dtype=torch.int32).cuda(), pos,
                         block_table=pool.table)
        st, code, _ = ctx.get_error()
        assert st == tri.TRI_EDEVICE and code == tri.TRI_DEV_BAD_RANGE, cu
        assert all(torch.equal(a, b) for a, b in zip(before, (pool.K, pool.V, pool.P, lens)))
    ctx.append_chunk(pool.K, pool.V, pool.P, lens, k, k, torch.tensor([2, 4, 4, 9], dtype=torch.int32).cuda(), pos,
                     block_table=pool.table)
    assert ctx.get_error()[0] == tri.TRI_OK and lens.tolist() == [5, 4, 10]
    ctx.close()
