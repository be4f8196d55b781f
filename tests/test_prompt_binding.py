"""What the torch-facing calls of the prompt side check before the library sees a pointer, without a GPU: tensors on the CPU are taken
for the context's device, and the library is handed no context, which it refuses (TRI_EINVAL) once every check has passed."""
import math
import types

import numpy as np
import pytest
import torch

from rope_aware_key_tri_b200 import tri

STREAM = types.SimpleNamespace(cuda_stream=0)


def _context(shape):
    ctx = tri.TriContext.__new__(tri.TriContext)
    ctx.device, ctx.handle, ctx.shape = -1, None, shape
    return ctx


def _append(ctx, L=1, H=2, d=64, page=16, pages=4, B=2, T=6, **kw):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    ints = lambda *s: torch.zeros(s, dtype=torch.int32)
    units, table = (pages, ints(B, 2)) if page else (B, None)
    a = dict(block_table=table, stream=STREAM, check=False)
    a.update(kw)
    return ctx.append_chunk(bf(L, units, H, page or 32, d), bf(L, units, H, page or 32, d), ints(L, units, H, page or 32), ints(B),
                            bf(L, T, H, d), bf(L, T, H, d), ints(B + 1), ints(T), **a)


@pytest.mark.parametrize("page", [0, 16])
def test_append_refuses_a_cache_of_other_heads(page):
    """The library takes heads and head_dim from the statistics: a cache that holds fewer would be written past its end."""
    assert _append(_context((1, 2, 4, 64)), page=page) == tri.TRI_EINVAL  # (no context)
    for shape in ((1, 8, 4, 128), (1, 8, 4, 64), (1, 2, 4, 128), (1, 1, 4, 64)):
        with pytest.raises(ValueError, match="statistics"):
            _append(_context(shape), page=page)
        with pytest.raises(ValueError, match="statistics"):
            _append(_context(shape), page=page, rotate=False)


def test_fewer_pages_than_the_pools_hold():
    """n_pages is the pools' layer stride: a part of the pools can be named in a cache of one layer only."""
    ctx = _context((2, 2, 4, 64))
    assert _append(ctx, L=1, n_pages=3) == tri.TRI_EINVAL  # (no context)
    assert _append(ctx, L=2, n_pages=4) == tri.TRI_EINVAL
    for L, n in ((2, 3), (1, 5), (2, 5)):
        with pytest.raises(ValueError, match="n_pages"):
            _append(ctx, L=L, n_pages=n)


def test_default_turns_of_the_scaled_tables():
    """"yarn" ramps up to 32 turns over the original length, "smooth" up to 4."""
    for kind, high in (("yarn", 32.0), ("smooth", 4.0)):
        for name in (kind, tri._SCALINGS[kind]):
            got, mag = tri.rope_frequencies(64, 1e6, name, 8.0, 8192)
            want, wmag = tri.rope_frequencies(64, 1e6, kind, 8.0, 8192, 1.0, high)
            assert (got == want).all() and mag == wmag


@pytest.mark.parametrize("r,base,factor,length,low,high", [(128, 1e6, 4.0, 8192, 1.0, 32.0), (64, 1e4, 8.0, 4096, 1.0, 32.0),
                                                           (96, 5e5, 2.0, 32768, 0.5, 16.0), (16, 1e4, 40.0, 2048, 1.0, 32.0)])
def test_yarn_ramp(r, base, factor, length, low, high):
    """Every band: omega / factor and omega mixed by a ramp over the band index, from the last band that turns at least `high`
    times over the length to the first that turns at most `low` times (as real indices, rounded outwards)."""
    f = np.arange(r // 2)
    omega = base ** (-2.0 * f / r)
    index = lambda turns: r * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base))
    first, last = max(math.floor(index(high)), 0), min(math.ceil(index(low)), r - 1)
    assert last > first
    mix = np.clip((f - first) / (last - first), 0.0, 1.0)
    got, magnitude = tri.rope_frequencies(r, base, "yarn", factor, length, low, high)
    np.testing.assert_allclose(got, omega / factor * mix + omega * (1 - mix), rtol=1e-12)
    assert math.isclose(magnitude, 1 + 0.1 * math.log(factor), rel_tol=1e-14)
