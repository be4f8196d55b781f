"""The prompt-side operators' host side: rotary tables against their formulas, and arguments that are refused before anything is
launched (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest

from rope_aware_key_tri_b200 import tri


@pytest.mark.parametrize("r", [16, 64, 96, 128])
def test_rope_frequencies(r):
    f = np.arange(r // 2)
    w = 1e6 ** (-2.0 * f / r)
    got, mag = tri.rope_frequencies(r, 1e6)
    np.testing.assert_allclose(got, w, rtol=1e-13)
    assert mag == 1.0
    got, mag = tri.rope_frequencies(r, 1e6, "linear", 8.0)
    np.testing.assert_allclose(got, w / 8.0, rtol=1e-13)
    got, mag = tri.rope_frequencies(r, 1e6, "ntk", 8.0)
    assert math.isclose(got[0], 1.0) and math.isclose(got[-1], w[-1] / 8.0, rel_tol=1e-12) and mag == 1.0
    for kind, low, high in (("yarn", 1.0, 32.0), ("smooth", 1.0, 4.0)):
        got, mag = tri.rope_frequencies(r, 1e6, kind, 8.0, 8192, low, high)
        turns = 8192 * w / (2 * math.pi)
        assert mag == (1.0 if kind == "smooth" else pytest.approx(0.1 * math.log(8.0) + 1.0))
        assert np.all(got <= w * (1 + 1e-12)) and np.all(got >= w / 8.0 * (1 - 1e-12))
        if kind == "smooth":
            np.testing.assert_allclose(got[turns >= high], w[turns >= high], rtol=1e-13)
            np.testing.assert_allclose(got[turns <= low], w[turns <= low] / 8.0, rtol=1e-13)
            mid = (turns > low) & (turns < high)
            m = (turns[mid] - low) / (high - low)
            np.testing.assert_allclose(got[mid], (1 - m) * w[mid] / 8.0 + m * w[mid], rtol=1e-12)
        else:
            lo = max(math.floor(r * math.log(8192 / (high * 2 * math.pi)) / (2 * math.log(1e6))), 0)
            hi = min(math.ceil(r * math.log(8192 / (low * 2 * math.pi)) / (2 * math.log(1e6))), r - 1)
            np.testing.assert_allclose(got[:lo + 1], w[:lo + 1], rtol=1e-13)
            np.testing.assert_allclose(got[min(hi, r // 2):], w[min(hi, r // 2):] / 8.0, rtol=1e-12)


@pytest.mark.parametrize("args", [(0, 1e4), (24, 1e4), (144, 1e4), (64, 1.0), (64, -2.0), (64, math.nan), (64, math.inf),
                                  (64, 1e4, "linear", 0.5), (64, 1e4, "ntk", math.inf), (64, 1e4, "yarn", 2.0, 0.0),
                                  (64, 1e4, "yarn", 2.0, 4096, 4.0, 4.0), (64, 1e4, "smooth", 2.0, 4096, -1.0, 4.0), (64, 1e4, 9),
                                  (64, 1e4, -1)])
def test_rope_frequencies_refuses(args):
    with pytest.raises(tri.TriError) as e:
        tri.rope_frequencies(*args)
    assert e.value.status == tri.TRI_EINVAL


def test_null_arguments_are_refused():
    L = tri.library()
    kv, rows = tri.tri_kv(), tri.tri_rows()
    R, K = ctypes.byref(rows), ctypes.byref(kv)
    om = (ctypes.c_double * 32)()
    assert L.tri_rope_load(None, 64, 0, om, 1.0) == tri.TRI_EINVAL
    assert L.tri_rope(None, R, R, 1, 1, 1, 64, None, 0, None) == tri.TRI_EINVAL
    assert L.tri_append_chunk(None, K, R, R, None, None, 1, 1, None, None, None) == tri.TRI_EINVAL
    assert L.tri_chunk_attention(None, K, R, None, 1, 1.0, 1, R, None, None) == tri.TRI_EINVAL
    mag = ctypes.c_double()
    assert L.tri_rope_frequencies(64, 1e4, 0, 1.0, 0.0, 1.0, 2.0, None, ctypes.byref(mag)) == tri.TRI_EINVAL
    assert L.tri_rope_frequencies(64, 1e4, 0, 1.0, 0.0, 1.0, 2.0, om, None) == tri.TRI_EINVAL


def test_rows_must_be_bf16_on_the_gpu():
    import torch
    with pytest.raises(ValueError):
        tri.make_rows(torch.zeros(2, 3, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        tri.make_rows(torch.zeros(2, 64))
