"""The check of attention results against mistakes planted in the 64-bit form: a value tile missing, taken twice, a page's rows taken from
the next page. Each must be rejected, and what the kernel's roundings give accepted."""
import pytest
import torch

import attention_check as ac


def _case(n, m, d, seed, aim):
    g = torch.Generator().manual_seed(seed)
    k = (0.6 * torch.randn((m, d), generator=g)).to(torch.bfloat16)
    v = torch.randn((m, d), generator=g).to(torch.bfloat16)
    if aim:
        q = ac.aimed(k, torch.randint(0, m, (n,), generator=g))
    else:
        q = (2.0 * torch.randn((n, d), generator=g)).to(torch.bfloat16)
    return q, k, v


def _zeroed(v, rows):
    w = v.clone()
    w[rows] = 0.0
    return w


def _shifted(v, rows, by):
    w = v.clone()
    w[rows] = v[slice(rows.start + by, rows.stop + by)]
    return w


@pytest.mark.parametrize("n,m,d", [(1, 9000, 64), (1, 9000, 128), (17, 5000, 128), (300, 7777, 64)])
def test_planted_mistakes_are_rejected(n, m, d):
    heads = 8 if n < 300 else 1  # query heads that share the keys
    q, k, v = _case(n * heads, m, d, n + d, False)
    p = ac.weights(q, k, None, d ** -0.5)
    assert ac.excess(ac.rounded(p, v), p, q, k, v, d ** -0.5) <= 1.0
    t = slice(2048, 2176)
    for bad in (_zeroed(v, t), _shifted(v, t, 128), _zeroed(v, slice(2048, 2080)), _shifted(v, slice(2064, 2080), 16)):
        assert ac.excess(ac.rounded(p, bad), p, q, k, v, d ** -0.5) > 1.0


@pytest.mark.parametrize("d", [64, 128])
def test_queries_aimed_at_single_keys(d):
    """Where one key has almost all the weight, a single misplaced row shows."""
    m = 5000
    g = torch.Generator().manual_seed(d)
    k = (0.6 * torch.randn((m, d), generator=g)).to(torch.bfloat16)
    v = torch.randn((m, d), generator=g).to(torch.bfloat16)
    targets = torch.arange(0, m, 17)
    q = ac.aimed(k, targets)
    p = ac.weights(q, k, None, d ** -0.5)
    assert (p.gather(1, targets[:, None]) > 0.5).all()
    assert ac.excess(ac.rounded(p, v), p, q, k, v, d ** -0.5) <= 1.0
    for bad in (_zeroed(v, slice(1700, 1701)), _shifted(v, slice(1700, 1701), 1), _shifted(v, slice(3200, 3216), 16),
                _zeroed(v, slice(4864, 5000))):
        assert ac.excess(ac.rounded(p, bad), p, q, k, v, d ** -0.5) > 5.0
