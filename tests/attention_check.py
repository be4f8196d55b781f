"""A check of attention results, row by row, that a misplaced or missing value row does not pass.

For one query head: weights p_j (64 bits), values v_j, out = sum_j p_j v_j. The kernel's error is at most, per dim,
  * weights rounded to bf16, d_j each, |d_j| <= 2^-8, as often up as down and independently from key to key: by Hoeffding's
    inequality |sum d_j p_j v_j| stays below T 2^-8 sqrt(sum p_j^2 v_j^2) but for a chance of 2 exp(-T^2 / 2); T = 9: 5e-18;
  * logits off by e in the log2 domain (prompt_util.attention_bounds), the exponential by 2^-18, and the fp32 sums: an MMA adds 16
    products in at most two steps of 2^-23, so M / 8 + 32 of them over M keys: w sum_j p_j |v_j|;
  * the result rounded to bf16: 2^-8 |out|.
"""
import math

import torch

T = 9.0


def weights(q, k, first, scale):
    """p [n][m] (64 bits) of the queries q [n][d], query i seeing the keys [0, first + i) (None: all)."""
    x = q.double() @ k.double().T * scale
    if first is not None:
        seen = torch.arange(k.shape[0], device=k.device)[None, :] < first + torch.arange(q.shape[0], device=k.device)[:, None]
        x = torch.where(seen, x, -math.inf)
    return torch.softmax(x, -1)


def tolerance(p, q, k, v, scale):
    """(want, tol) [n][d]."""
    M, d = k.shape
    vd = v.double()
    want = p @ vd
    e = (d + 2) * 2.0 ** -23 * float((q.double().abs() @ k.double().abs().T).max()) * scale * math.log2(math.e)
    w = 2 * math.log(2) * e + 2.0 ** -18 + (M / 8 + 32) * 2.0 ** -23
    return want, T * 2.0 ** -8 * torch.sqrt((p * p) @ (vd * vd)) + w * (p @ vd.abs()) + 2.0 ** -8 * want.abs()


def excess(got, p, q, k, v, scale):
    """The largest error in units of what is allowed: up to 1 passes."""
    want, tol = tolerance(p, q, k, v, scale)
    return float(((got.double() - want).abs() / tol).max())


def rounded(p, v):
    """What the kernel's arithmetic gives, but for its fp32 errors: weights relative to the largest, rounded to bf16, over the
    sum of the unrounded ones."""
    u = p / p.amax(-1, keepdim=True)
    return ((u.to(torch.bfloat16).double() @ v.double()) / u.sum(-1, keepdim=True)).to(torch.bfloat16)


def aimed(k, targets, strength=3.0):
    """Queries whose weight lies almost all on one key each: strength times that key, without its neighbours' help."""
    kt = k[targets].double()
    return (strength * kt / kt.pow(2).mean(-1, keepdim=True)).to(torch.bfloat16)
