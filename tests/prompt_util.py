"""Plain 64-bit forms of the prompt-side operators (rotary positions, chunk append, chunk attention) and the caches that their
tests run on. Everything here is torch float64 on the inputs' device, without the library."""
import math

import numpy as np
import torch

from rope_aware_key_tri_b200 import tri

HALF, INTERLEAVED = 0, 1
BASE = 1e6


def context(L=1, hkv=1, group=1, d=64, layout=HALF, base=BASE):
    ctx = tri.TriContext(0)
    hq, F = hkv * group, d // 2
    ctx.calibrate_load(L, hkv, group, d, base, layout, np.zeros((L, hq, d)), np.zeros((L, hq, F)), np.zeros((L, hq, F)), [1])
    return ctx


def bf16(gen, shape, sigma=1.0, device="cuda"):
    return (sigma * torch.randn(shape, generator=gen)).to(torch.bfloat16).to(device)


def rotate(x, pos, omega, layout, magnitude=1.0, inverse=False):
    """x [..., T, H, d] float64 rotated at pos [T]; omega [r/2]."""
    r = 2 * len(omega)
    om = torch.as_tensor(np.asarray(omega), dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None, None] * om
    c, s = torch.cos(ang) * magnitude, torch.sin(ang) * magnitude
    if inverse:
        c, s = torch.cos(ang) / magnitude, -torch.sin(ang) / magnitude
    ia = torch.arange(r // 2, device=x.device) * (1 if layout == HALF else 2)
    ib = ia + (r // 2 if layout == HALF else 1)
    out = x.clone()
    out[..., ia] = x[..., ia] * c - x[..., ib] * s
    out[..., ib] = x[..., ia] * s + x[..., ib] * c
    return out


def rope_error_bound(x, want, rot, layout, magnitude=1.0):
    """Half a bf16 step of the result, plus the fp32 steps before it: sine and cosine (2 ulp each), the two products
    and the sum, all of them relative to |x_a| + |x_b| of the band."""
    size = x.abs()
    part = size.clone()
    if layout == HALF:
        part[..., :rot] = (size[..., :rot // 2] + size[..., rot // 2:rot]).repeat_interleave(1, -1).repeat(
            (1,) * (x.dim() - 1) + (2,))
    else:
        part[..., :rot] = (size[..., 0:rot:2] + size[..., 1:rot:2]).repeat_interleave(2, -1)
    return 2.0 ** -8 * want.abs() + 2.0 ** -20 * magnitude * part + 1e-37


class Paged:
    """Pools of garbage with a permuted block table for sequences of the given capacity (page 0: dense)."""

    def __init__(self, gen, L, hkv, d, page, totals, spare=2, device="cuda", extra_pages=0):
        self.page, self.L, self.hkv, self.d = page, L, hkv, d
        B = len(totals)
        if page:
            need = [-(-t // page) for t in totals]
            n_pages = sum(need) + spare
            self.n_pages = n_pages
            perm = torch.randperm(n_pages, generator=gen).tolist()
            self.table_host = np.full((B, max(1, max(need)) + extra_pages), -1, dtype=np.int32)
            for b, k in enumerate(need):
                self.table_host[b, :k] = [perm.pop() for _ in range(k)]
            self.table = torch.from_numpy(self.table_host).to(device)
            shape = (L, n_pages, hkv, page)
        else:
            self.table = None
            shape = (L, B, hkv, max(1, max(totals)) + spare)
        self.K, self.V = bf16(gen, shape + (d,), 0.6, device), bf16(gen, shape + (d,), 1.0, device)
        self.P = torch.full(shape, -7, dtype=torch.int32, device=device)

    def places(self, b, n):
        """(unit index tensor, offset tensor) of slots 0..n-1 of sequence b."""
        slot = torch.arange(n)
        if self.page:
            return torch.from_numpy(self.table_host[b].astype(np.int64))[slot // self.page], slot % self.page
        return torch.full((n,), b, dtype=torch.int64), slot

    def rows(self, x, b, n):
        """Rows 0..n-1 of sequence b: [L][hkv][n][...]."""
        u, o = self.places(b, n)
        return x[:, u.to(x.device), :, o.to(x.device)].transpose(0, 1).transpose(1, 2)


def attention(q, k, v, first, scale):
    """float64: q [H][n][d] over k, v [m][d]; query i sees keys [0, first + i) if first is an int, all m if None.
    Returns out [H][n][d] and lse [H][n]; rows that see nothing: zeros and -inf. Keys a query does not see take no part."""
    H, n, d = q.shape
    m = k.shape[0]
    out = torch.zeros((H, n, d), dtype=torch.float64, device=q.device)
    lse = torch.full((H, n), -math.inf, dtype=torch.float64, device=q.device)
    if m == 0 or n == 0:
        return out, lse
    x = q.double() @ k.double().T * scale
    if first is not None:
        seen = torch.arange(m, device=q.device)[None, :] < first + torch.arange(n, device=q.device)[:, None]
        x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top) & (top < 0), 0.0, top))
    z = p.sum(-1, keepdim=True)
    vv = v.double()
    if torch.isfinite(vv).all():
        o = p @ vv
    else:  # a zero weight takes no part, whatever the value is
        o = torch.stack([torch.stack([(p[h, i][p[h, i] != 0][:, None] * vv[p[h, i] != 0]).sum(0) for i in range(n)])
                         for h in range(H)])
    some = z > 0
    out = torch.where(some | torch.isnan(z), o / z, 0.0)
    lse = torch.where(some, top + torch.log(z), -math.inf)[..., 0]
    return out, lse


def attention_bounds(q, k, v, scale):
    """(absolute part of the output's error, absolute error of lse), derived:
      * a logit: d products, each sum step rounded (or truncated: 2^-23) in fp32, in the log2 domain:
        e = (d + 2) 2^-23 max sum |q k| scale log2(e); a weight moves by 2 ln2 e, the maximum included;
      * a weight is rounded to bf16 (2^-8), the hardware's exp2 and the rescales add 2^-20, the fp32 sums (M + 8) 2^-23;
      * the quotient is rounded to bf16: 2^-8 |out|, added by the caller.
    """
    M, d = k.shape[0], q.shape[-1]
    if M == 0 or q.shape[1] == 0:
        return 0.0, 0.0
    e = (d + 2) * 2.0 ** -23 * float((q.double().abs() @ k.double().abs().T).max()) * scale * math.log2(math.e)
    w = 2 * math.log(2) * e + 2.0 ** -20 + (M + 8) * 2.0 ** -23
    return (2.0 ** -8 + w) * float(v.double().abs().max()), math.log(2) * e + w + 2.0 ** -20
