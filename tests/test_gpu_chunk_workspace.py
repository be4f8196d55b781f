"""The attention's workspace when an allocation fails on the way."""
import numpy as np
import pytest
import torch

import prompt_util as pu
from rope_aware_key_tri_b200 import tri

pytestmark = pytest.mark.gpu


def test_a_call_that_ran_out_of_memory_can_be_made_again():
    """The plan's memory is had, the parts' is not (TRI_ENOMEM); with memory free again the same call is right, with a plan of many
    CTAs, whatever the plan's memory held before."""
    g = torch.Generator().manual_seed(80)
    new, lens = [1] * 600, [1 + i % 50 for i in range(600)]
    ctx = pu.context(1, 1, 2, 128)
    pool = pu.Paged(g, 1, 1, 128, 16, lens)
    q = pu.bf16(g, (1, 600, 2, 128), 2.0)
    cu = torch.arange(601, dtype=torch.int32).cuda()
    lens_dev = torch.tensor(lens, dtype=torch.int32).cuda()
    out, lse = torch.empty_like(q), torch.empty((1, 600, 2), device="cuda")
    torch.cuda.synchronize()
    dirty = [torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    del dirty
    torch.cuda.empty_cache()
    room = 48 << 20  # for the plan, not for the parts (79 MB)
    hog = []
    for _ in range(64):
        size = (torch.cuda.mem_get_info()[0] - room) >> 21 << 21
        if size <= 0:
            break
        while size > 1 << 21:
            try:
                hog.append(torch.empty(size, dtype=torch.uint8, device="cuda"))
                break
            except torch.cuda.OutOfMemoryError:
                size = size // 2 >> 21 << 21
    try:
        assert torch.cuda.mem_get_info()[0] < 72 << 20
        st = ctx.chunk_attention(pool.K, pool.V, lens_dev, q, cu, out=out, lse=lse, block_table=pool.table, check=False)
    finally:
        del hog
        torch.cuda.empty_cache()
    assert st == tri.TRI_ENOMEM
    for _ in range(2):
        out.fill_(7.0)
        ctx.chunk_attention(pool.K, pool.V, lens_dev, q, cu, out=out, lse=lse, block_table=pool.table)
        assert ctx.get_error()[0] == tri.TRI_OK
        for b in range(600):
            k, v = pool.rows(pool.K, b, lens[b])[0, 0], pool.rows(pool.V, b, lens[b])[0, 0]
            qq = q[0, b:b + 1].transpose(0, 1)
            want, wlse = pu.attention(qq, k, v, lens[b], 128 ** -0.5)
            ta, tl = pu.attention_bounds(qq, k, v, 128 ** -0.5)
            assert ((out[0, b:b + 1].transpose(0, 1).double() - want).abs() <= ta + 2.0 ** -8 * want.abs()).all(), b
            assert ((lse[0, b:b + 1].T.double() - wlse).abs() <= tl).all(), b
    ctx.close()
