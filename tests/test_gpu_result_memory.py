"""Results that a call allocates belong to the stream that writes them (the caching allocator hands a stream's memory back to work
on that stream without waiting for others)."""
import pytest
import torch

import prompt_util as pu
from rope_aware_key_tri_b200 import tri

pytestmark = pytest.mark.gpu


def _stream_of(x):
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= x.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]


def test_results_belong_to_their_stream():
    g = torch.Generator().manual_seed(110)
    ctx = pu.context(1, 2, 2, 64)
    pool = pu.Paged(g, 1, 2, 64, 16, [40, 40])
    q = pu.bf16(g, (1, 2, 4, 64))
    cu, lens = torch.arange(3, dtype=torch.int32).cuda(), torch.full((2,), 40, dtype=torch.int32, device="cuda")
    pos = torch.arange(2, dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    for stream in (None, side):
        here = (stream or torch.cuda.current_stream()).cuda_stream
        side.wait_stream(torch.cuda.current_stream())
        results = [ctx.rope(q, pos, stream=stream),
                   ctx.chunk_attention(pool.K, pool.V, lens, q, cu, block_table=pool.table, stream=stream),
                   ctx.decode_attention(pool.K, pool.V, lens, q, block_table=pool.table, stream=stream),
                   *ctx.calibrate_estimate(q, pu.HALF, stream=stream)]
        torch.cuda.synchronize()
        assert [_stream_of(x) for x in results] == [here] * len(results)
        assert ctx.get_error()[0] == tri.TRI_OK
    ctx.close()
