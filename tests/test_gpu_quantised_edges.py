"""What quantize_fp8 writes past a matrix's edge, up to the whole group that its rows are stored in."""

import pytest
import torch

import thread_block_lds_amd as tbl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("rows,cols", [(3, 5), (130, 300), (1, 200), (257, 129)])
def test_bytes_past_the_edge_are_zero(rows, cols, dtype, block):
    """Also in groups that hold a NaN or an infinity."""
    x = torch.ones(rows, cols)
    x[-1, -1] = float("nan")
    x[0, cols // 2] = float("inf")
    q, t = tbl.quantize_fp8(x.to(dtype).cuda(), rows=block, transposed=True)
    one = tbl.quantize_fp8(x.to(dtype).cuda(), rows=block)
    for v in (q, t, one):
        r, c = v.codes.shape
        whole = torch.as_strided(v.codes.view(torch.uint8), (r, -(-c // 128) * 128), (v.codes.stride(0) if r > 1 else -(-c // 128) * 128, 1))
        assert bool((whole[:, c:] == 0).all())
        assert bool(v.codes.float()[-1, -1].isnan())
