"""newton_schulz on shapes that take 256 tiles, whole and split along k. Tolerances: _newton_schulz.py."""

import pytest
import torch

import thread_block_lds_amd as tbl
from _dispatch import ortho
from _newton_schulz import bound, check, exact, strong

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(1024, 8192), (16384, 520), (2305, 4100), (4100, 2305), (4097, 4100), (5888, 5700)])
def test_256_tiles(rows, cols):
    print(f"newton_schulz {rows}x{cols} {ortho(1, rows, cols)}", flush=True)
    for dtype in (torch.float32, torch.bfloat16):
        x = strong(rows, cols, dtype, 3)
        want, most = exact(x), bound(x)
        for out in (torch.float32, torch.bfloat16, torch.float16):
            check(tbl.newton_schulz(x, out_dtype=out), x, want, most)
        assert torch.equal(tbl.newton_schulz(x), tbl.newton_schulz(x))


@pytest.mark.parametrize("batch,rows,cols", [(12, 1100, 1300), (3, 1300, 8000)])
def test_256_tiles_of_a_batch(batch, rows, cols):
    print(f"newton_schulz {batch}x{rows}x{cols} {ortho(batch, rows, cols)}", flush=True)
    x = torch.stack([strong(rows, cols, torch.bfloat16, i) * 10.0 ** (i % 5 - 2) for i in range(batch)])
    y = tbl.newton_schulz(x, out_dtype=torch.float32)
    for i in (0, 1, batch - 1):
        check(y[i], x[i])
