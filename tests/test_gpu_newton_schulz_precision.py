"""How exact newton_schulz is: what it keeps beside fp16, and no more, is what its error shows. The bounds are derived in
_newton_schulz.py; without the diagonals, or without the remainder, the simulated error lies beyond them."""

import pytest
import torch

import thread_block_lds_amd as tbl
from _newton_schulz import bound, exact, normal, off, rounded, strong

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(20, 4000), (1926, 33), (100, 20000), (160, 5000), (20000, 160), (512, 16384), (1024, 4096)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_alike_singular_values(rows, cols, dtype):
    """Of a wide random matrix: alike diagonals, whose roundings shift every singular value the same way."""
    x = normal(rows, cols, dtype)
    print(f"newton_schulz {rows}x{cols} {dtype}", flush=True)
    want, most = exact(x), bound(x)
    assert off(rounded(x, diagonals=False), want) > 1.15 * most
    got = off(tbl.newton_schulz(x, out_dtype=torch.float32), want)
    assert got <= most, (got, most)


@pytest.mark.parametrize("rows,cols", [(100, 400), (300, 400), (400, 300), (1030, 1030), (2050, 2050)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_remainder(rows, cols, dtype):
    """Directions that noise alone fills: a multiplies what rounding X adds there in every step that follows."""
    x = strong(rows, cols, dtype)
    print(f"newton_schulz {rows}x{cols} {dtype}", flush=True)
    want, most = exact(x), bound(x)
    assert off(rounded(x, remainder=False), want) > 1.15 * most
    got = off(tbl.newton_schulz(x, out_dtype=torch.float32), want)
    assert got <= most, (got, most)
