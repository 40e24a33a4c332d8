"""newton_schulz on batches: against their matrices one by one, and on many of them. Tolerances: _newton_schulz.py."""

import pytest
import torch

import thread_block_lds_amd as tbl
from _dispatch import ortho
from _newton_schulz import check, off, strong

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,rows,cols", [(3, 128, 300), (5, 300, 40), (2, 16, 16), (12, 513, 257), (7, 60, 1000)])
def test_a_batch_gives_the_bits_of_its_matrices(batch, rows, cols):
    """Where a batch is run as its matrices alone are (the same tiles or as many chunks)."""
    x = torch.stack([strong(rows, cols, torch.bfloat16, i) for i in range(batch)])
    assert ortho(batch, rows, cols) == ortho(1, rows, cols)
    y = tbl.newton_schulz(x)
    for i in range(batch):
        assert torch.equal(y[i], tbl.newton_schulz(x[i].contiguous()))


@pytest.mark.parametrize("batch,rows,cols", [(16, 128, 1000), (40, 30, 700)])
def test_a_batch_against_its_matrices(batch, rows, cols):
    """Where a large batch's matrices are summed in fewer chunks: two sums' worth of the precision tests' 2^-13 apart."""
    x = torch.stack([strong(rows, cols, torch.bfloat16, i) for i in range(batch)])
    y = tbl.newton_schulz(x, out_dtype=torch.float32)
    for i in range(batch):
        assert off(y[i], tbl.newton_schulz(x[i].contiguous(), out_dtype=torch.float32).double()) <= 2.0 ** -12


def test_many_matrices_with_strided_rows():
    """A norm of many parts for each of many matrices: 2^32 threads if every matrix had as many as one alone."""
    batch, rows, cols = 16384, 1024, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(batch, rows, 24, generator=g, device="cuda").bfloat16()[:, :, 3:3 + cols]
    y = tbl.newton_schulz(x)
    for i in (0, 777, batch - 1):
        check(y[i], x[i].contiguous())
    assert bool(y.isfinite().all())
