"""Which kernels the GPU tests' shapes reach, by the library's own rules (CPU only): a change to a rule that took a kernel's
tests away would fail here."""

import pytest

from _dispatch import gemm8, ortho

F16, F32 = 0, 2


@pytest.mark.parametrize("batch,rows,cols,want", [
    (1, 1024, 8192, [(256, 16), (128, 1), (128, 1), (128, 1)]),      # P split
    (1, 16384, 520, [(256, 16), (128, 1), (256, 1), (256, 1)]),
    (1, 2305, 4100, [(128, 1), (128, 1), (256, 1), (256, 1)]),
    (1, 4097, 4100, [(256, 1), (256, 1), (256, 7), (256, 7)]),       # updates split
    (1, 5888, 5700, [(256, 12), (256, 12), (256, 15), (256, 15)]),
    (12, 1100, 1300, [(256, 1), (256, 1), (128, 1), (128, 1)]),
    (3, 1300, 8000, [(128, 1), (128, 1), (256, 4), (256, 4)]),
    (1, 128, 1000, [(0, 1)] * 4), (1, 129, 131, [(128, 1)] * 4),
])
def test_orthogonalisation(batch, rows, cols, want):
    assert ortho(batch, rows, cols) == want
    assert ortho(batch, cols, rows) == want


@pytest.mark.parametrize("M,N,K,out,want", [
    (3001, 4099, 1111, F16, (256, False)), (4500, 4700, 1234, F16, (256, True)), (4096, 4100, 3001, F16, (256, True)),
    (4097, 4095, 1100, F16, (256, True)), (300, 260, 300, F16, (128, False)), (200, 300, 8192, F16, (128, True)),
    (5, 64, 300, F16, (0, False)), (40, 64, 300, F16, (0, False)),
    (300, 260, 300, F32, (128, False)), (200, 300, 8192, F32, (128, True)), (40, 64, 300, F32, (0, False)),
])
def test_gemm(M, N, K, out, want):
    assert gemm8(M, N, K, out) == want
