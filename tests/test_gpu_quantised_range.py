"""gemm_fp8 where the product of two scales leaves fp32's range.

A group's sum may be zero or small however large its operands' scales are: where their product is beyond fp32's largest
value, the sum is taken by the smaller scale first. Bounds: test_gpu_quantised_gemm.py's."""

import pytest
import torch

import thread_block_lds_amd as tbl
from _dispatch import gemm8
from test_gpu_quantised_gemm import E4M3, E5M2
from test_gpu_quantised_gemm_large import check_product

pytestmark = pytest.mark.gpu

SHAPES = [(5, 64, 300), (40, 64, 300), (300, 260, 300), (200, 300, 8192), (3001, 4099, 300), (4097, 4095, 1100)]


def blocks(rows, cols, block, fmt, seed, scale):
    """Random codes; every scale is ``scale`` in group 0 and 1 in the others. Group 0 has zeros but for one column."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randn(rows, -(-cols // 128) * 128, generator=g, device="cuda")
    codes[:, :128] = 0
    codes[:, seed] = 4.0
    codes[:, 9] = 2.0 ** -9 if fmt == E4M3 else 2.0 ** -16
    groups = -(-cols // 128)
    s = torch.ones((groups, rows) if block == 1 else (-(-rows // 128), groups), device="cuda")
    if block == 1:
        s[0] = scale
    else:
        s[:, 0] = scale
    return tbl.Fp8Blocks(codes.to(fmt)[:, :cols], s, block)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("block", [1, 128])
def test_scales_beyond_fp32_together(M, N, K, block):
    """Their one common column makes 2^-25 (e4m3 x e5m2) x 1e40."""
    print(f"gemm_fp8 {M}x{N}x{K} block {block} {gemm8(M, N, K, 1)} {gemm8(M, N, K, 2)}", flush=True)
    a, b = blocks(M, K, 1, E4M3, 1, 1e30), blocks(N, K, block, E5M2, 2, 1e10)
    for out in (torch.bfloat16, torch.float32):
        add = torch.randn(M, N, device="cuda")
        check_product(tbl.gemm_fp8(a, b, add=add, out_dtype=out), a, b, add)
        a0, b0 = (tbl.Fp8Blocks(q.codes.clone(), q.scale, q.rows) for q in (a, b))
        a0.codes.view(torch.uint8)[:, 9] = 0     # nothing in common: the group's sum is 0
        c = tbl.gemm_fp8(a0, b0, out_dtype=out)
        assert bool(c.isfinite().all())
        check_product(c, a0, b0, None)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("sa,sb", [(1e35, 1e-20), (1e-20, 1e35), (1e-30, 1e30)])
def test_one_large_scale(M, N, K, sa, sb):
    """Whose product with a group's sum alone would leave the range."""
    a, b = blocks(M, K, 1, E4M3, 1, sa), blocks(N, K, 1, E4M3, 1, sb)
    a.codes.view(torch.uint8)[:, 1] = 0x7E       # 448
    b.codes.view(torch.uint8)[:, 1] = 0x7E
    for out in (torch.bfloat16, torch.float32):
        check_product(tbl.gemm_fp8(a, b, out_dtype=out), a, b, None)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_results_that_are_not_finite_stay(M, N, K):
    """An infinite or NaN scale, a NaN code, and a sum beyond the range, beside groups whose scales overflow together."""
    for scale in (1.0, 1e30):
        a, b = blocks(M, K, 1, E4M3, 1, scale), blocks(N, K, 1, E4M3, 1, 1e10)
        a.codes.view(torch.uint8)[:, 9] = 0
        a.codes.view(torch.uint8)[:, 1] = 0
        a.scale[1, 0] = float("inf")
        a.scale[2, 2] = float("nan")
        a.codes.view(torch.uint8)[3, 5] = 0x7F
        a.codes.view(torch.uint8)[4, 1] = 0x7E
        b.scale[0, 7] = 1e38
        for out in (torch.bfloat16, torch.float32):
            c = tbl.gemm_fp8(a, b, out_dtype=out)
            assert bool((~c[0].isfinite()).all()) and bool(c[2].isnan().all()) and bool(c[3].isnan().all())
            assert float(c[4, 7]) == float("inf") and (scale == 1 or bool((c[4] == float("inf")).all()))
            assert bool(c[1].isfinite().all()) and (M <= 5 or bool(c[5:].isfinite().all()))
