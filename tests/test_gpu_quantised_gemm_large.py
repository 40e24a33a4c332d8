"""gemm_fp8 with 256 tiles over many groups: whole and split along k, ragged in every size, scales of either layout, with
an added matrix. The bounds are those of test_gpu_quantised_gemm.py, the 64-bit products are taken on the GPU."""

import pytest
import torch

import thread_block_lds_amd as tbl
from _dispatch import gemm8
from test_gpu_quantised_gemm import E4M3, E5M2, TINY, U

pytestmark = pytest.mark.gpu


def stored(rows, cols, fmt, block, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-3, 4, (rows, cols), generator=g, device="cuda").float())
    return tbl.quantize_fp8(x, fmt=fmt, rows=block)


def dequantized(q):
    c, s = q.codes.float().double(), q.scale.double()
    rows, cols = c.shape
    full = s.t() if q.rows == 1 else s.repeat_interleave(128, 0)[:rows]
    return c * full.repeat_interleave(128, 1)[:, :cols]


def check_product(c, qa, qb, add):
    a, b = dequantized(qa), dequantized(qb).t().contiguous()
    K = a.shape[1]
    ref, size = torch.mm(a, b), torch.mm(a.abs(), b.abs())
    if add is not None:
        ref, size = ref + add.double(), size + add.double().abs()
    u = U[c.dtype]
    bound = (2 * K + 4) * 2.0 ** -24 * size + u * ref.abs() + TINY[c.dtype]
    if c.dtype != torch.float32:
        bound = (1 + u) * (bound + 2.0 ** -10 * size)
    bad = (~((c.double() - ref).abs() <= bound)).nonzero()
    assert len(bad) == 0, f"{len(bad)} elements beyond the bound, first at {bad[0].tolist()}: {c[tuple(bad[0])]} want {ref[tuple(bad[0])]}"


@pytest.mark.parametrize("M,N,K,fa,fb,ba,bb,out,add", [
    (3001, 4099, 1111, E4M3, E4M3, 1, 1, torch.float16, False),
    (3001, 4099, 1111, E4M3, E5M2, 128, 128, torch.bfloat16, True),
    (4500, 4700, 1234, E4M3, E4M3, 1, 128, torch.bfloat16, True),
    (4500, 4700, 1234, E5M2, E4M3, 1, 1, torch.float16, False),
    (4096, 4100, 3001, E5M2, E4M3, 1, 1, torch.bfloat16, True),
    (4096, 4100, 3001, E5M2, E5M2, 1, 128, torch.bfloat16, False),
    (4097, 4095, 1100, E4M3, E4M3, 128, 1, torch.bfloat16, False),
])
def test_256_tiles(M, N, K, fa, fb, ba, bb, out, add):
    print(f"gemm_fp8 {M}x{N}x{K} {fa} {fb} {ba} {bb} {out} {gemm8(M, N, K, 1)}", flush=True)
    a, b = stored(M, K, fa, ba, 1), stored(N, K, fb, bb, 2)
    plus = torch.randn(M, N, device="cuda") if add else None
    c = tbl.gemm_fp8(a, b, add=plus, out_dtype=out)
    check_product(c, a, b, plus)
    assert torch.equal(c, tbl.gemm_fp8(a, b, add=plus, out_dtype=out))


@pytest.mark.parametrize("M,N,K", [(3001, 4099, 1111), (4500, 4700, 1234)])
def test_256_tiles_ignore_what_lies_past_k(M, N, K):
    """Bytes of a row past K may hold NaN codes."""
    a, b = stored(M, 1280, E4M3, 1, 3), stored(N, 1280, E4M3, 1, 4)
    groups = -(-K // 128)
    sliced = []
    for q in (a, b):
        codes = q.codes.clone()
        codes[:, K:].view(torch.uint8).fill_(0x7F)
        sliced.append(tbl.Fp8Blocks(codes[:, :K], q.scale[:groups].contiguous(), 1))
    check_product(tbl.gemm_fp8(*sliced), *sliced, None)
