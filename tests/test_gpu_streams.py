"""Calls on a stream other than the current one take their buffers from that stream's pool, on the GPU: blocks that the
current stream has just given back, which its waiting kernels may still use, are not handed to them."""

import pytest
import torch

import thread_block_lds_amd as tbl
from test_gpu_quantised_gemm import values

pytestmark = pytest.mark.gpu


def given_back(*tensors):
    """The byte ranges of freshly freed blocks of the current stream's pool as large as ``tensors``, several of each."""
    held = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8, device="cuda") for t in tensors for _ in range(3)]
    ranges = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in held]
    torch.cuda.synchronize()
    return ranges


def outside(t, ranges):
    begin = t.data_ptr()
    end = begin + t.numel() * t.element_size()
    return all(end <= a or b <= begin for a, b in ranges)


def test_fp8_and_newton_schulz_outputs():
    x = values(300, 640, torch.bfloat16, 1).cuda()
    w = values(256, 640, torch.bfloat16, 2).cuda()
    want_x, want_t = tbl.quantize_fp8(x, transposed=True)
    want_w = tbl.quantize_fp8(w, rows=128)
    want_y, want_u = tbl.gemm_fp8(want_x, want_w), tbl.newton_schulz(x)
    ranges = given_back(want_x.codes, want_x.scale, want_t.codes, want_t.scale, want_y, want_u)
    side = torch.cuda.Stream()
    q, t = tbl.quantize_fp8(x, transposed=True, stream=side.cuda_stream)
    y = tbl.gemm_fp8(want_x, want_w, stream=side.cuda_stream)
    u = tbl.newton_schulz(x, stream=side.cuda_stream)
    for v in (q.codes, q.scale, t.codes, t.scale, y, u):
        assert outside(v, ranges)
    side.synchronize()
    assert torch.equal(q.codes.view(torch.uint8), want_x.codes.view(torch.uint8)) and torch.equal(t.scale, want_t.scale)
    assert torch.equal(t.codes.view(torch.uint8), want_t.codes.view(torch.uint8)) and torch.equal(q.scale, want_x.scale)
    assert torch.equal(y, want_y) and torch.equal(u, want_u)
