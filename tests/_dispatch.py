"""How the library runs a shape: the rules of gemm_fp8 and newton_schulz, asked through the library's own symbols."""

import ctypes

import thread_block_lds_amd as tbl


class _Gemm(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("floats", ctypes.c_int64)]


class _Ortho(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int), ("parts", ctypes.c_int)]


def gemm8(M, N, K, out):
    """(kernel, split): 0 streaming, 128 or 256 tiles; whether tiles are split along k."""
    f = tbl.lib()["_ZN3tbl10gemm8_planEllli"]
    f.restype, f.argtypes = _Gemm, [ctypes.c_int64] * 3 + [ctypes.c_int]
    p = f(M, N, K, out)
    return p.kernel, p.floats > 0


def ortho(batch, rows, cols):
    """(tile, parts) of P, Q, the update and the last update; tile 0: a short side."""
    f = tbl.lib()["_ZN3tbl13ortho_productEilll"]
    f.restype, f.argtypes = _Ortho, [ctypes.c_int] + [ctypes.c_int64] * 3
    return [(p.tile, p.parts) for p in (f(kind, batch, rows, cols) for kind in range(4))]
