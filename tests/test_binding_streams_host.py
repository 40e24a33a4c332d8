"""Where a call runs and where its own buffers come from, in the Python binding. CPU only: the library and
torch's streams are stood in for.

Memory is handed out by pools, one of each stream, and a block of the current stream's pool may still be in use by kernels that
wait there. A call on another stream therefore takes its outputs and workspaces from that stream's pool; an output,
which its caller may use and drop on the current stream, is recorded there."""

import contextlib

import pytest
import torch

import thread_block_lds_amd as tbl

CURRENT, SIDE = 0x1000, 0x2000


class Gpu(torch.Tensor):
    """A CPU tensor that says that it is on GPU ``at``."""

    is_cuda = property(lambda self: True)
    at = 0

    def get_device(self):
        return Gpu.at

    def record_stream(self, stream):
        Gpu.recorded.append((self.data_ptr(), stream.cuda_stream))


class Stream:
    def __init__(self, address, device=None):
        self.cuda_stream = int(address)


class Calls:
    """The library: sizes are the real one's, launches are noted."""

    def __init__(self, real):
        self.real, self.calls, self.on = real, [], []

    def __getattr__(self, name):
        if name.endswith("_workspace") or name in ("tbl_gemm_tile_shape", "tbl_status_string"):
            return getattr(self.real, name)
        if name == "tbl_device_info":
            return lambda *a: tbl.ERR_HIP

        def call(*args):
            self.calls.append((name, [getattr(a, "value", a) for a in args]))
            self.on.append(Gpu.current)
            return tbl.OK
        return call


@pytest.fixture
def gpu(monkeypatch):
    """(calls, made): the launches, and {address: stream that was current when the buffer was made}."""
    current, made = [CURRENT], {}
    Gpu.recorded, Gpu.at, Gpu.current = [], 0, 0
    calls = Calls(tbl.lib())

    @contextlib.contextmanager
    def on(stream):
        current.append(current[-1] if stream is None else stream.cuda_stream)
        yield
        current.pop()

    @contextlib.contextmanager
    def on_gpu(index):
        before, Gpu.current = Gpu.current, index
        yield
        Gpu.current = before

    def maker(make):
        def wrapped(*a, **k):
            k.pop("device", None)
            t = make(*a, **k)
            t = t if isinstance(t, Gpu) else t.as_subclass(Gpu)
            made[t.data_ptr()] = current[-1]
            wrapped.kept.append(t)   # so that no address comes twice
            return t
        wrapped.kept = []
        return wrapped

    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, maker(getattr(torch, name)))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "device", on_gpu)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: Gpu.current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(current[-1]))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: current[-1], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: Gpu.current, raising=False)
    monkeypatch.setattr(tbl, "lib", lambda: calls)
    return calls, made


def fake(shape, dtype):
    return torch.ones(shape).to(dtype).as_subclass(Gpu)


def quantized(rows, cols):
    return tbl.Fp8Blocks(fake((rows, cols), torch.float8_e4m3fn), fake((-(-cols // 128), rows), torch.float32))


def fp8_calls():
    x = fake((200, 300), torch.bfloat16)
    return {
        "quantize_fp8": lambda s: tbl.quantize_fp8(x, transposed=True, stream=s),
        "gemm_fp8": lambda s: tbl.gemm_fp8(quantized(200, 8192), quantized(300, 8192), stream=s),
        "gemm_fp8 of unaligned rows": lambda s: tbl.gemm_fp8(quantized(200, 300), quantized(300, 300), stream=s),
        "newton_schulz": lambda s: tbl.newton_schulz(x, stream=s),
    }


def other_calls():
    a, b = fake((512, 512), torch.float16), fake((512, 512), torch.float16)
    i = fake((64, 128), torch.int32)
    return {
        "gemm": lambda s: tbl.gemm(a, b, stream=s),
        "gemm of a tile": lambda s: tbl.gemm(a, b, tile=(256, 256, 32), stream=s),
        "gemm_dynamic": lambda s: tbl.gemm_dynamic(a, b, num_programs=3, stream=s),
        "gemm_dynamic_noalloc": lambda s: tbl.gemm_dynamic_noalloc(a, b, num_programs=3, stream=s),
        "gemm_lds_layout": lambda s: tbl.gemm_lds_layout(a, b, tbl.LDS_LAYOUTS[0], stream=s),
        "mfma_rate": lambda s: tbl.mfma_rate(a, b, workgroups=4, stream=s)[1:],
        "tile_map": lambda s: tbl.tile_map(tbl.ROW, 4, 4, stream=s)[:2],
        "transpose_i32": lambda s: tbl.transpose_i32(i, stream=s),
        "copy16": lambda s: tbl.copy16(i, stream=s),
    }


CALLS = {**fp8_calls(), **other_calls()}


def outputs(result):
    if isinstance(result, tbl.Fp8Blocks):
        return [result.codes, result.scale]
    if isinstance(result, tuple):
        return [t for r in result for t in outputs(r)]
    return [result] if isinstance(result, torch.Tensor) else []


@pytest.mark.parametrize("name", list(CALLS))
def test_buffers_come_from_the_stream_of_the_call(gpu, name):
    calls, made = gpu
    result = CALLS[name](SIDE)
    assert made and set(made.values()) == {SIDE}
    (_, args), = calls.calls
    assert args[-1] == SIDE
    for t in outputs(result):
        assert (t.data_ptr(), CURRENT) in Gpu.recorded


@pytest.mark.parametrize("stream", [None, CURRENT])
@pytest.mark.parametrize("name", list(CALLS))
def test_buffers_of_a_call_on_the_current_stream(gpu, name, stream):
    calls, made = gpu
    CALLS[name](stream)
    assert made and set(made.values()) == {CURRENT} and Gpu.recorded == []
    (_, args), = calls.calls
    assert args[-1] == CURRENT


@pytest.mark.parametrize("name", [n for n in CALLS if n != "tile_map"])
def test_a_call_runs_on_its_tensors_gpu(gpu, name):
    """A default stream's address is 0 on every GPU: it means the current GPU's."""
    calls, _ = gpu
    Gpu.at = 1
    CALLS[name](None)
    assert calls.on == [1] and Gpu.current == 0


def test_tile_map_runs_on_its_gpu(gpu):
    calls, _ = gpu
    tbl.tile_map(tbl.ROW, 4, 4, device="cuda:1")
    assert calls.on == [1] and Gpu.current == 0
