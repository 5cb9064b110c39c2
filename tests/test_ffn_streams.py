"""Where the calls with 4-bit weights and the layer norm take their memory, and on which stream they
run, without a GPU: a stand-in for torch and for the library that records both."""
import contextlib
import math
from types import SimpleNamespace

import pytest

MAIN, SIDE = 11, 22


class Tensor:
    """What the binding asks of a CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, device="cuda:0"):
        self.shape, self.dtype, self.device = tuple(shape), dtype, device

    def dim(self):
        return len(self.shape)

    def stride(self):
        return tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def numel(self):
        return math.prod(self.shape)

    def element_size(self):
        return {"bf16": 2, "f32": 4, "u8": 1}[self.dtype]

    def is_contiguous(self):
        return True

    def get_device(self):
        return int(self.device.split(":")[1]) if self.device != "cpu" else -1

    def data_ptr(self):
        return id(self)

    def unbind(self, _):
        return [Tensor(self.shape[1:], self.dtype, self.device) for _ in range(self.shape[0])]


class Stream:
    def __init__(self, cuda_stream, device="cuda:0"):
        self.cuda_stream, self.device = cuda_stream, device


@pytest.fixture
def world(monkeypatch):
    """The binding on the stand-ins; `taken`: the current stream at each allocation, `ran`: (call,
    stream argument) of each launch."""
    import precision_quantization_gb300 as qz
    w = SimpleNamespace(qz=qz, taken=[], ran=[], current=MAIN, device=0)

    def empty(shape, dtype, device):
        w.taken.append(w.current)
        return Tensor(shape, dtype, device)

    @contextlib.contextmanager
    def on(stream):
        before, w.current = w.current, stream.cuda_stream
        yield
        w.current = before

    @contextlib.contextmanager
    def at(device):
        before, w.device = w.device, device if isinstance(device, int) else int(str(device).split(":")[1])
        yield
        w.device = before

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("workspace"):
                    return 1024
                w.ran.append((name, args[-1], w.device))
                return 0
            return call

    torch = SimpleNamespace(
        bfloat16="bf16", float32="f32", uint8="u8", empty=empty, cuda=SimpleNamespace(stream=on, device=at),
        _C=SimpleNamespace(_cuda_getCurrentRawStream=lambda device: w.current + 100 * device,
                           _cuda_getDevice=lambda: w.device))
    monkeypatch.setattr(qz, "_torch", lambda: torch)
    monkeypatch.setattr(qz, "_lib", Lib())
    w.weight = lambda device="cuda:0": qz.Weight(qz.Quantized(
        Tensor((64, 64), "u8", device), Tensor((64, 8), "u8", device), Tensor((1,), "f32", device), qz.QZ_NVFP4,
        qz.QZ_GRAN_BLOCK, 0, 64, 128, 16))
    return w


def calls(w, device="cuda:0"):
    """Each public call on its own inputs, as functions of the keyword arguments left."""
    qz, h = w.qz, w.weight(device)
    x, y = Tensor((4, 128), "bf16", device), Tensor((4, 64), "bf16", device)
    row = Tensor((4,), "f32", device)
    return {
        "linear": lambda **k: qz.linear(x, h, **k),
        "linear_backward": lambda **k: qz.linear_backward(y, h, **k),
        "gated_ffn": lambda **k: qz.gated_ffn(x, h, h, save=True, **k),
        "gated_ffn_backward": lambda **k: qz.gated_ffn_backward(y, y, y, h, h, **k),
        "layer_norm": lambda **k: qz.layer_norm(x, **k),
        "layer_norm_backward": lambda **k: qz.layer_norm_backward(x, x, row, row, **k),
    }


NAMES = ["linear", "linear_backward", "gated_ffn", "gated_ffn_backward", "layer_norm", "layer_norm_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_comes_from_the_stream_that_uses_it(world, name):
    """A block of the current stream's pool may be in use there, and is handed out there again as soon
    as the call drops it; the kernels on the other stream wait for neither."""
    calls(world)[name](stream=Stream(SIDE))
    assert world.taken and set(world.taken) == {SIDE}
    assert [s for _, s, _ in world.ran] == [SIDE] and world.current == MAIN


@pytest.mark.parametrize("name", NAMES)
def test_current_stream_is_the_default(world, name):
    calls(world)[name]()
    assert set(world.taken) == {MAIN} and [s for _, s, _ in world.ran] == [MAIN]


def test_stream_of_another_device(world):
    with pytest.raises(ValueError):
        calls(world)["linear"](stream=Stream(SIDE, "cuda:1"))
    assert not world.ran


@pytest.mark.parametrize("name", NAMES)
def test_launches_on_the_device_of_the_inputs(world, name):
    """Inputs on a device that is not the current one: the call runs there, on its current stream."""
    calls(world, "cuda:1")[name]()
    assert [(s, d) for _, s, d in world.ran] == [(MAIN + 100, 1)] and world.device == 0


def test_other_devices_are_refused(world):
    qz, here, cpu, far = world.qz, world.weight(), world.weight("cpu"), world.weight("cuda:1")
    m = lambda rows, cols, device="cuda:0": Tensor((rows, cols), "bf16", device)  # noqa: E731
    v = lambda n, device="cuda:0": Tensor((n,), "f32", device)  # noqa: E731
    x, y = m(4, 128), m(4, 64)
    refused = [lambda w=w: qz.linear(x, w) for w in (cpu, far)]
    refused += [lambda w=w: qz.linear_backward(y, w) for w in (cpu, far)]
    refused += [lambda w=w: qz.gated_ffn(x, *w) for w in ((cpu, here), (here, cpu), (far, here), (here, far))]
    refused += [lambda w=w: qz.gated_ffn_backward(y, y, y, *w) for w in ((here, far), (cpu, here))]
    for d in ("cpu", "cuda:1"):
        mixed = qz.Quantized(Tensor((64, 64), "u8"), Tensor((64, 8), "u8", d), v(1), qz.QZ_NVFP4, qz.QZ_GRAN_BLOCK, 0, 64, 128, 16)
        scale = qz.Quantized(Tensor((64, 64), "u8"), Tensor((64, 8), "u8"), v(1, d), qz.QZ_NVFP4, qz.QZ_GRAN_BLOCK, 0, 64, 128, 16)
        refused += [lambda q=mixed: qz.Weight(q), lambda q=scale: qz.Weight(q),
                    lambda d=d: qz.linear(x, here, out=m(4, 64, d)), lambda d=d: qz.linear_backward(y, here, out=m(4, 128, d)),
                    lambda d=d: qz.gated_ffn(x, here, here, out=m(4, 64, d)),
                    lambda d=d: qz.gated_ffn(x, here, here, save=True, out=(y, y, m(4, 64, d))),
                    lambda d=d: qz.gated_ffn_backward(y, m(4, 64, d), y, here, here),
                    lambda d=d: qz.gated_ffn_backward(y, y, y, here, here, out=(x, y, m(4, 64, d))),
                    lambda d=d: qz.layer_norm(x, v(128, d)), lambda d=d: qz.layer_norm(x, out=(x, v(4, d), v(4))),
                    lambda d=d: qz.layer_norm_backward(m(4, 128, d), x, v(4), v(4)),
                    lambda d=d: qz.layer_norm_backward(x, x, v(4, d), v(4)),
                    lambda d=d: qz.layer_norm_backward(x, x, v(4), v(4), out=(x, v(128), v(128, d))),
                    lambda d=d: qz.layer_norm_backward(x, x, v(4), v(4), workspace=Tensor((1024,), "u8", d))]
    two_bytes = qz.Quantized(Tensor((64, 64), "u8"), Tensor((64, 8), "u8"), Tensor((1,), "bf16"), qz.QZ_NVFP4, qz.QZ_GRAN_BLOCK, 0, 64, 128, 16)
    gaps = Tensor((1024,), "u8")
    gaps.is_contiguous = lambda: False
    refused += [lambda: qz.Weight(two_bytes), lambda: qz.layer_norm_backward(x, x, v(4), v(4), workspace=gaps)]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    assert not world.ran


def test_a_weight_keeps_its_buffers(world):
    """Codes, scales and tensor scale live as long as the handle that points to them, whatever the
    Quantized they came from refers to by then."""
    import gc
    import weakref
    q = world.qz.Quantized(Tensor((64, 64), "u8"), Tensor((64, 8), "u8"), Tensor((1,), "f32"), world.qz.QZ_NVFP4,
                           world.qz.QZ_GRAN_BLOCK, 0, 64, 128, 16)
    refs = [weakref.ref(t) for t in (q.codes, q.scales, q.tensor_scale)]
    w = world.qz.Weight(q)
    q.codes, q.scales, q.tensor_scale = Tensor((64, 64), "u8"), Tensor((64, 8), "u8"), Tensor((1,), "f32")
    gc.collect()
    assert [r() is not None and r().data_ptr() for r in refs] == [w.desc.codes, w.desc.scales, w.desc.tensor_scale_dev]
    del w
    gc.collect()
    assert all(r() is None for r in refs)
