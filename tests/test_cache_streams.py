"""Where the calls around the 8-bit cache take their memory, and on which stream they run, without a GPU: a
stand-in for torch and for the library that records both."""
import contextlib
import math
from types import SimpleNamespace

import pytest

MAIN, SIDE = 11, 22


class Tensor:
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
        return {"bf16": 2, "f32": 4, "u8": 1, "i32": 4}[self.dtype]

    def is_contiguous(self):
        return True

    def get_device(self):
        return int(self.device.split(":")[1]) if self.device != "cpu" else -1

    def data_ptr(self):
        return id(self)


class Stream:
    def __init__(self, cuda_stream, device="cuda:0"):
        self.cuda_stream, self.device = cuda_stream, device


@pytest.fixture
def world(monkeypatch):
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
        before, w.device = w.device, int(str(device).split(":")[1])
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
        bfloat16="bf16", float32="f32", uint8="u8", int32="i32", empty=empty, empty_like=lambda t: empty(t.shape, t.dtype, t.device),
        cuda=SimpleNamespace(stream=on, device=at),
        _C=SimpleNamespace(_cuda_getCurrentRawStream=lambda device: w.current + 100 * device, _cuda_getDevice=lambda: w.device))
    monkeypatch.setattr(qz, "_torch", lambda: torch)
    monkeypatch.setattr(qz, "_lib", Lib())
    return w


def calls(w, device="cuda:0", other=None):
    """Each public call on inputs on `device`, its handles on `other`."""
    qz, T, far = w.qz, Tensor, other or device
    cache = qz.KVCache(T((4, 2, 32, 64), "u8", far), T((4, 2, 2), "f32", far), T((4, 2, 32, 64), "u8", far), T((4, 2, 2), "f32", far), "int8")
    table = qz.RotaryTable(T((100, 32), "f32", far), T((100, 32), "f32", far))
    q, k = T((3, 4, 64), "bf16", device), T((3, 2, 64), "bf16", device)
    pages, lengths = T((3, 2), "i32", device), T((3,), "i32", device)
    return {
        "rotary": lambda **a: qz.rotary(q, table, **a),
        "rotary_backward": lambda **a: qz.rotary_backward(q, table, **a),
        "cache_append": lambda **a: qz.cache_append(cache, k, k, pages, lengths, rotary=table, q=q, **a),
        "cache_attention": lambda **a: qz.cache_attention(q, cache, pages, lengths, lse=True, **a),
    }


NAMES = ["rotary", "rotary_backward", "cache_append", "cache_attention"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_comes_from_the_stream_that_uses_it(world, name):
    calls(world)[name](stream=Stream(SIDE))
    assert world.taken and set(world.taken) == {SIDE}
    assert [s for _, s, _ in world.ran] == [SIDE] and world.current == MAIN


@pytest.mark.parametrize("name", NAMES)
def test_current_stream_is_the_default(world, name):
    calls(world)[name]()
    assert set(world.taken) == {MAIN} and [s for _, s, _ in world.ran] == [MAIN]


@pytest.mark.parametrize("name", NAMES)
def test_launches_on_the_device_of_the_inputs(world, name):
    calls(world, "cuda:1")[name]()
    assert [(s, d) for _, s, d in world.ran] == [(MAIN + 100, 1)] and world.device == 0


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("other", ["cuda:1", "cpu"])
def test_other_devices_are_refused(world, name, other):
    with pytest.raises(ValueError):
        calls(world, other=other)[name]()
    with pytest.raises(ValueError):
        calls(world)[name](stream=Stream(SIDE, "cuda:1"))
    assert not world.ran
