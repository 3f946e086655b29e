"""Where the Python wrappers take memory when a stream is given (no GPU needed:
tensors, streams and the library are stand-ins that write down what is asked of
them).  Memory of torch's allocator belongs to the stream that is current when
it is asked for: a block that a call on stream A has given back may still be
written there, and only work on A is ordered behind that.  So the workspace and
the results of a call on stream B have to come from B."""
import contextlib
import types

import pytest
import torch

from bit_lifted_gemv_amd import lq

DEV = torch.device("cuda", 0)
SIZE = {torch.float32: 4, torch.float16: 2, torch.bfloat16: 2, torch.int32: 4, torch.uint8: 1}


class Tensor:
    is_cuda = True
    device = DEV

    def __init__(self, shape, dtype, owner=None):
        self.shape, self.dtype, self.owner, self.used_on = torch.Size(shape), dtype, owner, set()

    def stride(self, i=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000000

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return SIZE[self.dtype]

    def view(self, *_):
        return self

    def unbind(self):
        part = Tensor(self.shape[1:], self.dtype, self.owner)
        part.used_on = self.used_on                    # of one storage
        return (part,) * self.shape[0]

    def record_stream(self, stream):
        self.used_on.add(stream.cuda_stream)


class Stream(types.SimpleNamespace):
    pass


@pytest.fixture
def gpu(monkeypatch):
    """A machine with two streams, whose library succeeds and asks for workspaces."""
    g = types.SimpleNamespace(default=Stream(cuda_stream=0, device=DEV), made=[], handles=[])
    g.current = g.default
    g.other = Stream(cuda_stream=77, device=DEV)

    @contextlib.contextmanager
    def use(stream):
        before, g.current = g.current, stream
        yield
        g.current = before

    def empty(*shape, dtype=torch.float32, device=None):
        shape = shape[0] if isinstance(shape[0], (tuple, list)) else shape
        t = Tensor(shape, dtype, g.current)
        g.made.append(t)
        return t

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_size"):
                    args[-1]._obj.value = 1024
                else:
                    g.handles.append(args[-1])
                return 0
            return call

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "zeros", empty)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: g.current)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: g.current.cuda_stream)
    monkeypatch.setattr(lq, "lib", Library)
    monkeypatch.setattr(lq, "_bytes_needed", lambda *a: 1024)
    monkeypatch.setattr(lq, "_WS", {})
    return g


def calls():
    T = Tensor
    w, s, a = T((64, 4), torch.int32), T((64,), torch.float32), T((40, 128), torch.float16)
    we, se = T((4, 64, 4), torch.int32), T((4, 64), torch.float32)
    off = T((5,), torch.int32)
    pos, weight = T((20, 2), torch.int32), T((20, 2), torch.float32)
    return {
        "gemm_ep": lambda **k: lq.gemm_ep(w, s, a, **k),
        "gemm_grouped": lambda **k: lq.gemm_grouped(we, se, a, off, **k),
        "gemm_join": lambda **k: lq.gemm_join(we, se, a, off, pos, weight, **k),
        "route": lambda **k: lq.route(T((40, 8), torch.float32), 2, **k),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_memory_comes_from_the_stream_of_the_call(gpu, name):
    out = calls()[name](stream=gpu.other)
    assert gpu.handles == [77] and len(gpu.made) >= 2
    assert all(t.owner is gpu.other for t in gpu.made)
    assert gpu.current is gpu.default
    # results are the caller's, who may let go of them while its own stream still reads
    for t in out if isinstance(out, tuple) else (out,):
        assert gpu.default.cuda_stream in t.used_on
    gpu.made.clear()
    calls()[name]()
    assert gpu.handles == [77, 0] and all(t.owner is gpu.default for t in gpu.made)


def test_arguments_are_kept_for_the_stream_of_the_call(gpu):
    w, s = Tensor((64, 4), torch.int32), Tensor((64,), torch.float32)
    a, bias = Tensor((40, 128), torch.float16), Tensor((64,), torch.float32)
    out = Tensor((40, 64), torch.float16, gpu.default)
    assert lq.gemm_ep(w, s, a, bias, out=out, stream=gpu.other) is out
    assert all(t.used_on == {77} for t in (w, s, a, bias, out))
    lq.gemm_ep(w, s, a, bias, "none", False, None, None, out, gpu.other)        # all by position
    assert gpu.handles == [77, 77]


def test_stream_of_another_device_is_refused(gpu):
    other = Stream(cuda_stream=5, device=torch.device("cuda", 1))
    w, s, a = Tensor((64, 4), torch.int32), Tensor((64,), torch.float32), Tensor((40, 128), torch.float16)
    with pytest.raises(ValueError):
        lq.gemm_ep(w, s, a, stream=other)
    assert not gpu.handles
