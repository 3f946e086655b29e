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


def older_calls():
    T = Tensor
    f32, f16 = torch.float32, torch.float16
    w, s, M = T((64, 4), torch.int32), T((64,), f32), T((8, 8), f32)
    a, t_inv = T((8, 128), f16), T((1, 128, 128), f16)
    return {
        "pack_signs": lambda **k: lq.pack_signs(T((64, 128), torch.uint8), **k),
        "unpack_signs": lambda **k: lq.unpack_signs(w, 128, **k),
        "lift": lambda **k: lq.lift(a, t_inv, M, 8, 8, **k),
        "lift_parts": lambda **k: lq.lift_parts(a, t_inv, M, 8, 8, **k),
        "lift_kron": lambda **k: lq.lift_kron(a, T((128,), f32), T((16, 16), f32), T((8, 8), f32),
                                              T((16,), f32), M, 8, 8, **k),
        "encode": lambda **k: lq.encode(T((50, 8), f32), M, T((0, 8), f32), **k),
        "layer_b1": lambda **k: lq.layer_b1(T((1, 128), f16), t_inv, M, 8, 8, w, s, **k),
        "gemm_decoded": lambda **k: lq.gemm_decoded(w, s, M, 8, 8, a, **k),
        "softmin_grad": lambda **k: lq.softmin_grad(T((50, 8), f32), M, **k),
        "gemv": lambda **k: lq.gemv(w, s, T((8, 128), f32), **k),
        "gemv_parts": lambda **k: lq.gemv_parts(w, s, T((4096,), torch.uint8), 128, 8, **k),
        "gemm": lambda **k: lq.gemm(w, s, a, **k),
    }


@pytest.mark.parametrize("name", sorted(older_calls()))
def test_memory_of_the_other_wrappers_comes_from_the_stream_of_the_call(gpu, name):
    """Their workspaces are kept per stream and filled with zeros when made: on that stream too."""
    out = older_calls()[name](stream=gpu.other)
    assert gpu.handles == [77] and gpu.made
    assert all(t.owner is gpu.other for t in gpu.made)
    for t in out if isinstance(out, tuple) else (out,):
        assert gpu.default.cuda_stream in t.used_on
    older_calls()[name]()
    assert gpu.handles == [77, 0]


def test_wrappers_without_results_take_a_stream(gpu):
    buf, sink = Tensor((4096,), torch.uint8), Tensor((4096,), torch.int32)
    assert lq.stream_read(buf, sink, stream=gpu.other) is None and buf.used_on == {77}
    four = [Tensor((8, 8), torch.float32) for _ in range(4)]
    assert lq.adam_update(*four, 1, 0.01, stream=gpu.other) is None
    w, s, a, out = Tensor((64, 4), torch.int32), Tensor((64,), torch.float32), Tensor((8, 128), torch.float32), Tensor((8, 64), torch.float32)
    assert lq.gemv_noalloc(w, s, a, out, stream=gpu.other) is out and out.used_on == {77}
    assert gpu.handles == [77, 77, 77]


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


def test_tensors_in_lists_are_kept_too(gpu):
    a, b, c = (Tensor((8, 8), torch.float32) for _ in range(3))

    @lq._on_stream
    def call(x, several, stream=None):
        return a, [c, None]
    assert call(a, [b, (c, 3)], stream=gpu.other)[0] is a
    assert a.used_on == b.used_on == c.used_on == {77}        # given, so not made by the call
    d = Tensor((8, 8), torch.float32)
    call2 = lq._on_stream(lambda x, stream=None: (x, [d]))
    call2(a, stream=gpu.other)
    assert d.used_on == {0}
