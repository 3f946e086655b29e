"""Refusals of the 8-bit layers and of the rows sorted by expert, on the host and
before any HIP call, and where the Python wrappers take their memory (no GPU
needed)."""
import ctypes

import pytest
import torch

from bit_lifted_gemv_amd import lq
from test_streams_cpu import SIZE, Tensor, gpu  # noqa: F401

P = 0x10000000          # never dereferenced
MIS = P + 2
F32, F16, BF16, E4M3, E5M2, E8M0 = range(6)
NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5, 7


@pytest.fixture(scope="module")
def L():
    return lq.load_library()


def size(f, *args):
    n = ctypes.c_size_t(0)
    assert f(*args, ctypes.byref(n)) == 0
    return n.value


def quant(L, **over):
    a = dict(x=P, dt=F16, rows=5, K=300, ld=300, q=P, qdt=E4M3, ldq=384, e=P, lde=4)
    a.update(over)
    return L.lq_quant8(a["x"], a["dt"], a["rows"], a["K"], a["ld"], a["q"], a["qdt"], a["ldq"], a["e"], a["lde"], None)


@pytest.mark.parametrize("over,status", [
    (dict(x=None), NULL), (dict(q=None), NULL), (dict(e=None), NULL), (dict(dt=E4M3), DTYPE), (dict(dt=9), DTYPE),
    (dict(qdt=F16), DTYPE), (dict(qdt=E8M0), DTYPE), (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(K=0), SHAPE),
    (dict(K=(1 << 22) + 1, ld=1 << 23, ldq=1 << 23, lde=1 << 17), SHAPE), (dict(ld=299), SHAPE), (dict(ldq=368), SHAPE),
    (dict(lde=2), SHAPE), (dict(lde=5), ALIGN), (dict(ldq=392), ALIGN), (dict(q=P + 8), ALIGN), (dict(e=MIS), ALIGN),
    (dict(x=P + 1), ALIGN), (dict(dt=F32, x=MIS), ALIGN), (dict(rows=0, x=None), 0),
])
def test_quant_refusals(L, over, status):
    assert quant(L, **over) == status


def quant_blocks(L, **over):
    a = dict(w=P, dt=F32, E=2, m=200, K=300, ld=300, q=P, ldq=384, e=P, lde=4)
    a.update(over)
    return L.lq_quant8_blocks(a["w"], a["dt"], a["E"], a["m"], a["K"], a["ld"], a["q"], a["ldq"], a["e"], a["lde"], None)


@pytest.mark.parametrize("over,status", [
    (dict(w=None), NULL), (dict(q=None), NULL), (dict(e=None), NULL), (dict(dt=E4M3), DTYPE), (dict(E=0), SHAPE),
    (dict(E=1025), SHAPE), (dict(m=0), SHAPE), (dict(m=(1 << 22) + 1), SHAPE), (dict(K=0), SHAPE), (dict(ld=10), SHAPE),
    (dict(ldq=300), SHAPE), (dict(lde=3), ALIGN), (dict(ldq=408), ALIGN), (dict(q=MIS), ALIGN), (dict(w=MIS), ALIGN),
])
def test_quant_blocks_refusals(L, over, status):
    assert quant_blocks(L, **over) == status


def gemm8(L, **over):
    a = dict(w=P, m=4096, K=4000, ldw=4096, s=P, st=E8M0, lds=32, a=P + (1 << 28), adt=E4M3, lda=4096, e=P, lde=32, B=300,
             bias=None, act=0, gated=0, res=None, ldr=0, out=P, odt=BF16, ldo=4096, ws=P, n=1 << 32)
    a.update(over)
    return L.lq_gemm8(a["w"], a["m"], a["K"], a["ldw"], a["s"], a["st"], a["lds"], a["a"], a["adt"], a["lda"], a["e"],
                      a["lde"], a["B"], a["bias"], a["act"], a["gated"], a["res"], a["ldr"], a["out"], a["odt"], a["ldo"],
                      a["ws"], a["n"], None)


COMMON = [
    (dict(w=None), NULL), (dict(s=None), NULL), (dict(a=None), NULL), (dict(out=None), NULL), (dict(e=None), NULL),
    (dict(adt=F32), DTYPE), (dict(adt=E8M0), DTYPE), (dict(st=F16), DTYPE), (dict(st=E4M3), DTYPE), (dict(odt=E4M3), DTYPE),
    (dict(act=5), UNSUPPORTED), (dict(act=-1), UNSUPPORTED), (dict(m=0), SHAPE), (dict(m=65, gated=1), SHAPE),
    (dict(K=0), SHAPE), (dict(K=(1 << 22) + 1, ldw=1 << 23), SHAPE), (dict(ldw=3984), SHAPE), (dict(ldw=4104), ALIGN),
    (dict(m=1 << 20), SHAPE), (dict(lds=31), SHAPE), (dict(lds=33), ALIGN), (dict(lds=33, s=MIS, st=F32), ALIGN),
    (dict(lda=3984), SHAPE), (dict(lda=4104), ALIGN), (dict(lde=31), SHAPE), (dict(lde=34), ALIGN), (dict(w=P + 8), ALIGN),
    (dict(a=P + 8), ALIGN), (dict(e=MIS), ALIGN), (dict(s=MIS), ALIGN), (dict(bias=MIS), ALIGN), (dict(ldo=63), SHAPE),
    (dict(out=P + 1), ALIGN), (dict(adt=F16, lda=3999), SHAPE), (dict(adt=F16, a=P + (1 << 28) + 1), ALIGN),
    (dict(adt=F16, ws=None), WORKSPACE), (dict(adt=F16, n=100), WORKSPACE), (dict(adt=F16, ws=P + 16), ALIGN),
    (dict(lda=1 << 40), SHAPE),
]


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(B=0), SHAPE), (dict(B=-1), SHAPE), (dict(B=1 << 31), SHAPE), (dict(B=1 << 20, K=4096), SHAPE),
    (dict(res=P, ldr=63), SHAPE), (dict(res=P + 1, ldr=4096), ALIGN), (dict(out=P + (1 << 28)), UNSUPPORTED),
    (dict(out=P, res=P, ldr=8192), UNSUPPORTED),
])
def test_gemm8_refusals(L, over, status):
    assert gemm8(L, **over) == status
    assert L.lq_last_error()


def grouped(L, **over):
    a = dict(w=P, E=4, m=4096, K=4000, ldw=4096, s=P, st=E8M0, lds=32, a=P + (1 << 28), adt=E4M3, lda=4096, e=P, lde=32,
             ar=500, rows=P, off=P, R=1000, bias=None, act=0, gated=0, out=P, odt=BF16, ldo=4096, ws=P, n=1 << 32)
    a.update(over)
    return L.lq_gemm8_grouped(a["w"], a["E"], a["m"], a["K"], a["ldw"], a["s"], a["st"], a["lds"], a["a"], a["adt"],
                              a["lda"], a["e"], a["lde"], a["ar"], a["rows"], a["off"], a["R"], a["bias"], a["act"],
                              a["gated"], a["out"], a["odt"], a["ldo"], a["ws"], a["n"], None)


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(R=-1), SHAPE), (dict(R=1 << 31), SHAPE), (dict(rows=None), SHAPE),
    (dict(ar=0), SHAPE), (dict(ar=-1), SHAPE), (dict(ar=1 << 21), SHAPE), (dict(off=None), NULL), (dict(off=MIS), ALIGN), (dict(rows=MIS), ALIGN),
    (dict(R=0, w=None), 0),
])
def test_gemm8_grouped_refusals(L, over, status):
    assert grouped(L, **over) == status


def test_workspaces(L):
    n = ctypes.c_size_t(0)
    f, g = L.lq_gemm8_workspace_size, L.lq_gemm8_grouped_workspace_size
    assert size(f, 4096, 4096, BF16, 300) >= 300 * 4096
    assert gemm8(L, adt=BF16, n=size(f, 4096, 4000, BF16, 300) - 1) == WORKSPACE
    assert f(4096, 4096, F32, 3, ctypes.byref(n)) == DTYPE
    assert f(0, 4096, BF16, 3, ctypes.byref(n)) == SHAPE
    assert f(64, 128, BF16, 3, None) == NULL
    assert g(0, 64, 128, BF16, 3, 3, ctypes.byref(n)) == SHAPE
    assert g(4, 64, 128, BF16, 3, -1, ctypes.byref(n)) == SHAPE
    assert g(4, 64, 128, BF16, 3, 3, None) == NULL
    assert size(f, 1, 1, E4M3, 1) >= 0 and size(g, 4, 65, 128, E5M2, 0, 0) == 0   # an odd m has no gated form


def sort(L, **over):
    a = dict(x=P, size=2, T=10, n=64, ldx=64, rows=P, R=20, out=P + 4096, ldo=64)
    a.update(over)
    return L.lq_sort_rows(a["x"], a["size"], a["T"], a["n"], a["ldx"], a["rows"], a["R"], a["out"], a["ldo"], None)


@pytest.mark.parametrize("over,status", [
    (dict(x=None), NULL), (dict(rows=None), NULL), (dict(out=None), NULL), (dict(size=3), DTYPE), (dict(size=8), DTYPE),
    (dict(size=0), DTYPE), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(R=-1), SHAPE), (dict(R=1 << 31), SHAPE),
    (dict(n=0), SHAPE), (dict(n=(1 << 30) + 1, ldx=1 << 31, ldo=1 << 31), SHAPE), (dict(ldx=63), SHAPE), (dict(ldo=63), SHAPE),
    (dict(x=P + 1), ALIGN), (dict(out=P + 1), ALIGN), (dict(rows=MIS), ALIGN), (dict(out=P), UNSUPPORTED), (dict(R=0, x=None), 0),
])
def test_sort_refusals(L, over, status):
    assert sort(L, **over) == status


def join(L, **over):
    a = dict(z=P, dt=BF16, R=20, n=64, ldz=64, pos=P, wt=P, T=10, k=2, res=None, ldr=0, out=P + 4096, odt=BF16, ldo=64)
    a.update(over)
    return L.lq_join_rows(a["z"], a["dt"], a["R"], a["n"], a["ldz"], a["pos"], a["wt"], a["T"], a["k"], a["res"], a["ldr"],
                          a["out"], a["odt"], a["ldo"], None)


@pytest.mark.parametrize("over,status", [
    (dict(z=None), NULL), (dict(pos=None), NULL), (dict(out=None), NULL), (dict(dt=E4M3), DTYPE), (dict(odt=7), DTYPE),
    (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 30), SHAPE), (dict(R=-1), SHAPE), (dict(n=0), SHAPE),
    (dict(ldz=63), SHAPE), (dict(ldo=63), SHAPE), (dict(res=P, ldr=63), SHAPE), (dict(pos=MIS), ALIGN), (dict(wt=MIS), ALIGN),
    (dict(z=P + 1), ALIGN), (dict(out=P + 1), ALIGN), (dict(out=P), UNSUPPORTED), (dict(res=P + 4096, ldr=128), UNSUPPORTED),
    (dict(T=0, z=None), 0),
])
def test_join_refusals(L, over, status):
    assert join(L, **over) == status


def grad(L, **over):
    a = dict(dy=P, dt=F32, ldy=64, z=P + 4096, ldz=64, R=20, n=64, pos=P, wt=P, T=10, k=2, rows=P, dz=P + 8192, lddz=64, dw=P)
    a.update(over)
    return L.lq_join_rows_grad(a["dy"], a["dt"], a["ldy"], a["z"], a["ldz"], a["R"], a["n"], a["pos"], a["wt"], a["T"],
                               a["k"], a["rows"], a["dz"], a["lddz"], a["dw"], None)


@pytest.mark.parametrize("over,status", [
    (dict(dy=None), NULL), (dict(z=None), NULL), (dict(pos=None), NULL), (dict(wt=None), NULL), (dict(dz=None), NULL),
    (dict(dw=None), NULL), (dict(dt=E5M2), DTYPE), (dict(k=0), SHAPE), (dict(T=-1), SHAPE), (dict(R=1 << 31), SHAPE),
    (dict(n=0), SHAPE), (dict(ldy=63), SHAPE), (dict(ldz=63), SHAPE), (dict(lddz=63), SHAPE), (dict(dy=MIS), ALIGN),
    (dict(z=MIS), ALIGN), (dict(dz=MIS), ALIGN), (dict(pos=MIS), ALIGN), (dict(rows=MIS), ALIGN), (dict(dw=MIS), ALIGN),
    (dict(dz=P), UNSUPPORTED), (dict(dz=P + 4096), UNSUPPORTED), (dict(T=0, R=0, dy=None), 0), (dict(T=0, rows=None, dz=None), 0),
])
def test_grad_refusals(L, over, status):
    assert grad(L, **over) == status


def test_wrappers_refuse_what_they_cannot_take():
    z, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    w = lq.Blocks8(torch.zeros(8, 128, dtype=torch.float8_e4m3fn), torch.zeros(1, 4, dtype=torch.uint8)[:, :1])
    with pytest.raises(ValueError):
        lq.quantize8(z)
    with pytest.raises(ValueError):
        lq.quantize8_blocks(z)
    with pytest.raises(ValueError):
        lq.gemm8(w, torch.zeros(2, 128, dtype=torch.float16))
    with pytest.raises(ValueError):
        lq.gemm8_grouped(w._replace(values=w.values[None], scales=w.scales[None]), torch.zeros(2, 128, dtype=torch.float16), i[0])
    with pytest.raises(ValueError):
        lq.sort_rows(z, i[:, 0].contiguous())
    with pytest.raises(ValueError):
        lq.join_rows(z, i)
    with pytest.raises(ValueError):
        lq.join_rows_grad(z, z, i, torch.zeros(4, 2))


def test_scales_whose_rows_are_not_whole_words_are_refused():
    values = torch.zeros(200, 384, dtype=torch.float8_e4m3fn)
    ok = torch.zeros(2, 4, dtype=torch.uint8)[:, :3]
    assert lq._weights8(lq.Blocks8(values, ok), ()) == (E8M0, 4)
    assert lq._weights8(lq.Blocks8(values, torch.zeros(2, 3)), ()) == (F32, 3)
    for bad in (torch.zeros(2, 3, dtype=torch.uint8), torch.zeros(8, dtype=torch.uint8)[1:].as_strided((2, 3), (4, 1)),
                torch.zeros(3, 2, dtype=torch.uint8).t(), torch.zeros(2, 4, dtype=torch.uint8), torch.zeros(1, 3, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            lq._weights8(lq.Blocks8(values, bad), ())
    with pytest.raises(TypeError):
        lq._weights8(lq.Blocks8(values, torch.zeros(2, 3, dtype=torch.float16)), ())
    with pytest.raises(TypeError):
        lq._weights8(lq.Blocks8(values.view(torch.uint8), ok), ())
    with pytest.raises(ValueError):
        lq._weights8(lq.Blocks8(values[:, :300].contiguous(), ok), ())
    with pytest.raises(ValueError):                     # matrices apart
        lq._weights8(lq.Blocks8(torch.zeros(2, 200, 384, dtype=torch.float8_e4m3fn), torch.zeros(2, 3, 4, dtype=torch.uint8)[:, :2, :3]), (2,))


def test_transposed_weights():
    values = torch.arange(3 * 256).reshape(3, 256).to(torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros(1, 4, dtype=torch.uint8)
    scales[0, :2] = torch.tensor([7, 9], dtype=torch.uint8)
    for s in (scales[:, :2], torch.tensor([[0.5, 2.0]])):
        t = lq.Blocks8(values, s).transposed()
        assert t.values.shape == (256, 128) and t.values.is_contiguous()
        assert torch.equal(t.values.view(torch.uint8)[:, :3], values.view(torch.uint8).t())
        assert (t.values.view(torch.uint8)[:, 3:] == 0).all()
        assert torch.equal(t.scales, s.t())
        lq._weights8(t, ())


class Tensor8(Tensor):
    """A stand-in that also says what the new wrappers ask."""

    def __getitem__(self, _):
        return self

    def storage_offset(self):
        return 0

    def untyped_storage(self):
        class Storage:
            nbytes = staticmethod(lambda: 1 << 30)
        return Storage


def calls8():
    T = Tensor8
    f8, u8, i32, f16, f32 = torch.float8_e4m3fn, torch.uint8, torch.int32, torch.float16, torch.float32
    w, we = lq.Blocks8(T((64, 128), f8), T((1, 1), u8)), lq.Blocks8(T((4, 64, 128), f8), T((4, 1, 1), f32))
    a, pos, weight = T((40, 128), f16), T((20, 2), i32), T((20, 2), f32)
    return {
        "quantize8": lambda **k: lq.quantize8(a, **k),
        "quantize8_blocks": lambda **k: lq.quantize8_blocks(a, **k),
        "gemm8": lambda **k: lq.gemm8(w, a, **k),
        "gemm8_grouped": lambda **k: lq.gemm8_grouped(we, a, T((5,), i32), **k),
        "sort_rows": lambda **k: lq.sort_rows(a, T((80,), i32), **k),
        "join_rows": lambda **k: lq.join_rows(a, pos, weight, **k),
        "join_rows_grad": lambda **k: lq.join_rows_grad(T((20, 128), f16), a, pos, weight, T((40,), i32), **k),
    }


@pytest.fixture
def gpu8(gpu, monkeypatch):  # noqa: F811
    empty = torch.empty

    def empty8(*shape, **k):
        t = empty(*shape, **k)
        t.__class__ = Tensor8
        return t
    monkeypatch.setattr(torch, "empty", empty8)
    monkeypatch.setitem(SIZE, torch.float8_e4m3fn, 1)
    return gpu


@pytest.mark.parametrize("name", sorted(calls8()))
def test_memory_comes_from_the_stream_of_the_call(gpu8, name):
    out = calls8()[name](stream=gpu8.other)
    assert gpu8.handles == [77] and gpu8.made
    assert all(t.owner is gpu8.other for t in gpu8.made)
    assert gpu8.current is gpu8.default
    for t in out if isinstance(out, tuple) else (out,):
        assert gpu8.default.cuda_stream in t.used_on
    gpu8.made.clear()
    calls8()[name]()
    assert gpu8.handles == [77, 0] and all(t.owner is gpu8.default for t in gpu8.made)


@pytest.mark.parametrize("name", sorted(calls8()))
def test_stream_of_another_device_is_refused(gpu8, name):
    import types
    with pytest.raises(ValueError):
        calls8()[name](stream=types.SimpleNamespace(cuda_stream=5, device=torch.device("cuda", 1)))
    assert not gpu8.handles
