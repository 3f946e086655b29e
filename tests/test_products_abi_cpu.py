"""Refusals of lq_gemm_ep, lq_gemm_grouped, lq_gemm_join and lq_route: bad
arguments are rejected on the host, before any HIP call (no GPU needed)."""
import ctypes

import pytest

from bit_lifted_gemv_amd import lq

P = 0x10000000          # never dereferenced
MIS = P + 2
BF16, F16, F32 = lq.LQ_BF16, lq.LQ_F16, lq.LQ_F32
NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5, 7


@pytest.fixture(scope="module")
def L():
    return lq.load_library()


def size(f, *args):
    n = ctypes.c_size_t(0)
    assert f(*args, ctypes.byref(n)) == 0
    return n.value


def ep(L, **over):
    a = dict(w=P, m=4096, K=4096, ldw=128, s=P, a=P, dt=BF16, lda=4096, B=300, bias=None, act=0,
             gated=0, res=None, ldr=0, out=P, odt=BF16, ldo=4096, ws=P, n=1 << 30)
    a.update(over)
    return L.lq_gemm_ep(a["w"], a["m"], a["K"], a["ldw"], a["s"], a["a"], a["dt"], a["lda"], a["B"],
                        a["bias"], a["act"], a["gated"], a["res"], a["ldr"], a["out"], a["odt"],
                        a["ldo"], a["ws"], a["n"], None)


@pytest.mark.parametrize("over,status", [
    (dict(w=None), NULL), (dict(s=None), NULL), (dict(a=None), NULL), (dict(out=None), NULL),
    (dict(dt=F32), DTYPE), (dict(dt=7), DTYPE), (dict(odt=9), DTYPE), (dict(act=5), UNSUPPORTED),
    (dict(act=-1), UNSUPPORTED), (dict(m=0), SHAPE), (dict(m=63, gated=1), SHAPE), (dict(K=0), SHAPE),
    (dict(K=4092), SHAPE), (dict(K=(1 << 22) + 8, lda=1 << 23, ldw=1 << 18), SHAPE), (dict(B=0), SHAPE),
    (dict(B=-1), SHAPE), (dict(B=1 << 31), SHAPE), (dict(ldw=3), SHAPE), (dict(ldw=130), ALIGN),
    (dict(m=1 << 20, ldw=1024), SHAPE), (dict(lda=120), SHAPE), (dict(lda=4100), ALIGN),
    (dict(w=P + 8), ALIGN), (dict(a=P + 8), ALIGN), (dict(s=MIS), ALIGN), (dict(bias=MIS), ALIGN),
    (dict(ldo=63), SHAPE), (dict(res=P, ldr=63), SHAPE), (dict(out=P + 1), ALIGN),
    (dict(res=P + 1, ldr=4096), ALIGN), (dict(odt=F32, out=MIS), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(n=0), WORKSPACE), (dict(ws=P + 16), ALIGN), (dict(B=1 << 22, K=1024, ldw=32, lda=1024), SHAPE),
])
def test_gemm_ep_refusals(L, over, status):
    assert ep(L, **over) == status
    assert L.lq_last_error()


def test_gemm_ep_workspace(L):
    f = L.lq_gemm_ep_workspace_size
    assert size(f, 64, 128, 3, BF16) == 0          # few rows, short: none
    need = size(f, 4096, 4096, 300, BF16)
    assert need > 0
    assert ep(L, n=need - 1) == WORKSPACE
    assert size(f, 8192, 68096, 16, BF16) > 0      # sums of the slices
    assert size(f, 4096, 4096, 300, F32) > need
    n = ctypes.c_size_t(0)
    assert f(64, 128, 3, BF16, None) == NULL
    assert f(0, 128, 3, BF16, ctypes.byref(n)) == SHAPE
    assert f(64, 12, 3, BF16, ctypes.byref(n)) == SHAPE
    assert f(64, 128, 3, 4, ctypes.byref(n)) == DTYPE


def grouped(L, **over):
    a = dict(w=P, E=4, m=64, K=128, ldw=4, s=P, a=P, dt=BF16, lda=128, ar=500, rows=P, off=P, R=1000,
             bias=None, act=0, gated=0, out=P, odt=BF16, ldo=64, ws=P, n=1 << 30)
    a.update(over)
    return L.lq_gemm_grouped(a["w"], a["E"], a["m"], a["K"], a["ldw"], a["s"], a["a"], a["dt"],
                             a["lda"], a["ar"], a["rows"], a["off"], a["R"], a["bias"], a["act"],
                             a["gated"], a["out"], a["odt"], a["ldo"], a["ws"], a["n"], None)


@pytest.mark.parametrize("over,status", [
    (dict(w=None), NULL), (dict(off=None), NULL), (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(R=-1), SHAPE), (dict(R=1 << 31), SHAPE), (dict(rows=None), SHAPE), (dict(ar=0), SHAPE),
    (dict(off=MIS), ALIGN), (dict(rows=MIS), ALIGN), (dict(m=65, gated=1), SHAPE), (dict(n=64), WORKSPACE),
    (dict(dt=F32), DTYPE), (dict(ldo=10), SHAPE), (dict(lda=8), SHAPE), (dict(R=0, w=None), 0),
])
def test_gemm_grouped_refusals(L, over, status):
    assert grouped(L, **over) == status


def join(L, **over):
    a = dict(w=P, E=4, m=64, K=128, ldw=4, s=P, a=P, dt=BF16, lda=128, off=P, R=10, bias=None, pos=P,
             wt=P, T=5, k=2, res=None, ldr=0, out=P, odt=BF16, ldo=64, ws=P, n=1 << 30)
    a.update(over)
    return L.lq_gemm_join(a["w"], a["E"], a["m"], a["K"], a["ldw"], a["s"], a["a"], a["dt"], a["lda"],
                          a["off"], a["R"], a["bias"], a["pos"], a["wt"], a["T"], a["k"], a["res"],
                          a["ldr"], a["out"], a["odt"], a["ldo"], a["ws"], a["n"], None)


@pytest.mark.parametrize("over,status", [
    (dict(pos=None), NULL), (dict(wt=None), NULL), (dict(a=None), NULL), (dict(off=None), NULL),
    (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE),
    (dict(R=-1), SHAPE), (dict(pos=MIS), ALIGN), (dict(res=P, ldr=3), SHAPE), (dict(n=100), WORKSPACE),
    (dict(T=0, w=None), 0),
])
def test_gemm_join_refusals(L, over, status):
    assert join(L, **over) == status


def test_gemm_join_workspace(L):
    f = L.lq_gemm_join_workspace_size
    need = size(f, 4, 64, 128, 10, 5, 2, BF16)
    assert join(L, n=need - 1) == WORKSPACE


def route(L, **over):
    a = dict(x=P, dt=F32, T=100, E=8, ld=8, valid=None, k=2, ren=1, ids=P, wt=P, pos=P, rows=P, off=P,
             ws=P, n=1 << 20)
    a.update(over)
    return L.lq_route(a["x"], a["dt"], a["T"], a["E"], a["ld"], a["valid"], a["k"], a["ren"], a["ids"],
                      a["wt"], a["pos"], a["rows"], a["off"], a["ws"], a["n"], None)


@pytest.mark.parametrize("over,status", [
    (dict(x=None), NULL), (dict(off=None), NULL), (dict(ids=None), NULL), (dict(rows=None), NULL),
    (dict(dt=3), DTYPE), (dict(E=0), SHAPE), (dict(E=1025, ld=1025), SHAPE), (dict(k=9), SHAPE),
    (dict(k=0), SHAPE), (dict(E=64, ld=64, k=33), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 30), SHAPE),
    (dict(ld=7), SHAPE), (dict(x=MIS), ALIGN), (dict(ids=MIS), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(n=10), WORKSPACE), (dict(ws=P + 4), ALIGN),
])
def test_route_refusals(L, over, status):
    assert route(L, **over) == status


def test_route_workspace(L):
    assert size(L.lq_route_workspace_size, 64, 1024, 8) == 0
    assert size(L.lq_route_workspace_size, 65, 8, 8) > 0
    n = ctypes.c_size_t(0)
    assert L.lq_route_workspace_size(5, 8, 9, ctypes.byref(n)) == SHAPE
    assert L.lq_route_workspace_size(5, 8, 2, None) == NULL


def test_wrappers_refuse_tensors_on_the_host():
    import torch
    w = torch.zeros(8, 4, dtype=torch.int32)
    s = torch.zeros(8)
    a = torch.zeros(2, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        lq.gemm_ep(w, s, a)
    with pytest.raises(ValueError):
        lq.route(torch.zeros(2, 4), 2)


def test_outputs_over_the_activations_are_refused(L):
    """A workgroup writes outputs while others still read activations; the residual may be the output
    itself, but then row by row."""
    Q, W = P + (1 << 28), P + (2 << 28)
    for B in (1, 300):
        assert ep(L, m=4096, a=Q, out=Q, ws=W, B=B) == UNSUPPORTED
    assert grouped(L, a=Q, out=Q, ws=W) == UNSUPPORTED
    assert ep(L, a=P, out=Q, res=Q, ldr=8192, ws=W) == UNSUPPORTED
    assert join(L, R=10, a=P, out=Q, res=Q, ldr=128, ws=W) == UNSUPPORTED
