"""ctypes binding of liblq (include/lq.h): argument marshalling only.

Every function here passes device pointers, sizes and the current HIP stream
of torch to the C ABI; all arithmetic of the layer runs in the library's HIP
kernels.  Importing this module opens ``liblq.so`` next to it and raises if
the library is missing -- there is no fallback.

Packed weights are held in torch.int32 tensors (the same 32 bits as the ABI's
uint32 words).
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple, Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblq.so")

LQ_F32, LQ_F16, LQ_BF16, LQ_E4M3, LQ_E5M2, LQ_E8M0 = 0, 1, 2, 3, 4, 5
STATUS = {0: "LQ_OK", 1: "LQ_ERR_NULL", 2: "LQ_ERR_SHAPE", 3: "LQ_ERR_DTYPE", 4: "LQ_ERR_ALIGN",
          5: "LQ_ERR_UNSUPPORTED", 6: "LQ_ERR_HIP", 7: "LQ_ERR_WORKSPACE"}

EXPORTS = ("lq_status_string", "lq_last_error", "lq_version", "lq_pack_signs", "lq_unpack_signs",
           "lq_lift_activations", "lq_lift_kron_workspace_size", "lq_lift_kron",
           "lq_gemv_workspace_size", "lq_workspace_clear", "lq_gemv", "lq_gemm",
           "lq_encode_workspace_size", "lq_encode", "lq_softmin_workspace_size",
           "lq_softmin_grad", "lq_adam_update", "lq_gemm_decoded_workspace_size",
           "lq_gemm_decoded", "lq_layer_b1_workspace_size", "lq_layer_b1",
           "lq_gemv_noalloc", "lq_stream_read", "lq_lift_parts_size", "lq_lift_parts",
           "lq_gemv_parts_workspace_size", "lq_gemv_parts",
           "lq_gemm_ep_workspace_size", "lq_gemm_ep", "lq_route_workspace_size", "lq_route",
           "lq_gemm_grouped_workspace_size", "lq_gemm_grouped", "lq_gemm_join_workspace_size",
           "lq_gemm_join", "lq_quant8", "lq_quant8_blocks", "lq_gemm8_workspace_size", "lq_gemm8",
           "lq_gemm8_grouped_workspace_size", "lq_gemm8_grouped", "lq_sort_rows", "lq_join_rows",
           "lq_join_rows_grad")

# Activations of gemm_ep and gemm_grouped.
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_vp = ctypes.c_void_p
_sz = ctypes.c_size_t


class LQError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m bit_lifted_gemv_amd.build`")
    lib = ctypes.CDLL(path)
    sig = {
        "lq_status_string": (ctypes.c_char_p, [_i32]),
        "lq_last_error": (ctypes.c_char_p, []),
        "lq_version": (ctypes.c_char_p, []),
        "lq_pack_signs": (_i32, [_vp, _i64, _i64, _i64, _vp, _i64, _vp]),
        "lq_unpack_signs": (_i32, [_vp, _i64, _i64, _i64, _vp, _i64, _vp]),
        "lq_lift_activations": (_i32, [_vp, _i32, _i64, _i64, _vp, _i32, _i32, _vp, _i32, _i32,
                                       _vp, _i32, _vp]),
        "lq_lift_kron_workspace_size": (_i32, [_i64, _i64, ctypes.POINTER(_sz)]),
        "lq_lift_kron": (_i32, [_vp, _i32, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                                _vp, _i32, _vp, _sz, _vp]),
        "lq_gemv_workspace_size": (_i32, [_i64, _i64, _i64, ctypes.POINTER(_sz)]),
        "lq_workspace_clear": (_i32, [_vp, _sz, _vp]),
        "lq_gemv": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _sz, _vp]),
        "lq_gemm": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _vp]),
        "lq_gemv_noalloc": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp]),
        "lq_stream_read": (_i32, [_vp, _sz, _vp, _vp]),
        "lq_lift_parts_size": (_i32, [_i64, ctypes.POINTER(_sz)]),
        "lq_lift_parts": (_i32, [_vp, _i32, _i64, _i64, _vp, _i32, _i32, _vp, _i32, _i32, _vp,
                                 _sz, _vp]),
        "lq_gemv_parts_workspace_size": (_i32, [_i64, _i64, _i64, ctypes.POINTER(_sz)]),
        "lq_gemv_parts": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _sz, _i64, _vp, _vp, _sz, _vp]),
        "lq_encode_workspace_size": (_i32, [_i32, _i32, ctypes.POINTER(_sz)]),
        "lq_encode": (_i32, [_vp, _i64, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _sz, _vp]),
        "lq_softmin_workspace_size": (_i32, [_i64, _i32, _i32, ctypes.POINTER(_sz)]),
        "lq_gemm_decoded_workspace_size": (_i32, [_i64, _i64, ctypes.POINTER(_sz)]),
        "lq_layer_b1_workspace_size": (_i32, [_i64, _i64, _i32, _i32, ctypes.POINTER(_sz)]),
        "lq_layer_b1": (_i32, [_vp, _i32, _i64, _vp, _i32, _i32, _vp, _i32, _i32, _vp, _i64, _i64,
                               _vp, _vp, _vp, _sz, _vp]),
        "lq_gemm_decoded": (_i32, [_vp, _i64, _i64, _i64, _vp, _i32, _i32, _vp, _vp, _i32, _i64,
                                   _vp, _vp, _sz, _vp]),
        "lq_softmin_grad": (_i32, [_vp, _i64, _vp, _i32, _i32, ctypes.c_float, _vp, _vp, _vp,
                                   _sz, _vp]),
        "lq_gemm_ep_workspace_size": (_i32, [_i64, _i64, _i64, _i32, ctypes.POINTER(_sz)]),
        "lq_gemm_ep": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _i64, _vp, _i32, _i32,
                              _vp, _i64, _vp, _i32, _i64, _vp, _sz, _vp]),
        "lq_route_workspace_size": (_i32, [_i64, _i64, _i32, ctypes.POINTER(_sz)]),
        "lq_route": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                            _vp, _sz, _vp]),
        "lq_gemm_grouped_workspace_size": (_i32, [_i64, _i64, _i64, _i64, _i64, _i32,
                                                  ctypes.POINTER(_sz)]),
        "lq_gemm_grouped": (_i32, [_vp, _i64, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _i64, _vp,
                                   _vp, _i64, _vp, _i32, _i32, _vp, _i32, _i64, _vp, _sz, _vp]),
        "lq_gemm_join_workspace_size": (_i32, [_i64, _i64, _i64, _i64, _i64, _i32, _i32,
                                               ctypes.POINTER(_sz)]),
        "lq_gemm_join": (_i32, [_vp, _i64, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _i64, _vp,
                                _vp, _vp, _i64, _i32, _vp, _i64, _vp, _i32, _i64, _vp, _sz, _vp]),
        "lq_quant8": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i32, _i64, _vp, _i64, _vp]),
        "lq_quant8_blocks": (_i32, [_vp, _i32, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp]),
        "lq_gemm8_workspace_size": (_i32, [_i64, _i64, _i32, _i64, ctypes.POINTER(_sz)]),
        "lq_gemm8": (_i32, [_vp, _i64, _i64, _i64, _vp, _i32, _i64, _vp, _i32, _i64, _vp, _i64, _i64,
                            _vp, _i32, _i32, _vp, _i64, _vp, _i32, _i64, _vp, _sz, _vp]),
        "lq_gemm8_grouped_workspace_size": (_i32, [_i64, _i64, _i64, _i32, _i64, _i64,
                                                   ctypes.POINTER(_sz)]),
        "lq_gemm8_grouped": (_i32, [_vp, _i64, _i64, _i64, _i64, _vp, _i32, _i64, _vp, _i32, _i64,
                                    _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i32, _i32, _vp, _i32,
                                    _i64, _vp, _sz, _vp]),
        "lq_sort_rows": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp]),
        "lq_join_rows": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _i64, _i32, _vp, _i64, _vp,
                                _i32, _i64, _vp]),
        "lq_join_rows_grad": (_i32, [_vp, _i32, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _i32,
                                     _vp, _vp, _i64, _vp, _vp]),
        "lq_adam_update": (_i32, [_vp, _vp, _vp, _vp, _i64, _i32, ctypes.c_float,
                                  ctypes.c_float, ctypes.c_float, ctypes.c_float, _vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_LIB: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        _LIB = load_library()
    return _LIB


def check(status: int) -> None:
    if status != 0:
        raise LQError(status, lib().lq_last_error().decode())


# ----------------------------------------------------------------- helpers
def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LQ_F32
    if t.dtype == torch.float16:
        return LQ_F16
    if t.dtype == torch.bfloat16:
        return LQ_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _torch_dt(code: int) -> torch.dtype:
    return {LQ_F32: torch.float32, LQ_F16: torch.float16, LQ_BF16: torch.bfloat16}[code]


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dev(*ts: torch.Tensor) -> None:
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must live on the GPU")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _tensors(x) -> list:
    """The tensors among arguments or results, also in lists and tuples."""
    if isinstance(x, (tuple, list)):
        return [t for v in x for t in _tensors(v)]
    return [x] if hasattr(x, "record_stream") else []


def _on_stream(call):
    """A wrapper around the calls whose last parameter is `stream`.  A stream
    other than the current one becomes the current one for the call, so that
    its workspace and the tensors it makes are that stream's memory, in order
    with its kernels: a block that the caller's stream has given back may still
    be in use there.  What is passed in is kept until `stream` is through with
    it, and what is returned until the caller's stream is; that the one stream
    waits for the other's results is the caller's business."""
    last = call.__code__.co_argcount - 1

    @functools.wraps(call)
    def run(*args, **kwargs):
        stream = args[last] if len(args) > last else kwargs.get("stream")
        if stream is None:
            return call(*args, **kwargs)
        caller = torch.cuda.current_stream(stream.device)
        if caller == stream:
            return call(*args, **kwargs)
        with torch.cuda.stream(stream):
            result = call(*args, **kwargs)
        given = _tensors((args, list(kwargs.values())))
        for t in given:
            t.record_stream(stream)
        for t in _tensors(result):
            if not any(t is g for g in given):
                t.record_stream(caller)
        return result
    return run


# ----------------------------------------------------------------- C ABI wrappers
@_on_stream
def pack_signs(signs: torch.Tensor, ldw: Optional[int] = None, stream=None) -> torch.Tensor:
    """int8 signs [rows][K] -> int32 words [rows][ldw] (LSB-first, bit 1 = positive)."""
    _dev(signs)
    rows, K = signs.shape
    ldw = (K + 31) // 32 if ldw is None else ldw
    out = torch.empty((rows, ldw), dtype=torch.int32, device=signs.device)
    check(lib().lq_pack_signs(_ptr(signs), rows, K, K, _ptr(out), ldw, _stream(stream)))
    return out


@_on_stream
def unpack_signs(packed: torch.Tensor, K: int, stream=None) -> torch.Tensor:
    _dev(packed)
    rows, ldw = packed.shape
    out = torch.empty((rows, K), dtype=torch.int8, device=packed.device)
    check(lib().lq_unpack_signs(_ptr(packed), rows, K, ldw, _ptr(out), K, _stream(stream)))
    return out


@_on_stream
def lift(a: torch.Tensor, t_inv: torch.Tensor, M: torch.Tensor, d: int, D: int,
         out_dtype: torch.dtype = torch.float32, t_block: int = 128,
         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """a [B][n], t_inv [n/128][128][128], M float [d][D] -> a_lift [B][n*D/d]."""
    _dev(a, t_inv, M)
    B, n = a.shape
    K = n // d * D
    if out is None:
        out = torch.empty((B, K), dtype=out_dtype, device=a.device)
    check(lib().lq_lift_activations(_ptr(a), _dt(a), B, n, _ptr(t_inv), _dt(t_inv), t_block,
                                    _ptr(M), d, D, _ptr(out), _dt(out), _stream(stream)))
    return out


def lift_parts_size(K: int) -> int:
    n = _sz(0)
    check(lib().lq_lift_parts_size(K, ctypes.byref(n)))
    return n.value


@_on_stream
def lift_parts(a: torch.Tensor, t_inv: torch.Tensor, M: torch.Tensor, d: int, D: int,
               t_block: int = 128, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """a [B][n] and t_inv of one 16-bit type, M float [d][D] -> the operand
    image of lq_gemv_parts (uint8, lq_lift_parts_size(n*D/d) bytes)."""
    _dev(a, t_inv, M)
    B, n = a.shape
    nb = lift_parts_size(n // d * D)
    if out is None:
        out = torch.empty(nb, dtype=torch.uint8, device=a.device)
    check(lib().lq_lift_parts(_ptr(a), _dt(a), B, n, _ptr(t_inv), _dt(t_inv), t_block, _ptr(M),
                              d, D, _ptr(out), out.numel() * out.element_size(),
                              _stream(stream)))
    return out


@_on_stream
def lift_kron(a: torch.Tensor, s1: torch.Tensor, p1_inv: torch.Tensor, p2_inv: torch.Tensor,
              s2: torch.Tensor, M: torch.Tensor, d: int, D: int,
              out_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """a [B][n], Kronecker whitening factors (float32: s1 [n], P1^-1 [n1][n1],
    P2^-1 [n2][n2], s2 [n/d]), M float [d][D] -> a_lift [B][n*D/d]."""
    _dev(a, s1, p1_inv, p2_inv, s2, M)
    B, n = a.shape
    n1 = p1_inv.shape[0]
    K = n // d * D
    if out is None:
        out = torch.empty((B, K), dtype=out_dtype, device=a.device)
    nb = _sz(0)
    check(lib().lq_lift_kron_workspace_size(B, n, ctypes.byref(nb)))
    ws = workspace(nb.value, a.device, -1, stream)
    check(lib().lq_lift_kron(_ptr(a), _dt(a), B, n, n1, _ptr(s1), _ptr(p1_inv), _ptr(p2_inv),
                             _ptr(s2), _ptr(M), d, D, _ptr(out), _dt(out), _ptr(ws), nb.value,
                             _stream(stream)))
    return out


@_on_stream
def encode(w: torch.Tensor, M: torch.Tensor, A: Optional[torch.Tensor] = None,
           codes: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
           stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Lattice codes of float32 weight groups w [G][d] under M [d][D]:
    exhaustive when A is None, else the auxiliary-vector search with the
    completion A [D-d][D].  Returns (codes int8 [G][D], err float32 [G])."""
    _dev(w, M)
    G, d = w.shape
    D = M.shape[1]
    if codes is None:
        codes = torch.empty((G, D), dtype=torch.int8, device=w.device)
    if err is None:
        err = torch.empty((G,), dtype=torch.float32, device=w.device)
    ws, nbytes = None, 0
    if A is not None:
        _dev(A)
        if A.numel() == 0:    # D == d: A has no rows; any non-null pointer selects the search
            A = torch.zeros(1, dtype=torch.float32, device=w.device)
        nb = _sz(0)
        check(lib().lq_encode_workspace_size(d, D, ctypes.byref(nb)))
        nbytes = nb.value
        ws = workspace(nbytes, w.device, -2, stream)
    check(lib().lq_encode(_ptr(w), G, _ptr(M), _ptr(A), d, D, _ptr(codes), _ptr(err), _ptr(ws),
                          nbytes, _stream(stream)))
    return codes, err


@_on_stream
def layer_b1(a: torch.Tensor, t_inv: torch.Tensor, M: torch.Tensor, d: int, D: int,
             w_packed: torch.Tensor, s: torch.Tensor, out: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """The whole layer for one token (a [n] or [1][n]): lift inside the
    one-token product; out float32 [1][m]."""
    _dev(a, t_inv, M, w_packed, s)
    n = a.shape[-1]
    m, ldw = w_packed.shape
    if out is None:
        out = torch.empty((1, m), dtype=torch.float32, device=a.device)
    nb = _sz(0)
    check(lib().lq_layer_b1_workspace_size(m, n, d, D, ctypes.byref(nb)))
    ws = workspace(nb.value, a.device, m, stream) if nb.value else None
    check(lib().lq_layer_b1(_ptr(a), _dt(a), n, _ptr(t_inv), _dt(t_inv), 128, _ptr(M), d, D,
                            _ptr(w_packed), m, ldw, _ptr(s), _ptr(out), _ptr(ws), nb.value,
                            _stream(stream)))
    return out


@_on_stream
def gemm_decoded(w_packed: torch.Tensor, s: torch.Tensor, M: torch.Tensor, d: int, D: int,
                 u: torch.Tensor, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """out [B][m] = s * (W_hat @ u^T) with W_hat decoded from the signs and M
    (float16 u [B][n], the whitened activations)."""
    _dev(w_packed, s, M, u)
    m, ldw = w_packed.shape
    B, n = u.shape
    if out is None:
        out = torch.empty((B, m), dtype=torch.float32, device=u.device)
    nb = _sz(0)
    check(lib().lq_gemm_decoded_workspace_size(m, n, ctypes.byref(nb)))
    ws = workspace(nb.value, u.device, -4, stream) if nb.value else None
    check(lib().lq_gemm_decoded(_ptr(w_packed), m, n, ldw, _ptr(M), d, D, _ptr(s), _ptr(u),
                                _dt(u), B, _ptr(out), _ptr(ws) if ws is not None else None,
                                nb.value, _stream(stream)))
    return out


@_on_stream
def softmin_grad(w: torch.Tensor, M: torch.Tensor, T: float = 10.0,
                 loss: Optional[torch.Tensor] = None, grad: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Soft-argmin objective of samples w [N][d] under M [d][D] and its
    gradient: (loss float32 [1], grad float32 [d][D]), both on the device."""
    _dev(w, M)
    N, d = w.shape
    D = M.shape[1]
    if loss is None:
        loss = torch.empty((1,), dtype=torch.float32, device=w.device)
    if grad is None:
        grad = torch.empty((d, D), dtype=torch.float32, device=w.device)
    nb = _sz(0)
    check(lib().lq_softmin_workspace_size(N, d, D, ctypes.byref(nb)))
    ws = workspace(nb.value, w.device, -3, stream)
    check(lib().lq_softmin_grad(_ptr(w), N, _ptr(M), d, D, float(T), _ptr(loss), _ptr(grad),
                                _ptr(ws), nb.value, _stream(stream)))
    return loss, grad


@_on_stream
def adam_update(M: torch.Tensor, grad: torch.Tensor, m1: torch.Tensor, m2: torch.Tensor,
                step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                eps: float = 1e-8, stream=None) -> None:
    """One Adam step on M in place (m1, m2: moment buffers, zero at step 1)."""
    _dev(M, grad, m1, m2)
    check(lib().lq_adam_update(_ptr(M), _ptr(grad), _ptr(m1), _ptr(m2), M.numel(), step,
                               float(lr), float(beta1), float(beta2), float(eps),
                               _stream(stream)))


@_on_stream
def learn_m(M0: torch.Tensor, batches, T: float = 10.0, lr: float = 0.01,
            stream=None) -> Tuple[torch.Tensor, list]:
    """Adam on the soft-argmin objective from M0, one step per batch of
    samples (float32 [N][d] device tensors drawn by the caller).  Returns
    (M, the per-step loss tensors)."""
    M = M0.detach().clone().contiguous()
    m1 = torch.zeros_like(M)
    m2 = torch.zeros_like(M)
    grad = torch.empty_like(M)
    losses = []
    for i, w in enumerate(batches, start=1):
        loss, _ = softmin_grad(w, M, T, grad=grad, stream=stream)
        adam_update(M, grad, m1, m2, i, lr, stream=stream)
        losses.append(loss)
    return M, losses


_WS = {}


def workspace(nbytes: int, device: torch.device, tag: int = 0, stream=None) -> torch.Tensor:
    """A workspace of at least nbytes, cached per (device, stream, tag) and
    grown on demand, zero-filled when allocated.  Calls on one stream run in
    order, so they may share it; calls on different streams get their own.
    The GEMV uses its row count as tag, the Kronecker lift -1, the encoder -2,
    the soft-argmin objective -3, the decode-weights product -4, the GEMV on
    the parts image -5.  The zeros are written on the current stream, which is
    the call's (_on_stream)."""
    key = (device.type, device.index, _stream(stream), tag)
    ws = _WS.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        _WS[key] = ws
    return ws


def gemv_workspace_size(m: int, K: int, B: int) -> int:
    n = _sz(0)
    check(lib().lq_gemv_workspace_size(m, K, B, ctypes.byref(n)))
    return n.value


@_on_stream
def gemv(w_packed: torch.Tensor, s: torch.Tensor, a_lift: torch.Tensor, K: Optional[int] = None,
         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out [B][m] = s * (sigma @ a_lift^T), float32 lifted activations, 1 <= B <= 16."""
    _dev(w_packed, s, a_lift)
    m, ldw = w_packed.shape
    B, Ka = a_lift.shape
    K = Ka if K is None else K
    if K != Ka:
        raise ValueError(f"K={K} differs from the lifted activations' row length {Ka}")
    if out is None:
        out = torch.empty((B, m), dtype=torch.float32, device=a_lift.device)
    nws = gemv_workspace_size(m, K, B)
    ws = workspace(nws, a_lift.device, m, stream) if nws else None
    check(lib().lq_gemv(_ptr(w_packed), m, K, ldw, _ptr(s), _ptr(a_lift), B, _ptr(out), _ptr(ws),
                        nws, _stream(stream)))
    return out


@_on_stream
def gemv_parts(w_packed: torch.Tensor, s: torch.Tensor, parts: torch.Tensor, K: int, B: int,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out [B][m] = s * (sigma @ a_hat^T) from the image of lift_parts."""
    _dev(w_packed, s, parts)
    m, ldw = w_packed.shape
    if out is None:
        out = torch.empty((B, m), dtype=torch.float32, device=parts.device)
    n = _sz(0)
    check(lib().lq_gemv_parts_workspace_size(m, K, B, ctypes.byref(n)))
    ws = workspace(n.value, parts.device, -5, stream)
    check(lib().lq_gemv_parts(_ptr(w_packed), m, K, ldw, _ptr(s), _ptr(parts),
                              parts.numel() * parts.element_size(), B, _ptr(out), _ptr(ws),
                              n.value, _stream(stream)))
    return out


@_on_stream
def gemv_noalloc(w_packed: torch.Tensor, s: torch.Tensor, a_lift: torch.Tensor,
                 out: torch.Tensor, stream=None) -> torch.Tensor:
    """lq_gemv without a workspace (the library's per-GPU scratch; calls on
    one GPU must not overlap); out [B][m] float32 must be given."""
    _dev(w_packed, s, a_lift, out)
    m, ldw = w_packed.shape
    B, K = a_lift.shape
    check(lib().lq_gemv_noalloc(_ptr(w_packed), m, K, ldw, _ptr(s), _ptr(a_lift), B, _ptr(out),
                                _stream(stream)))
    return out


@_on_stream
def stream_read(buf: torch.Tensor, sink: torch.Tensor, stream=None) -> None:
    """Read every byte of buf once (the HBM read-rate reference); sink: a
    device int32 tensor of at least 4 x compute units."""
    _dev(buf, sink)
    check(lib().lq_stream_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                               _stream(stream)))


@_on_stream
def gemm(w_packed: torch.Tensor, s: torch.Tensor, a_lift: torch.Tensor, K: Optional[int] = None,
         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out [B][m] on the matrix cores; a_lift float16 or bfloat16 [B][K]."""
    _dev(w_packed, s, a_lift)
    m, ldw = w_packed.shape
    B, Ka = a_lift.shape
    K = Ka if K is None else K
    if K != Ka:
        raise ValueError(f"K={K} differs from the lifted activations' row length {Ka}")
    if out is None:
        out = torch.empty((B, m), dtype=torch.float32, device=a_lift.device)
    check(lib().lq_gemm(_ptr(w_packed), m, K, ldw, _ptr(s), _ptr(a_lift), _dt(a_lift), B,
                        _ptr(out), _stream(stream)))
    return out


# ------------------------------------- products with an epilogue, experts, router
def _elsewhere(device: torch.device) -> bool:
    """Whether the tensors' device is not the current one (the calls below then
    run under it)."""
    return device.index != torch.cuda.current_device()


def _handle(device: torch.device, stream) -> int:
    """The HIP stream of a call: `stream`, or the device's current one (its raw
    handle: torch.cuda.current_stream builds a Stream object, 2 us)."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


@functools.lru_cache(maxsize=4096)
def _bytes_needed(call: str, *sizes: int) -> int:
    n = _sz(0)
    check(getattr(lib(), call)(*sizes, ctypes.byref(n)))
    return n.value


def _temporary(nbytes: int, device: torch.device) -> Optional[torch.Tensor]:
    """A workspace from torch's allocator on the current stream, which is the
    call's (_on_stream), a new one for every call, so that calls on two streams
    or captured graphs never share one; returned memory is reused in stream
    order."""
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _same_device(device: torch.device, **tensors: Optional[torch.Tensor]) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


def _plain(name: str, t: Optional[torch.Tensor], dtype: torch.dtype, shape: tuple) -> None:
    """A contiguous tensor of this type and shape (or None)."""
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _pitch(name: str, t: torch.Tensor, shape: tuple, dtype: Optional[torch.dtype] = None) -> int:
    """Row pitch of a matrix whose rows are dense and may lie apart."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}'s rows must be dense")
    # the stride of a single row says nothing
    return t.stride(0) if shape[0] > 1 else shape[1] + -shape[1] % 8


def _experts(w_packed: torch.Tensor, s: torch.Tensor, bias: Optional[torch.Tensor],
             lead: tuple) -> None:
    if not w_packed.is_cuda:
        raise ValueError("tensors must live on the GPU")
    _plain("w_packed", w_packed, torch.int32, lead + (w_packed.shape[-1],))
    _plain("s", s, torch.float32, lead)
    _plain("bias", bias, torch.float32, lead)


def _lifted(a_lift: torch.Tensor) -> int:
    if a_lift.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"a_lift must be float16 or bfloat16, not {a_lift.dtype}")
    return _pitch("a_lift", a_lift, tuple(a_lift.shape))


def _target(out: Optional[torch.Tensor], rows: int, width: int, out_dtype: Optional[torch.dtype],
            a_lift: torch.Tensor) -> Tuple[torch.Tensor, int]:
    if out is None:
        dt = a_lift.dtype if out_dtype is None else out_dtype
        out = torch.empty((rows, width), dtype=dt, device=a_lift.device)
        return out, width
    if out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, not {out_dtype}")
    return out, _pitch("out", out, (rows, width))


def _act(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r} (one of {', '.join(ACTS)})")
    return ACTS[act]


@_on_stream
def gemm_ep(w_packed: torch.Tensor, s: torch.Tensor, a_lift: torch.Tensor,
            bias: Optional[torch.Tensor] = None, act: str = "none", gated: bool = False,
            residual: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """act(s * (sigma @ a_lift^T) + bias) + residual for any number of tokens
    (lq_gemm_ep).  a_lift float16 or bfloat16 [B][K] (rows may lie apart);
    `act` one of ACTS; `gated`: rows of w_packed are the gate's m/2, then the up
    projection's, and out [B][m/2] = act(gate) * up + residual.  out_dtype
    (default a_lift's): float32, float16 or bfloat16, also the residual's;
    `residual` may be `out`."""
    m, ldw = w_packed.shape
    B, K = a_lift.shape
    dev = a_lift.device
    _experts(w_packed, s, bias, (m,))
    _same_device(dev, w_packed=w_packed, s=s, bias=bias, residual=residual, out=out)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return gemm_ep(w_packed, s, a_lift, bias, act, gated, residual, out_dtype, out, stream)
    lda = _lifted(a_lift)
    width = m // 2 if gated else m
    code = _act(act)
    out, ldo = _target(out, B, width, out_dtype, a_lift)
    odt = _dt(out)
    ldr = 0 if residual is None else _pitch("residual", residual, (B, width), out.dtype)
    nb = _bytes_needed("lq_gemm_ep_workspace_size", m, K, B, odt)
    ws = _temporary(nb, dev)
    check(lib().lq_gemm_ep(_ptr(w_packed), m, K, ldw, _ptr(s), _ptr(a_lift), _dt(a_lift), lda, B,
                           _ptr(bias), code, int(gated), _ptr(residual), ldr, _ptr(out), odt, ldo,
                           _ptr(ws), nb, _handle(dev, stream)))
    return out


@_on_stream
def gemm_grouped(w_packed: torch.Tensor, s: torch.Tensor, a_lift: torch.Tensor,
                 offsets: torch.Tensor, rows: Optional[torch.Tensor] = None,
                 bias: Optional[torch.Tensor] = None, act: str = "none", gated: bool = False,
                 out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """The experts' products on ragged runs of rows (lq_gemm_grouped):
    w_packed [E][m][ldw], s and bias [E][m], offsets int32 [E + 1], rows int32
    [R] (which row of a_lift each sorted row is; None: its own).  Returns out
    [R][m], or [R][m/2] when gated; rows outside every run are not written."""
    E, m, ldw = w_packed.shape
    n_rows, K = a_lift.shape
    dev = a_lift.device
    R = n_rows if rows is None else rows.shape[0]
    _experts(w_packed, s, bias, (E, m))
    _plain("offsets", offsets, torch.int32, (E + 1,))
    _plain("rows", rows, torch.int32, (R,))
    _same_device(dev, w_packed=w_packed, s=s, bias=bias, offsets=offsets, rows=rows, out=out)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return gemm_grouped(w_packed, s, a_lift, offsets, rows, bias, act, gated, out_dtype,
                                out, stream)
    lda = _lifted(a_lift)
    code = _act(act)
    out, ldo = _target(out, R, m // 2 if gated else m, out_dtype, a_lift)
    odt = _dt(out)
    nb = _bytes_needed("lq_gemm_grouped_workspace_size", E, m, K, n_rows, R, odt)
    ws = _temporary(nb, dev)
    check(lib().lq_gemm_grouped(_ptr(w_packed), E, m, K, ldw, _ptr(s), _ptr(a_lift), _dt(a_lift),
                                lda, n_rows, _ptr(rows), _ptr(offsets), R, _ptr(bias), code,
                                int(gated), _ptr(out), odt, ldo, _ptr(ws), nb,
                                _handle(dev, stream)))
    return out


@_on_stream
def gemm_join(w_packed: torch.Tensor, s: torch.Tensor, a_lift: torch.Tensor,
              offsets: torch.Tensor, pos: torch.Tensor, weight: torch.Tensor,
              bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
              out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """The experts' products on the sorted rows a_lift [R][K] and their weighted
    sum per token (lq_gemm_join): out [T][m] = residual + sum_j weight[t][j]
    z[pos[t][j]], pos int32 and weight float32 [T][k].  `residual` may be `out`."""
    E, m, ldw = w_packed.shape
    R, K = a_lift.shape
    T, k = pos.shape
    dev = a_lift.device
    _experts(w_packed, s, bias, (E, m))
    _plain("offsets", offsets, torch.int32, (E + 1,))
    _plain("pos", pos, torch.int32, (T, k))
    _plain("weight", weight, torch.float32, (T, k))
    _same_device(dev, w_packed=w_packed, s=s, bias=bias, offsets=offsets, pos=pos, weight=weight,
                 residual=residual, out=out)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return gemm_join(w_packed, s, a_lift, offsets, pos, weight, bias, residual, out_dtype,
                             out, stream)
    lda = _lifted(a_lift)
    out, ldo = _target(out, T, m, out_dtype, a_lift)
    odt = _dt(out)
    ldr = 0 if residual is None else _pitch("residual", residual, (T, m), out.dtype)
    nb = _bytes_needed("lq_gemm_join_workspace_size", E, m, K, R, T, k, odt)
    ws = _temporary(nb, dev)
    check(lib().lq_gemm_join(_ptr(w_packed), E, m, K, ldw, _ptr(s), _ptr(a_lift), _dt(a_lift),
                             lda, _ptr(offsets), R, _ptr(bias), _ptr(pos), _ptr(weight), T, k,
                             _ptr(residual), ldr, _ptr(out), odt, ldo, _ptr(ws), nb,
                             _handle(dev, stream)))
    return out


class Routing(NamedTuple):
    """What lq_route gives: ids int32 and weight float32 [T][k] (largest logit
    first; -1 and 0 where a token has no further expert), pos int32 [T][k]
    (sorted position of each pair, or -1), rows int32 [T * k] (token of each
    sorted position, -1 behind the last), offsets int32 [E + 1]."""
    ids: torch.Tensor
    weight: torch.Tensor
    pos: torch.Tensor
    rows: torch.Tensor
    offsets: torch.Tensor


@_on_stream
def route(logits: torch.Tensor, k: int, valid: Optional[torch.Tensor] = None, renorm: bool = True,
          stream=None) -> Routing:
    """Each token's k experts, their weights and the pairs sorted by expert
    (lq_route).  logits [T][E] float32, float16 or bfloat16 (rows may lie
    apart); valid: uint8 or bool [T], 0 for tokens that go to no expert."""
    T, E = logits.shape
    dev = logits.device
    if not logits.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if valid is not None and valid.dtype == torch.bool:
        valid = valid.view(torch.uint8)
    _plain("valid", valid, torch.uint8, (T,))
    _same_device(dev, valid=valid)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return route(logits, k, valid, renorm, stream)
    ld = _pitch("logits", logits, (T, E))
    code = _dt(logits)
    nb = _bytes_needed("lq_route_workspace_size", T, E, k)
    ws = _temporary(nb, dev)
    ids, pos, rows = torch.empty((3, T, k), dtype=torch.int32, device=dev).unbind()
    rows = rows.view(-1)
    weight = torch.empty((T, k), dtype=torch.float32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    check(lib().lq_route(_ptr(logits), code, T, E, ld, _ptr(valid), k, int(renorm), _ptr(ids),
                         _ptr(weight), _ptr(pos), _ptr(rows), _ptr(offsets), _ptr(ws), nb,
                         _handle(dev, stream)))
    return Routing(ids, weight, pos, rows, offsets)


# ------------------------------------- 8-bit floating point layers
#: The 8-bit types of quantize8 and the products.
TYPES8 = {torch.float8_e4m3fn: LQ_E4M3, torch.float8_e5m2: LQ_E5M2}


class Rows8(NamedTuple):
    """Activations in 8 bits (lq_quant8): values float8_e4m3fn or float8_e5m2
    [B][K in whole 128] and exps uint8 [B][K / 128], a power of two 2^(exps - 127)
    for each 128 positions.  Rows of exps lie whole words apart."""
    values: torch.Tensor
    exps: torch.Tensor


class Blocks8(NamedTuple):
    """Weights in 8 bits: values float8_e4m3fn [m][K in whole 128] (zeros from K
    on), or [E][m][..] for E matrices, and a scale for each 128 x 128 block
    [ceil(m / 128)][K / 128] (or [E][..][..]): float32, or uint8 exponents
    (2^(scales - 127)) whose rows lie whole words apart."""
    values: torch.Tensor
    scales: torch.Tensor

    def transposed(self) -> "Blocks8":
        """The weights of the gradient: m and K exchanged (laid out anew)."""
        values = self.values.view(torch.uint8).transpose(-1, -2)
        m = self.values.shape[-2]
        values = torch.nn.functional.pad(values, (0, -m % 128)).contiguous().view(torch.float8_e4m3fn)
        scales = self.scales.transpose(-1, -2)
        if scales.dtype != torch.uint8:
            return Blocks8(values, scales.contiguous())
        held = _exponents(scales.shape, scales.device)
        held.copy_(scales)
        return Blocks8(values, held)


def _exponents(shape, device) -> torch.Tensor:
    """Room for exponents whose rows are whole words: a view of it."""
    blocks = shape[-1]
    held = torch.empty((*shape[:-1], blocks + -blocks % 4), dtype=torch.uint8, device=device)
    return held[..., :blocks] if blocks % 4 else held


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _on_gpu(*ts: torch.Tensor) -> None:
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must live on the GPU")


@_on_stream
def quantize8(x: torch.Tensor, dtype: torch.dtype = torch.float8_e4m3fn, stream=None) -> Rows8:
    """Rows x [B][K] (float32, float16 or bfloat16; rows may lie apart) in 8
    bits with a power of two for each 128 positions (lq_quant8)."""
    B, K = x.shape
    dev = x.device
    _on_gpu(x)
    if dtype not in TYPES8:
        raise TypeError(f"unsupported 8-bit type {dtype}")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return quantize8(x, dtype, stream)
    ld = _pitch("x", x, (B, K))
    values = torch.empty((B, _blocks(K) * 128), dtype=dtype, device=dev)
    exps = _exponents((B, _blocks(K)), dev)
    check(lib().lq_quant8(_ptr(x), _dt(x), B, K, ld, _ptr(values), TYPES8[dtype], values.shape[1],
                          _ptr(exps), _blocks(K) + -_blocks(K) % 4, _handle(dev, stream)))
    return Rows8(values, exps)


@_on_stream
def quantize8_blocks(w: torch.Tensor, stream=None) -> Blocks8:
    """Weights w [m][K] or [E][m][K] (float32, float16 or bfloat16, contiguous) in
    8 bits with a power of two for each 128 x 128 block (lq_quant8_blocks)."""
    *lead, m, K = w.shape
    dev = w.device
    _on_gpu(w)
    if len(lead) > 1:
        raise ValueError(f"w has shape {tuple(w.shape)}, not [m][K] or [E][m][K]")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return quantize8_blocks(w, stream)
    E = lead[0] if lead else 1
    values = torch.empty((*lead, m, _blocks(K) * 128), dtype=torch.float8_e4m3fn, device=dev)
    scales = _exponents((*lead, _blocks(m), _blocks(K)), dev)
    check(lib().lq_quant8_blocks(_ptr(w), _dt(w), E, m, K, K, _ptr(values), values.shape[-1],
                                 _ptr(scales), _blocks(K) + -_blocks(K) % 4, _handle(dev, stream)))
    return Blocks8(values, scales)


def _exponent_pitch(name: str, t: torch.Tensor, dtype: torch.dtype) -> int:
    """Row pitch of scales [..][rows][blocks]; rows of uint8 exponents are whole words
    (also the last one: the kernels read words)."""
    shape, stride = t.shape, t.stride()
    rows, blocks = shape[-2:]
    held = blocks + -blocks % 4
    if blocks > 1 and stride[-1] != 1:
        raise ValueError(f"{name}'s rows must be dense")
    # a stride along a single element says nothing
    pitch = stride[-2] if rows > 1 else held
    if len(shape) > 2 and shape[0] > 1:
        if rows == 1:
            pitch = stride[0]
        elif stride[0] != rows * pitch:
            raise ValueError(f"{name}'s matrices must follow one another")
    if dtype is torch.uint8 and t.numel():
        if pitch % 4 or (held != blocks and t.storage_offset() + (t.numel() // blocks - 1) * pitch + held
                         > t.untyped_storage().nbytes()):
            raise ValueError(f"{name}'s rows must be whole words (as quantize8 makes them)")
    return pitch


def _weights8(w: Blocks8, lead: tuple) -> Tuple[int, int]:
    """Checks weights of [lead] matrices; their scales' type and row pitch."""
    values, scales = w
    m, K = values.shape[-2:]
    _plain("w.values", values, torch.float8_e4m3fn, lead + (m, K))
    if K % 128:
        raise ValueError(f"w.values has {K} columns, not whole 128 (zeros behind the last)")
    shape, dtype = lead + (-(-m // 128), K // 128), scales.dtype
    if dtype is not torch.uint8 and dtype is not torch.float32:
        raise TypeError(f"w.scales must be uint8 exponents or float32, not {dtype}")
    if scales.shape != shape:
        raise ValueError(f"w.scales has shape {tuple(scales.shape)}, not {shape}")
    return LQ_E8M0 if dtype is torch.uint8 else LQ_F32, _exponent_pitch("w.scales", scales, dtype)


def _rows8(a, width: int):
    """(tensor, type code, pitch, exponents, their pitch) of 8- or 16-bit activations for
    weights of `width` columns; and K."""
    if isinstance(a, Rows8):
        values, exps = a
        if values.dtype not in TYPES8:
            raise TypeError(f"a.values must be float8_e4m3fn or float8_e5m2, not {values.dtype}")
        B = values.shape[0]
        lda = _pitch("a.values", values, (B, width))
        _pitch("a.exps", exps, (B, width // 128), torch.uint8)
        return (values, TYPES8[values.dtype], lda, exps, _exponent_pitch("a.exps", exps, torch.uint8),
                width)
    if a.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"a must be Rows8, float16 or bfloat16, not {a.dtype}")
    B, K = a.shape
    if _blocks(K) * 128 != width:
        raise ValueError(f"a has {K} columns, the weights {width}")
    return a, _dt(a), _pitch("a", a, (B, K)), None, 0, K


def _target8(out: Optional[torch.Tensor], rows: int, width: int, out_dtype: Optional[torch.dtype],
             a: torch.Tensor) -> Tuple[torch.Tensor, int]:
    if out is None and out_dtype is None and a.dtype in TYPES8:
        out_dtype = torch.bfloat16
    return _target(out, rows, width, out_dtype, a)


@_on_stream
def gemm8(w: Blocks8, a, bias: Optional[torch.Tensor] = None, act: str = "none",
          gated: bool = False, residual: Optional[torch.Tensor] = None,
          out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
          stream=None) -> torch.Tensor:
    """act(a @ w^T + bias) + residual for any number of tokens (lq_gemm8).  w:
    8-bit weights [m][K]; a: Rows8, or float16 or bfloat16 [B][K], which the
    call quantizes (to the same result).  Epilogue as gemm_ep; out_dtype: a's,
    bfloat16 for Rows8; float32 keeps 24 bits of every sum, at half the speed or
    less (lq_gemm8).  The gradient of the activations is
    gemm8(w.transposed(), quantize8(dz, torch.float8_e5m2))."""
    m, width = w.values.shape
    values = a.values if isinstance(a, Rows8) else a
    dev = values.device
    _on_gpu(values)
    kind, lds = _weights8(w, ())
    _plain("bias", bias, torch.float32, (m,))
    _same_device(dev, w=w.values, scales=w.scales, exps=a.exps if isinstance(a, Rows8) else None,
                 bias=bias, residual=residual, out=out)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return gemm8(w, a, bias, act, gated, residual, out_dtype, out, stream)
    values, code, lda, exps, lde, K = _rows8(a, width)
    B = values.shape[0]
    rows_out = m // 2 if gated else m
    out, ldo = _target8(out, B, rows_out, out_dtype, values)
    odt = _dt(out)
    ldr = 0 if residual is None else _pitch("residual", residual, (B, rows_out), out.dtype)
    nb = _bytes_needed("lq_gemm8_workspace_size", m, K, code, B)
    ws = _temporary(nb, dev)
    check(lib().lq_gemm8(_ptr(w.values), m, K, width, _ptr(w.scales), kind, lds, _ptr(values), code,
                         lda, _ptr(exps), lde, B, _ptr(bias), _act(act), int(gated), _ptr(residual),
                         ldr, _ptr(out), odt, ldo, _ptr(ws), nb, _handle(dev, stream)))
    return out


@_on_stream
def gemm8_grouped(w: Blocks8, a, offsets: torch.Tensor, rows: Optional[torch.Tensor] = None,
                  bias: Optional[torch.Tensor] = None, act: str = "none", gated: bool = False,
                  out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """The experts' products on ragged runs of rows (lq_gemm8_grouped): w 8-bit
    weights [E][m][K], a as in gemm8, offsets int32 [E + 1], rows int32 [R] (which
    row of a each sorted row is; None: its own), bias float32 [E][m].  Returns
    out [R][m], or [R][m/2] when gated; rows outside every run are not written."""
    E, m, width = w.values.shape
    values = a.values if isinstance(a, Rows8) else a
    dev = values.device
    _on_gpu(values)
    n_rows = values.shape[0]
    R = n_rows if rows is None else rows.shape[0]
    kind, lds = _weights8(w, (E,))
    _plain("bias", bias, torch.float32, (E, m))
    _plain("offsets", offsets, torch.int32, (E + 1,))
    _plain("rows", rows, torch.int32, (R,))
    _same_device(dev, w=w.values, scales=w.scales, exps=a.exps if isinstance(a, Rows8) else None,
                 offsets=offsets, rows=rows, bias=bias, out=out)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return gemm8_grouped(w, a, offsets, rows, bias, act, gated, out_dtype, out, stream)
    values, code, lda, exps, lde, K = _rows8(a, width)
    out, ldo = _target8(out, R, m // 2 if gated else m, out_dtype, values)
    odt = _dt(out)
    nb = _bytes_needed("lq_gemm8_grouped_workspace_size", E, m, K, code, n_rows, R)
    ws = _temporary(nb, dev)
    check(lib().lq_gemm8_grouped(_ptr(w.values), E, m, K, width, _ptr(w.scales), kind, lds,
                                 _ptr(values), code, lda, _ptr(exps), lde, n_rows, _ptr(rows),
                                 _ptr(offsets), R, _ptr(bias), _act(act), int(gated), _ptr(out), odt,
                                 ldo, _ptr(ws), nb, _handle(dev, stream)))
    return out


# ------------------------------------- rows sorted by expert and back
@_on_stream
def sort_rows(x, rows: torch.Tensor, out=None, stream=None):
    """x [T][n] in the experts' order (lq_sort_rows): out[r] = x[rows[r]], zeros
    where rows (int32 [R], route's) is outside [0, T).  x: float32, float16,
    bfloat16 or an 8-bit type, or Rows8 (values and exponents go along).  The
    gradient is join_rows(dout, pos)."""
    if isinstance(x, Rows8):
        _on_gpu(x.exps)
        held = Rows8(None, None) if out is None else out
        exps = held.exps
        if exps is None:
            exps = _exponents((rows.shape[0], x.exps.shape[1]), x.exps.device)
        return Rows8(sort_rows(x.values, rows, held.values, stream), sort_rows(x.exps, rows, exps, stream))
    T, n = x.shape
    R, dev = rows.shape[0], x.device
    _on_gpu(x)
    size = x.element_size()
    if size not in (1, 2, 4):
        raise TypeError(f"unsupported dtype {x.dtype}")
    _plain("rows", rows, torch.int32, (R,))
    _same_device(dev, rows=rows, out=out)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return sort_rows(x, rows, out, stream)
    ldx = _pitch("x", x, (T, n))
    out, ldo = _target(out, R, n, x.dtype, x)
    check(lib().lq_sort_rows(_ptr(x), size, T, n, ldx, _ptr(rows), R, _ptr(out), ldo,
                             _handle(dev, stream)))
    return out


@_on_stream
def join_rows(z: torch.Tensor, pos: torch.Tensor, weight: Optional[torch.Tensor] = None,
              residual: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The sorted rows z [R][n] back in the tokens' order, weighted and added
    (lq_join_rows): out[t] = residual[t] + sum_j weight[t][j] z[pos[t][j]], pos int32
    and weight float32 [T][k] (None: the plain sum); a position outside [0, R)
    adds nothing.  out_dtype (default z's), also the residual's: float32, float16
    or bfloat16; `residual` may be `out`."""
    R, n = z.shape
    T, k = pos.shape
    dev = z.device
    _on_gpu(z)
    _plain("pos", pos, torch.int32, (T, k))
    _plain("weight", weight, torch.float32, (T, k))
    _same_device(dev, pos=pos, weight=weight, residual=residual, out=out)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return join_rows(z, pos, weight, residual, out_dtype, out, stream)
    ldz = _pitch("z", z, (R, n))
    out, ldo = _target(out, T, n, out_dtype, z)
    ldr = 0 if residual is None else _pitch("residual", residual, (T, n), out.dtype)
    check(lib().lq_join_rows(_ptr(z), _dt(z), R, n, ldz, _ptr(pos), _ptr(weight), T, k,
                             _ptr(residual), ldr, _ptr(out), _dt(out), ldo, _handle(dev, stream)))
    return out


@_on_stream
def join_rows_grad(dy: torch.Tensor, z: torch.Tensor, pos: torch.Tensor, weight: torch.Tensor,
                   rows: Optional[torch.Tensor] = None, stream=None
                   ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gradients of join_rows with weights, from dy [T][n] (lq_join_rows_grad):
    (dz [R][n] of z's type, dweight float32 [T][k]).  With rows (route's) the
    rows of dz that no token has are zeros; without, every row must be named
    in pos, for the others are not written.  Positions of two pairs must differ,
    as route's do.  The residual's gradient is dy."""
    R, n = z.shape
    T, k = pos.shape
    dev = z.device
    _on_gpu(z)
    _plain("pos", pos, torch.int32, (T, k))
    _plain("weight", weight, torch.float32, (T, k))
    _plain("rows", rows, torch.int32, (R,))
    _same_device(dev, dy=dy, pos=pos, weight=weight, rows=rows)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return join_rows_grad(dy, z, pos, weight, rows, stream)
    ldy = _pitch("dy", dy, (T, n), z.dtype)
    ldz = _pitch("z", z, (R, n))
    dz = torch.empty((R, n), dtype=z.dtype, device=dev)
    dweight = torch.empty((T, k), dtype=torch.float32, device=dev)
    check(lib().lq_join_rows_grad(_ptr(dy), _dt(z), ldy, _ptr(z), ldz, R, n, _ptr(pos), _ptr(weight),
                                  T, k, _ptr(rows), _ptr(dz), n, _ptr(dweight),
                                  _handle(dev, stream)))
    return dz, dweight


# ----------------------------------------------------------------- layer
class DeviceLayer:
    """A layer's stored arrays resident on the GPU (uploaded once)."""

    def __init__(self, packed, M, t_inv, s, d: int, D: int, n: int, act_dtype: str,
                 device="cuda"):
        import numpy as np
        self.d, self.D, self.n = d, D, n
        self.K = n // d * D
        self.m = packed.shape[0]
        self.act_dtype = act_dtype
        self.w = torch.from_numpy(np.ascontiguousarray(packed).view(np.int32)).to(device)
        self.M = torch.from_numpy(np.ascontiguousarray(M, dtype=np.float32)).to(device)
        self.t_inv = to_torch_16(t_inv, act_dtype).to(device)
        self.s = torch.from_numpy(np.ascontiguousarray(s, dtype=np.float32)).to(device)

    @classmethod
    def from_synth(cls, L, device="cuda") -> "DeviceLayer":
        return cls(L.packed, L.M, L.t_inv, L.s, L.d, L.D, L.n, L.dtype, device)

    def _parts_ok(self, a: torch.Tensor) -> bool:
        """The lift into the GEMV's operand image takes a and T^-1 of one
        16-bit type and d in {4, 8, 16, 32}."""
        return (a.dtype in (torch.float16, torch.bfloat16) and a.dtype == self.t_inv.dtype
                and self.d in (4, 8, 16, 32) and self.d <= self.D <= 256)

    def forward(self, a: torch.Tensor, gemm_dtype: torch.dtype = torch.float16,
                path: str = "auto") -> torch.Tensor:
        """o [B][m]: lift then the GEMV (B <= 16) or the GEMM (larger B), the
        faster paths at the workload shapes (6 - 16 tokens: the lift into the
        GEMV's operand image, when it takes the shape).  Paths: "gemv" / "gemm" force
        those; "fused" the one-token layer with the lift inside the GEMV
        (lq_layer_b1); "decoded" u = T^-1 a (the lift with M = I_4) then the
        decode-weights product; "parts" the lift into the GEMV's float8-part
        operand image, then the GEMV on it (lq_lift_parts, lq_gemv_parts)."""
        B = a.shape[0]
        if path == "fused":
            return layer_b1(a, self.t_inv, self.M, self.d, self.D, self.w, self.s)
        if path == "decoded":
            eye = torch.eye(4, dtype=torch.float32, device=a.device)
            u = lift(a, self.t_inv, eye, 4, 4, out_dtype=torch.float16)
            return gemm_decoded(self.w, self.s, self.M, self.d, self.D, u)
        if path == "auto" and 6 <= B <= 16 and self._parts_ok(a):
            path = "parts"
        if path == "parts":
            img = lift_parts(a, self.t_inv, self.M, self.d, self.D)
            return gemv_parts(self.w, self.s, img, self.K, B)
        use_gemm = path == "gemm" or (path == "auto" and B > 16)
        if use_gemm:
            al = lift(a, self.t_inv, self.M, self.d, self.D, out_dtype=gemm_dtype)
            return gemm(self.w, self.s, al, self.K)
        al = lift(a, self.t_inv, self.M, self.d, self.D, out_dtype=torch.float32)
        return gemv(self.w, self.s, al, self.K)

    def forward_ep(self, a: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none",
                   gated: bool = False, residual: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None,
                   lift_dtype: torch.dtype = torch.float16) -> torch.Tensor:
        """act(o + bias) + residual (or the gated form) in out_dtype (default
        a's type) for any number of tokens: the lift into lift_dtype, then
        lq_gemm_ep.  float16 keeps 11 bits of the lifted values; past 65504 it
        overflows (a token with such a value gives NaN): layers whose
        lifted values may lie there take lift_dtype=torch.bfloat16, 8 bits
        (errors of 2.8e-3 of a token's largest output against 3.6e-4)."""
        if out_dtype is None:
            out_dtype = a.dtype
        al = lift(a, self.t_inv, self.M, self.d, self.D, out_dtype=lift_dtype)
        return gemm_ep(self.w, self.s, al, bias=bias, act=act, gated=gated, residual=residual,
                       out_dtype=out_dtype)


class DeviceExperts:
    """A mixture-of-experts MLP resident on the GPU: E experts of 1-bit lifted
    layers, w1 [E][2 f][ldw] (gate rows, then up rows) on n inputs, w2 [E][n][ldw]
    on f, their row scales s1 [E][2 f] and s2 [E][n], and the transforms that all
    experts share, t1 [n/128][128][128], t2 [f/128][128][128], M1 and M2 [d][D]."""

    def __init__(self, w1, s1, t1, M1, w2, s2, t2, M2, d: int, D: int, k: int, act: str = "silu",
                 bias1=None, bias2=None):
        self.w1, self.s1, self.t1, self.M1, self.bias1 = w1, s1, t1, M1, bias1
        self.w2, self.s2, self.t2, self.M2, self.bias2 = w2, s2, t2, M2, bias2
        self.d, self.D, self.k, self.act = d, D, k, act

    def forward(self, x: torch.Tensor, logits: torch.Tensor,
                residual: Optional[torch.Tensor] = None, valid: Optional[torch.Tensor] = None,
                renorm: bool = True) -> torch.Tensor:
        """x [T][n] (float16 or bfloat16), router logits [T][E] -> [T][n]: each token
        through its k experts, weighted, plus the residual.  valid[t] == 0: none.
        No tokens give no rows."""
        if x.shape[0] == 0:                        # the lift takes one row at least
            return torch.empty((0, self.w2.shape[1]), dtype=x.dtype, device=x.device)
        r = route(logits, self.k, valid=valid, renorm=renorm)
        a = lift(x, self.t1, self.M1, self.d, self.D, out_dtype=x.dtype)
        h = gemm_grouped(self.w1, self.s1, a, r.offsets, rows=r.rows, bias=self.bias1,
                         act=self.act, gated=True)
        hl = lift(h, self.t2, self.M2, self.d, self.D, out_dtype=x.dtype)
        return gemm_join(self.w2, self.s2, hl, r.offsets, r.pos, r.weight, bias=self.bias2,
                         residual=residual)


def to_torch_16(x, dtype: str) -> torch.Tensor:
    """Host array in storage format (float16, or bf16 bits as uint16) -> torch CPU tensor."""
    import numpy as np
    x = np.ascontiguousarray(x)
    if dtype == "f16":
        return torch.from_numpy(x.astype(np.float16))
    if dtype == "bf16":
        return torch.from_numpy(x.view(np.int16)).view(torch.bfloat16)
    if dtype == "f32":
        return torch.from_numpy(x.astype(np.float32))
    raise ValueError(dtype)
