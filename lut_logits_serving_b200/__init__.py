"""librqlut Python binding: LUT-based serving of a residual-product-quantized
(RQ) tied embedding on one B200.

Thin ctypes marshalling over the C ABI declared in ``include/rqlut.h``; every
step of the computation runs in the library's sm_100a CUDA kernels.  PyTorch
only provides device memory and the current stream.  The functions keep the C
names:

* ``rq_lut_build``  -- per-token tables T[p][k][b] = <h_b[m], C[m][l][k]>
* ``rq_lut_logits`` -- z[b][v] = sum_p T[p][code[v][p]][b], softcap, argmax
* ``rq_logits_from_hidden`` -- both, large batches in token groups of 32;
  a full group's rows are decoded and multiplied on the tensor cores
  (``rq_logits_from_hidden_path`` picks tables, FP32 or tensor cores)
* ``rq_decode_rows`` -- bf16 input rows rebuilt on demand
* ``rq_pack10`` -- uint16 codes -> 10-bit packed rows
* ``rq_xent``, ``rq_distill`` -- cross entropy and distillation from a
  teacher's top logits on the head, without keeping its logits;
  ``rq_xent_grad``, ``rq_distill_grad`` -- their gradients with respect to
  the hidden states and the codebooks (``rq_prepare_grad`` once per artifact)
* ``rq_prepare_sched``, ``rq_prepare_rot10`` -- the batch-1 layouts of
  uint16 and 10-bit codes (bank-scheduled, rotated slices)

(method: "Gemma-2 runtime compression: NF4 + LUT serving", LUT section.)
There is no CPU fallback: if the library or a GPU is missing, calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

__all__ = [
    "RqDims", "RqError", "U16", "PACKED10", "SCHED", "U8", "ROT10", "lib", "rq_pack8", "dims",
    "rq_prepare_sched", "rq_prepare_rot10",
    "rq_status_string", "rq_version", "rq_codes_bytes", "rq_lut_token_stride",
    "rq_lut_bytes", "rq_logits_workspace_bytes", "rq_fused_workspace_bytes",
    "rq_lut_build", "rq_lut_logits", "rq_logits_from_hidden", "rq_logits_from_hidden_path",
    "rq_decode_rows",
    "rq_pack10", "rq_device_error", "rq_set_profile_events", "rq_lut_logits_static",
    "rq_greedy_step", "rq_encode", "rq_topk_workspace_bytes", "rq_topk_sample",
    "rq_last_cuda_error", "rq_cuda_error_name", "PATH_AUTO", "PATH_TABLES", "PATH_DECODE_FP32",
    "PATH_DECODE_TC", "rq_loss_workspace_bytes", "rq_xent", "rq_xent_grad", "rq_distill",
    "rq_distill_grad", "rq_grad_index_bytes", "rq_prepare_grad", "rq_argmax_candidates", "rq_argmax_merge", "shard_rows", "rq_sharded_logits",
]

U16 = 0
PACKED10 = 1
SCHED = 2
U8 = 3
ROT10 = 4        # RQ_CODES_PACKED10_ROT
# kernel of full 32-token groups in rq_logits_from_hidden (rqlut.h RQ_PATH_*)
PATH_AUTO = 0
PATH_TABLES = 1
PATH_DECODE_FP32 = 2
PATH_DECODE_TC = 3

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "librqlut.so")


class RqDims(ctypes.Structure):
    _fields_ = [("V", ctypes.c_int64), ("D", ctypes.c_int32), ("M", ctypes.c_int32),
                ("L", ctypes.c_int32), ("K", ctypes.c_int32)]

    def __repr__(self):
        return f"RqDims(V={self.V}, D={self.D}, M={self.M}, L={self.L}, K={self.K})"


def dims(V, D, M, L, K) -> RqDims:
    return RqDims(int(V), int(D), int(M), int(L), int(K))


class RqError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        msg = f"{fn} failed: {rq_status_string(status)} ({status})"
        if status == 4:   # RQ_ERR_CUDA: name the runtime error behind it
            err = rq_last_cuda_error(clear=True)
            msg += f" [{rq_cuda_error_name(err)}]"
        super().__init__(msg)


_lib = None
_p = ctypes.c_void_p
_i = ctypes.c_int
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t
_f = ctypes.c_float

_SIGNATURES = {
    "rq_status_string": (ctypes.c_char_p, [_i]),
    "rq_version": (_i, []),
    "rq_codes_bytes": (_sz, [RqDims, _i]),
    "rq_lut_token_stride": (_i, [_i]),
    "rq_lut_bytes": (_sz, [RqDims, _i]),
    "rq_logits_workspace_bytes": (_sz, [RqDims, _i, _i, _i]),
    "rq_fused_workspace_bytes": (_sz, [RqDims, _i, _i, _i]),
    "rq_lut_build": (_i, [_p, _p, RqDims, _i, _p, _p]),
    "rq_lut_logits": (_i, [_p, _i, RqDims, _p, _i, _f, _p, _p, _p, _sz, _p]),
    "rq_logits_from_hidden": (_i, [_p, _p, _p, _i, RqDims, _i, _f, _p, _p, _p, _sz, _p]),
    "rq_logits_from_hidden_path": (_i, [_p, _p, _p, _i, RqDims, _i, _f, _p, _p, _p, _sz, _i,
                                        _p]),
    "rq_decode_rows": (_i, [_p, _i64, _p, _i, _p, RqDims, _f, _p, _p]),
    "rq_pack10": (_i, [_p, RqDims, _p, _p]),
    "rq_pack8": (_i, [_p, RqDims, _p, _p]),
    "rq_encode": (_i, [_p, RqDims, _p, _p, _p]),
    "rq_topk_workspace_bytes": (_sz, [_i64, _i, _i]),
    "rq_last_cuda_error": (_i, [_i]),
    "rq_cuda_error_name": (ctypes.c_char_p, [_i]),
    "rq_topk_sample": (_i, [_p, _i64, _i, _i, _f, ctypes.c_uint64, ctypes.c_uint64, _p, _p, _p,
                            _p, _sz, _p]),
    "rq_device_error": (_i, [ctypes.POINTER(ctypes.c_uint32), _i]),
    "rq_set_profile_events": (_i, [_p, _p]),
    "rq_prepare_sched": (_i, [_p, RqDims, _p, _p, _p]),
    "rq_prepare_rot10": (_i, [_p, RqDims, _p, _p, _p]),
    "rq_lut_logits_static": (_i, [_p, _i, RqDims, _p, _i, _f, _p, _p, _p]),
    "rq_greedy_step": (_i, [_p, _p, _p, _i, RqDims, _i, _f, _p, _p, _f, _p, _p, _sz, _p]),
    "rq_loss_workspace_bytes": (_sz, [RqDims, _i, _i, _i, _i]),
    "rq_xent": (_i, [_p, _i, _p, _p, _i, RqDims, _i, _f, _p, _p, _p, _p, _sz, _p]),
    "rq_xent_grad": (_i, [_p, _i, _p, _p, _i, RqDims, _i, _f, _p, _p, _p, _p, _p, _p, _p, _sz,
                          _p]),
    "rq_distill": (_i, [_p, _i, _p, _p, _i, RqDims, _i, _f, _p, _p, _i, _f, _p, _p, _p, _sz, _p]),
    "rq_distill_grad": (_i, [_p, _i, _p, _p, _i, RqDims, _i, _f, _p, _p, _i, _f, _p, _p, _p, _p,
                             _p, _p, _sz, _p]),
    "rq_grad_index_bytes": (_sz, [RqDims]),
    "rq_prepare_grad": (_i, [_p, _i, RqDims, _p, _p]),
    "rq_argmax_candidates": (_i, [_p, _p, _i, _i64, _i64, _p, _p, _p]),
    "rq_argmax_merge": (_i, [_p, _p, _i, _i, _p, _p]),
}


def lib() -> ctypes.CDLL:
    """Load librqlut.so (built in-tree by ``lut_logits_serving_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"librqlut.so not found at {LIB_PATH}; build it with "
                "`python -m lut_logits_serving_b200.build` (there is no CPU fallback)")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


# ------------------------------------------------------------ host queries

def rq_status_string(status: int) -> str:
    return lib().rq_status_string(int(status)).decode()


def rq_version() -> int:
    return lib().rq_version()


def rq_codes_bytes(d: RqDims, fmt: int) -> int:
    return lib().rq_codes_bytes(d, fmt)


def rq_lut_token_stride(B: int) -> int:
    return lib().rq_lut_token_stride(B)


def rq_lut_bytes(d: RqDims, B: int) -> int:
    return lib().rq_lut_bytes(d, B)


def rq_logits_workspace_bytes(d: RqDims, B: int, fmt: int, want_argmax: bool) -> int:
    return lib().rq_logits_workspace_bytes(d, B, fmt, int(bool(want_argmax)))


def rq_fused_workspace_bytes(d: RqDims, B: int, fmt: int, want_argmax: bool) -> int:
    return lib().rq_fused_workspace_bytes(d, B, fmt, int(bool(want_argmax)))


# ------------------------------------------------------------ device calls

def _torch():
    import torch
    return torch


def _stream(stream):
    torch = _torch()
    if stream is None:
        # without a Stream object around it, 2 us of a small call; not a public
        # name of torch, so where it is missing the public call serves
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return ctypes.c_void_p(raw(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _cuda(t, dtype, name, nbytes=None):
    """Device pointer of `t` after checking its type, layout and, with
    `nbytes`, that it holds at least that many bytes: the C calls take bare
    pointers, so a short buffer would otherwise be read or written past its
    end."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if nbytes is not None and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name}: {t.numel() * t.element_size()} bytes, "
                         f"the call needs {nbytes}")
    if not _on_device(t):
        raise ValueError(f"{name}: must be a CUDA tensor (no CPU fallback)")
    return ctypes.c_void_p(t.data_ptr())


def _on_device(t):
    return t.is_cuda


def _ptr_or_null(t, dtype, name, nbytes=None):
    return ctypes.c_void_p(None) if t is None else _cuda(t, dtype, name, nbytes)


def _book_bytes(d):
    """Bytes of the codebooks C [M, L, K, ds] (fp32)."""
    return d.M * d.L * d.K * (d.D // d.M if d.M > 0 else 0) * 4


def _tokens(h, d, name="h"):
    """B of hidden states h [B, D] (or [D] for one token)."""
    if h.dim() == 1 and h.shape[0] == d.D:
        return 1
    if h.dim() != 2 or h.shape[1] != d.D:
        raise ValueError(f"{name}: shape {tuple(h.shape)}, expected [B, {d.D}]")
    return h.shape[0]


def _check(fn, status):
    if status != 0:
        raise RqError(fn, status)


def _codes_dtype(fmt):
    torch = _torch()
    return torch.uint8 if fmt in (PACKED10, U8, ROT10) else torch.uint16


def _empty(shape, dtype, like):
    torch = _torch()
    return torch.empty(shape, dtype=dtype, device=like.device)


def _workspace(nbytes, like, ws):
    torch = _torch()
    if nbytes == 0:
        return ctypes.c_void_p(None), 0, ws
    if ws is None or ws.numel() * ws.element_size() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    return _cuda(ws, None, "ws"), ws.numel() * ws.element_size(), ws


def rq_lut_build(h, C, d: RqDims, lut=None, stream=None):
    """h float32 [B, D], C float32 [M, L, K, ds] -> lut float32 [P, K, Bs]."""
    torch = _torch()
    B = _tokens(h, d)
    Bs = rq_lut_token_stride(B)
    if lut is None:
        lut = _empty((d.M * d.L, d.K, Bs), torch.float32, h)
    _check("rq_lut_build", lib().rq_lut_build(
        _cuda(h, torch.float32, "h"), _cuda(C, torch.float32, "C", _book_bytes(d)), d, B,
        _cuda(lut, torch.float32, "lut", rq_lut_bytes(d, B)), _stream(stream)))
    return lut


def rq_lut_logits(codes, fmt: int, d: RqDims, lut, B: int, softcap: float = 30.0,
                  want_logits: bool = True, want_argmax: bool = False, logits=None,
                  argmax=None, ws=None, stream=None):
    """Returns (logits float32 [B, V] or None, argmax int32 [B] or None, ws)."""
    torch = _torch()
    if want_logits and logits is None:
        logits = _empty((B, d.V), torch.float32, lut)
    if want_argmax and argmax is None:
        argmax = _empty((B,), torch.int32, lut)
    nbytes = rq_logits_workspace_bytes(d, B, fmt, argmax is not None)
    wp, wn, ws = _workspace(nbytes, lut, ws)
    _check("rq_lut_logits", lib().rq_lut_logits(
        _cuda(codes, _codes_dtype(fmt), "codes", rq_codes_bytes(d, fmt)), fmt, d,
        _cuda(lut, torch.float32, "lut", rq_lut_bytes(d, B)), B,
        float(softcap), _ptr_or_null(logits, torch.float32, "logits", B * d.V * 4),
        _ptr_or_null(argmax, torch.int32, "argmax", B * 4), wp, wn, _stream(stream)))
    return logits, argmax, ws


def rq_logits_from_hidden(h, C, codes, fmt: int, d: RqDims, softcap: float = 30.0,
                          want_logits: bool = True, want_argmax: bool = False, logits=None,
                          argmax=None, ws=None, stream=None, path: int = None):
    """Returns (logits float32 [B, V] or None, argmax int32 [B] or None, ws).
    ``path`` (one of PATH_*) picks the kernel of full 32-token groups; None
    is the library's default (rq_logits_from_hidden)."""
    torch = _torch()
    B = _tokens(h, d)
    if want_logits and logits is None:
        logits = _empty((B, d.V), torch.float32, h)
    if want_argmax and argmax is None:
        argmax = _empty((B,), torch.int32, h)
    nbytes = rq_fused_workspace_bytes(d, B, fmt, argmax is not None)
    wp, wn, ws = _workspace(nbytes, h, ws)
    args = (_cuda(h, torch.float32, "h"), _cuda(C, torch.float32, "C", _book_bytes(d)),
            _cuda(codes, _codes_dtype(fmt), "codes", rq_codes_bytes(d, fmt)), fmt, d, B,
            float(softcap), _ptr_or_null(logits, torch.float32, "logits", B * d.V * 4),
            _ptr_or_null(argmax, torch.int32, "argmax", B * 4), wp, wn)
    if path is None:
        _check("rq_logits_from_hidden", lib().rq_logits_from_hidden(*args, _stream(stream)))
    else:
        _check("rq_logits_from_hidden_path",
               lib().rq_logits_from_hidden_path(*args, int(path), _stream(stream)))
    return logits, argmax, ws


def rq_logits_from_hidden_path(h, C, codes, fmt: int, d: RqDims, path: int,
                               softcap: float = 30.0, **kw):
    """rq_logits_from_hidden with an explicit kernel for full token groups."""
    return rq_logits_from_hidden(h, C, codes, fmt, d, softcap, path=path, **kw)


def rq_argmax_candidates(logits, argmax, row0: int, val=None, gidx=None, stream=None):
    """A vocabulary shard's winner per token: (value float32 [B], global row
    int32 [B]) from its logits [B, V_shard] and argmax [B]."""
    torch = _torch()
    if logits.dim() != 2:
        raise ValueError("logits: [B, V_shard] expected")
    B, V = logits.shape
    if val is None:
        val = _empty((B,), torch.float32, logits)
    if gidx is None:
        gidx = _empty((B,), torch.int32, logits)
    _check("rq_argmax_candidates", lib().rq_argmax_candidates(
        _cuda(logits, torch.float32, "logits"), _cuda(argmax, torch.int32, "argmax", B * 4),
        B, V, int(row0), _cuda(val, torch.float32, "val", B * 4),
        _cuda(gidx, torch.int32, "gidx", B * 4), _stream(stream)))
    return val, gidx


def rq_argmax_merge(val, gidx, out=None, stream=None):
    """Global argmax int32 [B] from n shards' candidates val, gidx [n, B]."""
    torch = _torch()
    if val.dim() != 2 or tuple(gidx.shape) != tuple(val.shape):
        raise ValueError("val, gidx: [n, B] expected")
    n, B = val.shape
    if out is None:
        out = _empty((B,), torch.int32, val)
    _check("rq_argmax_merge", lib().rq_argmax_merge(
        _cuda(val, torch.float32, "val"), _cuda(gidx, torch.int32, "gidx"), n, B,
        _cuda(out, torch.int32, "argmax", B * 4), _stream(stream)))
    return out


def shard_rows(V: int, rank: int, world: int):
    """Rows [row0, row1) of vocabulary shard `rank` of `world` (even split)."""
    if world < 1 or not 0 <= rank < world:
        raise ValueError("rank, world")
    return V * rank // world, V * (rank + 1) // world


def rq_sharded_logits(h, C, codes_shard, fmt: int, d_shard: RqDims, row0: int,
                      softcap: float = 30.0, group=None, ws=None, stream=None):
    """Logits of this rank's vocabulary rows and the global greedy pick: the
    fused call on the shard, its per-token winner, one all-gather of the
    winners over the process group (NCCL), and the merge.  Returns (logits
    [B, V_shard], argmax int32 [B] of global rows, ws)."""
    torch = _torch()
    logits, am, ws = rq_logits_from_hidden(h, C, codes_shard, fmt, d_shard, softcap,
                                           want_argmax=True, ws=ws, stream=stream)
    val, gidx = rq_argmax_candidates(logits, am, row0, stream=stream)
    world = 1
    import torch.distributed as dist
    if dist.is_available() and dist.is_initialized():
        world = dist.get_world_size(group)
    if world > 1:
        # flat [world * B] buffers, rank-major (the layout every backend takes);
        # the collectives are ordered after the candidates on the call's stream
        vals = _empty((world * val.numel(),), torch.float32, val)
        idxs = _empty((world * gidx.numel(),), torch.int32, gidx)
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            dist.all_gather_into_tensor(vals, val, group=group)
            dist.all_gather_into_tensor(idxs, gidx, group=group)
        vals, idxs = vals.view(world, -1), idxs.view(world, -1)
    else:
        vals, idxs = val.view(1, -1), gidx.view(1, -1)
    return logits, rq_argmax_merge(vals, idxs, stream=stream), ws


def rq_decode_rows(ids, codes, fmt: int, C, d: RqDims, scale: float, out=None, stream=None):
    """ids int32 [N] -> bf16 rows [N, D] (returned as torch.bfloat16)."""
    torch = _torch()
    N = ids.numel()
    if out is None:
        out = _empty((N, d.D), torch.bfloat16, ids)
    if out.dtype not in (torch.bfloat16, torch.uint16, torch.int16):
        raise ValueError("out: bf16 rows expected")
    _check("rq_decode_rows", lib().rq_decode_rows(
        _cuda(ids, torch.int32, "ids"), N,
        _cuda(codes, _codes_dtype(fmt), "codes", rq_codes_bytes(d, fmt)), fmt,
        _cuda(C, torch.float32, "C", _book_bytes(d)), d, float(scale),
        _cuda(out, None, "out", N * d.D * 2), _stream(stream)))
    return out


def rq_pack10(codes_u16, d: RqDims, out=None, stream=None):
    """uint16 [V, P] (or [V, M, L]) -> uint8 [V, ceil(10 P / 8)]."""
    torch = _torch()
    if out is None:
        out = _empty((d.V, rq_codes_bytes(d, PACKED10) // d.V), torch.uint8, codes_u16)
    _check("rq_pack10", lib().rq_pack10(
        _cuda(codes_u16, torch.uint16, "codes_u16", rq_codes_bytes(d, U16)), d,
        _cuda(out, torch.uint8, "packed", rq_codes_bytes(d, PACKED10)), _stream(stream)))
    return out


def rq_encode(X, C, d: RqDims, out=None, stream=None):
    """Rows float32 [V, D] -> uint16 codes [V, M*L]: greedy residual
    nearest-codeword assignment against C [M, L, K, ds]."""
    torch = _torch()
    if out is None:
        out = _empty((d.V, d.M * d.L), torch.uint16, X)
    _check("rq_encode", lib().rq_encode(
        _cuda(X, torch.float32, "X", d.V * d.D * 4), d,
        _cuda(C, torch.float32, "C", _book_bytes(d)),
        _cuda(out, torch.uint16, "codes", rq_codes_bytes(d, U16)), _stream(stream)))
    return out


def rq_last_cuda_error(clear: bool = False) -> int:
    return int(lib().rq_last_cuda_error(int(bool(clear))))


def rq_cuda_error_name(err: int) -> str:
    return lib().rq_cuda_error_name(int(err)).decode()


def rq_topk_workspace_bytes(V: int, B: int, k: int) -> int:
    return int(lib().rq_topk_workspace_bytes(V, B, k))


def rq_topk_sample(logits, k: int, temperature: float = 1.0, seed: int = 0, step: int = 0,
                   topk_val=None, topk_idx=None, token=None, want_topk: bool = True,
                   ws=None, stream=None):
    """logits float32 [B, V] (device) -> (topk_val [B, k], topk_idx [B, k], token [B]);
    the top-k outputs are None with want_topk=False."""
    torch = _torch()
    if logits.dim() != 2:
        raise ValueError("logits: [B, V] expected")
    B, V = logits.shape
    if want_topk:
        if topk_val is None:
            topk_val = _empty((B, k), torch.float32, logits)
        if topk_idx is None:
            topk_idx = _empty((B, k), torch.int32, logits)
    if token is None:
        token = _empty((B,), torch.int32, logits)
    nbytes = rq_topk_workspace_bytes(V, B, k)
    wsp, wsn, ws = _workspace(max(nbytes, 1), logits, ws)
    _check("rq_topk_sample", lib().rq_topk_sample(
        _cuda(logits, torch.float32, "logits"), V, B, k, float(temperature),
        ctypes.c_uint64(seed), ctypes.c_uint64(step),
        _ptr_or_null(topk_val, torch.float32, "topk_val", B * k * 4),
        _ptr_or_null(topk_idx, torch.int32, "topk_idx", B * k * 4),
        _cuda(token, torch.int32, "token", B * 4), wsp, wsn, _stream(stream)))
    return topk_val, topk_idx, token


def rq_pack8(codes_u16, d: RqDims, out=None, stream=None):
    """uint16 [V, P] (or [V, M, L]) -> uint8 [V, P] (RQ_CODES_U8, K <= 256)."""
    torch = _torch()
    if out is None:
        out = _empty((d.V, d.M * d.L), torch.uint8, codes_u16)
    _check("rq_pack8", lib().rq_pack8(
        _cuda(codes_u16, torch.uint16, "codes_u16", rq_codes_bytes(d, U16)), d,
        _cuda(out, torch.uint8, "packed", rq_codes_bytes(d, U8)), _stream(stream)))
    return out


# ------------------------------------------------------------ losses

def rq_loss_workspace_bytes(d: RqDims, N: int, fmt: int, k: int = 1, grad: bool = False) -> int:
    """Workspace of a loss on N tokens (and, with grad, of its gradient);
    k entries per teacher's list (0 or 1 for cross entropy)."""
    return int(lib().rq_loss_workspace_bytes(d, N, fmt, k, int(bool(grad))))


def rq_grad_index_bytes(d: RqDims) -> int:
    return int(lib().rq_grad_index_bytes(d))


@functools.lru_cache(maxsize=256)
def _loss_sizes(V, D, M, L, K, fmt, N, k, grad):
    """(codes, codebooks, index, workspace) bytes of a loss call: pure
    arithmetic, kept because a small call's time is its host side."""
    d = dims(V, D, M, L, K)
    return (rq_codes_bytes(d, fmt), _book_bytes(d), rq_grad_index_bytes(d) if grad else 0,
            rq_loss_workspace_bytes(d, N, fmt, k, grad))


def _stream_on(stream, device, name):
    if stream is not None and stream.device != device:
        raise ValueError(f"stream on {stream.device}, {name} on {device}")


class _LossCall:
    """Checks and pointers of one call of the losses: every tensor on h's
    device, which is made current with the call's stream for the call's time
    (what the call allocates then belongs to that stream)."""

    def __init__(self, h, d, fmt, k, grad, stream):
        torch = _torch()
        if not isinstance(h, torch.Tensor):
            raise ValueError("h: expected a torch.Tensor")
        if h.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"h: dtype {h.dtype}, expected float32 or bfloat16")
        self.tensor, self.h, self.device, self.N = torch.Tensor, h, h.device, _tokens(h, d)
        self.bf16 = int(h.dtype == torch.bfloat16)
        self.code_dtype = torch.uint16 if fmt in (U16, SCHED) else torch.uint8
        (self.codes_bytes, self.book_bytes, self.index_bytes,
         self.ws_bytes) = _loss_sizes(d.V, d.D, d.M, d.L, d.K, fmt, self.N, k, grad)
        self.stream, self.stack = stream, None

    def __enter__(self):
        if self.h.is_cuda:
            torch = _torch()
            if self.stream is not None or torch.cuda.current_device() != self.device.index:
                _stream_on(self.stream, self.device, "h")    # before anything is entered
                self.stack = contextlib.ExitStack()
                self.stack.enter_context(torch.cuda.device(self.device))
                if self.stream is not None:
                    self.stack.enter_context(torch.cuda.stream(self.stream))
        return self

    def __exit__(self, *exc):
        return self.stack.__exit__(*exc) if self.stack is not None else None

    def ptr(self, t, dtype, name, nbytes):
        """Address of `t` after the checks of _cuda and of its device (at once,
        then one by one to name what is wrong)."""
        if isinstance(t, self.tensor) and t.dtype is dtype and t.device == self.device and \
                t.nbytes >= nbytes and t.is_contiguous() and _on_device(t):
            return t.data_ptr()
        if not isinstance(t, self.tensor):
            raise ValueError(f"{name}: expected a torch.Tensor")
        if t.dtype is not dtype:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
        if t.nbytes < nbytes:
            raise ValueError(f"{name}: {t.nbytes} bytes, the call needs {nbytes}")
        if not _on_device(t):
            raise ValueError(f"{name}: must be a CUDA tensor (no CPU fallback)")
        raise ValueError(f"{name}: on {t.device}, h on {self.device}")

    def out(self, t, shape, dtype):
        return self.h.new_empty(shape, dtype=dtype) if t is None else t

    def workspace(self, ws):
        if ws is not None and not isinstance(ws, self.tensor):
            raise ValueError("ws: expected a torch.Tensor")
        if ws is None or ws.nbytes < self.ws_bytes:
            ws = self.h.new_empty((self.ws_bytes,), dtype=_torch().uint8)
        return ws, self.ptr(ws, ws.dtype, "ws", self.ws_bytes), ws.nbytes

    def head(self, C, codes, fmt, d, softcap):
        """The arguments every loss call begins with."""
        return (self.ptr(self.h, self.h.dtype, "h", 0), self.bf16,
                self.ptr(C, _torch().float32, "C", self.book_bytes),
                self.ptr(codes, self.code_dtype, "codes", self.codes_bytes), fmt, d, self.N,
                float(softcap))


def _lists(call, val, idx, temperature):
    """The arguments of a teacher's lists [N, k]."""
    torch = _torch()
    n = call.N * idx.shape[1] * 4
    return (call.ptr(val, torch.float32, "teacher_val", n),
            call.ptr(idx, torch.int32, "teacher_idx", n), idx.shape[1], float(temperature))


def _lists_k(h, val, idx):
    for t, name in ((h, "h"), (val, "teacher_val"), (idx, "teacher_idx")):
        if not isinstance(t, _torch().Tensor):
            raise ValueError(f"{name}: expected a torch.Tensor")
    if idx.dim() != 2 or idx.shape[0] != (h.shape[0] if h.dim() == 2 else 1) or \
            val.shape != idx.shape:
        raise ValueError("teacher_val, teacher_idx: [N, k] expected")
    return idx.shape[1]


def _run_loss(fn, h, C, codes, fmt, d, k, extra, softcap, loss, lse, ws, stream):
    f32 = _torch().float32
    with _LossCall(h, d, fmt, k, False, stream) as c:
        loss, lse = c.out(loss, (c.N,), f32), c.out(lse, (c.N,), f32)
        args = c.head(C, codes, fmt, d, softcap) + extra(c)
        ws, wp, wn = c.workspace(ws)
        _check(fn, getattr(lib(), fn)(*args, c.ptr(loss, f32, "loss", c.N * 4),
                                      c.ptr(lse, f32, "lse", c.N * 4), wp, wn, _stream(None)))
    return loss, lse, ws


def _run_grad(fn, h, C, codes, fmt, d, k, extra, lse, index, weight, softcap, want_dh, want_dC, dh,
              dC, ws, stream):
    torch = _torch()
    f32 = torch.float32
    with _LossCall(h, d, fmt, k, True, stream) as c:
        if want_dh:
            dh = c.out(dh, (c.N, d.D), h.dtype)
        if want_dC:
            dC = c.out(dC, (d.M, d.L, d.K, d.D // d.M), f32)
        args = c.head(C, codes, fmt, d, softcap) + extra(c)
        ws, wp, wn = c.workspace(ws)
        _check(fn, getattr(lib(), fn)(
            *args, c.ptr(lse, f32, "lse", c.N * 4),
            None if weight is None else c.ptr(weight, f32, "weight", c.N * 4),
            c.ptr(index, torch.uint8, "index", c.index_bytes),
            None if dh is None else c.ptr(dh, h.dtype, "dh", c.N * d.D * h.element_size()),
            None if dC is None else c.ptr(dC, f32, "dC", c.book_bytes), wp, wn, _stream(None)))
    return dh, dC, ws


def rq_prepare_grad(codes, fmt: int, d: RqDims, out=None, stream=None):
    """Codes in any layout -> the index uint8 [rq_grad_index_bytes(d)] that
    the gradients of the losses sum the vocabulary's rows by."""
    torch = _torch()
    if not isinstance(codes, torch.Tensor):
        raise ValueError("codes: expected a torch.Tensor")
    nbytes = rq_grad_index_bytes(d)
    _stream_on(stream, codes.device, "codes")
    with torch.cuda.device(codes.device) if codes.is_cuda else contextlib.nullcontext():
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            if out is None:
                out = _empty((nbytes,), torch.uint8, codes)
            args = (_cuda(codes, _codes_dtype(fmt), "codes", rq_codes_bytes(d, fmt)), fmt, d,
                    _cuda(out, torch.uint8, "index", nbytes))
            if out.device != codes.device:
                raise ValueError(f"out: on {out.device}, codes on {codes.device}")
            _check("rq_prepare_grad", lib().rq_prepare_grad(*args, _stream(None)))
    return out


def rq_xent(h, C, codes, fmt: int, d: RqDims, target, softcap: float = 30.0, loss=None, lse=None,
            ws=None, stream=None):
    """Softmax cross entropy of the head against target ids int32 [N] (below
    0: none, loss 0), h [N, D] float32 or bfloat16.  Returns (loss float32
    [N], lse float32 [N], ws)."""
    i32 = _torch().int32
    return _run_loss("rq_xent", h, C, codes, fmt, d, 1,
                     lambda c: (c.ptr(target, i32, "target", c.N * 4),), softcap, loss, lse, ws,
                     stream)


def rq_xent_grad(h, C, codes, fmt: int, d: RqDims, target, lse, index, weight=None,
                 softcap: float = 30.0, want_dh: bool = True, want_dC: bool = True, dh=None,
                 dC=None, ws=None, stream=None):
    """Gradient of sum_n weight[n] loss[n] of rq_xent (weight float32 [N],
    None: all 1), from its lse and rq_prepare_grad's index.  Returns (dh [N, D]
    in h's type or None, dC float32 [M, L, K, ds] or None, ws)."""
    i32 = _torch().int32
    return _run_grad("rq_xent_grad", h, C, codes, fmt, d, 1,
                     lambda c: (c.ptr(target, i32, "target", c.N * 4),), lse, index, weight,
                     softcap, want_dh, want_dC, dh, dC, ws, stream)


def rq_distill(h, C, codes, fmt: int, d: RqDims, teacher_val, teacher_idx,
               temperature: float = 1.0, softcap: float = 30.0, loss=None, lse=None, ws=None,
               stream=None):
    """Distillation from a teacher's top logits float32 [N, k] at ids int32
    [N, k] (below 0: none), as rq_topk_sample returns them.  Returns (loss
    float32 [N], lse float32 [N] at the temperature, ws)."""
    return _run_loss("rq_distill", h, C, codes, fmt, d, _lists_k(h, teacher_val, teacher_idx),
                     lambda c: _lists(c, teacher_val, teacher_idx, temperature), softcap, loss,
                     lse, ws, stream)


def rq_distill_grad(h, C, codes, fmt: int, d: RqDims, teacher_val, teacher_idx, lse, index,
                    weight=None, temperature: float = 1.0, softcap: float = 30.0,
                    want_dh: bool = True, want_dC: bool = True, dh=None, dC=None, ws=None,
                    stream=None):
    """Gradient of sum_n weight[n] loss[n] of rq_distill; see rq_xent_grad."""
    return _run_grad("rq_distill_grad", h, C, codes, fmt, d,
                     _lists_k(h, teacher_val, teacher_idx),
                     lambda c: _lists(c, teacher_val, teacher_idx, temperature), lse, index,
                     weight, softcap, want_dh, want_dC, dh, dC, ws, stream)


def rq_device_error(clear: bool = True) -> int:
    v = ctypes.c_uint32(0)
    _check("rq_device_error", lib().rq_device_error(ctypes.byref(v), int(bool(clear))))
    return v.value


def rq_set_profile_events(start=None, stop=None):
    """start/stop: torch.cuda.Event (enable_timing=True) or None to switch off."""
    sp = ctypes.c_void_p(start.cuda_event if start is not None else None)
    tp = ctypes.c_void_p(stop.cuda_event if stop is not None else None)
    _check("rq_set_profile_events", lib().rq_set_profile_events(sp, tp))


def rq_prepare_sched(codes_u16, d: RqDims, out=None, stats=None, stream=None):
    """uint16 codes [V, P] -> bank-scheduled uint16 codes [V, P] (RQ_CODES_SCHED).
    With stats=True returns (out, (steps, bank passes)) after a sync."""
    torch = _torch()
    if out is None:
        out = torch.empty((d.V, d.M * d.L), dtype=torch.uint16, device=codes_u16.device)
    st = None
    if stats:
        st = torch.zeros(2, dtype=torch.int64, device=codes_u16.device)
    _check("rq_prepare_sched", lib().rq_prepare_sched(
        _cuda(codes_u16, torch.uint16, "codes_u16", rq_codes_bytes(d, U16)), d,
        _cuda(out, torch.uint16, "out", rq_codes_bytes(d, SCHED)),
        _ptr_or_null(st, torch.int64, "stats", 16), _stream(stream)))
    if stats:
        v = st.cpu().tolist()
        return out, (v[0], v[1])
    return out


def rq_prepare_rot10(codes_u16, d: RqDims, out=None, stats=None, stream=None):
    """uint16 codes [V, P] -> RQ_CODES_PACKED10_ROT bytes (rotated 10-bit slices,
    then the rotations).  With stats=True returns (out, (steps, bank passes))
    after a sync."""
    torch = _torch()
    nbytes = rq_codes_bytes(d, ROT10)
    if out is None:
        out = torch.empty((nbytes,), dtype=torch.uint8, device=codes_u16.device)
    st = None
    if stats:
        st = torch.zeros(2, dtype=torch.int64, device=codes_u16.device)
    _check("rq_prepare_rot10", lib().rq_prepare_rot10(
        _cuda(codes_u16, torch.uint16, "codes_u16", rq_codes_bytes(d, U16)), d,
        _cuda(out, torch.uint8, "out", nbytes), _ptr_or_null(st, torch.int64, "stats", 16),
        _stream(stream)))
    if stats:
        v = st.cpu().tolist()
        return out, (v[0], v[1])
    return out


def rq_lut_logits_static(codes, fmt: int, d: RqDims, lut, B: int, softcap: float = 30.0,
                         want_logits: bool = True, want_argmax: bool = False, logits=None,
                         argmax=None, stream=None):
    """rq_lut_logits with the library's fixed device scratch as workspace
    (for callers that cannot allocate; see include/rqlut.h).
    Returns (logits or None, argmax or None)."""
    torch = _torch()
    if want_logits and logits is None:
        logits = _empty((B, d.V), torch.float32, lut)
    if want_argmax and argmax is None:
        argmax = _empty((B,), torch.int32, lut)
    _check("rq_lut_logits_static", lib().rq_lut_logits_static(
        _cuda(codes, _codes_dtype(fmt), "codes", rq_codes_bytes(d, fmt)), fmt, d,
        _cuda(lut, torch.float32, "lut", rq_lut_bytes(d, B)), B,
        float(softcap), _ptr_or_null(logits, torch.float32, "logits", B * d.V * 4),
        _ptr_or_null(argmax, torch.int32, "argmax", B * 4), _stream(stream)))
    return logits, argmax


def rq_greedy_step(h, C, codes, fmt: int, d: RqDims, softcap: float = 30.0, scale: float = 1.0,
                   want_logits: bool = True, logits=None, argmax=None, rows=None, ws=None,
                   stream=None):
    """Logits (optional), argmax and the bf16 input rows of the picked tokens.
    Returns (logits or None, argmax int32 [B], rows bf16 [B, D], ws)."""
    torch = _torch()
    B = _tokens(h, d)
    if want_logits and logits is None:
        logits = _empty((B, d.V), torch.float32, h)
    if argmax is None:
        argmax = _empty((B,), torch.int32, h)
    if rows is None:
        rows = _empty((B, d.D), torch.bfloat16, h)
    nbytes = rq_fused_workspace_bytes(d, B, fmt, True)
    wp, wn, ws = _workspace(nbytes, h, ws)
    _check("rq_greedy_step", lib().rq_greedy_step(
        _cuda(h, torch.float32, "h"), _cuda(C, torch.float32, "C", _book_bytes(d)),
        _cuda(codes, _codes_dtype(fmt), "codes", rq_codes_bytes(d, fmt)), fmt, d, B,
        float(softcap), _ptr_or_null(logits, torch.float32, "logits", B * d.V * 4),
        _cuda(argmax, torch.int32, "argmax", B * 4), float(scale),
        _cuda(rows, None, "rows", B * d.D * 2), wp, wn, _stream(stream)))
    return logits, argmax, rows, ws
