"""Python binding for libmmq.so, the MI355X (gfx950) prefill MMQ library.

Argument marshalling only: every step of the path (activation quantisation, weight repack,
the MMQ contraction, MoE grouping) runs in the library's HIP kernels. PyTorch provides device
memory and the stream. There is no CPU fallback: if the library is missing, every call raises.

The functions mirror include/mmq.h one to one (same names without the `mmq_` prefix):

    act_bytes, act_region_offsets, quantize_act, packed_bytes, repack_weights, gemm,
    gemm_id_workspace_bytes, gemm_id, gemm_id_noalloc, gemm_id_noalloc_max_workspace_bytes,
    group_bytes, group_region_offsets, group_rows, moe_gather, moe_combine, moe_combine_grad,
    lora_workspace_bytes, lora, lora_grad_workspace_bytes, lora_grad, cache_bytes, cache_write,
    cache_read, cache_attn_workspace_bytes, cache_attn, status_string

plus `group_views` (the regions of a plan as tensors), `cache_shape` (a cache's records as a
tensor's shape) and host-side encoders/decoders of the
documented act layouts (`act_to_host`, `act_q8_1_pack_host` and friends for q8_1,
`act_i8_pack_host` / `act_i8_to_host` for the per-token int8 form), used by tests and the bench
to fill or read act buffers.
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmmq.so")

# enums (include/mmq.h)
MMQ_OK, MMQ_EINVAL, MMQ_EUNSUPPORTED, MMQ_EALIGN, MMQ_EWORKSPACE, MMQ_EHIP = range(6)
WTYPE = {"q8_0": 0, "q4_0": 1, "q4_K": 2, "iq1t": 3, "i8_row": 4, "iq1c": 5, "q6_K": 6, "iq1s": 7}
ATYPE = {"q8_1": 0, "i8_token": 1}
OTYPE = {"f32": 0, "bf16": 1, "i32_partials": 2}


class MMQError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {status_string(code)} ({code})")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmmq.so (built in-tree by __graft_entry__.build()); raise if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built: run `python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    e = ctypes.c_int
    L.mmq_status_string.argtypes = [e]
    L.mmq_status_string.restype = ctypes.c_char_p
    L.mmq_act_bytes.argtypes = [e, I, I]
    L.mmq_act_bytes.restype = S
    L.mmq_act_region_offsets.argtypes = [e, I, I, ctypes.POINTER(S)]
    L.mmq_act_region_offsets.restype = e
    L.mmq_quantize_act.argtypes = [e, P, I, I, I, P, P]
    L.mmq_quantize_act.restype = e
    L.mmq_packed_bytes.argtypes = [e, I, I]
    L.mmq_packed_bytes.restype = S
    L.mmq_repack_weights.argtypes = [e, P, P, I, I, P, P]
    L.mmq_repack_weights.restype = e
    L.mmq_gemm.argtypes = [e, P, P, I, I, I, e, P, I, P]
    L.mmq_gemm.restype = e
    L.mmq_gemm_id_workspace_bytes.argtypes = [I, I, I]
    L.mmq_gemm_id_workspace_bytes.restype = S
    L.mmq_gemm_id.argtypes = [e, P, I, P, P, I, I, I, I, e, P, P, S, P]
    L.mmq_gemm_id.restype = e
    L.mmq_gemm_id_noalloc.argtypes = [e, P, I, P, P, I, I, I, I, e, P, P]
    L.mmq_gemm_id_noalloc.restype = e
    L.mmq_gemm_id_noalloc_max_workspace_bytes.argtypes = []
    L.mmq_gemm_id_noalloc_max_workspace_bytes.restype = S
    L.mmq_group_bytes.argtypes = [I, I, I]
    L.mmq_group_bytes.restype = S
    L.mmq_group_region_offsets.argtypes = [I, I, I, ctypes.POINTER(S)]
    L.mmq_group_region_offsets.restype = e
    L.mmq_group_rows.argtypes = [P, I, I, I, P, P]
    L.mmq_group_rows.restype = e
    L.mmq_moe_gather.argtypes = [e, P, I, P, I, I, I, I, P, I, P]
    L.mmq_moe_gather.restype = e
    L.mmq_moe_combine.argtypes = [e, P, I, e, P, P, I, I, I, I, P, I, P]
    L.mmq_moe_combine.restype = e
    L.mmq_moe_combine_grad.argtypes = [e, P, I, P, I, e, P, P, I, I, I, I, P, I, P, P]
    L.mmq_moe_combine_grad.restype = e
    L.mmq_lora_workspace_bytes.argtypes = [I, I, I, I, I]
    L.mmq_lora_workspace_bytes.restype = S
    L.mmq_lora.argtypes = [e, P, e, P, P, P, I, I, P, I, I, I, P, I, P, I, P, P, S, P]
    L.mmq_lora.restype = e
    L.mmq_lora_grad_workspace_bytes.argtypes = [I, I, I, I, I]
    L.mmq_lora_grad_workspace_bytes.restype = S
    L.mmq_lora_grad.argtypes = [e, P, e, P, P, P, I, I, P, I, I, I, P, P, I, P, I, P, I, P, P, P, S, P]
    L.mmq_lora_grad.restype = e
    L.mmq_cache_bytes.argtypes = [e, I, I, I, I]
    L.mmq_cache_bytes.restype = S
    L.mmq_cache_write.argtypes = [e, P, I, P, I, P, I, e, P, e, P, I, I, I, I, P]
    L.mmq_cache_write.restype = e
    L.mmq_cache_read.argtypes = [e, P, I, e, P, e, P, I, I, I, I, P, I, P, I, P]
    L.mmq_cache_read.restype = e
    L.mmq_cache_attn_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I]
    L.mmq_cache_attn_workspace_bytes.restype = S
    L.mmq_cache_attn.argtypes = [e, P, I, I, I, e, P, e, P, I, I, I, I, P, I, I, P, P, I, I, P, ctypes.c_float,
                                 P, I, P, S, P]
    L.mmq_cache_attn.restype = e
    _lib = L
    return L


def status_string(code: int) -> str:
    return lib().mmq_status_string(int(code)).decode()


def _check(fn: str, code: int):
    if code != MMQ_OK:
        raise MMQError(fn, code)


def _ptr(t) -> int | None:
    return None if t is None else int(t.data_ptr())


def _stream(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _wt(w) -> int:
    return WTYPE[w] if isinstance(w, str) else int(w)


def _at(a) -> int:
    return ATYPE[a] if isinstance(a, str) else int(a)


def _ot(o) -> int:
    return OTYPE[o] if isinstance(o, str) else int(o)


# -------------------------------------------------------------------------- sizes

def act_bytes(atype, M: int, K: int) -> int:
    return int(lib().mmq_act_bytes(_at(atype), M, K))


def act_region_offsets(atype, M: int, K: int) -> tuple[int, int, int, int, int]:
    arr = (ctypes.c_size_t * 5)()
    _check("mmq_act_region_offsets", lib().mmq_act_region_offsets(_at(atype), M, K, arr))
    return tuple(int(v) for v in arr)


def packed_bytes(wtype, N: int, K: int) -> int:
    return int(lib().mmq_packed_bytes(_wt(wtype), N, K))


def gemm_id_workspace_bytes(E: int, T: int, top_k: int) -> int:
    return int(lib().mmq_gemm_id_workspace_bytes(E, T, top_k))


# -------------------------------------------------------------------------- calls

def quantize_act(x, atype="q8_1", out=None, stream=None):
    """x: CUDA float32 [M, K] (row stride x.stride(0)); returns the act buffer (uint8)."""
    import torch
    assert x.is_cuda and x.dtype == torch.float32 and x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    nbytes = act_bytes(atype, M, K)
    if nbytes == 0:
        raise MMQError("mmq_act_bytes", MMQ_EINVAL)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    _check("mmq_quantize_act", lib().mmq_quantize_act(_at(atype), _ptr(x), M, K, x.stride(0),
                                                       _ptr(out), _stream(stream)))
    return out


def repack_weights(wtype, raw, N: int, K: int, row_scale=None, out=None, stream=None, grid=None):
    """raw: CUDA tensor holding the raw rows (uint8 bytes, or int8 [N,K] for i8_row).
    The repack's auxiliary input `aux` is row_scale (CUDA f32 [N]) for i8_row and grid (CUDA
    uint16/int16 [2048], the codebook) for iq1c and iq1s."""
    import torch
    nbytes = packed_bytes(wtype, N, K)
    if nbytes == 0:
        raise MMQError("mmq_packed_bytes", MMQ_EINVAL)
    if row_scale is not None and grid is not None:
        raise ValueError("pass row_scale (i8_row) or grid (iq1c, iq1s), not both")
    aux = row_scale if row_scale is not None else grid
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=raw.device)
    _check("mmq_repack_weights", lib().mmq_repack_weights(_wt(wtype), _ptr(raw), _ptr(aux), N, K,
                                                           _ptr(out), _stream(stream)))
    return out


def gemm(wtype, packed, act, M: int, N: int, K: int, otype="f32", out=None, ldo=None, stream=None):
    import torch
    o = _ot(otype)
    if out is None:
        if o == OTYPE["f32"]:
            out = torch.empty((M, N), dtype=torch.float32, device=packed.device)
        elif o == OTYPE["bf16"]:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=packed.device)
        else:
            w = _wt(wtype)
            shape = (M, N) if w == WTYPE["i8_row"] else (M, N, K // 16) if w == WTYPE["q6_K"] else (M, N, K // 32)
            out = torch.empty(shape, dtype=torch.int32, device=packed.device)
    if ldo is None:
        ldo = out.stride(0) if out.dim() == 2 else N
    _check("mmq_gemm", lib().mmq_gemm(_wt(wtype), _ptr(packed), _ptr(act), M, N, K, o, _ptr(out), ldo,
                                       _stream(stream)))
    return out


def gemm_id(wtype, packed, E: int, act, ids, T: int, top_k: int, N: int, K: int, out=None,
            workspace=None, stream=None):
    import torch
    if out is None:
        out = torch.empty((T, top_k, N), dtype=torch.float32, device=packed.device)
    ws = gemm_id_workspace_bytes(E, T, top_k)
    if workspace is None:
        workspace = torch.empty(max(ws, 16), dtype=torch.uint8, device=packed.device)
    _check("mmq_gemm_id", lib().mmq_gemm_id(_wt(wtype), _ptr(packed), E, _ptr(act), _ptr(ids), T, top_k, N, K,
                                             OTYPE["f32"], _ptr(out), _ptr(workspace), workspace.numel(),
                                             _stream(stream)))
    return out


def gemm_id_noalloc_max_workspace_bytes() -> int:
    return int(lib().mmq_gemm_id_noalloc_max_workspace_bytes())


def gemm_id_noalloc(wtype, packed, E: int, act, ids, T: int, top_k: int, N: int, K: int, out, stream=None):
    """mmq_gemm_id without a workspace argument: the library's static per-GPU scratch is used.
    `out` must be given (the call allocates nothing)."""
    _check("mmq_gemm_id_noalloc", lib().mmq_gemm_id_noalloc(_wt(wtype), _ptr(packed), E, _ptr(act), _ptr(ids), T,
                                                             top_k, N, K, OTYPE["f32"], _ptr(out), _stream(stream)))
    return out


# ------------------------------------------------------- rows grouped by adapter or expert

# A serving step makes these calls back to back, so the host's time per call counts: sizes that
# depend on (E, T, top_k) alone are looked up once, the checks read each tensor's shape once and
# build their messages only when they fail.

def _gpu(fn: str, *tensors) -> int:
    """The current GPU's index, on which every tensor (None skipped, not the first) has to be."""
    import torch
    at = tensors[0].get_device()
    if at >= 0 and at != torch._C._cuda_getDevice():
        at = -1
    for t in tensors:
        if t is not None and (at < 0 or t.get_device() != at):
            raise ValueError(f"{fn}: every tensor must be on the current GPU, got one on {t.device}")
    return at


def _raw_stream(stream, at: int) -> int:
    import torch
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(at)
    if stream.device_index != at:
        raise ValueError(f"the stream must be one of the current GPU ({at}), got one of GPU {stream.device_index}")
    return int(stream.cuda_stream)


def _scratch(fn: str, workspace) -> int:
    """The bytes of a caller's workspace."""
    if not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace must be contiguous, got strides {workspace.stride()}")
    return workspace.nbytes


def _ld(fn: str, name: str, t, rows: int, cols: int, dtype) -> int:
    """The row stride of a [rows, cols] tensor of `dtype` whose columns are contiguous."""
    if t.dtype is not dtype or t.shape != (rows, cols):
        raise ValueError(f"{fn}: {name} must be {dtype} {(rows, cols)}, got {t.dtype} {tuple(t.shape)}")
    ld, step = t.stride()
    if step != 1 and cols != 1:
        raise ValueError(f"{fn}: {name}'s columns must be contiguous, got strides {t.stride()}")
    return ld if rows > 1 else max(ld, cols)


def _flat(fn: str, name: str, t, shape, dtype):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be contiguous {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")


def _row_otype(fn: str, t) -> int:
    import torch
    if t.dtype is torch.float32:
        return 0
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{fn}: rows must be float32 or bfloat16, got {t.dtype}")
    return 1


def _plan_of(fn: str, plan, E: int, T: int, top_k: int):
    import torch
    nbytes = group_bytes(E, T, top_k)
    if nbytes == 0:
        raise MMQError("mmq_group_bytes", MMQ_EINVAL)
    if plan.dtype is not torch.uint8 or plan.numel() < nbytes or not plan.is_contiguous():
        raise ValueError(f"{fn}: plan must be the {nbytes} bytes that group_rows returns for E={E}, T={T}, top_k={top_k}")


def _new(like, shape, dtype, stream):
    """A tensor on `like`'s GPU for a call's result or workspace, from the memory of the call's own
    stream: what the current stream's earlier work still uses is not handed to another stream's
    call. shape None: of `like`'s shape."""
    import torch
    if stream is None:
        return torch.empty_like(like) if shape is None else like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return torch.empty_like(like) if shape is None else like.new_empty(shape, dtype=dtype)


def _zeros(like, stream):
    """As _new, of `like`'s shape and filled with zeros on the call's stream."""
    import torch
    if stream is None:
        return torch.zeros_like(like)
    with torch.cuda.stream(stream):
        return torch.zeros_like(like)


@functools.lru_cache(maxsize=4096)
def group_bytes(E: int, T: int, top_k: int) -> int:
    return int(lib().mmq_group_bytes(E, T, top_k))


@functools.lru_cache(maxsize=4096)
def group_region_offsets(E: int, T: int, top_k: int) -> tuple[int, int, int, int]:
    arr = (ctypes.c_size_t * 4)()
    _check("mmq_group_region_offsets", lib().mmq_group_region_offsets(E, T, top_k, arr))
    return tuple(int(v) for v in arr)


def group_rows(ids, E: int, out=None, stream=None):
    """Sort the pairs' ids (CUDA int32 [T, top_k], or [T] for one id a row) by group; returns the
    plan (uint8), shared by the calls on this batch."""
    import torch
    fn = "group_rows"
    at = _gpu(fn, ids, out)
    shape = ids.shape
    if ids.dtype is not torch.int32 or not 1 <= len(shape) <= 2 or not ids.is_contiguous():
        raise ValueError(f"{fn}: ids must be contiguous int32 [T] or [T, top_k], got {ids.dtype} {tuple(shape)}")
    T, top_k = shape[0], shape[1] if len(shape) == 2 else 1
    if out is None:
        nbytes = group_bytes(E, T, top_k)
        if nbytes == 0:
            raise MMQError("mmq_group_bytes", MMQ_EINVAL)
        out = _new(ids, nbytes, torch.uint8, stream)
    else:
        _plan_of(fn, out, E, T, top_k)
    _check("mmq_group_rows", lib().mmq_group_rows(ids.data_ptr(), E, T, top_k, out.data_ptr(), _raw_stream(stream, at)))
    return out


def group_views(plan, E: int, T: int, top_k: int = 1):
    """The plan's regions as int32 tensors sharing its memory: offs [E+1], order [P], pos [P],
    units [U, 4]."""
    import torch
    _plan_of("group_views", plan, E, T, top_k)
    P = T * top_k
    U = P // 64 + min(E + 1, P)
    _, order, pos, units = group_region_offsets(E, T, top_k)
    w = plan.view(torch.int32)
    return (w.as_strided((E + 1,), (1,)), w.as_strided((P,), (1,), w.storage_offset() + order // 4),
            w.as_strided((P,), (1,), w.storage_offset() + pos // 4),
            w.as_strided((U, 4), (4, 1), w.storage_offset() + units // 4))


def moe_gather(x, plan, E: int, top_k: int, out=None, stream=None):
    """Token rows x (CUDA float32 or bfloat16 [T, N]) in expert order: [T * top_k, N]. The rows past
    the last pair with an expert (from the plan's offs[E] on) are not written: in a tensor made here
    they hold whatever its memory held."""
    fn = "moe_gather"
    at = _gpu(fn, x, plan, out)
    o = _row_otype(fn, x)
    if x.dim() != 2:
        raise ValueError(f"{fn}: x must be [T, N], got {tuple(x.shape)}")
    T, N = x.shape
    _plan_of(fn, plan, E, T, top_k)
    if out is None:
        out = _new(x, (T * top_k, N), x.dtype, stream)
    ldx = _ld(fn, "x", x, T, N, x.dtype)
    ldr = _ld(fn, "out", out, T * top_k, N, x.dtype)
    _check("mmq_moe_gather", lib().mmq_moe_gather(o, x.data_ptr(), ldx, plan.data_ptr(), E, T, top_k, N,
                                                  out.data_ptr(), ldr, _raw_stream(stream, at)))
    return out


ROWORDER = {"pair": 0, "sorted": 1}


def _row_order(fn: str, order) -> int:
    r = ROWORDER.get(order)
    if r is None:
        raise ValueError(f"{fn}: order must be one of {list(ROWORDER)}, got {order!r}")
    return r


def _pair_rows(fn: str, z, P: int):
    """z [P, N], or [T, top_k, N] as gemm_id returns it, as [P, N]."""
    shape = z.shape
    if len(shape) == 3 and (shape[0] == 1 or shape[1] == 1 or z.stride(0) == shape[1] * z.stride(1)):
        z = z.view(shape[0] * shape[1], shape[2])
    if z.dim() != 2 or z.shape[0] != P:
        raise ValueError(f"{fn}: the pairs' rows must be [T * top_k, N], or [T, top_k, N] with one stride, and "
                         f"{P} pairs, got {tuple(shape)} with strides {z.stride()}")
    return z


def moe_combine(z, plan, E: int, T: int, top_k: int, weights=None, order="pair", out=None, stream=None):
    """The experts' rows z (CUDA float32 or bfloat16 [T * top_k, N], or [T, top_k, N] as gemm_id
    returns them) weighted and summed into tokens: [T, N]. weights: float32 [T, top_k] or None."""
    import torch
    fn = "moe_combine"
    at = _gpu(fn, z, plan, weights, out)
    o = _row_otype(fn, z)
    r = _row_order(fn, order)
    _plan_of(fn, plan, E, T, top_k)
    z = _pair_rows(fn, z, T * top_k)
    N = z.shape[1]
    ldz = _ld(fn, "z", z, T * top_k, N, z.dtype)
    if weights is not None:
        _flat(fn, "weights", weights, (T, top_k), torch.float32)
    if out is None:
        out = _new(z, (T, N), z.dtype, stream)
    ldy = _ld(fn, "out", out, T, N, z.dtype)
    _check("mmq_moe_combine", lib().mmq_moe_combine(o, z.data_ptr(), ldz, r, _ptr(weights),
                                                    plan.data_ptr(), E, T, top_k, N, out.data_ptr(), ldy,
                                                    _raw_stream(stream, at)))
    return out


def moe_combine_grad(dy, z, plan, E: int, top_k: int, weights, order="pair", dz=None, dw=None, stream=None):
    """Gradients of moe_combine for the rows and the weights: dz like z, dw float32 [T, top_k]. Rows of
    dz that no pair has (moe_combine does not read them) are zeros where dz is made here, and left as
    they are in a dz that is given, which saves the fill."""
    import torch
    fn = "moe_combine_grad"
    at = _gpu(fn, dy, z, plan, weights, dz, dw)
    o = _row_otype(fn, z)
    r = _row_order(fn, order)
    if dy.dim() != 2:
        raise ValueError(f"{fn}: dy must be [T, N], got {tuple(dy.shape)}")
    T, N = dy.shape
    P = T * top_k
    _plan_of(fn, plan, E, T, top_k)
    lddy = _ld(fn, "dy", dy, T, N, z.dtype)
    if dz is None:
        dz = _zeros(z, stream)
    if dw is None:
        dw = _new(weights, None, None, stream)
    z, rows = _pair_rows(fn, z, P), _pair_rows(fn, dz, P)
    ldz = _ld(fn, "z", z, P, N, z.dtype)
    lddz = _ld(fn, "dz", rows, P, N, z.dtype)
    _flat(fn, "weights", weights, (T, top_k), torch.float32)
    _flat(fn, "dw", dw, (T, top_k), torch.float32)
    _check("mmq_moe_combine_grad",
           lib().mmq_moe_combine_grad(o, dy.data_ptr(), lddy, z.data_ptr(), ldz, r, weights.data_ptr(),
                                      plan.data_ptr(), E, T, top_k, N, rows.data_ptr(), lddz, dw.data_ptr(),
                                      _raw_stream(stream, at)))
    return dz, dw


# ---------------------------------------------------- adapters beside a shared projection

ADTYPE = {"bf16": 0, "f16": 1}


@functools.lru_cache(maxsize=4096)
def lora_workspace_bytes(E: int, M: int, N: int, K: int, R: int) -> int:
    return int(lib().mmq_lora_workspace_bytes(E, M, N, K, R))


@functools.lru_cache(maxsize=4096)
def _act_need(atype: int, M: int, K: int) -> int:
    return int(lib().mmq_act_bytes(atype, M, K))


def _adapters(fn: str, act, A, B, scale, plan, M: int, at_: int):
    """Checks what both adapter calls read; returns (adapter type, E, R, K, N)."""
    import torch
    if A.dtype is torch.bfloat16:
        d = 0
    elif A.dtype is torch.float16:
        d = 1
    else:
        raise ValueError(f"{fn}: adapters must be bfloat16 or float16, got {A.dtype}")
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError(f"{fn}: A must be [E, R, K] and B [E, N, R], got {tuple(A.shape)} and {tuple(B.shape)}")
    E, R, K = A.shape
    N = B.shape[1]
    _flat(fn, "A", A, (E, R, K), A.dtype)
    _flat(fn, "B", B, (E, N, R), A.dtype)
    _flat(fn, "scale", scale, (E,), torch.float32)
    _plan_of(fn, plan, E, M, 1)
    need = _act_need(at_, M, K)
    if act.dtype is not torch.uint8 or act.numel() < max(need, 1) or not act.is_contiguous():
        raise ValueError(f"{fn}: act must be the {need} bytes that quantize_act returns for M={M}, K={K}")
    return d, E, R, K, N


def lora(act, A, B, scale, plan, M: int, atype="q8_1", base=None, out=None, v=None, workspace=None, stream=None):
    """Adds the rows' low-rank adapters to a projection's output: out = base + scale (x^ A^T) B^T,
    with A [E, R, K], B [E, N, R] (bfloat16 or float16), scale float32 [E] and the plan of the
    rows' adapters (group_rows of int32 [M]). base, out: [M, N] float32 (q8_1) or bfloat16
    (i8_token); out=base adds in place, base=None starts from zeros. Returns (out, v), v = x^ A^T
    float32 [M, R] being what lora_grad needs."""
    import torch
    fn = "lora"
    at = _gpu(fn, act, A, B, scale, plan, base, out, v, workspace)
    at_ = _at(atype)
    d, E, R, K, N = _adapters(fn, act, A, B, scale, plan, M, at_)
    dt = torch.float32 if at_ == 0 else torch.bfloat16
    if out is None:
        out = _new(act, (M, N), dt, stream) if base is None else _new(base, None, None, stream)
    if v is None:
        v = _new(scale, (M, R), torch.float32, stream)
    else:
        _flat(fn, "v", v, (M, R), torch.float32)
    if workspace is None:
        nbytes = lora_workspace_bytes(E, M, N, K, R)
        if nbytes:
            workspace = _new(act, nbytes, torch.uint8, stream)
    ldb = _ld(fn, "base", base, M, N, dt) if base is not None else 0
    ldo = _ld(fn, "out", out, M, N, dt)
    _check("mmq_lora", lib().mmq_lora(at_, act.data_ptr(), d, A.data_ptr(), B.data_ptr(), scale.data_ptr(), E, R,
                                      plan.data_ptr(), M, N, K, _ptr(base), ldb, out.data_ptr(), ldo, v.data_ptr(),
                                      _ptr(workspace), 0 if workspace is None else _scratch(fn, workspace),
                                      _raw_stream(stream, at)))
    return out, v


@functools.lru_cache(maxsize=4096)
def lora_grad_workspace_bytes(E: int, M: int, N: int, K: int, R: int) -> int:
    return int(lib().mmq_lora_grad_workspace_bytes(E, M, N, K, R))


def lora_grad(act, A, B, scale, plan, v, dy, atype="q8_1", dx_base=None, dx=None, dA=None, dB=None,
              want_dx: bool = True, workspace=None, stream=None):
    """Gradients of lora from its 8-bit activations: dy [M, N] float32 (q8_1) or bfloat16
    (i8_token), v as lora returned it, the other inputs as given to it. Returns (dx, dA, dB) in
    float32: dx [M, K] = dx_base + the adapters' part (dx=dx_base adds in place; with want_dx=False
    None, and a dx that is given is left as it is), dA and dB like A and B."""
    import torch
    fn = "lora_grad"
    at = _gpu(fn, act, A, B, scale, plan, v, dy, dx_base, dx, dA, dB, workspace)
    at_ = _at(atype)
    if dy.dim() != 2:
        raise ValueError(f"{fn}: dy must be [M, N], got {tuple(dy.shape)}")
    M = dy.shape[0]
    d, E, R, K, N = _adapters(fn, act, A, B, scale, plan, M, at_)
    f32 = torch.float32
    lddy = _ld(fn, "dy", dy, M, N, f32 if at_ == 0 else torch.bfloat16)
    _flat(fn, "v", v, (M, R), f32)
    if not want_dx:
        dx = None
    elif dx is None:
        dx = _new(scale, (M, K), f32, stream)
    if dA is None:
        dA = _new(scale, (E, R, K), f32, stream)
    else:
        _flat(fn, "dA", dA, (E, R, K), f32)
    if dB is None:
        dB = _new(scale, (E, N, R), f32, stream)
    else:
        _flat(fn, "dB", dB, (E, N, R), f32)
    lddx = _ld(fn, "dx", dx, M, K, f32) if dx is not None else 0
    ldxb = _ld(fn, "dx_base", dx_base, M, K, f32) if dx_base is not None else 0
    if workspace is None:
        workspace = _new(act, lora_grad_workspace_bytes(E, M, N, K, R), torch.uint8, stream)
    _check("mmq_lora_grad",
           lib().mmq_lora_grad(at_, act.data_ptr(), d, A.data_ptr(), B.data_ptr(), scale.data_ptr(), E, R,
                               plan.data_ptr(), M, N, K, v.data_ptr(), dy.data_ptr(), lddy, _ptr(dx_base), ldxb,
                               _ptr(dx), lddx, dA.data_ptr(), dB.data_ptr(), workspace.data_ptr(), _scratch(fn, workspace),
                               _raw_stream(stream, at)))
    return dx, dA, dB


# ------------------------------------------------------- the quantised key/value cache

CACHE_BLOCK = {"q8_0": 34, "q4_0": 18}      # bytes of 32 values


def cache_bytes(ctype, pages: int, page: int, heads: int, D: int) -> int:
    return int(lib().mmq_cache_bytes(_wt(ctype), pages, page, heads, D))


def cache_shape(ctype, pages: int, page: int, heads: int, D: int) -> tuple[int, int, int, int]:
    """The shape of a cache of keys or of values as a uint8 tensor: [pages, heads, page / 32, bytes of
    a record of 32 tokens], as the calls below take it. Allocated by the caller; nothing needs to be
    filled in."""
    nbytes = cache_bytes(ctype, pages, page, heads, D)
    if nbytes == 0:
        raise MMQError("mmq_cache_bytes", MMQ_EINVAL)
    return pages, heads, page // 32, nbytes // (pages * heads * (page // 32))


@functools.lru_cache(maxsize=256)
def _cache_dims(kshape, vshape, ktype, vtype):
    """(key type, value type, pages, page, heads, D) of caches of these shapes, None if they are not two of one size."""
    if len(kshape) != 4 or len(vshape) != 4:
        return None
    pages, heads, tiles, rec = kshape
    D = rec // CACHE_BLOCK[ktype]
    if heads == 0 or D == 0 or rec != D * CACHE_BLOCK[ktype] or vshape != (pages, heads, tiles, D * CACHE_BLOCK[vtype]):
        return None
    return WTYPE[ktype], WTYPE[vtype], pages, 32 * tiles, heads, D


def _caches(fn: str, kcache, vcache, ktype, vtype):
    """(key type, value type, pages, page, heads, D) of two caches."""
    import torch
    for name, t in (("ktype", ktype), ("vtype", vtype)):
        if t not in CACHE_BLOCK:
            raise ValueError(f"{fn}: {name} must be one of {list(CACHE_BLOCK)}, got {t!r}")
    dims = _cache_dims(kcache.shape, vcache.shape, ktype, vtype)
    if dims is None or kcache.dtype is not torch.uint8 or vcache.dtype is not torch.uint8 or not kcache.is_contiguous() or \
            not vcache.is_contiguous():
        raise ValueError(f"{fn}: kcache and vcache must be contiguous uint8 of cache_shape's shape with heads of one size, got "
                         f"{kcache.dtype} {tuple(kcache.shape)} of {ktype} and {vcache.dtype} {tuple(vcache.shape)} of {vtype}")
    return dims


def _heads_ld(fn: str, name: str, t, heads: int, D: int, dtype) -> tuple[int, int]:
    """(rows, row stride) of a [rows, heads, D] or [rows, heads * D] tensor whose heads lie one after another."""
    shape, strides = t.shape, t.stride()
    if t.dtype is not dtype or (shape[1:] != (heads, D) and shape[1:] != (heads * D,)):
        raise ValueError(f"{fn}: {name} must be {dtype} [rows, {heads}, {D}] or [rows, {heads * D}], got {t.dtype} {tuple(shape)}")
    if strides[-1] != 1 or (len(shape) == 3 and heads != 1 and strides[1] != D):
        raise ValueError(f"{fn}: {name}'s heads must lie one after another, got strides {strides}")
    return shape[0], strides[0] if shape[0] > 1 else max(strides[0], heads * D)


def cache_write(k, v, slots, kcache, vcache, ktype="q8_0", vtype="q8_0", stream=None):
    """Quantises rows of keys and values (CUDA float32 or bfloat16 [rows, heads, D] or [rows, heads * D],
    any row stride: a projection's output as it is) into the caches' slots (int32 [rows]: page * tokens
    of a page + place). Rows whose slot is -1, or outside the caches, are not written."""
    import torch
    fn = "cache_write"
    at = _gpu(fn, k, v, slots, kcache, vcache)
    tk, tv, pages, page, heads, D = _caches(fn, kcache, vcache, ktype, vtype)
    o = _row_otype(fn, k)
    rows, ldk = _heads_ld(fn, "k", k, heads, D, k.dtype)
    vrows, ldv = _heads_ld(fn, "v", v, heads, D, k.dtype)
    if vrows != rows:
        raise ValueError(f"{fn}: k and v must have as many rows, got {rows} and {vrows}")
    _flat(fn, "slots", slots, (rows,), torch.int32)
    _check("mmq_cache_write", lib().mmq_cache_write(o, k.data_ptr(), ldk, v.data_ptr(), ldv, slots.data_ptr(), rows, tk,
                                                    kcache.data_ptr(), tv, vcache.data_ptr(), pages, page, heads, D,
                                                    _raw_stream(stream, at)))


def cache_read(slots, kcache, vcache, ktype="q8_0", vtype="q8_0", dtype=None, k=None, v=None, stream=None):
    """The rows at slots (CUDA int32 [rows]) as values: (k, v), [rows, heads, D] in `dtype` (float32, or
    bfloat16). Rows whose slot is outside the caches are not written: in tensors made here they hold
    whatever their memory held. k, v: given together, they name the type."""
    import torch
    fn = "cache_read"
    at = _gpu(fn, slots, kcache, vcache, k, v)
    tk, tv, pages, page, heads, D = _caches(fn, kcache, vcache, ktype, vtype)
    if slots.dim() != 1:
        raise ValueError(f"{fn}: slots must be [rows], got {tuple(slots.shape)}")
    rows = slots.shape[0]
    _flat(fn, "slots", slots, (rows,), torch.int32)
    if (k is None) != (v is None) or (k is not None and dtype not in (None, k.dtype)):
        raise ValueError(f"{fn}: give k and v together, and no other dtype than theirs")
    if k is None:
        dtype = torch.float32 if dtype is None else dtype
        k = _new(slots, (rows, heads, D), dtype, stream)
        v = _new(slots, (rows, heads, D), dtype, stream)
    o = _row_otype(fn, k)
    krows, ldk = _heads_ld(fn, "k", k, heads, D, k.dtype)
    vrows, ldv = _heads_ld(fn, "v", v, heads, D, k.dtype)
    if krows != rows or vrows != rows:
        raise ValueError(f"{fn}: k and v must have a row for each of the {rows} slots, got {krows} and {vrows}")
    _check("mmq_cache_read", lib().mmq_cache_read(o, slots.data_ptr(), rows, tk, kcache.data_ptr(), tv, vcache.data_ptr(),
                                                  pages, page, heads, D, k.data_ptr(), ldk, v.data_ptr(), ldv,
                                                  _raw_stream(stream, at)))
    return k, v


@functools.lru_cache(maxsize=4096)
def cache_attn_workspace_bytes(rows: int, heads_q: int, page: int, heads: int, D: int, width: int, B: int, max_q: int) -> int:
    return int(lib().mmq_cache_attn_workspace_bytes(rows, heads_q, page, heads, D, width, B, max_q))


def cache_attn(q, kcache, vcache, table, lens, starts, max_q: int, ktype="q8_0", vtype="q8_0", mask=None, scale=None,
               out=None, workspace=None, stream=None):
    """Attention of the sequences' newest tokens over the cache: q (CUDA float32 or bfloat16 [rows, heads_q, D]
    or [rows, heads_q * D], any row stride), table int32 [B, width] of pages (columns contiguous), lens int32
    [B], starts int32 [B + 1]: sequence b's new tokens are its last ones, rows starts[b] .. starts[b + 1] - 1,
    at most max_q. A new token sees the tokens before the new ones and, of the new ones, those up to itself
    (mask None), or those whose bit its word of mask (int64 or uint64 [rows], bit j: new token j) has.
    scale: D ** -0.5 if None. Returns out, like q; rows of no sequence are not written."""
    import torch
    fn = "cache_attn"
    at = _gpu(fn, q, kcache, vcache, table, lens, starts, mask, out, workspace)
    tk, tv, pages, page, heads, D = _caches(fn, kcache, vcache, ktype, vtype)
    o = _row_otype(fn, q)
    rows = q.shape[0] if q.dim() else 0
    heads_q = q.shape[1] if q.dim() == 3 else q.shape[1] // D if q.dim() == 2 else 0
    if heads_q == 0 or heads_q % heads:
        raise ValueError(f"{fn}: q must have a multiple of {heads} heads of {D} values, got {tuple(q.shape)}")
    rows, ldq = _heads_ld(fn, "q", q, heads_q, D, q.dtype)
    if lens.dim() != 1 or table.dim() != 2:
        raise ValueError(f"{fn}: table must be [B, width] and lens [B], got {tuple(table.shape)} and {tuple(lens.shape)}")
    B, width = lens.shape[0], table.shape[1]
    ldt = _ld(fn, "table", table, B, width, torch.int32)
    _flat(fn, "lens", lens, (B,), torch.int32)
    _flat(fn, "starts", starts, (B + 1,), torch.int32)
    if mask is not None and (mask.dtype not in (torch.int64, torch.uint64) or mask.shape != (rows,) or not mask.is_contiguous()):
        raise ValueError(f"{fn}: mask must be contiguous int64 or uint64 [{rows}], got {mask.dtype} {tuple(mask.shape)}")
    if out is None:
        out = _new(q, tuple(q.shape), q.dtype, stream)
    orows, ldo = _heads_ld(fn, "out", out, heads_q, D, q.dtype)
    if orows != rows:
        raise ValueError(f"{fn}: out must have {rows} rows, got {orows}")
    if workspace is None:
        nbytes = cache_attn_workspace_bytes(rows, heads_q, page, heads, D, width, B, max_q)
        if nbytes:
            workspace = _new(kcache, nbytes, torch.uint8, stream)
    _check("mmq_cache_attn",
           lib().mmq_cache_attn(o, q.data_ptr(), ldq, rows, heads_q, tk, kcache.data_ptr(), tv, vcache.data_ptr(), pages,
                                page, heads, D, table.data_ptr(), ldt, width, lens.data_ptr(), starts.data_ptr(), B, max_q,
                                _ptr(mask), D ** -0.5 if scale is None else scale, out.data_ptr(), ldo, _ptr(workspace),
                                0 if workspace is None else _scratch(fn, workspace), _raw_stream(stream, at)))
    return out


# -------------------------------------------------------------------------- host helpers

def _act_dims(M: int, K: int):
    Mp = (M + 31) // 32 * 32
    KB = K // 32
    KBp = (KB + 7) // 8 * 8
    return Mp, KB, KBp, Mp // 32


def _act_regions(act_bytes_host: np.ndarray, M: int, K: int):
    """All four q8_1 regions, padding included, as row-major arrays: xq int8 [Mp, KBp*32],
    xs2 uint32 [Mp, KBp], xsx f32 [Mp, KBp], xg uint32 [Mp, KBp, 2] (the dword of half h of each
    block; all stored tiled, transposed back here)."""
    o = act_region_offsets("q8_1", M, K)
    Mp, KB, KBp, MT = _act_dims(M, K)
    buf = np.asarray(act_bytes_host, dtype=np.uint8)
    t = buf[o[0]:o[0] + MT * KBp * 1024].view(np.int8).reshape(MT, KBp, 2, 32, 16)   # [mt, b, h, r, 16]
    xq = t.transpose(0, 3, 1, 2, 4).reshape(Mp, KBp * 32)
    cells = Mp * KBp
    def tile_major(region, dt):
        return buf[region:region + 4 * cells].view(dt).reshape(MT, KBp, 32).transpose(0, 2, 1).reshape(Mp, KBp)
    xs2 = tile_major(o[1], np.uint32)
    xsx = tile_major(o[2], np.float32)
    xg = buf[o[3]:o[3] + 8 * cells].view(np.uint32).reshape(MT, KBp, 2, 32).transpose(0, 3, 1, 2).reshape(Mp, KBp, 2)
    return xq, xs2, xsx, xg


def _half_bits(v):
    return np.asarray(v, np.uint32).astype(np.uint16).view(np.float16).astype(np.float32)


def act_groups_host(act_bytes_host: np.ndarray, M: int, K: int):
    """Region 3 decoded: the integer 8-value group sums G as int32 [Mp, KBp, 4], padding
    included (G_j * 2^-13 is stored as f16, so G_j = f16 value * 2^13 exactly)."""
    _, _, _, xg = _act_regions(act_bytes_host, M, K)
    g = np.stack([_half_bits(xg & 0xFFFF), _half_bits(xg >> 16)], axis=-1).reshape(xg.shape[0], xg.shape[1], 4)
    return (g.astype(np.float64) * 8192.0).astype(np.int32)


def act_to_host(act_bytes_host: np.ndarray, M: int, K: int):
    """Decode a q8_1 act buffer (copied to host as uint8) into plain row-major
    (xq int8 [M,K], xs f32 [M,K/32], xsum int32 [M,K/32]) following the documented layout:
    xs is the low f16 half of region 1, xsum the sum of the four group sums of region 3."""
    xq, xs2, _, _ = _act_regions(act_bytes_host, M, K)
    KB = K // 32
    xs = _half_bits(xs2 & 0xFFFF)
    xsum = act_groups_host(act_bytes_host, M, K).sum(axis=2).astype(np.int32)
    return (np.ascontiguousarray(xq[:M, :K]), np.ascontiguousarray(xs[:M, :KB]),
            np.ascontiguousarray(xsum[:M, :KB]))


def act_derived_host(act_bytes_host: np.ndarray, M: int, K: int):
    """Regions 1 and 2 decoded to f32 [Mp, KBp] each (padding included): the low and high f16
    halves of xs2, and xsx. They must equal xs, xs and xs * xsum exactly."""
    _, xs2, xsx, _ = _act_regions(act_bytes_host, M, K)
    return _half_bits(xs2 & 0xFFFF), _half_bits(xs2 >> 16), xsx.copy()


def act_padding_host(act_bytes_host: np.ndarray, M: int, K: int):
    """The padded rows (m >= M) and padded blocks (b >= K/32) of every region of a q8_1 act
    buffer, as one flat array that must be all zero."""
    xq, xs2, xsx, xg = _act_regions(act_bytes_host, M, K)
    KB = K // 32
    pads = [xq[M:].ravel(), xq[:, K:].ravel()]
    for r in (xs2, xsx, xg):
        pads += [r[M:].ravel(), r[:, KB:].ravel()]
    return np.concatenate([p.astype(np.float64) for p in pads])


def act_q8_1_pack_host(xq: np.ndarray, xs: np.ndarray) -> np.ndarray:
    """Encode q8_1 activations (xq int8 [M, K], xs f32 [M, K/32], the f16-exact block scales)
    into the documented MMQ_ACT_Q8_1 layout (uint8 buffer of act_bytes("q8_1", M, K) bytes);
    xsum and the group sums are taken from xq."""
    xq = np.asarray(xq, dtype=np.int8)
    M, K = xq.shape
    o = act_region_offsets("q8_1", M, K)
    Mp, KB, KBp, MT = _act_dims(M, K)
    buf = np.zeros(act_bytes("q8_1", M, K), np.uint8)
    full = np.zeros((Mp, KBp * 32), np.int8)
    full[:M, :K] = xq
    buf[o[0]:o[0] + MT * KBp * 1024] = full.reshape(MT, 32, KBp, 2, 16).transpose(0, 2, 3, 1, 4).reshape(-1).view(np.uint8)
    g = full.reshape(Mp, KBp, 4, 8).astype(np.int64).sum(axis=3)                      # [Mp, KBp, 4]
    s = np.zeros((Mp, KBp), np.float32)
    s[:M, :KB] = xs
    h = s.astype(np.float16).view(np.uint16).astype(np.uint32)
    def tm(a):
        return a.reshape(MT, 32, KBp).transpose(0, 2, 1).reshape(-1)
    buf[o[1]:o[1] + 4 * Mp * KBp] = tm(h | (h << 16)).view(np.uint8)
    buf[o[2]:o[2] + 4 * Mp * KBp] = tm((s * g.sum(axis=2).astype(np.float32)).astype(np.float32)).view(np.uint8)
    gh = (g.astype(np.float32) * np.float32(2.0 ** -13)).astype(np.float16).view(np.uint16).astype(np.uint32)
    pair = gh[..., 0::2] | (gh[..., 1::2] << 16)                                      # [Mp, KBp, 2 halves]
    buf[o[3]:o[3] + 8 * Mp * KBp] = pair.reshape(MT, 32, KBp, 2).transpose(0, 2, 3, 1).reshape(-1).view(np.uint8)
    return buf


def act_i8_pack_host(a: np.ndarray, sa: np.ndarray) -> np.ndarray:
    """Encode int8 activations a [M, K] and per-token scales sa [M] into the documented
    MMQ_ACT_I8_TOKEN layout (uint8 buffer of act_bytes("i8_token", M, K) bytes)."""
    a = np.asarray(a, dtype=np.int8)
    M, K = a.shape
    o = act_region_offsets("i8_token", M, K)
    Mp, KB, KBp, MT = _act_dims(M, K)
    buf = np.zeros(act_bytes("i8_token", M, K), np.uint8)
    full = np.zeros((Mp, KBp * 32), np.int8)
    full[:M, :K] = a
    t = full.reshape(MT, 32, KBp, 2, 16).transpose(0, 2, 3, 1, 4)          # [mt, b, h, r, 16]
    buf[o[0]:o[0] + MT * KBp * 1024] = t.reshape(-1).view(np.uint8)
    sp = np.zeros(Mp, np.float32)
    sp[:M] = np.asarray(sa, dtype=np.float32)
    buf[o[1]:o[1] + 4 * Mp] = sp.view(np.uint8)
    return buf


def act_i8_to_host(act_bytes_host: np.ndarray, M: int, K: int, padded: bool = False):
    """Decode an MMQ_ACT_I8_TOKEN buffer (copied to host as uint8) into (a int8 [M, K],
    sa f32 [M]), or with padded=True into ([Mp, KBp*32], [Mp]) including the zero padding."""
    o = act_region_offsets("i8_token", M, K)
    Mp, KB, KBp, MT = _act_dims(M, K)
    buf = np.asarray(act_bytes_host, dtype=np.uint8)
    t = buf[o[0]:o[0] + MT * KBp * 1024].view(np.int8).reshape(MT, KBp, 2, 32, 16)
    full = t.transpose(0, 3, 1, 2, 4).reshape(Mp, KBp * 32)
    sa = buf[o[1]:o[1] + 4 * Mp].view(np.float32)
    if padded:
        return full.copy(), sa.copy()
    return np.ascontiguousarray(full[:M, :K]), sa[:M].copy()
