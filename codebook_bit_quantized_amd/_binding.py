"""ctypes binding of libcbq.so.

Argument marshalling only: every step of the path runs in the library's HIP kernels.
torch supplies device memory (output tensors are allocated here with torch) and the
current HIP stream.  There is no CPU or Python fallback: if the library is missing or
the GPU is absent, the calls raise.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import List, Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libcbq.so")

CBQ_OK, CBQ_EINVAL, CBQ_EUNSUPPORTED, CBQ_EWORKSPACE, CBQ_EHIP = 0, -1, -2, -3, -4
EPI_F32, EPI_SWIGLU_BF16 = 0, 1
PATH_AUTO, PATH_LUT, PATH_MFMA = 0, 1, 2
PATH_PAGES_PRODUCTS, PATH_PAGES_BUCKETS = 3, 4   # the table forms (4-bit, A4; never chosen by AUTO)
PATH_REG_TABLES = 0x10   # flags: where 2-/3-bit codebooks are looked up (default: per path)
PATH_LDS_TABLES = 0x20
AUTO_MAX_LUT_ROWS = 32
FEW_MAX_TOKENS = 32

# every symbol include/cbq.h declares
EXPORTED = ("cbq_rotate_quantize", "cbq_rotate_quantize_ex", "cbq_rotate_dense_workspace",
            "cbq_rotate_quantize_dense", "cbq_route_workspace", "cbq_moe_route_gather",
            "cbq_moe_route_gather_noalloc", "cbq_prepack_bytes", "cbq_prepack_weights",
            "cbq_gemm_workspace", "cbq_codebook_lut_gemm", "cbq_moe_combine",
            "cbq_kmeans_codebooks", "cbq_refit_codebooks", "cbq_cpu_lut_gemm", "cbq_status_string", "cbq_last_error",
            "cbq_version", "cbq_norm_rotate_quantize", "cbq_combine_norm_residual", "cbq_moe_few_workspace",
            "cbq_moe_ffn_few", "cbq_adapter_workspace", "cbq_codebook_adapter_gemm")


class CbqError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


LAYOUT_ROWS, LAYOUT_BLOCKED = 0, 1


class cbq_weights(ctypes.Structure):
    _fields_ = [("idx", ctypes.c_void_p), ("codebook", ctypes.c_void_p), ("E", ctypes.c_int32),
                ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("layout", ctypes.c_int32)]


TYPE_F32, TYPE_BF16 = 0, 1


class cbq_norm(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("eps", ctypes.c_float), ("had_block", ctypes.c_int32),
                ("act_bits", ctypes.c_int32), ("normed", ctypes.c_void_p), ("ldn", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libcbq.so (built in-tree by codebook_bit_quantized_amd.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libcbq.so not found at {path}; build it with "
                          "`python -m codebook_bit_quantized_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    W = ctypes.POINTER(cbq_weights)
    f32, Nrm = ctypes.c_float, ctypes.POINTER(cbq_norm)
    sig = {
        "cbq_rotate_quantize": (ctypes.c_int, [vp, i64, i32, i64, i32, i32, vp, vp, vp, vp]),
        "cbq_rotate_quantize_ex": (ctypes.c_int, [vp, i64, i32, i64, i32, i32, vp, vp, vp, vp, vp,
                                                  vp]),
        "cbq_rotate_dense_workspace": (sz, [i64, i32]),
        "cbq_rotate_quantize_dense": (ctypes.c_int, [vp, i64, i32, i64, vp, i32, vp, vp, vp, vp, sz,
                                                     vp]),
        "cbq_route_workspace": (sz, [i64, i32, i32, i32]),
        "cbq_moe_route_gather": (ctypes.c_int, [vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp,
                                                vp, sz, vp]),
        "cbq_moe_route_gather_noalloc": (ctypes.c_int, [vp, i64, i32, i32, i32, i32, vp, vp, vp,
                                                        vp, vp, vp]),
        "cbq_prepack_bytes": (sz, [W]),
        "cbq_prepack_weights": (ctypes.c_int, [W, vp, vp]),
        "cbq_gemm_workspace": (sz, [W, i32, i64, i32, i32]),
        "cbq_codebook_lut_gemm": (ctypes.c_int, [vp, vp, i32, i64, vp, vp, W, i32, i32, i32, vp,
                                                 i64, vp, sz, vp]),
        "cbq_moe_combine": (ctypes.c_int, [vp, vp, vp, i64, i32, i32, i32, vp, vp]),
        "cbq_kmeans_codebooks": (ctypes.c_int, [vp, i64, i32, i64, i32, i32, vp, vp, vp, vp]),
        "cbq_refit_codebooks": (ctypes.c_int, [vp, i64, i32, i64, i32, vp, vp, i32, i64, vp, vp]),
        "cbq_cpu_lut_gemm": (ctypes.c_int, [vp, vp, i32, i64, W, vp, i64, i32, i32]),
        "cbq_norm_rotate_quantize": (ctypes.c_int, [vp, i64, i32, i64, Nrm, vp]),
        "cbq_combine_norm_residual": (ctypes.c_int, [vp, i32, i64, vp, vp, i64, i32, i32, i32, vp, f32, vp, i64,
                                                     f32, vp, i64, vp, i64, Nrm, vp]),
        "cbq_moe_few_workspace": (sz, [i64, i32, i32, i32, i32, i32]),
        "cbq_moe_ffn_few": (ctypes.c_int, [vp, vp, i32, vp, i64, i32, i32, i32, i32, W, W, W, vp, i32, i64, vp, sz, vp]),
        "cbq_adapter_workspace": (sz, [i64, i32]),
        "cbq_codebook_adapter_gemm": (ctypes.c_int, [vp, vp, i32, i64, W, vp, i64, vp, vp, vp, i32, i32, vp, vp, i64, vp,
                                                     sz, vp]),
        "cbq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "cbq_last_error": (ctypes.c_char_p, []),
        "cbq_version": (ctypes.c_int, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _opt_ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check(status: int):
    if status != CBQ_OK:
        lib = load_library()
        raise CbqError(status, f"{lib.cbq_status_string(status).decode()}: "
                               f"{lib.cbq_last_error().decode()}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _require_gpu(*ts: Optional[torch.Tensor]):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("cbq operates on device tensors only")


# handle of a device's current stream: torch's own accessor where it has one (the public
# torch.cuda.current_stream() builds an object, 3 us of a call that takes 15)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on_stream(dev: torch.device, stream, call):
    """call(stream handle) with `dev` current and what it allocates belonging to the stream it
    launches on: the given one, or dev's current one."""
    if stream is None and dev.index == torch.cuda.current_device():
        return call(_raw_stream(dev.index))
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    if not hasattr(st, "cuda_stream"):
        st = torch.cuda.ExternalStream(int(st), device=dev)
    if st.device != dev:
        raise ValueError(f"the stream is on {st.device}, the tensors are on {dev}")
    with torch.cuda.device(dev), torch.cuda.stream(st):
        return call(st.cuda_stream)


def _tensor(name: str, t: Optional[torch.Tensor], dev: torch.device, dtype, shape=None,
            rows: bool = False, contiguous: bool = False):
    """Checks an argument tensor's place, type, shape and layout; None passes.  rows: unit
    stride along the last dimension."""
    if t is None or (t.dtype is dtype and t.device == dev and (shape is None or t.shape == shape)
                     and t.is_contiguous()):
        return
    if t.device != dev:
        raise ValueError(f"{name} must be on the same GPU as the other tensors (got {t.device}, {dev})")
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if rows and t.numel() > 0 and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _row_stride(t: torch.Tensor) -> int:
    """Elements between rows of a [T][K] tensor (its width where there is at most one row,
    whose stride torch leaves open)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 8 * ((t.shape[1] + 7) // 8))


_CODEBOOK_TYPES = (torch.int16, torch.float16, torch.uint16)


@dataclass
class CodebookWeights:
    """One weight matrix type for E experts: packed indices and fp16 codebooks (device).
    idx is [E][N][K*bits/8] in the row layout, or the blocked layout's bytes as
    [E][N][Kp*bits/8] (Kp = K rounded up to 128) after prepack_weights."""
    idx: torch.Tensor        # uint8 [E][N][row bytes]
    codebook: torch.Tensor   # int16/uint16/float16 [E][N][2^bits]
    K: int
    bits: int
    layout: int = LAYOUT_ROWS

    @property
    def E(self) -> int:
        return self.idx.shape[0]

    @property
    def N(self) -> int:
        return self.idx.shape[1]

    def _c_checked(self, dev: torch.device, name: str) -> cbq_weights:
        """c_struct() of tensors that are as it describes them: on dev, packed, of these sizes."""
        idx, cb, K, bits = self.idx, self.codebook, self.K, self.bits
        kp = K if self.layout == LAYOUT_ROWS else (K + 127) // 128 * 128
        if idx.dim() != 3:
            raise ValueError(f"{name}.idx must have three dimensions (got shape {tuple(idx.shape)})")
        E, N, _ = idx.shape
        _tensor(name + ".idx", idx, dev, torch.uint8, (E, N, kp * bits // 8), contiguous=True)
        if cb.dtype not in _CODEBOOK_TYPES:
            raise ValueError(f"{name}.codebook must hold fp16 patterns as float16, int16 or uint16 (got {cb.dtype})")
        _tensor(name + ".codebook", cb, dev, cb.dtype, (E, N, 1 << bits), contiguous=True)
        return cbq_weights(idx.data_ptr(), cb.data_ptr(), E, N, K, bits, self.layout)

    def c_struct(self) -> cbq_weights:
        return cbq_weights(self.idx.data_ptr(), self.codebook.data_ptr(), self.E, self.N, self.K,
                           self.bits, self.layout)


# ---------------------------------------------------------------------------
def rotate_quantize(x: torch.Tensor, act_bits: int = 4, had_block: int = 0,
                    codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                    precond: Optional[torch.Tensor] = None, smooth: Optional[torch.Tensor] = None,
                    signs: Optional[torch.Tensor] = None, stream=None):
    """x: bf16 (or int16 bit patterns) [T][K] on the GPU -> (codes uint8, scales fp32).

    smooth (fp32 [K]) and signs (uint8 [K/8] bitmask) select cbq_rotate_quantize_ex."""
    lib = load_library()
    _require_gpu(x, smooth, signs)
    T, K = x.shape
    ldx = x.stride(0)
    if x.stride(1) != 1:
        raise ValueError("x must have unit stride along channels")
    if codes is None:
        codes = torch.empty((T, K * act_bits // 8), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((T,), dtype=torch.float32, device=x.device)
    if smooth is None and signs is None:
        _check(lib.cbq_rotate_quantize(_ptr(x), T, K, ldx, had_block, act_bits, _ptr(codes),
                                       _ptr(scales), _ptr(precond), _stream(stream)))
    else:
        _check(lib.cbq_rotate_quantize_ex(_ptr(x), T, K, ldx, had_block, act_bits, _ptr(smooth),
                                          _ptr(signs), _ptr(codes), _ptr(scales), _ptr(precond),
                                          _stream(stream)))
    return codes, scales


def rotate_dense_workspace(T: int, K: int) -> int:
    """Bytes of device workspace rotate_quantize_dense needs (cbq_rotate_dense_workspace)."""
    return int(load_library().cbq_rotate_dense_workspace(T, K))


def rotate_quantize_dense(x: torch.Tensor, R: torch.Tensor, act_bits: int = 4,
                          codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                          precond: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                          stream=None):
    """x: bf16 [T][K], R: bf16 [K][K] (u = R x per token) on the GPU -> (codes, scales).

    ws: optional uint8 device workspace of rotate_dense_workspace(T, K) bytes."""
    lib = load_library()
    _require_gpu(x, R, ws)
    T, K = x.shape
    if (T > 0 and x.stride(1) != 1) or not R.is_contiguous() or tuple(R.shape) != (K, K):
        raise ValueError("x needs unit channel stride and R must be a contiguous [K][K] tensor")
    if codes is None:
        codes = torch.empty((T, K * act_bits // 8), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((T,), dtype=torch.float32, device=x.device)
    need = int(lib.cbq_rotate_dense_workspace(T, K))
    if ws is None and T > 0:
        ws = torch.empty((need,), dtype=torch.uint8, device=x.device)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.cbq_rotate_quantize_dense(_ptr(x), T, K, max(x.stride(0), K), _ptr(R), act_bits, _ptr(codes),
                                         _ptr(scales), _ptr(precond), _ptr(ws), nbytes,
                                         _stream(stream)))
    return codes, scales


def route_workspace(T: int, E: int, topk: int, n_shared: int = 0) -> int:
    """Bytes of device workspace moe_route_gather needs (cbq_route_workspace)."""
    return int(load_library().cbq_route_workspace(T, E, topk, n_shared))


def moe_route_gather(logits: torch.Tensor, topk: int, renormalize: bool = True, n_shared: int = 0,
                     out: Optional[dict] = None, stream=None) -> dict:
    """logits fp32 [T][E] -> dict(ids, weights, offsets, sorted_tokens, slot_of).

    ``out`` may hold preallocated outputs under those names and a workspace under "ws"."""
    lib = load_library()
    _require_gpu(logits)
    T, E = logits.shape
    dev = logits.device
    o = out or {}
    ids = o.get("ids") if o.get("ids") is not None else torch.empty((T, topk), dtype=torch.int32, device=dev)
    w = o.get("weights") if o.get("weights") is not None else torch.empty((T, topk), dtype=torch.float32, device=dev)
    offs = o.get("offsets") if o.get("offsets") is not None else torch.empty((E + n_shared + 1,), dtype=torch.int32, device=dev)
    R = T * topk + n_shared * T
    st = o.get("sorted_tokens") if o.get("sorted_tokens") is not None else torch.empty((max(R, 1),), dtype=torch.int32, device=dev)
    so = o.get("slot_of") if o.get("slot_of") is not None else torch.empty((T, topk), dtype=torch.int32, device=dev)
    need = int(lib.cbq_route_workspace(T, E, topk, n_shared))
    ws = o.get("ws")
    if need > 0 and (ws is None or ws.numel() * ws.element_size() < need):
        ws = torch.empty((need,), dtype=torch.uint8, device=dev)
    _check(lib.cbq_moe_route_gather(_ptr(logits), T, E, topk, int(bool(renormalize)), n_shared,
                                    _ptr(ids), _ptr(w), _ptr(offs), _ptr(st), _ptr(so),
                                    _ptr(ws) if need > 0 else None, need, _stream(stream)))
    return dict(ids=ids, weights=w, offsets=offs, sorted_tokens=st[:R], slot_of=so)


def moe_route_gather_noalloc(logits: torch.Tensor, topk: int, renormalize: bool = True,
                             n_shared: int = 0, out: Optional[dict] = None, stream=None) -> dict:
    """moe_route_gather through cbq_moe_route_gather_noalloc: the library's own scratch
    replaces the workspace.  ``out`` may hold preallocated outputs as for
    moe_route_gather (its "ws" entry is ignored)."""
    lib = load_library()
    _require_gpu(logits)
    T, E = logits.shape
    dev = logits.device
    o = out or {}

    def get(name, shape, dtype):
        t = o.get(name)
        return t if t is not None else torch.empty(shape, dtype=dtype, device=dev)

    R = T * topk + n_shared * T
    ids = get("ids", (T, topk), torch.int32)
    w = get("weights", (T, topk), torch.float32)
    offs = get("offsets", (E + n_shared + 1,), torch.int32)
    st = get("sorted_tokens", (max(R, 1),), torch.int32)
    so = get("slot_of", (T, topk), torch.int32)
    _check(lib.cbq_moe_route_gather_noalloc(_ptr(logits), T, E, topk, int(bool(renormalize)),
                                            n_shared, _ptr(ids), _ptr(w), _ptr(offs), _ptr(st),
                                            _ptr(so), _stream(stream)))
    return dict(ids=ids, weights=w, offsets=offs, sorted_tokens=st[:R], slot_of=so)


def prepack_weights(w: CodebookWeights, stream=None) -> CodebookWeights:
    """The blocked-layout copy of a row-layout weight set (cbq_prepack_weights); the
    codebooks are shared, not copied."""
    lib = load_library()
    _require_gpu(w.idx, w.codebook)
    if w.layout != LAYOUT_ROWS:
        raise ValueError("prepack_weights takes a row-layout weight set")
    s = w.c_struct()
    n = int(lib.cbq_prepack_bytes(ctypes.byref(s)))
    kp = (w.K + 127) // 128 * 128
    dst = torch.empty((w.E, w.N, kp * w.bits // 8), dtype=torch.uint8, device=w.idx.device)
    assert dst.numel() == n
    _check(lib.cbq_prepack_weights(ctypes.byref(s), _ptr(dst), _stream(stream)))
    return CodebookWeights(idx=dst, codebook=w.codebook, K=w.K, bits=w.bits, layout=LAYOUT_BLOCKED)


def gemm_workspace(weights: Sequence[CodebookWeights], n_rows: int, act_bits: int,
                   path: int = PATH_AUTO) -> int:
    """Bytes of optional GEMM workspace (cbq_gemm_workspace): with it, a single-matrix MFMA
    call whose tiles would leave CUs idle splits K in two, and a 4-bit gate/up call the
    column tiles of a half-empty last round; 0 when no call of these sizes can."""
    arr = (cbq_weights * len(weights))(*[w.c_struct() for w in weights])
    return int(load_library().cbq_gemm_workspace(arr, len(weights), n_rows, act_bits, path))


def codebook_lut_gemm(codes: torch.Tensor, scales: torch.Tensor, act_bits: int,
                      weights: Sequence[CodebookWeights], n_rows: Optional[int] = None,
                      expert_offsets: Optional[torch.Tensor] = None,
                      row_token: Optional[torch.Tensor] = None, epilogue: Optional[int] = None,
                      path: int = PATH_AUTO, out: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, stream=None):
    """Grouped codebook GEMM.  One weight set -> fp32 [R][N]; {gate, up} -> bf16 SwiGLU [R][N].

    ws: optional device workspace (a tensor of gemm_workspace(...) bytes or more)."""
    lib = load_library()
    _require_gpu(codes, scales, expert_offsets, row_token, ws)
    n_w = len(weights)
    if epilogue is None:
        epilogue = EPI_SWIGLU_BF16 if n_w == 2 else EPI_F32
    if n_rows is None:
        n_rows = row_token.shape[0] if row_token is not None else codes.shape[0]
    N = weights[0].N
    if out is None:
        dt = torch.bfloat16 if epilogue == EPI_SWIGLU_BF16 else torch.float32
        out = torch.empty((n_rows, N), dtype=dt, device=codes.device)
    arr = (cbq_weights * n_w)(*[w.c_struct() for w in weights])
    _check(lib.cbq_codebook_lut_gemm(_ptr(codes), _ptr(scales), act_bits, n_rows,
                                     _ptr(expert_offsets), _ptr(row_token), arr, n_w, epilogue,
                                     path, _ptr(out), out.stride(0), _ptr(ws),
                                     0 if ws is None else ws.numel() * ws.element_size(),
                                     _stream(stream)))
    return out


def moe_combine(expert_out: torch.Tensor, slot_of: torch.Tensor, topk_w: torch.Tensor,
                n_shared: int = 0, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    lib = load_library()
    _require_gpu(expert_out, slot_of, topk_w)
    T, topk = slot_of.shape
    H = expert_out.shape[1]
    if y is None:
        y = torch.empty((T, H), dtype=torch.float32, device=expert_out.device)
    _check(lib.cbq_moe_combine(_ptr(expert_out), _ptr(slot_of), _ptr(topk_w), T, topk, H, n_shared,
                               _ptr(y), _stream(stream)))
    return y


def _like_rows(x: torch.Tensor) -> torch.Tensor:
    """A contiguous bf16 tensor of x's shape."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _norm_outputs(x: torch.Tensor, act_bits: int, normed, codes, scales, want_normed: bool = True):
    if normed is None and want_normed:
        normed = _like_rows(x)
    T, K = x.shape
    dev = x.device
    if act_bits:
        if codes is None:
            codes = torch.empty((T, K * act_bits // 8), dtype=torch.uint8, device=dev)
        if scales is None:
            scales = torch.empty(T, dtype=torch.float32, device=dev)
    return normed, codes, scales


def _norm_struct(weight, eps, had_block, act_bits, normed, codes, scales) -> cbq_norm:
    return cbq_norm(weight.data_ptr(), eps, had_block, act_bits, _opt_ptr(normed),
                    0 if normed is None else _row_stride(normed), codes.data_ptr() if act_bits else None,
                    scales.data_ptr() if act_bits else None)


def _check_norm_args(T, K, dev, weight, act_bits, normed, codes, scales):
    _tensor("weight", weight, dev, torch.float32, (K,), contiguous=True)
    _tensor("normed", normed, dev, torch.bfloat16, (T, K), rows=True)
    if act_bits:
        _tensor("codes", codes, dev, torch.uint8, (T, K * act_bits // 8), contiguous=True)
        _tensor("scales", scales, dev, torch.float32, (T,), contiguous=True)
    elif codes is not None or scales is not None:
        raise ValueError("codes and scales are written with act_bits 4 or 8 only (got 0)")


def norm_rotate_quantize(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, act_bits: int = 4,
                         had_block: int = 0, want_normed: bool = True, normed: Optional[torch.Tensor] = None,
                         codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None, stream=None):
    """RMS norm of x (bf16 [T][K]) with weight (fp32 [K]), fused with rotate_quantize of its
    bf16 result: returns (normed, codes, scales).  act_bits = 0 leaves out the codes (codes
    and scales are None), want_normed = False the normed rows (cbq_norm_rotate_quantize)."""
    lib = load_library()
    _require_gpu(x)
    T, K = x.shape
    dev = x.device
    _tensor("x", x, dev, torch.bfloat16, rows=True)
    _check_norm_args(T, K, dev, weight, act_bits, normed, codes, scales)

    def call(st):
        n, c, s = _norm_outputs(x, act_bits, normed, codes, scales, want_normed)
        nrm = _norm_struct(weight, eps, had_block, act_bits, n, c, s)
        _check(lib.cbq_norm_rotate_quantize(x.data_ptr(), T, K, _row_stride(x), ctypes.byref(nrm), st))
        return (n, c, s) if act_bits else (n, None, None)

    return _on_stream(dev, stream, call)


def combine_norm_residual(rows: torch.Tensor, residual: torch.Tensor, slot_of: Optional[torch.Tensor] = None,
                          topk_w: Optional[torch.Tensor] = None, n_shared: Optional[int] = None,
                          post_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                          next_weight: Optional[torch.Tensor] = None, act_bits: int = 0, had_block: int = 0,
                          out: Optional[torch.Tensor] = None, normed: Optional[torch.Tensor] = None,
                          codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None, stream=None):
    """out = residual + scale * gate * norm(combined rows), bf16 [T][H]; with next_weight also
    the next block's norm of out: returns out, or (out, normed, codes, scales)
    (cbq_combine_norm_residual).

    rows: fp32 or bf16 [T*topk + n_shared*T][H] with slot_of and topk_w [T][topk] from
    moe_route_gather, or a block's output [T][H] without them.  post_weight (fp32 [H]) norms
    the combined row; gate is bf16 [T][H], or [H] / [1][H] for all tokens.  out may be
    residual.  act_bits = 0 leaves out the codes.  eps serves both norms."""
    lib = load_library()
    _require_gpu(rows, residual)
    dev = residual.device
    T, H = residual.shape
    if (slot_of is None) != (topk_w is None):
        raise ValueError("slot_of and topk_w go together")
    topk = 0 if slot_of is None else slot_of.shape[1]
    if n_shared is None:
        n_shared = 0 if topk else 1
    _tensor("residual", residual, dev, torch.bfloat16, rows=True)
    _tensor("rows", rows, dev, (torch.float32, torch.bfloat16), (T * topk + n_shared * T, H), rows=True)
    _tensor("slot_of", slot_of, dev, torch.int32, (T, topk), contiguous=True)
    _tensor("topk_w", topk_w, dev, torch.float32, (T, topk), contiguous=True)
    _tensor("post_weight", post_weight, dev, torch.float32, (H,), contiguous=True)
    _tensor("out", out, dev, torch.bfloat16, (T, H), rows=True)
    ldg = 0
    if gate is not None:
        shared_gate = gate.dim() == 1 or gate.shape[0] == 1 and T != 1
        _tensor("gate", gate, dev, torch.bfloat16, (H,) if gate.dim() == 1 else (1 if shared_gate else T, H), rows=True)
        ldg = 0 if shared_gate else _row_stride(gate)
    if next_weight is not None:
        _check_norm_args(T, H, dev, next_weight, act_bits, normed, codes, scales)
    elif normed is not None or codes is not None or scales is not None:
        raise ValueError("normed, codes and scales are written with next_weight only")

    def call(st):
        o = _like_rows(residual) if out is None else out
        nrm = None
        if next_weight is not None:
            n, c, s = _norm_outputs(residual, act_bits, normed, codes, scales)
            nrm = ctypes.byref(_norm_struct(next_weight, eps, had_block, act_bits, n, c, s))
        _check(lib.cbq_combine_norm_residual(
            rows.data_ptr(), TYPE_F32 if rows.dtype == torch.float32 else TYPE_BF16, _row_stride(rows), _opt_ptr(slot_of),
            _opt_ptr(topk_w), T, topk, n_shared, H, _opt_ptr(post_weight), eps, _opt_ptr(gate), ldg, scale, residual.data_ptr(),
            _row_stride(residual), o.data_ptr(), _row_stride(o), nrm, st))
        if next_weight is None:
            return o
        return (o, n, c, s) if act_bits else (o, n, None, None)

    return _on_stream(dev, stream, call)


def moe_few_workspace(T: int, topk: int, n_shared: int, H: int, F: int, act_bits: int = 4) -> int:
    """Bytes of device workspace moe_ffn_few needs (cbq_moe_few_workspace)."""
    return int(load_library().cbq_moe_few_workspace(T, topk, n_shared, H, F, act_bits))


def moe_ffn_few(codes: torch.Tensor, scales: torch.Tensor, logits: torch.Tensor, gate: CodebookWeights,
                up: CodebookWeights, down: CodebookWeights, topk: int, n_shared: int = 0, act_bits: int = 4,
                renormalize: bool = True, y: Optional[torch.Tensor] = None, y_dtype: torch.dtype = torch.bfloat16,
                ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The whole MoE FFN layer for at most FEW_MAX_TOKENS quantised tokens (cbq_moe_ffn_few):
    codes and scales from rotate_quantize or norm_rotate_quantize, router logits fp32 [T][E],
    gate/up/down of E + n_shared experts.  Returns y [T][H] in y_dtype (bf16 or fp32).

    h stays fp32 up to its quantiser, where moe_ffn rounds it to bf16.  ws: optional uint8
    device workspace of moe_few_workspace(...) bytes; calls that overlap need one each."""
    lib = load_library()
    _require_gpu(codes, scales, logits)
    dev = codes.device
    T, E = logits.shape
    H, F = gate.K, gate.N
    _tensor("codes", codes, dev, torch.uint8, (T, H * act_bits // 8), contiguous=True)
    _tensor("scales", scales, dev, torch.float32, (T,), contiguous=True)
    _tensor("logits", logits, dev, torch.float32, contiguous=True)
    g, u, d = gate._c_checked(dev, "gate"), up._c_checked(dev, "up"), down._c_checked(dev, "down")
    if y is not None:
        y_dtype = y.dtype
    if y_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"y must be float32 or bfloat16 (got {y_dtype})")
    _tensor("y", y, dev, y_dtype, (T, H), rows=True)
    _tensor("ws", ws, dev, torch.uint8, contiguous=True)

    def call(st):
        o = torch.empty((T, H), dtype=y_dtype, device=dev) if y is None else y
        w = ws if ws is not None else torch.empty((moe_few_workspace(T, topk, n_shared, H, F, act_bits),),
                                                  dtype=torch.uint8, device=dev)
        _check(lib.cbq_moe_ffn_few(codes.data_ptr(), scales.data_ptr(), act_bits, logits.data_ptr(), T, E, topk,
                                   int(bool(renormalize)), n_shared, ctypes.byref(g), ctypes.byref(u),
                                   ctypes.byref(d), o.data_ptr(),
                                   TYPE_F32 if y_dtype == torch.float32 else TYPE_BF16, _row_stride(o), w.data_ptr(),
                                   w.numel(), st))
        return o

    return _on_stream(dev, stream, call)


def adapter_workspace(T: int, rank: int) -> int:
    """Bytes of device workspace codebook_adapter_gemm needs (cbq_adapter_workspace)."""
    return int(load_library().cbq_adapter_workspace(T, rank))


def codebook_adapter_gemm(codes: torch.Tensor, scales: torch.Tensor, act_bits: int, weights: CodebookWeights,
                          x: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor, adapter_of: torch.Tensor,
                          adapter_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                          ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """A dense codebook projection with each token's low-rank adapter beside it
    (cbq_codebook_adapter_gemm): fp32 [T][N] = scale * q W^T + s_a (x A_a^T) B_a^T.

    x: bf16 [T][K], the unrotated activations; lora_a: bf16 [n][rank][K]; lora_b: bf16
    [n][N][rank]; adapter_of: int32 [T], -1 (or any id outside the set) for none;
    adapter_scale: fp32 [n] or None.  ws: optional uint8 device workspace of
    adapter_workspace(T, rank) bytes; calls that overlap need one each."""
    lib = load_library()
    _require_gpu(codes, scales, x)
    dev = codes.device
    T, K, N = x.shape[0], weights.K, weights.N
    n_ad, rank = lora_a.shape[0], lora_a.shape[1]
    _tensor("codes", codes, dev, torch.uint8, (T, K * act_bits // 8), contiguous=True)
    _tensor("scales", scales, dev, torch.float32, (T,), contiguous=True)
    W = weights._c_checked(dev, "weights")
    _tensor("x", x, dev, torch.bfloat16, (T, K), rows=True)
    _tensor("lora_a", lora_a, dev, torch.bfloat16, (n_ad, rank, K), contiguous=True)
    _tensor("lora_b", lora_b, dev, torch.bfloat16, (n_ad, N, rank), contiguous=True)
    _tensor("adapter_of", adapter_of, dev, torch.int32, (T,), contiguous=True)
    _tensor("adapter_scale", adapter_scale, dev, torch.float32, (n_ad,), contiguous=True)
    _tensor("out", out, dev, torch.float32, (T, N), rows=True)
    _tensor("ws", ws, dev, torch.uint8, contiguous=True)

    def call(st):
        o = torch.empty((T, N), dtype=torch.float32, device=dev) if out is None else out
        w = ws if ws is not None else torch.empty((adapter_workspace(T, rank),), dtype=torch.uint8, device=dev)
        _check(lib.cbq_codebook_adapter_gemm(
            codes.data_ptr(), scales.data_ptr(), act_bits, T, ctypes.byref(W), x.data_ptr(),
            _row_stride(x), lora_a.data_ptr(), lora_b.data_ptr(), _opt_ptr(adapter_scale), n_ad, rank,
            adapter_of.data_ptr(), o.data_ptr(), _row_stride(o), w.data_ptr(), w.numel(), st))
        return o

    return _on_stream(dev, stream, call)


def kmeans_codebooks(w: torch.Tensor, bits: int, max_iters: int = 50, idx: Optional[torch.Tensor] = None,
                     codebook: Optional[torch.Tensor] = None, iters_done: Optional[torch.Tensor] = None,
                     stream=None) -> CodebookWeights:
    """bf16 weight rows [R][K] (last dim contiguous) -> CodebookWeights (E = 1, N = R): one
    K-means per row (cbq_kmeans_codebooks)."""
    lib = load_library()
    _require_gpu(w)
    R, K = w.shape
    if w.stride(1) != 1:
        raise ValueError("w rows must be contiguous")
    dev = w.device
    if idx is None:
        idx = torch.empty((1, R, K * bits // 8), dtype=torch.uint8, device=dev)
    if codebook is None:
        codebook = torch.empty((1, R, 1 << bits), dtype=torch.int16, device=dev)
    _check(lib.cbq_kmeans_codebooks(_ptr(w), R, K, w.stride(0), bits, max_iters, _ptr(idx),
                                    _ptr(codebook), _ptr(iters_done), _stream(stream)))
    return CodebookWeights(idx=idx, codebook=codebook, K=K, bits=bits)


def refit_codebooks(w: torch.Tensor, cw: "CodebookWeights", x: torch.Tensor, stream=None) -> "CodebookWeights":
    """Output-aware refit of cw's centroids (in place) on bf16 calibration activations
    x [n][K] (cbq_refit_codebooks); w: the bf16 rows [R][K] that cw clusters."""
    lib = load_library()
    _require_gpu(w, x, cw.idx, cw.codebook)
    R, K = w.shape
    n = x.shape[0]
    if w.stride(1) != 1 or x.stride(1) != 1 or x.shape[1] != K or K != cw.K:
        raise ValueError("w and x need contiguous rows of the weights' K channels")
    if not cw.codebook.is_contiguous() or not cw.idx.is_contiguous():
        raise ValueError("the codebook and index tensors must be contiguous")
    _check(lib.cbq_refit_codebooks(_ptr(w), R, K, w.stride(0), cw.bits, _ptr(cw.idx), _ptr(x), n,
                                   x.stride(0), _ptr(cw.codebook), _stream(stream)))
    return cw


CPU_NO_AVX512 = 1


def cpu_lut_gemm(codes, scales, act_bits: int, idx, codebook, K: int, bits: int,
                 n_threads: int = 0, out=None, avx512: bool = True):
    """The LUT GEMM on host cores (cbq_cpu_lut_gemm).  numpy arrays: codes uint8
    [T][K*act_bits/8], scales float32 [T], idx uint8 [N][K*bits/8] (or [1][N][...]),
    codebook uint16 [N][2^bits]; returns float32 [T][N]."""
    import numpy as np
    lib = load_library()
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    scales = np.ascontiguousarray(scales, dtype=np.float32)
    idx = np.ascontiguousarray(idx, dtype=np.uint8).reshape(-1, K * bits // 8)
    codebook = np.ascontiguousarray(codebook).view(np.uint16).reshape(-1, 1 << bits)
    T, N = codes.shape[0], idx.shape[0]
    if out is None:
        out = np.empty((T, N), dtype=np.float32)
    w = cbq_weights(idx.ctypes.data, codebook.ctypes.data, 1, N, K, bits, LAYOUT_ROWS)
    _check(lib.cbq_cpu_lut_gemm(ctypes.c_void_p(codes.ctypes.data), ctypes.c_void_p(scales.ctypes.data),
                                act_bits, T, ctypes.byref(w), ctypes.c_void_p(out.ctypes.data),
                                out.strides[0] // 4, n_threads, 0 if avx512 else CPU_NO_AVX512))
    return out


def moe_ffn(x: torch.Tensor, logits: torch.Tensor, gate: CodebookWeights, up: CodebookWeights,
            down: CodebookWeights, topk: int, n_shared: int = 0, act_bits: int = 4,
            renormalize: bool = True, path: int = PATH_AUTO, keep: bool = False, stream=None):
    """One MoE FFN layer as a sequence of the four library calls (no compute here).

    gate/up/down hold E routed + n_shared shared experts.  Returns y fp32 [T][H], or
    (y, intermediates) when keep is True.  The GEMMs get the optional workspaces
    gemm_workspace asks for."""
    codes, scales = rotate_quantize(x, act_bits, stream=stream)
    rt = moe_route_gather(logits, topk, renormalize, n_shared, stream=stream)
    R = int(rt["sorted_tokens"].shape[0])

    def workspace(ws):
        n = gemm_workspace(ws, R, act_bits, path)
        return torch.empty((n,), dtype=torch.uint8, device=x.device) if n > 0 else None

    h = codebook_lut_gemm(codes, scales, act_bits, [gate, up], expert_offsets=rt["offsets"],
                          row_token=rt["sorted_tokens"], path=path, ws=workspace([gate, up]),
                          stream=stream)
    codes_h, scales_h = rotate_quantize(h, act_bits, stream=stream)
    out = codebook_lut_gemm(codes_h, scales_h, act_bits, [down], expert_offsets=rt["offsets"],
                            path=path, ws=workspace([down]), stream=stream)
    y = moe_combine(out, rt["slot_of"], rt["weights"], n_shared, stream=stream)
    if keep:
        return y, dict(codes=codes, scales=scales, route=rt, h=h, codes_h=codes_h,
                       scales_h=scales_h, out=out)
    return y
