"""Python binding of libmoe_exl3.so (MI355X / gfx950).

Argument marshalling only: every step of the layer runs in the HIP library
behind the C ABI declared in include/moe_exl3.h.  PyTorch provides device
memory and streams.  There is no fallback: if the library is missing or no
GPU is present, calls raise.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_exl3.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_MISALIGNED, ERR_HIP = 0, -1, -2, -3, -4, -5
DT_F32, DT_F16, DT_BF16, DT_FP8, DT_GEMV_F16, DT_MFMA_BIASED_F16 = 0, 1, 2, 3, 4, 5
CB_MCG, CB_MCG_E4M3 = 0, 1
HAS_SHARED, HAS_ROUTER_BIAS, FORCE_GEMV, FORCE_MFMA, FP8_MFMA = 1, 2, 4, 8, 16
DEBUG_CHECKS, DETERMINISTIC_COMBINE = 32, 64
HADAMARD, SHARED_TRELLIS, PER_TENSOR_K = 128, 256, 512
# status word of a workspace (int32 at byte STATUS_OFFSET)
STATUS_OFFSET = 8
(STATUS_BAD_INDEX, STATUS_TILE_OVERFLOW, STATUS_ACT_RANGE, STATUS_COUNTS, STATUS_TABLES,
 STATUS_NONFINITE_X, STATUS_BAD_WIDTH) = (1, 2, 4, 8, 16, 32, 64)

# every symbol the header declares
EXPORTS = ("moe_exl3_version", "moe_exl3_strerror", "moe_exl3_workspace_size",
           "moe_exl3_layer", "moe_exl3_layer_profiled", "moe_exl3_route", "moe_exl3_decode",
           "moe_exl3_repack", "moe_exl3_expand_block_scales", "moe_exl3_layer_noalloc",
           "moe_exl3_glu_workspace_size", "moe_exl3_glu_backward_workspace_size", "moe_exl3_glu",
           "moe_exl3_glu_backward", "moe_exl3_lora_workspace_size", "moe_exl3_lora_linear",
           "moe_exl3_sort_workspace_size", "moe_exl3_sort", "moe_exl3_dispatch", "moe_exl3_dispatch_backward",
           "moe_exl3_combine", "moe_exl3_combine_backward", "moe_exl3_dropout", "moe_exl3_w4_workspace_size",
           "moe_exl3_w4_linear", "moe_exl3_w4_glu")
ACT_SILU, ACT_GELU_TANH = 0, 1
SCRATCH_BYTES = 64 << 20
ORDER_ROWMAJOR, ORDER_COLMAJOR, ORDER_COLGROUPS128 = 0, 1, 2
# launch steps of moe_exl3_layer_profiled (events[i] is recorded before step i)
STEPS = ("route_logits", "topk", "segments", "convert_x", "gemv_gateup", "mfma_gateup",
         "gemv_down", "mfma_down", "shared", "combine")
STEP_END = len(STEPS)


class Desc(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("inter", C.c_int32), ("n_experts", C.c_int32),
                ("top_k", C.c_int32), ("K", C.c_int32), ("codebook", C.c_int32),
                ("mcg", C.c_uint32), ("act_dtype", C.c_int32), ("flags", C.c_uint32),
                ("gemv_max_rows", C.c_int32)]


class Weights(C.Structure):
    _fields_ = [("codes", C.c_void_p * 3), ("suh", C.c_void_p * 3), ("svh", C.c_void_p * 3),
                ("router_w", C.c_void_p), ("router_bias", C.c_void_p),
                ("shared_w", C.c_void_p * 3), ("signs", C.c_void_p), ("code_tab", C.c_void_p),
                ("k_tab", C.c_void_p)]


class GluDesc(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("inter", C.c_int32), ("act_dtype", C.c_int32), ("act", C.c_int32)]


class LoraDesc(C.Structure):
    _fields_ = [("n_in", C.c_int32), ("n_out", C.c_int32), ("n_adapters", C.c_int32), ("rank", C.c_int32),
                ("act_dtype", C.c_int32)]


class LoraAdapters(C.Structure):
    _fields_ = [("a", C.c_void_p), ("b", C.c_void_p), ("scales", C.c_void_p), ("ranks", C.c_void_p)]


class TokensDesc(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("n_experts", C.c_int32), ("top_k", C.c_int32), ("act_dtype", C.c_int32)]


class Drop(C.Structure):
    _fields_ = [("p", C.c_double), ("rng", C.c_void_p)]


class W4Desc(C.Structure):
    _fields_ = [("n_in", C.c_int32), ("n_out", C.c_int32), ("n_experts", C.c_int32), ("group", C.c_int32),
                ("act_dtype", C.c_int32), ("act", C.c_int32)]


class W4Weights(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("zeros", C.c_void_p)]


class MoeError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} ({code})")
        self.code = code


_lib = None


def lib():
    """Load the HIP library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m trellis_quantized_moe_exl3_amd.build`")
        l = C.CDLL(LIB_PATH)
        l.moe_exl3_version.restype = C.c_int
        l.moe_exl3_strerror.argtypes = [C.c_int]
        l.moe_exl3_strerror.restype = C.c_char_p
        l.moe_exl3_workspace_size.argtypes = [C.POINTER(Desc), C.c_int64, C.POINTER(C.c_size_t)]
        l.moe_exl3_layer.argtypes = [C.POINTER(Desc), C.POINTER(Weights), C.c_void_p, C.c_int64,
                                     C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]
        l.moe_exl3_layer_profiled.argtypes = [
            C.POINTER(Desc), C.POINTER(Weights), C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
            C.c_size_t, C.c_void_p, C.POINTER(C.c_void_p), C.c_int]
        l.moe_exl3_route.argtypes = [C.POINTER(Desc), C.POINTER(Weights), C.c_void_p, C.c_int64,
                                     C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                     C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]
        l.moe_exl3_decode.argtypes = [C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_uint32,
                                      C.c_int32, C.c_void_p, C.c_int32, C.c_void_p]
        l.moe_exl3_layer_noalloc.argtypes = [C.POINTER(Desc), C.POINTER(Weights), C.c_void_p, C.c_int64,
                                             C.c_void_p, C.c_void_p]
        l.moe_exl3_repack.argtypes = [C.c_void_p, C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_int32,
                                      C.c_int32, C.c_void_p]
        l.moe_exl3_expand_block_scales.argtypes = [C.c_void_p, C.c_int32, C.c_int32, C.c_int32,
                                                   C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.c_void_p]
        for f in ("moe_exl3_glu_workspace_size", "moe_exl3_glu_backward_workspace_size"):
            getattr(l, f).argtypes = [C.POINTER(GluDesc), C.c_int64, C.POINTER(C.c_size_t)]
        l.moe_exl3_lora_workspace_size.argtypes = [C.POINTER(LoraDesc), C.c_int64, C.POINTER(C.c_size_t)]
        l.moe_exl3_glu.argtypes = [C.POINTER(GluDesc), C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p, C.c_int64,
                                   C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]
        l.moe_exl3_glu_backward.argtypes = [
            C.POINTER(GluDesc), C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64,
            C.c_int64, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]
        l.moe_exl3_lora_linear.argtypes = [
            C.POINTER(LoraDesc), C.c_void_p, C.c_int64, C.c_void_p, C.POINTER(LoraAdapters), C.c_void_p, C.c_void_p,
            C.c_int64, C.c_int64, C.c_void_p, C.c_int64, C.c_void_p, C.c_size_t, C.c_void_p]
        p, i, z = C.c_void_p, C.c_int64, C.c_size_t
        td, dr, wd, ww = C.POINTER(TokensDesc), C.POINTER(Drop), C.POINTER(W4Desc), C.POINTER(W4Weights)
        l.moe_exl3_sort_workspace_size.argtypes = [td, i, C.POINTER(z)]
        l.moe_exl3_sort.argtypes = [td, p, i, p, p, p, p, p, z, p]
        l.moe_exl3_dispatch.argtypes = [td, p, i, p, p, i, i, p, i, p]
        l.moe_exl3_dispatch_backward.argtypes = [td, p, i, p, i, p, p, i, i, p, i, p, p]
        l.moe_exl3_combine.argtypes = [td, p, i, p, p, p, i, dr, i, i, p, i, p]
        l.moe_exl3_combine_backward.argtypes = [td, p, i, p, i, p, p, dr, i, i, p, i, p, p]
        l.moe_exl3_dropout.argtypes = [C.c_int32, p, i, p, i, dr, i, i, p, i, p]
        l.moe_exl3_w4_workspace_size.argtypes = [wd, i, C.POINTER(z)]
        l.moe_exl3_w4_linear.argtypes = [wd, p, i, ww, p, p, i, i, p, i, p, z, p]
        l.moe_exl3_w4_glu.argtypes = [wd, p, i, ww, ww, p, i, p, i, p, z, p]
        for f in EXPORTS[EXPORTS.index("moe_exl3_glu_workspace_size"):]:
            getattr(l, f).restype = C.c_int
        for f in ("moe_exl3_workspace_size", "moe_exl3_layer", "moe_exl3_layer_profiled",
                  "moe_exl3_route", "moe_exl3_decode", "moe_exl3_repack", "moe_exl3_expand_block_scales",
                  "moe_exl3_layer_noalloc"):
            getattr(l, f).restype = C.c_int
        _lib = l
    return _lib


def version() -> int:
    return lib().moe_exl3_version()


def strerror(code: int) -> str:
    return lib().moe_exl3_strerror(code).decode()


def _check(rc: int, what: str):
    if rc != OK:
        raise MoeError(rc, what)


def make_desc(hidden, inter, n_experts, top_k, K, codebook=CB_MCG, mcg=0x9E3779B1,
              act_dtype=DT_BF16, flags=0, gemv_max_rows=0) -> Desc:
    return Desc(hidden, inter, n_experts, top_k, K, codebook, mcg & 0xFFFFFFFF, act_dtype, flags,
                gemv_max_rows)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr()


def make_weights(codes: Sequence, suh: Sequence, svh: Sequence, router_w, router_bias=None,
                 shared: Optional[Sequence] = None, signs=None, code_tab=None, k_tab=None) -> Weights:
    """Weights struct from device tensors (the tensors must outlive its use).
    signs: int8 [2][H]; code_tab: int64 [3][EA] device addresses of the
    per-tensor codes; k_tab: int32 [3][EA] widths."""
    w = Weights()
    w.signs = _ptr(signs)
    w.code_tab = _ptr(code_tab)
    w.k_tab = _ptr(k_tab)
    for p in range(3):
        w.codes[p] = _ptr(codes[p]) if codes is not None else None
        w.suh[p] = _ptr(suh[p])
        w.svh[p] = _ptr(svh[p])
        w.shared_w[p] = _ptr(shared[p]) if shared is not None else None
    w.router_w = _ptr(router_w)
    w.router_bias = _ptr(router_bias)
    return w


def workspace_size(desc: Desc, max_tokens: int) -> int:
    n = C.c_size_t(0)
    _check(lib().moe_exl3_workspace_size(C.byref(desc), max_tokens, C.byref(n)), "workspace_size")
    return n.value


def _check_acts(desc: Desc, what: str, *tensors) -> None:
    """x and out must be contiguous 2-D device tensors [T][hidden] of a 2-byte
    dtype (bf16 or fp16 data, raw int16 accepted) matching act_dtype, all of
    the same shape: the kernels index them as such."""
    import torch
    want = {DT_BF16: (torch.bfloat16, torch.int16), DT_F16: (torch.float16, torch.int16)}[desc.act_dtype]
    shape = None
    for t in tensors:
        if t.dim() != 2 or t.shape[1] != desc.hidden:
            raise ValueError(f"{what}: expected [T][{desc.hidden}], got {tuple(t.shape)}")
        if t.dtype not in want:
            raise ValueError(f"{what}: dtype {t.dtype} does not match act_dtype {desc.act_dtype}")
        if not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{what}: tensors must be contiguous and on the GPU")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{what}: x and out shapes differ")
        shape = t.shape


def _check_ws(workspace) -> None:
    if workspace is None or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")


def status(workspace) -> int:
    """The status word of the last call that used `workspace` (synchronises)."""
    import torch
    torch.cuda.synchronize()
    return int(workspace.view(torch.uint8)[STATUS_OFFSET:STATUS_OFFSET + 4].cpu().view(torch.int32).item())


_torch_mod = _raw_stream = _current_device = None


def _torch():
    """torch, and its lookup of the current stream's handle (building a Stream
    object costs as much as a launch; used where torch has no such lookup)."""
    global _torch_mod, _raw_stream, _current_device
    if _torch_mod is None:
        import torch
        _current_device = torch.cuda.current_device
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda device: torch.cuda.current_stream(device).cuda_stream)
        _torch_mod = torch
    return _torch_mod


def _stream(stream, device: Optional[int] = None) -> int:
    """Handle of a stream; None: the current one (of `device`, if it is known
    to be the current GPU)."""
    if stream is not None:
        return stream.cuda_stream
    if device is None:
        device = _torch().cuda.current_device()
    return _raw_stream(device)


def layer(desc: Desc, weights: Weights, x, out, workspace, stream=None) -> None:
    """out = MoE layer(x); x, out: [T][H] device tensors of the activation dtype."""
    _check_acts(desc, "layer", x, out)
    _check_ws(workspace)
    T = x.shape[0]
    _check(lib().moe_exl3_layer(C.byref(desc), C.byref(weights), _ptr(x), T, _ptr(out),
                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream(stream)), "moe_exl3_layer")


def layer_noalloc(desc: Desc, weights: Weights, x, out, stream=None) -> None:
    """layer() with the library's own per-GPU scratch array as the workspace
    (moe_exl3_layer_noalloc): allocates nothing."""
    _check_acts(desc, "layer_noalloc", x, out)
    T = x.shape[0]
    _check(lib().moe_exl3_layer_noalloc(C.byref(desc), C.byref(weights), _ptr(x), T, _ptr(out),
                                        _stream(stream)), "moe_exl3_layer_noalloc")


def layer_profiled(desc: Desc, weights: Weights, x, out, workspace, events, stream=None) -> None:
    """layer() recording events[i] (hipEvent_t handles) before launch step i."""
    _check_acts(desc, "layer_profiled", x, out)
    _check_ws(workspace)
    T = x.shape[0]
    arr = (C.c_void_p * len(events))(*events)
    _check(lib().moe_exl3_layer_profiled(C.byref(desc), C.byref(weights), _ptr(x), T, _ptr(out),
                                         _ptr(workspace), workspace.numel() * workspace.element_size(),
                                         _stream(stream), arr, len(events)),
           "moe_exl3_layer_profiled")


def route(desc: Desc, weights: Weights, x, idx, w=None, counts=None, offsets=None,
          sorted_ids=None, pos=None, workspace=None, stream=None) -> None:
    """Routing tables of x (moe_exl3_route); outputs are int32/fp32 device
    tensors of T*k (idx, w, sorted_ids, pos), E (counts) or E+1 (offsets)
    elements, or None (idx is required)."""
    _check_acts(desc, "route", x)
    _check_ws(workspace)
    T = x.shape[0]
    n, E = T * desc.top_k, desc.n_experts
    for t, size, what in ((idx, n, "idx"), (w, n, "w"), (counts, E, "counts"), (offsets, E + 1, "offsets"),
                          (sorted_ids, n, "sorted_ids"), (pos, n, "pos")):
        if t is None:
            if what == "idx":
                raise ValueError("route: idx is required")
            continue
        if not t.is_cuda or not t.is_contiguous() or t.numel() < size or t.element_size() != 4:
            raise ValueError(f"route: {what} must be a contiguous 4-byte GPU tensor of >= {size} elements")
    _check(lib().moe_exl3_route(C.byref(desc), C.byref(weights), _ptr(x), T, _ptr(idx), _ptr(w),
                                _ptr(counts), _ptr(offsets), _ptr(sorted_ids), _ptr(pos),
                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream(stream)), "moe_exl3_route")


def decode(codes, n_in: int, n_out: int, K: int, mcg: int, codebook: int, dst, dst_dtype: int,
           stream=None) -> None:
    """Dense [n_in][n_out] decode of one trellis-coded matrix into `dst`."""
    nbytes = n_in * n_out * (4 if dst_dtype == DT_F32 else 1 if dst_dtype == DT_FP8 else 2)
    words = (n_in // 16) * (n_out // 16) * 16 * K
    if not (dst.is_cuda and codes.is_cuda and dst.is_contiguous() and codes.is_contiguous()):
        raise ValueError("decode: codes and dst must be contiguous GPU tensors")
    if dst.numel() * dst.element_size() < nbytes or codes.numel() * codes.element_size() < 2 * words:
        raise ValueError("decode: codes or dst smaller than the matrix")
    _check(lib().moe_exl3_decode(_ptr(codes), n_in, n_out, K, mcg & 0xFFFFFFFF, codebook,
                                 _ptr(dst), dst_dtype, _stream(stream)), "moe_exl3_decode")


def repack(src, dst, count: int, n_in: int, n_out: int, K: int, src_order: int, stream=None) -> None:
    """Reorder the tile grids of `count` trellis tensors from `src_order` into
    the kernels' row-major grid (moe_exl3_repack)."""
    words = count * (n_in // 16) * (n_out // 16) * 16 * K
    for t, what in ((src, "src"), (dst, "dst")):
        if not t.is_cuda or not t.is_contiguous() or t.numel() * t.element_size() < 2 * words:
            raise ValueError(f"repack: {what} must be a contiguous GPU tensor of >= {2 * words} bytes")
    _check(lib().moe_exl3_repack(_ptr(src), _ptr(dst), count, n_in, n_out, K, src_order, _stream(stream)),
           "moe_exl3_repack")


def expand_block_scales(block, n_trellis: int, hidden: int, inter: int, suh: Sequence, svh: Sequence,
                        stream=None) -> None:
    """Per-channel side vectors from the block table [n_trellis][3][hidden/128]
    (moe_exl3_expand_block_scales)."""
    if block.numel() < n_trellis * 3 * (hidden // 128):
        raise ValueError("expand_block_scales: block table too small")
    for p in range(3):
        n_in, n_out = (hidden, inter) if p < 2 else (inter, hidden)
        if suh[p].numel() < n_trellis * n_in or svh[p].numel() < n_trellis * n_out:
            raise ValueError("expand_block_scales: side vector too small")
    sp = (C.c_void_p * 3)(*[_ptr(t) for t in suh])
    vp = (C.c_void_p * 3)(*[_ptr(t) for t in svh])
    _check(lib().moe_exl3_expand_block_scales(_ptr(block), n_trellis, hidden, inter, sp, vp, _stream(stream)),
           "moe_exl3_expand_block_scales")


# ---- dense operators: the gated feed-forward block and the projection with adapters


def make_glu_desc(hidden: int, inter: int, act_dtype: int = DT_BF16, act: int = ACT_SILU) -> GluDesc:
    return GluDesc(hidden, inter, act_dtype, act)


def make_lora_desc(n_in: int, n_out: int, n_adapters: int, rank: int, act_dtype: int = DT_BF16) -> LoraDesc:
    return LoraDesc(n_in, n_out, n_adapters, rank, act_dtype)


def _size(fn: str, desc, max_tokens: int) -> int:
    n = C.c_size_t(0)
    _check(getattr(lib(), fn)(C.byref(desc), max_tokens, C.byref(n)), fn)
    return n.value


def glu_workspace_size(desc: GluDesc, max_tokens: int) -> int:
    return _size("moe_exl3_glu_workspace_size", desc, max_tokens)


def glu_backward_workspace_size(desc: GluDesc, max_tokens: int) -> int:
    return _size("moe_exl3_glu_backward_workspace_size", desc, max_tokens)


def lora_workspace_size(desc: LoraDesc, max_tokens: int) -> int:
    return _size("moe_exl3_lora_workspace_size", desc, max_tokens)


_dense_types = {}


def _dense_dtypes(act_dtype: int):
    """Tensor dtypes accepted for a 16-bit argument (its own, or raw int16)."""
    if not _dense_types:
        torch = _torch()
        _dense_types.update({DT_BF16: (torch.bfloat16, torch.int16), DT_F16: (torch.float16, torch.int16)})
    if act_dtype not in _dense_types:
        raise ValueError(f"act_dtype {act_dtype} is neither DT_F16 nor DT_BF16")
    return _dense_types[act_dtype]


def _rows(t, rows: int, cols: int, types, device: int, what: str) -> int:
    """Row stride of a [rows][cols] activation on a GPU (unit column stride,
    rows apart by any stride; a single row or column has none)."""
    if t.shape != (rows, cols) or t.dtype not in types or t.get_device() != device:
        raise ValueError(f"{what}: expected [{rows}][{cols}] {types[0]} on GPU {device}, got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device}")
    ld, step = t.stride()
    if rows <= 1:
        ld = cols
    if (step != 1 and cols != 1) or ld < cols:
        raise ValueError(f"{what}: rows must be contiguous and apart, got strides {t.stride()}")
    return ld


def _whole(t, shape, types, device: int, what: str):
    """A contiguous tensor of exactly this shape."""
    if t.shape != shape or t.dtype not in types or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous {shape} {types[0]} on GPU {device}, got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device}")


def _dense_device(x, workspace, stream, what: str) -> int:
    """The GPU of a call: that of x, which must be the current one, of the
    workspace and of the stream."""
    d = x.get_device()   # below 0: not on a GPU
    if d < 0 or d != _torch().cuda.current_device():
        raise ValueError(f"{what}: tensors must be on the current GPU, got {x.device}")
    if workspace is None or workspace.get_device() != d or not workspace.is_contiguous():
        raise ValueError(f"{what}: workspace must be a contiguous tensor on GPU {d}")
    if stream is not None and stream.device != x.device:
        raise ValueError(f"{what}: a stream of {stream.device}, tensors on {x.device}")
    return d


def glu(desc: GluDesc, x, w_gate, w_up, out, workspace, pre=None, stream=None) -> None:
    """out = act(x w_gate^T) * (x w_up^T) (moe_exl3_glu).  x [T][hidden], out
    [T][inter], weights [inter][hidden]; pre: optional fp32 [2][T][inter] that
    receives the two products for glu_backward()."""
    d = _dense_device(x, workspace, stream, "glu")
    types, T, H, I = _dense_dtypes(desc.act_dtype), x.shape[0], desc.hidden, desc.inter
    ldx, ldo = _rows(x, T, H, types, d, "glu: x"), _rows(out, T, I, types, d, "glu: out")
    _whole(w_gate, (I, H), types, d, "glu: w_gate")
    _whole(w_up, (I, H), types, d, "glu: w_up")
    if pre is not None:
        _whole(pre, (2, T, I), (_torch().float32,), d, "glu: pre")
    _check(lib().moe_exl3_glu(C.byref(desc), x.data_ptr(), ldx, w_gate.data_ptr(), w_up.data_ptr(), T,
                              out.data_ptr(), ldo, _ptr(pre), workspace.data_ptr(), workspace.nbytes,
                              _stream(stream, d)), "moe_exl3_glu")


def glu_backward(desc: GluDesc, x, w_gate, w_up, pre, dout, workspace, dx=None, dw_gate=None, dw_up=None,
                 stream=None) -> None:
    """Gradients of glu() from dout and its `pre` (moe_exl3_glu_backward): dx
    [T][hidden] and / or dw_gate and dw_up [inter][hidden], written."""
    d = _dense_device(x, workspace, stream, "glu_backward")
    types, T, H, I = _dense_dtypes(desc.act_dtype), x.shape[0], desc.hidden, desc.inter
    ldx, lddo = _rows(x, T, H, types, d, "glu_backward: x"), _rows(dout, T, I, types, d, "glu_backward: dout")
    _whole(pre, (2, T, I), (_torch().float32,), d, "glu_backward: pre")
    lddx = H
    if dx is not None:
        lddx = _rows(dx, T, H, types, d, "glu_backward: dx")
    for t, what in ((w_gate, "w_gate"), (w_up, "w_up"), (dw_gate, "dw_gate"), (dw_up, "dw_up")):
        if t is not None:
            _whole(t, (I, H), types, d, "glu_backward: " + what)
    _check(lib().moe_exl3_glu_backward(C.byref(desc), x.data_ptr(), ldx, _ptr(w_gate), _ptr(w_up), pre.data_ptr(),
                                       dout.data_ptr(), lddo, T, _ptr(dx), lddx, _ptr(dw_gate), _ptr(dw_up),
                                       workspace.data_ptr(), workspace.nbytes, _stream(stream, d)),
           "moe_exl3_glu_backward")


def lora_linear(desc: LoraDesc, x, w, lora_a, lora_b, ids, out, workspace, base=None, scales=None, ranks=None,
                stream=None) -> None:
    """out[t] = x[t] w^T + base[t] + scales[e] lora_b[e] (lora_a[e] x[t]), e =
    ids[t] (-1: no adapter) (moe_exl3_lora_linear).  x [T][n_in]; w
    [n_out][n_in] or None; lora_a [n_adapters][rank][n_in]; lora_b
    [n_adapters][n_out][rank]; ids int32 [T]; base [T][n_out] or None, may be
    out; scales fp32 and ranks int32 [n_adapters] or None.  status(workspace)
    reports ids and ranks out of range."""
    torch = _torch()
    d = _dense_device(x, workspace, stream, "lora_linear")
    types, T = _dense_dtypes(desc.act_dtype), x.shape[0]
    K, N, n, r = desc.n_in, desc.n_out, desc.n_adapters, desc.rank
    ldx, ldy = _rows(x, T, K, types, d, "lora_linear: x"), _rows(out, T, N, types, d, "lora_linear: out")
    ldb = N
    if base is not None:
        ldb = _rows(base, T, N, types, d, "lora_linear: base")
    if w is not None:
        _whole(w, (N, K), types, d, "lora_linear: w")
    _whole(lora_a, (n, r, K), types, d, "lora_linear: lora_a")
    _whole(lora_b, (n, N, r), types, d, "lora_linear: lora_b")
    _whole(ids, (T,), (torch.int32,), d, "lora_linear: ids")
    if scales is not None:
        _whole(scales, (n,), (torch.float32,), d, "lora_linear: scales")
    if ranks is not None:
        _whole(ranks, (n,), (torch.int32,), d, "lora_linear: ranks")
    ad = LoraAdapters(lora_a.data_ptr(), lora_b.data_ptr(), _ptr(scales), _ptr(ranks))
    _check(lib().moe_exl3_lora_linear(C.byref(desc), x.data_ptr(), ldx, _ptr(w), C.byref(ad), ids.data_ptr(),
                                      _ptr(base), ldb, T, out.data_ptr(), ldy, workspace.data_ptr(),
                                      workspace.nbytes, _stream(stream, d)), "moe_exl3_lora_linear")


# ---- operators around a MoE layer's own experts: sort, dispatch, combine,
# dropout, products with 4-bit weights


def make_tokens_desc(hidden: int, n_experts: int, top_k: int, act_dtype: int = DT_BF16) -> TokensDesc:
    return TokensDesc(hidden, n_experts, top_k, act_dtype)


def make_w4_desc(n_in: int, n_out: int, n_experts: int = 1, group: int = 128, act_dtype: int = DT_BF16,
                 act: int = ACT_SILU) -> W4Desc:
    return W4Desc(n_in, n_out, n_experts, group, act_dtype, act)


def sort_workspace_size(desc: TokensDesc, max_tokens: int) -> int:
    return _size("moe_exl3_sort_workspace_size", desc, max_tokens)


def w4_workspace_size(desc: W4Desc, max_rows: int) -> int:
    return _size("moe_exl3_w4_workspace_size", desc, max_rows)


def _call_device(x, stream, what: str) -> int:
    """The GPU of a call without a workspace: that of x, which must be the
    current one, and of the stream."""
    d = x.get_device()   # below 0: not on a GPU
    if _torch_mod is None:
        _torch()
    if d < 0 or d != _current_device():
        raise ValueError(f"{what}: tensors must be on the current GPU, got {x.device}")
    if stream is not None and stream.device != x.device:
        raise ValueError(f"{what}: a stream of {stream.device}, tensors on {x.device}")
    return d


def _table(t, n: int, dtype, device: int, what: str, name: str) -> int:
    """Address of a contiguous table of n entries, of any shape."""
    if t.numel() != n or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what}: {name}: expected {n} contiguous {dtype} on GPU {device}, got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device}")
    return t.data_ptr()


def _drop(p: float, rng, device: int, what: str):
    """The dropout argument of a call (None: nothing is dropped)."""
    if p == 0 and rng is None:
        return None
    if rng is None:
        raise ValueError(f"{what}: dropout needs rng, two int64 on the GPU (seed and offset)")
    torch = _torch()
    if rng.numel() != 2 or rng.dtype not in (torch.int64, torch.uint64) or rng.get_device() != device \
            or not rng.is_contiguous():
        raise ValueError(f"{what}: rng must be two contiguous int64 (seed, offset) on GPU {device}")
    return C.byref(Drop(p, rng.data_ptr()))


def sort(desc: TokensDesc, idx, counts, offsets, sorted_ids, pos, workspace, stream=None) -> None:
    """Tables of the slots sorted by expert (moe_exl3_sort).  idx int32 [T][k]
    (-1: no expert); counts [E] or None, offsets [E + 1], sorted_ids [T k] or
    None, pos [T k]: int32, written.  status(workspace) reports indexes out of
    range."""
    i32 = _torch().int32
    d = _dense_device(idx, workspace, stream, "sort")
    E, k, T = desc.n_experts, desc.top_k, idx.shape[0]
    _whole(idx, (T, k), (i32,), d, "sort: idx")
    offsets, pos = _table(offsets, E + 1, i32, d, "sort", "offsets"), _table(pos, T * k, i32, d, "sort", "pos")
    if counts is not None:
        counts = _table(counts, E, i32, d, "sort", "counts")
    if sorted_ids is not None:
        sorted_ids = _table(sorted_ids, T * k, i32, d, "sort", "sorted_ids")
    _check(lib().moe_exl3_sort(C.byref(desc), idx.data_ptr(), T, counts, offsets, sorted_ids, pos, workspace.data_ptr(),
                               workspace.nbytes, _stream(stream, d)), "moe_exl3_sort")


def _slots(desc: TokensDesc, T: int, pos, w, dw, device: int, what: str):
    """Addresses of the slots' tables (None: none)."""
    n = T * desc.top_k
    torch = _torch_mod
    return (_table(pos, n, torch.int32, device, what, "pos"),
            None if w is None else _table(w, n, torch.float32, device, what, "w"),
            None if dw is None else _table(dw, n, torch.float32, device, what, "dw"))


def dispatch(desc: TokensDesc, x, pos, out, w=None, stream=None) -> None:
    """out[pos[a]] = w[a] x[a // k] (moe_exl3_dispatch).  x [T][hidden], out
    [rows][hidden]; pos int32 and w fp32 (or None) [T][k]."""
    d = _call_device(x, stream, "dispatch")
    types, T, H = _dense_dtypes(desc.act_dtype), x.shape[0], desc.hidden
    ldx = _rows(x, T, H, types, d, "dispatch: x")
    ldo = _rows(out, out.shape[0], H, types, d, "dispatch: out")
    pos, w, _ = _slots(desc, T, pos, w, None, d, "dispatch")
    _check(lib().moe_exl3_dispatch(C.byref(desc), x.data_ptr(), ldx, pos, w, T, out.shape[0],
                                   out.data_ptr(), ldo, _stream(stream, d)), "moe_exl3_dispatch")


def dispatch_backward(desc: TokensDesc, dout, x, pos, dx, w=None, dw=None, stream=None) -> None:
    """Gradients of dispatch() from dout [rows][hidden]: dx [T][hidden], and dw
    fp32 [T][k] where it is given (x is read for it alone, else maybe None)."""
    d = _call_device(dx, stream, "dispatch_backward")
    types, T, H = _dense_dtypes(desc.act_dtype), dx.shape[0], desc.hidden
    lddx = _rows(dx, T, H, types, d, "dispatch_backward: dx")
    lddo = _rows(dout, dout.shape[0], H, types, d, "dispatch_backward: dout")
    ldx = H
    if x is not None:
        ldx = _rows(x, T, H, types, d, "dispatch_backward: x")
    pos, w, dw = _slots(desc, T, pos, w, dw, d, "dispatch_backward")
    _check(lib().moe_exl3_dispatch_backward(C.byref(desc), dout.data_ptr(), lddo, _ptr(x), ldx, pos, w, T, dout.shape[0],
                                            dx.data_ptr(), lddx, dw, _stream(stream, d)),
           "moe_exl3_dispatch_backward")


def combine(desc: TokensDesc, z, pos, y, w=None, base=None, p: float = 0.0, rng=None, stream=None) -> None:
    """y[t] = base[t] + D(sum_j w[a] z[pos[a]]) (moe_exl3_combine), D dropout with
    probability p from rng (int64 {seed, offset} on the GPU).  z [rows][hidden],
    y and base [T][hidden]; pos int32 and w fp32 (or None) [T][k]."""
    d = _call_device(y, stream, "combine")
    types, T, H = _dense_dtypes(desc.act_dtype), y.shape[0], desc.hidden
    ldy, ldz = _rows(y, T, H, types, d, "combine: y"), _rows(z, z.shape[0], H, types, d, "combine: z")
    ldb = H
    if base is not None:
        ldb = _rows(base, T, H, types, d, "combine: base")
    pos, w, _ = _slots(desc, T, pos, w, None, d, "combine")
    _check(lib().moe_exl3_combine(C.byref(desc), z.data_ptr(), ldz, pos, w, _ptr(base), ldb,
                                  _drop(p, rng, d, "combine"), T, z.shape[0], y.data_ptr(), ldy, _stream(stream, d)),
           "moe_exl3_combine")


def combine_backward(desc: TokensDesc, dy, z, pos, dz, w=None, dw=None, p: float = 0.0, rng=None, stream=None) -> None:
    """Gradients of combine() from dy [T][hidden], with the p and rng of its call:
    dz [rows][hidden] (may be z itself), and dw fp32 [T][k] where it is given (z
    is read for it alone, else maybe None)."""
    d = _call_device(dy, stream, "combine_backward")
    types, T, H = _dense_dtypes(desc.act_dtype), dy.shape[0], desc.hidden
    rows = dz.shape[0]
    lddy, lddz = _rows(dy, T, H, types, d, "combine_backward: dy"), _rows(dz, rows, H, types, d, "combine_backward: dz")
    ldz = H
    if z is not None:
        ldz = _rows(z, rows, H, types, d, "combine_backward: z")
    pos, w, dw = _slots(desc, T, pos, w, dw, d, "combine_backward")
    _check(lib().moe_exl3_combine_backward(C.byref(desc), dy.data_ptr(), lddy, _ptr(z), ldz, pos, w,
                                           _drop(p, rng, d, "combine_backward"), T, rows, dz.data_ptr(), lddz, dw,
                                           _stream(stream, d)), "moe_exl3_combine_backward")


def dropout(x, y, p: float, rng, residual=None, stream=None) -> None:
    """y = residual + D(x) (moe_exl3_dropout), D dropout with probability p from
    rng (int64 {seed, offset} on the GPU); with a gradient for x, D's gradient.  x,
    y, residual: [rows][cols] bf16, fp16 or fp32, rows apart by any stride, the
    first at a 16-byte aligned address."""
    torch = _torch()
    d = _call_device(x, stream, "dropout")
    dt = {torch.bfloat16: DT_BF16, torch.float16: DT_F16, torch.float32: DT_F32}.get(x.dtype)
    if dt is None or x.dim() != 2:
        raise ValueError(f"dropout: x must be [rows][cols] bf16, fp16 or fp32, got {tuple(x.shape)} {x.dtype}")
    rows, cols = x.shape
    types = (x.dtype,)
    ldx, ldy, ldr = _rows(x, rows, cols, types, d, "dropout: x"), _rows(y, rows, cols, types, d, "dropout: y"), cols
    if residual is not None:
        ldr = _rows(residual, rows, cols, types, d, "dropout: residual")
    drop = _drop(p, rng, d, "dropout") or C.byref(Drop(0.0, None))
    _check(lib().moe_exl3_dropout(dt, x.data_ptr(), ldx, _ptr(residual), ldr, drop, rows, cols, y.data_ptr(), ldy,
                                  _stream(stream, d)), "moe_exl3_dropout")


class W4:
    """A stack of 4-bit matrices: codes uint8 [E][N][K / 2], scales [E][N][K /
    group] of the activations' dtype, zeros uint8 [E][N][K / group] or None (8).
    One matrix may leave out E.  It holds the memory that the tensors have here:
    values written there later count, other memory given to the tensors does not."""

    def __init__(self, codes, scales, zeros=None):
        self._held = tuple(t if t is None else t.detach() if t.dim() == 3 else t.detach()[None]
                           for t in (codes, scales, zeros))
        self.weights = W4Weights(*(_ptr(t) for t in self._held))
        self._checked = None

    codes = property(lambda self: self._held[0])
    scales = property(lambda self: self._held[1])
    zeros = property(lambda self: self._held[2])

    def check(self, desc: W4Desc, device: int, what: str):
        key = (desc.n_in, desc.n_out, desc.n_experts, desc.group, desc.act_dtype, device)
        if self._checked != key:
            u8 = (_torch().uint8,)
            E, N, K, G = desc.n_experts, desc.n_out, desc.n_in, max(1, desc.group)
            _whole(self.codes, (E, N, K // 2), u8, device, what + ": codes")
            _whole(self.scales, (E, N, K // G), _dense_dtypes(desc.act_dtype), device, what + ": scales")
            if self.zeros is not None:
                _whole(self.zeros, (E, N, K // G), u8, device, what + ": zeros")
            self._checked = key
        return C.byref(self.weights)


def make_w4(codes, scales, zeros=None) -> W4:
    return W4(codes, scales, zeros)


def _w4_offsets(desc: W4Desc, offsets, device: int, what: str):
    if offsets is not None:
        return _table(offsets, desc.n_experts + 1, _torch().int32, device, what, "offsets")
    if desc.n_experts != 1:
        raise ValueError(f"{what}: {desc.n_experts} experts need offsets")
    return None


def w4_linear(desc: W4Desc, x, w: W4, y, workspace, offsets=None, base=None, stream=None) -> None:
    """y[r] = x[r] W_e^T + base[r] with 4-bit weights (moe_exl3_w4_linear), e the
    expert of row r: offsets[e] <= r < offsets[e + 1] (int32 [E + 1]; None: one
    expert).  x [rows][n_in], y and base [rows][n_out].  status(workspace)
    reports offsets that descend or leave the rows."""
    d = _dense_device(x, workspace, stream, "w4_linear")
    types, R = _dense_dtypes(desc.act_dtype), x.shape[0]
    ldx, ldy = _rows(x, R, desc.n_in, types, d, "w4_linear: x"), _rows(y, R, desc.n_out, types, d, "w4_linear: y")
    ldb = desc.n_out
    if base is not None:
        ldb = _rows(base, R, desc.n_out, types, d, "w4_linear: base")
    _check(lib().moe_exl3_w4_linear(C.byref(desc), x.data_ptr(), ldx, w.check(desc, d, "w4_linear"),
                                    _w4_offsets(desc, offsets, d, "w4_linear"), _ptr(base), ldb, R, y.data_ptr(), ldy,
                                    workspace.data_ptr(), workspace.nbytes, _stream(stream, d)), "moe_exl3_w4_linear")


def w4_glu(desc: W4Desc, x, w_gate: W4, w_up: W4, h, workspace, offsets=None, stream=None) -> None:
    """h[r] = act(x[r] Wg_e^T) * (x[r] Wu_e^T) with 4-bit weights
    (moe_exl3_w4_glu); otherwise as w4_linear()."""
    d = _dense_device(x, workspace, stream, "w4_glu")
    types, R = _dense_dtypes(desc.act_dtype), x.shape[0]
    ldx, ldh = _rows(x, R, desc.n_in, types, d, "w4_glu: x"), _rows(h, R, desc.n_out, types, d, "w4_glu: h")
    _check(lib().moe_exl3_w4_glu(C.byref(desc), x.data_ptr(), ldx, w_gate.check(desc, d, "w4_glu: w_gate"),
                                 w_up.check(desc, d, "w4_glu: w_up"), _w4_offsets(desc, offsets, d, "w4_glu"), R,
                                 h.data_ptr(), ldh, workspace.data_ptr(), workspace.nbytes, _stream(stream, d)),
           "moe_exl3_w4_glu")
