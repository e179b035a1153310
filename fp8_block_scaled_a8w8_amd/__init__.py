"""Python binding of libgemm_a8w8.so, the a8w8 block-scale GEMM for MI355X (gfx950).

Argument marshalling only: every step of the GEMM runs in the HIP kernels of
the library.  torch supplies device memory and the stream.  The names mirror
the C ABI in ``include/gemm_a8w8_blockscale.h``.

    Y[m,n] = bf16( sum_kb (A_fp8 . W_fp8^T)_kb * a_scale[m,kb] * w_scale[n//128,kb] )

A ``float8_e4m3fn`` (or uint8 bytes) [M,K]; a_scale float32 [M,K/128];
W ``float8_e4m3fn`` (or uint8) [N,K]; w_scale float32 [ceil(N/128),K/128];
Y bfloat16 [M,N].

The MX-scaled variant (``gemm_a8w8_mxscale`` and its batched and packed
forms) takes E8M0 scale bytes instead: a_scale uint8 [M,K/32] (one per row
per 32-wide K group), w_scale uint8 [ceil(N/32),K/32] (one per 32x32 block),
value 2^(e-127).  The row-wise variant (``gemm_a8w8_rowwise``) takes one fp32
scale per activation row (a_scale [M]) and per weight row (w_scale [N]).

Split K across workgroups needs a caller-owned workspace (``Workspace``):
every GEMM function takes ``workspace=``; without one it runs the fastest
plan that splits no K (what the plain C entries run), with one the fastest
plan of the table row (``gemm_a8w8_ex`` in the C ABI).  A workspace serves
calls in stream order; calls that may overlap in time need one each.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgemm_a8w8.so")

A8W8_OK = 0
A8W8_ERR_NULL = 1
A8W8_ERR_SHAPE = 2
A8W8_ERR_ALIGN = 3
A8W8_ERR_ARCH = 4
A8W8_ERR_HIP = 5
A8W8_ERR_PLAN = 6
A8W8_ERR_WORKSPACE = 7
SCALE_KINDS = {"block": 0, "mx": 1, "rowwise": 2}
SCORES = {"softmax": 0, "sigmoid": 1}
ROPE_LAYOUTS = {"halves": 0, "pairs": 1}
KERNEL_NAMES = {1: "skinny", 2: "tile", 3: "ptile", 4: "pskinny", 5: "tall", 6: "rskinny", 7: "sktile"}

EXPORTED = (
    "gemm_a8w8_blockscale",
    "gemm_a8w8_blockscale_plan",
    "gemm_a8w8_num_variants",
    "gemm_a8w8_describe_variant",
    "gemm_a8w8_blockscale_run_variant",
    "gemm_a8w8_variant_name",
    "gemm_a8w8_status_string",
    "gemm_a8w8_table_hash",
    "a8w8_quantize_1x128",
    "gemm_a8w8_blockscale_fused_quant",
    "gemm_a8w8_blockscale_fused_quant_plan",
    "a8w8_prepack_weights",
    "gemm_a8w8_blockscale_packed",
    "gemm_a8w8_blockscale_packed_run_variant",
    "gemm_a8w8_mxscale",
    "gemm_a8w8_mxscale_packed",
    "batched_gemm_a8w8_mxscale",
    "batched_gemm_a8w8_mxscale_packed",
    "gemm_a8w8_mxscale_plan",
    "gemm_a8w8_mxscale_run_variant",
    "gemm_a8w8_rowwise",
    "gemm_a8w8_rowwise_packed",
    "gemm_a8w8_rowwise_run_variant",
    "gemm_a8w8_ex",
    "gemm_a8w8_ex_plan",
    "gemm_a8w8_workspace_init",
    "gemm_a8w8_blockscale_noalloc",
    "a8w8_moe_route",
    "a8w8_moe_layer",
    "a8w8_moe_workspace_bytes",
    "gemm_a8w8_blockscale_lora",
    "gemm_a8w8_blockscale_lora_quantize_1x128",
    "gemm_a8w8_blockscale_lora_workspace_bytes",
    "a8w8_qk_norm_rope",
    "a8w8_paged_attention",
    "a8w8_paged_attention_workspace_bytes",
)


class A8W8Error(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {gemm_a8w8_status_string(status)} (status {status})")


class Plan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("variant", ctypes.c_int32),
                ("bm", ctypes.c_int32), ("bn", ctypes.c_int32),
                ("waves", ctypes.c_int32), ("kblocks", ctypes.c_int32),
                ("kpasses", ctypes.c_int32), ("fallback", ctypes.c_int32),
                ("grid", ctypes.c_int64), ("key_m", ctypes.c_int64),
                ("splits", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("workspace", ctypes.c_int64)]

    def as_dict(self) -> dict:
        d = {f: getattr(self, f) for f, _ in self._fields_ if f != "reserved"}
        d["kernel_name"] = KERNEL_NAMES.get(self.kernel, "?")
        return d


class GemmDesc(ctypes.Structure):
    """a8w8_gemm_desc of the C ABI."""
    _fields_ = [("A", ctypes.c_void_p), ("a_scale", ctypes.c_void_p), ("W", ctypes.c_void_p),
                ("w_scale", ctypes.c_void_p), ("Y", ctypes.c_void_p),
                ("batch", ctypes.c_int64), ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("scale_kind", ctypes.c_int32), ("w_packed", ctypes.c_int32),
                ("variant", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class MoeDesc(ctypes.Structure):
    """a8w8_moe_desc of the C ABI."""
    _fields_ = [("X", ctypes.c_void_p), ("logits", ctypes.c_void_p), ("W13", ctypes.c_void_p),
                ("w13_scale", ctypes.c_void_p), ("W2", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p),
                ("Y", ctypes.c_void_p), ("T", ctypes.c_int64), ("H", ctypes.c_int64), ("I", ctypes.c_int64),
                ("experts", ctypes.c_int32), ("topk", ctypes.c_int32), ("logits_dtype", ctypes.c_int32),
                ("score", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("w_packed", ctypes.c_int32),
                ("scale", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class LoraDesc(ctypes.Structure):
    """a8w8_lora_desc of the C ABI."""
    _fields_ = [("X", ctypes.c_void_p), ("W", ctypes.c_void_p), ("w_scale", ctypes.c_void_p), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("scaling", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("Y", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("adapters", ctypes.c_int32), ("rank", ctypes.c_int32), ("w_packed", ctypes.c_int32),
                ("variant", ctypes.c_int32), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class RopeDesc(ctypes.Structure):
    """a8w8_rope_desc of the C ABI."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64), ("k_row", ctypes.c_int64), ("k_head", ctypes.c_int64),
                ("v_row", ctypes.c_int64), ("v_head", ctypes.c_int64),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("inv_freq", ctypes.c_void_p), ("axis_of", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p), ("k_cache", ctypes.c_void_p),
                ("v_cache", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("T", ctypes.c_int64), ("cache_slots", ctypes.c_int64), ("q_heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("layout", ctypes.c_int32), ("cache_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class AttentionDesc(ctypes.Structure):
    """a8w8_attention_desc of the C ABI."""
    _fields_ = [("q", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("gate_row", ctypes.c_int64), ("gate_head", ctypes.c_int64), ("k_cache", ctypes.c_void_p),
                ("v_cache", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("q_start", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("T", ctypes.c_int64), ("B", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("table_pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("cache_dtype", ctypes.c_int32),
                ("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("scale", ctypes.c_float), ("reserved", ctypes.c_int32), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library.  Raises if it was not built (no fallback path exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                               "(python -m fp8_block_scaled_a8w8_amd.build or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        L.gemm_a8w8_blockscale.restype = ctypes.c_int
        L.gemm_a8w8_blockscale.argtypes = [vp] * 5 + [i64] * 3 + [vp]
        L.gemm_a8w8_blockscale_plan.restype = ctypes.c_int
        L.gemm_a8w8_blockscale_plan.argtypes = [i64, i64, i64, i32, ctypes.POINTER(Plan)]
        L.gemm_a8w8_num_variants.restype = ctypes.c_int
        L.gemm_a8w8_num_variants.argtypes = []
        L.gemm_a8w8_describe_variant.restype = ctypes.c_int
        L.gemm_a8w8_describe_variant.argtypes = [i32, i64, i64, i64, ctypes.POINTER(Plan)]
        L.gemm_a8w8_blockscale_run_variant.restype = ctypes.c_int
        L.gemm_a8w8_blockscale_run_variant.argtypes = [i32] + [vp] * 5 + [i64] * 3 + [vp]
        L.gemm_a8w8_variant_name.restype = ctypes.c_char_p
        L.gemm_a8w8_variant_name.argtypes = [i32]
        L.gemm_a8w8_status_string.restype = ctypes.c_char_p
        L.gemm_a8w8_status_string.argtypes = [ctypes.c_int]
        L.gemm_a8w8_table_hash.restype = ctypes.c_uint64
        L.gemm_a8w8_table_hash.argtypes = []
        L.a8w8_quantize_1x128.restype = ctypes.c_int
        L.a8w8_quantize_1x128.argtypes = [vp] * 3 + [i64] * 2 + [vp]
        L.a8w8_prepack_weights.restype = ctypes.c_int
        L.a8w8_prepack_weights.argtypes = [vp] * 2 + [i64] * 2 + [vp]
        L.gemm_a8w8_blockscale_packed.restype = ctypes.c_int
        L.gemm_a8w8_blockscale_packed.argtypes = [vp] * 5 + [i64] * 3 + [vp]
        L.gemm_a8w8_blockscale_packed_run_variant.restype = ctypes.c_int
        L.gemm_a8w8_blockscale_packed_run_variant.argtypes = [i32] + [vp] * 5 + [i64] * 3 + [vp]
        for name in ("gemm_a8w8_mxscale", "gemm_a8w8_mxscale_packed"):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = [vp] * 5 + [i64] * 3 + [vp]
        for name in ("batched_gemm_a8w8_mxscale", "batched_gemm_a8w8_mxscale_packed"):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = [vp] * 5 + [i64] * 4 + [vp]
        L.gemm_a8w8_mxscale_plan.restype = ctypes.c_int
        L.gemm_a8w8_mxscale_plan.argtypes = [i64, i64, i64, i32, ctypes.POINTER(Plan)]
        for name in ("gemm_a8w8_rowwise", "gemm_a8w8_rowwise_packed"):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = [vp] * 5 + [i64] * 3 + [vp]
        L.gemm_a8w8_rowwise_run_variant.restype = ctypes.c_int
        L.gemm_a8w8_rowwise_run_variant.argtypes = [i32] + [vp] * 5 + [i64] * 3 + [i32, vp]
        L.gemm_a8w8_mxscale_run_variant.restype = ctypes.c_int
        L.gemm_a8w8_mxscale_run_variant.argtypes = [i32] + [vp] * 5 + [i64] * 4 + [i32, vp]
        L.gemm_a8w8_ex.restype = ctypes.c_int
        L.gemm_a8w8_ex.argtypes = [ctypes.POINTER(GemmDesc), vp]
        L.gemm_a8w8_ex_plan.restype = ctypes.c_int
        L.gemm_a8w8_ex_plan.argtypes = [ctypes.POINTER(GemmDesc), i32, ctypes.POINTER(Plan)]
        L.gemm_a8w8_workspace_init.restype = ctypes.c_int
        L.gemm_a8w8_workspace_init.argtypes = [vp, i64, vp]
        L.gemm_a8w8_blockscale_noalloc.restype = ctypes.c_int
        L.gemm_a8w8_blockscale_noalloc.argtypes = [vp] * 5 + [i64] * 3 + [vp]
        L.gemm_a8w8_blockscale_fused_quant.restype = ctypes.c_int
        L.gemm_a8w8_blockscale_fused_quant.argtypes = [vp] * 4 + [i64] * 3 + [i32, i32, vp]
        L.gemm_a8w8_blockscale_fused_quant_plan.restype = ctypes.c_int
        L.gemm_a8w8_blockscale_fused_quant_plan.argtypes = [i64, i64, i64, i32, i32, ctypes.POINTER(Plan)]
        L.a8w8_moe_route.restype = ctypes.c_int
        L.a8w8_moe_route.argtypes = [vp, i32, i64, i64, i32, i32, i32, ctypes.c_float, vp, vp, vp]
        L.a8w8_moe_layer.restype = ctypes.c_int
        L.a8w8_moe_layer.argtypes = [ctypes.POINTER(MoeDesc), vp]
        L.a8w8_moe_workspace_bytes.restype = ctypes.c_int
        L.a8w8_moe_workspace_bytes.argtypes = [i64, i32, i32, i64, i64, i32, ctypes.POINTER(i64)]
        for f in (L.gemm_a8w8_blockscale_lora, L.gemm_a8w8_blockscale_lora_quantize_1x128):
            f.restype = ctypes.c_int
            f.argtypes = [ctypes.POINTER(LoraDesc), vp]
        L.gemm_a8w8_blockscale_lora_workspace_bytes.restype = ctypes.c_int
        L.gemm_a8w8_blockscale_lora_workspace_bytes.argtypes = [i64, i64, i64, i32, i32, ctypes.POINTER(i64)]
        L.a8w8_qk_norm_rope.restype = ctypes.c_int
        L.a8w8_qk_norm_rope.argtypes = [ctypes.POINTER(RopeDesc), vp]
        L.a8w8_paged_attention.restype = ctypes.c_int
        L.a8w8_paged_attention.argtypes = [ctypes.POINTER(AttentionDesc), vp]
        L.a8w8_paged_attention_workspace_bytes.restype = ctypes.c_int
        L.a8w8_paged_attention_workspace_bytes.argtypes = [i64, i64] + [i32] * 5 + [ctypes.POINTER(i64)]
        _lib = L
    return _lib


def gemm_a8w8_status_string(status: int) -> str:
    return lib().gemm_a8w8_status_string(int(status)).decode()


def gemm_a8w8_variant_name(variant: int) -> str | None:
    r = lib().gemm_a8w8_variant_name(int(variant))
    return r.decode() if r is not None else None


def gemm_a8w8_table_hash() -> int:
    return int(lib().gemm_a8w8_table_hash())


def gemm_a8w8_num_variants() -> int:
    return int(lib().gemm_a8w8_num_variants())


def gemm_a8w8_blockscale_plan(M: int, N: int, K: int, cu_count: int = 0) -> dict:
    p = Plan()
    rc = lib().gemm_a8w8_blockscale_plan(M, N, K, cu_count, ctypes.byref(p))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "gemm_a8w8_blockscale_plan")
    d = p.as_dict()
    d["name"] = gemm_a8w8_variant_name(d["variant"])
    return d


def gemm_a8w8_describe_variant(variant: int, M: int = 0, N: int = 1, K: int = 128) -> dict:
    p = Plan()
    rc = lib().gemm_a8w8_describe_variant(variant, M, N, K, ctypes.byref(p))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "gemm_a8w8_describe_variant")
    d = p.as_dict()
    d["name"] = gemm_a8w8_variant_name(variant)
    return d


# The current stream's handle without a Stream object around it (0.1 against 2.8 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _check_device(named, device) -> None:
    """Every tensor contiguous, on the GPU, on `device`, which must be the current device (the
    library launches on the current device)."""
    for name, t in named:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous GPU tensor")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, the other operands on {device}")
    if device.index is not None and device.index != torch.cuda.current_device():
        raise ValueError(f"operands are on {device} but the current device is cuda:{torch.cuda.current_device()}")


def _out(out, shape, device, what="out"):
    if out is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=device)
    if out.dtype != torch.bfloat16 or tuple(out.shape) != tuple(shape):
        raise ValueError(f"{what} must be a contiguous bfloat16 {tuple(shape)} tensor")
    _check_device(((what, out),), device)
    return out


def _check(A, a_scale, W, w_scale, out):
    if A.dtype not in (torch.float8_e4m3fn, torch.uint8) or W.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError("A and W must be float8_e4m3fn (or raw uint8 bytes)")
    if a_scale.dtype != torch.float32 or w_scale.dtype != torch.float32:
        raise TypeError("scales must be float32")
    if A.dim() != 2 or W.dim() != 2:
        raise ValueError("A and W must be 2-D")
    M, K = A.shape
    N, K2 = W.shape
    if K2 != K:
        raise ValueError(f"A is [M,{K}] but W is [N,{K2}]")
    if K % 128:
        raise ValueError("K must be a multiple of 128")
    KB, NB = K // 128, (N + 127) // 128
    if tuple(a_scale.shape) != (M, KB) or tuple(w_scale.shape) != (NB, KB):
        raise ValueError(f"scale shapes must be [{M},{KB}] and [{NB},{KB}], got "
                         f"{tuple(a_scale.shape)} and {tuple(w_scale.shape)}")
    _check_device((("A", A), ("a_scale", a_scale), ("W", W), ("w_scale", w_scale)), A.device)
    out = _out(out, (M, N), A.device)
    return M, N, K, out


class Workspace:
    """Split-K workspace: caller-owned device memory that split plans use for their fp32 partial
    tiles and per-tile counters.  Allocated here by torch (device memory is torch's part) and
    zero-filled once by the library's own kernel (gemm_a8w8_workspace_init); every call leaves it
    ready for the next.  Calls using one workspace must run in stream order (one stream, or
    properly ordered streams); calls or graph replays that may overlap in time need one each."""

    def __init__(self, nbytes: int = 64 << 20, device=None, stream=None):
        nbytes = max(256, (int(nbytes) + 255) // 256 * 256)
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device if device is not None else "cuda")
        self.nbytes = nbytes
        rc = lib().gemm_a8w8_workspace_init(self.buf.data_ptr(), nbytes, _stream_handle(stream))
        if rc != A8W8_OK:
            raise A8W8Error(rc, "gemm_a8w8_workspace_init")

    def ptr(self) -> int:
        return self.buf.data_ptr()


def _desc(A, a_scale, W, w_scale, out, batch, M, N, K, kind, w_packed, variant, workspace) -> GemmDesc:
    if workspace is not None and workspace.buf.device != A.device:
        raise ValueError(f"the workspace is on {workspace.buf.device}, the operands on {A.device}")
    return GemmDesc(A.data_ptr(), a_scale.data_ptr(), W.data_ptr(), w_scale.data_ptr(), out.data_ptr(),
                    batch, M, N, K, SCALE_KINDS[kind], 1 if w_packed else 0, -1 if variant is None else int(variant),
                    0, workspace.ptr() if workspace is not None else None,
                    workspace.nbytes if workspace is not None else 0)


def _ex_launch(desc: GemmDesc, stream, what: str) -> None:
    rc = lib().gemm_a8w8_ex(ctypes.byref(desc), _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, what)


def gemm_a8w8_blockscale(A: torch.Tensor, a_scale: torch.Tensor, W: torch.Tensor,
                         w_scale: torch.Tensor, out: torch.Tensor | None = None,
                         stream=None, workspace: Workspace | None = None) -> torch.Tensor:
    """Y = A . W^T with 1x128 activation / 128x128 weight fp32 block scales; returns bf16 [M,N].
    With a workspace the call may split K across workgroups (gemm_a8w8_ex)."""
    M, N, K, out = _check(A, a_scale, W, w_scale, out)
    if workspace is not None:
        _ex_launch(_desc(A, a_scale, W, w_scale, out, 1, M, N, K, "block", False, None, workspace), stream,
                   "gemm_a8w8_ex")
        return out
    rc = lib().gemm_a8w8_blockscale(A.data_ptr(), a_scale.data_ptr(), W.data_ptr(),
                                    w_scale.data_ptr(), out.data_ptr(), M, N, K,
                                    _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "gemm_a8w8_blockscale")
    return out


def gemm_a8w8_blockscale_noalloc(A, a_scale, W, w_scale, out=None, stream=None) -> torch.Tensor:
    """gemm_a8w8_blockscale_noalloc of the C ABI: the table's fastest plan (split K included) with
    the library's static scratch as workspace; the C call allocates nothing (``out`` may be given
    so that nothing is allocated here either).  Calls overlapping in time on one GPU race."""
    M, N, K, out = _check(A, a_scale, W, w_scale, out)
    rc = lib().gemm_a8w8_blockscale_noalloc(A.data_ptr(), a_scale.data_ptr(), W.data_ptr(), w_scale.data_ptr(),
                                            out.data_ptr(), M, N, K, _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "gemm_a8w8_blockscale_noalloc")
    return out


def gemm_a8w8_blockscale_run_variant(variant: int, A, a_scale, W, w_scale, out=None, stream=None, workspace=None):
    """Same as gemm_a8w8_blockscale with a fixed kernel instance (tuning and tests); split
    instances need a workspace."""
    M, N, K, out = _check(A, a_scale, W, w_scale, out)
    if workspace is not None:
        _ex_launch(_desc(A, a_scale, W, w_scale, out, 1, M, N, K, "block", False, variant, workspace), stream,
                   f"gemm_a8w8_ex(variant {variant})")
        return out
    rc = lib().gemm_a8w8_blockscale_run_variant(variant, A.data_ptr(), a_scale.data_ptr(),
                                                W.data_ptr(), w_scale.data_ptr(), out.data_ptr(),
                                                M, N, K, _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, f"gemm_a8w8_blockscale_run_variant({variant})")
    return out


def gemm_a8w8_ex(A, a_scale, W, w_scale, *, scale_kind: str = "block", packed_n: int | None = None,
                 variant: int | None = None, workspace: Workspace | None = None, out=None, stream=None):
    """gemm_a8w8_ex of the C ABI: any scale kind ("block", "mx", "rowwise"), row-major or packed W
    (packed_n = real row count), 2-D operands or batched 3-D MX operands, an optional forced
    instance and an optional workspace (split-K and stream-K plans)."""
    if scale_kind == "mx":
        batched = A.dim() == 3
        batch, M, N, K, out = _check_mx(A, a_scale, W, w_scale, out, batched, packed_n)
    elif scale_kind == "rowwise":
        M, N, K, out = _check_rowwise(A, a_scale, W, w_scale, out, packed_n)
        batch = 1
    elif scale_kind == "block":
        Wc = W if packed_n is None else _packed_view(W, packed_n)
        M, N, K, out = _check(A, a_scale, Wc, w_scale, out)
        batch = 1
    else:
        raise ValueError(f"scale_kind must be one of {sorted(SCALE_KINDS)}")
    _ex_launch(_desc(A, a_scale, W, w_scale, out, batch, M, N, K, scale_kind, packed_n is not None, variant,
                     workspace), stream, "gemm_a8w8_ex")
    return out


def gemm_a8w8_ex_plan(M: int, N: int, K: int, *, scale_kind: str = "block", batch: int = 1,
                      variant: int | None = None, workspace_bytes: int = 0, cu_count: int = 0,
                      packed: bool = False) -> dict:
    """The plan gemm_a8w8_ex launches for this shape with `workspace_bytes` of workspace
    (host only; packed: weights in the packed layout); plan["workspace"] is the workspace it uses."""
    d = GemmDesc(None, None, None, None, None, batch, M, N, K, SCALE_KINDS[scale_kind], 1 if packed else 0,
                 -1 if variant is None else int(variant), 0, None, int(workspace_bytes))
    p = Plan()
    rc = lib().gemm_a8w8_ex_plan(ctypes.byref(d), cu_count, ctypes.byref(p))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "gemm_a8w8_ex_plan")
    r = p.as_dict()
    r["name"] = gemm_a8w8_variant_name(r["variant"])
    return r


def quantize_1x128(X: torch.Tensor, out: torch.Tensor | None = None, scale_out: torch.Tensor | None = None,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """bf16 activations [M,K] -> (e4m3fn codes [M,K], fp32 scales [M,K/128]), one scale per 1x128 group.

    The A / a_scale operands of gemm_a8w8_blockscale (see a8w8_quantize_1x128 in the C header)."""
    if X.dtype != torch.bfloat16 or X.dim() != 2:
        raise ValueError("X must be a contiguous bfloat16 [M,K] GPU tensor")
    _check_device((("X", X),), X.device)
    M, K = X.shape
    if K % 128:
        raise ValueError("K must be a multiple of 128")
    if out is None:
        out = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=X.device)
    elif out.dtype not in (torch.float8_e4m3fn, torch.uint8) or tuple(out.shape) != (M, K):
        raise ValueError("out must be a contiguous float8_e4m3fn (or uint8) [M,K] tensor")
    if scale_out is None:
        scale_out = torch.empty((M, K // 128), dtype=torch.float32, device=X.device)
    elif scale_out.dtype != torch.float32 or tuple(scale_out.shape) != (M, K // 128):
        raise ValueError("scale_out must be a contiguous float32 [M,K/128] tensor")
    _check_device((("out", out), ("scale_out", scale_out)), X.device)
    rc = lib().a8w8_quantize_1x128(X.data_ptr(), out.data_ptr(), scale_out.data_ptr(), M, K, _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "a8w8_quantize_1x128")
    return out, scale_out


def gemm_a8w8_blockscale_fused_quant(X: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor,
                                     out: torch.Tensor | None = None, *, packed_n: int | None = None,
                                     variant: int | None = None, stream=None) -> torch.Tensor:
    """Decode (M <= 16): bf16 X [M,K] quantised per 1x128 group inside the GEMM kernel, times the
    block-scaled W; bitwise equal to quantize_1x128 then gemm_a8w8_blockscale_run_variant with the
    instance gemm_a8w8_blockscale_fused_quant_plan reports.  ``packed_n``: W is in the packed
    layout (prepack_weights) for N = packed_n rows."""
    if X.dtype != torch.bfloat16 or X.dim() != 2:
        raise ValueError("X must be a contiguous bfloat16 [M,K] GPU tensor")
    if W.dtype not in (torch.float8_e4m3fn, torch.uint8) or W.dim() != 2:
        raise TypeError("W must be a 2-D float8_e4m3fn (or raw uint8) tensor")
    if w_scale.dtype != torch.float32:
        raise TypeError("w_scale must be float32")
    Wv = W if packed_n is None else _packed_view(W, packed_n)
    M, K = X.shape
    N, K2 = Wv.shape
    if K2 != K or K % 128:
        raise ValueError(f"X is [M,{K}] and W is [N,{K2}]: K must agree and be a multiple of 128")
    if tuple(w_scale.shape) != ((N + 127) // 128, K // 128):
        raise ValueError(f"w_scale must be [{(N + 127) // 128},{K // 128}], got {tuple(w_scale.shape)}")
    _check_device((("X", X), ("W", W), ("w_scale", w_scale)), X.device)
    out = _out(out, (M, N), X.device)
    rc = lib().gemm_a8w8_blockscale_fused_quant(X.data_ptr(), W.data_ptr(), w_scale.data_ptr(), out.data_ptr(),
                                                M, N, K, 0 if packed_n is None else 1,
                                                -1 if variant is None else int(variant), _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "gemm_a8w8_blockscale_fused_quant")
    return out


def gemm_a8w8_blockscale_fused_quant_plan(M: int, N: int, K: int, cu_count: int = 0,
                                          variant: int | None = None) -> dict:
    p = Plan()
    rc = lib().gemm_a8w8_blockscale_fused_quant_plan(M, N, K, cu_count, -1 if variant is None else int(variant),
                                                     ctypes.byref(p))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "gemm_a8w8_blockscale_fused_quant_plan")
    d = p.as_dict()
    d["name"] = gemm_a8w8_variant_name(d["variant"])
    return d


def packed_rows(N: int) -> int:
    """Rows of the packed weight layout: N padded to a multiple of 16."""
    return (N + 15) // 16 * 16


def prepack_weights(W: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Row-major e4m3fn W [N,K] -> the packed layout (uint8 [16*ceil(N/16), K]); see the C header."""
    if W.dtype not in (torch.float8_e4m3fn, torch.uint8) or W.dim() != 2:
        raise ValueError("W must be a contiguous float8_e4m3fn (or uint8) [N,K] GPU tensor")
    _check_device((("W", W),), W.device)
    N, K = W.shape
    if K % 128:
        raise ValueError("K must be a multiple of 128")
    if out is None:
        out = torch.empty((packed_rows(N), K), dtype=torch.uint8, device=W.device)
    elif tuple(out.shape) != (packed_rows(N), K) or out.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise ValueError(f"out must be a contiguous uint8 [{packed_rows(N)},{K}] tensor")
    _check_device((("out", out),), W.device)
    rc = lib().a8w8_prepack_weights(W.data_ptr(), out.data_ptr(), N, K, _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "a8w8_prepack_weights")
    return out


def _packed_view(Wp, N):
    if Wp.dtype not in (torch.float8_e4m3fn, torch.uint8) or Wp.dim() != 2:
        raise TypeError("Wp must be a 2-D uint8 (or float8_e4m3fn) tensor")
    if Wp.shape[0] != packed_rows(N):
        raise ValueError(f"packed weights for N={N} have {packed_rows(N)} rows, got {Wp.shape[0]}")
    if not Wp.is_contiguous():
        raise ValueError("Wp must be a contiguous GPU tensor")
    return Wp[:N]


def _check_packed(A, a_scale, Wp, w_scale, N, out):
    return _check(A, a_scale, _packed_view(Wp, N), w_scale, out)


def gemm_a8w8_blockscale_packed(A: torch.Tensor, a_scale: torch.Tensor, Wp: torch.Tensor, w_scale: torch.Tensor,
                                N: int, out: torch.Tensor | None = None, stream=None,
                                workspace: Workspace | None = None) -> torch.Tensor:
    """Same result as gemm_a8w8_blockscale, with W given in the packed layout (prepack_weights)."""
    M, N, K, out = _check_packed(A, a_scale, Wp, w_scale, N, out)
    if workspace is not None:
        _ex_launch(_desc(A, a_scale, Wp, w_scale, out, 1, M, N, K, "block", True, None, workspace), stream,
                   "gemm_a8w8_ex")
        return out
    rc = lib().gemm_a8w8_blockscale_packed(A.data_ptr(), a_scale.data_ptr(), Wp.data_ptr(), w_scale.data_ptr(),
                                           out.data_ptr(), M, N, K, _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "gemm_a8w8_blockscale_packed")
    return out


def gemm_a8w8_blockscale_packed_run_variant(variant: int, A, a_scale, Wp, w_scale, N: int, out=None, stream=None,
                                            workspace=None):
    """gemm_a8w8_blockscale_packed with a fixed kernel instance (tuning and tests)."""
    M, N, K, out = _check_packed(A, a_scale, Wp, w_scale, N, out)
    if workspace is not None:
        _ex_launch(_desc(A, a_scale, Wp, w_scale, out, 1, M, N, K, "block", True, variant, workspace), stream,
                   f"gemm_a8w8_ex(variant {variant})")
        return out
    rc = lib().gemm_a8w8_blockscale_packed_run_variant(variant, A.data_ptr(), a_scale.data_ptr(), Wp.data_ptr(),
                                                       w_scale.data_ptr(), out.data_ptr(), M, N, K,
                                                       _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, f"gemm_a8w8_blockscale_packed_run_variant({variant})")
    return out


def variants() -> list[dict]:
    """Descriptions of every compiled kernel instance."""
    return [gemm_a8w8_describe_variant(i) for i in range(gemm_a8w8_num_variants())]


# ---------------------------------------------------------------------------
# MX-scaled variant (E8M0 scales: 1x32 activation groups, 32x32 weight blocks)

_E8M0_DTYPES = tuple(d for d in (torch.uint8, getattr(torch, "float8_e8m0fnu", None)) if d is not None)


def _check_mx(A, a_scale, W, w_scale, out, batched: bool, N: int | None = None):
    """Validate MX operands; W is row-major [.., N, K] or (N given) packed [.., 16*ceil(N/16), K]."""
    nd = 3 if batched else 2
    for name, t in (("A", A), ("W", W)):
        if t.dtype not in (torch.float8_e4m3fn, torch.uint8) or t.dim() != nd:
            raise TypeError(f"{name} must be a {nd}-D float8_e4m3fn (or uint8) tensor")
    for name, t in (("a_scale", a_scale), ("w_scale", w_scale)):
        if t.dtype not in _E8M0_DTYPES or t.dim() != nd:
            raise TypeError(f"{name} must be a {nd}-D uint8 (E8M0 code) tensor")
    batch = A.shape[0] if batched else 1
    M, K = A.shape[-2:]
    rows, K2 = W.shape[-2:]
    if N is None:
        N = rows
    elif rows != packed_rows(N):
        raise ValueError(f"packed weights for N={N} have {packed_rows(N)} rows, got {rows}")
    if K2 != K:
        raise ValueError(f"A is [..,M,{K}] but W is [..,N,{K2}]")
    if K % 128:
        raise ValueError("K must be a multiple of 128")
    lead = (batch,) if batched else ()
    if batched and (W.shape[0] != batch or a_scale.shape[0] != batch or w_scale.shape[0] != batch):
        raise ValueError("every operand needs the same batch count")
    if tuple(a_scale.shape) != lead + (M, K // 32) or tuple(w_scale.shape) != lead + ((N + 31) // 32, K // 32):
        raise ValueError(f"MX scale shapes must be {lead + (M, K // 32)} and {lead + ((N + 31) // 32, K // 32)}, "
                         f"got {tuple(a_scale.shape)} and {tuple(w_scale.shape)}")
    _check_device((("A", A), ("a_scale", a_scale), ("W", W), ("w_scale", w_scale)), A.device)
    out = _out(out, lead + (M, N), A.device)
    return batch, M, N, K, out


def _mx_call(name, A, a_scale, W, w_scale, out, batched, N, stream, workspace=None):
    packed = N is not None
    batch, M, N, K, out = _check_mx(A, a_scale, W, w_scale, out, batched, N)
    if workspace is not None:
        _ex_launch(_desc(A, a_scale, W, w_scale, out, batch, M, N, K, "mx", packed, None, workspace), stream,
                   "gemm_a8w8_ex")
        return out
    args = [A.data_ptr(), a_scale.data_ptr(), W.data_ptr(), w_scale.data_ptr(), out.data_ptr()]
    args += [batch, M, N, K] if batched else [M, N, K]
    rc = getattr(lib(), name)(*args, _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, name)
    return out


def gemm_a8w8_mxscale(A, a_scale, W, w_scale, out=None, stream=None, workspace=None) -> torch.Tensor:
    """MX-scaled Y = A . W^T (E8M0 scales per 1x32 activation group and 32x32 weight block); bf16 [M,N]."""
    return _mx_call("gemm_a8w8_mxscale", A, a_scale, W, w_scale, out, False, None, stream, workspace)


def gemm_a8w8_mxscale_packed(A, a_scale, Wp, w_scale, N: int, out=None, stream=None, workspace=None) -> torch.Tensor:
    """gemm_a8w8_mxscale with W in the packed layout (prepack_weights)."""
    return _mx_call("gemm_a8w8_mxscale_packed", A, a_scale, Wp, w_scale, out, False, N, stream, workspace)


def batched_gemm_a8w8_mxscale(A, a_scale, W, w_scale, out=None, stream=None, workspace=None) -> torch.Tensor:
    """Batched MX GEMM: A [b,M,K], a_scale [b,M,K/32], W [b,N,K], w_scale [b,ceil(N/32),K/32] -> bf16 [b,M,N]."""
    return _mx_call("batched_gemm_a8w8_mxscale", A, a_scale, W, w_scale, out, True, None, stream, workspace)


def batched_gemm_a8w8_mxscale_packed(A, a_scale, Wp, w_scale, N: int, out=None, stream=None, workspace=None) -> torch.Tensor:
    """batched_gemm_a8w8_mxscale with each batch's W packed (Wp [b,16*ceil(N/16),K])."""
    return _mx_call("batched_gemm_a8w8_mxscale_packed", A, a_scale, Wp, w_scale, out, True, N, stream, workspace)


def gemm_a8w8_mxscale_plan(M: int, N: int, K: int, cu_count: int = 0) -> dict:
    p = Plan()
    rc = lib().gemm_a8w8_mxscale_plan(M, N, K, cu_count, ctypes.byref(p))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "gemm_a8w8_mxscale_plan")
    d = p.as_dict()
    d["name"] = gemm_a8w8_variant_name(d["variant"])
    return d


def gemm_a8w8_mxscale_run_variant(variant: int, A, a_scale, W, w_scale, out=None, stream=None,
                                  packed_n: int | None = None, workspace=None) -> torch.Tensor:
    """MX GEMM with a fixed kernel instance; 2-D operands or 3-D (batched); packed W when packed_n is given."""
    batched = A.dim() == 3
    batch, M, N, K, out = _check_mx(A, a_scale, W, w_scale, out, batched, packed_n)
    if workspace is not None:
        _ex_launch(_desc(A, a_scale, W, w_scale, out, batch, M, N, K, "mx", packed_n is not None, variant,
                         workspace), stream, f"gemm_a8w8_ex(variant {variant})")
        return out
    rc = lib().gemm_a8w8_mxscale_run_variant(variant, A.data_ptr(), a_scale.data_ptr(), W.data_ptr(),
                                             w_scale.data_ptr(), out.data_ptr(), batch, M, N, K,
                                             1 if packed_n is not None else 0, _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, f"gemm_a8w8_mxscale_run_variant({variant})")
    return out


# ---------------------------------------------------------------------------
# Row-wise variant (fp32 scale per activation row and per weight row)

def _check_rowwise(A, a_scale, W, w_scale, out, N=None):
    for name, t in (("A", A), ("W", W)):
        if t.dtype not in (torch.float8_e4m3fn, torch.uint8) or t.dim() != 2:
            raise TypeError(f"{name} must be a 2-D float8_e4m3fn (or uint8) tensor")
    M, K = A.shape
    rows, K2 = W.shape
    if N is None:
        N = rows
    elif rows != packed_rows(N):
        raise ValueError(f"packed weights for N={N} have {packed_rows(N)} rows, got {rows}")
    if K2 != K or K % 128:
        raise ValueError("A and W must agree on K, a multiple of 128")
    if a_scale.dtype != torch.float32 or w_scale.dtype != torch.float32 or \
            tuple(a_scale.shape) != (M,) or tuple(w_scale.shape) != (N,):
        raise ValueError(f"row-wise scales must be float32 [{M}] and [{N}]")
    _check_device((("A", A), ("a_scale", a_scale), ("W", W), ("w_scale", w_scale)), A.device)
    out = _out(out, (M, N), A.device)
    return M, N, K, out


def gemm_a8w8_rowwise(A, a_scale, W, w_scale, out=None, stream=None, workspace=None) -> torch.Tensor:
    """Row-wise scaled Y = a_scale[m] * w_scale[n] * (A . W^T) (per-token / per-channel); bf16 [M,N]."""
    M, N, K, out = _check_rowwise(A, a_scale, W, w_scale, out)
    if workspace is not None:
        _ex_launch(_desc(A, a_scale, W, w_scale, out, 1, M, N, K, "rowwise", False, None, workspace), stream,
                   "gemm_a8w8_ex")
        return out
    rc = lib().gemm_a8w8_rowwise(A.data_ptr(), a_scale.data_ptr(), W.data_ptr(), w_scale.data_ptr(),
                                 out.data_ptr(), M, N, K, _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "gemm_a8w8_rowwise")
    return out


def gemm_a8w8_rowwise_packed(A, a_scale, Wp, w_scale, N: int, out=None, stream=None,
                             workspace=None) -> torch.Tensor:
    """gemm_a8w8_rowwise with W in the packed layout (prepack_weights)."""
    M, N, K, out = _check_rowwise(A, a_scale, Wp, w_scale, out, N)
    if workspace is not None:
        _ex_launch(_desc(A, a_scale, Wp, w_scale, out, 1, M, N, K, "rowwise", True, None, workspace), stream,
                   "gemm_a8w8_ex")
        return out
    rc = lib().gemm_a8w8_rowwise_packed(A.data_ptr(), a_scale.data_ptr(), Wp.data_ptr(), w_scale.data_ptr(),
                                        out.data_ptr(), M, N, K, _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "gemm_a8w8_rowwise_packed")
    return out


def gemm_a8w8_rowwise_run_variant(variant: int, A, a_scale, W, w_scale, out=None, stream=None,
                                  packed_n: int | None = None, workspace=None) -> torch.Tensor:
    """Row-wise GEMM with a fixed kernel instance; packed W when packed_n is given."""
    M, N, K, out = _check_rowwise(A, a_scale, W, w_scale, out, packed_n)
    if workspace is not None:
        _ex_launch(_desc(A, a_scale, W, w_scale, out, 1, M, N, K, "rowwise", packed_n is not None, variant,
                         workspace), stream, f"gemm_a8w8_ex(variant {variant})")
        return out
    rc = lib().gemm_a8w8_rowwise_run_variant(variant, A.data_ptr(), a_scale.data_ptr(), W.data_ptr(),
                                             w_scale.data_ptr(), out.data_ptr(), M, N, K,
                                             1 if packed_n is not None else 0, _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, f"gemm_a8w8_rowwise_run_variant({variant})")
    return out


# ---------------------------------------------------------------------------
# Mixture of experts for a few tokens: routing, and the whole layer on fp8
# block-scaled expert weights

def _check_logits(logits: torch.Tensor) -> int:
    if logits.dim() != 2 or logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("logits must be a contiguous float32 or bfloat16 [T,E] GPU tensor")
    return 1 if logits.dtype == torch.bfloat16 else 0


def _score(score: str) -> int:
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}")
    return SCORES[score]


def moe_route(logits: torch.Tensor, topk: int, *, score: str = "softmax", renormalize: bool = True,
              scale: float = 1.0, weights_out: torch.Tensor | None = None, ids_out: torch.Tensor | None = None,
              stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The topk experts of each token's logits [T,E] (float32 or bfloat16): (weights float32 [T,topk], ids
    int32 [T,topk]), best first, ties to the lowest index.  Weights are the softmax over the row or the
    sigmoid of the chosen logits, divided by the chosen ones' sum if ``renormalize``, times ``scale``.  A
    logit of -inf or NaN masks its expert; slots left without one have id -1 and weight 0."""
    dtype, sc = _check_logits(logits), _score(score)
    _check_device((("logits", logits),), logits.device)
    T, E = logits.shape
    if weights_out is None:
        weights_out = torch.empty((T, topk), dtype=torch.float32, device=logits.device)
    elif weights_out.dtype != torch.float32 or tuple(weights_out.shape) != (T, topk):
        raise ValueError(f"weights_out must be a contiguous float32 [{T},{topk}] tensor")
    else:
        _check_device((("weights_out", weights_out),), logits.device)
    if ids_out is None:
        ids_out = torch.empty((T, topk), dtype=torch.int32, device=logits.device)
    elif ids_out.dtype != torch.int32 or tuple(ids_out.shape) != (T, topk):
        raise ValueError(f"ids_out must be a contiguous int32 [{T},{topk}] tensor")
    else:
        _check_device((("ids_out", ids_out),), logits.device)
    rc = lib().a8w8_moe_route(logits.data_ptr(), dtype, T, E, topk, sc, 1 if renormalize else 0, scale,
                              weights_out.data_ptr(), ids_out.data_ptr(), _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "a8w8_moe_route")
    return weights_out, ids_out


class MoeExperts:
    """The weights of a mixture-of-experts layer, checked once and kept by the caller's program.

    W13 float8_e4m3fn (or uint8) [E,2I,H] (each expert's I gate rows, then its I up rows) with w13_scale
    float32 [E,2I/128,H/128]; W2 [E,H,I] with w2_scale float32 [E,H/128,I/128]; one scale per 128x128 block.
    ``packed``: W13 and W2 are in the packed layout (``MoeExperts.pack`` or prepack_weights on the experts'
    rows one after another)."""

    def __init__(self, W13, w13_scale, W2, w2_scale, packed: bool = False):
        for name, w in (("W13", W13), ("W2", W2)):
            if w.dtype not in (torch.float8_e4m3fn, torch.uint8) or w.dim() != 3:
                raise TypeError(f"{name} must be a 3-D float8_e4m3fn (or raw uint8) tensor")
        if w13_scale.dtype != torch.float32 or w2_scale.dtype != torch.float32:
            raise TypeError("scales must be float32")
        E, I2, H = W13.shape
        I = I2 // 2
        if I2 % 256 or H % 128 or I2 == 0 or H == 0:
            raise ValueError(f"W13 is [E,2I,H] with H and I multiples of 128, got {tuple(W13.shape)}")
        if tuple(W2.shape) != (E, H, I):
            raise ValueError(f"W2 must be [{E},{H},{I}], got {tuple(W2.shape)}")
        if tuple(w13_scale.shape) != (E, I2 // 128, H // 128) or tuple(w2_scale.shape) != (E, H // 128, I // 128):
            raise ValueError(f"scale shapes must be {(E, I2 // 128, H // 128)} and {(E, H // 128, I // 128)}, got "
                             f"{tuple(w13_scale.shape)} and {tuple(w2_scale.shape)}")
        _check_device((("W13", W13), ("w13_scale", w13_scale), ("W2", W2), ("w2_scale", w2_scale)), W13.device)
        self.W13, self.w13_scale, self.W2, self.w2_scale = W13, w13_scale, W2, w2_scale
        self.E, self.H, self.I, self.packed, self.device = E, H, I, bool(packed), W13.device

    @classmethod
    def pack(cls, W13, w13_scale, W2, w2_scale, stream=None) -> "MoeExperts":
        """Row-major weights converted to the packed layout."""
        e = cls(W13, w13_scale, W2, w2_scale)
        packed = [prepack_weights(w.reshape(-1, w.shape[2]), stream=stream).view(w.shape) for w in (W13, W2)]
        return cls(packed[0], e.w13_scale, packed[1], e.w2_scale, packed=True)


def moe_workspace_bytes(T: int, topk: int, experts: MoeExperts, cu_count: int = 0) -> int:
    """Workspace bytes moe_layer_a16w8_blockscale needs for any number of tokens up to T (Workspace(nbytes))."""
    n = ctypes.c_int64(0)
    rc = lib().a8w8_moe_workspace_bytes(T, topk, experts.E, experts.H, experts.I, cu_count, ctypes.byref(n))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "a8w8_moe_workspace_bytes")
    return n.value


def moe_layer_a16w8_blockscale(X: torch.Tensor, logits: torch.Tensor, experts: MoeExperts, topk: int,
                               workspace: Workspace, *, score: str = "softmax", renormalize: bool = True,
                               scale: float = 1.0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """A whole mixture-of-experts layer for a few tokens: X bf16 [T,H] routed by logits [T,E] as moe_route
    does it, Y[t] = sum_j w[t,j] W2[e] (silu(W13[e] gate . x_t) * (W13[e] up . x_t)); returns bf16 [T,H].
    Activations stay bf16; the workspace needs moe_workspace_bytes."""
    dtype, sc = _check_logits(logits), _score(score)
    if X.dtype != torch.bfloat16 or X.dim() != 2:
        raise ValueError("X must be a contiguous bfloat16 [T,H] GPU tensor")
    T, H = X.shape
    if H != experts.H or tuple(logits.shape) != (T, experts.E):
        raise ValueError(f"X must be [T,{experts.H}] and logits [T,{experts.E}], got {tuple(X.shape)} and "
                         f"{tuple(logits.shape)}")
    _check_device((("X", X), ("logits", logits)), experts.device)
    if workspace.buf.device != X.device:
        raise ValueError(f"the workspace is on {workspace.buf.device}, the operands on {X.device}")
    out = _out(out, (T, H), X.device)
    d = MoeDesc(X.data_ptr(), logits.data_ptr(), experts.W13.data_ptr(), experts.w13_scale.data_ptr(),
                experts.W2.data_ptr(), experts.w2_scale.data_ptr(), out.data_ptr(), T, H, experts.I, experts.E, topk,
                dtype, sc, 1 if renormalize else 0, 1 if experts.packed else 0, scale, 0, workspace.ptr(),
                workspace.nbytes)
    rc = lib().a8w8_moe_layer(ctypes.byref(d), _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "a8w8_moe_layer")
    return out


# ---------------------------------------------------------------------------
# Low-rank adapters of many requests beside one shared projection

class LoraAdapters:
    """A stack of low-rank adapters, checked once and kept by the caller's program: A bf16 [L,R,K],
    B bf16 [L,N,R], scaling float32 [L]; R a multiple of 8 up to 256 (smaller ranks padded with zeros)."""

    def __init__(self, A, B, scaling):
        if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16 or A.dim() != 3 or B.dim() != 3:
            raise TypeError("A and B must be 3-D bfloat16 tensors")
        L, R, K = A.shape
        if B.shape[0] != L or B.shape[2] != R:
            raise ValueError(f"A is [{L},{R},K] but B is {tuple(B.shape)}")
        if R % 8 or not 8 <= R <= 256:
            raise ValueError(f"the rank must be a multiple of 8 from 8 to 256, got {R}")
        if scaling.dtype != torch.float32 or tuple(scaling.shape) != (L,):
            raise ValueError(f"scaling must be a float32 [{L}] tensor")
        _check_device((("A", A), ("B", B), ("scaling", scaling)), A.device)
        self.A, self.B, self.scaling = A, B, scaling
        self.L, self.R, self.K, self.N, self.device = L, R, K, B.shape[1], A.device


def lora_workspace_bytes(M: int, N: int, K: int, adapters: LoraAdapters) -> int:
    """Workspace bytes gemm_a8w8_blockscale_lora needs for any number of rows up to M (Workspace(nbytes))."""
    n = ctypes.c_int64(0)
    rc = lib().gemm_a8w8_blockscale_lora_workspace_bytes(M, N, K, adapters.L, adapters.R, ctypes.byref(n))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "gemm_a8w8_blockscale_lora_workspace_bytes")
    return n.value


def gemm_a8w8_blockscale_lora(X: torch.Tensor, W: torch.Tensor, w_scale: torch.Tensor, adapters: LoraAdapters,
                              ids: torch.Tensor, workspace: Workspace, *, packed_n: int | None = None,
                              variant: int | None = None, scales: str = "reciprocal", out: torch.Tensor | None = None,
                              stream=None) -> torch.Tensor:
    """Y[m] = a8w8(X[m] quantised per 1x128 group, W) + scaling[a] B[a] (A[a] X[m]), a = ids[m] (int32 [M];
    negative: the projection alone), rounded once; returns bf16 [M,N].  The groups' scales are
    amax * fp32(1/448) (``scales="reciprocal"``), at most one ulp from quantize_1x128's amax / 448, or those quotients
    (``"quotient"``: a row without an adapter gets the bits of quantize_1x128 and the same instance's GEMM).
    ``packed_n``: W is in the packed layout for N = packed_n rows.  The workspace needs lora_workspace_bytes."""
    if scales not in ("reciprocal", "quotient"):
        raise ValueError(f"scales must be 'reciprocal' or 'quotient', got {scales!r}")
    if X.dtype != torch.bfloat16 or X.dim() != 2:
        raise ValueError("X must be a contiguous bfloat16 [M,K] GPU tensor")
    if W.dtype not in (torch.float8_e4m3fn, torch.uint8) or W.dim() != 2:
        raise TypeError("W must be a 2-D float8_e4m3fn (or raw uint8) tensor")
    if w_scale.dtype != torch.float32:
        raise TypeError("w_scale must be float32")
    Wv = W if packed_n is None else _packed_view(W, packed_n)
    M, K = X.shape
    N, K2 = Wv.shape
    if K2 != K or K % 128:
        raise ValueError(f"X is [M,{K}] and W is [N,{K2}]: K must agree and be a multiple of 128")
    if tuple(w_scale.shape) != ((N + 127) // 128, K // 128):
        raise ValueError(f"w_scale must be [{(N + 127) // 128},{K // 128}], got {tuple(w_scale.shape)}")
    if adapters.N != N or adapters.K != K:
        raise ValueError(f"the adapters are for N={adapters.N}, K={adapters.K}; the projection has N={N}, K={K}")
    if ids.dtype != torch.int32 or tuple(ids.shape) != (M,):
        raise ValueError(f"ids must be a contiguous int32 [{M}] tensor")
    _check_device((("X", X), ("W", W), ("w_scale", w_scale), ("ids", ids)), adapters.device)
    if workspace.buf.device != X.device:
        raise ValueError(f"the workspace is on {workspace.buf.device}, the operands on {X.device}")
    out = _out(out, (M, N), X.device)
    d = LoraDesc(X.data_ptr(), W.data_ptr(), w_scale.data_ptr(), adapters.A.data_ptr(), adapters.B.data_ptr(),
                 adapters.scaling.data_ptr(), ids.data_ptr(), out.data_ptr(), M, N, K, adapters.L, adapters.R,
                 0 if packed_n is None else 1, -1 if variant is None else int(variant), workspace.ptr(),
                 workspace.nbytes)
    name = "gemm_a8w8_blockscale_lora" if scales == "reciprocal" else "gemm_a8w8_blockscale_lora_quantize_1x128"
    rc = getattr(lib(), name)(ctypes.byref(d), _stream_handle(stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, name)
    return out


# ---------------------------------------------------------------------------
# The attention half of a decoder block: norms and rotation of queries and keys
# into a paged cache, and attention of new tokens over it

class _Handle:
    """Attributes are as they were checked: another tensor needs a handle of its own."""

    def __setattr__(self, name, value):
        if name in self.__dict__:
            raise AttributeError(f"{type(self).__name__}.{name} was checked when the handle was made: make a new one instead")
        super().__setattr__(name, value)


class KvCache(_Handle):
    """A paged cache, checked once and kept by the caller's program: k and v bfloat16 or float8_e4m3fn
    [pages,page_size,kv_heads,head_dim], page_size a power of two, head_dim 64, 128 or 256; 8-bit entries stand for
    code * scale, k_scale and v_scale float32 [kv_heads] (None: 1)."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or v.dtype != k.dtype or k.dim() != 4:
            raise TypeError("k and v must be 4-D bfloat16 or float8_e4m3fn tensors of one type")
        if k.shape != v.shape:
            raise ValueError(f"k is {tuple(k.shape)} but v is {tuple(v.shape)}")
        pages, page_size, heads, D = k.shape
        if D not in (64, 128, 256):
            raise ValueError(f"head_dim must be 64, 128 or 256, got {D}")
        if page_size < 1 or page_size & (page_size - 1) or page_size > 65536:
            raise ValueError(f"page_size must be a power of two up to 65536, got {page_size}")
        if pages < 1 or heads < 1 or pages * page_size > 2 ** 31 - 1:
            raise ValueError(f"a cache has 1 to 2^31 - 1 slots and at least one head, got {tuple(k.shape)}")
        named = [("k", k), ("v", v)]
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is None:
                continue
            if k.dtype == torch.bfloat16:
                raise ValueError("scales belong to 8-bit caches")
            if s.dtype != torch.float32 or tuple(s.shape) != (heads,):
                raise ValueError(f"{name} must be a float32 [{heads}] tensor")
            named.append((name, s))
        _check_device(named, k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.page_size, self.kv_heads, self.head_dim = pages, page_size, heads, D
        self.dtype, self.device, self.index = 0 if k.dtype == torch.bfloat16 else 1, k.device, k.get_device()

    def operands(self) -> tuple:
        """Addresses of k, v and their scales, as the descriptors take them."""
        return self.k.data_ptr(), self.v.data_ptr(), _ptr(self.k_scale), _ptr(self.v_scale)

    @classmethod
    def empty(cls, pages: int, page_size: int, kv_heads: int, head_dim: int, dtype=torch.bfloat16, k_scale=None,
              v_scale=None, device="cuda") -> "KvCache":
        """Pages of zeros."""
        shape = (pages, page_size, kv_heads, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype, device=device) for _ in "kv")
        if dtype == torch.float8_e4m3fn:
            k, v = k.view(dtype), v.view(dtype)
        return cls(k, v, k_scale, v_scale)


class Rope(_Handle):
    """The position rotation, checked once and kept by the caller's program: inv_freq float32 [rotary_dim/2];
    ``axes`` int32 [rotary_dim/2], the row of the positions that turns each pair (None: row 0); ``layout`` "halves"
    (pairs (i, i + rotary_dim/2)) or "pairs" ((2i, 2i+1))."""

    def __init__(self, inv_freq, axes=None, layout: str = "halves"):
        if layout not in ROPE_LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
        if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not 8 <= inv_freq.shape[0] <= 128 or inv_freq.shape[0] % 8:
            raise ValueError("inv_freq must be a float32 [rotary_dim/2] tensor, rotary_dim a multiple of 16 up to 256")
        named = [("inv_freq", inv_freq)]
        if axes is not None:
            if axes.dtype != torch.int32 or axes.shape != inv_freq.shape:
                raise ValueError(f"axes must be an int32 [{inv_freq.shape[0]}] tensor")
            named.append(("axes", axes))
        _check_device(named, inv_freq.device)
        self.inv_freq, self.axes, self.layout, self.rotary_dim = inv_freq, axes, layout, 2 * len(inv_freq)
        self.device, self.index = inv_freq.device, inv_freq.get_device()

    def operands(self) -> tuple:
        """Addresses, dimensions and layout, as the descriptor takes them."""
        return self.inv_freq.data_ptr(), _ptr(self.axes), self.rotary_dim, ROPE_LAYOUTS[self.layout]


# The current device's index without torch.cuda's own checks (0.1 against 0.5 us a call).
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _check_current(index: int) -> None:
    current = _raw_device() if _raw_device is not None else torch.cuda.current_device()
    if index != current:
        raise ValueError(f"operands are on cuda:{index} but the current device is cuda:{current}")


def _stream_on(index: int, stream) -> int:
    """_stream_handle on the current device, which _check_current has looked up already."""
    return _raw_stream(index) if stream is None and _raw_stream is not None else _stream_handle(stream)


def _check_heads(name, x, shape, index):
    """A bf16 [T,heads,head_dim] view on GPU `index` (None: any) whose heads are contiguous and start on 16 bytes; returns
    its shape, token and head strides and address."""
    if x.dtype != torch.bfloat16 or x.dim() != 3 or (shape is not None and x.shape != shape):
        raise ValueError(f"{name} must be a bfloat16 {'[T,heads,head_dim]' if shape is None else tuple(shape)} tensor, "
                         f"got {x.dtype} {tuple(x.shape)}")
    if not x.is_cuda or (index is not None and x.get_device() != index):
        raise ValueError(f"{name} must be a GPU tensor on the others' device, it is on {x.device}")
    row, head, unit = x.stride()
    ptr = x.data_ptr()
    if unit != 1 or row % 8 or head % 8 or ptr % 16:
        raise ValueError(f"{name}: heads must be contiguous and start on 16 bytes, got strides {x.stride()}")
    return x.shape, row, head, ptr


def _check_ints(name, x, shape, index):
    """A contiguous int32 tensor of `shape` on GPU `index`; returns its address."""
    if x.dtype != torch.int32 or x.shape != shape or not x.is_contiguous() or not x.is_cuda or x.get_device() != index:
        raise ValueError(f"{name} must be a contiguous int32 {tuple(shape)} tensor on cuda:{index}, got {x.dtype} "
                         f"{tuple(x.shape)} on {x.device}")
    return x.data_ptr()


def _check_counts(**named) -> None:
    """Whole numbers from 0 that fit the descriptors' 32-bit fields (which would take 2^32 + 1 for 1)."""
    for name, x in named.items():
        if not 0 <= x < 2 ** 31:
            raise ValueError(f"{name} must be from 0 to 2^31 - 1, got {x}")


def _check_weight(name, w, D, index):
    """A float32 [D] tensor on GPU `index` or None; returns its address."""
    if w is None:
        return None
    if w.dtype != torch.float32 or w.shape != (D,) or not w.is_contiguous() or not w.is_cuda or w.get_device() != index:
        raise ValueError(f"{name} must be a contiguous float32 [{D}] tensor on cuda:{index}")
    return w.data_ptr()


def _heads_out(name, out, like, shape, index):
    if out is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=like.device)
    if out.dtype != torch.bfloat16 or out.shape != shape or not out.is_contiguous() or not out.is_cuda or out.get_device() != index:
        raise ValueError(f"{name} must be a contiguous bfloat16 {tuple(shape)} tensor on cuda:{index}")
    return out


def _ptr(t):
    return None if t is None else t.data_ptr()


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, rope: Rope | None = None, positions: torch.Tensor | None = None, *,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 v: torch.Tensor | None = None, cache: KvCache | None = None, slots: torch.Tensor | None = None,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Norms of each head of q [T,Hq,D] and k [T,Hkv,D] (bf16, views into the projection's rows as well), times q_weight and
    k_weight (float32 [D]; None: no norm), and the rotation by ``positions`` int32 [T] or [axes,T], in one pass.  With a
    ``cache`` the keys and v [T,Hkv,D] go to ``slots`` int32 [T] of it (page * page_size + offset; -1: not stored) in its
    type; without one the keys are returned.  Returns (q bf16 [T,Hq,D], k bf16 [T,Hkv,D] or None)."""
    (T, Hq, D), q_row, q_head, q_ptr = _check_heads("q", q, None, None)
    index = q.get_device()
    Hkv = k.shape[1] if k.dim() == 3 else 0
    _, k_row, k_head, k_ptr = _check_heads("k", k, (T, Hkv, D), index)
    wq, wk = _check_weight("q_weight", q_weight, D, index), _check_weight("k_weight", k_weight, D, index)
    axes, turn = 1, (None, None, None, 0, 0)
    if rope is not None:
        if positions is None or positions.dim() not in (1, 2):
            raise ValueError(f"positions must be an int32 [{T}] or [axes,{T}] tensor")
        if rope.rotary_dim > D:
            raise ValueError(f"the rotation has {rope.rotary_dim} dimensions, the heads {D}")
        if rope.index != index:
            raise ValueError(f"the rotation is on cuda:{rope.index}, q on cuda:{index}")
        axes = positions.shape[0] if positions.dim() == 2 else 1
        turn = (_check_ints("positions", positions, (T,) if positions.dim() == 1 else (axes, T), index), *rope.operands())
    if cache is not None:
        if k_out is not None:
            raise ValueError("the keys go to the cache or to k_out, not to both")
        if v is None or slots is None:
            raise ValueError("a cache needs v and slots")
        if cache.kv_heads != Hkv or cache.head_dim != D or cache.index != index:
            raise ValueError(f"the cache has {cache.kv_heads} heads of {cache.head_dim} on cuda:{cache.index}, k {Hkv} of {D} "
                             f"on cuda:{index}")
        _, v_row, v_head, v_ptr = _check_heads("v", v, (T, Hkv, D), index)
        at, k_new = _check_ints("slots", slots, (T,), index), None
        kept = (*cache.operands(), cache.pages * cache.page_size, cache.dtype)
    else:
        if v is not None or slots is not None:
            raise ValueError("v and slots belong to a cache")
        k_out = _heads_out("k_out", k_out, k, (T, Hkv, D), index)
        v_row = v_head = 0
        v_ptr = at = None
        k_new, kept = k_out.data_ptr(), (None, None, None, None, 0, 0)
    _check_current(index)
    q_out = _heads_out("q_out", q_out, q, (T, Hq, D), index)
    positions_ptr, inv_freq, axis_of, rotary_dim, layout = turn
    d = RopeDesc(q_ptr, k_ptr, v_ptr, q_row, q_head, k_row, k_head, v_row, v_head, wq, wk, positions_ptr, inv_freq, axis_of, at,
                 q_out.data_ptr(), k_new, *kept[:4], T, kept[4], Hq, Hkv, D, rotary_dim, axes, layout, kept[5], eps)
    rc = lib().a8w8_qk_norm_rope(ctypes.byref(d), _stream_on(index, stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "a8w8_qk_norm_rope")
    return q_out, k_out


def paged_attention_workspace_bytes(T: int, B: int, q_heads: int, cache: KvCache, cu_count: int = 0) -> int:
    """Workspace bytes paged_attention needs for up to T rows of up to B sequences (Workspace(nbytes))."""
    _check_counts(q_heads=q_heads, cu_count=max(cu_count, 0))
    n = ctypes.c_int64(0)
    rc = lib().a8w8_paged_attention_workspace_bytes(T, B, q_heads, cache.kv_heads, cache.head_dim, cache.dtype, cu_count,
                                                    ctypes.byref(n))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "a8w8_paged_attention_workspace_bytes")
    return n.value


def paged_attention(q: torch.Tensor, cache: KvCache, page_table: torch.Tensor, q_start: torch.Tensor,
                    kv_lens: torch.Tensor, workspace: Workspace, *, scale: float | None = None, window: int = 0,
                    sinks: int = 0, gate: torch.Tensor | None = None, max_new: int = 0, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Attention of new tokens, q bf16 [T,Hq,D], over a paged cache; returns bf16 [T,Hq,D].  Sequence b has the rows
    q_start[b] .. q_start[b+1] (int32 [B+1]) and kv_lens[b] (int32 [B]) cached tokens, the new ones included, in the pages
    page_table[b] (int32 [B,pages of a sequence], -1 where unused).  Row i of its n rows stands at kv_lens[b] - n + i and
    sees the keys up to there, with ``window`` > 0 only the last ``window`` of them and the first ``sinks`` tokens.  ``scale``
    (default D^-1/2) multiplies the scores, sigmoid(``gate``) [T,Hq,D] the result.  The softmax's numerators have 16 bits in
    sequences with up to 16 rows per key head (rows times Hq / Hkv) and 8 bits in longer ones.  ``max_new``: a hint, the most
    rows of one sequence (0: unknown); a hint of at most 16 rows per key head takes all sequences for such short ones,
    which costs those that are not time.  Rows outside every sequence stay as they were in ``out``.  The workspace needs
    paged_attention_workspace_bytes."""
    index = cache.index
    (T, Hq, D), q_row, q_head, q_ptr = _check_heads("q", q, None, index)
    if D != cache.head_dim or Hq % cache.kv_heads:
        raise ValueError(f"q has {Hq} heads of {D}, the cache {cache.kv_heads} of {cache.head_dim}")
    _check_counts(window=window, sinks=sinks, max_new=max_new)
    if page_table.dim() != 2:
        raise ValueError("page_table must be a contiguous int32 [B,pages] GPU tensor")
    B, P = page_table.shape
    table = _check_ints("page_table", page_table, (B, P), index)
    starts, lens = _check_ints("q_start", q_start, (B + 1,), index), _check_ints("kv_lens", kv_lens, (B,), index)
    g_row = g_head = 0
    g_ptr = None
    if gate is not None:
        _, g_row, g_head, g_ptr = _check_heads("gate", gate, (T, Hq, D), index)
    if workspace.buf.get_device() != index:
        raise ValueError(f"the workspace is on {workspace.buf.device}, the operands on cuda:{index}")
    _check_current(index)
    out = _heads_out("out", out, q, (T, Hq, D), index)
    d = AttentionDesc(q_ptr, g_ptr, q_row, q_head, g_row, g_head, *cache.operands(), table, starts, lens, out.data_ptr(), T, B,
                      cache.pages, P, cache.page_size, Hq, cache.kv_heads, D, cache.dtype, window, sinks, max_new,
                      D ** -0.5 if scale is None else scale, 0, workspace.ptr(), workspace.nbytes)
    rc = lib().a8w8_paged_attention(ctypes.byref(d), _stream_on(index, stream))
    if rc != A8W8_OK:
        raise A8W8Error(rc, "a8w8_paged_attention")
    return out
