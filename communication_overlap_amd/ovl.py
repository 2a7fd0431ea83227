"""ctypes binding of libovl.so: the same entry points as include/ovl.h.

Argument marshalling only.  Tensors are passed as raw device pointers
(their data_ptr()), streams as their HIP handle; every step of the path runs
in the library's kernels.  There is no fallback: if the library is missing,
loading fails loudly.
"""

from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, Structure, byref, c_char_p, c_float, c_int32, c_int64, c_size_t, c_uint32, c_uint64, c_void_p

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libovl.so")

OVL_OK = 0
OVL_EINVAL = -1
OVL_ESHAPE = -2
OVL_EALIGN = -3
OVL_EEPOCH = -4
OVL_EHIP = -5
OVL_ETIMEOUT = -6
OVL_EUNSUPPORTED = -7

MODE_FUSED = 0
MODE_COPY_ONLY = 1
MODE_GEMM_ONLY = 2
MODE_BARRIER = 3

ERROR_RECORD_BYTES = 64

BF16, F32, FP8 = 0, 1, 2
TYPES = {"bf16": BF16, "f32": F32, "fp8": FP8}
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(5)
ACTS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "silu": ACT_SILU}

EXPORTS = (
    "ag_gemm_plan", "ag_gemm_plan_destroy", "ag_gemm_num_units", "ag_gemm_flags_bytes",
    "ag_gemm_workspace_bytes", "ag_gemm_splits", "ag_gemm_run",
    "gemm_rs_flags_bytes", "gemm_rs_workspace_bytes", "gemm_rs_run",
    "a2a_flags_bytes", "a2a_workspace_bytes", "a2a_trace_bytes", "a2a_dispatch_grouped_gemm_run",
    "a2a_combine_flags_bytes", "a2a_combine_workspace_bytes", "a2a_combine_run",
    "ovl_flags_reset", "ovl_check", "ovl_strerror", "ovl_copy",
    "ring_allreduce_flags_bytes", "ring_allreduce_workspace_bytes", "ring_allreduce_run",
    "fp8_quantize_rows", "a2a_dispatch_grouped_gemm_fp8_run", "ag_gemm_trace_bytes",
    "ag_gemm_row_tiles", "ag_gemm_tile_rows", "ag_gemm_consumer_order", "ag_gemm_run_noalloc",
    "gemm_epilogue_workspace_bytes", "gemm_epilogue_run", "gemm_epilogue_grad_workspace_bytes",
    "gemm_epilogue_grad_run", "moe_layer_workspace_bytes", "moe_layer_run",
    "grad_clip_plan", "grad_clip_plan_destroy", "grad_clip_workspace_bytes", "grad_clip_upload", "grad_norm_clip_run",
)


class OvlError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} ({status})")


class Opts(Structure):
    _fields_ = [("mode", c_uint32), ("producers", c_uint32), ("spin_limit", c_uint64), ("trace", c_void_p),
                ("jitter", c_uint32), ("reserved", c_uint32)]


class AgGemmDesc(Structure):
    _fields_ = [("ranks", c_int32), ("rank", c_int32), ("shard_m", c_int64), ("k", c_int64), ("n", c_int64),
                ("tile_m", c_int32), ("tile_n", c_int32), ("tiles_per_flag", c_int32), ("flag_stride", c_int32),
                ("unit_producers", c_int32)]


class GemmRsDesc(Structure):
    _fields_ = [("ranks", c_int32), ("rank", c_int32), ("m", c_int64), ("n", c_int64), ("k", c_int64),
                ("tile_m", c_int32), ("tile_n", c_int32), ("flag_stride", c_int32)]


class A2aDesc(Structure):
    _fields_ = [("ranks", c_int32), ("rank", c_int32), ("tokens", c_int64), ("hidden", c_int64), ("n", c_int64),
                ("topk", c_int32), ("num_experts", c_int32), ("experts_per_rank", c_int32),
                ("flag_stride", c_int32), ("tile_m", c_int32), ("tile_n", c_int32)]


class RingDesc(Structure):
    _fields_ = [("ranks", c_int32), ("n", c_int64), ("tile", c_int64), ("flag_stride", c_int32)]


class GemmEpilogueDesc(Structure):
    _fields_ = [(f, c_int64) for f in ("m", "n", "k", "lda", "ldb", "ldo", "ldz", "ldr")] + \
               [(f, c_int32) for f in ("act", "out_type", "res_type", "reserved")]


class GemmEpilogueGradDesc(Structure):
    _fields_ = [(f, c_int64) for f in ("m", "n", "k", "lda", "ldb", "lddz", "lddy", "ldz", "ldz_in", "ldda", "lddb")] + \
               [(f, c_int32) for f in ("act", "act_in", "dy_type", "da_type", "db_type", "reserved")]


class MoeLayerDesc(Structure):
    _fields_ = [(f, c_int64) for f in ("tokens", "hidden", "inter")] + \
               [(f, c_int32) for f in ("experts", "topk", "act", "gated", "w_type", "out_type", "norm_topk", "reserved")]


class GradClipTensor(Structure):
    _fields_ = [("src", c_void_p), ("dst", c_void_p), ("count", c_int64), ("type", c_int32), ("reserved", c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """Loads libovl.so once (after torch, so that both share one HIP runtime)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m communication_overlap_amd.build`")
    import torch  # noqa: F401  (loads the HIP runtime the library links against)
    L = ctypes.CDLL(LIB_PATH, mode=ctypes.RTLD_GLOBAL)
    st = c_int32
    L.ag_gemm_plan.argtypes = [POINTER(AgGemmDesc), POINTER(c_void_p)]
    L.ag_gemm_plan.restype = st
    L.ag_gemm_plan_destroy.argtypes = [c_void_p]
    L.ag_gemm_plan_destroy.restype = st
    L.ag_gemm_num_units.argtypes = [c_void_p]
    L.ag_gemm_num_units.restype = c_int64
    L.ag_gemm_flags_bytes.argtypes = [c_void_p]
    L.ag_gemm_flags_bytes.restype = c_size_t
    L.ag_gemm_workspace_bytes.argtypes = [c_void_p]
    L.ag_gemm_workspace_bytes.restype = c_size_t
    L.ag_gemm_splits.argtypes = [c_void_p]
    L.ag_gemm_splits.restype = c_int32
    L.ag_gemm_trace_bytes.argtypes = [c_void_p]
    L.ag_gemm_trace_bytes.restype = c_size_t
    L.ag_gemm_row_tiles.argtypes = [c_void_p]
    L.ag_gemm_row_tiles.restype = c_int32
    L.ag_gemm_tile_rows.argtypes = [c_void_p]
    L.ag_gemm_tile_rows.restype = c_int32
    L.ag_gemm_run.argtypes = [c_void_p, POINTER(c_void_p), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                              c_int64, c_void_p, POINTER(Opts), c_void_p]
    L.ag_gemm_run.restype = st
    L.ag_gemm_run_noalloc.argtypes = [c_void_p, POINTER(c_void_p), c_void_p, c_void_p, c_void_p, c_void_p,
                                      c_int64, c_void_p, POINTER(Opts), c_void_p]
    L.ag_gemm_run_noalloc.restype = st
    L.gemm_rs_flags_bytes.argtypes = [POINTER(GemmRsDesc)]
    L.gemm_rs_flags_bytes.restype = c_size_t
    L.gemm_rs_workspace_bytes.argtypes = [POINTER(GemmRsDesc)]
    L.gemm_rs_workspace_bytes.restype = c_size_t
    L.gemm_rs_run.argtypes = [POINTER(GemmRsDesc), c_void_p, c_void_p, POINTER(c_void_p), POINTER(c_void_p),
                              c_void_p, c_void_p, c_void_p, c_void_p, c_int64, POINTER(Opts), c_void_p]
    L.gemm_rs_run.restype = st
    L.a2a_flags_bytes.argtypes = [POINTER(A2aDesc)]
    L.a2a_flags_bytes.restype = c_size_t
    L.a2a_workspace_bytes.argtypes = [POINTER(A2aDesc)]
    L.a2a_workspace_bytes.restype = c_size_t
    L.a2a_trace_bytes.argtypes = [POINTER(A2aDesc)]
    L.a2a_trace_bytes.restype = c_size_t
    L.a2a_dispatch_grouped_gemm_run.argtypes = [POINTER(A2aDesc), POINTER(c_void_p), POINTER(c_void_p), c_void_p,
                                                c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                                c_int64, POINTER(Opts), c_void_p]
    L.a2a_dispatch_grouped_gemm_run.restype = st
    L.a2a_combine_flags_bytes.argtypes = [POINTER(A2aDesc)]
    L.a2a_combine_flags_bytes.restype = c_size_t
    L.a2a_combine_workspace_bytes.argtypes = [POINTER(A2aDesc)]
    L.a2a_combine_workspace_bytes.restype = c_size_t
    L.a2a_combine_run.argtypes = [POINTER(A2aDesc), c_void_p, c_void_p, POINTER(c_void_p), POINTER(c_void_p),
                                  c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int64,
                                  POINTER(Opts), c_void_p]
    L.a2a_combine_run.restype = st
    L.ovl_flags_reset.argtypes = [c_void_p, c_size_t, c_void_p, c_size_t, c_void_p]
    L.ovl_flags_reset.restype = st
    L.ovl_check.argtypes = [c_void_p, POINTER(c_int64), c_void_p]
    L.ovl_check.restype = st
    L.ovl_strerror.argtypes = [c_int32]
    L.ovl_strerror.restype = c_char_p
    L.ovl_copy.argtypes = [c_void_p, c_void_p, c_size_t, c_int32, c_void_p]
    L.ovl_copy.restype = st
    L.ring_allreduce_flags_bytes.argtypes = [POINTER(RingDesc)]
    L.ring_allreduce_flags_bytes.restype = c_size_t
    L.ring_allreduce_workspace_bytes.argtypes = [POINTER(RingDesc)]
    L.ring_allreduce_workspace_bytes.restype = c_size_t
    L.ring_allreduce_run.argtypes = [POINTER(RingDesc), POINTER(c_void_p), POINTER(c_void_p), c_void_p, c_void_p,
                                     c_int64, POINTER(Opts), c_void_p]
    L.ring_allreduce_run.restype = st
    L.fp8_quantize_rows.argtypes = [c_void_p, c_void_p, c_void_p, c_int64, c_int64, c_void_p]
    L.fp8_quantize_rows.restype = st
    L.a2a_dispatch_grouped_gemm_fp8_run.argtypes = [POINTER(A2aDesc), POINTER(c_void_p), POINTER(c_void_p),
                                                    POINTER(c_void_p), c_void_p, c_void_p, c_void_p, c_void_p,
                                                    c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int64,
                                                    POINTER(Opts), c_void_p]
    L.a2a_dispatch_grouped_gemm_fp8_run.restype = st
    L.gemm_epilogue_workspace_bytes.argtypes = [POINTER(GemmEpilogueDesc)]
    L.gemm_epilogue_workspace_bytes.restype = c_size_t
    L.gemm_epilogue_run.argtypes = [POINTER(GemmEpilogueDesc)] + [c_void_p] * 8
    L.gemm_epilogue_run.restype = st
    L.gemm_epilogue_grad_workspace_bytes.argtypes = [POINTER(GemmEpilogueGradDesc)]
    L.gemm_epilogue_grad_workspace_bytes.restype = c_size_t
    L.gemm_epilogue_grad_run.argtypes = [POINTER(GemmEpilogueGradDesc)] + [c_void_p] * 13
    L.gemm_epilogue_grad_run.restype = st
    L.moe_layer_workspace_bytes.argtypes = [POINTER(MoeLayerDesc)]
    L.moe_layer_workspace_bytes.restype = c_size_t
    L.moe_layer_run.argtypes = [POINTER(MoeLayerDesc)] + [c_void_p] * 11
    L.moe_layer_run.restype = st
    L.grad_clip_plan.argtypes = [POINTER(GradClipTensor), c_int64, POINTER(c_void_p)]
    L.grad_clip_plan.restype = st
    L.grad_clip_plan_destroy.argtypes = [c_void_p]
    L.grad_clip_plan_destroy.restype = st
    L.grad_clip_workspace_bytes.argtypes = [c_void_p]
    L.grad_clip_workspace_bytes.restype = c_size_t
    L.grad_clip_upload.argtypes = [c_void_p, c_void_p, c_void_p]
    L.grad_clip_upload.restype = st
    L.grad_norm_clip_run.argtypes = [c_void_p, c_float, c_void_p, c_void_p, c_void_p]
    L.grad_norm_clip_run.restype = st
    _lib = L
    return L


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_torch_module = None


def strerror(status: int) -> str:
    try:
        return lib().ovl_strerror(status).decode()
    except ImportError:
        return f"status {status}"


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        # torch.cuda.current_stream() makes a Stream object (2.9 us a call); the
        # handle alone takes 0.1.
        torch = _torch()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _opts(mode: int, producers: int, spin_limit: int, trace=None, jitter: int = 0) -> Opts:
    return Opts(mode, producers, spin_limit, _ptr(trace), jitter, 0)


def _check(status: int, where: str, raise_on_error: bool) -> int:
    if status != OVL_OK and raise_on_error:
        raise OvlError(status, where)
    return status


def _ptr_array(ts):
    arr = (c_void_p * len(ts))()
    for i, t in enumerate(ts):
        arr[i] = _ptr(t)
    return arr


# ------------------------------------------------------------------ AG-GEMM

class AgGemmPlan:
    """Owns an ag_gemm_plan_t."""

    def __init__(self, ranks, rank, shard_m, k, n, tile_m, tile_n, tiles_per_flag=0, flag_stride=8,
                 unit_producers=1):
        self.desc = AgGemmDesc(ranks, rank, shard_m, k, n, tile_m, tile_n, tiles_per_flag, flag_stride,
                               unit_producers)
        h = c_void_p()
        _check(lib().ag_gemm_plan(byref(self.desc), byref(h)), "ag_gemm_plan", True)
        self.handle = h

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.ag_gemm_plan_destroy(h)
            self.handle = None

    @property
    def num_units(self) -> int:
        return lib().ag_gemm_num_units(self.handle)

    @property
    def flags_bytes(self) -> int:
        return lib().ag_gemm_flags_bytes(self.handle)

    @property
    def workspace_bytes(self) -> int:
        return lib().ag_gemm_workspace_bytes(self.handle)

    @property
    def splits(self) -> int:
        return lib().ag_gemm_splits(self.handle)

    @property
    def trace_bytes(self) -> int:
        return lib().ag_gemm_trace_bytes(self.handle)

    @property
    def tile_rows(self) -> int:
        """Rows of the consumer's output tile (chosen by the library)."""
        return lib().ag_gemm_tile_rows(self.handle)

    @property
    def row_tiles(self) -> int:
        return lib().ag_gemm_row_tiles(self.handle)


def ag_gemm_plan(*args, **kw) -> AgGemmPlan:
    return AgGemmPlan(*args, **kw)


def ag_gemm_run(plan: AgGemmPlan, shards, b, gathered, c, flags, workspace, epoch: int, producer_order=None,
                mode: int = MODE_FUSED, producers: int = 0, spin_limit: int = 0, stream=None,
                raise_on_error: bool = True, trace=None, jitter: int = 0) -> int:
    arr = _ptr_array(shards)
    o = _opts(mode, producers, spin_limit, trace, jitter)
    st = lib().ag_gemm_run(plan.handle, arr, _ptr(b), _ptr(gathered), _ptr(c), _ptr(flags), _ptr(workspace),
                           epoch, _ptr(producer_order), byref(o), _stream(stream))
    return _check(st, "ag_gemm_run", raise_on_error)


def ag_gemm_run_noalloc(plan: AgGemmPlan, shards, b, gathered, c, flags, epoch: int, producer_order=None,
                        mode: int = MODE_FUSED, producers: int = 0, spin_limit: int = 0, stream=None,
                        raise_on_error: bool = True, trace=None, jitter: int = 0) -> int:
    arr = _ptr_array(shards)
    o = _opts(mode, producers, spin_limit, trace, jitter)
    st = lib().ag_gemm_run_noalloc(plan.handle, arr, _ptr(b), _ptr(gathered), _ptr(c), _ptr(flags), epoch,
                                   _ptr(producer_order), byref(o), _stream(stream))
    return _check(st, "ag_gemm_run_noalloc", raise_on_error)


# ------------------------------------------------------------------ GEMM-RS

def gemm_rs_desc(ranks, rank, m, n, k, tile_m=256, tile_n=256, flag_stride=8) -> GemmRsDesc:
    return GemmRsDesc(ranks, rank, m, n, k, tile_m, tile_n, flag_stride)


def gemm_rs_flags_bytes(desc: GemmRsDesc) -> int:
    return lib().gemm_rs_flags_bytes(byref(desc))


def gemm_rs_workspace_bytes(desc: GemmRsDesc) -> int:
    return lib().gemm_rs_workspace_bytes(byref(desc))


def gemm_rs_run(desc: GemmRsDesc, a, b, peer_out, peer_in, out, out_flags, in_flags, workspace, epoch: int,
                mode: int = MODE_FUSED, producers: int = 0, spin_limit: int = 0, stream=None,
                raise_on_error: bool = True) -> int:
    o = _opts(mode, producers, spin_limit)
    st = lib().gemm_rs_run(byref(desc), _ptr(a), _ptr(b), _ptr_array(peer_out), _ptr_array(peer_in), _ptr(out),
                           _ptr(out_flags), _ptr(in_flags), _ptr(workspace), epoch, byref(o), _stream(stream))
    return _check(st, "gemm_rs_run", raise_on_error)


# ------------------------------------------------------------------ dispatch + grouped GEMM

def a2a_desc(ranks, rank, tokens, hidden, n, topk, num_experts, experts_per_rank, flag_stride=8,
             tile_m=0, tile_n=0) -> A2aDesc:
    return A2aDesc(ranks, rank, tokens, hidden, n, topk, num_experts, experts_per_rank, flag_stride, tile_m, tile_n)


def a2a_flags_bytes(desc: A2aDesc) -> int:
    return lib().a2a_flags_bytes(byref(desc))


def a2a_workspace_bytes(desc: A2aDesc) -> int:
    return lib().a2a_workspace_bytes(byref(desc))


def a2a_trace_bytes(desc: A2aDesc) -> int:
    return lib().a2a_trace_bytes(byref(desc))


def a2a_dispatch_grouped_gemm_run(desc: A2aDesc, x, topk_idx, w, recv_x, recv_src, recv_count, y, flags,
                                  workspace, epoch: int, mode: int = MODE_FUSED, producers: int = 0,
                                  spin_limit: int = 0, stream=None, raise_on_error: bool = True, trace=None) -> int:
    o = _opts(mode, producers, spin_limit, trace)
    st = lib().a2a_dispatch_grouped_gemm_run(byref(desc), _ptr_array(x), _ptr_array(topk_idx), _ptr(w),
                                             _ptr(recv_x), _ptr(recv_src), _ptr(recv_count), _ptr(y), _ptr(flags),
                                             _ptr(workspace), epoch, byref(o), _stream(stream))
    return _check(st, "a2a_dispatch_grouped_gemm_run", raise_on_error)


def fp8_quantize_rows(in_bf16, codes, scale, rows: int, cols: int, stream=None, raise_on_error: bool = True) -> int:
    st = lib().fp8_quantize_rows(_ptr(in_bf16), _ptr(codes), _ptr(scale), rows, cols, _stream(stream))
    return _check(st, "fp8_quantize_rows", raise_on_error)


def a2a_dispatch_grouped_gemm_fp8_run(desc: A2aDesc, x8, x_scale, topk_idx, w8, w_scale, recv_x8, recv_scale,
                                      recv_src, recv_count, y, flags, workspace, epoch: int, mode: int = MODE_FUSED,
                                      producers: int = 0, spin_limit: int = 0, stream=None,
                                      raise_on_error: bool = True, trace=None) -> int:
    o = _opts(mode, producers, spin_limit, trace)
    st = lib().a2a_dispatch_grouped_gemm_fp8_run(byref(desc), _ptr_array(x8), _ptr_array(x_scale),
                                                 _ptr_array(topk_idx), _ptr(w8), _ptr(w_scale), _ptr(recv_x8),
                                                 _ptr(recv_scale), _ptr(recv_src), _ptr(recv_count), _ptr(y),
                                                 _ptr(flags), _ptr(workspace), epoch, byref(o), _stream(stream))
    return _check(st, "a2a_dispatch_grouped_gemm_fp8_run", raise_on_error)


def a2a_combine_flags_bytes(desc: A2aDesc) -> int:
    return lib().a2a_combine_flags_bytes(byref(desc))


def a2a_combine_workspace_bytes(desc: A2aDesc) -> int:
    return lib().a2a_combine_workspace_bytes(byref(desc))


def a2a_combine_run(desc: A2aDesc, y, recv_count, ret_out, ret_in, topk_idx, gates, out, out_flags, in_flags,
                    workspace, epoch: int, mode: int = MODE_FUSED, spin_limit: int = 0, stream=None,
                    raise_on_error: bool = True) -> int:
    o = _opts(mode, 0, spin_limit)
    st = lib().a2a_combine_run(byref(desc), _ptr(y), _ptr(recv_count), _ptr_array(ret_out), _ptr_array(ret_in),
                               _ptr(topk_idx), _ptr(gates), _ptr(out), _ptr(out_flags), _ptr(in_flags),
                               _ptr(workspace), epoch, byref(o), _stream(stream))
    return _check(st, "a2a_combine_run", raise_on_error)


# ------------------------------------------------------------------ ring all-reduce

def ring_desc(ranks, n, tile, flag_stride=8) -> RingDesc:
    return RingDesc(ranks, n, tile, flag_stride)


def ring_allreduce_flags_bytes(desc: RingDesc) -> int:
    return lib().ring_allreduce_flags_bytes(byref(desc))


def ring_allreduce_workspace_bytes(desc: RingDesc) -> int:
    return lib().ring_allreduce_workspace_bytes(byref(desc))


def ring_allreduce_run(desc: RingDesc, inputs, outputs, flags, workspace, epoch: int, mode: int = MODE_FUSED,
                       spin_limit: int = 0, stream=None, raise_on_error: bool = True) -> int:
    o = _opts(mode, 0, spin_limit)
    st = lib().ring_allreduce_run(byref(desc), _ptr_array(inputs), _ptr_array(outputs), _ptr(flags),
                                  _ptr(workspace), epoch, byref(o), _stream(stream))
    return _check(st, "ring_allreduce_run", raise_on_error)


# ------------------------------------------------------------------ feed-forward layers

def _act(act) -> int:
    return ACTS[act] if isinstance(act, str) else act


def _type(t) -> int:
    return TYPES[t] if isinstance(t, str) else t


# Element types of buffers beside BF16, F32 and FP8.
_INT32, _BYTES = 16, 17


def _dtypes() -> dict:
    global _dtype_table
    if _dtype_table is None:
        t = _torch()
        _dtype_table = {BF16: (t.bfloat16, t.int16, t.uint16), F32: (t.float32,), FP8: (t.uint8, t.float8_e4m3fn),
                        _INT32: (t.int32,), _BYTES: (t.uint8, t.int8, t.bool)}
    return _dtype_table


_dtype_table = None


class _Buffers:
    """Marshals the buffers of one call of the feed-forward calls.  A tensor
    has to lie on the current device, hold elements of the right type (bf16 or
    its bits as int16 or uint16; E4M3 or its codes as uint8) and be as large as
    the call takes it to be (dense, or a two-dimensional view with the
    descriptor's row stride); raw addresses pass unchecked."""

    __slots__ = ("where", "device", "kinds")

    def __init__(self, where: str):
        torch = _torch()
        self.where = where
        self.kinds = _dtypes()
        self.device = torch.cuda.current_device() if torch.cuda.is_initialized() or torch.cuda.is_available() else -2

    def refuse(self, name: str, why: str):
        raise OvlError(OVL_EINVAL, f"{self.where}: {name} {why}")

    def __call__(self, name: str, t, kind: int, rows: int, cols: int, ld: int = 0):
        if t is None or isinstance(t, int):
            return t
        kinds = self.kinds.get(kind)
        if kinds and t.dtype not in kinds:  # (of a type that the library refuses anything goes)
            self.refuse(name, f"has elements of type {t.dtype}, not {' or '.join(str(k) for k in kinds)}")
        if t.get_device() != self.device:  # -1: host memory
            self.refuse(name, "is not on the current device")
        if t.is_contiguous():
            if rows > 0 and t.numel() < (rows - 1) * (ld or cols) + cols:
                self.refuse(name, "is too small")
        elif not (t.dim() == 2 and t.stride(1) == 1 and t.stride(0) == (ld or cols) and t.shape[0] >= rows
                  and t.shape[1] >= cols):
            self.refuse(name, "is neither dense nor a matrix with the descriptor's row stride")
        return t.data_ptr()


def _workspace(buf, workspace, nbytes, desc):
    """The workspace's address; its size is asked of the library once for a descriptor's contents."""
    if workspace is None or isinstance(workspace, int):
        return workspace
    key = bytes(desc)
    known = getattr(desc, "_workspace", None)
    if known is None or known[0] != key:
        known = desc._workspace = (key, nbytes(byref(desc)))
    return buf("workspace", workspace, _BYTES, 1, known[1])


def gemm_epilogue_desc(m, n, k, act="none", out_type="bf16", res_type="bf16", lda=0, ldb=0, ldo=0, ldz=0,
                       ldr=0) -> GemmEpilogueDesc:
    return GemmEpilogueDesc(m, n, k, lda, ldb, ldo, ldz, ldr, _act(act), _type(out_type), _type(res_type), 0)


def gemm_epilogue_workspace_bytes(desc: GemmEpilogueDesc) -> int:
    return lib().gemm_epilogue_workspace_bytes(byref(desc))


def gemm_epilogue_run(desc: GemmEpilogueDesc, a, b, bias, residual, out, z, workspace, stream=None,
                      raise_on_error: bool = True) -> int:
    """out = act(a @ b + bias) + residual; z: the rounded pre-activation (bias, residual and z may be None)."""
    buf = _Buffers("gemm_epilogue_run")
    m, n, k = desc.m, desc.n, desc.k
    st = lib().gemm_epilogue_run(
        byref(desc), buf("a", a, BF16, m, k, desc.lda), buf("b", b, BF16, k, n, desc.ldb), buf("bias", bias, F32, 1, n),
        buf("residual", residual, desc.res_type, m, n, desc.ldr), buf("out", out, desc.out_type, m, n, desc.ldo),
        buf("z", z, BF16, m, n, desc.ldz),
        _workspace(buf, workspace, lib().gemm_epilogue_workspace_bytes, desc), _stream(stream))
    return _check(st, "gemm_epilogue_run", raise_on_error)


def gemm_epilogue_grad_desc(m, n, k, act="none", act_in="none", dy_type="bf16", da_type="bf16", db_type="f32", lda=0,
                            ldb=0, lddz=0, lddy=0, ldz=0, ldz_in=0, ldda=0, lddb=0) -> GemmEpilogueGradDesc:
    return GemmEpilogueGradDesc(m, n, k, lda, ldb, lddz, lddy, ldz, ldz_in, ldda, lddb, _act(act), _act(act_in),
                                _type(dy_type), _type(da_type), _type(db_type), 0)


def gemm_epilogue_grad_workspace_bytes(desc: GemmEpilogueGradDesc) -> int:
    return lib().gemm_epilogue_grad_workspace_bytes(byref(desc))


def gemm_epilogue_grad_run(desc: GemmEpilogueGradDesc, dz, a, b, z_in, da, db, db_in, dbias, dbias_in, workspace,
                           dy=None, z=None, stream=None, raise_on_error: bool = True) -> int:
    """da = (dz @ b^T) * act_in'(z_in), db = db_in + a^T @ dz, dbias = dbias_in + column sums of dz; with the
    descriptor's act, dz = dy * act'(z) is computed first.  Any of da, db, dbias may be None."""
    buf = _Buffers("gemm_epilogue_grad_run")
    m, n, k = desc.m, desc.n, desc.k
    st = lib().gemm_epilogue_grad_run(
        byref(desc), buf("dy", dy, desc.dy_type, m, n, desc.lddy), buf("z", z, BF16, m, n, desc.ldz),
        buf("dz", dz, BF16, m, n, desc.lddz), buf("a", a, BF16, m, k, desc.lda), buf("b", b, BF16, k, n, desc.ldb),
        buf("z_in", z_in, BF16, m, k, desc.ldz_in), buf("da", da, desc.da_type, m, k, desc.ldda),
        buf("db", db, desc.db_type, k, n, desc.lddb), buf("db_in", db_in, desc.db_type, k, n, desc.lddb),
        buf("dbias", dbias, F32, 1, n), buf("dbias_in", dbias_in, F32, 1, n),
        _workspace(buf, workspace, lib().gemm_epilogue_grad_workspace_bytes, desc), _stream(stream))
    return _check(st, "gemm_epilogue_grad_run", raise_on_error)


def moe_layer_desc(tokens, hidden, inter, experts, topk, act="silu", gated=True, w_type="bf16", out_type="bf16",
                   norm_topk=True) -> MoeLayerDesc:
    return MoeLayerDesc(tokens, hidden, inter, experts, topk, _act(act), int(gated), _type(w_type), _type(out_type),
                        int(norm_topk), 0)


def moe_layer_workspace_bytes(desc: MoeLayerDesc) -> int:
    return lib().moe_layer_workspace_bytes(byref(desc))


def moe_layer_run(desc: MoeLayerDesc, x, router, topk_idx, gates, w1, w1_scale, w2, w2_scale, out, workspace,
                  stream=None, raise_on_error: bool = True) -> int:
    """The whole layer for a few tokens; with a router, topk_idx and gates are written, else read."""
    buf = _Buffers("moe_layer_run")
    t, h, i, e, k = desc.tokens, desc.hidden, desc.inter, desc.experts, desc.topk
    n1, w = (2 * i if desc.gated else i), desc.w_type
    st = lib().moe_layer_run(
        byref(desc), buf("x", x, BF16, t, h), buf("router", router, BF16, h, e), buf("topk_idx", topk_idx, _INT32, t, k),
        buf("gates", gates, F32, t, k), buf("w1", w1, w, e * h, n1), buf("w1_scale", w1_scale, F32, e, n1),
        buf("w2", w2, w, e * i, h), buf("w2_scale", w2_scale, F32, e, h), buf("out", out, desc.out_type, t, h),
        _workspace(buf, workspace, lib().moe_layer_workspace_bytes, desc), _stream(stream))
    return _check(st, "moe_layer_run", raise_on_error)


class GradClipPlan:
    """Owns a grad_clip_plan_t, and keeps the tensors it was made of."""

    def __init__(self, src, dst=None):
        """src: tensors (bfloat16 or float32); dst: as many (None entries: only in the norm), or None to clip in place."""
        import torch
        src = list(src)
        dst = list(src) if dst is None else list(dst)
        if len(src) != len(dst):
            raise OvlError(OVL_EINVAL, "grad_clip_plan: as many outputs as inputs")
        buf = _Buffers("grad_clip_plan")
        arr = (GradClipTensor * max(1, len(src)))()
        for i, (s, d) in enumerate(zip(src, dst)):
            if s.dtype not in (torch.bfloat16, torch.float32) or (d is not None and d.dtype != s.dtype):
                buf.refuse(f"tensor {i}", "is not bfloat16 or float32, or its output is of another type")
            if not s.is_contiguous() or (d is not None and (not d.is_contiguous() or d.numel() != s.numel())):
                buf.refuse(f"tensor {i}", "is not dense, or its output is of another size")
            n, kind = s.numel(), F32 if s.dtype == torch.float32 else BF16
            arr[i] = GradClipTensor(buf(f"tensor {i}", s, kind, 1, n) or None, buf(f"output {i}", d, kind, 1, n) or None,
                                    n, kind, 0)
        self.tensors = (src, dst)
        self.device = buf.device
        h = c_void_p()
        _check(lib().grad_clip_plan(arr, len(src), byref(h)), "grad_clip_plan", True)
        self.handle = h
        self.workspace_bytes = lib().grad_clip_workspace_bytes(h)

    def _here(self, buf):
        if buf.device != self.device:
            buf.refuse("plan", "is of tensors on another device than the current one")

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.grad_clip_plan_destroy(h)
            self.handle = None


def grad_clip_plan(src, dst=None) -> GradClipPlan:
    return GradClipPlan(src, dst)


def grad_clip_upload(plan: GradClipPlan, workspace, stream=None, raise_on_error: bool = True) -> int:
    buf = _Buffers("grad_clip_upload")
    plan._here(buf)
    ws = buf("workspace", workspace, _BYTES, 1, plan.workspace_bytes)
    return _check(lib().grad_clip_upload(plan.handle, ws, _stream(stream)), "grad_clip_upload", raise_on_error)


def grad_norm_clip_run(plan: GradClipPlan, max_norm: float, norm, workspace, stream=None,
                       raise_on_error: bool = True) -> int:
    """norm (float32 [1]) = the global norm; every dst = src * min(1, max_norm / (norm + 1e-6))."""
    buf = _Buffers("grad_norm_clip_run")
    plan._here(buf)
    st = lib().grad_norm_clip_run(plan.handle, max_norm, buf("norm", norm, F32, 1, 1),
                                  buf("workspace", workspace, _BYTES, 1, plan.workspace_bytes), _stream(stream))
    return _check(st, "grad_norm_clip_run", raise_on_error)


# ------------------------------------------------------------------ flags, errors, copy

def ovl_flags_reset(flags, flag_bytes: int, workspace, ws_bytes: int, stream=None) -> None:
    _check(lib().ovl_flags_reset(_ptr(flags), flag_bytes, _ptr(workspace), ws_bytes, _stream(stream)),
           "ovl_flags_reset", True)


def ovl_check(workspace, stream=None, raise_on_error: bool = True):
    """Returns (status, (site, flag index, observed, awaited))."""
    detail = (c_int64 * 4)()
    st = lib().ovl_check(_ptr(workspace), detail, _stream(stream))
    _check(st, "ovl_check", raise_on_error)
    return st, tuple(detail)


def ovl_copy(dst, src, nbytes: int, blocks: int = 0, stream=None) -> None:
    _check(lib().ovl_copy(_ptr(dst), _ptr(src), nbytes, blocks, _stream(stream)), "ovl_copy", True)
