"""ctypes binding of libulysses.so: argument marshalling only.

Every function has the name of the C entry point it calls and takes torch
tensors (device memory), plain ints and an optional CUDA stream; all work
happens in the library's kernels.  There is no fallback: if the library
cannot be loaded, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build


# return codes, as in include/ulysses.h
ULYSSES_OK = 0
ULYSSES_ERR_ARG = 1
ULYSSES_ERR_DIVISIBILITY = 2
ULYSSES_ERR_ALIGN = 3
ULYSSES_ERR_WINDOW = 4
ULYSSES_ERR_WORKSPACE = 5
ULYSSES_ERR_CUDA = 6
ULYSSES_ERR_DEVICE = 7
ULYSSES_ERR_UNSUPPORTED = 8
ULYSSES_PLAN_CAUSAL = 1
ULYSSES_PLAN_PAIR_ATTENTION = 2
ULYSSES_PLAN_DETERMINISTIC = 4
ULYSSES_KV4_CAUSAL = 1
ULYSSES_KV4_WEIGHTS = 2
MAX_SEQS = 64
MAX_WINDOW_BYTES = 1024 ** 3

EXPORTS = (
    "ulysses_plan", "ulysses_plan_ex", "ulysses_plan_destroy", "ulysses_plan_padded_tokens", "ulysses_plan_plane_chunk",
    "ulysses_plan_window_bytes_per_plane", "ulysses_workspace_bytes", "ulysses_repack_fwd",
    "ulysses_repack_bwd", "ulysses_attn_fwd", "ulysses_layer_fwd", "ulysses_layer_fwd_host",
    "ulysses_last_device_error", "ulysses_strerror",
    "ulysses_layer_fwd_fused_noalloc", "ulysses_prologue_repack_fwd",
    "ulysses_lse_bytes", "ulysses_attn_fwd_lse", "ulysses_attn_bwd_workspace_bytes", "ulysses_attn_bwd",
    "ulysses_layer_bwd_workspace_bytes", "ulysses_layer_bwd", "ulysses_repack_fwd_fp8", "ulysses_attn_fwd_fp8",
    "ulysses_workspace_bytes_fp8", "ulysses_layer_fwd_fp8", "ulysses_repack_fwd_push", "ulysses_attn_fwd_push",
    "ulysses_repack_bwd_push", "ulysses_attn_fwd_lse_slab", "ulysses_attn_bwd_slab", "ulysses_a2a_pack",
    "ulysses_a2a_unpack", "ulysses_layer_fwd_fp8_host",
    "ulysses_kv4_plan", "ulysses_kv4_plan_destroy", "ulysses_kv4_cache_bytes", "ulysses_kv4_weight_offset",
    "ulysses_kv4_position_offset", "ulysses_kv4_append", "ulysses_kv4_load", "ulysses_kv4_attn_workspace_bytes",
    "ulysses_kv4_attn", "ulysses_kv4_evict", "ulysses_kv4_last_device_error",
)


class UlyssesError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: error {code}: {strerror(code)}")


_lock = threading.Lock()
_handle: ctypes.CDLL | None = None


def library_path() -> str:
    """The library this process loads: $ULYSSES_LIBRARY when set (for
    example the bounds-checked libulysses_debug.so), else the in-tree
    libulysses.so."""
    return os.environ.get("ULYSSES_LIBRARY") or _build.LIB


def load() -> ctypes.CDLL:
    """Load (building first if the sources are newer) and type the library."""
    global _handle
    with _lock:
        if _handle is not None:
            return _handle
        path = os.environ.get("ULYSSES_LIBRARY") or _build.ensure_built()
        if not os.path.exists(path):
            raise ImportError(f"libulysses library missing at {path}")
        lib = ctypes.CDLL(path)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        lib.ulysses_plan.argtypes = [ctypes.POINTER(vp), i64, i32, i32, i32, i32, i64, i64, i64,
                                     ctypes.POINTER(ctypes.c_int32), i32]
        lib.ulysses_plan.restype = ctypes.c_int
        lib.ulysses_plan_ex.argtypes = [ctypes.POINTER(vp), i64, i32, i32, i32, i32, i64, i64, i64,
                                        ctypes.POINTER(ctypes.c_int32), i32, ctypes.c_uint32]
        lib.ulysses_plan_ex.restype = ctypes.c_int
        lib.ulysses_plan_destroy.argtypes = [vp]
        lib.ulysses_plan_destroy.restype = None
        lib.ulysses_plan_padded_tokens.argtypes = [vp]
        lib.ulysses_plan_padded_tokens.restype = i64
        lib.ulysses_plan_plane_chunk.argtypes = [vp]
        lib.ulysses_plan_plane_chunk.restype = i32
        lib.ulysses_plan_window_bytes_per_plane.argtypes = [vp]
        lib.ulysses_plan_window_bytes_per_plane.restype = i64
        lib.ulysses_workspace_bytes.argtypes = [vp]
        lib.ulysses_workspace_bytes.restype = sz
        lib.ulysses_repack_fwd.argtypes = [vp, vp, vp, vp]
        lib.ulysses_repack_fwd.restype = ctypes.c_int
        lib.ulysses_prologue_repack_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, ctypes.c_float, vp]
        lib.ulysses_prologue_repack_fwd.restype = ctypes.c_int
        lib.ulysses_lse_bytes.argtypes = [vp]
        lib.ulysses_lse_bytes.restype = sz
        lib.ulysses_attn_fwd_lse.argtypes = [vp, vp, vp, vp, ctypes.c_float, vp]
        lib.ulysses_attn_fwd_lse.restype = ctypes.c_int
        lib.ulysses_attn_bwd_workspace_bytes.argtypes = [vp]
        lib.ulysses_attn_bwd_workspace_bytes.restype = sz
        lib.ulysses_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, sz, ctypes.c_float, vp]
        lib.ulysses_attn_bwd.restype = ctypes.c_int
        lib.ulysses_layer_bwd_workspace_bytes.argtypes = [vp]
        lib.ulysses_layer_bwd_workspace_bytes.restype = sz
        lib.ulysses_layer_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ulysses_layer_bwd.restype = ctypes.c_int
        lib.ulysses_repack_bwd.argtypes = [vp, vp, vp, i32, vp]
        lib.ulysses_repack_bwd.restype = ctypes.c_int
        lib.ulysses_attn_fwd.argtypes = [vp, vp, vp, ctypes.c_float, vp]
        lib.ulysses_attn_fwd.restype = ctypes.c_int
        lib.ulysses_layer_fwd.argtypes = [vp, vp, vp, vp, sz, i32, vp]
        lib.ulysses_layer_fwd.restype = ctypes.c_int
        lib.ulysses_layer_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, sz, i32, vp]
        lib.ulysses_layer_fwd_host.restype = ctypes.c_int
        lib.ulysses_last_device_error.argtypes = [vp, vp]
        lib.ulysses_last_device_error.restype = ctypes.c_int
        lib.ulysses_strerror.argtypes = [ctypes.c_int]
        lib.ulysses_strerror.restype = ctypes.c_char_p
        lib.ulysses_layer_fwd_fused_noalloc.argtypes = [vp, vp, i64, i32, i32, i32, i32, i64, i64,
                                                        ctypes.POINTER(ctypes.c_int32), i32,
                                                        ctypes.POINTER(ctypes.c_int32), vp]
        lib.ulysses_layer_fwd_fused_noalloc.restype = ctypes.c_int
        lib.ulysses_repack_fwd_fp8.argtypes = [vp, vp, vp, vp]
        lib.ulysses_repack_fwd_fp8.restype = ctypes.c_int
        lib.ulysses_attn_fwd_fp8.argtypes = [vp, vp, vp, ctypes.c_float, vp]
        lib.ulysses_attn_fwd_fp8.restype = ctypes.c_int
        lib.ulysses_workspace_bytes_fp8.argtypes = [vp]
        lib.ulysses_workspace_bytes_fp8.restype = sz
        lib.ulysses_layer_fwd_fp8.argtypes = [vp, vp, vp, vp, sz, vp]
        lib.ulysses_layer_fwd_fp8.restype = ctypes.c_int
        lib.ulysses_repack_fwd_push.argtypes = [vp, i32, vp, ctypes.POINTER(vp), i32, vp]
        lib.ulysses_repack_fwd_push.restype = ctypes.c_int
        lib.ulysses_attn_fwd_push.argtypes = [vp, i32, vp, ctypes.POINTER(vp), ctypes.c_float, vp]
        lib.ulysses_attn_fwd_push.restype = ctypes.c_int
        lib.ulysses_repack_bwd_push.argtypes = [vp, i32, vp, ctypes.POINTER(vp), i32, vp]
        lib.ulysses_repack_bwd_push.restype = ctypes.c_int
        lib.ulysses_layer_fwd_fp8_host.argtypes = [vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ulysses_layer_fwd_fp8_host.restype = ctypes.c_int
        lib.ulysses_a2a_pack.argtypes = [vp, vp, i32, i32, vp, vp]
        lib.ulysses_a2a_pack.restype = ctypes.c_int
        lib.ulysses_a2a_unpack.argtypes = [vp, vp, vp, i32, i32, vp]
        lib.ulysses_a2a_unpack.restype = ctypes.c_int
        lib.ulysses_attn_fwd_lse_slab.argtypes = [vp, vp, vp, vp, ctypes.c_float, vp]
        lib.ulysses_attn_fwd_lse_slab.restype = ctypes.c_int
        lib.ulysses_attn_bwd_slab.argtypes = [vp, vp, vp, vp, vp, vp, vp, sz, ctypes.c_float, vp]
        lib.ulysses_attn_bwd_slab.restype = ctypes.c_int
        lib.ulysses_kv4_plan.argtypes = [ctypes.POINTER(vp), i32, i32, i32, i64]
        lib.ulysses_kv4_plan.restype = ctypes.c_int
        lib.ulysses_kv4_plan_destroy.argtypes = [vp]
        lib.ulysses_kv4_plan_destroy.restype = None
        for name in ("ulysses_kv4_cache_bytes", "ulysses_kv4_weight_offset", "ulysses_kv4_position_offset"):
            getattr(lib, name).argtypes = [vp]
            getattr(lib, name).restype = sz
        lib.ulysses_kv4_append.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i32, vp, vp, vp, vp]
        lib.ulysses_kv4_append.restype = ctypes.c_int
        lib.ulysses_kv4_load.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i32, vp, vp, vp]
        lib.ulysses_kv4_load.restype = ctypes.c_int
        lib.ulysses_kv4_attn_workspace_bytes.argtypes = [vp, i32, i32, ctypes.c_uint32]
        lib.ulysses_kv4_attn_workspace_bytes.restype = sz
        lib.ulysses_kv4_attn.argtypes = [vp, vp, vp, i32, i32, i64, i64, vp, vp, vp, ctypes.c_float, ctypes.c_uint32,
                                         vp, sz, vp]
        lib.ulysses_kv4_attn.restype = ctypes.c_int
        lib.ulysses_kv4_evict.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, vp]
        lib.ulysses_kv4_evict.restype = ctypes.c_int
        lib.ulysses_kv4_last_device_error.argtypes = [vp, vp]
        lib.ulysses_kv4_last_device_error.restype = ctypes.c_int
        _handle = lib
        return lib


def strerror(code: int) -> str:
    return load().ulysses_strerror(int(code)).decode()


def _check(code: int, where: str) -> None:
    if code != ULYSSES_OK:
        raise UlyssesError(code, where)


def _ptr(t) -> int | None:
    """Device (or host) address of a tensor, or an int address as given."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Plan:
    """Owner of a ulysses_plan_t*; destroyed with the object."""

    def __init__(self, handle: int, N: int, H: int, D: int, P: int, planes: int, cu_seqlens, causal: bool = False):
        self._h = ctypes.c_void_p(handle)
        self.N, self.H, self.D, self.P, self.planes = N, H, D, P, planes
        self.causal = bool(causal)
        self.cu_seqlens = None if cu_seqlens is None else [int(x) for x in cu_seqlens]

    @property
    def handle(self) -> ctypes.c_void_p:
        if not self._h:
            raise ValueError("plan destroyed")
        return self._h

    @property
    def padded_tokens(self) -> int:
        return load().ulysses_plan_padded_tokens(self.handle)

    @property
    def rows_per_rank(self) -> int:
        """Nl = Np / P: the sequence rows each rank owns."""
        return self.padded_tokens // self.P

    @property
    def plane_chunk(self) -> int:
        return load().ulysses_plan_plane_chunk(self.handle)

    @property
    def window_bytes_per_plane(self) -> int:
        return load().ulysses_plan_window_bytes_per_plane(self.handle)

    @property
    def workspace_bytes(self) -> int:
        return load().ulysses_workspace_bytes(self.handle)

    @property
    def workspace_bytes_fp8(self) -> int:
        return load().ulysses_workspace_bytes_fp8(self.handle)

    @property
    def lse_bytes(self) -> int:
        return load().ulysses_lse_bytes(self.handle)

    @property
    def lse_row_stride(self) -> int:
        """Floats between the lse rows of consecutive (rank, local head) pairs."""
        return self.lse_bytes // 4 // self.H

    @property
    def attn_bwd_workspace_bytes(self) -> int:
        return load().ulysses_attn_bwd_workspace_bytes(self.handle)

    @property
    def slab_lse_bytes(self) -> int:
        """lse bytes of one rank's slab (ulysses_attn_fwd_lse_slab)."""
        return self.lse_bytes // self.P

    @property
    def slab_attn_bwd_workspace_bytes(self) -> int:
        """Workspace of ulysses_attn_bwd_slab."""
        return self.attn_bwd_workspace_bytes // self.P

    @property
    def layer_bwd_workspace_bytes(self) -> int:
        return load().ulysses_layer_bwd_workspace_bytes(self.handle)

    def destroy(self) -> None:
        if self._h:
            load().ulysses_plan_destroy(self._h)
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.destroy()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass


def ulysses_plan(N: int, H: int, D: int, P: int, planes: int, token_stride: int = 0, plane_stride: int = 0,
                 plane_chunk: int = 0, cu_seqlens=None, causal: bool = False, pair_cta: bool = False,
                 deterministic: bool = False) -> Plan:
    """ulysses_plan (or ulysses_plan_ex with ULYSSES_PLAN_CAUSAL when causal,
    ULYSSES_PLAN_PAIR_ATTENTION when pair_cta, ULYSSES_PLAN_DETERMINISTIC when
    deterministic)."""
    lib = load()
    h = ctypes.c_void_p()
    if cu_seqlens is None:
        arr, ns = None, 0
    else:
        vals = [int(x) for x in cu_seqlens]
        arr = (ctypes.c_int32 * len(vals))(*vals)
        ns = len(vals) - 1
    flags = ((ULYSSES_PLAN_CAUSAL if causal else 0) | (ULYSSES_PLAN_PAIR_ATTENTION if pair_cta else 0)
             | (ULYSSES_PLAN_DETERMINISTIC if deterministic else 0))
    if flags:
        code = lib.ulysses_plan_ex(ctypes.byref(h), int(N), int(H), int(D), int(P), int(planes), int(token_stride),
                                   int(plane_stride), int(plane_chunk), arr, ns, flags)
    else:
        code = lib.ulysses_plan(ctypes.byref(h), int(N), int(H), int(D), int(P), int(planes), int(token_stride),
                                int(plane_stride), int(plane_chunk), arr, ns)
    _check(code, "ulysses_plan")
    return Plan(h.value, N, H, D, P, planes, cu_seqlens, causal)


def ulysses_repack_fwd(plan: Plan, src_seq, dst_heads, stream=None) -> None:
    _check(load().ulysses_repack_fwd(plan.handle, _ptr(src_seq), _ptr(dst_heads), _stream(stream)),
           "ulysses_repack_fwd")


def ulysses_prologue_repack_fwd(plan: Plan, src_seq, dst_heads, norm_q_weight, norm_k_weight, cos, sin,
                                rotary_dim: int, eps: float = 1e-5, stream=None) -> None:
    _check(load().ulysses_prologue_repack_fwd(plan.handle, _ptr(src_seq), _ptr(dst_heads), _ptr(norm_q_weight),
                                              _ptr(norm_k_weight), _ptr(cos), _ptr(sin), int(rotary_dim),
                                              float(eps), _stream(stream)), "ulysses_prologue_repack_fwd")


def ulysses_attn_fwd_lse(plan: Plan, qkv_heads, out_heads, lse, softmax_scale: float, stream=None) -> None:
    _check(load().ulysses_attn_fwd_lse(plan.handle, _ptr(qkv_heads), _ptr(out_heads), _ptr(lse),
                                       float(softmax_scale), _stream(stream)), "ulysses_attn_fwd_lse")


def ulysses_attn_bwd(plan: Plan, qkv_heads, out_heads, dout_heads, lse, dqkv_heads, workspace,
                     softmax_scale: float, workspace_bytes: int | None = None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(load().ulysses_attn_bwd(plan.handle, _ptr(qkv_heads), _ptr(out_heads), _ptr(dout_heads), _ptr(lse),
                                   _ptr(dqkv_heads), _ptr(workspace), int(workspace_bytes), float(softmax_scale),
                                   _stream(stream)), "ulysses_attn_bwd")


def ulysses_a2a_pack(plan: Plan, src_shard, planes: int, plane: int, send, stream=None) -> None:
    """Plane `plane` of a shard [Nl, planes, H, D] -> all-to-all send buffer [P, Nl, Hl, D]."""
    _check(load().ulysses_a2a_pack(plan.handle, _ptr(src_shard), int(planes), int(plane), _ptr(send),
                                   _stream(stream)), "ulysses_a2a_pack")


def ulysses_a2a_unpack(plan: Plan, recv, out_shard, planes: int, plane: int, stream=None) -> None:
    """All-to-all receive buffer [P, Nl, Hl, D] -> plane `plane` of a shard [Nl, planes, H, D]."""
    _check(load().ulysses_a2a_unpack(plan.handle, _ptr(recv), _ptr(out_shard), int(planes), int(plane),
                                     _stream(stream)), "ulysses_a2a_unpack")


def ulysses_attn_fwd_lse_slab(plan: Plan, heads, out_heads, lse, softmax_scale: float, stream=None) -> None:
    """Attention over one rank's head slab [C, Np, Hl, D] with its lse."""
    _check(load().ulysses_attn_fwd_lse_slab(plan.handle, _ptr(heads), _ptr(out_heads), _ptr(lse),
                                            float(softmax_scale), _stream(stream)), "ulysses_attn_fwd_lse_slab")


def ulysses_attn_bwd_slab(plan: Plan, heads, out_heads, dout_heads, lse, dqkv_heads, workspace,
                          softmax_scale: float, workspace_bytes: int | None = None, stream=None) -> None:
    """The attention backward of one rank's head slab: dqkv_heads [3, Np, Hl, D]."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(load().ulysses_attn_bwd_slab(plan.handle, _ptr(heads), _ptr(out_heads), _ptr(dout_heads), _ptr(lse),
                                        _ptr(dqkv_heads), _ptr(workspace), int(workspace_bytes),
                                        float(softmax_scale), _stream(stream)), "ulysses_attn_bwd_slab")


def ulysses_layer_bwd(plan: Plan, qkv_heads, out_heads, lse, dout_seq, dqkv_seq, workspace,
                      workspace_bytes: int | None = None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(load().ulysses_layer_bwd(plan.handle, _ptr(qkv_heads), _ptr(out_heads), _ptr(lse), _ptr(dout_seq),
                                    _ptr(dqkv_seq), _ptr(workspace), int(workspace_bytes), _stream(stream)),
           "ulysses_layer_bwd")


def ulysses_repack_bwd(plan: Plan, src_heads, dst_seq, planes: int, stream=None) -> None:
    _check(load().ulysses_repack_bwd(plan.handle, _ptr(src_heads), _ptr(dst_seq), int(planes), _stream(stream)),
           "ulysses_repack_bwd")


def ulysses_attn_fwd(plan: Plan, qkv_heads, out_heads, softmax_scale: float, stream=None) -> None:
    _check(load().ulysses_attn_fwd(plan.handle, _ptr(qkv_heads), _ptr(out_heads), float(softmax_scale),
                                   _stream(stream)), "ulysses_attn_fwd")


def _ptr_table(ptrs):
    """Host array of device pointers (tensors or int addresses), indexed by rank."""
    if ptrs is None:
        return None
    vals = [_ptr(t) for t in ptrs]
    return (ctypes.c_void_p * max(1, len(vals)))(*vals)


def ulysses_repack_fwd_push(plan: Plan, rank: int, src_shard, dst_heads, planes: int | None = None,
                            stream=None) -> None:
    """Rank `rank` pushes its shard [Nl, planes, H, D] into every rank's head
    slab dst_heads[r] = T_r [planes, Np, Hl, D] (device pointers, one per
    rank); planes defaults to the plan's C."""
    if dst_heads is not None and len(dst_heads) != plan.P:
        raise UlyssesError(ULYSSES_ERR_ARG, "ulysses_repack_fwd_push: one destination per rank")
    planes = plan.planes if planes is None else int(planes)
    _check(load().ulysses_repack_fwd_push(plan.handle, int(rank), _ptr(src_shard), _ptr_table(dst_heads), planes,
                                          _stream(stream)), "ulysses_repack_fwd_push")


def ulysses_attn_fwd_push(plan: Plan, rank: int, heads, dst_seq, softmax_scale: float, stream=None) -> None:
    """Attention over rank `rank`'s head slab T_r with each output row stored
    into its owning rank's shard dst_seq[q] = O_q [Nl, H, D]."""
    if dst_seq is not None and len(dst_seq) != plan.P:
        raise UlyssesError(ULYSSES_ERR_ARG, "ulysses_attn_fwd_push: one destination per rank")
    _check(load().ulysses_attn_fwd_push(plan.handle, int(rank), _ptr(heads), _ptr_table(dst_seq),
                                        float(softmax_scale), _stream(stream)), "ulysses_attn_fwd_push")


def ulysses_repack_bwd_push(plan: Plan, rank: int, src_heads, dst_seq, planes: int, stream=None) -> None:
    """Rank `rank` pushes its head rows [planes, Np, Hl, D] into every rank's
    shard dst_seq[q] = [Nl, planes, H, D]."""
    if dst_seq is not None and len(dst_seq) != plan.P:
        raise UlyssesError(ULYSSES_ERR_ARG, "ulysses_repack_bwd_push: one destination per rank")
    _check(load().ulysses_repack_bwd_push(plan.handle, int(rank), _ptr(src_heads), _ptr_table(dst_seq), int(planes),
                                          _stream(stream)), "ulysses_repack_bwd_push")


def ulysses_repack_fwd_fp8(plan: Plan, src_seq, dst_heads_fp8, stream=None) -> None:
    _check(load().ulysses_repack_fwd_fp8(plan.handle, _ptr(src_seq), _ptr(dst_heads_fp8), _stream(stream)),
           "ulysses_repack_fwd_fp8")


def ulysses_attn_fwd_fp8(plan: Plan, qkv_heads_fp8, out_heads, softmax_scale: float, stream=None) -> None:
    _check(load().ulysses_attn_fwd_fp8(plan.handle, _ptr(qkv_heads_fp8), _ptr(out_heads), float(softmax_scale),
                                       _stream(stream)), "ulysses_attn_fwd_fp8")


def ulysses_layer_fwd_fp8(plan: Plan, qkv_seq, out_seq, workspace, workspace_bytes: int | None = None,
                          stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().ulysses_layer_fwd_fp8(plan.handle, _ptr(qkv_seq), _ptr(out_seq), _ptr(workspace),
                                        int(workspace_bytes), _stream(stream)), "ulysses_layer_fwd_fp8")


def ulysses_layer_fwd(plan: Plan, qkv_seq, out_seq, workspace=None, workspace_bytes: int | None = None,
                      fused: int = 0, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().ulysses_layer_fwd(plan.handle, _ptr(qkv_seq), _ptr(out_seq), _ptr(workspace),
                                    int(workspace_bytes), int(fused), _stream(stream)), "ulysses_layer_fwd")


def ulysses_layer_fwd_host(plan: Plan, host_qkv_seq, host_out_seq, dev_qkv_seq, dev_out_seq, workspace=None,
                           workspace_bytes: int | None = None, fused: int = 0, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().ulysses_layer_fwd_host(plan.handle, _ptr(host_qkv_seq), _ptr(host_out_seq), _ptr(dev_qkv_seq),
                                         _ptr(dev_out_seq), _ptr(workspace), int(workspace_bytes), int(fused),
                                         _stream(stream)), "ulysses_layer_fwd_host")


def ulysses_layer_fwd_fp8_host(plan: Plan, host_qkv_seq, host_out_seq, dev_qkv_seq, dev_out_seq, workspace,
                               workspace_bytes: int | None = None, stream=None) -> None:
    """The FP8 layer from host buffers, streamed by head groups (workspace_bytes_fp8)."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().ulysses_layer_fwd_fp8_host(plan.handle, _ptr(host_qkv_seq), _ptr(host_out_seq), _ptr(dev_qkv_seq),
                                             _ptr(dev_out_seq), _ptr(workspace), int(workspace_bytes),
                                             _stream(stream)), "ulysses_layer_fwd_fp8_host")


def ulysses_last_device_error(plan: Plan, stream=None) -> int:
    return load().ulysses_last_device_error(plan.handle, _stream(stream))


def ulysses_layer_fwd_fused_noalloc(qkv_seq, out_seq, N: int, H: int, D: int, P: int, planes: int,
                                    token_stride: int = 0, plane_stride: int = 0, cu_seqlens=None,
                                    check: bool = False, stream=None) -> int:
    """The fused layer without a plan and without any device allocation.

    Returns the kernel's error bits when ``check`` is true (the call then
    synchronises the stream; non-zero bits are returned, not raised), else 0.
    Argument and CUDA errors raise UlyssesError.
    """
    if cu_seqlens is None:
        arr, ns = None, 0
    else:
        vals = [int(x) for x in cu_seqlens]
        arr = (ctypes.c_int32 * len(vals))(*vals)
        ns = len(vals) - 1
    status = ctypes.c_int32(0)
    code = load().ulysses_layer_fwd_fused_noalloc(_ptr(qkv_seq), _ptr(out_seq), int(N), int(H), int(D), int(P),
                                                  int(planes), int(token_stride), int(plane_stride), arr, ns,
                                                  ctypes.byref(status) if check else None, _stream(stream))
    if check and code == ULYSSES_ERR_DEVICE:
        return status.value
    _check(code, "ulysses_layer_fwd_fused_noalloc")
    return status.value


# ---------------------------------------------------------------- 4-bit K/V cache


class KV4Plan:
    """Owner of a ulysses_kv4_t*: the geometry of 4-bit K/V caches."""

    def __init__(self, handle: int, batch: int, heads: int, D: int, capacity: int):
        self._h = ctypes.c_void_p(handle)
        self.batch, self.heads, self.D, self.capacity = batch, heads, D, capacity
        lib = load()
        self.cache_bytes: int = lib.ulysses_kv4_cache_bytes(self._h)
        self.weight_offset: int = lib.ulysses_kv4_weight_offset(self._h)
        self.position_offset: int = lib.ulysses_kv4_position_offset(self._h)

    @property
    def handle(self) -> ctypes.c_void_p:
        if not self._h:
            raise ValueError("plan destroyed")
        return self._h

    def workspace_bytes(self, q_heads: int, q_len: int, weights: bool = False) -> int:
        """Workspace of ulysses_kv4_attn."""
        return load().ulysses_kv4_attn_workspace_bytes(self.handle, _kv4_int(q_heads), _kv4_int(q_len),
                                                       ULYSSES_KV4_WEIGHTS if weights else 0)

    def destroy(self) -> None:
        if self._h:
            load().ulysses_kv4_plan_destroy(self._h)
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.destroy()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass


def ulysses_kv4_plan(batch: int, heads: int, D: int, capacity: int) -> KV4Plan:
    """The geometry of 4-bit K/V caches: `capacity` slots (a multiple of 32)
    for each of `batch` sequences and `heads` K/V heads of D = 128."""
    h = ctypes.c_void_p()
    _check(load().ulysses_kv4_plan(ctypes.byref(h), _kv4_int(batch), _kv4_int(heads), _kv4_int(D),
                                   max(-1, min(int(capacity), 2 ** 63 - 1))), "ulysses_kv4_plan")
    return KV4Plan(h.value, int(batch), int(heads), int(D), int(capacity))


# A decoding step makes these calls once a layer, so what they check of their
# tensors is kept to a few microseconds.
_types: dict = {}


def _kv4_types() -> dict:
    if not _types:
        import torch
        _types.update(tensor=torch.Tensor, uint8=torch.uint8, bf16=torch.bfloat16, int32=torch.int32,
                      fp32=torch.float32, device=torch.cuda.current_device,
                      raw_stream=getattr(torch._C, "_cuda_getCurrentRawStream", None))
    return _types


def _kv4_stream(stream, t: dict):
    if stream is None and t["raw_stream"] is not None:
        return t["raw_stream"](t["device"]())
    return _stream(stream)


def _kv4_flat(where: str, name: str, x, tensor, dtype, numel: int, dev: int):
    """The address of a contiguous CUDA tensor on device dev of this type with at least numel elements."""
    if not isinstance(x, tensor) or not x.is_cuda or x.dtype is not dtype:
        raise TypeError(f"{where}: {name} must be a CUDA tensor of type {dtype}")
    if x.numel() < numel or not x.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous with at least {numel} elements")
    if x.get_device() != dev:
        raise ValueError(f"{where}: {name} is not on the current device")
    return x.data_ptr()


def _kv4_cache(where: str, name: str, kv: KV4Plan, x, t: dict):
    """The address of a cache of this plan, and the current device, which has to be its own."""
    if not isinstance(x, t["tensor"]) or not x.is_cuda:
        raise TypeError(f"{where}: {name} must be a CUDA tensor of type {t['uint8']}")
    dev = t["device"]()
    return _kv4_flat(where, name, x, t["tensor"], t["uint8"], kv.cache_bytes, dev), dev


def _kv4_strides(shape, stride) -> tuple:
    return tuple(0 if n == 1 else d for n, d in zip(shape, stride))


def _kv4_int(x) -> int:
    """An int32 argument; what is outside int32 becomes its end, which the library refuses."""
    return max(-1, min(int(x), 2 ** 31 - 1))


def _kv4_rows(where: str, kv: KV4Plan, cache, k, v, cu, start, t: dict):
    """The common arguments of append and load: K and V of one shape and
    layout, [rows, heads, D] or, split over ranks, [P, rows, heads / P, D]."""
    T, i32, bf16 = t["tensor"], t["int32"], t["bf16"]
    c, dev = _kv4_cache(where, "cache", kv, cache, t)
    for name, x in (("k", k), ("v", v)):
        if not isinstance(x, T) or not x.is_cuda or x.dtype is not bf16:
            raise TypeError(f"{where}: {name} must be a CUDA tensor of type {bf16}")
        if x.get_device() != dev:
            raise ValueError(f"{where}: {name} is not on the current device")
    shape, stride = k.shape, k.stride()
    n = len(shape)
    if n not in (3, 4) or shape[-1] != kv.D or stride[-1] != 1:
        raise ValueError(f"{where}: k and v are [rows, heads, {kv.D}] or [ranks, rows, heads / ranks, {kv.D}]")
    if 1 in shape:   # the stride of a single row or head says nothing
        stride = _kv4_strides(shape, stride)
        same = v.shape == shape and stride == _kv4_strides(shape, v.stride())
    else:
        same = v.shape == shape and v.stride() == stride
    if not same:
        raise ValueError(f"{where}: k and v must have one shape and layout")
    ranks, rank_stride = (shape[0], stride[0]) if n == 4 else (1, 0)
    if ranks * shape[-2] != kv.heads:
        raise ValueError(f"{where}: {ranks * shape[-2]} heads, the plan has {kv.heads}")
    return (kv.handle, c, k.data_ptr(), v.data_ptr(), shape[-3], stride[-3], stride[-2], rank_stride, shape[-2],
            _kv4_flat(where, "cu", cu, T, i32, kv.batch + 1, dev),
            _kv4_flat(where, "start", start, T, i32, kv.batch, dev))


def ulysses_kv4_append(kv: KV4Plan, cache, k, v, cu, start, pos0=None, stream=None) -> None:
    """Quantise rows of K and V into the cache: rows cu[b] .. cu[b+1]-1 go to
    slots start[b] on of sequence b.  k, v: bf16 [rows, heads, D] (a plane of
    packed rows will do) or [P, rows, heads / P, D] (planes of a head slab).
    pos0: int32 [batch], the position of each sequence's first new row
    (default: its slot)."""
    t = _kv4_types()
    args = _kv4_rows("ulysses_kv4_append", kv, cache, k, v, cu, start, t)
    p = None
    if pos0 is not None:
        p = _kv4_flat("ulysses_kv4_append", "pos0", pos0, t["tensor"], t["int32"], kv.batch, t["device"]())
    if args[4]:
        _check(load().ulysses_kv4_append(*args, p, _kv4_stream(stream, t)), "ulysses_kv4_append")


def ulysses_kv4_load(kv: KV4Plan, cache, k, v, cu, start, stream=None) -> None:
    """Bring slots start[b] on back as bf16 rows cu[b] .. cu[b+1]-1 of k and v
    (layouts as ulysses_kv4_append)."""
    t = _kv4_types()
    args = _kv4_rows("ulysses_kv4_load", kv, cache, k, v, cu, start, t)
    if args[4]:
        _check(load().ulysses_kv4_load(*args, _kv4_stream(stream, t)), "ulysses_kv4_load")


def ulysses_kv4_attn(kv: KV4Plan, cache, q, out, lengths, softmax_scale: float, lse=None, causal: bool = False,
                     weights: bool = False, workspace=None, stream=None) -> None:
    """Attention of q, bf16 [batch, q_len, q_heads, D] (any strides of rows and
    heads), over the cache's slots below lengths [batch] (int32) into out, the
    same shape, contiguous; lse: optional fp32 [batch, q_heads, q_len].
    weights: add each slot's attention weight to the cache's.  workspace: uint8,
    at least kv.workspace_bytes(q_heads, q_len, weights)."""
    where, t = "ulysses_kv4_attn", _kv4_types()
    T = t["tensor"]
    c, dev = _kv4_cache(where, "cache", kv, cache, t)
    if not isinstance(q, T) or not q.is_cuda or q.dtype is not t["bf16"]:
        raise TypeError(f"{where}: q must be a CUDA tensor of type {t['bf16']}")
    if q.get_device() != dev:
        raise ValueError(f"{where}: q is not on the current device")
    shape, stride = q.shape, q.stride()
    if len(shape) != 4 or shape[0] != kv.batch or shape[3] != kv.D or stride[3] != 1:
        raise ValueError(f"{where}: q is [{kv.batch}, q_len, q_heads, {kv.D}]")
    B, q_len, q_heads, D = shape
    if q_len > 1 and B > 1 and stride[0] != q_len * stride[1]:
        raise ValueError(f"{where}: the rows of q must be evenly spaced over sequences and queries")
    token_stride = stride[1] if q_len > 1 else (stride[0] if B > 1 else 0)
    o = _kv4_flat(where, "out", out, T, t["bf16"], B * q_len * q_heads * D, dev)
    if out.shape != shape:
        raise ValueError(f"{where}: out has q's shape")
    ls = None if lse is None else _kv4_flat(where, "lse", lse, T, t["fp32"], B * q_heads * q_len, dev)
    ws, nbytes = None, 0
    if workspace is not None:
        ws, nbytes = _kv4_flat(where, "workspace", workspace, T, t["uint8"], 0, dev), workspace.numel()
    _check(load().ulysses_kv4_attn(kv.handle, c, q.data_ptr(), q_heads, q_len, token_stride,
                                   stride[2] if q_heads > 1 else 0, o, ls, _kv4_flat(where, "lengths", lengths, T, t["int32"], B, dev),
                                   softmax_scale,
                                   (ULYSSES_KV4_CAUSAL if causal else 0) | (ULYSSES_KV4_WEIGHTS if weights else 0),
                                   ws, nbytes, _kv4_stream(stream, t)), where)


def ulysses_kv4_evict(src_kv: KV4Plan, src_cache, dst_kv: KV4Plan, dst_cache, lengths, new_lengths, keep: int,
                      sink: int = 0, recent: int = 0, stream=None) -> None:
    """Move the slots worth keeping (the first `sink`, the last `recent` and
    those of largest accumulated weight, `keep` in all) into dst_cache, in
    their order; new_lengths [batch] gets min(lengths, keep)."""
    where, t = "ulysses_kv4_evict", _kv4_types()
    T, i32 = t["tensor"], t["int32"]
    src, dev = _kv4_cache(where, "src_cache", src_kv, src_cache, t)
    dst, _ = _kv4_cache(where, "dst_cache", dst_kv, dst_cache, t)
    _check(load().ulysses_kv4_evict(src_kv.handle, src, dst_kv.handle, dst,
                                    _kv4_flat(where, "lengths", lengths, T, i32, src_kv.batch, dev),
                                    _kv4_flat(where, "new_lengths", new_lengths, T, i32, src_kv.batch, dev),
                                    _kv4_int(keep), _kv4_int(sink), _kv4_int(recent), _kv4_stream(stream, t)), where)


def ulysses_kv4_last_device_error(kv: KV4Plan, stream=None) -> int:
    return load().ulysses_kv4_last_device_error(kv.handle, _stream(stream))
