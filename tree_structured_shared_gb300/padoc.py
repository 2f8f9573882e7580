"""ctypes binding over libpadoc.so: argument marshalling only.

Every computation runs in the library's CUDA kernels.  The names mirror the C
functions declared in include/padoc.h.  Tensors may be torch tensors (their
data_ptr() is passed) or raw integer device addresses.  There is no CPU path:
if the compiled library is missing, loading fails with an error.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
import sys
from typing import Optional, Sequence

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpadoc.so")

OK, ERR_INVALID, ERR_OOM, ERR_CUDA, ERR_UNSUPPORTED, ERR_DEVICE_TIMEOUT = 0, -1, -2, -3, -4, -5
F32, BF16, I4 = 0, 1, 2
PACK_CANONICAL, PACK_DOCUMENT = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_BANDS, ROPE_RAMP = 0, 1, 2, 3, 4

EXPORTED = [
    "padoc_last_error", "padoc_version", "padoc_tree_desc_build", "padoc_tree_desc_free",
    "padoc_tree_desc_info", "padoc_tree_desc_segments", "padoc_tree_desc_upload",
    "padoc_tree_attn_varlen", "padoc_kv_pool_create", "padoc_kv_pool_destroy", "padoc_kv_alloc",
    "padoc_kv_append", "padoc_kv_fork", "padoc_kv_release", "padoc_kv_seq_info", "padoc_kv_seq_blocks",
    "padoc_kv_block_refcount", "padoc_kv_pool_stats", "padoc_kv_pool_sync", "padoc_kv_pool_device",
    "padoc_debug_kv_pool_rehome", "padoc_debug_set_wait_limit", "padoc_branch_decode_ws_size", "padoc_branch_decode", "padoc_tree_mask_build", "padoc_depths",
    "padoc_device_status", "padoc_decode_plan_create", "padoc_decode_plan_ws_size", "padoc_decode_plan_fused", "padoc_decode_plan_upload",
    "padoc_decode_prefix_pass", "padoc_decode_own_pass", "padoc_decode_plan_free", "padoc_branch_decode_noalloc",
    "padoc_verify_accept", "padoc_kv_commit", "padoc_draft_index_create", "padoc_draft_index_free",
    "padoc_draft_trie", "padoc_draft_trie_batch", "padoc_tree_attn_varlen_bwd_ws_size",
    "padoc_tree_attn_varlen_bwd", "padoc_tree_desc_bwd_plan", "padoc_kv_reserve", "padoc_kv_advance", "padoc_kv_trim",
    "padoc_sched_create", "padoc_sched_destroy", "padoc_sched_submit", "padoc_sched_schedule", "padoc_sched_update",
    "padoc_sched_request", "padoc_sched_output", "padoc_kv_storage_bytes", "padoc_kv_rows_create",
    "padoc_kv_rows_ws_size", "padoc_kv_rows_upload", "padoc_kv_rows_free", "padoc_kv_write", "padoc_kv_gather",
    "padoc_kv_append_rope", "padoc_rope_table", "padoc_rope_apply", "padoc_lm_loss_ws_size", "padoc_lm_loss",
    "padoc_lm_loss_bwd", "padoc_act_bytes", "padoc_act_keep", "padoc_act_restore",
    "padoc_tree_attn_varlen_bwd_kept_ws_size", "padoc_tree_attn_varlen_bwd_kept",
]
NOALLOC_SCRATCH_BYTES = 32 << 20


class PadocError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libpadoc error {code}: {msg}")
        self.code = code


class TreeSpec(C.Structure):
    _fields_ = [("n_pages", C.c_int32), ("prefix_len", C.POINTER(C.c_int32)),
                ("n_regions", C.POINTER(C.c_int32)), ("layout_len", C.POINTER(C.c_int32)),
                ("content_len", C.POINTER(C.c_int32)), ("order", C.c_int32)]


class SchedConfig(C.Structure):
    _fields_ = [("tau", C.c_float), ("n_max", C.c_int32), ("window", C.c_int32), ("max_len", C.c_int32),
                ("fork_token", C.c_int32), ("child_token", C.c_int32), ("eos_token", C.c_int32)]


class SchedStep(C.Structure):
    _fields_ = [("cap", C.c_int32), ("n_admitted", C.c_int32), ("n_preempted", C.c_int32), ("n_active", C.c_int32),
                ("n_pages", C.c_int32), ("admitted", C.POINTER(C.c_int32)), ("preempted", C.POINTER(C.c_int32)),
                ("active", C.POINTER(C.c_int32)), ("active_seq", C.POINTER(C.c_int32)),
                ("page_seq", C.POINTER(C.c_int32)), ("branch_offsets", C.POINTER(C.c_int32))]


class DecodeBatch(C.Structure):
    _fields_ = [("n_pages", C.c_int32), ("n_branches", C.c_int32), ("page_seq", C.POINTER(C.c_int32)),
                ("branch_offsets", C.POINTER(C.c_int32)), ("branch_seq", C.POINTER(C.c_int32)),
                ("q_offsets", C.POINTER(C.c_int32))]


class RopeSpec(C.Structure):
    _fields_ = [("cos_sin", C.c_void_p), ("n_pos", C.c_int32), ("rot_dim", C.c_int32), ("interleaved", C.c_int32)]


class KVStep(C.Structure):
    _fields_ = [("q", C.c_void_p), ("q_stride", C.c_int64), ("Hq", C.c_int32), ("q_rot", C.c_void_p),
                ("k", C.c_void_p), ("k_stride", C.c_int64), ("v", C.c_void_p), ("v_stride", C.c_int64),
                ("k_rot", C.c_void_p)]


class RopeScaling(C.Structure):
    _fields_ = [("base", C.c_double), ("rot_dim", C.c_int32), ("kind", C.c_int32), ("factor", C.c_double),
                ("context", C.c_double), ("turns_lo", C.c_double), ("turns_hi", C.c_double),
                ("amplitude", C.c_double)]


class RopePart(C.Structure):
    _fields_ = [("x", C.c_void_p), ("stride", C.c_int64), ("out", C.c_void_p), ("out_stride", C.c_int64),
                ("heads", C.c_int32)]


class LmHead(C.Structure):
    _fields_ = [("h", C.c_void_p), ("h_stride", C.c_int64), ("w", C.c_void_p), ("w_stride", C.c_int64),
                ("targets", C.c_void_p), ("n", C.c_int32), ("D", C.c_int32), ("V", C.c_int32)]


class Act(C.Structure):
    _fields_ = [("rows", C.c_void_p), ("stride", C.c_int64), ("n", C.c_int64), ("width", C.c_int32),
                ("kept", C.c_void_p)]


# the same two as packed bytes, which cost a tenth to make: two parts, and one act
_PARTS = struct.Struct("@PqPqi4xPqPqi4x").pack
_ACT = struct.Struct("@Pqqi4xP").pack

_lib = None


def lib() -> C.CDLL:
    """Loads libpadoc.so (built by tree_structured_shared_gb300.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run tree_structured_shared_gb300.build first")
        L = C.CDLL(LIB_PATH)
        vp, i32, i64, f32 = C.c_void_p, C.c_int32, C.c_int64, C.c_float
        p32, p64 = C.POINTER(C.c_int32), C.POINTER(C.c_int64)
        sig = {
            "padoc_last_error": (C.c_char_p, []),
            "padoc_version": (C.c_int, []),
            "padoc_tree_desc_build": (C.c_int, [C.POINTER(TreeSpec), C.POINTER(vp)]),
            "padoc_tree_desc_free": (C.c_int, [vp]),
            "padoc_tree_desc_info": (C.c_int, [vp, p64, p64, p64, p64]),
            "padoc_tree_desc_segments": (C.c_int, [vp, p32, p32]),
            "padoc_tree_desc_upload": (C.c_int, [vp, i32]),
            "padoc_tree_attn_varlen": (C.c_int, [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, vp]),
            "padoc_kv_pool_create": (C.c_int, [C.POINTER(vp), vp, vp, i32, i32, i32, i32, i32, i32, i32]),
            "padoc_kv_pool_destroy": (C.c_int, [vp]),
            "padoc_kv_alloc": (C.c_int, [vp, i32, p32]),
            "padoc_kv_append": (C.c_int, [vp, i32, vp, vp, i32, vp]),
            "padoc_kv_fork": (C.c_int, [vp, i32, i32, p32]),
            "padoc_kv_release": (C.c_int, [vp, i32]),
            "padoc_kv_seq_info": (C.c_int, [vp, i32, p32, p32, p32]),
            "padoc_kv_seq_blocks": (C.c_int, [vp, i32, p32, i32]),
            "padoc_kv_block_refcount": (C.c_int, [vp, i32, p32]),
            "padoc_kv_pool_stats": (C.c_int, [vp, p32, p32]),
            "padoc_kv_pool_sync": (C.c_int, [vp, vp]),
            "padoc_kv_pool_device": (C.c_int, [vp, p32]),
            "padoc_debug_kv_pool_rehome": (C.c_int, [vp, i32]),
            "padoc_debug_set_wait_limit": (C.c_int, [C.c_uint64]),
            "padoc_branch_decode_ws_size": (C.c_int, [vp, C.POINTER(DecodeBatch), i32, C.POINTER(C.c_size_t)]),
            "padoc_branch_decode": (C.c_int, [vp, C.POINTER(DecodeBatch), i32, vp, vp, vp, vp, vp, vp, f32, vp,
                                              C.c_size_t, vp]),
            "padoc_tree_mask_build": (C.c_int, [p32, i32, C.POINTER(C.c_uint16)]),
            "padoc_depths": (C.c_int, [p32, p32, i32, p64, p64]),
            "padoc_device_status": (C.c_int, [vp]),
            "padoc_decode_plan_create": (C.c_int, [vp, C.POINTER(DecodeBatch), i32, C.POINTER(vp)]),
            "padoc_decode_plan_ws_size": (C.c_int, [vp, C.POINTER(C.c_size_t)]),
            "padoc_decode_plan_fused": (C.c_int, [vp, C.POINTER(C.c_int32)]),
            "padoc_decode_plan_upload": (C.c_int, [vp, vp, C.c_size_t, vp]),
            "padoc_decode_prefix_pass": (C.c_int, [vp, vp, f32, vp, vp]),
            "padoc_decode_own_pass": (C.c_int, [vp, vp, vp, vp, vp, vp, vp, f32, vp, vp]),
            "padoc_decode_plan_free": (C.c_int, [vp]),
            "padoc_branch_decode_noalloc": (C.c_int, [vp, C.POINTER(DecodeBatch), i32, vp, vp, vp, vp, vp, vp, f32,
                                                      vp]),
            "padoc_verify_accept": (C.c_int, [vp, i32, i32, vp, vp, vp, i32, i32, f32, vp, vp, vp, vp]),
            "padoc_kv_commit": (C.c_int, [vp, i32, p32, p32, p32, i32, vp, vp, vp, C.c_size_t, vp]),
            "padoc_kv_reserve": (C.c_int, [vp, i32, i32]),
            "padoc_kv_advance": (C.c_int, [vp, i32, i32]),
            "padoc_kv_trim": (C.c_int, [vp, i32]),
            "padoc_sched_create": (C.c_int, [vp, C.POINTER(SchedConfig), C.POINTER(vp)]),
            "padoc_sched_destroy": (C.c_int, [vp]),
            "padoc_sched_submit": (C.c_int, [vp, i32, i64, p32]),
            "padoc_sched_schedule": (C.c_int, [vp, C.POINTER(SchedStep)]),
            "padoc_sched_update": (C.c_int, [vp, i64, i32, p32, p32, p32]),
            "padoc_sched_request": (C.c_int, [vp, i32, p32, p32, p32, p64]),
            "padoc_sched_output": (C.c_int, [vp, i32, p32, i64, p64]),
            "padoc_tree_attn_varlen_bwd_ws_size": (C.c_int, [vp, i32, C.POINTER(C.c_size_t)]),
            "padoc_tree_attn_varlen_bwd": (C.c_int, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                                     f32, vp, C.c_size_t, vp]),
            "padoc_tree_desc_bwd_plan": (C.c_int, [vp, p32, p32, p64, p64]),
            "padoc_kv_storage_bytes": (C.c_int, [i32, i32, i32, i32, C.POINTER(C.c_size_t)]),
            "padoc_kv_rows_create": (C.c_int, [vp, i32, p32, p32, p32, p32, C.POINTER(vp)]),
            "padoc_kv_rows_ws_size": (C.c_int, [vp, C.POINTER(C.c_size_t)]),
            "padoc_kv_rows_upload": (C.c_int, [vp, vp, C.c_size_t, vp]),
            "padoc_kv_rows_free": (C.c_int, [vp]),
            "padoc_kv_write": (C.c_int, [vp, C.POINTER(RopeSpec), C.POINTER(KVStep), vp, vp]),
            "padoc_kv_gather": (C.c_int, [vp, vp, vp, vp, vp]),
            "padoc_kv_append_rope": (C.c_int, [vp, i32, p32, p32, p32, C.POINTER(RopeSpec), C.POINTER(KVStep), vp,
                                               C.c_size_t, vp]),
            "padoc_rope_table": (C.c_int, [C.POINTER(RopeScaling), i64, i32, vp, vp]),
            "padoc_rope_apply": (C.c_int, [C.POINTER(RopeSpec), i32, vp, i32, i32, i64, vp, i32, vp]),
            "padoc_lm_loss_ws_size": (C.c_int, [i32, i32, i32, i32, C.POINTER(C.c_size_t)]),
            "padoc_lm_loss": (C.c_int, [C.POINTER(LmHead), vp, vp, vp, C.c_size_t, vp]),
            "padoc_lm_loss_bwd": (C.c_int, [C.POINTER(LmHead), vp, vp, vp, vp, vp, C.c_size_t, vp]),
            "padoc_act_bytes": (C.c_int, [i64, i32, C.POINTER(C.c_size_t)]),
            "padoc_act_keep": (C.c_int, [i32, vp, vp]),
            "padoc_act_restore": (C.c_int, [i32, vp, vp]),
            "padoc_tree_attn_varlen_bwd_kept_ws_size": (C.c_int, [vp, i32, i32, i32, C.POINTER(C.c_size_t)]),
            "padoc_tree_attn_varlen_bwd_kept": (C.c_int, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, f32,
                                                          vp, C.c_size_t, vp]),
            "padoc_draft_index_create": (C.c_int, [p32, p64, i32, i32, C.POINTER(vp)]),
            "padoc_draft_index_free": (C.c_int, [vp]),
            "padoc_draft_trie": (C.c_int, [vp, p32, i32, i32, i32, p32, p32, p32]),
            "padoc_draft_trie_batch": (C.c_int, [C.POINTER(vp), i32, p32, p32, i32, i32, p32, p32, p32,
                                                 C.POINTER(C.c_uint16)]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(rc: int):
    if rc != OK:
        raise PadocError(rc, lib().padoc_last_error().decode(errors="replace"))


def _ptr(x) -> Optional[int]:
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


_current_stream = None  # () -> the current CUDA stream's handle, once torch sees a GPU


def _find_current_stream():
    global _current_stream
    try:
        import torch
        if not torch.cuda.is_available():
            return None
        torch.cuda.init()
        raw, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    except Exception:
        return None
    if raw is not None and dev is not None:  # a tenth of the public call's time
        _current_stream = lambda: raw(dev())  # noqa: E731
    else:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _current_stream


def _stream(stream) -> Optional[int]:
    if stream is None:
        f = _current_stream or _find_current_stream()
        return (f() or None) if f else None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _p32(a: np.ndarray):
    return a.ctypes.data_as(C.POINTER(C.c_int32))


# ------------------------------------------------------------------ tree descriptor


class TreeDesc:
    """Host descriptor of packed pages (padoc_tree_desc_build)."""

    def __init__(self, pages, order: int = PACK_CANONICAL):
        self._keep = [
            _i32([p.prefix_len for p in pages]),
            _i32([len(p.layout_len) for p in pages]),
            _i32([x for p in pages for x in p.layout_len] or [0]),
            _i32([x for p in pages for x in p.content_len] or [0]),
        ]
        spec = TreeSpec(len(pages), _p32(self._keep[0]), _p32(self._keep[1]), _p32(self._keep[2]),
                        _p32(self._keep[3]), order)
        h = C.c_void_p()
        _check(lib().padoc_tree_desc_build(C.byref(spec), C.byref(h)))
        self.handle = h

    def info(self):
        v = [C.c_int64() for _ in range(4)]
        _check(lib().padoc_tree_desc_info(self.handle, *[C.byref(x) for x in v]))
        return {"n_tokens": v[0].value, "n_qsegs": v[1].value, "n_kvsegs": v[2].value,
                "ancestor_pairs": v[3].value}

    def segments(self):
        inf = self.info()
        qs = np.zeros((max(inf["n_qsegs"], 1), 4), np.int32)
        kv = np.zeros((max(inf["n_kvsegs"], 1), 3), np.int32)
        _check(lib().padoc_tree_desc_segments(self.handle, _p32(qs), _p32(kv)))
        return qs[: inf["n_qsegs"]], kv[: inf["n_kvsegs"]]

    def bwd_plan(self):
        """Key-stationary backward plan: items [n, 4], entries [m, 5]."""
        n, m = C.c_int64(), C.c_int64()
        _check(lib().padoc_tree_desc_bwd_plan(self.handle, None, None, C.byref(n), C.byref(m)))
        it = np.zeros((max(n.value, 1), 4), np.int32)
        en = np.zeros((max(m.value, 1), 5), np.int32)
        _check(lib().padoc_tree_desc_bwd_plan(self.handle, _p32(it), _p32(en), None, None))
        return it[: n.value], en[: m.value]

    def upload(self, group: int):
        _check(lib().padoc_tree_desc_upload(self.handle, group))

    def free(self):
        if self.handle:
            lib().padoc_tree_desc_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def tree_attn_varlen(desc: TreeDesc, q, k, v, o, lse, dtype: int, Hq: int, Hkv: int, d: int,
                     scale: float = 0.0, stream=None):
    _check(lib().padoc_tree_attn_varlen(desc.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), dtype, Hq,
                                        Hkv, d, float(scale), _stream(stream)))


def tree_attn_varlen_bwd_ws_size(desc: TreeDesc, Hq: int) -> int:
    n = C.c_size_t()
    _check(lib().padoc_tree_attn_varlen_bwd_ws_size(desc.handle, Hq, C.byref(n)))
    return n.value


def tree_attn_varlen_bwd(desc: TreeDesc, q, k, v, o, lse, d_o, dq, dk, dv, dtype: int, Hq: int, Hkv: int, d: int,
                         ws, ws_bytes: int, scale: float = 0.0, stream=None):
    _check(lib().padoc_tree_attn_varlen_bwd(desc.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(d_o),
                                            _ptr(dq), _ptr(dk), _ptr(dv), dtype, Hq, Hkv, d, float(scale), _ptr(ws),
                                            int(ws_bytes), _stream(stream)))


# ------------------------------------------------------------------ around the attention of a training step


def tree_attn_varlen_bwd_kept_ws_size(desc: TreeDesc, Hq: int, Hkv: int, d: int) -> int:
    n = C.c_size_t()
    _check(lib().padoc_tree_attn_varlen_bwd_kept_ws_size(desc.handle, Hq, Hkv, d, C.byref(n)))
    return n.value


def tree_attn_varlen_bwd_kept(desc: TreeDesc, q_kept, k_kept, v_kept, o_kept, lse, d_o, dq, dk, dv, Hq: int, Hkv: int,
                              d: int, ws, ws_bytes: int, scale: float = 0.0, stream=None):
    """padoc_tree_attn_varlen_bwd_kept: the backward from checkpoints of q, k, v and o."""
    _check(lib().padoc_tree_attn_varlen_bwd_kept(desc.handle, _ptr(q_kept), _ptr(k_kept), _ptr(v_kept), _ptr(o_kept),
                                                 _ptr(lse), _ptr(d_o), _ptr(dq), _ptr(dk), _ptr(dv), Hq, Hkv, d,
                                                 float(scale), _ptr(ws), int(ws_bytes), _stream(stream)))


def rope_table(cos_sin, n_pos: int, rot_dim: int, base: float, *, kind: int = ROPE_PLAIN, factor: float = 1.0,
               context: float = 0.0, turns_lo: float = 1.0, turns_hi: float = 32.0, amplitude: float = 1.0,
               first: int = 0, stream=None):
    """padoc_rope_table: device f32 cos_sin [n_pos, rot_dim] out."""
    if not (cos_sin is None or isinstance(cos_sin, int)) and (
            cos_sin.dtype is not sys.modules["torch"].float32 or cos_sin.numel() < n_pos * rot_dim or not cos_sin.is_contiguous()):
        raise PadocError(ERR_INVALID, "rope_table: cos_sin must be n_pos * rot_dim dense f32 values")
    sc = RopeScaling(base, rot_dim, kind, factor, context, turns_lo, turns_hi, amplitude)
    _check(lib().padoc_rope_table(C.byref(sc), int(first), n_pos, _ptr(cos_sin), _stream(stream)))


_NO_TYPE = (None, 0)
_DTYPES = {}  # F32, BF16 -> torch's type and its bytes, once a tensor was seen


def _row_stride(x, n: int, row: int) -> int:
    """Elements between the n rows of `row` values that x holds, where no stride was given."""
    if x.dim() >= 2 and x.size(0) >= n and x[0].numel() >= row and x[0].is_contiguous():
        return x.stride(0)  # a row each, or the head of a wider one
    if x.is_contiguous() and (x.dim() < 2 or x[0].numel() <= row):
        return row
    raise PadocError(ERR_INVALID, "rope_apply: rows must be dense, or their stride be given")


def _rows(x, n: int, row: int, nbytes: int, stride, dtype):
    """Address and row stride of n rows of `row` values, `nbytes` in all, of a tensor or an
    address."""
    if x is None or type(x) is int:
        return x or 0, row if stride is None else stride
    # a step of few tokens takes as long as the host's calls: a dense tensor meets three here
    m = x.nbytes
    if x.dtype is not dtype or m < nbytes:
        raise PadocError(ERR_INVALID, f"rope_apply: a tensor must be {dtype} and hold n rows of its heads")
    if stride is None:
        stride = row if m == nbytes and x.is_contiguous() else _row_stride(x, n, row)
    return x.data_ptr(), stride


def rope_apply(rope: "Rope", n: int, d: int, q, q_out, Hq: int, k=None, k_out=None, Hkv: int = 0, *, positions=None,
               dtype: int = BF16, backward: bool = False, q_stride: Optional[int] = None, k_stride: Optional[int] = None,
               q_out_stride: Optional[int] = None, k_out_stride: Optional[int] = None, stream=None):
    """padoc_rope_apply on q and, where given, k, whose type is dtype; strides in elements
    between rows are taken as they are, and a tensor's own where None.  positions: int32."""
    if not _DTYPES and (t := sys.modules.get("torch")):
        _DTYPES.update({F32: (t.float32, 4), BF16: (t.bfloat16, 2), "positions": t.int32})
    dt, size = _DTYPES.get(dtype, _NO_TYPE)
    hq = Hq * d
    m = n * hq * size
    x, xs = _rows(q, n, hq, m, q_stride, dt)
    y, ys = _rows(q_out, n, hq, m, q_out_stride, dt)
    if k is None:
        count, parts = 1, _PARTS(x, xs, y, ys, Hq, 0, 0, 0, 0, 0)
    else:
        hk = Hkv * d
        m = n * hk * size
        v, vs = _rows(k, n, hk, m, k_stride, dt)
        w, ws = _rows(k_out, n, hk, m, k_out_stride, dt)
        count, parts = 2, _PARTS(x, xs, y, ys, Hq, v, vs, w, ws, Hkv)
    if positions is not None and type(positions) is not int:
        if positions.dtype is not _DTYPES["positions"] or positions.nbytes < 4 * n or not positions.is_contiguous():
            raise PadocError(ERR_INVALID, "rope_apply: positions must be n dense int32 values")
        positions = positions.data_ptr()
    s = _current_stream() or None if stream is None and _current_stream else _stream(stream)
    rc = (_lib or lib()).padoc_rope_apply(rope.ref, count, parts, dtype, d, n, positions, 1 if backward else 0, s)
    if rc:
        _check(rc)


class LmLoss:
    """Cross entropy of rows h [n, D] against weights w [V, D], device bf16, and
    int32 targets [n] (negative: none); padoc_lm_loss and its backward."""

    def __init__(self, h, w, targets):
        self._keep = (h, w, targets)
        (n, D), V = h.shape, w.shape[0]
        if w.shape[1] != D or targets.shape[0] != n:
            raise PadocError(ERR_INVALID, "LmLoss: h [n, D], w [V, D] and targets [n] do not fit together")
        if h.stride(1) != 1 or w.stride(1) != 1 or (n > 1 and targets.stride(0) != 1):
            raise PadocError(ERR_INVALID, "LmLoss: a row's values and the targets must follow one another")
        if not (_is_bf16(h) and _is_bf16(w)) or targets.dtype is not sys.modules["torch"].int32:
            raise PadocError(ERR_INVALID, "LmLoss: h and w must be bf16 and the targets int32")
        if h.device != w.device or h.device != targets.device:
            raise PadocError(ERR_INVALID, "LmLoss: h, w and targets must be on one device")
        self.c = LmHead(_ptr(h), h.stride(0) if n > 1 else D, _ptr(w), w.stride(0) if V > 1 else D, _ptr(targets), n, D, V)
        self.ref = C.byref(self.c)

    def ws_size(self, backward: bool = False) -> int:
        b = C.c_size_t()
        _check(lib().padoc_lm_loss_ws_size(self.c.n, self.c.D, self.c.V, int(bool(backward)), C.byref(b)))
        return b.value

    def _dense(self, **tensors):
        """Refuses tensors (name=(x, bf16 or else f32, values)) that the library would read or
        write past their end, or as another type or layout than theirs."""
        torch, at = sys.modules["torch"], self._keep[0].device
        for name, (x, bf16, m) in tensors.items():
            if x is None or isinstance(x, int):
                continue
            if x.dtype is not (torch.bfloat16 if bf16 else torch.float32) or x.numel() < m or not x.is_contiguous() or x.device != at:
                raise PadocError(ERR_INVALID, f"LmLoss: {name} must be {m} dense {'bf16' if bf16 else 'f32'} values beside h")

    def _room(self, ws, ws_bytes: int):
        if not (ws is None or isinstance(ws, int)) and (ws.nbytes < ws_bytes or not ws.is_contiguous()):
            raise PadocError(ERR_INVALID, "LmLoss: ws is smaller than ws_bytes, or not dense")

    def forward(self, loss, lse, ws, ws_bytes: int, stream=None):
        """loss and lse: dense f32 of n values."""
        n = self.c.n
        self._dense(loss=(loss, False, n), lse=(lse, False, n))
        self._room(ws, ws_bytes)
        _check(lib().padoc_lm_loss(self.ref, _ptr(loss), _ptr(lse), _ptr(ws), int(ws_bytes), _stream(stream)))

    def backward(self, lse, d_loss, dh, dw, ws, ws_bytes: int, stream=None):
        """lse and d_loss: dense f32 of n values (an expanded one is refused: make it
        contiguous); dh, dw: dense bf16 of n * D and V * D, or None."""
        n, D = self.c.n, self.c.D
        self._dense(lse=(lse, False, n), d_loss=(d_loss, False, n), dh=(dh, True, n * D), dw=(dw, True, self.c.V * D))
        self._room(ws, ws_bytes)
        _check(lib().padoc_lm_loss_bwd(self.ref, _ptr(lse), _ptr(d_loss), _ptr(dh), _ptr(dw), _ptr(ws), int(ws_bytes),
                                       _stream(stream)))


def act_bytes(n: int, width: int) -> int:
    """Bytes of the checkpoint of n rows of `width` values."""
    b = C.c_size_t()
    _check(lib().padoc_act_bytes(int(n), int(width), C.byref(b)))
    return b.value


_BF16 = None  # torch.bfloat16, once a tensor was seen


def _is_bf16(x) -> bool:
    global _BF16
    if _BF16 is None:
        _BF16 = sys.modules["torch"].bfloat16  # a tensor is there, so torch is
    return x.dtype is _BF16


def _acts(rows, kept) -> bytes:
    """The padoc_act array of the tensors and their checkpoints."""
    if len(rows) != len(kept):
        raise PadocError(ERR_INVALID, "act: one checkpoint a tensor is needed")
    out = b""
    for x, b in zip(rows, kept):
        if x.dim() != 2 or not _is_bf16(x):
            raise PadocError(ERR_INVALID, "act: rows must be bf16 [n, width]")
        (n, width), (step, one) = x.shape, x.stride()
        if one != 1 and width > 1:
            raise PadocError(ERR_INVALID, "act: a row's values must follow one another")
        if b.nbytes < n * width + n * width // 32 or not b.is_contiguous():
            raise PadocError(ERR_INVALID, "act: a checkpoint is smaller than act_bytes(n, width), or not dense")
        out += _ACT(x.data_ptr(), step if n > 1 else width, n, width, b.data_ptr())
    return out


def act_keep(rows, kept, stream=None):
    """padoc_act_keep: bf16 tensors [n, width] into their checkpoints (device
    bytes, act_bytes(n, width) each); one launch for up to eight."""
    rc = lib().padoc_act_keep(len(rows), _acts(rows, kept), _stream(stream))
    if rc:
        _check(rc)


def act_restore(kept, rows, stream=None):
    """padoc_act_restore: checkpoints back into bf16 tensors [n, width]."""
    rc = lib().padoc_act_restore(len(rows), _acts(rows, kept), _stream(stream))
    if rc:
        _check(rc)


# ------------------------------------------------------------------ KV pool


class KVPool:
    """Refcounted paged KV pool over caller-owned storage (padoc_kv_pool_*)."""

    def __init__(self, k_pool, v_pool, num_blocks: int, Hkv: int, d: int = 128, max_seqs: int = 1024,
                 max_blocks_per_seq: int = 512, block_size: int = 16, dtype: int = BF16):
        h = C.c_void_p()
        _check(lib().padoc_kv_pool_create(C.byref(h), _ptr(k_pool), _ptr(v_pool), num_blocks, block_size, Hkv, d,
                                          dtype, max_seqs, max_blocks_per_seq))
        self.handle = h
        self.Hkv = Hkv
        self.d = d
        self._storage = (k_pool, v_pool)

    def alloc(self, n_tokens: int = 0) -> int:
        s = C.c_int32()
        _check(lib().padoc_kv_alloc(self.handle, n_tokens, C.byref(s)))
        return s.value

    def fork(self, parent: int, fork_len: int) -> int:
        s = C.c_int32()
        _check(lib().padoc_kv_fork(self.handle, parent, fork_len, C.byref(s)))
        return s.value

    def append(self, seq: int, k, v, n: int, stream=None):
        _check(lib().padoc_kv_append(self.handle, seq, _ptr(k), _ptr(v), n, _stream(stream)))

    def release(self, seq: int):
        _check(lib().padoc_kv_release(self.handle, seq))

    def seq_info(self, seq: int):
        a, b, c = C.c_int32(), C.c_int32(), C.c_int32()
        _check(lib().padoc_kv_seq_info(self.handle, seq, C.byref(a), C.byref(b), C.byref(c)))
        return {"length": a.value, "fork_len": b.value, "n_blocks": c.value}

    def seq_blocks(self, seq: int):
        n = self.seq_info(seq)["n_blocks"]
        out = np.zeros(max(n, 1), np.int32)
        _check(lib().padoc_kv_seq_blocks(self.handle, seq, _p32(out), len(out)))
        return out[:n]

    def refcount(self, block: int) -> int:
        r = C.c_int32()
        _check(lib().padoc_kv_block_refcount(self.handle, block, C.byref(r)))
        return r.value

    def stats(self):
        a, b = C.c_int32(), C.c_int32()
        _check(lib().padoc_kv_pool_stats(self.handle, C.byref(a), C.byref(b)))
        return {"free_blocks": a.value, "live_seqs": b.value}

    def sync(self, stream=None):
        _check(lib().padoc_kv_pool_sync(self.handle, _stream(stream)))

    def device(self) -> int:
        d = C.c_int32()
        _check(lib().padoc_kv_pool_device(self.handle, C.byref(d)))
        return d.value

    def debug_rehome(self, device: int):
        """Testing aid (padoc_debug_kv_pool_rehome): relabels the pool's device."""
        _check(lib().padoc_debug_kv_pool_rehome(self.handle, device))

    def reserve(self, seq: int, n_tokens: int):
        _check(lib().padoc_kv_reserve(self.handle, seq, n_tokens))

    def advance(self, seq: int, n: int):
        _check(lib().padoc_kv_advance(self.handle, seq, n))

    def trim(self, seq: int):
        _check(lib().padoc_kv_trim(self.handle, seq))

    def commit(self, seqs: Sequence[int], row_offsets: Sequence[int], rows: Sequence[int], n_src_rows: int,
               k_new, v_new, ws, ws_bytes: int, stream=None):
        """padoc_kv_commit: appends rows[row_offsets[i]:row_offsets[i+1]] of
        k_new / v_new to sequence seqs[i]."""
        a, b, c = _i32(seqs if len(seqs) else [0]), _i32(row_offsets if len(row_offsets) else [0]), \
            _i32(rows if len(rows) else [0])
        _check(lib().padoc_kv_commit(self.handle, len(seqs), _p32(a), _p32(b), _p32(c), n_src_rows, _ptr(k_new),
                                     _ptr(v_new), _ptr(ws), int(ws_bytes), _stream(stream)))

    def append_rope(self, seqs: Sequence[int], row_offsets: Sequence[int], k, v, ws=None, ws_bytes: int = 0, *,
                    positions=None, rope: Optional["Rope"] = None, stream=None, **step):
        """padoc_kv_append_rope: reserve, write and advance; step as in KVRows.write."""
        a, _, b, p = _row_lists(seqs, None, row_offsets, positions)
        st = _kv_step(self, k, v, **step)
        _check(lib().padoc_kv_append_rope(self.handle, len(seqs), _p32(a), _p32(b), None if p is None else _p32(p),
                                          None if rope is None else C.byref(rope.c), C.byref(st), _ptr(ws),
                                          int(ws_bytes), _stream(stream)))

    def destroy(self):
        if self.handle:
            lib().padoc_kv_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def kv_storage_bytes(num_blocks: int, Hkv: int, d: int = 128, dtype: int = BF16) -> int:
    """Bytes of a pool's K storage (and, again, of its V storage)."""
    n = C.c_size_t()
    _check(lib().padoc_kv_storage_bytes(num_blocks, Hkv, d, dtype, C.byref(n)))
    return n.value


class Rope:
    """Rotation by position (padoc_rope): cos_sin is a device f32 table
    [n_pos, rot_dim], cosines then sines."""

    def __init__(self, cos_sin, rot_dim: int, interleaved: bool = False, n_pos: Optional[int] = None):
        self._table = cos_sin
        if n_pos is None:
            n_pos = int(cos_sin.shape[0])
        self.c = RopeSpec(_ptr(cos_sin), n_pos, rot_dim, int(bool(interleaved)))
        self.ref = C.byref(self.c)


def _kv_step(pool: "KVPool", k, v, *, k_stride=None, v_stride=None, q=None, Hq: int = 0, q_stride=None, q_rot=None,
             k_rot=None) -> KVStep:
    row = pool.Hkv * pool.d
    return KVStep(_ptr(q), Hq * pool.d if q_stride is None else int(q_stride), Hq, _ptr(q_rot),
                  _ptr(k), row if k_stride is None else int(k_stride), _ptr(v),
                  row if v_stride is None else int(v_stride), _ptr(k_rot))


def _row_lists(seqs, first, row_offsets, positions):
    """The host arrays of a row list; the library reads len(seqs) of first, one
    more of row_offsets and a position a row, so shorter ones are refused."""
    n = len(seqs)
    a, b = _i32(seqs if n else [0]), _i32(row_offsets)
    f = None if first is None else _i32(first if len(first) else [0])
    p = None if positions is None else _i32(positions)
    if n and (b.size <= n or (f is not None and f.size < n) or (p is not None and p.size < b[n])):
        raise PadocError(ERR_INVALID, "first, row_offsets or positions is shorter than the sequences and rows need")
    return a, f, b, p


class KVRows:
    """Token ranges of sequences (padoc_kv_rows): written from, or read back
    into, packed rows in one launch."""

    def __init__(self, pool: KVPool, seqs: Sequence[int], first: Optional[Sequence[int]], row_offsets: Sequence[int],
                 positions=None):
        a, f, b, p = _row_lists(seqs, first, row_offsets, positions)
        h = C.c_void_p()
        _check(lib().padoc_kv_rows_create(pool.handle, len(seqs), _p32(a), None if f is None else _p32(f), _p32(b),
                                          None if p is None else _p32(p), C.byref(h)))
        self.handle = h
        self.n = int(b[len(seqs)]) if len(seqs) else 0
        self._pool, self._row, self._lib = pool, pool.Hkv * pool.d, lib()

    def ws_size(self) -> int:
        n = C.c_size_t()
        _check(lib().padoc_kv_rows_ws_size(self.handle, C.byref(n)))
        return n.value

    def upload(self, ws=None, ws_bytes: int = 0, stream=None):
        _check(lib().padoc_kv_rows_upload(self.handle, _ptr(ws), int(ws_bytes), _stream(stream)))

    def write(self, k, v, ws=None, *, rope: Optional[Rope] = None, stream=None, q=None, Hq: int = 0, q_rot=None,
              k_rot=None, q_stride=None, k_stride=None, v_stride=None):
        """padoc_kv_write.  Optional: q with Hq and q_rot, k_rot, and the row
        strides k_stride, v_stride, q_stride in elements (dense by default)."""
        # a step of few rows takes as long as this call: no detours
        row = self._row
        st = KVStep(_ptr(q), Hq * self._pool.d if q_stride is None else q_stride, Hq, _ptr(q_rot), _ptr(k),
                    row if k_stride is None else k_stride, _ptr(v), row if v_stride is None else v_stride, _ptr(k_rot))
        rc = self._lib.padoc_kv_write(self.handle, None if rope is None else rope.ref, C.byref(st), _ptr(ws),
                                      _stream(stream))
        if rc != OK:
            _check(rc)

    def gather(self, k, v, ws=None, stream=None):
        _check(lib().padoc_kv_gather(self.handle, _ptr(k), _ptr(v), _ptr(ws), _stream(stream)))

    def free(self):
        if self.handle:
            lib().padoc_kv_rows_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class Batch:
    """Host arrays of one decode/verify step (padoc_decode_batch)."""

    def __init__(self, page_seq: Sequence[int], branch_offsets: Sequence[int], branch_seq: Sequence[int],
                 q_offsets: Sequence[int]):
        self._keep = [_i32(page_seq if len(page_seq) else [0]), _i32(branch_offsets), _i32(branch_seq or [0]),
                      _i32(q_offsets)]
        self.c = DecodeBatch(len(page_seq), len(branch_seq), _p32(self._keep[0]), _p32(self._keep[1]),
                             _p32(self._keep[2]), _p32(self._keep[3]))
        self.nq = int(self._keep[3][-1]) if len(branch_seq) else 0


def branch_decode_ws_size(pool: KVPool, batch: Batch, Hq: int) -> int:
    n = C.c_size_t()
    _check(lib().padoc_branch_decode_ws_size(pool.handle, C.byref(batch.c), Hq, C.byref(n)))
    return n.value


def branch_decode(pool: KVPool, batch: Batch, Hq: int, q, k_new, v_new, tree_bits, o, lse, ws, ws_bytes: int,
                  scale: float = 0.0, stream=None):
    _check(lib().padoc_branch_decode(pool.handle, C.byref(batch.c), Hq, _ptr(q), _ptr(k_new), _ptr(v_new),
                                     _ptr(tree_bits), _ptr(o), _ptr(lse), float(scale), _ptr(ws), int(ws_bytes),
                                     _stream(stream)))


def branch_decode_noalloc(pool: KVPool, batch: Batch, Hq: int, q, k_new, v_new, tree_bits, o, lse,
                          scale: float = 0.0, stream=None):
    """padoc_branch_decode with the workspace taken from the library's fixed
    device array (no device allocation; for callers that may not allocate)."""
    _check(lib().padoc_branch_decode_noalloc(pool.handle, C.byref(batch.c), Hq, _ptr(q), _ptr(k_new), _ptr(v_new),
                                             _ptr(tree_bits), _ptr(o), _ptr(lse), float(scale), _stream(stream)))


def verify_accept(logits, nq: int, vocab: int, tokens, parents, q_offsets, n_branches: int, max_nodes: int,
                  tau: float, n_acc, path, free_token, stream=None):
    """padoc_verify_accept: device arrays in, device n_acc [B], path [B, 16]
    and free_token [B] out."""
    _check(lib().padoc_verify_accept(_ptr(logits), nq, vocab, _ptr(tokens), _ptr(parents), _ptr(q_offsets),
                                     n_branches, max_nodes, float(tau), _ptr(n_acc), _ptr(path), _ptr(free_token),
                                     _stream(stream)))


class DraftIndex:
    """A request's fixed drafts with their window table (padoc_draft_index)."""

    def __init__(self, drafts: Sequence[Sequence[int]], window: int = 3):
        toks = _i32([t for d in drafts for t in d] or [0])
        offs = np.zeros(len(drafts) + 1, np.int64)
        offs[1:] = np.cumsum([len(d) for d in drafts])
        h = C.c_void_p()
        _check(lib().padoc_draft_index_create(_p32(toks), offs.ctypes.data_as(C.POINTER(C.c_int64)), len(drafts),
                                              window, C.byref(h)))
        self.handle = h

    def trie(self, accepted: Sequence[int], max_nodes: int = 16, max_depth: int = 7):
        """One step's verify block: (tokens, parents) lists."""
        acc = _i32(accepted)
        t = np.zeros(max_nodes, np.int32)
        p = np.zeros(max_nodes, np.int32)
        n = C.c_int32()
        _check(lib().padoc_draft_trie(self.handle, _p32(acc), len(acc), max_nodes, max_depth, _p32(t), _p32(p),
                                      C.byref(n)))
        return t[: n.value].tolist(), p[: n.value].tolist()

    def free(self):
        if self.handle:
            lib().padoc_draft_index_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def draft_trie_batch(indexes: Sequence[DraftIndex], accepted: Sequence[Sequence[int]], max_nodes: int = 16,
                     max_depth: int = 7):
    """padoc_draft_trie_batch: returns tokens [nq], parents [nq], q_offsets
    [B + 1] and tree bits [nq] (uint16) as numpy arrays."""
    B = len(indexes)
    hs = (C.c_void_p * max(B, 1))(*[ix.handle.value for ix in indexes])
    acc = _i32([t for a in accepted for t in a] or [0])
    aoff = np.zeros(B + 1, np.int32)
    aoff[1:] = np.cumsum([len(a) for a in accepted])
    cap = max(B * max_nodes, 1)
    t, p = np.zeros(cap, np.int32), np.zeros(cap, np.int32)
    q = np.zeros(B + 1, np.int32)
    bits = np.zeros(cap, np.uint16)
    _check(lib().padoc_draft_trie_batch(hs, B, _p32(acc), _p32(aoff), max_nodes, max_depth, _p32(t), _p32(p),
                                        _p32(q), bits.ctypes.data_as(C.POINTER(C.c_uint16))))
    nq = int(q[-1])
    return t[:nq], p[:nq], q, bits[:nq]


class Scheduler:
    """The branch scheduler over a KV pool (padoc_sched_*)."""

    STATES = ("waiting", "running", "ended", "done")

    def __init__(self, pool: "KVPool", tau: float, n_max: int, window: int, max_len: int, fork_token: int,
                 child_token: int, eos_token: int, cap: int = 4096):
        self.pool = pool
        cfg = SchedConfig(tau, n_max, window, max_len, fork_token, child_token, eos_token)
        h = C.c_void_p()
        _check(lib().padoc_sched_create(pool.handle, C.byref(cfg), C.byref(h)))
        self.handle = h
        self.cap = cap
        self._bufs = [np.zeros(cap + 1, np.int32) for _ in range(6)]

    def submit(self, prompt_len: int, arrival: int) -> int:
        r = C.c_int32()
        _check(lib().padoc_sched_submit(self.handle, prompt_len, arrival, C.byref(r)))
        return r.value

    def schedule(self):
        """admitted, preempted, and the batch as [(page_seq, [(request, seq), ...]), ...]."""
        b = self._bufs
        st = SchedStep(self.cap, 0, 0, 0, 0, *[_p32(x) for x in b])
        _check(lib().padoc_sched_schedule(self.handle, C.byref(st)))
        pages = []
        for p in range(st.n_pages):
            lo, hi = b[5][p], b[5][p + 1]
            pages.append((int(b[4][p]), [(int(b[2][i]), int(b[3][i])) for i in range(lo, hi)]))
        return b[0][: st.n_admitted].tolist(), b[1][: st.n_preempted].tolist(), pages

    def update(self, now: int, accepted):
        """accepted: [(request, [tokens...]), ...] in processing order."""
        req = _i32([r for r, _ in accepted] or [0])
        off = np.zeros(len(accepted) + 1, np.int32)
        off[1:] = np.cumsum([len(t) for _, t in accepted])
        toks = _i32([t for _, ts in accepted for t in ts] or [0])
        _check(lib().padoc_sched_update(self.handle, now, len(accepted), _p32(req), _p32(off), _p32(toks)))

    def request(self, rid: int):
        st, seq, par = C.c_int32(), C.c_int32(), C.c_int32()
        n = C.c_int64()
        _check(lib().padoc_sched_request(self.handle, rid, C.byref(st), C.byref(seq), C.byref(par), C.byref(n)))
        return {"state": self.STATES[st.value], "seq": seq.value, "parent": par.value, "n_out": n.value}

    def output(self, rid: int):
        n = C.c_int64()
        _check(lib().padoc_sched_output(self.handle, rid, None, 0, C.byref(n)))
        out = np.zeros(max(n.value, 1), np.int32)
        _check(lib().padoc_sched_output(self.handle, rid, _p32(out), len(out), C.byref(n)))
        return out[: n.value].tolist()

    def destroy(self):
        if self.handle:
            lib().padoc_sched_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


class DecodePlan:
    """A planned decode step (padoc_decode_plan_*): host plan, upload, and the
    two device passes."""

    def __init__(self, pool: KVPool, batch: Batch, Hq: int):
        h = C.c_void_p()
        _check(lib().padoc_decode_plan_create(pool.handle, C.byref(batch.c), Hq, C.byref(h)))
        self.handle = h
        self._refs = (pool, batch)

    def ws_size(self) -> int:
        n = C.c_size_t()
        _check(lib().padoc_decode_plan_ws_size(self.handle, C.byref(n)))
        return n.value

    def fused(self) -> bool:
        """True when the step runs as one kernel (the prefix pass launches nothing)."""
        f = C.c_int32()
        _check(lib().padoc_decode_plan_fused(self.handle, C.byref(f)))
        return bool(f.value)

    def upload(self, ws, ws_bytes: int, stream=None):
        _check(lib().padoc_decode_plan_upload(self.handle, _ptr(ws), int(ws_bytes), _stream(stream)))

    def prefix_pass(self, q, ws, scale: float = 0.0, stream=None):
        _check(lib().padoc_decode_prefix_pass(self.handle, _ptr(q), float(scale), _ptr(ws), _stream(stream)))

    def own_pass(self, q, k_new, v_new, tree_bits, o, lse, ws, scale: float = 0.0, stream=None):
        _check(lib().padoc_decode_own_pass(self.handle, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(tree_bits),
                                           _ptr(o), _ptr(lse), float(scale), _ptr(ws), _stream(stream)))

    def free(self):
        if self.handle:
            lib().padoc_decode_plan_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


# ------------------------------------------------------------------ small helpers


def tree_mask_build(parent: Sequence[int]) -> np.ndarray:
    p = _i32(parent if len(parent) else [0])
    out = np.zeros(max(len(parent), 1), np.uint16)
    _check(lib().padoc_tree_mask_build(_p32(p), len(parent), out.ctypes.data_as(C.POINTER(C.c_uint16))))
    return out[: len(parent)]


def depths(layout_len: Sequence[int], content_len: Sequence[int]):
    a, b = _i32(list(layout_len) or [0]), _i32(list(content_len) or [0])
    s, t = C.c_int64(), C.c_int64()
    _check(lib().padoc_depths(_p32(a), _p32(b), len(layout_len), C.byref(s), C.byref(t)))
    return {"D_seq": s.value, "D_tree": t.value}


def device_status(stream=None):
    _check(lib().padoc_device_status(_stream(stream)))


def debug_set_wait_limit(ns: int):
    """Testing aid (padoc_debug_set_wait_limit): the wait limit of the
    verify own pass's keys-on-M kernel and of the 4-bit prefix pass's tcgen05
    kernel on the current device; 0 restores the default."""
    _check(lib().padoc_debug_set_wait_limit(int(ns)))
