"""Python binding of libengram.so, the Engram per-layer forward step on one GB300.

Argument marshalling only: every function below forwards to the C function of
the same name declared in ``include/engram.h``; every step of the forward path
runs in the library's CUDA kernels.  Pointers may be given as ints, torch
tensors (``data_ptr()``) or numpy arrays (host memory); streams as ints,
``torch.cuda.Stream`` objects or None (legacy default stream).  A non-zero
status raises ``EngramError`` with the library's message.  If the library has
not been built the first call raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libengram.so")

DEAD = 0xFFFFFFFF
MASKED = 0xFFFFFFFF

STATUS = {0: "OK", 1: "EINVAL", 2: "ENOMEM", 3: "ECUDA", 4: "ESTATE", 5: "ETIMEOUT",
          6: "EUNSUPPORTED", 7: "EBOUNDS"}
OK, EINVAL, ENOMEM, ECUDA, ESTATE, ETIMEOUT, EUNSUPPORTED, EBOUNDS = range(8)

# Names exported by the library (the declarations of include/engram.h).
EXPORTS = (
    "engram_ctx_create", "engram_ctx_destroy", "engram_layer_params",
    "engram_layer_set_multipliers", "engram_layer_bind", "engram_layer_refresh",
    "engram_layer_info",
    "engram_table_fill", "engram_table_fill_bf16",
    "engram_session_create", "engram_session_fork", "engram_session_reset",
    "engram_session_destroy", "engram_session_append", "engram_batch_append",
    "engram_workspace_bytes", "engram_hash", "engram_gather_dequant", "engram_project",
    "engram_gate", "engram_forward", "engram_forward_noalloc", "engram_forward_staged",
    "engram_forward_staged_workspace_bytes", "engram_stage_rows", "engram_forward_staged_rows",
    "engram_project_windows", "engram_prepass", "engram_gate_bf16kv",
    "engram_layer_bind_shard", "engram_scale_range", "engram_hash_by_bucket",
    "engram_raw_row_bytes", "engram_host_table_alloc", "engram_host_table_free",
    "engram_shard_gather_raw", "engram_stage_raw_rows",
    "engram_embed", "engram_embed_grad", "engram_embed_grad_workspace_bytes",
    "engram_gate_checkpoint", "engram_gate_backward", "engram_gate_backward_checkpoint",
    "engram_gate_backward_workspace_bytes", "engram_project_backward",
    "engram_project_backward_workspace_bytes", "engram_loss", "engram_loss_workspace_bytes",
    "engram_loss_backward", "engram_loss_backward_workspace_bytes",
    "engram_norm", "engram_norm_backward", "engram_norm_backward_workspace_bytes",
    "engram_grad_norm", "engram_grad_norm_workspace_bytes", "engram_adamw", "engram_adamw_rows",
    "engram_sync", "engram_ctx_set_wait_limit", "engram_debug_starve_operand",
    "engram_last_error",
)


class EngramError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status
        self.message = message


class CtxDesc(C.Structure):
    _fields_ = [
        ("vocab", C.c_uint32), ("vc", C.c_uint32), ("min_n", C.c_uint32), ("max_n", C.c_uint32),
        ("heads", C.c_uint32), ("row_dim", C.c_uint32), ("hc", C.c_uint32), ("d", C.c_uint32),
        ("pad_cid", C.c_uint32), ("n_layers", C.c_uint32), ("eps", C.c_double),
        ("layer_seeds", C.POINTER(C.c_uint64)), ("bucket_bases", C.POINTER(C.c_uint64)),
    ]


BIND_BF16_OPERANDS = 1
BIND_TABLE_BF16 = 2
KV_F32, KV_BF16 = 0, 1  # engram_prepass: kv as fp32, or rounded once to BF16
EMBED_F32, EMBED_BF16 = 0, 1  # engram_embed: the table's type
F32, BF16, MXFP8 = 0, 1, 2  # engram_norm and the calls after it


class LayerWeights(C.Structure):
    _fields_ = [
        ("table", C.c_void_p), ("scales", C.c_void_p), ("rows", C.c_uint64),
        ("wkv", C.c_void_p), ("wq", C.c_void_p), ("wk", C.c_void_p), ("flags", C.c_uint32),
    ]


class LayerInfo(C.Structure):
    _fields_ = [
        ("rows", C.c_uint64), ("bound", C.c_int32), ("fp16_operands", C.c_int32),
        ("scale_min", C.c_uint32), ("scale_max", C.c_uint32), ("wkv_exp", C.c_int32),
        ("a_exp_shift", C.c_int32), ("bucket_gather", C.c_int32), ("table_bf16", C.c_int32),
    ]


class GradPart(C.Structure):
    _fields_ = [("grad", C.c_void_p), ("count", C.c_void_p), ("n", C.c_uint64), ("dim", C.c_uint32),
                ("format", C.c_int32)]


class _AdamWStep(C.Structure):
    _fields_ = [("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double), ("eps", C.c_double),
                ("seed", C.c_uint64), ("d_lr", C.c_void_p), ("d_step", C.c_void_p),
                ("d_factor", C.c_void_p), ("step", C.c_uint32), ("state_format", C.c_int32)]


class AdamWTensor(C.Structure):
    _fields_ = [("param", C.c_void_p), ("master", C.c_void_p), ("grad", C.c_void_p), ("m", C.c_void_p),
                ("v", C.c_void_p), ("m_scales", C.c_void_p), ("v_scales", C.c_void_p),
                ("n", C.c_uint64), ("lr_scale", C.c_float), ("weight_decay", C.c_float),
                ("param_format", C.c_int32), ("grad_format", C.c_int32)]


class _AdamWTable(C.Structure):
    _fields_ = [("table", C.c_void_p), ("scales", C.c_void_p), ("master", C.c_void_p),
                ("m", C.c_void_p), ("v", C.c_void_p), ("m_scales", C.c_void_p),
                ("v_scales", C.c_void_p), ("rows", C.c_uint64), ("dim", C.c_uint32),
                ("table_format", C.c_int32), ("lr_scale", C.c_float), ("weight_decay", C.c_float)]


_lib = None


def lib() -> C.CDLL:
    """Load libengram.so (built in-tree by ``build.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build the CUDA library first "
                               "(engram_gram_conditional_gb300.build.build())")
        L = C.CDLL(LIB_PATH)
        vp, i64, st = C.c_void_p, C.c_int64, C.c_int
        u32, u64, f32 = C.c_uint32, C.c_uint64, C.c_float
        sig = {
            "engram_ctx_create": [C.POINTER(CtxDesc), vp, C.POINTER(vp)],
            "engram_ctx_destroy": [vp],
            "engram_layer_params": [vp, C.c_int, vp, vp, vp, vp],
            "engram_layer_set_multipliers": [vp, C.c_int, vp],
            "engram_layer_bind": [vp, C.c_int, C.POINTER(LayerWeights)],
            "engram_layer_refresh": [vp, C.c_int, vp],
            "engram_layer_info": [vp, C.c_int, C.POINTER(LayerInfo)],
            "engram_table_fill": [vp, C.c_uint64, vp, vp, C.c_uint64, C.c_uint64, vp],
            "engram_table_fill_bf16": [vp, C.c_uint64, vp, C.c_uint64, C.c_uint64, vp],
            "engram_session_create": [vp, C.POINTER(vp)],
            "engram_session_fork": [vp, C.POINTER(vp)],
            "engram_session_reset": [vp],
            "engram_session_destroy": [vp],
            "engram_session_append": [vp, vp, vp, i64, vp],
            "engram_batch_append": [vp, vp, vp, i64, vp],
            "engram_hash": [vp, C.c_int, vp, i64, vp, vp],
            "engram_gather_dequant": [vp, C.c_int, vp, i64, vp, vp],
            "engram_project": [vp, C.c_int, vp, i64, vp, vp],
            "engram_gate": [vp, C.c_int, vp, vp, i64, vp, vp, vp],
            "engram_forward": [vp, C.c_int, vp, i64, vp, vp, vp, vp],
            "engram_project_windows": [vp, C.c_int, vp, i64, vp, vp],
            "engram_prepass": [vp, C.c_int, vp, i64, vp, C.c_int, vp, vp],
            "engram_gate_bf16kv": [vp, C.c_int, vp, vp, i64, vp, vp, vp],
            "engram_forward_noalloc": [vp, C.c_int, vp, i64, vp, vp, vp],
            "engram_forward_staged": [vp, C.c_int, vp, i64, vp, vp, vp, vp],
            "engram_stage_rows": [vp, C.c_int, vp, i64, vp, vp],
            "engram_forward_staged_rows": [vp, C.c_int, vp, i64, vp, vp, vp, vp],
            "engram_sync": [vp, vp],
            "engram_ctx_set_wait_limit": [vp, i64],
            "engram_layer_bind_shard": [vp, C.c_int, C.POINTER(LayerWeights), C.c_uint64,
                                        C.c_uint32, C.c_uint32],
            "engram_scale_range": [vp, vp, C.c_uint64, C.POINTER(C.c_uint32),
                                   C.POINTER(C.c_uint32)],
            "engram_host_table_alloc": [C.c_uint64, C.POINTER(vp)],
            "engram_host_table_free": [vp, C.c_uint64],
            "engram_hash_by_bucket": [vp, C.c_int, vp, i64, vp, vp],
            "engram_shard_gather_raw": [vp, C.c_int, vp, i64, vp, vp],
            "engram_stage_raw_rows": [vp, C.c_int, vp, vp, i64, vp, vp],
            "engram_debug_starve_operand": [vp, C.c_int],
            "engram_embed": [vp, vp, C.c_int, u64, u32, vp, i64, f32, u32, vp, vp],
            "engram_embed_grad": [vp, u64, u32, vp, i64, f32, u32, vp, vp, vp, vp, C.c_int, vp, vp],
            "engram_gate_checkpoint": [vp, C.c_int, vp, C.c_int, vp, i64, vp, vp, vp, vp, vp, vp],
            "engram_gate_backward": [vp, C.c_int, vp, C.c_int, vp, vp, i64, vp, vp, vp, vp, vp, vp,
                                     vp],
            "engram_gate_backward_checkpoint": [vp, C.c_int, vp, vp, vp, i64, vp, vp, vp, vp, vp,
                                                vp, vp],
            "engram_project_backward": [vp, C.c_int, vp, vp, i64, vp, vp, vp, vp],
            "engram_loss": [vp, vp, vp, u32, u32, vp, i64, vp, vp, vp, vp],
            "engram_loss_backward": [vp, vp, vp, u32, u32, vp, i64, vp, vp, vp, vp, vp, vp],
            "engram_norm": [vp, vp, C.c_int, u32, f32, vp, vp, i64, u32, f32, vp, vp, C.c_int, vp, vp],
            "engram_norm_backward": [vp, vp, C.c_int, vp, i64, u32, f32, vp, vp, u32, f32, vp, vp, vp,
                                     vp, vp],
            "engram_grad_norm": [vp, C.POINTER(GradPart), C.c_int32, f32, vp, vp, vp, vp, vp],
            "engram_adamw": [vp, C.POINTER(AdamWTensor), C.c_int32, C.POINTER(_AdamWStep), vp],
            "engram_adamw_rows": [vp, C.POINTER(_AdamWTable), vp, vp, i64, vp, C.POINTER(_AdamWStep),
                                  vp],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = st
        for name in ("engram_workspace_bytes", "engram_forward_staged_workspace_bytes",
                     "engram_gate_backward_workspace_bytes",
                     "engram_project_backward_workspace_bytes"):
            getattr(L, name).argtypes = [vp, i64]
            getattr(L, name).restype = C.c_size_t
        for name, args in (("engram_embed_grad_workspace_bytes", [i64, u64, u32]),
                           ("engram_loss_workspace_bytes", [i64, u32, u32]),
                           ("engram_loss_backward_workspace_bytes", [i64, u32, u32]),
                           ("engram_norm_backward_workspace_bytes", [i64, u32]),
                           ("engram_grad_norm_workspace_bytes", [C.POINTER(GradPart), C.c_int32])):
            getattr(L, name).argtypes = args
            getattr(L, name).restype = C.c_size_t
        L.engram_raw_row_bytes.argtypes = [vp]
        L.engram_raw_row_bytes.restype = C.c_size_t
        L.engram_last_error.argtypes = []
        L.engram_last_error.restype = C.c_char_p
        _lib = L
    return _lib


def engram_last_error() -> str:
    return lib().engram_last_error().decode()


def _check(status: int):
    if status != OK:
        raise EngramError(status, engram_last_error())


def _ptr(x):
    """Address of a buffer: int, None, torch tensor, numpy array or ctypes object."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if isinstance(x, np.ndarray):
        assert x.flags["C_CONTIGUOUS"], "numpy buffers must be C-contiguous"
        return x.ctypes.data
    if isinstance(x, C.c_void_p):
        return x.value
    raise TypeError(f"cannot take the address of {type(x)}")


def _stream(s):
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream  # torch.cuda.Stream


# ---- context and layers ---------------------------------------------------------------

def engram_ctx_create(vocab, vc, token_map, layer_seeds, bucket_bases, *, min_n=2, max_n=4,
                      heads=8, row_dim=256, hc=4, d=5120, pad_cid=0, eps=1e-6):
    seeds = np.ascontiguousarray(layer_seeds, dtype=np.uint64)
    bases = np.ascontiguousarray(bucket_bases, dtype=np.uint64)
    tmap = np.ascontiguousarray(token_map, dtype=np.uint32)
    if tmap.size != vocab:
        raise EngramError(EINVAL, "token_map must have vocab entries")
    desc = CtxDesc(vocab, vc, min_n, max_n, heads, row_dim, hc, d, pad_cid, len(seeds), eps,
                   seeds.ctypes.data_as(C.POINTER(C.c_uint64)),
                   bases.ctypes.data_as(C.POINTER(C.c_uint64)))
    out = C.c_void_p()
    _check(lib().engram_ctx_create(C.byref(desc), tmap.ctypes.data, C.byref(out)))
    return out


def engram_ctx_destroy(ctx):
    _check(lib().engram_ctx_destroy(ctx))


def engram_layer_params(ctx, layer: int, nb: int):
    mult = np.zeros((nb, 4), np.uint64)
    prime = np.zeros(nb, np.uint64)
    offset = np.zeros(nb, np.uint64)
    rows = np.zeros(1, np.uint64)
    _check(lib().engram_layer_params(ctx, layer, mult.ctypes.data, prime.ctypes.data,
                                     offset.ctypes.data, rows.ctypes.data))
    return mult, prime, offset, int(rows[0])


def engram_layer_set_multipliers(ctx, layer: int, mult):
    m = np.ascontiguousarray(mult, dtype=np.uint64)
    _check(lib().engram_layer_set_multipliers(ctx, layer, m.ctypes.data))


def engram_layer_bind(ctx, layer: int, table, scales, rows: int, wkv, wq, wk, flags: int = 0):
    w = LayerWeights(_ptr(table), _ptr(scales), rows, _ptr(wkv), _ptr(wq), _ptr(wk), flags)
    _check(lib().engram_layer_bind(ctx, layer, C.byref(w)))


def engram_layer_refresh(ctx, layer: int, stream=None):
    _check(lib().engram_layer_refresh(ctx, layer, _stream(stream)))


def engram_layer_info(ctx, layer: int) -> dict:
    info = LayerInfo()
    _check(lib().engram_layer_info(ctx, layer, C.byref(info)))
    return {name: getattr(info, name) for name, _ in LayerInfo._fields_}


def engram_table_fill(ctx, seed: int, data, scale, row_begin: int, row_end: int, stream=None):
    _check(lib().engram_table_fill(ctx, seed, _ptr(data), _ptr(scale), row_begin, row_end,
                                   _stream(stream)))


def engram_table_fill_bf16(ctx, seed: int, data, row_begin: int, row_end: int, stream=None):
    _check(lib().engram_table_fill_bf16(ctx, seed, _ptr(data), row_begin, row_end,
                                        _stream(stream)))


# ---- sessions -------------------------------------------------------------------------

def engram_session_create(ctx):
    out = C.c_void_p()
    _check(lib().engram_session_create(ctx, C.byref(out)))
    return out


def engram_session_fork(session):
    out = C.c_void_p()
    _check(lib().engram_session_fork(session, C.byref(out)))
    return out


def engram_session_reset(session):
    _check(lib().engram_session_reset(session))


def engram_session_destroy(session):
    _check(lib().engram_session_destroy(session))


def engram_session_append(session, tokens, is_image=None, windows_out=None):
    """Append tokens; returns the windows (uint32 [n][4], host)."""
    tk = np.ascontiguousarray(tokens, dtype=np.int32)
    im = None if is_image is None else np.ascontiguousarray(is_image, dtype=np.uint8)
    out = np.empty((tk.size, 4), np.uint32) if windows_out is None else windows_out
    _check(lib().engram_session_append(session, tk.ctypes.data,
                                       None if im is None else im.ctypes.data, tk.size,
                                       _ptr(out)))
    return out


def engram_batch_append(sessions, tokens, is_image=None, windows_out=None):
    """Append one token to each session; returns the windows (uint32 [n][4], host)."""
    arr = (C.c_void_p * len(sessions))(*[s.value if isinstance(s, C.c_void_p) else s
                                         for s in sessions])
    tk = np.ascontiguousarray(tokens, dtype=np.int32)
    im = None if is_image is None else np.ascontiguousarray(is_image, dtype=np.uint8)
    out = np.empty((len(sessions), 4), np.uint32) if windows_out is None else windows_out
    _check(lib().engram_batch_append(C.cast(arr, C.c_void_p), tk.ctypes.data,
                                     None if im is None else im.ctypes.data, len(sessions),
                                     _ptr(out)))
    return out


# ---- device steps -----------------------------------------------------------------------

def engram_workspace_bytes(ctx, T: int) -> int:
    return int(lib().engram_workspace_bytes(ctx, T))


def engram_hash(ctx, layer, d_windows, T, d_rows, stream=None):
    _check(lib().engram_hash(ctx, layer, _ptr(d_windows), T, _ptr(d_rows), _stream(stream)))


def engram_gather_dequant(ctx, layer, d_rows, T, d_emb, stream=None):
    _check(lib().engram_gather_dequant(ctx, layer, _ptr(d_rows), T, _ptr(d_emb), _stream(stream)))


def engram_project(ctx, layer, d_emb, T, d_kv, stream=None):
    _check(lib().engram_project(ctx, layer, _ptr(d_emb), T, _ptr(d_kv), _stream(stream)))


def engram_gate(ctx, layer, d_kv, d_windows, T, d_hidden, d_gates=None, stream=None):
    _check(lib().engram_gate(ctx, layer, _ptr(d_kv), _ptr(d_windows), T, _ptr(d_hidden),
                             _ptr(d_gates), _stream(stream)))


def engram_forward(ctx, layer, d_windows, T, d_hidden, d_workspace, d_gates=None, stream=None):
    _check(lib().engram_forward(ctx, layer, _ptr(d_windows), T, _ptr(d_hidden), _ptr(d_workspace),
                                _ptr(d_gates), _stream(stream)))


def engram_forward_staged_workspace_bytes(ctx, T: int) -> int:
    return int(lib().engram_forward_staged_workspace_bytes(ctx, T))


def engram_forward_staged(ctx, layer, d_windows, T, d_hidden, d_workspace, d_gates=None,
                          stream=None):
    _check(lib().engram_forward_staged(ctx, layer, _ptr(d_windows), T, _ptr(d_hidden),
                                       _ptr(d_workspace), _ptr(d_gates), _stream(stream)))


def engram_stage_rows(ctx, layer, d_windows, T, d_workspace, stream=None):
    _check(lib().engram_stage_rows(ctx, layer, _ptr(d_windows), T, _ptr(d_workspace),
                                   _stream(stream)))


def engram_forward_staged_rows(ctx, layer, d_windows, T, d_hidden, d_workspace, d_gates=None,
                               stream=None):
    _check(lib().engram_forward_staged_rows(ctx, layer, _ptr(d_windows), T, _ptr(d_hidden),
                                            _ptr(d_workspace), _ptr(d_gates), _stream(stream)))


def engram_forward_noalloc(ctx, layer, d_windows, T, d_hidden, d_gates=None, stream=None):
    """engram_forward without a workspace argument, for callers that cannot allocate:
    the scratch is the library's built-in 8 MiB device buffer (see include/engram.h)."""
    _check(lib().engram_forward_noalloc(ctx, layer, _ptr(d_windows), T, _ptr(d_hidden),
                                        _ptr(d_gates), _stream(stream)))


def engram_project_windows(ctx, layer, d_windows, T, d_kv, stream=None):
    _check(lib().engram_project_windows(ctx, layer, _ptr(d_windows), T, _ptr(d_kv),
                                        _stream(stream)))


def engram_prepass(ctx, layer, d_windows, T, d_kv, kv_format, d_workspace, stream=None):
    _check(lib().engram_prepass(ctx, layer, _ptr(d_windows), T, _ptr(d_kv), int(kv_format),
                                _ptr(d_workspace), _stream(stream)))


def engram_gate_bf16kv(ctx, layer, d_kv, d_windows, T, d_hidden, d_gates=None, stream=None):
    _check(lib().engram_gate_bf16kv(ctx, layer, _ptr(d_kv), _ptr(d_windows), T, _ptr(d_hidden),
                                    _ptr(d_gates), _stream(stream)))


def engram_layer_bind_shard(ctx, layer: int, table, scales, rows: int, wkv, wq, wk, row_lo: int,
                            scale_min: int, scale_max: int, flags: int = 0):
    w = LayerWeights(_ptr(table), _ptr(scales), rows, _ptr(wkv), _ptr(wq), _ptr(wk), flags)
    _check(lib().engram_layer_bind_shard(ctx, layer, C.byref(w), row_lo, scale_min, scale_max))


def engram_scale_range(ctx, scales, n: int):
    """(min, max) of n E8M0 bytes on the device (255, 0 for n = 0)."""
    lo, hi = C.c_uint32(), C.c_uint32()
    _check(lib().engram_scale_range(ctx, _ptr(scales), n, C.byref(lo), C.byref(hi)))
    return lo.value, hi.value


def engram_host_table_alloc(nbytes: int) -> int:
    """Registered, huge-page-advised host memory for a table read through UVA
    (see include/engram.h); returns its address (host and device)."""
    out = C.c_void_p()
    _check(lib().engram_host_table_alloc(nbytes, C.byref(out)))
    return out.value


def engram_host_table_free(ptr: int, nbytes: int):
    _check(lib().engram_host_table_free(ptr, nbytes))


def engram_hash_by_bucket(ctx, layer, d_windows, T, d_rows_bm, stream=None):
    _check(lib().engram_hash_by_bucket(ctx, layer, _ptr(d_windows), T, _ptr(d_rows_bm),
                                       _stream(stream)))


def engram_raw_row_bytes(ctx) -> int:
    return int(lib().engram_raw_row_bytes(ctx))


def engram_shard_gather_raw(ctx, layer, d_ids, n, d_raw, stream=None):
    _check(lib().engram_shard_gather_raw(ctx, layer, _ptr(d_ids), n, _ptr(d_raw), _stream(stream)))


def engram_stage_raw_rows(ctx, layer, d_rows_bm, d_raw_bm, T, d_workspace, stream=None):
    _check(lib().engram_stage_raw_rows(ctx, layer, _ptr(d_rows_bm), _ptr(d_raw_bm), T,
                                       _ptr(d_workspace), _stream(stream)))


# ---- training ----------------------------------------------------------------------------

def engram_embed(ctx, d_table, table_format, rows, dim, d_ids, n, scale, copies, d_out,
                 stream=None):
    _check(lib().engram_embed(ctx, _ptr(d_table), int(table_format), rows, dim, _ptr(d_ids), n,
                              scale, copies, _ptr(d_out), _stream(stream)))


def engram_embed_grad_workspace_bytes(n: int, rows: int, dim: int) -> int:
    return int(lib().engram_embed_grad_workspace_bytes(n, rows, dim))


def engram_embed_grad(ctx, rows, dim, d_ids, n, scale, copies, d_dout, d_unique, d_count, d_grad,
                      accumulate, d_workspace, stream=None):
    _check(lib().engram_embed_grad(ctx, rows, dim, _ptr(d_ids), n, scale, copies, _ptr(d_dout),
                                   _ptr(d_unique), _ptr(d_count), _ptr(d_grad), int(accumulate),
                                   _ptr(d_workspace), _stream(stream)))


def engram_gate_checkpoint(ctx, layer, d_kv, kv_format, d_windows, T, d_hidden, d_hidden_out,
                           d_gates, d_codes, d_scales, stream=None):
    _check(lib().engram_gate_checkpoint(ctx, layer, _ptr(d_kv), int(kv_format), _ptr(d_windows), T,
                                        _ptr(d_hidden), _ptr(d_hidden_out), _ptr(d_gates),
                                        _ptr(d_codes), _ptr(d_scales), _stream(stream)))


def engram_gate_backward_workspace_bytes(ctx, T: int) -> int:
    return int(lib().engram_gate_backward_workspace_bytes(ctx, T))


def engram_gate_backward(ctx, layer, d_kv, kv_format, d_hidden, d_windows, T, d_dout, d_dhidden,
                         d_dkv, d_dwq, d_dwk, d_workspace, stream=None):
    _check(lib().engram_gate_backward(ctx, layer, _ptr(d_kv), int(kv_format), _ptr(d_hidden),
                                      _ptr(d_windows), T, _ptr(d_dout), _ptr(d_dhidden),
                                      _ptr(d_dkv), _ptr(d_dwq), _ptr(d_dwk), _ptr(d_workspace),
                                      _stream(stream)))


def engram_gate_backward_checkpoint(ctx, layer, d_codes, d_scales, d_windows, T, d_dout, d_dhidden,
                                    d_dkv, d_dwq, d_dwk, d_workspace, stream=None):
    _check(lib().engram_gate_backward_checkpoint(ctx, layer, _ptr(d_codes), _ptr(d_scales),
                                                 _ptr(d_windows), T, _ptr(d_dout), _ptr(d_dhidden),
                                                 _ptr(d_dkv), _ptr(d_dwq), _ptr(d_dwk),
                                                 _ptr(d_workspace), _stream(stream)))


def engram_project_backward_workspace_bytes(ctx, T: int) -> int:
    return int(lib().engram_project_backward_workspace_bytes(ctx, T))


def engram_project_backward(ctx, layer, d_emb, d_dkv, T, d_demb, d_dwkv, d_workspace, stream=None):
    _check(lib().engram_project_backward(ctx, layer, _ptr(d_emb), _ptr(d_dkv), T, _ptr(d_demb),
                                         _ptr(d_dwkv), _ptr(d_workspace), _stream(stream)))


def engram_loss_workspace_bytes(T: int, vocab: int, dim: int) -> int:
    return int(lib().engram_loss_workspace_bytes(T, vocab, dim))


def engram_loss(ctx, d_x, d_head, vocab, dim, d_labels, T, d_loss, d_lse, d_workspace, stream=None):
    _check(lib().engram_loss(ctx, _ptr(d_x), _ptr(d_head), vocab, dim, _ptr(d_labels), T,
                             _ptr(d_loss), _ptr(d_lse), _ptr(d_workspace), _stream(stream)))


def engram_loss_backward_workspace_bytes(T: int, vocab: int, dim: int) -> int:
    return int(lib().engram_loss_backward_workspace_bytes(T, vocab, dim))


def engram_loss_backward(ctx, d_x, d_head, vocab, dim, d_labels, T, d_lse, d_dloss, d_dx, d_dhead,
                         d_workspace, stream=None):
    _check(lib().engram_loss_backward(ctx, _ptr(d_x), _ptr(d_head), vocab, dim, _ptr(d_labels), T,
                                      _ptr(d_lse), _ptr(d_dloss), _ptr(d_dx), _ptr(d_dhead),
                                      _ptr(d_workspace), _stream(stream)))


def engram_norm(ctx, d_x, format, copies, scale, d_residual, d_weight, n, dim, eps, d_sum, d_y, y_format,
                d_y_scales=None, stream=None):
    _check(lib().engram_norm(ctx, _ptr(d_x), int(format), copies, scale, _ptr(d_residual),
                             _ptr(d_weight), n, dim, eps, _ptr(d_sum), _ptr(d_y), int(y_format),
                             _ptr(d_y_scales), _stream(stream)))


def engram_norm_backward_workspace_bytes(n: int, dim: int) -> int:
    return int(lib().engram_norm_backward_workspace_bytes(n, dim))


def engram_norm_backward(ctx, d_sum, format, d_weight, n, dim, eps, d_dy, d_dsum, copies, scale, d_dx,
                         d_dresidual, d_dweight, d_workspace, stream=None):
    _check(lib().engram_norm_backward(ctx, _ptr(d_sum), int(format), _ptr(d_weight), n, dim, eps,
                                      _ptr(d_dy), _ptr(d_dsum), copies, scale, _ptr(d_dx),
                                      _ptr(d_dresidual), _ptr(d_dweight), _ptr(d_workspace),
                                      _stream(stream)))


def _format(x) -> int:
    """F32 or BF16 of a tensor (BF16 ones may be viewed as 16-bit whole numbers)."""
    kind = str(x.dtype).replace("torch.", "")
    if kind not in ("float32", "bfloat16", "int16", "uint16"):
        raise EngramError(EINVAL, f"fp32 or BF16 values expected, got {x.dtype}")
    return F32 if kind == "float32" else BF16


def _flat(name, x, n):
    """The address of a contiguous tensor of n values."""
    if x is None:
        return None
    if not x.is_contiguous() or x.numel() != n:
        raise EngramError(EINVAL, f"{name}: {n} contiguous values expected, got {list(x.shape)}")
    return x.data_ptr()


def _held(name, x, n, sizes):
    """The address of a contiguous tensor of at least n values of `sizes` (a tuple) bytes each; other
    buffers' as they are."""
    if x is None or isinstance(x, int):
        return x
    if not hasattr(x, "data_ptr"):
        return _ptr(x)
    if x.numel() < n or x.element_size() not in sizes or not x.is_contiguous():
        raise EngramError(EINVAL, f"{name}: {n} contiguous values of {' or '.join(map(str, sizes))} bytes expected, "
                                  f"got {x.dtype} {list(x.shape)}")
    return x.data_ptr()


def _place(buffers, place=None):
    """The index of the CUDA device that all tensors among `buffers` (and those of `place`) are on, None
    where there are only addresses, -1 where one is elsewhere."""
    for x in buffers:
        if x is None or isinstance(x, int):
            continue
        at = x.get_device() if hasattr(x, "get_device") else -1 if isinstance(x, np.ndarray) else place
        if place is None:
            place = at
        elif at != place:
            return -1
    return place


_current_device = None  # torch's function, from the first call that has tensors on


def _on_device(name, place):
    """Refuses buffers that the kernels would not find on the current device."""
    global _current_device
    if place is None:
        return
    if _current_device is None:
        import torch

        _current_device = torch.cuda.current_device
    if place < 0 or _current_device() != place:
        raise EngramError(EINVAL, f"{name}: tensors on the current CUDA device expected")


def grad_parts(parts):
    """engram_grad_norm's list from dicts: ``grad`` (a tensor, fp32 or BF16), and for the sparse
    gradient of a table ``count`` (a device uint32) and ``dim`` (values of a row).  The list
    keeps the tensors alive."""
    out = (GradPart * len(parts))()
    out.kept = [dict(p) for p in parts]
    out.place = _place([x for p in parts for x in (p["grad"], p.get("count"))])
    for c, p in zip(out, parts):
        grad, dim = p["grad"], p.get("dim", 1)
        if grad.numel() % dim:
            raise EngramError(EINVAL, f"grad: rows of {dim} values expected, got {list(grad.shape)}")
        c.grad, c.count = _flat("grad", grad, grad.numel()), _held("count", p.get("count"), 1, (4,))
        c.n, c.dim, c.format = grad.numel() // dim, dim, _format(grad)
    return out


def engram_grad_norm_workspace_bytes(parts) -> int:
    """``parts``: grad_parts()'s list."""
    return int(lib().engram_grad_norm_workspace_bytes(parts, len(parts)))


def engram_grad_norm(ctx, parts, max_norm, d_norms, d_norm, d_factor, d_workspace, stream=None):
    """``parts``: grad_parts()'s list."""
    _on_device("parts", getattr(parts, "place", None))
    _check(lib().engram_grad_norm(ctx, parts, len(parts), max_norm, _ptr(d_norms), _ptr(d_norm),
                                  _ptr(d_factor), _ptr(d_workspace), _stream(stream)))


def adamw_tensors(tensors):
    """engram_adamw's list from dicts of tensors: ``param``, ``grad``, ``m``, ``v``, and, where there
    are such, ``master``, ``m_scales``, ``v_scales``, ``lr_scale`` (1) and ``weight_decay`` (0).  The
    list keeps the tensors alive."""
    out = (AdamWTensor * len(tensors))()
    out.kept = [dict(t) for t in tensors]
    out.place = _place([x for t in tensors for x in t.values() if not isinstance(x, float)])
    sizes = {t[name].element_size() for t in tensors for name in ("m", "v")}
    if len(sizes) > 1 or not sizes <= {1, 4}:
        raise EngramError(EINVAL, "m and v: all fp32, or all 8-bit codes")
    out.state_format = MXFP8 if sizes == {1} else F32 if sizes else None
    for c, t in zip(out, tensors):
        n = t["param"].numel()
        if t.get("master") is not None and t["master"].element_size() != 4:
            raise EngramError(EINVAL, "master: fp32 values expected")
        for name in ("param", "master", "grad", "m", "v"):
            setattr(c, name, _flat(name, t.get(name), n))
        for name in ("m_scales", "v_scales"):
            setattr(c, name, _flat(name, t.get(name), (n + 31) // 32))
        c.n, c.lr_scale, c.weight_decay = n, t.get("lr_scale", 1.0), t.get("weight_decay", 0.0)
        c.param_format, c.grad_format = _format(t["param"]), _format(t["grad"])
    return out


def _word(name, x, floating):
    """The address of a device word: fp32, or a whole number of 32 bits."""
    if x is None or not hasattr(x, "data_ptr"):
        return _ptr(x)
    if x.element_size() != 4 or x.is_floating_point() != floating or x.numel() < 1:
        raise EngramError(EINVAL, f"{name}: {'fp32' if floating else 'int32'} expected, got {x.dtype} {list(x.shape)}")
    return x.data_ptr()


def AdamWStep(lr=0.0, beta1=0.9, beta2=0.999, eps=1e-8, step=0, seed=0, state_format=F32, d_lr=None,
              d_step=None, d_factor=None):
    """engram_adamw_step; d_lr, d_step and d_factor: device tensors (or addresses) or None."""
    out = _AdamWStep(lr, beta1, beta2, eps, seed, _word("d_lr", d_lr, True), _word("d_step", d_step, False),
                     _word("d_factor", d_factor, True), step, int(state_format))
    out.kept = d_lr, d_step, d_factor
    out.place = _place(out.kept)
    return out


_SIZES = {F32: (4,), BF16: (2,), MXFP8: (1,)}


def AdamWTable(table, rows, dim, table_format, m, v, scales=None, master=None, m_scales=None,
               v_scales=None, lr_scale=1.0, weight_decay=0.0):
    """engram_adamw_table; the buffers are device tensors (or addresses)."""
    n, one, four = rows * dim, (1,), (4,)
    state = one if hasattr(m, "data_ptr") and m.element_size() == 1 else four
    out = _AdamWTable(_held("table", table, n, _SIZES.get(table_format, (1, 2, 4))), _held("scales", scales, n // 32, one),
                      _held("master", master, n, four), _held("m", m, n, state), _held("v", v, n, state),
                      _held("m_scales", m_scales, n // 32, one), _held("v_scales", v_scales, n // 32, one),
                      rows, dim, int(table_format), lr_scale, weight_decay)
    out.kept = table, scales, master, m, v, m_scales, v_scales
    out.place = _place(out.kept)
    out.state_format = None if not hasattr(m, "data_ptr") else MXFP8 if state is one else F32
    return out


def _goes_with(step, out, name, buffers=()):
    """Refuses a list or table whose states are not the step's, and buffers that are not on the device."""
    kept = getattr(out, "state_format", None)
    if step is not None and kept is not None and kept != step.state_format:
        raise EngramError(EINVAL, f"state_format: the states of {name} have the other one")
    place, other = getattr(out, "place", None), getattr(step, "place", None)
    _on_device(name, _place(buffers, other if place is None else place if other is None or other == place else -1))


def engram_adamw(ctx, tensors, step, stream=None):
    """``tensors``: adamw_tensors()'s list; ``step``: AdamWStep()."""
    _goes_with(step, tensors, "tensors")
    _check(lib().engram_adamw(ctx, tensors, len(tensors), None if step is None else C.byref(step),
                              _stream(stream)))


def engram_adamw_rows(ctx, table, d_ids, d_count, n, d_grad, step, stream=None):
    """``table``: AdamWTable(); ``step``: AdamWStep()."""
    _goes_with(step, table, "table, step and gradient", (d_ids, d_count, d_grad))
    dim = 0 if table is None else table.dim
    _check(lib().engram_adamw_rows(ctx, None if table is None else C.byref(table), _held("ids", d_ids, n, (4,)),
                                   _held("count", d_count, 1, (4,)), n, _held("grad", d_grad, n * dim, (4,)),
                                   None if step is None else C.byref(step), _stream(stream)))


def engram_ctx_set_wait_limit(ctx, ns: int):
    _check(lib().engram_ctx_set_wait_limit(ctx, ns))


def engram_debug_starve_operand(ctx, on: bool):
    _check(lib().engram_debug_starve_operand(ctx, 1 if on else 0))


def engram_sync(ctx, stream=None):
    _check(lib().engram_sync(ctx, _stream(stream)))
