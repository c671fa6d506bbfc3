"""Thin ctypes binding of ``libttsdecode.so`` (declared in ``include/tts_decode.h``).

Argument marshalling only: every function takes device tensors, passes their
pointers, strides and the current CUDA stream to the C entry point of the same name,
and raises ``TtsError`` on a non-OK status.  There is no fallback: if the library has
not been built, importing this module raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("TTS_LIBRARY") or os.path.join(_HERE, "_build", "libttsdecode.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the CUDA library first "
        "(python -m autoregressive_codebook_tts_gb300.build)")

_lib = ctypes.CDLL(LIB_PATH)

TTS_F32, TTS_BF16, TTS_Q8_0, TTS_I8, TTS_E4M3 = 0, 1, 2, 3, 4
Q8_0_BLOCK, Q8_0_BYTES = 32, 34  # entries and bytes of a Q8_0 block
TTS_MAX_TABLES = 16
TTS_MAX_TREE_NODES = 64
TTS_MAX_NORM_WIDTH, TTS_MAX_ADAPTER_RANK, TTS_MAX_PLAN_STREAMS = 16384, 128, 4096
TTS_KV_PREFETCH_BEFORE_WAIT = 1

EFLAG_ID_RANGE = 1
EFLAG_POS_RANGE = 2
EFLAG_PAGE = 4
EFLAG_NVALID = 8
EFLAG_TIMEOUT = 16

EXPORTED = [
    "tts_abi_version", "tts_abi_min_version", "tts_abi_check", "tts_status_str", "tts_frame_embed",
    "tts_rope_table", "tts_qk_norm_rope", "tts_kv_set_rows", "tts_decode_attn_workspace_size",
    "tts_decode_attn_default_splits", "tts_workspace_init", "tts_decode_attn", "tts_decode_step",
    "tts_decode_step_noalloc",
    "tts_prefill_workspace_size",
    "tts_prefill_launch_count",
    "tts_prefill_step",
    "tts_sample",
    "tts_sample_embed",
    "tts_counter_advance",
    "tts_check_wait_timeout",
    "tts_decode_layer_scratch_size",
    "tts_decode_layer_launch_count",
    "tts_decode_layer",
    "tts_rope_table_scaled",
    "tts_rope_rows",
    "tts_kv_write_rows",
    "tts_kv_read_rows",
    "tts_tree_attn_workspace_size",
    "tts_tree_attn",
    "tts_tree_commit",
    "tts_add_rms_norm",
    "tts_project_workspace_size",
    "tts_project_rows",
    "tts_page_plan",
    "tts_kv_write_slots",
]


class TtsTables(ctypes.Structure):
    _fields_ = [("tab", ctypes.c_void_p * TTS_MAX_TABLES), ("n_tables", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("hidden", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class TtsKvDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("window_quantum", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("paged", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("bt_stride", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("block_table", ctypes.c_void_p)]


class TtsLayerWeights(ctypes.Structure):
    _fields_ = [("w_qkv", ctypes.c_void_p), ("w_o", ctypes.c_void_p), ("w_gu", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("gamma_attn", ctypes.c_void_p),
                ("gamma_mlp", ctypes.c_void_p), ("gamma_q", ctypes.c_void_p),
                ("gamma_k", ctypes.c_void_p), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32)]


class TtsRopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("original_max_pos", ctypes.c_int32),
                ("factor", ctypes.c_double), ("low_rotations", ctypes.c_double),
                ("high_rotations", ctypes.c_double), ("attn_scale", ctypes.c_double)]


class TtsKvCache(ctypes.Structure):
    """Built by kv_cache, which also notes what the tensors behind it are."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]

    def get_device(self):
        return self.device_index


class TtsAdapters(ctypes.Structure):
    """Built by adapters, which also notes what the tensors behind it are."""
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("rank", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("n_adapters", ctypes.c_int32), ("rank_max", ctypes.c_int32)]

    def get_device(self):
        return self.device_index


_P, _I32, _I64, _F, _D, _SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                               ctypes.c_double, ctypes.c_size_t)
_sigs = {
    "tts_abi_version": ([], _I32),
    "tts_abi_min_version": ([], _I32),
    "tts_abi_check": ([_I32], _I32),
    "tts_status_str": ([_I32], ctypes.c_char_p),
    "tts_frame_embed": ([ctypes.POINTER(TtsTables), _P, _I64, _P, _I64, _P, _I32, _P, _P], _I32),
    "tts_rope_table": ([_P, _I32, _I32, _D, _P], _I32),
    "tts_qk_norm_rope": ([_P, _I64, _P, _I64, _P, _P, _P, _I32, _I32, _I32, _I32, _F, _P, _I32,
                          _P, _P], _I32),
    "tts_kv_set_rows": ([_P, _P, _I64, _P, _P, ctypes.POINTER(TtsKvDesc), _P, _P, _P], _I32),
    "tts_decode_attn_workspace_size": ([ctypes.POINTER(TtsKvDesc), _I32], _SZ),
    "tts_decode_attn_default_splits": ([ctypes.POINTER(TtsKvDesc)], _I32),
    "tts_workspace_init": ([_P, _SZ, _P], _I32),
    "tts_decode_attn": ([_P, _I64, _P, _P, ctypes.POINTER(TtsKvDesc), _P, _F, _P, _P, _SZ, _I32,
                         _P, _P], _I32),
    "tts_decode_step": ([_P, _P, _P, _I64, _P, _P, _F, _P, _I32, _P, _P,
                         ctypes.POINTER(TtsKvDesc), _P, _F, _P, _P, _SZ, _I32, _P, _P], _I32),
    "tts_decode_step_noalloc": ([_P, _P, _P, _I64, _P, _P, _F, _P, _I32, _P, _P,
                                 ctypes.POINTER(TtsKvDesc), _P, _F, _P, _I32, _P, _P], _I32),
    "tts_prefill_workspace_size": ([ctypes.POINTER(TtsKvDesc), _I32, _I32], _SZ),
    "tts_prefill_launch_count": ([ctypes.POINTER(TtsKvDesc), _I32, _I32], _I32),
    "tts_sample": ([_P, _I64, _I32, _I32, _I32, _F, ctypes.c_uint64, _P, ctypes.c_uint32, _P, _I64, _P],
                   _I32),
    "tts_sample_embed": ([_P, _I64, _I32, _I32, _I32, _F, ctypes.c_uint64, _P, ctypes.c_uint32, _P, _I64,
                          ctypes.POINTER(TtsTables), _P, _P], _I32),
    "tts_counter_advance": ([_P, ctypes.c_uint64, _P], _I32),
    "tts_check_wait_timeout": ([_P, _P], _I32),
    "tts_decode_layer_scratch_size": ([ctypes.POINTER(TtsKvDesc), _I32, _I32, _I32], _SZ),
    "tts_decode_layer_launch_count": ([ctypes.POINTER(TtsKvDesc)], _I32),
    "tts_decode_layer": ([_P, ctypes.POINTER(TtsLayerWeights), _F, _P, _I32, _P, _P,
                          ctypes.POINTER(TtsKvDesc), _P, _F, _P, _SZ, _I32, _P, _P], _I32),
    "tts_prefill_step": ([_P, _P, _P, _I64, _P, _P, _F, _P, _I32, _P, _P,
                          ctypes.POINTER(TtsKvDesc), _P, _I32, _F, _P, _P, _SZ, _I32, _P, _P], _I32),
    "tts_rope_table_scaled": ([_P, _I32, _I32, _D, ctypes.POINTER(TtsRopeScaling), _P], _I32),
    "tts_rope_rows": ([_P, _I64, _P, _I64, _I32, _P, _I64, _P, _I64, _I32, _P, _P, _F, _P, _I32,
                       _I32, _I32, _I32, _I32, _I32, _P, _I32, _P, _P], _I32),
    "tts_kv_write_rows": ([_P, _P, _I32, _I64, ctypes.POINTER(TtsKvCache),
                           ctypes.POINTER(TtsKvDesc), _P, _P, _I32, _P, _P], _I32),
    "tts_kv_read_rows": ([ctypes.POINTER(TtsKvCache), ctypes.POINTER(TtsKvDesc), _P, _P, _I32, _P,
                          _P, _I32, _I64, _P, _P], _I32),
    "tts_tree_attn_workspace_size": ([ctypes.POINTER(TtsKvDesc), _I32, _I32], _SZ),
    "tts_tree_attn": ([_P, _I32, _I64, ctypes.POINTER(TtsKvCache), ctypes.POINTER(TtsKvDesc), _P,
                       _P, _P, _I32, _F, _P, _P, _SZ, _P, _P], _I32),
    "tts_tree_commit": ([ctypes.POINTER(TtsKvCache), ctypes.POINTER(TtsKvDesc), _P, _P, _I64, _P,
                         _I32, _P, _P], _I32),
    "tts_add_rms_norm": ([_P, _I64, _I32, _P, _I64, _I32, _P, _I64, _P, _F, _I32, _I32, _P, _I64, _I32, _P, _P], _I32),
    "tts_project_workspace_size": ([_I32, _I32, _I32, _I32, ctypes.POINTER(TtsAdapters)], _SZ),
    "tts_project_rows": ([_P, _I64, _I32, _P, _P, _P, _I32, _I32, ctypes.POINTER(TtsAdapters), _P, _P, _I32, _I32,
                          _P, _I64, _I32, _P, _SZ, _P, _P], _I32),
    "tts_page_plan": ([ctypes.POINTER(TtsKvDesc), _P, _P, _P, _P, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P], _I32),
    "tts_kv_write_slots": ([_P, _P, _I32, _I64, ctypes.POINTER(TtsKvCache), ctypes.POINTER(TtsKvDesc), _P, _I32, _P,
                            _P], _I32),
}
for _name, (_args, _ret) in _sigs.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _ret


class TtsError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_lib.tts_status_str(status).decode()}")


def _check(status: int, where: str):
    if status != 0:
        raise TtsError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _row_stride(t):
    """Elements between consecutive stream rows of a [B, ...] tensor whose rows are
    contiguous inside (e.g. a column slice of a fused projection buffer)."""
    return t.stride(0)


def abi_version() -> int:
    return _lib.tts_abi_version()


def abi_min_version() -> int:
    return _lib.tts_abi_min_version()


def abi_check(caller_version: int) -> int:
    """The library's own range test of a caller's ABI version: 0 (TTS_OK) or TTS_ERR_ABI."""
    return int(_lib.tts_abi_check(int(caller_version)))


def status_str(status: int) -> str:
    return _lib.tts_status_str(status).decode()


# ---------------------------------------------------------------------------
# Descriptors
# ---------------------------------------------------------------------------
_KV_CODES = {"f32": TTS_F32, "bf16": TTS_BF16, "i8": TTS_I8, "e4m3": TTS_E4M3,
             "float32": TTS_F32, "bfloat16": TTS_BF16, "int8": TTS_I8, "float8_e4m3fn": TTS_E4M3,
             torch.float32: TTS_F32, torch.bfloat16: TTS_BF16, torch.int8: TTS_I8,
             torch.float8_e4m3fn: TTS_E4M3}


def kv_desc(B, n_q_heads, n_kv_heads, head_dim, capacity, kv_dtype="f32", window_quantum=256,
            paged=False, page_size=16, n_pages=0, block_table=None, flags=0) -> TtsKvDesc:
    """A layer's cache.  kv_dtype: "f32", "bf16", "i8" or "e4m3", or the torch dtype (its name).
    block_table: int32 [B or more rows][pages], entries of a row contiguous."""
    if kv_dtype not in _KV_CODES:
        raise ValueError("kv_dtype must be \"f32\", \"bf16\", \"i8\", \"e4m3\" or the torch dtype")
    if paged and block_table is not None:
        if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] < B or \
                (block_table.shape[1] > 1 and block_table.stride(1) != 1):
            raise ValueError("block_table must be int32 with a contiguous row of page ids per stream")
    d = TtsKvDesc()
    d.B, d.n_q_heads, d.n_kv_heads, d.head_dim, d.capacity = B, n_q_heads, n_kv_heads, head_dim, capacity
    d.window_quantum = window_quantum
    d.kv_dtype = _KV_CODES[kv_dtype]
    d.paged = 1 if paged else 0
    d.page_size = page_size if paged else 0
    d.n_pages = n_pages if paged else 0
    d.bt_stride = block_table.stride(0) if (paged and block_table is not None) else 0
    d.flags = flags
    d.block_table = block_table.data_ptr() if (paged and block_table is not None) else None
    d.table_device = block_table.get_device() if (paged and block_table is not None) else None
    return d


def tables(tabs) -> TtsTables:
    """Table descriptor for f32, bf16 or Q8_0 tables (all of one dtype).  A Q8_0 table is
    a uint8 tensor [vocab][hidden / 32 * 34] of 34-byte blocks (binary16 scale, then 32
    int8 quants)."""
    t = TtsTables()
    dts = {x.dtype for x in tabs}
    if len(dts) != 1 or not dts <= {torch.float32, torch.bfloat16, torch.uint8}:
        raise ValueError("codebook tables must all be float32, all bfloat16 or all uint8 (Q8_0)")
    for i, x in enumerate(tabs):
        t.tab[i] = x.data_ptr()
    t.n_tables = len(tabs)
    if tabs[0].dtype == torch.uint8:
        if tabs[0].shape[1] % Q8_0_BYTES:
            raise ValueError("a Q8_0 row is a whole number of 34-byte blocks")
        t.vocab, t.hidden = tabs[0].shape[0], tabs[0].shape[1] // Q8_0_BYTES * Q8_0_BLOCK
        t.dtype = TTS_Q8_0
    else:
        t.vocab, t.hidden = tabs[0].shape
        t.dtype = TTS_BF16 if tabs[0].dtype == torch.bfloat16 else TTS_F32
    return t


# ---------------------------------------------------------------------------
# Entry points
# ---------------------------------------------------------------------------
def tts_frame_embed(tabs, ids, overlay, out, err_flag=None, stream=None):
    """out[b] = ((E_0[ids[b,0]] + ...) + overlay[b]); tabs: list of [vocab, hidden] f32."""
    t = tables(tabs) if not isinstance(tabs, TtsTables) else tabs
    _check(_lib.tts_frame_embed(ctypes.byref(t), _ptr(ids), ids.stride(0), _ptr(overlay),
                                0 if overlay is None else overlay.stride(0), _ptr(out),
                                out.shape[0], _ptr(err_flag), _stream(stream)), "tts_frame_embed")


def tts_rope_table(cs, max_pos, head_dim, base, stream=None):
    _check(_lib.tts_rope_table(_ptr(cs), max_pos, head_dim, float(base), _stream(stream)),
           "tts_rope_table")


def tts_qk_norm_rope(q, k, gamma_q, gamma_k, pos, n_q_heads, n_kv_heads, head_dim, eps, cs,
                     max_pos, err_flag=None, stream=None):
    _check(_lib.tts_qk_norm_rope(_ptr(q), _row_stride(q), _ptr(k), _row_stride(k), _ptr(gamma_q),
                                 _ptr(gamma_k), _ptr(pos), q.shape[0], n_q_heads, n_kv_heads,
                                 head_dim, float(eps), _ptr(cs), max_pos, _ptr(err_flag),
                                 _stream(stream)), "tts_qk_norm_rope")


def tts_kv_set_rows(k, v, k_cache, v_cache, desc: TtsKvDesc, dst_pos, err_flag=None, stream=None):
    assert k.stride(0) == v.stride(0), "k and v rows must share one stride"
    _check(_lib.tts_kv_set_rows(_ptr(k), _ptr(v), _row_stride(k), _ptr(k_cache), _ptr(v_cache),
                                ctypes.byref(desc), _ptr(dst_pos), _ptr(err_flag),
                                _stream(stream)), "tts_kv_set_rows")


def tts_decode_attn_workspace_size(desc: TtsKvDesc, n_splits=0) -> int:
    return int(_lib.tts_decode_attn_workspace_size(ctypes.byref(desc), n_splits))


def tts_decode_attn_default_splits(desc: TtsKvDesc) -> int:
    return int(_lib.tts_decode_attn_default_splits(ctypes.byref(desc)))


def tts_workspace_init(ws, stream=None):
    _check(_lib.tts_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "tts_workspace_init")


def workspace(desc: TtsKvDesc, n_splits=0, device="cuda", stream=None):
    """Allocate (through torch) and clear a workspace for desc/n_splits."""
    n = max(tts_decode_attn_workspace_size(desc, n_splits), 256)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    tts_workspace_init(ws, stream)
    return ws


def tts_decode_attn(q, k_cache, v_cache, desc: TtsKvDesc, n_valid, scale, out, ws, n_splits=0,
                    err_flag=None, stream=None):
    _check(_lib.tts_decode_attn(_ptr(q), _row_stride(q), _ptr(k_cache), _ptr(v_cache),
                                ctypes.byref(desc), _ptr(n_valid), float(scale), _ptr(out),
                                _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                n_splits, _ptr(err_flag), _stream(stream)), "tts_decode_attn")


def tts_decode_step(q, k, v, gamma_q, gamma_k, eps, cs, max_pos, k_cache, v_cache,
                    desc: TtsKvDesc, cur_len, scale, out, ws, n_splits=0, err_flag=None,
                    stream=None):
    stride = _row_stride(q)
    assert k.stride(0) == stride and v.stride(0) == stride, "q, k, v rows must share one stride"
    _check(_lib.tts_decode_step(_ptr(q), _ptr(k), _ptr(v), stride, _ptr(gamma_q), _ptr(gamma_k),
                                float(eps), _ptr(cs), max_pos, _ptr(k_cache), _ptr(v_cache),
                                ctypes.byref(desc), _ptr(cur_len), float(scale), _ptr(out),
                                _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                n_splits, _ptr(err_flag), _stream(stream)), "tts_decode_step")


def tts_decode_step_noalloc(q, k, v, gamma_q, gamma_k, eps, cs, max_pos, k_cache, v_cache,
                            desc: TtsKvDesc, cur_len, scale, out, n_splits=0, err_flag=None,
                            stream=None):
    """tts_decode_step with the library's built-in scratch instead of a workspace (for
    callers that cannot allocate device memory); see include/tts_decode.h."""
    stride = _row_stride(q)
    assert k.stride(0) == stride and v.stride(0) == stride, "q, k, v rows must share one stride"
    _check(_lib.tts_decode_step_noalloc(_ptr(q), _ptr(k), _ptr(v), stride, _ptr(gamma_q),
                                        _ptr(gamma_k), float(eps), _ptr(cs), max_pos,
                                        _ptr(k_cache), _ptr(v_cache), ctypes.byref(desc),
                                        _ptr(cur_len), float(scale), _ptr(out), n_splits,
                                        _ptr(err_flag), _stream(stream)), "tts_decode_step_noalloc")


def tts_prefill_workspace_size(desc: TtsKvDesc, T: int, n_splits=0) -> int:
    return int(_lib.tts_prefill_workspace_size(ctypes.byref(desc), T, n_splits))


def tts_prefill_launch_count(desc: TtsKvDesc, T: int, n_splits=0) -> int:
    return int(_lib.tts_prefill_launch_count(ctypes.byref(desc), T, n_splits))


def prefill_workspace(desc: TtsKvDesc, T: int, n_splits=0, device="cuda", stream=None):
    """Allocate (through torch) and clear a workspace for a prefill of T positions."""
    n = max(tts_prefill_workspace_size(desc, T, n_splits), 256)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    tts_workspace_init(ws, stream)
    return ws


def tts_prefill_step(q, k, v, gamma_q, gamma_k, eps, cs, max_pos, k_cache, v_cache,
                     desc: TtsKvDesc, start_pos, T, scale, out, ws, n_splits=0, err_flag=None,
                     stream=None):
    """q, k, v: [B*T, ...] row views (row r = b*T + t), read only."""
    stride = _row_stride(q)
    assert k.stride(0) == stride and v.stride(0) == stride, "q, k, v rows must share one stride"
    _check(_lib.tts_prefill_step(_ptr(q), _ptr(k), _ptr(v), stride, _ptr(gamma_q), _ptr(gamma_k),
                                 float(eps), _ptr(cs), max_pos, _ptr(k_cache), _ptr(v_cache),
                                 ctypes.byref(desc), _ptr(start_pos), int(T), float(scale),
                                 _ptr(out), _ptr(ws),
                                 0 if ws is None else ws.numel() * ws.element_size(),
                                 n_splits, _ptr(err_flag), _stream(stream)), "tts_prefill_step")


def tts_sample(logits, top_k, temperature, seed, counter, out_ids, draw=0, stream=None):
    """logits [B, V] f32 (rows may be strided); out_ids: int32 tensor whose first dim
    indexes streams (a column view of an ids buffer is fine); draw: the third Philox
    counter word (e.g. the sub-step within a frame)."""
    B, V = logits.shape
    _check(_lib.tts_sample(_ptr(logits), logits.stride(0), B, V, int(top_k), float(temperature),
                           ctypes.c_uint64(int(seed) & ((1 << 64) - 1)), _ptr(counter),
                           ctypes.c_uint32(int(draw)), _ptr(out_ids), out_ids.stride(0),
                           _stream(stream)), "tts_sample")


def tts_sample_embed(logits, top_k, temperature, seed, counter, out_ids, table, out_rows, draw=0,
                     stream=None):
    """tts_sample, then the drawn tokens' rows of one table into out_rows [B, hidden] f32,
    in one launch; table: a TtsTables of one table or a list of one tensor."""
    B, V = logits.shape
    t = tables(table) if not isinstance(table, TtsTables) else table
    _check(_lib.tts_sample_embed(_ptr(logits), logits.stride(0), B, V, int(top_k), float(temperature),
                                 ctypes.c_uint64(int(seed) & ((1 << 64) - 1)), _ptr(counter),
                                 ctypes.c_uint32(int(draw)), _ptr(out_ids), out_ids.stride(0),
                                 ctypes.byref(t), _ptr(out_rows), _stream(stream)), "tts_sample_embed")


def tts_counter_advance(counter, by=1, stream=None):
    _check(_lib.tts_counter_advance(_ptr(counter), ctypes.c_uint64(int(by)), _stream(stream)),
           "tts_counter_advance")


def tts_check_wait_timeout(err_flag, stream=None):
    """One bounded wait that nothing ends: sets TTS_EFLAG_TIMEOUT in err_flag after about
    a second."""
    _check(_lib.tts_check_wait_timeout(_ptr(err_flag), _stream(stream)), "tts_check_wait_timeout")


def layer_weights(w_qkv, w_o, w_gu, w_down, gamma_attn, gamma_mlp, gamma_q, gamma_k) -> TtsLayerWeights:
    """Descriptor of one layer's weights: bf16 matrices, f32 norm weights (device tensors;
    the caller keeps them alive)."""
    for m in (w_qkv, w_o, w_gu, w_down):
        if m.dtype != torch.bfloat16 or not m.is_contiguous():
            raise ValueError("layer weight matrices must be contiguous bfloat16")
    t = TtsLayerWeights()
    t.w_qkv, t.w_o, t.w_gu, t.w_down = (m.data_ptr() for m in (w_qkv, w_o, w_gu, w_down))
    t.gamma_attn, t.gamma_mlp, t.gamma_q, t.gamma_k = (
        g.data_ptr() for g in (gamma_attn, gamma_mlp, gamma_q, gamma_k))
    t.hidden = w_qkv.shape[1]
    t.inter = w_down.shape[1]
    return t


def tts_decode_layer_launch_count(desc: TtsKvDesc) -> int:
    return int(_lib.tts_decode_layer_launch_count(ctypes.byref(desc)))


def tts_decode_layer_scratch_size(desc: TtsKvDesc, hidden, inter, n_splits=0) -> int:
    return int(_lib.tts_decode_layer_scratch_size(ctypes.byref(desc), hidden, inter, n_splits))


def layer_scratch(desc: TtsKvDesc, hidden, inter, n_splits=0, device="cuda", stream=None):
    """Allocate (through torch) and clear the scratch of a decode layer."""
    n = max(tts_decode_layer_scratch_size(desc, hidden, inter, n_splits), 256)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    tts_workspace_init(ws, stream)
    return ws


def tts_decode_layer(h, weights: TtsLayerWeights, eps, cs, max_pos, k_cache, v_cache,
                     desc: TtsKvDesc, cur_len, scale, scratch, n_splits=0, err_flag=None,
                     stream=None):
    _check(_lib.tts_decode_layer(_ptr(h), ctypes.byref(weights), float(eps), _ptr(cs), max_pos,
                                 _ptr(k_cache), _ptr(v_cache), ctypes.byref(desc), _ptr(cur_len),
                                 float(scale), _ptr(scratch), scratch.numel() * scratch.element_size(),
                                 n_splits, _ptr(err_flag), _stream(stream)), "tts_decode_layer")


# ---------------------------------------------------------------------------
# Drafted decoding over a quantised cache
# ---------------------------------------------------------------------------
_ROW_CODES = {torch.float32: TTS_F32, torch.bfloat16: TTS_BF16}
_KV_TORCH = {TTS_F32: torch.float32, TTS_BF16: torch.bfloat16, TTS_I8: torch.int8,
             TTS_E4M3: torch.float8_e4m3fn}
_ROPE_KINDS = {"none": 0, "linear": 1, "base": 2, "parts": 3}


def _rows(t, what, width=None):
    """Checks a [rows, width] view whose rows are contiguous; returns (dtype code, stride)."""
    code = _ROW_CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be float32 or bfloat16")
    if t.dim() != 2 or t.stride(1) != 1 or (width is not None and t.shape[1] != width):
        raise ValueError(f"{what} must be a 2-d view of contiguous rows"
                         + ("" if width is None else f" of {width} entries"))
    # one row has no stride of its own
    return code, t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _ints(t, what, n, dtype=torch.int32):
    if t is None:
        return   # optional arguments only; the library refuses a missing required one
    if t.dtype != dtype or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of {n} entries")


def _p(t):
    """A tensor's address as a plain int (ctypes converts it), None for None."""
    return None if t is None else t.data_ptr()


def _on_device(stream, first, *others):
    """Every tensor on first's device, and that device the current one (launches go there);
    returns the stream's handle (default: the current one)."""
    d = first.get_device()
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError("all tensors must be on one device")
    if d < 0 or d != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on {first.device}, which is not the current CUDA device")
    return torch._C._cuda_getCurrentRawStream(d) if stream is None else stream.cuda_stream


def kv_cache(k, v, k_scale=None, v_scale=None) -> TtsKvCache:
    """A layer's cache: K and V tensors (float32, bfloat16, or 8-bit codes as int8 or
    float8_e4m3fn), and for 8-bit codes the float32 scales of their rows (the shape of K
    without its last dimension).  The caller keeps them alive."""
    scaled = k.dtype in (torch.int8, torch.float8_e4m3fn)
    if k.dtype not in _KV_TORCH.values() or v.dtype != k.dtype or v.shape != k.shape or \
            not k.is_contiguous() or not v.is_contiguous():
        raise ValueError("K and V must be contiguous tensors of one cache dtype and shape")
    for s in (k_scale, v_scale):
        if scaled != (s is not None):
            raise ValueError("8-bit caches, and only they, take k_scale and v_scale")
        if scaled and (s.dtype != torch.float32 or s.shape != k.shape[:-1] or not s.is_contiguous()):
            raise ValueError("scales must be contiguous float32, one per cache row")
    for t in (v, k_scale, v_scale):
        if t is not None and t.device != k.device:
            raise ValueError("K, V and their scales must be on one device")
    c = TtsKvCache(k.data_ptr(), v.data_ptr(), None if k_scale is None else k_scale.data_ptr(),
                   None if v_scale is None else v_scale.data_ptr())
    c.dtype, c.shape, c.device_index = k.dtype, tuple(k.shape), k.get_device()
    return c


def _cache_fits(cache: TtsKvCache, desc: TtsKvDesc):
    """The tensors behind `cache` are what `desc` says (the library only sees pointers)."""
    rows = ((desc.n_pages, desc.n_kv_heads, desc.page_size, desc.head_dim) if desc.paged
            else (desc.B, desc.n_kv_heads, desc.capacity, desc.head_dim))
    if cache.dtype != _KV_TORCH.get(desc.kv_dtype) or cache.shape != rows:
        raise ValueError(f"the descriptor's cache is {_KV_TORCH.get(desc.kv_dtype)} {rows}, "
                         f"the tensors are {cache.dtype} {cache.shape}")
    if getattr(desc, "table_device", None) not in (None, cache.device_index):
        raise ValueError("the block table and the cache must be on one device")


def tts_rope_table_scaled(cs, max_pos, rot_dim, base, kind="none", factor=1.0, original_max_pos=1,
                          low_rotations=1.0, high_rotations=32.0, attn_scale=1.0, stream=None):
    """A (cos, sin) table cs [max_pos, rot_dim / 2, 2] for a longer window: kind "none",
    "linear", "base" or "parts" (include/tts_decode.h states the formulas)."""
    if kind not in _ROPE_KINDS:
        raise ValueError(f"kind must be one of {sorted(_ROPE_KINDS)}")
    if cs.dtype != torch.float32 or not cs.is_contiguous() or cs.numel() < max_pos * rot_dim:
        raise ValueError("cs must be contiguous float32 of max_pos * rot_dim entries")
    st = _on_device(stream, cs)
    s = TtsRopeScaling(_ROPE_KINDS[kind], original_max_pos, float(factor), float(low_rotations),
                       float(high_rotations), float(attn_scale))
    _check(_lib.tts_rope_table_scaled(_p(cs), max_pos, rot_dim, float(base), ctypes.byref(s), st),
           "tts_rope_table_scaled")


def tts_rope_rows(q, k, q_out, k_out, pos, n_q_heads, n_kv_heads, head_dim, cs, gamma_q=None,
                  gamma_k=None, eps=1e-6, interleaved=False, err_flag=None, stream=None):
    """q [rows, n_q_heads * head_dim] and k (or None) rotated into q_out and k_out at pos
    [rows]; cs [max_pos, rot_dim / 2, 2] sets how much of each head turns.  Rows may be
    strided views; float32 or bfloat16 in and out; q_out and k_out may be q and k."""
    if k is None:
        n_kv_heads, k_out = 0, None
    qd, kd = n_q_heads * head_dim, n_kv_heads * head_dim
    dt, qs = _rows(q, "q", qd)
    odt, qos = _rows(q_out, "q_out", qd)
    ks = kos = 0
    n = q.shape[0]
    if k is not None:
        kdt, ks = _rows(k, "k", kd)
        kodt, kos = _rows(k_out, "k_out", kd)
        if kdt != dt or kodt != odt or k.shape[0] != n or k_out.shape[0] != n:
            raise ValueError("q and k must be of one dtype and row count, and so their outputs")
    if q_out.shape[0] != n:
        raise ValueError("q_out must have q's rows")
    _ints(pos, "pos", n)
    for gm in (gamma_q, gamma_k):
        if gm is not None:
            _ints(gm, "gamma", head_dim, torch.float32)
    if cs.dim() != 3 or cs.dtype != torch.float32 or not cs.is_contiguous() or cs.shape[2] != 2:
        raise ValueError("cs must be a contiguous float32 [max_pos, rot_dim / 2, 2] table")
    _ints(err_flag, "err_flag", 1)
    st = _on_device(stream, q, k, q_out, k_out, pos, cs, gamma_q, gamma_k, err_flag)
    _check(_lib.tts_rope_rows(_p(q), qs, _p(k), ks, dt, _p(q_out), qos, _p(k_out), kos, odt,
                              _p(gamma_q), _p(gamma_k), float(eps), _p(pos), n, n_q_heads,
                              n_kv_heads, head_dim, 2 * cs.shape[1], int(bool(interleaved)), _p(cs),
                              cs.shape[0], _p(err_flag), st), "tts_rope_rows")


def tts_kv_write_rows(k, v, cache: TtsKvCache, desc: TtsKvDesc, start_pos, T, n_rows=None,
                      err_flag=None, stream=None):
    """k, v [B * T, n_kv_heads * head_dim] (row b * T + t) into the cache at start_pos[b] + t,
    quantised to its dtype; n_rows [B]: only the first n_rows[b] of stream b."""
    kd = desc.n_kv_heads * desc.head_dim
    dt, ks = _rows(k, "k", kd)
    vdt, vs = _rows(v, "v", kd)
    if vdt != dt or vs != ks or k.shape[0] != desc.B * T or v.shape[0] != desc.B * T:
        raise ValueError("k and v must share dtype and stride and hold B * T rows")
    _cache_fits(cache, desc)
    _ints(start_pos, "start_pos", desc.B)
    _ints(n_rows, "n_rows", desc.B)
    _ints(err_flag, "err_flag", 1)
    st = _on_device(stream, k, v, cache, start_pos, n_rows, err_flag)
    _check(_lib.tts_kv_write_rows(_p(k), _p(v), dt, ks, ctypes.byref(cache), ctypes.byref(desc),
                                  _p(start_pos), _p(n_rows), T, _p(err_flag), st), "tts_kv_write_rows")


def tts_kv_read_rows(cache: TtsKvCache, desc: TtsKvDesc, start_pos, T, k_out, v_out, n_rows=None,
                     err_flag=None, stream=None):
    """Cache rows start_pos[b] + t, t < min(T, n_rows[b]), as values into rows b * T + t of
    k_out and v_out [B * T, n_kv_heads * head_dim]; other rows are left as they were."""
    kd = desc.n_kv_heads * desc.head_dim
    dt, ks = _rows(k_out, "k_out", kd)
    vdt, vs = _rows(v_out, "v_out", kd)
    if vdt != dt or vs != ks or k_out.shape[0] != desc.B * T or v_out.shape[0] != desc.B * T:
        raise ValueError("k_out and v_out must share dtype and stride and hold B * T rows")
    _cache_fits(cache, desc)
    _ints(start_pos, "start_pos", desc.B)
    _ints(n_rows, "n_rows", desc.B)
    _ints(err_flag, "err_flag", 1)
    st = _on_device(stream, k_out, v_out, cache, start_pos, n_rows, err_flag)
    _check(_lib.tts_kv_read_rows(ctypes.byref(cache), ctypes.byref(desc), _p(start_pos), _p(n_rows), T,
                                 _p(k_out), _p(v_out), dt, ks, _p(err_flag), st), "tts_kv_read_rows")


def _row_code(q_dtype):
    code = {"f32": TTS_F32, "bf16": TTS_BF16}.get(q_dtype, _ROW_CODES.get(q_dtype))
    if code is None:
        raise ValueError("q_dtype must be \"f32\", \"bf16\" or the torch dtype")
    return code


def tts_tree_attn_workspace_size(desc: TtsKvDesc, T: int, q_dtype="f32") -> int:
    return int(_lib.tts_tree_attn_workspace_size(ctypes.byref(desc), T, _row_code(q_dtype)))


def tree_workspace(desc: TtsKvDesc, T: int, q_dtype="f32", device="cuda"):
    """Allocate (through torch) a workspace for trees of up to T nodes."""
    n = max(tts_tree_attn_workspace_size(desc, t, q_dtype) for t in range(1, T + 1))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def tts_tree_attn(q, cache: TtsKvCache, desc: TtsKvDesc, n_past, T, scale, out, ws, n_nodes=None,
                  tree_mask=None, err_flag=None, stream=None):
    """Attention of T drafted nodes a stream: q [B * T, n_q_heads * head_dim] (float32 or
    bfloat16), out dense of q's dtype, tree_mask int64 [B, T] (bit u: node t sees node u; None:
    the chain), n_nodes [B] (None: T each).  T = 1 without a mask decodes one token."""
    dt, qs = _rows(q, "q", desc.n_q_heads * desc.head_dim)
    if q.shape[0] != desc.B * T:
        raise ValueError("q must hold B * T rows")
    if out.dtype != q.dtype or out.numel() != q.shape[0] * q.shape[1] or not out.is_contiguous():
        raise ValueError("out must be contiguous, of q's dtype and size")
    _cache_fits(cache, desc)
    _ints(n_past, "n_past", desc.B)
    _ints(n_nodes, "n_nodes", desc.B)
    _ints(tree_mask, "tree_mask", desc.B * T, torch.int64)
    if ws is not None and not ws.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    _ints(err_flag, "err_flag", 1)
    st = _on_device(stream, q, cache, n_past, n_nodes, tree_mask, out, ws, err_flag)
    _check(_lib.tts_tree_attn(_p(q), dt, qs, ctypes.byref(cache), ctypes.byref(desc), _p(n_past),
                              _p(n_nodes), _p(tree_mask), T, float(scale), _p(out), _p(ws),
                              0 if ws is None else ws.numel() * ws.element_size(), _p(err_flag), st),
           "tts_tree_attn")


def tts_tree_commit(cache: TtsKvCache, desc: TtsKvDesc, n_past, path, n_accept, T, err_flag=None,
                    stream=None):
    """The accepted path's rows to the front of the tree's: path [B, T] int32 (rows may be
    strided), its first n_accept[b] entries strictly ascending node indices."""
    if path.dtype != torch.int32 or path.dim() != 2 or path.shape != (desc.B, T) or path.stride(1) != 1:
        raise ValueError("path must be an int32 [B, T] view of contiguous rows")
    _cache_fits(cache, desc)
    _ints(n_past, "n_past", desc.B)
    _ints(n_accept, "n_accept", desc.B)
    _ints(err_flag, "err_flag", 1)
    st = _on_device(stream, path, cache, n_past, n_accept, err_flag)
    _check(_lib.tts_tree_commit(ctypes.byref(cache), ctypes.byref(desc), _p(n_past), _p(path),
                                path.stride(0) if desc.B > 1 else T, _p(n_accept), T, _p(err_flag), st),
           "tts_tree_commit")


# ---------------------------------------------------------------------------
# One step of many requests
# ---------------------------------------------------------------------------
_ROW8_CODES = {torch.float32: TTS_F32, torch.bfloat16: TTS_BF16, torch.float8_e4m3fn: TTS_E4M3}
_X_CODES = {"bf16": TTS_BF16, "e4m3": TTS_E4M3, torch.bfloat16: TTS_BF16, torch.float8_e4m3fn: TTS_E4M3}


def _rows_of(t, what, codes, shape):
    """Checks a view of `shape` whose rows are contiguous; returns (dtype code, stride)."""
    code = codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be one of {', '.join(str(c) for c in codes if not isinstance(c, str))}")
    if t.shape != shape or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be a [{shape[0]}, {shape[1]}] view of contiguous rows")
    # one row has no stride of its own: any that keeps it aligned
    return code, t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // 16) * 16


def tts_add_rms_norm(x, residual, sum_out, gamma, eps, out, out_scale=None, stream=None):
    """residual + x into sum_out (None: not stored; may be residual), and the RMS norm of that sum
    times gamma into out, [rows, n] each: x, residual and sum_out float32 or bfloat16, out
    float32, bfloat16 or float8_e4m3fn with out_scale [rows].  residual None: the norm of x."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, n]")
    n, width = x.shape
    dt, xs = _rows_of(x, "x", _ROW_CODES, x.shape)
    odt, os_ = _rows_of(out, "out", _ROW8_CODES, x.shape)
    rdt = rs = ss = 0
    if residual is not None:
        rdt, rs = _rows_of(residual, "residual", _ROW_CODES, x.shape)
        if sum_out is not None:
            sdt, ss = _rows_of(sum_out, "sum_out", _ROW_CODES, x.shape)
            if sdt != rdt:
                raise ValueError("sum_out must be of residual's dtype")
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    if (odt == TTS_E4M3) != (out_scale is not None):
        raise ValueError("float8_e4m3fn outputs, and only they, take out_scale")
    _ints(gamma, "gamma", width, torch.float32)
    _ints(out_scale, "out_scale", n, torch.float32)
    st = _on_device(stream, x, residual, sum_out, gamma, out, out_scale)
    _check(_lib.tts_add_rms_norm(_p(x), xs, dt, _p(residual), rs, rdt, _p(sum_out), ss, _p(gamma), float(eps), n, width,
                                 _p(out), os_, odt, _p(out_scale), st), "tts_add_rms_norm")


def adapters(a, b, rank=None, scale=None) -> TtsAdapters:
    """A pool of low-rank adapters of a projection [n, k]: a [adapters, rank_max, k] and b
    [adapters, n, rank_max], bfloat16; rank int32 and scale float32 [adapters] (None: rank_max and
    1 each).  The caller keeps the tensors alive."""
    for t in (a, b):
        if t.dtype != torch.bfloat16 or t.dim() != 3 or not t.is_contiguous():
            raise ValueError("a and b must be contiguous bfloat16 of three dimensions")
    if a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
        raise ValueError("a is [adapters, rank_max, k], b [adapters, n, rank_max]")
    _ints(rank, "rank", a.shape[0])
    _ints(scale, "scale", a.shape[0], torch.float32)
    for t in (b, rank, scale):
        if t is not None and t.device != a.device:
            raise ValueError("the adapters' tensors must be on one device")
    p = TtsAdapters(a.data_ptr(), b.data_ptr(), _p(rank), _p(scale), a.shape[0], a.shape[1])
    p.n, p.k, p.device_index = b.shape[1], a.shape[2], a.get_device()
    return p


def tts_project_workspace_size(rows, n, k, x_dtype, adapters=None) -> int:
    if x_dtype not in _X_CODES:
        raise ValueError("x_dtype must be \"bf16\", \"e4m3\" or the torch dtype")
    ad = None if adapters is None else ctypes.byref(adapters)
    return int(_lib.tts_project_workspace_size(rows, n, k, _X_CODES[x_dtype], ad))


def project_workspace(rows, n, k, x_dtype, adapters=None, device="cuda"):
    """Allocate (through torch) a workspace for projections of up to `rows` rows."""
    return torch.empty(max(tts_project_workspace_size(rows, n, k, x_dtype, adapters), 256), dtype=torch.uint8,
                       device=device)


def tts_project_rows(x, w, out, ws, x_scale=None, w_scale=None, adapters=None, stream_adapter=None,
                     row_stream=None, err_flag=None, stream=None):
    """out [rows, n] = x [rows, k] times w [n, k] transposed, and to each row its request's
    adapter: row r is of request row_stream[r] (None: r; negative: the row is left as it was),
    which has adapter stream_adapter[request] (negative: none).  x and w bfloat16, or
    float8_e4m3fn with x_scale [rows] and w_scale [n]; out float32 or bfloat16."""
    if x.dim() != 2 or w.dim() != 2 or not w.is_contiguous() or w.dtype != x.dtype or w.shape[1] != x.shape[1]:
        raise ValueError("x is [rows, k], w contiguous [n, k], of one dtype")
    rows, k = x.shape
    n = w.shape[0]
    dt, xs = _rows_of(x, "x", _X_CODES, x.shape)
    odt, os_ = _rows_of(out, "out", _ROW_CODES, (rows, n))
    if (dt == TTS_E4M3) != (x_scale is not None) or (dt == TTS_E4M3) != (w_scale is not None):
        raise ValueError("float8_e4m3fn rows and weights, and only they, take x_scale and w_scale")
    _ints(x_scale, "x_scale", rows, torch.float32)
    _ints(w_scale, "w_scale", n, torch.float32)
    _ints(row_stream, "row_stream", rows)
    n_streams = 0
    if adapters is not None:
        if adapters.n != n or adapters.k != k:
            raise ValueError("the adapters are of another projection")
        if stream_adapter is None:
            raise ValueError("adapters need stream_adapter")
        _ints(stream_adapter, "stream_adapter", rows if row_stream is None else 1)
        n_streams = stream_adapter.numel()
    if ws is not None and not ws.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    _ints(err_flag, "err_flag", 1)
    st = _on_device(stream, x, w, out, ws, x_scale, w_scale, adapters, stream_adapter, row_stream, err_flag)
    _check(_lib.tts_project_rows(_p(x), xs, dt, _p(x_scale), _p(w), _p(w_scale), n, k,
                                 None if adapters is None else ctypes.byref(adapters), _p(row_stream),
                                 _p(stream_adapter), n_streams, rows, _p(out), os_, odt, _p(ws),
                                 0 if ws is None else ws.numel() * ws.element_size(), _p(err_flag), st),
           "tts_project_rows")


def tts_page_plan(desc: TtsKvDesc, block_table, free_pages, n_free, n_past, n_new, n_rows, row_start, row_stream,
                  row_pos, row_slot, T=0, err_flag=None, stream=None):
    """Pages and row maps of a step: block_table (desc's own, updated), free_pages [n_pages] and
    n_free [1] (updated), n_past and n_new [B]; n_rows [B], row_start [B + 1], and row_stream,
    row_pos and row_slot (int64) of max_rows = row_stream's entries each.  T 0: packed rows,
    else T rows a stream (include/tts_decode.h states the rules)."""
    if not desc.paged or block_table.data_ptr() != desc.block_table:
        raise ValueError("block_table must be the descriptor's own, of a paged cache")
    for t, what, n in ((free_pages, "free_pages", desc.n_pages), (n_free, "n_free", 1), (n_past, "n_past", desc.B),
                       (n_new, "n_new", desc.B), (n_rows, "n_rows", desc.B), (row_start, "row_start", desc.B + 1)):
        _ints(t, what, n)
    max_rows = row_stream.numel()
    _ints(row_stream, "row_stream", max_rows)
    _ints(row_pos, "row_pos", max_rows)
    _ints(row_slot, "row_slot", max_rows, torch.int64)
    _ints(err_flag, "err_flag", 1)
    st = _on_device(stream, block_table, free_pages, n_free, n_past, n_new, n_rows, row_start, row_stream, row_pos,
                    row_slot, err_flag)
    _check(_lib.tts_page_plan(ctypes.byref(desc), _p(block_table), _p(free_pages), _p(n_free), _p(n_past), _p(n_new), T,
                              max_rows, _p(n_rows), _p(row_start), _p(row_stream), _p(row_pos), _p(row_slot),
                              _p(err_flag), st), "tts_page_plan")


def tts_kv_write_slots(k, v, cache: TtsKvCache, desc: TtsKvDesc, row_slot, err_flag=None, stream=None):
    """k, v [rows, n_kv_heads * head_dim] into the cache at row_slot [rows] (int64; negative: the
    row is skipped), converted or quantised as by tts_kv_write_rows."""
    kd = desc.n_kv_heads * desc.head_dim
    dt, ks = _rows(k, "k", kd)
    vdt, vs = _rows(v, "v", kd)
    if vdt != dt or vs != ks or v.shape[0] != k.shape[0]:
        raise ValueError("k and v must share dtype, stride and row count")
    _cache_fits(cache, desc)
    _ints(row_slot, "row_slot", k.shape[0], torch.int64)
    _ints(err_flag, "err_flag", 1)
    st = _on_device(stream, k, v, cache, row_slot, err_flag)
    _check(_lib.tts_kv_write_slots(_p(k), _p(v), dt, ks, ctypes.byref(cache), ctypes.byref(desc), _p(row_slot),
                                   k.shape[0], _p(err_flag), st), "tts_kv_write_slots")


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)
