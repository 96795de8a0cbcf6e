"""ctypes binding of libgk.so: the C ABI of include/gk.h under the same names.

Argument marshalling only.  Device buffers are passed as torch CUDA tensors (or
raw integer addresses); every computation runs in the library's kernels.  A
missing or unloadable library raises at import of the first call, never falls
back to anything else.
"""
from __future__ import annotations

import ctypes
import os
import sys
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# GK_LIB_PATH selects another build of the same library (the sanitizer build in the tests)
LIB_PATH = os.environ.get("GK_LIB_PATH") or os.path.join(_HERE, "libgk.so")

GK_OK = 0
GK_ERR_INVALID = 1
GK_ERR_OOM = 2
GK_ERR_HOT_FULL = 3
GK_ERR_CUDA = 4
GK_ERR_DEVICE_BOUNDS = 5
GK_ERR_TIMEOUT = 6
GK_ERR_UNSUPPORTED = 7
GK_BACKEND_DENSE = 0
GK_BACKEND_CASCADE = 1

c_i32, c_i64, c_u64, c_dbl, c_vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_double, ctypes.c_void_p


class GkError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"gk status {status}: {message}")
        self.status = status


class gk_pool_config(ctypes.Structure):
    _fields_ = [("num_layers", c_i32), ("num_q_heads", c_i32), ("num_kv_heads", c_i32), ("head_dim", c_i32),
                ("hot_tokens", c_i64), ("cold_slots", c_i64), ("cold_page_size", c_i32), ("reserved0", c_i32),
                ("seed", c_u64), ("hot_k", c_vp), ("hot_v", c_vp), ("cold_k", c_vp), ("cold_v", c_vp)]


class gk_batch(ctypes.Structure):
    _fields_ = [("num_requests", c_i32), ("max_blocks", c_i32),
                ("prefix_hot_base", ctypes.POINTER(c_i64)), ("prefix_len", ctypes.POINTER(c_i32)),
                ("suffix_len", ctypes.POINTER(c_i32)), ("d_block_table", c_vp), ("d_q", c_vp),
                ("d_out", c_vp), ("d_lse", c_vp), ("d_new_k", c_vp), ("d_new_v", c_vp)]


class gk_plan_summary(ctypes.Structure):
    _fields_ = [("num_requests", c_i32), ("num_groups", c_i32), ("max_m_eff", c_i32), ("prefix_ctas", c_i32),
                ("suffix_ctas", c_i32), ("dense_ctas", c_i32), ("num_partials", c_i32), ("dense_merge", c_i32),
                ("prefix_bytes", c_i64), ("prefix_flops", c_i64), ("suffix_bytes", c_i64), ("dense_bytes", c_i64),
                ("cascade_split", c_i32), ("prefix_tiles_per_item", c_i32), ("prefix_kernel", c_i32),
                ("prefix_rows_per_item", c_i32), ("prefix_row_groups", c_i32), ("prefix_ctas_gather", c_i32),
                ("sm_slots", c_i32)]


class gk_cost_model(ctypes.Structure):
    _fields_ = [("c_flat_us", c_dbl), ("bw_flat_gbs", c_dbl), ("c_cascade_us", c_dbl), ("bw_prefix_gbs", c_dbl),
                ("bw_suffix_gbs", c_dbl), ("c_merge_us", c_dbl), ("prefix_tile_us", c_dbl), ("prefix_item_us", c_dbl),
                ("gather_sm_gbs", c_dbl), ("c_gather_us", c_dbl), ("prefix_tile_split_us", c_dbl),
                ("warp_tile_us", c_dbl), ("warp_group_us", c_dbl), ("warp_item_us", c_dbl),
                ("warp_split_ratio", c_dbl), ("prefix_cta_ramp_us", c_dbl), ("prefix_cta_gather_ratio", c_dbl),
                ("c_merge_state_us", c_dbl), ("prefix_item_split_us", c_dbl), ("warp_item_split_us", c_dbl),
                ("prefix_item_crowd_us", c_dbl), ("split_gather_ratio_tensor", c_dbl), ("c_gather_split_us", c_dbl),
                ("split_tensor_us", c_dbl)]


class gk_tables(ctypes.Structure):
    _fields_ = [("num_rows", c_i32), ("max_blocks", c_i32), ("capacity", c_i32), ("reserved0", c_i32), ("d_table", c_vp),
                ("d_free", c_vp), ("d_len", c_vp), ("d_len_out", c_vp), ("d_num_free", c_vp), ("d_num_free_out", c_vp),
                ("d_work", c_vp)]


GK_TABLES_WORK_PER_ROW = 32


class gk_prompt_batch(ctypes.Structure):
    _fields_ = [("num_requests", c_i32), ("max_blocks", c_i32), ("new_len", ctypes.POINTER(c_i32)),
                ("prefix_hot_base", ctypes.POINTER(c_i64)), ("prefix_len", ctypes.POINTER(c_i32)),
                ("context_len", ctypes.POINTER(c_i32)), ("d_block_table", c_vp), ("d_q", c_vp), ("d_k", c_vp),
                ("d_v", c_vp), ("d_out", c_vp), ("d_lse", c_vp), ("q_stride", c_i64), ("k_stride", c_i64),
                ("v_stride", c_i64), ("out_stride", c_i64)]


class gk_prompt_plan_summary(ctypes.Structure):
    _fields_ = [("tokens", c_i64), ("flops", c_i64), ("bytes", c_i64), ("items", c_i32), ("ctas", c_i32),
                ("stacked_requests", c_i32), ("partials", c_i32), ("max_pieces", c_i32), ("max_cta_tiles", c_i32),
                ("scratch_bytes", c_i64)]


class gk_qkv(ctypes.Structure):
    _fields_ = [("num_tokens", c_i32), ("rot_dim", c_i32), ("interleaved", c_i32), ("eps", ctypes.c_float), ("num_positions", c_i64),
                ("d_cos_sin", c_vp), ("d_positions", c_vp), ("d_q_weight", c_vp), ("d_k_weight", c_vp), ("d_q", c_vp), ("d_k", c_vp),
                ("d_v", c_vp), ("d_q_out", c_vp), ("d_k_out", c_vp), ("q_stride", c_i64), ("k_stride", c_i64), ("v_stride", c_i64),
                ("q_out_stride", c_i64), ("k_out_stride", c_i64)]


P = ctypes.POINTER
_SIGS = {
    "gk_pool_create": (c_i32, [P(gk_pool_config), P(c_vp)]),
    "gk_pool_create_kv4": (c_i32, [P(gk_pool_config), P(c_vp)]),
    "gk_kv4_row_bytes": (c_i64, [c_i32, c_i32]),
    "gk_pool_destroy": (None, [c_vp]),
    "gk_last_error": (ctypes.c_char_p, [c_vp]),
    "gk_status_string": (ctypes.c_char_p, [c_i32]),
    "gk_prefix_alloc": (c_i32, [c_vp, c_i64, P(c_i64)]),
    "gk_prefix_release": (c_i32, [c_vp, c_i64]),
    "gk_hot_stats": (c_i32, [c_vp, P(c_i64), P(c_i64), P(c_i64)]),
    "gk_prefix_acquire": (c_i32, [c_vp, c_u64, c_i64, P(c_i64), P(c_i32)]),
    "gk_prefix_unref": (c_i32, [c_vp, c_u64]),
    "gk_hot_cache_stats": (c_i32, [c_vp, P(c_i64), P(c_i64), P(c_i64)]),
    "gk_seq_create_cached": (c_i32, [c_vp, c_i32, c_vp, P(c_i32), P(c_i64)]),
    "gk_seq_cache_blocks": (c_i32, [c_vp, c_i32, c_i32, c_vp, P(c_i32)]),
    "gk_cold_cache_stats": (c_i32, [c_vp, P(c_i64), P(c_i64)]),
    "gk_seq_create": (c_i32, [c_vp, P(c_i32)]),
    "gk_seq_fork": (c_i32, [c_vp, c_i32, P(c_i32)]),
    "gk_seq_release": (c_i32, [c_vp, c_i32]),
    "gk_seq_table": (c_i32, [c_vp, c_i32, P(P(c_i32)), P(c_i32), P(c_i64)]),
    "gk_seq_append_slots": (c_i32, [c_vp, c_i32, P(c_i32), P(c_i64), P(c_i32), P(c_i32), P(c_i32)]),
    "gk_seq_tables": (c_i32, [c_vp, c_i32, P(c_i32), c_i32, P(c_i32), P(c_i32)]),
    "gk_cold_stats": (c_i32, [c_vp, P(c_i64), P(c_i64)]),
    "gk_block_refcount": (c_i32, [c_vp, c_i32, P(c_i32)]),
    "gk_append_kv": (c_i32, [c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_i32, c_vp]),
    "gk_write_prefix_kv": (c_i32, [c_vp, c_vp, c_i32, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp]),
    "gk_qk_norm_rope": (c_i32, [c_vp, c_vp, P(gk_qkv)]),
    "gk_append_qkv": (c_i32, [c_vp, c_vp, c_i32, P(gk_qkv), c_vp, c_i32, c_vp]),
    "gk_read_kv": (c_i32, [c_vp, c_vp, c_i32, c_i64, c_vp, c_vp, c_vp, c_i64, c_i64]),
    "gk_decode_kv4": (c_i32, [c_vp, c_vp, c_i32, P(gk_batch), c_vp, c_vp]),
    "gk_plan_build": (c_i32, [c_vp, P(gk_batch), c_vp, P(c_vp)]),
    "gk_plan_update": (c_i32, [c_vp, P(gk_batch), c_vp]),
    "gk_plan_destroy": (None, [c_vp]),
    "gk_plan_info": (c_i32, [c_vp, P(gk_plan_summary)]),
    "gk_plan_segments": (c_i32, [c_vp, c_i32, P(c_i32), P(c_i32), c_vp, c_vp]),
    "gk_decode_dense": (c_i32, [c_vp, c_vp, c_i32, P(gk_batch), c_vp]),
    "gk_decode_cascade": (c_i32, [c_vp, c_vp, c_i32, P(gk_batch), c_vp]),
    "gk_decode_dense_static": (c_i32, [c_vp, c_vp, c_i32, P(gk_batch)]),
    "gk_cascade_levels": (c_i32, [c_vp, c_vp, c_i32, P(gk_batch), c_vp]),
    "gk_cascade_prefix": (c_i32, [c_vp, c_vp, c_i32, P(gk_batch), c_vp]),
    "gk_cascade_suffix": (c_i32, [c_vp, c_vp, c_i32, P(gk_batch), c_vp]),
    "gk_cascade_merge": (c_i32, [c_vp, c_vp, c_i32, P(gk_batch), c_vp]),
    "gk_tables_step": (c_i32, [c_vp, c_vp, P(gk_tables), c_vp, c_vp, c_i64, c_vp, c_vp]),
    "gk_prompt_plan_build": (c_i32, [c_vp, P(gk_prompt_batch), c_vp, P(c_vp)]),
    "gk_prompt_plan_update": (c_i32, [c_vp, P(gk_prompt_batch), c_vp]),
    "gk_prompt_plan_destroy": (None, [c_vp]),
    "gk_prompt_plan_info": (c_i32, [c_vp, P(gk_prompt_plan_summary)]),
    "gk_prompt_plan_items": (c_i32, [c_vp, P(c_i32), P(c_i32), c_vp, c_vp]),
    "gk_prompt_attn": (c_i32, [c_vp, c_vp, c_i32, P(gk_prompt_batch), c_vp]),
    "gk_dispatch": (c_i32, [c_vp, c_vp, P(c_i32), P(c_dbl), P(c_dbl)]),
    "gk_cost_model_set": (c_i32, [c_vp, P(gk_cost_model)]),
    "gk_cost_model_get": (c_i32, [c_vp, P(gk_cost_model)]),
    "gk_cost_model_load": (c_i32, [c_vp, ctypes.c_char_p]),
    "gk_pool_set_cascade_mode": (c_i32, [c_vp, c_i32, c_i32]),
    "gk_pool_set_gather_partition": (c_i32, [c_vp, c_i32]),
    "gk_pool_set_prefix_kernel": (c_i32, [c_vp, c_i32]),
    "gk_pool_set_sm_speeds": (c_i32, [c_vp, P(ctypes.c_float), c_i32]),
    "gk_pool_get_sm_speeds": (c_i32, [c_vp, P(ctypes.c_float), P(c_i32)]),
    "gk_sm_speeds_measure": (c_i32, [c_vp, c_vp, c_i32, P(gk_batch), c_vp, c_i32, P(ctypes.c_float)]),
    "gk_calibrate": (c_i32, [c_vp, c_vp, ctypes.c_char_p]),
    "gk_device_error": (c_i32, [c_vp, c_vp, P(c_i32)]),
}

_lib = None


def lib():
    """The loaded libgk.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run __graft_entry__.build() (or python paged_kv_cache_pool_gb300/build.py)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(x):
    """Device address of a torch tensor, an int, or None."""
    if x is None or isinstance(x, int):    # first: a failed attribute look-up costs 0.4 us a call
        return x
    return x.data_ptr()


def _stream(s):
    if s is None or isinstance(s, int):
        return s
    return s.cuda_stream


def _check(st, pool=None):
    if st != GK_OK:
        msg = lib().gk_last_error(pool).decode() if pool else ""
        if not msg:
            msg = lib().gk_status_string(st).decode()
        raise GkError(st, msg)


def _i64p(a):
    return a.ctypes.data_as(P(c_i64))


def _i32p(a):
    return a.ctypes.data_as(P(c_i32))


# what the checks of tensors need to know: (query heads, KV heads, channels) by pool, and behind the tokens by prompt plan
_geometry, _prompt_shape = {}, {}


# ---- pool ----------------------------------------------------------------------
def gk_pool_create(num_layers, num_q_heads, num_kv_heads, head_dim, hot_tokens, cold_slots, cold_page_size,
                   seed=0, hot_k=None, hot_v=None, cold_k=None, cold_v=None):
    cfg = gk_pool_config(num_layers, num_q_heads, num_kv_heads, head_dim, hot_tokens, cold_slots, cold_page_size, 0,
                         seed, _ptr(hot_k), _ptr(hot_v), _ptr(cold_k), _ptr(cold_v))
    out = c_vp()
    _check(lib().gk_pool_create(ctypes.byref(cfg), ctypes.byref(out)))
    _geometry[out.value] = (num_q_heads, num_kv_heads, head_dim)
    return out.value


def gk_pool_create_kv4(num_layers, num_q_heads, num_kv_heads, head_dim, hot_tokens, cold_slots, cold_page_size, seed=0, hot_k=None,
                       hot_v=None, cold=None):
    """cold: uint8 [num_layers, cold_slots, gk_kv4_row_bytes(num_kv_heads, head_dim)] or its address."""
    cfg = gk_pool_config(num_layers, num_q_heads, num_kv_heads, head_dim, hot_tokens, cold_slots, cold_page_size, 0, seed,
                         _ptr(hot_k), _ptr(hot_v), _ptr(cold), None)
    if cold is not None and not isinstance(cold, int):
        row = gk_kv4_row_bytes(num_kv_heads, head_dim)
        if cold.numel() * cold.element_size() < num_layers * cold_slots * row or not cold.is_contiguous():
            raise ValueError(f"cold must be contiguous and hold {num_layers} layers of {cold_slots} rows of {row} bytes")
    out = c_vp()
    _check(lib().gk_pool_create_kv4(ctypes.byref(cfg), ctypes.byref(out)))
    _geometry[out.value] = (num_q_heads, num_kv_heads, head_dim)
    return out.value


def gk_kv4_row_bytes(num_kv_heads, head_dim):
    """Bytes of a 4-bit row of K and V (0: no pool has this geometry)."""
    return lib().gk_kv4_row_bytes(num_kv_heads, head_dim)


def gk_pool_destroy(pool):
    _geometry.pop(pool, None)
    lib().gk_pool_destroy(pool)


def gk_last_error(pool):
    return lib().gk_last_error(pool).decode()


def gk_status_string(status):
    return lib().gk_status_string(status).decode()


# ---- HOT pool --------------------------------------------------------------------
def gk_prefix_alloc(pool, prefix_len):
    base = c_i64()
    _check(lib().gk_prefix_alloc(pool, prefix_len, ctypes.byref(base)), pool)
    return base.value


def gk_prefix_release(pool, hot_base):
    _check(lib().gk_prefix_release(pool, hot_base), pool)


def gk_hot_stats(pool):
    a, b, c = c_i64(), c_i64(), c_i64()
    _check(lib().gk_hot_stats(pool, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)), pool)
    return a.value, b.value, c.value


def gk_prefix_acquire(pool, key, prefix_len):
    """-> (hot_base, hit): a reference on the cached slab of key, allocated (evicting idle slabs) on a miss."""
    base, hit = c_i64(), c_i32()
    _check(lib().gk_prefix_acquire(pool, int(key) & ((1 << 64) - 1), int(prefix_len), ctypes.byref(base),
                                   ctypes.byref(hit)), pool)
    return base.value, bool(hit.value)


def gk_prefix_unref(pool, key):
    _check(lib().gk_prefix_unref(pool, int(key) & ((1 << 64) - 1)), pool)


def gk_hot_cache_stats(pool):
    """-> (cached slabs, idle slabs, tokens held by idle slabs)."""
    a, b, c = c_i64(), c_i64(), c_i64()
    _check(lib().gk_hot_cache_stats(pool, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)), pool)
    return a.value, b.value, c.value


# ---- COLD block manager ----------------------------------------------------------
def gk_seq_create(pool):
    s = c_i32()
    _check(lib().gk_seq_create(pool, ctypes.byref(s)), pool)
    return s.value


def gk_seq_fork(pool, parent):
    s = c_i32()
    _check(lib().gk_seq_fork(pool, parent, ctypes.byref(s)), pool)
    return s.value


def gk_seq_release(pool, seq):
    _check(lib().gk_seq_release(pool, seq), pool)


def gk_seq_table(pool, seq):
    """-> (block table as a numpy int32 copy, length in tokens)."""
    t = P(c_i32)()
    nb, ln = c_i32(), c_i64()
    _check(lib().gk_seq_table(pool, seq, ctypes.byref(t), ctypes.byref(nb), ctypes.byref(ln)), pool)
    arr = np.ctypeslib.as_array(t, shape=(nb.value,)).copy() if nb.value else np.zeros(0, np.int32)
    return arr, ln.value


def gk_seq_append_slots(pool, seqs):
    """-> (slot_mapping int64 [n], cow_pairs int32 [n_cow, 2]).  Raises GkError(GK_ERR_OOM) with .n_done set."""
    seqs = np.ascontiguousarray(seqs, dtype=np.int32)
    n = len(seqs)
    slots = np.empty(n, dtype=np.int64)
    cow = np.empty(2 * max(n, 1), dtype=np.int32)
    ncow, ndone = c_i32(), c_i32()
    st = lib().gk_seq_append_slots(pool, n, _i32p(seqs), _i64p(slots), ctypes.byref(ncow), _i32p(cow),
                                   ctypes.byref(ndone))
    if st != GK_OK:
        err = GkError(st, gk_last_error(pool))
        err.n_done = ndone.value
        err.slots = slots[:ndone.value]
        err.cow_pairs = cow[:2 * ncow.value].reshape(-1, 2)
        raise err
    return slots, cow[:2 * ncow.value].reshape(-1, 2).copy()


def gk_seq_tables(pool, seqs, max_blocks, table_out=None, len_out=None):
    """Fill (or allocate) int32 [n, max_blocks] tables and int32 [n] lengths; returns both."""
    seqs = np.ascontiguousarray(seqs, dtype=np.int32)
    n = len(seqs)
    if table_out is None:
        table_out = np.empty((n, max_blocks), dtype=np.int32)
    if len_out is None:
        len_out = np.empty(n, dtype=np.int32)
    assert table_out.dtype == np.int32 and table_out.flags.c_contiguous and table_out.size >= n * max_blocks
    _check(lib().gk_seq_tables(pool, n, _i32p(seqs), max_blocks, _i32p(table_out), _i32p(len_out)), pool)
    return table_out, len_out


def gk_seq_create_cached(pool, tokens):
    """-> (seq, n_cached): a new sequence starting with the longest cached chain of tokens' full blocks."""
    t = np.ascontiguousarray(tokens, dtype=np.int32)
    s, n = c_i32(), c_i64()
    _check(lib().gk_seq_create_cached(pool, len(t), t.ctypes.data_as(c_vp), ctypes.byref(s), ctypes.byref(n)), pool)
    return s.value, n.value


def gk_seq_cache_blocks(pool, seq, tokens):
    """Cache seq's full blocks covering tokens; -> blocks newly cached."""
    t = np.ascontiguousarray(tokens, dtype=np.int32)
    n = c_i32()
    _check(lib().gk_seq_cache_blocks(pool, int(seq), len(t), t.ctypes.data_as(c_vp), ctypes.byref(n)), pool)
    return n.value


def gk_cold_cache_stats(pool):
    """-> (cached blocks, evictable blocks)."""
    a, b = c_i64(), c_i64()
    _check(lib().gk_cold_cache_stats(pool, ctypes.byref(a), ctypes.byref(b)), pool)
    return a.value, b.value


def gk_cold_stats(pool):
    a, b = c_i64(), c_i64()
    _check(lib().gk_cold_stats(pool, ctypes.byref(a), ctypes.byref(b)), pool)
    return a.value, b.value


def gk_block_refcount(pool, block):
    r = c_i32()
    _check(lib().gk_block_refcount(pool, block, ctypes.byref(r)), pool)
    return r.value


class Tables:
    """A gk_tables over int32 torch tensors: table [rows, max_blocks], free [capacity], length [rows],
    num_free [1]; the step's outputs go to length_out and num_free_out (default: in place)."""

    def __init__(self, table, free, length, num_free, length_out=None, num_free_out=None):
        self.length_out = length if length_out is None else length_out
        self.num_free_out = num_free if num_free_out is None else num_free_out
        self.table, self.free, self.length, self.num_free = table, free, length, num_free
        rows, width = table.shape
        self.rows, self.i32, self.i64 = rows, sys.modules["torch"].int32, sys.modules["torch"].int64
        for x, n in ((table, rows * width), (free, free.numel()), (length, rows), (num_free, 1), (self.length_out, rows),
                     (self.num_free_out, 1)):
            if x.numel() != n or x.dtype is not self.i32 or not x.is_contiguous():
                raise ValueError("tables are contiguous int32 tensors: table [rows, max_blocks], free, length [rows], num_free [1]")
        # int32 words: allocations are at least 16-byte aligned
        self.work = table.new_empty((rows + 1) * (GK_TABLES_WORK_PER_ROW // 4))
        self.c = gk_tables(rows, width, free.numel(), 0, _ptr(table), _ptr(free), _ptr(length), _ptr(self.length_out),
                           _ptr(num_free), _ptr(self.num_free_out), _ptr(self.work))
        self.ref = ctypes.byref(self.c)


def _row_of(x, n, dtype, what):
    """Address of x, a contiguous tensor of at least n elements, or an address."""
    if x is None or isinstance(x, int):
        return x
    if x.dtype is not dtype or x.numel() < n or not x.is_contiguous():
        raise ValueError(f"{what} must be contiguous {dtype} with {n} elements or more")
    return x.data_ptr()


def gk_tables_step(pool, stream, tables, d_add, d_slot_mapping, d_done, d_release=None, n_slots=None):
    """int32 [rows] add, done and release (flags), int64 [n_slots] slot mapping: torch tensors or addresses."""
    rows, n, i32, i64 = tables.rows, d_slot_mapping.numel() if n_slots is None else n_slots, tables.i32, tables.i64
    st = lib().gk_tables_step(pool, _stream(stream), tables.ref, _row_of(d_release, rows, i32, "release"),
                              _row_of(d_add, rows, i32, "add"), n, _row_of(d_slot_mapping, n, i64, "the slot mapping"),
                              _row_of(d_done, rows, i32, "done"))
    if st:
        _check(st, pool)


# ---- device work -------------------------------------------------------------------
def gk_append_kv(pool, stream, layer, d_slot_mapping, d_k, d_v, d_cow_pairs=None, n=None, n_cow=None):
    n = d_slot_mapping.numel() if n is None else n
    n_cow = (0 if d_cow_pairs is None else d_cow_pairs.numel() // 2) if n_cow is None else n_cow
    _check(lib().gk_append_kv(pool, _stream(stream), layer, n, _ptr(d_slot_mapping), _ptr(d_k), _ptr(d_v), n_cow,
                              _ptr(d_cow_pairs) if n_cow else None), pool)


def gk_write_prefix_kv(pool, stream, layer, hot_base, prefix_len, t0, d_k, d_v, n=None):
    n = d_k.shape[0] if n is None else n
    _check(lib().gk_write_prefix_kv(pool, _stream(stream), layer, hot_base, prefix_len, t0, n, _ptr(d_k), _ptr(d_v)),
           pool)


# ---- from a layer's projections to its cache and attention -----------------------------
def _gpu_row(x, n, dtype, what):
    """As _row_of, of a tensor that is on the GPU."""
    if x is not None and not isinstance(x, int) and not x.is_cuda:
        raise ValueError(f"{what} must be on the GPU")
    return _row_of(x, n, dtype, what)


class _Call(threading.local):
    """The gk_qkv that a thread's calls fill in, a copy of c: the library reads it while other threads may run."""

    def __init__(self, c):
        self.c = gk_qkv.from_buffer_copy(c)
        self.ref = ctypes.byref(self.c)
        self.seen = None


class Rope:
    """How the queries and keys of a layer are normed and rotated: cos_sin fp32 [positions, rot_dim] (cosines, then sines),
    bf16 weights [head_dim] or None (no norm).  Kept by the caller; the tensors stay alive with it.  Pools of several threads
    may share one."""

    def __init__(self, cos_sin=None, rot_dim=None, interleaved=False, q_weight=None, k_weight=None, eps=1e-6):
        import torch
        self.torch = torch
        if cos_sin is not None:
            if cos_sin.dim() != 2 or cos_sin.dtype is not torch.float32 or not cos_sin.is_contiguous() or not cos_sin.is_cuda:
                raise ValueError("cos_sin must be contiguous fp32 [positions, rot_dim] on the GPU")
            if rot_dim is not None and rot_dim != cos_sin.shape[1]:
                raise ValueError(f"cos_sin has rows of {cos_sin.shape[1]}, not of rot_dim {rot_dim}")
            rot_dim = cos_sin.shape[1]
        elif rot_dim:
            raise ValueError("a rotation needs cos_sin")
        self.dims = set()
        for w in (q_weight, k_weight):
            if w is None:
                continue
            if w.dim() != 1 or w.dtype is not torch.bfloat16 or not w.is_contiguous() or not w.is_cuda:
                raise ValueError("a norm's weight must be contiguous bf16 [head_dim] on the GPU")
            self.dims.add(w.shape[0])
        self.tensors = cos_sin, q_weight, k_weight
        self.rotates = bool(rot_dim)
        self.call = _Call(gk_qkv(0, rot_dim or 0, int(bool(interleaved)), eps, 0 if cos_sin is None else cos_sin.shape[0],
                                 _ptr(cos_sin), None, _ptr(q_weight), _ptr(k_weight)))

    @property
    def c(self):
        return self.call.c

    def set(self, pool, positions, q, k, v, q_out, k_out, n):
        """Fill the call's rows in: bf16 [n, heads, d] tensors (tokens may be strided) or addresses of packed rows."""
        call = self.call
        c = call.c
        # what a layout was found to be when it came last (strides, heads and types: not what the tensors hold or where)
        seen = (_geometry.get(pool), n, _layout(q), _layout(q_out), _layout(k), _layout(k_out), _layout(v), _layout(positions))
        if seen != call.seen:
            call.seen = None
            self._check(c, pool, positions, q, k, v, q_out, k_out, n)
            call.seen = seen
        c.d_q, c.d_q_out, c.d_k, c.d_k_out, c.d_v = _ptr(q), _ptr(q_out), _ptr(k), _ptr(k_out), _ptr(v)
        if self.rotates:
            c.d_positions = _ptr(positions)
        return call.ref

    def _check(self, c, pool, positions, q, k, v, q_out, k_out, n):
        torch = self.torch
        hq, hkv, dim = _geometry.get(pool, (None, None, None))
        if dim is not None and any(d != dim for d in self.dims):
            raise ValueError(f"the norms' weights are of {self.dims} channels, the pool's heads of {dim}")
        strides = []
        for x, heads, what in ((q, hq, "q"), (q_out, hq, "q_out"), (k, hkv, "k"), (k_out, hkv, "k_out"), (v, hkv, "v")):
            h, d, stride, _ = _token_rows(x, n, what, torch)
            if h is not None and heads is not None and (h != heads or d != dim):
                raise ValueError(f"{what} must have the pool's {heads} heads of {dim}")
            strides.append(stride)
        if self.rotates:
            if positions is None and n:
                raise ValueError("a rotation needs positions")
            _gpu_row(positions, n, torch.int32, "positions")
        c.num_tokens = n
        c.q_stride, c.q_out_stride, c.k_stride, c.k_out_stride, c.v_stride = strides


def _layout(x):
    """All that the checks of a tensor look at (an address and None: themselves)."""
    return x if x is None or isinstance(x, int) else (x.shape, x.stride(), x.dtype, x.is_cuda)


def gk_qk_norm_rope(pool, stream, rope, positions, q, k, q_out=None, k_out=None, n=None):
    """q [n, Hq, d] and k [n, Hkv, d] (either may be None), normed and rotated, to q_out and k_out (default: in place)."""
    n = (k if q is None else q).shape[0] if n is None else n
    ref = rope.set(pool, positions, q, k, None, q if q_out is None else q_out, k if k_out is None else k_out, n)
    st = (_lib or lib()).gk_qk_norm_rope(pool, _stream(stream), ref)
    if st:
        _check(st, pool)


def gk_append_qkv(pool, stream, layer, rope, positions, d_slot_mapping, q, k, v, q_out=None, k_out=None, d_cow_pairs=None, n=None):
    """As gk_qk_norm_rope, and K and V into the cache; q may be None, q_out defaults to in place, k_out to none."""
    n = k.shape[0] if n is None else n
    ref = rope.set(pool, positions, q, k, v, q if q_out is None else q_out, k_out, n)
    i32, i64 = rope.torch.int32, rope.torch.int64
    n_cow = 0 if d_cow_pairs is None else d_cow_pairs.numel() // 2
    st = (_lib or lib()).gk_append_qkv(pool, _stream(stream), layer, ref, _gpu_row(d_slot_mapping, n, i64, "the slot mapping"), n_cow,
                                       _gpu_row(d_cow_pairs, 2 * n_cow, i32, "copy-on-write pairs") if n_cow else None)
    if st:
        _check(st, pool)


_read_seen = {}      # (geometry, layouts) of reads that were checked: the token strides of k and v


def gk_read_kv(pool, stream, layer, d_slot_mapping, d_k, d_v, n=None):
    """K and V of the slots as bf16 [n, Hkv, d] (tokens may be strided)."""
    n = d_slot_mapping.numel() if n is None else n
    seen = (_geometry.get(pool), n, _layout(d_slot_mapping), _layout(d_k), _layout(d_v))
    strides = _read_seen.get(seen)
    if strides is None:
        torch = sys.modules.get("torch")
        heads, dim = (seen[0] or (None, None, None))[1:]
        strides = []
        for x, what in ((d_k, "k"), (d_v, "v")):
            h, d, stride, _ = _token_rows(x, n, what, torch)
            if h is not None and heads is not None and (h != heads or d != dim):
                raise ValueError(f"{what} must have the pool's {heads} heads of {dim}")
            strides.append(stride)
        if not isinstance(d_slot_mapping, int):
            _gpu_row(d_slot_mapping, n, torch.int64, "the slot mapping")
        if len(_read_seen) >= 256:
            _read_seen.clear()
        _read_seen[seen] = strides
    st = (_lib or lib()).gk_read_kv(pool, _stream(stream), layer, n, _ptr(d_slot_mapping), _ptr(d_k), _ptr(d_v), *strides)
    if st:
        _check(st, pool)


def _packed(x, what, hint=""):
    """Address of x, a contiguous tensor or an address, and what a call that knows its size checks of it (None of an address)."""
    if x is None or isinstance(x, int):
        return x, None
    if not x.is_contiguous():
        raise ValueError(f"{what} must be contiguous{hint}")
    return x.data_ptr(), (x.numel(), x.dtype, x.is_cuda)


_FUSED = ": queries in the rows of a fused projection need an output of their own (q_out)"


class Batch:
    """Keeps the host arrays of a gk_batch alive; .set_device() swaps the per-layer device pointers."""

    def __init__(self, prefix_hot_base, prefix_len, suffix_len, d_block_table=None, max_blocks=0, d_q=None,
                 d_out=None, d_lse=None):
        self.prefix_hot_base = np.ascontiguousarray(prefix_hot_base, dtype=np.int64)
        self.prefix_len = np.ascontiguousarray(prefix_len, dtype=np.int32)
        self.suffix_len = np.ascontiguousarray(suffix_len, dtype=np.int32)
        q, self.q = _packed(d_q, "q", _FUSED)
        lse, self.lse = _packed(d_lse, "lse")
        self.c = gk_batch(len(self.prefix_len), max_blocks, _i64p(self.prefix_hot_base), _i32p(self.prefix_len),
                          _i32p(self.suffix_len), _ptr(d_block_table), q, _ptr(d_out), lse, None, None)
        self.ref = ctypes.byref(self.c)

    def set_device(self, d_block_table=None, max_blocks=None, d_q=None, d_out=None, d_lse=None, d_new_k=None,
                   d_new_v=None):
        """d_lse, d_new_k and d_new_v are set on every call (None clears them: no LSE
        output, no fused append); the others keep their value when None.  ValueError, with the
        batch as it was, for a q or lse that is not contiguous."""
        lse, lse_seen = _packed(d_lse, "lse")
        if d_q is not None:
            self.c.d_q, self.q = _packed(d_q, "q", _FUSED)
        if d_block_table is not None:
            self.c.d_block_table = _ptr(d_block_table)
        if max_blocks is not None:
            self.c.max_blocks = max_blocks
        if d_out is not None:
            self.c.d_out = _ptr(d_out)
        self.c.d_lse, self.lse = lse, lse_seen
        self.c.d_new_k = _ptr(d_new_k)
        self.c.d_new_v = _ptr(d_new_v)
        return self


def gk_plan_build(pool, batch, stream=None):
    out = c_vp()
    _check(lib().gk_plan_build(pool, ctypes.byref(batch.c), _stream(stream), ctypes.byref(out)), pool)
    return out.value


def gk_plan_update(pool, plan, batch, stream=None):
    _check(lib().gk_plan_update(plan, ctypes.byref(batch.c), _stream(stream)), pool)


def gk_plan_destroy(plan):
    lib().gk_plan_destroy(plan)


def gk_plan_info(plan):
    s = gk_plan_summary()
    _check(lib().gk_plan_info(plan, ctypes.byref(s)))
    return {name: getattr(s, name) for name, _ in gk_plan_summary._fields_}


def gk_plan_segments(plan, dense=False):
    """(begin [n_ctas + 1], segs [n_segs, 4] = request, t0, t1, entry): the plan's gather partition."""
    n_ctas, n_segs = c_i32(), c_i32()
    _check(lib().gk_plan_segments(plan, int(bool(dense)), ctypes.byref(n_ctas), ctypes.byref(n_segs), None, None))
    begin = np.zeros(n_ctas.value + 1, dtype=np.int32)
    segs = np.zeros((n_segs.value, 4), dtype=np.int32)
    _check(lib().gk_plan_segments(plan, int(bool(dense)), ctypes.byref(n_ctas), ctypes.byref(n_segs),
                                  begin.ctypes.data_as(c_vp), segs.ctypes.data_as(c_vp)))
    return begin, segs


def gk_decode_dense(pool, stream, layer, batch, plan):
    _check(lib().gk_decode_dense(pool, _stream(stream), layer, ctypes.byref(batch.c), plan), pool)


def gk_decode_cascade(pool, stream, layer, batch, plan):
    _check(lib().gk_decode_cascade(pool, _stream(stream), layer, ctypes.byref(batch.c), plan), pool)


def gk_decode_kv4(pool, stream, layer, batch, plan, d_out):
    """bf16 out [B, Hq, d] of a decode step over a 4-bit pool (the batch's q [B, Hq, d], lse and block table; its d_out is not used).
    All are packed: append_qkv's queries in place, in a fused projection's rows, are not."""
    n, torch = batch.c.num_requests, sys.modules.get("torch")
    hq, _, d = _geometry.get(pool, (None, None, None))
    if not isinstance(d_out, int):
        shape = (n, d_out.shape[1] if hq is None else hq, d_out.shape[2] if d is None else d)
        if d_out.shape != shape or d_out.dtype is not torch.bfloat16 or not d_out.is_contiguous() or not d_out.is_cuda:
            raise ValueError("out must be contiguous bf16 [%d, %d, %d] on the GPU" % shape)
        d_out = d_out.data_ptr()
    if hq is not None:
        if batch.q is not None and (batch.q[0] < n * hq * d or batch.q[1] is not torch.bfloat16 or not batch.q[2]):
            raise ValueError(f"q must be bf16 [{n}, {hq}, {d}] on the GPU")
        if batch.lse is not None and (batch.lse[0] < n * hq or batch.lse[1] is not torch.float32 or not batch.lse[2]):
            raise ValueError(f"lse must be fp32 [{n}, {hq}] on the GPU")
    st = (_lib or lib()).gk_decode_kv4(pool, _stream(stream), layer, batch.ref, plan, d_out)
    if st:
        _check(st, pool)


def gk_decode_dense_static(pool, stream, layer, batch):
    _check(lib().gk_decode_dense_static(pool, _stream(stream), layer, ctypes.byref(batch.c)), pool)


def gk_cascade_levels(pool, stream, layer, batch, plan):
    _check(lib().gk_cascade_levels(pool, _stream(stream), layer, ctypes.byref(batch.c), plan), pool)


def gk_cascade_prefix(pool, stream, layer, batch, plan):
    _check(lib().gk_cascade_prefix(pool, _stream(stream), layer, ctypes.byref(batch.c), plan), pool)


def gk_cascade_suffix(pool, stream, layer, batch, plan):
    _check(lib().gk_cascade_suffix(pool, _stream(stream), layer, ctypes.byref(batch.c), plan), pool)


def gk_cascade_merge(pool, stream, layer, batch, plan):
    _check(lib().gk_cascade_merge(pool, _stream(stream), layer, ctypes.byref(batch.c), plan), pool)


# ---- prompt step ---------------------------------------------------------------------
def _token_rows(x, tokens, what, torch):
    """heads, d, elements from one token to the next (0: packed) and address of x, a bf16 CUDA tensor [tokens, heads, d];
    no heads and no d for the address of packed rows."""
    if x is None or isinstance(x, int):
        return None, None, 0, x
    n, heads, d = x.shape
    row, head, channel = x.stride()
    if n != tokens or x.dtype is not torch.bfloat16 or not x.is_cuda or n and (channel != 1 or heads > 1 and head != d):
        raise ValueError(f"{what} must be bf16 [{tokens}, heads, d] on the GPU, with a token's heads and channels contiguous")
    if n > 1 and row < heads * d:
        raise ValueError(f"{what}'s tokens overlap: a row of a token's own is read for each of {n}, which expand() does not give")
    return heads, d, row if n > 1 else 0, x.data_ptr()


class PromptBatch:
    """Keeps the host arrays of a gk_prompt_batch alive; .set_device() swaps the per-layer device pointers."""

    def __init__(self, new_len, prefix_hot_base=None, prefix_len=None, context_len=None, d_block_table=None,
                 max_blocks=0):
        self.new_len = np.ascontiguousarray(new_len, dtype=np.int32)
        n = len(self.new_len)

        def host(a, t):
            if a is None:
                return None
            a = np.ascontiguousarray(a, dtype=t)
            if a.shape != (n,):
                raise ValueError("one entry per request")
            return a
        self.prefix_hot_base, self.prefix_len = host(prefix_hot_base, np.int64), host(prefix_len, np.int32)
        self.context_len = host(context_len, np.int32)
        self.tokens = int(self.new_len.astype(np.int64).sum())
        self.c = gk_prompt_batch(n, max_blocks, _i32p(self.new_len),
                                 None if self.prefix_hot_base is None else _i64p(self.prefix_hot_base),
                                 None if self.prefix_len is None else _i32p(self.prefix_len),
                                 None if self.context_len is None else _i32p(self.context_len))
        self._check_table(d_block_table, max_blocks)
        self._table = d_block_table
        self.c.d_block_table = _ptr(d_block_table)
        self.shape = self.tokens, None, None, None   # and query heads, KV heads and channels of the tensors set last
        self.ref = ctypes.byref(self.c)

    def set_device(self, d_q, d_k, d_v, d_out, d_lse=None, d_block_table=None, max_blocks=None):
        """bf16 [T, Hq, d] q and out, [T, Hkv, d] k and v, fp32 [T, Hq] lse, int32 [B, max_blocks] table: torch tensors
        (tokens may be strided, as views of a fused projection are; lse is contiguous, and the table's rows max_blocks
        apart) or addresses of packed rows.  ValueError, with the batch as it was, for tensors of another type or shape."""
        c, T, torch = self.c, self.tokens, sys.modules.get("torch")    # who passes tensors has imported it
        hq, d, q_stride, q = _token_rows(d_q, T, "q", torch)
        ho, do, out_stride, out = _token_rows(d_out, T, "out", torch)
        hkv, dk, k_stride, k = _token_rows(d_k, T, "k", torch)
        hv, dv, v_stride, v = _token_rows(d_v, T, "v", torch)
        if hq != ho or hkv != hv or not d == do == dk == dv:       # or some of them are addresses
            hq, hkv, d = (hq, ho), (hkv, hv), (d, do, dk, dv)
            hq, hkv, d = (next((x for x in same if x is not None), None) for same in (hq, hkv, d))
            if any(x not in (None, y) for x, y in zip((ho, hv, do, dk, dv), (hq, hkv, d, d, d))):
                raise ValueError("out has the heads of q, v those of k, and all four the same channels")
        if d_lse is not None and not isinstance(d_lse, int):
            if d_lse.shape != (T, hq) and (hq is not None or d_lse.dim() != 2 or d_lse.shape[0] != T) or \
                    d_lse.dtype is not torch.float32 or not d_lse.is_contiguous() or not d_lse.is_cuda:
                raise ValueError(f"lse must be contiguous fp32 [{T}, query heads] on the GPU")
        if d_block_table is not None or max_blocks is not None:
            table = self._table if d_block_table is None else d_block_table
            width = c.max_blocks if max_blocks is None else max_blocks
            self._check_table(table, width)
            c.d_block_table, c.max_blocks, self._table = _ptr(table), width, table
        c.q_stride, c.out_stride, c.k_stride, c.v_stride = q_stride, out_stride, k_stride, v_stride
        c.d_q, c.d_k, c.d_v, c.d_out, c.d_lse = q, k, v, out, _ptr(d_lse)
        self.shape = T, hq, hkv, d
        return self

    def _check_table(self, table, width):
        if table is None or isinstance(table, int):
            return
        n = len(self.new_len)
        rows = table.is_contiguous() and table.numel() >= n * width or \
            table.dim() == 2 and table.shape[0] >= n and table.stride() == (width, 1)    # the first columns of a wider table
        if table.dtype is not sys.modules["torch"].int32 or not rows or not table.is_cuda:
            raise ValueError(f"the block table must be int32 [{n}, {width}] on the GPU, or columns of one with rows of {width}")

    def check_plan(self, plan):
        """The plan is of as many tokens, and its pool has the tensors' heads (None: an address's are not known)."""
        want = _prompt_shape.get(plan, self.shape)
        if want[0] != self.tokens:
            raise ValueError("the plan is of another number of tokens than the batch")
        if any(None is not a != b is not None for a, b in zip(self.shape, want)):
            raise ValueError("the pool has %s query heads and %s KV heads of %s" % want[1:])


def gk_prompt_plan_build(pool, batch, stream=None):
    out = c_vp()
    _check(lib().gk_prompt_plan_build(pool, ctypes.byref(batch.c), _stream(stream), ctypes.byref(out)), pool)
    _prompt_shape[out.value] = (batch.tokens, *_geometry.get(pool, (None, None, None)))
    return out.value


def gk_prompt_plan_update(pool, plan, batch, stream=None):
    _check(lib().gk_prompt_plan_update(plan, ctypes.byref(batch.c), _stream(stream)), pool)
    _prompt_shape[plan] = (batch.tokens, *_prompt_shape.get(plan, (0, None, None, None))[1:])


def gk_prompt_plan_destroy(plan):
    _prompt_shape.pop(plan, None)
    lib().gk_prompt_plan_destroy(plan)


def gk_prompt_plan_info(plan):
    s = gk_prompt_plan_summary()
    _check(lib().gk_prompt_plan_info(plan, ctypes.byref(s)))
    return {name: getattr(s, name) for name, _ in gk_prompt_plan_summary._fields_}


def gk_prompt_plan_items(plan):
    """(begin [n_ctas + 1], items [n_items, 8] = request, run tokens, head, first token, first tile, tiles, partial, HOT tiles)."""
    n_ctas, n_items = c_i32(), c_i32()
    _check(lib().gk_prompt_plan_items(plan, ctypes.byref(n_ctas), ctypes.byref(n_items), None, None))
    begin = np.zeros(n_ctas.value + 1, dtype=np.int32)
    items = np.zeros((n_items.value, 8), dtype=np.int32)
    _check(lib().gk_prompt_plan_items(plan, ctypes.byref(n_ctas), ctypes.byref(n_items), begin.ctypes.data_as(c_vp),
                                      items.ctypes.data_as(c_vp)))
    return begin, items


def gk_prompt_attn(pool, stream, layer, batch, plan):
    if _prompt_shape.get(plan) != batch.shape:
        batch.check_plan(plan)
    st = lib().gk_prompt_attn(pool, _stream(stream), layer, batch.ref, plan)
    if st:
        _check(st, pool)


def gk_dispatch(pool, plan):
    """-> (GK_BACKEND_*, predicted dense us, predicted cascade us)."""
    ch, td, tc = c_i32(), c_dbl(), c_dbl()
    _check(lib().gk_dispatch(pool, plan, ctypes.byref(ch), ctypes.byref(td), ctypes.byref(tc)), pool)
    return ch.value, td.value, tc.value


def gk_cost_model_get(pool):
    cm = gk_cost_model()
    _check(lib().gk_cost_model_get(pool, ctypes.byref(cm)), pool)
    return {k: getattr(cm, k) for k in COST_MODEL_KEYS}


COST_MODEL_KEYS = ("c_flat_us", "bw_flat_gbs", "c_cascade_us", "bw_prefix_gbs", "bw_suffix_gbs", "c_merge_us",
                   "prefix_tile_us", "prefix_item_us", "gather_sm_gbs", "c_gather_us", "prefix_tile_split_us",
                   "warp_tile_us", "warp_group_us", "warp_item_us", "warp_split_ratio", "prefix_cta_ramp_us",
                   "prefix_cta_gather_ratio", "c_merge_state_us", "prefix_item_split_us", "warp_item_split_us",
                   "prefix_item_crowd_us", "split_gather_ratio_tensor", "c_gather_split_us",
                   "split_tensor_us")


def gk_cost_model_set(pool, cm: dict):
    c = gk_cost_model()
    for k in COST_MODEL_KEYS:
        setattr(c, k, float(cm[k]))
    _check(lib().gk_cost_model_set(pool, ctypes.byref(c)), pool)


GK_CASCADE_AUTO, GK_CASCADE_SEQUENTIAL, GK_CASCADE_SPLIT = 0, 1, 2


def gk_pool_set_cascade_mode(pool, mode, tiles_per_item=0):
    _check(lib().gk_pool_set_cascade_mode(pool, int(mode), int(tiles_per_item)), pool)


GK_PARTITION_STREAM, GK_PARTITION_PER_REQUEST = 0, 1


def gk_pool_set_gather_partition(pool, partition):
    _check(lib().gk_pool_set_gather_partition(pool, int(partition)), pool)


GK_PREFIX_AUTO, GK_PREFIX_TENSOR, GK_PREFIX_WARP = 0, 1, 2


def gk_pool_set_prefix_kernel(pool, kernel):
    _check(lib().gk_pool_set_prefix_kernel(pool, int(kernel)), pool)


def gk_pool_set_sm_speeds(pool, speeds):
    """speeds: one per SM of the device, or None / empty to clear."""
    if speeds is None or len(speeds) == 0:
        _check(lib().gk_pool_set_sm_speeds(pool, None, 0), pool)
        return
    a = np.ascontiguousarray(speeds, dtype=np.float32)
    _check(lib().gk_pool_set_sm_speeds(pool, a.ctypes.data_as(P(ctypes.c_float)), len(a)), pool)


def gk_pool_get_sm_speeds(pool):
    n = c_i32()
    _check(lib().gk_pool_get_sm_speeds(pool, None, ctypes.byref(n)), pool)
    a = np.zeros(n.value, np.float32)
    if n.value:
        _check(lib().gk_pool_get_sm_speeds(pool, a.ctypes.data_as(P(ctypes.c_float)), ctypes.byref(n)), pool)
    return a


def gk_sm_speeds_measure(pool, stream, layer, batch, plan, reps=5):
    """-> the measured per-SM speeds (installed in the pool)."""
    n = c_i32()
    _check(lib().gk_pool_get_sm_speeds(pool, None, ctypes.byref(n)), pool)
    _check(lib().gk_sm_speeds_measure(pool, _stream(stream), layer, ctypes.byref(batch.c), plan, reps, None), pool)
    return gk_pool_get_sm_speeds(pool)


def gk_calibrate(pool, stream=None, json_out=None):
    _check(lib().gk_calibrate(pool, _stream(stream), json_out.encode() if json_out else None), pool)


def gk_cost_model_load(pool, json_text: str):
    _check(lib().gk_cost_model_load(pool, json_text.encode()), pool)


def gk_device_error(pool, stream=None):
    code = c_i32()
    _check(lib().gk_device_error(pool, _stream(stream), ctypes.byref(code)), pool)
    return code.value
