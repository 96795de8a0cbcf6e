/*
 * gk.h -- C ABI of the shared-prefix paged decode-attention library (libgk.so).
 *
 * Storage follows "GraniKV: Asymmetric Granularity KV-Cache Paging for
 * Multi-Agent Systems with Long Shared Prefix": a shared prefix lives in a
 * contiguous HOT pool (Section 3.2) and each request's own tokens live in a
 * token-granular COLD pool (Section 3.3) reached through a block table whose
 * bookkeeping is the refcounted copy-on-write block manager of "Paged KV cache"
 * (How it works; Code).
 *
 * Conventions for every call:
 *  - The return value is a gk_status; GK_OK is 0.  On failure the pool's
 *    gk_last_error() text says what was wrong.  No C++ exception crosses the ABI.
 *  - "device" pointers are CUDA global-memory addresses owned by the caller;
 *    the library never frees them.  "host" pointers are ordinary memory.
 *  - Device work is enqueued on the caller's stream (a cudaStream_t passed as
 *    void*; NULL is the legacy default stream) and returns before it finishes.
 *  - Host metadata (block tables, refcounts, HOT free list, plans) is owned by
 *    the library.  A pool and its plans are not thread-safe.
 *  - bf16 is passed as raw 16-bit storage (void*); fp32 as float*.
 *
 * Layouts (all row-major, d = head_dim, Hkv = num_kv_heads, L = num_layers):
 *  - HOT K and V: [hot_tokens * L * Hkv * d] bf16 each.  A prefix at token base
 *    b with Lp tokens owns elements [b*L*Hkv*d, (b+Lp)*L*Hkv*d), laid out
 *    [L][Hkv][Lp][d], so the (layer, head) slice is one contiguous [Lp][d]
 *    block ("base + l*Lp*Hkv + h*Lp" of Section 3.2 with the allocator
 *    counting tokens).
 *  - COLD K and V: [L][cold_slots][Hkv][d] bf16 each; the slot of token t of a
 *    sequence is table[t / P] * P + t % P with P = cold_page_size
 *    ("Paged KV cache", How it works).
 *  - COLD in 4 bits (gk_pool_create_kv4): [L][cold_slots][gk_kv4_row_bytes], one row
 *    of codes and scales for a token's K and V together (the call gives the layout).
 *  - Queries [B][Hq][d] bf16, outputs [B][Hq][d] fp32, LSE [B][Hq] fp32
 *    (natural log).  Query head qh reads KV head qh / (Hq / Hkv).
 */
#ifndef GK_H_
#define GK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gk_status {
  GK_OK = 0,
  GK_ERR_INVALID = 1,        /* bad argument, unknown id, inconsistent sizes */
  GK_ERR_OOM = 2,            /* COLD pool out of blocks: preempt a sequence ("Paged KV cache", step 4) */
  GK_ERR_HOT_FULL = 3,       /* no HOT range fits: place the prefix in COLD (GraniKV Appendix B.10) */
  GK_ERR_CUDA = 4,           /* a CUDA runtime or driver call failed */
  GK_ERR_DEVICE_BOUNDS = 5,  /* a kernel met an out-of-range block or slot id and skipped it */
  GK_ERR_TIMEOUT = 6,        /* a kernel's bounded wait ran out; its results are not valid */
  GK_ERR_UNSUPPORTED = 7     /* geometry the kernels were not built for */
} gk_status;

typedef enum gk_backend {
  GK_BACKEND_DENSE = 0,      /* flat paged attention: every request reads its whole context */
  GK_BACKEND_CASCADE = 1     /* shared-prefix contraction + suffix gather + LSE merge */
} gk_backend;

typedef struct gk_pool gk_pool;
typedef struct gk_plan gk_plan;

typedef struct gk_pool_config {
  int32_t num_layers;
  int32_t num_q_heads;
  int32_t num_kv_heads;      /* 1..8, divides num_q_heads */
  int32_t head_dim;          /* 64 or 128; Hq/Hkv in {1,2,4} at 64, {1,2,4,5,8} at 128 */
  int64_t hot_tokens;        /* HOT capacity in tokens */
  int64_t cold_slots;        /* COLD capacity in token slots; a multiple of cold_page_size, at most 2^31 - 1 */
  int32_t cold_page_size;    /* P: tokens per COLD block (GraniKV uses 1; "Paged KV cache" uses 16) */
  int32_t reserved0;
  uint64_t seed;             /* 0: blocks are handed out 0,1,2,...; otherwise in a splitmix64-driven
                                Fisher-Yates order (shuffled physical slots) */
  void *hot_k, *hot_v;       /* device, layouts above; all four NULL = host-only pool (bookkeeping,
                                planning and dispatch work without a GPU) */
  void *cold_k, *cold_v;
} gk_pool_config;

/* ---- pool ------------------------------------------------------------------ */

/* Create a pool over caller-allocated storage.  Does not touch the device
 * contents.  *out is owned by the caller and freed with gk_pool_destroy. */
gk_status gk_pool_create(const gk_pool_config* cfg, gk_pool** out);

/* A pool whose COLD side holds K and V in 4 bits, 4.5 bits an element (5 where a row is
 * padded) instead of 16; HOT stays bf16.  cfg->cold_k is the store of every layer's rows,
 * [num_layers][cold_slots][gk_kv4_row_bytes(Hkv, d)], cold_v NULL; the rest is gk_pool_create's.
 * Each 64 channels of a token's K and of its V, per KV head, are one group: with lo its least
 * value (a bf16 value of the group itself) and span = bf16(greatest - lo),
 *   code = min(15, round((x - lo) * 15 / span)), ties to even,   x is held as lo + code * (span / 15).
 * A span under 2^-100 counts as 0 (every code 0).  A group that holds an infinity or NaN, or whose span
 * reaches 2^120, is held as NaN throughout (lo NaN, span 0).
 * A row: per KV head K's codes then V's (d / 2 bytes each: 32-bit words of eight channels, the first in
 * the lowest four bits; word w has channels 8 w .. 8 w + 7 at d = 64 and 8 (w / 2) + 64 (w % 2) .. + 7 at
 * d = 128, so that a thread's loads hold what its tensor-core fragments take), then per KV head the bf16
 * pairs (lo, span) of K's groups, then of V's; padded to 16 bytes.
 * The block manager, gk_tables_step, the HOT calls and plans work as on any pool; in a plan's summary
 * suffix_ctas are the 4-bit gather's, dense_ctas is 0, and levels never share a launch (gk_pool_set_cascade_mode
 * and gk_pool_set_gather_partition change nothing).  Written by
 * gk_append_kv and gk_append_qkv, read by gk_read_kv and gk_decode_kv4; the other calls that read or
 * write COLD (gk_decode_dense, gk_decode_dense_static, gk_decode_cascade and its stages,
 * gk_sm_speeds_measure, gk_calibrate, gk_dispatch, prompt plans with a COLD context) return
 * GK_ERR_UNSUPPORTED. */
gk_status gk_pool_create_kv4(const gk_pool_config* cfg, gk_pool** out);
/* Bytes of one 4-bit row; 0 for a geometry that no pool takes. */
int64_t gk_kv4_row_bytes(int32_t num_kv_heads, int32_t head_dim);
void gk_pool_destroy(gk_pool* pool);
/* Text of the pool's last error ("" if none); valid until the next call on the pool. */
const char* gk_last_error(const gk_pool* pool);
const char* gk_status_string(gk_status s);

/* ---- HOT pool (GraniKV Section 3.2; first-fit packing, Appendix B.8b) -------- */

/* Reserve prefix_len contiguous tokens: first fit over the address-ordered,
 * coalesced free list, else the bump pointer.  GK_ERR_HOT_FULL when nothing fits
 * (the caller keeps the prefix in COLD; no demotion, Appendix B.10). */
gk_status gk_prefix_alloc(gk_pool* pool, int64_t prefix_len, int64_t* hot_base);
/* Return a prefix's range; it merges with adjacent free ranges, and a range
 * ending at the bump pointer lowers it.  GK_ERR_INVALID for a range held by the
 * prefix cache below (those leave through gk_prefix_unref and eviction). */
gk_status gk_prefix_release(gk_pool* pool, int64_t hot_base);
gk_status gk_hot_stats(const gk_pool* pool, int64_t* bump_top, int64_t* free_ranges,
                       int64_t* free_tokens);

/* HOT prefix cache (GraniKV Section 3.2: a prefix's slab is reference counted;
 * at zero references it becomes evictable, and LRU eviction returns its range
 * to the free list, merged with its neighbours, under memory pressure).
 * key names the prefix's contents (the caller's hash of its tokens).
 * gk_prefix_acquire: a cached key gains a reference and *hit = 1 (its K/V are
 * already in the slab).  Otherwise a range is allocated as gk_prefix_alloc
 * does; while nothing fits, the slab idle longest (no reference since its last
 * use) is evicted and the allocation retried; the new slab has one reference
 * and *hit = 0 (the caller writes its K/V, gk_write_prefix_kv).  GK_ERR_HOT_FULL
 * when nothing fits even after every idle slab is evicted (those stay
 * evicted); GK_ERR_INVALID when key is cached with another prefix_len.  gk_prefix_unref drops one reference (GK_ERR_INVALID if
 * the key holds none).  Acquire and unref both count as a use for the LRU
 * order.  Host only. */
gk_status gk_prefix_acquire(gk_pool* pool, uint64_t key, int64_t prefix_len, int64_t* hot_base, int32_t* hit);
gk_status gk_prefix_unref(gk_pool* pool, uint64_t key);
/* Slabs in the cache, those of them idle, and the tokens the idle ones hold. */
gk_status gk_hot_cache_stats(const gk_pool* pool, int64_t* cached, int64_t* idle, int64_t* idle_tokens);

/* ---- COLD pool block manager ("Paged KV cache", How it works steps 1-4; Code) - */

gk_status gk_seq_create(gk_pool* pool, int32_t* seq);
/* Child shares every block of parent (refcount + 1); nothing is copied. */
gk_status gk_seq_fork(gk_pool* pool, int32_t parent, int32_t* child);
/* Drop one reference to every block of seq; blocks reaching zero return to the
 * free list (most recently freed is handed out first).  The id becomes invalid. */
gk_status gk_seq_release(gk_pool* pool, int32_t seq);
/* Borrow seq's block table (valid until the next call that changes the pool). */
gk_status gk_seq_table(const gk_pool* pool, int32_t seq, const int32_t** table, int32_t* nblocks,
                       int64_t* len);
/* Reserve one slot for each entry of seqs[0..n) in order (a sequence may repeat).
 * slot_mapping_out[i] receives the slot of that token.  When the token lands in
 * a shared partial block, the sequence first takes a fresh block; the pair
 * (shared, fresh) is appended to cow_pairs_out (capacity 2*n int32) and counted
 * in *n_cow.  GK_ERR_OOM: the first failing entry is reported in *n_done and the
 * entries before it stay applied (so the caller can preempt and retry the rest);
 * *n_done = n on success.  n_done may be NULL. */
gk_status gk_seq_append_slots(gk_pool* pool, int32_t n, const int32_t* seqs, int64_t* slot_mapping_out,
                              int32_t* n_cow, int32_t* cow_pairs_out, int32_t* n_done);
/* Block tables of n sequences as one row-major [n][max_blocks] int32 array
 * (rows padded with block 0 past each table's end; the padding is never read
 * because a request reads only its own length) and their lengths in tokens.
 * GK_ERR_INVALID if a table is longer than max_blocks. */
gk_status gk_seq_tables(const gk_pool* pool, int32_t n, const int32_t* seqs, int32_t max_blocks,
                        int32_t* table_out, int32_t* len_out);
gk_status gk_cold_stats(const gk_pool* pool, int64_t* free_blocks, int64_t* total_blocks);
/* A block's references: one per sequence holding it, plus one while it is cached. */
gk_status gk_block_refcount(const gk_pool* pool, int32_t block, int32_t* refcount);

/* COLD prefix caching ("Paged KV cache", How it works, step 5): each full block
 * is keyed by a hash of its parent block's key and its page_size token ids,
 *   key(block i) = H(key(block i - 1), tokens[i P .. i P + P)),  key(block -1) = 0,
 *   H(parent, t[0..P)) = h_P where h_0 = mix(parent + G) and h_{j+1} = mix(h_j XOR t_j * G)
 * (64-bit arithmetic, t_j taken as an unsigned 32-bit value, G = 0x9E3779B97F4A7C15,
 * mix = the output function of splitmix64).  The cache holds one reference on
 * each cached block, so a cached block outlives the sequences that used it;
 * when the free list is empty, taking a block first releases the least
 * recently used cached block that no sequence holds (creation of a cached
 * sequence and caching count as uses).
 * gk_seq_create_cached: a new sequence that starts with the longest chain of
 * cached blocks matching tokens[0..n) block by block (each gains a reference);
 * *n_cached = its length in tokens (a multiple of the page size; their K/V are
 * already in the pool).  The caller appends and writes the remaining tokens.
 * gk_seq_cache_blocks: caches seq's full blocks covering tokens[0..n) (at most
 * its length), skipping keys already cached and blocks cached under another
 * key; *n_new (may be NULL) = blocks added.  Host only. */
gk_status gk_seq_create_cached(gk_pool* pool, int32_t n_tokens, const int32_t* tokens, int32_t* seq, int64_t* n_cached);
gk_status gk_seq_cache_blocks(gk_pool* pool, int32_t seq, int32_t n_tokens, const int32_t* tokens, int32_t* n_new);
/* Blocks in the cache, and those of them no sequence holds (evictable). */
gk_status gk_cold_cache_stats(const gk_pool* pool, int64_t* cached_blocks, int64_t* evictable_blocks);

/* Block tables and slot maps built on the device: the same bookkeeping for rows
 * (one per request slot of an engine) that share no block, without a host loop
 * per token or a copy of tables and slots, so a captured graph can contain it.
 * The caller owns the arrays.  The blocks on the stack are the caller's to hand
 * out: taken from the pool beforehand (a sequence that holds them keeps the
 * pool's own manager off them) and given back when the rows are done.  Forked and
 * cached sequences, whose blocks are shared, stay with gk_seq_*. */
typedef struct gk_tables {
  int32_t num_rows;       /* R, at most 2^20 */
  int32_t max_blocks;     /* row stride of d_table: the most blocks a row can hold */
  int32_t capacity;       /* entries of d_free */
  int32_t reserved0;
  int32_t* d_table;       /* device [R][max_blocks]: block ids, valid up to each row's length */
  int32_t* d_free;        /* device [capacity]: stack of free block ids; the last one below the count is
                             handed out next */
  const int32_t* d_len;   /* device [R]: tokens of each row before the step ... */
  int32_t* d_len_out;     /* ... and after it (may be d_len) */
  const int32_t* d_num_free; /* device [1]: ids on the stack before the step ... */
  int32_t* d_num_free_out;   /* ... and after it (may be d_num_free) */
  void* d_work;           /* device, GK_TABLES_WORK_PER_ROW * (R + 1) bytes, 16-byte aligned: scratch of a step */
} gk_tables;
#define GK_TABLES_WORK_PER_ROW 32

/* One step.  First every row r with d_release[r] != 0 (d_release NULL: none) gives
 * its blocks back, in row order, and has length 0 (gk_seq_release).  Then every
 * row r, in row order, gets d_add[r] tokens (gk_seq_append_slots): the slots of
 * all rows' tokens follow one another in d_slot_mapping [n_slots] (gk_append_kv's
 * input), places past the last token are -1.  When the stack runs empty, the token
 * that needed the next block and every later one are not placed: their slots are
 * -1, and d_done[r] tells how many tokens of each row were.  Lengths, tables, the
 * stack and the slots come out bit for bit as from those calls.
 * d_release, d_add, d_done: device int32 [R]; d_slot_mapping: device int64.
 * A row with a negative length or add, a table too long for its row or for
 * max_blocks after the append, or tokens past n_slots appends nothing; an id on
 * the stack outside the pool gives slots of -1; a count outside [0, capacity], or
 * releases past it, counts as an empty stack or releases nothing: each is reported
 * as GK_ERR_DEVICE_BOUNDS by gk_device_error().  Nothing happens when R = 0.  Calls
 * that share any of the arrays must be ordered.  The pool's device must be the
 * current one (else GK_ERR_INVALID). */
gk_status gk_tables_step(gk_pool* pool, void* stream, const gk_tables* t, const int32_t* d_release,
                         const int32_t* d_add, int64_t n_slots, int64_t* d_slot_mapping, int32_t* d_done);

/* ---- KV writes (device) ---------------------------------------------------- */

/* reshape_and_cache ("Paged KV cache", step 1) for one layer: first copy every
 * copy-on-write pair's whole source block to its destination block, then write
 * token i's K and V [Hkv][d] to COLD slot d_slot_mapping[i].
 * d_slot_mapping: device int64 [n]; d_k, d_v: device bf16 [n][Hkv][d];
 * d_cow_pairs: device int32 [n_cow][2] (src, dst) or NULL when n_cow = 0.
 * Out-of-range slots or blocks are skipped and reported as GK_ERR_DEVICE_BOUNDS
 * by gk_device_error().  On a 4-bit pool the rows are encoded (gk_pool_create_kv4); d_k and d_v are then
 * 16-byte aligned and the pool's device the current one (else GK_ERR_INVALID). */
gk_status gk_append_kv(gk_pool* pool, void* stream, int32_t layer, int32_t n, const int64_t* d_slot_mapping,
                       const void* d_k, const void* d_v, int32_t n_cow, const int32_t* d_cow_pairs);
/* Write prefix tokens [t0, t0+n) of one layer into the HOT slab at hot_base
 * (a range from gk_prefix_alloc of prefix_len tokens).  d_k, d_v: device bf16
 * [n][Hkv][d] (token-major, the same input layout as gk_append_kv). */
gk_status gk_write_prefix_kv(gk_pool* pool, void* stream, int32_t layer, int64_t hot_base,
                             int64_t prefix_len, int64_t t0, int64_t n, const void* d_k, const void* d_v);

/* ---- from a layer's projections to its cache and attention (device) ------------ */

/* The rows of n tokens between the q, k, v projection of a layer and its attention: each head of q and k
 * is normed, then rotated by its token's position.  The pages' caches hold keys after the rotation
 * (queries and keys reach them post-RoPE) and leave both to the engine.
 *   norm (weight not NULL):  x <- x / sqrt(mean_i x_i^2 + eps) * weight
 *   rotation of the first rot_dim channels, with (c, s) the cosine and sine of pair i at the position:
 *     (x_a, x_b) <- (x_a c - x_b s, x_b c + x_a s),  (a, b) = (i, i + rot_dim / 2), or (2 i, 2 i + 1)
 *     where interleaved; the channels from rot_dim on pass.
 * Everything is computed in fp32 and rounded to bf16 once.  Where a token's position is outside
 * [0, num_positions), nothing of the token is written, and it is reported as GK_ERR_DEVICE_BOUNDS by
 * gk_device_error(). */
typedef struct gk_qkv {
  int32_t num_tokens;         /* n, at most 2^27 */
  int32_t rot_dim;            /* 0 (no rotation) to head_dim, a multiple of 16 */
  int32_t interleaved;        /* 0 or 1 */
  float eps;                  /* of the norms, >= 0 */
  int64_t num_positions;      /* rows of d_cos_sin */
  const float* d_cos_sin;     /* device fp32 [num_positions][rot_dim], 16-byte aligned: rot_dim / 2 cosines,
                                 then as many sines; NULL when rot_dim is 0 */
  const int32_t* d_positions; /* device [n]; NULL when rot_dim is 0 */
  const void* d_q_weight;     /* device bf16 [d], 16-byte aligned, or NULL: no norm of queries */
  const void* d_k_weight;     /* ... of keys */
  const void* d_q;            /* device bf16 [n][Hq][d], 16-byte aligned like all rows here; NULL: no queries */
  const void* d_k;            /* device bf16 [n][Hkv][d] */
  const void* d_v;            /* device bf16 [n][Hkv][d] (gk_append_qkv) */
  void* d_q_out;              /* device bf16 [n][Hq][d], may be d_q with its stride; NULL when d_q is */
  void* d_k_out;              /* device bf16 [n][Hkv][d], may be d_k with its stride; gk_append_qkv: may be NULL */
  int64_t q_stride;           /* elements from one token's row to the next (views of a fused projection): */
  int64_t k_stride;           /* a multiple of 8, at least heads * d; 0 = packed rows */
  int64_t v_stride;
  int64_t q_out_stride;
  int64_t k_out_stride;
} gk_qkv;                     /* outputs overlap no input but their own, row for row */

/* q and k of n tokens, normed and rotated, to d_q_out and d_k_out (d_v is not read).  d_q or d_k may be
 * NULL with its output.  GK_ERR_INVALID for missing or misaligned pointers, a stride or count that does not
 * fit, a negative eps; GK_ERR_UNSUPPORTED for a rot_dim that is no multiple of 16 or above head_dim.  May
 * be captured.  The pool gives the geometry; its device must be the current one (else GK_ERR_INVALID). */
gk_status gk_qk_norm_rope(gk_pool* pool, void* stream, const gk_qkv* x);
/* The same, and the tokens' K (normed and rotated) and V into the slots of one layer's COLD cache,
 * in place of gk_qk_norm_rope and gk_append_kv: one pass over the projection's output.  d_k and d_v are
 * required, queries and d_k_out optional.  Copy-on-write pairs are copied first.  Slots are distinct.
 * Out-of-range slots or blocks are skipped and reported as by gk_append_kv (the token's q and k rows are
 * still written).  On a 4-bit pool the stored keys are the codes of the bf16 keys that d_k_out gets. */
gk_status gk_append_qkv(gk_pool* pool, void* stream, int32_t layer, const gk_qkv* x, const int64_t* d_slot_mapping,
                        int32_t n_cow, const int32_t* d_cow_pairs);
/* K and V of n COLD slots of one layer, as bf16 rows: a context that moves to a HOT prefix
 * (gk_write_prefix_kv), or a 4-bit context that the next chunk of its prompt attends there.  d_slot_mapping:
 * device int64 [n], n at most 2^27, any order, slots may repeat.  d_k, d_v: device bf16 [n][Hkv][d], 16-byte aligned, with
 * token strides as in gk_qkv.  4-bit rows give bf16(lo + code * (span / 15)), the bracket and the sum rounded to
 * fp32.  An out-of-range slot gives zeros and is reported as GK_ERR_DEVICE_BOUNDS by gk_device_error().
 * May be captured.  The pool's device must be the current one (else GK_ERR_INVALID). */
gk_status gk_read_kv(gk_pool* pool, void* stream, int32_t layer, int64_t n, const int64_t* d_slot_mapping, void* d_k,
                     void* d_v, int64_t k_stride, int64_t v_stride);

/* ---- one decode step ------------------------------------------------------- */

typedef struct gk_batch {
  int32_t num_requests;           /* B */
  int32_t max_blocks;             /* row stride of d_block_table */
  const int64_t* prefix_hot_base; /* host [B]: HOT base of the request's shared prefix, -1 = none */
  const int32_t* prefix_len;      /* host [B]: its length in tokens (0 when the base is -1) */
  const int32_t* suffix_len;      /* host [B]: tokens the request reads from COLD */
  const int32_t* d_block_table;   /* device [B][max_blocks]: COLD block ids of each request */
  const void* d_q;                /* device bf16 [B][Hq][d] (this layer's queries) */
  float* d_out;                   /* device fp32 [B][Hq][d] */
  float* d_lse;                   /* device fp32 [B][Hq], natural log; may be NULL */
  /* Optional fused append ("Paged KV cache", How it works step 2: reshape_and_cache),
   * both NULL or both set: this layer's new token of every request, device bf16
   * [B][Hkv][d].  Each request's last COLD token (suffix position suffix_len - 1,
   * reserved by gk_seq_append_slots and present in the block table) is then read
   * from here instead of the pool, and the decode writes it into the pool slot the
   * table gives -- what gk_append_kv would have written -- so no separate scatter
   * launch is needed.  Copy-on-write pairs of the step must be copied first
   * (gk_append_kv with n = 0).  Requests with suffix_len 0 are unaffected. */
  const void* d_new_k;
  const void* d_new_v;
} gk_batch;

typedef struct gk_plan_summary {
  int32_t num_requests;
  int32_t num_groups;             /* distinct HOT prefixes in the step */
  int32_t max_m_eff;              /* largest M_eff = B_g * Hq/Hkv over the groups (GraniKV Eq. 2) */
  int32_t prefix_ctas;            /* cascade prefix-kernel CTAs per layer */
  int32_t suffix_ctas;            /* suffix-gather CTAs per layer */
  int32_t dense_ctas;             /* flat-gather CTAs per layer */
  int32_t num_partials;           /* partial (O, LSE) states the merge combines per layer */
  int32_t dense_merge;            /* 1 if gk_decode_dense launches a merge (a request spans CTAs) */
  int64_t prefix_bytes;           /* algorithmic bytes per layer: HOT K+V read once per group */
  int64_t prefix_flops;           /* 4 * B_g * Hq * Lp * d summed over groups */
  int64_t suffix_bytes;           /* COLD K+V of all suffixes */
  int64_t dense_bytes;            /* K+V of every request's whole context */
  int32_t cascade_split;          /* 1: gk_decode_cascade runs the prefix items (prefix_ctas SMs) and
                                     the suffix gather (suffix_ctas SMs) side by side in one launch;
                                     0: one after the other, each over every SM */
  int32_t prefix_tiles_per_item;  /* 128-key tiles of the longest prefix work item */
  int32_t prefix_kernel;          /* prefix work items: GK_PREFIX_TENSOR or GK_PREFIX_WARP */
  int32_t prefix_rows_per_item;   /* stacked query rows per prefix work item: 256 or 128 */
  int32_t prefix_row_groups;      /* warp items: 16-row groups of the fullest item, rounded up to
                                     1, 2, 4 or 8; 0 for tensor-core items */
  int32_t prefix_ctas_gather;     /* split plans: 1 when the prefix CTAs also gather a share of the
                                     suffix after their items, 0 when only the other CTAs gather */
  int32_t sm_slots;               /* split plans: 1 when the slots are planned per SM from the pool's
                                     SM speeds (gk_pool_set_sm_speeds), 0 when CTA b takes slot b */
} gk_plan_summary;

/* Plan one decode step: group requests by HOT prefix (stable, first appearance),
 * split the prefix contraction and the gathers into balanced CTA work lists,
 * and lay out the partial states.  The grouping is GraniKV Section 3.6's: the
 * requests that share one HOT prefix stack their B_g * Hq/Hkv query rows per KV
 * head into one matrix (M_eff of Eq. 2, which also drives gk_dispatch).  Depends
 * only on the host arrays of the batch, which every layer of a step shares, so
 * one plan serves every layer of the step.  When the pool has device
 * storage the plan's tables are copied to the device on `stream` and scratch
 * for the partial states is allocated (owned by the plan).  Calls that use a
 * plan must be ordered on one stream. */
gk_status gk_plan_build(gk_pool* pool, const gk_batch* batch, void* stream, gk_plan** out);
/* Re-plan an existing plan for the next step (same pool), reusing its host and
 * device buffers when they are large enough.  Must be called on the stream the
 * plan's earlier work was enqueued on: the new tables are copied after that work. */
gk_status gk_plan_update(gk_plan* plan, const gk_batch* batch, void* stream);
/* Frees the plan's buffers; its enqueued work must have completed. */
void gk_plan_destroy(gk_plan* plan);
gk_status gk_plan_info(const gk_plan* plan, gk_plan_summary* out);
/* The gather partition of a plan (its host copy): which tokens each CTA gathers.
 * dense = 0: the cascade suffix partition, 1: the flat one.  The counts come
 * first: *n_ctas gather CTAs and *n_segs segments.  Then, when begin and segs
 * are not NULL, begin[0 .. n_ctas] receives the offsets of each CTA's
 * segments (CTA b: [begin[b], begin[b + 1])) and segs[4 * i .. 4 * i + 3]
 * segment i: request, first token, end token (in the request's own order: the
 * dense partition counts the HOT prefix first), and the partial state it
 * writes (-1: the request's output).  Host only; GK_ERR_INVALID for a NULL
 * plan or count pointer. */
gk_status gk_plan_segments(const gk_plan* plan, int32_t dense, int32_t* n_ctas, int32_t* n_segs, int32_t* begin,
                           int32_t* segs);

/* Flat paged attention (the dense backend): each request attends its prefix
 * (read from HOT, once per request) and its COLD suffix in one online-softmax
 * pass; writes d_out and d_lse of the batch for this layer.  This is the decode
 * of "Paged KV cache", How it works step 3 (the kernel walks each sequence's
 * block table and reads its K/V in place, token slot by slot), and the
 * baseline GraniKV compares against (Section 4, the SGLang default: every
 * request re-reads the shared prefix).  A request split over several CTAs is
 * merged by GraniKV Eq. 1 (gk_plan_summary.dense_merge). */
gk_status gk_decode_dense(gk_pool* pool, void* stream, int32_t layer, const gk_batch* batch,
                          const gk_plan* plan);
/* Cascade backend: (a) per prefix group and KV head, all query rows sharing the
 * prefix are stacked into one QK^T / PV contraction on the tensor cores, read
 * once from HOT (GraniKV Section 2.3, shared-prefix matmul; Section 3.5);
 * (b) the suffix is gathered through the block table; (c) the partial states
 * are merged by log-sum-exp (GraniKV Eq. 1).  A split plan
 * (gk_plan_summary.cascade_split) runs (a) and (b) in one launch on disjoint
 * SMs, then (c); otherwise (a), (b), (c) are three launches.  Both give the
 * same bits as the three stage calls below. */
gk_status gk_decode_cascade(gk_pool* pool, void* stream, int32_t layer, const gk_batch* batch,
                            const gk_plan* plan);
/* Allocation-free dense decode.  No counterpart in the paper: it exists for
 * callers that cannot allocate device memory while serving -- an engine that
 * hands all free HBM to its KV pool at start-up, or one whose allocator is
 * owned by a framework that rejects allocations made outside it.  Same result
 * as gk_plan_build + gk_decode_dense on this batch (see those calls for the
 * arguments), but the work tables and split-K partial states live in one
 * 8 MiB array compiled into libgk (every GPU that loads the library keeps it
 * until the process exits) and no call allocates device or pinned memory.
 *  - The first call on each device looks the array's address up
 *    (cudaGetSymbolAddress) with that device current; make that first call
 *    before any stream capture.  The pool's device must be the current device
 *    (else GK_ERR_INVALID).
 *  - Each call copies its work tables from host memory that it frees on
 *    return, so on a stream that is capturing it does nothing and returns
 *    GK_ERR_UNSUPPORTED.
 *  - A batch whose tables and partial states exceed 8 MiB is refused with
 *    GK_ERR_INVALID (gk_last_error gives the bytes needed); use the plan path.
 *  - Every call reuses the same array: calls that overlap on the GPU (two
 *    streams, or two pools on one device) race and give wrong results; order
 *    them on one stream.  Nothing in the array needs to start at zero.
 *  - The pool must already have done device work (any KV write), which is when
 *    its error word is created; otherwise GK_ERR_INVALID. */
gk_status gk_decode_dense_static(gk_pool* pool, void* stream, int32_t layer, const gk_batch* batch);
/* Stages (a) and (b) of gk_decode_cascade as the plan arranges them: one split
 * launch, or the prefix then the suffix kernel.  gk_decode_cascade is exactly
 * this followed by gk_cascade_merge. */
gk_status gk_cascade_levels(gk_pool* pool, void* stream, int32_t layer, const gk_batch* batch,
                            const gk_plan* plan);
/* The three stages of gk_decode_cascade, for callers that time them or run
 * (a) and (b) on two streams: the prefix and suffix stages write disjoint
 * partial states, and the merge must follow both.  They run the plan's work
 * lists (for a split plan: prefix_ctas long items, suffix_ctas gather CTAs). */
gk_status gk_cascade_prefix(gk_pool* pool, void* stream, int32_t layer, const gk_batch* batch,
                            const gk_plan* plan);
gk_status gk_cascade_suffix(gk_pool* pool, void* stream, int32_t layer, const gk_batch* batch,
                            const gk_plan* plan);
gk_status gk_cascade_merge(gk_pool* pool, void* stream, int32_t layer, const gk_batch* batch,
                           const gk_plan* plan);

/* One layer of a planned decode step over a 4-bit pool: each request's query attends its HOT prefix (bf16)
 * and its COLD tokens as the codes hold them, with s_j = q.k_j / sqrt(d):
 *   out = sum_j e^(s_j) v_j / Z,   lse = ln Z,   Z = sum_j e^(s_j).
 * The plan is gk_plan_build's on the 4-bit pool: prefix items, the COLD gather and the log-sum-exp join one
 * after the other (a join is launched only where a request has several partial states or no token).
 * d_out: device bf16 [B][Hq][d], 16-byte aligned, like the batch's d_q; the batch's d_out is not used, d_lse
 * may be NULL, d_new_k and d_new_v must be (GK_ERR_UNSUPPORTED: append first, gk_append_qkv).  Products and sums
 * are held in fp32; the weights are rounded to bf16 over the prefix and to fp16, times the group's span, over COLD,
 * the output to bf16 at the end.  (fp16 holds the products of weight and span scaled by a power of two: one below 2^-24 of the
 * largest in its 64 channels, over the queries that share the KV head, is off by up to 2^-35 of that largest.)
 * A score over COLD is a part from lo and a part from codes, each in fp32, which may cancel: it is off by up to 2^-18 of
 * sum_c |q_c| (|lo| + span) / sqrt(d), and lse by as much as the key whose sum is largest.
 * Queries of magnitude up to 2^100 are in range; a row that has a query of infinity or NaN, or attends a key that is held as NaN, comes out NaN, lse
 * too; channels whose attended values include NaN come out NaN.  A request without a token gives 0 and
 * minus infinity.  An out-of-range block id counts as zero K and V and is reported as GK_ERR_DEVICE_BOUNDS
 * by gk_device_error().  The batch's lengths and HOT bases are the plan's; only its device pointers and
 * max_blocks are read.  May be captured.  The pool's device must be the current one (else GK_ERR_INVALID). */
gk_status gk_decode_kv4(gk_pool* pool, void* stream, int32_t layer, const gk_batch* batch, const gk_plan* plan,
                        void* d_out);

/* ---- one prompt step ------------------------------------------------------- */

/* The new tokens of every request of a step: whole prompts, turns behind a
 * cached context, or chunks of prompts, of different lengths.  Request r has
 * n = new_len[r] new tokens, whose rows of q, k, v, out and lse follow those of
 * request r - 1 (packed; T = the sum of new_len rows), a HOT prefix of
 * prefix_len[r] tokens and context_len[r] tokens in COLD.  New token i attends
 * the whole HOT prefix, the COLD tokens and the new tokens 0 .. i, in that order
 * of positions; n = 0 is allowed (no rows).  The pages leave the prompt's own
 * attention to the engine ("Paged KV cache", How it works, step 1 only writes
 * its K/V; GraniKV Section 3.2 fills the HOT slab from it). */
typedef struct gk_prompt_batch {
  int32_t num_requests;           /* B */
  int32_t max_blocks;             /* row stride of d_block_table */
  const int32_t* new_len;         /* host [B] */
  const int64_t* prefix_hot_base; /* host [B]: HOT base, -1 = none; NULL = none for any request */
  const int32_t* prefix_len;      /* host [B]: 0 when the base is -1; NULL exactly when the base is NULL */
  const int32_t* context_len;     /* host [B]: earlier tokens of the request in COLD; NULL = 0 for all */
  const int32_t* d_block_table;   /* device [B][max_blocks]; read where context_len > 0, else may be NULL */
  const void* d_q;                /* device bf16 [T][Hq][d], 16-byte aligned, like the next three */
  const void* d_k;                /* device bf16 [T][Hkv][d]: the new tokens' keys (gk_append_kv's input) */
  const void* d_v;                /* device bf16 [T][Hkv][d] */
  void* d_out;                    /* device bf16 [T][Hq][d] */
  float* d_lse;                   /* device fp32 [T][Hq], natural log; may be NULL */
  /* out and lse overlap no input */
  int64_t q_stride;               /* elements from one token's row to the next (views of a fused q k v */
  int64_t k_stride;               /* projection): a multiple of 8, at least heads * d; 0 = packed rows */
  int64_t v_stride;
  int64_t out_stride;
} gk_prompt_batch;

typedef struct gk_prompt_plan gk_prompt_plan;

typedef struct gk_prompt_plan_summary {
  int64_t tokens;                 /* T */
  int64_t flops;                  /* 4 * d * Hq * (visible row-key pairs per query head), per layer */
  int64_t bytes;                  /* per layer: q, k, v, out and lse once, each HOT prefix once, COLD tokens */
  int32_t items;                  /* work items: two 128-row query tiles x one KV head x a range of key tiles */
  int32_t ctas;                   /* CTAs that run them */
  int32_t stacked_requests;       /* requests whose HOT keys are read by items that stack several requests' rows */
  int32_t partials;               /* partial states the join combines (0: no join launch) */
  int32_t max_pieces;             /* most items over one block of rows' keys */
  int32_t max_cta_tiles;          /* 128-key tiles of the CTA with the most */
  int64_t scratch_bytes;          /* of the partial states: 4 * (d + 1) for each row of each, at most 32 states a row */
} gk_prompt_plan_summary;

/* Plan a prompt step: cut the rows into items, balance them over the SMs by their key
 * tiles (long key ranges of steps with few rows are split and joined by log-sum-exp,
 * GraniKV Eq. 1; neighbouring requests with the same HOT prefix and few rows each are
 * stacked over it, Section 2.3; requests of one prefix that others stand between are
 * not, and each reads it by itself: 64 requests of 1 to 16 tokens over four prefixes
 * of 16384 take five times the key tiles in round robin that they take sorted by
 * prefix).  Depends only on the host arrays, so one plan serves every layer and may
 * be replayed from a captured graph.  Tables and partial states are owned by the
 * plan; calls that use a plan must be ordered on one stream.  GK_ERR_INVALID for a
 * negative length, a HOT prefix that is not live with that length, a context longer
 * than its block-table row, or more than 2^31 - 1 tokens.  Allocates device memory
 * (the tables, some hundred bytes an item, and scratch_bytes; a plan that grows takes
 * up to half as much again, and keeps it until it is destroyed) and uploads from a
 * buffer that the next plan rewrites: on a stream that is capturing it does nothing
 * and returns GK_ERR_UNSUPPORTED.  The pool's device must be the current one, here
 * and in gk_prompt_attn (else GK_ERR_INVALID). */
gk_status gk_prompt_plan_build(gk_pool* pool, const gk_prompt_batch* batch, void* stream, gk_prompt_plan** out);
/* Re-plan for the next step, reusing the buffers; on the stream of the plan's earlier
 * work.  A graph captured with the plan holds the launch of the step planned then:
 * after an update it must not be replayed, but captured again. */
gk_status gk_prompt_plan_update(gk_prompt_plan* plan, const gk_prompt_batch* batch, void* stream);
/* Frees the plan's buffers; its enqueued work must have completed. */
void gk_prompt_plan_destroy(gk_prompt_plan* plan);
gk_status gk_prompt_plan_info(const gk_prompt_plan* plan, gk_prompt_plan_summary* out);
/* The plan's work list (its host copy).  The counts come first: *n_ctas CTAs and
 * *n_items items.  Then, when begin and items are not NULL, begin[0 .. n_ctas]
 * receives the offsets of each CTA's items and items[8 * i .. 8 * i + 7] item i:
 * request (the first of a stacked run), tokens of the stacked run (0: an item of
 * one request), KV head, first token (of the request or run; an item covers
 * 2 * floor(128 * Hkv / Hq)), first key tile, key tiles (128 keys each: the HOT
 * prefix's, then COLD's, then the new tokens'), partial state (-1: the output),
 * and the HOT prefix's tiles.  Host only. */
gk_status gk_prompt_plan_items(const gk_prompt_plan* plan, int32_t* n_ctas, int32_t* n_items, int32_t* begin,
                               int32_t* items);
/* Attention of one layer of a planned prompt step: with s_j = q.k_j / sqrt(d) over
 * the keys the row attends, out = sum_j e^(s_j) v_j / Z and lse = ln Z, Z = sum_j
 * e^(s_j).  Products and sums are held in fp32; the weights are rounded to bf16
 * before the product with V, the output to bf16 at the end.  Out of range are scores
 * of magnitude 2^28 and more, which fp32 holds to whole tens only, and finite values
 * of V of magnitude 2^63 and more, whose products with weights of up to 2^64 before
 * the division by Z could overflow.  A row that attends a score of NaN (or of plus
 * infinity) comes out NaN, lse too; where every score is minus infinity out is 0 and
 * lse minus infinity.  Keys a row does not attend contribute nothing, whatever their
 * K and V hold (infinities and NaN included).  Reads COLD through the block table (an
 * out-of-range block id counts as zero K and V and is reported as
 * GK_ERR_DEVICE_BOUNDS by gk_device_error()) and does not write the pool:
 * gk_append_kv (or gk_write_prefix_kv) stores the new tokens, before or after.  The
 * batch's lengths and HOT bases are the plan's; only its device pointers and strides
 * are read.  May be captured. */
gk_status gk_prompt_attn(gk_pool* pool, void* stream, int32_t layer, const gk_prompt_batch* batch,
                         const gk_prompt_plan* plan);

/* ---- per-step dispatch (GraniKV Section 3.6, Eq. 2) -------------------------- */

typedef struct gk_cost_model {
  double c_flat_us;               /* fixed cost of the dense backend per layer */
  double bw_flat_gbs;             /* its sustained gather bandwidth */
  double c_cascade_us;            /* fixed cost of the cascade backend per layer */
  double bw_prefix_gbs;           /* bandwidth bound of the prefix contraction (HOT reads) */
  double bw_suffix_gbs;           /* suffix gather bandwidth over every SM */
  double c_merge_us;              /* merge cost per (request, query head) */
  double prefix_tile_us;          /* one 128-key tile of a 256-row prefix work item on one SM */
  double prefix_item_us;          /* fixed cost of a prefix work item (of each wave of them) */
  double gather_sm_gbs;           /* suffix gather bandwidth one SM sustains (split plans) */
  double c_gather_us;             /* fixed cost of a separate suffix-gather launch (sequential plans) */
  double prefix_tile_split_us;    /* prefix_tile_us for an item of a split plan, which runs beside a
                                     gather that keeps HBM busy (its K/V tiles wait longer) */
  double warp_tile_us;            /* one 128-key tile of a warp-MMA prefix item alone: the part that does
                                     not grow with its rows ... */
  double warp_group_us;           /* ... plus this much per group of 16 rows (rounded up to 1, 2, 4, 8) */
  double warp_item_us;            /* fixed cost of a warp-MMA prefix item (of each wave of them) */
  double warp_split_ratio;        /* a warp item's tile beside the gather of a split plan, over alone */
  double prefix_cta_ramp_us;      /* split plans: a prefix CTA starts gathering this long after its item */
  double prefix_cta_gather_ratio; /* ... and gathers at this fraction of a gather-only CTA's rate */
  double c_merge_state_us;        /* merge cost per partial state of a request (a merge warp's round trips) */
  double prefix_item_split_us;    /* fixed cost of a tensor-core prefix item inside a split launch */
  double warp_item_split_us;      /* fixed cost of a warp-MMA prefix item inside a split launch */
  double prefix_item_crowd_us;    /* ... plus this much per prefix item of the launch (their first loads
                                     contend with each other) */
  double split_gather_ratio_tensor; /* gather rate in a split launch of tensor-core items, over gather_sm
                                     (that launch's 320-thread blocks hold the gather to fewer registers) */
  double c_gather_split_us;       /* fixed cost of the gather inside a split launch: when its gather-only
                                     CTAs start (c_gather_us is the stand-alone gather launch's) */
  double split_tensor_us;         /* what a split launch of tensor-core items costs over one of warp-MMA
                                     items (its 320-thread blocks, tensor memory, tensor maps) */
} gk_cost_model;

/* Predict both backends for the plan and pick the smaller:
 *   T_dense   = c_flat + dense_bytes / bw_flat
 *   T_cascade = c_cascade + T_levels + c_merge * B * Hq + c_merge_state * num_partials / B
 * with C = gk_plan_summary.prefix_tiles_per_item key tiles per prefix item,
 * (tile, tile_split, item) = (prefix_tile, prefix_tile_split, prefix_item) for
 * tensor-core items and, for warp-MMA items (gk_plan_summary.prefix_kernel),
 * tile = warp_tile + R * warp_group with R = gk_plan_summary.prefix_row_groups,
 * tile_split = warp_split_ratio * tile and item = warp_item; item_split =
 * (prefix_item_split or warp_item_split) + prefix_item_crowd * prefix_ctas is an
 * item's fixed cost in a split launch; and
 *   sequential plan (W = ceil(prefix_ctas / SMs) waves of prefix items):
 *     T_levels = max(prefix_bytes / bw_prefix, W * (C * tile + item))
 *                + c_gather + suffix_bytes / bw_suffix
 *   split plan (see gk_plan_summary.cascade_split; it = C * tile_split + item_split,
 *   n = prefix_ctas, A = SMs - n gather-only CTAs, G = suffix_bytes / gather_sm
 *   the gather's SM-time (gather_sm times split_gather_ratio_tensor for
 *   tensor-core items), e = prefix_cta_gather_ratio, r = prefix_cta_ramp):
 *     T_gather = (G + A * c_gather + n * e * (it + r)) / (A + n * e)
 *                when the prefix CTAs gather too (gk_plan_summary.prefix_ctas_gather),
 *              = c_gather + G / A otherwise, and at least c_gather + suffix_bytes / bw_suffix;
 *     T_levels = max(it, T_gather, (suffix_bytes + prefix_bytes) / bw_suffix)
 *   (gather-only CTAs start after c_gather, prefix CTAs r after their items,
 *   and all end together; the gather is held to HBM as a whole, and so is the launch).
 * A plan without prefix work has no prefix term, one without suffix work no
 * gather term.  GraniKV's M_eff (Eq. 2) enters through the items: a group of
 * M_eff stacked rows gives ceil(M_eff / rows per item) items per KV head and key
 * split.  The plan has already chosen the prefix kernel and the arrangement
 * with the smallest predicted time (GraniKV Section 3.6's routing between its
 * two prefix kernels, with the threshold replaced by the measured model), so
 * this call completes the three-way choice: flat, cascade over tensor-core
 * items, cascade over warp-MMA items.  Dense is chosen only when strictly
 * faster; a negative prediction (a negative c_cascade on a tiny step) counts as
 * zero.  Host only. */
gk_status gk_dispatch(const gk_pool* pool, const gk_plan* plan, gk_backend* choice, double* t_dense_us,
                      double* t_cascade_us);
gk_status gk_cost_model_set(gk_pool* pool, const gk_cost_model* cm);

/* Cascade arrangement of the plans the pool builds from now on.
 *  GK_CASCADE_AUTO (default): split when the cost model predicts it faster.
 *  GK_CASCADE_SEQUENTIAL: prefix items over every SM, then the suffix gather.
 *  GK_CASCADE_SPLIT: prefix items beside the suffix gather in one launch, with
 *    tiles_per_item 128-key tiles per item (0: the cost model's best split).
 *    A step without prefix or suffix work, or whose items would leave no SM
 *    for the gather, is planned sequentially.
 * The choice changes the work lists and the partial states, not the
 * attention computed.  Host only.  GK_ERR_INVALID for an unknown mode or a
 * negative tiles_per_item. */
typedef enum gk_cascade_mode {
  GK_CASCADE_AUTO = 0,
  GK_CASCADE_SEQUENTIAL = 1,
  GK_CASCADE_SPLIT = 2
} gk_cascade_mode;
gk_status gk_pool_set_cascade_mode(gk_pool* pool, gk_cascade_mode mode, int32_t tiles_per_item);

/* How the stand-alone gathers (the flat backend, and the suffix of a sequential
 * cascade plan) split their tokens over CTAs, in the plans the pool builds from
 * now on (a split cascade plan always gives each SM one slot of the stream).
 *  GK_PARTITION_STREAM (default): the requests' tokens as one stream cut into
 *    equal quotas (at least 64 tokens, multiples of 16) over at most one CTA per
 *    SM; a quota that crosses a request boundary yields one segment per request.
 *  GK_PARTITION_PER_REQUEST: Tangram's ahead-of-time partitioning (Algorithm 1,
 *    with requests as its head groups and their tokens as budgets): target
 *    tau = max(1, ceil(total / SMs)); request r gets S_r = max(1, ceil(n_r / tau))
 *    segments of its own tokens, the first n_r mod S_r of them one token longer,
 *    one CTA each (so up to SMs + B CTAs, in waves).
 * The choice changes the work lists and the partial states, not the attention
 * computed.  Host only.  GK_ERR_INVALID for an unknown value. */
typedef enum gk_gather_partition {
  GK_PARTITION_STREAM = 0,
  GK_PARTITION_PER_REQUEST = 1
} gk_gather_partition;
gk_status gk_pool_set_gather_partition(gk_pool* pool, gk_gather_partition partition);

/* Which kernel runs the shared-prefix level of the cascade in the plans the
 * pool builds from now on.  GraniKV Section 3.5 pairs two: the shared-prefix
 * matmul ("GKV-dense": every row sharing the prefix stacked into one
 * tensor-core contraction) and the cascade backend's level-0 kernel
 * ("GKV-cascade": a FlashAttention-style tiled online softmax that reads the
 * prefix once), and Section 3.6 routes between them on M_eff.
 *  GK_PREFIX_AUTO (default): per step, the one whose cascade the cost model
 *    predicts faster, the tensor-core items only when predicted at least 10 %
 *    faster (their predictions at small steps run low) and never when every
 *    group stacks at most 64 rows per KV head (M_eff <= 64, which a tensor-core
 *    item pads to 256).
 *  GK_PREFIX_TENSOR: tcgen05 items of 256 stacked rows (two 128-row tiles).
 *  GK_PREFIX_WARP: warp-MMA items of 128 stacked rows (8 warps x 16 rows), no
 *    tensor memory; meant for small M_eff.
 * Either kind writes the same partial states (one per request, query head and
 * key split); the arrangement (gk_pool_set_cascade_mode) applies to both.
 * Host only.  GK_ERR_INVALID for an unknown value. */
typedef enum gk_prefix_kernel {
  GK_PREFIX_AUTO = 0,
  GK_PREFIX_TENSOR = 1,
  GK_PREFIX_WARP = 2
} gk_prefix_kernel;
gk_status gk_pool_set_prefix_kernel(gk_pool* pool, gk_prefix_kernel kernel);
/* SM-aware split launches (no counterpart in the pages: they assume a uniform
 * GPU).  On GB300 some SMs gather COLD rows 5-10 % slower than others, the same
 * from launch to launch, so equal gather slots end at different times and the
 * launch waits for the slowest.  With SM speeds set, split plans size each
 * SM's slot by its speed, give the prefix items to the slowest SMs (the longest
 * item to the slowest), and the split launch's CTA on SM s takes the slot
 * planned for s (an atomic claim per launch; a slot already taken sends the CTA
 * to the next free one, so every slot is run exactly once whatever SMs the
 * CTAs land on).  The results are the same attention whichever slots run where;
 * the partial-state boundaries, and so the last bits, follow the speeds.
 *  - gk_pool_set_sm_speeds: n speeds (relative; any positive scale) for SM ids
 *    0 .. n-1, n = the device's SM count (152 for a pool without device
 *    storage, which plans as for one GB300); n = 0 clears them (plans as
 *    without).  Host only.  GK_ERR_INVALID for another n or a speed that is not
 *    positive and finite.  Plans built before keep their slots.
 *  - gk_pool_get_sm_speeds: *n = the count set (0 when none) and, when speeds is
 *    not NULL, the speeds (normalised to mean 1).
 *  - gk_sm_speeds_measure: runs the plan's gather `reps` times on `stream`,
 *    each launch alone, with each CTA's SM id and times recorded by the kernel:
 *    a split plan's own launch (gk_cascade_levels; a slot's rate counts its
 *    gather, after its item, and prefix and gather-only slots are each scaled
 *    to their own mean in the launch) or a sequential plan's stand-alone suffix
 *    gather (gk_cascade_suffix).  An SM's speed is the median over the launches
 *    of the scaled tokens per us of the slots it ran (slots with under a quarter
 *    of the largest one's tokens are left out), normalised to mean 1; SMs
 *    without a sample get 1.  Installs the speeds in the pool and, when speeds
 *    is not NULL, writes them there (dev SM count entries).  The launches write
 *    the plan's partial states (and the outputs of requests one CTA covers) and,
 *    with a fused append, the step's tokens, as the decode calls do.  Blocking;
 *    allocates and frees its own 32 bytes per CTA of device memory.
 *    GK_ERR_INVALID when the plan has no suffix segments or reps is not in
 *    1 .. 64. */
gk_status gk_pool_set_sm_speeds(gk_pool* pool, const float* speeds, int32_t n);
gk_status gk_pool_get_sm_speeds(const gk_pool* pool, float* speeds, int32_t* n);
gk_status gk_sm_speeds_measure(gk_pool* pool, void* stream, int32_t layer, const gk_batch* batch,
                               const gk_plan* plan, int32_t reps, float* speeds);
gk_status gk_cost_model_get(const gk_pool* pool, gk_cost_model* cm);
/* Re-fit the cost model on this GPU (GraniKV Section 3.6: the routing rule stays
 * and its numbers are re-fit per GPU; Appendix B.4b's sweep).  Times, with CUDA
 * events on `stream` and L2 emptied before every launch, the flat backend, the
 * suffix gather, the merge, tensor-core and warp-MMA prefix items of several
 * key-tile counts (warp items with 1, 2 and 8 groups of 16 rows), the gather
 * beside long items, and whole cascades, on layer 0 of this pool with a
 * synthetic batch of one shared prefix; fits each gk_cost_model term by least
 * squares (the flat backend's and the suffix gather's terms by relative error,
 * so that the smallest steps count as much as the largest); installs the model in the pool; and, if json_out is not
 * NULL, writes it to that file in gk_cost_model_load's format with the
 * measured points under "measured".  Blocking; a few seconds.
 *  - The pool needs device storage; its K/V contents are read as they are (the
 *    timings do not depend on the values) and never written.  Cases that do not
 *    fit its free HOT and COLD space are skipped; with at least 16384 free HOT
 *    tokens and 262144 free COLD token slots every case runs.  GK_ERR_INVALID
 *    when too few cases fit to fit every term (the model is left as it was).
 *  - HOT ranges, sequences and COLD blocks are taken from the pool's allocators
 *    and given back: afterwards the same blocks are free, though the order in
 *    which free blocks are handed out may differ.  The pool's cascade mode,
 *    prefix kernel and gather partition are restored.
 *  - The calibration's own scratch (queries, outputs, tables, 512 MiB to empty
 *    L2) is allocated with cudaMalloc and freed before returning.
 *  - The terms of the split arrangement (prefix_tile_split_us / prefix_tile_us,
 *    warp_split_ratio, prefix_item_split_us, warp_item_split_us,
 *    prefix_item_crowd_us, prefix_cta_ramp_us, gather_sm_gbs,
 *    split_gather_ratio_tensor, c_gather_split_us, split_tensor_us) and c_cascade_us are fitted
 *    to the whole cascades it times (sequential and split plans, forced and as
 *    the planner arranges them, both prefix kernels, a grid of steps with
 *    16..512-token suffixes, that grid planned again with the first fit): a
 *    coordinate search over candidate values of each term that minimises the
 *    largest plus half the mean relative error of T_cascade, the other terms
 *    held at their own fits.  c_cascade_us may come out negative
 *    (the terms timed alone each carry a launch that the cascade overlaps).
 *    prefix_cta_gather_ratio is set to 1: once it starts, a prefix CTA gathers
 *    at a gather-only CTA's rate. */
gk_status gk_calibrate(gk_pool* pool, void* stream, const char* json_out);
/* Same as gk_cost_model_set from JSON text: {"c_flat_us": .., "bw_flat_gbs": ..,
 * "c_cascade_us": .., "bw_prefix_gbs": .., "bw_suffix_gbs": .., "c_merge_us": ..,
 * "prefix_tile_us": .., "prefix_item_us": .., "gather_sm_gbs": .., "c_gather_us": ..,
 * "prefix_tile_split_us": .., "warp_tile_us": .., "warp_group_us": .., "warp_item_us": ..,
 * "warp_split_ratio": .., "prefix_cta_ramp_us": .., "prefix_cta_gather_ratio": ..,
 * "c_merge_state_us": .., "prefix_item_split_us": .., "warp_item_split_us": ..,
 * "prefix_item_crowd_us": .., "split_gather_ratio_tensor": .., "c_gather_split_us": ..,
 * "split_tensor_us": ..}.
 * Keys left out keep their current values; other keys are skipped. */
gk_status gk_cost_model_load(gk_pool* pool, const char* json);

/* ---- device error word -------------------------------------------------------- */

/* Synchronize `stream`, read and clear the pool's device error word.  *code is
 * GK_OK, GK_ERR_DEVICE_BOUNDS or GK_ERR_TIMEOUT; the return value reports
 * failures of the read itself. */
gk_status gk_device_error(gk_pool* pool, void* stream, int32_t* code);

#ifdef __cplusplus
}
#endif

#endif /* GK_H_ */
