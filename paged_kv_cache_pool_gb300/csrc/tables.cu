// Block tables and slot maps on the device: one step of the COLD block manager
// ("Paged KV cache", How it works, steps 1-3) for rows that share no block.
//
// State: a stack of free block ids, a length and a block-table row per request
// row.  A step releases the flagged rows (their blocks are pushed in row order,
// each row in table order), then appends add[r] tokens to every row in row order:
//   have_r = ceil(len_r / P),  need_r = ceil((len_r + add_r) / P) - have_r,
//   B_r = sum_{q < r} need_q,  block i of row r's new ones = stack[n - 1 - (B_r + i)],
// what gk_seq_release and gk_seq_append_slots do one token at a time: the k-th
// block taken is the k-th from the top.  When the stack is empty the token that
// asks for the next block and every later one get nothing, as there:
//   done_r = min(add_r, (have_r + n - B_r) P - len_r) where B_r <= n, else 0.
//
// One launch of one thread-block cluster.  Up to 1024 rows, every CTA scans all of
// them (one row a thread) and keeps their records in shared memory; with more, each
// CTA sums its share, the CTAs exchange their totals through distributed shared
// memory, and the records go through the workspace.  Released blocks are copied to
// the stack by all threads of the cluster; behind a cluster barrier every thread
// writes up to four consecutive slots and at most a table entry for each.  No order depends
// on scheduling.  A step moves 8 bytes per token and 8 per block: it is bound by round
// trips to L2 and by its launch, which is why it is one launch (three of them, a scan,
// a push and a fill kernel, took 9-13 us on the GPU and 13 us of the host's time).
// What it measured (GB300, CUDA graph replays): a decode step of 368 rows of which eight
// give back 10900 blocks 6.2 us; 48 rows taking 20 thousand slots in pages of 16 6.8 us;
// 24 rows taking 119 thousand slots 11.4 us; 1024 rows running out of blocks 7.5 us.
#include <algorithm>

#include "device_common.cuh"
#include "gk_internal.h"

namespace gk {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxCtas = 16;
constexpr int kUnroll = 4;         // independent loads in flight per thread

// per row, for the kernel's later phases
struct TableRowDev {
  int64_t tok0;      // its first token's place in the slot map
  int32_t len;       // tokens before the append (0 for a released row)
  int32_t done;      // tokens appended
  int32_t pop0;      // blocks the rows before it took
  int32_t have;      // blocks before the append
  int32_t pad[2];
};
static_assert(sizeof(TableRowDev) == GK_TABLES_WORK_PER_ROW, "workspace size in gk.h");

struct StepParams {
  int32_t rows, max_blocks, capacity, page;
  int32_t page_shift;               // log2(page), -1 where it is no power of two
  int64_t n_blocks;                 // COLD blocks of the pool
  int64_t n_slots;
  int32_t* table;
  int32_t* free;
  const int32_t* len;
  int32_t* len_out;
  const int32_t* n_free;
  int32_t* n_free_out;
  const int32_t* release;
  const int32_t* add;
  int64_t* slots;
  int32_t* done;
  TableRowDev* work;
  int32_t* err;
};

// 32-bit quotients, by shifts for the usual pages: 64-bit division held the fill to 9 us
// for 119 thousand tokens
__device__ __forceinline__ int32_t page_of(const StepParams& p, int32_t pos) {
  return p.page_shift >= 0 ? pos >> p.page_shift : (int32_t)((uint32_t)pos / (uint32_t)p.page);
}
// blocks of tokens in [0, 2^31)
__device__ __forceinline__ int32_t blocks_of(const StepParams& p, int32_t tokens) {
  return tokens > 0 ? page_of(p, tokens - 1) + 1 : 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 64-bit value at shared address `addr` of CTA `rank` of the cluster
__device__ __forceinline__ int64_t ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t a;
  int64_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

// exclusive sums over the CTA of three values per thread; the totals in sum[]
__device__ __forceinline__ void scan3(int64_t v[3], int64_t sum[3], int64_t (*warp_sum)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    int64_t x = v[i];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    inc[i] = x;
    if (lane == 31) warp_sum[warp][i] = x;
  }
  __syncthreads();
  if (warp < 3) {
    int64_t x = warp_sum[lane][warp];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    warp_sum[lane][warp] = x;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int64_t before = warp ? warp_sum[warp - 1][i] : 0;
    v[i] = before + inc[i] - v[i];
    sum[i] = warp_sum[31][i];
  }
  __syncthreads();
}

// last i of [0, n) with key(i) <= x (key ascending, key(0) <= x)
template <typename Key>
__device__ __forceinline__ int last_at_most(int n, int64_t x, Key key) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (key(mid) <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// what a row asks for
struct RowAsk {
  int64_t asked;     // its places in the slot map
  int32_t need;      // new blocks
  int32_t pushed;    // released blocks
  int32_t len;       // tokens it starts the append with
  int32_t have;      // their blocks
  bool bad;          // its length or table cannot be: it keeps both
  bool skip;         // it appends nothing
  bool wrong;        // ... and asked for something
};
__device__ __forceinline__ RowAsk row_ask(const StepParams& p, int r, bool releases) {
  RowAsk a{0, 0, 0, 0, 0, false, true, false};
  if (r >= p.rows) return a;
  const int32_t len = p.len[r], add = p.add[r], rel = releases ? p.release[r] : 0;
  a.asked = add > 0 ? add : 0;
  a.len = len;
  a.bad = len < 0 || blocks_of(p, len) > p.max_blocks;
  if (!a.bad && rel != 0) {
    a.pushed = blocks_of(p, len);
    a.len = 0;
  }
  a.skip = a.bad || add < 0 || a.len + a.asked > INT32_MAX || blocks_of(p, a.len + (int32_t)a.asked) > p.max_blocks;
  a.wrong = a.skip && add != 0;
  if (!a.bad) a.have = blocks_of(p, a.len);
  if (!a.skip) a.need = blocks_of(p, a.len + (int32_t)a.asked) - a.have;
  return a;
}

// kFit: the rows are at most kThreads
template <bool kFit>
__global__ void __launch_bounds__(kThreads) tables_step_kernel(const StepParams p) {
  __shared__ int64_t warp_sum[32][3];
  __shared__ int64_t total[2][3];           // this CTA's rows: tokens, new blocks, released blocks
  __shared__ int64_t totals[kMaxCtas][3];
  __shared__ int32_t push_at[kThreads];     // released blocks of the chunk's rows before each
  __shared__ TableRowDev rows_s[kFit ? kThreads : 1];  // every row's record
  const int tid = (int)threadIdx.x;
  const int rank = (int)cluster_rank(), ctas = (int)cluster_ctas();
  griddep_launch_dependents();
  griddep_wait();
  const int span = kFit ? p.rows : (p.rows + ctas - 1) / ctas;   // rows that this CTA scans
  const int r_begin = kFit ? 0 : min(p.rows, rank * span), r_end = min(p.rows, r_begin + span);
  const int32_t n_in = *p.n_free;
  const bool stack_ok = n_in >= 0 && n_in <= p.capacity;
  const int32_t n0 = stack_ok ? n_in : 0;

  // ---- totals: this CTA's, then everyone's -------------------------------------------
  bool releases = p.release != nullptr;
  int64_t base[3], all[3];
  RowAsk a;                                 // the last chunk's row, and its place in the chunk
  int64_t v[3], sum[3];
  for (int pass = 0;; ++pass) {
    int64_t mine[3] = {0, 0, 0};
    for (int r0 = r_begin; r0 < r_end || r0 == r_begin; r0 += kThreads) {
      a = row_ask(p, r0 + tid < r_end ? r0 + tid : p.rows, releases);
      v[0] = a.asked;
      v[1] = a.need;
      v[2] = a.pushed;
      scan3(v, sum, warp_sum);
#pragma unroll
      for (int i = 0; i < 3; ++i) mine[i] += sum[i];
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      base[i] = 0;
      all[i] = mine[i];
    }
    if (!kFit && ctas > 1) {
      // the totals stay until the cluster barrier behind the rows' results, so no CTA changes or
      // leaves them while another reads
      if (tid < 3) total[pass][tid] = tid == 0 ? mine[0] : tid == 1 ? mine[1] : mine[2];
      cluster_sync();
      if (tid < 3 * ctas) totals[tid / 3][tid % 3] = ld_cluster(smem_u32(&total[pass][tid % 3]), (uint32_t)(tid / 3));
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        all[i] = 0;
        for (int c = 0; c < ctas; ++c) {
          if (c < rank) base[i] += totals[c][i];
          all[i] += totals[c][i];
        }
      }
      __syncthreads();
    }
    if (stack_ok && n0 + all[2] <= p.capacity) break;
    if (pass == 0 && rank == 0 && tid == 0) report_error(p.err, kErrBounds);
    if (!releases || pass == 1) break;
    releases = false;                       // the stack cannot take them: nothing is released
  }
  const int64_t top = n0 + all[2];          // blocks on the stack after the releases

  // ---- per-row results, and released blocks to the stack -------------------------------
  const bool once = kFit || r_end - r_begin <= kThreads;   // a, v and sum are still those of the only chunk
  int32_t done = 0;
  int64_t taken = 0;
  bool overflow = false;
  auto write_row = [&](int r) {
    p.done[r] = done;
    p.len_out[r] = a.bad ? a.len : a.len + done;
    if (overflow && stack_ok) *p.n_free_out = (int32_t)(top - taken);
  };
  for (int r0 = r_begin; r0 < r_end; r0 += kThreads) {
    const int r = r0 + tid, n_here = min(kThreads, r_end - r0);
    if (!once) {
      a = row_ask(p, r < r_end ? r : p.rows, releases);
      v[0] = a.asked;
      v[1] = a.need;
      v[2] = a.pushed;
      scan3(v, sum, warp_sum);
    }
    const int64_t tok0 = base[0] + v[0], pop0 = base[1] + v[1];
    if (r < r_end) {
      const int64_t end = tok0 + a.asked;
      done = 0;
      if (!a.skip && end <= p.n_slots && pop0 <= top)
        done = (int32_t)min(a.asked, (a.have + top - pop0) * p.page - a.len);
      if ((!kFit || rank == 0) && (a.bad || a.wrong || end > p.n_slots)) report_error(p.err, kErrBounds);
      // the first row without room in the slot map: no row from there on takes a block
      overflow = end > p.n_slots && tok0 <= p.n_slots;
      taken = min(pop0, top);
      const TableRowDev w{tok0, a.len, done, (int32_t)min(pop0, (int64_t)INT32_MAX), a.have, {0, 0}};
      if (kFit) {
        rows_s[r] = w;
      } else {
        p.work[r] = w;
        write_row(r);
      }
    }
    if (releases) {
      push_at[tid] = (int32_t)v[2];
      __syncthreads();
      int32_t* dst = p.free + n0 + base[2];
      const uint32_t n_push = (uint32_t)sum[2];            // below 2^31: the strides cannot wrap
      const uint32_t stride = kFit ? ctas * kThreads : kThreads;
      for (uint32_t i0 = (kFit ? rank * kThreads : 0) + tid; i0 < n_push; i0 += kUnroll * stride) {
        int32_t id[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          const uint32_t i = i0 + k * stride;
          if (i < n_push) {
            const int q = last_at_most(n_here, i, [&](int x) { return (int64_t)push_at[x]; });
            id[k] = p.table[(int64_t)(r0 + q) * p.max_blocks + ((int32_t)i - push_at[q])];
          }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
          if (i0 + k * stride < n_push) dst[i0 + k * stride] = id[k];
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) base[i] += sum[i];
  }
  if (ctas > 1) cluster_sync();
  else __syncthreads();
  // outputs that may be the inputs' own arrays: behind everyone's reads
  if (kFit && rank == 0 && tid < p.rows) write_row(tid);
  if (rank == 0 && tid == 0 && (!stack_ok || all[0] <= p.n_slots))
    *p.n_free_out = stack_ok ? (int32_t)(top - min(all[1], top)) : n_in;

  // ---- a slot and at most a table entry per token ----------------------------------------
  const TableRowDev* rows = kFit ? rows_s : p.work;
  auto row_of = [&](int64_t t) { return last_at_most(p.rows, t, [&](int x) { return rows[x].tok0; }); };
  const bool wide = (uintptr_t)p.slots % 16 == 0;
  // consecutive tokens a thread takes at a time: few where the threads outnumber the tokens, as
  // each may need a search of its own (a decode step's tokens are all of different rows)
  const int64_t threads = (int64_t)ctas * kThreads;
  const int per = (int)min((int64_t)kUnroll, (p.n_slots + threads - 1) / threads);
  for (int64_t t0 = ((int64_t)rank * kThreads + tid) * per; t0 < p.n_slots; t0 += threads * per) {
    int32_t id[kUnroll], pos[kUnroll];
    int64_t cell[kUnroll];                  // -1: nothing to place, -2: nothing to write
    int64_t slot[kUnroll];
    int r = 0;
    int64_t next = t0;                      // first token of the row after r
    TableRowDev w;
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int64_t t = t0 + k;
      cell[k] = -1;
      id[k] = -1;
      pos[k] = 0;
      if (k >= per || t >= p.n_slots || t >= all[0]) continue;
      if (t >= next) {
        r = row_of(t);
        w = rows[r];
        next = r + 1 < p.rows ? rows[r + 1].tok0 : all[0];
      }
      const int64_t j = t - w.tok0;
      if (j >= w.done) continue;
      pos[k] = w.len + (int32_t)j;
      const int32_t b = page_of(p, pos[k]);
      pos[k] -= b * p.page;                 // within the block
      cell[k] = (int64_t)r * p.max_blocks + b;
      const int64_t from = top - 1 - ((int64_t)w.pop0 + b - w.have);
      if (b < w.have) id[k] = p.table[cell[k]];
      else if (from >= 0 && from < p.capacity) id[k] = p.free[from];
      // a new block's first token writes its table entry
      if (b < w.have || pos[k] != 0) cell[k] = -2;
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (cell[k] >= 0) p.table[cell[k]] = id[k];
      slot[k] = -1;
      if (cell[k] != -1) {
        if (id[k] >= 0 && id[k] < p.n_blocks) slot[k] = (int64_t)id[k] * p.page + pos[k];
        else report_error(p.err, kErrBounds);
      }
    }
    if (wide && per == kUnroll && t0 + kUnroll <= p.n_slots) {
#pragma unroll
      for (int k = 0; k < kUnroll; k += 2)
        *reinterpret_cast<longlong2*>(p.slots + t0 + k) = make_longlong2(slot[k], slot[k + 1]);
    } else {
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (k < per && t0 + k < p.n_slots) p.slots[t0 + k] = slot[k];
    }
  }
}

}  // namespace

int launch_tables_step(const LaunchCommon& lc, void* stream, const gk_tables* t, const int32_t* d_release,
                       const int32_t* d_add, int64_t n_slots, int64_t* d_slots, int32_t* d_done) {
  const gk_pool_config& c = *lc.cfg;
  StepParams p{};
  p.rows = t->num_rows;
  p.max_blocks = t->max_blocks;
  p.capacity = t->capacity;
  p.page = c.cold_page_size;
  p.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (c.cold_page_size == 1 << s) p.page_shift = s;
  p.n_blocks = c.cold_slots / c.cold_page_size;
  p.n_slots = n_slots;
  p.table = t->d_table;
  p.free = t->d_free;
  p.len = t->d_len;
  p.len_out = t->d_len_out;
  p.n_free = t->d_num_free;
  p.n_free_out = t->d_num_free_out;
  p.release = d_release;
  p.add = d_add;
  p.slots = d_slots;
  p.done = d_done;
  p.work = (TableRowDev*)t->d_work;
  p.err = lc.d_error;
  // The CTAs of the cluster: one for few tokens and no releases, else sixteen (the most a
  // cluster has).  One against sixteen on a GB300: 64 rows of a token each 4.6 / 4.8 us, 1000
  // rows of a token each 6.5 / 7.0, 64 rows of 64 tokens 6.4 / 5.4, 64 rows of 500 tokens
  // 21.9 / 5.8, 368 rows of a token each while eight rows give back 10900 blocks 12.4 / 6.3.
  // Eight CTAs were no faster than sixteen anywhere (119 thousand tokens: 16.8 against 11.4).
  const bool fit = p.rows <= kThreads;
  const int ctas = d_release || n_slots > 2 * kThreads || !fit ? kMaxCtas : 1;
  auto kern = fit ? tables_step_kernel<true> : tables_step_kernel<false>;
  if (ctas > 1) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return (int)e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return (int)cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace gk

extern "C" gk_status gk_tables_step(gk_pool* pool, void* stream, const gk_tables* t, const int32_t* d_release,
                                    const int32_t* d_add, int64_t n_slots, int64_t* d_slot_mapping, int32_t* d_done) {
  if (!pool || !t) return GK_ERR_INVALID;
  gk::Pool* p = &pool->impl;
  if (t->num_rows < 0 || t->max_blocks < 0 || t->capacity < 0 || n_slots < 0)
    return gk::fail(p, GK_ERR_INVALID, "negative size");
  if (t->num_rows > (1 << 20)) return gk::fail(p, GK_ERR_INVALID, "more than 2^20 rows");
  if (t->num_rows > 0) {
    if (!t->d_len || !t->d_len_out || !t->d_num_free || !t->d_num_free_out || !t->d_work || !d_add || !d_done ||
        (t->max_blocks > 0 && !t->d_table) || (t->capacity > 0 && !t->d_free) || (n_slots > 0 && !d_slot_mapping))
      return gk::fail(p, GK_ERR_INVALID, "null device pointer");
    for (const void* ptr : {(const void*)t->d_table, (const void*)t->d_free, (const void*)t->d_len, (const void*)t->d_len_out,
                            (const void*)t->d_num_free, (const void*)t->d_num_free_out, (const void*)d_release,
                            (const void*)d_add, (const void*)d_done})
      if ((uintptr_t)ptr % 4 != 0) return gk::fail(p, GK_ERR_INVALID, "int32 arrays must be 4-byte aligned");
    if ((uintptr_t)d_slot_mapping % 8 != 0) return gk::fail(p, GK_ERR_INVALID, "the slot map must be 8-byte aligned");
    if ((uintptr_t)t->d_work % 16 != 0) return gk::fail(p, GK_ERR_INVALID, "d_work must be 16-byte aligned");
  }
  gk_status st = gk::ensure_device(p);
  if (st == GK_OK) st = gk::device_is_current(p);
  if (st != GK_OK) return st;
  if (t->num_rows == 0) return GK_OK;
  gk::LaunchCommon lc{&p->cfg, p->d_error, p->dev.num_sms};
  int e = gk::launch_tables_step(lc, stream, t, d_release, d_add, n_slots, d_slot_mapping, d_done);
  return e ? gk::cuda_fail(p, e, "block-table kernels") : GK_OK;
}
