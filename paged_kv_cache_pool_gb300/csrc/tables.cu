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
// tables_scan_kernel (one CTA) does the three exclusive sums over the rows
// (tokens, new blocks, released blocks), writes lengths, counts and, per row, what
// the wide kernels need; tables_push_kernel copies released blocks to the stack;
// tables_fill_kernel writes one slot and at most one table entry per token.
// Nothing is computed twice and no order depends on scheduling.  A step moves at
// most 8 bytes per token and 8 per block: it is bound by launches and by the scan's
// round trips.
#include <algorithm>

#include "device_common.cuh"
#include "gk_internal.h"

namespace gk {
namespace {

constexpr int kScanThreads = 1024;

// per row, written by the scan for the kernels after it
struct TableRowDev {
  int64_t tok0;      // its first token's place in the slot map
  int32_t len;       // tokens before the append (0 for a released row)
  int32_t done;      // tokens appended
  int32_t pop0;      // blocks the rows before it took
  int32_t push0;     // released blocks of the rows before it
  int32_t pushed;    // released blocks of this row
  int32_t pad0;
};
static_assert(sizeof(TableRowDev) == GK_TABLES_WORK_PER_ROW, "workspace size in gk.h");

struct StepParams {
  int32_t rows, max_blocks, capacity, page;
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
  int32_t* top;                     // blocks on the stack after the releases
  int32_t* err;
};

__device__ __forceinline__ int32_t blocks_of(int64_t tokens, int32_t page) { return (int32_t)((tokens + page - 1) / page); }

// one token of row r, k-th of its new ones, at place t of the slot map
__device__ __forceinline__ void place(const StepParams& p, const TableRowDev& w, int r, int32_t k, int64_t t, int32_t top) {
  int64_t slot = -1;
  if (k < w.done) {
    const int32_t pos = w.len + k, b = pos / p.page, have = blocks_of(w.len, p.page);
    int32_t* cell = p.table + (int64_t)r * p.max_blocks + b;
    int32_t id;
    if (b >= have) {
      const int32_t from = top - 1 - (w.pop0 + (b - have));
      id = from >= 0 && from < p.capacity ? p.free[from] : -1;
      if (pos % p.page == 0) *cell = id;       // a new block's first token writes its table entry
    } else {
      id = *cell;
    }
    if (id >= 0 && id < p.n_blocks) slot = (int64_t)id * p.page + pos % p.page;
    else report_error(p.err, kErrBounds);
  }
  p.slots[t] = slot;
}

// exclusive sums over the CTA of three values per thread; total in sum[]
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
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      int64_t x = warp_sum[lane][i];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      warp_sum[lane][i] = x;
    }
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

__global__ void __launch_bounds__(kScanThreads) tables_scan_kernel(const StepParams p) {
  __shared__ int64_t warp_sum[32][3];
  griddep_launch_dependents();
  griddep_wait();
  int64_t base[3] = {0, 0, 0};      // tokens, new blocks, released blocks of the rows before this chunk
  const int32_t n_in = *p.n_free;
  const bool stack_ok = n_in >= 0 && n_in <= p.capacity;
  const int32_t n0 = stack_ok ? n_in : 0;
  // the released blocks first: how high the stack is before any append
  int64_t released = 0;
  if (p.release) {
    for (int r0 = 0; r0 < p.rows; r0 += kScanThreads) {
      const int r = r0 + (int)threadIdx.x;
      int64_t v[3] = {0, 0, 0}, sum[3];
      if (r < p.rows && p.release[r] != 0) {
        const int32_t len = p.len[r];
        if (len >= 0 && blocks_of(len, p.page) <= p.max_blocks) v[2] = blocks_of(len, p.page);
      }
      scan3(v, sum, warp_sum);
      released += sum[2];
    }
  }
  const bool push_ok = stack_ok && n0 + released <= p.capacity;
  const int64_t top = push_ok ? n0 + released : n0;
  if (!push_ok && threadIdx.x == 0) report_error(p.err, kErrBounds);
  int64_t taken_all = 0;
  for (int r0 = 0; r0 < p.rows; r0 += kScanThreads) {
    const int r = r0 + (int)threadIdx.x;
    int32_t len = 0, add = 0, pushed = 0;
    bool bad = false;
    if (r < p.rows) {
      len = p.len[r];
      add = p.add[r];
      bad = len < 0 || blocks_of(len, p.page) > p.max_blocks;
      if (!bad && p.release && p.release[r] != 0 && push_ok) {
        pushed = blocks_of(len, p.page);
        len = 0;
      }
    }
    const int64_t asked = add > 0 ? add : 0;
    // a row whose length or table cannot hold the append takes no part in it
    bool skip = bad || add < 0 || (int64_t)len + asked > INT32_MAX || blocks_of((int64_t)len + asked, p.page) > p.max_blocks;
    int64_t v[3] = {asked, skip ? 0 : blocks_of((int64_t)len + asked, p.page) - blocks_of(len, p.page), pushed}, sum[3];
    const int64_t need = v[1];
    scan3(v, sum, warp_sum);
    const int64_t tok0 = base[0] + v[0], pop0 = base[1] + v[1], push0 = base[2] + v[2];
    int64_t taken = 0;
    if (r < p.rows) {
      if (tok0 + asked > p.n_slots) skip = true;      // no room in the slot map
      int32_t done = 0;
      if (!skip && pop0 <= top) {
        const int64_t fits = ((int64_t)blocks_of(len, p.page) + top - pop0) * p.page - len;
        done = (int32_t)min(asked, fits);
        taken = min(need, top - pop0);
      }
      if (bad || (skip && (add != 0))) report_error(p.err, kErrBounds);
      p.work[r] = {tok0, len, done, (int32_t)min(pop0, (int64_t)INT32_MAX), (int32_t)push0, pushed, 0};
      p.done[r] = done;
      p.len_out[r] = bad ? p.len[r] : len + done;
    }
    int64_t t3[3] = {taken, 0, 0}, tsum[3];
    scan3(t3, tsum, warp_sum);
    taken_all += tsum[0];
#pragma unroll
    for (int i = 0; i < 3; ++i) base[i] += sum[i];
  }
  if (threadIdx.x == 0) {
    *p.n_free_out = stack_ok ? (int32_t)(top - taken_all) : n_in;
    *p.top = (int32_t)top;
    p.top[1] = n0;
  }
}

// one CTA per released row: its blocks onto the stack
__global__ void tables_push_kernel(const StepParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const TableRowDev w = p.work[blockIdx.x];
  const int32_t* row = p.table + (int64_t)blockIdx.x * p.max_blocks;
  int32_t* dst = p.free + p.top[1] + w.push0;
  for (int i = threadIdx.x; i < w.pushed; i += blockDim.x) dst[i] = row[i];
}

__global__ void tables_fill_kernel(const StepParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int32_t top = *p.top;
  for (int64_t t = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; t < p.n_slots; t += (int64_t)gridDim.x * blockDim.x) {
    // the last row that starts at or before t holds it, or t is past them all
    int lo = 0, hi = p.rows - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.work[mid].tok0 <= t) lo = mid;
      else hi = mid - 1;
    }
    const TableRowDev w = p.work[lo];
    const int64_t k = t - w.tok0;
    place(p, w, lo, (int32_t)min(k, (int64_t)INT32_MAX), t, top);
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
  p.top = (int32_t*)t->d_work;
  p.work = (TableRowDev*)((uint8_t*)t->d_work + GK_TABLES_WORK_PER_ROW);
  p.err = lc.d_error;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = launch_pdl(tables_scan_kernel, dim3(1), dim3(kScanThreads), 0, st, p);
  if (e == cudaSuccess && d_release) e = launch_pdl(tables_push_kernel, dim3((unsigned)p.rows), dim3(256), 0, st, p);
  if (e == cudaSuccess && n_slots > 0) {
    const int64_t blocks = std::min<int64_t>((n_slots + 255) / 256, (int64_t)lc.num_sms * 8);
    e = launch_pdl(tables_fill_kernel, dim3((unsigned)blocks), dim3(256), 0, st, p);
  }
  return (int)e;
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
    if ((uintptr_t)t->d_work % 16 != 0) return gk::fail(p, GK_ERR_INVALID, "d_work must be 16-byte aligned");
  }
  gk_status st = gk::ensure_device(p);
  if (st != GK_OK) return st;
  if (t->num_rows == 0) return GK_OK;
  gk::LaunchCommon lc{&p->cfg, p->d_error, p->dev.num_sms};
  int e = gk::launch_tables_step(lc, stream, t, d_release, d_add, n_slots, d_slot_mapping, d_done);
  return e ? gk::cuda_fail(p, e, "block-table kernels") : GK_OK;
}
