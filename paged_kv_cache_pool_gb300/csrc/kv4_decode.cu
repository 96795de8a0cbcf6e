// Decode over 4-bit COLD rows (gk_decode_kv4): the suffix gather over codes, and the
// log-sum-exp join of its partial states with those of the prefix items.
//
// With k_c = lo + code_c * (span / 15) in each group of 64 channels,
//   q . k = sum_groups span / 15 * (q_g . code_g) + lo * sum(q_g)
//   sum_j p_j v_j = sum_j (p_j span_j / 15) code_j + sum_j p_j lo_j   in each group's channels.
#include <cmath>

#include "device_common.cuh"
#include "gk_internal.h"
#include "kv4.cuh"
#include "max_nan.cuh"

namespace gk {
namespace {

struct Kv4Params {
  const uint8_t* rows;        // the layer's
  int64_t num_blocks;
  int32_t page;
  int32_t Hkv, Hq;
  const int32_t* table;
  int32_t max_blocks;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  float* part_o;
  float* part_l;
  const int32_t* seg_begin;
  const SegmentDev* segs;
  float scale;                // log2(e) / sqrt(d)
  int32_t* err;
};

// Warp h of a CTA is KV head h; it takes the CTA's segments one by one, each query
// head over the segment's tokens, 32 at a time: a thread scores a token, then the
// warp adds the tokens' values, D / 32 channels a thread.
template <int D>
__global__ void __launch_bounds__(32 * kMaxKvHeads) kv4_gather_kernel(const Kv4Params p) {
  constexpr int C = D / 32, W = D / 8;
  __shared__ float qs[kMaxKvHeads][D];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, h = threadIdx.x >> 5, g = p.Hq / p.Hkv;
  const int64_t row_bytes = kv4::row_bytes(p.Hkv, D);
  for (int sg = p.seg_begin[blockIdx.x]; sg < p.seg_begin[blockIdx.x + 1]; ++sg) {
    const SegmentDev seg = p.segs[sg];
    for (int qi = 0; qi < g; ++qi) {
      const int qh = h * g + qi;
      const uint16_t* qrow = p.q + ((int64_t)seg.req * p.Hq + qh) * D;
      __syncwarp();
      float sum[D / 64] = {};
      for (int c = lane; c < D; c += 32) {
        const float x = __uint_as_float((uint32_t)qrow[c] << 16);
        qs[h][c] = x;
        sum[c / 64] += x;
      }
#pragma unroll
      for (int gr = 0; gr < D / 64; ++gr)
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], off);
      __syncwarp();
      float m = -INFINITY, l = 0.f, o[C] = {};
      for (int t = seg.t0; t < seg.t1; t += 32) {
        const bool live = t + lane < seg.t1;
        int64_t slot = -1;
        if (live) {
          const int32_t b = p.table[(int64_t)seg.req * p.max_blocks + (t + lane) / p.page];
          if (b >= 0 && b < p.num_blocks)
            slot = (int64_t)b * p.page + (t + lane) % p.page;
          else
            report_error(p.err, kErrBounds);
        }
        const uint8_t* row = p.rows + slot * row_bytes;
        float s = live ? 0.f : -INFINITY;
        if (slot >= 0) {
          const uint32_t* codes = reinterpret_cast<const uint32_t*>(row + kv4::codes_at(h, D));
          const uint32_t* sc = reinterpret_cast<const uint32_t*>(row + kv4::scales_at(p.Hkv, h, D));
          float dot[D / 64] = {};
          for (int w = 0; w < W; ++w) {
            const uint32_t x = codes[w];
            const int gr = D == 64 ? 0 : w & 1, c0 = D == 64 ? 8 * w : 8 * (w >> 1) + 64 * gr;
            for (int i = 0; i < 8; ++i) dot[gr] = fmaf((float)((x >> (4 * i)) & 15u), qs[h][c0 + i], dot[gr]);
          }
#pragma unroll
          for (int gr = 0; gr < D / 64; ++gr)
            s += fmaf(bf_hi(sc[gr]) * (1.f / 15.f), dot[gr], bf_lo(sc[gr]) * sum[gr]);
          s *= p.scale;
        }
        float mx = s;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = max_nan(m, mx);
        const float a = ex2(m - mn), pr = ex2(s - mn);
        m = mn;
        float ps = pr;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, off);
        l = l * a + ps;
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] *= a;
        for (int u = 0; u < 32 && t + u < seg.t1; ++u) {
          const float pu = __shfl_sync(0xffffffffu, pr, u);
          const int64_t su = __shfl_sync(0xffffffffu, slot, u);
          if (su < 0) continue;
          const uint8_t* ru = p.rows + su * row_bytes;
          const int w = lane * C / 8;
          const uint32_t x = reinterpret_cast<const uint32_t*>(ru + kv4::codes_at(h, D) + D / 2)[w];
          const uint32_t sc = reinterpret_cast<const uint32_t*>(ru + kv4::scales_at(p.Hkv, h, D) + D / 16)[D == 64 ? 0 : w & 1];
#pragma unroll
          for (int c = 0; c < C; ++c)
            o[c] = fmaf(pu, fmaf((float)((x >> (4 * (lane * C % 8 + c))) & 15u), bf_hi(sc) * (1.f / 15.f), bf_lo(sc)), o[c]);
        }
      }
      const float inv = 1.f / l;
      const int w = lane * C / 8, ch = (D == 64 ? 8 * w : 8 * (w >> 1) + 64 * (w & 1)) + lane * C % 8;
      if (seg.entry >= 0) {
        const int64_t r = (int64_t)seg.entry * p.Hq + qh;
        for (int c = 0; c < C; ++c) p.part_o[r * D + ch + c] = o[c] * inv;
        if (lane == 0) p.part_l[r] = m + __log2f(l);
      } else {
        const int64_t r = (int64_t)seg.req * p.Hq + qh;
        for (int c = 0; c < C; c += 2)
          *reinterpret_cast<uint32_t*>(p.out + r * D + ch + c) = pack_bf16x2(o[c] * inv, o[c + 1] * inv);
        if (lane == 0 && p.lse) p.lse[r] = (m + __log2f(l)) * kLn2;
      }
    }
  }
}

// O = sum_e 2^(l_e - m) O_e / sum_e 2^(l_e - m), LSE = (m + log2 sum_e 2^(l_e - m)) ln 2 over the partial
// states of a request, m the largest l_e; a warp for each request and query head.
__global__ void __launch_bounds__(256) kv4_join_kernel(const float* part_o, const float* part_l, const RequestDev* reqs, int32_t B,
                                                       int32_t Hq, int32_t D, uint16_t* out, float* lse) {
  griddep_launch_dependents();
  griddep_wait();
  const int w = (int)((blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (w >= B * Hq) return;
  const int r = w / Hq, qh = w % Hq;
  const int e0 = reqs[r].entry_cas, ne = reqs[r].n_entry_cas;
  if (ne < 0) return;  // written by its only segment
  float m = -INFINITY, z = 0.f, o[4] = {};
  for (int e = 0; e < ne; ++e) m = max_nan(m, __ldcg(part_l + (int64_t)(e0 + e) * Hq + qh));
  if (m != -INFINITY)
    for (int e = 0; e < ne; ++e) {
      const int64_t row = (int64_t)(e0 + e) * Hq + qh;
      const float x = ex2(__ldcg(part_l + row) - m);
      if (x == 0.f) continue;      // an empty state, whose row may never have been written
      z += x;
      for (int c = 0; c < D / 32; ++c) o[c] = fmaf(x, __ldcg(part_o + row * D + lane * (D / 32) + c), o[c]);
    }
  const float inv = m == -INFINITY ? 0.f : 1.f / z;
  for (int c = 0; c < D / 32; c += 2)
    *reinterpret_cast<uint32_t*>(out + ((int64_t)r * Hq + qh) * D + lane * (D / 32) + c) = pack_bf16x2(o[c] * inv, o[c + 1] * inv);
  if (lane == 0 && lse) lse[(int64_t)r * Hq + qh] = m == -INFINITY ? -INFINITY : (m + __log2f(z)) * kLn2;
}

}  // namespace

int kv4_ctas_per_sm(const gk_pool_config* cfg) { return 16 / cfg->num_kv_heads; }

int launch_kv4_gather(const LaunchCommon& lc, void* stream, int32_t layer, const gk_batch* b, const Plan* pl, void* d_out) {
  const gk_pool_config& c = *lc.cfg;
  if (pl->suf_segs.empty()) return 0;
  Kv4Params p{};
  p.rows = (const uint8_t*)c.cold_k + layer * c.cold_slots * (int64_t)kv4::row_bytes(c.num_kv_heads, c.head_dim);
  p.num_blocks = c.cold_slots / c.cold_page_size;
  p.page = c.cold_page_size;
  p.Hkv = c.num_kv_heads;
  p.Hq = c.num_q_heads;
  p.table = b->d_block_table;
  p.max_blocks = b->max_blocks;
  p.q = (const uint16_t*)b->d_q;
  p.out = (uint16_t*)d_out;
  p.lse = b->d_lse;
  p.part_o = pl->d_part_o;
  p.part_l = pl->d_part_l;
  const uint8_t* base = (const uint8_t*)pl->d_buf;
  p.seg_begin = (const int32_t*)(base + pl->off_suf_begin);
  p.segs = (const SegmentDev*)(base + pl->off_suf_segs);
  p.scale = kLog2e / sqrtf((float)c.head_dim);
  p.err = lc.d_error;
  auto kern = c.head_dim == 128 ? kv4_gather_kernel<128> : kv4_gather_kernel<64>;
  return (int)launch_pdl(kern, dim3(pl->summary.suffix_ctas), dim3(32 * c.num_kv_heads), 0, (cudaStream_t)stream, p);
}

int launch_kv4_join(const LaunchCommon& lc, void* stream, const gk_batch* b, const Plan* pl, void* d_out) {
  const gk_pool_config& c = *lc.cfg;
  const int64_t warps = (int64_t)pl->B * c.num_q_heads;
  return (int)launch_pdl(kv4_join_kernel, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, (cudaStream_t)stream, pl->d_part_o,
                         pl->d_part_l, (const RequestDev*)((const uint8_t*)pl->d_buf + pl->off_reqs), pl->B, c.num_q_heads, c.head_dim,
                         (uint16_t*)d_out, b->d_lse);
}

}  // namespace gk

extern "C" gk_status gk_decode_kv4(gk_pool* pool, void* stream, int32_t layer, const gk_batch* b, const gk_plan* plan, void* d_out) {
  if (!pool || !b || !plan) return GK_ERR_INVALID;
  gk::Pool* p = &pool->impl;
  const gk::Plan* pl = &plan->impl;
  if (!p->kv4) return gk::fail(p, GK_ERR_UNSUPPORTED, "gk_decode_kv4 reads a 4-bit pool (gk_pool_create_kv4)");
  if (layer < 0 || layer >= p->cfg.num_layers) return gk::fail(p, GK_ERR_INVALID, "layer out of range");
  if (pl->pool != p) return gk::fail(p, GK_ERR_INVALID, "plan belongs to another pool");
  if (!pl->uploaded) return gk::fail(p, GK_ERR_INVALID, "plan has no device tables");
  if (b->num_requests != pl->B) return gk::fail(p, GK_ERR_INVALID, "batch size differs from the plan");
  if (b->d_new_k || b->d_new_v) return gk::fail(p, GK_ERR_UNSUPPORTED, "no fused append: append first (gk_append_qkv)");
  if (pl->B > 0 && (!b->d_q || !d_out || (pl->suffix_blocks > 0 && !b->d_block_table)))
    return gk::fail(p, GK_ERR_INVALID, "batch device pointers missing");
  if (b->max_blocks < pl->suffix_blocks) return gk::fail(p, GK_ERR_INVALID, "block-table row shorter than the planned suffixes");
  if ((uintptr_t)b->d_q % 16 != 0 || (uintptr_t)d_out % 16 != 0)
    return gk::fail(p, GK_ERR_INVALID, "q and out must be 16-byte aligned");
  if ((uintptr_t)b->d_lse % 4 != 0 || (uintptr_t)b->d_block_table % 4 != 0)
    return gk::fail(p, GK_ERR_INVALID, "lse and the block table must be 4-byte aligned");
  gk_status st = gk::ensure_device(p);
  if (st == GK_OK) st = gk::device_is_current(p);
  if (st != GK_OK || pl->B == 0) return st;
  gk::LaunchCommon lc{&p->cfg, p->d_error, p->dev.num_sms};
  int e = 0;
  if (!pl->prefix_items.empty() && (e = gk::launch_prefix(lc, stream, layer, b, pl)))
    return gk::cuda_fail(p, e, "cascade prefix kernel");
  if ((e = gk::launch_kv4_gather(lc, stream, layer, b, pl, d_out))) return gk::cuda_fail(p, e, "4-bit gather kernel");
  if (pl->kv4_join && (e = gk::launch_kv4_join(lc, stream, b, pl, d_out))) return gk::cuda_fail(p, e, "join kernel");
  return GK_OK;
}
