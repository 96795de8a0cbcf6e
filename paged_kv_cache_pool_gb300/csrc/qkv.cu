// From a layer's q, k, v projection to its attention and cache: norms of the heads of q
// and k, the rotation of positions, the writes into the paged COLD cache (bf16 rows or
// 4-bit rows), and the way back from the cache to bf16 rows.
//
// Per head x of d channels, in fp32 (gk_qkv in gk.h gives the formulas): the sum of squares
// is one pass over registers and log2(d / 16) shuffles; the rotation multiplies with the
// cosines and sines of the token's position from a table.  About ten operations a channel
// against 4 bytes, so HBM bounds it: each input is read once and each output written once.
//
// A warp takes the heads of one token 256 channels at a time (8 heads of 64 or 4 of 128), 16
// channels a thread in two 16-byte chunks: chunk j and chunk j + d / 16 of the head, the two
// that a rotation of the whole head pairs, and at d = 128 one of either group of 64 that 4-bit
// rows scale together.
#include <cstdint>

#include "device_common.cuh"
#include "gk_internal.h"
#include "kv4.cuh"

namespace gk {
namespace {

constexpr int kWarps = 4;  // warps of a block

// how channels rotate: not at all, whole heads in halves, neighbouring pairs, a part of the head in halves
enum Rotation { kNone, kHalves, kPairs, kPart };

struct QkvParams {
  const uint16_t *q, *k, *v;
  uint16_t *q_out, *k_out;
  int64_t qs, ks, vs, qos, kos;   // elements from token to token
  const uint16_t *wq, *wk;
  const float* table;
  const int32_t* pos;
  int64_t num_pos;
  int32_t rot;
  float eps;
  int32_t n, Hq, Hkv;
  // cache of the layer (slots null: none)
  const int64_t* slots;
  int64_t num_slots;
  uint16_t *cold_k, *cold_v;      // bf16 rows
  uint8_t* rows;                  // 4-bit rows
  int32_t* err;
};

__device__ __forceinline__ void unpack8(uint4 w, float* x) {
  x[0] = bf_lo(w.x); x[1] = bf_hi(w.x); x[2] = bf_lo(w.y); x[3] = bf_hi(w.y);
  x[4] = bf_lo(w.z); x[5] = bf_hi(w.z); x[6] = bf_lo(w.w); x[7] = bf_hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float m;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// (a, b) <- (a c - b s, b c + a s), each product and sum rounded by itself: the bits that
// elementary fp32 operations give, so that 4-bit codes do not depend on contraction
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

// lo and span (as bf16 bits, lo in the low half) of a group whose least and greatest values are given
__device__ __forceinline__ uint32_t group_scale(float lo, float hi, float& span) {
  const uint32_t w = pack_bf16x2(lo, __fsub_rn(hi, lo));
  span = bf_hi(w);
  if (!(span < kv4::kMostSpan)) {  // an infinity or NaN among the values, or a span too wide
    span = 0.f;
    return 0x7fffu;              // lo NaN: the group reads as NaN
  }
  if (span < kv4::kLeastSpan) {
    span = 0.f;
    return w & 0xffffu;
  }
  return w;
}

// eight codes, the first in the lowest nibble
__device__ __forceinline__ uint32_t codes8(const float* x, float lo, float span) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // round(15 (x - lo) / span) to even
    const float c = rintf(__fdiv_rn(__fmul_rn(__fsub_rn(x[i], lo), 15.f), span));
    w |= (uint32_t)fminf(c, 15.f) << (4 * i);
  }
  return span > 0.f ? w : 0u;
}

template <int D, int ROT, bool KV4>
__global__ void __launch_bounds__(32 * kWarps) qkv_kernel(const QkvParams p, int passes) {
  constexpr int LPH = D / 16;       // lanes of a head
  constexpr int HPW = 32 / LPH;     // heads of a pass
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, j = lane % LPH;
  const int64_t w = blockIdx.x * (int64_t)kWarps + (threadIdx.x >> 5);
  const int64_t tok = w / passes;
  if (tok >= p.n) return;
  int64_t at = 0;
  if (ROT != kNone) {
    at = p.pos[tok];
    if (at < 0 || at >= p.num_pos) {
      if (lane == 0) report_error(p.err, kErrBounds);
      return;
    }
  }
  // the heads of q, k and v in one row: head hh is this thread's
  const int hh = (int)(w % passes) * HPW + lane / LPH;
  const int kind = hh < p.Hq ? 0 : hh < p.Hq + p.Hkv ? 1 : p.slots && hh < p.Hq + 2 * p.Hkv ? 2 : 3;
  const int h = kind == 0 ? hh : kind == 1 ? hh - p.Hq : hh - p.Hq - p.Hkv;
  const uint16_t* src = kind == 0 ? p.q + tok * p.qs : kind == 1 ? p.k + tok * p.ks : p.v + tok * p.vs;
  const uint16_t* wgt = kind == 0 ? p.wq : kind == 1 ? p.wk : nullptr;
  float x[16];
  if (kind < 3) {
    unpack8(reinterpret_cast<const uint4*>(src + h * D)[j], x);
    unpack8(reinterpret_cast<const uint4*>(src + h * D)[j + LPH], x + 8);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
  }
  if (p.wq || p.wk) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int off = 1; off < LPH; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    if (wgt) {
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
      float g[16];
      unpack8(reinterpret_cast<const uint4*>(wgt)[j], g);
      unpack8(reinterpret_cast<const uint4*>(wgt)[j + LPH], g + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], r), g[i]);
    }
  }
  if (ROT != kNone) {
    const float* cs = p.table + at * p.rot;
    const int half = p.rot / 2;
    if (ROT == kHalves) {
      float c[8], s[8];
      load8(cs + 8 * j, c);
      load8(cs + half + 8 * j, s);
      if (kind < 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn(x[i], x[i + 8], c[i], s[i]);
      }
    } else if (ROT == kPairs) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int ch = j + b * LPH;            // chunk: pairs 4 ch .. 4 ch + 3
        if (kind < 2 && ch * 8 < p.rot) {
          const float4 c = __ldg(reinterpret_cast<const float4*>(cs + 4 * ch));
          const float4 s = __ldg(reinterpret_cast<const float4*>(cs + half + 4 * ch));
          float* y = x + 8 * b;
          turn(y[0], y[1], c.x, s.x);
          turn(y[2], y[3], c.y, s.y);
          turn(y[4], y[5], c.z, s.z);
          turn(y[6], y[7], c.w, s.w);
        }
      }
    } else {
      // chunk ch < half / 8 pairs with chunk ch + half / 8, which another thread of the head holds
      const int hc = half / 8;
      float other[16];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int ch = j + b * LPH;
        const int pc = ch < hc ? ch + hc : ch < 2 * hc ? ch - hc : ch;
        const int from = (lane & ~(LPH - 1)) | (pc & (LPH - 1));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float lo = __shfl_sync(0xffffffffu, x[i], from), hi = __shfl_sync(0xffffffffu, x[i + 8], from);
          other[8 * b + i] = pc < LPH ? lo : hi;
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int ch = j + b * LPH;
        if (kind < 2 && ch < 2 * hc) {
          float c[8], s[8];
          load8(cs + 8 * (ch < hc ? ch : ch - hc), c);
          load8(cs + half + 8 * (ch < hc ? ch : ch - hc), s);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float mine = x[8 * b + i], theirs = other[8 * b + i];
            if (ch < hc)
              turn(mine, theirs, c[i], s[i]);
            else
              turn(theirs, mine, c[i], s[i]);
            x[8 * b + i] = mine;
          }
        }
      }
    }
  }
  const uint4 y0 = pack8(x), y1 = pack8(x + 8);
  if (kind < 2) {
    uint16_t* out = kind == 0 ? p.q_out + tok * p.qos : p.k_out ? p.k_out + tok * p.kos : nullptr;
    if (out) {
      reinterpret_cast<uint4*>(out + h * D)[j] = y0;
      reinterpret_cast<uint4*>(out + h * D)[j + LPH] = y1;
    }
  }
  if (!p.slots) return;
  if (__all_sync(0xffffffffu, kind == 0)) return;
  const int64_t slot = p.slots[tok];
  const bool ok = slot >= 0 && slot < p.num_slots;
  if (!ok && kind == 1 && h == 0 && j == 0) report_error(p.err, kErrBounds);
  if (!KV4) {
    if (ok && (kind == 1 || kind == 2)) {
      uint16_t* out = (kind == 1 ? p.cold_k : p.cold_v) + (slot * p.Hkv + h) * D;
      reinterpret_cast<uint4*>(out)[j] = y0;
      reinterpret_cast<uint4*>(out)[j + LPH] = y1;
    }
    return;
  }
  // 4-bit rows: of the bf16 values
  unpack8(y0, x);
  unpack8(y1, x + 8);
  float lo[2] = {x[0], x[8]}, hi[2] = {x[0], x[8]};
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo[0] = min_nan(lo[0], x[i]);
    hi[0] = max_nan(hi[0], x[i]);
    lo[1] = min_nan(lo[1], x[8 + i]);
    hi[1] = max_nan(hi[1], x[8 + i]);
  }
  if (D == 64) {     // both chunks are of the head's one group
    lo[0] = min_nan(lo[0], lo[1]);
    hi[0] = max_nan(hi[0], hi[1]);
  }
#pragma unroll
  for (int g = 0; g < D / 64; ++g)
#pragma unroll
    for (int off = 1; off < LPH; off <<= 1) {
      lo[g] = min_nan(lo[g], __shfl_xor_sync(0xffffffffu, lo[g], off));
      hi[g] = max_nan(hi[g], __shfl_xor_sync(0xffffffffu, hi[g], off));
    }
  if (!ok || kind == 0 || kind == 3) return;
  uint8_t* row = p.rows + slot * kv4::row_bytes(p.Hkv, D);
  uint8_t* codes = row + kv4::codes_at(h, D) + (kind == 2 ? D / 2 : 0);
  uint8_t* scales = row + kv4::scales_at(p.Hkv, h, D) + (kind == 2 ? D / 16 : 0);
  float span;
  const uint32_t s0 = group_scale(lo[0], hi[0], span);
  const uint32_t c0 = codes8(x, lo[0], span);
  if (D == 64) {
    reinterpret_cast<uint32_t*>(codes)[j] = c0;
    reinterpret_cast<uint32_t*>(codes)[j + LPH] = codes8(x + 8, lo[0], span);
    if (j == 0) *reinterpret_cast<uint32_t*>(scales) = s0;
  } else {
    const uint32_t s1 = group_scale(lo[1], hi[1], span);
    reinterpret_cast<uint2*>(codes)[j] = make_uint2(c0, codes8(x + 8, lo[1], span));
    if (j == 0) *reinterpret_cast<uint2*>(scales) = make_uint2(s0, s1);
  }
}

struct ReadParams {
  const int64_t* slots;
  int64_t n, num_slots;
  const uint16_t *cold_k, *cold_v;
  const uint8_t* rows;
  uint16_t *k, *v;
  int64_t ks, vs;
  int32_t Hkv;
  int32_t* err;
};

// bf16(lo + code * step) of the eight codes of a word
__device__ __forceinline__ uint4 values8(uint32_t w, float lo, float step) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(lo, __fmul_rn((float)((w >> (4 * i)) & 15u), step));
  return pack8(x);
}

template <int D, bool KV4>
__global__ void __launch_bounds__(32 * kWarps) read_kernel(const ReadParams p, int passes) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, j = lane % LPH;
  const int64_t w = blockIdx.x * (int64_t)kWarps + (threadIdx.x >> 5);
  const int64_t tok = w / passes;
  const int hh = (int)(w % passes) * HPW + lane / LPH;
  if (tok >= p.n || hh >= 2 * p.Hkv) return;
  const bool is_v = hh >= p.Hkv;
  const int h = is_v ? hh - p.Hkv : hh;
  const int64_t slot = p.slots[tok];
  uint4 y0 = make_uint4(0, 0, 0, 0), y1 = y0;
  if (slot < 0 || slot >= p.num_slots) {
    if (hh == 0 && j == 0) report_error(p.err, kErrBounds);
  } else if (KV4) {
    const uint8_t* row = p.rows + slot * kv4::row_bytes(p.Hkv, D);
    const uint8_t* codes = row + kv4::codes_at(h, D) + (is_v ? D / 2 : 0);
    const uint32_t* scales = reinterpret_cast<const uint32_t*>(row + kv4::scales_at(p.Hkv, h, D) + (is_v ? D / 16 : 0));
    const uint32_t s0 = scales[0], s1 = scales[D / 64 - 1];
    uint2 c;
    if (D == 64) {
      c.x = reinterpret_cast<const uint32_t*>(codes)[j];
      c.y = reinterpret_cast<const uint32_t*>(codes)[j + LPH];
    } else {
      c = reinterpret_cast<const uint2*>(codes)[j];
    }
    y0 = values8(c.x, bf_lo(s0), __fdiv_rn(bf_hi(s0), 15.f));
    y1 = values8(c.y, bf_lo(s1), __fdiv_rn(bf_hi(s1), 15.f));
  } else {
    const uint4* src = reinterpret_cast<const uint4*>((is_v ? p.cold_v : p.cold_k) + (slot * p.Hkv + h) * D);
    y0 = src[j];
    y1 = src[j + LPH];
  }
  uint4* out = reinterpret_cast<uint4*>((is_v ? p.v + tok * p.vs : p.k + tok * p.ks) + h * D);
  out[j] = y0;
  out[j + LPH] = y1;
}

// One CTA per copy-on-write pair: the rows of a block, 16 bytes at a time.
__global__ void kv4_cow_kernel(uint4* layer, int64_t block_vecs, int64_t n_blocks, const int32_t* __restrict__ pairs,
                               int32_t* err) {
  griddep_launch_dependents();
  griddep_wait();
  const int32_t src = pairs[2 * blockIdx.x], dst = pairs[2 * blockIdx.x + 1];
  if (src < 0 || dst < 0 || src >= n_blocks || dst >= n_blocks) {
    if (threadIdx.x == 0) report_error(err, kErrBounds);
    return;
  }
  for (int64_t i = threadIdx.x; i < block_vecs; i += blockDim.x)
    layer[dst * block_vecs + i] = layer[src * block_vecs + i];
}

template <int D, int ROT>
int launch_qkv_t(bool kv4, const QkvParams& p, cudaStream_t st) {
  const int heads = p.Hq + p.Hkv * (p.slots ? 2 : 1);
  const int passes = (heads + 512 / D - 1) / (512 / D);
  const int64_t blocks = ((int64_t)p.n * passes + kWarps - 1) / kWarps;
  auto kern = kv4 ? qkv_kernel<D, ROT, true> : qkv_kernel<D, ROT, false>;
  return (int)launch_pdl(kern, dim3((unsigned)blocks), dim3(32 * kWarps), 0, st, p, passes);
}

template <int D>
int launch_qkv_d(bool kv4, const QkvParams& p, bool interleaved, cudaStream_t st) {
  if (p.rot == 0) return launch_qkv_t<D, kNone>(kv4, p, st);
  if (interleaved) return launch_qkv_t<D, kPairs>(kv4, p, st);
  return p.rot == D ? launch_qkv_t<D, kHalves>(kv4, p, st) : launch_qkv_t<D, kPart>(kv4, p, st);
}

}  // namespace

int64_t kv4_row_bytes(int32_t hkv, int32_t d) { return kv4::row_bytes(hkv, d); }

int launch_kv4_cow_copy(const LaunchCommon& lc, void* stream, int32_t layer, int32_t n_cow, const int32_t* d_pairs) {
  const gk_pool_config& c = *lc.cfg;
  const int64_t row_vecs = kv4::row_bytes(c.num_kv_heads, c.head_dim) / 16;
  return (int)launch_pdl(kv4_cow_kernel, dim3(n_cow), dim3(256), 0, (cudaStream_t)stream,
                         (uint4*)c.cold_k + layer * c.cold_slots * row_vecs, c.cold_page_size * row_vecs,
                         (int64_t)(c.cold_slots / c.cold_page_size), d_pairs, lc.d_error);
}

int launch_qkv(const LaunchCommon& lc, void* stream, bool kv4, int32_t layer, const gk_qkv* x, const int64_t* d_slots) {
  const gk_pool_config& c = *lc.cfg;
  const int64_t d = c.head_dim, q_row = c.num_q_heads * d, kv_row = c.num_kv_heads * d;
  auto stride = [](int64_t s, int64_t row) { return s ? s : row; };
  QkvParams p{};
  p.q = (const uint16_t*)x->d_q;
  p.k = (const uint16_t*)x->d_k;
  p.v = (const uint16_t*)x->d_v;
  p.q_out = (uint16_t*)x->d_q_out;
  p.k_out = (uint16_t*)x->d_k_out;
  p.qs = stride(x->q_stride, q_row);
  p.ks = stride(x->k_stride, kv_row);
  p.vs = stride(x->v_stride, kv_row);
  p.qos = stride(x->q_out_stride, q_row);
  p.kos = stride(x->k_out_stride, kv_row);
  p.wq = p.q ? (const uint16_t*)x->d_q_weight : nullptr;
  p.wk = p.k ? (const uint16_t*)x->d_k_weight : nullptr;
  p.table = x->d_cos_sin;
  p.pos = x->d_positions;
  p.num_pos = x->num_positions;
  p.rot = x->rot_dim;
  p.eps = x->eps;
  p.n = x->num_tokens;
  p.Hq = p.q ? c.num_q_heads : 0;
  p.Hkv = p.k ? c.num_kv_heads : 0;
  p.slots = d_slots;
  p.num_slots = c.cold_slots;
  if (d_slots && kv4) {
    p.rows = (uint8_t*)c.cold_k + layer * c.cold_slots * (int64_t)kv4::row_bytes(c.num_kv_heads, c.head_dim);
  } else if (d_slots) {
    p.cold_k = (uint16_t*)c.cold_k + layer * c.cold_slots * kv_row;
    p.cold_v = (uint16_t*)c.cold_v + layer * c.cold_slots * kv_row;
  }
  p.err = lc.d_error;
  cudaStream_t st = (cudaStream_t)stream;
  return c.head_dim == 128 ? launch_qkv_d<128>(kv4, p, x->interleaved != 0, st)
                           : launch_qkv_d<64>(kv4, p, x->interleaved != 0, st);
}

int launch_read_kv(const LaunchCommon& lc, void* stream, bool kv4, int32_t layer, int64_t n, const int64_t* d_slots,
                   void* d_k, void* d_v, int64_t k_stride, int64_t v_stride) {
  const gk_pool_config& c = *lc.cfg;
  const int64_t kv_row = (int64_t)c.num_kv_heads * c.head_dim;
  ReadParams p{};
  p.slots = d_slots;
  p.n = n;
  p.num_slots = c.cold_slots;
  if (kv4) {
    p.rows = (const uint8_t*)c.cold_k + layer * c.cold_slots * (int64_t)kv4::row_bytes(c.num_kv_heads, c.head_dim);
  } else {
    p.cold_k = (const uint16_t*)c.cold_k + layer * c.cold_slots * kv_row;
    p.cold_v = (const uint16_t*)c.cold_v + layer * c.cold_slots * kv_row;
  }
  p.k = (uint16_t*)d_k;
  p.v = (uint16_t*)d_v;
  p.ks = k_stride ? k_stride : kv_row;
  p.vs = v_stride ? v_stride : kv_row;
  p.Hkv = c.num_kv_heads;
  p.err = lc.d_error;
  const int per = 512 / c.head_dim, passes = (2 * c.num_kv_heads + per - 1) / per;
  const int64_t blocks = (n * passes + kWarps - 1) / kWarps;
  auto kern = c.head_dim == 128 ? (kv4 ? read_kernel<128, true> : read_kernel<128, false>)
                                : (kv4 ? read_kernel<64, true> : read_kernel<64, false>);
  return (int)launch_pdl(kern, dim3((unsigned)blocks), dim3(32 * kWarps), 0, (cudaStream_t)stream, p, passes);
}

}  // namespace gk

using gk::Pool;

namespace {

constexpr int32_t kMostTokens = 1 << 27;  // so that a launch's blocks fit its grid

// null and misaligned pointers, strides and the rotation of x; cache: as gk_append_qkv takes it
gk_status check_qkv(Pool* p, const gk_qkv* x, bool cache) {
  const gk_pool_config& c = p->cfg;
  const int64_t q_row = (int64_t)c.num_q_heads * c.head_dim, kv_row = (int64_t)c.num_kv_heads * c.head_dim;
  if (x->num_tokens < 0 || x->num_tokens > kMostTokens)
    return gk::fail(p, GK_ERR_INVALID, "num_tokens must be in [0, 2^27]");
  if (x->rot_dim < 0 || x->rot_dim % 16 != 0 || x->rot_dim > c.head_dim)
    return gk::fail(p, GK_ERR_UNSUPPORTED, "rot_dim must be a multiple of 16 up to head_dim");
  if (x->interleaved != 0 && x->interleaved != 1) return gk::fail(p, GK_ERR_INVALID, "interleaved must be 0 or 1");
  if (!(x->eps >= 0.f)) return gk::fail(p, GK_ERR_INVALID, "eps must not be negative");
  if (x->num_positions < 0) return gk::fail(p, GK_ERR_INVALID, "negative num_positions");
  const bool some = x->num_tokens > 0;
  if (some && x->rot_dim > 0 && (!x->d_cos_sin || !x->d_positions))
    return gk::fail(p, GK_ERR_INVALID, "a rotation needs d_cos_sin and d_positions");
  if (some && (x->d_q == nullptr) != (x->d_q_out == nullptr))
    return gk::fail(p, GK_ERR_INVALID, "d_q and d_q_out go together");
  if (some && cache && (!x->d_k || !x->d_v)) return gk::fail(p, GK_ERR_INVALID, "an append needs d_k and d_v");
  if (some && !cache && (x->d_k == nullptr) != (x->d_k_out == nullptr))
    return gk::fail(p, GK_ERR_INVALID, "d_k and d_k_out go together");
  for (const void* ptr : {x->d_q, x->d_k, cache ? x->d_v : nullptr, (const void*)x->d_q_out, (const void*)x->d_k_out, x->d_q_weight,
                          x->d_k_weight, (const void*)x->d_cos_sin})
    if ((uintptr_t)ptr % 16 != 0) return gk::fail(p, GK_ERR_INVALID, "rows, weights and the table must be 16-byte aligned");
  if ((uintptr_t)x->d_positions % 4 != 0) return gk::fail(p, GK_ERR_INVALID, "positions must be 4-byte aligned");
  const int64_t s[5] = {x->q_stride, x->q_out_stride, x->k_stride, x->k_out_stride, x->v_stride};
  for (int i = 0; i < 5; ++i)
    if (s[i] != 0 && (s[i] < (i < 2 ? q_row : kv_row) || s[i] % 8 != 0 || s[i] > ((int64_t)1 << 38)))
      return gk::fail(p, GK_ERR_INVALID, "a token stride must be 0 or a multiple of 8 that holds the token's heads");
  return GK_OK;
}

gk_status on_device(Pool* p) {
  gk_status st = gk::ensure_device(p);
  return st == GK_OK ? gk::device_is_current(p) : st;
}

}  // namespace

extern "C" {

gk_status gk_qk_norm_rope(gk_pool* pool, void* stream, const gk_qkv* x) {
  if (!pool || !x) return GK_ERR_INVALID;
  Pool* p = &pool->impl;
  gk_status st = check_qkv(p, x, false);
  if (st == GK_OK) st = on_device(p);
  if (st != GK_OK) return st;
  if (x->num_tokens == 0 || (!x->d_q && !x->d_k)) return GK_OK;
  gk::LaunchCommon lc{&p->cfg, p->d_error, p->dev.num_sms};
  int e = gk::launch_qkv(lc, stream, false, 0, x, nullptr);
  return e ? gk::cuda_fail(p, e, "norm and rotation kernel") : GK_OK;
}

gk_status gk_append_qkv(gk_pool* pool, void* stream, int32_t layer, const gk_qkv* x, const int64_t* d_slot_mapping,
                        int32_t n_cow, const int32_t* d_cow_pairs) {
  if (!pool || !x) return GK_ERR_INVALID;
  Pool* p = &pool->impl;
  if (layer < 0 || layer >= p->cfg.num_layers || n_cow < 0) return gk::fail(p, GK_ERR_INVALID, "bad layer or count");
  gk_status st = check_qkv(p, x, true);
  if (st != GK_OK) return st;
  if ((x->num_tokens > 0 && !d_slot_mapping) || (n_cow > 0 && !d_cow_pairs))
    return gk::fail(p, GK_ERR_INVALID, "null device pointer");
  if ((uintptr_t)d_slot_mapping % 8 != 0 || (uintptr_t)d_cow_pairs % 4 != 0)
    return gk::fail(p, GK_ERR_INVALID, "slots must be 8-byte and copy-on-write pairs 4-byte aligned");
  st = on_device(p);
  if (st != GK_OK) return st;
  gk::LaunchCommon lc{&p->cfg, p->d_error, p->dev.num_sms};
  if (n_cow > 0) {
    int e = p->kv4 ? gk::launch_kv4_cow_copy(lc, stream, layer, n_cow, d_cow_pairs)
                   : gk::launch_cow_copy(lc, stream, layer, n_cow, d_cow_pairs);
    if (e) return gk::cuda_fail(p, e, "copy-on-write kernel");
  }
  if (x->num_tokens == 0) return GK_OK;
  int e = gk::launch_qkv(lc, stream, p->kv4, layer, x, d_slot_mapping);
  return e ? gk::cuda_fail(p, e, "append kernel") : GK_OK;
}

gk_status gk_read_kv(gk_pool* pool, void* stream, int32_t layer, int64_t n, const int64_t* d_slot_mapping, void* d_k,
                     void* d_v, int64_t k_stride, int64_t v_stride) {
  if (!pool) return GK_ERR_INVALID;
  Pool* p = &pool->impl;
  const int64_t kv_row = (int64_t)p->cfg.num_kv_heads * p->cfg.head_dim;
  if (layer < 0 || layer >= p->cfg.num_layers || n < 0 || n > kMostTokens)
    return gk::fail(p, GK_ERR_INVALID, "bad layer or count");
  if (n > 0 && (!d_slot_mapping || !d_k || !d_v)) return gk::fail(p, GK_ERR_INVALID, "null device pointer");
  if ((uintptr_t)d_k % 16 != 0 || (uintptr_t)d_v % 16 != 0 || (uintptr_t)d_slot_mapping % 8 != 0)
    return gk::fail(p, GK_ERR_INVALID, "rows must be 16-byte and slots 8-byte aligned");
  for (int64_t s : {k_stride, v_stride})
    if (s != 0 && (s < kv_row || s % 8 != 0 || s > ((int64_t)1 << 38)))
      return gk::fail(p, GK_ERR_INVALID, "a token stride must be 0 or a multiple of 8 that holds the token's heads");
  gk_status st = on_device(p);
  if (st != GK_OK || n == 0) return st;
  gk::LaunchCommon lc{&p->cfg, p->d_error, p->dev.num_sms};
  int e = gk::launch_read_kv(lc, stream, p->kv4, layer, n, d_slot_mapping, d_k, d_v, k_stride, v_stride);
  return e ? gk::cuda_fail(p, e, "read-back kernel") : GK_OK;
}

}  // extern "C"
