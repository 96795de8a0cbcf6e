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
// rows scale together.  Where a part of the head rotates in halves the chunks are dealt out so
// that a thread still holds both of a pair.
#include <cstdint>

#include "device_common.cuh"
#include "gk_internal.h"
#include "kv4.cuh"

namespace gk {
namespace {

constexpr int kWarps = 4;  // warps of a block
constexpr int kChunk = 7;  // most passes of a warp (5, 12 or 14 a warp: 3 - 10 % slower)
// Blocks of an SM, as registers allow (72 a thread).  16384 tokens of 32/8 heads of 128, normed, that rotate in halves, in pairs, in
// halves of 64 channels: into bf16 rows 64, 68, 68 us (by six blocks 68, 71, 70), into 4-bit rows 66, 71, 78 (69, 71, 72: the
// last form spills 24 bytes a thread under this bound).
constexpr int kBlocks = 7;
constexpr int kFewWarps = 64;  // warps of an SM at most

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
  float one;                      // 1, which the compiler must not know: a packed product and a packed sum it contracts, for
                                  // all their .rn, while a product times this plus a term keeps its own rounding
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
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
// 16 bytes that this call reads once
__device__ __forceinline__ uint4 load_once(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
// of two bf16 each, NaN where either is
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// (a, b) <- (a c - b s, b c + a s), each product and sum rounded by itself: the bits that
// elementary fp32 operations give, so that 4-bit codes do not depend on contraction
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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

// Eight codes round(15 (x - lo) / span), ties to even, the first in the lowest nibble.  With q0 = t inv, t = 15 (x - lo)
// rounded and inv the reciprocal to 2^-23, q = q0 + (t - q0 span) inv, its bracket exact, is off by about 2^-45 before it is
// rounded to fp32.  So where t / span is an integer and a half q is that too; where it is not, t is at least an ulp from
// (k + 1/2) span, which fp32 holds (span has eight bits), and q rounds to its side.  Two values an instruction.
__device__ __forceinline__ uint32_t codes8(const float* x, float lo, float span) {
  constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: a sum with it is rounded to an integer, in its low bits
  constexpr uint32_t kBits = 0x4b400000u;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(span));   // the span is between 2^-100 and 2^120, or 0
  const uint64_t nlo = f2pack(-lo, -lo), nspan = f2pack(-span, -span), ii = f2pack(inv, inv);
  const uint64_t fifteen = f2pack(15.f, 15.f), magic = f2pack(kMagic, kMagic);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t t = mul2(fadd2(f2pack(x[i], x[i + 1]), nlo), fifteen), q0 = mul2(t, ii);
    f2unpack(fadd2(ffma2(ffma2(q0, nspan, t), ii, q0), magic), y[i], y[i + 1]);
  }
  uint32_t w = __float_as_uint(y[7]);
#pragma unroll
  for (int i = 6; i >= 0; --i) w = w * 16u + __float_as_uint(y[i]);
  return span == 0.f ? 0u : w - kBits * 0x11111111u;
}

// The two chunks of a head that lane j of its LPH holds: j and j + LPH; where a part of the head rotates in halves, of hc chunks
// each, the first hc lanes hold the chunks that pair, j and j + hc, and the others the rest in order.
template <int D, int ROT>
__device__ __forceinline__ void chunks_of(int j, int hc, int& c0, int& c1) {
  constexpr int LPH = D / 16;
  c0 = ROT == kPart && j >= hc ? j + hc : j;
  c1 = ROT == kPart && j < hc ? j + hc : j + LPH;
}

// What the rotation of a thread's two chunks takes: eight cosines and sines, in halves of the pairs (i, i + 8) of its 16
// channels, of neighbouring pairs four for each chunk.
struct Angles {
  float c[8], s[8];
};

template <int D, int ROT>
__device__ __forceinline__ void load_angles(const QkvParams& p, int64_t at, int j, Angles& w) {
  constexpr int LPH = D / 16;
  const float* cs = p.table + at * p.rot;
  const int half = p.rot / 2;
  if (ROT == kHalves || (ROT == kPart && 8 * j < half)) {
    load8(cs + 8 * j, w.c);
    load8(cs + half + 8 * j, w.s);
  } else if (ROT == kPairs) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int ch = j + b * LPH;                // pairs 4 ch .. 4 ch + 3
      if (ch * 8 >= p.rot) continue;
      const float4 x = *reinterpret_cast<const float4*>(cs + 4 * ch);
      const float4 y = *reinterpret_cast<const float4*>(cs + half + 4 * ch);
      w.c[4 * b] = x.x; w.c[4 * b + 1] = x.y; w.c[4 * b + 2] = x.z; w.c[4 * b + 3] = x.w;
      w.s[4 * b] = y.x; w.s[4 * b + 1] = y.y; w.s[4 * b + 2] = y.z; w.s[4 * b + 3] = y.w;
    }
  }
}

// x: the thread's two chunks
template <int D, int ROT>
__device__ __forceinline__ void rotate(const QkvParams& p, int j, const Angles& w, float* x) {
  constexpr int LPH = D / 16;
  if (ROT == kHalves || (ROT == kPart && 16 * j < p.rot)) {
    const uint64_t one = f2pack(p.one, p.one), minus = f2pack(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t a = f2pack(x[i], x[i + 1]), b = f2pack(x[i + 8], x[i + 9]);
      const uint64_t c = f2pack(w.c[i], w.c[i + 1]), s = f2pack(w.s[i], w.s[i + 1]);
      f2unpack(ffma2(mul2(b, s), minus, mul2(a, c)), x[i], x[i + 1]);
      f2unpack(ffma2(mul2(a, s), one, mul2(b, c)), x[i + 8], x[i + 9]);
    }
  } else if (ROT == kPairs) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((j + i / 4 * LPH) * 8 < p.rot) turn(x[2 * i], x[2 * i + 1], w.c[i], w.s[i]);
  }
}

// Codes and scales of a thread's chunks c0 and c1 (y0 and y1, bf16) of head h, K or V, to its token's row; all threads of
// the warp call it, those with ok store.  ANY: the chunks are not j and j + LPH.
template <int D, bool ANY>
__device__ __forceinline__ void store_codes(uint4 y0, uint4 y1, uint8_t* row, int hkv, int h, bool is_v, int j, int c0, int c1, bool ok) {
  constexpr int LPH = D / 16;
  float x[16];
  unpack8(y0, x);
  unpack8(y1, x + 8);
  // least and greatest: of both chunks in a word's halves, then of the group's threads
  const uint32_t a0 = min2(min2(y0.x, y0.y), min2(y0.z, y0.w)), a1 = min2(min2(y1.x, y1.y), min2(y1.z, y1.w));
  const uint32_t b0 = max2(max2(y0.x, y0.y), max2(y0.z, y0.w)), b1 = max2(max2(y1.x, y1.y), max2(y1.z, y1.w));
  uint32_t lo = min2(__byte_perm(a0, a1, 0x5410), __byte_perm(a0, a1, 0x7632));
  uint32_t hi = max2(__byte_perm(b0, b1, 0x5410), __byte_perm(b0, b1, 0x7632));
  const bool second0 = ANY && D == 128 && c0 >= LPH, first1 = ANY && D == 128 && c1 < LPH;
  if (D == 64) {     // both chunks are of the head's one group
    lo = min2(lo, __byte_perm(lo, 0, 0x1032));
    hi = max2(hi, __byte_perm(hi, 0, 0x1032));
  } else if (second0 || first1) {  // of one group, the halves' other one gets an infinity
    const uint32_t l = min2(lo, __byte_perm(lo, 0, 0x1032)), g = max2(hi, __byte_perm(hi, 0, 0x1032));
    lo = __byte_perm(l, 0x7f80u, second0 ? 0x1054 : 0x5410);
    hi = __byte_perm(g, 0xff80u, second0 ? 0x1054 : 0x5410);
  }
#pragma unroll
  for (int off = 1; off < LPH; off <<= 1) {
    lo = min2(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = max2(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
  if (!ok) return;
  uint8_t* codes = row + kv4::codes_at(h, D) + (is_v ? D / 2 : 0);
  uint8_t* scales = row + kv4::scales_at(hkv, h, D) + (is_v ? D / 16 : 0);
  float span;
  const uint32_t s0 = group_scale(bf_lo(lo), bf_lo(hi), span);
  if (D == 64) {
    reinterpret_cast<uint32_t*>(codes)[c0] = codes8(x, bf_lo(lo), span);
    reinterpret_cast<uint32_t*>(codes)[c1] = codes8(x + 8, bf_lo(lo), span);
    if (j == 0) *reinterpret_cast<uint32_t*>(scales) = s0;
  } else {
    float span1;
    const uint32_t s1 = group_scale(bf_hi(lo), bf_hi(hi), span1);
    const uint32_t w0 = codes8(x, second0 ? bf_hi(lo) : bf_lo(lo), second0 ? span1 : span);
    const uint32_t w1 = codes8(x + 8, first1 ? bf_lo(lo) : bf_hi(lo), first1 ? span : span1);
    if (ANY) {       // word 2 (c % LPH) + c / LPH is chunk c's
      reinterpret_cast<uint32_t*>(codes)[second0 ? 2 * (c0 - LPH) + 1 : 2 * c0] = w0;
      reinterpret_cast<uint32_t*>(codes)[first1 ? 2 * c1 : 2 * (c1 - LPH) + 1] = w1;
    } else {
      reinterpret_cast<uint2*>(codes)[j] = make_uint2(w0, w1);
    }
    if (j == 0) *reinterpret_cast<uint2*>(scales) = make_uint2(s0, s1);
  }
}

// A warp takes passes [part * chunk, (part + 1) * chunk) of a token's: its heads of q, of k and of v, HPW at a time.  Their
// rows are asked for at once, into shared memory; angles and weights are loaded once for all.
// GB300, 16384 tokens of 32/8 heads of 128, normed (344 MB): 77 us with a pass a warp, 75 with four a warp unrolled (290
// instructions a pass), 66 with two passes ahead in registers, 56 as it is, 6.1 TB/s; a copy of the same bytes takes 50.
// Small blocks and many of them (seven of four warps an SM) hide the chain position -> angles -> first pass.
template <int D, int ROT, bool KV4>
__global__ void __launch_bounds__(32 * kWarps, kBlocks) qkv_kernel(const QkvParams p, int passes, uint32_t parts, int chunk) {
  constexpr int LPH = D / 16;       // lanes of a head
  constexpr int HPW = 32 / LPH;     // heads of a pass
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, j = lane % LPH;
  const uint32_t w = blockIdx.x * kWarps + (threadIdx.x >> 5);   // of at most 2^27 tokens' few
  const uint32_t of_token = w / parts;
  const int64_t tok = of_token;
  if (tok >= p.n) return;
  const int first = (int)(w - of_token * parts) * chunk, end = min(passes, first + chunk);
  const int q_passes = (p.Hq + HPW - 1) / HPW, k_end = q_passes + (p.Hkv + HPW - 1) / HPW;
  int c0, c1;                       // this thread's chunks of a head
  chunks_of<D, ROT>(j, p.rot / 16, c0, c1);
  const int apart = 8 * (c1 - c0);
  const uint16_t* const src_q = p.q + tok * p.qs + 8 * c0;
  const uint16_t* const src_k = p.k + tok * p.ks + 8 * c0;
  const uint16_t* const src_v = p.v + tok * p.vs + 8 * c0;
  // pass i is of q, k or v (kind 0, 1, 2), head h this thread's
  auto kind_of = [&](int i) { return i < q_passes ? 0 : i < k_end ? 1 : 2; };
  auto head_of = [&](int i, int kind) {
    return (i - (kind == 0 ? 0 : kind == 1 ? q_passes : k_end)) * HPW + lane / LPH;
  };
  // every pass's rows are asked for at once, each thread's chunks to its own places: no thread waits for another's
  extern __shared__ __align__(16) uint4 rows[];
  uint4* const buf = rows + (threadIdx.x >> 5) * chunk * 64 + lane;
#pragma unroll 1
  for (int i = first; i < end; ++i) {
    const int kind = kind_of(i), h = head_of(i, kind);
    const uint16_t* src = (kind == 0 ? src_q : kind == 1 ? src_k : src_v) + h * D;
    if (h < (kind == 0 ? p.Hq : p.Hkv)) {
      const uint32_t dst = smem_u32(buf + (i - first) * 64);
      cp_async16(dst, src);
      cp_async16(dst + 512, src + apart);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  for (int i = end - first; i < kChunk; ++i) asm volatile("cp.async.commit_group;" ::: "memory");
  int64_t slot = -1;
  if (p.slots) slot = p.slots[tok];
  Angles angles;
  if (ROT != kNone) {
    const int64_t at = p.pos[tok];
    if (at < 0 || at >= p.num_pos) {
      if (lane == 0) report_error(p.err, kErrBounds);
      return;
    }
    if (first < k_end) load_angles<D, ROT>(p, at, j, angles);
  }
  const bool stored = slot >= 0 && slot < p.num_slots;
  if (p.slots && !stored && first == 0 && lane == 0) report_error(p.err, kErrBounds);
  float g[16];                      // the weights of the kind that was normed last
  int of = -1;
#pragma unroll 1
  for (int i = first; i < end; ++i) {
    const int kind = kind_of(i), h = head_of(i, kind);
    const bool mine = h < (kind == 0 ? p.Hq : p.Hkv);
    // a group a pass, and one more ahead of each pass: all but the last kChunk - 1 have landed, this pass's rows and the next one's
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group %0;" ::"n"(kChunk - 1) : "memory");
    uint4 y0 = buf[(i - first) * 64], y1 = buf[(i - first) * 64 + 32];
    if (kind < 2) {
      float x[16];
      unpack8(y0, x);
      unpack8(y1, x + 8);
      const uint16_t* weight = kind == 0 ? p.wq : p.wk;
      if (weight) {
        if (of != kind) {
          of = kind;
          unpack8(reinterpret_cast<const uint4*>(weight)[c0], g);
          unpack8(reinterpret_cast<const uint4*>(weight)[c1], g + 8);
        }
        uint64_t sum = 0;
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const uint64_t v = f2pack(x[k], x[k + 1]);
          sum = ffma2(v, v, sum);
        }
        float ss, odd;
        f2unpack(sum, ss, odd);
        ss += odd;
#pragma unroll
        for (int off = 1; off < LPH; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        const uint64_t rr = f2pack(r, r);
#pragma unroll
        for (int k = 0; k < 16; k += 2)
          f2unpack(mul2(mul2(f2pack(x[k], x[k + 1]), rr), f2pack(g[k], g[k + 1])), x[k], x[k + 1]);
      }
      rotate<D, ROT>(p, j, angles, x);
      y0 = pack8(x);
      y1 = pack8(x + 8);
      uint16_t* out = kind == 0 ? p.q_out + tok * p.qos : p.k_out ? p.k_out + tok * p.kos : nullptr;
      if (out && mine) {
        *reinterpret_cast<uint4*>(out + h * D + 8 * c0) = y0;
        *reinterpret_cast<uint4*>(out + h * D + 8 * c1) = y1;
      }
      if (kind == 0 || !p.slots) continue;
    }
    if (KV4) {
      store_codes<D, ROT == kPart>(y0, y1, p.rows + slot * kv4::row_bytes(p.Hkv, D), p.Hkv, h, kind == 2, j, c0, c1, stored && mine);
    } else if (stored && mine) {
      uint16_t* out = (kind == 1 ? p.cold_k : p.cold_v) + (slot * p.Hkv + h) * D + 8 * c0;
      *reinterpret_cast<uint4*>(out) = y0;
      *reinterpret_cast<uint4*>(out + apart) = y1;
    }
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
  float one;                      // as in QkvParams
  int32_t* err;
};

// bf16(lo + code * step) of the eight codes of a word, product and sum rounded to fp32.  A nibble becomes a number where it
// stands: the low bits of 2^23, less 2^23, are the code times a power of 16, and that power's part of the step meets it.
__device__ __forceinline__ uint4 values8(uint32_t w, float lo, float step, uint64_t one) {
  constexpr uint32_t kBits = 0x4b000000u;  // 2^23
  const uint64_t base = f2pack(-8388608.f, -8388608.f), ll = f2pack(lo, lo);
  const uint64_t s01 = f2pack(step, step * 0x1p-4f), s23 = f2pack(step * 0x1p-8f, step * 0x1p-12f);
  auto pair = [&](uint32_t v, uint32_t m0, uint32_t m1, uint64_t s) {
    float a, b;
    f2unpack(ffma2(mul2(fadd2(f2pack(__uint_as_float((v & m0) | kBits), __uint_as_float((v & m1) | kBits)), base), s), one, ll), a, b);
    return pack_bf16x2(a, b);
  };
  const uint32_t h = w >> 16;
  return make_uint4(pair(w, 0xfu, 0xf0u, s01), pair(w, 0xf00u, 0xf000u, s23), pair(h, 0xfu, 0xf0u, s01), pair(h, 0xf00u, 0xf000u, s23));
}

template <int D, bool KV4, int U>
__global__ void __launch_bounds__(32 * kWarps) read_kernel(const ReadParams p, uint32_t warps_per_token) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, j = lane % LPH;
  // (at most 2^27 tokens of four warps)
  const uint32_t w = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t tok = w / warps_per_token;
  if (tok >= p.n) return;
  const int hh0 = (int)(w % warps_per_token) * HPW * U + lane / LPH;
  const int64_t slot = p.slots[tok];
  const bool ok = slot >= 0 && slot < p.num_slots;
  if (!ok && hh0 == 0 && j == 0) report_error(p.err, kErrBounds);
  // every pass's loads before the first is used
  uint4 y[U][2];
  uint32_t sc[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int hh = hh0 + u * HPW;
    const bool is_v = hh >= p.Hkv;
    const int h = is_v ? hh - p.Hkv : hh;
    y[u][0] = y[u][1] = make_uint4(0, 0, 0, 0);
    sc[u][0] = sc[u][1] = 0;
    if (!ok || hh >= 2 * p.Hkv) continue;
    if (KV4) {
      const uint8_t* row = p.rows + slot * kv4::row_bytes(p.Hkv, D);
      const uint32_t* codes = reinterpret_cast<const uint32_t*>(row + kv4::codes_at(h, D) + (is_v ? D / 2 : 0));
      const uint32_t* scales = reinterpret_cast<const uint32_t*>(row + kv4::scales_at(p.Hkv, h, D) + (is_v ? D / 16 : 0));
      if (D == 64) {
        y[u][0].x = codes[j];
        y[u][1].x = codes[j + LPH];
        sc[u][0] = sc[u][1] = scales[0];
      } else {
        const uint2 c = reinterpret_cast<const uint2*>(codes)[j], s = *reinterpret_cast<const uint2*>(scales);
        y[u][0].x = c.x;
        y[u][1].x = c.y;
        sc[u][0] = s.x;
        sc[u][1] = s.y;
      }
    } else {
      const uint16_t* src = (is_v ? p.cold_v : p.cold_k) + (slot * p.Hkv + h) * D;
      y[u][0] = load_once(src + 8 * j);
      y[u][1] = load_once(src + 8 * (j + LPH));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int hh = hh0 + u * HPW;
    if (hh >= 2 * p.Hkv) continue;
    const bool is_v = hh >= p.Hkv;
    uint4* out = reinterpret_cast<uint4*>(is_v ? p.v + tok * p.vs + (hh - p.Hkv) * D : p.k + tok * p.ks + hh * D);
    if (KV4) {
#pragma unroll
      for (int b = 0; b < 2; ++b) y[u][b] = values8(y[u][b].x, bf_lo(sc[u][b]), __fdiv_rn(bf_hi(sc[u][b]), 15.f), f2pack(p.one, p.one));
    }
    out[j] = y[u][0];
    out[j + LPH] = y[u][1];
  }
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

template <int D, int ROT, bool KV4>
int launch_qkv_u(const QkvParams& p, int num_sms, cudaStream_t st) {
  const int per = 512 / D, kv = (p.Hkv + per - 1) / per, passes = (p.Hq + per - 1) / per + kv * (p.slots ? 2 : 1);
  // The fewest passes a warp with which one wave of warps takes all, up to four; else kChunk.  40/8 heads of 128, against
  // one pass while an SM has up to 64 of them: bf16 rows of 512 tokens 4.4 -> 3.6 us, 768 6.4 -> 4.5, 1024 6.8 -> 5.2; from
  // five on (1500 tokens) 10.4 where seven take 10.0.
  const int64_t room = (int64_t)num_sms * kWarps * kBlocks, waves = ((int64_t)p.n * passes + room - 1) / room;
  const int chunk = waves > 4 ? kChunk : (int)waves;
  const int parts = (passes + chunk - 1) / chunk, each = (passes + parts - 1) / parts;
  const int64_t blocks = ((int64_t)p.n * parts + kWarps - 1) / kWarps;
  return (int)launch_pdl(qkv_kernel<D, ROT, KV4>, dim3((unsigned)blocks), dim3(32 * kWarps), kWarps * each * 1024, st, p, passes, (uint32_t)parts, each);
}

template <int D, int ROT>
int launch_qkv_t(bool kv4, const QkvParams& p, int num_sms, cudaStream_t st) {
  return kv4 ? launch_qkv_u<D, ROT, true>(p, num_sms, st) : launch_qkv_u<D, ROT, false>(p, num_sms, st);
}

template <int D>
int launch_qkv_d(bool kv4, const QkvParams& p, bool interleaved, int num_sms, cudaStream_t st) {
  if (p.rot == 0) return launch_qkv_t<D, kNone>(kv4, p, num_sms, st);
  if (interleaved) return launch_qkv_t<D, kPairs>(kv4, p, num_sms, st);
  return p.rot == D ? launch_qkv_t<D, kHalves>(kv4, p, num_sms, st) : launch_qkv_t<D, kPart>(kv4, p, num_sms, st);
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
  p.one = 1.f;
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
  return c.head_dim == 128 ? launch_qkv_d<128>(kv4, p, x->interleaved != 0, lc.num_sms, st)
                           : launch_qkv_d<64>(kv4, p, x->interleaved != 0, lc.num_sms, st);
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
  p.one = 1.f;
  p.err = lc.d_error;
  const int per = 512 / c.head_dim, passes = (2 * c.num_kv_heads + per - 1) / per;
  // a warp of each pass while the SMs hold them all, or where a token has only one (65536 tokens of 4 heads of 64 in 4 bits: 18
  // us, 21 with loops of four); else four a warp (of 8 heads of 128: 53, 68 with one)
  const int u = passes == 1 || n * passes <= (int64_t)lc.num_sms * kFewWarps ? 1 : 4;
  const int warps = (passes + u - 1) / u;
  const int64_t blocks = (n * warps + kWarps - 1) / kWarps;
  auto kern = c.head_dim == 128
                  ? (u == 1 ? (kv4 ? read_kernel<128, true, 1> : read_kernel<128, false, 1>)
                            : (kv4 ? read_kernel<128, true, 4> : read_kernel<128, false, 4>))
                  : (u == 1 ? (kv4 ? read_kernel<64, true, 1> : read_kernel<64, false, 1>)
                            : (kv4 ? read_kernel<64, true, 4> : read_kernel<64, false, 4>));
  return (int)launch_pdl(kern, dim3((unsigned)blocks), dim3(32 * kWarps), 0, (cudaStream_t)stream, p, (uint32_t)warps);
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
