// Decode over 4-bit COLD rows (gk_decode_kv4): the suffix gather over codes, and the
// log-sum-exp join of its partial states with those of the prefix items.
//
// With k_c = lo + code_c * (span / 15) in each group of 64 channels,
//   q . k = sum_groups span / 15 * (q_g . code_g) + lo * sum(q_g)
//   sum_j p_j v_j = sum_j (p_j span_j / 15) code_j + sum_j p_j lo_j   in each group's channels,
// so the two products run on codes alone and a token's scales meet its score and its weight.
//
// What bounds it: 4.5 bits an element, (d + d / 8) bytes a token and KV head, from HBM; 4 g d operations
// for them on the warp-level tensor cores.  At HBM speed an SM has about 800 instruction slots for 32 tokens of
// one head (d = 128), so the instructions a token costs decide how near the gather comes.  Codes become
// operands by one logic instruction a pair: the pair (code & 0x000f000f) read as fp16 is the subnormal pair
// code * 2^-24, and (code & 0x00f000f0) is 16 * code * 2^-24, both exact, and the tensor core multiplies
// subnormals exactly; the factor 16 goes into the query's fragment.  For V the second operand is the whole byte,
// code + 16 * code', from whose sum the first one's is taken in the end.  (As 8-bit floats four codes would take one
// mask, but the warp-level products of 8-bit operands cost several times the fp16 ones on this chip: 608 requests of
// 2048 tokens took 450 us so and 265 with fp16.)
//
// GB300, 4 requests of 262144 tokens, 32/8 heads of 128, pages of 16 (1.2 GB of rows): 210 us, 5.8 TB/s, 85 % of the
// measured copy rate; the same work on rows that stay in L2 takes 177, so instructions bind it next to HBM, half
// of the issue slots and of the ALU pipe's (masks, byte permutes, integer tests) busy.
#include <cmath>

#include "device_common.cuh"
#include "gk_internal.h"
#include "kv4.cuh"
#include "max_nan.cuh"

namespace gk {
namespace {

constexpr int kTok = kKv4Tokens;
constexpr int kSmWarps = 16;   // warps of an SM: 128 registers a thread
constexpr size_t kSmSmem = 228 * 1024;  // shared memory of an SM, 1 KB of it taken by each resident CTA

struct Kv4Params {
  const uint8_t* rows;        // the layer's
  int64_t num_blocks;
  int32_t page, page_shift;   // log2(page), or -1
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

constexpr int kSegCache = 32;  // segment records a CTA keeps in shared memory

constexpr int kStages = 2;     // of a warp's ring (three cost 2 %)

// a stage of one warp: K codes, V codes, scales of kTok tokens
__host__ __device__ constexpr int stage_bytes(int d) { return kTok * (d + d / 8); }

// D (16x8, fp32) += A (16x16, row) . B (16x8, col), fp16
__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same onto zeros
__device__ __forceinline__ void mma_f16_first(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// D (16x8, fp32) = A (16x8, row) . B (8x8, col), bf16
__device__ __forceinline__ void mma_bf16_first(float* d, uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
// D (16x8, fp32) = A (16x16, row) . B (16x8, col), bf16
__device__ __forceinline__ void mma_bf16_first(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// of two fp16 each, NaN where either is
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
// 2^e as fp32, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// floor(log2 x) of a normal x >= 0; -127 for 0
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }

constexpr float kSlack = 4.f;
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u, kByte = 0x00ff00ffu;

// Warp h of a CTA is KV head h and its G query heads, and moves its own data: it copies its head's codes and
// scales of 32 tokens a stage with cp.async into a private ring, kStages - 1 ahead of its compute, so no
// warp waits for another; 16 warps share an SM.  Block ids are loaded a stage before its copies.
//
// A stage is two tiles of 16 tokens.  S^T[16 tok x 8] = K . Q^T: a thread's 16 bytes of a token's K row are the
// A fragments of all eight k16 steps (the row's order, kv4.cuh, is made for that).  Rows r = 0 .. 7 of a
// tile are tokens (r >> 1) + 4 (r & 1) of its half, which lets the V loads below go without bank conflicts.
// O^T[d x 8] += V^T . P^T: a thread's 8 bytes of each of four tokens, paired by two byte permutes, are the A fragments
// of all m16 tiles; P^T is the weights of both heads a thread scored, times the token's span, through movmatrix.
//
// Up to four query heads fill half of the eight columns, so the columns are paired: column c + 4 is head c again, and
// of the scores a column c < 4 takes the first tile's and c + 4 the second's.  A thread then scales, weighs and sums half as many scores,
// none of them idle; P^T meets a tile with the other tile's columns masked, and the two halves of O are added in
// the end.  On rows in L2 4 requests of 262144 tokens (g = 4) take 187 us without it and 171 with it, from HBM 212 and 210.
template <int D, int G>
__global__ void __launch_bounds__(32 * kMaxKvHeads, kSmWarps / kMaxKvHeads) kv4_gather_kernel(const Kv4Params p) {
  constexpr int NG = D / 64;         // groups
  constexpr int KW = D / 32;         // words of K a thread takes of a token
  constexpr int MT = D / 16;         // m16 tiles of O^T
  constexpr int NST = kStages;
  constexpr int CPT = D / 16;        // 16-byte chunks of a token's codes (K and V)
  constexpr int TPI = 32 / CPT;      // tokens a copy instruction of the warp covers
  constexpr bool PAIR = G <= 4;
  constexpr int NS = PAIR ? 1 : 2;   // score fragments of a thread
  constexpr int SHARE = PAIR ? 2 : 4;  // lanes that far apart and further hold the same heads
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int4 cache[kSegCache];
  const int lane = threadIdx.x & 31, h = threadIdx.x >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  // The CTA's segments: the plan's tables are not written by the kernels of a step, so the records are read while the
  // kernel ahead ends, and a change of segment costs no trip to memory.
  const int sg0 = p.seg_begin[blockIdx.x], sg1 = p.seg_begin[blockIdx.x + 1];
  for (int i = threadIdx.x; i < min(sg1 - sg0, kSegCache); i += blockDim.x)
    cache[i] = *reinterpret_cast<const int4*>(p.segs + sg0 + i);
  __syncthreads();
  auto seg_at = [&](int i) {         // request, first and end token, partial state
    return i - sg0 < kSegCache ? cache[i - sg0] : *reinterpret_cast<const int4*>(p.segs + i);
  };
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t ring = smem_u32(smem) + h * NST * stage_bytes(D);
  const int row_bytes = kv4::row_bytes(p.Hkv, D);
  const uint8_t* const code_src = p.rows + kv4::codes_at(h, D) + (lane % CPT) * 16;
  const uint8_t* const scale_src = p.rows + kv4::scales_at(p.Hkv, h, D);

  // ---- copies ----
  // where this thread's chunk of the tokens it copies lands: token T's K row at place T ^ bit 2 of T (d = 128; at d = 64
  // T ^ 2 * bit 2), its V row at T with the halves swapped by bit 1 (d = 128), for conflict-free loads
  uint32_t dst0, dst1;
  {
    const int t = lane / CPT, c = lane % CPT;
    if (c < CPT / 2) {
      if (D == 128) {                // t = 0 .. 3; a step adds 4, which flips bit 2
        dst0 = t * 64 + c * 16;
        dst1 = (t ^ 1) * 64 + c * 16;
      } else {                       // t = 0 .. 7; a step adds 8
        dst0 = dst1 = (t ^ ((t >> 2 & 1) << 1)) * 32 + c * 16;
      }
    } else {
      const int cv = c - CPT / 2;
      dst0 = dst1 = kTok * (D / 2) + (D == 128 ? t * 64 + (cv ^ ((t >> 1 & 1) << 1)) * 16 : t * 32 + cv * 16);
    }
  }
  // a segment's query rows to L1, a 128-byte line a thread, when its first stage is looked up
  auto prefetch_q = [&](int32_t req) {
    const char* row = reinterpret_cast<const char*>(p.q + ((int64_t)req * p.Hq + h * G) * D) + lane * 128;
    if (lane * 128 < G * D * 2) asm volatile("prefetch.global.L1 [%0];" ::"l"(row));
  };
  int lsg = sg0, lt = 0, lt1 = 0;     // the look-up's segment and tokens
  const int32_t* ltab = nullptr;
  auto look_at = [&]() {
    if (lsg < sg1) {
      const int4 s = seg_at(lsg);
      lt = s.y;
      lt1 = s.z;
      ltab = p.table + (int64_t)s.x * p.max_blocks;
      prefetch_q(s.x);
    }
  };
  // tokens of the next stage (0: none left), and this thread's token's block id and place in the block
  auto lookup = [&](int& n, int32_t& id, int32_t& in_page) {
    n = 0;
    if (lsg < sg1) {
      n = min(kTok, lt1 - lt);
      const int t = lt + lane;
      const int b = p.page_shift >= 0 ? t >> p.page_shift : t / p.page;
      in_page = t - b * p.page;
      if (lane < n) id = __ldcg(ltab + b);
      lt += n;
      if (lt == lt1) {
        ++lsg;
        look_at();
      }
    }
  };
  int next = 0;
  auto issue = [&](int idn, int32_t id, int32_t in_page) {
    if (idn > 0) {
      const bool bad = lane < idn && (id < 0 || id >= p.num_blocks);
      int32_t slot = lane < idn && !bad ? id * p.page + in_page : 0;
      if (idn < kTok) slot = __shfl_sync(0xffffffffu, slot, min(lane, idn - 1));
      const uint32_t st = ring + (uint32_t)next * stage_bytes(D);
      // places past the stage's tokens get its last token's row: they meet weights and spans of 0
      const uint32_t sdst = st + kTok * D;
      // Pages of one token: 32 places at once cost address translations that one instruction for the stage's scales waits
      // for in turn (608 requests of 2048 tokens, 8 KV heads of 128: 463 us), so the threads that copy a few tokens' codes next
      // touch those rows' scales first (253; 280 behind the codes, 385 a copy later).  At d = 64, 304 requests of 4096: 8 KV heads
      // 195 so and 260 by one instruction, 4 heads 87 and 85.  From pages of two on the one instruction takes 238, the other 255.
      if (p.page > 1) {
#pragma unroll
        for (int j = 0; j < kTok / TPI; ++j) {
          const int32_t s = __shfl_sync(0xffffffffu, slot, j * TPI + lane / CPT);
          copy_async<16>(st + (j & 1 ? dst1 : dst0) + j * TPI * (D / 2), code_src + (int64_t)s * row_bytes);
        }
        copy_async<D / 8>(sdst + lane * (D / 8), scale_src + (int64_t)slot * row_bytes);
      } else {
#pragma unroll
        for (int j = 0; j < kTok / TPI; ++j) {
          const int32_t s = __shfl_sync(0xffffffffu, slot, j * TPI + lane / CPT);
          if (lane % CPT == 0)
            copy_async<D / 8>(sdst + (j * TPI + lane / CPT) * (D / 8), scale_src + (int64_t)s * row_bytes);
          copy_async<16>(st + (j & 1 ? dst1 : dst0) + j * TPI * (D / 2), code_src + (int64_t)s * row_bytes);
        }
      }
      uint32_t zero = __ballot_sync(0xffffffffu, bad);
      if (zero) {
        // ids outside the pool: their tokens' rows count as zeros, and the last token's so do in the places past the stage's, as a
        // NaN there, though it meets weights of 0, would reach the scores of the other tile's row through the product with lo
        if (zero >> (idn - 1)) zero |= ~0u << (idn - 1);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        if (bad) report_error(p.err, kErrBounds);
        for (uint32_t left = zero; left; left &= left - 1) {
          const int t = __ffs(left) - 1;
          const uint32_t k = D == 128 ? st + (t ^ (t >> 2 & 1)) * 64 : st + (t ^ (t >> 2 & 1) << 1) * 32;
          const uint32_t v = st + kTok * (D / 2) + t * (D / 2) - D / 2;
          if (lane < D / 16) sts128((lane < D / 32 ? k : v) + lane * 16, make_uint4(0, 0, 0, 0));
          if (lane < D / 64) asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(st + kTok * D + t * (D / 8) + lane * 8), "r"(0) : "memory");
        }
        __syncwarp();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++next == NST) next = 0;
  };
  look_at();
  int nid;                           // the stage whose ids are on their way
  int32_t id = 0, in_page = 0;
  {
    int n[NST - 1];
    int32_t ids[NST - 1] = {}, at[NST - 1] = {};
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) lookup(n[i], ids[i], at[i]);
    lookup(nid, id, in_page);
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) issue(n[i], ids[i], at[i]);
  }

  // ---- compute ----
  const int ta = (gq >> 1) + 4 * (gq & 1);                 // this thread's row of a half tile, as a token
  const uint32_t k_at = D == 128 ? (uint32_t)((ta ^ (gq & 1)) * 64 + tq * 16) : (uint32_t)((ta ^ ((gq & 1) << 1)) * 32 + tq * 8);
  const uint32_t v_at = kTok * (D / 2) +
                        (D == 128 ? tq * 64 + ((gq >> 1) ^ ((tq >> 1) << 1)) * 16 + (gq & 1) * 8 : tq * 32 + gq * 4);
  const uint32_t first = gq < 4 ? ~0u : 0u;                // paired: of weights, whose column is the first tile's
  // of the query's fragments; columns without a head repeat another's, so that what a warp finds over all of them (the largest
  // product of weight and span) is of rows that count
  const int head = (PAIR ? gq & 3 : gq) % G;
  const int half = PAIR ? tq >> 1 : 0;                     // this thread's tile
  const uint32_t s_at = kTok * D + (ta + 16 * half) * (D / 8);
  int cslot = 0;
  for (int sg = sg0; sg < sg1; ++sg) {
    const int4 seg = seg_at(sg);
    const int32_t dest = seg.w >= 0 ? seg.w : ~seg.x;
    // Q as B fragments: the channels of a thread's word i of K, paired (c, c + 4); scaled by a power of two to
    // between 2^13 and 2^14, and the odd channels, whose codes come 16 times as large, by 2^-4 of it: fp16 holds a head's bf16
    // values to half a step of 2^-24, 2^-38 of the largest in the even channels and 2^-34 in the odd ones
    uint32_t qf[KW][4];
    float F[2];
    // sum(q) of each group (times scale) as the B fragment that meets lo: column gq, rows 2 tq and 2 tq + 1 the groups' tq-th
    // bf16 terms, three of which make fp32 (paired: rows of the column's own tile, terms tq & 1 and 2 + (tq & 1))
    uint32_t zf[2] = {};
    {
      uint4 raw[KW];
      float top = 0.f, sum[NG] = {};
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const int w = KW * tq + i, ch = D == 128 ? 8 * (w >> 1) + 64 * (w & 1) : 8 * w;   // channels ch .. ch + 7
        raw[i] = *reinterpret_cast<const uint4*>(p.q + ((int64_t)seg.x * p.Hq + h * G + head) * D + ch);
      }
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const uint32_t r[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          top = fmaxf(top, fmaxf(fabsf(bf_lo(r[c])), fabsf(bf_hi(r[c]))));
          sum[D == 128 ? i & 1 : 0] += bf_lo(r[c]) + bf_hi(r[c]);
        }
      }
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
#pragma unroll
        for (int g = 0; g < NG; ++g) sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], off);
      }
      const int e = min(120, 13 - exponent(top));
      const float s = pow2(e), s16 = pow2(e - 4);
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const uint4 r = raw[i];
        qf[i][0] = pack_f16x2(bf_lo(r.x) * s, bf_lo(r.z) * s);
        qf[i][1] = pack_f16x2(bf_hi(r.x) * s16, bf_hi(r.z) * s16);
        qf[i][2] = pack_f16x2(bf_lo(r.y) * s, bf_lo(r.w) * s);
        qf[i][3] = pack_f16x2(bf_hi(r.y) * s16, bf_hi(r.w) * s16);
      }
      const float f = p.scale * (16777216.f / 15.f) * pow2(-e);
#pragma unroll
      for (int k = 0; k < 2; ++k) F[k] = __shfl_sync(0xffffffffu, f, 4 * (2 * tq + k));   // of query heads 2 tq and 2 tq + 1
      float z[2] = {sum[0] * p.scale, NG == 2 ? sum[NG - 1] * p.scale : 0.f};
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const uint32_t term = pack_bf16x2(z[0], z[1]);
        if (PAIR ? (gq >> 2) == half && (tq & 1) == (k & 1) : tq == k) zf[PAIR ? k >> 1 : 0] = term;
        z[0] -= bf_lo(term);
        z[1] -= bf_hi(term);
      }
    }
    float o[MT][4], R[NG][2] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {};
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    // fp16 holds a token's weight times its group's span, scaled by the group's power of two vs: the largest product of the stage that
    // chose vs is below 2^11, those of later stages below 2^15, or vs is chosen again.  One below fp16's normal range is off by
    // 2^-35 of that largest product at most.  (The product, not the span: a token of wide values and no weight must not take the
    // others' bits.  4 requests of 262144 tokens take 209 us by either, on rows in L2 171 by spans and 177 by products.)
    float vs[NG];                      // 0: not chosen yet
#pragma unroll
    for (int g = 0; g < NG; ++g) vs[g] = 0.f;

    for (int left = seg.z - seg.y; left > 0; left -= kTok) {
      const int n = min(kTok, left);
      issue(nid, id, in_page);
      lookup(nid, id, in_page);
      asm volatile("cp.async.wait_group %0;" ::"n"(NST - 1) : "memory");
      __syncwarp();
      const uint32_t st = ring + (uint32_t)cslot * stage_bytes(D);
      if (++cslot == NST) cslot = 0;
      // scores
      float sc[NS][4];                 // rows ta and ta + 8 of a tile, heads 2 tq and 2 tq + 1 (paired: 2 (tq & 1) and the next)
      uint32_t vscale[NS][2][NG];      // V's (lo, span) of those tokens
      // K's (lo, span) of a fragment's tokens, and V's
      auto scales = [&](uint32_t at, uint32_t* ka, uint32_t* kb, uint32_t (*v)[NG]) {
        if (D == 128) {
          const uint4 a = lds128(at), b = lds128(at + 8 * (D / 8));
          ka[0] = a.x; ka[NG - 1] = a.y; v[0][0] = a.z; v[0][NG - 1] = a.w;
          kb[0] = b.x; kb[NG - 1] = b.y; v[1][0] = b.z; v[1][NG - 1] = b.w;
        } else {
          const uint2 a = lds64(at), b = lds64(at + 8 * (D / 8));
          ka[0] = a.x; v[0][0] = a.y;
          kb[0] = b.x; v[1][0] = b.y;
        }
      };
      auto both_lo = [&](const uint32_t* k) { return NG == 2 ? __byte_perm(k[0], k[NG - 1], 0x5410) : k[0] & 0xffffu; };
      auto products = [&](int u, float (*acc)[4]) {
        uint32_t wa[KW], wb[KW];
        const uint32_t kt = st + k_at + u * 16 * (D / 2);
        if (D == 128) {
          const uint4 a = lds128(kt), b = lds128(kt + 8 * (D / 2));
          wa[0] = a.x; wa[1] = a.y; wa[KW - 2] = a.z; wa[KW - 1] = a.w;
          wb[0] = b.x; wb[1] = b.y; wb[KW - 2] = b.z; wb[KW - 1] = b.w;
        } else {
          const uint2 a = lds64(kt), b = lds64(kt + 8 * (D / 2));
          wa[0] = a.x; wa[1] = a.y;
          wb[0] = b.x; wb[1] = b.y;
        }
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          float* d = acc[D == 128 ? i & 1 : 0];
          if (i < NG)
            mma_f16_first(d, wa[i] & kLow, wb[i] & kLow, wa[i] & kHigh, wb[i] & kHigh, qf[i][0], qf[i][1]);
          else
            mma_f16(d, wa[i] & kLow, wb[i] & kLow, wa[i] & kHigh, wb[i] & kHigh, qf[i][0], qf[i][1]);
          const uint32_t xa = wa[i] >> 8, xb = wb[i] >> 8;
          mma_f16(d, xa & kLow, xb & kLow, xa & kHigh, xb & kHigh, qf[i][2], qf[i][3]);
        }
      };
      auto scaled = [&](float* s, const uint32_t* ka, const uint32_t* kb, const float (*acc)[4]) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float da = bf_hi(ka[0]) * acc[0][k], db = bf_hi(kb[0]) * acc[0][2 + k];
          if (NG == 2) {
            da = fmaf(bf_hi(ka[NG - 1]), acc[NG - 1][k], da);
            db = fmaf(bf_hi(kb[NG - 1]), acc[NG - 1][2 + k], db);
          }
          s[k] = fmaf(da, F[k], s[k]);
          s[2 + k] = fmaf(db, F[k], s[2 + k]);
        }
      };
      uint32_t ka[NG], kb[NG];
      if (PAIR) {
        float acc[NG][4], other[NG][4];
        scales(st + s_at, ka, kb, vscale[0]);
        const uint32_t la = both_lo(ka), lb = both_lo(kb);
        mma_bf16_first(sc[0], la, lb, la, lb, zf[0], zf[1]);
        products(0, acc);
        products(1, other);
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (half) acc[g][i] = other[g][i];
        scaled(sc[0], ka, kb, acc);
      } else {
#pragma unroll
        for (int u = 0; u < NS; ++u) {
          float acc[NG][4];
          scales(st + s_at + u * 16 * (D / 8), ka, kb, vscale[u]);
          // the part of lo: k = 2 tq and 2 tq + 1 are the row's two groups
          mma_bf16_first(sc[u], both_lo(ka), both_lo(kb), zf[0]);
          products(u, acc);
          scaled(sc[u], ka, kb, acc);
        }
      }
      if (n < kTok) {
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (16 * (u + half) + 8 * r + ta >= n) {
              sc[u][2 * r] = sc[u][2 * r + 1] = -INFINITY;
#pragma unroll
              for (int g = 0; g < NG; ++g) vscale[u][r][g] = 0;
            }
      }
      // The exponents' reference m is raised only where a score passes it by kSlack (a vote in place of a
      // maximum over the warp).
      float d[NS][4];
#pragma unroll
      for (int u = 0; u < NS; ++u)
#pragma unroll
        for (int i = 0; i < 4; i += 2)
          f2unpack(fadd2(f2pack(sc[u][i], sc[u][i + 1]), f2pack(-m[0], -m[1])), d[u][i], d[u][i + 1]);
      float past = fmaxf(fmax3(d[0][0], d[0][1], d[0][2]), d[0][3]);
      if (!PAIR) past = fmax3(fmax3(past, d[NS - 1][0], d[NS - 1][1]), d[NS - 1][2], d[NS - 1][3]);
      bool again = false;              // choose vs: weights of before are smaller now, and so may be all that is to come
      if (__any_sync(0xffffffffu, past > kSlack)) {
        float x0 = fmaxf(fmaxf(sc[0][0], sc[0][2]), fmaxf(sc[NS - 1][0], sc[NS - 1][2]));
        float x1 = fmaxf(fmaxf(sc[0][1], sc[0][3]), fmaxf(sc[NS - 1][1], sc[NS - 1][3]));
#pragma unroll
        for (int off = SHARE; off < 32; off <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
        }
        x0 = fmaxf(m[0], x0);
        x1 = fmaxf(m[1], x1);
        float a0 = ex2(m[0] - x0), a1 = ex2(m[1] - x1);
        if (x0 == m[0]) a0 = 1.f;      // -inf - -inf
        if (x1 == m[1]) a1 = 1.f;
        l[0] *= a0;
        l[1] *= a1;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          R[g][0] *= a0;
          R[g][1] *= a1;
        }
        if (vs[0] != 0.f) {
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            o[i][0] *= a0; o[i][1] *= a1; o[i][2] *= a0; o[i][3] *= a1;
          }
        }
        m[0] = x0;
        m[1] = x1;
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) d[u][i] = sc[u][i] - m[i & 1];
        again = true;
      }
      float e[NS][4];                  // rows a and b of the first head, then of the second
#pragma unroll
      for (int u = 0; u < NS; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) e[u][i] = ex2(d[u][i]);
        l[0] += e[u][0];
        l[0] += e[u][2];
        l[1] += e[u][1];
        l[1] += e[u][3];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float la = bf_lo(vscale[u][0][g]), lb = bf_lo(vscale[u][1][g]);
          R[g][0] = fmaf(e[u][0], la, R[g][0]);
          R[g][1] = fmaf(e[u][1], la, R[g][1]);
          R[g][0] = fmaf(e[u][2], lb, R[g][0]);
          R[g][1] = fmaf(e[u][3], lb, R[g][1]);
        }
      }
      // products of weight and span, scaled, of rows a and b, both heads a word
      uint32_t ws[NS][NG][2], high = 0;
      auto weigh = [&](bool wide) {
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const uint64_t span = f2pack(bf_hi(vscale[u][0][g]), bf_hi(vscale[u][1][g])), by = f2pack(vs[g], vs[g]);
            const uint64_t e0 = f2pack(e[u][0], e[u][2]), e1 = f2pack(e[u][1], e[u][3]);
            float a0, b0, a1, b1;
            f2unpack(wide ? mul2(mul2(e0, span), by) : mul2(e0, mul2(span, by)), a0, b0);
            f2unpack(wide ? mul2(mul2(e1, span), by) : mul2(e1, mul2(span, by)), a1, b1);
            ws[u][g][0] = pack_f16x2(a0, a1);
            ws[u][g][1] = pack_f16x2(b0, b1);
            high = max_f16x2(max_f16x2(ws[u][g][0], ws[u][g][1]), high);
          }
      };
      if (!again) {
        weigh(false);
        // 2^15 (0x7800) and more, infinity and NaN (a span that overflows times its scale, on a weight of 0); not one is negative
        again = __any_sync(0xffffffffu, ((high + 0x08000800u) & 0x80008000u) != 0);
      }
      if (again) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float top = 0.f, held = 0.f;
#pragma unroll
          for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, e[u][i] * bf_hi(vscale[u][i >> 1][g]));
          top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
          int to = min(113, 10 - exponent(top));
          if (vs[g] != 0.f) {
            // what O holds, in a new scale too
            int by = to - exponent(vs[g]);
            if (by > 0) {
#pragma unroll
              for (int i = 4 * g; i < 4 * g + 4; ++i) held = fmaxf(fmaxf(fmaxf(fabsf(o[i][0]), fabsf(o[i][1])), fmaxf(fabsf(o[i][2]), fabsf(o[i][3]))), held);
              held = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(held)));
              by = min(by, 96 - exponent(held));
              to = exponent(vs[g]) + by;
            }
            const int half = by / 2;
            const float f = pow2(half), f2 = pow2(by - half);
#pragma unroll
            for (int i = 4 * g; i < 4 * g + 4; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k) o[i][k] = o[i][k] * f * f2;
          }
          vs[g] = pow2(to);
        }
        weigh(true);
      }
      uint32_t b[2][NG][2];            // P^T times the spans, of either tile
#pragma unroll
      for (int u = 0; u < NS; ++u)
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            b[u][g][k] = transpose8x8(ws[u][g][k]);
            if (PAIR) {
              b[1][g][k] = b[0][g][k] & ~first;
              b[0][g][k] &= first;
            }
          }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        // tokens tq, tq + 4, tq + 8, tq + 12 of the tile
        uint32_t w[4][NG];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t at = st + v_at + (u * 16 + 4 * k) * (D / 2);
          if (D == 128) {
            const uint2 x = lds64(at);
            w[k][0] = x.x;
            w[k][NG - 1] = x.y;
          } else {
            w[k][0] = lds32(at);
          }
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {      // channels 0 .. 3, then 4 .. 7
            const uint32_t x = __byte_perm(w[0][g], w[1][g], hf ? 0x7632 : 0x5410);
            const uint32_t y = __byte_perm(w[2][g], w[3][g], hf ? 0x7632 : 0x5410);
            const uint32_t x1 = __byte_perm(x, 0, 0x4341), y1 = __byte_perm(y, 0, 0x4341);
            mma_f16(o[4 * g + 2 * hf], x & kLow, x & kByte, y & kLow, y & kByte, b[u][g][0], b[u][g][1]);
            mma_f16(o[4 * g + 2 * hf + 1], x1 & kLow, x1, y1 & kLow, y1, b[u][g][0], b[u][g][1]);
          }
        }
      }
      __syncwarp();                    // every lane has read the stage before it is refilled
    }

    // the sums over tokens live on the threads that share a head, O's on the two that share its rows too
#pragma unroll
    for (int off = SHARE; off < 32; off <<= 1)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], off);
#pragma unroll
        for (int g = 0; g < NG; ++g) R[g][k] += __shfl_xor_sync(0xffffffffu, R[g][k], off);
      }
    if (PAIR) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] += __shfl_xor_sync(0xffffffffu, o[i][k], 2);
    }
    float back[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) back[g] = 1.f / vs[g];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int hh = 2 * tq + k;       // (paired: lanes from tq = 2 on hold what the others do)
      if (hh >= G) continue;
      const float inv = 1.f / l[k], f = inv * (16777216.f / 15.f);
      const int64_t row = (int64_t)(dest >= 0 ? dest : ~dest) * p.Hq + h * G + hh;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float y[8];                    // channels 64 g + 8 gq .. + 7
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[2 * i] = fmaf(o[4 * g + i][k] * f, back[g], R[g][k] * inv);
          y[2 * i + 1] = fmaf((o[4 * g + i][2 + k] - o[4 * g + i][k]) * (f * 0.0625f), back[g], R[g][k] * inv);
        }
        const int64_t at = row * D + 64 * g + 8 * gq;
        if (dest >= 0) {
          *reinterpret_cast<float4*>(p.part_o + at) = make_float4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<float4*>(p.part_o + at + 4) = make_float4(y[4], y[5], y[6], y[7]);
        } else {
          *reinterpret_cast<uint4*>(p.out + at) =
              make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
        }
      }
      if (gq == 0) {
        const float lse = m[k] + __log2f(l[k]);
        if (dest >= 0)
          p.part_l[row] = lse;
        else if (p.lse)
          p.lse[row] = lse * kLn2;
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// O = sum_e 2^(l_e - m) O_e / sum_e 2^(l_e - m), LSE = (m + log2 sum_e 2^(l_e - m)) ln 2 over the partial
// states of a request, m the largest l_e, for each query head.  WARPS warps share a row: each joins the states
// e = its index + WARPS i, then the first one theirs.  A state of LSE -inf (weight 0) may hold anything.
// SPLIT blocks share a row's channels (one request of 131072 tokens, 32 rows of 293 states: the step 36.7 us, 35.7 by four).
// Bound by latency: a warp asks for eight states' rows before it uses any.
template <int D, int WARPS, int SPLIT = 1>
__global__ void __launch_bounds__(WARPS > 8 ? 32 * WARPS : 256) kv4_join_kernel(const float* part_o, const float* part_l, const RequestDev* __restrict__ reqs,
                                                       int32_t B, int32_t Hq, uint16_t* out, float* lse) {
  constexpr int C = D / 32 / SPLIT;    // channels of a thread
  constexpr int N = WARPS > 8 ? WARPS : 8;  // warps of a block
  __shared__ float sm[N], sz[N], so[N][D / SPLIT];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % WARPS;
  const int64_t w = SPLIT > 1 ? blockIdx.x / SPLIT : blockIdx.x * (int64_t)(N / WARPS) + warp / WARPS;
  const int ch = (SPLIT > 1 ? blockIdx.x % SPLIT * (D / SPLIT) : 0) + lane * C;   // the thread's first
  const bool row = w < (int64_t)B * Hq;
  const int r = row ? (int)(w / Hq) : 0, qh = (int)(w % Hq);
  const int e0 = reqs[r].entry_cas, ne = row ? reqs[r].n_entry_cas : -1;
  griddep_wait();
  float m = -INFINITY, z = 0.f, o[C] = {};
  for (int eb = part; eb < ne; eb += 8 * WARPS) {
    float l[8], v[8][C];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int e = eb + k * WARPS;
      const int64_t at = (int64_t)(e0 + min(e, ne - 1)) * Hq + qh;
      l[k] = e < ne ? __ldcg(part_l + at) : -INFINITY;
      if (C == 4) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(part_o + at * D + ch));
        v[k][0] = x.x; v[k][1 % C] = x.y; v[k][C < 2 ? 0 : C - 2] = x.z; v[k][C - 1] = x.w;
      } else if (C == 2) {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(part_o + at * D + ch));
        v[k][0] = x.x; v[k][C - 1] = x.y;
      } else {
        v[k][0] = __ldcg(part_o + at * D + ch);
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max_nan(top, l[k]);
    if (top == -INFINITY) continue;
    const float a = ex2(m - top);
    m = top;
    z *= a;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] *= a;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = ex2(l[k] - m);
      if (x == 0.f) continue;
      z += x;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = fmaf(x, v[k][c], o[c]);
    }
  }
  if (WARPS > 1) {
    sm[warp] = m;
    sz[warp] = z;
#pragma unroll
    for (int c = 0; c < C; ++c) so[warp][lane * C + c] = o[c];
    __syncthreads();
    if (part > 0) return;
    float top = m;
#pragma unroll
    for (int k = 1; k < WARPS; ++k) top = max_nan(top, sm[warp + k]);
    if (top != -INFINITY) {
      const float a = ex2(m - top);
      z *= a;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = a == 0.f ? 0.f : o[c] * a;
#pragma unroll
      for (int k = 1; k < WARPS; ++k) {
        const float x = ex2(sm[warp + k] - top);
        if (x == 0.f) continue;
        z = fmaf(x, sz[warp + k], z);
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] = fmaf(x, so[warp + k][lane * C + c], o[c]);
      }
    }
    m = top;
  }
  if (ne < 0) return;                  // written by its only segment
  const float inv = m == -INFINITY ? 0.f : 1.f / z;
  if (C == 1) {
    out[w * D + ch] = (uint16_t)pack_bf16x2(o[0] * inv, 0.f);
  } else {
    uint32_t* dst = reinterpret_cast<uint32_t*>(out + w * D + ch);
#pragma unroll
    for (int c = 0; c < C; c += 2) dst[c / 2] = pack_bf16x2(o[c] * inv, o[(c + 1) % C] * inv);
  }
  if (ch == 0 && lse) lse[w] = m == -INFINITY ? -INFINITY : (m + __log2f(z)) * kLn2;
}

size_t gather_smem(int hkv, int d) { return (size_t)hkv * kStages * stage_bytes(d); }

template <int D, int G>
int launch_gather_t(Pool* pool, const Kv4Params& p, int ctas, cudaStream_t st) {
  const size_t smem = gather_smem(p.Hkv, D);
  auto kern = kv4_gather_kernel<D, G>;
  if (!pool->kv4_smem_set) {
    // (the most that any pool of these heads takes: the attribute is the kernel's, not the pool's)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)gather_smem(kMaxKvHeads, D));
    if (e != cudaSuccess) return (int)e;
    pool->kv4_smem_set = true;
  }
  return (int)launch_pdl(kern, dim3(ctas), dim3(32 * p.Hkv), smem, st, p);
}

}  // namespace

// As many CTAs of Hkv warps as an SM's registers (kSmWarps warps) and shared memory hold.
int kv4_ctas_per_sm(const gk_pool_config* cfg) {
  const int by_smem =
      (int)(kSmSmem / (gather_smem(cfg->num_kv_heads, cfg->head_dim) + sizeof(int4) * kSegCache + 1024));
  const int by_warps = kSmWarps / cfg->num_kv_heads;
  return by_smem < by_warps ? by_smem : by_warps;
}

int launch_kv4_gather(const LaunchCommon& lc, void* stream, int32_t layer, const gk_batch* b, const Plan* pl, void* d_out) {
  const gk_pool_config& c = *lc.cfg;
  if (pl->suf_segs.empty()) return 0;
  Kv4Params p{};
  p.rows = (const uint8_t*)c.cold_k + layer * c.cold_slots * (int64_t)kv4::row_bytes(c.num_kv_heads, c.head_dim);
  p.num_blocks = c.cold_slots / c.cold_page_size;
  p.page = c.cold_page_size;
  p.page_shift = -1;
  for (int sh = 0; sh < 31; ++sh)
    if ((1 << sh) == c.cold_page_size) p.page_shift = sh;
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
  const int ctas = pl->summary.suffix_ctas, g = c.num_q_heads / c.num_kv_heads;
  cudaStream_t st = (cudaStream_t)stream;
  if (c.head_dim == 128) {
    switch (g) {
      case 1: return launch_gather_t<128, 1>(pl->pool, p, ctas, st);
      case 2: return launch_gather_t<128, 2>(pl->pool, p, ctas, st);
      case 4: return launch_gather_t<128, 4>(pl->pool, p, ctas, st);
      case 5: return launch_gather_t<128, 5>(pl->pool, p, ctas, st);
      case 8: return launch_gather_t<128, 8>(pl->pool, p, ctas, st);
    }
  } else {
    switch (g) {
      case 1: return launch_gather_t<64, 1>(pl->pool, p, ctas, st);
      case 2: return launch_gather_t<64, 2>(pl->pool, p, ctas, st);
      case 4: return launch_gather_t<64, 4>(pl->pool, p, ctas, st);
    }
  }
  return (int)cudaErrorInvalidValue;
}

int launch_kv4_join(const LaunchCommon& lc, void* stream, const gk_batch* b, const Plan* pl, void* d_out) {
  const gk_pool_config& c = *lc.cfg;
  const int64_t rows = (int64_t)pl->B * c.num_q_heads;
  const int most = pl->kv4_most_states;
  // A warp a row while two rounds hold its states, or while the rows alone fill the SMs.  Steps of one request, 32 rows, by 1, 8
  // and 32 warps a row: 16 states 7.9, 8.0, 7.5 us, 32 10.3, 8.0, 10.1, 64 15.3, 8.6, 10.4, 128 (not by 1) 8.6, 10.2; 16 requests
  // of 19 61.1, 59.7, 67.3, 8 of 38 40.5, 35.3, 40.1, 4 of 73 23.7 by 8 and 23.3 by 32.
  const int warps = most <= 16 || rows >= 32 * (int64_t)lc.num_sms ? 1 : most <= 64 ? 8 : 32;
  // as many blocks a row as one wave holds (of 32 warps; 128 rows by four, in four waves, cost the step 10 %)
  const int most_split = c.head_dim / 32, sms = lc.num_sms;
  const int split = warps < 32 ? 1 : rows * most_split <= sms ? most_split : rows * 2 <= sms ? 2 : 1;
  auto kern = c.head_dim == 128
                  ? (warps == 1   ? kv4_join_kernel<128, 1>
                     : warps == 8 ? kv4_join_kernel<128, 8>
                     : split == 4 ? kv4_join_kernel<128, 32, 4>
                     : split == 2 ? kv4_join_kernel<128, 32, 2>
                                  : kv4_join_kernel<128, 32>)
                  : (warps == 1   ? kv4_join_kernel<64, 1>
                     : warps == 8 ? kv4_join_kernel<64, 8>
                     : split == 2 ? kv4_join_kernel<64, 32, 2>
                                  : kv4_join_kernel<64, 32>);
  return (int)launch_pdl(kern, dim3((unsigned)(warps == 1 ? (rows + 7) / 8 : rows * split)), dim3(warps == 32 ? 1024 : 256), 0,
                         (cudaStream_t)stream, pl->d_part_o, pl->d_part_l,
                         (const RequestDev*)((const uint8_t*)pl->d_buf + pl->off_reqs), pl->B, c.num_q_heads, (uint16_t*)d_out,
                         b->d_lse);
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
