// Prompt attention: causal attention of packed new tokens over their request's
// HOT prefix, its COLD tokens and themselves, on 5th-generation tensor cores.
//
// For request r with Lp HOT, c COLD and n new tokens, token i and query head h
// (KV head h / g), over the keys HOT 0..Lp-1, COLD 0..c-1, new 0..i:
//   s_j = q.k_j / sqrt(d),  m = max_j s_j,  Z = sum_j e^(s_j - m),
//   O = sum_j e^(s_j - m) v_j / Z,  LSE = m + ln Z.
// A key of one KV head is 4 d bytes and 4 d flop for each of the n g rows of the
// request's n tokens: n g flop per byte where the keys are its own, so that it is
// bound by the tensor cores above some 292 / g tokens (73 at g = 4; 1950 TFLOP/s
// against 6.69 TB/s), and by HBM or a chain of latencies below.  New tokens and
// shared prefixes are read again from L2 by each 256 rows.
//
// One work item = one KV head x 2 * tpt consecutive tokens of one request (tpt =
// floor(128 / g); the g query heads of a token are g consecutive rows, so an item
// is two 128-row Q tiles) x a range of 128-key tiles.  Keys come in tiles of one
// source each: HOT tiles (2D tensor map over the whole HOT pool), COLD tiles
// (rows gathered through the block table by four warps with 16-byte cp.async, whose
// completion arrives at the tile's barrier),
// then tiles of new tokens (3D tensor maps over the caller's packed tensors).
// S_i = Q_i K^T and O_i += P_i V accumulate in tensor memory (512 columns: S_0
// S_1 O_0 O_1; P_i overwrites S_i as bf16).  Softmax warpgroup i owns Q tile i, one
// thread per row, and one warp issues PV_0(j) S_0(j+1), PV_1(j) S_1(j+1), so that
// one tile's softmax runs under the other's products.  A tile's two products take
// 1024 tensor cycles, so its softmax has to come back in about as long; there is
// no pass for the maximum: exponents are taken against a reference that is the
// maximum over the row's first keys, raised between tiles when a tile's sum passed
// 2^8 and within one (its exponentials are then done again) when it passed 2^64,
// so that every value stays in fp32 and bf16 range.  O and LSE use the same
// reference as P, so this changes neither beyond fp32 rounding.
// P is rounded to bf16 (half a step, 2^-9 to 2^-8 of the value) because V is
// bf16 and both operands of the product have one type; the row sum adds the
// unrounded fp32 values.
//
// CTAs are persistent (one per SM: 512 tensor-memory columns and 224 KB of
// shared memory) and run the lists of items that the plan balanced.  K and V tiles
// share one ring of stages, and the loads of the next item start while the
// softmax of the last one ends.  The elements after an item's last V tile, one for each
// Q tile, stage its output: a warp of its own stores them (whole Q tiles by TMA), so
// that the softmax warps are at the next item 1300 cycles after the last product.
//
// What it measured (GB300, one layer, CUDA graph replays): 16384 tokens on 40/8 heads of
// 128 in 1630-1770 us as the power cap sets the clock, 1.55-1.68 PFLOP/s; 8192 tokens on
// 32/8 heads 331 us, 1.66 PFLOP/s, 85 % of the measured bf16 peak.  A key tile of two Q tiles takes 1.48 us, about 3050 cycles, where
// its four products alone are 2048: what bounds it is the chain S -> softmax (1400) -> PV
// and next S (1400) -> softmax with its hand-overs (250), of which the two Q tiles overlap
// all but the products.  An item costs about 3.5 us besides (first Q and S, first
// reference, output), which is what bounds short prompts: 64 prompts of 256 tokens on 32/8
// heads take 82-87 us.  COLD tiles cost 1.60 us: their copies share the schedulers with the
// softmax (two chunks of 2048 tokens over 6000-12000 in pages of 16: 465 us, 1.40 PFLOP/s).
// In short prompts a fifth of the stalls wait for instructions: the roles' code is
// 110 KB, so variants of the softmax share one copy of it.  Tried and slower, in ns a key
// tile: an issuing warp per Q tile (24 % more), its loop over the Q tiles not unrolled
// (1526 -> 1683: descriptors leave the uniform registers), two threads a row (2516,
// spilling), probabilities stored as they come (1643 -> 1876), handed over in two halves
// (1542 -> 1674: the issuing warp's waits queue behind its own products), the first
// reference from registers already loaded (1542 -> 1677, spilling), and at d = 64 P in
// columns of its own with S issued a tile ahead (6 %).
//
// Masked keys.  Scores are masked by selection, so whatever K holds in a masked
// place does no harm; the product P V, though, would turn a masked 0 times an
// infinity or NaN in V into NaN.  So V tiles with masked places (the end of a HOT
// prefix, the diagonal and the end of the new tokens) pass through the gather
// warps, which zero the rows past the end (another request's tokens) and rows that
// hold an infinity or NaN and are hidden from some row of the item; the rows that
// do see such a key add its term in the epilogue (add_hidden_values, never taken
// for finite values).
//
// Warp roles (512 threads): 0 TMA, 1 MMA and tensor memory, 2-3 and 13-14 gather
// and scan, 4-7 and 8-11 softmax of Q tiles 0 and 1, 12 operand relay, 15 output.  The
// block starts with 128 registers a thread; the softmax warpgroups take 152 and the
// other two keep 104 (spills in the softmax loop were measured to halve the kernel's
// speed, spills in the other roles to cost 6 %).
#include <cuda.h>

#include <cmath>
#include <cstring>
#include <type_traits>

#include "max_nan.cuh"
#include "prefix_body.cuh"
#include "prompt.h"

namespace gk {
namespace prompt {

using prefix::BM;
using prefix::BN;
using prefix::idesc;
using prefix::kRegionKV;
using prefix::kRegionQ;
using prefix::kTmemCols;
using prefix::sdesc;
using prefix::tc_mma_ts;

constexpr int kThreads = 512;
constexpr int kSoftmaxRegs = 152, kOtherRegs = 104;   // 128 * (2 * 152 + 2 * 104) = 512 * 128


struct Params {
  CUtensorMap tq, tk, tv, tout;   // the call's packed tensors
  CUtensorMap thk, thv;           // the HOT pool
  const PromptReqDev* reqs;
  const PromptItemDev* items;
  const int32_t* cta_begin;       // [gridDim.x + 1]
  const int32_t* block_table;
  const uint16_t *cold_k, *cold_v;
  const uint16_t *q, *k, *v;      // add_hidden_values only
  uint16_t* out;
  float* lse;
  float* part_o;                  // [rows of the partial states][D]
  float* part_l;                  // [rows], log2
  int64_t q_stride, k_stride, v_stride, out_stride;
  int64_t cold_slots;
  int64_t cold_blocks;
  int32_t page, max_blocks;
  int32_t Hq, Hkv, G, tpt, layer;
  int32_t* err;
  float scale_log2;               // log2(e) / sqrt(d)
};

template <int D>
struct Layout {
  static constexpr int NST = D == 128 ? 5 : 8;           // K/V tiles in the ring
  static constexpr uint32_t kTile = BN * D * 2;
  static constexpr uint32_t kQTile = BM * D * 2;
  static constexpr uint32_t kRing = 2 * kQTile;
  static constexpr uint32_t kData = kRing + NST * kTile;
};

enum : int {
  B_QFULL = 0,                    // one per Q tile, also the next four
  B_QEMPTY = 2,
  B_SFULL = 4,
  B_PFULL = 6,
  B_OFULL = 8,
  B_FINAL = 10,
  B_RFULL = 11,                   // 8 each
  B_REMPTY = 19,
  B_RSCAN = 27,
  B_ROUT = 35,
  B_COUNT = 43
};
constexpr uint32_t kCtlTmemSlot = B_COUNT * 8;
constexpr uint32_t kCtlAbort = kCtlTmemSlot + 4;
constexpr uint32_t kCtlHidden = kCtlAbort + 4;   // an infinity or NaN was hidden in this CTA's V tiles
constexpr uint32_t kCtlBytes = 512;
static_assert(kCtlHidden + 4 <= kCtlBytes, "prompt control block");
// dynamic shared memory starts 1024-byte aligned (checked by the kernel)
static_assert(Layout<128>::kData + kCtlBytes <= 232448 && Layout<64>::kData + kCtlBytes <= 232448, "shared memory");

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(tmap), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// a whole tile from shared memory to global memory, in the thread's current bulk group
__device__ __forceinline__ void tma_store_3d(const void* tmap, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(tmap), "r"(x),
               "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// the thread's bulk stores have read their sources; or are done
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// 16-byte copy, or 16 zero bytes when !valid (the source is then not read)
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, uint64_t src, bool valid) {
  const uint32_t n = valid ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// Bounded wait; the clock and the CTA's abort flag are looked at every 256 tries only,
// as reading the timer at each try delays what follows the barrier by 100 cycles and more.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, int32_t* err, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if (n & 255u) continue;
    if (*abort_flag) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitLimitNs) {
      report_error(err, kErrTimeout);
      *abort_flag = 1;
      return false;
    }
  }
}

// ring position: stage and phase parity of the current element
template <int NST>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == NST) {
      st = 0;
      ph ^= 1u;
    }
  }
  __device__ __forceinline__ void skip(int n) {
    const int at = st + n, laps = at / NST;
    st = at - laps * NST;
    ph ^= (uint32_t)laps & 1u;
  }
};

// key tiles of Q tile i of an item, counted from the item's first
__device__ __forceinline__ int tile_count(const PromptItemDev& it, const PromptReqDev& rq, int tpt, int i) {
  const int a = it.tok0 + i * tpt;
  if (a >= rq.n) return 0;
  const int last = min(rq.n, a + tpt) - 1;
  const int total = rq.nt_hot + rq.nt_cold + last / BN + 1;
  return max(0, min(it.tile0 + it.ntile, total) - it.tile0);
}

// the ring's elements that stage an item's output: one for each Q tile with key tiles
__device__ __forceinline__ int staging_count(const PromptItemDev& it, const PromptReqDev& rq, int tpt) {
  return (tile_count(it, rq, tpt, 0) > 0) + (tile_count(it, rq, tpt, 1) > 0);
}
// Partial rows staged kRowBytes at a time: the byte of 16-byte chunk c of row r.  Neither a
// thread's row nor the chunks that a quarter warp reads of one meet in a bank.
template <int kRowBytes>
__device__ __forceinline__ uint32_t staged(int r, int c) {
  return (uint32_t)(r * kRowBytes + ((c ^ (kRowBytes >= 128 ? r & 7 : (r >> 1) & 3)) << 4));
}
// Output rows staged as TMA's 128-byte swizzle has them, 64 columns a region
__device__ __forceinline__ uint32_t staged_out(int r, int c) {
  return (uint32_t)(c >> 3) * kRegionQ + (uint32_t)(r * 128 + (((c ^ r) & 7) << 4));
}

// does a V tile hold places that some row of the item must not see?
__device__ __forceinline__ bool scanned(const PromptItemDev& it, const PromptReqDev& rq, int t) {
  if (t < rq.nt_hot) return (t + 1) * BN > rq.lp;
  return (t - rq.nt_hot - rq.nt_cold + 1) * BN - 1 > it.tok0;
}

// The terms of new keys in (tok0, tk] whose V row holds an infinity or NaN: those
// rows were zeroed in shared memory because other rows of the item must not see
// them.  p_j v_j is added to O (tensor memory) for the rows that do.
template <int D>
__device__ __forceinline__ void add_hidden_values(const Params& p, int item, int token, int hr, bool valid, float m, uint32_t tO) {
  const PromptItemDev it = p.items[item];
  const PromptReqDev rq = p.reqs[it.req];
  const int tk = it.tok0 + token, qh = it.head * p.G + hr;
  const int hi = valid ? tk : -1;
  const int top = __reduce_max_sync(0xffffffffu, hi);
#pragma unroll 1
  for (int j = it.tok0 + 1; j <= top; ++j) {
    const int tile = j / BN + rq.nt_hot + rq.nt_cold;
    if (tile < it.tile0 || tile >= it.tile0 + it.ntile) continue;
    const uint16_t* vr = p.v + (int64_t)(rq.t0 + j) * p.v_stride + it.head * D;
    bool bad = false;
#pragma unroll 1
    for (int c = 0; c < D; ++c) bad |= (vr[c] & 0x7F80) == 0x7F80;
    if (!bad) continue;   // warp-uniform: every lane read the same row
    float w = 0.f;
    if (j <= hi) {
      const uint16_t* qr = p.q + (int64_t)(rq.t0 + tk) * p.q_stride + qh * D;
      const uint16_t* kr = p.k + (int64_t)(rq.t0 + j) * p.k_stride + it.head * D;
      float s = 0.f;
#pragma unroll 1
      for (int c = 0; c < D; ++c) s = fmaf(bf_lo(qr[c]), bf_lo(kr[c]), s);
      w = ex2(s * p.scale_log2 - m);
    }
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
      float o[32];
      tmem_ld32(tO + c0, o);
      tc_wait_ld();
      if (j <= hi)
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = fmaf(w, bf_lo(vr[c0 + e]), o[e]);
      __syncwarp();
      tmem_st32(tO + c0, o);
      tc_wait_st();
    }
  }
}

// a value every lane holds, in a form the compiler knows to be warp-uniform
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }
// true on one lane of the (converged) warp, always the same one
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

__device__ __forceinline__ void stg128_if(bool doit, uint64_t addr, uint4 v) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t@p st.global.v4.b32 [%1], {%2,%3,%4,%5};\n\t}" ::"r"(
                   (int)doit),
               "l"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// keeps uses of the registers of a tcgen05.ld behind its wait
__device__ __forceinline__ void tie32(float* v) {
#pragma unroll
  for (int e = 0; e < 32; e += 8)
    asm volatile("" : "+f"(v[e]), "+f"(v[e + 1]), "+f"(v[e + 2]), "+f"(v[e + 3]), "+f"(v[e + 4]), "+f"(v[e + 5]),
                 "+f"(v[e + 6]), "+f"(v[e + 7]));
}

__device__ __forceinline__ float max32(const float* s) {
  float a[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) a[k] = fmax3(s[k], s[k + 4], s[k + 8]);
#pragma unroll
  for (int c = 12; c < 28; c += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = fmax3(a[k], s[c + k], s[c + 4 + k]);
#pragma unroll
  for (int k = 0; k < 4; ++k) a[k] = fmaxf(a[k], s[28 + k]);
  return fmaxf(fmax3(a[0], a[1], a[2]), a[3]);
}

// 2^(s * scale - m) of 64 scores as 32 bf16 pairs, added to the running sums in fp32
__device__ __forceinline__ void exp64(const float* s, uint32_t* pk, uint64_t* sum4, uint64_t sc2, uint64_t nm2) {
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    float xa, xb;
    f2unpack(ffma2(f2pack(s[2 * c], s[2 * c + 1]), sc2, nm2), xa, xb);
    const float a = ex2(xa), b = ex2(xb);
    sum4[c & 3] = fadd2(sum4[c & 3], f2pack(a, b));
    pk[c] = pack_bf16x2(a, b);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ Params p) {
  using Lay = Layout<D>;
  constexpr int NST = Lay::NST;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  if (raw & 1023u) {              // the operand layouts need it
    if (threadIdx.x == 0) report_error(p.err, kErrTimeout);
    return;
  }
  const uint32_t base = raw;
  const uint32_t ctl = base + Lay::kData;
  uint8_t* ctl_ptr = smem_raw + Lay::kData;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl_ptr + kCtlAbort);
  volatile int* hidden_flag = reinterpret_cast<volatile int*>(ctl_ptr + kCtlHidden);
  auto bar = [&](int i) { return ctl + 8u * (uint32_t)i; };
  const uint32_t sQ = base, sR = base + Lay::kRing;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    *hidden_flag = 0;
    mbar_init(bar(B_FINAL), 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar(B_REMPTY + s), 8);  // one arrival of the MMAs' end and seven of the relay; for a staging element,
                                        // eight of the output warp or two of each softmax warp
      mbar_init(bar(B_RFULL + s), 128); // the TMA thread arrives 128 times, or each gather thread once
      mbar_init(bar(B_RSCAN + s), 1);
      mbar_init(bar(B_ROUT + s), 4);    // a Q tile's softmax warps: its output is staged
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_QFULL + i), 1);
      mbar_init(bar(B_QEMPTY + i), 1);    // a softmax warp has seen the Q tile's last S
      mbar_init(bar(B_SFULL + i), 1);
      mbar_init(bar(B_PFULL + i), 129);   // the softmax threads and the relay
      mbar_init(bar(B_OFULL + i), 1);
    }
    fence_mbar_init();
  }
  // rows of a Q tile that no token has (g = 5) stay zero
  for (int c = threadIdx.x; c < 2 * (D / 64) * (BM - p.tpt * p.G) * 8; c += kThreads) {
    const int per = (BM - p.tpt * p.G) * 8;
    sts128(sQ + (uint32_t)(c / per) * kRegionQ + (uint32_t)(p.tpt * p.G * 8 + c % per) * 16, make_uint4(0, 0, 0, 0));
  }
  fence_async_shared();
  if (warp == 1) {
    tmem_alloc(ctl + kCtlTmemSlot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(ctl_ptr + kCtlTmemSlot);
  // The plan's tables are written before the kernel ahead of this one starts and by no kernel,
  // so they are read while it still runs; what reads or writes a call's data waits for it
  // (griddep_wait in the roles below).
  const int i0 = p.cta_begin[blockIdx.x], i1 = p.cta_begin[blockIdx.x + 1];
  auto tS = [&](int i) { return tmem + (uint32_t)(i * 128); };
  auto tO = [&](int i) { return tmem + 256u + (uint32_t)(i * 128); };

  // a wait of a whole warp, with a warp-uniform answer
  auto wait = [&](int b, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_or_abort(bar(b), parity, p.err, abort_flag)) != 0;
  };

  if (warp < 4 || warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    if (lane == 0) {
      Ring<NST> ring;                              // over the elements K0 V0 K1 V1 ...
      uint32_t scan_ph = 0;                        // bit s: parity of RSCAN[s]'s current phase
      uint32_t in_ring = 0, in_scan = 0, full_ph = 0;  // the last load of each stage, for the drain below
      uint32_t staged = 0;                         // stages that an epilogue wrote to last
      uint32_t qn[2] = {0, 0};
      bool ok = true;
      PromptItemDev next_it = {};
      PromptReqDev next_rq = {};
      if (i0 < i1) {
        next_it = p.items[i0];
        next_rq = p.reqs[next_it.req];
      }
      for (const CUtensorMap* tm : {&p.tq, &p.tk, &p.tv, &p.tout})
        asm volatile("prefetch.tensormap [%0];" ::"l"(tm) : "memory");
      griddep_wait();
      for (int ii = i0; ok && ii < i1; ++ii) {
        const PromptItemDev it = next_it;
        const PromptReqDev rq = next_rq;
        if (ii + 1 < i1) {
          next_it = p.items[ii + 1];
          next_rq = p.reqs[next_it.req];
        }
        const int nctx = rq.nt_hot + rq.nt_cold;
        const int n_el = 2 * it.ntile + staging_count(it, rq, p.tpt);
        for (int j = 0; j < n_el; ++j) {
          if (j == 1) {
            // each Q tile, once the last product with the one before has read it
            for (int i = 0; i < 2; ++i) {
              if (tile_count(it, rq, p.tpt, i) == 0) continue;
              if (!wait_or_abort(bar(B_QEMPTY + i), (qn[i] & 1u) ^ 1u, p.err, abort_flag)) { ok = false; break; }
              ++qn[i];
              mbar_arrive_expect_tx(bar(B_QFULL + i), (uint32_t)(p.tpt * p.G) * 128u * (D / 64));
              for (int h = 0; h < D / 64; ++h)
                tma_load_3d(sQ + i * Lay::kQTile + h * kRegionQ, &p.tq, h * 64, it.head * p.G,
                            rq.t0 + it.tok0 + i * p.tpt, bar(B_QFULL + i));
            }
            if (!ok) break;
          }
          const int t = it.tile0 + (j >> 1);
          const bool is_v = j & 1;
          const int st = ring.st;
          const uint32_t ph = ring.ph;
          ring.next();
          // waited for whoever fills the stage: a parity wait may be neither a phase ahead nor one
          // behind.  The gather warps, which would fall behind over tiles that are none of theirs,
          // learn through B_RSCAN which stage is theirs.
          if (!wait_or_abort(bar(B_REMPTY + st), ph ^ 1u, p.err, abort_flag)) { ok = false; break; }
          if (j >= 2 * it.ntile) {                 // a staging element
            in_ring &= ~(1u << st);
            in_scan &= ~(1u << st);
            if (it.entry >= 0) staged |= 1u << st;   // written and read by the softmax warps only
            mbar_arrive_n(bar(B_RFULL + st), 128);
          } else if (t >= rq.nt_hot && t < nctx) { // COLD: to the gather warps
            in_ring &= ~(1u << st);
            in_scan &= ~(1u << st);
            scan_ph ^= 1u << st;
            mbar_arrive(bar(B_RSCAN + st));
          } else {
            const bool scan = is_v && scanned(it, rq, t);
            const uint32_t b = bar((scan ? B_RSCAN : B_RFULL) + st);
            const uint32_t tile = sR + (uint32_t)st * Lay::kTile;
            if (staged >> st & 1u) {
              // the epilogue's ordinary writes before TMA's (a fence by the warps that wrote, behind
              // their stores to global memory, took them 1500 cycles)
              fence_async_shared();
              staged &= ~(1u << st);
            }
            if (!scan) mbar_arrive_n(b, 127);
            mbar_arrive_expect_tx(b, Lay::kTile);
            if (t < rq.nt_hot) {
              const int row = (int)(rq.hot_row + ((int64_t)p.layer * p.Hkv + it.head) * rq.lp + t * BN);
              for (int h = 0; h < D / 64; ++h) tma_load_2d(tile + h * kRegionKV, is_v ? &p.thv : &p.thk, h * 64, row, b);
            } else {
              const int row = rq.t0 + (t - nctx) * BN;
              for (int h = 0; h < D / 64; ++h)
                tma_load_3d(tile + h * kRegionKV, is_v ? &p.tv : &p.tk, h * 64, it.head, row, b);
            }
            const uint32_t bit = 1u << st;
            in_ring = scan ? in_ring & ~bit : in_ring | bit;
            in_scan = scan ? in_scan | bit : in_scan & ~bit;
            full_ph = (full_ph & ~bit) | (ph << st);
            if (scan) scan_ph ^= bit;
          }
        }
      }
      if (!ok) {
        // let the loads already issued land before shared memory goes away
        for (int s = 0; s < NST; ++s) {
          if (in_ring >> s & 1u) mbar_wait(bar(B_RFULL + s), full_ph >> s & 1u, nullptr);
          if (in_scan >> s & 1u) mbar_wait(bar(B_RSCAN + s), (scan_ph >> s & 1u) ^ 1u, nullptr);
        }
        for (int i = 0; i < 2; ++i)
          if (qn[i]) mbar_wait(bar(B_QFULL + i), (qn[i] - 1) & 1u, nullptr);
      }
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer --------------------------------
    // The whole warp walks the loop with warp-uniform values and one elected lane
    // issues: the descriptors then stay in uniform registers, where a loop of one
    // lane moves each of them there for every MMA (84 cycles per MMA measured, 64
    // being the tensor cores' own).
    constexpr uint32_t kIdQK = idesc(BN, false);
    constexpr uint32_t kIdPV = idesc(D, true);
    const uint64_t dQ = sdesc(sQ, 16, 1024), dK = sdesc(sR, 16, 1024), dV = sdesc(sR, kRegionKV, 1024);
    auto issue_s = [&](int i, int st) {
      const uint64_t a0 = dQ + ((uint32_t)i * Lay::kQTile >> 4);
      const uint64_t b0 = dK + ((uint32_t)st * Lay::kTile >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        tc_mma_ss(tS(i), a0 + (((kk / 4) * kRegionQ + (kk % 4) * 32) >> 4),
                  b0 + (((kk / 4) * kRegionKV + (kk % 4) * 32) >> 4), kIdQK, kk > 0 ? 1u : 0u);
      tc_commit(bar(B_SFULL + i));
    };
    auto issue_pv = [&](int i, int st, bool first) {
      const uint64_t b0 = dV + ((uint32_t)st * Lay::kTile >> 4);
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk)
        tc_mma_ts(tO(i), tS(i) + kk * 8, b0 + ((kk * 2048) >> 4), kIdPV, (!first || kk > 0) ? 1u : 0u);
    };
    Ring<NST> k;                   // the next element: K0 V0 K1 V1 ...
    uint32_t qn[2] = {0, 0}, pn[2] = {0, 0};
    bool ok = true;
    const int u0 = uniform(i0), u1 = uniform(i1);
    for (int ii = u0; ok && ii < u1; ++ii) {
      const PromptItemDev it = p.items[ii];
      const PromptReqDev rq = p.reqs[it.req];
      const int ntile = uniform(it.ntile);
      const int cnt[2] = {uniform(tile_count(it, rq, p.tpt, 0)), uniform(tile_count(it, rq, p.tpt, 1))};
      if (!wait(B_RFULL + k.st, k.ph)) { ok = false; break; }
      fence_async_shared();        // K_0 may have been gathered
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (cnt[i] == 0) continue;
        if (!wait(B_QFULL + i, qn[i] & 1u)) { ok = false; break; }
        ++qn[i];
        tc_fence_after();
        if (elect_one()) issue_s(i, k.st);
        __syncwarp();
      }
      if (!ok) break;
      if (elect_one()) tc_commit(bar(B_REMPTY + k.st));
      __syncwarp();
      for (int j = 0; ok && j < ntile; ++j) {
        Ring<NST> v = k;
        v.next();
        k = v;
        k.next();
        const bool last = j + 1 == ntile;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (j >= cnt[i]) continue;
          // P, and through the relay V_j and K_(j+1)
          if (!wait(B_PFULL + i, pn[i] & 1u)) { ok = false; break; }
          ++pn[i];
          tc_fence_after();
          if (elect_one()) {
            issue_pv(i, v.st, j == 0);
            // S(j+1) over P(j), once the product has read it (one thread's MMAs run in order)
            if (j + 1 < cnt[i]) issue_s(i, k.st);
            else tc_commit(bar(B_OFULL + i));
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) {
          tc_commit(bar(B_REMPTY + v.st));
          if (!last) tc_commit(bar(B_REMPTY + k.st));
        }
        __syncwarp();
      }
      k.skip((cnt[0] > 0) + (cnt[1] > 0));
    }
    // arrives once every MMA issued above has finished, aborted or not
    if (elect_one()) tc_commit(bar(B_FINAL));
    __syncwarp();
  } else if (warp == 2 || warp == 3 || warp == 13 || warp == 14) {
    // ----------------------- COLD gather and V tile scan -----------------------
    constexpr int kChunks = D / 8;               // 16-byte chunks per row
    constexpr int kRowsPerCopy = 32 / kChunks;   // rows per warp instruction
    const int row0 = (warp < 4 ? warp - 2 : warp - 11) * 32;   // this warp's rows of a tile
    const int ch = lane % kChunks, sub = lane / kChunks;
    const uint32_t slot_bytes = (uint32_t)(p.Hkv * D) * 2u;
    griddep_wait();
    Ring<NST> ring;
    uint32_t scan_ph = 0;
    bool ok = true;
    for (int ii = i0; ok && ii < i1; ++ii) {
      const PromptItemDev it = p.items[ii];
      const PromptReqDev rq = p.reqs[it.req];
      const int nctx = rq.nt_hot + rq.nt_cold;
      // block id of row row0 + lane of COLD tile t, fetched one tile ahead
      int id = -1, slot = -1;
      auto fetch_ids = [&](int t) {
        const int pos = (t - rq.nt_hot) * BN + row0 + lane;
        id = t >= rq.nt_hot && t < nctx && t < it.tile0 + it.ntile && pos < rq.ctx
                 ? p.block_table[(int64_t)rq.row * p.max_blocks + pos / p.page]
                 : -1;
      };
      fetch_ids(max(it.tile0, rq.nt_hot));
      for (int j = 0; j < 2 * it.ntile; ++j) {
        const int t = it.tile0 + (j >> 1);
        const bool is_v = j & 1;
        const int st = ring.st;
        ring.next();
        const bool cold = t >= rq.nt_hot && t < nctx;
        if (!cold && !(is_v && scanned(it, rq, t))) continue;
        // the stage is free (COLD), or TMA has filled it
        if (!wait(B_RSCAN + st, scan_ph >> st & 1u)) { ok = false; break; }
        scan_ph ^= 1u << st;
        const uint32_t tile = sR + (uint32_t)st * Lay::kTile;
        if (cold) {
          if (!is_v) {
            const int pos = (t - rq.nt_hot) * BN + row0 + lane;
            const bool in = pos < rq.ctx;
            slot = in && id >= 0 && id < p.cold_blocks ? id * p.page + pos % p.page : -1;
            if (in && slot < 0) report_error(p.err, kErrBounds);
            fetch_ids(t + 1);
          }
          // four instructions a copy where every row exists: the gather warps share their schedulers
          // with the softmax warps (a tile of COLD keys took 1837 ns with a dozen, 1603 so)
          const uint64_t src0 = (uint64_t)((is_v ? p.cold_v : p.cold_k) +
                                           ((int64_t)p.layer * p.cold_slots * p.Hkv + it.head) * D + ch * 8);
          const uint32_t dst0 = tile + (uint32_t)(ch >> 3) * kRegionKV + (uint32_t)(row0 + sub) * 128;
          const bool all = __all_sync(0xffffffffu, slot >= 0);
          if (all) {
#pragma unroll
            for (int r = 0; r < 32; r += kRowsPerCopy)     // row0 is a multiple of 8
              cp_async16(dst0 + r * 128 + (((ch ^ (r + sub)) & 7) << 4),
                         (const void*)(src0 + (uint64_t)(uint32_t)__shfl_sync(0xffffffffu, slot, r + sub) * slot_bytes));
          } else {
#pragma unroll 1
            for (int r = 0; r < 32; r += kRowsPerCopy) {
              const int s = __shfl_sync(0xffffffffu, slot, r + sub);
              cp_async16_or_zero(dst0 + r * 128 + (((ch ^ (r + sub)) & 7) << 4),
                                 src0 + (uint64_t)(uint32_t)max(s, 0) * slot_bytes, s >= 0);
            }
          }
          cp_async_mbar_arrive(bar(B_RFULL + st));
        } else {
          const bool hot = t < rq.nt_hot;
          const int key0 = (hot ? t : t - nctx) * BN;
          const int end = hot ? rq.lp : rq.n;
          const int row = row0 + lane, key = key0 + row;
          const uint32_t src = tile + row * 128;
          bool zero = key >= end;
          if (!zero && !hot && key > it.tok0) {
            uint32_t top = 0;
#pragma unroll 4
            for (int c = 0; c < kChunks; ++c) {
              const uint4 w = lds128(src + (c >> 3) * kRegionKV + (((c & 7) ^ (row & 7)) << 4));
              // exponent bits all ones carry into the sign bit of their half
              top |= ((w.x & 0x7F807F80u) + 0x00800080u) | ((w.y & 0x7F807F80u) + 0x00800080u) |
                     ((w.z & 0x7F807F80u) + 0x00800080u) | ((w.w & 0x7F807F80u) + 0x00800080u);
            }
            if (top & 0x80008000u) {
              zero = true;
              *hidden_flag = 1;
            }
          }
          if (zero) {
#pragma unroll 4
            for (int c = 0; c < kChunks; ++c)
              sts128(src + (c >> 3) * kRegionKV + (((c & 7) ^ (row & 7)) << 4), make_uint4(0, 0, 0, 0));
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive_n(bar(B_RFULL + st), 32);
        }
      }
      if (!ok) break;
      ring.skip(staging_count(it, rq, p.tpt));
    }
    cp_async_wait_all();
  } else if (warp == 12) {
    // ------------------------------ operand relay -------------------------------
    // Waits for V_j and K_(j+1) and arrives for them on the barriers of P(j): the MMA
    // warp then waits once per Q tile and key tile.  (Its own waits queue behind the
    // MMAs that it has issued: two more cost it 500 cycles a key tile, with P ready.)
    if (lane == 0) {
      Ring<NST> ring;
      uint32_t pn[2] = {0, 0};
      bool ok = true;
      auto full = [&](bool cold) {
        if (!wait_or_abort(bar(B_RFULL + ring.st), ring.ph, p.err, abort_flag)) return false;
        if (cold) fence_async_shared();            // the gathered rows before the products' reads
        mbar_arrive_n(bar(B_REMPTY + ring.st), 7);
        ring.next();
        return true;
      };
      for (int ii = i0; ok && ii < i1; ++ii) {
        const PromptItemDev it = p.items[ii];
        const PromptReqDev rq = p.reqs[it.req];
        const int cnt[2] = {tile_count(it, rq, p.tpt, 0), tile_count(it, rq, p.tpt, 1)};
        auto cold = [&](int j) { return it.tile0 + j >= rq.nt_hot && it.tile0 + j < rq.nt_hot + rq.nt_cold; };
        ok = full(cold(0));            // K_0: the MMA warp waits for it too
        for (int j = 0; ok && j < it.ntile; ++j) {
          ok = full(cold(j)) && (j + 1 == it.ntile || full(cold(j + 1)));
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (ok && j < cnt[i]) {
              // one arrival a phase: not before the last P's phase is over
              if (pn[i] > 0) ok = wait_or_abort(bar(B_PFULL + i), (pn[i] - 1) & 1u, p.err, abort_flag);
              ++pn[i];
              if (ok) mbar_arrive(bar(B_PFULL + i));
            }
        }
        ring.skip((cnt[0] > 0) + (cnt[1] > 0));
      }
    }
  } else {
    // ------------------------------- output rows --------------------------------
    // Staged bf16 rows to global memory while the softmax warps are at the next item (they
    // took 2300 cycles an item to write them themselves): whole Q tiles by TMA (1400 cycles a
    // tile, 3000 by this warp's own stores), the last rows of a request, whose tile holds
    // another's behind them, 512 bytes an instruction.
    constexpr int kChunks = D / 8, kRows = 32 / kChunks;
    const int ch = lane % kChunks, sub = lane / kChunks;
    const uint32_t inv_g = 65536u / (uint32_t)p.G + 1u;   // r * inv_g >> 16 = r / G for r < 128
    griddep_wait();
    Ring<NST> ring;
    uint32_t out_ph = 0;
    bool ok = true;
    for (int ii = i0; ok && ii < i1; ++ii) {
      const PromptItemDev it = p.items[ii];
      const PromptReqDev rq = p.reqs[it.req];
      ring.skip(2 * it.ntile);
      for (int i = 0; i < 2; ++i) {
        if (tile_count(it, rq, p.tpt, i) == 0) continue;
        const int st = ring.st;
        ring.next();
        if (it.entry >= 0) continue;               // a partial state: the softmax warps write it
        if (!wait(B_ROUT + st, out_ph >> st & 1u)) { ok = false; break; }
        out_ph ^= 1u << st;
        const uint32_t tile = sR + (uint32_t)st * Lay::kTile;
        const int tok0 = it.tok0 + i * p.tpt;
        if (lane == 0) fence_async_shared();       // the softmax warps' writes before TMA's reads, now or later
        if (tok0 + p.tpt <= rq.n) {
          if (lane == 0) {
            for (int h = 0; h < D / 64; ++h)
              tma_store_3d(&p.tout, h * 64, it.head * p.G, rq.t0 + tok0, tile + h * kRegionQ);
            bulk_commit();
            bulk_wait_read();
          }
        } else {
          const int n = (rq.n - tok0) * p.G;
          uint16_t* const out0 = p.out + (int64_t)(rq.t0 + tok0) * p.out_stride + it.head * p.G * D + ch * 8;
#pragma unroll 1
          for (int r0 = sub; r0 - sub < n; r0 += 8 * kRows) {
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = lds128(tile + staged_out(r0 + k * kRows, ch));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int r = r0 + k * kRows, tok = (int)((uint32_t)r * inv_g >> 16);
              stg128_if(r < n, (uint64_t)(out0 + (int64_t)tok * p.out_stride + (r - tok * p.G) * D), v[k]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_n(bar(B_REMPTY + st), 8);
      }
    }
    if (lane == 0) bulk_wait();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---------------------- softmax / correction / epilogue ---------------------
    const int qi = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const int tr = row / p.G, hr = row % p.G;     // token within the Q tile, query head within the group
    const uint32_t tSr = tS(qi) + lane_off, tOr = tO(qi) + lane_off;
    griddep_wait();
    uint32_t sn = 0, on = 0;
    Ring<NST> ring;                               // moved to the Q tile's staging element of each item
    bool ok = true;
    // what the warp keeps of an item: the Q tile's key tiles, its staging element's place behind
    // the item before and the elements after it, where the row's output goes (0: nowhere; the
    // output warp has the address of an output row itself), the tiles with masked places counted
    // from the item's first (the last HOT and COLD ones, and those on the diagonal), and how many
    // keys the row sees there (rows of no token: as the last one)
    int cnt = 0, skip = 0, rest = 0, j_hot = -1, j_cold = -1, j_new = 0, lim_hot = 0, lim_cold = 0, lim_new = 0;
    bool part_row = false;
    uint64_t dst = 0, lse_dst = 0;
    auto open_item = [&](int ii) {
      const PromptItemDev it = p.items[ii];
      const PromptReqDev rq = p.reqs[it.req];
      const int nctx = rq.nt_hot + rq.nt_cold;
      cnt = tile_count(it, rq, p.tpt, qi);
      const bool other = tile_count(it, rq, p.tpt, qi ^ 1) > 0;
      skip = 2 * it.ntile + (qi && other);
      rest = (cnt > 0) + (!qi && other);
      const int tk = it.tok0 + qi * p.tpt + tr;
      part_row = it.entry >= 0;
      dst = lse_dst = 0;
      if (tr < p.tpt && tk < rq.n) {
        const int qh = it.head * p.G + hr;
        const int64_t prow = it.part_row + qi * p.tpt * p.G + row, orow = rq.t0 + tk;
        dst = part_row ? (uint64_t)(p.part_o + prow * D) : 1;
        lse_dst = part_row ? (uint64_t)(p.part_l + prow) : p.lse ? (uint64_t)(p.lse + orow * p.Hq + qh) : 0;
      }
      j_hot = rq.lp % BN ? rq.nt_hot - 1 - it.tile0 : -1;
      j_cold = rq.ctx % BN ? nctx - 1 - it.tile0 : -1;
      j_new = nctx - it.tile0 + (it.tok0 + qi * p.tpt + 1) / BN;
      lim_hot = rq.lp % BN;
      lim_cold = rq.ctx % BN;
      lim_new = min(tk, rq.n - 1) + 1 + (nctx - it.tile0) * BN;
    };
    if (i0 < i1) open_item(i0);
    for (int ii = i0; ok && ii < i1; ++ii) {
      ring.skip(skip);
      // m: the reference of every exponent so far (-inf: no key seen), part: the last tile's sum, l: the row's
      float m = -INFINITY, part = 0.f, l = 0.f;
      bool adjust = true;                         // some row of the warp needs another reference
      // raise the reference to m_new: O and l hold the keys so far scaled by 2^-m
      auto raise = [&](float m_new, bool have_o) {
        const float f = m == -INFINITY ? 1.f : ex2(m - m_new);
        if (have_o) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(tOr + c, o);
            tc_wait_ld();
            tie32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f;
            tmem_st32(tOr + c, o);
          }
          tc_wait_st();
        }
        l *= f;
        m = m_new;
      };
      for (int j = 0; j < cnt; ++j) {
        // warp-uniform: a lane that gave up takes its whole warp out of the loop
        if (!wait(B_SFULL + qi, sn & 1u)) { ok = false; break; }
        ++sn;
        tc_fence_after();
        if (j + 1 == cnt && (warp & 3) == 0 && lane == 0) mbar_arrive(bar(B_QEMPTY + qi));   // Q was read for the last time
        if (j == j_hot || j == j_cold || j >= j_new) {
          // minus infinity over the hidden scores, in tensor memory: one copy of the code below then
          // serves every tile (with two, the second one's instructions were fetched anew each item)
          const int lim = j == j_hot ? lim_hot : j == j_cold ? lim_cold : lim_new - j * BN;
#pragma unroll 1
          for (int c = 0; c < BN; c += 32) {
            if (__all_sync(0xffffffffu, lim >= c + 32)) continue;
            float s[32];
            tmem_ld32(tSr + c, s);
            tc_wait_ld();
            tie32(s);
#pragma unroll
            for (int e = 0; e < 32; ++e) s[e] = e < lim - c ? s[e] : -INFINITY;
            tmem_st32(tSr + c, s);
          }
          tc_wait_st();
        }
        // the row's maximum over the tile's first keys, in log2 units, rounded up: no exponent against it is above 0
        auto maximum = [&](int keys) {
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < keys; c += 32) {
            float s[32];
            tmem_ld32(tSr + c, s);
            tc_wait_ld();
            tie32(s);
            mx = fmaxf(mx, max32(s));
          }
          return __fmul_ru(mx, p.scale_log2);
        };
        // S(j) completed after PV(j-1), so O may be rescaled here
        if (adjust) {
          float m_new = part > 256.f ? m + __log2f(part) : m;
          if (__any_sync(0xffffffffu, m == -INFINITY)) {
            // rows without one start from 32 keys' maximum, or the tile's where they see none of those
            float mx = maximum(32);
            if (__any_sync(0xffffffffu, mx == -INFINITY)) mx = maximum(BN);
            if (m == -INFINITY) m_new = mx;
          }
          raise(m_new, j > 0);
        }
        uint32_t pk[BN / 2];
        // P and the row's sum in the tile
        auto exponentials = [&]() {
          const float m_sub = m == -INFINITY ? 0.f : m;     // a row that sees no key yet: -inf - 0
          const uint64_t sc2 = f2pack(p.scale_log2, p.scale_log2), nm2 = f2pack(-m_sub, -m_sub);
          uint64_t sum4[4] = {0, 0, 0, 0};
          float sa[64], sb[64];
          tmem_ld32(tSr, sa);
          tmem_ld32(tSr + 32, sa + 32);
          tc_wait_ld();
          tie32(sa);
          tie32(sa + 32);
          tmem_ld32(tSr + 64, sb);
          tmem_ld32(tSr + 96, sb + 32);
          exp64(sa, pk, sum4, sc2, nm2);
          tc_wait_ld();
          tie32(sb);
          tie32(sb + 32);
          exp64(sb, pk + 32, sum4, sc2, nm2);
          float s0, s1, s2, s3;
          f2unpack(fadd2(sum4[0], sum4[1]), s0, s1);
          f2unpack(fadd2(sum4[2], sum4[3]), s2, s3);
          part = (s0 + s1) + (s2 + s3);
        };
        for (bool again = false;; again = true) {
          exponentials();
          if (again || !__any_sync(0xffffffffu, part > 0x1p64f)) break;
          // far above the reference: raise it and take the tile again (its S is still there)
          raise(fmaxf(m, maximum(BN)), j > 0);
        }
        l += part;
#pragma unroll
        for (int c = 0; c < BN / 2; c += 32) tmem_st32(tSr + c, reinterpret_cast<const float*>(pk + c));
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(bar(B_PFULL + qi));
        adjust = __any_sync(0xffffffffu, m == -INFINITY || part > 256.f);
      }
      if (!ok) break;
      // the next item's records while the last product runs
      const int cnt_now = cnt, rest_now = rest;
      const bool part_now = part_row;
      const uint64_t dst_now = dst, lse_now = lse_dst;
      if (ii + 1 < i1) open_item(ii + 1);
      if (cnt_now > 0) {
        if (!wait(B_OFULL + qi, on & 1u)) { ok = false; break; }
        ++on;
        tc_fence_after();
        if (__any_sync(0xffffffffu, *hidden_flag))
          add_hidden_values<D>(p, ii, qi * p.tpt + tr, hr, dst_now != 0, m, tOr);
      }
      const float inv = l > 0.f || l != l ? __fdividef(1.f, l) : 0.f;   // no key in this range: O = 0, LSE = -inf
      const float lse2 = m + __log2f(l);
      if (lse_now) *reinterpret_cast<float*>(lse_now) = part_now ? lse2 : lse2 * kLn2;
      if (cnt_now > 0) {
        // the staging element (its stage's earlier tiles were used by this Q tile, or by an earlier
        // item: the wait cannot be a phase behind)
        if (!wait(B_RFULL + ring.st, ring.ph)) { ok = false; break; }
        const uint32_t stage = sR + (uint32_t)ring.st * Lay::kTile;
        if (part_now) {
          // fp32 rows, kRow bytes of each of the warp's 32 at a time
          constexpr int kRow = D, kChunks = kRow / 16;
          const uint32_t mine = stage + (uint32_t)(warp & 3) * (32 * kRow);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32(tOr + c, o);
            tc_wait_ld();
            tie32(o);
#pragma unroll
            for (int h = 0; h < 32; h += kRow / 4) {
#pragma unroll
              for (int e = 0; e < kRow / 4; e += 4)
                sts128(mine + staged<kRow>(lane, e / 4),
                       make_uint4(__float_as_uint(o[h + e] * inv), __float_as_uint(o[h + e + 1] * inv),
                                  __float_as_uint(o[h + e + 2] * inv), __float_as_uint(o[h + e + 3] * inv)));
              __syncwarp();
              uint4 v[kChunks];
              uint64_t to[kChunks];
#pragma unroll
              for (int k = 0; k < kChunks; ++k) {      // all on their way before the first is used
                const int r = (k * 32 + lane) / kChunks;
                v[k] = lds128(mine + staged<kRow>(r, lane % kChunks));
                to[k] = __shfl_sync(0xffffffffu, dst_now, r);
              }
#pragma unroll
              for (int k = 0; k < kChunks; ++k) stg128_if(to[k] != 0, to[k] + (c + h) * 4 + (lane % kChunks) * 16, v[k]);
              __syncwarp();
            }
          }
          if (lane == 0) mbar_arrive_n(bar(B_REMPTY + ring.st), 2);
        } else {
#pragma unroll 1
          for (int c = 0; c < D; c += 64) {
            float o[64];
            tmem_ld32(tOr + c, o);
            tmem_ld32(tOr + c + 32, o + 32);
            tc_wait_ld();
            tie32(o);
            tie32(o + 32);
#pragma unroll
            for (int e = 0; e < 64; e += 8)
              sts128(stage + staged_out(row, (c + e) / 8),
                     make_uint4(pack_bf16x2(o[e] * inv, o[e + 1] * inv), pack_bf16x2(o[e + 2] * inv, o[e + 3] * inv),
                                pack_bf16x2(o[e + 4] * inv, o[e + 5] * inv),
                                pack_bf16x2(o[e + 6] * inv, o[e + 7] * inv)));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_ROUT + ring.st));   // to the output warp
        }
      }
      ring.skip(rest_now);
    }
    tc_fence_before();
  }
  // every MMA has finished (the MMA thread commits B_FINAL on every path, and its
  // waits are bounded) and the loads have landed before memory is released
  if (threadIdx.x == 0) mbar_wait(bar(B_FINAL), 0, nullptr);
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the partial states of rows whose keys several items covered: with l_e the
// states' LSE (log2), m = max l_e, w_e = 2^(l_e - m): O = sum w_e O_e / sum w_e,
// LSE = (m + log2 sum w_e) ln 2.  A state whose LSE is NaN makes its row NaN, as
// it is where one item covers the keys.  One warp per row, 32 rows per CTA, at most 32
// states per row (lane e holds state e's weight); bound by the read of the states
// (4 d bytes each), four in flight per warp.
template <int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptJoinDev* __restrict__ joins,
                                                          const PromptReqDev* __restrict__ reqs,
                                                          const float* __restrict__ part_o,
                                                          const float* __restrict__ part_l, uint16_t* __restrict__ out,
                                                          float* __restrict__ lse, int64_t out_stride, int32_t Hq,
                                                          int32_t G, int32_t tpt) {
  griddep_launch_dependents();
  griddep_wait();
  const PromptJoinDev jn = joins[blockIdx.x];
  const PromptReqDev rq = reqs[jn.req];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = jn.own_n + jn.hot_n;
  const int own_rows = min(2 * tpt, rq.n - jn.tok0) * G;   // of each of the block's own states
#pragma unroll 1
  for (int u = 0; u < 4; ++u) {
    const int r = jn.row0 + u * 8 + warp;          // row of the block, counted token by token
    const int local = r / G, h = r % G;            // token of the block, head of the group
    const int tk = jn.tok0 + local;
    if (local >= 2 * tpt || tk >= rq.n) break;     // warp-uniform
    // the stacked prefix: whole blocks before the token's, hot_n states each, then its own block's states
    const int ht = jn.hot_tok + local, hb = ht / (2 * tpt), hl = ht % (2 * tpt);
    const int hot_rows = min(2 * tpt, jn.hot_len - hb * 2 * tpt) * G;
    const int64_t hot_row = jn.hot0 + (int64_t)hb * 2 * tpt * G * jn.hot_n + hl * G + h;
    auto entry_row = [&](int e) {
      return e < jn.own_n ? jn.own0 + (int64_t)e * own_rows + r : hot_row + (int64_t)(e - jn.own_n) * hot_rows;
    };
    const float le = lane < n ? __ldcg(part_l + entry_row(lane)) : -INFINITY;
    float mx = le;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    float w = mx == -INFINITY ? 0.f : ex2(le - mx);
    if (lane >= n) w = 0.f;
    float z = w;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool has = lane < D / 4;
    for (int e0 = 0; e0 < n; e0 += 4) {
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = has && e0 + k < n ? __ldcg(reinterpret_cast<const float4*>(part_o + entry_row(e0 + k) * D) + lane)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, (e0 + k) & 31);
        if (wk != 0.f) {                           // an empty state's row may never have been written
          o.x = fmaf(wk, v[k].x, o.x);
          o.y = fmaf(wk, v[k].y, o.y);
          o.z = fmaf(wk, v[k].z, o.z);
          o.w = fmaf(wk, v[k].w, o.w);
        }
      }
    }
    const float inv = z > 0.f || z != z ? 1.f / z : 0.f;
    const int64_t orow = rq.t0 + tk;
    const int qh = jn.head * G + h;
    if (has)
      reinterpret_cast<uint2*>(out + orow * out_stride + qh * D)[lane] =
          make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (lane == 0 && lse) lse[orow * Hq + qh] = (mx + __log2f(z)) * kLn2;
  }
}

namespace {

template <int D>
int launch_t(const Params& pp, const PromptPlan* pl, const uint8_t* base, cudaStream_t st) {
  auto kern = prompt_kernel<D>;
  constexpr size_t smem = Layout<D>::kData + kCtlBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return (int)e;
  const int ctas = (int)pl->cta_begin.size() - 1;
  if (ctas > 0) {
    e = launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, st, pp);
    if (e != cudaSuccess) return (int)e;
  }
  if (!pl->joins.empty())
    e = launch_pdl(prompt_join_kernel<D>, dim3((unsigned)pl->joins.size()), dim3(256), 0, st,
                   (const PromptJoinDev*)(base + pl->off_joins), pp.reqs, (const float*)pp.part_o,
                   (const float*)pp.part_l, pp.out, pp.lse, pp.out_stride, pp.Hq, pp.G, pp.tpt);
  return (int)e;
}

}  // namespace
}  // namespace prompt

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// the driver's tensor-map encoder; null when the driver has none
EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? (EncodeTiledFn)p
               : nullptr;
  }();
  return fn;
}

// 3D map over a packed tensor [tokens][heads][d] with a token stride, 128-byte
// swizzle; tokens past the end read as zeros
int encode_packed(CUtensorMap* tm, const void* ptr, int d, int heads, int64_t tokens, int64_t stride,
                         int box_heads, int box_tokens) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return 1;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? 0
             : 2;
}

// 2D map over a whole HOT pool as rows of d elements
int encode_hot(CUtensorMap* tm, const void* ptr, int d, int64_t rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return 1;
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)d * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)kPrefixTileN};
  cuuint32_t estr[2] = {1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? 0
             : 2;
}

}  // namespace

int encode_hot_maps(const gk_pool_config* cfg, uint8_t* out) {
  const int64_t rows = cfg->hot_tokens * cfg->num_layers * cfg->num_kv_heads;
  const void* pools[2] = {cfg->hot_k, cfg->hot_v};
  for (int i = 0; i < 2; ++i) {
    CUtensorMap tm;
    if (encode_hot(&tm, pools[i], cfg->head_dim, rows)) return 1;
    std::memcpy(out + i * sizeof(CUtensorMap), &tm, sizeof(CUtensorMap));
  }
  return 0;
}

int launch_prompt(const LaunchCommon& lc, void* stream, int32_t layer, const gk_prompt_batch* b, const PromptPlan* pl) {
  const gk_pool_config& c = *lc.cfg;
  const uint8_t* base = (const uint8_t*)pl->d_buf;
  const int D = c.head_dim, G = c.num_q_heads / c.num_kv_heads;
  prompt::Params pp = {};
  pp.Hq = c.num_q_heads;
  pp.Hkv = c.num_kv_heads;
  pp.G = G;
  pp.tpt = kPrefixTileM / G;
  pp.layer = layer;
  pp.q_stride = b->q_stride ? b->q_stride : (int64_t)pp.Hq * D;
  pp.k_stride = b->k_stride ? b->k_stride : (int64_t)pp.Hkv * D;
  pp.v_stride = b->v_stride ? b->v_stride : (int64_t)pp.Hkv * D;
  pp.out_stride = b->out_stride ? b->out_stride : (int64_t)pp.Hq * D;
  int e = encode_packed(&pp.tq, b->d_q, D, pp.Hq, pl->tokens, pp.q_stride, G, pp.tpt);
  if (!e) e = encode_packed(&pp.tk, b->d_k, D, pp.Hkv, pl->tokens, pp.k_stride, 1, kPrefixTileN);
  if (!e) e = encode_packed(&pp.tv, b->d_v, D, pp.Hkv, pl->tokens, pp.v_stride, 1, kPrefixTileN);
  if (!e) e = encode_packed(&pp.tout, b->d_out, D, pp.Hq, pl->tokens, pp.out_stride, G, pp.tpt);
  if (e) return (int)cudaErrorInvalidValue;
  std::memcpy(&pp.thk, pl->hot_maps, sizeof(CUtensorMap));
  std::memcpy(&pp.thv, pl->hot_maps + sizeof(CUtensorMap), sizeof(CUtensorMap));
  pp.reqs = (const PromptReqDev*)(base + pl->off_reqs);
  pp.items = (const PromptItemDev*)(base + pl->off_items);
  pp.cta_begin = (const int32_t*)(base + pl->off_begin);
  pp.block_table = b->d_block_table;
  pp.cold_k = (const uint16_t*)c.cold_k;
  pp.cold_v = (const uint16_t*)c.cold_v;
  pp.q = (const uint16_t*)b->d_q;
  pp.k = (const uint16_t*)b->d_k;
  pp.v = (const uint16_t*)b->d_v;
  pp.out = (uint16_t*)b->d_out;
  pp.lse = b->d_lse;
  pp.part_o = pl->d_part_o;
  pp.part_l = pl->d_part_l;
  pp.cold_slots = c.cold_slots;
  pp.cold_blocks = c.cold_slots / c.cold_page_size;
  pp.page = c.cold_page_size;
  pp.max_blocks = b->max_blocks;
  pp.err = lc.d_error;
  pp.scale_log2 = kLog2e / sqrtf((float)D);
  if (D == 128) return prompt::launch_t<128>(pp, pl, base, (cudaStream_t)stream);
  if (D == 64) return prompt::launch_t<64>(pp, pl, base, (cudaStream_t)stream);
  return (int)cudaErrorInvalidValue;
}

}  // namespace gk
