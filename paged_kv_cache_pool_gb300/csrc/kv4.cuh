// 4-bit COLD rows: where a row keeps what, and the code of a value.
//
// A row holds one token's K and V of every KV head: per head K's codes then V's,
// d / 2 bytes each, then per head the (lo, span) pairs of K's groups of 64 channels,
// then of V's.  Value = lo + code * (span / 15).
//
// The order of channels inside the codes is the one in which the attention's warp
// tiles take them: eight channels a 32-bit word, and at d = 128 the words of the two
// groups in turn, so that a thread's 16 bytes of K, and its 8 bytes of V, hold as many
// channels of either group (a tensor-core step must stay inside a group, whose
// span is applied to its sum).
#pragma once

#include <cstdint>

namespace gk {
namespace kv4 {

constexpr int kGroup = 64;  // channels that share lo and span
// a span below 2^-100 is held as 0, so that its reciprocal and products stay in fp32's normal range
constexpr float kLeastSpan = 7.888609052210118e-31f;
// from 2^120 on a group is held as NaN: 15 times a wider span could pass fp32
constexpr float kMostSpan = 1.329227995784916e36f;

__host__ __device__ constexpr int row_bytes(int hkv, int d) { return (hkv * d + hkv * d / 8 + 15) / 16 * 16; }
// byte of a head's codes (K's; V's are d / 2 further) and of its scales (K's; V's are d / 16 further)
__host__ __device__ constexpr int codes_at(int h, int d) { return h * d; }
__host__ __device__ constexpr int scales_at(int hkv, int h, int d) { return hkv * d + h * (d / 8); }

}  // namespace kv4
}  // namespace gk
