// Rotary positions shared by the query rotation (mla_rope.cu) and the cache append
// (mla_append.cu).
//
// Pair i of the 64-wide rotary part turns by freq[i] radians a position:
//     (a, b) -> (a cos t - b sin t, a sin t + b cos t) * amplitude,   t = p * freq[i]
// A position of 10^5 with a frequency near 1 is tens of thousands of turns, of which
// fp32 would keep two digits.  Only the fraction of a turn counts, so a frequency is kept as
// its fraction of a turn a position, cut on the host from extended precision to 2^-63 of a turn
// (towards zero; in units of 2^-64, whose last bit is 0), and p times it modulo 2^64 is the
// angle's fraction, off by less than p 2^-63 of a turn for frequencies up to a turn a position
// (2^-32 of a turn at the largest p; a frequency of k turns keeps log2 k bits less): one integer
// product instead of fp64 arithmetic and its conversions.  The upper 32 bits as a
// signed number are the angle in [-1/2, 1/2) turns, which goes to fp32 (angle error
// pi 2^-24) and, being within [-pi, pi], to the fast sine and cosine (absolute error 2^-21.2
// there by CUDA's documentation).  Together under 2^-20.5 of the pair's length, 2^12 times below
// a bf16 half step of it; a component that the rotation takes close to 0 keeps that absolute
// error.  The accurate functions took 45 of the append's 290 instructions a row.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>
#include "mla_internal.h"
#include "../../include/mla_decode.h"

namespace mla {

// A rotation as the kernels take it (by value).
struct RopeTurns {
  uint64_t turns[kDRope / 2];  // turns a position of each pair modulo 1, in 2^-64
  float amplitude;
};

// Division of a row number (< 2^31) by the tokens a sequence: row / d = row * mul >> shift
// with mul = floor(2^shift / d) + 1 and 2^(shift - 31) the power of two at or above d.
struct RowDiv {
  uint32_t d, mul;
  int shift;
  explicit RowDiv(int d_) : d((uint32_t)d_) {
    int l = 0;
    while ((1u << l) < d) ++l;
    shift = 31 + l;
    mul = (uint32_t)((uint64_t(1) << shift) / d + 1);
  }
  __host__ __device__ int quotient(uint32_t row) const { return (int)(((uint64_t)row * mul) >> shift); }
};

// Host side: false when the caller's rotation is not usable.
bool rope_turns(const mla_rope_t* rope, RopeTurns* out);

#ifdef __CUDACC__
// cos and sin of pair `pair` at position pos, times the amplitude.
__device__ __forceinline__ void rope_cos_sin(const RopeTurns& r, int pair, int pos, float* c, float* s) {
  const uint64_t t = static_cast<uint64_t>(static_cast<uint32_t>(pos)) * r.turns[pair];
  const float angle = static_cast<float>(static_cast<int32_t>(t >> 32)) * (6.2831853071795865f * 0x1p-32f);
  *c = __cosf(angle) * r.amplitude;
  *s = __sinf(angle) * r.amplitude;
}

// Position of new token i of a sequence with n cached tokens (the new ones counted), q of
// them new.  kTokenNone: padding (i >= q) or no place in the sequence (n < q: a negative
// position); kTokenBad: n or q invalid.
constexpr int kTokenNone = -1, kTokenBad = -2;
__device__ __forceinline__ int token_position(int n, int q, int i, int s_q) {
  if (n < 0 || q < 0 || q > s_q) return kTokenBad;
  if (i >= q) return kTokenNone;
  const int p = n - q + i;
  return p < 0 ? kTokenNone : p;
}
#endif

}  // namespace mla
