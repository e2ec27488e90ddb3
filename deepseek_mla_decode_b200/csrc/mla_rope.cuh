// Rotary positions shared by the query rotation (mla_rope.cu) and the cache append
// (mla_append.cu).
//
// Pair i of the 64-wide rotary part turns by freq[i] radians a position:
//     (a, b) -> (a cos t - b sin t, a sin t + b cos t) * amplitude,   t = p * freq[i]
// A position of 10^5 with a frequency near 1 is tens of thousands of turns, of which
// fp32 would keep two digits.  The angle is therefore kept in turns in fp64 and reduced
// there, exactly, to a fraction in [-1/2, 1/2]; only that fraction goes to fp32 and to
// sincospif (angle error pi * 2^-25, 2^16 times below a bf16 step).
#pragma once
#include <cuda_runtime.h>
#include <cstdint>
#include "mla_internal.h"
#include "../../include/mla_decode.h"

namespace mla {

// A rotation as the kernels take it (by value).
struct RopeTurns {
  double turns[kDRope / 2];  // turns a position of each pair
  float amplitude;
};

// Host side: false when the caller's rotation is not usable.
bool rope_turns(const mla_rope_t* rope, RopeTurns* out);

#ifdef __CUDACC__
// cos and sin of pair `pair` at position pos, times the amplitude.
__device__ __forceinline__ void rope_cos_sin(const RopeTurns& r, int pair, int pos, float* c, float* s) {
  double t = static_cast<double>(pos) * r.turns[pair];
  t -= rint(t);
  float sn, cs;
  sincospif(2.0f * static_cast<float>(t), &sn, &cs);
  *c = cs * r.amplitude;
  *s = sn * r.amplitude;
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
