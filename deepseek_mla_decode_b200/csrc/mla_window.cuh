// Shared by the windowed decode kernels (mla_decode_kernel.cu over the bf16 cache,
// mla_window_fp8.cu over the FP8 cache).
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "mla_internal.h"
#include "pair_ptx.cuh"

namespace mla {

// Rows that no piece covers: a unit without a visible key (0 / -inf; the padding tokens of a
// ragged batch), with an invalid length or count (NaN and MLA_DEVICE_ERR_SEQLEN) or with a
// block count in the metadata that is not its length's (NaN and MLA_DEVICE_ERR_METADATA).
// Partition `part` of P takes the units u with u % P == part.  One warp, whose CTA has no
// other use for it, writes them from the kernel's start on: at the end of the kernel this
// was on its critical path (three units of eight are padding when one to four of four draft
// tokens are kept).  The lanes look at 32 units at a time.
template <class UnitLen>
__device__ __forceinline__ void write_orphan_units(const int32_t* meta, int units, int M, int window, int sinks,
                                                   int part, int P, int lane, UnitLen unit_len, __nv_bfloat16* out,
                                                   float* lse, int32_t* status) {
  const float nan = __int_as_float(0x7fc00000);
  for (int base = part; base < units; base += 32 * P) {
    const int u = base + lane * P;
    int bits = 0;
    bool orphan = false;
    if (u < units) {
      const int n = unit_len(u);
      if (n < 0)
        bits = kErrSeqlen;
      else if (meta[off_nblk() + u] != window_blocks(n, window, sinks).count)
        bits = kErrMetadata;
      orphan = bits != 0 || n == 0;
    }
    if (bits != 0 && status) atomicOr(status, bits);
    uint32_t left = __ballot_sync(0xffffffffu, orphan);
    const uint32_t bad = __ballot_sync(0xffffffffu, bits != 0);
    while (left) {
      const int k = __ffs(left) - 1;
      left &= left - 1;
      const int64_t row0 = ((int64_t)base + (int64_t)k * P) * M;
      const float v = (bad >> k) & 1 ? nan : 0.0f;
      const uint32_t pv = ptx::pack_bf16x2(v, v);
      uint4* o = reinterpret_cast<uint4*>(out + row0 * kDLatent);
#pragma unroll 4
      for (int i = lane; i < M * (kDLatent / 8); i += 32) o[i] = make_uint4(pv, pv, pv, pv);
      for (int r = lane; r < M; r += 32) lse[row0 + r] = (bad >> k) & 1 ? nan : -INFINITY;
    }
  }
}

}  // namespace mla
