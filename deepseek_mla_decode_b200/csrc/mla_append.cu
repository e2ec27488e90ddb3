// Appending new tokens' rows to the paged latent cache, bf16 or packed FP8.
//
// A new row arrives as the down-projection left it, x = [c (512) | k (64)], and is stored
// at position p = n_b - q_b + i of its sequence as
//     [ c * w / sqrt(mean(c^2) + eps) | rot_p(k) ]        (norm and rotation optional)
// rounded once: to bf16, or to the packed FP8 row of mla_fp8.cu, whose scale, codes and
// scaled rotary keys come from the 32-bit row.  Memory-bound: 1152 bytes read and 1152 or
// 656 written a row.
//
// Measured: 65536 rows with norm and rotation in 29.7 us, 5.1 TB/s, 78 % of a plain copy
// (25.4 us without the two); 20 k FP8 rows in 12.6 us, whose 16 codes a lane are products
// instead of divisions where that decides them (17.2 us with divisions); a decode step's 256
// rows in 2.4 us, a launch.  Two rows a warp (30.5 us) and persistent warps that load a row
// ahead (36 us) lose to more warps: 48 registers keep 40 of them on an SM.  What bounds both
// is latency: 33 warps run at a time, an instruction waits 14 to 15 cycles, 4 to 5 of them for
// loads and 4 for the butterflies, and the issue slots are busy in 54 % (bf16) and 58 % (FP8) of
// the cycles, DRAM at 42 % and 16 % of its rate.
//
// One warp per row.  Lane l holds c[8l..8l+7] and c[256+8l..256+8l+7] (two 16-byte loads,
// and 8- or 16-byte stores, contiguous over the warp) and pair l of k; the sum of squares
// and the row maximum are butterflies over the warp, in a fixed order.
#include <cuda_bf16.h>
#include <cmath>
#include "mla_rope.cuh"
#include "ptx_sm100.cuh"

namespace mla {

using namespace ptx;

namespace {

constexpr int kWarpsPerBlock = 4;

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7]));
}
// two fp32 -> two e4m3 (nearest even, saturating), lo in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// maximum that keeps a NaN: a row that holds one gets a NaN scale and reads back as NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Codes of 16 values over scale, as IEEE quotients rounded to e4m3.  Products by 1/scale
// shrunk and stretched by 2^-21 (1/scale and the product are each off by 2^-24) bracket the
// quotient, and rounding keeps order: where both give the same codes, those are the
// quotient's.  That holds for all but about one value in 2^16; the others are divided.
__device__ __forceinline__ uint32_t codes4(const float* f, float r) {
  return e4m3x2(f[0] * r, f[1] * r) | (e4m3x2(f[2] * r, f[3] * r) << 16);
}
__device__ __forceinline__ uint32_t divided_codes4(const float* f, float scale) {
  return e4m3x2(__fdiv_rn(f[0], scale), __fdiv_rn(f[1], scale)) |
         (e4m3x2(__fdiv_rn(f[2], scale), __fdiv_rn(f[3], scale)) << 16);
}
__device__ __forceinline__ void codes16(const float (&c0)[8], const float (&c1)[8], float scale, uint32_t (&q)[4]) {
  const float r = __frcp_rn(scale);
  const float below = r * (1.0f - 0x1p-21f), above = r * (1.0f + 0x1p-21f);
  bool same = scale > 0x1p-100f && scale < 0x1p100f;  // 1/scale is a normal number
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* f = (i < 2 ? c0 : c1) + 4 * (i & 1);
    q[i] = codes4(f, below);
    same = same && q[i] == codes4(f, above);
  }
  if (!same) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = divided_codes4((i < 2 ? c0 : c1) + 4 * (i & 1), scale);
  }
}

struct AppendParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* weight;  // norm weight, or null: no norm
  const int32_t* block_table;
  const int32_t* seqlens;
  const int32_t* q_lens;
  int32_t* status;
  uint8_t* cache;
  int64_t row_stride, num_blocks;
  uint32_t rows;
  int max_blocks;
  float eps;
  int rotate;  // 0: store k as given
  int half_layout;
  RowDiv per_seq;  // tokens a sequence
  RopeTurns rope;
};

// kSkipPadding: the row's loads wait for the sequence's words, and padding is not read; else
// they go out at once.  Waiting pays where many rows may be padding and their bytes count:
// 32764 rows of which half are real 13.1 us against 14.0, 512 rows of which 5 in 8 are real
// 3.3 us against 3.1.
template <bool kFp8, bool kSkipPadding>
__global__ void __launch_bounds__(kWarpsPerBlock * 32) append_kernel(const __grid_constant__ AppendParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const uint32_t row = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  const int i0 = p.half_layout ? lane : 2 * lane, i1 = p.half_layout ? lane + 32 : 2 * lane + 1;
  uint4 v0, v1;
  __nv_bfloat16 k0, k1;
  auto load = [&]() {
    const __nv_bfloat16* src = p.x + (int64_t)row * p.row_stride;
    v0 = reinterpret_cast<const uint4*>(src)[lane];
    v1 = reinterpret_cast<const uint4*>(src)[lane + 32];
    k0 = src[kDLatent + i0];
    k1 = src[kDLatent + i1];
  };
  if constexpr (!kSkipPadding) load();
  const int s_q = (int)p.per_seq.d, b = p.per_seq.quotient(row), i = (int)(row - (uint32_t)b * p.per_seq.d);
  const int n = p.seqlens[b];
  int pos = token_position(n, p.q_lens ? p.q_lens[b] : s_q, i, s_q);
  if ((int64_t)n > (int64_t)p.max_blocks * kBlockSize) pos = kTokenBad;
  const int32_t block = pos >= 0 ? p.block_table[(int64_t)b * p.max_blocks + pos / kBlockSize] : -1;
  if (pos < 0 || block < 0 || (int64_t)block >= p.num_blocks) {
    if (lane == 0 && p.status && pos != kTokenNone) atomicOr(p.status, pos < 0 ? kErrSeqlen : kErrBlockId);
    return;
  }
  if constexpr (kSkipPadding) load();
  float a = __bfloat162float(k0), d = __bfloat162float(k1);
  float c0[8], c1[8];
  unpack8(v0, c0);
  unpack8(v1, c1);
  if (p.weight) {  // in packed pairs: half the issue slots of the scalar form
    float w0[8], w1[8];
    unpack8(reinterpret_cast<const uint4*>(p.weight)[lane], w0);
    unpack8(reinterpret_cast<const uint4*>(p.weight)[lane + 32], w1);
    uint64_t s0 = pack_f32x2(0.f, 0.f), s1 = s0;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint64_t x0 = pack_f32x2(c0[e], c0[e + 1]), x1 = pack_f32x2(c1[e], c1[e + 1]);
      s0 = fma2(x0, x0, s0);
      s1 = fma2(x1, x1, s1);
    }
    float ss, odd;
    unpack_f32x2(add2(s0, s1), ss, odd);
    ss += odd;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * (1.0f / kDLatent) + p.eps);
    const uint64_t rr = pack_f32x2(r, r);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      unpack_f32x2(mul2(mul2(pack_f32x2(c0[e], c0[e + 1]), rr), pack_f32x2(w0[e], w0[e + 1])), c0[e], c0[e + 1]);
      unpack_f32x2(mul2(mul2(pack_f32x2(c1[e], c1[e + 1]), rr), pack_f32x2(w1[e], w1[e + 1])), c1[e], c1[e + 1]);
    }
  }
  if (p.rotate) {
    float cs, sn;
    rope_cos_sin(p.rope, lane, pos, &cs, &sn);
    const float a0 = a, d0 = d;
    a = a0 * cs - d0 * sn;
    d = a0 * sn + d0 * cs;
  }
  const int64_t slot = (int64_t)block * kBlockSize + pos % kBlockSize;
  if constexpr (kFp8) {
    float amax = max_nan(fabsf(a), fabsf(d));
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max_nan(amax, max_nan(fabsf(c0[e]), fabsf(c1[e])));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float scale = __fdiv_rn(amax, 448.0f);
    uint32_t q[4] = {0u, 0u, 0u, 0u};
    float ka = 0.f, kd = 0.f;
    if (scale > 0.f) {
      codes16(c0, c1, scale, q);
      ka = __fdiv_rn(a, scale);
      kd = __fdiv_rn(d, scale);
    }
    uint8_t* dst = p.cache + slot * kRowBytes8;
    reinterpret_cast<uint2*>(dst)[lane] = make_uint2(q[0], q[1]);
    reinterpret_cast<uint2*>(dst)[lane + 32] = make_uint2(q[2], q[3]);
    __nv_bfloat16* kp = reinterpret_cast<__nv_bfloat16*>(dst + kOffKpe8);
    kp[i0] = __float2bfloat16_rn(ka);
    kp[i1] = __float2bfloat16_rn(kd);
    if (lane == 0) reinterpret_cast<uint4*>(dst + kOffScale8)[0] = make_uint4(__float_as_uint(scale), 0u, 0u, 0u);
  } else {
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.cache) + slot * kDQK;
    reinterpret_cast<uint4*>(dst)[lane] = pack8(c0);
    reinterpret_cast<uint4*>(dst)[lane + 32] = pack8(c1);
    dst[kDLatent + i0] = __float2bfloat16_rn(a);
    dst[kDLatent + i1] = __float2bfloat16_rn(d);
  }
}

mla_status_t append_any(bool fp8, const void* kv_a, int64_t row_stride, const void* norm_weight, float eps,
                        const int32_t* block_table, int max_blocks, const int32_t* cache_seqlens,
                        const int32_t* q_lens, int B, int s_q, const mla_rope_t* rope, void* cache,
                        int64_t num_blocks, int32_t* status, void* stream) {
  if (!kv_a || !block_table || !cache_seqlens || !cache) return MLA_ERR_INVALID_ARG;
  if (B < 1 || s_q < 1 || (int64_t)B * s_q > 0x7fffffffLL) return MLA_ERR_INVALID_ARG;
  if (num_blocks < 1 || num_blocks > (int64_t)INT32_MAX || max_blocks < 1) return MLA_ERR_INVALID_ARG;
  if (row_stride < kDQK || (row_stride & 7)) return MLA_ERR_INVALID_ARG;
  if (norm_weight && !(eps >= 0.f && eps < 1e30f)) return MLA_ERR_INVALID_ARG;
  const uintptr_t wide = reinterpret_cast<uintptr_t>(kv_a) | reinterpret_cast<uintptr_t>(norm_weight) |
                         reinterpret_cast<uintptr_t>(cache);
  const uintptr_t words = reinterpret_cast<uintptr_t>(cache_seqlens) | reinterpret_cast<uintptr_t>(q_lens) |
                          reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(status);
  if ((wide & 15u) || (words & 3u)) return MLA_ERR_INVALID_ARG;
  AppendParams p = {.per_seq = RowDiv(s_q)};
  if (rope && !rope_turns(rope, &p.rope)) return MLA_ERR_INVALID_ARG;
  int sms = 0;
  mla_status_t st = mla_device_sm_count(&sms);
  if (st != MLA_OK) return st;
  p.x = static_cast<const __nv_bfloat16*>(kv_a);
  p.weight = static_cast<const __nv_bfloat16*>(norm_weight);
  p.block_table = block_table;
  p.seqlens = cache_seqlens;
  p.q_lens = q_lens;
  p.status = status;
  p.cache = static_cast<uint8_t*>(cache);
  p.row_stride = row_stride;
  p.rows = (uint32_t)B * (uint32_t)s_q;
  p.num_blocks = num_blocks;
  p.max_blocks = max_blocks;
  p.eps = eps;
  p.rotate = rope != nullptr;
  p.half_layout = rope ? rope->half_layout : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.rows + kWarpsPerBlock - 1) / kWarpsPerBlock);
  cfg.blockDim = dim3(kWarpsPerBlock * 32);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // more rows than the GPU holds warps (40 an SM)
  const bool skip = q_lens != nullptr && p.rows > (uint32_t)sms * 40;
  auto* kernel = fp8 ? (skip ? append_kernel<true, true> : append_kernel<true, false>)
                     : (skip ? append_kernel<false, true> : append_kernel<false, false>);
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return MLA_ERR_CUDA;
  return MLA_OK;
}

}  // namespace
}  // namespace mla

extern "C" {

mla_status_t mla_append_kv(const void* kv_a, int64_t row_stride, const void* norm_weight, float eps,
                           const int32_t* block_table, int max_blocks, const int32_t* cache_seqlens,
                           const int32_t* q_lens, int B, int s_q, const mla_rope_t* rope, void* kv_cache,
                           int64_t num_blocks, int32_t* status, void* stream) {
  return mla::append_any(false, kv_a, row_stride, norm_weight, eps, block_table, max_blocks, cache_seqlens, q_lens, B,
                         s_q, rope, kv_cache, num_blocks, status, stream);
}

mla_status_t mla_append_kv_fp8(const void* kv_a, int64_t row_stride, const void* norm_weight, float eps,
                               const int32_t* block_table, int max_blocks, const int32_t* cache_seqlens,
                               const int32_t* q_lens, int B, int s_q, const mla_rope_t* rope, void* kv_fp8,
                               int64_t num_blocks, int32_t* status, void* stream) {
  return mla::append_any(true, kv_a, row_stride, norm_weight, eps, block_table, max_blocks, cache_seqlens, q_lens, B,
                         s_q, rope, kv_fp8, num_blocks, status, stream);
}

}  // extern "C"
