// Rotary positions of the queries, and the frequencies of a rotation.
//
// mla_rope_q splits 192-wide heads [128 without position | 64 rotary] into the operands of
// the absorption GEMM (the 128) and of the decode (the 64, rotated); mla_rope_inplace
// rotates the 64 where they lie.  Memory-bound: 384 bytes read and written a head.
//
// Measured: 8192 tokens x 128 heads in 127.9 us, 6.30 TB/s, 96 % of a plain copy; a decode
// step's 256 tokens x 128 heads in 4.4-4.9 us (floor 3.8); one token 2.5 us, a launch.  In
// place 68.4 us (floor 41: 128 of every 384 bytes, 60 % of a copy) and 3.7 us (floor 1.3).
//
// Eight lanes take a head: two 16-byte pieces of its 128 and one of its 64 each, so a warp
// moves four heads with three loads a lane.  A warp stays on one row (one position): lane i
// computes pair i's angle once and the eight lanes of a head fetch the cosines and sines of
// their pairs by shuffles.
#include <cuda_bf16.h>
#include <cmath>
#include <type_traits>
#include "mla_rope.cuh"

namespace mla {
namespace {

constexpr int kDNope = 128, kDHead = kDNope + kDRope;
constexpr int kWarpsPerBlock = 8;
constexpr int kHeadsPerPass = 4;
constexpr int kHeadsPerWarp = 16;

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// kSplit: q [R][H][192] -> q_heads [R][H][128], q_pe [R][H][64]; else q_pe = q and the
// rotary part is rotated in place.  kHalf: pair i = (x[i], x[i + 32]), else (x[2i], x[2i+1]).
// kSkipPadding: q's loads wait for the sequence's words and padding is not read (its heads are
// read and dropped otherwise): 8192 tokens x 128 heads of which half are real 105 us against
// 128; waiting costs 2 % where all are real (131 us against 128).
template <bool kHalf, bool kSplit, bool kSkipPadding>
__global__ void __launch_bounds__(kWarpsPerBlock * 32) rope_q_kernel(
    const __nv_bfloat16* q, int64_t row_stride, const int32_t* seqlens, const int32_t* q_lens, uint32_t rows,
    const __grid_constant__ RowDiv per_seq, int H, const __grid_constant__ RopeTurns rope, __nv_bfloat16* q_heads,
    __nv_bfloat16* q_pe, int32_t* status) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  // block (x, y): rows of a group of kHeadsPerWarp heads
  const uint32_t row32 = blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
  if (row32 >= rows) return;
  const int64_t row = row32;
  const int h0 = (int)blockIdx.y * kHeadsPerWarp, s_q = (int)per_seq.d;
  const int b = per_seq.quotient(row32), i = (int)(row32 - (uint32_t)b * per_seq.d);
  const int pos = token_position(seqlens[b], q_lens ? q_lens[b] : s_q, i, s_q);
  if (pos == kTokenBad && h0 == 0 && lane == 0 && status) atomicOr(status, kErrSeqlen);
  // no position: zeros; an invalid length or count: NaN
  const uint32_t fill = pos == kTokenBad ? 0x7fc07fc0u : 0u;
  if (kSkipPadding && pos < 0) {
    const uint4 v = make_uint4(fill, fill, fill, fill);
    const int heads = min(H - h0, kHeadsPerWarp);
    if (kSplit) {
      uint4* dn = reinterpret_cast<uint4*>(q_heads + (row * H + h0) * kDNope);
      uint4* dp = reinterpret_cast<uint4*>(q_pe + (row * H + h0) * kDRope);
      for (int k = lane; k < heads * (kDNope / 8); k += 32) dn[k] = v;
      for (int k = lane; k < heads * (kDRope / 8); k += 32) dp[k] = v;
    } else {
      for (int k = lane; k < heads * (kDRope / 8); k += 32)
        reinterpret_cast<uint4*>(q_pe + row * row_stride + (int64_t)(h0 + k / 8) * kDHead)[kDNope / 8 + k % 8] = v;
    }
    return;
  }
  float c = 0.f, s = 0.f;
  if (pos >= 0) rope_cos_sin(rope, lane, pos, &c, &s);
  const int j = lane & 7;  // 16-byte piece of the rotary part
  constexpr int kPairs = kHalf ? 8 : 4;
  float cs[kPairs], sn[kPairs];
#pragma unroll
  for (int e = 0; e < kPairs; ++e) {
    const int pair = kHalf ? 8 * (j & 3) + e : 4 * j + e;
    cs[e] = __shfl_sync(0xffffffffu, c, pair);
    sn[e] = __shfl_sync(0xffffffffu, s, pair);
    if (kHalf && j < 4) sn[e] = -sn[e];
  }
#pragma unroll
  for (int g = 0; g < kHeadsPerWarp; g += kHeadsPerPass) {
    const int h = h0 + g + (lane >> 3);
    const bool on = h < H;
    const int hc = on ? h : H - 1;
    const uint4* src = reinterpret_cast<const uint4*>(q + row * row_stride + (int64_t)hc * kDHead);
    uint4 n0, n1, x;
    if (kSplit) {
      n0 = src[j];
      n1 = src[j + 8];
    }
    x = src[kDNope / 8 + j];
    uint4 y;
    if (kHalf) {
      uint4 o;  // the pairs' other members
      o.x = __shfl_xor_sync(0xffffffffu, x.x, 4);
      o.y = __shfl_xor_sync(0xffffffffu, x.y, 4);
      o.z = __shfl_xor_sync(0xffffffffu, x.z, 4);
      o.w = __shfl_xor_sync(0xffffffffu, x.w, 4);
      y.x = pack(lo_f(x.x) * cs[0] + lo_f(o.x) * sn[0], hi_f(x.x) * cs[1] + hi_f(o.x) * sn[1]);
      y.y = pack(lo_f(x.y) * cs[2] + lo_f(o.y) * sn[2], hi_f(x.y) * cs[3] + hi_f(o.y) * sn[3]);
      y.z = pack(lo_f(x.z) * cs[kPairs - 4] + lo_f(o.z) * sn[kPairs - 4],
                 hi_f(x.z) * cs[kPairs - 3] + hi_f(o.z) * sn[kPairs - 3]);
      y.w = pack(lo_f(x.w) * cs[kPairs - 2] + lo_f(o.w) * sn[kPairs - 2],
                 hi_f(x.w) * cs[kPairs - 1] + hi_f(o.w) * sn[kPairs - 1]);
    } else {
      y.x = pack(lo_f(x.x) * cs[0] - hi_f(x.x) * sn[0], lo_f(x.x) * sn[0] + hi_f(x.x) * cs[0]);
      y.y = pack(lo_f(x.y) * cs[1] - hi_f(x.y) * sn[1], lo_f(x.y) * sn[1] + hi_f(x.y) * cs[1]);
      y.z = pack(lo_f(x.z) * cs[2] - hi_f(x.z) * sn[2], lo_f(x.z) * sn[2] + hi_f(x.z) * cs[2]);
      y.w = pack(lo_f(x.w) * cs[3] - hi_f(x.w) * sn[3], lo_f(x.w) * sn[3] + hi_f(x.w) * cs[3]);
    }
    if (!kSkipPadding && pos < 0) n0 = n1 = y = make_uint4(fill, fill, fill, fill);
    if (!on) continue;
    if (kSplit) {
      const int64_t head = row * H + h;
      uint4* dn = reinterpret_cast<uint4*>(q_heads + head * kDNope);
      dn[j] = n0;
      dn[j + 8] = n1;
      reinterpret_cast<uint4*>(q_pe + head * kDRope)[j] = y;
    } else {
      reinterpret_cast<uint4*>(q_pe + row * row_stride + (int64_t)h * kDHead)[kDNope / 8 + j] = y;
    }
  }
}

mla_status_t rope_q_any(const void* q, int64_t row_stride, const int32_t* cache_seqlens, const int32_t* q_lens, int B,
                        int s_q, int H, const mla_rope_t* rope, void* q_heads, void* q_pe, int32_t* status,
                        void* stream) {
  if (!q || !cache_seqlens || !rope) return MLA_ERR_INVALID_ARG;
  if (B < 1 || s_q < 1 || H < 1 || H > 65535 || (int64_t)B * s_q > 0x7fffffffLL) return MLA_ERR_INVALID_ARG;
  if (row_stride < (int64_t)H * kDHead || (row_stride & 7)) return MLA_ERR_INVALID_ARG;
  const uintptr_t wide = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q_heads) |
                         reinterpret_cast<uintptr_t>(q_pe);
  const uintptr_t words = reinterpret_cast<uintptr_t>(cache_seqlens) | reinterpret_cast<uintptr_t>(q_lens) |
                          reinterpret_cast<uintptr_t>(status);
  if ((wide & 15u) || (words & 3u)) return MLA_ERR_INVALID_ARG;
  RopeTurns turns;
  if (!rope_turns(rope, &turns)) return MLA_ERR_INVALID_ARG;
  int sms = 0;
  mla_status_t st = mla_device_sm_count(&sms);
  if (st != MLA_OK) return st;
  const int64_t rows = (int64_t)B * s_q;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + kWarpsPerBlock - 1) / kWarpsPerBlock),
                     (unsigned)((H + kHeadsPerWarp - 1) / kHeadsPerWarp));
  cfg.blockDim = dim3(kWarpsPerBlock * 32);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool split = q_heads != nullptr;
  // more warps than the GPU holds (40 an SM): bytes count, not the first load's delay
  const bool skip = q_lens != nullptr && (int64_t)cfg.gridDim.x * cfg.gridDim.y * kWarpsPerBlock > (int64_t)sms * 40;
  auto pick = [&](auto half) {
    constexpr bool kHalf = decltype(half)::value;
    if (split) return skip ? rope_q_kernel<kHalf, true, true> : rope_q_kernel<kHalf, true, false>;
    return skip ? rope_q_kernel<kHalf, false, true> : rope_q_kernel<kHalf, false, false>;
  };
  auto* kernel = rope->half_layout ? pick(std::true_type{}) : pick(std::false_type{});
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<const __nv_bfloat16*>(q), row_stride, cache_seqlens, q_lens,
                         (uint32_t)rows, RowDiv(s_q), H, turns, static_cast<__nv_bfloat16*>(q_heads),
                         static_cast<__nv_bfloat16*>(q_pe), status) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}

}  // namespace

bool rope_turns(const mla_rope_t* rope, RopeTurns* out) {
  constexpr long double kTurn = 1.0L / 6.283185307179586476925286766559L;
  if (rope->half_layout != 0 && rope->half_layout != 1) return false;
  if (!std::isfinite(rope->amplitude)) return false;
  for (int i = 0; i < kDRope / 2; ++i) {
    // beyond this extended precision keeps too little of a turn's fraction
    if (!(std::fabs(rope->freq[i]) <= 1e6)) return false;
    // whole turns of either sign drop out, and the fraction is kept to 2^-63 of a turn
    long double t = rope->freq[i] * kTurn;
    t -= static_cast<long double>(static_cast<int64_t>(t));
    out->turns[i] = static_cast<uint64_t>(static_cast<int64_t>(t * 0x1p63L)) << 1;
  }
  out->amplitude = rope->amplitude;
  return true;
}

}  // namespace mla

extern "C" {

mla_status_t mla_rope_init(mla_rope_t* rope, double base, int half_layout, int scaling, double factor,
                           double original_len, double beta_fast, double beta_slow, double amplitude) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (!rope || !(base > 1.0) || !std::isfinite(base) || (half_layout != 0 && half_layout != 1) ||
      !std::isfinite(amplitude))
    return MLA_ERR_INVALID_ARG;
  if (scaling != MLA_ROPE_PLAIN && scaling != MLA_ROPE_LINEAR && scaling != MLA_ROPE_YARN) return MLA_ERR_INVALID_ARG;
  if (scaling != MLA_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return MLA_ERR_INVALID_ARG;
  double lo = 0.0, hi = 0.0;
  if (scaling == MLA_ROPE_YARN) {
    if (!(original_len > 0.0) || !std::isfinite(original_len) || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) ||
        !std::isfinite(beta_fast))
      return MLA_ERR_INVALID_ARG;
    // (fractional) pair index whose wave turns `turns` times within original_len
    const auto pair_of = [&](double turns) {
      return MLA_D_ROPE * std::log(original_len / (turns * kTwoPi)) / (2.0 * std::log(base));
    };
    lo = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
    hi = std::fmin(std::ceil(pair_of(beta_slow)), MLA_D_ROPE - 1.0);
  }
  for (int i = 0; i < MLA_D_ROPE / 2; ++i) {
    double f = std::pow(base, -2.0 * i / MLA_D_ROPE);
    if (scaling == MLA_ROPE_LINEAR) f /= factor;
    if (scaling == MLA_ROPE_YARN) {
      const double g = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      f = f * (1.0 - g) + f / factor * g;
    }
    rope->freq[i] = f;
  }
  rope->amplitude = static_cast<float>(amplitude);
  rope->half_layout = half_layout;
  return std::isfinite(rope->amplitude) ? MLA_OK : MLA_ERR_INVALID_ARG;
}

mla_status_t mla_rope_q(const void* q, int64_t row_stride, const int32_t* cache_seqlens, const int32_t* q_lens, int B,
                        int s_q, int H, const mla_rope_t* rope, void* q_heads, void* q_pe, int32_t* status,
                        void* stream) {
  if (!q_heads || !q_pe) return MLA_ERR_INVALID_ARG;
  return mla::rope_q_any(q, row_stride, cache_seqlens, q_lens, B, s_q, H, rope, q_heads, q_pe, status, stream);
}

mla_status_t mla_rope_inplace(void* q, int64_t row_stride, const int32_t* cache_seqlens, const int32_t* q_lens, int B,
                              int s_q, int H, const mla_rope_t* rope, int32_t* status, void* stream) {
  return mla::rope_q_any(q, row_stride, cache_seqlens, q_lens, B, s_q, H, rope, nullptr, q, status, stream);
}

}  // extern "C"
