// Windowed decode over the packed FP8 cache, on its codes as they are.
//
// Math: mla_decode_kernel.cu's, over the token schedule and a window's visible blocks
// (window_blocks).  A cache row is s * [code | k'], code e4m3 (512), k' bf16 (64), s fp32.
//
// Both products are of 8-bit floats (tcgen05 kind::f8f6f4, fp32 accumulators), and the operand
// that is not a code goes in as two terms: hi, the value rounded to e4m3, and lo, what hi's code
// left of it (its smallest steps included) rounded to e5m2.  Four bits, three and lo's sign are
// the eight of a bf16 value, and e5m2's range carries on where e4m3's ends: off by at most
// 2^-8 of the value down to 2^-6, 2^-14 below that, 2^-17 and less below 2^-14.
//   QK:  q * 2^j = q_hi + q_lo, the power of two taking the row's largest value to
//        [128, 256): exact down to 2^-6, 2^-13 of the row's largest.  k' splits the same way
//        into [k'_hi | k'_lo], a fifth 128-wide chunk beside the four of codes, against
//        [q_hi | q_hi] and [q_lo | q_lo].
//   PV:  P = 2^(x - m) * s = P_hi + P_lo.  Every key counts: where one key takes most of the
//        weight (the first keys, which are kept visible for that), thousands share the rest, and
//        a grid fixed by the largest loses them.  So m follows the largest x + log2 s of each
//        tile, up and down, lazily: a tile's largest P stays in [2^6, 2^8.5), O is rescaled
//        when it would leave that, and a weight is off by at most 2^-8 of itself or 2^-20 of
//        its tile's largest (a tile's 256 keys together lose less than 2^-12 of that one).  The
//        normaliser l = sum 2^(x - m) is fp32, in the unit of the row's largest.
// Two 8-bit MMAs take the time of one bf16 MMA, so this costs no tensor time over the bf16
// cache, moves half its bytes through the ring, and converts nothing but the 64 rotary
// values a key.
//
// Unit, TMEM, ring order, softmax thread map, epilogue and failure path are those of
// mla_decode_kernel.cu: a pair of CTAs takes 128 rows (here one token's heads), CTA r rows
// [64r, 64r + 64), keys [128r, 128r + 128) of a 256-key tile as its half of the QK operand
// and dims 256h + 128r + (0..127) as its half of the PV operand.  One box of the cache, 64
// rows x 128 code bytes, serves both: K-major for QK, MN-major for PV.
//
// Measured (192 sequences, 128 heads, window 4096, attention and combine): 262-272 us,
// 49 % of the tensor floor, against 432 us for the kernel that converts codes to
// bf16; with scores six times as wide 265-281 us.  128 sequences with up to four draft tokens,
// window 512: 134-146 us against a floor of 33, and 256 sequences, window 1024: 145 us against
// 44, both more than the bf16 cache's 100 and 117 us: a piece of five tiles or less is mostly
// its switch.  No unit is busy half the time (tensor pipe 45 %, issue 35 %, DRAM 27 %); a tile of
// 9.7 k cycles is the softmax's two passes (5 k), its hand-offs (3 k) and, spread over 13
// tiles, the switch of pieces (0.9 k: the new query's terms and the old output).  The
// instruction stream is part of it: with both passes unrolled over 64 keys and the terms made
// by unrolled code the kernel took 346 us, for the warps waited for instructions; so the
// passes run over groups of 16 and 32 keys and read the scores from tensor memory twice.  128
// registers a thread at compile time leave 24 bytes of spills.
//
// Warps: 0, 2, 3 producers, 1 MMA issue (leader) and TMEM, 4..11 softmax and epilogue,
// 12..15 preparation (the query rows' terms once a piece; the rotary keys' terms and the
// scale tables once a tile).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstdint>
#include <cstring>
#include "mla_internal.h"
#include "mla_window.cuh"
#include "pair_ptx.cuh"
#include "ptx_sm100.cuh"

namespace mla {

using namespace ptx;

namespace {

constexpr int kThreads = 512;
constexpr int kNumProducers = 3;
constexpr int kMmaWarp = 1;
constexpr int kSoftmaxWarp0 = 4;
constexpr int kNumSoftmaxThreads = 256;
constexpr int kPrepWarp0 = 12;
constexpr int kNumPrepThreads = 128;
constexpr int kStages = 5;
constexpr int kBoxBytes = 8192;       // 64 rows x 128 bytes, 128-byte swizzle
constexpr int kStageBytes = 2 * kBoxBytes;
constexpr int kCodeChunks = 4;        // 512 codes / 128
constexpr int kChunks = kCodeChunks + 1;  // and the rotary one
constexpr int kSmemQ = 0;             // box 2c: q_hi of chunk c, box 2c + 1: q_lo
constexpr int kSmemP = kSmemQ + 2 * kChunks * kBoxBytes;  // P_hi (2 boxes of 128 keys), P_lo
constexpr int kSmemRing = kSmemP + 4 * kBoxBytes;
constexpr int kSmemRot = kSmemRing + kStages * kStageBytes;  // rotary keys' terms of this CTA's 128 keys
constexpr int kSmemTab = kSmemRot + kStageBytes;             // two tables of 2 x 256 floats
constexpr int kTabBytes = 2 * kTileKeys * 4;
constexpr int kSmemDyn = kSmemTab + 2 * kTabBytes;
constexpr int kEpiRoundBytes = 4 * kBoxBytes;
static_assert(4 * kEpiRoundBytes <= kSmemRot, "the last epilogue's staging stays inside Q, P and the ring");
// setmaxnreg split: warps 0-3, 4-11, 12-15 draw on the 512 x 128 registers of the launch
constexpr int kRegsIssue = 88, kRegsPrep = 88, kRegsSoftmax = 168;
static_assert(128 * (kRegsIssue + kRegsPrep) + 256 * kRegsSoftmax == kThreads * 128, "register split");
constexpr uint32_t kTmemO = 0, kTmemS0 = 256, kTmemCols = 512;
// The largest P of a tile is 2^kHeadroom where a unit is taken and stays in
// [2^(kHeadroom - kFall), 2^(kHeadroom + kRise)) = [2^6, 2^8.5) while it is kept: below e4m3's
// 448, and as far above e5m2's smallest steps as that allows.  O is rescaled the more often, which
// costs little: 269.4 us (192 sequences) against 268.1 with the unit at 2^6 in [2^2, 2^8.5), and
// 269.1 against 267.9 where every other tile's scales are 2^-12 of the others', so that each
// tile takes a new unit.
constexpr float kHeadroom = 8.0f, kRise = 0.5f, kFall = 2.0f;
// The unit falls at most this far below the row's largest: what a tile below that adds is not
// worth its exponent (2^-40 a key), and O stays far from fp32's range.
constexpr float kUnitFloor = 40.0f;
// Scales below this count as it: a row of zeros (scale 0) still weighs 2^x in the
// normaliser, and 2^x is kept in units of the largest x + log2 s.
constexpr float kMinScale = 0x1p-100f;
constexpr int kMaxUp = 100;  // largest power of two of a query row
constexpr uint32_t kIdescQK = make_idesc_e4m3(128, 256, false, false);
constexpr uint32_t kIdescPV = make_idesc_e4m3(128, 256, false, true);
constexpr uint32_t kLoA = kIdescAE5M2, kLoB = kIdescBE5M2;  // the operand is of low terms
constexpr int kBarSoftmax = 1, kBarPrep = 2;
constexpr uint64_t kDrainWaitNs = 100000000ull;  // bound on the post-abort wait for tensor-core work
constexpr uint64_t kQuiesceNs = 500000ull;       // post-abort wait for TMA loads in flight

struct Params {
  CUtensorMap tm_rows;  // packed rows as bytes [num_blocks][64][656], box {128, 64, 1}, SW128
  CUtensorMap tm_qn;    // q_nope as [units * M][512] bf16, box {64, 64}, SW128
  CUtensorMap tm_qp;    // q_pe as [units * M][64] bf16, box {64, 64}, SW128
  CUtensorMap tm_out;   // out as [units][M][512] bf16, box {64, 64, 1}, SW128 (TMA store)
  CUtensorMap tm_part;  // partial outputs as [slots][M][512] fp32, box {32, 64, 1}, SW128
  const uint8_t* rows;
  const int32_t* block_table;
  const int32_t* seqlens;
  const int32_t* q_lens;
  const int32_t* meta;
  __nv_bfloat16* out;
  float* lse;
  float* part_lse;
  int32_t* status;
  int64_t num_blocks;
  uint64_t timeout_ns;
  int max_blocks;
  int B, rep, M;  // units (tokens), tokens a sequence, rows a unit (heads)
  int window, sinks;
  float scale_log2;
  int inject_stall;
};

struct __align__(8) Ctrl {
  uint64_t full[kStages];   // leader: stage landed in both CTAs (count 1 + tx of both)
  uint64_t empty[kStages];  // both: stage consumed by the MMAs (commit)
  uint64_t q_full;          // leader: both CTAs' query terms written (count 2)
  uint64_t q_empty;         // both: last QK of the piece done (commit)
  uint64_t q_raw;           // this CTA's query rows landed as bf16 (count 1 + tx)
  uint64_t k_raw;           // this CTA's rotary keys landed as bf16 (count 1 + tx)
  uint64_t k_full;          // leader: both CTAs' rotary keys written (count 2)
  uint64_t k_empty;         // both: rotary QK of the tile done (commit)
  uint64_t sc_full[2];      // scale table of a tile written (count 1)
  uint64_t sc_empty[2];     // scale table of a tile used by the softmax (count 1)
  uint64_t s_full[2];       // both: S buffer written (commit)
  uint64_t p_full;          // leader: P written in both CTAs (count 2)
  uint64_t p_free;          // both: PV done (commit)
  uint64_t o_free;          // leader: O read out by both CTAs (count 2)
  uint64_t drain;           // both: every tensor-core op issued before an abort completed (commit)
  uint64_t never;           // nothing arrives: the injected stall waits on it
  uint32_t tmem_base;
  volatile int abort;
  volatile int peer_abort;  // written by the peer CTA at teardown
  float red_max[2][4][64];
  float red_sum[4][64];
  // 2^-j of the rows of piece k at k & 3.  Piece k + 4's are written after at least three
  // later tiles' tables, the second of which waited for the softmax of piece k's last tile.
  float row_scale[4][64];
  int bad_piece;
  int block_ids[kNumProducers][128];
};
constexpr int kIdRing = 128;

struct Piece {
  int b, k_lo, k_hi, split, n;
  WindowBlocks w;
};

// Keys in the visible prefix of unit u (token u % rep of sequence u / rep), -1: invalid.
__device__ __forceinline__ int unit_len(const Params& p, int u) {
  const int r = u / p.rep;
  const int n = p.seqlens[r];
  if ((int64_t)n > (int64_t)p.max_blocks * kBlockSize) return -1;
  return token_seq_len(n, p.q_lens ? p.q_lens[r] : p.rep, u - r * p.rep, p.rep, 1);
}
__device__ __forceinline__ int unit_blocks(const Params& p, int n) {
  return n < 0 ? -1 : window_blocks(n, p.window, p.sinks).count;
}
__device__ __forceinline__ const int32_t* unit_table(const Params& p, int u) {
  return p.block_table + (int64_t)(u / p.rep) * p.max_blocks;
}

// Walks the pieces of one partition; units with an invalid length, or a block count in the
// metadata that is not the one their length needs, are skipped by every role alike (an idle
// warp writes their NaN rows).
struct Walker {
  const Params* p;
  int cb, ck, be, ke;
  const int32_t* nblk;
  const int32_t* first_part;
  int part;
  __device__ Walker(const Params& prm, int part_) : p(&prm), part(part_) {
    const int32_t* m = prm.meta;
    cb = m[off_part_start() + 2 * part];
    ck = m[off_part_start() + 2 * part + 1];
    be = m[off_part_end() + 2 * part];
    ke = m[off_part_end() + 2 * part + 1];
    nblk = m + off_nblk();
    first_part = m + off_first_part(prm.B);
  }
  __device__ bool next(Piece& pc) {
    if (cb < 0) cb = p->B;  // malformed start: no pieces
    while (cb < p->B && (cb < be || (cb == be && ck < ke))) {
      const int nb = nblk[cb];
      const int hi = min((cb == be) ? ke : nb, nb);
      const int b = cb, lo = max(ck, 0);
      cb += 1;
      ck = 0;
      if (lo >= hi) continue;
      const int n = unit_len(*p, b);
      if (unit_blocks(*p, n) != nb) continue;
      pc.b = b;
      pc.k_lo = lo;
      pc.k_hi = hi;
      pc.split = part - first_part[b];
      pc.n = n;
      pc.w = window_blocks(n, p->window, p->sinks);
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ int num_tiles(const Piece& pc) {
  return (pc.k_hi - pc.k_lo + kBlocksPerTile - 1) / kBlocksPerTile;
}
__device__ __forceinline__ int blocks_in_tile(const Piece& pc, int t) {
  const int r = pc.k_hi - pc.k_lo - t * kBlocksPerTile;
  return r < kBlocksPerTile ? r : kBlocksPerTile;
}
// visible rows [lo, hi) of block kb of tile t
__device__ __forceinline__ void rows_in_block(const Piece& pc, int t, int kb, int* lo, int* hi) {
  window_rows(pc.w, pc.n, pc.k_lo + t * kBlocksPerTile + kb, lo, hi);
}
__device__ __forceinline__ void set_status(const Params& p, int bits) {
  if (p.status) atomicOr(p.status, bits);
}
__device__ __forceinline__ bool valid_id(const Params& p, int32_t id) { return id >= 0 && (int64_t)id < p.num_blocks; }
// invalid ids read block 0; the epilogue turns the piece's rows into NaN
__device__ __forceinline__ int clamp_block_id(const Params& p, int32_t id) {
  if (valid_id(p, id)) return id;
  set_status(p, kErrBlockId);
  return 0;
}

// Bounded wait that also gives up when another role of this CTA aborted.
__device__ __forceinline__ bool wait_bar(Ctrl* c, const Params& p, uint32_t bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t deadline = globaltimer_ns() + p.timeout_ns;
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i) {
      if (mbar_try_wait(bar, parity)) return true;
    }
    if (c->abort) return false;
    if (globaltimer_ns() > deadline) {
      c->abort = 1;
      set_status(p, kErrTimeout);
      return false;
    }
  }
}

// Four values as two terms each: hi the value rounded to e4m3, lo what hi left, read back off
// the codes, rounded to e5m2.
__device__ __forceinline__ void split2(float a, float b, uint16_t& hi, uint16_t& lo) {
  asm("{\n\t.reg .b32 h;\n\t.reg .b16 x, y, m;\n\t.reg .f32 p, q;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 %0, %3, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 h, %0;\n\t"
      "mov.b32 {x, y}, h;\n\t"
      "mov.b16 m, 0xBC00;\n\t"  // -1
      "fma.rn.f32.f16 p, x, m, %2;\n\t"
      "fma.rn.f32.f16 q, y, m, %3;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 %1, q, p;\n\t}"
      : "=&h"(hi), "=&h"(lo)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ void split4(float a, float b, float c, float d, uint32_t& hi, uint32_t& lo) {
  uint16_t h0, l0, h1, l1;
  split2(a, b, h0, l0);
  split2(c, d, h1, l1);
  hi = h0 | ((uint32_t)h1 << 16);
  lo = l0 | ((uint32_t)l1 << 16);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t* w) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t w;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(addr) : "memory");
  return w;
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"((uint16_t)v) : "memory");
}

// ===========================================================================
// the kernel
// ===========================================================================
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    window_fp8_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Ctrl ctrl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + kSmemQ, sP = sbase + kSmemP, sRing = sbase + kSmemRing, sRot = sbase + kSmemRot;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = (rank == 0);
  const int part = blockIdx.x >> 1;

  // ---- setup (reads no input: it overlaps the previous kernel's tail) --------------
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&ctrl.full[s]), 1);
      mbar_init(smem_u32(&ctrl.empty[s]), 1);
    }
    mbar_init(smem_u32(&ctrl.q_full), 2);
    mbar_init(smem_u32(&ctrl.q_empty), 1);
    mbar_init(smem_u32(&ctrl.q_raw), 1);
    mbar_init(smem_u32(&ctrl.k_raw), 1);
    mbar_init(smem_u32(&ctrl.k_full), 2);
    mbar_init(smem_u32(&ctrl.k_empty), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&ctrl.sc_full[s]), 1);
      mbar_init(smem_u32(&ctrl.sc_empty[s]), 1);
      mbar_init(smem_u32(&ctrl.s_full[s]), 1);
    }
    mbar_init(smem_u32(&ctrl.p_full), 2);
    mbar_init(smem_u32(&ctrl.p_free), 1);
    mbar_init(smem_u32(&ctrl.o_free), 2);
    mbar_init(smem_u32(&ctrl.drain), 1);
    mbar_init(smem_u32(&ctrl.never), 1);
    ctrl.abort = 0;
    ctrl.peer_abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&ctrl.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&p.tm_rows);
    prefetch_tmap(&p.tm_qn);
    prefetch_tmap(&p.tm_qp);
    prefetch_tmap(&p.tm_out);
    prefetch_tmap(&p.tm_part);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = ctrl.tmem_base;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int P = p.meta[kHdrNumParts];
  const bool bad_meta = p.meta[kHdrMagic] != kMetaMagicWin || p.meta[kHdrB] != p.B || p.meta[kHdrSq] != 1 ||
                        p.meta[kHdrH] != p.M || p.meta[kHdrNumTiles] != 1 || P * 2 != (int)gridDim.x ||
                        p.meta[kHdrTokens] != p.rep || p.meta[kHdrTokCausal] != 1 ||
                        p.meta[kHdrWindow] != p.window || p.meta[kHdrSinks] != p.sinks;
  if (bad_meta && tid == 0 && blockIdx.x == 0) set_status(p, kErrMetadata);

  if (!bad_meta) {  // else every role skips; the CTA still joins the cluster barriers below
    // =======================================================================
    // producers: warps 0, 2, 3 own ring stages k % 3 == 0, 1, 2
    // =======================================================================
    if (warp == 0 || warp == 2 || warp == 3) {
      regs_dec<kRegsIssue>();
      const int pi = (warp == 0) ? 0 : warp - 1;
      int32_t* idwin = ctrl.block_ids[pi];
      Walker walk(p, part);
      uint32_t it = 0;
      bool ok = true;
      auto mine = [&]() { return (int)(it % kNumProducers) == pi; };
      auto acquire = [&](uint32_t& slot) -> bool {
        slot = it % kStages;
        const uint32_t use = it / kStages;
        return use == 0 || wait_bar(&ctrl, p, smem_u32(&ctrl.empty[slot]), (use - 1) & 1);
      };
      // block ids of the current piece: as in mla_decode_kernel.cu, 32 at a time one chunk
      // ahead into this warp's window
      Piece cur{};
      int cur_base = 0, id_pending = 0, id_chunks = 0;
      const int32_t* bt = nullptr;
      auto fetch_id = [&](const Piece& pc, const int32_t* table, int i) -> int {
        return (i < pc.k_hi - pc.k_lo) ? clamp_block_id(p, table[window_block(pc.w, pc.k_lo + i)]) : 0;
      };
      auto ensure_ids = [&](int last) {
        while (last >= 32 * id_chunks) {
          idwin[(cur_base + 32 * id_chunks + lane) % kIdRing] = id_pending;
          ++id_chunks;
          id_pending = fetch_id(cur, bt, 32 * id_chunks + lane);
          __syncwarp();
        }
      };
      // QK of tile t: this CTA's (up to) two blocks, 128 code columns a stage.  A CTA
      // without keys in the tile loads its first block (those columns of S are masked), so
      // that every stage carries bytes of both CTAs.
      auto issue_qk = [&](int t) {
        const int nb = blocks_in_tile(cur, t);
        const int own0 = 2 * (int)rank;
        ensure_ids(t * kBlocksPerTile + nb - 1);
        const int own = min(max(nb - own0, 0), 2);
        const int nbox = own > 0 ? own : 1;
        const int first = own > 0 ? own0 + (lane & 1) : 0;
        const int my_id = idwin[(cur_base + t * kBlocksPerTile + first) % kIdRing];
        const int boxes = (nb < 2 ? nb : 2) + (nb > 2 ? nb - 2 : 1);
        for (int c = 0; c < kCodeChunks && ok; ++c) {
          if (!mine()) {
            ++it;
            continue;
          }
          uint32_t slot;
          ok = __shfl_sync(0xffffffffu, acquire(slot), 0);
          if (!ok) break;
          const uint32_t fb = smem_u32(&ctrl.full[slot]);
          expect_tx_if(lane == 0 && leader, fb, kBoxBytes * boxes);
          tma_load_3d_cg2_if(lane < nbox, sRing + slot * kStageBytes + (lane & 1) * kBoxBytes, &p.tm_rows,
                             mapa_shared(fb, 0), 128 * c, 0, my_id);
          ++it;
        }
      };
      // PV of tile t of piece pc: two blocks a stage.  A block whose last or first rows are
      // hidden is loaded from row hi - 64 or lo on; what lies outside it is zero-filled.
      auto issue_pv = [&](const Piece& pc, int base, int t) {
        const int nb = blocks_in_tile(pc, t);
        for (int h = 0; h < 2 && ok; ++h) {
          for (int kb0 = 0; kb0 < nb && ok; kb0 += 2) {
            if (!mine()) {
              ++it;
              continue;
            }
            const int nbox = min(nb - kb0, 2), kb = kb0 + min(lane & 1, nbox - 1);
            const int id = idwin[(base + t * kBlocksPerTile + kb) % kIdRing];
            int lo, hi;
            rows_in_block(pc, t, kb, &lo, &hi);
            uint32_t slot;
            ok = __shfl_sync(0xffffffffu, acquire(slot), 0);
            if (!ok) break;
            const uint32_t fb = smem_u32(&ctrl.full[slot]);
            expect_tx_if(lane == 0 && leader, fb, 2 * kBoxBytes * nbox);
            tma_load_3d_cg2_if(lane < nbox, sRing + slot * kStageBytes + (lane & 1) * kBoxBytes, &p.tm_rows,
                               mapa_shared(fb, 0), 256 * h + 128 * (int)rank, hi < kBlockSize ? hi - kBlockSize : lo,
                               id);
            ++it;
          }
        }
      };
      // one ring order for the whole partition: QK of each tile, then PV of the tile before
      Piece nxt{}, prv{};
      int prv_base = 0, prv_t = -1;
      bool have = walk.next(cur);
      bool have_nxt = have && walk.next(nxt);
      if (have) {
        bt = unit_table(p, cur.b);
        id_pending = fetch_id(cur, bt, lane);
      }
      while (ok && have) {
        id_chunks = 0;
        const int nt = num_tiles(cur);
        int id_next = 0;
        for (int t = 0; t < nt && ok; ++t) {
          if (t == nt - 1 && have_nxt) id_next = fetch_id(nxt, unit_table(p, nxt.b), lane);
          issue_qk(t);
          if (ok && prv_t >= 0) issue_pv(prv, prv_base, prv_t);
          prv = cur;
          prv_base = cur_base;
          prv_t = t;
        }
        cur_base = (cur_base + 32 * id_chunks) % kIdRing;
        have = have_nxt;
        if (have) {
          cur = nxt;
          bt = unit_table(p, cur.b);
          id_pending = id_next;
          have_nxt = walk.next(nxt);
        }
      }
      if (ok && prv_t >= 0) issue_pv(prv, prv_base, prv_t);
    }
    // =======================================================================
    // MMA issuer (leader CTA only)
    // =======================================================================
    else if (warp == kMmaWarp && leader) {
      regs_dec<kRegsIssue>();
      Walker walk(p, part);
      uint32_t slot = 0, phase = 0, qk_count = 0, pv_count = 0;
      int npieces = 0;
      bool ok = true;
      const bool elected = elect_one();
      // start fields hold address >> 4; a K step of 32 codes is 32 bytes of a K-major row,
      // of 32 keys 32 rows of 128 bytes
      constexpr uint64_t kBoxD = kBoxBytes >> 4, kStageD = kStageBytes >> 4;
      const uint64_t dq0 = make_smem_desc(sQ, 16, 1024, kSwizzle128B);
      const uint64_t dp0 = make_smem_desc(sP, 16, 1024, kSwizzle128B);
      const uint64_t dk0 = make_smem_desc(sRing, 16, 1024, kSwizzle128B);
      const uint64_t dr0 = make_smem_desc(sRot, 16, 1024, kSwizzle128B);
      const uint64_t dv0 = make_smem_desc(sRing, kBoxBytes, 1024, kSwizzle128B);
      auto next_stage = [&]() {
        if (++slot == kStages) {
          slot = 0;
          phase ^= 1;
        }
      };
      auto mma_chunk = [&](uint32_t d, int c, uint64_t b0) {
        const uint64_t a0 = dq0 + 2 * c * kBoxD;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t b = (c == kCodeChunks && ks >= 2) ? kLoB : 0u;
          umma8_2sm_if(elected, d, a0 + 2 * ks, b0 + 2 * ks, kIdescQK | b, (c | ks) != 0);
          umma8_2sm_if(elected, d, a0 + kBoxD + 2 * ks, b0 + 2 * ks, kIdescQK | kLoA | b, 1);
        }
      };
      auto mma_qk = [&](int nt, int t) {
        const uint32_t buf = qk_count & 1;
        const uint32_t d = tmem + kTmemS0 + 128 * buf;
        for (int c = 0; c < kCodeChunks && ok; ++c) {
          ok = wait_bar(&ctrl, p, smem_u32(&ctrl.full[slot]), phase);
          if (!ok) break;
          mma_chunk(d, c, dk0 + slot * kStageD);
          commit_2sm_if(elected, smem_u32(&ctrl.empty[slot]));
          next_stage();
        }
        if (ok) ok = wait_bar(&ctrl, p, smem_u32(&ctrl.k_full), qk_count & 1);
        if (ok) {
          tc_fence_after();
          mma_chunk(d, kCodeChunks, dr0);
          commit_2sm_if(elected, smem_u32(&ctrl.k_empty));
          commit_2sm_if(elected, smem_u32(&ctrl.s_full[buf]));
          if (t == nt - 1) commit_2sm_if(elected, smem_u32(&ctrl.q_empty));
        }
        ++qk_count;
      };
      auto mma_pv = [&](const Piece& pc, int piece_idx, int t) {
        if (!ok) return;
        ok = wait_bar(&ctrl, p, smem_u32(&ctrl.p_full), pv_count & 1);
        if (ok && t == 0 && piece_idx > 0) ok = wait_bar(&ctrl, p, smem_u32(&ctrl.o_free), (piece_idx - 1) & 1);
        if (!ok) return;
        tc_fence_after();
        const int nb = blocks_in_tile(pc, t);
        for (int h = 0; h < 2 && ok; ++h) {
          for (int kb0 = 0; kb0 < nb && ok; kb0 += 2) {
            ok = wait_bar(&ctrl, p, smem_u32(&ctrl.full[slot]), phase);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int kb = kb0 + i;
              if (kb >= nb) break;
              // keys in rows [64 - hi, 64) or [0, 64 - lo): skip a step that holds none
              int lo, hi;
              rows_in_block(pc, t, kb, &lo, &hi);
              const int ks0 = (kBlockSize - hi) >> 5, ks1 = (kBlockSize - lo + 31) >> 5;
              const bool first = (t == 0 && kb == 0);
              const uint64_t a0 = dp0 + (kb >> 1) * kBoxD + 4 * (kb & 1);
              const uint64_t b0 = dv0 + slot * kStageD + i * kBoxD;
#pragma unroll
              for (int ks = 0; ks < 2; ++ks) {
                const bool on = elected && ks >= ks0 && ks < ks1;
                umma8_2sm_if(on, tmem + kTmemO + 128 * h, a0 + 2 * ks, b0 + 256 * ks, kIdescPV, !(first && ks == ks0));
                umma8_2sm_if(on, tmem + kTmemO + 128 * h, a0 + 2 * kBoxD + 2 * ks, b0 + 256 * ks, kIdescPV | kLoA, 1);
              }
            }
            commit_2sm_if(elected, smem_u32(&ctrl.empty[slot]));
            next_stage();
          }
        }
        if (ok) commit_2sm_if(elected, smem_u32(&ctrl.p_free));
        ++pv_count;
      };
      Piece cur, prv{};
      int prv_t = -1, prv_idx = 0;
      if (p.inject_stall) ok = wait_bar(&ctrl, p, smem_u32(&ctrl.never), 0);
      while (ok && walk.next(cur)) {
        ok = wait_bar(&ctrl, p, smem_u32(&ctrl.q_full), npieces & 1);
        tc_fence_after();
        const int nt = num_tiles(cur);
        for (int t = 0; t < nt && ok; ++t) {
          mma_qk(nt, t);
          if (prv_t >= 0) mma_pv(prv, prv_idx, prv_t);
          prv = cur;
          prv_t = t;
          prv_idx = npieces;
        }
        ++npieces;
      }
      if (prv_t >= 0) mma_pv(prv, prv_idx, prv_t);
    }
    // =======================================================================
    // softmax / correction / epilogue
    // =======================================================================
    else if (warp >= kSoftmaxWarp0 && warp < kSoftmaxWarp0 + 8) {
      regs_inc<kRegsSoftmax>();
      const int st = tid - kSoftmaxWarp0 * 32;  // 0..255
      const int g = st >> 7;                    // keys 64g.. of each half; O half g
      const int L = st & 127;                   // TMEM lane
      const int quad = (warp & 3);
      const int m = L & 63;    // row within the CTA
      const int hk = L >> 6;   // key half
      const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
      const int y0 = kRowsPerCta * (int)rank;
      const int grow = y0 + m;
      const bool row_valid = grow < p.M;
      const uint32_t p_full_l = mapa_shared(smem_u32(&ctrl.p_full), 0);
      const uint32_t o_free_l = mapa_shared(smem_u32(&ctrl.o_free), 0);
      Walker walk(p, part);
      Piece pc;
      uint32_t qk_count = 0, pv_count = 0;
      int npieces = 0;
      // ok: this thread's waits all completed; go: the same for all 256 threads, refreshed
      // only by named barriers that AND ok
      bool ok = true, go = true;
      bool pend = false, pend_direct = true;
      int pend_b = 0, pend_slot = 0;
      float pend_sc = 0.f, pend_lse = 0.f;
      auto epilogue = [&](bool drain) {
        const uint32_t to = tmem + kTmemO + 128 * g + lane_off;
        // per round every thread writes 128 bytes of its row (64 bf16 or 32 fp32 columns)
        // into box 2g + hk, laid out [64 rows][128 B] with the 128-byte swizzle, and one
        // thread stores the four boxes; rows past M are clipped by the tensor map
        const int rounds = pend_direct ? 2 : 4;
        auto stage = [&](int r) -> uint32_t { return drain ? sQ + r * kEpiRoundBytes : sP; };
        auto store_round = [&](int r) {
#pragma unroll
          for (int bx = 0; bx < 4; ++bx) {
            const int gg = bx >> 1, hh = bx & 1;
            if (pend_direct)
              tma_store_3d(&p.tm_out, stage(r) + bx * kBoxBytes, 256 * gg + 128 * hh + 64 * r, y0, pend_b);
            else
              tma_store_3d(&p.tm_part, stage(r) + bx * kBoxBytes, 256 * gg + 128 * hh + 32 * r, y0, pend_slot);
          }
        };
#pragma unroll 1
        for (int r = 0; r < rounds; ++r) {
          const uint32_t srow = stage(r) + (2 * g + hk) * kBoxBytes + m * 128;
          uint32_t w[32];
          if (pend_direct) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t o[32];
              tmem_ld32_wait(to + 64 * r + 32 * hf, o);
#pragma unroll
              for (int k = 0; k < 16; ++k)
                w[16 * hf + k] =
                    pack_bf16x2(__uint_as_float(o[2 * k]) * pend_sc, __uint_as_float(o[2 * k + 1]) * pend_sc);
            }
          } else {
            tmem_ld32_wait(to + 32 * r, w);
#pragma unroll
            for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * pend_sc);
          }
          if (r > 0 && !drain) named_bar_sync(kBarSoftmax, kNumSoftmaxThreads);  // previous round's boxes were read
#pragma unroll
          for (int q = 0; q < 8; ++q)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(srow + ((q ^ (m & 7)) << 4)),
                         "r"(w[4 * q]), "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                         : "memory");
          fence_proxy_async_smem();
          if (drain) continue;
          if (r == 0) {
            go = named_bar_and(kBarSoftmax, kNumSoftmaxThreads, ok);
            if (!go) return;
          } else {
            named_bar_sync(kBarSoftmax, kNumSoftmaxThreads);
          }
          if (st == 0 && y0 < p.M) {  // a CTA whose 64 rows all lie past M stores nothing
            store_round(r);
            bulk_commit();
            bulk_wait_read_all();
          }
        }
        if (drain) {
          go = named_bar_and(kBarSoftmax, kNumSoftmaxThreads, ok);
          if (!go) return;
          if (st == 0 && y0 < p.M) {  // completion is awaited at teardown
            for (int r = 0; r < rounds; ++r) store_round(r);
            bulk_commit();
          }
        }
        if (row_valid && hk == 0 && g == 0) {
          if (pend_direct)
            p.lse[(int64_t)pend_b * p.M + grow] = pend_lse;
          else
            p.part_lse[(int64_t)pend_slot * p.M + grow] = pend_lse;
        }
        // every O read and the staging reads of the last round are done
        tc_fence_before();
        named_bar_sync(kBarSoftmax, kNumSoftmaxThreads);
        if (st == 0) {
          if (leader)
            mbar_arrive(smem_u32(&ctrl.o_free));
          else
            mbar_arrive_remote(o_free_l);
        }
        pend = false;
      };
      while (go && walk.next(pc)) {
        const int nt = num_tiles(pc);
        // m_used: the unit of P and O, m_l: that of l, the largest m_used so far
        float m_used = -INFINITY, m_l = -INFINITY, l_part = 0.f, rs = 0.f;
        const int nsplit = p.meta[off_num_splits(p.B) + pc.b];
        const int split_base = p.meta[off_split_prefix(p.B) + pc.b];
        int bad_ids = 0;
        {
          const int32_t* bt = unit_table(p, pc.b);
          for (int k = pc.k_lo + st; k < pc.k_hi; k += kNumSoftmaxThreads)
            bad_ids |= !valid_id(p, bt[window_block(pc.w, k)]);
        }
        for (int t = 0; t < nt && go; ++t) {
          const uint32_t buf = qk_count & 1;
          ok = wait_bar(&ctrl, p, smem_u32(&ctrl.sc_full[buf]), (qk_count >> 1) & 1) && ok;
          ok = wait_bar(&ctrl, p, smem_u32(&ctrl.s_full[buf]), (qk_count >> 1) & 1) && ok;
          // (at least the smallest normal number: times a hidden key's -inf it stays -inf)
          if (t == 0) {
            rs = ctrl.row_scale[npieces & 3][m] * p.scale_log2;
            if (rs < 0x1p-126f) rs = 0x1p-126f;
          }
          tc_fence_after();
          const uint32_t ts = tmem + kTmemS0 + 128 * buf + lane_off + 64 * g;
          // of this thread's block, keys [c0, c0 + cnt) are visible
          int c0 = 0, hi = kBlockSize, cnt = 0;
          if (2 * hk + g < blocks_in_tile(pc, t)) {
            rows_in_block(pc, t, 2 * hk + g, &c0, &hi);
            if (row_valid) cnt = hi - c0;
          }
          auto seen = [&](int c) -> bool { return (uint32_t)(c - c0) < (uint32_t)cnt; };
          const bool full = __all_sync(0xffffffffu, cnt == kBlockSize);
          // x = S * s * rs with the key's scale s and rs = 2^-j * scale * log2 e; the maximum is
          // of z = x + log2 s.  The table holds s and log2 s.
          const float4* tab = reinterpret_cast<const float4*>(smem + kSmemTab + buf * kTabBytes) + 16 * (2 * hk + g);
          // hidden keys of a group that starts at key c score -inf: their weight is 2^-inf = 0
          auto hide = [&](uint32_t* s, int c, int count) {
            if (!full) {
#pragma unroll
              for (int i = 0; i < count; ++i)
                if (!seen(c + i)) s[i] = 0xff800000u;
            }
          };
          auto score = [](uint32_t s) -> float { return __uint_as_float(s); };
          float mx0 = -INFINITY, mx1 = -INFINITY;
          const uint64_t rs2 = pack_f32x2(rs, rs);
#pragma unroll 1
          for (int c = 0; c < 64; c += 16) {
            uint32_t s[16];
            tmem_ld16_wait(ts + c, s);
            hide(s, c, 16);
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 f = tab[(c + i) >> 2], lg = tab[64 + ((c + i) >> 2)];
              const uint64_t y01 = mul2(pack_f32x2(score(s[i]), score(s[i + 1])), pack_f32x2(f.x, f.y));
              const uint64_t y23 = mul2(pack_f32x2(score(s[i + 2]), score(s[i + 3])), pack_f32x2(f.z, f.w));
              float z0, z1, z2, z3;
              unpack_f32x2(fma2(y01, rs2, pack_f32x2(lg.x, lg.y)), z0, z1);
              unpack_f32x2(fma2(y23, rs2, pack_f32x2(lg.z, lg.w)), z2, z3);
              mx0 = max3(mx0, z0, z1);
              mx1 = max3(mx1, z2, z3);
            }
          }
          ctrl.red_max[buf][2 * hk + g][m] = fmaxf(mx0, mx1);
          go = named_bar_and(kBarSoftmax, kNumSoftmaxThreads, ok);
          if (!go) break;
          const float top = fmaxf(fmaxf(ctrl.red_max[buf][0][m], ctrl.red_max[buf][1][m]),
                                  fmaxf(ctrl.red_max[buf][2][m], ctrl.red_max[buf][3][m]));
          // the unit this tile's largest weight asks for
          const float want = fmaxf(top, m_l - kUnitFloor);
          const bool rescale = want > m_used + kRise || want < m_used - kFall;
          float alpha = 1.f;
          if (rescale) {
            alpha = (m_used == -INFINITY) ? 0.f : fast_exp2(m_used - want);
            m_used = want;
            if (m_used > m_l) {
              l_part *= (m_l == -INFINITY) ? 0.f : fast_exp2(m_l - m_used);
              m_l = m_used;
            }
          }
          const float beta = (m_used == m_l) ? 1.f : fast_exp2(m_used - m_l);
          const float nref = (m_used == -INFINITY) ? 0.f : kHeadroom - m_used;
          // weights: P of keys 0..31 in pa, of 32..63 in pb (8 words of hi, 8 of lo terms)
          uint64_t l01 = pack_f32x2(0.f, 0.f), l23 = l01;
          const uint64_t nref2 = pack_f32x2(nref, nref);
          uint32_t pa[16], pb[16] = {};
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
#pragma unroll
            for (int q = 0; q < 16; ++q) pa[q] = pb[q];
            uint32_t s[32];
            tmem_ld32_wait(ts + c, s);
            hide(s, c, 32);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float4 f = tab[(c >> 2) + q];
              const uint64_t f01 = pack_f32x2(f.x, f.y), f23 = pack_f32x2(f.z, f.w);
              float e0, e1, e2, e3;
              unpack_f32x2(fma2(mul2(pack_f32x2(score(s[4 * q]), score(s[4 * q + 1])), f01), rs2, nref2), e0, e1);
              unpack_f32x2(fma2(mul2(pack_f32x2(score(s[4 * q + 2]), score(s[4 * q + 3])), f23), rs2, nref2), e2, e3);
              const uint64_t e01 = pack_f32x2(fast_exp2(e0), fast_exp2(e1));
              const uint64_t e23 = pack_f32x2(fast_exp2(e2), fast_exp2(e3));
              l01 = add2(l01, e01);
              l23 = add2(l23, e23);
              unpack_f32x2(mul2(e01, f01), e0, e1);
              unpack_f32x2(mul2(e23, f23), e2, e3);
              split4(e0, e1, e2, e3, pb[q], pb[8 + q]);
            }
          }
          {
            float l0, l1;
            unpack_f32x2(add2(l01, l23), l0, l1);
            l_part = fmaf(beta, l0 + l1, l_part);
          }
          // PV of the previous tile (possibly the previous piece's last) must be done before
          // P is overwritten, O is rescaled or the previous piece's O is read
          if (qk_count >= 1) {
            ok = wait_bar(&ctrl, p, smem_u32(&ctrl.p_free), pv_count & 1) && ok;
            ++pv_count;
            tc_fence_after();
            if (t == 0) {
              if (pend) {
                epilogue(false);
                if (!go) break;
              }
            } else if (__any_sync(0xffffffffu, rescale)) {
              const uint32_t to = tmem + kTmemO + 128 * g + lane_off;
#pragma unroll 1
              for (int c = 0; c < 128; c += 32) {
                uint32_t o[32];
                tmem_ld32_wait(to + c, o);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                asm volatile(
                    "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
                    "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
                    "%29, %30, %31, %32};" ::"r"(to + c),
                    "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]),
                    "r"(o[8]), "r"(o[9]), "r"(o[10]), "r"(o[11]), "r"(o[12]), "r"(o[13]), "r"(o[14]),
                    "r"(o[15]), "r"(o[16]), "r"(o[17]), "r"(o[18]), "r"(o[19]), "r"(o[20]), "r"(o[21]),
                    "r"(o[22]), "r"(o[23]), "r"(o[24]), "r"(o[25]), "r"(o[26]), "r"(o[27]), "r"(o[28]),
                    "r"(o[29]), "r"(o[30]), "r"(o[31])
                    : "memory");
              }
              tmem_wait_st();
            }
          }
          // P -> shared memory: K-major, box hk holds keys 128hk.. of all 64 rows, this thread's
          // 64 keys are granules 4g..4g+3 of its row (granule j at j ^ (m & 7)).  A block with
          // hidden rows has its keys where its V rows were loaded, 64 - hi further on or c0
          // further back: as a rotation, for the hidden keys' zeros belong where these leave.
          const uint32_t prow = sP + hk * kBoxBytes + m * 128;
          const int turn = hi < kBlockSize ? kBlockSize - hi : kBlockSize - c0;  // 64: none
          auto put = [&](const uint32_t (&w)[16], int c) {
            if (turn == kBlockSize) {  // warp-uniform
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t a = prow + (((4 * g + (c >> 4) + j) ^ (m & 7)) << 4);
                st_shared_v4(a, w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                st_shared_v4(a + 2 * kBoxBytes, w[8 + 4 * j], w[8 + 4 * j + 1], w[8 + 4 * j + 2], w[8 + 4 * j + 3]);
              }
            } else {
#pragma unroll
              for (int q = 0; q < 8; ++q) {
#pragma unroll 1
                for (int e = 0; e < 4; ++e) {
                  const int k = (c + 4 * q + e + turn) & 63;
                  const uint32_t a = prow + (((4 * g + (k >> 4)) ^ (m & 7)) << 4) + (k & 15);
                  st_shared_u8(a, w[q] >> (8 * e));
                  st_shared_u8(a + 2 * kBoxBytes, w[8 + q] >> (8 * e));
                }
              }
            }
          };
          put(pa, 0);
          put(pb, 32);
          fence_proxy_async_smem();
          tc_fence_before();
          named_bar_sync(kBarSoftmax, kNumSoftmaxThreads);
          if (st == 0) {
            if (leader)
              mbar_arrive(smem_u32(&ctrl.p_full));
            else
              mbar_arrive_remote(p_full_l);
            mbar_arrive(smem_u32(&ctrl.sc_empty[buf]));  // the table has been read
          }
          ++qk_count;
        }
        if (!go) break;
        ++npieces;
        // row sums and the block-id verdict, while the piece's last PV is still running
        ctrl.red_sum[2 * hk + g][m] = l_part;
        if (st == 0) ctrl.bad_piece = 0;
        named_bar_sync(kBarSoftmax, kNumSoftmaxThreads);
        if (bad_ids) ctrl.bad_piece = 1;
        const float l_row = ctrl.red_sum[0][m] + ctrl.red_sum[1][m] + ctrl.red_sum[2][m] + ctrl.red_sum[3][m];
        named_bar_sync(kBarSoftmax, kNumSoftmaxThreads);
        const bool bad = ctrl.bad_piece != 0;
        const float nanf_ = __int_as_float(0x7fc00000);
        // NaN scales make the row NaN; so does a NaN among the visible scores (l is NaN then)
        const float unit = (m_used == m_l) ? 1.f : fast_exp2(m_used - m_l);  // O's in l's
        pend_sc = (bad || l_row != l_row) ? nanf_ : ((l_row > 0.f) ? unit / l_row : 0.f);
        const float lse2 = m_l - kHeadroom + __log2f(l_row);
        pend_lse = (bad || l_row != l_row) ? nanf_ : ((l_row > 0.f) ? lse2 * 0.69314718055994531f : -INFINITY);
        pend_direct = (nsplit == 1);
        pend_b = pc.b;
        pend_slot = split_base + pc.split;
        pend = true;
      }
      go = named_bar_and(kBarSoftmax, kNumSoftmaxThreads, ok && go);
      if (go && pend) {
        ok = wait_bar(&ctrl, p, smem_u32(&ctrl.p_free), pv_count & 1) && ok;
        ++pv_count;
        tc_fence_after();
        epilogue(true);
      }
    }
    // =======================================================================
    // preparation
    // =======================================================================
    else if (warp >= kPrepWarp0) {
      regs_dec<kRegsPrep>();
      const int pt = tid - kPrepWarp0 * 32;  // 0..127
      const int pw = warp - kPrepWarp0;
      const uint32_t q_full_l = mapa_shared(smem_u32(&ctrl.q_full), 0);
      const uint32_t k_full_l = mapa_shared(smem_u32(&ctrl.k_full), 0);
      float* const tables = reinterpret_cast<float*>(smem + kSmemTab);
      bool ok = true, go = true;
      // makes this role's writes visible and joins its threads; false: a wait ran out
      auto publish = [&]() -> bool {
        fence_proxy_async_smem();
        go = named_bar_and(kBarPrep, kNumPrepThreads, ok);
        return go;
      };
      auto arrive = [&](uint64_t* bar, uint32_t leader_bar) {
        if (leader)
          mbar_arrive(smem_u32(bar));
        else
          mbar_arrive_remote(leader_bar);
      };
      // ---- query rows: they land as nine 64-column bf16 boxes and become terms in place.
      // A warp takes a row at a time (two rows in flight): lane l holds values 16l.. of
      // q_nope, whose hi and lo terms are granule l % 8 of boxes 2 (l / 8) and 2 (l / 8) + 1,
      // where values of the same row lay, and 2l.. of q_pe.
      constexpr int kQBytes = 9 * kBoxBytes;
      auto load_q = [&](int b) {  // by warp kPrepWarp0
        const int row = b * p.M + kRowsPerCta * (int)rank;
        const uint32_t bar = smem_u32(&ctrl.q_raw);
        expect_tx_if(lane == 0, bar, kQBytes);
        __syncwarp();
        tma_load_2d_if(lane < 9, sQ + (lane < 9 ? lane : 0) * kBoxBytes,
                       lane < 8 ? (const void*)&p.tm_qn : (const void*)&p.tm_qp, bar, lane < 8 ? 64 * lane : 0, row);
      };
      auto split_rows = [&](int piece) {
#pragma unroll 1
        for (int m0 = 16 * pw; m0 < 16 * pw + 16; m0 += 2) {
          uint32_t w[2][8], wr[2];
          float up[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int m = m0 + i;
            const uint32_t a = sQ + (lane >> 2) * kBoxBytes + m * 128;
            ld_shared_v4(a + (((2 * (lane & 3)) ^ (m & 7)) << 4), &w[i][0]);
            ld_shared_v4(a + (((2 * (lane & 3) + 1) ^ (m & 7)) << 4), &w[i][4]);
            wr[i] = ld_shared_u32(sQ + 8 * kBoxBytes + m * 128 + (((lane >> 2) ^ (m & 7)) << 4) + 4 * (lane & 3));
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t mx = wr[i] & 0x7fff7fffu;  // magnitudes order as integers
#pragma unroll
            for (int k = 0; k < 8; ++k) mx = __vmaxu2(mx, w[i][k] & 0x7fff7fffu);
            mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
            const int E = (int)(mx >> 7);  // biased exponent of the row's largest value
            const int j = min(134 - E, kMaxUp);
            up[i] = __int_as_float((j + 127) << 23);
            if (lane == 0)
              ctrl.row_scale[piece & 3][m0 + i] =
                  E == 255 ? __int_as_float(0x7fc00000) : __int_as_float((127 - j) << 23);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int m = m0 + i;
            const float u = up[i];
            uint32_t h[4], l[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              split4(bf_lo(w[i][2 * k]) * u, bf_hi(w[i][2 * k]) * u, bf_lo(w[i][2 * k + 1]) * u,
                     bf_hi(w[i][2 * k + 1]) * u, h[k], l[k]);
            const uint32_t a = sQ + 2 * (lane >> 3) * kBoxBytes + m * 128 + (((lane & 7) ^ (m & 7)) << 4);
            st_shared_v4(a, h[0], h[1], h[2], h[3]);
            st_shared_v4(a + kBoxBytes, l[0], l[1], l[2], l[3]);
            // rotary chunk: the 64 terms twice, against [k'_hi | k'_lo]
            uint32_t rh, rl;
            split4(bf_lo(wr[i]) * u, bf_hi(wr[i]) * u, 0.f, 0.f, rh, rl);
            const uint32_t row = sQ + 2 * kCodeChunks * kBoxBytes + m * 128 + 2 * (lane & 7);
            const uint32_t g0 = ((lane >> 3) ^ (m & 7)) << 4, g1 = ((4 + (lane >> 3)) ^ (m & 7)) << 4;
            st_shared_u16(row + g0, rh);
            st_shared_u16(row + g1, rh);
            st_shared_u16(row + kBoxBytes + g0, rl);
            st_shared_u16(row + kBoxBytes + g1, rl);
          }
        }
      };
      // ---- a tile: thread pt holds the scales of the tile's keys pt and 128 + pt; the rotary
      // parts of this CTA's keys land as bf16 and become [k'_hi | k'_lo] in place, eight lanes
      // a row
      float sA = 0.f, sB = 0.f;
      int idA = 0, idB = 0;                // blocks of those two keys
      bool seenA = false, seenB = false;   // whether they are visible
      const int r = pt & 63;
      auto scale_of = [&](int id) -> float {
        const uint8_t* row = p.rows + ((int64_t)id * kBlockSize + r) * kRowBytes8;
        return __ldg(reinterpret_cast<const float*>(row + kOffScale8));
      };
      auto load_tile = [&](const Piece& pc, const int32_t* bt, int t) {
        const int nb = blocks_in_tile(pc, t), v0 = pc.k_lo + t * kBlocksPerTile, kb = pt >> 6;
        seenA = seenB = false;
        sA = sB = 0.f;
        if (kb < nb) {
          const int32_t id = bt[window_block(pc.w, v0 + kb)];
          idA = valid_id(p, id) ? id : 0;
          int lo, hi;
          rows_in_block(pc, t, kb, &lo, &hi);
          seenA = r >= lo && r < hi;
          sA = scale_of(idA);
        }
        if (kb + 2 < nb) {
          const int32_t id = bt[window_block(pc.w, v0 + kb + 2)];
          idB = valid_id(p, id) ? id : 0;
          int lo, hi;
          rows_in_block(pc, t, kb + 2, &lo, &hi);
          seenB = r >= lo && r < hi;
          sB = scale_of(idB);
        }
      };
      auto table_entry = [&](float* tab, int key, float s, bool seen) {
        float f = seen ? s : 1.0f;         // a hidden key's scale may be anything
        if (f < kMinScale) f = kMinScale;  // a NaN stays one
        tab[key] = f;
        tab[kTileKeys + key] = __log2f(f);
      };
      auto split_rotary = [&]() {
        const int j = lane & 7;
#pragma unroll 1
        for (int k0 = 0; k0 < 8; k0 += 2) {
          uint32_t w[2][4];
          const uint32_t box = sRot + (pw >> 1) * kBoxBytes;
          const int m0 = 32 * (pw & 1) + 4 * k0 + (lane >> 3);
#pragma unroll
          for (int k = 0; k < 2; ++k) ld_shared_v4(box + (m0 + 4 * k) * 128 + ((j ^ ((m0 + 4 * k) & 7)) << 4), &w[k][0]);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int m = m0 + 4 * k;
            uint32_t h0, l0, h1, l1;
            split4(bf_lo(w[k][0]), bf_hi(w[k][0]), bf_lo(w[k][1]), bf_hi(w[k][1]), h0, l0);
            split4(bf_lo(w[k][2]), bf_hi(w[k][2]), bf_lo(w[k][3]), bf_hi(w[k][3]), h1, l1);
            // this lane's 8 values: half of granule j / 2 of the hi terms, 4 + j / 2 of the lo
            const uint32_t row = box + m * 128 + 8 * (j & 1);
            st_shared_v2(row + (((j >> 1) ^ (m & 7)) << 4), h0, h1);
            st_shared_v2(row + (((4 + (j >> 1)) ^ (m & 7)) << 4), l0, l1);
          }
        }
      };
      Walker walk(p, part);
      Piece cur;
      uint32_t tiles = 0, raws = 0;
      int npieces = 0;
      while (go && walk.next(cur)) {
        const int32_t* bt = unit_table(p, cur.b);
        if (npieces > 0) ok = wait_bar(&ctrl, p, smem_u32(&ctrl.q_empty), (npieces - 1) & 1) && ok;
        // a wait that ran out in another warp shows at the next publish; this one loads only
        // after its own wait, so the buffer is free
        if (pw == 0 && __all_sync(0xffffffffu, ok)) load_q(cur.b);
        load_tile(cur, bt, 0);
        ok = wait_bar(&ctrl, p, smem_u32(&ctrl.q_raw), npieces & 1) && ok;
        if (__all_sync(0xffffffffu, ok)) split_rows(npieces);  // (whole warps: it shuffles)
        if (!publish()) break;
        if (pt == 0) arrive(&ctrl.q_full, q_full_l);
        const int nt = num_tiles(cur);
        for (int t = 0; t < nt && go; ++t) {
          const uint32_t buf = tiles & 1;
          const int own = min(max(blocks_in_tile(cur, t) - 2 * (int)rank, 0), 2);
          if (tiles >= 1) ok = wait_bar(&ctrl, p, smem_u32(&ctrl.k_empty), (tiles - 1) & 1) && ok;
          if (own > 0) {
            // lane 0 of the two even warps brings the block whose scales it holds
            const uint32_t bar = smem_u32(&ctrl.k_raw);
            const bool all = __all_sync(0xffffffffu, ok);
            expect_tx_if(all && pt == 0, bar, own * kBoxBytes);
            tma_load_3d_if(all && lane == 0 && !(pw & 1) && (pw >> 1) < own, sRot + (pw >> 1) * kBoxBytes, &p.tm_rows,
                           bar, kOffKpe8, 0, leader ? idA : idB);
          }
          if (tiles >= 2) ok = wait_bar(&ctrl, p, smem_u32(&ctrl.sc_empty[buf]), ((tiles >> 1) - 1) & 1) && ok;
          if (ok) {
            float* tab = tables + buf * (kTabBytes / 4);
            table_entry(tab, pt, sA, seenA);
            table_entry(tab, 128 + pt, sB, seenB);
          }
          if (t + 1 < nt) load_tile(cur, bt, t + 1);
          if (own > 0) {
            ok = wait_bar(&ctrl, p, smem_u32(&ctrl.k_raw), raws & 1) && ok;
            ++raws;
            if ((pw >> 1) < own && __all_sync(0xffffffffu, ok)) split_rotary();
          }
          if (!publish()) break;
          if (pt == 0) {
            mbar_arrive(smem_u32(&ctrl.sc_full[buf]));
            arrive(&ctrl.k_full, k_full_l);
          }
          ++tiles;
        }
        ++npieces;
      }
    }
    // the peer CTA's MMA warp has no role; it joins its warpgroup's register release and
    // writes the rows of units that no piece covers
    else if (warp == kMmaWarp) {
      regs_dec<kRegsIssue>();
      write_orphan_units(p.meta, p.B, p.M, p.window, p.sinks, part, P, lane, [&](int u) { return unit_len(p, u); },
                         p.out, p.lse, p.status);
    }
  }

  // ---- teardown ------------------------------------------------------------
  if (warp == kSoftmaxWarp0 && lane == 0) bulk_wait_all();  // the epilogue's TMA stores landed
  tc_fence_before();
  __syncthreads();
  // Every role has stopped issuing (all waits are bounded).  Each CTA tells the other
  // whether it aborted; then both drain together or neither does.
  if (tid == 0) st_cluster_u32(mapa_shared(smem_u32((const void*)&ctrl.peer_abort), rank ^ 1u), (uint32_t)ctrl.abort);
  cluster_sync();
  tc_fence_after();
  if (ctrl.abort || ctrl.peer_abort) {
    // A wait ran out somewhere in the pair: asynchronous work issued before it may still
    // be in flight.  Tensor-core work (MMAs) has a completion handle: a commit issued
    // after it arrives on both CTAs' drain barriers once all of it has completed.  TMA
    // loads have none besides the stage barriers that did not complete, so both CTAs
    // also wait out their latency (at most a few microseconds even under full load)
    // with a 500 us margin before the TMEM and the shared memory are released.
    if (warp == kMmaWarp) {
      const bool el = elect_one();
      if (leader) commit_2sm_if(el, smem_u32(&ctrl.drain));
      const uint64_t dl = globaltimer_ns() + kDrainWaitNs;
      while (!mbar_try_wait(smem_u32(&ctrl.drain), 0) && globaltimer_ns() < dl) {
      }
    }
    if (tid == 0) {
      const uint64_t until = globaltimer_ns() + kQuiesceNs;
      while (globaltimer_ns() < until) {
      }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

}  // namespace

cudaError_t window_fp8_setup() {
  return cudaFuncSetAttribute(window_fp8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemDyn + 1024);
}

cudaError_t launch_window_fp8(const CUtensorMap& tm_rows, const CUtensorMap& tm_qn, const CUtensorMap& tm_qp,
                              const CUtensorMap& tm_out, const CUtensorMap& tm_part, const void* rows,
                              const int32_t* block_table, int max_blocks, const int32_t* seqlens,
                              const int32_t* q_lens, const int32_t* meta, int64_t num_blocks, int units, int rep,
                              int H, float scale, int window, int sinks, void* out, float* lse, float* part_lse,
                              int32_t* status, int num_ctas, uint64_t wait_timeout_ns, int inject_stall,
                              cudaStream_t stream) {
  Params prm;
  std::memset(&prm, 0, sizeof(prm));
  prm.tm_rows = tm_rows;
  prm.tm_out = tm_out;
  prm.tm_part = tm_part;
  prm.rows = static_cast<const uint8_t*>(rows);
  prm.tm_qn = tm_qn;
  prm.tm_qp = tm_qp;
  prm.block_table = block_table;
  prm.seqlens = seqlens;
  prm.q_lens = q_lens;
  prm.meta = meta;
  prm.out = static_cast<__nv_bfloat16*>(out);
  prm.lse = lse;
  prm.part_lse = part_lse;
  prm.status = status;
  prm.num_blocks = num_blocks;
  prm.timeout_ns = wait_timeout_ns;
  prm.max_blocks = max_blocks;
  prm.B = units;
  prm.rep = rep;
  prm.M = H;
  prm.window = window;
  prm.sinks = sinks;
  prm.scale_log2 = scale * 1.4426950408889634f;
  prm.inject_stall = inject_stall;
  // programmatic dependent launch, as for the other attention kernel
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemDyn + 1024;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, window_fp8_kernel, prm);
}

}  // namespace mla
