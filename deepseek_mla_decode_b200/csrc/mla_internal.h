// Internal layout shared by the host entry points and the kernels of libmla.so.
#pragma once
#include <cstdint>

namespace mla {

constexpr int kBlockSize = 64;     // cache rows per physical block
constexpr int kDLatent = 512;      // c_kv / output width
constexpr int kDRope = 64;         // k_pe / q_pe width
constexpr int kDQK = 576;          // cache row width
constexpr int kRowsPerTile = 128;  // query rows (token-major: row = i * H + h) per CTA pair
constexpr int kRowsPerCta = 64;    // each CTA of the pair owns 64 of them
constexpr int kTileKeys = 256;     // keys per pipeline step (4 cache blocks)
constexpr int kBlocksPerTile = kTileKeys / kBlockSize;

// Packed FP8 cache row (bytes): [0, 512) e4m3 codes of c_kv / scale, [512, 640) k_pe /
// scale as 64 bf16, [640, 644) the fp32 scale, [644, 656) zero.
constexpr int kRowBytes8 = 656;
constexpr int kOffKpe8 = 512;
constexpr int kOffScale8 = 640;

// Split-KV scheduler constants (the same values are stated in the float64 oracle).
constexpr int kSchedOverheadTiles = 1;  // cost of starting a sequence, in 256-key tiles
constexpr int kSchedMinCap = 2;         // smallest partition cost, in tiles
constexpr int kMaxWorkers = 256;         // CTA pairs the metadata can describe

// ---------------------------------------------------------------------------
// Metadata buffer (int32 words), written by mla_get_metadata:
//   [0, kHdrWords)                      header (see kHdr*)
//   part_start [kMaxWorkers][2]         (b, k) of each partition's first block
//   part_end   [kMaxWorkers][2]         exclusive end (next partition's start)
//   nblk[B], first_part[B], num_splits[B], split_prefix[B]
// ---------------------------------------------------------------------------
constexpr int kHdrWords = 16;
enum HdrField : int {
  kHdrMagic = 0,
  kHdrB = 1,
  kHdrSq = 2,
  kHdrH = 3,
  kHdrNumParts = 4,   // P: partitions per row tile
  kHdrNumTiles = 5,   // T: row tiles of 128 query rows
  kHdrCap = 6,        // partition cost cap (256-key tiles)
  kHdrTotalSlots = 7, // sum of num_splits
  kHdrNumWorkers = 8, // CTA pairs available on the device
  kHdrOverhead = 9,
  kHdrTokens = 10,    // token schedule: the call's s_q (query tokens per sequence); 0 otherwise
  kHdrTokCausal = 11, // token schedule: the causal flag the lengths were built with
  kHdrWindow = 12,    // windowed schedule: keys in the window; 0 otherwise
  kHdrSinks = 13,     // windowed schedule: first keys that stay visible
  kHdrSignature = 14, // two words: schedule_signature of what the schedule was made for
};
constexpr int32_t kMetaMagic = 0x4D4C4131;     // "MLA1"
constexpr int32_t kMetaMagicWin = 0x4D4C4157;  // "MLAW": a windowed schedule

// What a schedule was made for, in one 64-bit word for the LSE combine: the attention kernel
// checks the header's fields and runs no piece of another call's schedule, whose slots then
// hold nothing and may lie outside the workspace.  (The combine's own check of the fields
// made a decode of 64 sequences 1 us longer: its few registers are all in use.)
inline uint64_t schedule_signature(int B, int s_q, int H, int P, int tok_rep, int tok_causal, int window, int sinks) {
  uint64_t h = static_cast<uint32_t>(kMetaMagic);
  for (int v : {B, s_q, H, P, tok_rep, tok_rep ? tok_causal : 0, window, sinks}) {
    h = (h ^ static_cast<uint32_t>(v)) * 0x9E3779B97F4A7C15u;
    h ^= h >> 32;
  }
  return h;
}

// Token schedule: the decode of B sequences with up to `rep` query tokens each (q of
// them real) runs as an s_q = 1 decode of B * rep sequences; sequence u = b * rep + t
// is token t of b.  With the causal mask token t sees the first n - q + t + 1 keys of
// b (all n without it); a padding token (t >= q) sees none.  -1 marks an invalid query
// count or a negative length.  The schedule, the attention kernel and the combine all
// take a token's length from here.
__host__ __device__ inline int token_seq_len(int n, int q, int t, int rep, int causal) {
  if (q < 0 || q > rep || n < 0) return -1;
  if (t >= q) return 0;
  if (!causal) return n;
  const int v = n - q + t + 1;
  return v > 0 ? v : 0;
}

// Sliding window.  The token at position n - 1 sees the keys t < n with t >= n - window or
// t < sinks.  Its blocks are numbered through without the hidden ones: `sink_blocks` blocks
// of first keys, then the blocks from `first` to the sequence's last.  Where nothing is
// hidden between them (n - window <= sinks) the numbers are the sequence's own.  Hidden
// rows are a block's last (the last sink block keeps sink_rows, the sequence's last block
// the rows before n) or its first (block `first` hides `skip`), never both: a window of at
// least one block does not end in the block it starts in unless it fills it.
struct WindowBlocks {
  int sink_blocks, sink_rows, first, skip, count;
};
constexpr int kMinWindow = kBlockSize;
__host__ __device__ inline WindowBlocks window_blocks(int n, int window, int sinks) {
  WindowBlocks w{0, 0, 0, 0, n / kBlockSize + (n % kBlockSize != 0)};
  const int lo = n - window;
  if (lo <= sinks) return w;
  w.sink_blocks = sinks / kBlockSize + (sinks % kBlockSize != 0);
  w.sink_rows = sinks - (w.sink_blocks - 1) * kBlockSize;
  w.first = lo / kBlockSize;
  w.skip = lo % kBlockSize;
  w.count += w.sink_blocks - w.first;
  return w;
}
// The sequence's block behind number v, and the rows [lo, hi) of it that are visible.
__host__ __device__ inline int window_block(const WindowBlocks& w, int v) {
  return v < w.sink_blocks ? v : w.first + v - w.sink_blocks;
}
__host__ __device__ inline void window_rows(const WindowBlocks& w, int n, int v, int* lo, int* hi) {
  if (v < w.sink_blocks) {
    *lo = 0;
    *hi = v == w.sink_blocks - 1 ? w.sink_rows : kBlockSize;
  } else {
    const int left = n - window_block(w, v) * kBlockSize;
    *lo = v == w.sink_blocks ? w.skip : 0;
    *hi = left < kBlockSize ? left : kBlockSize;
  }
}

__host__ __device__ inline int64_t meta_words(int B) {
  return kHdrWords + 4LL * kMaxWorkers + 4LL * B;
}
__host__ __device__ inline int off_part_start() { return kHdrWords; }
__host__ __device__ inline int off_part_end() { return kHdrWords + 2 * kMaxWorkers; }
__host__ __device__ inline int off_nblk() { return kHdrWords + 4 * kMaxWorkers; }
__host__ __device__ inline int64_t off_first_part(int B) { return off_nblk() + (int64_t)B; }
__host__ __device__ inline int64_t off_num_splits(int B) { return off_nblk() + 2LL * B; }
__host__ __device__ inline int64_t off_split_prefix(int B) { return off_nblk() + 3LL * B; }

// ---------------------------------------------------------------------------
// Workspace: partial outputs of split sequences.
//   partial_o   fp32 [slots][M_total][512]   (normalised by the piece's own sum)
//   partial_lse fp32 [slots][M_total]
// with slots = B + P*T upper bound (each partition boundary cuts one sequence).
// ---------------------------------------------------------------------------
__host__ __device__ inline int64_t ws_slots(int B, int num_workers) { return (int64_t)B + num_workers; }

// Kernel error bits (mirror MLA_DEVICE_ERR_* of the public header).
constexpr int kErrBlockId = 1;
constexpr int kErrSeqlen = 2;
constexpr int kErrTimeout = 4;
constexpr int kErrMetadata = 8;

}  // namespace mla
