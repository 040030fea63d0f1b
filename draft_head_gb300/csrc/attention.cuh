// What the attention kernels share: the packed query rows of a tile, which
// cache slots they see, the split of a long cache over CTAs and the join of the
// splits' partial results.
#pragma once

#include "common.cuh"
#include "rows.cuh"

namespace domino {

// A tile is `BM` packed query rows of one kv head of one request: packed row r
// is row i = r / G of the block and query head kvh * G + r % G (G query heads
// read one kv head), so that all the rows that need a key tile share its load.
//
// Which slots a tile sees: [0, sinks) and [low, end), taken in key tiles of BN
// slots: first the tiles from floor(low / BN) on, then the sink tiles (few of their
// slots are seen, so a maximum begun there would have to be raised).
struct KeyTiles {
  int main_begin, main_count;  // tiles main_begin .. main_begin + main_count - 1 first
  int count;                   // then tiles 0 .. count - main_count - 1
  __device__ __forceinline__ int slot(int k, int BN) const {
    return (k < main_count ? main_begin + k : k - main_count) * BN;
  }
};

// First slot of the window of a row at position p.
__device__ __forceinline__ int window_low(int p, int window) {
  if (window == 0) return 0;
  const int64_t low = (int64_t)p - window + 1;
  return low < 0 ? 0 : (low > 0x7fffffff ? 0x7fffffff : (int)low);
}

// low: the smallest window_low of the tile's rows; i_last: its last row.
__device__ __forceinline__ KeyTiles key_tiles(int mode, int sinks, int low, int ctx, int n, int i_last, int BN) {
  const int end = mode == DOMINO_MASK_CAUSAL ? ctx + i_last + 1 : ctx + n;
  // Outside the causal mode the window does not reach into the block.
  const int start = mode == DOMINO_MASK_CAUSAL ? min(low, end) : min(low, ctx);
  KeyTiles k;
  // A window that begins past the row itself (positions ahead of the slots) leaves all tiles to the sinks.
  k.main_begin = start < end ? start / BN : (end + BN - 1) / BN;
  k.main_count = (end + BN - 1) / BN - k.main_begin;
  k.count = k.main_count + min((min(sinks, end) + BN - 1) / BN, k.main_begin);
  return k;
}

// Whether a row (place i, window from `low`) sees slot s.
__device__ __forceinline__ bool sees(int mode, int sinks, int low, int ctx, int n, int i, const uint8_t* mask_row, int s) {
  const bool near = s >= low || s < sinks;
  const int j = s - ctx;
  if (j < 0) return near;
  if (mode == DOMINO_MASK_CAUSAL) return j <= i && near;
  if (mode == DOMINO_MASK_FULL) return j < n;
  return j < n && mask_row[j] != 0;
}

// The split of a tile's key tiles over `splits` CTAs at most: none gets fewer
// than `least` key tiles, so a short past (known on the device only) is not
// cut into pieces that cost more to join than they save.
__device__ __forceinline__ int splits_used(int splits, int count, int least) {
  return max(1, min(splits, count / least));
}

// Partial results of the splits of a tile in the workspace: per (tile, split)
// BM x D sums of exp2(s - m) v (fp32) and BM pairs (m, l).
struct Partials {
  float* o;
  float2* ml;
  unsigned int* arrived;  // per tile, zero between calls
};

// Splits of each of `tiles` tiles so that about `want` CTAs run (kCountersPerSm per SM at most); 1 from
// `want` tiles on. tiles * splits stays below 2 * want, which sizes the workspace for every smaller
// block too.
inline int splits_for(int64_t tiles, int64_t want, int64_t most) {
  int64_t s = (want + tiles - 1) / tiles;
  s = s < most ? s : most;
  return (int)(s < 1 ? 1 : s);
}
// The workspace behind its control block: the counters, whose place is the same for every attention kernel (they are
// zero between calls, and a workspace may go from one kernel to another), then what a kernel needs for itself.
constexpr int kCountersPerSm = 8;  // tiles that are cut, at most, for each SM
inline size_t counter_bytes() { return ((size_t)kCountersPerSm * num_sms() * 4 + 255) & ~(size_t)255; }
inline size_t partial_bytes(int64_t want, int BM, int D) {
  return counter_bytes() + (size_t)(2 * want) * BM * (8 + (size_t)D * 4);
}
inline Partials partials_at(void* scratch, int64_t want, int BM) {
  uint8_t* w = (uint8_t*)scratch;
  Partials p;
  p.arrived = (unsigned int*)w;
  w += counter_bytes();
  p.ml = (float2*)w;
  p.o = (float*)(w + (size_t)(2 * want) * BM * 8);
  return p;
}

}  // namespace domino
