// Attention of a few rows over the cache (domino_block_attention and
// domino_paged_attention; the definitions are in domino.h): bf16 or codes, head_dim <= 128,
// at most 16 packed rows of a kv head, as when a token is decoded.
//
// Bound by the cache's bytes, or with one request by the time from launch to the last join.
// So: no shared memory, barriers or tensor memory on the way of the keys and values, and a
// short program (a cold instruction costs more than a cold byte here). A warp takes 16 slots
// at a time, the next ones' loads in flight. It computes S^T = K Q^T and O^T += V^T P^T with
// mma.m16n8k16: 16 slots (or 16 columns of V) against 8 rows, so that eight rows waste nothing.
// The order of the terms of a dot product is free, and so is that of the columns of O, so
// every operand is read in 16-byte pieces as it lies in memory:
//   K  lane (n = lane / 4, c = lane % 4) reads elements [32 j + 8 c, + 8) of slots n, n + 8; two
//      pairs of them are one K = 16 step, and Q is read with the same order;
//   V  the lane reads elements [64 j + 8 n, + 8) of slots 2 c, 2 c + 1, 2 c + 8, 2 c + 9; byte
//      permutes pair the slots, and O's rows 2 c, 2 c + 1 end up with eight neighbouring columns.
// P goes from the accumulators' layout to the operand's by movmatrix. Maxima as in the tensor
// core kernel: raised only when a score passes them by 2^kLazy.
// Four warps of a CTA share its slots and join in shared memory; CTAs that share a row tile
// write their sums to the workspace, and the last one joins them in order.
//
// One token, 32 heads of 128 over 8 of the cache: over 4000 slots 12.2 us (20 with the tensor core
// kernel), over 30,000 slots 28.1 us (4.4 TB/s); 64 tokens over up to 4000 slots each 117 us
// (4.6 TB/s).
//
// Pages hold 16 slots at least, so a tile of 16 lies in one: one table entry a tile, read a tile ahead.
// Codes (e4m3 with a power of two per slot and head) are fp16 to the mma: a conversion instruction makes two of them at once, exactly
// (in bf16 it takes a permute, a shift, a mask and a product), and no scale is applied to them. A key's scale multiplies its score, a
// value's its weight, as an addition to the logarithm, in fp32: P is rounded to fp16, 2^-12 of a weight where bf16 gives 2^-9. As the weights
// carry the scales, the maximum that they are relative to is that of score + scale, 2^11 there and 2^15 at most, so that products down to
// 2^-35 of the largest count; the softmax's own weights are summed in fp32 relative to the scores' maximum (an exponential more, 229 us both).
// Queries are brought to fp16's range by a power of two per row. A value that is no number has that in its scale, so a
// row that does not see it cannot get it: there is nothing to clear. The codes wait in a warp's ring in shared memory (cp.async), which
// frees the registers of the tiles on their way: one token over 4000 quantised slots 11.7 us, 128 tokens over up to 8000 229 us, 4.8 TB/s of
// half the bytes (bf16 pages 393 us, 5.6 TB/s).
#include <math.h>
#include <algorithm>

#include "attention.cuh"
#include "packed.cuh"
#include "pages.cuh"

namespace domino {

namespace {

constexpr int kBN = 16, kWarps = 4, kThr = 32 * kWarps;
constexpr int kLeast = 8;  // key tiles per CTA at least: two per warp
// From kManyTiles row tiles on, pieces of at least kLeastMany key tiles, about kWaves times as many as are
// resident at once: the lengths are unlike, and one round and a half of whole row tiles leaves SMs idle. Tokens
// of 16 / 32 / 64 / 128 requests over up to 4000 slots: 37.8 / 61.6 / 116.7 / 198.8 us; with one round of pieces
// 42.6 / 69.9 / 126.8 / 206.8. Of 8 requests (64 row tiles, fewer pieces than SMs) 33.8, with the other rule 28.6.
constexpr int kManyTiles = 96, kLeastMany = 64, kWaves = 4;
constexpr int kMostPieces = 64;  // of a row tile: their join takes a round trip for every eight
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazyBf16 = 32.0f;
// Codes: weights with their values' scales in fp16, 2^kAtMost at the maximum and 2^(kAtMost + kLazyCodes) at most.
constexpr float kLazyCodes = 4.0f, kAtMost = 11.0f;
constexpr float kRoom = 10.0f;  // a warp's sum of weights is left between 2^-kRoom and twice that: no join passes fp32's range
constexpr int kCodesCtas = 3, kDepth = 2;  // of one group of rows, on an SM; tiles of a warp's ring (3 and 2: 128 tokens 229 us, one 11.7; 3 and 3: 231 and 11.8; 4 and 2: 224 and 13.0)

struct RowsP {
  AttnArgs a;
  Partials part;
  int splits, least;  // CTAs per row tile at most; key tiles that each has at least
  float c;  // scale log2(e)
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <int CACHE>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (CACHE == kPagedE4m3)
    mma16816_f16(d, a0, a1, a2, a3, b0, b1);
  else
    mma16816(d, a0, a1, a2, a3, b0, b1);
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint4 ldg16(const __nv_bfloat16* p) {
  uint4 x;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
  return x;
}
// Eight elements of a slot.
struct Piece {
  uint4 x;
  __device__ __forceinline__ void load(const void* base, int64_t at) { x = ldg16((const __nv_bfloat16*)base + at); }
  __device__ __forceinline__ void zero() { x = make_uint4(0, 0, 0, 0); }
};
// Codes wait in a warp's ring in shared memory: a tile's keys, values and scales, rows padded so that the lanes' 8-byte reads
// meet every bank once.
template <int JJ>
struct Tile {
  static constexpr int DP = 64 * JJ, kKeyRow = DP + 32, kValueRow = DP + 16;
  static constexpr int kValues = kBN * kKeyRow, kScales = kValues + kBN * kValueRow, kBytes = kScales + 2 * kBN;
};
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, bool there) {  // zeros where it is not
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint2 lds8(const uint8_t* p) { return *(const uint2*)p; }
__device__ __forceinline__ uint4 pairs8(uint2 x) {
  const uint2 a = codes_f16(x.x), b = codes_f16(x.y);
  return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ uint32_t part(const uint4& x, int t) { return t == 0 ? x.x : t == 1 ? x.y : t == 2 ? x.z : x.w; }
__device__ __forceinline__ bool bad16(uint32_t x) {  // a bf16 pair with an infinity or a NaN in it
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t clear16(uint32_t x) {
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
  return x;
}

// NT: groups of 8 rows; KS: 32-element pieces of a head; JJ: 64-element pieces.
template <int NT, int KS, int JJ, int CACHE>
__global__ void __launch_bounds__(kThr, CACHE == kPagedE4m3 && NT == 1 ? kCodesCtas : 2) attn_rows_kernel(const __grid_constant__ RowsP p) {
  constexpr int kRows = 8 * NT, DP = 64 * JJ;
  constexpr bool kCodes = CACHE == kPagedE4m3;
  constexpr float kLazy = kCodes ? kLazyCodes : kLazyBf16;
  using Codes = Tile<JJ>;
  // The warps' sums, and before them the rings of codes.
  constexpr int kRing = kCodes ? kDepth * Codes::kBytes : 0, kSums = kRows * (DP + 4) * 4;
  constexpr int kMine = (kRing > kSums ? kRing : kSums);
  extern __shared__ __align__(16) uint8_t s_dyn[];
  __shared__ __align__(16) uint8_t s_fixed[kCodes ? 16 : kWarps * kMine];
  uint8_t* s_all = kCodes ? s_dyn : s_fixed;
  auto s_o = [&](int w, int r, int e) { return (float*)(s_all + w * kMine) + r * (DP + 4) + e; };
  __shared__ float2 s_ml[kWarps][kRows];
  __shared__ int s_low[kRows], s_i[kRows], s_last;
  const AttnArgs& a = p.a;
  const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
  const int G = a.hq / a.hkv;
  int q0, rows_n, ctx;
  if (!request_rows(a.rows, b, q0, rows_n, ctx, threadIdx.x == 0, a.ctl)) return;
  const int rows = rows_n * G;
  if (rows == 0) return;
  if (threadIdx.x < kRows) {
    const int i = min((int)threadIdx.x, rows - 1) / G;
    s_i[threadIdx.x] = i;
    s_low[threadIdx.x] = window_low(a.rows.positions ? a.rows.positions[q0 + i] : ctx + i, a.window);
  }
  // Q, rows n (+ 8): the terms in the order in which K is read.
  uint32_t q[NT][KS][4];
#pragma unroll
  for (int g = 0; g < NT; ++g) {
    const int r = g * 8 + n, i = min(r, rows - 1) / G;
    const __nv_bfloat16* src = (const __nv_bfloat16*)a.q + ((int64_t)(q0 + i) * a.hq + h * G + (min(r, rows - 1) - i * G)) * a.D;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (r < rows && 32 * j + 8 * c < a.D) x = *(const uint4*)(src + 32 * j + 8 * c);
      q[g][j][0] = x.x; q[g][j][1] = x.y; q[g][j][2] = x.z; q[g][j][3] = x.w;
    }
  }
  float qc[NT][2];  // scale log2(e), and the power of two that a row's queries were divided by
#pragma unroll
  for (int g = 0; g < NT; ++g) {
    int e = 0;
    if (kCodes) {
      uint32_t most = 0;
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) most = max(most, max((q[g][j][x] << 16) & 0x7fff0000u, q[g][j][x] & 0x7fff0000u));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
      e = query_exponent(most);
      const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) q[g][j][x] = query_f16(q[g][j][x], f);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int of = kCodes ? __shfl_sync(0xffffffffu, e, (2 * c + x) * 4) : 0;
      qc[g][x] = kCodes ? p.c * __uint_as_float((uint32_t)(of + 127) << 23) : p.c;
    }
  }
  __syncthreads();
  int low_min = 0x7fffffff, low_max = 0;
  for (int r = 0; r < kRows; ++r) {
    low_min = min(low_min, s_low[r]);
    low_max = max(low_max, s_low[r]);
  }
  const KeyTiles kt = key_tiles(a.mode, a.sinks, low_min, ctx, rows_n, rows_n - 1, kBN);
  const int used = splits_used(p.splits, kt.count, p.least);
  if (split >= used) return;
  const int k_begin = (int)((int64_t)kt.count * split / used), k_end = (int)((int64_t)kt.count * (split + 1) / used);
  // Slots that every row sees: from all_low (or among the sinks) up to all_hi.
  const int all_hi = a.mode == DOMINO_MASK_CAUSAL ? ctx + 1 : a.mode == DOMINO_MASK_FULL ? ctx + rows_n : ctx;
  const int all_low = a.mode == DOMINO_MASK_CAUSAL ? low_max : min(low_max, ctx);
  const uint8_t* mask = a.mask ? a.mask + (int64_t)b * a.rows.max_q * a.rows.max_q : nullptr;

  const int end = ctx + rows_n;
  Piece kx[2][KS], vx[4][JJ];
  int64_t tile_at = 0;  // elements from the caches' begin to the tile's first slot
  bool tile_there = true;
  // Where in a tile the lane's first piece of keys and of values is.
  const int64_t k_lane = (int64_t)n * a.ss + 8 * c, v_lane = (int64_t)(2 * c) * a.ss + 8 * n;
  const uint32_t ring = smem_u32(s_all) + (uint32_t)(warp * kMine);
  int in_ring = 0, out_ring = 0;
  // Pages are as large as tiles at least, so a tile lies in one: its number is read one tile ahead of the tile.
  auto page_at = [&](int k) { return CACHE == kWhole ? 0 : page_of(a.pages, b, kt.slot(k, kBN)); };
  auto fetch = [&](int k, int page) {
    const int s0 = kt.slot(k, kBN);
    if (CACHE == kWhole)
      tile_at = (int64_t)b * a.rs + (int64_t)h * a.hs + (int64_t)s0 * a.ss;
    else
      tile_at = (int64_t)page * a.pages.page_stride + (int64_t)h * a.hs + (int64_t)slot_in_page(a.pages, s0) * a.ss;
    tile_there = CACHE == kWhole || page >= 0;
    if (!tile_there && lane == 0) dev_error(a.ctl, DEV_ERR_DATA);
    const int there = tile_there ? end - s0 : 0;  // slots of the tile
    if constexpr (kCodes) {
      const uint32_t to = ring + (uint32_t)(in_ring * Codes::kBytes);
      constexpr int kPieces = DP / 16, kStep = 32 / kPieces;  // of a row; rows at a time
      const int piece = lane % kPieces, r0 = lane / kPieces;
      const uint8_t* kp = (const uint8_t*)a.k + tile_at + (int64_t)r0 * a.ss + piece * 16;
      const uint8_t* vp = (const uint8_t*)a.v + tile_at + (int64_t)r0 * a.ss + piece * 16;
      const bool in_head = piece * 16 < a.D;
#pragma unroll
      for (int r = 0; r < kBN; r += kStep) {
        const bool here = r0 + r < there && in_head;
        copy16(to + (r0 + r) * Codes::kKeyRow + piece * 16, here ? kp + (int64_t)r * a.ss : (const uint8_t*)a.k, here);
        copy16(to + Codes::kValues + (r0 + r) * Codes::kValueRow + piece * 16, here ? vp + (int64_t)r * a.ss : (const uint8_t*)a.v, here);
      }
      if (lane < 2) {
        const uint8_t* from = lane == 0 ? a.pages.k_scale : a.pages.v_scale;
        copy16(to + Codes::kScales + lane * kBN, tile_there ? from + scale_at(a.pages, a.hkv, page, h, s0) : from, tile_there);
      }
      if (++in_ring == kDepth) in_ring = 0;
      return;
    }
    const int64_t k_at = tile_at + k_lane, v_at = tile_at + v_lane;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int s = n + 8 * x;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        if (s < there && 32 * j + 8 * c < a.D)
          kx[x][j].load(a.k, k_at + x * (8 * (int64_t)a.ss) + 32 * j);
        else
          kx[x][j].zero();
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int s = 2 * c + (x & 1) + 8 * (x >> 1);
#pragma unroll
      for (int j = 0; j < JJ; ++j) {
        if (s < there && 64 * j + 8 * n < a.D)
          vx[x][j].load(a.v, v_at + ((x & 1) + 8 * (x >> 1)) * (int64_t)a.ss + 64 * j);
        else
          vx[x][j].zero();
      }
    }
  };

  // Codes: l, the sum of the softmax's own weights, is relative to the maximum of the scores, ms, and o to m above it: kAtMost below
  // the maximum of score + the value's exponent. (From one of them, weights or their sum would leave fp32's range beside values
  // whose exponents are far apart; and added to scores that are large themselves, m would be lost in them.) ms begins below every
  // score, so that -inf alone has weight 0.
  float o[NT][4 * JJ][4], m[NT][2], l[NT][2], ms[NT][2];
#pragma unroll
  for (int g = 0; g < NT; ++g) {
#pragma unroll
    for (int t = 0; t < 4 * JJ; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[g][t][e] = 0.0f;
    m[g][0] = m[g][1] = kCodes ? 0.0f : -INFINITY;
    ms[g][0] = ms[g][1] = -3.402823466e+38f;
    l[g][0] = l[g][1] = 0.0f;
  }
  int page = 0;
  constexpr int kAhead = kCodes ? kDepth * kWarps : kWarps;  // the tile that is asked for while one is worked on
#pragma unroll
  for (int d = 0; d < kAhead; d += kWarps) {
    const int k = k_begin + warp + d;
    if (k < k_end) fetch(k, page_at(k));
    if (kCodes) asm volatile("cp.async.commit_group;" ::: "memory");
  }
  if (!kCodes && k_begin + warp + kAhead < k_end) page = page_at(k_begin + warp + kAhead);
#pragma unroll 1
  for (int k = k_begin + warp; k < k_end; k += kWarps) {
    const int s0 = kt.slot(k, kBN);
    const int64_t here = tile_at;
    const bool gone = CACHE != kWhole && !tile_there;  // no such page: nothing was read
    Piece kr[2][KS], vr[4][JJ];
    const uint8_t* codes = nullptr;
    // Codes: the keys' scales of slots n and n + 8 (e / 2 of the scores below), and the values' as exponents.
    float ks[2], ve[2];
    if constexpr (kCodes) {
      if (k + kAhead < k_end) page = page_at(k + kAhead);
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
      __syncwarp();
      codes = s_all + warp * kMine + out_ring * Codes::kBytes;
      if (++out_ring == kDepth) out_ring = 0;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        ks[x] = scale_f32(codes[Codes::kScales + n + 8 * x]);
        const int v = codes[Codes::kScales + kBN + n + 8 * x];
        ve[x] = v == kScaleNan ? scale_f32(v) : (float)(v - 127);
      }
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int j = 0; j < KS; ++j) kr[x][j] = kx[x][j];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int j = 0; j < JJ; ++j) vr[x][j] = vx[x][j];
      if (k + kAhead < k_end) {
        fetch(k + kAhead, page);
        if (k + 2 * kAhead < k_end) page = page_at(k + 2 * kAhead);
      }
    }
    const bool whole = s0 + kBN <= all_hi && (s0 >= all_low || s0 + kBN <= a.sinks);
    bool mend = false;
    if constexpr (kCodes) {
      if (!whole) {  // a value that is no number has that in its scale, and so in its weight; slots without one may hold anything
        uint32_t* v = (uint32_t*)(codes + Codes::kValues);
        for (int x = lane; x < kBN * Codes::kValueRow / 4; x += 32) v[x] = codes_that_are_numbers(v[x]);
        __syncwarp();
      }
    } else {
      if (!whole) {
        // A weight of 0 does not stop an infinity or a NaN in the product: they are cleared here
        // and added below to the rows that see them.
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int j = 0; j < JJ; ++j) {
            uint4& v = vr[x][j].x;
            mend |= bad16(v.x) | bad16(v.y) | bad16(v.z) | bad16(v.w);
            v = make_uint4(clear16(v.x), clear16(v.y), clear16(v.z), clear16(v.w));
          }
        mend = __any_sync(0xffffffffu, mend) && !gone;
      }
    }
    float s[NT][4];  // slots n, n, n + 8, n + 8 of rows 2c, 2c + 1, 2c, 2c + 1
#pragma unroll
    for (int g = 0; g < NT; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[g][e] = 0.0f;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      const uint8_t* at = codes + n * Codes::kKeyRow + 32 * j + 8 * c;
      const uint4 k0 = kCodes ? pairs8(lds8(at)) : kr[0][j].x, k1 = kCodes ? pairs8(lds8(at + 8 * Codes::kKeyRow)) : kr[1][j].x;
#pragma unroll
      for (int g = 0; g < NT; ++g) {
        mma<CACHE>(s[g], k0.x, k1.x, k0.y, k1.y, q[g][j][0], q[g][j][1]);
        mma<CACHE>(s[g], k0.z, k1.z, k0.w, k1.w, q[g][j][2], q[g][j][3]);
      }
    }
    uint32_t pw[NT][2];
#pragma unroll
    for (int g = 0; g < NT; ++g) {
      bool hidden[4] = {};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // Codes: the factors first, as large queries may have small keys; and a product that no subtraction takes up, or large
        // scores would be their rounding away from their own maximum.
        s[g][e] = kCodes ? __fmul_rn(s[g][e], qc[g][e & 1] * ks[e >> 1]) : s[g][e] * qc[g][e & 1];
        if (!whole) {
          const int r = g * 8 + 2 * c + (e & 1), slot = s0 + n + 8 * (e >> 1);
          hidden[e] = !(slot < end && sees(a.mode, a.sinks, s_low[r], ctx, rows_n, s_i[r],
                                           mask ? mask + (int64_t)s_i[r] * a.rows.max_q : nullptr, slot));
          if (hidden[e]) s[g][e] = -INFINITY;
        }
      }
      if constexpr (kCodes) {
        float x[4], y[4];  // the weights' logarithms: of the products', of the softmax's own
        auto relative = [&] {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[e] = s[g][e] - ms[g][e & 1];
            x[e] = y[e] + (ve[e >> 1] - m[g][e & 1]);
          }
        };
        relative();
        if (__any_sync(0xffffffffu, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) > kAtMost + kLazy ||
                                        fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) > kLazy)) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float high = fmaxf(s[g][e], s[g][2 + e]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, d));
            const float now_s = high - ms[g][e] > kLazy ? high : ms[g][e], by = ms[g][e] - now_s;
            float top = fmaxf(s[g][e] - now_s + ve[0], s[g][2 + e] - now_s + ve[1]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float same = m[g][e] + by, now = top - same > kAtMost + kLazy ? top - kAtMost : same;
            f[e] = ex2(same - now);
            l[g][e] *= ex2(by);
            m[g][e] = now;
            ms[g][e] = now_s;
          }
#pragma unroll
          for (int t = 0; t < 4 * JJ; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[g][t][e] *= f[e & 1];
          relative();
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          l[g][e & 1] += ex2(y[e]);
          s[g][e] = hidden[e] ? 0.0f : ex2(x[e]);
        }
      } else {
        const float top[2] = {fmaxf(s[g][0], s[g][2]), fmaxf(s[g][1], s[g][3])};
        if (__any_sync(0xffffffffu, top[0] > m[g][0] + kLazy || top[1] > m[g][1] + kLazy)) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = top[e];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            const float now = x > m[g][e] + kLazy ? x : m[g][e];
            f[e] = now == m[g][e] || m[g][e] == -INFINITY ? 1.0f : ex2(m[g][e] - now);
            m[g][e] = now;
            l[g][e] *= f[e];
          }
#pragma unroll
          for (int t = 0; t < 4 * JJ; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[g][t][e] *= f[e & 1];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[g][e] = ex2(s[g][e] - (m[g][e & 1] == -INFINITY ? 0.0f : m[g][e & 1]));
          l[g][e & 1] += s[g][e];
        }
      }
      pw[g][0] = transpose8(kCodes ? pack_f16(s[g][0], s[g][1]) : pack_bf16(s[g][0], s[g][1]));
      pw[g][1] = transpose8(kCodes ? pack_f16(s[g][2], s[g][3]) : pack_bf16(s[g][2], s[g][3]));
    }
#pragma unroll
    for (int j = 0; j < JJ; ++j) {
      uint2 w[4];
      if constexpr (kCodes) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          w[x] = lds8(codes + Codes::kValues + (2 * c + (x & 1) + 8 * (x >> 1)) * Codes::kValueRow + 64 * j + 8 * n);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        // Elements 2 t and 2 t + 1 of slots 2 c and 2 c + 1 (a0, a1), 2 c + 8 and 2 c + 9 (a2, a3); codes are paired as bytes.
        uint32_t a0, a1, a2, a3;
        if constexpr (kCodes) {
          const uint32_t select = t & 1 ? 0x7362 : 0x5140;
          auto word = [&](int x) { return t < 2 ? w[x].x : w[x].y; };
          const uint2 lo = codes_f16(__byte_perm(word(0), word(1), select)), hi = codes_f16(__byte_perm(word(2), word(3), select));
          a0 = lo.x; a1 = lo.y; a2 = hi.x; a3 = hi.y;
        } else {
          const uint32_t v0 = part(vr[0][j].x, t), v1 = part(vr[1][j].x, t), v2 = part(vr[2][j].x, t), v3 = part(vr[3][j].x, t);
          a0 = __byte_perm(v0, v1, 0x5410); a1 = __byte_perm(v0, v1, 0x7632);
          a2 = __byte_perm(v2, v3, 0x5410); a3 = __byte_perm(v2, v3, 0x7632);
        }
#pragma unroll
        for (int g = 0; g < NT; ++g) mma<CACHE>(o[g][4 * j + t], a0, a1, a2, a3, pw[g][0], pw[g][1]);
      }
    }
    if (kCodes) {
      __syncwarp();  // everyone has read the tile
      if (k + kAhead < k_end) fetch(k + kAhead, page);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    if (!kCodes && mend) {
#pragma unroll
      for (int g = 0; g < NT; ++g)
        for (int x = 0; x < kBN && s0 + x < end; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = g * 8 + 2 * c + e;
            const bool sees_it = sees(a.mode, a.sinks, s_low[r], ctx, rows_n, s_i[r],
                                      mask ? mask + (int64_t)s_i[r] * a.rows.max_q : nullptr, s0 + x);
#pragma unroll
            for (int d = 0; d < 8 * JJ; ++d) {
              const int col = 64 * (d >> 3) + 8 * n + (d & 7);
              const float v = col < a.D ? __bfloat162float(((const __nv_bfloat16*)a.v)[here + (int64_t)x * a.ss + col]) : 0.0f;
              if (sees_it && !isfinite(v)) o[g][(d >> 3) * 4 + ((d & 7) >> 1)][(d & 1) * 2 + e] += v;
            }
          }
    }
  }

  if (kCodes) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  }
  // The warps' results, in shared memory.
#pragma unroll
  for (int g = 0; g < NT; ++g)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = g * 8 + 2 * c + e;
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[g][e] += __shfl_xor_sync(0xffffffffu, l[g][e], d);
      if (kCodes) {
        // Both relative to one point, kRoom above the logarithm of l (which is 1 at least where a slot counts at all). The factor
        // of o may be below fp32's range where the result is not.
        const float to = ms[g][e] + (kRoom + (float)((int)(__float_as_uint(l[g][e]) >> 23) - 127)), by = ms[g][e] - to;
        const float half = l[g][e] == 0.0f ? 1.0f : ex2(0.5f * (m[g][e] + by));
        m[g][e] = l[g][e] == 0.0f ? -INFINITY : to;
        l[g][e] *= ex2(by);
#pragma unroll
        for (int t = 0; t < 4 * JJ; ++t) {
          o[g][t][e] = o[g][t][e] * half * half;
          o[g][t][2 + e] = o[g][t][2 + e] * half * half;
        }
      }
      if (n == 0) s_ml[warp][r] = make_float2(m[g][e], l[g][e]);
#pragma unroll
      for (int j = 0; j < JJ; ++j) {
        float* dst = s_o(warp, r, 64 * j + 8 * n);
        *(float4*)dst = make_float4(o[g][4 * j][e], o[g][4 * j][2 + e], o[g][4 * j + 1][e], o[g][4 * j + 1][2 + e]);
        *(float4*)(dst + 4) = make_float4(o[g][4 * j + 2][e], o[g][4 * j + 2][2 + e], o[g][4 * j + 3][e], o[g][4 * j + 3][2 + e]);
      }
    }
  __syncthreads();
  const int64_t tile = (int64_t)b * a.hkv + h;
  auto finish = [&](int r, int e, float4 x, float mm, float ll) {
    const int i = r / G;
    const int64_t row = (int64_t)(q0 + i) * a.hq + h * G + (r - i * G);
    const float inv = ll > 0.0f ? 1.0f / ll : (ll == 0.0f ? 0.0f : NAN);
    *(uint2*)((__nv_bfloat16*)a.out + row * a.D + e) = make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
    if (e == 0 && a.lse) a.lse[row] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
  };
  for (int x = threadIdx.x; x < rows * (DP / 4); x += kThr) {
    const int r = x / (DP / 4), e = (x - r * (DP / 4)) * 4;
    if (e >= a.D) continue;  // a piece's rows lie head_dim apart in the workspace
    float mm = -INFINITY, ll = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_ml[w][r].x);
    float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 v = s_ml[w][r];
      const float4 y = *(const float4*)s_o(w, r, e);
      const float f = v.x == -INFINITY || v.x == mm ? 1.0f : ex2(v.x - mm);  // a warp that saw nothing has sums of 0
      ll += v.y * f;
      acc.x += y.x * f; acc.y += y.y * f; acc.z += y.z * f; acc.w += y.w * f;
    }
    if (used == 1) {
      finish(r, e, acc, mm, ll);
    } else {
      const int64_t at = (tile * p.splits + split) * kRows + r;
      *(float4*)(p.part.o + at * a.D + e) = acc;
      if (e == 0) p.part.ml[at] = make_float2(mm, ll);
    }
  }
  if (used == 1) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    s_last = atomicAdd(p.part.arrived + tile, 1u) == (unsigned)used - 1u;
    if (s_last) p.part.arrived[tile] = 0u;  // ready for the next call
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // A thread has up to kX groups of four columns, in rows that are kThr / (DP / 4) apart: one pass over the
  // pieces in order, kU in flight for every group, the maximum raised as they come.
  constexpr int kX = kRows * (DP / 4) / kThr, kApart = kThr / (DP / 4), kU = kX > 2 ? 4 : 8;
  const int e = (threadIdx.x % (DP / 4)) * 4, r0 = threadIdx.x / (DP / 4);
  if (e >= a.D) return;
  float mm[kX], ll[kX];
  float4 acc[kX];
#pragma unroll
  for (int x = 0; x < kX; ++x) {
    mm[x] = -INFINITY;
    ll[x] = 0.0f;
    acc[x] = make_float4(0, 0, 0, 0);
  }
  for (int s = 0; s < used; s += kU) {
    float2 ml[kX][kU];
    float4 y[kX][kU];
#pragma unroll
    for (int x = 0; x < kX; ++x)
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        ml[x][u] = make_float2(-INFINITY, 0.0f);
        if (s + u < used && r0 + x * kApart < rows) {
          const int64_t at = (tile * p.splits + s + u) * kRows + r0 + x * kApart;
          ml[x][u] = __ldcg(&p.part.ml[at]);
          y[x][u] = __ldcg((const float4*)(p.part.o + at * a.D + e));
        }
      }
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      float now = mm[x];
#pragma unroll
      for (int u = 0; u < kU; ++u) now = fmaxf(now, ml[x][u].x);
      const float keep = now == mm[x] || mm[x] == -INFINITY ? 1.0f : ex2(mm[x] - now);
      ll[x] *= keep;
      acc[x].x *= keep; acc[x].y *= keep; acc[x].z *= keep; acc[x].w *= keep;
      mm[x] = now;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (ml[x][u].x == -INFINITY && ml[x][u].y == 0.0f) continue;  // saw nothing
        const float f = ml[x][u].x == now || ml[x][u].x == -INFINITY ? 1.0f : ex2(ml[x][u].x - now);
        ll[x] += ml[x][u].y * f;
        acc[x].x += y[x][u].x * f; acc[x].y += y[x][u].y * f; acc[x].z += y[x][u].z * f; acc[x].w += y[x][u].w * f;
      }
    }
  }
#pragma unroll
  for (int x = 0; x < kX; ++x)
    if (r0 + x * kApart < rows) finish(r0 + x * kApart, e, acc[x], mm[x], ll[x]);
}

int64_t resident() { return 2 * (int64_t)num_sms(); }
int64_t want_ctas() { return kWaves * resident(); }
static_assert(2 * kWaves <= kCountersPerSm, "a counter for every tile that is cut");

template <int NT, int KS, int JJ, int CACHE>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
  RowsP p;
  p.a = a;
  p.c = a.scale * kLog2e;
  const int64_t key_tiles = ((int64_t)a.rows.max_ctx + a.rows.max_q) / kBN, row_tiles = (int64_t)a.hkv * a.rows.batch;
  const bool many = row_tiles >= kManyTiles;
  p.least = many ? kLeastMany : kLeast;
  p.splits = splits_for(row_tiles, many ? want_ctas() : resident(), std::min<int64_t>(key_tiles / p.least, kMostPieces));
  p.part = partials_at(a.scratch, want_ctas(), 16);
  const dim3 grid((unsigned)p.splits, (unsigned)a.hkv, (unsigned)a.rows.batch);
  size_t smem = 0;
  if (CACHE == kPagedE4m3) {
    smem = (size_t)kWarps * std::max(kDepth * Tile<JJ>::kBytes, 8 * NT * (64 * JJ + 4) * 4);
    static FuncOnce once;
    const cudaError_t e = once.set((const void*)attn_rows_kernel<NT, KS, JJ, CACHE>, (int)smem, false);
    if (e != cudaSuccess) return e;
  }
  attn_rows_kernel<NT, KS, JJ, CACHE><<<grid, kThr, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

// Up to 8 packed rows it is the faster one or as fast (64 tokens over up to 4000 slots 117 us, the tensor core
// kernel 118; over up to 500 slots 24 and 50). From 9 to 16 its products are twice as many, and with every SM busy over
// long caches the tensor core kernel wins, from pasts of about 2500 on: 64 requests of 4 rows in groups of 4, up to 500 /
// 2000 / 2500 / 3000 / 4000 slots, 31 / 76 / 80 / 96 / 120 us and 47 / 76 / 81 / 92 / 112; 32 requests 18 / 47 / 48 / 55 / 72
// and 28 / 46 / 50 / 54 / 67. Fewer, which leave SMs idle: 16 requests up to 4000 slots 43.7 and 43.1; one 21 and 21.
// Codes, which the tensor core kernel has to turn into bf16 first, are this one's up to 16 rows: 64 requests of 4 rows in groups of 4, up to
// 500 / 2000 / 8000 slots, 30 / 71 / 193 us and 57 / 106 / 270, and 2 rows in groups of 8, 3 in groups of 5, 8 in groups of 2 or 16 rows of
// a head of its own within 3 us of either; 16 requests 15 / 39 / 64 and 27 / 45 / 100. (From 9 rows on two CTAs, 8 warps, run on an SM; the bytes
// of the longest would take 82 us.)
bool attn_rows_applies(const AttnArgs& a) {
  const int64_t rows = (int64_t)a.rows.max_q * (a.hq / a.hkv);
  if (a.dtype != DOMINO_BF16 || a.D > 128 || rows > 16) return false;
  return rows <= 8 || a.cache == kPagedE4m3 || a.rows.max_ctx < 2500 || (int64_t)a.hkv * a.rows.batch <= num_sms();
}
size_t attn_rows_ws_bytes(const AttnArgs& a) { return partial_bytes(want_ctas(), 16, a.D); }

template <int CACHE>
static cudaError_t launch_on(const AttnArgs& a, cudaStream_t stream) {
  const bool many = a.rows.max_q * (a.hq / a.hkv) > 8;
  if (a.D > 64) return many ? launch<2, 4, 2, CACHE>(a, stream) : launch<1, 4, 2, CACHE>(a, stream);
  return many ? launch<2, 2, 1, CACHE>(a, stream) : launch<1, 2, 1, CACHE>(a, stream);
}
cudaError_t launch_attention_rows(const AttnArgs& a, cudaStream_t stream) {
  return a.cache == kWhole ? launch_on<kWhole>(a, stream) : a.cache == kPaged ? launch_on<kPaged>(a, stream)
                                                                             : launch_on<kPagedE4m3>(a, stream);
}

}  // namespace domino
