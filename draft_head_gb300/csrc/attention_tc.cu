// Attention of a block's rows over the cache on the tensor cores
// (domino_block_attention and domino_paged_attention; the definitions are in domino.h): bf16 or
// codes, head_dim <= 128.
//
// One pass over the keys with the running maximum and sum of the softmax. Per key
// tile of 128 slots and query tile of 128 packed rows (row and query head of one kv
// head): S = Q K^T (tcgen05.mma, fp32 in TMEM), a thread per row takes its 128
// scores to registers, P = 2^(S c - m) goes back over S in TMEM as bf16 (the operand's type: the sum that
// divides adds the weights before this rounding, which takes the output's error against 64 bits from 0.0017 to 0.0022 of its
// size), and O += P V with P as the TMEM operand and V as it lies in the cache (slots x head_dim,
// head_dim contiguous: the MN-major operand). P is handed over in two halves, so the first
// half's product runs under the second half's exponentials. (Scores in halves of 64 slots with
// an S each, so that nothing waits for a product, measured slower: an N = 64 MMA takes 48
// cycles, not 32, and every hand-over costs the MMA warp about 150.) O stays in TMEM; it is
// rescaled only when a row's maximum has grown by more than 2^kLazy since the last time: P is
// then up to 2^kLazy, which fp32 sums and bf16 (fp32's exponents) hold without loss.
//
//   warp 0       TMA: key and value tiles into one ring of buffers
//   warp 1       TMEM and the MMAs. The whole warp runs the loop and one elected thread issues:
//                under elect.sync an M = 128, N = 128, K = 16 MMA issues every 64 cycles (the
//                full rate), from a branch on the lane number every 120 to 220 (measured)
//   warps 2, 3   query tiles, one row tile ahead; clear non-finite values of tiles that some
//                row does not see (both count in every barrier that they signal: the parity wait of a
//                warp that did not could miss a phase)
//   warps 4-7, 8-11  two groups of 128 threads: softmax and epilogue
//
// NQ = 2 (prompts): bound by the exponentials and the MMAs. Each group has a query tile of
// its own; both read the same key and value buffers and take turns: one's MMAs run under the
// other's softmax.
// NQ = 1 (few rows: one token, a draft block, a tree): bound by the cache's bytes. The groups
// take the key tiles of one query tile in turn, each with its own maximum, sum and O, which the
// epilogue joins.
//
// The work is the list of all (request, row tile, kv head, key tile), cut into equal pieces, one
// per CTA of a grid of one CTA per SM; lengths live on the device, so every CTA counts the list
// itself. Every (request, row tile, kv head) counts kItem key tiles more, about what its start and
// its epilogue cost. A row tile cut over CTAs is joined by the last of them to finish, in piece
// order, from fp32 sums in the workspace: the result does not depend on the order of arrival.
//
// 32 query heads of 128 over 8: draft blocks of 16 rows for 64 requests over up to 8000 slots with a
// window of 4096: 173 us, 5.4 TB/s; trees of 17 rows for 16 requests over up to 6000 slots: 64 us, 3.7
// TB/s; two prompts of 8192 rows with a window of 2048:
// 449 us, 1.05 PFLOP/s of seen pairs; one prompt of 16,384 rows: 1.48 ms, 1.49 PFLOP/s. In prompts the
// tensor pipe is busy 43 % of the time in a short call (4096 rows with the window); a softmax group's own path
// (scores to registers, exponentials, weights back) sets the pace. A polynomial on the FMA pipe for part
// of the exponentials made it longer (a quarter of them: 450 -> 537 us).
//
// Pages: warp 0 reads the table a tile ahead and brings a tile page by page. Codes (e4m3 with a power of two per slot and head)
// arrive in buffers of their own, and
//   warps 12-15  turn them into bf16 in the ring: code x scale is exact there (4 significant bits), so all that follows is the
//                same. A code's fields at bf16's places are 2^-120 of it, and one product with the scale does the rest.
// They share the SM's issue slots and shared memory with the softmax, and set the pace where the cache's bytes would: 64
// blocks over pages of 64 slots 229 us (bf16 pages 169, of 16 slots 201, 256 181), 16 trees 85 us (66), chunks of 2048 rows for 4 requests
// 473 us (400), 0.99 PFLOP/s. With the conversion left out, a copy in its place, they took 200, 77 and 463 (the chunks 490 then): it is the
// passes through shared memory, not the arithmetic, that cost. (Products of codes as fp16 with scales relative to a tile's largest: 210, 79 and 502, and
// small scales beside large ones would lose bits. Keys by two of the warps and values by the other two: 244, 90 and 654.)
#include <cuda.h>
#include <math.h>
#include <string.h>
#include <algorithm>
#include <mutex>

#include "attention.cuh"
#include "packed.cuh"
#include "pages.cuh"
#include "waits.cuh"

namespace domino {

namespace {

constexpr int kBN = 128;   // slots of a key tile
constexpr int kHalf = 64;  // and of the halves in which the weights are handed over
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 32.0f;  // growth of the maximum (log2) that forces a rescale of O
// A weight's logarithm is one multiply-add, score x c - m, with m the maximum's product with c as it is rounded, half a unit of its last
// place off: 32 at most below this. From here on that could be more than the exponential holds, and scores that differ at all
// differ by 2^6 there: c is replaced by the power of two at or below it, whose products are exact (and by which they differ by 2^5).
constexpr float kExactFrom = 1073741824.0f;  // 2^30
constexpr int kBadRing = 8;    // items the roles may be apart, at most (the ring holds fewer tiles)

struct TcAttnP {
  CUtensorMap tmK, tmV, tmQ, tmO;
  int q_boxes;    // 1: a query tile is one box of tmQ (the group divides 128)
  int o_boxes;    // 1: 32 packed rows of the output are one box of tmO (it divides 32)
  AttnArgs a;
  int row_tiles;  // per request, of 128 NQ packed rows
  int slots;      // ring buffers
  int staged;     // codes: buffers in which they arrive
  int folded;     // pages: tmK and tmV are of whole heads (make_pages_tmap)
  int64_t page_step, head_step;  // pages: their places along the last axis of tmK and tmV, and the first place behind it
  int no_page;
  uint64_t timeout_ns;
  float c;        // scale log2(e)
  float c_exact;  // the power of two at or below it
  unsigned int* arrived;  // per CTA: pieces in, of the row tile that begins in it and goes on
  float2* ml;             // [2 grid][128 NQ]
  float4* o;              // [2 grid][NQ][DP / 4][128]: four columns of a row, rows next to each other
};

// A row tile of one request: its rows and the slots they see. `cnt` is 0 when it has
// no rows.
struct Unit {
  int q0, n, ctx, r0, rows, i_first, i_last, low_min, low_max, cnt;
  KeyTiles kt;
};

template <int BMT>
__device__ __forceinline__ Unit load_unit(const AttnArgs& a, int row_tiles, int u, bool report) {
  Unit w;
  w.cnt = 0;
  const int b = u / row_tiles, tile = u - b * row_tiles, G = a.hq / a.hkv;
  if (!request_rows(a.rows, b, w.q0, w.n, w.ctx, report, a.ctl)) return w;
  w.r0 = tile * BMT;
  w.rows = min(BMT, w.n * G - w.r0);
  if (w.rows <= 0) return w;
  w.i_first = w.r0 / G;
  w.i_last = (w.r0 + w.rows - 1) / G;
  if (a.window == 0) {
    w.low_min = w.low_max = 0;
  } else if (a.rows.positions) {
    w.low_min = 0x7fffffff;
    w.low_max = 0;
    for (int i = w.i_first; i <= w.i_last; ++i) {
      const int low = window_low(__ldg(a.rows.positions + w.q0 + i), a.window);
      w.low_min = min(w.low_min, low);
      w.low_max = max(w.low_max, low);
    }
  } else {
    w.low_min = window_low(w.ctx + w.i_first, a.window);
    w.low_max = window_low(w.ctx + w.i_last, a.window);
  }
  w.kt = key_tiles(a.mode, a.sinks, w.low_min, w.ctx, w.n, w.i_last, kBN);
  // Rows that see nothing at all take a key tile, masked whole, on the way to their output of 0 and lse of -inf.
  if (w.kt.count == 0) w.kt.main_begin = 0, w.kt.main_count = w.kt.count = 1;
  w.cnt = w.kt.count;
  return w;
}

// Whether every row of the tile sees every slot of the key tile at s0.
__device__ __forceinline__ bool all_seen(const AttnArgs& a, const Unit& w, int s0) {
  const int hi = a.mode == DOMINO_MASK_CAUSAL ? w.ctx + w.i_first + 1 : a.mode == DOMINO_MASK_FULL ? w.ctx + w.n : w.ctx;
  const int low = a.mode == DOMINO_MASK_CAUSAL ? w.low_max : min(w.low_max, w.ctx);
  return s0 + kBN <= hi && (s0 >= low || s0 + kBN <= a.sinks);
}

// A bounded wait that all lanes of a warp leave together, with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* s_abort, Ctl* ctl, uint64_t timeout_ns) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, s_abort, ctl, timeout_ns));
}
// Barrier of N threads that tells all of them whether every one was `ok`.
template <int N>
__device__ __forceinline__ bool group_all(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.and.pred q, %1, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)ok), "n"(N)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e != 0;
}

// The CTA's part of the work list, walked by every role alike.
template <int kItem>
struct Walk {
  int u, h, k, len;
  int64_t x;  // place in the list
  // Key tiles [k0, k1) of the row tile are the CTA's (may be none).
  __device__ __forceinline__ void part(int cnt, int& k0, int& k1) const {
    k0 = max(0, k - kItem);
    k1 = max(0, k + min(len, cnt + kItem - k) - kItem);
  }
  __device__ __forceinline__ void next(int cnt, int hkv) {
    const int piece = min(len, cnt + kItem - k);
    len -= piece;
    x += piece;
    k += piece;
    if (k == cnt + kItem) {
      k = 0;
      if (++h == hkv) {
        h = 0;
        ++u;
      }
    }
  }
};

__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};\n" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, int x, int s, int h, int b, uint64_t* bar,
                                            uint64_t policy, bool hint) {
  if (hint)
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
        "l"((uint64_t)tmap), "r"(x), "r"(s), "r"(h), "r"(b), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"((uint64_t)tmap), "r"(x), "r"(s), "r"(h), "r"(b), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"((uint64_t)tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const void* tmap, int x, int y, int z, const void* src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"((uint64_t)tmap), "r"(x),
               "r"(y), "r"(z), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void tma_load_5d(void* dst, const void* tmap, int x, int y, int z, int u, int v, uint64_t* bar,
                                            uint64_t policy, bool hint) {
  if (hint)
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(smem_u32(dst)),
        "l"((uint64_t)tmap), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"((uint64_t)tmap), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(smem_u32(bar))
        : "memory");
}
// How a key or value tile's atoms (8 slots of 64 elements, 1024 bytes) lie: from one to that of the next 8 slots, and to
// that of the next 64 elements.
struct Atoms {
  uint32_t slots, elements;
};
// Shared-memory descriptor of an MN-major operand with 128-byte swizzle: rows of 64
// elements of N, 8 rows (of K) per 1024-byte atom; the next 8 rows follow at the
// stride offset, the next 64 elements of N at the leading offset.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, Atoms at) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(at.elements >> 4) << 16) | ((uint64_t)(at.slots >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// The same of a K-major one, whose leading offset is unused.
__device__ __forceinline__ uint64_t sdesc_k_atoms(uint32_t saddr, Atoms at) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(at.slots >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
__device__ __forceinline__ bool bad16(uint32_t x) {  // a bf16 pair with an infinity or a NaN in it
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t clear16(uint32_t x) {
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
  return x;
}

// The page of the `n` slots from s0 + x on, which lie in one, of the key tile at s0: -1 for one that is not there, -2 where the row tile
// looks at none of them.
constexpr int kLeastPage = 16;
__device__ __forceinline__ int tile_page(const AttnArgs& a, const Unit& w, int b, int s0, int x, int n) {
  const int end = a.mode == DOMINO_MASK_CAUSAL ? w.ctx + w.i_last + 1 : w.ctx + w.n, s = s0 + x;
  const bool needed = x < kBN && s < end && (s < a.sinks || s + n > first_slot(a.mode, w.low_min, w.ctx, end));
  return needed ? page_of(a.pages, b, s) : -2;
}

// Codes: what goes with a tile to those who turn it into bf16.
constexpr uint32_t kNotePlain = 1, kNoteClean = 2, kNoteEnd = 4;  // all scales take one factor; values that some row does not see; no tile
constexpr int kNoteItem = 3;                                      // from this bit on: the row tile's number
constexpr uint32_t kSecondFactor = 0xffff0000u;  // with a scale's byte: it takes two factors, or is NaN

// Visibility of the 128 slots from s0 for one row, as bits.
__device__ __forceinline__ void seen_bits(const AttnArgs& a, const Unit& w, int i, int low, const uint8_t* mask_row, int s0,
                                          uint32_t (&bits)[4]) {
  const int end = a.mode == DOMINO_MASK_CAUSAL ? w.ctx + i + 1 : a.mode == DOMINO_MASK_FULL ? w.ctx + w.n : w.ctx;
  const int from = a.mode == DOMINO_MASK_CAUSAL ? low : min(low, w.ctx);
  auto below = [&](int x, int word) -> uint32_t {  // slots of the word below slot x
    const int d = x - (s0 + word * 32);
    return d <= 0 ? 0u : d >= 32 ? 0xffffffffu : (1u << d) - 1u;
  };
#pragma unroll
  for (int j = 0; j < 4; ++j) bits[j] = (~below(from, j) | below(a.sinks, j)) & below(end, j);
  if (a.mode == DOMINO_MASK_TREE) {
    const int j0 = max(0, s0 - w.ctx), j1 = min(w.n, s0 + kBN - w.ctx);
    for (int j = j0; j < j1; ++j) {
      const int at = w.ctx + j - s0;
      const uint32_t bit = __ldg(mask_row + j) ? 1u << (at & 31) : 0u;
#pragma unroll
      for (int q = 0; q < 4; ++q) bits[q] |= (at >> 5) == q ? bit : 0u;
    }
  }
}

// Adds the non-finite values that the row sees in the piece's partly seen tiles to columns [e0, e1) of its
// result in memory (bf16 `out`, or the piece's sums `sums`): the tiles had them cleared, because the product
// with V would have spread them to the rows that do not see them.
template <int CACHE>
__device__ __noinline__ void add_non_finite(const AttnArgs& a, const Unit& w, int b, int h, int k0, int k1, int i, int low,
                                            const uint8_t* mask_row, int e0, int e1, __nv_bfloat16* out, float4* sums) {
  for (int k = k0; k < k1; ++k) {
    const int s0 = w.kt.slot(k, kBN);
    if (all_seen(a, w, s0)) continue;
    uint32_t bits[4];
    seen_bits(a, w, i, low, mask_row, s0, bits);
    for (int j = 0; j < kBN; ++j) {
      const uint32_t word = j < 32 ? bits[0] : j < 64 ? bits[1] : j < 96 ? bits[2] : bits[3];
      if (!((word >> (j & 31)) & 1u)) continue;
      const int page = CACHE == kWhole ? 0 : page_of(a.pages, b, s0 + j);
      if (page < 0) continue;
      const int64_t row = CACHE == kWhole
                              ? (int64_t)b * a.rs + (int64_t)h * a.hs + (int64_t)(s0 + j) * a.ss
                              : (int64_t)page * a.pages.page_stride + (int64_t)h * a.hs + (int64_t)slot_in_page(a.pages, s0 + j) * a.ss;
      Scale2 scale = {0, 0};
      if (CACHE == kPagedE4m3) scale = scale_bf16(a.pages.v_scale[scale_at(a.pages, a.hkv, page, h, s0 + j)]);
      for (int e = e0; e < e1 && e < a.D; ++e) {
        uint32_t x;
        if (CACHE == kPagedE4m3) {
          x = codes8_bf16(make_uint2(((const uint8_t*)a.v)[row + e], 0), scale).x & 0xffffu;
        } else {
          x = ((const uint16_t*)a.v)[row + e];
        }
        if ((x & 0x7f80u) != 0x7f80u) continue;
        if (out)
          out[e] = __float2bfloat16(__bfloat162float(out[e]) + __uint_as_float(x << 16));
        else
          ((float*)(sums + (e >> 2) * 128))[e & 3] += __uint_as_float(x << 16);
      }
    }
  }
}

template <int NQ, int KB, int CACHE>
struct Cfg {
  static constexpr int DP = 64 * KB;
  static constexpr bool kCodes = CACHE == kPagedE4m3;
  static constexpr uint32_t kStaged = (uint32_t)kBN * DP;  // bytes of a tile of codes
  static constexpr int kThreads = kCodes ? 512 : 384;
  // Registers: launched with 65,536 / kThreads a thread; the softmax's 8 warps take kMore, the others keep kLess
  // (256 x 208 + 128 x 88 = 64,512 = 384 x 168; 256 x (200 + 56) = 256 x (192 + 64) = 65,536: over codes chunks take 474 us with
  // 200 and 489 with 192, 64 blocks 229 and 241, 16 trees 84 and 85).
  static constexpr int kMore = kCodes ? 200 : 208, kLess = kCodes ? 56 : 88;
  static constexpr int BMT = 128 * NQ;
  // List places of a row tile beside its key tiles: its start and epilogue take about 11,000 cycles, a key
  // tile 2,000 (NQ = 1) or 3,200. Two more than that for prompts measured best (2: 497 us, 6: 465, 8: 450,
  // 10: 460 for two prompts of 8192 rows with a window; 64 blocks 195 us at 2 and 169 at 6).
  static constexpr int kItem = NQ == 1 ? 6 : 8;
  static constexpr uint32_t kTile = (uint32_t)KB * kBN * 128;    // bytes of a key or value tile
  static constexpr uint32_t kQBytes = (uint32_t)KB * 128 * 128;  // bytes of a query tile
  static constexpr uint32_t kStage = NQ == 2 ? 8 * 4096 : 0;     // output on its way out
};
constexpr uint32_t kOCol = 256;  // TMEM: S of group g at 128 g, O of group g at kOCol + DP g

template <int NQ, int KB, int CACHE>
__global__ void __launch_bounds__(Cfg<NQ, KB, CACHE>::kThreads, 1) attn_tc_kernel(const __grid_constant__ TcAttnP p) {
  using C = Cfg<NQ, KB, CACHE>;
  constexpr int kThreads = C::kThreads;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* ring = sQ + NQ * C::kQBytes;
  const int slots = p.slots;
  uint8_t* stage = ring + (size_t)slots * C::kTile;  // NQ = 2: 4 KB per softmax warp
  // The buffers that copies fill, `full` once they have: the ring's own, or codes on their way to it.
  const int in_slots = C::kCodes ? p.staged : slots;
  uint8_t* in = C::kCodes ? stage + C::kStage : ring;
  uint32_t* in_factors = (uint32_t*)(in + (C::kCodes ? (size_t)in_slots * C::kStaged : 0));  // codes: [in_slots][kBN] factors
  volatile uint32_t* in_notes = in_factors + (C::kCodes ? in_slots * kBN : 0);                // and [8] notes
  uint64_t* full = C::kCodes ? (uint64_t*)(in_notes + 8) : (uint64_t*)(stage + C::kStage);
  uint64_t* empty = full + in_slots;
  // The ring's: keys ready, values ready, buffers read.
  uint64_t* v_clean = empty + in_slots;
  uint64_t* k_ready = C::kCodes ? v_clean : full;
  uint64_t* freed = C::kCodes ? v_clean + slots : empty;
  uint64_t* s_ready = (C::kCodes ? freed : v_clean) + slots;  // [2]: per group
  uint64_t* p_ready = s_ready + 2;      // [4]: per group and half
  uint64_t* o_done = p_ready + 4;       // [2]: per group, once per row tile
  uint64_t* q_ready = o_done + 2;
  uint64_t* q_free = q_ready + 1;
  uint64_t* drain = q_free + 1;
  int64_t* s_prefix = (int64_t*)(drain + 1);
  int64_t* s_scan = s_prefix + 1;       // [kThreads / 32]
  float2* s_ml = (float2*)(s_scan + kThreads / 32);  // [2][128] NQ = 1: the groups' (m, l)
  int* s_unit = (int*)(s_ml + (NQ == 1 || !C::kCodes ? 256 : 0));
  int* s_cnt = s_unit + 1;
  int* s_last = s_cnt + 1;              // [2]
  volatile int* s_bad = s_last + 2;     // [2][kBadRing]
  uint32_t* tmem_slot = (uint32_t*)(s_last + 2 + 2 * kBadRing);
  volatile int* s_abort = (volatile int*)(tmem_slot + 1);

  const AttnArgs& a = p.a;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int hkv = a.hkv, G = a.hq / a.hkv;
  Ctl* ctl = a.ctl;

  if (threadIdx.x == 0) {
    for (int s = 0; s < in_slots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::kCodes ? 4 : 1);
    }
    for (int s = 0; s < slots; ++s) {
      mbar_init(&v_clean[s], C::kCodes ? 4 : 2);
      if (C::kCodes) mbar_init(&freed[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_ready[s], 1);
      mbar_init(&p_ready[2 * s], 4);
      mbar_init(&p_ready[2 * s + 1], 4);
      mbar_init(&o_done[s], 1);
    }
    mbar_init(q_ready, 2);
    mbar_init(q_free, 1);
    mbar_init(drain, 1);
    *s_abort = 0;
    for (int i = 0; i < 2 * kBadRing; ++i) s_bad[i] = 0;
    mbar_fence_init();
    tma_prefetch_desc(&p.tmK);
    tma_prefetch_desc(&p.tmV);
    if (p.q_boxes) tma_prefetch_desc(&p.tmQ);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // Columns of the query tiles past head_dim stay zero.
  if (a.D < C::DP) {
    for (uint32_t x = threadIdx.x; x < NQ * C::kQBytes / 16; x += kThreads) ((uint4*)sQ)[x] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }

  // Count the work list (places of one kv head) and find this CTA's part of it.
  auto places = [](const Unit& w) { return w.cnt > 0 ? w.cnt + C::kItem : 0; };
  const int units = a.rows.batch * p.row_tiles;
  const int chunk = (units + kThreads - 1) / kThreads;
  const int u_begin = min(units, (int)threadIdx.x * chunk), u_end = min(units, u_begin + chunk);
  int64_t mine = 0;
  int last_places = 0;
  for (int u = u_begin; u < u_end; ++u) {
    last_places = places(load_unit<C::BMT>(a, p.row_tiles, u, blockIdx.x == 0 && u % p.row_tiles == 0));
    mine += last_places;
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t s = s_scan[w];
    before += w < warp ? s : 0;
    total += s;
  }
  before += incl - mine;
  const int64_t list = total * hkv;
  // CTAs with work: no more than places, so that none of them is empty.
  const int ctas = (int)min((int64_t)gridDim.x, max(list, (int64_t)1));
  const bool idle = (int)blockIdx.x >= ctas || list == 0;
  const int64_t x0 = idle ? 0 : list * blockIdx.x / ctas, x1 = idle ? 0 : list * (blockIdx.x + 1) / ctas;
  if (!idle && mine > 0 && before <= x0 / hkv && x0 / hkv < before + mine) {
    int64_t at = before;
    for (int u = u_begin; u < u_end; ++u) {
      const int c = u + 1 == u_end ? last_places : places(load_unit<C::BMT>(a, p.row_tiles, u, false));
      if (x0 < (at + c) * hkv) {
        *s_unit = u;
        *s_cnt = c;
        *s_prefix = at;
        break;
      }
      at += c;
    }
  }
  __syncthreads();
  Walk<C::kItem> walk;
  walk.len = (int)(x1 - x0);
  walk.x = x0;
  walk.u = 0; walk.h = 0; walk.k = 0;
  if (walk.len > 0) {
    walk.u = *s_unit;
    const int c = *s_cnt;
    const int64_t in = x0 - *s_prefix * hkv;
    walk.h = (int)(in / c);
    walk.k = (int)(in - (int64_t)walk.h * c);
  }

  if (warp < 4 || warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kLess));
    if (C::kCodes && warp >= 12) {
      // Keys and values from codes to bf16, exactly: 16 codes of a slot at a time, swizzled as the MMA reads them. What these warps
      // need to know of a tile comes with it, so that nothing else takes their registers.
      constexpr int kPer = C::DP / 16, kRows = 128 / kPer;  // pieces of a slot, slots at a time (whole swizzle atoms)
      const int piece = (threadIdx.x & 127) % kPer, r0 = (threadIdx.x & 127) / kPer;
      // A piece is two units of 16 bytes; neighbours of the other half of the head begin with the second one, so that eight
      // threads reach all banks.
      const int odd = KB == 2 ? piece >> 2 : 0, unit = (piece & 3) * 2, sw = r0 & 7;
      const uint32_t src0 = (uint32_t)(r0 * C::DP + piece * 16);
      const uint32_t dst0 = (uint32_t)((piece >> 2) * (kBN * 128) + r0 * 128 + (((unit + odd) ^ sw) << 4));
      const uint32_t dst1 = (uint32_t)((piece >> 2) * (kBN * 128) + r0 * 128 + (((unit + 1 - odd) ^ sw) << 4));
      int from = 0, to = 0;  // the buffer that codes are in, and the one that they go to
      uint32_t from_phase = 0, to_phase = 0;
      while (warp_wait(&full[from], from_phase, s_abort, ctl, p.timeout_ns)) {
        const uint32_t note = in_notes[from];
        if (note & kNoteEnd) break;
        if (!warp_wait(&freed[to], to_phase ^ 1u, s_abort, ctl, p.timeout_ns)) break;
        const uint8_t* src = in + (size_t)from * C::kStaged + src0;
        const uint32_t* factor = in_factors + from * kBN + r0;
        uint8_t* dst = ring + (size_t)to * C::kTile;
        if (note & kNotePlain) {
          constexpr int kU = 4;
#pragma unroll 1
          for (int i0 = 0; i0 < kBN / kRows; i0 += kU) {
            uint4 x[kU];
            uint32_t f[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
              x[u] = *(const uint4*)(src + (i0 + u) * (kRows * C::DP));
              f[u] = factor[(i0 + u) * kRows];
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
              const uint2 y[4] = {codes_bf16(x[u].x, f[u]), codes_bf16(x[u].y, f[u]), codes_bf16(x[u].z, f[u]), codes_bf16(x[u].w, f[u])};
              const uint4 y0 = make_uint4(y[0].x, y[0].y, y[1].x, y[1].y), y1 = make_uint4(y[2].x, y[2].y, y[3].x, y[3].y);
              *(uint4*)(dst + dst0 + (i0 + u) * (kRows * 128)) = odd ? y1 : y0;
              *(uint4*)(dst + dst1 + (i0 + u) * (kRows * 128)) = odd ? y0 : y1;
            }
          }
        } else {
          bool bad = false;
#pragma unroll 1
          for (int i = 0; i < kBN / kRows; ++i) {
            const uint4 x = *(const uint4*)(src + i * (kRows * C::DP));
            const uint32_t f = factor[i * kRows];
            const Scale2 scale = f >= kSecondFactor ? scale_bf16((int)(f & 255u)) : Scale2{f, 0};
            uint4 y[2] = {codes8_bf16(make_uint2(x.x, x.y), scale), codes8_bf16(make_uint2(x.z, x.w), scale)};
            if (note & kNoteClean) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                bad |= bad16(y[e].x) | bad16(y[e].y) | bad16(y[e].z) | bad16(y[e].w);
                y[e] = make_uint4(clear16(y[e].x), clear16(y[e].y), clear16(y[e].z), clear16(y[e].w));
              }
            }
            *(uint4*)(dst + dst0 + i * (kRows * 128)) = odd ? y[1] : y[0];
            *(uint4*)(dst + dst1 + i * (kRows * 128)) = odd ? y[0] : y[1];
          }
          if (bad) {
            s_bad[(note >> kNoteItem) & (kBadRing - 1)] = 1;
            s_bad[kBadRing + ((note >> kNoteItem) & (kBadRing - 1))] = 1;
            __threadfence_block();
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&empty[from]);
          mbar_arrive(&v_clean[to]);
        }
        if (++from == in_slots) { from = 0; from_phase ^= 1u; }
        if (++to == slots) { to = 0; to_phase ^= 1u; }
      }
    } else if (CACHE != kWhole && warp == 0) {
      // Pages: the whole warp walks the list and one elected lane issues (from a branch on the lane number a copy takes about
      // 280 cycles: 64 blocks over pages of 16 slots 415 us). Lane i has the number of a tile's i-th page, read a tile ahead.
      // Codes: the lane has the scales of slots 4 lane .. 4 lane + 3 of the tile's keys and values too, read a tile ahead, the
      // number of their page two tiles ahead; 2^0 where no row looks.
      const uint64_t pol = l2_policy_evict_first();
      const bool once = p.row_tiles == 1, leader = elect_one();
      const int shift = min(a.pages.shift, 7);
      int slot = 0;
      uint32_t phase = 0, item = 0;
      long issued = 0;
      bool ok = true;
      Unit w;
      int cur = -1;
      while (walk.len > 0 && walk.u < units && ok) {
        if (walk.u != cur) w = load_unit<C::BMT>(a, p.row_tiles, cur = walk.u, false);
        if (w.cnt == 0) { ++walk.u; continue; }
        const int b = walk.u / p.row_tiles;
        int k0, k1;
        walk.part(w.cnt, k0, k1);
        int page = k0 < k1 ? tile_page(a, w, b, w.kt.slot(k0, kBN), lane << shift, 1 << shift) : -2;
        uint32_t scales[2] = {}, scales_next[2] = {};
        int scale_page = -2;
        auto scales_at = [&](int k, int in_page, uint32_t (&x)[2]) {
          const int64_t at = in_page < 0 ? 0 : scale_at(a.pages, hkv, in_page, walk.h, w.kt.slot(k, kBN) + 4 * lane);
          x[0] = in_page < 0 ? 0x7f7f7f7fu : __ldg((const uint32_t*)(a.pages.k_scale + at));
          x[1] = in_page < 0 ? 0x7f7f7f7fu : __ldg((const uint32_t*)(a.pages.v_scale + at));
        };
        if (C::kCodes && k0 < k1) {
          scales_at(k0, tile_page(a, w, b, w.kt.slot(k0, kBN), 4 * lane, 4), scales_next);
          if (k0 + 1 < k1) scale_page = tile_page(a, w, b, w.kt.slot(k0 + 1, kBN), 4 * lane, 4);
        }
        for (int k = k0; k < k1 && ok; ++k) {
          const int s0 = w.kt.slot(k, kBN), at = slot_in_page(a.pages, s0);
          if (page == -1) dev_error(ctl, DEV_ERR_DATA);
          const int place = page < 0 ? p.no_page : (int)(page * p.page_step + walk.h * p.head_step);
          int places[kBN / kLeastPage];
#pragma unroll
          for (int i = 0; i < kBN / kLeastPage; ++i) places[i] = __shfl_sync(0xffffffffu, place, i);
          page = k + 1 < k1 ? tile_page(a, w, b, w.kt.slot(k + 1, kBN), lane << shift, 1 << shift) : -2;
          if (C::kCodes) {
            scales[0] = scales_next[0];
            scales[1] = scales_next[1];
            if (k + 1 < k1) scales_at(k + 1, scale_page, scales_next);
            if (k + 2 < k1) scale_page = tile_page(a, w, b, w.kt.slot(k + 2, kBN), 4 * lane, 4);
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            ok = ok && warp_wait(&empty[slot], phase ^ 1u, s_abort, ctl, p.timeout_ns);
            if (!ok) break;
            const void* tm = kv ? &p.tmV : &p.tmK;
            if (C::kCodes) {
              uint32_t f[4], most = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t byte = (scales[kv] >> (8 * i)) & 255u;
                most = max(most, byte);
                f[i] = byte > 134u ? kSecondFactor | byte : (byte + 120u) * 0x00800080u;
              }
              *(uint4*)(in_factors + slot * kBN + 4 * lane) = make_uint4(f[0], f[1], f[2], f[3]);
              const bool plain = __all_sync(0xffffffffu, most <= 134u);
              if (lane == 0)
                in_notes[slot] = (plain ? kNotePlain : 0u) | (kv && !all_seen(a, w, s0) ? kNoteClean : 0u) |
                                 item << kNoteItem;
              __syncwarp();
            }
            if (leader) {
              mbar_expect_tx(&full[slot], C::kCodes ? C::kStaged : C::kTile);
#pragma unroll
              for (int i = 0; i < kBN / kLeastPage; ++i) {
                if (i << shift >= kBN) break;
                if (C::kCodes) {
                  tma_load_3d(in + (size_t)slot * C::kStaged + (size_t)(i << shift) * C::DP, tm, 0, at, places[i], &full[slot]);
                } else if (KB == 2 && p.folded) {
                  tma_load_5d(ring + (size_t)slot * C::kTile + (size_t)(i << shift) * 256, tm, 0, 0, 0, at / 8, places[i], &full[slot], pol,
                              once);
                } else {
#pragma unroll
                  for (int kb = 0; kb < KB; ++kb)
                    tma_load_3d(ring + (size_t)slot * C::kTile + kb * (kBN * 128) + (size_t)(i << shift) * 128, tm, kb * 64, at, places[i],
                                &full[slot]);
                }
              }
            }
            __syncwarp();
            ++issued;
            if (++slot == in_slots) { slot = 0; phase ^= 1u; }
          }
        }
        walk.next(w.cnt, hkv);
        if (k0 < k1) ++item;
      }
      if (C::kCodes) {  // no more tiles
        ok = ok && warp_wait(&empty[slot], phase ^ 1u, s_abort, ctl, p.timeout_ns);
        if (ok && lane == 0) {
          in_notes[slot] = kNoteEnd;
          mbar_arrive(&full[slot]);
        }
      }
      // The last copies land before the block ends, as below. (The one that was in the end's buffer has been read.)
      for (long j = issued - 1; j >= 0 && j >= issued - in_slots + (C::kCodes && ok ? 1 : 0); --j)
        mbar_land(&full[j % in_slots], (uint32_t)((j / in_slots) & 1), ctl);
    } else if (warp == 0 && lane == 0) {
      const uint64_t pol = l2_policy_evict_first();
      const bool once = p.row_tiles == 1;  // no other row tile reads this cache again
      int slot = 0;
      uint32_t phase = 0;
      long issued = 0;
      bool ok = true;
      Unit w;
      int cur = -1;
      while (walk.len > 0 && walk.u < units && ok) {
        if (walk.u != cur) w = load_unit<C::BMT>(a, p.row_tiles, cur = walk.u, false);
        if (w.cnt == 0) { ++walk.u; continue; }
        const int b = walk.u / p.row_tiles;
        int k0, k1;
        walk.part(w.cnt, k0, k1);
        for (int k = k0; k < k1 && ok; ++k) {
          const int s0 = w.kt.slot(k, kBN);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            if (!mbar_wait(&empty[slot], phase ^ 1u, s_abort, ctl, p.timeout_ns)) { ok = false; break; }
            mbar_expect_tx(&full[slot], C::kTile);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
              tma_load_4d(ring + (size_t)slot * C::kTile + kb * (kBN * 128), kv ? &p.tmV : &p.tmK, kb * 64, s0, walk.h, b,
                          &full[slot], pol, once);
            ++issued;
            if (++slot == slots) { slot = 0; phase ^= 1u; }
          }
        }
        walk.next(w.cnt, hkv);
      }
      // The last copies land before the block ends, also where those who wait for them have given up.
      for (long j = issued - 1; j >= 0 && j >= issued - slots; --j)
        mbar_land(&full[j % slots], (uint32_t)((j / slots) & 1), ctl);
    } else if (warp == 1) {
      const uint32_t id_s = idesc_bf16_f32(128, kBN);
      const uint32_t id_o = idesc_bf16_f32(128, C::DP) | (1u << 16);  // B is MN-major
      const bool leader = elect_one();
      uint32_t item = 0, done[2] = {0, 0};  // key tiles each group has had
      bool ok = true;
      // The ring holds K_0, V_0, K_1, V_1, ...; two cursors over it.
      int ks = 0, vs = 1;
      uint32_t kph = 0, vph = 0;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && warp_wait(bar, parity, s_abort, ctl, p.timeout_ns);
        tc_fence_after();
      };
      auto step = [&](int& s, uint32_t& ph) {
        s += 2;
        if (s >= slots) { s -= slots; ph ^= 1u; }
      };
      const uint32_t q_addr = smem_u32(sQ), ring_addr = smem_u32(ring);
      const Atoms atoms = CACHE == kPaged && KB == 2 && p.folded ? Atoms{KB * 1024, 1024} : Atoms{1024, kBN * 128};
      auto scores = [&](int qt, int g) {  // S_g = Q K^T
        const uint64_t ad = sdesc_k_sw128(q_addr + (uint32_t)qt * C::kQBytes);
        const uint64_t bd = sdesc_k_atoms(ring_addr + (uint32_t)ks * C::kTile, atoms);
        if (leader) {
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16(tmem + (uint32_t)(g * 128), ad + (uint64_t)(kb * (128 * 128 / 16) + 2 * k),
                        bd + (uint64_t)(kb * (atoms.elements / 16) + 2 * k), id_s, (kb | k) ? 1u : 0u);
          umma_commit(&s_ready[g]);
        }
        __syncwarp();
      };
      auto values = [&](int g, bool first, bool last) {  // O_g += P_g V
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          wait(&p_ready[g * 2 + half], done[g] & 1u);
          if (!ok) return;
          const uint64_t bd = sdesc_mn_sw128(ring_addr + (uint32_t)vs * C::kTile + (uint32_t)half * (kHalf / 8) * atoms.slots, atoms);
          if (leader) {
#pragma unroll
            for (int k = 0; k < kHalf / 16; ++k)
              umma_bf16_ts(tmem + kOCol + (uint32_t)(g * C::DP), tmem + (uint32_t)(g * 128 + half * (kHalf / 2) + 8 * k),
                           bd + (uint64_t)(k * (2 * atoms.slots / 16)), id_o, (first && half == 0 && k == 0) ? 0u : 1u);
            if (half == 1 && last) umma_commit(&o_done[g]);
          }
          __syncwarp();
        }
        ++done[g];
      };
      auto release = [&](uint64_t* bar) {
        if (leader) umma_commit(bar);
        __syncwarp();
      };
      Unit w;
      int cur = -1;
      while (walk.len > 0 && walk.u < units && ok) {
        if (walk.u != cur) w = load_unit<C::BMT>(a, p.row_tiles, cur = walk.u, false);
        if (w.cnt == 0) { ++walk.u; continue; }
        int k0, k1;
        walk.part(w.cnt, k0, k1);
        walk.next(w.cnt, hkv);
        const int n = k1 - k0;
        if (n == 0) continue;
        wait(q_ready, item & 1u);
        // A tile's scores go out once the product of the tile before in its S has been issued:
        // NQ = 2: tile t + 1 of both groups after tile t; NQ = 1: tile t + 2 after tile t.
        constexpr int kAhead = NQ == 2 ? 1 : 2;
        for (int t = 0; t < kAhead && t < n && ok; ++t) {
          wait(&k_ready[ks], kph);
          if (!ok) break;
          if (NQ == 2) {
            scores(0, 0);
            scores(1, 1);
          } else {
            scores(0, t);
          }
          if (t + 1 == n) release(q_free);
          release(&freed[ks]);
          step(ks, kph);
        }
        for (int t = 0; t < n && ok; ++t) {
          const bool more = t + kAhead < n;
          wait(&v_clean[vs], vph);  // and so it is full
          if (NQ == 2) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              values(g, t == 0, t + 1 == n);
              if (more && g == 0) wait(&k_ready[ks], kph);
              if (!ok) break;
              if (more) scores(g, g);
            }
          } else {
            const int g = t & 1;
            values(g, t < 2, t + 2 >= n);
            if (more) wait(&k_ready[ks], kph);
            if (!ok) break;
            if (more) scores(0, g);
          }
          if (!ok) break;
          release(&freed[vs]);
          step(vs, vph);
          if (more) {
            if (t + kAhead + 1 == n) release(q_free);
            release(&freed[ks]);
            step(ks, kph);
          }
        }
        ++item;
      }
      // Every MMA issued above has finished before TMEM is freed.
      release(drain);
      mbar_land(drain, 0, ctl);
    } else if (warp >= 2) {
    const int t64 = threadIdx.x - 64;
    int slot = 1;
    uint32_t phase = 0, item = 0, boxes = 0;
    bool ok = true;
    Unit w;
    int cur = -1;
    while (walk.len > 0 && walk.u < units && ok) {
      if (walk.u != cur) w = load_unit<C::BMT>(a, p.row_tiles, cur = walk.u, false);
      if (w.cnt == 0) { ++walk.u; continue; }
      const int h = walk.h;
      int k0, k1;
      walk.part(w.cnt, k0, k1);
      walk.next(w.cnt, hkv);
      if (k0 == k1) continue;
      // The query rows, swizzled as the MMA reads them; the scores before have read theirs. Rows that
      // there are none of hold anything: no other row's result depends on them.
      if (item > 0 && !warp_wait(q_free, (item - 1u) & 1u, s_abort, ctl, p.timeout_ns)) break;
      if (p.q_boxes) {
        // Packed rows of a tile are `G` heads of each of 128 / G rows: one box.
        if (threadIdx.x == 64) {
          ++boxes;
          mbar_expect_tx(q_ready, NQ * C::kQBytes);
#pragma unroll
          for (int g = 0; g < NQ; ++g)
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
              tma_load_3d(sQ + g * C::kQBytes + kb * (128 * 128), &p.tmQ, kb * 64, h * G, w.q0 + w.i_first + g * (128 / G), q_ready);
        } else if (threadIdx.x == 96) {
          // The other warp counts too: a row tile of a key tile or two has all its scores before any value tile is
          // asked of it, and q_free could be two phases on before it has seen the one it waits for.
          mbar_arrive(q_ready);
        }
      } else {
        const int x = t64 & (8 * KB - 1);
        constexpr int kStep = 64 / (8 * KB);
        int r = t64 / (8 * KB), i = (w.r0 + r) / G, gq = w.r0 + r - i * G;
        if (x * 8 < a.D)
          for (; r < w.rows; r += kStep) {
            const __nv_bfloat16* src = (const __nv_bfloat16*)a.q + ((int64_t)(w.q0 + i) * a.hq + h * G + gq) * a.D + x * 8;
            const uint32_t dst = smem_u32(sQ) + (uint32_t)((r >> 7) * C::kQBytes + (x >> 3) * (128 * 128) + (r & 127) * 128 +
                                                           (((x & 7) ^ (r & 7)) << 4));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
            for (gq += kStep; gq >= G; gq -= G) ++i;
          }
        asm volatile("cp.async.wait_all;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(q_ready);
      }
      // Values of tiles that not every row sees: a weight of 0 does not stop an infinity
      // or a NaN in the product, so these are cleared here and the row tile is marked.
      for (int k = k0; k < k1 && !C::kCodes; ++k) {  // codes: whoever turns them into bf16 clears them
        ok = warp_wait(&full[slot], phase, s_abort, ctl, p.timeout_ns);
        if (!ok) break;
        if (!all_seen(a, w, w.kt.slot(k, kBN))) {
          uint4* v = (uint4*)(ring + (size_t)slot * C::kTile);
          bool bad = false;
#pragma unroll 8
          for (uint32_t x = t64; x < C::kTile / 16; x += 64) {
            uint4 y = v[x];
            if (bad16(y.x) | bad16(y.y) | bad16(y.z) | bad16(y.w)) {
              bad = true;
              uint16_t* e = (uint16_t*)&v[x];
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if ((e[j] & 0x7f80u) == 0x7f80u) e[j] = 0;
            }
          }
          if (bad) {
            s_bad[item & (kBadRing - 1)] = 1;
            s_bad[kBadRing + (item & (kBadRing - 1))] = 1;
            __threadfence_block();
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_clean[slot]);
        slot += 2;
        if (slot >= slots) { slot -= slots; phase ^= 1u; }
      }
      ++item;
    }
    if (boxes > 0) mbar_land(q_ready, (boxes - 1u) & 1u, ctl);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kMore));
    const int g = (warp - 4) >> 2;  // group
    const int quarter = warp & 3;   // TMEM lanes this warp reaches
    const int trow = quarter * 32 + lane, r_in = (NQ == 2 ? g * 128 : 0) + trow;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_col = tmem + lanes + (uint32_t)(g * 128);
    const uint32_t o_col = tmem + lanes + kOCol + (uint32_t)(g * C::DP);
    uint8_t* my_stage = stage + (warp - 4) * 4096;
    uint32_t item = 0, tiles = 0, done_items = 0;
    bool ok = true;
    Unit w;
    int cur = -1, i = 0, low = 0;
    bool live = false;
    int64_t row0 = 0;  // this thread's row for kv head 0, in rows of head_dim
    const uint8_t* mask_row = nullptr;
    // NQ = 2: where this lane stores 16 bytes of 8 of its warp's rows (kv head 0), and which there are.
    int out_at[8] = {};  // from the row tile's first row
    uint32_t out_rows = 0;
    while (walk.len > 0 && walk.u < units && ok) {
      const int b = walk.u / p.row_tiles, h = walk.h;
      if (walk.u != cur) {
        w = load_unit<C::BMT>(a, p.row_tiles, cur = walk.u, false);
        if (w.cnt > 0) {
          live = r_in < w.rows;
          const int pr = w.r0 + min(r_in, w.rows - 1);
          i = pr / G;
          row0 = (int64_t)(w.q0 + i) * a.hq + (pr - i * G);
          low = a.window == 0 ? 0 : window_low(a.rows.positions ? __ldg(a.rows.positions + w.q0 + i) : w.ctx + i, a.window);
          mask_row = a.mask ? a.mask + ((int64_t)b * a.rows.max_q + i) * a.rows.max_q : nullptr;
          if (NQ == 2) {
            out_rows = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int r = j * 4 + (lane >> 3);
              const int pq = w.r0 + g * 128 + quarter * 32 + r;
              out_at[j] = ((pq / G - w.i_first) * a.hq + pq % G) * a.D + (lane & 7) * 8;
              out_rows |= g * 128 + quarter * 32 + r < w.rows ? 1u << j : 0u;
            }
          }
        }
      }
      if (w.cnt == 0) { ++walk.u; continue; }
      const int64_t first_x = walk.x - walk.k + C::kItem, last_x = first_x + w.cnt - 1;
      int k0, k1;
      walk.part(w.cnt, k0, k1);
      walk.next(w.cnt, hkv);
      if (k0 == k1) continue;
      const int64_t row = row0 + h * G;
      __nv_bfloat16* out_tile = (__nv_bfloat16*)a.out + ((int64_t)(w.q0 + w.i_first) * a.hq + h * G) * a.D;
      float m = -INFINITY, l = 0.0f;  // m: log2 units
      float by = p.c, less = 3.402823466e+38f;  // a weight's logarithm is score x by + less; before a score has been seen, above every one
      bool first = true;
      for (int k = NQ == 2 ? k0 : k0 + g; k < k1; k += NQ == 2 ? 1 : 2, ++tiles, first = false) {
        const int s0 = w.kt.slot(k, kBN);
        // With these scores the group's product before is done too: it was issued before them.
        ok = warp_wait(&s_ready[g], tiles & 1u, s_abort, ctl, p.timeout_ns);
        if (!ok) break;
        tc_fence_after();
        if (NQ == 1 && r_in - lane >= w.rows) {  // no row of the tile is this warp's: its weights may be anything
          tc_fence_before();
          __syncwarp();
          if (lane < 2) mbar_arrive(&p_ready[g * 2 + lane]);
          continue;
        }
        uint32_t s[kBN];
#pragma unroll
        for (int c = 0; c < kBN; c += 32) tmem_ld32_nowait(s_col + c, s + c);
        tmem_wait_ld();
        if (!all_seen(a, w, s0)) {
          uint32_t bits[4];
          seen_bits(a, w, i, low, mask_row, s0, bits);
#pragma unroll
          for (int c = 0; c < kBN; ++c)
            if (!((bits[c >> 5] >> (c & 31)) & 1u)) s[c] = 0xff800000u;
        }
        float m4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) m4[c] = max3(__uint_as_float(s[c]), __uint_as_float(s[c + 4]), __uint_as_float(s[c + 8]));
#pragma unroll
        for (int c = 12; c < 124; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) m4[e] = max3(m4[e], __uint_as_float(s[c + e]), __uint_as_float(s[c + 4 + e]));
#pragma unroll
        for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], __uint_as_float(s[124 + e]));
        const float top = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]), over = fmaf(top, by, less);
        const bool grow = live && over > kLazy;  // at first: any finite maximum
        if (__any_sync(0xffffffffu, grow)) {
          const float m_new = grow ? top * p.c : m;
          const bool exact = fabsf(m_new) >= kExactFrom;
          const float f = !grow || m == -INFINITY ? 1.0f : ex2(exact ? -over : m - m_new);
          m = m_new;
          by = grow && exact ? p.c_exact : grow ? p.c : by;
          less = grow ? -(exact ? top * p.c_exact : m_new) : less;
          l *= f;
          if (!first) {
#pragma unroll 1
            for (int c = 0; c < C::DP; c += 32) {
              uint32_t o[32];
              tmem_ld32_nowait(o_col + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(o_col + c, o);
            }
            tmem_wait_st();
          }
        }
        const float2 c2 = make_float2(by, by), n2 = make_float2(less, less);
        float2 sum2[2] = {make_float2(0, 0), make_float2(0, 0)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int e = half * kHalf + 2 * c;
            float2 x = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, n2);
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            // To bf16, 2^-9 of a weight at most: an MMA's operands have one type, and V's is bf16. The sum takes the weights as they
            // are, in fp32, so that the log-sum is no worse for it. Outputs are off by 0.0022 of their size, by their own rounding alone
            // 0.0017.
            pk[c] = pack_bf16(x.x, x.y);
            sum2[c & 1] = add2(sum2[c & 1], x);
          }
          tmem_st32(s_col + 32 * half, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_ready[g * 2 + half]);
        }
        l += (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
      }
      if (ok && !first) ok = warp_wait(&o_done[g], done_items++ & 1u, s_abort, ctl, p.timeout_ns);
      // Whoever shares the epilogue goes on together or not at all: nobody is left at a barrier.
      if (NQ == 1) s_ml[g * 128 + trow] = make_float2(m, l);
      ok = NQ == 1 ? group_all<256>(1, ok) : group_all<128>(1 + g, ok);
      if (!ok) break;
      tc_fence_after();
      const int bad_at = g * kBadRing + (int)(item & (kBadRing - 1));
      const bool bad = s_bad[bad_at] != 0;

      // NQ = 1: the two groups' results are one; each group takes half of the columns of both O.
      float f0 = 1.0f, f1 = 0.0f;
      if (NQ == 1) {
        const float2 x = s_ml[trow], y = s_ml[128 + trow];
        m = fmaxf(x.x, y.x);
        f0 = x.x == m ? 1.0f : ex2(x.x - m);
        f1 = y.x == m ? 1.0f : ex2(y.x - m);
        l = x.y * f0 + y.y * f1;  // a sum may be NaN (of NaN scores) beside a maximum of -inf
      }
      const bool two = NQ == 1 && k1 - k0 > 1;  // the second O has been written
      const bool o_boxes = p.o_boxes && !bad && g * 128 + quarter * 32 + 32 <= w.rows;
      // CTA c holds list places [list c / ctas, list (c + 1) / ctas).
      int c_first = blockIdx.x, pieces = 1;
      if (k0 > 0 || k1 < w.cnt) {
        c_first = (int)(((first_x + 1) * ctas - 1) / list);
        pieces = (int)(((last_x + 1) * ctas - 1) / list) - c_first + 1;
      }
      const int64_t mine_at = (int64_t)blockIdx.x * 2 + ((int)blockIdx.x == c_first ? 1 : 0);
      const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : NAN);
      constexpr int kCols = NQ == 2 ? C::DP : C::DP / 2;
      constexpr int kPart = NQ == 2 ? 64 : 32;  // columns at a time
      const int col0 = NQ == 2 ? 0 : g * kCols;
      const uint32_t o_base = tmem + lanes + kOCol + (uint32_t)(NQ == 2 ? g * C::DP : col0);
#pragma unroll 1
      for (int c = 0; c < kCols; c += kPart) {
        uint32_t o[kPart];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < kPart; e += 32) tmem_ld32_nowait(o_base + c + e, o + e);
        tmem_wait_ld();
        if (NQ == 1) {
          uint32_t o1[kPart];
          if (two) tmem_ld32_nowait(o_base + C::DP + c, o1);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < kPart; ++e)
            o[e] = __float_as_uint(__uint_as_float(o[e]) * f0 + (two ? __uint_as_float(o1[e]) * f1 : 0.0f));
        }
        __syncwarp();
        if (pieces > 1) {
          if (live) {
            float4* dst = p.o + ((mine_at * NQ + (NQ == 2 ? g : 0)) * (C::DP / 4) + (col0 + c) / 4) * 128 + trow;
#pragma unroll
            for (int e = 0; e < kPart / 4; ++e)
              dst[e * 128] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                                         __uint_as_float(o[4 * e + 3]));
          }
        } else {
          uint4 y[kPart / 8];
#pragma unroll
          for (int e = 0; e < kPart / 8; ++e) {
            uint32_t z[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              z[j] = pack_bf16(__uint_as_float(o[8 * e + 2 * j]) * inv, __uint_as_float(o[8 * e + 2 * j + 1]) * inv);
            y[e] = make_uint4(z[0], z[1], z[2], z[3]);
          }
          if (NQ == 2 && o_boxes) {
            // As a box, from shared memory.
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
#pragma unroll
            for (int e = 0; e < kPart / 8; ++e) *(uint4*)(my_stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = y[e];
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&p.tmO, c, h * G, w.q0 + w.i_first + (g * 128 + quarter * 32) / G, my_stage);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          } else if (NQ == 2) {
            // Through shared memory, so that 128 bytes of a row leave together.
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
#pragma unroll
            for (int e = 0; e < kPart / 8; ++e) *(uint4*)(my_stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = y[e];
            __syncwarp();
            const int x = lane & 7;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int r = j * 4 + (lane >> 3);
              if (((out_rows >> j) & 1) && c + x * 8 < a.D)
                *(uint4*)(out_tile + out_at[j] + c) = *(const uint4*)(my_stage + r * 128 + ((x ^ (r & 7)) << 4));
            }
            __syncwarp();
          } else if (live) {
#pragma unroll
            for (int e = 0; e < kPart / 8; ++e)
              if (col0 + c + 8 * e < a.D) *(uint4*)((__nv_bfloat16*)a.out + row * a.D + col0 + c + 8 * e) = y[e];
          }
        }
      }
      tc_fence_before();  // these reads of O before the next item's first product
      if (bad) {
        __threadfence_block();
        __syncwarp();  // a row's result may have been stored by other lanes
        if (live)
          add_non_finite<CACHE>(a, w, b, h, k0, k1, i, low, mask_row, col0, col0 + kCols,
                         pieces > 1 ? nullptr : (__nv_bfloat16*)a.out + row * a.D,
                         p.o + (mine_at * NQ + (NQ == 2 ? g : 0)) * (C::DP / 4) * 128 + trow);
      }
      if (pieces == 1) {
        if (live && a.lse && (NQ == 2 || g == 0)) a.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
      } else {
        if (live && (NQ == 2 || g == 0)) p.ml[mine_at * C::BMT + r_in] = make_float2(m, l);
        __threadfence();
      }
      // Done with O, s_ml, s_bad, the query tile and (when cut) the partial rows.
      constexpr int kGroup = NQ == 1 ? 256 : 128;
      const int bar_id = NQ == 1 ? 1 : 1 + g;
      group_all<kGroup>(bar_id, true);
      if (trow == 0) s_bad[bad_at] = 0;
      if (pieces > 1) {
        const int me = NQ == 1 ? g * 128 + trow : trow;
        if (me == 0) {
          // Every query tile of the row tile counts one arrival per piece.
          unsigned* cnt = p.arrived + c_first * NQ + (NQ == 2 ? g : 0);
          const bool last = atomicAdd(cnt, 1u) == (unsigned)pieces - 1u;
          if (last) *cnt = 0u;  // ready for the next call
          s_last[NQ == 2 ? g : 0] = last;
        }
        group_all<kGroup>(bar_id, true);
        if (s_last[NQ == 2 ? g : 0]) {
          __threadfence();
          // The pieces in order. Neighbouring threads take rows, a thread the same row in every round.
          const int qt = NQ == 2 ? g : 0;
          const int rows_q = min(128, w.rows - qt * 128);
          int rp = 1;
          while (rp < rows_q) rp <<= 1;
          const int r = me & (rp - 1);
          auto piece_at = [&](int pc) { return (int64_t)(c_first + pc) * 2 + (pc == 0 ? 1 : 0); };
          if (r < rows_q && me / rp < C::DP / 4) {
            float mm = -INFINITY, ll = 0.0f;
#pragma unroll 8
            for (int pc = 0; pc < pieces; ++pc) mm = fmaxf(mm, __ldcg(&p.ml[piece_at(pc) * C::BMT + qt * 128 + r]).x);
            const int prr = w.r0 + qt * 128 + r, ii = prr / G;
            const int64_t orow = (int64_t)(w.q0 + ii) * a.hq + h * G + (prr - ii * G);
            constexpr int kE = 4;  // groups of four columns in flight
            for (int e4 = me / rp; e4 < C::DP / 4; e4 += kE * (kGroup / rp)) {
              float4 acc[kE];
              ll = 0.0f;
#pragma unroll
              for (int e = 0; e < kE; ++e) acc[e] = make_float4(0, 0, 0, 0);
#pragma unroll 4
              for (int pc = 0; pc < pieces; ++pc) {
                const float2 v = __ldcg(&p.ml[piece_at(pc) * C::BMT + qt * 128 + r]);
                const float4* src = p.o + ((piece_at(pc) * NQ + qt) * (C::DP / 4)) * 128 + r;
                const bool none = v.x == -INFINITY && v.y == 0.0f;  // saw nothing
                const float f = none ? 0.0f : v.x == mm ? 1.0f : ex2(v.x - mm);
                ll += none ? 0.0f : v.y * f;
#pragma unroll
                for (int e = 0; e < kE; ++e) {
                  const int at = e4 + e * (kGroup / rp);
                  if (at < C::DP / 4 && !none) {
                    const float4 y = __ldcg(src + at * 128);
                    acc[e].x += y.x * f; acc[e].y += y.y * f; acc[e].z += y.z * f; acc[e].w += y.w * f;
                  }
                }
              }
              const float iv = ll > 0.0f ? 1.0f / ll : (ll == 0.0f ? 0.0f : NAN);
#pragma unroll
              for (int e = 0; e < kE; ++e) {
                const int at = e4 + e * (kGroup / rp);
                if (at * 4 < a.D)
                  *(uint2*)((__nv_bfloat16*)a.out + orow * a.D + at * 4) =
                      make_uint2(pack_bf16(acc[e].x * iv, acc[e].y * iv), pack_bf16(acc[e].z * iv, acc[e].w * iv));
              }
            }
            if (me / rp == 0 && a.lse) a.lse[orow] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
          }
        }
      }
      ++item;
    }
    if (NQ == 2 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                  const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (EncodeTiledFn)ptr;
  });
  return fn;
}

// The cache as {head_dim, slot, kv head, request}, boxes of 64 x 128 slots. An axis of one
// entry gets any valid stride. Elements past head_dim read as zero.
bool make_tmap(CUtensorMap* tm, const void* base, const AttnArgs& a) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.rows.capacity, (cuuint64_t)a.hkv, (cuuint64_t)a.rows.batch};
  const int64_t st[3] = {a.ss, a.hs, a.rs};
  cuuint64_t strides[3];
  for (int i = 0; i < 3; ++i) strides[i] = dims[i + 1] == 1 ? (cuuint64_t)((a.D * 2 + 15) / 16 * 16) : (cuuint64_t)(st[i] * 2);
  cuuint32_t box[4] = {64, (cuuint32_t)kBN, 1, 1}, estr[4] = {1, 1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same for pages. A copy has a cost of its own, so a page's heads are taken whole: pages and kv heads are one axis, in steps of their
// strides' common divisor, and bf16 heads of 128 are {64 elements, 8 slots, half, groups of 8 slots, place}, which lands as swizzle
// atoms of the two halves in turn. Codes are {head_dim, slot, place}, not swizzled; other heads {head_dim, slot, place} in
// boxes of 64.
int64_t divisor(int64_t x, int64_t y) { return y == 0 ? x : divisor(y, x % y); }
bool page_places(const AttnArgs& a, int64_t* unit, int64_t* places) {
  const int64_t ps = a.pages.n_pages > 1 ? a.pages.page_stride : 0, hs = a.hkv > 1 ? a.hs : 0;
  *unit = divisor(ps, hs);
  if (*unit == 0) *unit = 16;  // one head of one page
  *places = (a.pages.n_pages - 1) * (ps / *unit) + (a.hkv - 1) * (hs / *unit) + 1;
  return *places < 0x7fffffff;
}
bool make_pages_tmap(TcAttnP& p, CUtensorMap* tm, const void* base, const AttnArgs& a) {
  EncodeTiledFn fn = encode_fn();
  int64_t unit, places;
  if (!fn || !page_places(a, &unit, &places)) return false;
  const bool codes = a.cache == kPagedE4m3;
  const int size = codes ? 1 : 2, page = 1 << a.pages.shift, box_slots = page < kBN ? page : kBN;
  p.folded = !codes && a.D == 128;
  p.no_page = (int)places;
  p.page_step = a.pages.n_pages > 1 ? a.pages.page_stride / unit : 0;
  p.head_step = a.hkv > 1 ? a.hs / unit : 0;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const auto type = codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto swizzle = codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
  if (p.folded) {
    const cuuint64_t dims[5] = {64, 8, 2, (cuuint64_t)(page / 8), (cuuint64_t)places};
    const cuuint64_t strides[4] = {(cuuint64_t)(a.ss * 2), 128, (cuuint64_t)(a.ss * 16), (cuuint64_t)(unit * 2)};
    const cuuint32_t box[5] = {64, 8, 2, (cuuint32_t)(box_slots / 8), 1};
    return fn(tm, type, 5, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)page, (cuuint64_t)places};
  const cuuint64_t strides[2] = {(cuuint64_t)(a.ss * size), (cuuint64_t)(unit * size)};
  const cuuint32_t box[3] = {(cuuint32_t)(codes && a.D > 64 ? 128 : 64), (cuuint32_t)box_slots, 1};
  return fn(tm, type, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries or the output as {head_dim, head, row}, boxes of 64 elements of a group's heads of
// packed / G rows.
bool make_row_tmap(CUtensorMap* tm, const void* base, int packed, const AttnArgs& a) {
  EncodeTiledFn fn = encode_fn();
  const int G = a.hq / a.hkv;
  if (!fn || packed % G) return false;
  cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.hq, (cuuint64_t)a.rows.tokens};
  cuuint64_t strides[2] = {(cuuint64_t)a.D * 2, (cuuint64_t)a.hq * a.D * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(packed / G)}, estr[3] = {1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NQ, int KB, int CACHE>
cudaError_t launch_tc(const AttnArgs& a, cudaStream_t stream) {
  using C = Cfg<NQ, KB, CACHE>;
  TcAttnP p;
  memset(&p, 0, sizeof(p));
  if (CACHE == kWhole ? !make_tmap(&p.tmK, a.k, a) || !make_tmap(&p.tmV, a.v, a)
                      : !make_pages_tmap(p, &p.tmK, a.k, a) || !make_pages_tmap(p, &p.tmV, a.v, a))
    return cudaErrorInvalidValue;
  p.q_boxes = make_row_tmap(&p.tmQ, a.q, 128, a) ? 1 : 0;
  p.o_boxes = NQ == 2 && make_row_tmap(&p.tmO, a.out, 32, a) ? 1 : 0;
  p.a = a;
  p.row_tiles = (int)(((int64_t)a.rows.max_q * (a.hq / a.hkv) + C::BMT - 1) / C::BMT);
  p.timeout_ns = wait_timeout_ns();
  // Masked scores are -inf before they are multiplied and have to stay so with a scale of 0: the smallest normal factor
  // instead, which brings products of up to 2^120 to within 2^-6 of 0.
  p.c = fmaxf(a.scale * kLog2e, 1.17549435e-38f);
  p.c_exact = ldexpf(1.0f, ilogbf(fminf(p.c, 3.402823466e+38f)));
  // Beside the tiles: barriers, notes and (NQ = 1) the groups' maxima and sums.
  constexpr uint32_t kSmall = NQ == 2 && C::kCodes ? 1024 : 3 * 1024;
  const uint32_t budget = 227 * 1024 - kSmall;
  int slots = (int)((budget - NQ * C::kQBytes - C::kStage) / C::kTile);
  // Even: a buffer is always a key or always a value buffer, so every phase of a value
  // buffer is waited for by those who clear it.
  p.slots = slots > 12 ? 12 : slots & ~1;
  size_t staged = 0;
  if (C::kCodes) {
    // Of the room for four buffers or more, codes take what is left beside three (prompts; with two, the next tile's values wait for
    // the last product with this one's) or four of the MMA's. Three in turn are keys and values alike, which prompts may: their
    // products take the buffers in the order in which they are filled.
    p.slots = NQ == 2 && KB == 2 ? 3 : 4;
    p.staged = std::min(8, (int)((budget - NQ * C::kQBytes - C::kStage - p.slots * C::kTile) / (C::kStaged + kBN * 4)));
    staged = (size_t)p.staged * (C::kStaged + kBN * 4);
  }
  const size_t smem = (size_t)NQ * C::kQBytes + (size_t)p.slots * C::kTile + C::kStage + staged + kSmall;
  const int grid = num_sms();
  static_assert(NQ <= kCountersPerSm, "a counter for every tile that is cut");
  if ((int64_t)a.rows.batch * p.row_tiles > (1 << 30)) return cudaErrorInvalidConfiguration;
  uint8_t* w = (uint8_t*)a.scratch;
  p.arrived = (unsigned int*)w;
  w += counter_bytes();
  p.ml = (float2*)w;
  p.o = (float4*)(w + (size_t)2 * grid * C::BMT * 8);
  static FuncOnce once;
  cudaError_t e = once.set((const void*)attn_tc_kernel<NQ, KB, CACHE>, 227 * 1024, false);
  if (e != cudaSuccess) return e;
  attn_tc_kernel<NQ, KB, CACHE><<<grid, C::kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t attn_tc_ws_bytes(const AttnArgs& a) {
  const size_t dp = a.D > 64 ? 128 : 64;
  return counter_bytes() + (size_t)2 * num_sms() * 256 * (8 + dp * 4);
}

// bf16, head_dim <= 128, and a cache that a tensor map can describe: no axis of more than
// one entry with a stride of 0 (requests that share a cache), strides below 2^40 bytes.
bool attn_tc_applies(const AttnArgs& a) {
  if (a.dtype != DOMINO_BF16 || a.D > 128) return false;
  const bool whole = a.cache == kWhole;
  const int64_t st[3] = {a.ss, a.hs, whole ? a.rs : a.pages.page_stride};
  const int n[3] = {whole ? a.rows.capacity : 1 << a.pages.shift, a.hkv, whole ? a.rows.batch : a.pages.n_pages};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (st[i] == 0 || st[i] * 2 >= ((int64_t)1 << 40))) return false;
  int64_t unit, places;
  return whole || page_places(a, &unit, &places);
}

template <int CACHE>
static cudaError_t launch_on(const AttnArgs& a, cudaStream_t stream) {
  const bool wide = a.D > 64;
  if ((int64_t)a.rows.max_q * (a.hq / a.hkv) > 128) return wide ? launch_tc<2, 2, CACHE>(a, stream) : launch_tc<2, 1, CACHE>(a, stream);
  return wide ? launch_tc<1, 2, CACHE>(a, stream) : launch_tc<1, 1, CACHE>(a, stream);
}
cudaError_t launch_attention_tc(const AttnArgs& a, cudaStream_t stream) {
  return a.cache == kWhole ? launch_on<kWhole>(a, stream) : a.cache == kPaged ? launch_on<kPaged>(a, stream)
                                                                             : launch_on<kPagedE4m3>(a, stream);
}

}  // namespace domino
