// Attention of a few rows over the cache (domino_block_attention; the definition
// is in domino.h): bf16, head_dim <= 128, at most 16 packed rows of a kv head,
// as when a token is decoded.
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
#include <math.h>
#include <algorithm>

#include "attention.cuh"
#include "packed.cuh"

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
constexpr float kLazy = 32.0f;

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
template <int NT, int KS, int JJ>
__global__ void __launch_bounds__(kThr, 2) attn_rows_kernel(const __grid_constant__ RowsP p) {
  constexpr int kRows = 8 * NT, DP = 64 * JJ;
  __shared__ __align__(16) float s_o[kWarps][kRows][DP + 4];
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

  const __nv_bfloat16* kb = (const __nv_bfloat16*)a.k + (int64_t)b * a.rs + (int64_t)h * a.hs;
  const __nv_bfloat16* vb = (const __nv_bfloat16*)a.v + (int64_t)b * a.rs + (int64_t)h * a.hs;
  const int end = ctx + rows_n;
  uint4 kx[2][KS], vx[4][JJ];
  auto fetch = [&](int k) {
    const int s0 = kt.slot(k, kBN);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int s = s0 + n + 8 * x;
#pragma unroll
      for (int j = 0; j < KS; ++j)
        kx[x][j] = s < end && 32 * j + 8 * c < a.D ? ldg16(kb + (int64_t)s * a.ss + 32 * j + 8 * c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int s = s0 + 2 * c + (x & 1) + 8 * (x >> 1);
#pragma unroll
      for (int j = 0; j < JJ; ++j)
        vx[x][j] = s < end && 64 * j + 8 * n < a.D ? ldg16(vb + (int64_t)s * a.ss + 64 * j + 8 * n) : make_uint4(0, 0, 0, 0);
    }
  };

  float o[NT][4 * JJ][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int g = 0; g < NT; ++g) {
#pragma unroll
    for (int t = 0; t < 4 * JJ; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[g][t][e] = 0.0f;
    m[g][0] = m[g][1] = -INFINITY;
    l[g][0] = l[g][1] = 0.0f;
  }
  if (k_begin + warp < k_end) fetch(k_begin + warp);
#pragma unroll 1
  for (int k = k_begin + warp; k < k_end; k += kWarps) {
    const int s0 = kt.slot(k, kBN);
    uint4 kc[2][KS], vc[4][JJ];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int j = 0; j < KS; ++j) kc[x][j] = kx[x][j];
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int j = 0; j < JJ; ++j) vc[x][j] = vx[x][j];
    if (k + kWarps < k_end) fetch(k + kWarps);
    const bool whole = s0 + kBN <= all_hi && (s0 >= all_low || s0 + kBN <= a.sinks);
    bool mend = false;
    if (!whole) {
      // A weight of 0 does not stop an infinity or a NaN in the product: they are cleared here
      // and added below to the rows that see them.
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int j = 0; j < JJ; ++j) {
          mend |= bad16(vc[x][j].x) | bad16(vc[x][j].y) | bad16(vc[x][j].z) | bad16(vc[x][j].w);
          vc[x][j] = make_uint4(clear16(vc[x][j].x), clear16(vc[x][j].y), clear16(vc[x][j].z), clear16(vc[x][j].w));
        }
      mend = __any_sync(0xffffffffu, mend);
    }
#pragma unroll
    for (int g = 0; g < NT; ++g) {
      float s[4] = {0, 0, 0, 0};  // slots n, n, n + 8, n + 8 of rows 2c, 2c + 1, 2c, 2c + 1
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        mma16816(s, kc[0][j].x, kc[1][j].x, kc[0][j].y, kc[1][j].y, q[g][j][0], q[g][j][1]);
        mma16816(s, kc[0][j].z, kc[1][j].z, kc[0][j].w, kc[1][j].w, q[g][j][2], q[g][j][3]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[e] *= p.c;
        if (!whole) {
          const int r = g * 8 + 2 * c + (e & 1), slot = s0 + n + 8 * (e >> 1);
          if (!(slot < end && sees(a.mode, a.sinks, s_low[r], ctx, rows_n, s_i[r],
                                   mask ? mask + (int64_t)s_i[r] * a.rows.max_q : nullptr, slot)))
            s[e] = -INFINITY;
        }
      }
      const float top[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
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
        s[e] = ex2(s[e] - (m[g][e & 1] == -INFINITY ? 0.0f : m[g][e & 1]));
        l[g][e & 1] += s[e];
      }
      const uint32_t b0 = transpose8(pack_bf16(s[0], s[1])), b1 = transpose8(pack_bf16(s[2], s[3]));
#pragma unroll
      for (int j = 0; j < JJ; ++j) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t v0 = part(vc[0][j], t), v1 = part(vc[1][j], t), v2 = part(vc[2][j], t), v3 = part(vc[3][j], t);
          mma16816(o[g][4 * j + t], __byte_perm(v0, v1, 0x5410), __byte_perm(v0, v1, 0x7632), __byte_perm(v2, v3, 0x5410),
                   __byte_perm(v2, v3, 0x7632), b0, b1);
        }
      }
      if (mend) {
        for (int x = 0; x < kBN && s0 + x < end; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = g * 8 + 2 * c + e;
            const bool sees_it = sees(a.mode, a.sinks, s_low[r], ctx, rows_n, s_i[r],
                                      mask ? mask + (int64_t)s_i[r] * a.rows.max_q : nullptr, s0 + x);
#pragma unroll
            for (int d = 0; d < 8 * JJ; ++d) {
              const int col = 64 * (d >> 3) + 8 * n + (d & 7);
              const float v = col < a.D ? __bfloat162float(vb[(int64_t)(s0 + x) * a.ss + col]) : 0.0f;
              if (sees_it && !isfinite(v)) o[g][(d >> 3) * 4 + ((d & 7) >> 1)][(d & 1) * 2 + e] += v;
            }
          }
      }
    }
  }

  // The warps' results, in shared memory.
#pragma unroll
  for (int g = 0; g < NT; ++g)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = g * 8 + 2 * c + e;
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[g][e] += __shfl_xor_sync(0xffffffffu, l[g][e], d);
      if (n == 0) s_ml[warp][r] = make_float2(m[g][e], l[g][e]);
#pragma unroll
      for (int j = 0; j < JJ; ++j) {
        float* dst = &s_o[warp][r][64 * j + 8 * n];
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
      const float4 y = *(const float4*)&s_o[w][r][e];
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

template <int NT, int KS, int JJ>
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
  attn_rows_kernel<NT, KS, JJ><<<grid, kThr, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

// Up to 8 packed rows it is the faster one or as fast (64 tokens over up to 4000 slots 117 us, the tensor core
// kernel 118; over up to 500 slots 24 and 50). From 9 to 16 its products are twice as many, and with every SM busy over
// long caches the tensor core kernel wins, from pasts of about 2500 on: 64 requests of 4 rows in groups of 4, up to 500 /
// 2000 / 2500 / 3000 / 4000 slots, 31 / 76 / 80 / 96 / 120 us and 47 / 76 / 81 / 92 / 112; 32 requests 18 / 47 / 48 / 55 / 72
// and 28 / 46 / 50 / 54 / 67. Fewer, which leave SMs idle: 16 requests up to 4000 slots 43.7 and 43.1; one 21 and 21.
bool attn_rows_applies(const AttnArgs& a) {
  const int64_t rows = (int64_t)a.rows.max_q * (a.hq / a.hkv);
  if (a.dtype != DOMINO_BF16 || a.D > 128 || rows > 16) return false;
  return rows <= 8 || a.rows.max_ctx < 2500 || (int64_t)a.hkv * a.rows.batch <= num_sms();
}
size_t attn_rows_ws_bytes(const AttnArgs& a) { return partial_bytes(want_ctas(), 16, a.D); }

cudaError_t launch_attention_rows(const AttnArgs& a, cudaStream_t stream) {
  const bool many = a.rows.max_q * (a.hq / a.hkv) > 8;
  if (a.D > 64) return many ? launch<2, 4, 2>(a, stream) : launch<1, 4, 2>(a, stream);
  return many ? launch<2, 2, 1>(a, stream) : launch<1, 2, 1>(a, stream);
}

}  // namespace domino
