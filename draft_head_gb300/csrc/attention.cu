// Attention of a block's rows over the cache (domino_block_attention and
// domino_paged_attention; the definitions are in domino.h): the kernel on CUDA cores, for
// fp32 and for every head size.
//
// One pass over the keys with the running maximum m and sum l of the softmax:
// per key tile s = scale q.k, m' = max(m, s), o = o 2^(m - m') + 2^(s - m') v
// (scores in units of log2(e), so that one exp2 is the exponential). A CTA holds
// 32 packed rows (row and query head of one kv head) and takes key tiles of 32
// slots. A thread has 4 rows x 2 keys of the scores and 4 rows x D / 16 columns of o.
// Few tiles and a long cache: the key tiles are split over CTAs, each writes its
// (o, m, l), and the last one of a tile to arrive joins them in split order, so the
// result does not depend on the arrival order.
//
// A few rows: bound by latency (a key tile's loads, products and barriers behind one another), so the key
// tiles are spread as thin as two per CTA. Three requests of 40 rows over 1500 slots, 6 heads of 80, window 700: 39 us,
// 2.2 TFLOP/s; one row over 3000 slots 32.5 us (53 and 71 us with scalar loads and arithmetic and pieces joined one
// by one). Prompts: bound by shared memory (six 16-byte reads for 16 packed multiply-adds of the scores). 2000
// rows: 8 heads of 128 in fp32 666 us, 8 heads of 256 in bf16 1348 us, 12 TFLOP/s both.
#include <math.h>
#include <algorithm>

#include "attention.cuh"
#include "packed.cuh"
#include "pages.cuh"

namespace domino {

namespace {

constexpr int kBM = 32, kBN = 32, kThr = 128;
constexpr int kLeast = 2;  // key tiles per split at least
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct SimtP {
  AttnArgs a;
  Partials part;
  int splits, row_tiles;
};

__device__ __forceinline__ float4 load4(const float* p) { return *(const float4*)p; }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *(const uint2*)p;
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}

// Four elements of slot s of kv head h of request b; zeros where its page is not there (`page` < 0).
template <typename T, int CACHE>
__device__ __forceinline__ float4 slot4(const AttnArgs& a, const void* kv, const uint8_t* scale, int page, int h, int s, int e) {
  if (page < 0) return make_float4(0, 0, 0, 0);
  const int64_t at = (int64_t)page * a.pages.page_stride + (int64_t)h * a.hs + (int64_t)slot_in_page(a.pages, s) * a.ss + e;
  if (CACHE == kPaged) return load4((const T*)kv + at);
  const float4 x = codes_f32(*(const uint32_t*)((const uint8_t*)kv + at));
  const float f = scale_f32(scale[scale_at(a.pages, a.hkv, page, h, s)]);
  return make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
}

template <typename T, int CACHE>
__global__ void __launch_bounds__(kThr) attn_simt_kernel(const __grid_constant__ SimtP p) {
  extern __shared__ float sm[];
  __shared__ int s_last;
  const AttnArgs& a = p.a;
  const int D = a.D, ldq = D + 4;
  float* sq = sm;                 // [kBM][D + 4]
  float* sk = sq + kBM * ldq;     // [kBN][D + 4]
  float* sv = sk + kBN * ldq;     // [kBN][D]
  float* sp = sv + kBN * D;       // [kBM][kBN + 1]
  int* s_i = (int*)(sp + kBM * (kBN + 1));  // place, window begin of each row
  int* s_low = s_i + kBM;
  const int tile = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
  const int h = blockIdx.y, b = blockIdx.z, t = threadIdx.x;
  const int G = a.hq / a.hkv;
  int q0, n, ctx;
  if (!request_rows(a.rows, b, q0, n, ctx, t == 0, a.ctl)) return;
  const int r0 = tile * kBM, rows = min(kBM, n * G - r0);
  if (rows <= 0) return;

  if (t < kBM) {
    const int i = min(r0 + t, n * G - 1) / G;
    const int pos = a.rows.positions ? a.rows.positions[q0 + i] : ctx + i;
    s_i[t] = i;
    s_low[t] = window_low(pos, a.window);
  }
  const T* q = (const T*)a.q;
  // Four elements a thread; its place moves on by kThr of them without a division.
  const int nv = D / 4, row_step = kThr / nv, col_step = kThr - row_step * nv, row_1 = t / nv, col_1 = t - row_1 * nv;
  auto each = [&](int rows_of, auto f) {
    for (int r = row_1, e = col_1; r < rows_of;) {
      f(r, e * 4);
      r += row_step;
      e += col_step;
      if (e >= nv) {
        e -= nv;
        ++r;
      }
    }
  };
  each(kBM, [&](int r, int e) {
    float4 x = make_float4(0, 0, 0, 0);
    if (r < rows) {
      const int pr = r0 + r;
      x = load4(q + ((int64_t)(q0 + pr / G) * a.hq + h * G + pr % G) * D + e);
    }
    const float c = a.scale * kLog2e;
    *(float4*)(sq + r * ldq + e) = make_float4(x.x * c, x.y * c, x.z * c, x.w * c);
  });
  __syncthreads();
  int low = 0x7fffffff, low_max = 0;
  for (int r = 0; r < rows; ++r) {
    low = min(low, s_low[r]);
    low_max = max(low_max, s_low[r]);
  }
  // Slots that every row sees: from all_low (or among the sinks) up to all_hi.
  const int all_hi = a.mode == DOMINO_MASK_CAUSAL ? ctx + s_i[0] + 1 : a.mode == DOMINO_MASK_FULL ? ctx + n : ctx;
  const int all_low = a.mode == DOMINO_MASK_CAUSAL ? low_max : min(low_max, ctx);
  const KeyTiles kt = key_tiles(a.mode, a.sinks, low, ctx, n, s_i[rows - 1], kBN);
  const int used = splits_used(p.splits, kt.count, kLeast);
  if (split >= used) return;
  const int k_begin = (int)((int64_t)kt.count * split / used), k_end = (int)((int64_t)kt.count * (split + 1) / used);

  const int tr = t >> 4, tc = t & 15;
  float m[4], l[4], o[4][16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.0f;
#pragma unroll
    for (int c = 0; c < 16; ++c) o[i][c] = 0.0f;
  }
  const T* kb = (const T*)a.k + (int64_t)b * a.rs + (int64_t)h * a.hs;
  const T* vb = (const T*)a.v + (int64_t)b * a.rs + (int64_t)h * a.hs;
  const uint8_t* mask = a.mask ? a.mask + (int64_t)b * a.rows.max_q * a.rows.max_q : nullptr;
  for (int k = k_begin; k < k_end; ++k) {
    const int s0 = kt.slot(k, kBN);
    __syncthreads();
    each(kBN, [&](int r, int e) {
      // Slots past the request's rows are not read.
      const bool in = s0 + r < ctx + n;
      if (CACHE == kWhole) {
        *(float4*)(sk + r * ldq + e) = in ? load4(kb + (int64_t)(s0 + r) * a.ss + e) : make_float4(0, 0, 0, 0);
        *(float4*)(sv + r * D + e) = in ? load4(vb + (int64_t)(s0 + r) * a.ss + e) : make_float4(0, 0, 0, 0);
      } else {
        // Pages before the window may be gone.
        const bool needed = in && (s0 + r < a.sinks || s0 + r >= first_slot(a.mode, low, ctx, ctx + n));
        const int page = needed ? page_of(a.pages, b, s0 + r) : -1;
        if (needed && page < 0 && e == 0) dev_error(a.ctl, DEV_ERR_DATA);
        *(float4*)(sk + r * ldq + e) = slot4<T, CACHE>(a, a.k, a.pages.k_scale, page, h, s0 + r, e);
        *(float4*)(sv + r * D + e) = slot4<T, CACHE>(a, a.v, a.pages.v_scale, page, h, s0 + r, e);
      }
    });
    __syncthreads();
    const bool whole = s0 + kBN <= all_hi && (s0 >= all_low || s0 + kBN <= a.sinks);
    float2 s2[4][2] = {};  // even and odd terms
    for (int e = 0; e < D; e += 4) {
      float4 kq[2], qq[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) kq[j] = *(const float4*)(sk + (tc + 16 * j) * ldq + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) qq[i] = *(const float4*)(sq + (tr * 4 + i) * ldq + e);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          s2[i][j] = fma2(make_float2(qq[i].x, qq[i].y), make_float2(kq[j].x, kq[j].y),
                         fma2(make_float2(qq[i].z, qq[i].w), make_float2(kq[j].z, kq[j].w), s2[i][j]));
    }
    float s[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) s[i][j] = s2[i][j].x + s2[i][j].y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = tr * 4 + i;
      bool in[2];
      float mx = m[i];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int slot = s0 + tc + 16 * j;
        in[j] = r < rows && (whole || (slot < ctx + n &&
                sees(a.mode, a.sinks, s_low[r], ctx, n, s_i[r], mask ? mask + (int64_t)s_i[r] * a.rows.max_q : nullptr, slot)));
        if (in[j]) mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      // A row that has seen nothing, or scores of -inf alone, keeps m = -inf and l = 0.
      const float keep = mx == -INFINITY || m[i] == mx ? 1.0f : exp2f(m[i] - mx);
      const float base = fmaxf(mx, -3.402823466e+38f);  // not -inf: scores of -inf have no weight
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float w = in[j] ? exp2f(s[i][j] - base) : -0.0f;  // the sign says that the slot is not seen
        sp[r * (kBN + 1) + tc + 16 * j] = w;
        sum += w;
      }
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      l[i] = l[i] * keep + sum;
      m[i] = mx;
#pragma unroll
      for (int c = 0; c < 16; ++c) o[i][c] *= keep;
    }
    __syncwarp();  // a row's weights are written and read by one warp
    for (int j = 0; j < kBN; ++j) {
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = sp[(tr * 4 + i) * (kBN + 1) + j];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int e = c * 64 + tc * 4;
        if (e < D) {
          float4 v = *(const float4*)(sv + j * D + e);
          // What a row does not see has weight 0 and must not be multiplied if it is no number; what it sees is added as
          // it is then, as the weight may have vanished. A slot that all rows see may be anything.
          if (!whole && !(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w))) {
            const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (__float_as_int(w[i]) >= 0) {
#pragma unroll
                for (int y = 0; y < 4; ++y) o[i][4 * c + y] = isfinite(x[y]) ? fmaf(w[i], x[y], o[i][4 * c + y]) : o[i][4 * c + y] + x[y];
              }
            continue;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 w2 = make_float2(w[i], w[i]);
            const float2 x = fma2(w2, make_float2(v.x, v.y), make_float2(o[i][4 * c], o[i][4 * c + 1]));
            const float2 y = fma2(w2, make_float2(v.z, v.w), make_float2(o[i][4 * c + 2], o[i][4 * c + 3]));
            o[i][4 * c] = x.x; o[i][4 * c + 1] = x.y; o[i][4 * c + 2] = y.x; o[i][4 * c + 3] = y.y;
          }
        }
      }
    }
  }

  T* out = (T*)a.out;
  if (used > 1) {
    const int64_t tl = ((int64_t)b * a.hkv + h) * p.row_tiles + tile;
    const int64_t base = (tl * p.splits + split) * kBM;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = tr * 4 + i;
      if (r >= rows) continue;
      if (tc == 0) p.part.ml[base + r] = make_float2(m[i], l[i]);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c * 64 + tc * 4 < D)
          *(float4*)(p.part.o + (base + r) * D + c * 64 + tc * 4) =
              make_float4(o[i][4 * c], o[i][4 * c + 1], o[i][4 * c + 2], o[i][4 * c + 3]);
    }
    __threadfence();
    __syncthreads();
    if (t == 0) {
      const unsigned int was = atomicAdd(p.part.arrived + tl, 1u);
      s_last = was == (unsigned)used - 1u;
      if (s_last) p.part.arrived[tl] = 0u;  // ready for the next call
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    // Four columns of a row at a time, one pass over the pieces in order, eight in flight, the maximum raised as
    // they come.
    for (int x = t; x < rows * nv; x += kThr) {
      const int r = x / nv, e = (x - r * nv) * 4;
      const int64_t first = tl * p.splits * kBM + r;
      float mm = -INFINITY, ll = 0.0f;
      float4 acc = make_float4(0, 0, 0, 0);
      for (int s = 0; s < used; s += 8) {
        float2 ml[8];
        float4 y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          ml[u] = make_float2(-INFINITY, 0.0f);
          if (s + u < used) {
            ml[u] = __ldcg(&p.part.ml[first + (int64_t)(s + u) * kBM]);
            y[u] = __ldcg((const float4*)(p.part.o + (first + (int64_t)(s + u) * kBM) * D + e));
          }
        }
        float now = mm;
#pragma unroll
        for (int u = 0; u < 8; ++u) now = fmaxf(now, ml[u].x);
        const float keep = now == mm || mm == -INFINITY ? 1.0f : exp2f(mm - now);
        ll *= keep;
        acc.x *= keep; acc.y *= keep; acc.z *= keep; acc.w *= keep;
        mm = now;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (ml[u].x == -INFINITY && ml[u].y == 0.0f) continue;  // saw nothing
          const float f = ml[u].x == mm || ml[u].x == -INFINITY ? 1.0f : exp2f(ml[u].x - mm);
          ll += ml[u].y * f;
          acc.x += y[u].x * f; acc.y += y[u].y * f; acc.z += y[u].z * f; acc.w += y[u].w * f;
        }
      }
      const int pr = r0 + r;
      const int64_t row = (int64_t)(q0 + pr / G) * a.hq + h * G + pr % G;
      const float inv = ll > 0.0f ? 1.0f / ll : (ll == 0.0f ? 0.0f : NAN);
      if (a.lse && e == 0) a.lse[row] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
      T* dst = out + row * D + e;
      dst[0] = (T)(acc.x * inv);
      dst[1] = (T)(acc.y * inv);
      dst[2] = (T)(acc.z * inv);
      dst[3] = (T)(acc.w * inv);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = tr * 4 + i, pr = r0 + r;
    if (r >= rows) continue;
    const int64_t row = (int64_t)(q0 + pr / G) * a.hq + h * G + pr % G;
    const float inv = l[i] > 0.0f ? 1.0f / l[i] : (l[i] == 0.0f ? 0.0f : NAN);
    if (a.lse && tc == 0) a.lse[row] = l[i] == 0.0f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const int e = (c >> 2) * 64 + tc * 4 + (c & 3);
      if (e < D) out[row * D + e] = (T)(o[i][c] * inv);
    }
  }
}

// Two CTAs per SM.
int64_t simt_want() { return 2 * (int64_t)num_sms(); }

int simt_row_tiles(const AttnArgs& a) {
  return (int)(((int64_t)a.rows.max_q * (a.hq / a.hkv) + kBM - 1) / kBM);
}

}  // namespace

// Of every kernel that a block with these bounds or smaller ones may run on.
size_t attn_ws_bytes(const AttnArgs& a) {
  const size_t simt = partial_bytes(simt_want(), kBM, a.D);
  if (a.dtype != DOMINO_BF16 || a.D > 128) return simt;
  const size_t rows = attn_rows_ws_bytes(a), tc = attn_tc_ws_bytes(a);
  if (a.cache != kWhole) return std::max(simt, std::max(rows, tc));
  return std::max(rows, attn_tc_applies(a) ? tc : simt);
}

cudaError_t launch_attention(const AttnArgs& a, cudaStream_t stream) {
  if (attn_rows_applies(a)) return launch_attention_rows(a, stream);
  if (attn_tc_applies(a)) return launch_attention_tc(a, stream);
  SimtP p;
  p.a = a;
  p.row_tiles = simt_row_tiles(a);
  p.splits = splits_for((int64_t)p.row_tiles * a.hkv * a.rows.batch, simt_want(),
                        ((int64_t)a.rows.max_ctx + a.rows.max_q) / kBN / kLeast);
  p.part = partials_at(a.scratch, simt_want(), kBM);
  const size_t smem = sizeof(float) * (kBM * (a.D + 4) + kBN * (a.D + 4) + kBN * a.D + kBM * (kBN + 1)) + 8 * kBM;
  const dim3 grid((unsigned)(p.row_tiles * p.splits), (unsigned)a.hkv, (unsigned)a.rows.batch);
  auto run = [&](auto kernel, FuncOnce& once) {
    const cudaError_t e = once.set((const void*)kernel, 120 * 1024, false);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThr, smem, stream>>>(p);
    return cudaGetLastError();
  };
  static FuncOnce once_bf16, once_f32, once_paged_bf16, once_paged_f32, once_e4m3;
  if (a.cache == kPagedE4m3) return run(attn_simt_kernel<__nv_bfloat16, kPagedE4m3>, once_e4m3);
  if (a.cache == kPaged)
    return a.dtype == DOMINO_BF16 ? run(attn_simt_kernel<__nv_bfloat16, kPaged>, once_paged_bf16)
                                  : run(attn_simt_kernel<float, kPaged>, once_paged_f32);
  return a.dtype == DOMINO_BF16 ? run(attn_simt_kernel<__nv_bfloat16, kWhole>, once_bf16)
                                : run(attn_simt_kernel<float, kWhole>, once_f32);
}

}  // namespace domino
