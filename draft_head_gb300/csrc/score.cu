// What a row of logits says of a given token: its log-probability and rank, the row's entropy and its most likely tokens
// (domino_token_logprobs; the definition is in domino.h).
//
// One pass over the row. With m the maximum so far, d = (x - m) / T in log2 units and w = 2^d, a thread keeps S = sum w and
// E = sum w d; when m rises by r, E' = 2^-r (E - r S) and S' = 2^-r S. Then
//   log sum exp = m / T + log S,   entropy = log S - E / S,   log p(t) = (x_t - m) / T - log S,
// and as m is the true maximum d <= 0, so that both terms of the entropy are >= 0 and nothing cancels.
//   Rank: the given token's logit is known beforehand; tokens before it in (logit, id) are counted, in the batches of a warp that
//     have one.
//   Most likely tokens: a warp holds its best 32 (value, id) keys, one a lane, sorted. A batch of 32 lanes' values is looked at
//     only if one reaches the bound, the largest that any warp of the block knows: its n-th key, or the n-th largest of its
//     lanes' maxima, which n tokens reach.
// A cluster of CTAs takes a row when there are few; their results meet in the first one's shared memory.
#include <math.h>

#include "common.cuh"
#include "packed.cuh"

namespace domino {

namespace {

typedef unsigned long long u64;

constexpr int kThr = 256, kWarps = kThr / 32;
constexpr int kMaxCluster = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLeastD = -1000.0f;  // weights below 2^-149 are 0; takes the place of -inf and NaN, so that w d is 0
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Another CTA's shared memory, at the place of p.
__device__ __forceinline__ uint32_t dsmem(const void* p, uint32_t rank) {
  uint32_t ra;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(p)), "r"(rank));
  return ra;
}
__device__ __forceinline__ u64 dsmem_u64(uint32_t at) {
  u64 x;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ float4 dsmem_f4(uint32_t at) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(at) : "memory");
  return x;
}

// The sums of part of a row; `m` the maximum of its logits, S and E in units of log2.
struct Sums {
  float m, S, E;
  __device__ __forceinline__ void raise(float to, float c) {  // to >= m
    if (to == m) return;
    const float r = (m - to) * c, f = ex2(r);
    E = f == 0.0f ? 0.0f : f * fmaf(r, S, E);
    S *= f;
    m = to;
  }
  __device__ __forceinline__ void join(Sums o, float c) {
    const float to = fmaxf(m, o.m);
    raise(to, c);
    o.raise(to, c);
    S += o.S;
    E += o.E;
  }
};

// Keys of (value descending, id ascending), one a lane; 0 for none.
__device__ __forceinline__ u64 shfl_xor(u64 x, int d) { return __shfl_xor_sync(kAll, x, d); }
__device__ __forceinline__ u64 sorted_down(u64 x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int d = k / 2; d > 0; d >>= 1) {
      const u64 y = shfl_xor(x, d);
      const bool upper = ((lane & d) == 0) == ((lane & k) == 0);  // this lane keeps the larger one
      x = (x > y) == upper ? x : y;
    }
  return x;
}
__device__ __forceinline__ float sorted_down(float x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int d = k / 2; d > 0; d >>= 1) {
      const float y = __shfl_xor_sync(kAll, x, d);
      x = ((lane & d) == 0) == ((lane & k) == 0) ? fmaxf(x, y) : fminf(x, y);
    }
  return x;
}
// The 32 largest of two sorted lists, sorted.
__device__ __forceinline__ u64 merged(u64 a, u64 b) {
  const int lane = threadIdx.x & 31;
  const u64 r = __shfl_sync(kAll, b, 31 - lane);
  u64 x = a > r ? a : r;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const u64 y = shfl_xor(x, d);
    x = (x > y) == ((lane & d) == 0) ? x : y;
  }
  return x;
}

// A row's elements in units of 16 aligned bytes: unit u holds elements [u kVec - skew, + kVec).
template <typename T>
struct Units {
  static constexpr int kVec = 16 / sizeof(T);
  const T* row;
  int V, skew, units;
  __device__ __forceinline__ Units(const T* r, int n) : row(r), V(n) {
    skew = (int)(((uintptr_t)r & 15) / sizeof(T));
    units = (int)(((int64_t)skew + V + kVec - 1) / kVec);
  }
  __device__ __forceinline__ int64_t first(int u) const { return (int64_t)u * kVec - skew; }
  // Elements that are not the row's are -inf, and not read.
  __device__ __forceinline__ uint4 load(int u, int end) const {
    const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    uint4 x = make_uint4(none, none, none, none);
    if (u >= end) return x;
    const int64_t i0 = first(u);
    if (i0 >= 0 && i0 + kVec <= V) {
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(row + i0));
    } else {
      uint32_t w[4] = {none, none, none, none};
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        if (i0 + e < 0 || i0 + e >= V) continue;
        if (sizeof(T) == 2) {
          const uint32_t y = *(const uint16_t*)(row + i0 + e);
          w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | y << 16 : (w[e / 2] & 0xffff0000u) | y;
        } else {
          w[e & 3] = *(const uint32_t*)(row + i0 + e);
        }
      }
      x = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return x;
  }
  static __device__ __forceinline__ void values(const uint4& x, float* v) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      v[e] = sizeof(T) == 4 ? __uint_as_float(w[e & 3]) : __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
};

struct Smem {
  u64 buf[kWarps][64];
  u64 list[kWarps][32];
  u64 bound;       // keys that are not above it are not among the best
  Sums sums[kWarps];
  int count[kWarps];
  float4 part;     // the CTA's m, S, E and rank (its bits)
  u64 best[32];
};

// The value just below x.
__device__ __forceinline__ float below(float x) {
  return x == 0.0f ? __uint_as_float(0x80000001u) : order_key_float(float_order_key(x) - 1u);
}

template <typename T, int kUnits>
__global__ void __launch_bounds__(kThr, 4) score_kernel(const ScoreArgs a, int size) {
  using U = Units<T>;
  constexpr int kVec = U::kVec, kN = kUnits * kVec;
  __shared__ Smem s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = size > 1 ? (int)cluster_rank() : 0, r = blockIdx.x / size;
  const T* row = (const T*)a.logits + (int64_t)r * a.ls;
  const U u(row, a.V);
  const int u0 = (int)((int64_t)u.units * rank / size), u1 = (int)((int64_t)u.units * (rank + 1) / size);
  const float temp = a.temperature ? a.temperature[r] : 1.0f;
  const bool fine = temp >= 1e-30f && isfinite(temp);
  const float c = kLog2e / temp;
  const int token = a.tokens ? a.tokens[r] : -1;
  const bool given = token >= 0 && token < a.V;
  const float xt = given ? fmaxf(to_f<T>(row[token]), -INFINITY) : INFINITY;  // a NaN counts as -inf
  const float xt_below = below(xt);
  const int n = a.top_n;
  const u64 least = value_id_key(-INFINITY, 0);
  if (threadIdx.x == 0) s.bound = least;
  __syncthreads();

  Sums q = {-INFINITY, 0.0f, 0.0f};
  int before = 0, held = 0;
  float lane_top = -INFINITY;
  u64 best = 0, bound = least;
  volatile u64* s_bound = &s.bound;
  u64* buf = s.buf[warp];

  auto take = [&](int count) {  // the first `count` (32 at most) of the buffer into the list
    __syncwarp();
    const u64 x = lane < count ? buf[lane] : 0;
    best = merged(best, sorted_down(x));
    const u64 nth = __shfl_sync(kAll, best, n - 1);
    if (nth > bound) bound = nth;
    __syncwarp();
    if (lane < held - count) buf[lane] = buf[count + lane];
    held -= count;
    __syncwarp();
    if (lane == 0) atomicMax(&s.bound, bound);
  };

  uint4 next[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) next[j] = u.load(u0 + j * kThr + (int)threadIdx.x, u1);
#pragma unroll 1
  for (int ub = u0; ub < u1; ub += kUnits * kThr) {
    float x[kN];
#pragma unroll
    for (int j = 0; j < kUnits; ++j) U::values(next[j], x + j * kVec);
    const int mine = ub + (int)threadIdx.x;  // unit j of this thread: mine + j kThr
    if (ub + kUnits * kThr < u1) {
#pragma unroll
      for (int j = 0; j < kUnits; ++j) next[j] = u.load(mine + (kUnits + j) * kThr, u1);
    }
    float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < kN; e += 8)
#pragma unroll
      for (int k = 0; k < 4; ++k) t4[k] = max3(t4[k], x[e + k], x[e + 4 + k]);
    const float top = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);

    if (__any_sync(kAll, top >= xt)) {
      if (xt == -INFINITY) {
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const int64_t id = u.first(mine + (e / kVec) * kThr) + e % kVec;
          const bool there = mine + (e / kVec) * kThr < u1 && id >= 0 && id < a.V;
          before += there && (x[e] > xt || id < token) ? 1 : 0;
        }
      } else {
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
          const int64_t id = u.first(mine + j * kThr);
          const float over = id + kVec <= token ? xt_below : xt;
#pragma unroll
          for (int e = 0; e < kVec; ++e) before += x[j * kVec + e] > over ? 1 : 0;
          if (id < token && id + kVec > token) {  // the unit of the token itself: its equals before it
#pragma unroll
            for (int e = 0; e < kVec; ++e) before += x[j * kVec + e] == xt && id + e < token ? 1 : 0;
          }
        }
      }
    }

    if (n > 0) {
      const u64 known = __shfl_sync(kAll, *s_bound, 0);
      if (known > bound) bound = known;
      if (__any_sync(kAll, top >= key_value(bound))) {
        lane_top = fmaxf(lane_top, top);
        // n tokens at least reach the n-th largest of the lanes' maxima.
        const float nth = __shfl_sync(kAll, sorted_down(lane_top), n - 1);
        const u64 reached = (u64)float_order_key(nth) << 32;  // before every token of that value
        if (nth > -INFINITY && reached > bound) bound = reached;
        if (lane == 0) atomicMax(&s.bound, bound);
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
          const float at_least = key_value(bound);
          float unit_top = x[j * kVec];
#pragma unroll
          for (int e = 1; e < kVec; ++e) unit_top = fmaxf(unit_top, x[j * kVec + e]);
          if (!__any_sync(kAll, unit_top >= at_least)) continue;
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            const float v = x[j * kVec + e];
            const unsigned hit = __ballot_sync(kAll, v >= at_least);
            if (!hit) continue;
            const u64 key = v >= at_least ? value_id_key(v, (uint32_t)(u.first(mine + j * kThr) + e)) : 0;
            const unsigned in = __ballot_sync(kAll, key > bound);
            if (key > bound) buf[held + __popc(in & ((1u << lane) - 1u))] = key;
            held += __popc(in);
            if (held >= 32) take(32);
          }
        }
      } else {
        lane_top = fmaxf(lane_top, top);
      }
    }

    q.raise(fmaxf(q.m, top), c);
    if (top == INFINITY) {  // they share everything
#pragma unroll
      for (int e = 0; e < kN; ++e) q.S += x[e] == INFINITY ? 1.0f : 0.0f;
    } else {
      const float m = q.m == -INFINITY ? 0.0f : q.m;
      const float2 m2 = make_float2(-m, -m), c2 = make_float2(c, c);
      float2 S2 = make_float2(q.S, 0.0f), E2 = make_float2(q.E, 0.0f);
#pragma unroll
      for (int e = 0; e < kN; e += 2) {
        float2 d = mul2(add2(make_float2(x[e], x[e + 1]), m2), c2);
        d.x = fmaxf(d.x, kLeastD);
        d.y = fmaxf(d.y, kLeastD);
        const float2 w = make_float2(ex2(d.x), ex2(d.y));
        S2 = add2(S2, w);
        E2 = fma2(w, d, E2);
      }
      q.S = S2.x + S2.y;
      q.E = E2.x + E2.y;
    }
  }
  while (held > 0) take(min(held, 32));

  // The warp's, the block's, the cluster's.
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    Sums o;
    o.m = __shfl_xor_sync(kAll, q.m, d);
    o.S = __shfl_xor_sync(kAll, q.S, d);
    o.E = __shfl_xor_sync(kAll, q.E, d);
    q.join(o, c);
    before += __shfl_xor_sync(kAll, before, d);
  }
  s.list[warp][lane] = best;
  if (lane == 0) {
    s.sums[warp] = q;
    s.count[warp] = before;
  }
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < kWarps; ++w) {
      q.join(s.sums[w], c);
      before += s.count[w];
      if (n > 0) best = merged(best, s.list[w][lane]);
    }
    s.best[lane] = best;
    if (lane == 0) s.part = make_float4(q.m, q.S, q.E, __int_as_float(before));
  }
  if (size > 1) {
    cluster_sync();
    if (rank == 0 && warp == 0) {
      for (int k = 1; k < size; ++k) {
        const float4 p = dsmem_f4(dsmem(&s.part, (uint32_t)k));
        Sums o = {p.x, p.y, p.z};
        q.join(o, c);
        before += __float_as_int(p.w);
        if (n > 0) best = merged(best, dsmem_u64(dsmem(&s.best[lane], (uint32_t)k)));
      }
    }
    cluster_sync();  // the others' shared memory has been read
  }
  if (rank != 0 || warp != 0) return;
  const float log_s = logf(q.S);
  auto logprob = [&](float x) {
    if (!fine) return __uint_as_float(0x7fffffffu);
    return (x == q.m ? 0.0f : (x - q.m) / temp) - (q.m == -INFINITY ? INFINITY : log_s);
  };
  if (lane == 0) {
    const bool none = token == -1;
    if (!fine || (!given && !none)) dev_error(a.ctl, DEV_ERR_DATA);
    if (a.logprob) a.logprob[r] = none && fine ? 0.0f : given ? logprob(xt) : NAN;
    if (a.rank) a.rank[r] = none ? 0 : given ? before : -1;
    if (a.entropy) a.entropy[r] = !fine ? NAN : q.m == -INFINITY ? 0.0f : log_s - q.E / q.S * kLn2;
    if (a.lse) a.lse[r] = !fine ? NAN : q.m == -INFINITY ? -INFINITY : q.m / temp + log_s;
  }
  if (lane < n) {
    const bool there = best > least;
    if (a.top_ids) a.top_ids[(int64_t)r * n + lane] = there ? (int)key_id(best) : -1;
    if (a.top_logprob) a.top_logprob[(int64_t)r * n + lane] = there ? logprob(key_value(best)) : fine ? -INFINITY : NAN;
  }
}

template <typename T, int kUnits>
cudaError_t launch(const ScoreArgs& a, cudaStream_t stream) {
  // CTAs of a row: as many as still leave each a few batches, while the rows do not fill the SMs.
  const int units = a.V / (16 / (int)sizeof(T)) + 1;
  int size = 1;
  while (size < kMaxCluster && (int64_t)a.rows * size < 4 * (int64_t)num_sms() && units / (2 * size) >= kUnits * kThr) size <<= 1;
  if ((int64_t)a.rows * size > 0x7fffffff) return cudaErrorInvalidConfiguration;
  static FuncOnce once;
  cudaError_t e = once.set((const void*)score_kernel<T, kUnits>, 0, true);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows * size));
  cfg.blockDim = dim3(kThr);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)size;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, score_kernel<T, kUnits>, a, size);
}

}  // namespace

cudaError_t launch_score(const ScoreArgs& a, cudaStream_t stream) {
  return a.dtype == DOMINO_BF16 ? launch<__nv_bfloat16, 4>(a, stream) : launch<float, 4>(a, stream);
}

}  // namespace domino
