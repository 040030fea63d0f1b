// What a row of logits says of a given token: its log-probability and rank, the row's entropy and its most likely tokens
// (domino_token_logprobs; the definition is in domino.h).
//
// One pass over the row. With m the maximum so far, d = (x - m) / T in log2 units and w = 2^d, a thread keeps S = sum w and
// E = sum w d; when m / T rises by r, E' = 2^-r (E - r S) and S' = 2^-r S. Then
//   log sum exp = m / T + log S,   entropy = log S - E / S,   log p(t) = (x_t - m) / T - log S,
// where m is the true maximum, so that d <= 0 but for what m's product with log2(e) / T is rounded by (half a unit at most): log S and E / S share
// that and lose no more to it than its last bits. What they leave of a row that one token has, on the wrong side of 0, is set to 0.
//   Rank: the given token's logit is known beforehand; tokens before it in (logit, id) are counted, in the batches of a warp that
//     have one.
//   Most likely tokens: the pass leaves every thread's maxima of up to 16 stretches of its tokens in shared memory. The n-th largest of
//     the threads' maxima is reached by n tokens, so only stretches that reach it (hardly more than n) are read again, and what
//     reaches it there is sorted. (Collected on the way, in 32 (value, id) keys a warp, they took longer than the rest: 1088
//     rows 109 us without and 182 with the 8 most likely.)
// A cluster of CTAs takes a row when there are few; their results meet in the first one's shared memory.
//
// Many rows: 1088 of 151,936 in bf16 with the 8 most likely tokens 97 us, 3.4 TB/s (without them 84), at 12.7 instructions a logit, 71 % of the issue
// slots and 45 % of memory. The rest is unlike blocks, in 1.8 rounds that take 2: a row whose token is the most likely counts its
// rank in a batch or two, one whose token lies in the bulk in nearly all (all rows of the first kind 76 us, of the second 125). Four
// blocks an SM (measured at 95 us; three: 98, five: 107; twice as many of 128 threads: 98); a row over two blocks 105. One row: 12.3 us a call,
// launch, two batches, three joins and a cluster barrier behind one another.
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
__device__ __forceinline__ int dsmem_s32(uint32_t at) {
  int x;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ float4 dsmem_f4(uint32_t at) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(at) : "memory");
  return x;
}

// Where a maximum's product with c is below this, its weights are in units of log2 from the product as it is rounded: d is one
// multiply-add from the logit, and the rounding, half a unit at most, is nobody's error. Beyond it (temperatures of 1e-6 and less,
// logits of 1e8), where the rounding may be more than the exponential holds, they are from the maximum itself: d = (x - m) c.
constexpr float kRoundedBelow = 16777216.0f;  // 2^24
__device__ __forceinline__ bool rounded(float at) { return fabsf(at) < kRoundedBelow; }

// The sums of part of a row; `m` the maximum of its logits.
// S is held with what its additions round away, r: where one token has nearly all, the logarithm of S is that of the rest.
struct Sums {
  float m, S, E, r;
  __device__ __forceinline__ void add(float x) {
    const float t = S + x, y = t - S;
    r += (S - (t - y)) + (x - y);
    S = t;
  }
  __device__ __forceinline__ void raise(float to, float c) {  // to >= m
    if (to == m) return;
    // From one point to the other, each rounded or not: products that no addition may take up.
    const float at = __fmul_rn(to, c), was = __fmul_rn(m, c);
    float d = __fsub_rn(was, at);
    if (!rounded(at) || !rounded(was)) d = rounded(at) ? fmaf(m, c, -at) : rounded(was) ? -fmaf(to, c, -was) : (m - to) * c;
    const float f = ex2(d);
    E = f == 0.0f ? 0.0f : f * fmaf(d, S, E);
    S *= f;
    r *= f;
    m = to;
  }
  __device__ __forceinline__ void join(Sums o, float c) {
    const float to = fmaxf(m, o.m);
    raise(to, c);
    o.raise(to, c);
    add(o.S);
    r += o.r;
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
__device__ __forceinline__ float merged(float a, float b) {
  const int lane = threadIdx.x & 31;
  float x = fmaxf(a, __shfl_sync(kAll, b, 31 - lane));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const float y = __shfl_xor_sync(kAll, x, d);
    x = (lane & d) == 0 ? fmaxf(x, y) : fminf(x, y);
  }
  return x;
}
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

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A row's elements in units of 16 aligned bytes: unit u holds elements [u kVec - skew, + kVec).
template <typename T>
struct Units {
  static constexpr int kVec = 16 / sizeof(T);
  const T* row;
  int V, skew, units;
  int whole0, whole1;  // units [whole0, whole1) are the row's alone
  __device__ __forceinline__ Units(const T* r, int n) : row(r), V(n) {
    skew = (int)(((uintptr_t)r & 15) / sizeof(T));
    units = (int)(((int64_t)skew + V + kVec - 1) / kVec);
    whole0 = skew ? 1 : 0;
    whole1 = (int)(((int64_t)skew + V) / kVec);
  }
  __device__ __forceinline__ int64_t first(int u) const { return (int64_t)u * kVec - skew; }
  // Units u, u + kThr, ... of which those from `end` on are -inf, as are elements that are not the row's; neither is read.
  template <int kUnits>
  __device__ __forceinline__ void load(int batch, int end, uint4 (&x)[kUnits]) const {
    const int u = batch + (int)threadIdx.x;
    if (batch >= whole0 && batch + kUnits * kThr <= min(whole1, end)) {
      const uint4* at = (const uint4*)(row - skew) + u;
#pragma unroll
      for (int j = 0; j < kUnits; ++j)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(x[j].x), "=r"(x[j].y), "=r"(x[j].z), "=r"(x[j].w)
                     : "l"(at + j * kThr));
    } else {
#pragma unroll
      for (int j = 0; j < kUnits; ++j) x[j] = load_some(u + j * kThr, end);
    }
  }
  __device__ __noinline__ uint4 load_some(int u, int end) const {
    const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    if (u >= end) return make_uint4(none, none, none, none);
    if (u >= whole0 && u < whole1) return __ldg((const uint4*)(row - skew) + u);
    const int64_t i0 = first(u);
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
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float value(const uint4& x, int e) {
    const uint32_t w = sizeof(T) == 4 ? (e == 0 ? x.x : e == 1 ? x.y : e == 2 ? x.z : x.w)
                                      : (e < 2 ? x.x : e < 4 ? x.y : e < 6 ? x.z : x.w);
    return sizeof(T) == 4 ? __uint_as_float(w) : __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
  }
  // The largest of kUnits units; a NaN counts as -inf.
  template <int kUnits>
  static __device__ __forceinline__ float largest(const uint4 (&x)[kUnits]) {
    if (sizeof(T) == 2) {
      uint32_t m = 0xff80ff80u;
#pragma unroll
      for (int j = 0; j < kUnits; ++j) m = max_bf16x2(m, max_bf16x2(max_bf16x2(x[j].x, x[j].y), max_bf16x2(x[j].z, x[j].w)));
      return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kUnits; ++j)
      m = max3(m, max3(__uint_as_float(x[j].x), __uint_as_float(x[j].y), -INFINITY),
               max3(__uint_as_float(x[j].z), __uint_as_float(x[j].w), -INFINITY));
    return m;
  }
};

constexpr int kStretches = 16;
struct Smem {
  union {
    float tops[kStretches][kThr];  // of each stretch of a thread's tokens
    u64 list[kWarps][32];          // after them
  };
  u64 buf[kWarps][64];
  float warp_tops[kWarps][32];
  float reached;
  Sums sums[kWarps];
  int count[kWarps];
  int works;
  uint16_t work[kStretches * kThr];  // stretches to be read again
  alignas(16) Sums part;             // the CTA's, read as four floats, and
  int part_count;
  u64 best[32];
};

// The value just below x.
__device__ __forceinline__ float below(float x) {
  return x == 0.0f ? __uint_as_float(0x80000001u) : order_key_float(float_order_key(x) - 1u);
}

template <typename T, int kUnits>
__global__ void __launch_bounds__(kThr, 4) score_kernel(const ScoreArgs a, int size) {
  using U = Units<T>;
  constexpr int kVec = U::kVec;
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
  const int n = a.top_n;
  const u64 least = value_id_key(-INFINITY, 0);
  if (threadIdx.x == 0) s.works = 0;

  Sums q = {-INFINITY, 0.0f, 0.0f, 0.0f};
  int before = 0;
  constexpr int kBatch = kUnits * kThr;  // units
  const int batches = (u1 - u0 + kBatch - 1) / kBatch, stretch = max(1, (batches + kStretches - 1) / kStretches);  // in batches
  float here = -INFINITY, thread_top = -INFINITY;  // of the stretch, of all
  int in_stretch = 0, stretches = 0;

  uint4 cur[kUnits], next[kUnits];
  // One of them by a number that the compiler does not know: the paths that few batches take are loops over units, or
  // their code, once for every element, would not fit the instruction cache (1088 rows 235 us).
  auto unit = [&](int j) {
    uint4 x = cur[0];
#pragma unroll
    for (int i = 1; i < kUnits; ++i)
      if (i == j) x = cur[i];
    return x;
  };
  u.template load<kUnits>(u0, u1, next);
#pragma unroll 2
  for (int ub = u0; ub < u1; ub += kBatch) {
#pragma unroll
    for (int j = 0; j < kUnits; ++j) cur[j] = next[j];
    if (ub + kBatch < u1) u.template load<kUnits>(ub + kBatch, u1, next);
    const float top = U::template largest<kUnits>(cur);

    if (__any_sync(kAll, top >= xt)) {
      const int mine = ub + (int)threadIdx.x;  // unit j of this thread: mine + j kThr
      const float xt_below = below(xt);
#pragma unroll 1
      for (int j = 0; j < kUnits; ++j) {
        const uint4 x = unit(j);
        const int64_t id = u.first(mine + j * kThr);
        if (xt == -INFINITY) {
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            const bool there = mine + j * kThr < u1 && id + e >= 0 && id + e < a.V;
            before += there && (U::value(x, e) > xt || id + e < token) ? 1 : 0;
          }
        } else {
          const float over = id + kVec <= token ? xt_below : xt;
#pragma unroll
          for (int e = 0; e < kVec; ++e) before += U::value(x, e) > over ? 1 : 0;
          if (id < token && id + kVec > token) {  // the unit of the token itself: its equals before it
#pragma unroll
            for (int e = 0; e < kVec; ++e) before += U::value(x, e) == xt && id + e < token ? 1 : 0;
          }
        }
      }
    }

    here = fmaxf(here, top);
    if (n > 0 && (++in_stretch == stretch || ub + kBatch >= u1)) {
      s.tops[stretches++][threadIdx.x] = here;
      thread_top = fmaxf(thread_top, here);
      here = -INFINITY;
      in_stretch = 0;
    }

    q.raise(fmaxf(q.m, top), c);
    const float m = q.m == -INFINITY ? 0.0f : q.m, at = __fmul_rn(m, c);
    if (!rounded(at)) {
#pragma unroll 1
      for (int j = 0; j < kUnits; ++j) {
        const uint4 x = unit(j);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {  // infinities share everything
          const float v = U::value(x, e), d = v == m ? 0.0f : fmaxf((v - m) * c, kLeastD), w = ex2(d);
          q.add(w);
          q.E = fmaf(w, d, q.E);
        }
      }
    } else {
      const float2 c2 = make_float2(c, c), n2 = make_float2(-at, -at);
      float2 S2 = make_float2(0.0f, 0.0f), E2 = make_float2(q.E, 0.0f);
#pragma unroll
      for (int j = 0; j < kUnits; ++j)
#pragma unroll
        for (int e = 0; e < kVec; e += 2) {
          float2 d = fma2(make_float2(U::value(cur[j], e), U::value(cur[j], e + 1)), c2, n2);
          d.x = fmaxf(d.x, kLeastD);
          d.y = fmaxf(d.y, kLeastD);
          const float2 w = make_float2(ex2(d.x), ex2(d.y));
          S2 = add2(S2, w);
          E2 = fma2(w, d, E2);
        }
      q.add(S2.x);
      q.add(S2.y);
      q.E = E2.x + E2.y;
    }
  }

  u64 best = 0;
  if (n > 0) {
    // n tokens at least reach the n-th largest of the threads' maxima.
    float t = sorted_down(thread_top);
    s.warp_tops[warp][lane] = t;
    __syncthreads();
#pragma unroll 1
    for (int step = kWarps / 2; step > 0; step >>= 1) {
      if (warp < step) {
        t = merged(t, s.warp_tops[warp + step][lane]);
        s.warp_tops[warp][lane] = t;
      }
      if (step == 1 && warp == 0 && lane == n - 1) s.reached = t;
      __syncthreads();
    }
    const float reached = s.reached;
    for (int k = 0; k < stretches && thread_top >= reached; ++k) {
      const float top = s.tops[k][threadIdx.x];
      if (top >= reached && top > -INFINITY) s.work[atomicAdd(&s.works, 1)] = (uint16_t)(k * kThr + threadIdx.x);
    }
    __syncthreads();
    // A warp reads a stretch again, an element a lane; what is not below the bound goes to a buffer, which is sorted by 32.
    u64 bound = max((u64)float_order_key(reached) << 32, least);
    u64* buf = s.buf[warp];
    int held = 0;
    const int works = s.works;
    for (int i = warp; i < works || held > 0; i += kWarps) {
      if (i < works) {
        const int k = s.work[i] / kThr, t = s.work[i] % kThr;
        for (int b = k * stretch; b < min((k + 1) * stretch, batches); ++b) {
          const int at = u0 + b * kBatch + (lane / kVec) * kThr + t;
          const int64_t id = u.first(at) + lane % kVec;
          u64 key = 0;
          if (lane < kUnits * kVec && at < u1 && id >= 0 && id < a.V) {
            const float v = to_f<T>(row[id]);
            if (v > -INFINITY) key = value_id_key(v, (uint32_t)id);  // and no NaN
          }
          const unsigned in = __ballot_sync(kAll, key > bound);
          if (key > bound) buf[held + __popc(in & ((1u << lane) - 1u))] = key;
          held += __popc(in);
          if (held >= 32) {
            __syncwarp();
            held -= 32;
            best = merged(best, sorted_down(buf[held + lane]));
            bound = max(bound, __shfl_sync(kAll, best, n - 1));
            __syncwarp();
          }
        }
      } else {
        __syncwarp();
        best = merged(best, sorted_down(lane < held ? buf[lane] : 0ull));
        held = 0;
      }
    }
    __syncthreads();  // the stretches' maxima have been read
  }

  // The warp's, the block's, the cluster's. Blocks of a cluster by the warps of the first one, whose reads of the others' memory are
  // then on their way together.
  {
    float m = q.m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, d));
    q.raise(m, c);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float S = __shfl_xor_sync(kAll, q.S, d), r = __shfl_xor_sync(kAll, q.r, d);
      q.add(S);
      q.r += r;
      q.E += __shfl_xor_sync(kAll, q.E, d);
    }
    before = __reduce_add_sync(kAll, before);
  }
  auto join_warps = [&] {
#pragma unroll 1
    for (int step = kWarps / 2; step > 0; step >>= 1) {
      if (warp < 2 * step) {
        s.list[warp][lane] = best;
        if (lane == 0) {
          s.sums[warp] = q;
          s.count[warp] = before;
        }
      }
      __syncthreads();
      if (warp < step) {
        q.join(s.sums[warp + step], c);
        before += s.count[warp + step];
        if (n > 0) best = merged(best, s.list[warp + step][lane]);
      }
    }
  };
  join_warps();
  if (size > 1) {
    if (warp == 0) {
      s.best[lane] = best;
      if (lane == 0) {
        s.part = q;
        s.part_count = before;
      }
    }
    cluster_sync();
    if (rank == 0) {
      float4 p[kMaxCluster / kWarps];
      int counts[kMaxCluster / kWarps];
      u64 x[kMaxCluster / kWarps];
#pragma unroll
      for (int i = 0; i < kMaxCluster / kWarps; ++i) {
        const int k = warp + i * kWarps;
        p[i] = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
        x[i] = 0;
        counts[i] = 0;
        if (k < size) {
          p[i] = dsmem_f4(dsmem(&s.part, (uint32_t)k));
          counts[i] = dsmem_s32(dsmem(&s.part_count, (uint32_t)k));
          x[i] = dsmem_u64(dsmem(&s.best[lane], (uint32_t)k));
        }
      }
      q = Sums{p[0].x, p[0].y, p[0].z, p[0].w};
      before = counts[0];
      best = x[0];
#pragma unroll
      for (int i = 1; i < kMaxCluster / kWarps; ++i) {
        q.join(Sums{p[i].x, p[i].y, p[i].z, p[i].w}, c);
        before += counts[i];
        if (n > 0) best = merged(best, x[i]);
      }
      __syncthreads();
      join_warps();
    }
    cluster_sync();  // the others' shared memory has been read
  }
  if (rank != 0 || warp != 0) return;
  // log2 of the sum from m c as it is rounded, or from m, and the logarithm from m itself.
  const float log_s = log2f(q.S) + (q.r != 0.0f ? q.r / q.S * kLog2e : 0.0f), at = __fmul_rn(q.m, c);
  const float log_m = (rounded(at) ? log_s - fmaf(q.m, c, -at) : log_s) * kLn2;
  auto logprob = [&](float x) {
    if (!fine) return __uint_as_float(0x7fffffffu);
    if (q.m == -INFINITY || x == -INFINITY) return -INFINITY;
    const float d = x == q.m ? 0.0f : x - q.m;  // beyond fp32 the quotients' difference need not be
    return fminf((isinf(d) ? x / temp - q.m / temp : d / temp) - log_m, 0.0f);
  };
  if (lane == 0) {
    const bool none = token == -1;
    if (!fine || (!given && !none)) dev_error(a.ctl, DEV_ERR_DATA);
    if (a.logprob) a.logprob[r] = none && fine ? 0.0f : given ? logprob(xt) : NAN;
    if (a.rank) a.rank[r] = none ? 0 : given ? before : -1;
    if (a.entropy) a.entropy[r] = !fine ? NAN : q.m == -INFINITY ? 0.0f : fmaxf((log_s - q.E / q.S) * kLn2, 0.0f);
    if (a.lse) a.lse[r] = !fine ? NAN : rounded(at) ? (at + log_s) * kLn2 : q.m / temp + log_s * kLn2;
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
