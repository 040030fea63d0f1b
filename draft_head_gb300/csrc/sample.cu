// The draw from a row of logits under top-k, top-p and min-p with given
// Gumbel noise (domino_sample; the definition is in domino.h).
//
// What stays of a row under top-k and top-p is a prefix of its order (logit
// descending, id ascending), so each is a bound on the 64-bit key of (value,
// id): top-k by counting the keys above a bound, top-p by summing their weights
// exp((logit - max) / T). min-p is a test of the weight itself. The draw is the
// argmax of logit / T + noise over what stayed.
//
// A cluster of up to 16 CTAs takes a row, each a slice that it reads once from
// memory and keeps in shared memory (fp32). Steps, each over the slice:
//   maximum            merged over the cluster; ends a greedy row
//   histogram          of (max - logit) / T: 1/64 nat a bin up to 12, then half
//                      a nat, with counts and weights (integers of 2^-30, so that no order
//                      of the atomics changes them); summed over the cluster, and
//                      every CTA finds the bins of the two bounds in the sums
//   short list         when all that can stay are at most kList tokens (peaked
//                      rows): they go to CTA 0, which orders them and does the rest
//   otherwise          the bin of each bound alone goes to CTA 0, which finds the
//                      exact key; a bin of more than kList tokens (equal logits, say)
//                      is first split by the bits of the keys. Every CTA then draws
//                      from what stayed of its slice, reading its noise.
// Bound by memory (the logits once, the noise where tokens stay) when there are many
// rows, and by the cluster's barriers (about a microsecond each) for one row.
#include <math.h>

#include "common.cuh"

namespace domino {

namespace {

constexpr int kThr = 256, kWarps = kThr / 32;
constexpr int kMaxCluster = 16;
constexpr int kBins = 1024, kNear = 768;  // 64 bins a nat up to 12 nats, then 2 a nat; the last: the rest
constexpr int kList = 2048, kPer = kList / kThr;
constexpr int kMaxSlice = 48 * 1024;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t dsmem(const void* p, uint32_t rank) {
  uint32_t ra;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(p)), "r"(rank));
  return ra;
}
__device__ __forceinline__ uint32_t ld_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ unsigned long long ld_u64(uint32_t a) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_u32(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void st_u64(uint32_t a, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_u32(uint32_t a, uint32_t v) {
  uint32_t o;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(o) : "r"(a), "r"(v) : "memory");
  return o;
}

typedef unsigned long long u64;

// Shared memory of a CTA before its slice.
struct Smem {
  union {
    uint32_t hist[3][kBins];  // counts; weights in two 15-bit halves
    u64 list[kList];          // CTA 0: keys gathered from the cluster
  };
  u64 mass[kBins];  // sums over the cluster (a CTA holds those of its bins before they are shared)
  uint32_t cnt[kBins];
  u64 part_key[kMaxCluster];  // from each CTA
  u64 part_lo[kMaxCluster];
  float part_sum[kMaxCluster];
  u64 red[kWarps];
  u64 red2[kWarps];
  float redf[kWarps];
  u64 result[4];  // CTA 0's answer
  int n_list;
  int found_bin;
  u64 found_cnt, found_mass;
};

struct Row {
  float lmax, inv_t, temp;
  float min_p;
  __device__ __forceinline__ float dist(float l) const { return l == lmax ? 0.0f : (lmax - l) * inv_t; }
  // Weight of a token in units of 2^-30.
  __device__ __forceinline__ uint32_t fixed(float d) const {
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(d * -1.4426950408889634f));
    return (uint32_t)__float2uint_rn(w * 1073741824.0f);
  }
  __device__ __forceinline__ float weight(float l) const { return l == lmax ? 1.0f : expf((l - lmax) * inv_t); }
};

__device__ __forceinline__ int bin_of(float d) {
  // Monotone in d, so in the order of the logits.
  if (d < 12.0f) return (int)(d * 64.0f);
  const float b = (d - 12.0f) * 2.0f + (float)kNear;
  return b < (float)(kBins - 1) ? (int)b : kBins - 1;
}

__device__ __forceinline__ u64 block_max(u64 v, u64* red) {
  v = warp_max_u64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v = red[w] > v ? red[w] : v;
  return v;
}
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += red[w];
  return v;
}
// Exclusive prefix sums of (a, b) over the block's threads, in thread order.
__device__ __forceinline__ void block_scan(u64& a, u64& b, u64* red, u64* red2) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 p = __shfl_up_sync(0xffffffffu, x, o), q = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) { x += p; y += q; }
  }
  __syncthreads();
  if (lane == 31) { red[warp] = x; red2[warp] = y; }
  __syncthreads();
  u64 bx = 0, by = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) { bx += red[w]; by += red2[w]; }
  a = bx + x - a;
  b = by + y - b;
}

// First place in cnt / mass (as `by_mass` says) where the sum up to and with it reaches
// `target` (the last one if none does). All threads get it, and the sums before it.
__device__ __forceinline__ void find(Smem& s, bool by_mass, double target, int& bin, u64& cnt_before, u64& mass_before) {
  constexpr int kEach = kBins / kThr;
  const int b0 = threadIdx.x * kEach;
  u64 c = 0, m = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) { c += s.cnt[b0 + j]; m += s.mass[b0 + j]; }
  u64 cb = c, mb = m;
  block_scan(cb, mb, s.red, s.red2);
  const double before = by_mass ? (double)mb : (double)cb, after = by_mass ? (double)(mb + m) : (double)(cb + c);
  if ((threadIdx.x == 0 || before < target) && (after >= target || threadIdx.x == kThr - 1)) {
    int j = 0;
    for (; j < kEach - 1; ++j) {
      const u64 nc = cb + s.cnt[b0 + j], nm = mb + s.mass[b0 + j];
      if ((by_mass ? (double)nm : (double)nc) >= target) break;
      cb = nc;
      mb = nm;
    }
    s.found_bin = b0 + j;
    s.found_cnt = cb;
    s.found_mass = mb;
  }
  __syncthreads();
  bin = s.found_bin;
  cnt_before = s.found_cnt;
  mass_before = s.found_mass;
  __syncthreads();
}

// Sums the CTAs' histograms: each CTA takes kBins / size bins, then all read all sums.
__device__ __forceinline__ void share_histogram(Smem& s, uint32_t rank, uint32_t size) {
  cluster_sync();
  const int per = kBins / (int)size;
  // A thread sums up to four CTAs' counts of a bin, all loads in flight at once.
  const int tpb = size > 4 ? (int)size / 4 : 1;  // threads per bin
  const int first = threadIdx.x % tpb;
  for (int x = threadIdx.x / tpb; x < per; x += kThr / tpb) {
    const int b = (int)rank * per + x;
    uint32_t c[4], hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t k = (uint32_t)(first + tpb * j);
      const bool on = k < size;
      c[j] = on ? ld_u32(dsmem(&s.hist[0][b], k)) : 0u;
      hi[j] = on ? ld_u32(dsmem(&s.hist[1][b], k)) : 0u;
      lo[j] = on ? ld_u32(dsmem(&s.hist[2][b], k)) : 0u;
    }
    uint32_t cs = c[0] + c[1] + c[2] + c[3];
    u64 m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m += ((u64)hi[j] << 15) + lo[j];
    for (int o = 1; o < tpb; o <<= 1) {
      cs += __shfl_xor_sync(0xffffffffu, cs, o);
      m += __shfl_xor_sync(0xffffffffu, m, o);
    }
    if (first == 0) {
      s.cnt[b] = cs;
      s.mass[b] = m;
    }
  }
  cluster_sync();
  if (size > 1) {
    uint32_t c[kBins / kThr];
    u64 m[kBins / kThr];
#pragma unroll
    for (int j = 0; j < kBins / kThr; ++j) {
      const int b = threadIdx.x + j * kThr;
      c[j] = ld_u32(dsmem(&s.cnt[b], (uint32_t)(b / per)));
      m[j] = ld_u64(dsmem(&s.mass[b], (uint32_t)(b / per)));
    }
#pragma unroll
    for (int j = 0; j < kBins / kThr; ++j) {
      const int b = threadIdx.x + j * kThr;
      if ((uint32_t)(b / per) != rank) {
        s.cnt[b] = c[j];
        s.mass[b] = m[j];
      }
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void add_weight(Smem& s, int b, uint32_t w) {
  atomicAdd(&s.hist[0][b], 1u);
  if (w >> 15) atomicAdd(&s.hist[1][b], w >> 15);
  if (w & 0x7fffu) atomicAdd(&s.hist[2][b], w & 0x7fffu);
}
__device__ __forceinline__ void clear_histogram(Smem& s) {
  for (int x = threadIdx.x; x < 3 * kBins; x += kThr) (&s.hist[0][0])[x] = 0u;
}

// Gathers the keys for which `in` holds in CTA 0's list.
template <typename In>
__device__ __forceinline__ void gather(Smem& s, const float* vals, int n, int id0, In in) {
  const uint32_t counter = dsmem(&s.n_list, 0);
  for (int p = threadIdx.x; p < n; p += kThr) {
    const float l = vals[p];
    if (l == l && in(l, id0 + p)) {
      const uint32_t at = add_u32(counter, 1u);
      if (at < (uint32_t)kList) st_u64(dsmem(&s.list[at], 0), value_id_key(l, (uint32_t)(id0 + p)));
    }
  }
}

// CTA 0: orders the list (largest key first), in place. Up to a key per thread, each is ranked
// against all; beyond, a bitonic sort (66 short steps for 2048 keys).
__device__ __forceinline__ void order_list(Smem& s, int n) {
  if (n <= kThr) {
    const u64 key = (int)threadIdx.x < n ? s.list[threadIdx.x] : 0;
    int rank = 0, x = 0;
    for (; x + 8 <= n; x += 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) rank += s.list[x + j] > key;
    }
    for (; x < n; ++x) rank += s.list[x] > key;
    __syncthreads();
    if ((int)threadIdx.x < n) s.list[rank] = key;
    __syncthreads();
    return;
  }
  int size = 2 * kThr;
  while (size < n) size <<= 1;
  for (int x = n + threadIdx.x; x < size; x += kThr) s.list[x] = 0;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
#pragma unroll 4
      for (int i = threadIdx.x; i < size / 2; i += kThr) {
        const int lo = ((i & ~(j - 1)) << 1) | (i & (j - 1)), hi = lo | j;
        const u64 x = s.list[lo], y = s.list[hi];
        if ((x < y) == ((lo & k) == 0)) {
          s.list[lo] = y;
          s.list[hi] = x;
        }
      }
      __syncthreads();
    }
  }
}

// CTA 0, ordered list of n keys: the key of the last that stays, when `cnt` more may stay (cnt > 0),
// or when those stay whose weight before them is below `aim` (by_mass). In `mass`, the weight of what stays.
__device__ __forceinline__ u64 cut_list(Smem& s, const Row& r, int n, bool by_mass, u64 cnt, double aim, u64* mass) {
  u64 own[kPer], c = 0, m = 0;
  const int x0 = threadIdx.x * kPer;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    own[j] = x0 + j < n ? (u64)r.fixed(r.dist(key_value(s.list[x0 + j]))) : 0;
    m += own[j];
  }
  block_scan(m, c, s.red, s.red2);
  u64 last = ~0ull, sum = 0;  // smallest key that stays
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int x = x0 + j;
    const bool stays = x < n && (by_mass ? (double)m < aim : (u64)x < cnt);
    if (stays) {
      last = s.list[x];
      sum = m + own[j];
    }
    m += own[j];
  }
  // The keys fall and the sums grow with the place, so the last one has the extremes.
  const u64 inv = block_max(~last, s.red);
  *mass = block_max(sum, s.red);
  return ~inv;
}

template <typename T>
__global__ void __launch_bounds__(kThr) sample_kernel(const SampleArgs a, int slice) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& s = *(Smem*)smem_raw;
  float* vals = (float*)(smem_raw + ((sizeof(Smem) + 15) & ~(size_t)15));
  const uint32_t rank = cluster_rank(), size = cluster_size();
  // All CTAs of the cluster are there before one writes to another (waited for below).
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int row = blockIdx.x / (int)size, t = threadIdx.x, V = a.V;
  const int s0 = min(V, (int)rank * slice), s1 = min(V, s0 + slice);
  const T* src = (const T*)a.logits + (int64_t)row * a.ls + s0;
  const float* g = a.gumbel ? a.gumbel + (int64_t)row * a.gs : nullptr;

  // The slice, in 16-byte units from the one that holds its first element: position p of
  // `vals` is token id0 + p; what lies outside the slice is marked with a NaN.
  constexpr int kVec = 16 / (int)sizeof(T);
  const int skew = (int)(((uintptr_t)src & 15u) / sizeof(T));
  const uint4* vec = (const uint4*)(src - skew);
  const int id0 = s0 - skew, n = s1 > s0 ? (skew + s1 - s0 + kVec - 1) / kVec * kVec : 0;
  float top = -INFINITY;
  int top_id = 0;  // the lowest id of this thread's largest logit: its ids rise
  constexpr int kUnroll = 8;
  for (int q0 = t; q0 < n / kVec; q0 += kThr * kUnroll) {
    uint4 x[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      if (q0 + j * kThr < n / kVec) x[j] = __ldcs(vec + q0 + j * kThr);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int q = q0 + j * kThr;
      if (q >= n / kVec) break;
      float f[kVec];
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        f[e] = sizeof(T) == 4 ? __uint_as_float(w[e & 3])
                              : __uint_as_float((e & 1) ? w[(e >> 1) & 3] & 0xffff0000u : w[(e >> 1) & 3] << 16);
        f[e] = fmaxf(f[e], -INFINITY);  // NaN counts as -inf
        const int id = id0 + q * kVec + e;
        if (id < s0 || id >= s1) {
          f[e] = __uint_as_float(0x7fffffffu);
        } else if (f[e] > top) {
          top = f[e];
          top_id = id;
        }
      }
#pragma unroll
      for (int e = 0; e < kVec; e += 4) *(float4*)(vals + q * kVec + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    }
  }
  Row r;
  r.temp = a.temperature ? a.temperature[row] : 1.0f;
  int top_k = a.top_k ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.0f;
  r.min_p = a.min_p ? a.min_p[row] : 0.0f;
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  // The same for every CTA of the cluster, as every branch on the way to a cluster barrier.
  if (!(r.temp >= 0.0f && r.temp < INFINITY) || top_k < 0 || !(top_p > 0.0f && top_p <= 1.0f) ||
      !(r.min_p >= 0.0f && r.min_p <= 1.0f) || (r.temp > 0.0f && !g)) {
    if (t == 0 && rank == 0) {
      dev_error(a.ctl, DEV_ERR_DATA);
      a.tokens[row] = -1;
      if (a.logprob) a.logprob[row] = NAN;
    }
    return;
  }
  u64 best = block_max(value_id_key(top, (uint32_t)top_id), s.red);
  if (t < (int)size) st_u64(dsmem(&s.part_key[rank], (uint32_t)t), best);
  if (t == 0) s.n_list = 0;
  clear_histogram(s);
  cluster_sync();
  best = 0;
  for (uint32_t k = 0; k < size; ++k) best = s.part_key[k] > best ? s.part_key[k] : best;
  r.lmax = key_value(best);
  if (r.lmax == -INFINITY || r.temp == 0.0f) {
    if (t == 0 && rank == 0) {
      a.tokens[row] = r.lmax == -INFINITY ? -1 : (int)key_id(best);
      if (a.logprob) a.logprob[row] = r.lmax == -INFINITY ? -INFINITY : 0.0f;
    }
    return;
  }
  r.inv_t = 1.0f / r.temp;
  if (top_k >= V) top_k = 0;

  u64 bound = 0;  // keys from here on stay
  if (top_k > 0 || top_p < 1.0f) {
    uint32_t rest = 0;
    u64 rest_w = 0;
    for (int p = t; p < n; p += kThr) {
      const float l = vals[p];
      if (l != l) continue;
      const float d = r.dist(l);
      const int b = bin_of(d);
      if (b < kBins - 1) {
        if (top_p < 1.0f)
          add_weight(s, b, r.fixed(d));
        else
          atomicAdd(&s.hist[0][b], 1u);
      } else {
        ++rest;
        rest_w += r.fixed(d);
      }
    }
    if (rest) {
      atomicAdd(&s.hist[0][kBins - 1], rest);
      atomicAdd(&s.hist[1][kBins - 1], (uint32_t)(rest_w >> 15));
      atomicAdd(&s.hist[2][kBins - 1], (uint32_t)(rest_w & 0x7fffu));
    }
    share_histogram(s, rank, size);
    int bin_k = kBins - 1, bin_p = kBins - 1;
    u64 cnt_k = 0, mass_k = 0, cnt_p = 0, mass_p = 0;
    if (top_k > 0) find(s, false, (double)top_k, bin_k, cnt_k, mass_k);
    // With no top-k the whole weight is the sum of all bins.
    double total = 0.0;
    if (top_p < 1.0f && top_k == 0) {
      u64 m = 0, z = 0;
      for (int b = t; b < kBins; b += kThr) m += s.mass[b];
      u64 before = m;
      block_scan(before, z, s.red, s.red2);
      if (t == kThr - 1) s.found_mass = before + m;
      __syncthreads();
      total = (double)s.found_mass;
      __syncthreads();
      find(s, true, (double)top_p * total, bin_p, cnt_p, mass_p);
    }
    const int bin_all = min(bin_k, bin_p);
    const u64 most = (top_k > 0 ? cnt_k + s.cnt[bin_k] : cnt_p + s.cnt[bin_p]);
    if (most <= (u64)kList) {
      // All that can stay, to CTA 0.
      gather(s, vals, n, id0, [&](float l, int) { return bin_of(r.dist(l)) <= bin_all; });
      cluster_sync();
      if (rank != 0) return;
      int m = s.n_list;
      order_list(s, m);
      u64 mass;
      if (top_k > 0) {
        bound = cut_list(s, r, m, false, (u64)top_k, 0.0, &mass);
        m = min(m, top_k);
        total = (double)mass;
      }
      if (top_p < 1.0f) {
        const u64 k = cut_list(s, r, m, true, 0, (double)top_p * total, &mass);
        bound = k > bound ? k : bound;
      }
      u64 key = 0;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int x = t + j * kThr;
        if (x < m && s.list[x] >= bound) {
          const float l = key_value(s.list[x]), w = r.weight(l);
          if (w >= r.min_p) {
            const uint32_t id = key_id(s.list[x]);
            const u64 c = value_id_key(l / r.temp + g[id], id);
            key = c > key ? c : key;
            sum += w;
          }
        }
      }
      sum = block_sum(sum, s.redf);
      key = block_max(key, s.red);
      // The drawn token's logit, from the thread that has it.
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int x = t + j * kThr;
        if (x < m && key_id(s.list[x]) == key_id(key)) {
          const float l = key_value(s.list[x]);
          a.tokens[row] = (int)key_id(key);
          if (a.logprob) a.logprob[row] = (l == r.lmax ? 0.0f : (l - r.lmax) * r.inv_t) - logf(sum);
        }
      }
      return;
    }

    // The bound of one of the two filters: the bin's keys in CTA 0's list, ordered.
    auto select = [&](int bin, u64 cnt_before, u64 mass_before, bool by_mass, u64 count, double aim, u64 floor_key, u64* mass_out) {
      u64 lo = 0, hi = ~0ull;  // keys of the bin in question
      u64 in_bin = s.cnt[bin];
      bool whole = true;       // all keys of the bin
      while (in_bin > (u64)kList) {
        // Split the keys between the smallest and the largest by their bits.
        u64 kmax = 0, kmin = 0;
        for (int p = t; p < n; p += kThr) {
          const float l = vals[p];
          if (l != l || bin_of(r.dist(l)) != bin) continue;
          const u64 k = value_id_key(l, (uint32_t)(id0 + p));
          if (!whole && (k < lo || k > hi)) continue;
          kmax = k > kmax ? k : kmax;
          kmin = ~k > kmin ? ~k : kmin;
        }
        kmax = block_max(kmax, s.red);
        kmin = block_max(kmin, s.red);
        __syncthreads();
        if (t < (int)size) {
          st_u64(dsmem(&s.part_key[rank], (uint32_t)t), kmax);
          st_u64(dsmem(&s.part_lo[rank], (uint32_t)t), kmin);
        }
        clear_histogram(s);
        cluster_sync();
        hi = 0;
        lo = 0;
        for (uint32_t k = 0; k < size; ++k) {
          hi = s.part_key[k] > hi ? s.part_key[k] : hi;
          lo = s.part_lo[k] > lo ? s.part_lo[k] : lo;
        }
        lo = ~lo;
        int shift = 0;
        while (((hi - lo) >> shift) >= (u64)kBins) ++shift;
        for (int p = t; p < n; p += kThr) {
          const float l = vals[p];
          if (l != l) continue;
          const float d = r.dist(l);
          if (bin_of(d) != bin) continue;
          const u64 k = value_id_key(l, (uint32_t)(id0 + p));
          if (k < lo || k > hi) continue;
          add_weight(s, (int)((hi - k) >> shift), r.fixed(d));
        }
        share_histogram(s, rank, size);
        int sub;
        u64 c, m;
        find(s, by_mass, by_mass ? aim - (double)mass_before : (double)(count - cnt_before), sub, c, m);
        cnt_before += c;
        mass_before += m;
        in_bin = s.cnt[sub];
        const u64 top = hi - ((u64)sub << shift);
        const u64 width = ((u64)1 << shift) - 1;
        hi = top;
        lo = top > width ? top - width : 0;
        whole = false;
      }
      gather(s, vals, n, id0, [&](float l, int id) {
        if (bin_of(r.dist(l)) != bin) return false;
        const u64 k = value_id_key(l, (uint32_t)id);
        return k >= floor_key && (whole || (k >= lo && k <= hi));
      });
      cluster_sync();
      if (rank == 0) {
        const int m = s.n_list;
        order_list(s, m);
        u64 mass;
        const u64 k = cut_list(s, r, m, by_mass, by_mass ? 0 : count - cnt_before, by_mass ? aim - (double)mass_before : 0.0, &mass);
        if (t == 0) {
          s.result[0] = k;
          s.result[1] = mass_before + mass;
          s.n_list = 0;
        }
      }
      cluster_sync();
      *mass_out = ld_u64(dsmem(&s.result[1], 0));
      const u64 k = ld_u64(dsmem(&s.result[0], 0));
      cluster_sync();
      return k;
    };
    u64 mass;
    if (top_k > 0) {
      // The sums that the second search needs are replaced if this one has to split a bin.
      if (top_p < 1.0f) {
        const bool splits = s.cnt[bin_k] > (uint32_t)kList;
        bound = select(bin_k, cnt_k, mass_k, false, (u64)top_k, 0.0, 0, &mass);
        total = (double)mass;
        if (splits) {
          clear_histogram(s);
          cluster_sync();
          for (int p = t; p < n; p += kThr) {
            const float l = vals[p];
            if (l != l) continue;
            const float d = r.dist(l);
            const int b = bin_of(d);
            if (value_id_key(l, (uint32_t)(id0 + p)) >= bound) add_weight(s, b, r.fixed(d));
          }
          share_histogram(s, rank, size);
        }
        find(s, true, (double)top_p * total, bin_p, cnt_p, mass_p);
        bin_p = min(bin_p, bin_k);
      } else {
        bound = select(bin_k, cnt_k, mass_k, false, (u64)top_k, 0.0, 0, &mass);
      }
    }
    if (top_p < 1.0f) {
      const u64 k = select(bin_p, cnt_p, mass_p, true, 0, (double)top_p * total, bound, &mass);
      bound = k > bound ? k : bound;
    }
  }

  // The draw over what stayed of the slice.
  u64 key = 0;
  float sum = 0.0f;
  for (int p0 = t; p0 < n; p0 += kThr * 8) {
    float z[8];
    bool in[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = p0 + j * kThr;
      in[j] = false;
      if (p < n) {
        const float l = vals[p];
        in[j] = l == l && value_id_key(l, (uint32_t)(id0 + p)) >= bound;
      }
      z[j] = in[j] ? __ldcs(g + id0 + p) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!in[j]) continue;
      const int p = p0 + j * kThr;
      const float l = vals[p], w = r.weight(l);
      if (w < r.min_p) continue;
      sum += w;
      const u64 c = value_id_key(l / r.temp + z[j], (uint32_t)(id0 + p));
      key = c > key ? c : key;
    }
  }
  sum = block_sum(sum, s.redf);
  key = block_max(key, s.red);
  if (t == 0) {
    st_u64(dsmem(&s.part_lo[rank], 0), key);
    st_u32(dsmem(&s.part_sum[rank], 0), __float_as_uint(sum));
  }
  cluster_sync();
  if (rank == 0 && t == 0) {
    sum = 0.0f;
    key = 0;
    for (uint32_t k = 0; k < size; ++k) {
      sum += s.part_sum[k];
      key = s.part_lo[k] > key ? s.part_lo[k] : key;
    }
    const int id = (int)key_id(key);
    a.tokens[row] = id;
    if (a.logprob) {
      const float l = fmaxf(to_f<T>(((const T*)a.logits)[(int64_t)row * a.ls + id]), -INFINITY);
      a.logprob[row] = (l == r.lmax ? 0.0f : (l - r.lmax) * r.inv_t) - logf(sum);
    }
  }
}

template <typename T>
cudaError_t launch(const SampleArgs& a, cudaStream_t stream) {
  // Slices of about 10,000 tokens: short enough for several CTAs on an SM and for one row to
  // be read by many SMs, long enough that the barriers do not outweigh the passes.
  int size = 1;
  while (size < kMaxCluster && (a.V + size - 1) / size > 10240) size <<= 1;
  const int slice = ((a.V + size - 1) / size + 31) / 32 * 32;
  if (slice > kMaxSlice || (int64_t)a.rows * size > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const size_t smem = ((sizeof(Smem) + 15) & ~(size_t)15) + (size_t)(slice + 16) * 4;
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows * size));
  cfg.blockDim = dim3(kThr);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)size;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, slice);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream) {
  return a.dtype == DOMINO_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

}  // namespace domino
