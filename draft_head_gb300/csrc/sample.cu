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
// memory; it keeps it in shared memory, or with many rows reads it again from L2. Steps, each
// over the slice:
//   no filter          one pass over logits and noise with a running maximum and sum, and done
//   maximum            of the slice and of 256 groups of the row's tokens, merged over the
//                      cluster; ends a greedy row
//   candidates         a top-k of up to 128: k groups reach the k-th largest group maximum, so
//                      no token below it stays, and about as many tokens as k are not below
//                      it (n of 256 (1 - exp(-n / 256)) = k). top-p alone tries the 128th:
//                      in a peaked row these tokens have the weight that stays. They go to
//                      CTA 0, which does the rest by itself. All other rows:
//   histogram          of (max - logit) / T in kNear bins, and one for the rest, with
//                      counts and (top-p without top-k) weights; integers, so that no
//                      order of the atomics changes them. A bin's weight is kept as what its
//                      tokens lack to the weight at its edge, 2^-21 of that a unit: one 32-bit
//                      atomic, where a sum of weights would need two. Summed over the
//                      cluster; every CTA finds the bounds' bins in the sums
//   short list         when all that can stay are at most kList tokens (peaked
//                      rows): they go to CTA 0, which does the rest by itself
//   otherwise          the bin of each bound alone goes to CTA 0, which finds the
//                      exact key; a bin of more than kList tokens (equal logits, say)
//                      is first split by the bits of the keys. Every CTA then draws
//                      from what stayed of its slice, reading its noise.
// In CTA 0's list, which it holds in registers, a bound is found by histograms over the keys' bits,
// each 1024 times finer than the one before.
// Bound by the instructions of the passes over the slice when there are many rows (memory next: the
// logits once, the noise where tokens stay), and by the cluster's barriers (about a microsecond each)
// for one row.
//
// Vocabulary 151,936, fp32. One row: greedy 4.5 us, top-k 64 with top-p 13, top-k 1000 22 us. 1024 rows: greedy
// 113 us (5.5 TB/s), no filter 218 (5.7 TB/s with the noise; in two passes 404), top-k 64 227, min-p 210, top-p alone
// 416 (peaked rows), mixed settings 320 us; 272 flat rows at top-p of 0.8 to 0.95 alone, where most of the vocabulary
// stays: 317 us.
#include <math.h>

#include "common.cuh"
#include "packed.cuh"

namespace domino {

namespace {

constexpr int kMaxWarps = 16;
constexpr int kMaxCluster = 16;
constexpr int kGroups = 256;  // groups of a row's tokens with a maximum each
constexpr int kBins = 1024, kNear = 1023;  // the first histogram: kNear bins, then one for the rest
constexpr int kList = 2048;
constexpr int kMaxSlice = 48 * 1024;  // shared memory; a bin's lack (below 2^16 a token) stays within 32 bits up to 64 K
constexpr int kManyCtas = 5;          // on an SM with many rows

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
typedef unsigned long long u64;

// Shared memory of a CTA before its slice.
struct Smem {
  union {
    uint32_t hist[4][kBins];  // counts; lacks, or weights in parts
    u64 list[kList];          // CTA 0: keys gathered from the cluster
  };
  u64 mass[kBins];  // sums over the cluster (a CTA holds those of its bins before they are shared)
  uint32_t cnt[kBins];
  u64 part_key[kMaxCluster];  // from each CTA
  u64 part_lo[kMaxCluster];
  float part_sum[kMaxCluster];
  u64 red[kMaxWarps];
  u64 red2[kMaxWarps];
  int part_n[kMaxCluster];
  u64 part_all[kMaxCluster], part_in[kMaxCluster];  // weight of the slice, and of what was gathered
  alignas(16) float group[kGroups];
  float redg[kGroups];
  float redf[kMaxWarps];
  u64 result;  // CTA 0's answer
  float floor;
  int n_local;
  int found_bin;
  u64 found_cnt, found_mass, found_here;
  u64 all_w, in_w;
};

// A weight of up to 16 in units of 2^-kUnit, in two halves that convert as 32 bits.
constexpr int kUnit = 40;
__device__ __forceinline__ u64 units(float w) {
  const float high = floorf(w * 1048576.0f);
  return ((u64)__float2uint_rz(high) << 20) + __float2uint_rn(fmaf(w, 1048576.0f, -high) * 1048576.0f);
}

struct Row {
  float lmax, inv_t, temp;
  float min_p;
  float scale;  // bins per nat
  __device__ __forceinline__ float dist(float l) const { return l == lmax ? 0.0f : (lmax - l) * inv_t; }
  // Weight of a token at distance d, and in the units in which top-p counts: sums of them are the same in any order, and
  // a whole vocabulary's rounding is below what fp32 tells of a top-p.
  static __device__ __forceinline__ float falling(float d) {
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(d * -1.4426950408889634f));
    return w;
  }
  static __device__ __forceinline__ u64 fixed(float d) { return units(falling(d)); }
  // The place of a logit among the bins: bin b holds [b, b + 1), bin kNear all from kNear on.
  // Monotone, so in the order of the logits.
  __device__ __forceinline__ float place(float l) const { return dist(l) * scale; }
  __device__ __forceinline__ bool in_bin(float l, int b) const {
    const float x = place(l);
    return x >= (float)b && (x < (float)(b + 1) || b == kNear);
  }
  __device__ __forceinline__ int bin(float d) const {
    const float b = d * scale;
    return b < (float)kNear ? (int)__float2uint_rz(b) : kNear;  // 0 below 0: a logit that has risen under the call
  }
  __device__ __forceinline__ float near_weight(float l) const {  // to 2^-22 and 2^-24 of (max - l) / T
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"((l - lmax) * (inv_t * 1.4426950408889634f)));
    return l == lmax ? 1.0f : w;
  }
  // Weight at a bin's upper edge, and what a token of the bin lacks to it, in units of 2^-21 of it
  // (a bin is at most 1/16 nat, so below 2^17).
  __device__ __forceinline__ float edge(int b) const { return exp2f((float)b * (-1.4426950408889634f / scale)); }
  __device__ __forceinline__ uint32_t lack(float d, int b) const {
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(((float)b - d * scale) * (1.4426950408889634f / scale)));
    return (uint32_t)__float2uint_rn((1.0f - w) * 2097152.0f);
  }
  __device__ __forceinline__ float weight(float l) const { return l == lmax ? 1.0f : expf((l - lmax) * inv_t); }
};

// top_p of a whole weight: what has at least this before it does not stay.
__device__ __forceinline__ u64 share_of(float top_p, u64 whole) { return (u64)ceil((double)top_p * (double)whole); }

__device__ __forceinline__ u64 warp_max(u64 v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((u64)hi << 32) | lo;
}
__device__ __forceinline__ float max16(const float (&l)[16]) {  // NaNs are passed over
  float m[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) m[j] = max3(l[j], l[j + 4], fmaxf(l[j + 8], l[j + 12]));
  return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// A CTA's slice of a row, in 16-byte units from the one that holds its first element; a unit that lies only partly in
// the slice is read element by element, so nothing outside the row is. kStage: raw in shared memory; otherwise
// read again, from L2.
template <typename T, int kThr, bool kStage>
struct Slice {
  static constexpr int kVec = 16 / (int)sizeof(T), kUnits = 16 / kVec;
  const uint4* from;
  uint4* stage;
  int units, id0, s0, s1;
  int whole0, wholes;  // the first unit that lies in the slice whole, and their number

  __device__ __forceinline__ Slice(const T* row, uint4* shared, int begin, int end) : stage(shared), s0(begin), s1(end) {
    const int skew = (int)(((uintptr_t)(row + s0) & 15u) / sizeof(T));
    from = (const uint4*)(row + s0 - skew);
    id0 = s0 - skew;
    units = s1 > s0 ? (skew + s1 - s0 + kVec - 1) / kVec : 0;
    whole0 = skew ? 1 : 0;
    wholes = max(0, (skew + s1 - s0) / kVec - whole0);
  }
  __device__ __forceinline__ bool whole(int q) const { return (unsigned)(q - whole0) < (unsigned)wholes; }
  // A unit that is not whole: its elements in the slice, and zeros.
  __device__ __forceinline__ uint4 ragged(int q) const {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const int id = id0 + q * kVec + e;
      if (id < s0 || id >= s1) continue;
      if (sizeof(T) == 4)
        w[e & 3] = __ldcg((const uint32_t*)from + q * kVec + e);
      else
        w[(e >> 1) & 3] |= (uint32_t)__ldcg((const unsigned short*)from + q * kVec + e) << (16 * (e & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }

  // What lies outside the slice is marked with one NaN; a NaN logit counts as -inf.
  static __device__ __forceinline__ float outside() { return __uint_as_float(0x7fffffffu); }
  static __device__ __forceinline__ float cleared(float l) {
    return __float_as_uint(l) == 0x7fffffffu ? l : fmaxf(l, -INFINITY);
  }
  // The values of a whole unit from its bits.
  static __device__ __forceinline__ void decode(uint4 x, float* l) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      l[e] = sizeof(T) == 4 ? __uint_as_float(w[e & 3])
                            : __uint_as_float((e & 1) ? w[(e >> 1) & 3] & 0xffff0000u : w[(e >> 1) & 3] << 16);
    }
  }
  // What of unit q's values lies outside the slice, marked.
  __device__ __forceinline__ void mark(int q, float* l) const {
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const int id = id0 + q * kVec + e;
      if (id < s0 || id >= s1) l[e] = outside();
    }
  }
  // The values of units q0, q0 + kThr, ... (kN / kVec of them), which `get` reads where they are whole. Most batches are whole
  // throughout, and go without a test a unit.
  template <int kN, bool kShared, typename Get>
  __device__ __forceinline__ void read(int q0, Get get, float (&l)[kN]) const {
    constexpr int kU = kN / kVec, kSpan = (kU - 1) * kThr;
    uint4 x[kU];
    if (wholes > kSpan && (unsigned)(q0 - whole0) < (unsigned)(wholes - kSpan)) {
#pragma unroll
      for (int j = 0; j < kU; ++j) x[j] = get(q0 + j * kThr);
#pragma unroll
      for (int j = 0; j < kU; ++j) decode(x[j], l + j * kVec);
    } else {
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        const int q = q0 + j * kThr;
        x[j] = make_uint4(0, 0, 0, 0);
        if (kShared ? q < units : whole(q)) x[j] = get(q);
      }
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        const int q = q0 + j * kThr;
        if (!kShared && q < units && !whole(q)) x[j] = ragged(q);
        decode(x[j], l + j * kVec);
        mark(q, l + j * kVec);
      }
    }
  }
  // f(16 values, their ids) until the slice is through, where one of the 16 is `least` at the least; a
  // thread's ids rise.
  template <typename F>
  __device__ __forceinline__ void batches(float least, F f) const {
    for (int q0 = threadIdx.x; q0 < units; q0 += kThr * kUnits) {
      float l[16];
      read<16, kStage>(q0, [&](int q) { return kStage ? stage[q] : __ldcg(from + q); }, l);
      if (least > -INFINITY && !(max16(l) >= least)) continue;
#pragma unroll
      for (int j = 0; j < 16; ++j) l[j] = cleared(l[j]);
      f(l, [&](int x16) { return id0 + (q0 + x16 / kVec * kThr) * kVec + x16 % kVec; });
    }
  }
};

// What a block of kThr threads does together.
template <int kThr>
struct Block {
static constexpr int kWarps = kThr / 32, kPer = kList / kThr;

static __device__ __forceinline__ u64 block_max(u64 v, u64* red) {
  v = warp_max(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_max(red[threadIdx.x & (kWarps - 1)]);
}
static __device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[threadIdx.x & (kWarps - 1)];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Exclusive prefix sums of (a, b) over the block's threads, in thread order.
static __device__ __forceinline__ void block_scan(u64& a, u64& b, u64* red, u64* red2) {
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

// First bin where the sum up to and with it reaches `target` (the last one with a count if none does: the sums of two
// passes may differ in their last bits), of kBins bins whose count and weight `at(bin, count, weight)` gives. All threads
// get the bin, the sums before it and its count.
template <typename At>
static __device__ __forceinline__ void find(Smem& s, At at, bool by_mass, u64 target, int& bin, u64& cnt_before, u64& mass_before, u64& here) {
  constexpr int kEach = kBins / kThr;
  const int b0 = threadIdx.x * kEach;
  u64 c[kEach], m[kEach], cs = 0, ms = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    at(b0 + j, c[j], m[j]);
    cs += c[j];
    ms += m[j];
  }
  u64 cb = cs, mb = ms;
  block_scan(cb, mb, s.red, s.red2);
  while (true) {
    const u64 before = by_mass ? mb : cb, after = by_mass ? mb + ms : cb + cs;
    if (threadIdx.x == kThr - 1 && after < target) {
      s.found_bin = -1;
      s.found_cnt = cb + cs;
    }
    if ((threadIdx.x == 0 || before < target) && after >= target) {
      u64 x = cb, y = mb;
      bool done = false;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        if (!done) {
          done = (by_mass ? y + m[j] : x + c[j]) >= target;
          if (done) {
            s.found_bin = b0 + j;
            s.found_cnt = x;
            s.found_mass = y;
            s.found_here = c[j];
          }
          x += c[j];
          y += m[j];
        }
      }
    }
    __syncthreads();
    bin = s.found_bin;
    cnt_before = s.found_cnt;
    mass_before = s.found_mass;
    here = s.found_here;
    __syncthreads();
    if (bin >= 0) return;
    by_mass = false;
    target = cnt_before;
  }
}

// Sums the CTAs' histograms (their first kArrays arrays): each CTA takes kBins / size bins, `mass_of`
// gives a bin's weight from the sums, then all read all.
template <int kArrays, typename MassOf>
static __device__ __forceinline__ void share_histogram(Smem& s, uint32_t rank, uint32_t size, MassOf mass_of) {
  cluster_sync();
  const int per = kBins / (int)size;
  // A thread sums up to four CTAs' counts of a bin, all loads in flight at once.
  const int tpb = size > 4 ? (int)size / 4 : 1;  // threads per bin
  const int first = threadIdx.x % tpb;
  for (int x = threadIdx.x / tpb; x < per; x += kThr / tpb) {
    const int b = (int)rank * per + x;
    uint32_t v[kArrays][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t k = (uint32_t)(first + tpb * j);
#pragma unroll
      for (int y = 0; y < kArrays; ++y) v[y][j] = k < size ? ld_u32(dsmem(&s.hist[y][b], k)) : 0u;
    }
    u64 sum[kArrays];
#pragma unroll
    for (int y = 0; y < kArrays; ++y) {
      sum[y] = (u64)v[y][0] + v[y][1] + v[y][2] + v[y][3];
      for (int o = 1; o < tpb; o <<= 1) sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], o);
    }
    if (first == 0) {
      s.cnt[b] = (uint32_t)sum[0];
      s.mass[b] = mass_of(b, sum);
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
      m[j] = kArrays > 1 ? ld_u64(dsmem(&s.mass[b], (uint32_t)(b / per))) : 0;
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

// A token of weight w in bin b: 16 bits of it an array (a slice's sums of 2^16 tokens stay within 32 bits).
static __device__ __forceinline__ void add_weight(Smem& s, int b, u64 w) {
  atomicAdd(&s.hist[0][b], 1u);
#pragma unroll
  for (int y = 1; y < 4; ++y) {
    const uint32_t part = (uint32_t)(w >> (48 - 16 * y)) & 0xffffu;
    if (part) atomicAdd(&s.hist[y][b], part);
  }
}
static __device__ __forceinline__ u64 whole_mass(int, const u64 (&sum)[4]) { return (sum[1] << 32) + (sum[2] << 16) + sum[3]; }
// The same for a token of a list of up to 2^11: two arrays hold its weights.
static __device__ __forceinline__ void add_listed(Smem& s, int b, u64 w) {
  atomicAdd(&s.hist[0][b], 1u);
  const uint32_t high = (uint32_t)(w >> 20), low = (uint32_t)w & 0xfffffu;
  if (high) atomicAdd(&s.hist[1][b], high);
  if (low) atomicAdd(&s.hist[2][b], low);
}
static __device__ __forceinline__ u64 listed_mass(const Smem& s, int b) { return ((u64)s.hist[1][b] << 20) + s.hist[2][b]; }
template <int kArrays>
static __device__ __forceinline__ void clear_histogram(Smem& s) {
  for (int x = threadIdx.x; x < kArrays * kBins; x += kThr) (&s.hist[0][0])[x] = 0u;
}

// Gathers the keys for which `in` holds in this CTA's list, and makes their number known to the
// cluster, with the weights `all` and `inside` of the whole block. Returns how many the cluster has.
template <typename S, typename In>
static __device__ __forceinline__ int collect(Smem& s, const S& slice, uint32_t rank, uint32_t size, float least, In in, bool weigh,
                                              const Row& r) {
  if (threadIdx.x == 0) s.n_local = 0;
  __syncthreads();
  u64 all = 0, inside = 0;
  slice.batches(weigh ? -INFINITY : least, [&](const float(&l)[16], auto id_of) {
    unsigned hits = 0;
    float part = 0.0f;  // a batch's sum has the weights' own precision
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const bool hit = l[j] == l[j] && in(l[j], id_of(j));
      hits |= hit ? 1u << j : 0u;
      if (weigh && l[j] == l[j]) part += r.falling(r.dist(l[j]));
    }
    if (weigh) all += units(part);
    if (hits) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if ((hits >> j) & 1u) {
          if (weigh) inside += r.fixed(r.dist(l[j]));
          const int at = atomicAdd(&s.n_local, 1);
          if (at < kList) s.list[at] = value_id_key(l[j], (uint32_t)id_of(j));
        }
    }
  });
  if (weigh) {
    u64 a = all, b = inside;
    block_scan(a, b, s.red, s.red2);
    if (threadIdx.x == kThr - 1) {
      s.all_w = a + all;
      s.in_w = b + inside;
    }
  }
  __syncthreads();
  if (threadIdx.x < size) {
    st_u32(dsmem(&s.part_n[rank], threadIdx.x), (uint32_t)s.n_local);
    if (weigh) {
      st_u64(dsmem(&s.part_all[rank], threadIdx.x), s.all_w);
      st_u64(dsmem(&s.part_in[rank], threadIdx.x), s.in_w);
    }
  }
  cluster_sync();
  int sum = 0;
  for (uint32_t k = 0; k < size; ++k) sum += s.part_n[k];
  return sum;
}
// The CTAs' lists (kList keys at most in all, unless logits change under the call: the rest is left out then) to CTA 0's,
// CTA after CTA.
static __device__ __forceinline__ void join(Smem& s, uint32_t rank) {
  int base = 0;
  for (uint32_t k = 0; k < rank; ++k) base += s.part_n[k];
  if (rank > 0)
    for (int x = threadIdx.x; x < min(s.n_local, kList - base); x += kThr) st_u64(dsmem(&s.list[base + x], 0), s.list[x]);
  cluster_sync();
}

// CTA 0's list of n keys, each thread's in registers.
struct List {
  u64 key[kPer];
};

// The key of the last that stays of the list, and the weight of what stays: the largest key with
// `target` keys at or above it, or (by_mass) with that weight; the smallest if the whole list has less.
// The list's shared memory is taken for the histograms.
static __device__ __forceinline__ u64 cut_list(Smem& s, const Row& r, const List& v, bool by_mass, u64 target, u64* mass_out) {
  u64 lo = 0, hi = ~0ull, mass = 0;
  while (true) {
    u64 top = 0, bottom = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (v.key[j] && v.key[j] >= lo && v.key[j] <= hi) {
        top = v.key[j] > top ? v.key[j] : top;
        bottom = ~v.key[j] > bottom ? ~v.key[j] : bottom;
      }
    }
    hi = block_max(top, s.red);
    lo = ~block_max(bottom, s.red2);
    if (top == 0 && hi == 0) {  // an empty list
      *mass_out = 0;
      return 0;
    }
    const int shift = max(0, 64 - __clzll((long long)(hi - lo)) - 10);
    clear_histogram<3>(s);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (v.key[j] && v.key[j] >= lo && v.key[j] <= hi)
        add_listed(s, (int)((hi - v.key[j]) >> shift), r.fixed(r.dist(key_value(v.key[j]))));
    __syncthreads();
    int bin;
    u64 c, m, here;
    find(s, [&](int b, u64& cc, u64& mm) {
      cc = s.hist[0][b];
      mm = listed_mass(s, b);
    }, by_mass, target, bin, c, m, here);
    const u64 in_bin = listed_mass(s, bin);
    target -= by_mass ? m : c;
    mass += m;
    hi -= (u64)bin << shift;
    lo = hi - (((u64)1 << shift) - 1) > hi ? 0 : hi - (((u64)1 << shift) - 1);
    if (here == 1 || shift == 0) {
      u64 k = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (v.key[j] && v.key[j] >= lo && v.key[j] <= hi) k = v.key[j];
      *mass_out = mass + in_bin;
      return block_max(k, s.red);
    }
    __syncthreads();  // before the histogram is cleared
  }
}

static __device__ __forceinline__ void load_list(const Smem& s, int n, List& v) {
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int x = threadIdx.x + j * kThr;
    v.key[j] = x < n ? s.list[x] : 0;
  }
}

// CTA 0: the draw from a list that holds all that can stay. `aim` is the weight for top-p when no top-k
// fixes it.
static __device__ __forceinline__ void draw_from_list(Smem& s, const SampleArgs& a, const Row& r, int row, int m, int top_k, float top_p,
                                               u64 aim) {
  const float* g = a.gumbel + (int64_t)row * a.gs;
  u64 key = 0;
  float sum = 0.0f;
  if (m <= 256) {
    // A key per thread, each ranked against all; then every bound is a matter of places and sums.
    u64 own = (int)threadIdx.x < m ? s.list[threadIdx.x] : 0;
    int rank = 0;
    if ((threadIdx.x & ~31u) < (unsigned)m) {
      int x = 0;
      for (; x + 8 <= m; x += 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) rank += s.list[x + j] > own;
      }
      for (; x < m; ++x) rank += s.list[x] > own;
    }
    __syncthreads();
    if ((int)threadIdx.x < m) s.list[rank] = own;
    __syncthreads();
    own = (int)threadIdx.x < m ? s.list[threadIdx.x] : 0;
    if (top_k > 0 && (int)threadIdx.x >= top_k) own = 0;
    const float l = key_value(own);
    const u64 w = own ? r.fixed(r.dist(l)) : 0;
    u64 before = w, z = 0;
    block_scan(before, z, s.red, s.red2);
    if (top_k > 0 && top_p < 1.0f) {
      if (threadIdx.x == kThr - 1) s.found_mass = before + w;
      __syncthreads();
      aim = share_of(top_p, s.found_mass);
    }
    if (own && (top_p >= 1.0f || before < aim)) {
      const float wt = r.weight(l);
      if (wt >= r.min_p) {
        const uint32_t id = key_id(own);
        key = value_id_key(l / r.temp + g[id], id);
        sum = wt;
      }
    }
    const u64 mine = key;
    sum = block_sum(sum, s.redf);
    key = block_max(key, s.red);
    if (mine && mine == key) {
      a.tokens[row] = (int)key_id(key);
      if (a.logprob) a.logprob[row] = (l == r.lmax ? 0.0f : (l - r.lmax) * r.inv_t) - logf(sum);
    }
    return;
  }
  List v;
  load_list(s, m, v);
  u64 mass, bound = 0;
  if (top_k > 0) {
    bound = cut_list(s, r, v, false, (u64)top_k, &mass);
    aim = share_of(top_p, mass);
  }
  if (top_p < 1.0f) {
    if (top_k > 0) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (v.key[j] < bound) v.key[j] = 0;
    }
    const u64 k = cut_list(s, r, v, true, aim, &mass);
    bound = k > bound ? k : bound;
  }
  // The list's order is that of the atomics that filled it, so its weights are summed as integers.
  u64 whole = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (v.key[j] && v.key[j] >= bound) {
      const float l = key_value(v.key[j]), w = r.weight(l);
      if (w >= r.min_p) {
        const uint32_t id = key_id(v.key[j]);
        const u64 c = value_id_key(l / r.temp + g[id], id);
        key = c > key ? c : key;
        whole += units(w);
      }
    }
  }
  u64 before = whole, z = 0;
  block_scan(before, z, s.red, s.red2);
  if (threadIdx.x == kThr - 1) s.found_mass = before + whole;
  key = block_max(key, s.red);  // a barrier before found_mass is read
  sum = (float)((double)s.found_mass * (1.0 / (double)(1ull << kUnit)));
  // From the thread that has the drawn token's logit.
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (v.key[j] && key_id(v.key[j]) == key_id(key)) {
      const float l = key_value(v.key[j]);
      a.tokens[row] = (int)key_id(key);
      if (a.logprob) a.logprob[row] = (l == r.lmax ? 0.0f : (l - r.lmax) * r.inv_t) - logf(sum);
    }
  }
}
};

// A row without a filter: one pass with a running maximum, the noise read beside the logits. False (and nothing written)
// for a row with +inf logits. A function of its own, as its registers would be spilled in the other passes' loops.
template <typename T, int kThr, bool kStage>
__device__ __noinline__ bool draw_unfiltered(Smem& s, const SampleArgs& a, int s0, int s1, int row, float temp) {
  using B = Block<kThr>;
  constexpr int kVec = 16 / (int)sizeof(T);
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const int t = threadIdx.x;
  const float* g = a.gumbel + (int64_t)row * a.gs;
  const Slice<T, kThr, kStage> slice((const T*)a.logits + (int64_t)row * a.ls, nullptr, s0, s1);
  Row r;
  r.temp = temp;
  r.inv_t = 1.0f / r.temp;
  const float c = r.inv_t * 1.4426950408889634f;
  const bool noise4 = ((uintptr_t)(g + slice.id0) & 15u) == 0;
  float m = -3.402823466e+38f, most = -INFINITY, sum = 0.0f, top_score = -INFINITY;
  int drawn = -1;
  constexpr int kN = kStage ? 16 : 8, kU = kN / kVec;  // in flight, of each
  for (int q0 = t; q0 < slice.units; q0 += kThr * kU) {
    float l[kN], z[kN], now = -INFINITY;
    slice.template read<kN, false>(q0, [&](int q) { return __ldcs(slice.from + q); }, l);
#pragma unroll
    for (int e = 0; e < kN; e += 4) {
      const int id = slice.id0 + (q0 + e / kVec * kThr) * kVec + e % kVec;
      const bool four = noise4 && id >= s0 && id + 4 <= s1;
      const float4 n = four ? __ldcs((const float4*)(g + id)) : make_float4(0, 0, 0, 0);
      z[e] = n.x; z[e + 1] = n.y; z[e + 2] = n.z; z[e + 3] = n.w;
      if (!four) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (id + k >= s0 && id + k < s1) z[e + k] = __ldcs(g + id + k);
      }
    }
#pragma unroll
    for (int j = 0; j < kN; ++j) now = fmaxf(now, l[j]);  // NaNs are passed over
    most = fmaxf(most, now);
    if (now > m) {
      sum *= ex2((m - now) * c);
      m = now;
    }
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      if (!(l[j] > -INFINITY)) continue;
      sum += ex2((l[j] - m) * c);
      const float near = l[j] * r.inv_t;
      if (near + z[j] + 1e-6f * (fabsf(near) + fabsf(z[j])) < top_score) continue;  // as in the draw below
      const float score = l[j] / r.temp + z[j];
      if (score > top_score || drawn < 0) {
        top_score = score;
        drawn = slice.id0 + (q0 + j / kVec * kThr) * kVec + j % kVec;
      }
    }
  }
  const u64 key = B::block_max(drawn < 0 ? 0 : value_id_key(top_score, (uint32_t)drawn), s.red);
  const float part = key_value(B::block_max(value_id_key(most, 0u), s.red));
  sum = B::block_sum(most == -INFINITY ? 0.0f : sum * ex2((m - part) * c), s.redf);
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (t < (int)size) st_u64(dsmem(&s.part_key[rank], (uint32_t)t), value_id_key(part, 0u));
  if (t == 0) {
    st_u64(dsmem(&s.part_lo[rank], 0), key);
    st_u32(dsmem(&s.part_sum[rank], 0), __float_as_uint(sum));
  }
  cluster_sync();
  r.lmax = -INFINITY;
  for (uint32_t k = 0; k < size; ++k) r.lmax = fmaxf(r.lmax, key_value(s.part_key[k]));
  if (r.lmax < INFINITY) {
    if (rank == 0 && t == 0) {
      u64 best = 0;
      sum = 0.0f;
      for (uint32_t k = 0; k < size; ++k) {
        if (s.part_sum[k] > 0.0f) sum += s.part_sum[k] * ex2((key_value(s.part_key[k]) - r.lmax) * c);
        best = s.part_lo[k] > best ? s.part_lo[k] : best;
      }
      const int id = best ? (int)key_id(best) : -1;  // -1: no logit above -inf
      a.tokens[row] = id;
      if (a.logprob) {
        const float l = id < 0 ? 0.0f : to_f<T>(((const T*)a.logits)[(int64_t)row * a.ls + id]);
        a.logprob[row] = id < 0 ? -INFINITY : (l == r.lmax ? 0.0f : (l - r.lmax) * r.inv_t) - logf(sum);
      }
    }
    return true;
  }
  cluster_sync();  // every CTA has read these
  return false;
}

template <typename T, int kThr, bool kStage>
__global__ void __launch_bounds__(kThr, kStage ? 2 : kManyCtas) sample_kernel(const __grid_constant__ SampleArgs a, int length) {
  using B = Block<kThr>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& s = *(Smem*)smem_raw;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  // All CTAs of the cluster are there before one writes to another (waited for below).
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int row = blockIdx.x / (int)size, t = threadIdx.x, V = a.V;
  const int s0 = min(V, (int)rank * length), s1 = min(V, s0 + length);
  const float* g = a.gumbel ? a.gumbel + (int64_t)row * a.gs : nullptr;

  constexpr int kVec = 16 / (int)sizeof(T);
  const Slice<T, kThr, kStage> slice((const T*)a.logits + (int64_t)row * a.ls, (uint4*)(smem_raw + ((sizeof(Smem) + 15) & ~(size_t)15)),
                                     s0, s1);
  bool there = false;  // all CTAs of the cluster have been seen
  {
    const float temp = a.temperature ? a.temperature[row] : 1.0f;
    const int k = a.top_k ? a.top_k[row] : 0;
    if (temp > 0.0f && temp < INFINITY && (k == 0 || k >= V) && g && !(a.top_p && a.top_p[row] != 1.0f) &&
        !(a.min_p && a.min_p[row] != 0.0f)) {
      if (draw_unfiltered<T, kThr, kStage>(s, a, s0, s1, row, temp)) return;
      there = true;
    }
  }
  float top = -INFINITY;
  int top_id = 0;  // the lowest id of this thread's largest logit: its ids rise
  if (kStage) {
    constexpr int kLoads = 8;  // in flight
    const int end = slice.whole0 + slice.wholes;
    for (int q0 = slice.whole0 + t; q0 < end; q0 += kThr * kLoads) {
      uint4 x[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        if (q0 + j * kThr < end) x[j] = __ldcs(slice.from + q0 + j * kThr);
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int q = q0 + j * kThr;
        if (q >= end) break;
        slice.stage[q] = x[j];
        float l[kVec], m = -INFINITY;
        slice.decode(x[j], l);
#pragma unroll
        for (int e = 0; e < kVec; ++e) m = fmaxf(m, l[e]);
        if (m > top) {
          top = m;
#pragma unroll
          for (int e = kVec - 1; e >= 0; --e)
            if (l[e] == m) top_id = slice.id0 + q * kVec + e;
        }
      }
    }
    // The units that are not whole: the first, of the lowest ids, and the last.
    if (t < 2 && t < slice.units) {
      const int q = t == 0 ? 0 : slice.units - 1;
      if (!slice.whole(q)) {
        const uint4 x = slice.ragged(q);
        slice.stage[q] = x;
        float l[kVec], m = -INFINITY;
        slice.decode(x, l);
        slice.mark(q, l);
#pragma unroll
        for (int e = 0; e < kVec; ++e) m = fmaxf(m, l[e]);
        if (t == 0 ? m >= top : m > top) {
          top = m;
#pragma unroll
          for (int e = kVec - 1; e >= 0; --e)
            if (l[e] == m) top_id = slice.id0 + q * kVec + e;
        }
      }
    }
  } else {
    // Before the first batch `top` is -inf, and a batch of nothing but -inf changes nothing.
    slice.batches(-INFINITY, [&](const float(&l)[16], auto id_of) {
      const float m = max16(l);
      if (m > top) {
        top = m;
#pragma unroll
        for (int j = 15; j >= 0; --j)
          if (l[j] == m) top_id = id_of(j);
      }
    });
  }
  Row r;
  r.temp = a.temperature ? a.temperature[row] : 1.0f;
  int top_k = a.top_k ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.0f;
  r.min_p = a.min_p ? a.min_p[row] : 0.0f;
  if (!there) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
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
  {
    // The groups: the same number of neighbouring threads' tokens each, kGroups / size in a CTA.
    const int lanes = kThr * (int)size / kGroups, per = kGroups / (int)size;
    float m = top;
    for (int o = 1; o < lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (t % lanes == 0) s.redg[t / lanes] = m;
    __syncthreads();
    if (t < kGroups)
      st_u32(dsmem(&s.group[(int)rank * per + t % per], (uint32_t)(t / per)), __float_as_uint(s.redg[t % per]));
  }
  u64 best = B::block_max(value_id_key(top, (uint32_t)top_id), s.red);
  if (t < (int)size) st_u64(dsmem(&s.part_key[rank], (uint32_t)t), best);
  B::template clear_histogram<2>(s);
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
  // 32 nats, and 64 where many tokens may stay, so that a bound inside a peaked row's bulk still
  // falls into a bin of few; a flat row of 150,000 tokens has about 1,500 in its fullest bin.
  r.scale = top_k > 128 ? 16.0f : 32.0f;

  u64 bound = 0;  // keys from here on stay
  if (top_k > 0 ? top_k <= kGroups / 2 : top_p < 1.0f) {
    // The candidates: tokens not below the k-th largest group maximum.
    const int k = top_k > 0 ? top_k : kGroups / 2;
    if (t < 32) {
      // The largest order key that k maxima reach, bit by bit; a warp, eight maxima a lane.
      uint32_t own[kGroups / 32], key = 0;
#pragma unroll
      for (int j = 0; j < kGroups / 32; ++j) own[j] = float_order_key(s.group[t + 32 * j]);
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t c = key | (1u << bit);
        uint32_t reach = 0;
#pragma unroll
        for (int j = 0; j < kGroups / 32; ++j) reach += own[j] >= c;
        if (__reduce_add_sync(0xffffffffu, reach) >= (uint32_t)k) key = c;
      }
      if (t == 0) s.floor = order_key_float(key);
    }
    __syncthreads();
    const float floor_l = s.floor;
    // top-p alone: a flat row's tokens below the candidates would hold most of its weight.
    const bool likely = top_k > 0 || r.near_weight(floor_l) * (float)V < 20.0f;
    if (likely) {
    const int m = B::collect(s, slice, rank, size, floor_l, [&](float l, int) { return l >= floor_l; }, top_k == 0, r);
    u64 aim = 0, inside = 0;
    if (top_k == 0) {
      u64 all = 0;
      for (uint32_t q = 0; q < size; ++q) {
        all += s.part_all[q];
        inside += s.part_in[q];
      }
      aim = share_of(top_p, all);
    }
    if (m <= kList && inside >= aim) {
      B::join(s, rank);
      if (rank == 0) B::draw_from_list(s, a, r, row, m, top_k, top_p, aim);
      return;
    }
    cluster_sync();  // the numbers are read before the next ones arrive
    B::template clear_histogram<2>(s);
    }
  }
  if (top_k > 0 || top_p < 1.0f) {
    const bool weigh = top_k == 0;  // with a top-k, its set is weighed once it is known
    uint32_t rest = 0;
    __syncthreads();
    slice.batches(-INFINITY, [&](const float(&l)[16], auto) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (l[j] != l[j]) continue;
        const float d = r.dist(l[j]);
        const int b = r.bin(d);
        if (b < kNear) {
          atomicAdd(&s.hist[0][b], 1u);
          if (weigh) atomicAdd(&s.hist[1][b], r.lack(d, b));
        } else {
          ++rest;
        }
      }
    });
    rest = __reduce_add_sync(0xffffffffu, rest);
    if (rest && (t & 31) == 0) atomicAdd(&s.hist[0][kNear], rest);
    if (weigh) {
      // Tokens past the last near bin, 32 nats down, weigh nothing: a whole vocabulary of them is less than 2^-26 of a row,
      // and no fp32 top-p below 1 is as near to it.
      B::template share_histogram<2>(s, rank, size, [&](int b, const u64 (&sum)[2]) {
        const double w = ((double)sum[0] - (double)sum[1] * (1.0 / 2097152.0)) * (double)r.edge(b);
        return b == kNear ? 0 : (u64)llrint(w * (double)(1ull << kUnit));
      });
    } else {
      B::template share_histogram<1>(s, rank, size, [](int, const u64 (&)[1]) { return (u64)0; });
    }
    auto sums = [&](int b, u64& c, u64& m) {
      c = s.cnt[b];
      m = s.mass[b];
    };
    int bin_k = kNear, bin_p = kNear;
    u64 cnt_k = 0, mass_k = 0, cnt_p = 0, mass_p = 0, here_k = 0, here_p = 0;
    if (top_k > 0) B::find(s, sums, false, (u64)top_k, bin_k, cnt_k, mass_k, here_k);
    // With no top-k the whole weight is the sum of all bins.
    u64 aim = 0;  // the weight before which a token stays; in whole units, so the least integer not below
    if (weigh) {
      u64 m = 0, z = 0;
      for (int b = t; b < kBins; b += kThr) m += s.mass[b];
      u64 before = m;
      B::block_scan(before, z, s.red, s.red2);
      if (t == kThr - 1) s.found_mass = before + m;
      __syncthreads();
      aim = share_of(top_p, s.found_mass);
      __syncthreads();
      B::find(s, sums, true, aim, bin_p, cnt_p, mass_p, here_p);
    }
    const int bin_all = min(bin_k, bin_p);
    const u64 most = top_k > 0 ? cnt_k + here_k : cnt_p + here_p;
    if (most <= (u64)kList) {
      // All that can stay, to CTA 0.
      const int m = B::collect(s, slice, rank, size, -INFINITY,
                            [&](float l, int) { return r.place(l) < (float)(bin_all + 1) || bin_all == kNear; }, false, r);
      B::join(s, rank);
      if (rank == 0) B::draw_from_list(s, a, r, row, m, top_k, top_p, aim);
      return;
    }

    // The bound of one of the two filters: the bin's keys in CTA 0's list, ordered.
    auto select = [&](int bin, u64 in_bin, u64 before, bool by_mass, u64 target, u64 floor_key) {
      u64 lo = 0, hi = ~0ull;  // keys of the bin in question
      bool whole = true;       // all keys of the bin
      while (in_bin > (u64)kList) {
        // Split the keys between the smallest and the largest by their bits.
        u64 kmax = 0, kmin = 0;
        slice.batches(-INFINITY, [&](const float(&l)[16], auto id_of) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (l[j] != l[j] || !r.in_bin(l[j], bin)) continue;
            const u64 k = value_id_key(l[j], (uint32_t)id_of(j));
            if (!whole && (k < lo || k > hi)) continue;
            kmax = k > kmax ? k : kmax;
            kmin = ~k > kmin ? ~k : kmin;
          }
        });
        kmax = B::block_max(kmax, s.red);
        kmin = B::block_max(kmin, s.red);
        __syncthreads();
        if (t < (int)size) {
          st_u64(dsmem(&s.part_key[rank], (uint32_t)t), kmax);
          st_u64(dsmem(&s.part_lo[rank], (uint32_t)t), kmin);
        }
        B::template clear_histogram<4>(s);
        cluster_sync();
        hi = 0;
        lo = 0;
        for (uint32_t k = 0; k < size; ++k) {
          hi = s.part_key[k] > hi ? s.part_key[k] : hi;
          lo = s.part_lo[k] > lo ? s.part_lo[k] : lo;
        }
        lo = ~lo;
        const int shift = max(0, 64 - __clzll((long long)(hi - lo)) - 10);
        slice.batches(-INFINITY, [&](const float(&l)[16], auto id_of) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (l[j] != l[j] || !r.in_bin(l[j], bin)) continue;
            const u64 k = value_id_key(l[j], (uint32_t)id_of(j));
            if (k >= lo && k <= hi) B::add_weight(s, (int)((hi - k) >> shift), r.fixed(r.dist(l[j])));
          }
        });
        B::template share_histogram<4>(s, rank, size, B::whole_mass);
        int sub;
        u64 c, m;
        B::find(s, sums, by_mass, target - before, sub, c, m, in_bin);
        before += by_mass ? m : c;
        const u64 top = hi - ((u64)sub << shift);
        const u64 width = ((u64)1 << shift) - 1;
        hi = top;
        lo = top > width ? top - width : 0;
        whole = false;
      }
      const int m = B::collect(s, slice, rank, size, -INFINITY, [&](float l, int id) {
        if (!r.in_bin(l, bin)) return false;
        const u64 k = value_id_key(l, (uint32_t)id);
        return k >= floor_key && (whole || (k >= lo && k <= hi));
      }, false, r);
      B::join(s, rank);
      if (rank == 0) {
        typename B::List v;
        B::load_list(s, m, v);
        u64 mass;
        const u64 k = B::cut_list(s, r, v, by_mass, target - before, &mass);
        if (t == 0) s.result = k;
      }
      cluster_sync();
      const u64 k = ld_u64(dsmem(&s.result, 0));
      cluster_sync();
      return k;
    };
    if (top_k > 0) {
      bound = select(bin_k, here_k, cnt_k, false, (u64)top_k, 0);
      if (top_p < 1.0f) {
        // Weigh the top-k set.
        B::template clear_histogram<4>(s);
        cluster_sync();
        slice.batches(-INFINITY, [&](const float(&l)[16], auto id_of) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (l[j] != l[j] || value_id_key(l[j], (uint32_t)id_of(j)) < bound) continue;
            const float d = r.dist(l[j]);
            B::add_weight(s, r.bin(d), r.fixed(d));
          }
        });
        B::template share_histogram<4>(s, rank, size, B::whole_mass);
        u64 m = 0, z = 0;
        for (int b = t; b < kBins; b += kThr) m += s.mass[b];
        u64 before = m;
        B::block_scan(before, z, s.red, s.red2);
        if (t == kThr - 1) s.found_mass = before + m;
        __syncthreads();
        aim = share_of(top_p, s.found_mass);
        __syncthreads();
        B::find(s, sums, true, aim, bin_p, cnt_p, mass_p, here_p);
      }
    }
    if (top_p < 1.0f) {
      const u64 k = select(bin_p, here_p, mass_p, true, aim, bound);
      bound = k > bound ? k : bound;
    }
  }

  // The draw over what stayed of the slice.
  const float b_val = bound ? key_value(bound) : -INFINITY;
  const int b_id = bound ? (int)key_id(bound) : V;
  float sum = 0.0f, top_score = -INFINITY;
  int drawn = -1;
  // Nothing below this passes min_p either (with room for the rounding; the test itself follows), so its
  // noise is not read.
  const float least = r.min_p > 0.0f ? fmaxf(b_val, r.lmax + r.temp * (logf(r.min_p) - 1e-3f) - 1e-5f * fabsf(r.lmax)) : b_val;
  slice.batches(least, [&](const float(&l)[16], auto id_of) {
    float z[16];
    unsigned in = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const bool stays = l[j] >= least && (l[j] > b_val || id_of(j) <= b_id);
      in |= stays ? 1u << j : 0u;
      z[j] = stays ? __ldcs(g + id_of(j)) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (!((in >> j) & 1u)) continue;
      const float w = r.near_weight(l[j]);
      if (w < r.min_p) continue;
      sum += w;
      // The exact score only where one within rounding of it does not lose.
      const float near = l[j] * r.inv_t;
      if (near + z[j] + 1e-6f * (fabsf(near) + fabsf(z[j])) < top_score) continue;
      const float score = l[j] / r.temp + z[j];
      if (score > top_score || drawn < 0) {  // ties stay with the lowest id
        top_score = score;
        drawn = id_of(j);
      }
    }
  });
  u64 key = drawn < 0 ? 0 : value_id_key(top_score, (uint32_t)drawn);
  sum = B::block_sum(sum, s.redf);
  key = B::block_max(key, s.red);
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
    const int id = key ? (int)key_id(key) : -1;  // -1: logits that changed between the passes
    a.tokens[row] = id;
    if (a.logprob && id < 0) a.logprob[row] = NAN;
    if (a.logprob && id >= 0) {
      const float l = fmaxf(to_f<T>(((const T*)a.logits)[(int64_t)row * a.ls + id]), -INFINITY);
      a.logprob[row] = (l == r.lmax ? 0.0f : (l - r.lmax) * r.inv_t) - logf(sum);
    }
  }
}

template <typename T, int kThr, bool kStage>
cudaError_t launch(const SampleArgs& a, int size, cudaStream_t stream) {
  const int length = ((a.V + size - 1) / size + 31) / 32 * 32;
  const size_t smem = ((sizeof(Smem) + 15) & ~(size_t)15) + (kStage ? (size_t)(length + 16) * sizeof(T) : 0);
  if (length > kMaxSlice || smem > 227 * 1024 || (int64_t)a.rows * size > 0x7fffffff) return cudaErrorInvalidConfiguration;
  static FuncOnce once;
  cudaError_t e = once.set((const void*)sample_kernel<T, kThr, kStage>, 227 * 1024, true);
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
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, kThr, kStage>, a, length);
}

template <typename T>
cudaError_t launch(const SampleArgs& a, cudaStream_t stream) {
  // Slices of up to 20,480 tokens; when the rows do not fill the SMs, of half that, so that more of
  // them read a row.
  int size = 1;
  while (size < kMaxCluster && (a.V + size - 1) / size > 20480) size <<= 1;
  const int64_t ctas = (int64_t)a.rows * size;
  if (size < kMaxCluster && a.V > 4096 * size && ctas * 2 <= num_sms()) size <<= 1;
  // All figures: rows of 151,936, mixed settings if nothing else is said, the same inputs again and again.
  // Few rows: the slices stay in shared memory, two CTAs on an SM. Many: a row's time is mostly barriers,
  // and what hides them is more rows in flight than shared memory holds, so the slices are read again
  // from L2 (1024 rows 540 us from shared memory and 292 from L2, 272 rows 160 and 138, 64 rows 51 and 43, 37 rows 32
  // and 39, 16 rows 28 and 40; one flat row at top-p 32 and 46).
  // Five CTAs on an SM, whose 48 registers do not hold the filters' passes (750 bytes are spilled): 1024 rows 292 us, 272
  // 138, flat ones 317, 1024 at min-p 210, without a filter 218, greedy 113. Four: 291, 124, 293, 176, 254 and 119; three:
  // 322, 119 and 328; six: 355, 169 and 415.
  // Where half as many CTAs still fill the SMs, the slices are twice as long: fewer barriers and searches for the same
  // tokens (1024 rows 334 us and 292 so, 272 flat rows at top-p 353 and 317, though 272 mixed ones 115 and 138). 64 rows,
  // which do not fill them: 43 us and 57, flat at top-p 94 and 112.
  if (ctas > 2 * (int64_t)num_sms()) {
    const bool longer = size > 1 && ctas / 2 > kManyCtas * num_sms() && (a.V + size / 2 - 1) / (size / 2) <= kMaxSlice - 32;
    return launch<T, 256, false>(a, longer ? size / 2 : size, stream);
  }
  return launch<T, 512, true>(a, size, stream);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream) {
  return a.dtype == DOMINO_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

}  // namespace domino
