// The draw from a row of logits under top-k, top-p and min-p with given
// Gumbel noise (domino_sample; the definition is in domino.h).
//
// What stays of a row is a prefix of its order (logit descending, id
// ascending), so it is one threshold: the order key K of the last value in
// it and the number n of tokens with that very value that are in it (the
// lowest ids). top-k and top-p each give such a pair by bisection over the 32
// bits of the key: k counts the tokens above a key, p sums their weights
// exp((logit - max) / T) (in 64 bits: what is compared with top_p decides which
// tokens stay). min-p is a test of the weight itself. The draw is
// then one pass: argmax of logit / T + noise over what stayed.
//
// One CTA per row; the row is read again from L2 by every bisection step.
#include <math.h>

#include "common.cuh"

namespace domino {

namespace {

constexpr int kSaThreads = 1024;
constexpr int kSaWarps = kSaThreads / 32;

template <typename T>
__device__ __forceinline__ float load_logit(const T* row, int v) {
  return fmaxf(to_f<T>(row[v]), -INFINITY);  // NaN counts as -inf
}

struct RowSet {
  float lmax, inv_t;
  __device__ __forceinline__ float weight(float l) const { return l == lmax ? 1.0f : expf((l - lmax) * inv_t); }
};

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(red[threadIdx.x & 31]);
}
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ int block_sum(int v, int* red) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, red[threadIdx.x & 31]);
}
__device__ __forceinline__ unsigned long long block_max(unsigned long long v, unsigned long long* red) {
  v = warp_max_u64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_max_u64(red[threadIdx.x & 31]);
}

template <typename T>
__global__ void __launch_bounds__(kSaThreads) sample_kernel(const SampleArgs a) {
  __shared__ unsigned long long red64[kSaWarps];
  __shared__ float redf[kSaWarps];
  __shared__ double redd[kSaWarps];
  __shared__ int redi[kSaWarps];
  __shared__ int s_base[kSaThreads];
  const int r = blockIdx.x, t = threadIdx.x, V = a.V;
  const T* row = (const T*)a.logits + (int64_t)r * a.ls;
  const float* g = a.gumbel ? a.gumbel + (int64_t)r * a.gs : nullptr;
  const float temp = a.temperature ? a.temperature[r] : 1.0f;
  const int top_k = a.top_k ? a.top_k[r] : 0;
  const float top_p = a.top_p ? a.top_p[r] : 1.0f, min_p = a.min_p ? a.min_p[r] : 0.0f;
  if (!(temp >= 0.0f && temp < INFINITY) || top_k < 0 || !(top_p > 0.0f && top_p <= 1.0f) ||
      !(min_p >= 0.0f && min_p <= 1.0f) || (temp > 0.0f && !g)) {
    if (t == 0) {
      dev_error(a.ctl, DEV_ERR_DATA);
      a.tokens[r] = -1;
      if (a.logprob) a.logprob[r] = NAN;
    }
    return;
  }
  unsigned long long best = 0;
  for (int v = t; v < V; v += kSaThreads) {
    const unsigned long long k = value_id_key(load_logit(row, v), (uint32_t)v);
    best = k > best ? k : best;
  }
  best = block_max(best, red64);
  RowSet s;
  s.lmax = key_value(best);
  if (s.lmax == -INFINITY || temp == 0.0f) {
    if (t == 0) {
      a.tokens[r] = s.lmax == -INFINITY ? -1 : (int)key_id(best);
      if (a.logprob) a.logprob[r] = s.lmax == -INFINITY ? -INFINITY : 0.0f;
    }
    return;
  }
  s.inv_t = 1.0f / temp;

  // What stays: keys above `key`, and the first n_tie tokens at `key`.
  uint32_t key = 0;
  int n_tie = V;
  if (top_k > 0 && top_k < V) {
    uint32_t lo = 0;  // the largest key with at least top_k tokens at or above it
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t c = lo | (1u << bit);
      int n = 0;
      for (int v = t; v < V; v += kSaThreads) n += float_order_key(load_logit(row, v)) >= c;
      if (block_sum(n, redi) >= top_k) lo = c;
    }
    int above = 0;
    for (int v = t; v < V; v += kSaThreads) above += float_order_key(load_logit(row, v)) > lo;
    key = lo;
    n_tie = top_k - block_sum(above, redi);
  }
  if (top_p < 1.0f) {
    // n_tie tokens at `key` are in the set; each has the weight of its value.
    const float w_key = key ? s.weight(order_key_float(key)) : 0.0f;
    double m = 0.0;
    for (int v = t; v < V; v += kSaThreads) {
      const float l = load_logit(row, v);
      if (float_order_key(l) > key) m += s.weight(l);
    }
    const double aim = (double)top_p * (block_sum(m, redd) + (key ? (double)n_tie * w_key : 0.0));
    // The smallest key with less than `aim` above it: its first tokens still stay.
    uint32_t lo = 0, hi = float_order_key(s.lmax);
    for (int bit = 31; bit >= 0; --bit) {
      // lo: prefix known to have at least `aim` above it (or 0)
      const uint32_t c = lo | (1u << bit);
      if (c > hi) continue;
      m = 0.0;
      for (int v = t; v < V; v += kSaThreads) {
        const float l = load_logit(row, v);
        const uint32_t kk = float_order_key(l);
        if (kk >= c && kk > key) m += s.weight(l);
      }
      double w = block_sum(m, redd);
      if (c <= key) w += (double)n_tie * w_key;
      if (w >= aim) lo = c;  // the mass at or above c reaches the aim
    }
    // At or above lo the mass reaches the aim, above it it does not.
    m = 0.0;
    for (int v = t; v < V; v += kSaThreads) {
      const float l = load_logit(row, v);
      if (float_order_key(l) > lo && float_order_key(l) > key) m += s.weight(l);
    }
    const double above = block_sum(m, redd);
    if (lo > key) {
      key = lo;
      const float w = s.weight(order_key_float(lo));
      n_tie = w > 0.0f ? (int)fmin(ceil((aim - above) / w), (double)V) : V;
    } else if (lo == key && key) {
      n_tie = w_key > 0.0f ? min(n_tie, (int)fmin(ceil((aim - above) / w_key), (double)V)) : n_tie;
    }
    if (n_tie < 1) n_tie = 1;
  }

  // Ids of the tokens at `key`: each thread takes a contiguous chunk, so that
  // its first tie's rank is the count of the chunks before it.
  const int chunk = (V + kSaThreads - 1) / kSaThreads;
  const int v0 = min(V, t * chunk), v1 = min(V, v0 + chunk);
  int rank = 0;
  if (n_tie < V) {
    int mine = 0;
    for (int v = v0; v < v1; ++v) mine += float_order_key(load_logit(row, v)) == key;
    s_base[t] = mine;
    __syncthreads();
    for (int o = 1; o < kSaThreads; o <<= 1) {
      const int x = t >= o ? s_base[t - o] : 0;
      __syncthreads();
      s_base[t] += x;
      __syncthreads();
    }
    rank = s_base[t] - mine;
  }
  float total = 0.0f;
  best = 0;
  for (int v = v0; v < v1; ++v) {
    const float l = load_logit(row, v);
    const uint32_t kk = float_order_key(l);
    if (kk < key || (kk == key && rank++ >= n_tie)) continue;
    const float w = s.weight(l);
    if (w < min_p) continue;
    total += w;
    const unsigned long long c = value_id_key(l / temp + g[v], (uint32_t)v);
    best = c > best ? c : best;
  }
  total = block_sum(total, redf);
  best = block_max(best, red64);
  if (t == 0) {
    const int v = (int)key_id(best);
    a.tokens[r] = v;
    if (a.logprob) {
      const float l = load_logit(row, v);
      a.logprob[r] = (l == s.lmax ? 0.0f : (l - s.lmax) * s.inv_t) - logf(total);
    }
  }
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream) {
  if (a.dtype == DOMINO_BF16)
    sample_kernel<__nv_bfloat16><<<a.rows, kSaThreads, 0, stream>>>(a);
  else
    sample_kernel<float><<<a.rows, kSaThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace domino
