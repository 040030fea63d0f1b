// Norm and rotation of a block's queries and keys, and the keys' and values'
// place in the cache, in one pass (domino_qk_norm_rope; the definition is in
// domino.h).
//
// Memory bound: every element is read once and written once. One CTA takes a
// row of the block. A group of lanes holds one head, eight elements a lane (16
// bytes of bf16), and the CTA's groups take the row's q, k and v heads in turn.
// Mean square by shuffles within the group; the rotation's partner elements
// come from the group's own fp32 copy in shared memory. All arithmetic is fp32,
// rounded once on the store.
#include "common.cuh"
#include "rows.cuh"

namespace domino {

namespace {

constexpr int kNrThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
  const float4 a = ((const float4*)p)[0], b = ((const float4*)p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 u = *(const uint4*)p;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  ((float4*)p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  ((float4*)p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *(const uint32_t*)&h;
  }
  *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NormRopeArgs a, int width) {
  extern __shared__ float s_y[];  // [groups][D]
  const int t = blockIdx.x;
  int b, i, ctx;
  if (!find_row(a.rows, t, b, i, ctx, a.ctl)) return;
  const int pos = a.rows.positions ? a.rows.positions[t] : ctx + i;
  if (a.rot > 0 && (pos < 0 || pos >= a.max_pos)) {
    if (threadIdx.x == 0) dev_error(a.ctl, DEV_ERR_DATA);
    return;
  }
  const float* cs = a.rope + (int64_t)pos * a.rot;
  const int group = threadIdx.x / width, lane = threadIdx.x % width, groups = kNrThreads / width;
  const int e0 = lane * 8;
  const bool live = e0 < a.D;
  const int half = a.rot / 2, heads = a.hq + 2 * a.hkv;
  const int64_t slot = (int64_t)b * a.rs + (int64_t)(ctx + i) * a.ss;
  float* y = s_y + group * a.D;
  for (int h0 = 0; h0 < heads; h0 += groups) {  // block-uniform bounds: every lane meets every shuffle
    const int h = h0 + group;
    const bool on = live && h < heads;
    const bool is_v = h >= a.hq + a.hkv, is_q = h < a.hq;
    float x[8] = {};
    const T* src = is_q ? (const T*)a.q + (int64_t)t * a.q_stride + (int64_t)h * a.D
                        : is_v ? (const T*)a.v + (int64_t)t * a.v_stride + (int64_t)(h - a.hq - a.hkv) * a.D
                               : (const T*)a.k + (int64_t)t * a.k_stride + (int64_t)(h - a.hq) * a.D;
    if (on) load8<T>(src + e0, x);
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
    for (int o = width / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (on && !is_v) {
      const float rstd = rsqrtf(ss / (float)a.D + a.eps);
      const T* w = (const T*)(is_q ? a.q_weight : a.k_weight);
      float wt[8] = {1, 1, 1, 1, 1, 1, 1, 1};
      if (w) load8<T>(w + e0, wt);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[e0 + j] = x[j] * rstd * wt[j];
    }
    __syncwarp();
    if (on) {
      if (!is_v) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = e0 + j;
          if (e >= a.rot) {
            x[j] = y[e];
          } else if (a.interleaved) {
            const float c = cs[e >> 1], s = cs[half + (e >> 1)];
            x[j] = (e & 1) ? y[e] * c + y[e - 1] * s : y[e] * c - y[e + 1] * s;
          } else {
            const int p = e < half ? e : e - half;
            const float c = cs[p], s = cs[half + p];
            x[j] = e < half ? y[e] * c - y[e + half] * s : y[e] * c + y[e - half] * s;
          }
        }
      }
      T* dst = is_q ? (T*)a.q_out + ((int64_t)t * a.hq + h) * a.D
                    : is_v ? (T*)a.v_cache + slot + (int64_t)(h - a.hq - a.hkv) * a.hs
                           : (T*)a.k_cache + slot + (int64_t)(h - a.hq) * a.hs;
      store8(dst + e0, x);
    }
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  int width = 1;
  while (width * 8 < a.D) width <<= 1;
  const size_t smem = (size_t)(kNrThreads / width) * a.D * 4;
  if (a.dtype == DOMINO_BF16)
    norm_rope_kernel<__nv_bfloat16><<<a.rows.tokens, kNrThreads, smem, stream>>>(a, width);
  else
    norm_rope_kernel<float><<<a.rows.tokens, kNrThreads, smem, stream>>>(a, width);
  return cudaGetLastError();
}

}  // namespace domino
