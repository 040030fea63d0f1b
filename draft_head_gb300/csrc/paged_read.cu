// Slots of a cache in pages as they are, or scaled back from their codes, in one piece (domino_paged_read; the definition is in
// domino.h).
//
// Memory bound: every code or element is read once, every element written once. A thread takes 16 bytes of a slot's vector;
// a CTA takes 64 slots of one kv head, keys and values, with all its loads in flight before the first store.
#include "common.cuh"
#include "pages.cuh"

namespace domino {

namespace {

constexpr int kThr = 256, kSlots = 64;

template <bool E4M3>
__global__ void __launch_bounds__(kThr) paged_read_kernel(const PagedReadArgs a) {
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t first = a.first ? a.first[b] : 0, count = a.count[b];
  if (first < 0 || count < 0 || count > a.max_count || count > a.out_capacity || first + count > a.capacity) {
    if (threadIdx.x == 0 && h == 0 && blockIdx.x == 0) dev_error(a.ctl, DEV_ERR_DATA);
    return;
  }
  const int j0 = blockIdx.x * kSlots;
  if (j0 >= count) return;
  const int n = min(kSlots, (int)count - j0), size = E4M3 ? 1 : a.dtype == DOMINO_BF16 ? 2 : 4;
  const int pieces = a.D * size / 16;  // of a slot's vector
  constexpr int kU = 2;
  for (int x0 = threadIdx.x; x0 < n * pieces; x0 += kU * kThr) {
    uint4 k[kU], v[kU];
    int scale[kU] = {}, at[kU], page[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int x = x0 + u * kThr, j = x / pieces;
      at[u] = x - j * pieces;
      page[u] = -1;
      if (x >= n * pieces) continue;
      const int s = (int)first + j0 + j;
      page[u] = page_of(a.pages, b, s);
      if (page[u] < 0) {
        if (at[u] == 0) dev_error(a.ctl, DEV_ERR_DATA);
        continue;
      }
      const int64_t from = ((int64_t)page[u] * a.pages.page_stride + (int64_t)h * a.hs + (int64_t)slot_in_page(a.pages, s) * a.ss) * size +
                           at[u] * 16;
      k[u] = *(const uint4*)((const uint8_t*)a.k + from);
      v[u] = *(const uint4*)((const uint8_t*)a.v + from);
      if (E4M3) {
        const int64_t to = scale_at(a.pages, a.hkv, page[u], h, s);
        scale[u] = a.pages.k_scale[to] | a.pages.v_scale[to] << 8;
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (page[u] < 0) continue;
      const int j = (x0 + u * kThr) / pieces;
      const int64_t to = (int64_t)b * a.out_rs + (int64_t)h * a.out_hs + (int64_t)(j0 + j) * a.out_ss;
      if (E4M3) {
        __nv_bfloat16* ko = (__nv_bfloat16*)a.k_out + to + at[u] * 16;
        __nv_bfloat16* vo = (__nv_bfloat16*)a.v_out + to + at[u] * 16;
        const Scale2 ks = scale_bf16(scale[u] & 255), vs = scale_bf16(scale[u] >> 8);
        ((uint4*)ko)[0] = codes8_bf16(make_uint2(k[u].x, k[u].y), ks);
        ((uint4*)ko)[1] = codes8_bf16(make_uint2(k[u].z, k[u].w), ks);
        ((uint4*)vo)[0] = codes8_bf16(make_uint2(v[u].x, v[u].y), vs);
        ((uint4*)vo)[1] = codes8_bf16(make_uint2(v[u].z, v[u].w), vs);
      } else {
        *(uint4*)((uint8_t*)a.k_out + to * size + at[u] * 16) = k[u];
        *(uint4*)((uint8_t*)a.v_out + to * size + at[u] * 16) = v[u];
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_read(const PagedReadArgs& a, cudaStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)a.max_count + kSlots - 1) / kSlots), (unsigned)a.hkv, (unsigned)a.batch);
  if (a.e4m3)
    paged_read_kernel<true><<<grid, kThr, 0, stream>>>(a);
  else
    paged_read_kernel<false><<<grid, kThr, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace domino
