// Norm and rotation of a block's queries and keys, and the keys' and values'
// place in the cache, in one pass (domino_qk_norm_rope and domino_paged_append; the
// definitions are in domino.h).
//
// Memory bound: every element is read once and written once. A group of lanes holds one head,
// eight elements a lane (16 bytes of bf16). A lane has the same eight places of every head, so a
// row's cosines and sines and the weights are read once and multiplied once. The mean square and
// the rotation's partners come by shuffles within the group; only where half of rot_dim is no
// multiple of eight do the partners go through shared memory. All arithmetic is fp32, rounded once
// on the store.
//
// Few rows: a CTA takes a row, or some of its heads, with the loads of several heads in flight. One
// draft block of 16 rows: 3.6 us, nearly all of it the launch.
// Many rows: a CTA takes a run of rows; bulk copies bring the next row to shared memory while it
// works on one, so that the loads wait for nothing. Prompts of 4 requests, 19,700 rows of 32 + 8 + 8
// heads of 128 in bf16: 86 us, 5.5 TB/s (without the copies ahead 114 us: too few bytes in flight; rows of which two
// do not fit the ring's 55 KB, 55 heads of 128 in fp32 say, go without them).
// Four CTAs an SM with two rows each measured best (three rows 87, four rows 89, three CTAs 97,
// five, whose registers spill, 98 us).
//
// Pages: a row's page is one table entry. Quantised: a head's largest magnitude by shuffles gives the scale's exponent by integer
// tests on its fp32 fields, and each element is rounded once, from fp32. 18,900 rows of the same heads into quantised pages 113 us, 3.9
// TB/s, into bf16 pages 101 us, into fp32 ones 164 (5.7 TB/s). With 15 warps an SM, codes fill neither memory (43 % of its peak) nor the issue
// slots (56 %, about 1100 instructions a row and warp): of 6.6 cycles that a warp takes for an instruction, 1.7 wait for the one before, 1.6 for
// shuffles and shared memory, 0.7 for global memory and 0.4 at the row's two barriers. (Fewer table reads, or the maximum by one reduction
// instruction, changed nothing: 115 and 116 us.)
#include <algorithm>

#include "common.cuh"
#include "packed.cuh"
#include "pages.cuh"
#include "rows.cuh"
#include "waits.cuh"

namespace domino {

namespace {

constexpr int kNrThreads = 128;
constexpr int kRunCtas = 4;     // of the kernel for many rows, on an SM
constexpr int kMostStages = 2;  // rows in a CTA's ring, at most
constexpr int kRunSmem = 55 * 1024;
// Rows per CTA of the kernel for few rows from which the kernel for many is taken. 32 + 8 + 8 heads of 128, first and second
// kernel: bf16, 1500 rows (two) 8.8 and 9.2 us, 2000 (three) 11.4 and 11.3, 2700 (four) 15.0 and 13.4, 4000 (six) 25.6 and 19.7;
// fp32, 2000 rows 17.9 and 20.2 us, 2700 27.5 and 28.3, 3300 (five) 33.4 and 33.5, 4000 39.1 and 38.0.
template <typename T>
constexpr int kRunRows = sizeof(T) == 2 ? 3 : 6;

// Eight elements as they lie in memory; in arithmetic, four fp32 pairs.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = ((const float4*)p)[0];
    b = ((const float4*)p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float2 (&x)[4]) const {
    x[0] = make_float2(a.x, a.y); x[1] = make_float2(a.z, a.w);
    x[2] = make_float2(b.x, b.y); x[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ void set(const float2 (&x)[4]) {
    a = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    b = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
  }
  __device__ __forceinline__ Raw8 of(int lane) const {  // another lane's
    Raw8 o;
    const float* x = (const float*)&a;
    float* y = (float*)&o.a;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], lane);
    x = (const float*)&b;
    y = (float*)&o.b;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], lane);
    return o;
  }
  __device__ __forceinline__ void store(float* p) const {
    ((float4*)p)[0] = a;
    ((float4*)p)[1] = b;
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *(const uint4*)p; }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float2 (&x)[4]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void set(const float2 (&x)[4]) {
    u = make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y), pack_bf16(x[2].x, x[2].y), pack_bf16(x[3].x, x[3].y));
  }
  __device__ __forceinline__ Raw8 of(int lane) const {  // another lane's
    Raw8 o;
    o.u.x = __shfl_sync(0xffffffffu, u.x, lane);
    o.u.y = __shfl_sync(0xffffffffu, u.y, lane);
    o.u.z = __shfl_sync(0xffffffffu, u.z, lane);
    o.u.w = __shfl_sync(0xffffffffu, u.w, lane);
    return o;
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *(uint4*)p = u; }
};

enum { kPairs = 0, kHalves = 1, kHalvesShared = 2 };

// What a lane does with its eight places of a head.
template <typename T, int MODE, int kWidth, int CACHE>
struct Places {
  const NormRopeArgs& a;
  const int e0, half;
  const bool live, low;  // within the head; in the first half of what turns
  const int partner_lane;
  const float inv_d;
  float* x;  // kHalvesShared: the group's head
  float c[8], s[8];
  float2 wc[4], ws[4];

  __device__ __forceinline__ Places(const NormRopeArgs& args, float* shared)
      : a(args), e0((int)(threadIdx.x % kWidth) * 8), half(args.rot / 2), live(e0 < args.D), low(e0 < half),
        partner_lane((int)(threadIdx.x & 31) + (e0 >= args.rot ? 0 : low ? half : -half) / 8), inv_d(1.0f / (float)args.D),
        x(shared) {}

  // A place's partner in the rotation (itself where it does not turn).
  __device__ __forceinline__ int partner_of(int e) const {
    return e >= a.rot ? e : MODE == kPairs ? e ^ 1 : e < half ? e + half : e - half;
  }
  // The angle of each of the lane's places: eight neighbours of a half, or four pairs. `raw` is what is read of the
  // table: up to eight cosines and eight sines.
  __device__ __forceinline__ void read_angles(int pos, float (&raw)[16]) const {
    const float* cs = a.rope + (int64_t)pos * a.rot;
    if (MODE == kHalves || (MODE == kPairs && a.rot % 8 == 0)) {
      constexpr int kN = MODE == kHalves ? 8 : 4;
      const float* at = cs + (MODE == kPairs ? e0 / 2 : low ? e0 : e0 - half);
      const bool turns = e0 < a.rot;
#pragma unroll
      for (int j = 0; j < kN; j += 4) {
        const float4 x4 = turns ? __ldg((const float4*)(at + j)) : make_float4(1, 1, 1, 1);
        const float4 y4 = turns ? __ldg((const float4*)(at + half + j)) : make_float4(0, 0, 0, 0);
        raw[j] = x4.x; raw[j + 1] = x4.y; raw[j + 2] = x4.z; raw[j + 3] = x4.w;
        raw[8 + j] = y4.x; raw[9 + j] = y4.y; raw[10 + j] = y4.z; raw[11 + j] = y4.w;
      }
    } else {
      constexpr int kN = MODE == kPairs ? 4 : 8;
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const int e = MODE == kPairs ? e0 + 2 * j : e0 + j, p = MODE == kPairs ? e >> 1 : e < half ? e : e - half;
        raw[j] = e < a.rot ? __ldg(cs + p) : 1.0f;
        raw[8 + j] = e < a.rot ? __ldg(cs + half + p) : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void set_angles(const float (&raw)[16]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = raw[MODE == kPairs ? j / 2 : j];
      s[j] = raw[8 + (MODE == kPairs ? j / 2 : j)];
      if (MODE == kPairs ? (j & 1) == 0 : e0 + j < half) s[j] = -s[j];
    }
  }
  // Weights times cosines and the partners' weights times sines.
  __device__ __forceinline__ void weigh(const float* w) {
    const int e = live ? e0 : 0;
    float x[8], y[8];
#pragma unroll
    for (int j = 0; j < 8; j += 4) *(float4*)&x[j] = *(const float4*)&w[e + j];
    if (MODE == kHalves) {
      const int p = partner_of(e);
#pragma unroll
      for (int j = 0; j < 8; j += 4) *(float4*)&y[j] = *(const float4*)&w[p + j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = MODE == kPairs ? x[j ^ 1] : w[partner_of(e + j)];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      wc[j] = make_float2(x[2 * j] * c[2 * j], x[2 * j + 1] * c[2 * j + 1]);
      ws[j] = make_float2(y[2 * j] * s[2 * j], y[2 * j + 1] * s[2 * j + 1]);
    }
  }
  // z = rstd (x (w c) + x' (w' s)), x' the partner. (An infinity makes rstd 0 and a NaN makes it a
  // NaN, so that a partner's value times 0 adds nothing to what the head's own values do.)
  __device__ __forceinline__ void turn(Raw8<T>& v, bool on, T* dst) {
    float2 z[4];
    turned(v, on, z);
    v.set(z);
    if (on) v.store(dst);
  }
  __device__ __forceinline__ void turned(Raw8<T>& v, bool on, float2 (&z)[4]) {
    float2 y[4];
    if (!on) v.zero();
    v.get(z);
    float2 sq = mul2(z[0], z[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) sq = fma2(z[e], z[e], sq);
    float ss = sq.x + sq.y;
#pragma unroll
    for (int o = kWidth / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float rstd = CACHE == kWhole || a.norm ? rsqrtf(ss * inv_d + a.eps) : 1.0f;
    if (MODE == kPairs) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = make_float2(z[e].y, z[e].x);
    } else if (MODE == kHalves) {
      v.of(partner_lane).get(y);
    } else {
      __syncwarp();
      if (on) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e0 + 2 * e] = z[e].x;
          x[e0 + 2 * e + 1] = z[e].y;
        }
      }
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y[e] = on ? make_float2(x[partner_of(e0 + 2 * e)], x[partner_of(e0 + 2 * e + 1)]) : make_float2(0, 0);
    }
    if (CACHE != kWhole) {  // without the norm, an infinity that does not turn stays one
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e0 + 2 * e >= a.rot) y[e] = make_float2(0, 0);
    }
    const float2 r2 = make_float2(rstd, rstd);
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = mul2(r2, fma2(z[e], wc[e], mul2(y[e], ws[e])));
  }
  // A head's vector as codes and their scale (pages.cuh).
  __device__ __forceinline__ void store_codes(const float2 (&z)[4], bool on, uint8_t* dst, uint8_t* scale) const {
    uint32_t most = 0;
    if (on) {
#pragma unroll
      for (int e = 0; e < 4; ++e) most = max(most, max(__float_as_uint(z[e].x) & 0x7fffffffu, __float_as_uint(z[e].y) & 0x7fffffffu));
    }
#pragma unroll
    for (int o = kWidth / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (!on) return;
    const int byte = scale_byte(most);
    const float f = scale_inverse(byte);
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = byte == kScaleNan ? 0u : pack_e4m3(z[e].x * f, z[e].y * f);
    *(uint2*)dst = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    if (e0 == 0) *scale = (uint8_t)byte;
  }
  // A key head, and a value head as it is, into the cache: `slot` is the row's place there (elements, with e0), page and
  // s where that is.
  __device__ __forceinline__ void cache_kv(Raw8<T>& xk, const Raw8<T>& xv, bool on, int h, int64_t slot, int page, int s) {
    const int64_t at = slot + (int64_t)h * a.hs;
    if (CACHE == kPagedE4m3) {
      const int64_t to = scale_at(a.pages, a.hkv, page, h, s);
      float2 z[4];
      xv.get(z);
      store_codes(z, on, (uint8_t*)a.v_cache + at, a.pages.v_scale + to);
      turned(xk, on, z);
      store_codes(z, on, (uint8_t*)a.k_cache + at, a.pages.k_scale + to);
    } else {
      if (on) xv.store((T*)a.v_cache + at);
      turn(xk, on, (T*)a.k_cache + at);
    }
  }
  // The row's place in the cache: false where its page is not there.
  __device__ __forceinline__ bool place(int b, int s, int64_t& slot, int& page) const {
    if (CACHE == kWhole) {
      page = 0;
      slot = (int64_t)b * a.rs + (int64_t)s * a.ss + e0;
      return true;
    }
    page = page_of(a.pages, b, s);
    slot = (int64_t)page * a.pages.page_stride + (int64_t)slot_in_page(a.pages, s) * a.ss + e0;
    return page >= 0;
  }
};

template <typename T>
__device__ __forceinline__ void read_weights(const NormRopeArgs& a, float* s_w) {
  for (int e = threadIdx.x; e < 2 * a.D; e += kNrThreads) {
    const T* w = (const T*)(e < a.D ? a.q_weight : a.k_weight);
    s_w[e] = w ? to_f<T>(w[e < a.D ? e : e - a.D]) : 1.0f;
  }
}

// Few rows: one or two per CTA, or the heads of one over several. (Also rows too long for the other kernel's ring.)
template <typename T, int MODE, int kWidth, int CACHE>
__global__ void __launch_bounds__(kNrThreads, 5) norm_rope_kernel(const NormRopeArgs a, int chunk) {
  constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;  // q heads in flight, beside one of k and one of v
  extern __shared__ __align__(16) float s_w[];    // [2][D] weights; kHalvesShared: [groups][D] heads
  constexpr int groups = kNrThreads / kWidth;
  const int group = threadIdx.x / kWidth;
  Places<T, MODE, kWidth, CACHE> at(a, s_w + 2 * a.D + group * a.D);
  const bool live = at.live;
  const int e0 = at.e0, first = blockIdx.y * groups + group, step = groups * gridDim.y;
  // Loops over heads have the same bounds for the whole block: every lane meets every shuffle.
  const int first_u = blockIdx.y * groups;
  int t = blockIdx.x * chunk;
  const int t_end = min(a.rows.tokens, t + chunk);
  Raw8<T> xq[kBatch], xk, xv;
  auto fetch_q = [&](int h0) {
    const T* p = (const T*)a.q + (int64_t)t * a.q_stride + e0;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (live && h0 + j * step < a.hq) xq[j].load(p + (h0 + j * step) * a.D);
  };
  auto fetch_kv = [&](int h) {
    if (live && h < a.hkv) {
      xk.load((const T*)a.k + (int64_t)t * a.k_stride + h * a.D + e0);
      xv.load((const T*)a.v + (int64_t)t * a.v_stride + h * a.D + e0);
    }
  };
  fetch_q(first);  // these need no lengths
  fetch_kv(first);
  read_weights<T>(a, s_w);
  if (blockIdx.y == 0) report_requests(a.rows, a.ctl);
  int b, i, ctx, rows;
  bool mine = find_row(a.rows, t, b, i, ctx, rows, a.ctl);
  __syncthreads();
  while (true) {
    const int pos = !mine ? 0 : a.rows.positions ? a.rows.positions[t] : ctx + i;
    int64_t slot = 0;
    int page = 0;
    const bool placed = mine && (a.rot == 0 || (pos >= 0 && pos < a.max_pos)) && at.place(b, ctx + i, slot, page);
    if (mine && !placed && threadIdx.x == 0) dev_error(a.ctl, DEV_ERR_DATA);
    if (placed) {
      float raw[16];
      at.read_angles(pos, raw);
      at.set_angles(raw);
      at.weigh(s_w + a.D);
      for (int h0 = first_u; h0 < a.hkv; h0 += step) {
        const int h = h0 + group;
        if (h0 > first_u) fetch_kv(h);
        at.cache_kv(xk, xv, live && h < a.hkv, h, slot, page, ctx + i);
      }
      at.weigh(s_w);
      T* q_out = (T*)a.q_out + (int64_t)t * a.hq * a.D + e0;
      for (int h0 = first_u; h0 < a.hq; h0 += kBatch * step) {
        if (h0 > first_u) fetch_q(h0 + group);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          // All of the batch at once, so that the heads' chains overlap; one beyond the last is not stored.
          const int h = h0 + j * step + group;
          at.turn(xq[j], live && h < a.hq, q_out + h * a.D);
        }
      }
    }
    if (++t == t_end) break;
    fetch_q(first);
    fetch_kv(first);
    if (mine && i + 1 < rows)
      ++i;
    else
      mine = find_row(a.rows, t, b, i, ctx, rows, a.ctl);
  }
}

// Many rows: a CTA takes a run of rows, which bulk copies bring to a ring of `stages` rows in shared memory while
// earlier ones are worked on; a row's angles are read one row ahead.
template <typename T, int MODE, int kWidth, int CACHE>
__global__ void __launch_bounds__(kNrThreads, kRunCtas) norm_rope_run_kernel(const NormRopeArgs a, int chunk, int stages, uint64_t timeout_ns) {
  constexpr int kBatch = 4;
  extern __shared__ __align__(16) float s_w[];  // [2][D] weights; kHalvesShared: [groups][D] heads; rows
  __shared__ __align__(8) uint64_t full[kMostStages];
  constexpr int groups = kNrThreads / kWidth;
  const int group = threadIdx.x / kWidth;
  Places<T, MODE, kWidth, CACHE> at(a, s_w + 2 * a.D + group * a.D);
  const bool live = at.live;
  const int e0 = at.e0;
  T* ring = (T*)(s_w + (2 + (MODE == kHalvesShared ? groups : 0)) * a.D);
  const int nq = a.hq * a.D, nk = a.hkv * a.D, row = nq + 2 * nk;  // elements
  const int t0 = blockIdx.x * chunk, t_end = min(a.rows.tokens, t0 + chunk);
  auto bring = [&](int t, int st) {
    T* to = ring + (int64_t)st * row;
    mbar_expect_tx(&full[st], (uint32_t)(row * sizeof(T)));
    if (nq) bulk_copy_g2s(to, (const T*)a.q + (int64_t)t * a.q_stride, (uint32_t)(nq * sizeof(T)), &full[st]);
    bulk_copy_g2s(to + nq, (const T*)a.k + (int64_t)t * a.k_stride, (uint32_t)(nk * sizeof(T)), &full[st]);
    bulk_copy_g2s(to + nq + nk, (const T*)a.v + (int64_t)t * a.v_stride, (uint32_t)(nk * sizeof(T)), &full[st]);
  };
  if (threadIdx.x == 0) {
    for (int st = 0; st < stages; ++st) mbar_init(&full[st], 1);
    mbar_fence_init();
    for (int st = 0; st < stages && t0 + st < t_end; ++st) bring(t0 + st, st);
  }
  read_weights<T>(a, s_w);
  report_requests(a.rows, a.ctl);
  int b, i, ctx, rows;
  bool mine, placed;
  int64_t slot = 0;  // the row's place in pages
  int page = 0, s = 0;
  float raw[16];
  auto look = [&](int t) {  // the row's place and angles
    const int pos = !mine ? 0 : a.rows.positions ? __ldg(a.rows.positions + t) : ctx + i;
    placed = mine && (a.rot == 0 || (pos >= 0 && pos < a.max_pos));
    if (CACHE != kWhole) {
      s = ctx + i;
      if (placed) placed = at.place(b, s, slot, page);
    }
    if (mine && !placed && threadIdx.x == 0) dev_error(a.ctl, DEV_ERR_DATA);
    if (placed) at.read_angles(pos, raw);
  };
  mine = find_row(a.rows, t0, b, i, ctx, rows, a.ctl);
  look(t0);
  __syncthreads();
  int st = 0;
  uint32_t phase = 0;
  bool ok = true;
  int t = t0;
  for (; t < t_end; ++t) {
    const bool on_row = placed;
    const int64_t row_slot = CACHE == kWhole ? (int64_t)b * a.rs + (int64_t)(ctx + i) * a.ss + e0 : slot;
    const int row_page = page, row_s = s;
    if (on_row) at.set_angles(raw);
    if (t + 1 < t_end) {
      if (mine && i + 1 < rows)
        ++i;
      else
        mine = find_row(a.rows, t + 1, b, i, ctx, rows, a.ctl);
      look(t + 1);
    }
    ok = __syncthreads_and(mbar_wait(&full[st], phase, nullptr, a.ctl, timeout_ns));
    if (!ok) break;
    if (on_row) {
      const T* x = ring + (int64_t)st * row + e0;
      at.weigh(s_w + a.D);
      for (int h0 = 0; h0 < a.hkv; h0 += groups) {
        const int h = h0 + group;
        const bool on = live && h < a.hkv;
        Raw8<T> xk, xv;
        if (on) {
          xk.load(x + nq + h * a.D);
          xv.load(x + nq + nk + h * a.D);
        }
        at.cache_kv(xk, xv, on, h, row_slot, row_page, row_s);
      }
      at.weigh(s_w);
      T* q_out = (T*)a.q_out + (int64_t)t * nq + e0;
      for (int h0 = 0; h0 < a.hq; h0 += kBatch * groups) {
        Raw8<T> xq[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (live && h0 + j * groups + group < a.hq) xq[j].load(x + (h0 + j * groups + group) * a.D);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int h = h0 + j * groups + group;
          at.turn(xq[j], live && h < a.hq, q_out + h * a.D);
        }
      }
    }
    __syncthreads();
    if (threadIdx.x == 0 && t + stages < t_end) bring(t + stages, st);
    if (++st == stages) {
      st = 0;
      phase ^= 1u;
    }
  }
  // After a wait that ran out for any thread: the rows on their way land before the memory is given up.
  if (!ok && threadIdx.x == 0)
    for (int k = 0; k < stages && t + k < t_end; ++k) {
      mbar_land(&full[st], phase, a.ctl);
      if (++st == stages) {
        st = 0;
        phase ^= 1u;
      }
    }
}

template <typename T, int MODE, int CACHE>
cudaError_t launch_on(const NormRopeArgs& a, cudaStream_t stream) {
  // Lanes per head: 8 (a head of up to 64), 16 or 32.
  const int width = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32, groups = kNrThreads / width;
  const int rounds = ((a.hq > a.hkv ? a.hq : a.hkv) + groups - 1) / groups;
  // A row's heads over several CTAs while the rows do not fill the SMs; past the five CTAs that an SM holds, a CTA
  // takes neighbouring rows one after the other: their lengths are then at hand.
  const int most = 5 * num_sms();
  int chunk = (a.rows.tokens + most - 1) / most;
  const size_t smem = (size_t)(2 + (MODE == kHalvesShared ? groups : 0)) * a.D * 4;
  const size_t row = (size_t)(a.hq + 2 * a.hkv) * a.D * sizeof(T);
  const int stages = (int)std::min<size_t>(kMostStages, (kRunSmem - smem) / row);
  if (chunk >= kRunRows<T> && stages >= 2) {
    const int ctas = kRunCtas * num_sms();
    chunk = (a.rows.tokens + ctas - 1) / ctas;
    const unsigned grid = (unsigned)((a.rows.tokens + chunk - 1) / chunk);
    const size_t bytes = smem + stages * row;
    auto run = [&](auto kernel, FuncOnce& once) {
      const cudaError_t e = once.set((const void*)kernel, kRunSmem, false);
      if (e != cudaSuccess) return e;
      kernel<<<grid, kNrThreads, bytes, stream>>>(a, chunk, stages, wait_timeout_ns());
      return cudaGetLastError();
    };
    static FuncOnce once8, once16, once32;
    if (width == 8) return run(norm_rope_run_kernel<T, MODE, 8, CACHE>, once8);
    if (width == 16) return run(norm_rope_run_kernel<T, MODE, 16, CACHE>, once16);
    return run(norm_rope_run_kernel<T, MODE, 32, CACHE>, once32);
  }
  const dim3 grid((unsigned)((a.rows.tokens + chunk - 1) / chunk),
                  (int64_t)a.rows.tokens * rounds <= 2 * num_sms() ? (unsigned)rounds : 1u);
  if (width == 8)
    norm_rope_kernel<T, MODE, 8, CACHE><<<grid, kNrThreads, smem, stream>>>(a, chunk);
  else if (width == 16)
    norm_rope_kernel<T, MODE, 16, CACHE><<<grid, kNrThreads, smem, stream>>>(a, chunk);
  else
    norm_rope_kernel<T, MODE, 32, CACHE><<<grid, kNrThreads, smem, stream>>>(a, chunk);
  return cudaGetLastError();
}

template <typename T, int MODE>
cudaError_t launch(const NormRopeArgs& a, cudaStream_t stream) {
  return launch_on<T, MODE, kWhole>(a, stream);
}
template <typename T>
cudaError_t launch(const NormRopeArgs& a, cudaStream_t stream) {
  if (a.interleaved) return launch<T, kPairs>(a, stream);
  return a.rot % 16 == 0 ? launch<T, kHalves>(a, stream) : launch<T, kHalvesShared>(a, stream);
}
template <typename T, int CACHE>
cudaError_t launch_paged(const NormRopeArgs& a, cudaStream_t stream) {
  if (a.interleaved) return launch_on<T, kPairs, CACHE>(a, stream);
  return a.rot % 16 == 0 ? launch_on<T, kHalves, CACHE>(a, stream) : launch_on<T, kHalvesShared, CACHE>(a, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  return a.dtype == DOMINO_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

cudaError_t launch_paged_append(const NormRopeArgs& a, cudaStream_t stream) {
  if (a.e4m3) return launch_paged<__nv_bfloat16, kPagedE4m3>(a, stream);
  return a.dtype == DOMINO_BF16 ? launch_paged<__nv_bfloat16, kPaged>(a, stream) : launch_paged<float, kPaged>(a, stream);
}

}  // namespace domino
