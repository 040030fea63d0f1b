// The packed rows of a block (domino_block in domino.h) on the device: which
// request a row belongs to, and a request's checked lengths.
#pragma once

#include "common.cuh"

namespace domino {

// Request b's first row, rows and past. False (with DEV_ERR_DATA recorded by
// the calling threads for which `report` is set) when a length is outside its
// bound: nothing of the request may then be touched.
__device__ __forceinline__ bool request_rows(const RowsArgs& r, int b, int& q0, int& n, int& ctx, bool report, Ctl* ctl) {
  int64_t first, rows;
  if (r.q_start) {
    first = r.q_start[b];
    rows = (int64_t)r.q_start[b + 1] - first;
  } else {
    first = (int64_t)b * r.max_q;
    rows = r.max_q;
  }
  const int64_t c = r.ctx_len[b];
  q0 = (int)first;
  n = (int)rows;
  ctx = (int)c;
  if (first < 0 || rows < 0 || rows > r.max_q || first + rows > r.tokens || c < 0 || c > r.max_ctx ||
      c + rows > r.capacity) {
    if (report) dev_error(ctl, DEV_ERR_DATA);
    return false;
  }
  return true;
}

// Looks at the lengths of all requests, also of those that no row leads to (without rows, or with fewer than none), once over
// the blocks of a grid's first axis.
__device__ __forceinline__ void report_requests(const RowsArgs& r, Ctl* ctl) {
  int q0, n, ctx;
  for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < r.batch; b += gridDim.x * blockDim.x) request_rows(r, b, q0, n, ctx, true, ctl);
}

// The request b and place i of packed row t, and the request's past and rows. Called by
// whole warps; every lane gets the result. A 32-way search: each round, the
// lanes look at 32 requests spread over what is left; in the last round a lane
// has its request's lengths at hand.
__device__ __forceinline__ bool find_row(const RowsArgs& r, int t, int& b, int& i, int& ctx, int& rows, Ctl* ctl) {
  const int lane = threadIdx.x & 31;
  if (!r.q_start) {
    b = t / r.max_q;
    int q0;
    if (!request_rows(r, b, q0, rows, ctx, lane == 0, ctl)) return false;
    i = t - q0;
    return i >= 0 && i < rows;
  }
  int lo = 0, n = r.batch;  // the last b in [lo, lo + n) with q_start[b] <= t
  while (n > 32) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, at < n && r.q_start[lo + at] <= t);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  int q0 = 0, c = 0;
  rows = 0;
  bool fine = true;
  if (lane < n) fine = request_rows(r, lo + lane, q0, rows, c, false, ctl);
  const unsigned m = __ballot_sync(0xffffffffu, lane < n && q0 <= t);
  const int k = m ? 31 - __clz(m) : 0;
  b = lo + k;
  i = t - __shfl_sync(0xffffffffu, q0, k);
  ctx = __shfl_sync(0xffffffffu, c, k);
  rows = __shfl_sync(0xffffffffu, rows, k);
  if (!__shfl_sync(0xffffffffu, (int)fine, k)) {
    if (lane == 0) dev_error(ctl, DEV_ERR_DATA);
    return false;
  }
  return i >= 0 && i < rows;  // or a row of no request
}

}  // namespace domino
