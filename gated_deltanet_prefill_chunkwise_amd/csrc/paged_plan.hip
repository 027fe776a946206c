// Page bookkeeping of a serving step: sgdn_paged_release and sgdn_paged_plan.
//
// Both are sums over the requests in front of a request (pages, rows) and a
// few integers written per page and per row; there is nothing to compute and
// little to move, so what counts is the number of launches and of dependent
// memory accesses.  One workgroup makes the sums (wave scans joined through
// LDS) because the counters and lengths may be updated in place: it has read
// everything before it writes.  A page that a request takes is found from the
// sums alone, so the thread that describes a page's first row also enters the
// page in the table and no row waits for the table of a new page.  Measured:
// 128 requests with a token each 4.4 us; 64 requests of which 8 end and 8
// begin with prompts, 95418 rows in all: release 5.2, sums 3.4, rows 4.5.
#include "common.h"
#include "paged.h"

namespace sgdn {

namespace {

constexpr int MAXW = 16;   // waves of the largest workgroup here

// Inclusive sums of x and y over the workgroup; tot_x, tot_y the totals.
// `part` is LDS of 2 * MAXW, free again when the call returns.
__device__ __forceinline__ void scan2(int64_t& x, int64_t& y, int64_t& tot_x, int64_t& tot_y, int64_t* part) {
  const int lane = lane_id(), wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t px = __shfl_up(x, o, 64), py = __shfl_up(y, o, 64);
    if (lane >= o) { x += px; y += py; }
  }
  if (lane == 63) { part[2 * wave] = x; part[2 * wave + 1] = y; }
  __syncthreads();
  tot_x = tot_y = 0;
  int64_t bx = 0, by = 0;
  for (int w = 0; w < nw; ++w) {
    if (w == wave) { bx = tot_x; by = tot_y; }
    tot_x += part[2 * w];
    tot_y += part[2 * w + 1];
  }
  x += bx;
  y += by;
  __syncthreads();
}

__device__ __forceinline__ int64_t wrap(int64_t i, int n) {
  const int64_t m = i % n;
  return m < 0 ? m + n : m;
}

__global__ __launch_bounds__(1024) void release_kernel(ReleaseArgs a) {
  __shared__ int64_t part[2 * MAXW];
  __shared__ int64_t first[1024];
  __shared__ int32_t count[1024];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6, nw = blockDim.x >> 6;
  const int64_t taken = a.pos[0];
  int64_t back = a.pos[1];
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + tid;
    int32_t len = 0;
    int64_t n = 0, zero = 0, tot, tz;
    if (b < a.B) {
      len = a.lens[b];
      if (a.done[b] != 0) {
        if (len > 0) n = min(((int64_t)len + a.P - 1) / a.P, (int64_t)a.W);
        len = 0;
      }
    }
    int64_t incl = n;
    scan2(incl, zero, tot, tz, part);
    first[tid] = back + incl - n;
    count[tid] = (int32_t)n;
    if (b < a.B) a.lens_out[b] = len;
    __syncthreads();
    if (tot > 0) {
      const int here = min((int)blockDim.x, a.B - b0);
      for (int i = wave; i < here; i += nw) {       // a wave per ended request
        const int c = count[i];
        const int32_t* row = a.table + (size_t)(b0 + i) * a.W;
        const int64_t at = first[i];
        for (int j = lane; j < c; j += 256) {        // four pages in flight per lane
          int32_t page[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) page[u] = j + 64 * u < c ? row[j + 64 * u] : 0;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (j + 64 * u < c) a.ring[wrap(at + j + 64 * u, a.F)] = page[u];
        }
      }
    }
    back += tot;
    __syncthreads();
  }
  if (tid == 0) {
    a.pos_out[0] = taken;
    a.pos_out[1] = back;
  }
}

// Describes row r and enters the page that it begins, from the sums.
__device__ __forceinline__ void fill_row(const PagePlanArgs& a, int r, const int32_t* cu, int64_t taken) {
  if (r >= cu[a.B]) {
    a.slot[r] = -1;
    a.row_req[r] = -1;
    a.row_len[r] = 0;
    return;
  }
  int lo = 0, hi = a.B;                 // the last b with cu[b] <= r has rows, as r < cu[B]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= r) lo = mid; else hi = mid;
  }
  const int b = lo;
  const int old = a.lens_out[b] - (cu[b + 1] - cu[b]);
  const int t = old + r - cu[b];
  const int lp = 31 - __builtin_clz(a.P);
  const int held = (old + a.P - 1) >> lp, j = t >> lp;
  int32_t* cell = a.table + (size_t)b * a.W + j;
  int32_t page;
  if (j >= held) {
    page = a.ring[wrap(taken + a.page_cu[b] + j - held, a.F)];
    if ((t & (a.P - 1)) == 0) *cell = page;      // t runs through every place of a new page
  } else {
    page = *cell;
  }
  // a page number that is none (a damaged ring or table) gives no slot
  a.slot[r] = page < 0 || page > (0x7fffffff >> lp) - 1 ? -1 : page * a.P + (t & (a.P - 1));
  a.row_req[r] = b;
  a.row_len[r] = t + 1;
}

// Sums and admission; with FILL the rows as well.
template <bool FILL>
__global__ __launch_bounds__(1024) void plan_kernel(PagePlanArgs a) {
  __shared__ int64_t part[2 * MAXW];
  __shared__ int32_t cu_l[1025];
  const int tid = threadIdx.x;
  const int64_t taken = a.pos[0], returned = a.pos[1];
  const int64_t avail = returned - taken;
  int64_t pages = 0, rows = 0, used = 0, made = 0;   // sums up to here: asked for, given
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + tid;
    int64_t len = 0, add = 0, need = 0, want = 0;
    int st = 0;
    if (b < a.B) {
      len = a.lens[b];
      add = a.add[b];
      const int64_t after = (len + add + a.P - 1) / a.P;
      st = len < 0 || add < 0 ? 8 : after > a.W ? 2 : 0;
      if (st == 0) {
        need = after - (len + a.P - 1) / a.P;
        want = add;
      }
    }
    int64_t np = need, nr = want, tot_p, tot_r;
    scan2(np, nr, tot_p, tot_r, part);
    if (st == 0 && need > 0 && pages + np > avail) st = 1;
    if (st == 0 && want > 0 && rows + nr > a.R) st = 4;
    pages += tot_p;
    rows += tot_r;
    if (st != 0) need = want = 0;
    int64_t gp = need, gr = want;
    scan2(gp, gr, tot_p, tot_r, part);
    if (b < a.B) {
      a.lens_out[b] = (int32_t)(len + want);
      a.cu[b + 1] = (int32_t)(made + gr);
      a.page_cu[b + 1] = (int32_t)(used + gp);
      a.status[b] = st;
      if (FILL && b0 == 0) cu_l[b + 1] = (int32_t)(made + gr);
    }
    used += tot_p;
    made += tot_r;
  }
  if (tid == 0) {
    a.cu[0] = 0;
    a.page_cu[0] = 0;
    cu_l[0] = 0;
    a.pos_out[0] = taken + used;
    a.pos_out[1] = returned;
  }
  if (FILL) {
    __syncthreads();                                 // cu, page_cu and lens_out of this workgroup
    for (int r = tid; r < a.R; r += blockDim.x) fill_row(a, r, cu_l, taken);
  }
}

// The rows of a long plan, behind plan_kernel<false>.
__global__ __launch_bounds__(256) void fill_kernel(PagePlanArgs a) {
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r < a.R) fill_row(a, r, a.cu, a.pos_out[0] - a.page_cu[a.B]);
}

}  // namespace

hipError_t launch_paged_release(const ReleaseArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(release_kernel, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}

// One launch while one workgroup's loop over the rows costs less than a second
// launch does, and the row sums of all requests fit its LDS: 128 requests with
// 128 rows take 4.1 us in one and 5.5 in two, with 1024 rows 6.6 and 6.4; 256
// with 2048 rows 10.6 and 7.0.
hipError_t launch_paged_plan(const PagePlanArgs& a, hipStream_t s) {
  const bool one = a.B <= 1024 && a.R <= 1024;
  if (one) {
    hipLaunchKernelGGL((plan_kernel<true>), dim3(1), dim3(a.B <= 256 ? 256 : 1024), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((plan_kernel<false>), dim3(1), dim3(a.B <= 256 ? 256 : 1024), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.R == 0) return e;
  hipLaunchKernelGGL(fill_kernel, dim3((a.R + 255) / 256), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace sgdn
