// New keys and values into their cache slots, and the 8-bit summary of each
// page that a row completes (sgdn_paged_write).
//
// A copy of 2 R Hkv D elements: bound by HBM for prompts, by latency for a
// decode step.  A workgroup copies TR rows of one head (16-byte accesses; the
// rows of a prompt follow each other in a page, so it writes one run of
// TR D elements), then looks for rows that fill the last place of their page.
// The page's other keys were written by earlier calls, or are rows of this
// call, which stand right before it: the sum takes the former from the cache
// and the latter from the input, so that it waits for no other workgroup.
//
// Summary: m = sum / P (P a power of two, the sum in binary64: for 16-bit
// keys it is exact and free of order), scale = 2^e with max |m| < 2^(e+7),
// codes = rint(m 2^-e).  Every step but the sum is exact.
//
// Measured: 8 prompts, 50275 rows in all, 8 heads of 128, bf16: 88 us for
// 313 MB read (a page's keys come again, from the L2 or HBM, for its summary)
// and 207 MB written, 5.9 TB/s.  With TR = 8, 32 and 64 100, 95 and 102 us;
// heads fastest in the grid 109, a run of rows for each XCD 99, non-temporal
// copies 136.  A step of 128 rows: 4.1 us with TR = 8, 5.0 with 16.
#include "common.h"
#include "paged.h"

namespace sgdn {

namespace {

template <typename E, int D, int TR>
__global__ __launch_bounds__(256) void write_kernel(PageWriteArgs a) {
  constexpr int EV = 16 / sizeof(E);        // elements of a 16-byte access
  constexpr int U = D / EV;                 // accesses per row
  constexpr int CG = D / 8, RG = 256 / CG;  // column groups of 8, row groups of the sum
  __shared__ int32_t slots[TR];
  __shared__ double sums[RG][D];
  __shared__ float top[4];
  const int tid = threadIdx.x, h = blockIdx.y;
  const int64_t r0 = (int64_t)blockIdx.x * TR;
  const int P = 1 << a.lp, n_slots = a.n_pages << a.lp;
  const E* k = static_cast<const E*>(a.k) + (size_t)h * D;
  const E* v = static_cast<const E*>(a.v) + (size_t)h * D;
  E* kc = static_cast<E*>(a.kc);
  E* vc = static_cast<E*>(a.vc);
  if (tid < TR) {
    const int32_t s = r0 + tid < a.R ? a.slot[r0 + tid] : -1;
    slots[tid] = s >= 0 && s < n_slots ? s : -1;
  }
  __syncthreads();
  for (int i = tid; i < TR * U; i += 256) {
    const int r = i / U, u = i % U, s = slots[r];
    if (s < 0) continue;
    const size_t to = (((size_t)(s >> a.lp) * a.Hkv + h) * P + (s & (P - 1))) * D + u * EV;
    const V16 x = ldv(k + (r0 + r) * a.ldk + u * EV), y = ldv(v + (r0 + r) * a.ldv + u * EV);
    stv(kc + to, x);
    stv(vc + to, y);
  }
  if (a.codes == nullptr) return;
  for (int r = 0; r < TR; ++r) {
    const int s = slots[r];
    if (s < 0 || (s & (P - 1)) != P - 1) continue;     // the same for all threads
    const int page = s >> a.lp;
    const int c = tid % CG, rg = tid / CG;
    const E* old = kc + ((size_t)page * a.Hkv + h) * P * D + c * 8;
    double acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0;
    for (int t = rg; t < P; t += RG) {
      const int64_t i = r0 + r - (P - 1 - t);          // its row, if it is one of this call
      const E* from = i >= 0 && a.slot[i] == s - (P - 1 - t) ? k + i * a.ldk + c * 8 : old + (size_t)t * D;
      union { V16 w[sizeof(E) / 2]; E x[8]; } f;
#pragma unroll
      for (int w = 0; w < (int)sizeof(E) / 2; ++w) f.w[w] = ldv(from + w * EV);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += (double)to_f(f.x[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[rg][c * 8 + e] = acc[e];
    __syncthreads();
    double m = 0.0;
    if (tid < D) {
      for (int g = 0; g < RG; ++g) m += sums[g][tid];
      m *= 1.0 / P;
      if (!__builtin_isfinite(m)) m = 0.0;
    }
    // max |m| as the exponent of the largest: frexp's x with |m| < 2^x
    int x = m == 0.0 ? -10000 : ilogb(m) + 1;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x = max(x, __shfl_xor(x, o, 64));
    if (lane_id() == 0) top[tid >> 6] = (float)x;
    __syncthreads();
    const int xm = (int)fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    const int e = xm == -10000 ? 0 : min(max(xm - 7, -126), 127);
    if (tid < D) {
      const double z = rint(ldexp(m, -e));
      a.codes[((size_t)page * a.Hkv + h) * D + tid] = (int8_t)fmin(fmax(z, -127.0), 127.0);
    }
    if (tid == 0) a.scale[(size_t)page * a.Hkv + h] = ldexpf(1.f, e);
    __syncthreads();
  }
}

// Rows of a workgroup: 8 for a few rows, where more workgroups end sooner
// (128 rows of 8 heads of 128: 4.1 us against 5.0 with 16), else 16 (50275
// rows: 88 us against 100 with 8, 95 with 32, 102 with 64).
template <typename E, int D> hipError_t launch_write_d(const PageWriteArgs& a, hipStream_t s) {
  if (a.R <= 1024)
    hipLaunchKernelGGL((write_kernel<E, D, 8>), dim3((a.R + 7) / 8, a.Hkv), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((write_kernel<E, D, 16>), dim3((a.R + 15) / 16, a.Hkv), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename E> hipError_t launch_write_e(const PageWriteArgs& a, int d, hipStream_t s) {
  if (d == 64) return launch_write_d<E, 64>(a, s);
  if (d == 128) return launch_write_d<E, 128>(a, s);
  return launch_write_d<E, 256>(a, s);
}

}  // namespace

hipError_t launch_paged_write(const PageWriteArgs& a, int dtype, int d, hipStream_t s) {
  if (dtype == 1) return launch_write_e<bf16>(a, d, s);
  if (dtype == 2) return launch_write_e<fp16>(a, d, s);
  return launch_write_e<float>(a, d, s);
}

}  // namespace sgdn
