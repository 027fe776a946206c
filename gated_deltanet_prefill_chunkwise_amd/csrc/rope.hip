// Rotary positions of queries and keys (sgdn_rope), with a norm of every head
// in the same pass (sgdn_norm_rope).
//
//   v = x / sqrt(mean x^2 + eps) (w + w_offset), or x;  t = p f_i
//   (a, b) -> m (a cos t - b sin t, b cos t + a sin t)
//
// Bound: HBM, every head read and written once (2 R (Hq + Hk) D elements).  A
// wave takes a row, or a slice of its heads.  It makes the row's rot / 2
// angles once, a lane each, and keeps what its lanes' elements and the other
// elements of their pairs are multiplied by in registers, the weights taken in;
// then it walks the heads, 64 / (lanes of a head) at a time, 16 bytes a lane,
// the next ones on their way.  The other element of a pair is in the same lane
// (interleaved), in a lane at a fixed distance (halves of whole 16-byte units),
// or anywhere (other halves: by way of LDS); it is fetched before the norm, as
// both have the same, so that 16-bit elements move two to a word.
//
// Measured, 32 + 8 heads of 128, bf16: 797 MB of rows turned in 154 us (5.2 TB/s),
// 958 MB normed and turned in 193 us (5.0 TB/s; a copy reaches 4.99).  The
// weights come by way of LDS, once a workgroup: read by each row from memory,
// 2 bytes a load, they cost 237 us, and 316 us for those of both elements.
// Halves by way of LDS (38932 rows, 60 of 128 turned): turned 155 us like the
// others, normed and turned 227, where pairs in a lane take 170.
// Waves that walk several rows, 8192 at a time: 166 and 226 us.
//
// Angles: t = p f in fp64 with the rounding error of the product carried
// along, minus the nearest multiple n of pi/2 (as two fp64 numbers); what is
// left, at most pi/4, goes to fp32 and into Taylor polynomials (the first
// dropped terms are under 2e-9), and n mod 4 says which is which.  (Positions
// give angles far below 2^50, up to where n is the nearest but for a quarter.)
//
// Norm: squares are summed in fp64, so that heads of any magnitude are normed
// alike (fp32 sums: 188 us of 193); where 1 / norm may lie outside fp32, x is
// scaled by the power of two of the norm first.  What follows is fp32.
#include "common.h"
#include "serve.h"

namespace sgdn {

namespace {

constexpr int NW = 4;                      // waves of a workgroup
enum { INTERLEAVED, HALF_UNITS, HALF_ANY };

// cos and sin of p f.
__device__ __forceinline__ float2 turn(double p, double f) {
  const double t = p * f, low = fma(p, f, -t);
  const double n = rint(t * 0.63661977236758134308);                  // 2 / pi
  double r = fma(-n, 1.57079632679489655800e+00, t);                  // pi / 2: the nearest fp64 number
  r = fma(-n, 6.12323399573676603587e-17, r) + low;                   // and what it leaves
  if (fabs(r) > 2.0) r = 0.0;              // t past 2^52: n is off by more than the angle is known to, any turn will do
  const float x = (float)r, y = x * x;
  const float s = x * (1.f + y * (-1.f / 6 + y * (1.f / 120 + y * (-1.f / 5040 + y * (1.f / 362880)))));
  const float c = 1.f + y * (-0.5f + y * (1.f / 24 + y * (-1.f / 720 + y * (1.f / 40320 + y * (-1.f / 3628800)))));
  const int q = (int)(n - 4.0 * floor(0.25 * n)) & 3;                 // 64 bits may not hold n
  return float2{q == 0 ? c : q == 1 ? -s : q == 2 ? -c : s, q == 0 ? s : q == 1 ? c : q == 2 ? -s : -c};
}

template <typename E> struct Unit { static constexpr int N = 16 / (int)sizeof(E); };
template <typename E> union Bits { V16 v; E x[Unit<E>::N]; };

template <typename E, typename W, bool NORM, int MODE>
__global__ __launch_bounds__(64 * NW) void rope_kernel(RopeArgs a, int lanes_log) {
  constexpr int N = Unit<E>::N;            // elements of a lane
  __shared__ float2 angles[NW][128];
  __shared__ float weights[NORM ? 2 : 1][NORM ? 256 : 1];
  __shared__ float staged[MODE == HALF_ANY ? NW : 1][64 * N];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if constexpr (NORM) {
    for (int i = threadIdx.x; i < a.D; i += 64 * NW) {
      weights[0][i] = (a.wq != nullptr ? to_f(static_cast<const W*>(a.wq)[i]) : 0.f) + a.w_offset;
      weights[1][i] = (a.wk != nullptr ? to_f(static_cast<const W*>(a.wk)[i]) : 0.f) + a.w_offset;
    }
    __syncthreads();
  }
  const int64_t at = (int64_t)blockIdx.x * NW + wave;
  const int r = __builtin_amdgcn_readfirstlane((int)(at / a.slices));
  const int slice = __builtin_amdgcn_readfirstlane((int)(at - (int64_t)r * a.slices));
  if (r >= a.R) return;
  const int64_t p = (int64_t)a.pos[r] + a.pos_offset;
  if (p < 0) return;
  const int half = a.rot >> 1;
  const int per = 64 >> lanes_log;         // heads of a step, all of q or all of k
  const int u = lane & ((1 << lanes_log) - 1), e0 = u * N;
  const bool in_head = e0 < a.D;
  const int q_steps = (a.Hq + per - 1) / per, steps = q_steps + (a.Hk + per - 1) / per;
  const int g0 = (int)((int64_t)steps * slice / a.slices), g1 = (int)((int64_t)steps * (slice + 1) / a.slices);

  const auto head = [&](int g) { return (g < q_steps ? g : g - q_steps) * per + (lane >> lanes_log); };
  const auto load = [&](int g) -> V16 {
    const bool is_q = g < q_steps;
    const int h = head(g);
    if (!in_head || g >= g1 || h >= (is_q ? a.Hq : a.Hk)) return zv();
    return ldv(static_cast<const E*>(is_q ? a.q.in : a.k.in) + r * (is_q ? a.q.in_row : a.k.in_row) + h * (is_q ? a.q.in_head : a.k.in_head) + e0);
  };
  V16 next = load(g0);

  for (int i = lane; i < half; i += 64) {
    float2 cs = turn((double)p, a.freqs[i]);
    angles[wave][i] = float2{cs.x * a.magnitude, cs.y * a.magnitude};
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");

  // the lane that holds the other elements of this lane's pairs (HALF_UNITS)
  const int distance = half / N;
  const int other = e0 < half ? lane + distance : e0 < a.rot ? lane - distance : lane;

  const double inv_d = 1.0 / a.D;
  // What an element and the other one of its pair are multiplied by: cosine,
  // and sine with the sign of the place in the pair, each times the weight.
  float own[N], cross[N];
  for (int g = g0; g < g1; ++g) {
    const bool is_q = g < q_steps;
    if (g == g0 || (NORM && g == q_steps)) {
      const float* w = weights[NORM && !is_q];
      const bool turned0 = e0 < a.rot, first0 = e0 < half;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = e0 + j;
        const bool turned = MODE == HALF_UNITS ? turned0 : e < a.rot;
        const bool first = MODE == INTERLEAVED ? (e & 1) == 0 : MODE == HALF_UNITS ? first0 : e < half;
        const int i = MODE == INTERLEAVED ? e >> 1 : (first ? e0 : e0 - half) + j;
        const float2 cs = turned ? angles[wave][i] : float2{1.f, 0.f};
        own[j] = cs.x;
        cross[j] = first ? -cs.y : cs.y;
        if (NORM) {
          const int o = MODE == INTERLEAVED ? e ^ 1 : (first ? e0 + half : e0 - half) + j;
          own[j] *= in_head ? w[e] : 0.f;
          cross[j] *= turned ? w[o] : 0.f;
        }
      }
    }
    Bits<E> x;
    x.v = next;
    next = load(g + 1);
    float y[N], z[N];                      // the lane's elements, the other ones of their pairs
#pragma unroll
    for (int j = 0; j < N; ++j) y[j] = to_f(x.x[j]);
    if constexpr (MODE == INTERLEAVED) {
#pragma unroll
      for (int j = 0; j < N; ++j) z[j] = y[j ^ 1];
    } else if constexpr (MODE == HALF_UNITS) {
      Bits<E> t;
#pragma unroll
      for (int w = 0; w < 4; ++w) t.v.w[w] = (uint32_t)__shfl((int)x.v.w[w], other, 64);
#pragma unroll
      for (int j = 0; j < N; ++j) z[j] = to_f(t.x[j]);
    } else {
      float* mine = staged[wave] + (lane >> lanes_log << lanes_log) * N;
#pragma unroll
      for (int j = 0; j < N; ++j) mine[e0 + j] = y[j];
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = e0 + j;
        z[j] = e < a.rot ? mine[e < half ? e + half : e - half] : 0.f;
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    if (NORM) {
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < N; ++j) sum = fma((double)y[j], (double)y[j], sum);
      for (int o = 1; o < 1 << lanes_log; o <<= 1) sum += __shfl_xor(sum, o, 64);
      const double mean = sum * inv_d + (double)a.eps;
      // mean is 4^k times 1/2 .. 2; zero, infinite and NaN as they are
      const int k = mean > 0.0 && mean < 1e300 ? (ilogb(mean) + 1) >> 1 : 0;
      const float inv = 1.f / sqrtf((float)ldexp(mean, -2 * k));
      if (__ballot(k > 60 || k < -60) == 0ull) {
        const float scale = ldexpf(inv, -k);
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] *= scale, z[j] *= scale;
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = ldexpf(y[j], -k) * inv, z[j] = ldexpf(z[j], -k) * inv;
      }
    }
    const int h = head(g);
    if (in_head && h < (is_q ? a.Hq : a.Hk)) {
#pragma unroll
      for (int j = 0; j < N; ++j) x.x[j] = from_f<E>(e0 + j < a.rot ? fmaf(z[j], cross[j], y[j] * own[j]) : y[j] * own[j]);
      stv(static_cast<E*>(is_q ? a.q.out : a.k.out) + r * (is_q ? a.q.out_row : a.k.out_row) + h * (is_q ? a.q.out_head : a.k.out_head) + e0, x.v);
    }
  }
}

int lanes_log_of(int d, int dtype) {
  const int units = d / (dtype == 0 ? 4 : 8);
  int l = 0;
  while (1 << l < units) ++l;
  return l;
}

template <typename E, typename W, bool NORM> hipError_t launch_mode(const RopeArgs& a, int lanes_log, bool interleaved, hipStream_t s) {
  const unsigned grid = (unsigned)(((int64_t)a.R * a.slices + NW - 1) / NW);
  if (interleaved)
    hipLaunchKernelGGL((rope_kernel<E, W, NORM, INTERLEAVED>), dim3(grid), dim3(64 * NW), 0, s, a, lanes_log);
  else if ((a.rot >> 1) % Unit<E>::N == 0)
    hipLaunchKernelGGL((rope_kernel<E, W, NORM, HALF_UNITS>), dim3(grid), dim3(64 * NW), 0, s, a, lanes_log);
  else
    hipLaunchKernelGGL((rope_kernel<E, W, NORM, HALF_ANY>), dim3(grid), dim3(64 * NW), 0, s, a, lanes_log);
  return hipGetLastError();
}

template <typename E> hipError_t launch_e(const RopeArgs& a, int lanes_log, int w_dtype, bool norm, bool interleaved, hipStream_t s) {
  if (!norm) return launch_mode<E, float, false>(a, lanes_log, interleaved, s);
  if (w_dtype == 1) return launch_mode<E, bf16, true>(a, lanes_log, interleaved, s);
  if (w_dtype == 2) return launch_mode<E, fp16, true>(a, lanes_log, interleaved, s);
  return launch_mode<E, float, true>(a, lanes_log, interleaved, s);
}

}  // namespace

// Few rows: their heads are dealt out to as many waves as there are steps of
// heads, until there are enough rows to fill the chip (4096 waves).
int rope_slices(int R, int Hq, int Hk, int d, int dtype) {
  const int per = 64 >> lanes_log_of(d, dtype), steps = (Hq + per - 1) / per + (Hk + per - 1) / per;
  const int want = R >= 4096 ? 1 : (4096 + R - 1) / R;
  return want < steps ? want : steps;
}

hipError_t launch_rope(const RopeArgs& a, int dtype, int w_dtype, bool norm, bool interleaved, hipStream_t s) {
  const int l = lanes_log_of(a.D, dtype);
  if (dtype == 1) return launch_e<bf16>(a, l, w_dtype, norm, interleaved, s);
  if (dtype == 2) return launch_e<fp16>(a, l, w_dtype, norm, interleaved, s);
  return launch_e<float>(a, l, w_dtype, norm, interleaved, s);
}

}  // namespace sgdn
