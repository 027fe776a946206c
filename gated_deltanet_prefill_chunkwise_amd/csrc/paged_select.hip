// Choice of blocks for each row by a cheap score over the page summaries
// (sgdn_paged_select).
//
//   score(r, h, j) = max over the group's heads of (q8 . codes_j) sq scale_j
// q8 and sq: the query's elements as 8-bit codes with a power of two, formed
// as a page's summary is.  The products run on the 8-bit matrix cores with
// 32-bit sums: |q8 . codes| <= 127^2 256 < 2^24, so the sum is exact, stays
// exact as fp32 and under both powers of two; hence every evaluation order
// gives the same score and the choice has no border cases.
//
// score_kernel: 16 rows of A are (token, head) pairs, 16 columns of B pages;
// tokens of one tile that belong to different requests are taken request by
// request.  pick_kernel: the K largest of a row by halving the range of
// their bit patterns (counts by ballot), written in rising order.  Bound: latency for a
// decode step (the codes of a request are read once: 1/128 of its keys and
// values at P = 64), the counting for prompts.
#include "common.h"
#include "paged.h"

namespace sgdn {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// 16 neighbouring elements as fp32.
template <typename E> __device__ __forceinline__ void ld16f(const E* p, float (&x)[16]) {
  union { V16 w[sizeof(E)]; E e[16]; } f;
#pragma unroll
  for (int i = 0; i < (int)sizeof(E); ++i) f.w[i] = ldv(p + i * (16 / (int)sizeof(E)));
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = to_f(f.e[i]);
}

constexpr int SW = 4;      // waves of a score workgroup

// Grid: (groups of token tiles, heads, page splits).  GP: the rows of a tile
// that a token takes, G rounded up to a power of two, or 16 (larger groups in
// several passes).  SHARE: the waves take a tile of tokens each and all walk
// the same pages (rows that mostly belong to one request: prompts); otherwise
// the waves share a tile and divide the pages (a few rows of many requests).
// Eight page groups are looked up at a time and requested one ahead.
template <typename E, int D, bool SHARE>
__global__ __launch_bounds__(64 * SW) void score_kernel(PageSelectArgs a, int GP) {
  constexpr int NS = D / 64;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int n = lane & 15, g = lane >> 4;
  const int TT = 16 / GP;                               // tokens of a tile
  const int row0 = (SHARE ? blockIdx.x * SW + wave : blockIdx.x) * TT, h = blockIdx.y;
  const int MT = (a.G + 15) / 16;
  const int my_row = row0 + n / GP, my_head = n % GP;   // of the A operand
  const int first = 16 * (SHARE ? blockIdx.z : blockIdx.z * SW + wave);
  const int step = 16 * (SHARE ? gridDim.z : SW * gridDim.z);

  for (int mt = 0; mt < MT; ++mt) {
    // codes of the queries: A operand, lane (n, g) elements 64 s + 16 g ..
    i32x4 qc[NS];
    float sq;
    {
      const int hd = 16 * mt + my_head;
      const bool real = my_row < a.R && hd < a.G;
      const E* q = static_cast<const E*>(a.q) + (real ? my_row * a.ldq + (size_t)(h * a.G + hd) * D : 0) + 16 * g;
      float x[NS][16], top = 0.f;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        ld16f(q + 64 * s, x[s]);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (!real || !__builtin_isfinite(x[s][i])) x[s][i] = 0.f;
          top = fmaxf(top, fabsf(x[s][i]));
        }
      }
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const int e = top == 0.f ? 0 : max(ilogbf(top) - 6, -126);
      sq = ldexpf(1.f, e);
      const float inv = ldexpf(1.f, -e);                // a normal number: e <= 121
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t u = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float z = fminf(fmaxf(rintf(x[s][4 * w + i] * inv), -127.f), 127.f);
            u |= ((uint32_t)(int)z & 255u) << (8 * i);
          }
          qc[s][w] = (int)u;
        }
    }
    float sr[4];                                        // sq of D's rows 4g + j
#pragma unroll
    for (int j = 0; j < 4; ++j) sr[j] = __shfl(sq, 4 * g + j, 64);

    for (int tok = 0; tok < TT; ++tok) {                // uniform
      const int r = row0 + tok;
      if (r >= a.R) break;
      const int req = a.row_req == nullptr ? r : a.row_req[r];
      if (req < 0 || req >= a.B) continue;
      if (tok > 0 && a.row_req != nullptr && a.row_req[r - 1] == req) continue;   // taken with the token before
      // the run of tokens of this request in the tile, and the longest of them
      int last = tok, len = min(a.row_len[r], a.max_len);
      while (last + 1 < TT && row0 + last + 1 < a.R && a.row_req != nullptr && a.row_req[row0 + last + 1] == req) {
        ++last;
        len = max(len, min(a.row_len[row0 + last], a.max_len));
      }
      if (len <= 0) continue;
      const int nb = (len + (1 << a.lp) - 1) >> a.lp;
      const int32_t* table = a.table + (size_t)req * a.W;
      auto put = [&](int j, int t, float x) {
        if (t < tok || t > last || j >= nb) return;
        float* to = a.score + ((size_t)(row0 + t) * a.Hkv + h) * a.NB + j;
        *to = mt == 0 ? x : fmaxf(*to, x);
      };
      for (int p0 = first; p0 < nb; p0 += 4 * step) {
        int page[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int j = p0 + u * step + n;
          page[u] = j < nb ? table[j] : -1;
        }
        i32x4 kc[4][NS];
        float sk[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bool ok = page[u] >= 0 && page[u] < a.n_pages;
          const size_t at = (size_t)(ok ? page[u] : 0) * a.Hkv + h;
          const int8_t* cp = a.codes + at * D + 16 * g;
          if (p0 + u * step < nb) {                     // uniform
#pragma unroll
            for (int s = 0; s < NS; ++s) kc[u][s] = *reinterpret_cast<const i32x4*>(cp + 64 * s);
            sk[u] = a.scale[at];
          }
          if (!ok) sk[u] = __builtin_nanf("");
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (p0 + u * step >= nb) break;
          i32x4 acc = {0, 0, 0, 0};
#pragma unroll
          for (int s = 0; s < NS; ++s) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(qc[s], kc[u][s], acc, 0, 0, 0);
          const int j = p0 + u * step + n;
          float v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool head = 16 * mt + (4 * g + i) % GP < a.G;
            const float x = ((float)acc[i] * sr[i]) * sk[u];
            v[i] = head && x == x ? x : -INFINITY;
          }
          if (GP == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) put(j, 4 * g + i, v[i]);
          } else if (GP == 2) {
            put(j, 2 * g, fmaxf(v[0], v[1]));
            put(j, 2 * g + 1, fmaxf(v[2], v[3]));
          } else {
            float x = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
            if (GP >= 8) x = fmaxf(x, __shfl_xor(x, 16, 64));
            if (GP == 16) x = fmaxf(x, __shfl_xor(x, 32, 64));
            if ((4 * g) % GP == 0) put(j, 4 * g / GP, x);
          }
        }
      }
    }
  }
}

// One workgroup of NT threads per (row, head), up to NR scores per thread.
template <int NT, int NR>
__global__ __launch_bounds__(NT) void pick_kernel(PageSelectArgs a) {
  constexpr int NWV = NT / 64;
  __shared__ int part[2][NWV][3];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const size_t rh = blockIdx.x;
  const int row = (int)(rh / a.Hkv);
  const int req = a.row_req == nullptr ? row : a.row_req[row];
  int len = min(a.row_len[row], a.max_len);
  if (req < 0 || req >= a.B) len = 0;
  const int nb = len <= 0 ? 0 : (len + (1 << a.lp) - 1) >> a.lp;
  int32_t* out = a.blocks + rh * a.K;
  const int want = min(a.K, nb);
  for (int i = want + threadIdx.x; i < a.K; i += NT) out[i] = -1;
  if (nb <= a.K) {
    for (int i = threadIdx.x; i < nb; i += NT) out[i] = i;
    return;
  }
  // Scores as whole numbers of the same order; wave w holds a run of 64 NR.
  const float* score = a.score + rh * a.NB;
  const int base = wave * 64 * NR;
  uint32_t key[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int j = base + 64 * i + lane;
    key[i] = 0u;                                       // beyond the row: under every score
    if (j < nb) {
      const uint32_t u = __builtin_bit_cast(uint32_t, score[j] + 0.f);   // -0 counts as 0
      key[i] = (u & 0x80000000u) ? ~u : u | 0x80000000u;
      if (j < a.n_sink || j >= nb - a.n_local) key[i] = 0xffffffffu;
    }
  }
  int flip = 0;
  auto total = [&](int (&x)[3]) {                      // sums over the waves of uniform counts
    if (NWV == 1) return;
    if (lane < 3) part[flip][wave][lane] = lane == 0 ? x[0] : lane == 1 ? x[1] : x[2];
    __syncthreads();
    x[0] = x[1] = x[2] = 0;
#pragma unroll
    for (int w = 0; w < NWV; ++w)
#pragma unroll
      for (int u = 0; u < 3; ++u) x[u] += part[flip][w][u];
    flip ^= 1;
  };
  // A T with `want` keys >= T, or the largest with more; two bits at a time,
  // as a round of several waves costs a barrier.
  uint32_t T = 0u;
  bool exact = false;
  for (int bit = 30; bit >= 0 && !exact; bit -= 2) {
    int c[3] = {0, 0, 0};
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int u = 0; u < 3; ++u) c[u] += __builtin_popcountll(__ballot(key[i] >= (T | ((uint32_t)(u + 1) << bit))));
    total(c);
    const int u = c[2] >= want ? 3 : c[1] >= want ? 2 : c[0] >= want ? 1 : 0;
    T |= (uint32_t)u << bit;
    exact = u > 0 && c[u - 1] == want;
  }
  int above = 0, equal = 0;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    above += __builtin_popcountll(__ballot(key[i] > T));
    equal += __builtin_popcountll(__ballot(key[i] == T));
  }
  int above0 = 0, equal0 = 0, all_above = above;
  if (NWV > 1) {
    if (lane == 0) { part[flip][wave][0] = above; part[flip][wave][1] = equal; }
    __syncthreads();
    all_above = 0;
#pragma unroll
    for (int w = 0; w < NWV; ++w) {
      if (w == wave) above0 = all_above;
      all_above += part[flip][w][0];
      if (w < wave) equal0 += part[flip][w][1];
    }
  }
  const int ties = want - all_above;                   // of the equal ones, the first
  const uint64_t below = (1ull << lane) - 1ull;
  int done_a = above0, done_e = equal0;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const bool is_a = key[i] > T, is_e = key[i] == T;
    const uint64_t ba = __ballot(is_a), be = __ballot(is_e);
    const int ra = done_a + __builtin_popcountll(ba & below);
    const int re = done_e + __builtin_popcountll(be & below);
    if (is_a || (is_e && re < ties)) out[ra + min(re, ties)] = base + 64 * i + lane;
    done_a += __builtin_popcountll(ba);
    done_e += __builtin_popcountll(be);
  }
}

template <typename E, bool SHARE>
hipError_t launch_score_s(const PageSelectArgs& a, int d, int gp, dim3 grid, hipStream_t s) {
  if (d == 64) hipLaunchKernelGGL((score_kernel<E, 64, SHARE>), grid, dim3(64 * SW), 0, s, a, gp);
  else if (d == 128) hipLaunchKernelGGL((score_kernel<E, 128, SHARE>), grid, dim3(64 * SW), 0, s, a, gp);
  else hipLaunchKernelGGL((score_kernel<E, 256, SHARE>), grid, dim3(64 * SW), 0, s, a, gp);
  return hipGetLastError();
}

template <typename E> hipError_t launch_score(const PageSelectArgs& a, int d, hipStream_t s) {
  // Rows that share requests (more rows than requests) fill a tile; a row of
  // its own request takes one alone, so that no wave walks several tables.
  const bool share = a.R > a.B;
  int gp = 16;
  if (share)
    for (gp = 1; gp < a.G && gp < 16;) gp <<= 1;
  const int tt = 16 / gp;
  const long long tiles = ((long long)a.R + tt - 1) / tt;
  const long long gx = share ? (tiles + SW - 1) / SW : tiles;
  // page splits: enough workgroups for the chip, each wave its four page groups
  const int run = share ? 64 : 64 * SW;
  const long long most = (a.NB + run - 1) / run, want = (2048 + gx * a.Hkv - 1) / (gx * a.Hkv);
  const dim3 grid((unsigned)gx, a.Hkv, (unsigned)(want < most ? want : most));
  return share ? launch_score_s<E, true>(a, d, gp, grid, s) : launch_score_s<E, false>(a, d, gp, grid, s);
}

}  // namespace

hipError_t launch_paged_select(const PageSelectArgs& a, int dtype, int d, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (a.NB > a.K)                                      // otherwise no row has a choice
    e = dtype == 1 ? launch_score<bf16>(a, d, s) : dtype == 2 ? launch_score<fp16>(a, d, s) : launch_score<float>(a, d, s);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((size_t)a.R * a.Hkv));
  if (a.NB <= 64) hipLaunchKernelGGL((pick_kernel<64, 1>), grid, dim3(64), 0, s, a);
  else if (a.NB <= 256) hipLaunchKernelGGL((pick_kernel<64, 4>), grid, dim3(64), 0, s, a);
  else if (a.NB <= 1024) hipLaunchKernelGGL((pick_kernel<256, 4>), grid, dim3(256), 0, s, a);
  else if (a.NB <= 4096) hipLaunchKernelGGL((pick_kernel<256, 16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((pick_kernel<1024, 16>), grid, dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace sgdn
