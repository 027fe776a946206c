// Choice of blocks for each row by a cheap score over the page summaries
// (sgdn_paged_select).
//
//   score(r, h, j) = max over the group's heads of (q8 . codes_j) sq scale_j
// q8 and sq: the query's elements as 8-bit codes with a power of two, formed
// as a page's summary is.  The products run on the 8-bit matrix cores with
// 32-bit sums: |q8 . codes| <= 127^2 256 < 2^22, so the sum is exact, also as
// fp32.  Only the order of a row's scores matters, so sq is taken over 2^16
// times the group's largest: whatever the queries' size, no score passes fp32
// (2^22 2^-16 2^121, the largest scale that a page has), and it is exact, all
// multiples of 2^-149 being fp32 numbers, as long as sq / (largest sq) and that
// times scale_j are >= 2^-133.  Hence every evaluation order gives the same
// score and the choice has no border cases.
//
// score_*_kernel: 16 rows of A are (token, head) pairs, 16 columns of B pages.
// pick_kernel: the K largest of a row by halving the range of
// their bit patterns (counts by ballot), written in rising order.
//
// Bound and measured: a decode step by latency (32 rows of 534 to 2048 pages of
// 64, 32/8 heads of 128: 18.3 us for 45 MB of codes and scales, 1/128 of the
// keys and values, then 11.6 to pick 64).  Prompts (6378 rows of 4 requests, up to
// 256 pages, 16/2 of 256: 31 us, and 14 to pick 16) by vector instructions first,
// scales, a maximum over heads and a store for each score that the products make:
// about half of the time (8192 rows, 1024 pages: 22.3 million of them, four
// cycles each on 1024 SIMDs, are 36 of 74 us).  The other half, LDS reads, the
// barrier of each stage of 32 pages and stores, has not been told apart.
#include <type_traits>

#include "common.h"
#include "paged.h"

namespace sgdn {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int SW = 4;      // waves of a score workgroup

// Maximum of two numbers (no NaN here): fmaxf would first quiet both.
__device__ __forceinline__ float max2(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, INFINITY); }

// Maximum over lanes l and l ^ 16, l and l ^ 32.
__device__ __forceinline__ float max_x16(float x) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const u32x2 r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t p = r[0], q = r[1];
  return max2(__builtin_bit_cast(float, p), __builtin_bit_cast(float, q));
}
__device__ __forceinline__ float max_x32(float x) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const u32x2 r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t p = r[0], q = r[1];
  return max2(__builtin_bit_cast(float, p), __builtin_bit_cast(float, q));
}

// A query tile as the A operand: lane (n, g) elements 64 s + 16 g .. + 15 of
// row n, as codes; sr: the powers of two of D's rows 4g + j, over 2^16 times
// their group's largest.
template <typename E, int NS> struct Query {
  i32x4 c[NS];
  float sr[4];
};
// Raw elements of a lane.  (Loads here take a place that can be read where
// they have none of their own: under a condition each would wait for itself.)
template <typename E, int NS> struct RawQ {
  V16 w[NS][sizeof(E)];
  __device__ __forceinline__ void load(const E* q) {
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int i = 0; i < (int)sizeof(E); ++i) w[s][i] = ldv(q + 64 * s + i * (16 / (int)sizeof(E)));
  }
  __device__ __forceinline__ float at(int s, int i) const {
    constexpr int PER = 16 / (int)sizeof(E);
    const uint32_t x = w[s][i / PER].w[(i % PER) * (int)sizeof(E) / 4];
    if constexpr (sizeof(E) == 4) {
      return __builtin_bit_cast(float, x);
    } else {
      const uint16_t half = (uint16_t)((i & 1) ? x >> 16 : x);
      return to_f(__builtin_bit_cast(E, half));
    }
  }
};
// Largest |x| of row n; elements that are not finite count as 0.  `odd` (uniform):
// there are some.
template <typename E, int NS> __device__ __forceinline__ float peak(const RawQ<E, NS>& raw, bool& odd) {
  uint32_t top = 0u;                                    // |x| by its bits: NaN over infinity over numbers
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __builtin_bit_cast(uint32_t, raw.at(s, i)) & 0x7fffffffu);
  odd = __ballot(top >= 0x7f800000u) != 0ull;
  if (odd) {
    top = 0u;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t u = __builtin_bit_cast(uint32_t, raw.at(s, i)) & 0x7fffffffu;
        if (u < 0x7f800000u) top = max(top, u);
      }
  }
  return max_x32(max_x16(__builtin_bit_cast(float, top)));
}
// Power of two of a row's codes by its peak.  (The codes of a row of zeros have
// any; the least, as it takes part in its group's largest.)
__device__ __forceinline__ int power_of(float t) { return t == 0.f ? -126 : max(ilogbf(t) - 6, -126); }
// Largest of the rows n of a group, GP (a power of two) next to each other.
template <int GP> __device__ __forceinline__ int group_max(int e) {
#pragma unroll
  for (int o = 1; o < GP; o <<= 1) e = max(e, __shfl_xor(e, o, 64));
  return e;
}
constexpr int ROOM = 16;   // powers of two over the group's largest: |q8 . codes| 2^-ROOM 2^121 < 2^127

// Codes with the power e, as the low byte of x 2^-e + 1.5 2^23, whose last place
// is 1: the sum rounds to the nearest whole number, ties to even, in two's
// complement.  `base`: the group's largest power.
template <typename E, int NS> __device__ __forceinline__ void quantise(const RawQ<E, NS>& raw, int g, int e, int base, bool odd, Query<E, NS>& q) {
  const float inv = ldexpf(1.f, -e);                    // a normal number: -126 <= e <= 121
  const float sq = ldexpf(1.f, e - base - ROOM);
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x = raw.at(s, 4 * w + i);
        if (odd && (__builtin_bit_cast(uint32_t, x) & 0x7fffffffu) >= 0x7f800000u) x = 0.f;
        z[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_fmed3f(x * inv, -127.f, 127.f) + 12582912.f);
      }
      const uint32_t lo = __builtin_amdgcn_perm(z[1], z[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(z[3], z[2], 0x04000c0cu);
      q.c[s][w] = (int)(lo | hi);
    }
#pragma unroll
  for (int j = 0; j < 4; ++j) q.sr[j] = __shfl(sq, 4 * g + j, 64);
}

// Summaries of 16 pages as the B operand: lane (n, g) bytes 64 s + 16 g .. of
// page n.  A page that is none has the scale NaN, which no maximum takes.
template <int NS> struct Pages {
  i32x4 c[NS];
  float sk;
};
template <int NS> __device__ __forceinline__ void load_pages(const PageSelectArgs& a, int page, int h, int g, Pages<NS>& p) {
  const bool ok = page >= 0 && page < a.n_pages;
  const size_t at = (size_t)(ok ? page : 0) * a.Hkv + h;
  const int8_t* cp = a.codes + at * (64 * NS) + 16 * g;
#pragma unroll
  for (int s = 0; s < NS; ++s) p.c[s] = *reinterpret_cast<const i32x4*>(cp + 64 * s);
  p.sk = a.scale[at];
  if (!ok) p.sk = __builtin_nanf("");
}

// The products of a tile: v[j] = (q8 . codes) sq 2^-base-16 for row 4g + j and page n.
// The page's scale is positive, so the maximum over heads may come before it.
template <typename E, int NS> __device__ __forceinline__ void products(const Query<E, NS>& q, const Pages<NS>& p, float (&v)[4]) {
  i32x4 acc = {0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < NS; ++s) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(q.c[s], p.c[s], acc, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = (float)acc[j] * q.sr[j];
}
__device__ __forceinline__ float scaled(float x, float sk) {
  return fmaxf(x * sk, -INFINITY);                       // NaN: -infinity
}

// One wave's share of the pages of row r and head h.  It has a batch of PG
// page groups on its way and looks up the next, the first before it turns to
// its query, as nearly all of its time is waiting.
template <typename E, int D, int PG>
__device__ __forceinline__ void score_row(const PageSelectArgs& a, int r, int h, int share, int shares) {
  constexpr int NS = D / 64;
  const int lane = lane_id(), n = lane & 15, g = lane >> 4;
  const int req = a.row_req == nullptr ? r : a.row_req[r];
  const int len = min(a.row_len[r], a.max_len);
  if (req < 0 || req >= a.B || len <= 0) return;
  const int nb = (len + (1 << a.lp) - 1) >> a.lp;
  const int32_t* table = a.table + (size_t)req * a.W;
  float* to = a.score + ((size_t)r * a.Hkv + h) * a.NB;
  const int step = 16 * PG * shares, first = 16 * PG * share;
  if (first >= nb) return;
  const E* query = static_cast<const E*>(a.q) + r * a.ldq + (size_t)(h * a.G) * D + 16 * g;
  int base = -126;                                       // the group's largest power, of all its tiles
  if (a.G > 16) {
    for (int h0 = 0; h0 < a.G; h0 += 16) {
      RawQ<E, NS> raw;
      raw.load(query + (size_t)min(h0 + n, a.G - 1) * D);
      bool odd;
      base = max(base, group_max<16>(power_of(peak<E, NS>(raw, odd))));
    }
  }
  for (int h0 = 0; h0 < a.G; h0 += 16) {
    RawQ<E, NS> raw;                                     // heads beyond the group: the last one again
    raw.load(query + (size_t)min(h0 + n, a.G - 1) * D);
    int page[PG];
    auto look_up = [&](int p0) {
#pragma unroll
      for (int u = 0; u < PG; ++u) {
        const int j = p0 + 16 * u + n;
        page[u] = table[min(j, nb - 1)];
      }
    };
    Pages<NS> pg[PG];
    look_up(first);
#pragma unroll
    for (int u = 0; u < PG; ++u) load_pages<NS>(a, page[u], h, g, pg[u]);
    look_up(first + step);
    bool odd;
    const int e = power_of(peak<E, NS>(raw, odd));
    Query<E, NS> q;
    quantise<E, NS>(raw, g, e, a.G > 16 ? base : group_max<16>(e), odd, q);
    for (int p0 = first; p0 < nb; p0 += step) {
      float x[PG], sk[PG];
#pragma unroll
      for (int u = 0; u < PG; ++u) {
        float v[4];
        products<E, NS>(q, pg[u], v);
        x[u] = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[u] = max2(x[u], v[j]);
        sk[u] = pg[u].sk;
      }
      if (p0 + step < nb) {
#pragma unroll
        for (int u = 0; u < PG; ++u) load_pages<NS>(a, page[u], h, g, pg[u]);
        look_up(p0 + 2 * step);
      }
#pragma unroll
      for (int u = 0; u < PG; ++u) {
        const float y = scaled(max_x32(max_x16(x[u])), sk[u]);
        const int j = p0 + 16 * u + n;
        if (g == 0 && j < nb) to[j] = h0 == 0 ? y : fmaxf(to[j], y);   // written by this lane
      }
    }
  }
}

// Rows of a request each (decode): the waves of a workgroup take HS heads,
// whose codes of a page are neighbours, and divide the row's pages by what is
// left.  A workgroup takes one of Z shares of the pages; the shares of all
// heads follow each other on one XCD (workgroup id mod 8), which then reads a
// page's scales once.
template <typename E, int D>
__global__ __launch_bounds__(64 * SW) void score_row_kernel(PageSelectArgs a, int HS, int Z) {
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int HB = (a.Hkv + HS - 1) / HS, PS = SW / HS;
  const int k = blockIdx.x >> 3, unit = (k / HB) * 8 + (blockIdx.x & 7);
  const int r = unit / Z, share = unit - r * Z;
  const int h = (k % HB) * HS + wave % HS;
  if (r < a.R && h < a.Hkv) score_row<E, D, 4>(a, r, h, share * PS + wave / HS, PS * Z);
}

// Many rows of a request (prompts), G <= 16: a tile holds 16 / GP tokens (GP: G
// rounded up to a power of two), a wave QT tiles.  The workgroup takes pages in
// stages of 32 through registers into two LDS buffers, the next on its way.
// (Read by each wave from global memory, a page's 16 bytes for each lane are an
// access of the L1 each: 45 million for 8192 rows and 1024 pages of two heads,
// 73 us of 99; now 74 us.  4 tiles a wave: 117, though fewer workgroups read the
// codes; 64 pages a stage and 8 waves: 67 there and no change below 4000 rows.)
// Tokens of different requests are taken request by request, and where they are
// more than a few (new tokens of other requests behind a prompt), row by row,
// each wave its own: 2048 and 100 such rows take 155 us in one call, 62 and 27
// in two (32/8 heads of 128, 512 blocks).
constexpr int QT = 2;      // 16-row tiles of a wave
constexpr int SP = 32;     // pages of a stage

// Position of 16-byte unit c of page p's codes: an LDS access reads the pages
// whose bit 2 is the same, and finds its units in different banks.
template <int D> __device__ __forceinline__ int unit_at(int p, int c) {
  return p * (D / 16) + (c ^ (D == 64 ? ((p >> 1) & 1) | ((p >> 2) & 2) : (p & 3) | ((p >> 1) & 4)));
}

template <typename E, int D, int GP>
__global__ __launch_bounds__(64 * SW, sizeof(E) == 4 ? 2 : 4) void score_rows_kernel(PageSelectArgs a) {
  constexpr int NS = D / 64, TT = 16 / GP, TW = QT * TT;
  constexpr int ROWS = SW * TW, RW = (ROWS + 63) / 64;   // of the workgroup; a lane's of them
  constexpr int RU = D / 16, NU = (SP * RU + 255) / 256; // units of a page; a thread's of a stage
  __shared__ V16 codes[2][SP * RU];
  __shared__ float scales[2][SP];
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int n = lane & 15, g = lane >> 4;
  const int wg0 = blockIdx.x * ROWS, row0 = wg0 + wave * TW, h = blockIdx.y;
  // every wave goes through the rows of the workgroup; lane l: rows l and l + 64
  int req[RW], len[RW];
  uint64_t todo[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int l = 64 * i + lane;
    req[i] = -1;
    len[i] = 0;
    if (l < ROWS && wg0 + l < a.R) {
      req[i] = a.row_req[wg0 + l];
      len[i] = min(a.row_len[wg0 + l], a.max_len);
      if (req[i] < 0 || req[i] >= a.B || len[i] <= 0) req[i] = -1;
    }
    todo[i] = __ballot(req[i] >= 0);
  }
  int runs = 0, last = -1;                               // runs of rows of one request
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    int before = __shfl_up(req[i], 1, 64);
    if (lane == 0) before = last;
    last = __builtin_amdgcn_readlane(req[i], 63);
    runs += __builtin_popcountll(__ballot(req[i] >= 0 && req[i] != before));
  }
  if (runs > 4) {
    for (int i = 0; i < TW && row0 + i < a.R; ++i) score_row<E, D, D == 256 ? 2 : 4>(a, row0 + i, h, blockIdx.z, gridDim.z);
    return;
  }
  Query<E, NS> q[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int r = min(row0 + t * TT + n / GP, a.R - 1), hd = min(n % GP, a.G - 1);
    RawQ<E, NS> raw;                                     // rows and heads beyond the last: the last again
    raw.load(static_cast<const E*>(a.q) + r * a.ldq + (size_t)(h * a.G + hd) * D + 16 * g);
    bool odd;
    const int e = power_of(peak<E, NS>(raw, odd));
    quantise<E, NS>(raw, g, e, group_max<GP>(e), odd, q[t]);
    if (sizeof(E) == 4) asm volatile("" ::: "memory");   // not all tiles' raw elements at once
  }
  while (true) {
    int now = -1;
#pragma unroll
    for (int i = RW - 1; i >= 0; --i)
      if (todo[i] != 0) now = __builtin_amdgcn_readlane(req[i], __builtin_ctzll(todo[i]));
    if (now < 0) return;
    int most = 0;
    uint32_t mine = 0;                                   // by the wave's tokens
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const uint64_t of = __ballot(req[i] == now) & todo[i];
      todo[i] &= ~of;
      if ((wave * TW) >> 6 == i) mine = (uint32_t)(of >> ((wave * TW) & 63)) & (uint32_t)((1ull << TW) - 1);
      if (req[i] == now) most = max(most, len[i]);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) most = max(most, __shfl_xor(most, o, 64));
    const int nb = __builtin_amdgcn_readfirstlane((most + (1 << a.lp) - 1) >> a.lp);
    const int32_t* table = a.table + (size_t)now * a.W;
    const int step = SP * gridDim.z, first = SP * blockIdx.z;
    if (first >= nb) continue;
    // where this lane's scores go, by tile, and whether they are of this request
    constexpr int PER = GP >= 4 ? 1 : 4 / GP;            // tokens of a lane's four rows
    float* to[QT][PER];
    bool ours[QT][PER];
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int tok = t * TT + 4 * g / GP + i;
        ours[t][i] = (4 * g) % GP == 0 || GP < 4 ? ((mine >> tok) & 1) != 0 : false;
        to[t][i] = a.score + ((size_t)(row0 + tok) * a.Hkv + h) * a.NB + n;
      }
    // this thread's units tid, tid + 256 of a stage; wave 0 has the scales too
    int page[NU], spage = 0, held = 0;
    V16 unit[NU];
    float scale = 0.f;
    auto look_up = [&](int p0) {
#pragma unroll
      for (int i = 0; i < NU; ++i) page[i] = table[min(p0 + ((tid + 256 * i) / RU) % SP, nb - 1)];
      if (wave == 0) spage = table[min(p0 + tid % SP, nb - 1)];
    };
    auto fetch = [&]() {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const size_t at = (size_t)(page[i] >= 0 && page[i] < a.n_pages ? page[i] : 0) * a.Hkv + h;
        unit[i] = ldv(a.codes + at * D + 16 * ((tid + 256 * i) % RU));
      }
      if (wave == 0) scale = a.scale[(size_t)(spage >= 0 && spage < a.n_pages ? spage : 0) * a.Hkv + h];
      held = spage;
    };
    auto store = [&](int buf) {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int u = tid + 256 * i;
        if (u < SP * RU) codes[buf][unit_at<D>(u / RU, u % RU)] = unit[i];
      }
      if (tid < SP) scales[buf][tid] = held >= 0 && held < a.n_pages ? scale : __builtin_nanf("");   // which no maximum takes
    };
    look_up(first);
    fetch();
    look_up(first + step);
    lds_barrier();                                       // the last request's stages have been read
    store(0);
    lds_barrier();
    int buf = 0;
    for (int p0 = first; p0 < nb; p0 += step) {
      const bool more = p0 + step < nb;
      if (more) {
        fetch();
        look_up(p0 + 2 * step);
      }
      float x[2][QT][PER];
      if (mine != 0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          Pages<NS> pg;
#pragma unroll
          for (int s = 0; s < NS; ++s) pg.c[s] = __builtin_bit_cast(i32x4, codes[buf][unit_at<D>(16 * u + n, 4 * s + g)]);
          pg.sk = scales[buf][16 * u + n];
#pragma unroll
          for (int t = 0; t < QT; ++t) {
            float v[4];
            products<E, NS>(q[t], pg, v);
            float (&y)[PER] = x[u][t];
            if constexpr (GP >= 4) {
              y[0] = max2(max2(v[0], v[1]), max2(v[2], v[3]));
              if (GP >= 8) y[0] = max_x16(y[0]);
              if (GP == 16) y[0] = max_x32(y[0]);
            } else if constexpr (GP == 2) {
              y[0] = max2(v[0], v[1]);
              y[1] = max2(v[2], v[3]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) y[i] = v[i];
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) y[i] = scaled(y[i], pg.sk);
          }
        }
      }
      // The next stage before the scores go out: a wait for what was fetched
      // would wait for them as well.
      if (more) store(buf ^ 1);
      if (mine != 0) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int t = 0; t < QT; ++t)
#pragma unroll
            for (int i = 0; i < PER; ++i)
              if (p0 + 16 * u + n < nb && ours[t][i]) to[t][i][p0 + 16 * u] = x[u][t][i];
      }
      lds_barrier();
      buf ^= 1;
    }
  }
}

// Orders a wave's own LDS writes before its reads.
__device__ __forceinline__ void lds_wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Maximum over a wave's lanes (all active) by row shifts and broadcasts.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  auto step = [&](auto ctrl) {
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, decltype(ctrl)::value, 0xf, 0xf, false));
  };
  step(std::integral_constant<int, 0x111>{});         // row_shr 1, 2, 4, 8
  step(std::integral_constant<int, 0x112>{});
  step(std::integral_constant<int, 0x114>{});
  step(std::integral_constant<int, 0x118>{});
  step(std::integral_constant<int, 0x142>{});         // row_bcast 15, 31
  step(std::integral_constant<int, 0x143>{});
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// NWV waves per (row, head), up to NR scores per lane; single waves come four
// to a workgroup.
template <int NWV, int NR>
__global__ __launch_bounds__(NWV == 1 ? 256 : 64 * NWV) void pick_kernel(PageSelectArgs a) {
  constexpr int NT = 64 * NWV;
  constexpr int ROWS = NWV == 1 ? 4 : 1;
  // Candidates that are ranked one against all: a step of the ranking costs a
  // wave about what NR / 4 + 4 steps of narrowing do, without their barriers.
  constexpr int FEW = NWV == 1 ? 8 : 16;
  __shared__ uint32_t part[2][NWV][2];
  __shared__ uint32_t cands[ROWS][64];
  const int lane = lane_id(), w0 = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wave = NWV == 1 ? 0 : w0, tid = NWV == 1 ? lane : (int)threadIdx.x;
  uint32_t* cand = cands[NWV == 1 ? w0 : 0];
  const int64_t rh = (int64_t)blockIdx.x * ROWS + (NWV == 1 ? w0 : 0);
  const int row = (int)(rh / a.Hkv);
  if (row >= a.R) return;
  const int req = a.row_req == nullptr ? row : a.row_req[row];
  int len = min(a.row_len[row], a.max_len);
  if (req < 0 || req >= a.B) len = 0;
  const int nb = len <= 0 ? 0 : (len + (1 << a.lp) - 1) >> a.lp;
  int32_t* out = a.blocks + rh * a.K;
  const int want = min(a.K, nb);
  for (int i = want + tid; i < a.K; i += NT) out[i] = -1;
  if (nb <= a.K) {
    for (int i = tid; i < nb; i += NT) out[i] = i;
    return;
  }
  // Scores as whole numbers of the same order; wave w holds a run of 64 NR.
  const float* score = a.score + rh * a.NB;
  const int base = wave * 64 * NR;
  uint32_t key[NR];
  float raw[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) raw[i] = score[min(base + 64 * i + lane, nb - 1)];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int j = base + 64 * i + lane;
    const uint32_t u = __builtin_bit_cast(uint32_t, raw[i] + 0.f);       // -0 counts as 0
    key[i] = (u & 0x80000000u) ? ~u : u | 0x80000000u;
    if (j < a.n_sink || j >= nb - a.n_local) key[i] = 0xffffffffu;
    if (j >= nb) key[i] = 0u;                            // beyond the row: under every score
  }
  int flip = 0;
  auto share = [&](uint32_t x, uint32_t y) {             // two uniform numbers of each wave, for all to read
    if (lane == 0) { part[flip][wave][0] = x; part[flip][wave][1] = y; }
    __syncthreads();
    flip ^= 1;                                           // the other buffer is free: all have passed it
  };
  uint32_t top = 0u, low = 0u;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    if (key[i] != 0xffffffffu) top = max(top, key[i]);
    if (key[i] != 0u) low = max(low, ~key[i]);
  }
  top = wave_max(top);
  low = wave_max(low);
  if (NWV > 1) {
    share(top, low);
#pragma unroll
    for (int w = 0; w < NWV; ++w) {
      top = max(top, part[flip ^ 1][w][0]);
      low = max(low, part[flip ^ 1][w][1]);
    }
  }
  // Narrow lo < hi, clo = count(key >= lo) > want > chi = count(key >= hi), in
  // turn where the two counts put the wanted rank and in the middle, until at
  // most FEW keys lie between (or more, all equal).
  const int forced = a.n_sink + a.n_local;               // nb > K >= forced: the two runs do not meet
  uint32_t lo = ~low, hi = top + 1;                      // scores stay under 0xff800001
  int clo = nb, chi = forced;
  bool even = true;
  while (clo - chi > FEW && clo != want && chi != want && lo + 1 < hi) {
    uint32_t mid = lo + ((hi - lo) >> 1);
    if (even) {
      const float f = (float)(clo - want) * __builtin_amdgcn_rcpf((float)(clo - chi));
      mid = lo + (uint32_t)((float)(hi - lo) * f);
      mid = min(max(mid, lo + 1), hi - 1);
    }
    even = !even;
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < NR; ++i) cnt += __builtin_popcountll(__ballot(key[i] >= mid));
    if (NWV > 1) {
      share((uint32_t)cnt, 0u);
      cnt = 0;
#pragma unroll
      for (int w = 0; w < NWV; ++w) cnt += (int)part[flip ^ 1][w][0];
    }
    if (cnt >= want) { lo = mid; clo = cnt; } else { hi = mid; chi = cnt; }
  }
  // Everything >= hi is picked, and want - chi of the m = clo - chi candidates
  // in lo .. hi - 1: rank them, the first of equal ones in front.
  const int m = clo - chi, need = want - chi;
  int above = 0, between = 0;                            // of this wave
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    above += __builtin_popcountll(__ballot(key[i] >= hi));
    between += __builtin_popcountll(__ballot(key[i] >= lo && key[i] < hi));
  }
  int above0 = 0, between0 = 0;
  if (NWV > 1) {
    share((uint32_t)above, (uint32_t)between);
#pragma unroll
    for (int w = 0; w < NWV; ++w)
      if (w < wave) { above0 += (int)part[flip ^ 1][w][0]; between0 += (int)part[flip ^ 1][w][1]; }
  }
  const uint64_t below = (1ull << lane) - 1ull;
  uint64_t picked = ~0ull;                               // by a candidate's place, where m <= 64
  if (need > 0 && m <= 64) {
    int c = between0;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const bool is = key[i] >= lo && key[i] < hi;
      const uint64_t b = __ballot(is);
      if (b == 0ull) continue;
      if (is) cand[c + __builtin_popcountll(b & below)] = key[i];
      c += __builtin_popcountll(b);
    }
    if (NWV > 1) __syncthreads(); else lds_wave_fence();
    const uint32_t mine = lane < m ? cand[lane] : 0u;
    int rank = 0;
    for (int j = 0; j < m; ++j) {
      const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)mine, j);
      rank += other > mine || (other == mine && j < lane) ? 1 : 0;
    }
    picked = __ballot(lane < m && rank < need);
  }
  const bool by_place = m > 64;                          // all candidates are equal
  int done = above0, seen = between0;                    // picked so far, candidates so far
  if (by_place) done += min(between0, need);
  else if (need > 0) done += __builtin_popcountll(between0 >= 64 ? picked : picked & ((1ull << between0) - 1ull));
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const bool is = key[i] >= lo && key[i] < hi;
    const uint64_t ca = __ballot(is), ge = __ballot(key[i] >= hi);
    if ((ca | ge) == 0ull) continue;
    const int c = seen + __builtin_popcountll(ca & below);
    const bool take = key[i] >= hi || (is && need > 0 && (by_place ? c < need : (picked >> c) & 1));
    const uint64_t b = __ballot(take);
    if (take) out[done + __builtin_popcountll(b & below)] = base + 64 * i + lane;
    done += __builtin_popcountll(b);
    seen += __builtin_popcountll(ca);
  }
}

template <typename E, int D> hipError_t launch_score_d(const PageSelectArgs& a, hipStream_t s) {
  // Rows of a request share its pages if they fill a quarter of a workgroup
  // (which takes its requests one after the other) and all rows the chip;
  // otherwise, or with more heads than a tile, a row at a time.  Shared and
  // alone, 512 blocks, 32/8 heads of 128: 32 requests with 2, 4, 6, 8 and 32 rows
  // each 55 and 19, 39 and 29, 37 and 36, 31 and 38, 39 and 104 us; 1 request
  // with 16, 64, 128 rows 14 and 12, 16 and 19, 18 and 26; 16/2 heads of 256: 16
  // with 16 each (1000 blocks) 20 and 35; 8/8 of 64: 64 with 8 each 87 and 46.
  // (All requests of these had rows.  B counts the block table's: 2048 rows of one
  // request take 39 us with its row alone for a table and 102 in a table of 512.)
  int gp = 1;
  while (gp < a.G) gp <<= 1;
  if ((int64_t)a.R * gp >= 32 * (int64_t)a.B && (int64_t)a.R * a.Hkv * D >= 1 << 16 && a.G <= 16) {
    const unsigned per = QT * SW * (16 / gp), gx = (a.R + per - 1) / per;
    const unsigned want = (512 + gx * a.Hkv - 1) / (gx * a.Hkv), most = (a.NB + 127) / 128;
    const dim3 grid(gx, a.Hkv, want < most ? want : most);
    switch (gp) {
      case 1: hipLaunchKernelGGL((score_rows_kernel<E, D, 1>), grid, dim3(64 * SW), 0, s, a); break;
      case 2: hipLaunchKernelGGL((score_rows_kernel<E, D, 2>), grid, dim3(64 * SW), 0, s, a); break;
      case 4: hipLaunchKernelGGL((score_rows_kernel<E, D, 4>), grid, dim3(64 * SW), 0, s, a); break;
      case 8: hipLaunchKernelGGL((score_rows_kernel<E, D, 8>), grid, dim3(64 * SW), 0, s, a); break;
      default: hipLaunchKernelGGL((score_rows_kernel<E, D, 16>), grid, dim3(64 * SW), 0, s, a); break;
    }
    return hipGetLastError();
  }
  const int hs = a.Hkv >= 4 ? 4 : a.Hkv >= 2 ? 2 : 1, hb = (a.Hkv + hs - 1) / hs;
  const long long rh = (long long)a.R * hb;
  const long long want = (1024 + rh - 1) / rh, most = (a.NB + 64 * (SW / hs) - 1) / (64 * (SW / hs));
  const int z = (int)(want < most ? want : most);
  const long long units = ((long long)a.R * z + 7) / 8 * 8;
  hipLaunchKernelGGL((score_row_kernel<E, D>), dim3((unsigned)(units * hb)), dim3(64 * SW), 0, s, a, hs, z);
  return hipGetLastError();
}

template <typename E> hipError_t launch_score(const PageSelectArgs& a, int d, hipStream_t s) {
  if (d == 64) return launch_score_d<E, 64>(a, s);
  if (d == 128) return launch_score_d<E, 128>(a, s);
  return launch_score_d<E, 256>(a, s);
}

}  // namespace

hipError_t launch_paged_select(const PageSelectArgs& a, int dtype, int d, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (a.NB > a.K)                                      // otherwise no row has a choice
    e = dtype == 1 ? launch_score<bf16>(a, d, s) : dtype == 2 ? launch_score<fp16>(a, d, s) : launch_score<float>(a, d, s);
  if (e != hipSuccess) return e;
  // One wave for each row while it holds the scores in 4 registers, or in 16
  // where the rows alone fill the chip (1000 blocks, scores included: 2048 rows
  // 66.9 us with one wave and 68.3 with four, 256 rows 21.2 and 18.6); else as
  // many waves as that takes.
  const long long rows = (long long)a.R * a.Hkv;
  const dim3 many((unsigned)rows), four((unsigned)((rows + 3) / 4));
  if (a.NB <= 64) hipLaunchKernelGGL((pick_kernel<1, 1>), four, dim3(256), 0, s, a);
  else if (a.NB <= 256) hipLaunchKernelGGL((pick_kernel<1, 4>), four, dim3(256), 0, s, a);
  else if (a.NB <= 1024 && rows >= 2048) hipLaunchKernelGGL((pick_kernel<1, 16>), four, dim3(256), 0, s, a);
  else if (a.NB <= 1024) hipLaunchKernelGGL((pick_kernel<4, 4>), many, dim3(256), 0, s, a);
  else if (a.NB <= 2048) hipLaunchKernelGGL((pick_kernel<4, 8>), many, dim3(256), 0, s, a);
  else if (a.NB <= 4096) hipLaunchKernelGGL((pick_kernel<4, 16>), many, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((pick_kernel<16, 16>), many, dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace sgdn
