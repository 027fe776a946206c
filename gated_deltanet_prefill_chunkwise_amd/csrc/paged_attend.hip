// Attention of single rows (new tokens) over a paged cache, whole
// (sgdn_paged_attend) or by a list of blocks (sgdn_paged_attend_sparse).
//
// For one row, key/value head and tile of up to 16 of the group's query heads
// the keys are walked in tiles of 32.  With x = scale log2(e) K q and a running
// reference c >= max x - const per query head:
//   p = 2^(x - c),  l += sum p,  A += V^T p;   c' > c: l, A *= 2^(c - c')
//   o = A / l,  lse = (c + log2 l) ln 2
// Partial results (c, l, A) of waves and splits join by the same rule.
//
// Both products run transposed, so that nothing crosses lanes between them:
//   S^T [32 keys x 16 heads] = K Q^T: the keys enter as the rows of A in the
//     order  row 4m + j of tile a = key 8m + 4a + j,  so that lane (n, g)
//     receives keys 8g .. 8g+7 of head n: the B operand of the next product;
//   A^T [D x 16 heads] += V^T P^T: V^T needs eight keys per lane.  Lane (n, g)
//     loads D/16 neighbouring elements of keys 8g .. 8g+7 (whole rows by the
//     16 lanes of a g) and transposes its 8 x D/16 square with byte
//     permutations; row i of product c then is element i D/16 + c.
// K and V go from global memory to registers, without LDS: no two waves of a
// workgroup read the same keys.  The next tile's K is requested when the
// scores are done and the next V when the weights are applied, so that a wave
// has 16 KiB (D = 128) on its way at all times.
//
// The reference c moves only where x exceeds it by 4 + BIAS, which after a few
// tiles is rare.  fp16 weights are kept up to 2^(BIAS + 4) instead of 2^4: the
// type holds 2^-14 with full accuracy, and BIAS = 10 puts that at 2^-24 of the
// largest weight.
//
// 16-bit weights enter the second product in two parts, the number rounded to
// the type and what that left, itself rounded: a weight errs by 2^-17 of itself
// (bf16: a remainder of at most 2^-8, of which 8 bits are held) or 2^-23 (fp16,
// and 2^-35 of the row's largest weight, as nothing lies below 2^-24), so o by
// that part of sum p |v|.  Far under a 16-bit o's own rounding; an fp32 o of bf16
// inputs is good to 2^-17, not to fp32.  The time of the first three calls below
// stays what it is with one part.
//
// Bound: HBM, each key and value once per row.  (At most 16 of 16 columns of
// the products are used; at 16 heads a group that is 4 flops a byte.)  Rows of
// one request read it once each: 32 requests of 4096 tokens take 100, 151, 298
// and 589 us with 1, 2, 4 and 8 rows each, a prompt of 4096 tokens 2.29 ms (32/8
// heads of 128, bf16).  A list's empty entries cost what listed ones do but for
// the reads' misses: 32 rows of 8 blocks 47 us in lists of 64 and 19 in lists of 8.
// Measured: 128 rows of 2071 to 8192 tokens, 32/8 heads of 128, bf16: 516 us for
// 2.67 GB (5.2 TB/s, what a copy of 1 GiB reaches); 2 rows of 106635 and 131072
// tokens, 16/2 heads of 256, fp16: 87 us for 489 MB and 5 for the join; 32 rows
// of 64 of up to 512 blocks of 64, 32/8 of 128: 95 us for 536 MB and 5.  One
// row of 4096 tokens, 32/8 of 128: 6.9 and 3.8 us, latency.
#include <type_traits>

#include "common.h"
#include "paged.h"

namespace sgdn {

namespace {

constexpr int NW = 4;        // waves of a workgroup
constexpr int KT = 32;       // keys of a tile
constexpr int MAX_SPLITS = 256;
constexpr unsigned LEFT_GRID = 2048;   // of the rows that tiles left

template <typename E> struct Bias { static constexpr float V = 0.f; };
template <> struct Bias<fp16> { static constexpr float V = 10.f; };

// V^T fragment of element c of every lane's D/16 (16-bit elements, two per word).
template <typename E, int DW> __device__ __forceinline__ frag_t<E> v_frag(const uint32_t (&v)[8][DW], int c) {
  if constexpr (sizeof(E) == 2) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const uint32_t sel = (c & 1) ? 0x07060302u : 0x05040100u;
    u32x4 w;
#pragma unroll
    for (int d = 0; d < 4; ++d) w[d] = __builtin_amdgcn_perm(v[2 * d + 1][c >> 1], v[2 * d][c >> 1], sel);
    return __builtin_bit_cast(frag_t<E>, w);
  } else {
    frag_t<E> f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __builtin_bit_cast(float, v[j][c]);
    return f;
  }
}

template <typename E> __device__ __forceinline__ frag_t<E> ld8a(const E* p) {   // 16-byte aligned
  if constexpr (sizeof(E) == 2) {
    return ld8(p);
  } else {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
    return cat44(a, b);
  }
}

// Where 16 keys lie: their first row (of D elements) in the caches, and how
// many of them take part.
struct Half { size_t row; int n; };

template <int D> struct Joined {
  float o[NW][16][D + 4];      // the pad spreads heads over banks
  float ml[NW][16][2];
};

// One split of one (head tile, row, key/value head).
template <typename E, typename O, int D, bool SPARSE, bool LOOP>
__device__ __forceinline__ void attend_unit(const PageAttendArgs& a, int unit, int split, Joined<D>& lds) {
  constexpr int NS = D / 32;                     // reduction steps of the scores
  constexpr int EPL = D / 16;                    // elements of V per lane and key
  constexpr int DW = EPL * (int)sizeof(E) / 4;   // the same in words
  constexpr bool TWO = sizeof(E) == 2;           // weights in two parts
  constexpr float BIAS = Bias<E>::V;
  auto& joined = lds.o;
  auto& ml = lds.ml;

  int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if (LOOP) asm volatile("" : "+v"(lane), "+s"(wave));   // keep nothing made of them from unit to unit
  const int n = lane & 15, g = lane >> 4;
  const int mt = unit % a.MT;
  const int rh = unit / a.MT;
  const int h = rh / a.R, row = rh - h * a.R;
  const int req = a.row_req == nullptr ? row : a.row_req[row];
  const int P = 1 << a.lp;
  int len = min(a.row_len[row], a.max_len);
  if (req < 0 || req >= a.B) len = 0;
  const int heads = min(16, a.G - 16 * mt);      // of this tile
  const int head0 = h * a.G + 16 * mt;
  const int32_t* table = a.table + (size_t)(len > 0 ? req : 0) * a.W;
  const int32_t* list = SPARSE ? a.blocks + ((size_t)row * a.Hkv + h) * a.n_blocks : nullptr;
  const int vkeys = len <= 0 ? 0 : SPARSE ? a.n_blocks << a.lp : len;   // < 2^31: 4096 * 128
  const int nt = (int)(((int64_t)vkeys + KT - 1) / KT);
  const int t0 = (int)((int64_t)nt * split / a.S) + wave, t1 = (int)((int64_t)nt * (split + 1) / a.S);
  const E* kc = static_cast<const E*>(a.kc);
  const E* vc = static_cast<const E*>(a.vc);

  frag_t<E> qf[NS];
  {
    const E* q = static_cast<const E*>(a.q) + row * a.ldq + (size_t)(head0 + n) * D + 8 * g;
#pragma unroll
    for (int s = 0; s < NS; ++s) qf[s] = n < heads ? ld8a(q + 32 * s) : zero_frag<E>();
  }

  // Lane l looks up half l % 2 of this wave's tile number l / 2 (of the next
  // 32); the loop reads the answers lane by lane.
  int pg = 0, at = 0, cnt = 0;
  auto look_up = [&](int t) {
    const int tile = t + NW * (lane >> 1);
    const int64_t vk = (int64_t)tile * KT + 16 * (lane & 1);
    cnt = 0; pg = 0; at = 0;
    if (tile < t1 && vk < vkeys) {
      int j = (int)vk >> a.lp;
      at = (int)vk & (P - 1);
      bool ok = true;
      if (SPARSE) {
        j = list[j];
        ok = j >= 0 && j <= (len - 1) >> a.lp;
      }
      if (ok) {
        const int page = table[j];
        if (page >= 0 && page < a.n_pages) {
          pg = page;
          cnt = min(max(len - ((j << a.lp) + at), 0), 16);
        }
      }
    }
    if (cnt == 0) { pg = 0; at = 0; }   // a place that can be read: page 0
  };
  auto half = [&](int i) {              // i: lane that looked it up
    const int p = __builtin_amdgcn_readlane(pg, i), o = __builtin_amdgcn_readlane(at, i);
    return Half{((size_t)p * a.Hkv + h) * P + o, __builtin_amdgcn_readlane(cnt, i)};
  };

  frag_t<E> kf[2][NS];
  uint32_t vf[8][DW];
  auto load_k = [&](const Half& h0, const Half& h1) {
    const E* p = kc + (n < 8 ? h0.row : h1.row) * D + ((8 * (n >> 2) + (n & 3)) & 15) * D + 8 * g;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int s = 0; s < NS; ++s) kf[t][s] = ld8a(p + 4 * t * D + 32 * s);
  };
  auto load_v = [&](const Half& h0, const Half& h1) {
    const E* p = vc + (g < 2 ? h0.row : h1.row) * D + (size_t)(8 * (g & 1)) * D + n * EPL;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (DW == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(p + j * D);
        vf[j][0] = x.x; vf[j][1] = x.y;
      } else {
#pragma unroll
        for (int w = 0; w < DW / 4; ++w) {
          const V16 x = ldv(p + j * D + w * (16 / (int)sizeof(E)));
#pragma unroll
          for (int u = 0; u < 4; ++u) vf[j][4 * w + u] = x.w[u];
        }
      }
    }
  };

  float c = -INFINITY, l = 0.f;       // reference and (this lane's part of the) sum of head n
  bool seen = false;                  // uniform: some key took part
  f32x4 acc[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) acc[i] = zero4();

  int slot = 0;                       // lane of the current tile's look-up
  look_up(t0);
  // The query, here: waited for inside the loop it would wait for what follows it too.
  __builtin_amdgcn_s_waitcnt(0x0F70);                    // vmcnt(0)
  Half h0 = half(0), h1 = half(1);
  if (t0 < t1) { load_k(h0, h1); load_v(h0, h1); }
  // A tile, and (MORE) the requests of the next one.  The last tile is a copy
  // of its own: where a request may or may not follow another, a wait for the
  // older one has to be a wait for both (1 to 2% of a call).
  auto step = [&](int t, auto MORE) {
    f32x4 s0 = zero4(), s1 = zero4();
#pragma unroll
    for (int s = 0; s < NS; ++s) { s0 = mma(kf[0][s], qf[s], s0); s1 = mma(kf[1][s], qf[s], s1); }
    const Half c0 = h0, c1 = h1;
    slot += 2;
    if constexpr (MORE) {
      if (slot == 64) { look_up(t + NW); slot = 0; }
      h0 = half(slot);
      h1 = half(slot + 1);
      load_k(h0, h1);
    }
    const bool some = c0.n + c1.n > 0;
    if (some) {
      seen = true;
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) { x[j] = s0[j] * a.scale; x[4 + j] = s1[j] * a.scale; }
      if (c0.n + c1.n < 32) {
        const int live = (g < 2 ? c0.n : c1.n) - 8 * (g & 1);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j >= live) {
            x[j] = -INFINITY;
#pragma unroll
            for (int w = 0; w < DW; ++w) vf[j][w] = 0u;    // 0 * NaN would reach the sum
          }
        }
      }
      float mx = x[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) mx = fmaxf(mx, x[j]);
      if (__ballot(mx > c + (BIAS + 4.f)) != 0ull) {
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float cn = fmaxf(c, mx - BIAS);
        const float f = cn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(c - cn);
        c = cn;
        l *= f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) acc[i] *= f;
      }
      const float cs = c == -INFINITY ? 0.f : c;           // every x so far is -inf
      f32x8 p;
#pragma unroll
      for (int j = 0; j < 8; ++j) { p[j] = __builtin_amdgcn_exp2f(x[j] - cs); l += p[j]; }
      frag_t<E> ph, pl;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ph[j] = from_f<E>(p[j]);
        if (TWO) pl[j] = from_f<E>(p[j] - to_f(ph[j]));
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const frag_t<E> vt = v_frag<E, DW>(vf, i);
        acc[i] = mma(vt, ph, acc[i]);
        if (TWO) acc[i] = mma(vt, pl, acc[i]);
      }
    }
    if constexpr (MORE) load_v(h0, h1);
  };
  int t = t0;
  for (; t + NW < t1; t += NW) step(t, std::true_type{});
  if (t < t1) step(t, std::false_type{});

  // join the four waves
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  if (g == 0) { ml[wave][n][0] = c; ml[wave][n][1] = seen ? l : -1.f; }
  __syncthreads();
  float top = -INFINITY;
#pragma unroll
  for (int w = 0; w < NW; ++w) top = fmaxf(top, ml[w][n][0]);
  const float mine = c == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(c - top);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < EPL; i += 4)
      st4f(&joined[wave][n][(4 * g + j) * EPL + i],
           f32x4{acc[i][j] * mine, acc[i + 1][j] * mine, acc[i + 2][j] * mine, acc[i + 3][j] * mine});
  __syncthreads();
  for (int i = threadIdx.x; i < heads * (D / 4); i += 64 * NW) {
    const int hd = i / (D / 4), e = 4 * (i % (D / 4));
    float m = -INFINITY, sum = 0.f;
    bool any = false;
#pragma unroll
    for (int w = 0; w < NW; ++w) m = fmaxf(m, ml[w][hd][0]);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float lw = ml[w][hd][1], cw = ml[w][hd][0];
      any = any || !(lw == -1.f);
      if (cw != -INFINITY) sum += lw * __builtin_amdgcn_exp2f(cw - m);
      else if (!(lw <= 0.f)) sum = lw;                     // NaN
    }
    f32x4 o = zero4();
#pragma unroll
    for (int w = 0; w < NW; ++w) o += *reinterpret_cast<const f32x4*>(&joined[w][hd][e]);
    const size_t rq = (size_t)row * a.Hq + head0 + hd;
    if (a.S > 1) {
      const size_t to = rq * a.S + split;
      st4f(a.part_o + to * D + e, o);
      if (e == 0) { a.part_ml[2 * to] = m; a.part_ml[2 * to + 1] = any ? sum : -1.f; }
    } else {
      if (any) o /= sum;
      st4o(static_cast<O*>(a.o) + rq * D + e, o);
      if (a.lse != nullptr && e == 0)
        a.lse[rq] = any ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    }
  }
}

// Rows next to each other (SPARSE) and the head tiles of a group read the same
// pages: with one split each XCD (workgroup id mod 8) gets one run of the units.
// With S splits a workgroup's XCD is (unit' S + split) mod 8, unit' the number
// before it is permuted: for S a multiple of 8, few units, the same split of
// every unit, so that head tiles meet there as well; for other S units and splits
// are spread.  The splits outermost in the grid, a unit's on one XCD, part the head
// tiles of 8 units or fewer: one row of 32768 tokens, 64/2 heads of 128 24.2 us
// and not 15.8, 128/1 27.6 and 19.7; sparse steps of 2 to 16 splits the same
// within 2%.
__device__ __forceinline__ int unit_of_xcd(int i, int units) { return (i & 7) * ((units + 7) >> 3) + (i >> 3); }

template <typename E, typename O, int D, bool SPARSE>
__global__ __launch_bounds__(64 * NW, sizeof(E) == 2 ? 2 : 1) void attend_kernel(PageAttendArgs a, int units) {
  __shared__ Joined<D> lds;
  int unit = blockIdx.x / a.S;
  const int split = blockIdx.x - unit * a.S;
  if (SPARSE || a.MT > 1) {
    unit = unit_of_xcd(unit, units);
    if (unit >= units) return;
  }
  attend_unit<E, O, D, SPARSE, false>(a, unit, split, lds);
}

// The rows that the tiles left, S = MT = 1.  Most often there are none, and a
// workgroup for each row takes 28 us to find that out (8192 rows and heads);
// so 2048 workgroups look 64 of their units up at a time.  Whole calls of 4096
// rows of 16 of 256 blocks, a workgroup a row and so (tiles with weights in one
// part): 171 and 146 us (32/8 heads of 128, nothing left), 160 and 155 (16/2 of
// 256); 1208 and 1247, 715 and 761 where every row is left, as the work is dealt
// out ahead.  (D = 256: one wave a SIMD, as two leave too few registers for the
// loop.)
template <typename E, typename O, int D>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void left_kernel(PageAttendArgs a, int units) {
  __shared__ Joined<D> lds;
  const int all = (units + 7) / 8 * 8;                   // a multiple of 8, like the grid
  for (int64_t first = blockIdx.x; first < all; first += 64 * (int64_t)gridDim.x) {
    const int64_t at = first + lane_id() * (int64_t)gridDim.x;
    const int u = unit_of_xcd((int)min(at, (int64_t)all - 1), units);
    const int h = min(u, units - 1) / a.R, row = min(u, units - 1) - h * a.R;
    uint64_t left = __ballot(at < all && u < units && a.done[(size_t)(row / a.TQ) * a.Hkv + h] == 0);
    while (left != 0) {
      const int i = __builtin_ctzll(left);
      left &= left - 1;
      attend_unit<E, O, D, true, true>(a, unit_of_xcd((int)(first + i * (int64_t)gridDim.x), units), 0, lds);
      __syncthreads();                                   // before the next unit writes lds
    }
  }
}

// Joins the S <= 256 splits of 64 elements of a (row, query head): thread t
// sums elements 4 (t % 16) .. of the splits t / 16 + 16 i.
template <typename O, int D>
__global__ __launch_bounds__(256) void join_kernel(PageAttendArgs a) {
  __shared__ float weight[MAX_SPLITS];
  __shared__ f32x4 joined[4][16];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
  const size_t rq = blockIdx.x / (D / 64);
  const int e0 = (int)(blockIdx.x % (D / 64)) * 64 + 4 * (lane & 15);
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + rq * a.S;
  // every wave makes the maximum and the sum for itself
  float c[MAX_SPLITS / 64], l[MAX_SPLITS / 64], m = -INFINITY;
#pragma unroll
  for (int i = 0; i < MAX_SPLITS / 64; ++i) {
    const int s = 64 * i + lane;
    const float2 x = s < a.S ? ml[s] : float2{-INFINITY, -1.f};
    c[i] = x.x;
    l[i] = x.y;
    m = fmaxf(m, x.x);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  float sum = 0.f;
  bool any = false;
#pragma unroll
  for (int i = 0; i < MAX_SPLITS / 64; ++i) {
    any = any || !(l[i] == -1.f);
    const float w = c[i] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(c[i] - m);
    if (c[i] != -INFINITY) sum += l[i] * w;
    else if (!(l[i] <= 0.f)) sum += l[i];                  // NaN
    if (wave == 0) weight[64 * i + lane] = w;
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o, 64);
  any = __ballot(any) != 0ull;
  __syncthreads();
  const float* p = a.part_o + rq * a.S * D + e0;
  f32x4 acc = zero4();
#pragma unroll 4
  for (int s = tid >> 4; s < a.S; s += 16) {
    const float w = weight[s];
    if (w != 0.f) acc += w * *reinterpret_cast<const f32x4*>(p + (size_t)s * D);
  }
#pragma unroll
  for (int o = 16; o < 64; o <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], o, 64);
  if (lane < 16) joined[wave][lane] = acc;
  __syncthreads();
  if (tid < 16) {
    f32x4 o = (joined[0][tid] + joined[1][tid]) + (joined[2][tid] + joined[3][tid]);
    if (any) o /= sum;
    st4o(static_cast<O*>(a.o) + rq * D + e0, o);
    if (a.lse != nullptr && e0 == 0)
      a.lse[rq] = any ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
  }
}

template <typename E, typename O, int D> hipError_t launch_d(const PageAttendArgs& a, hipStream_t s) {
  const int units = a.R * a.Hkv * a.MT;
  const unsigned grid = (unsigned)((a.blocks != nullptr || a.MT > 1 ? (units + 7) / 8 * 8 : units) * a.S);
  if constexpr (sizeof(E) == 2) {
    if (a.done != nullptr) {
      hipLaunchKernelGGL((left_kernel<E, O, D>), dim3(grid < LEFT_GRID ? grid : LEFT_GRID), dim3(64 * NW), 0, s, a, units);
      return hipGetLastError();
    }
  }
  if (a.blocks != nullptr)
    hipLaunchKernelGGL((attend_kernel<E, O, D, true>), dim3(grid), dim3(64 * NW), 0, s, a, units);
  else
    hipLaunchKernelGGL((attend_kernel<E, O, D, false>), dim3(grid), dim3(64 * NW), 0, s, a, units);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.S == 1) return e;
  hipLaunchKernelGGL((join_kernel<O, D>), dim3((unsigned)(a.R * a.Hq * (D / 64))), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename E, typename O> hipError_t launch_o(const PageAttendArgs& a, int d, hipStream_t s) {
  if (d == 64) return launch_d<E, O, 64>(a, s);
  if (d == 128) return launch_d<E, O, 128>(a, s);
  return launch_d<E, O, 256>(a, s);
}

template <typename E> hipError_t launch_e(const PageAttendArgs& a, int o_dtype, int d, hipStream_t s) {
  if (o_dtype == 1) return launch_o<E, bf16>(a, d, s);
  if (o_dtype == 2) return launch_o<E, fp16>(a, d, s);
  return launch_o<E, float>(a, d, s);
}

}  // namespace

// Splits of each unit's keys: `groups` workgroups to keep every CU's memory
// pipeline busy, but a tile at least for each wave of one.  More groups mean
// more to join: with rows of 512 bytes 256 groups take 48 and 102 us and 512
// take 51 and 105 (1 and 2 sequences of 131072, 2 heads of 256, fp16); with
// shorter rows 512 take 16.9 and 256 17.7 (4 of 4096, 8 heads of 128, bf16;
// 1024: 19.0), 20.0 and 20.8 (7 of 5001, 3 heads of 64, fp32; 1024: 19.7).
// The lengths are on the device, so rows count alike, whatever they see: where
// rows alone make the groups, the longest is walked by one workgroup a head.
// One row of 131072 tokens and 63 of 512, or of none (32/8 heads of 128, bf16):
// 2.69 ms, the long one by itself 99 us.  Calls that split such rows off lose
// nothing.
int paged_splits(long long units, int tiles, int row_bytes) {
  const int groups = row_bytes >= 512 ? 256 : 512;
  const long long want = (groups + units - 1) / units;
  const long long most = (tiles + NW - 1) / NW;
  const long long s = want < most ? want : most;
  return (int)(s < 1 ? 1 : s > MAX_SPLITS ? MAX_SPLITS : s);
}

hipError_t launch_paged_attend(const PageAttendArgs& a, int dtype, int o_dtype, int d, hipStream_t s) {
  if (dtype == 1) return launch_e<bf16>(a, o_dtype, d, s);
  if (dtype == 2) return launch_e<fp16>(a, o_dtype, d, s);
  return launch_e<float>(a, o_dtype, d, s);
}

}  // namespace sgdn
