// Attention of chunks of new tokens over a paged cache (sgdn_paged_attend_chunk):
// the plan, the kernel for fp32 and the join.  chunk16.hip has the 16-bit types.
//
// For a tile of columns ((row, query head) pairs of one request and key/value
// head) the keys are walked in blocks.  With x = scale log2(e) K q and a running
// reference c >= max x - const per column:
//   p = 2^(x - c),  l += sum p,  A += V^T p;   c' > c: l, A *= 2^(c - c')
//   o = A / l,  lse = (c + log2 l) ln 2
//
// Work: a tile costs a unit for each block of 64 keys and CHUNK_TILE more.  The costs of
// all tiles, one after the other, are cut into S equal shares, a workgroup for
// each share and head tile: whatever the lengths, all end together.  A tile
// that a cut goes through is made in parts (at most two a workgroup that are not
// whole tiles), which the join adds up by the rule above.  Shares are larger than
// that where the longest tile would fall into more parts than are worth joining.
//
// Measured (plan, attention, join): 16 rows over 4096 tokens, 32 / 8 heads of 128,
// bf16: 5.1, 13.2 and 7.6 us; fp32, 3 prompts of up to 301 rows over up to 1501 tokens,
// 15 / 3 heads of 64: 6.4, 64 and 7.2 us.  The plan is latency (a chain of sums), the join
// reads the parts once, four at a time (one by one: 13.4 us for the 16 rows) and by
// four sets of waves (one set: 9.2).
#include "chunk.h"
#include "chunk_rules.h"

namespace sgdn {

namespace {

// Units of cost: a part of fewer blocks costs more to join than it saves (the 16
// rows above, all three kernels: shares of 2, 4, 8 units 33, 25 and 26 us).
constexpr int MIN_SHARE = 4;

// Tiles of every request, in order; then those of the rows that belong to none
// (they write zeros).  One workgroup: the requests come in steps of NT, a thread
// each, and so do each step's tiles, which find their request in the sums of
// tiles by bisection.  Latency: 256 threads, where they hold all requests and
// tiles, sooner agree on a sum.
template <int NT>
__global__ __launch_bounds__(NT) void plan_kernel(ChunkArgs a) {
  constexpr int NW = NT / 64;
  __shared__ int row0[NT], rows[NT], most;
  __shared__ int64_t first[NT], sees[NT], part[NW];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
  // exclusive sums over the workgroup
  auto scan = [&](int64_t x, int64_t& total) {
    int64_t s = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t y = __shfl_up(s, o, 64);
      if (lane >= o) s += y;
    }
    if (lane == 63) part[wave] = s;
    __syncthreads();
    int64_t before = s - x;
    total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) { if (w < wave) before += part[w]; total += part[w]; }
    return before;
  };
  if (tid == 0) most = 0;              // units of the longest tile
  int base = 0, mine = -1;             // this thread's tile of the last step
  int64_t cost = 0, from = 0, to = 0;  // ... and what it takes
  for (int64_t b0 = 0; b0 < (int64_t)a.B + 2; b0 += NT) {
    const int64_t b = b0 + tid;
    int r0 = 0, r1 = 0;                // B: behind the last request, B + 1: in front of the first
    int64_t ahead = -(INT64_C(1) << 40);   // rows of none see none
    if (b < a.B) { r0 = a.cu[b]; r1 = a.cu[b + 1]; ahead = (int64_t)a.lens[b] - r1; }
    else if (b == a.B) { r0 = a.cu[a.B]; r1 = a.R; }
    else if (b == (int64_t)a.B + 1) { r1 = a.cu[0]; }
    r0 = min(max(r0, 0), a.R);
    r1 = min(max(r1, r0), a.R);
    int64_t total;                     // where cu falls, more than 32 bits may hold
    const int64_t before = scan((r1 - r0 + a.TR - 1) / a.TR, total);
    row0[tid] = r0;
    rows[tid] = r1 - r0;
    sees[tid] = ahead;
    first[tid] = before;
    __syncthreads();
    for (int64_t t0 = 0; t0 < min(total, (int64_t)a.cap - base); t0 += NT) {
      const int64_t t = t0 + tid;
      ChunkTile x{0, 0, -1, 0, 0, 0};  // stays so where cu falls and the sums mean nothing
      mine = t < min(total, (int64_t)a.cap - base) ? (int)(base + t) : -1;
      if (mine >= 0) {
        int lo = 0, hi = NT - 1;       // the last request whose first tile is t or one in front
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (first[mid] <= t) lo = mid; else hi = mid - 1;
        }
        const int64_t at = (t - first[lo]) * a.TR;
        if (at >= 0 && at < rows[lo]) {
          x.row0 = row0[lo] + (int)at;
          x.rows = min(a.TR, rows[lo] - (int)at);
          x.req = b0 + lo < a.B ? (int)(b0 + lo) : -1;
          x.ahead = sees[lo];
          x.longest = (int)min(max(sees[lo] + x.row0 + x.rows, (int64_t)0), (int64_t)a.max_len);
        }
      }
      int64_t all;
      const int64_t takes = mine >= 0 ? (int64_t)chunk_blocks(x.longest) + CHUNK_TILE : 0;
      x.at = cost + scan(takes, all);
      if (mine >= 0) {
        a.tiles[mine] = x;
        atomicMax(&most, (int)takes);
      }
      from = x.at;
      to = x.at + takes;
      cost += all;
      __syncthreads();                 // before the next sums
    }
    base = (int)min(base + total, (int64_t)a.cap);
    __syncthreads();
  }
  const int64_t share = max((cost + a.S - 1) / a.S, (int64_t)max(MIN_SHARE, (int)sqrtf((float)most * a.balance)));
  if (tid == 0) *a.head = ChunkHead{share, base, 0};
  for (int s = tid; s < a.S; s += NT)
    if (s * share >= cost) a.start[s] = base;               // nothing to do
  // The slots that begin inside of a tile.
  auto begins = [&](int t, int64_t from, int64_t to) {
    for (int64_t s = (from + share - 1) / share; s * share < to; ++s) a.start[s] = t;
  };
  if (base <= NT && (int64_t)a.B + 2 <= NT) {               // a step of requests and one of tiles: they are at hand
    if (mine >= 0) begins(mine, from, to);
    return;
  }
  for (int t = tid; t < base; t += NT) {
    const int64_t at = a.tiles[t].at;
    begins(t, at, at + chunk_blocks(a.tiles[t].longest) + CHUNK_TILE);
  }
}

// Joins the parts of a tile, of slots s, s + 1, ..: a workgroup takes the cut
// between slots s and s + 1, if it is the first of its tile, a head tile and the
// CW columns of a wave.  Parts lie as in that wave's registers, 4 elements a lane:
// run i of 64 lanes holds, of column n = lane % CW, elements e(i, lane) .. + 3.
// A wave takes a quarter of the runs.  Of PG sets of four waves each takes every
// PG-th AT_ONCE parts, and the first adds up what the others have.
template <typename O, int D, int COLS, int CW, int PG>
__global__ __launch_bounds__(256 * PG) void join_kernel(ChunkArgs a) {
  constexpr int NR = CW * D / 256;                           // runs of a wave's columns
  constexpr int OTHERS = PG > 1 ? PG - 1 : 1;
  __shared__ f32x4 sums[OTHERS][PG > 1 ? 4 : 1][NR / 4][64];
  __shared__ float2 stats[OTHERS][4][64];
  const int heads = a.Hkv * a.MT, waves = COLS / CW;
  const int wave = blockIdx.x % waves, hm = blockIdx.x / waves % heads, s = blockIdx.x / waves / heads;
  const int tile = a.start[s + 1];
  if (tile >= a.head->tiles) return;
  const ChunkTile t = a.tiles[tile];
  const int64_t share = a.head->share, to = t.at + chunk_blocks(t.longest) + CHUNK_TILE;
  if (t.at >= (s + 1) * share || t.at / share != s) return;  // begins at the cut, or has one in front
  const int last = (int)((to - 1) / share);
  const int h = hm / a.MT, mt = hm - h * a.MT, gt = min(a.GT, a.G - mt * a.GT);
  const int lane = lane_id(), i0 = (threadIdx.x >> 6) & 3, set = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int col = wave * CW + lane % CW, my_row = col / a.GT, my_head = col - my_row * a.GT;
  const bool mine = my_row < t.rows && my_head < gt;
  if (PG == 1 && !mine) return;
  auto part = [&](int i) { return ((size_t)(i == s ? 2 * s + 1 : 2 * i) * heads + hm) * COLS; };
  // A running reference, as the keys have: one pass, the next parts on their way.
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
  float m = -INFINITY, sum = 0.f;
  bool any = false;
  f32x4 acc[NR / 4];
#pragma unroll
  for (int k = 0; k < NR / 4; ++k) acc[k] = zero4();
  auto add = [&](float c, float l, const f32x4 (&o)[NR / 4]) {
    if (l == -1.f) return;                                   // saw nothing
    any = true;
    if (c == -INFINITY) {                                    // scores of -inf alone, or NaN: sums of 0, or NaN
      if (!(l <= 0.f)) sum += l;
#pragma unroll
      for (int k = 0; k < NR / 4; ++k) acc[k] += o[k];
      return;
    }
    const float top = fmaxf(m, c), w = __builtin_amdgcn_exp2f(c - top), f = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - top);
    m = top;
    sum = fmaf(l, w, sum * f);
#pragma unroll
    for (int k = 0; k < NR / 4; ++k) acc[k] = acc[k] * f + w * o[k];
  };
  constexpr int AT_ONCE = NR > 16 ? 2 : 4;
  for (int i = s + set * AT_ONCE; i <= last; i += PG * AT_ONCE) {
    float2 x[AT_ONCE];
    f32x4 o[AT_ONCE][NR / 4];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      const size_t p = part(min(i + j, last));
      x[j] = ml[p + col];
      const float* from = a.part_o + (p + wave * CW) * D + 4 * lane;
#pragma unroll
      for (int k = 0; k < NR / 4; ++k) o[j][k] = *reinterpret_cast<const f32x4*>(from + (i0 + 4 * k) * 256);
    }
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j)
      if (i + j <= last) add(x[j].x, x[j].y, o[j]);
  }
  if (PG > 1 && last - s >= AT_ONCE) {                                 // more than one set has parts
    if (set > 0) {
      stats[set - 1][i0][lane] = float2{m, any ? sum : -1.f};
#pragma unroll
      for (int k = 0; k < NR / 4; ++k) sums[set - 1][i0][k][lane] = acc[k];
    }
    __syncthreads();
    if (set == 0)
#pragma unroll
      for (int j = 0; j < PG - 1; ++j) {
        const float2 x = stats[j][i0][lane];
        f32x4 o[NR / 4];
#pragma unroll
        for (int k = 0; k < NR / 4; ++k) o[k] = sums[j][i0][k][lane];
        add(x.x, x.y, o);
      }
  }
  if (set > 0 || !mine) return;
  const size_t rq = (size_t)(t.row0 + my_row) * a.Hq + h * a.G + mt * a.GT + my_head;
#pragma unroll
  for (int k = 0; k < NR / 4; ++k) {
    const int i = i0 + 4 * k, e = CW == 32 ? 32 * (i >> 2) + 8 * (i & 3) + 4 * (lane >> 5) : 16 * i + 4 * (lane >> 4);
    f32x4 o = acc[k];
    if (any) o /= sum;
    st4o(static_cast<O*>(a.o) + rq * D + e, o);
  }
  if (i0 == 0 && lane < CW && a.lse != nullptr) a.lse[rq] = any ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// fp32: 64 columns a tile, 16 a wave; keys and values in stages of 32 through
// LDS; 16 x 16 x 4 products (the 3.6 GFLOP above would take 23 us at the 154 TFLOP/s
// of a large product).  The next stage on its way through registers while one is
// used: 117 us -> 80 for all three kernels, four workgroups a CU instead of two: 71 to
// 73.  A prompt of 4096, 32 / 8 heads of 128: 1490 us, products alone 893; 16 / 2 of
// 256: 2600 us, as its accumulators lie in scratch (272 bytes a lane) and every stage
// loads and stores them: the loops over values that are not finite are too large to
// unroll there, so that they index the accumulators at run time.
constexpr int SK = 32, COLS32 = 64;

template <typename O, int D>
__global__ __launch_bounds__(256, D == 64 ? 4 : 2) void chunk32_kernel(ChunkArgs a) {
  constexpr int NS = D / 32, DT = D / 16, LD = D + 4, RU = D / 4;
  __shared__ __attribute__((aligned(16))) float ks[SK * LD];
  __shared__ __attribute__((aligned(16))) float vs[SK * LD];
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int heads = a.Hkv * a.MT;
  const int slot = blockIdx.x / heads, hm = blockIdx.x - slot * heads, h = hm / a.MT, mt = hm - h * a.MT;
  const int head0 = h * a.G + mt * a.GT, gt = min(a.GT, a.G - mt * a.GT);
  const int P = 1 << a.lp;
  const float* kc = static_cast<const float*>(a.kc);
  const float* vc = static_cast<const float*>(a.vc);
  auto ld = [](const float* p) { return cat44(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4)); };

  const int64_t share = a.head->share, begin = slot * share, end = begin + share;
  const int tiles = a.head->tiles;
  for (int ti = a.start[slot]; ti < tiles; ++ti) {
    const ChunkTile t = a.tiles[ti];
    if (t.at >= end) break;
    if (t.rows <= 0) continue;
    const ChunkPart part = chunk_part(t, begin, end);
    const int col = 16 * wave + n, my_row = col / a.GT, my_head = col - my_row * a.GT;
    const bool real = my_row < t.rows && my_head < gt;
    const int row = t.row0 + min(my_row, t.rows - 1), head = head0 + min(my_head, gt - 1);
    const int len = real ? chunk_sees(a, t, row) : 0;
    const int32_t* table = a.table + (size_t)max(t.req, 0) * a.W;
    frag_t<float> qf[NS];
    {
      const float* q = static_cast<const float*>(a.q) + row * a.ldq + (size_t)head * D + 8 * g;
#pragma unroll
      for (int s = 0; s < NS; ++s) qf[s] = ld(q + 32 * s);
    }
    float c = -INFINITY, l = 0.f;
    bool seen = false;
    f32x4 acc[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[d] = zero4();

    const int k1 = (int)min((int64_t)part.b1 * CHUNK_KEYS, (int64_t)t.longest);
    // Pages of the halves of 16 keys, none beyond the table.
    struct Pages { int p[2]; };
    auto pages = [&](int k0) {
      Pages x;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int64_t j = ((int64_t)k0 + 16 * hf) >> a.lp;
        const int p = j < a.W ? table[j] : -1;
        x.p[hf] = p >= 0 && p < a.n_pages ? p : -1;
      }
      return x;
    };
    // A stage goes through registers: the next one is on its way while this one is used.
    constexpr int NU = 2 * SK * RU / 256;                  // 16-byte units of a thread
    V16 units[NU];
    auto fetch = [&](int k0, const Pages& pg) {
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int i = tid + 256 * u, key = i % (SK * RU) / RU, p = key < 16 ? pg.p[0] : pg.p[1];
        units[u] = zv();
        if (p >= 0 && k0 + key < t.longest)
          units[u] = ldv((u >= NU / 2 ? vc : kc) + (((size_t)p * a.Hkv + h) * P + ((k0 + key) & (P - 1))) * D + (i % RU) * 4);
      }
    };
    const int all_see = chunk_sees(a, t, t.row0);          // keys that every column sees
    Pages next{{-1, -1}};
    if (part.b0 < part.b1) {
      next = pages(part.b0 * CHUNK_KEYS);
      fetch(part.b0 * CHUNK_KEYS, next);
    }
    for (int k0 = part.b0 * CHUNK_KEYS; k0 < k1; k0 += SK) {
      const int page[2] = {next.p[0], next.p[1]};
      __syncthreads();
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int i = tid + 256 * u, key = i % (SK * RU) / RU;
        stv((u >= NU / 2 ? vs : ks) + key * LD + (i % RU) * 4, units[u]);
      }
      __syncthreads();
      if (k0 + SK < k1) {
        next = pages(k0 + SK);
        fetch(k0 + SK, next);
      }
      f32x4 s0 = zero4(), s1 = zero4();
      const int key = 8 * (n >> 2) + (n & 3);              // of K's row n in the first product; 4 more in the second
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        s0 = mma(ld(ks + key * LD + 32 * s + 8 * g), qf[s], s0);
        s1 = mma(ld(ks + (key + 4) * LD + 32 * s + 8 * g), qf[s], s1);
      }
      // lane (n, g): keys 8 g .. 8 g + 7 of column n
      float x[8];
      bool mine[8], any = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        mine[j] = k0 + 8 * g + j < len && (g < 2 ? page[0] : page[1]) >= 0;
        any = any || mine[j];
        x[j] = mine[j] ? (j < 4 ? s0[j] : s1[j - 4]) * a.scale : -INFINITY;
      }
      seen = seen || any;
      float mx = x[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) mx = fmaxf(mx, x[j]);
      mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
      mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
      const float cn = fmaxf(c, mx);
      const float f = cn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(c - cn);
      c = cn;
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d) acc[d] *= f;
      const float cs = c == -INFINITY ? 0.f : c;
      f32x8 p;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = __builtin_amdgcn_exp2f(x[j] - cs);
        l += p[j];
      }
      // A value that is not finite counts only for columns that see its key: key by key there.
      bool odd = false;
      if (k0 + SK > all_see) {
        for (int i = lane; i < SK * D; i += 64) odd |= !__builtin_isfinite(vs[(i / D) * LD + i % D]);
      }
      if (__ballot(odd) != 0ull) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              for (int k = 0; k < 4; ++k) {                // key 8 k + j
                const float w = __shfl(p[j], n + 16 * k, 64);
                if (__shfl((int)mine[j], n + 16 * k, 64)) acc[d][r] = fmaf(w, vs[(8 * k + j) * LD + 16 * d + 4 * g + r], acc[d][r]);
              }
      } else {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          f32x8 vf;
#pragma unroll
          for (int j = 0; j < 8; ++j) vf[j] = vs[(8 * g + j) * LD + 16 * d + n];
          acc[d] = mma(vf, p, acc[d]);
        }
      }
    }

    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    int some = seen;                   // of any lane of the column
    some |= __shfl_xor(some, 16, 64);
    some |= __shfl_xor(some, 32, 64);
    if (!real) continue;
    if (part.whole) {
      const size_t rq = (size_t)row * a.Hq + head;
      O* out = static_cast<O*>(a.o) + rq * D + 4 * g;
#pragma unroll
      for (int d = 0; d < DT; ++d) st4o(out + 16 * d, some ? acc[d] / l : zero4());
      if (g == 0 && a.lse != nullptr) a.lse[rq] = some ? (c + log2f(l)) * 0.6931471805599453f : -INFINITY;
    } else {
      const size_t at = ((size_t)(2 * slot + part.first) * heads + hm) * COLS32 + 16 * wave;
#pragma unroll
      for (int d = 0; d < DT; ++d) st4f(a.part_o + at * D + d * 256 + 4 * lane, acc[d]);
      if (g == 0) { a.part_ml[2 * (at + n)] = c; a.part_ml[2 * (at + n) + 1] = some ? l : -1.f; }
    }
  }
}

template <typename O, int D> hipError_t launch32(const ChunkArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((chunk32_kernel<O, D>), dim3((unsigned)(a.S * a.Hkv * a.MT)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename O, int D, int COLS, int CW> hipError_t launch_join(const ChunkArgs& a, hipStream_t s) {
  constexpr int SETS = CW * D / 256 > 16 ? 2 : 4;            // what LDS holds
  const int groups = (a.S - 1) * a.Hkv * a.MT * (COLS / CW);
  if (chunk_many_parts(a.S, a.cap)) hipLaunchKernelGGL((join_kernel<O, D, COLS, CW, SETS>), dim3(groups), dim3(256 * SETS), 0, s, a);
  else hipLaunchKernelGGL((join_kernel<O, D, COLS, CW, 1>), dim3(groups), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename O, int D> hipError_t launch_d(const ChunkArgs& a, int dtype, int o_dtype, hipStream_t s) {
  if (chunk_small(a.B, a.cap)) hipLaunchKernelGGL(plan_kernel<CHUNK_SMALL_PLAN>, dim3(1), dim3(CHUNK_SMALL_PLAN), 0, s, a);
  else hipLaunchKernelGGL(plan_kernel<1024>, dim3(1), dim3(1024), 0, s, a);
  hipError_t e = dtype == 0 ? launch32<O, D>(a, s) : launch_chunk16(a, dtype, o_dtype, D, s);
  if (e != hipSuccess || a.S == 1) return e;
  return dtype == 0 ? launch_join<O, D, COLS32, 16>(a, s) : launch_join<O, D, CHUNK16_COLS, 32>(a, s);
}

template <typename O> hipError_t launch_o(const ChunkArgs& a, int dtype, int o_dtype, int d, hipStream_t s) {
  if (d == 64) return launch_d<O, 64>(a, dtype, o_dtype, s);
  if (d == 128) return launch_d<O, 128>(a, dtype, o_dtype, s);
  return launch_d<O, 256>(a, dtype, o_dtype, s);
}

}  // namespace

int chunk_columns(int dtype) { return dtype == 0 ? COLS32 : CHUNK16_COLS; }

// Two workgroups a CU, one where its LDS holds no more (16 bits, D = 256), four
// where registers and LDS hold them (fp32, D = 64: 73 us for the prompts above, 80 with two).
int chunk_groups(int dtype, int d) { return dtype == 0 ? (d == 64 ? 1024 : 512) : d == 256 ? 256 : 512; }

// A tile of n blocks in shares of b is n / b parts for the join, which takes as
// long as b blocks do where b^2 is about this much of n.  (1/8, 1/3, 1/2: 4 rows
// over 30000 tokens, 32 / 8 heads of 128, bf16, 48, 45 and 40 us; 2 rows over 131072,
// 16 / 2 of 256, 131, 121 and 124; 16 over 4096 23.7, 23.7 and 24.4 (these with weights
// in one part, a tenth faster or less); fp32, 4 rows over 8000, 8 / 2 of 64, 32, 38 and
// 46.)
float chunk_balance(int dtype) { return dtype == 0 ? 1.f / 8 : 1.f / 3; }

hipError_t launch_chunk(const ChunkArgs& a, int dtype, int o_dtype, int d, hipStream_t s) {
  if (o_dtype == 1) return launch_o<bf16>(a, dtype, o_dtype, d, s);
  if (o_dtype == 2) return launch_o<fp16>(a, dtype, o_dtype, d, s);
  return launch_o<float>(a, dtype, o_dtype, d, s);
}

}  // namespace sgdn
