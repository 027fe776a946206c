// Attention of chunks of new tokens over a paged cache (sgdn_paged_attend_chunk).
//
// For a tile of columns ((row, query head) pairs of one request and key/value
// head) the keys are walked in stages of 32.  With x = scale log2(e) K q and a
// running reference c >= max x - const per column:
//   p = 2^(x - c),  l += sum p,  A += V^T p;   c' > c: l, A *= 2^(c - c')
//   o = A / l,  lse = (c + log2 l) ln 2
#include "common.h"
#include "serve.h"

namespace sgdn {

namespace {

constexpr int SK = 32;                 // keys of a stage
constexpr int COLS = 64;               // columns of a tile, 16 a wave

// Tiles of every request, in order; then those of the rows that belong to none.
__global__ __launch_bounds__(1024) void tiles_kernel(ChunkArgs a) {
  __shared__ int first[1025], row0[1024], rows[1024], wsum[16];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
  int base = 0;
  for (int64_t b0 = 0; b0 < (int64_t)a.B + 2; b0 += 1024) {
    const int64_t b = b0 + tid;
    int r0 = 0, r1 = 0;                // B: behind the last request, B + 1: in front of the first
    if (b < a.B) { r0 = a.cu[b]; r1 = a.cu[b + 1]; }
    else if (b == a.B) { r0 = a.cu[a.B]; r1 = a.R; }
    else if (b == (int64_t)a.B + 1) { r1 = a.cu[0]; }
    r0 = min(max(r0, 0), a.R);
    r1 = min(max(r1, r0), a.R);
    const int n = (r1 - r0 + a.TR - 1) / a.TR;
    row0[tid] = r0;
    rows[tid] = r1 - r0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(sum, o, 64);
      if (lane >= o) sum += x;
    }
    if (lane == 63) wsum[wave] = sum;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < 16; ++w) { if (w < wave) before += wsum[w]; total += wsum[w]; }
    first[tid] = before + sum - n;
    if (tid == 1023) first[1024] = total;
    __syncthreads();
    for (int t = tid; t < total && base + t < a.cap; t += 1024) {
      int lo = 0, hi = 1023;           // the last request whose first tile is t or one in front
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int at = (t - first[lo]) * a.TR;
      a.tiles[base + t] = ChunkTile{row0[lo] + at, min(a.TR, rows[lo] - at), b0 + lo < a.B ? (int)(b0 + lo) : -1, 0};
    }
    base = (int)min((int64_t)base + total, (int64_t)a.cap);
    __syncthreads();
  }
  if (tid == 0) a.count[0] = base;
}

template <typename E> __device__ __forceinline__ frag_t<E> ld8s(const E* p) {   // from LDS, 16-byte aligned
  if constexpr (sizeof(E) == 2) return ld8(p);
  else return cat44(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4));
}

template <typename E, typename O, int D>
__global__ __launch_bounds__(256) void chunk_kernel(ChunkArgs a) {
  constexpr int NS = D / 32, DT = D / 16, PAD = 16 / (int)sizeof(E), LD = D + PAD;
  constexpr int RU = D * (int)sizeof(E) / 16, EV = 16 / (int)sizeof(E);     // 16-byte units of a row
  constexpr bool TWO = sizeof(E) == 2;
  constexpr float BIAS = __is_same(E, fp16) ? 10.f : 0.f;
  __shared__ __attribute__((aligned(16))) E ks[SK * LD];
  __shared__ __attribute__((aligned(16))) E vs[SK * LD];
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int heads = a.Hkv * a.MT;
  const int tile = blockIdx.x / heads, hm = blockIdx.x - tile * heads, h = hm / a.MT, mt = hm - h * a.MT;
  if (tile >= a.count[0]) return;
  const ChunkTile t = a.tiles[tile];
  const int head0 = h * a.G + mt * a.GT, gt = min(a.GT, a.G - mt * a.GT);
  const int P = 1 << a.lp;
  // this lane's column
  const int col = 16 * wave + n, my_row = col / a.GT, my_head = col - my_row * a.GT;
  const bool real = my_row < t.rows && my_head < gt;
  const int row = t.row0 + min(my_row, t.rows - 1), head = head0 + min(my_head, gt - 1);
  auto sees = [&](int r) {             // tokens that row r sees
    if (t.req < 0) return 0;
    const int64_t x = (int64_t)a.lens[t.req] - a.cu[t.req + 1] + r + 1;
    return (int)min(max(x, (int64_t)0), (int64_t)a.max_len);
  };
  const int len = real ? sees(row) : 0, longest = sees(t.row0 + t.rows - 1);
  const int32_t* table = a.table + (size_t)max(t.req, 0) * a.W;
  const E* kc = static_cast<const E*>(a.kc);
  const E* vc = static_cast<const E*>(a.vc);

  frag_t<E> qf[NS];
  {
    const E* q = static_cast<const E*>(a.q) + row * a.ldq + (size_t)head * D + 8 * g;
#pragma unroll
    for (int s = 0; s < NS; ++s) qf[s] = ld8s(q + 32 * s);
  }
  float c = -INFINITY, l = 0.f;
  bool seen = false;
  f32x4 acc[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = zero4();

  for (int k0 = 0; k0 < longest; k0 += SK) {
    // Halves of 16 keys: page of each, none beyond the table.
    int page[2];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int64_t j = ((int64_t)k0 + 16 * hf) >> a.lp;
      const int x = j < a.W ? table[j] : -1;
      page[hf] = x >= 0 && x < a.n_pages ? x : -1;
    }
    __syncthreads();
    for (int i = tid; i < 2 * SK * RU; i += 256) {
      const bool is_v = i >= SK * RU;
      const int key = i % (SK * RU) / RU, u = i % RU, pg = key < 16 ? page[0] : page[1];
      V16 x = zv();
      if (pg >= 0 && k0 + key < longest) {
        const size_t from = (((size_t)pg * a.Hkv + h) * P + ((k0 + key) & (P - 1))) * D + u * EV;
        x = ldv((is_v ? vc : kc) + from);
      }
      stv((is_v ? vs : ks) + key * LD + u * EV, x);
    }
    __syncthreads();
    f32x4 s0 = zero4(), s1 = zero4();
    const int key = 8 * (n >> 2) + (n & 3);                // of K's row n in the first product; 4 more in the second
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      s0 = mma(ld8s(ks + key * LD + 32 * s + 8 * g), qf[s], s0);
      s1 = mma(ld8s(ks + (key + 4) * LD + 32 * s + 8 * g), qf[s], s1);
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
    const float cn = fmaxf(c, mx - BIAS);
    const float f = cn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(c - cn);
    c = cn;
    l *= f;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[d] *= f;
    const float cs = c == -INFINITY ? 0.f : c;
    f32x8 p;
    frag_t<E> ph, pl;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = __builtin_amdgcn_exp2f(x[j] - cs);
      l += p[j];
      ph[j] = from_f<E>(p[j]);
      if (TWO) pl[j] = from_f<E>(p[j] - to_f(ph[j]));
    }
    // A value that is not finite counts only for columns that see its key: key by key there.
    bool odd = false;
    for (int i = tid; i < SK * D; i += 256) odd = odd || !__builtin_isfinite(to_f(vs[(i / D) * LD + i % D]));
    if (__syncthreads_or(odd)) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            for (int k = 0; k < 4; ++k) {                  // key 8 k + j
              const float w = __shfl(p[j], n + 16 * k, 64);
              if (__shfl((int)mine[j], n + 16 * k, 64)) acc[d][r] = fmaf(w, to_f(vs[(8 * k + j) * LD + 16 * d + 4 * g + r]), acc[d][r]);
            }
    } else {
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        frag_t<E> vf;
#pragma unroll
        for (int j = 0; j < 8; ++j) vf[j] = vs[(8 * g + j) * LD + 16 * d + n];
        acc[d] = mma(vf, ph, acc[d]);
        if (TWO) acc[d] = mma(vf, pl, acc[d]);
      }
    }
  }

  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  int some = seen;                     // of any lane of the column
  some |= __shfl_xor(some, 16, 64);
  some |= __shfl_xor(some, 32, 64);
  seen = some != 0;
  if (!real) return;
  const float inv = seen ? 1.f / l : 0.f;
  const size_t rq = (size_t)row * a.Hq + head;
  O* out = static_cast<O*>(a.o) + rq * D + 4 * g;
#pragma unroll
  for (int d = 0; d < DT; ++d) st4o(out + 16 * d, seen ? acc[d] * inv : zero4());
  if (g == 0 && a.lse != nullptr) a.lse[rq] = seen ? (c + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <typename E, typename O> hipError_t launch_d(const ChunkArgs& a, int d, hipStream_t s) {
  hipLaunchKernelGGL(tiles_kernel, dim3(1), dim3(1024), 0, s, a);
  const dim3 grid((unsigned)(a.cap * a.Hkv * a.MT));
  if (d == 64) hipLaunchKernelGGL((chunk_kernel<E, O, 64>), grid, dim3(256), 0, s, a);
  else if (d == 128) hipLaunchKernelGGL((chunk_kernel<E, O, 128>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((chunk_kernel<E, O, 256>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename E> hipError_t launch_o(const ChunkArgs& a, int o_dtype, int d, hipStream_t s) {
  if (o_dtype == 1) return launch_d<E, bf16>(a, d, s);
  if (o_dtype == 2) return launch_d<E, fp16>(a, d, s);
  return launch_d<E, float>(a, d, s);
}

}  // namespace

int chunk_columns(int, int) { return COLS; }

hipError_t launch_chunk(const ChunkArgs& a, int dtype, int o_dtype, int d, hipStream_t s) {
  if (dtype == 1) return launch_o<bf16>(a, o_dtype, d, s);
  if (dtype == 2) return launch_o<fp16>(a, o_dtype, d, s);
  return launch_o<float>(a, o_dtype, d, s);
}

}  // namespace sgdn
