// Block-sparse attention of many neighbouring rows (prompts): rows of one
// request that follow each other look mostly for the same blocks, so a
// workgroup takes 128 columns of (row, query head) pairs of one key/value
// head, walks the union of its rows' lists once and lets each column use the
// blocks that its row listed.  Where 16 rows list 16 blocks each and share
// most, a block is fetched once instead of a dozen times.  Rows that share
// little are better off alone: such a tile is left to the kernel for single rows.
//
// A wave owns 32 columns (16 at D = 256); both products run transposed with
// 16 x 16 x 32 matrix instructions as in paged_attend.hip.  Keys and values come in stages of 32
// keys through registers into two LDS buffers, the next stage requested before
// the products of this one; K is read from LDS row by row, V by the transposing
// read.  Both are stored with the 16-byte units (V: pairs of them) of a row
// permuted by the key's number, so that the rows that are read at once lie in
// different banks.  (Copies straight to LDS were slower: the compiler lets
// every later LDS read wait for them.)
//
// Shared lists may not change what a row sees: weights of places that a row
// does not see are exactly 0, but 0 times a value that is not finite is not.
// A tile whose result is not finite anywhere, or whose rows belong to
// different requests, is left (done = 0) as well: that kernel runs behind and
// reads for each row its own blocks only.
//
// The softmax weights enter in two parts, as in paged_attend.hip, so that a
// row errs alike whichever kernel takes it.  (One part is 241 us in the call
// below, but rounds every weight to 16 bits: 1.4 times the error of a 16-bit o.)
//
// Bound: the steps of a stage, which follow each other, and LDS, which a wave
// reads whole for its 16 or 32 columns.  3189 rows of 16 of up to 256 blocks of
// 64 keys in four requests (16/2 heads of 256, bf16): 281 us, of which 171 are
// the products at the unions' size (32 blocks in the mean, 55 at most) and 41
// would be with each row's own blocks alone and each product once.  Tried and
// slower at D = 256, when it took 272 with one part: 32 x 32 x 16 instructions
// (300), 64 columns a workgroup (285), copies straight to LDS (395); 64-key stages
// of wave pairs that share weights: 243, but 147 and not 118 at D = 128.
#include "common.h"
#include "paged.h"

namespace sgdn {

namespace {

constexpr int COLS = 128;              // of a workgroup
constexpr int SK = 32;                 // keys of a stage
// 16-column tiles of a wave.  Two read LDS half as often for a product; with
// 256 elements their accumulators do not fit the registers.
constexpr int tiles_of_wave(int d) { return d == 256 ? 1 : 2; }

// What is left alone.  A block of the union costs a tile as much as gain / 4
// blocks of single rows' lists cost the kernel for these while the chip is
// full; with fewer than `full` tiles the tiles still take as long as `full`
// would, as a tile walks its union alone.  All tiles and all single rows, 4096
// rows of 16 of 256 blocks of 64 keys, where 32, 4, 3, 2 or 1 neighbouring rows
// have one list: 32/8 heads of 128 173, 791, 1053, 1253, 1709 and 1137 to 1164
// us; 16/2 of 256 154, 353, 517, 606, 990 and 599 to 639; 32/8 of 64 619, 920,
// 1259 (4, 2, 1) and 684 to 694; 8/8 of 64 682 (1) and 679, with 16384 rows 1486
// and 2697.  256 rows where 32 have one list: 66 and 77 (32/8 of 128), 52 and 48
// (of 64), 70 and 45 (16/2 of 256; 512 rows 73 and 84).  Near the border a call of
// which some tiles are left and some are not pays for both (16/2 of 256, 2 rows
// alike, with gain 10: 1035), so 256 keeps 9, where these are all taken.
constexpr int gain_of(int d) { return d == 256 ? 9 : d == 128 ? 14 : 16; }
constexpr int full_of(int d) { return d == 256 ? 384 : 512; }
constexpr int LIST = 256;              // blocks of the union that are listed at a time (8 words of bits)

// Position of 16-byte unit c of row `key`.  An access reads the keys whose bit 2
// is the same: the other bits of the number tell their rows apart.
template <int D> __device__ __forceinline__ int k_unit(int key, int c) {
  return D == 64 ? c ^ (((key >> 1) & 1) | ((key >> 2) & 6)) : c ^ ((key & 3) | ((key >> 1) & 12));
}
template <int D> __device__ __forceinline__ int v_unit(int key, int c) {
  const int f = D == 64 ? ((key >> 1) & 1) | ((key >> 2) & 2) : (key & 3) | ((key >> 1) & 4);
  return c ^ (f << 1);
}

// lgp: log2 of a row's columns (G rounded up to a power of two).
template <typename E, typename O, int D>
__global__ __launch_bounds__(64 * (8 / tiles_of_wave(D)), 2) void tile_kernel(PageAttendArgs a, int tiles, int words, int lgp) {
  const int TQ = COLS >> lgp;          // rows of a tile
  constexpr int CT = tiles_of_wave(D), TW = COLS / 16 / CT, NT = 64 * TW;
  constexpr int NS = D / 32, DT = D / 16, KB = NS < 4 ? NS : 4;
  constexpr int BUF = 2 * SK * D;      // elements of a stage: K, then V
  constexpr int RU = D / 8;            // 16-byte units of a row
  constexpr int NU = SK * 2 * RU / NT; // of a stage, for a thread
  constexpr float BIAS = sizeof(E) == 2 && __is_same(E, fp16) ? 10.f : 0.f;   // see paged_attend.hip
  extern __shared__ __attribute__((aligned(16))) char lds[];
  E* stage = reinterpret_cast<E*>(lds);
  uint32_t* rowbits = reinterpret_cast<uint32_t*>(lds + 2 * BUF * sizeof(E));   // [TQ][words]
  uint32_t* uni = rowbits + TQ * words;                                          // [words]
  __shared__ int row_len[COLS];
  __shared__ int req_max, req_min, len_max, more, bad, n_list, n_entries;
  __shared__ int2 list[LIST];

  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  // each XCD (workgroup id mod 8) takes a run of tiles of one head after the other
  const int units = tiles * a.Hkv, per = (units + 7) >> 3;
  const int unit = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if (unit >= units || (int)(blockIdx.x >> 3) >= per) return;
  const int h = unit / tiles, tile = unit - h * tiles, row0 = tile * TQ;
  int32_t* done = a.done + (size_t)tile * a.Hkv + h;

  if (tid == 0) { req_max = -1; req_min = 0x7fffffff; len_max = 0; bad = 0; n_entries = 0; }
  lds_barrier();
  if (tid < TQ) {
    const int r = row0 + tid;
    int len = 0, req = -1;
    if (r < a.R) {
      req = a.row_req[r];
      len = min(a.row_len[r], a.max_len);
    }
    if (req < 0 || req >= a.B || len <= 0) len = 0;
    row_len[tid] = len;
    if (len > 0) { atomicMax(&req_max, req); atomicMin(&req_min, req); atomicMax(&len_max, len); }
  }
  lds_barrier();
  const int req = __builtin_amdgcn_readfirstlane(req_max);
  if (req < 0 || req != req_min) {                       // nothing to see, or several requests
    if (tid == 0) *done = 0;
    return;
  }
  const int P = 1 << a.lp, longest = __builtin_amdgcn_readfirstlane(len_max);
  const int nw = (((longest - 1) >> a.lp) >> 5) + 1;     // words in use
  const int32_t* table = a.table + (size_t)req * a.W;
  const E* kc = static_cast<const E*>(a.kc);
  const E* vc = static_cast<const E*>(a.vc);

  // this lane's columns
  int my[CT], len[CT];                                   // row of the tile, what it sees
  frag_t<E> qf[CT][NS];
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    const int col = 16 * (CT * wave + t) + n, head = col & ((1 << lgp) - 1);
    my[t] = col >> lgp;
    len[t] = row_len[my[t]];
    const E* q = static_cast<const E*>(a.q) + min(row0 + my[t], a.R - 1) * a.ldq + (size_t)(h * a.G + min(head, a.G - 1)) * D + 8 * g;
#pragma unroll
    for (int s = 0; s < NS; ++s) qf[t][s] = ld8(q + 32 * s);
  }
  // Here, once: a wait for them inside the loop would also wait for the
  // requests of the next stage, every time.
  __builtin_amdgcn_s_waitcnt(0x0F70);                    // vmcnt(0)
  // A negative scale turns the query's sign, so that the largest product is the largest score.
  // A scale of 0 goes into the query whole, as 0 times a masked score is no score.
  if (a.scale <= 0.f) {
#pragma unroll
    for (int s = 0; s < CT * NS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) qf[s / NS][s % NS][e] = a.scale == 0.f ? from_f<E>(0.f) : -qf[s / NS][s % NS][e];
  }
  const float scale = a.scale == 0.f ? 1.f : fabsf(a.scale);
  // This thread's 16-byte units tid, tid + NT, .. of a stage: K's units, then
  // V's.  A wave's share of one lies in one matrix and in 16 keys of it.
  const int u_at = tid % RU;
  float c[CT], l[CT];
  bool seen[CT];
  f32x4 acc[CT][DT];
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    c[t] = -INFINITY; l[t] = 0.f; seen[t] = false;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[t][d] = zero4();
  }

  // Entries tid, tid + NT, .. of the tile's lists that have not been taken: a
  // block that a row lists again waits for the next pass.
  const int entries = TQ * a.n_blocks;
  uint32_t pending = ~0u;
  for (int pass = 0;; ++pass) {
    for (int i = tid; i < TQ * words + words; i += NT) rowbits[i] = 0u;
    if (tid == 0) more = 0;
    lds_barrier();
    int mine = 0;                                         // valid entries of this thread
    for (int i = 0, e = tid; e < entries; ++i, e += NT) {
      if (!((pending >> i) & 1)) continue;
      const int er = e / a.n_blocks;
      bool keep = false;
      if (row0 + er < a.R && row_len[er] > 0) {
        const int j = a.blocks[((size_t)(row0 + er) * a.Hkv + h) * a.n_blocks + (e - er * a.n_blocks)];
        if (j >= 0 && j <= (row_len[er] - 1) >> a.lp) {
          const int page = table[j];
          if (page >= 0 && page < a.n_pages) {
            const uint32_t bit = 1u << (j & 31);
            keep = (atomicOr(&rowbits[er * words + (j >> 5)], bit) & bit) != 0u;
            atomicOr(&uni[j >> 5], bit);
            ++mine;
          }
        }
      }
      if (keep) more = 1; else pending &= ~(1u << i);
    }
    if (pass == 0 && mine > 0) atomicAdd(&n_entries, mine);
    lds_barrier();
    if (pass == 0) {
      int blocks = 0;                                     // of the union
      for (int i = lane; i < nw; i += 64) blocks += __builtin_popcount(uni[i]);
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) blocks += __shfl_xor(blocks, o, 64);
      if (gain_of(D) * (int64_t)__builtin_amdgcn_readfirstlane(blocks) * max(units, full_of(D)) > 4 * (int64_t)units * n_entries) {
        if (tid == 0) *done = 0;
        return;
      }
    }

    for (int w0 = 0; w0 < nw; w0 += LIST / 32) {
      // List the blocks of 8 words of the union, with their pages.
      if (tid < LIST) {
        const int w = w0 + (tid >> 5), b = tid & 31;      // a thread a block
        const uint32_t bits = w < nw ? uni[w] : 0u;
        int before = 0;                                   // blocks of the words in front
        for (int i = w0; i < w; ++i) before += __builtin_popcount(i < nw ? uni[i] : 0u);
        if ((bits >> b) & 1u) list[before + __builtin_popcount(bits & ((1u << b) - 1u))] = int2{32 * w + b, table[32 * w + b]};
        if (tid == LIST - 1) n_list = before + __builtin_popcount(bits);
      }
      lds_barrier();
      const int n_blocks = __builtin_amdgcn_readfirstlane(n_list);
      // A stage: 32 keys of one block, or two blocks at P = 16.
      const int stages = P >= SK ? n_blocks << (a.lp - 5) : (n_blocks + 1) >> 1;
      const int per_block = a.lp - 5;                     // log2 of a block's stages (P >= 32)
      // Entry of half `hf` of stage i: block and page, (-1, 0) for none.
      auto half_of = [&](int i, int hf) {
        const int e = P >= SK ? i >> per_block : 2 * i + hf;
        const int2 x = list[min(e, n_blocks - 1)];
        return e < n_blocks ? x : int2{-1, 0};
      };
      auto place = [&](int i) { return P >= SK ? (i << 5) & (P - 1) : 0; };
      auto uniform = [](int2 x) { return int2{__builtin_amdgcn_readfirstlane(x.x), __builtin_amdgcn_readfirstlane(x.y)}; };
      // How many of the first and second 16 keys of a stage the columns see,
      // from their rows' bits of the two blocks.
      int n0[CT], n1[CT];
      auto sees = [&](int i, int2 b0, int2 b1, const uint32_t (&m0)[CT], const uint32_t (&m1)[CT]) {
        const int base = (b0.x << a.lp) + place(i);
#pragma unroll
        for (int t = 0; t < CT; ++t) {
          const bool in0 = (m0[t] >> (b0.x & 31)) & 1u, in1 = P >= SK ? in0 : b1.x >= 0 && ((m1[t] >> (b1.x & 31)) & 1u);
          n0[t] = in0 ? min(max(len[t] - base, 0), 16) : 0;
          n1[t] = in1 ? min(max(len[t] - (P >= SK ? base + 16 : b1.x << a.lp), 0), 16) : 0;
        }
      };
      auto words_of = [&](int2 b0, int2 b1, uint32_t (&m0)[CT], uint32_t (&m1)[CT]) {
#pragma unroll
        for (int t = 0; t < CT; ++t) {
          m0[t] = rowbits[my[t] * words + (max(b0.x, 0) >> 5)];
          m1[t] = rowbits[my[t] * words + (max(b1.x, 0) >> 5)];
        }
      };
      V16 units_r[NU];
      auto fetch = [&](int i, int2 b0, int2 b1) {
        const size_t r0 = ((size_t)b0.y * a.Hkv + h) * P + place(i);
        const size_t r1 = P >= SK ? r0 + 16 : ((size_t)b1.y * a.Hkv + h) * P;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          const int x0 = 64 * wave + NT * u;              // of the wave
          const E* from = x0 < SK * RU ? kc : vc;
          const int key0 = x0 % (SK * RU) / RU;
          const uint32_t in_half = (uint32_t)(((x0 % (SK * RU) + lane) / RU & 15) * D + 8 * u_at);
          units_r[u] = ldv(from + (key0 < 16 ? r0 : r1) * D + in_half);
        }
      };
      // Into buffer `buf`.  Places that no row sees may hold anything: their
      // values become 0.
      auto put = [&](int i, int2 b0, int2 b1, int buf) {
        E* to = stage + buf * BUF;
        const int live0 = longest - (b0.x << a.lp) - place(i);
        const int live1 = P >= SK ? live0 - 16 : b1.x >= 0 ? longest - (b1.x << a.lp) : 0;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          const int x0 = 64 * wave + NT * u, key = (x0 % (SK * RU) + lane) / RU;
          if (x0 < SK * RU) {
            stv(to + key * D + 8 * k_unit<D>(key, u_at), units_r[u]);
          } else {
            if (min(live0, live1) < 16 && (key & 15) >= (key < 16 ? live0 : live1)) units_r[u] = zv();
            stv(to + SK * D + key * D + 8 * v_unit<D>(key, u_at), units_r[u]);
          }
        }
      };

      if (stages > 0) {
        // Entries of the stage to request (one ahead) and what the column sees
        // of this stage are at hand when it begins.
        int2 a0 = uniform(half_of(0, 0)), a1 = uniform(half_of(0, 1));
        fetch(0, a0, a1);
        put(0, a0, a1, 0);
        uint32_t m0[CT], m1[CT];
        words_of(a0, a1, m0, m1);
        sees(0, a0, a1, m0, m1);
        a0 = uniform(half_of(1, 0));
        a1 = uniform(half_of(1, 1));
        for (int i = 0; i < stages; ++i) {
        const int buf = i & 1;
        lds_barrier();                                    // this buffer is whole, the other one free
        const bool more_stages = i + 1 < stages;
        if (more_stages) fetch(i + 1, a0, a1);
        const int2 c0 = half_of(i + 2, 0), c1 = half_of(i + 2, 1);
        words_of(a0, a1, m0, m1);
        __builtin_amdgcn_sched_barrier(0);                // the requests stay in front of the products
        bool some = false, full = true;
#pragma unroll
        for (int t = 0; t < CT; ++t) {
          some = some || n0[t] + n1[t] > 0;
          full = full && n0[t] + n1[t] == 32;
          seen[t] = seen[t] || n0[t] + n1[t] > 0;
        }
        const bool all = __ballot(full) == ~0ull;
        if (__ballot(some) != 0ull) {
          const E* kb = stage + buf * BUF;
          const int key = 8 * (n >> 2) + (n & 3);         // of K's row n in the first tile; 4 more in the second
          f32x4 s0[CT], s1[CT];
#pragma unroll
          for (int t = 0; t < CT; ++t) s0[t] = s1[t] = zero4();
#pragma unroll
          for (int s = 0; s < NS; s += KB) {
            frag_t<E> kf[2 * KB];
#pragma unroll
            for (int u = 0; u < KB; ++u) {
              kf[2 * u] = ld8(kb + key * D + 8 * k_unit<D>(key, 4 * (s + u) + g));
              kf[2 * u + 1] = ld8(kb + (key + 4) * D + 8 * k_unit<D>(key + 4, 4 * (s + u) + g));
            }
            __builtin_amdgcn_sched_barrier(0);            // all reads requested before the products
#pragma unroll
            for (int u = 0; u < KB; ++u)
#pragma unroll
              for (int t = 0; t < CT; ++t) {
                s0[t] = mma(kf[2 * u], qf[t][s + u], s0[t]);
                s1[t] = mma(kf[2 * u + 1], qf[t][s + u], s1[t]);
              }
          }
          const E* vb = stage + buf * BUF + SK * D;
          const int k0 = 8 * g + (n >> 2);
          auto value = [&](int d) {                       // 16 elements: 16-byte units 2d, 2d + 1
            typedef short s16x8 __attribute__((ext_vector_type(8)));
            const E* v0 = vb + k0 * D + 8 * v_unit<D>(k0, 2 * d) + 4 * (n & 3);
            const E* v1 = vb + (k0 + 4) * D + 8 * v_unit<D>(k0 + 4, 2 * d) + 4 * (n & 3);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)v0);
            const s16x4 up = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)v1);
            const s16x8 v = __builtin_shufflevector(lo, up, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(frag_t<E>, v);
          };
          // The values' reads: all before the weights are formed where the
          // registers hold them that long (D = 128, one part: 126 -> 118 us), else two, and
          // the next two in front of the products of these (307 -> 276 us for the
          // whole call above, with weights in one part; four: 279, eight: 290).
          constexpr int VB = D < 256 ? DT : 2;
          frag_t<E> vf[2][VB];
#pragma unroll
          for (int d = 0; d < VB; ++d) vf[0][d] = value(d);
          __builtin_amdgcn_sched_barrier(0);
          frag_t<E> ph[CT], pl[CT];
#pragma unroll
          for (int t = 0; t < CT; ++t) {
            float x[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) { x[r] = s0[t][r]; x[4 + r] = s1[t][r]; }
            if (!all) {
              const int live = (g < 2 ? n0[t] : n1[t]) - 8 * (g & 1);
#pragma unroll
              for (int r = 0; r < 8; ++r)
                if (r >= live) x[r] = -INFINITY;
            }
            float mx = x[0];
#pragma unroll
            for (int r = 1; r < 8; ++r) mx = fmaxf(mx, x[r]);
            mx *= scale;                                  // scale >= 0: its sign is in q
            if (__ballot(mx > c[t] + (BIAS + 4.f)) != 0ull) {
              mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
              mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
              const float cn = fmaxf(c[t], mx - BIAS);
              const float f = cn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(c[t] - cn);
              c[t] = cn;
              l[t] *= f;
#pragma unroll
              for (int d = 0; d < DT; ++d) acc[t][d] *= f;
            }
            const float cs = c[t] == -INFINITY ? 0.f : c[t];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              const float p = __builtin_amdgcn_exp2f(fmaf(x[r], scale, -cs));
              l[t] += p;
              ph[t][r] = from_f<E>(p);
              pl[t][r] = from_f<E>(p - to_f(ph[t][r]));
            }
          }
#pragma unroll
          for (int d0 = 0; d0 < DT; d0 += VB) {
            if (d0 + VB < DT) {
#pragma unroll
              for (int d = 0; d < VB; ++d) vf[(d0 / VB + 1) & 1][d] = value(d0 + VB + d);
              __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int d = 0; d < VB; ++d)
#pragma unroll
              for (int t = 0; t < CT; ++t) {
                acc[t][d0 + d] = mma(vf[(d0 / VB) & 1][d], ph[t], acc[t][d0 + d]);
                acc[t][d0 + d] = mma(vf[(d0 / VB) & 1][d], pl[t], acc[t][d0 + d]);
              }
          }
        }
        if (more_stages) put(i + 1, a0, a1, buf ^ 1);
        sees(i + 1, a0, a1, m0, m1);
        a0 = uniform(c0);
        a1 = uniform(c1);
        }
      }
      lds_barrier();                                    // the list is free
    }
    lds_barrier();                                      // `more` is whole, the bits are free
    if (__builtin_amdgcn_readfirstlane(more) == 0) break;
    lds_barrier();
  }

#pragma unroll
  for (int t = 0; t < CT; ++t) {
    l[t] += __shfl_xor(l[t], 16, 64);
    l[t] += __shfl_xor(l[t], 32, 64);
    const float inv = seen[t] ? 1.f / l[t] : 0.f;
    const int row = row0 + my[t], head = (16 * (CT * wave + t) + n) & ((1 << lgp) - 1);
    const bool real = row < a.R && head < a.G;
    const size_t rq = (size_t)row * a.Hq + h * a.G + head;
    O* out = static_cast<O*>(a.o) + rq * D + 4 * g;
    float zero = 0.f;                                     // 0, or NaN where an output is not finite
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const f32x4 o = acc[t][d] * inv;
      zero += (o[0] * 0.f + o[1] * 0.f) + (o[2] * 0.f + o[3] * 0.f);
      if (real) st4o(out + 16 * d, o);
    }
    if (real && g == 0 && a.lse != nullptr) a.lse[rq] = seen[t] ? (c[t] + log2f(l[t])) * 0.6931471805599453f : -INFINITY;
    if (real && !(zero == 0.f)) bad = 1;
  }
  lds_barrier();
  if (tid == 0) *done = bad == 0 ? 1 : 0;
}

template <typename E, typename O, int D> hipError_t launch_tiles(const PageAttendArgs& a, int words, hipStream_t s) {
  int lgp = 0;
  while (1 << lgp < a.G) ++lgp;
  const int tiles = (a.R + a.TQ - 1) / a.TQ, units = tiles * a.Hkv;
  const size_t bytes = 2 * 2 * SK * D * sizeof(E) + (size_t)(a.TQ + 1) * words * 4;
  hipLaunchKernelGGL((tile_kernel<E, O, D>), dim3((unsigned)((units + 7) / 8 * 8)), dim3(64 * (COLS / 16 / tiles_of_wave(D))), bytes, s, a, tiles, words, lgp);
  return hipGetLastError();
}

template <typename E, typename O> hipError_t launch_d(const PageAttendArgs& a, int d, int words, hipStream_t s) {
  if (d == 64) return launch_tiles<E, O, 64>(a, words, s);
  if (d == 128) return launch_tiles<E, O, 128>(a, words, s);
  return launch_tiles<E, O, 256>(a, words, s);
}

template <typename E> hipError_t launch_o(const PageAttendArgs& a, int o_dtype, int d, int words, hipStream_t s) {
  if (o_dtype == 1) return launch_d<E, bf16>(a, d, words, s);
  if (o_dtype == 2) return launch_d<E, fp16>(a, d, words, s);
  return launch_d<E, float>(a, d, words, s);
}

}  // namespace

// Rows of a tile, or 0 where the tiles do not serve: 32-bit types, more heads
// than columns of a tile's row share, no or few rows of a request each, so few
// that tiles lose even if all rows have one list, lists and contexts beyond the
// tile's tables in LDS.  B counts the block table's rows, as the host does not
// know which of them have tokens: 1024 rows of one request take 72 us with its
// row alone for a table and 299 in a table of 512 (32/8 heads of 128).  Prompts of
// 2048 rows without tiles, of 16 of 256 blocks, 32 rows alike: fp32 1473 us (32/8
// of 128; bf16 with tiles 87), 64/2 of 128 303 (32/2: 84), 8/8 of 64 with 1024
// blocks 345 (256: 164).
int paged_tile_rows(int R, int B, int G, int Hkv, int d, bool has_req, int dtype, int lp, int max_len, int n_blocks) {
  if (dtype == 0 || G > 16 || !has_req || R < 4 * (long long)B) return 0;
  int gp = 1;
  while (gp < G) gp <<= 1;
  const int tq = COLS / gp;
  const long long words = ((((long long)max_len - 1) >> lp) >> 5) + 1;
  if (4 * (long long)R * Hkv < gain_of(d) * full_of(d) || (long long)tq * n_blocks > 32 * 256 || (tq + 1) * words * 4 > 15 * 1024) return 0;
  return tq;
}

hipError_t launch_paged_tiles(const PageAttendArgs& a, int dtype, int o_dtype, int d, hipStream_t s) {
  const int words = (((a.max_len - 1) >> a.lp) >> 5) + 1;
  return dtype == 1 ? launch_o<bf16>(a, o_dtype, d, words, s) : launch_o<fp16>(a, o_dtype, d, words, s);
}

}  // namespace sgdn
