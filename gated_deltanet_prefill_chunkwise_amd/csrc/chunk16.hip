// Attention of chunks over a paged cache, 16-bit types (plan, join and the
// formulas: chunk.hip).
//
// A workgroup takes 128 columns, 32 a wave, and walks the keys in blocks of 64
// that lie in LDS, the next block on its way while this one is used.  Both
// products run transposed with 32 x 32 x 16 matrix instructions:
//   S^T [64 keys x 32 columns] = K Q^T: lane l = 32 f + n holds, of column n and of
//     each 32 keys, keys 8 i + 4 f + j (i, j = 0 .. 3);
//   A^T [D x 32 columns] += V^T P^T: the B operand of 16 keys takes eight of a
//     lane's weights as they stand, keys 4 f + j and 8 + 4 f + j, and V^T comes
//     in that order by two transposing reads.
// So nothing crosses lanes between the products, and the running maximum, which
// moves only where a score exceeds it by a threshold, is rarely shared.
//
// Weights enter the second product in two parts, the number rounded to the type
// and what that left, itself rounded, whatever the output's type: errors as in
// paged_attend.hip.  In one part a 16-bit output errs by 1.4 times its own
// rounding (2.3e-3 of a prompt in bf16, 1.7e-3 with two).  All else is fp32.
//
// Measured, 32 / 8 heads of 128, bf16, page 64:
//   a prompt of 8192 tokens    720 to 775 us, 763 TFLOP/s (a library product of
//                              8192^3: 1240 to 1273; half as many products
//                              again are the weights' second parts)
//   4 x up to 1024 tokens over 16384 cached and 60 single rows over as many
//                              1304 to 1417 us; 2.7 GB and 694 GFLOP would each take 545
//   127 single rows over up to 8192 tokens   409 us, what reading the cache takes
// and 16 / 2 heads of 256, 512 tokens over 131072: 1571 to 1702 us, 700 TFLOP/s.
// Bound: the prompt by both pipes together.  Of the cycles the matrix units are
// busy 62 %, vector instructions issue in 55 %, any instruction in 74 %; waves wait
// 17 % of their time; the clock falls from 2.2 to 1.6 GHz as calls follow each
// other.  The fast loop is 48 products, 33 exponentials and some 430 others a
// block, without spills (D = 128; 24 registers of the rare case lie in scratch);
// no LDS bank conflicts.  Heads of 256: one wave a SIMD, matrix 50 %, vector 31 %,
// any 44 %: what a wave does follows on itself.  Prompts and single rows: 49, 42
// and 60 %, waits 33 %, and 7.4 GB read past the L2 (5.7 TB/s), where 2.7 would do;
// which of the two holds it is not settled.  Heads of 64: 31, 51 and 68 %.
// Tried, with weights in one part (the prompt; boxes differ by 7 %): 8 waves and
// 256 columns 578 us against 569, though the step of prompts and rows then reads
// 4.4 GB of HBM and not 7.3; those 8 in halves half a block apart 1057 against 906
// (prompts and rows); the scores of the next 64 keys between the weights of these
// 710 against 618, of the next 32 790 against 624 (registers).  A raised priority
// of waves that form weights: 589 -> 581 us, prompts and rows 1150 -> 1115.  Waves
// that divide the keys of single rows among them: 526 against 510 us (127 rows of
// other lengths).
#include <type_traits>

#include "chunk.h"

namespace sgdn {

namespace {

constexpr int KB = CHUNK_KEYS, COLS = CHUNK16_COLS, NW = 4;
constexpr int GROUP = 6;               // instructions behind a product (6, 8, 10: 785, 790, 793 us)

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mma32(const bf16x8& a, const bf16x8& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma32(const fp16x8& a, const fp16x8& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// Two numbers rounded to E in a word, and each of them.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <typename E> __device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef E e2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, e2));
}
// What the first of two numbers leaves of p, and the second.
template <typename E> __device__ __forceinline__ float rest_low(float p, uint32_t w) {
  if constexpr (__is_same(E, bf16)) return p - __builtin_bit_cast(float, w << 16);
  else return p - to_f(__builtin_bit_cast(fp16, (uint16_t)w));
}
template <typename E> __device__ __forceinline__ float rest_high(float p, uint32_t w) {
  if constexpr (__is_same(E, bf16)) return p - __builtin_bit_cast(float, w & 0xFFFF0000u);
  else return p - to_f(__builtin_bit_cast(fp16, (uint16_t)(w >> 16)));
}

// 16-byte units of a row are permuted by the key's number, so that rows that are
// read at once lie in different banks: unit u of key k is stored at u ^ f(k).
// K is read 16 rows at once, one unit of each; V 4 or 8 rows, 64 or 32 bytes of each.
// f's bits are bits of k, so that f(k ^ k') = f(k) ^ f(k'): an address of another
// unit or key is this one with some bits turned, and needs no register of its own.
template <int D> __device__ __forceinline__ constexpr int k_swap(int key) { return D == 64 ? (key >> 1) & 7 : key & 15; }
template <int D> __device__ __forceinline__ constexpr int v_swap(int key) {
  return D == 64 ? ((key & 2) << 1) | ((key & 4) >> 1) : ((key & 3) << 2) | ((key & 4) >> 1);
}

// 16 bytes a lane from global memory to LDS (lane l to byte 16 l from `lds`), both
// AT bytes on.  In asm, so that the compiler does not let every read of LDS wait
// for it: the kernel waits itself, before the barrier in front of the block's
// first use.
template <int AT> __device__ __forceinline__ void copy_to_lds(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 offset:%3" ::"s"(lds), "v"(offset), "s"(base), "n"(AT) : "memory", "m0");
}
// The J-th and later ones of 16 rows of keys (or values): 1 KiB each.
template <int D, bool V, int J = 0> __device__ __forceinline__ void copy_rows(const char* base, uint32_t offset, uint32_t lds) {
  constexpr int RPI = 512 / D;                       // rows of a copy
  if constexpr (J * RPI < 16) {
    copy_to_lds<(J & 3) * 1024>(base + (J >> 2) * 4096, offset ^ (16u * (V ? v_swap<D>(J * RPI) : k_swap<D>(J * RPI))), lds + (J >> 2) * 4096);
    copy_rows<D, V, J + 1>(base, offset, lds);
  }
}

template <typename E, typename O, int D>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void chunk16_kernel(ChunkArgs a) {
  constexpr int NS = D / 16, DT = D / 32;            // reduction steps of the scores, 32-element tiles of an output
  constexpr int U = D / 8;                           // 16-byte units of a row
  constexpr int TILE = KB * D;                       // elements of a block of keys
  constexpr float BIAS = __is_same(E, fp16) ? 10.f : 0.f;   // see paged_attend.hip
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  E* const vbuf = reinterpret_cast<E*>(lds) + 2 * TILE;   // two blocks of values, behind two of keys

  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, f = lane >> 5;
  const int heads = a.Hkv * a.MT;
  const int slot = blockIdx.x / heads, hm = blockIdx.x - slot * heads, h = hm / a.MT, mt = hm - h * a.MT;
  const int head0 = h * a.G + mt * a.GT, gt = min(a.GT, a.G - mt * a.GT);
  const int P = 1 << a.lp;
  const E* kc = static_cast<const E*>(a.kc);
  const E* vc = static_cast<const E*>(a.vc);

  // bytes at which this lane's parts of the first copy begin, and its reads of a block
  const uint32_t k_off = ((lane / U) * U + ((lane % U) ^ k_swap<D>(lane / U))) * 16;
  const uint32_t v_off = ((lane / U) * U + ((lane % U) ^ v_swap<D>(lane / U))) * 16;
  const int k_at = n * D * 2 + 16 * (f ^ k_swap<D>(n));
  const int m = lane & 15, v_key = 4 * f + (m >> 2);
  const int v_at = v_key * D * 2 + 16 * ((2 * ((lane >> 4) & 1) + ((m & 3) >> 1)) ^ v_swap<D>(v_key)) + 8 * (m & 1);

  const int64_t share = a.head->share, begin = slot * share, end = begin + share;
  const int tiles = a.head->tiles;
  int ti = a.start[slot];
  ChunkTile next;
  if (ti < tiles) next = a.tiles[ti];
  while (ti < tiles) {
    const ChunkTile t = next;
    if (t.at >= end) break;
    if (++ti < tiles) next = a.tiles[ti];              // here, so that it is there when it is wanted
    if (t.rows <= 0) continue;
    const ChunkPart part = chunk_part(t, begin, end);
    int len;                                           // that this lane's column sees
    const E* q;
    {                                                  // columns that are none see what their row does: they change nothing
      const int col = 32 * wave + n, my_row = col / a.GT, my_head = col - my_row * a.GT;
      const int row = t.row0 + min(my_row, t.rows - 1), head = head0 + min(my_head, gt - 1);
      len = chunk_sees(a, t, row);
      q = static_cast<const E*>(a.q) + row * a.ldq + (size_t)head * D + 8 * f;
    }
    const int len_lo = __builtin_amdgcn_readlane(len, 0), len_hi = __builtin_amdgcn_readlane(len, 31);
    const bool active = 32 * wave < t.rows * a.GT;
    const int32_t* table = a.table + (size_t)max(t.req, 0) * a.W;

    frag_t<E> qf[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) qf[s] = ld8(q + 16 * s);
    // Here, once: a wait for them inside the loop would also wait for the copies there.
    __builtin_amdgcn_s_waitcnt(0x0F70);                // vmcnt(0)
    // A negative scale turns the query's sign, so that the largest product is the largest score.
    // A scale of 0 goes into the query whole, as 0 times a masked score is no score
    // (and 0 times an element that is not finite is NaN, as the scaled score would be).
    if (a.scale <= 0.f) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) qf[s][e] = a.scale == 0.f ? from_f<E>(0.f * to_f(qf[s][e])) : -qf[s][e];
    }
    const float scale = a.scale == 0.f ? 1.f : fabsf(a.scale);
    float c = -INFINITY, l = 0.f;
    bool seen = false;
    f32x16 acc[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[d] = zero16();

    // Lane l looks up the page of 16 keys number l of the next 16 blocks, -1 for none.
    const int groups = (int)(((int64_t)t.longest + 15) >> 4);
    int pages = -1;
    auto look_up = [&](int block) {
      const int g = 4 * block + lane;
      int x = -1;
      if (g < groups) x = table[(int)(((int64_t)g << 4) >> a.lp)];
      pages = x >= 0 && x < a.n_pages ? x : -1;
    };
    // Wave w copies 16 keys number w of a block.
    auto copy = [&](int block, int buf) {
      const int g = 4 * block + wave;
      const int page = max(__builtin_amdgcn_readlane(pages, g & 63), 0);      // a place that can be read
      const size_t from = ((size_t)page * a.Hkv + h) * P + (((int64_t)g << 4) & (P - 1));
      const uint32_t to = lds0 + (uint32_t)(buf * TILE + wave * 16 * D) * 2;
      copy_rows<D, false>(reinterpret_cast<const char*>(kc + from * D), k_off, to);
      copy_rows<D, true>(reinterpret_cast<const char*>(vc + from * D), v_off, to + 2 * TILE * 2);
    };

    if (part.b0 < part.b1) {
      look_up(part.b0 & ~15);
      lds_barrier();                                   // the last tile's blocks have been read
      copy(part.b0, 0);
    }
    // which of a block's 16 keys each lie in a page
    auto valid_of = [&](int b) { return (uint32_t)(__ballot(pages >= 0) >> ((4 * b) & 63)) & 15u; };
    // A block.  PLAIN: every column sees all of it.  (Copies of their own: the
    // other case's rare branch costs the registers of the products 128 moves.)
    auto step = [&](int b, uint32_t valid, auto PLAIN) {
      // What the rare case needs is formed there: kept from block to block it
      // would cost registers (and, spilled, waits for the copies).
      int lane = lane_id();
      if (!PLAIN) asm volatile("" : "+v"(lane));
      const int n = lane & 31, f = lane >> 5;
      const int buf = (b - part.b0) & 1;
      __builtin_amdgcn_s_waitcnt(0x0F70);              // vmcnt(0)
      lds_barrier();                                   // this block is whole, the other buffer free
      if (b + 1 < part.b1) {
        if (((b + 1) & 15) == 0) look_up(b + 1);
        copy(b + 1, buf ^ 1);
      }
      const int key0 = b * KB;
      // Places behind the last token and pages that are none may hold anything.
      if (!PLAIN && (valid != 15u || key0 + KB > t.longest)) {
        for (int i = tid; i < TILE / 8; i += 64 * NW) {
          const int key = i / U;
          if (!((valid >> (key >> 4)) & 1u) || key0 + key >= t.longest) stv(vbuf + buf * TILE + 8 * i, zv());
        }
        lds_barrier();
      }
      if (!active || (!PLAIN && key0 >= len_hi)) return;
      const bool full = PLAIN || (valid == 15u && key0 + KB <= len_lo);

      f32x16 s[2];
      s[0] = zero16();
      s[1] = zero16();
      int k_from = k_at + buf * TILE * 2, v_from = v_at + (2 + buf) * TILE * 2;
      asm volatile("" : "+v"(k_from), "+v"(v_from));   // formed anew for every block: their registers are few
      constexpr int KS = NS < 4 ? NS : 4;              // steps whose keys are read at once
      frag_t<E> kf[2][2 * KS];
      auto keys = [&](int i0) {
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          const E* k = reinterpret_cast<const E*>(lds + (k_from ^ (32 * (i0 + i))));
          kf[(i0 / KS) & 1][2 * i] = ld8(k);
          kf[(i0 / KS) & 1][2 * i + 1] = ld8(k + 32 * D);
        }
      };
      __builtin_amdgcn_s_setprio(0);
      keys(0);
#pragma unroll
      for (int i0 = 0; i0 < NS; i0 += KS) {
        if (i0 + KS < NS) keys(i0 + KS);
        __builtin_amdgcn_sched_barrier(0);             // the reads are requested in front of the products
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          s[0] = mma32(kf[(i0 / KS) & 1][2 * i], qf[i0 + i], s[0]);
          s[1] = mma32(kf[(i0 / KS) & 1][2 * i + 1], qf[i0 + i], s[1]);
        }
      }
      auto value = [&](int i, int d) {                 // V^T of 16 keys and 32 elements
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const E* p = reinterpret_cast<const E*>(lds + (v_from ^ (64 * (d & 3)))) + (d >> 2) * 128 + 16 * i * D;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
        const s16x4 up = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 8 * D));
        const s16x8 v = __builtin_shufflevector(lo, up, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(frag_t<E>, v);
      };
      frag_t<E> vf[2][DT];
#pragma unroll
      for (int d = 0; d < DT; ++d) vf[0][d] = value(0, d);
      __builtin_amdgcn_sched_barrier(0);
      // Of 16 keys number g this lane's column sees key 8 i + 4 f + j (i = 0, 1) where 8 i + j < left(g).
      auto left = [&](int g) { return (valid >> g) & 1u ? len - key0 - 16 * g - 4 * f : 0; };
      if (!full) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int x = left(g);
          seen = seen || x > 0;
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (8 * (r >> 2) + (r & 3) >= x) s[g >> 1][8 * (g & 1) + r] = -INFINITY;
        }
      } else {
        seen = true;
      }
      __builtin_amdgcn_s_setprio(1);                   // a wave that forms weights goes first: products of others hide behind it
      float mx = s[0][0];
#pragma unroll
      for (int r = 1; r < 16; ++r) mx = fmaxf(mx, s[0][r]);
#pragma unroll
      for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[1][r]);
      mx *= scale;                                     // its sign is in q
      if (__ballot(mx > c + (BIAS + 4.f)) != 0ull) {
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float cn = fmaxf(c, mx - BIAS);
        const float g = cn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(c - cn);
        c = cn;
        l *= g;
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[d] *= g;
      }
      const float cs = c == -INFINITY ? 0.f : c;
      const E* vb = vbuf + buf * TILE;
      uint32_t odd = 0u;                               // a value that is not finite, where some column does not see all
      if (!full) {
        for (int i = 0; i < TILE / 8; i += 64) {
          const V16 x = ldv(vb + 8 * (i + lane));
          const uint32_t e = __is_same(E, fp16) ? 0x7C007C00u : 0x7F807F80u, one = __is_same(E, fp16) ? 0x04000400u : 0x00800080u;
#pragma unroll
          for (int w = 0; w < 4; ++w) odd |= ((x.w[w] & e) + one) & 0x80008000u;
        }
      }
      auto weight = [&](int i, int r) { return __builtin_amdgcn_exp2f(fmaf(s[i >> 1][8 * (i & 1) + r], scale, -cs)); };
      if (!PLAIN && __ballot(odd != 0u) != 0ull) {
        // Such values count only for the columns that see their keys (0 times
        // them would be NaN): key by key, the weights by way of LDS.
        float* w = reinterpret_cast<float*>(lds + 4 * TILE * sizeof(E)) + wave * 16 * 32;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          int x = left(i);
          asm volatile("" : "+v"(x));                  // compared anew: 32 masks do not fit the registers
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const float p = weight(i, r);
            l += p;
            w[(8 * (r >> 2) + 4 * f + (r & 3)) * 32 + n] = 8 * (r >> 2) + (r & 3) < x ? p : -1.f;
          }
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
          __builtin_amdgcn_wave_barrier();
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll 1
          for (int k = 0; k < 16; ++k) {
            const float p = w[k * 32 + n];
            const bool sees = !(p < 0.f);
            const int key = 16 * i + k;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
              for (int r = 0; r < 16; r += 4) {
                const f32x4 v = ld4f(vb + key * D + 8 * ((4 * d + (r >> 2)) ^ v_swap<D>(key)) + 4 * f);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[d][r + j] = sees ? fmaf(p, v[j], acc[d][r + j]) : acc[d][r + j];
                asm volatile("" ::: "memory");               // not all values at once
              }
          }
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
          __builtin_amdgcn_wave_barrier();
        }
        return;
      }
      // The weights of 16 keys are formed while those of the 16 before are multiplied.
      frag_t<E> ph[2], pl[2];
      auto weights = [&](int i) {
        u32x4 hi, lo;
#pragma unroll
        for (int r = 0; r < 8; r += 2) {
          const float p0 = weight(i, r), p1 = weight(i, r + 1);
          l += p0 + p1;
          hi[r >> 1] = pack2<E>(p0, p1);
          lo[r >> 1] = pack2<E>(rest_low<E>(p0, hi[r >> 1]), rest_high<E>(p1, hi[r >> 1]));
        }
        ph[i & 1] = __builtin_bit_cast(frag_t<E>, hi);
        pl[i & 1] = __builtin_bit_cast(frag_t<E>, lo);
      };
      weights(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < 3) {
#pragma unroll
          for (int d = 0; d < DT; ++d) vf[(i + 1) & 1][d] = value(i + 1, d);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[d] = mma32(vf[i & 1][d], ph[i & 1], acc[d]);
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[d] = mma32(vf[i & 1][d], pl[i & 1], acc[d]);
        if (i < 3) {
          weights(i + 1);
#pragma unroll
          for (int m = 0; m < 2 * DT; ++m) {       // a product, then as many others as hide behind it
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x402, GROUP, 0);
          }
        }
      }
    };
    const int plain = min(part.b1, chunk_sees(a, t, t.row0) / KB);
    for (int b = part.b0; b < part.b1; ++b) {
      uint32_t valid = valid_of(b);
      for (; b < plain && valid == 15u; valid = valid_of(++b)) step(b, valid, std::true_type{});
      if (b < part.b1) step(b, valid, std::false_type{});
    }

    l += __shfl_xor(l, 32, 64);
    int some = seen;
    some |= __shfl_xor(some, 32, 64);
    int lane = lane_id();
    asm volatile("" : "+v"(lane));                     // as in the rare case above
    const int n = lane & 31, f = lane >> 5;
    if (part.whole) {
      // By way of LDS, so that a wave writes whole rows: 16-byte unit u of column k at u ^ k.
      constexpr int OU = D * (int)sizeof(O) / 16, SWAP = OU < 16 ? OU - 1 : 15;
      char* mine = lds + wave * 32 * D * (int)sizeof(O);
      const float inv = some ? 1.f / l : 0.f;
      lds_barrier();                                   // all waves are done with the last block
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const int at = (32 * d + 2 * r + 4 * f) * (int)sizeof(O);
          st4o(reinterpret_cast<O*>(mine + n * D * (int)sizeof(O) + ((at >> 4) ^ (n & SWAP)) * 16 + (at & 15)),
               f32x4{acc[d][r] * inv, acc[d][r + 1] * inv, acc[d][r + 2] * inv, acc[d][r + 3] * inv});
        }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      auto place = [&](int k) {                        // of the wave's column k among the call's rows and heads, -1 for none
        const int col = 32 * wave + k, my_row = col / a.GT, my_head = col - my_row * a.GT;
        return my_row < t.rows && my_head < gt ? (int64_t)(t.row0 + my_row) * a.Hq + head0 + my_head : (int64_t)-1;
      };
      for (int i = lane; i < 32 * OU; i += 64) {
        const int k = i / OU, u = i % OU;
        const int64_t rq = place(k);
        if (rq >= 0) stv(static_cast<char*>(a.o) + (rq * OU + u) * 16, ldv(mine + (k * OU + (u ^ (k & SWAP))) * 16));
      }
      if (f == 0 && a.lse != nullptr) {
        const int64_t rq = place(n);
        if (rq >= 0) a.lse[rq] = some ? (c + log2f(l)) * 0.6931471805599453f : -INFINITY;
      }
    } else {
      // Parts as they lie in the registers: the join reads them so.
      const size_t at = ((size_t)(2 * slot + part.first) * heads + hm) * COLS + 32 * wave;
      if (active) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int r = 0; r < 16; r += 4)
            st4f(a.part_o + at * D + (4 * d + (r >> 2)) * 256 + 4 * lane, f32x4{acc[d][r], acc[d][r + 1], acc[d][r + 2], acc[d][r + 3]});
        if (f == 0) { a.part_ml[2 * (at + n)] = c; a.part_ml[2 * (at + n) + 1] = some ? l : -1.f; }
      }
    }
  }
}

template <typename E, typename O, int D> hipError_t launch_d(const ChunkArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((chunk16_kernel<E, O, D>), dim3((unsigned)(a.S * a.Hkv * a.MT)), dim3(64 * NW), 4 * KB * D * sizeof(E) + NW * 16 * 32 * sizeof(float), s, a);
  return hipGetLastError();
}

template <typename E, typename O> hipError_t launch_o(const ChunkArgs& a, int d, hipStream_t s) {
  if (d == 64) return launch_d<E, O, 64>(a, s);
  if (d == 128) return launch_d<E, O, 128>(a, s);
  return launch_d<E, O, 256>(a, s);
}

template <typename E> hipError_t launch_e(const ChunkArgs& a, int o_dtype, int d, hipStream_t s) {
  if (o_dtype == 1) return launch_o<E, bf16>(a, d, s);
  if (o_dtype == 2) return launch_o<E, fp16>(a, d, s);
  return launch_o<E, float>(a, d, s);
}

}  // namespace

hipError_t launch_chunk16(const ChunkArgs& a, int dtype, int o_dtype, int d, hipStream_t s) {
  return dtype == 1 ? launch_e<bf16>(a, o_dtype, d, s) : launch_e<fp16>(a, o_dtype, d, s);
}

}  // namespace sgdn
