// C ABI of the operators around the paged cache (declared in
// include/sgdn_serve.h): argument validation, workspace carve-up and launches.
// Nothing here allocates device memory or synchronises.
#include <math.h>

#include "../../include/sgdn_serve.h"
#include "check.h"
#include "serve.h"

namespace {

using namespace sgdn;

bool known(int dtype) { return dtype == SGDN_F32 || dtype == SGDN_BF16 || dtype == SGDN_F16; }

int check_rope(const sgdn_rope_shape* p) {
  if (p == nullptr) return SGDN_EINVAL;
  if (p->rows < 0 || p->n_q < 0 || p->n_k < 0 || p->d < 1 || p->rot < 0) return SGDN_EINVAL;
  if (!known(p->dtype)) return SGDN_EINVAL;
  if (p->layout != SGDN_ROPE_HALF && p->layout != SGDN_ROPE_INTERLEAVED) return SGDN_EINVAL;
  if (p->rot > p->d) return SGDN_EINVAL;
  const int unit = p->dtype == SGDN_F32 ? 4 : 8;
  if (p->d > 256 || p->d % unit != 0 || p->rot % 2 != 0) return SGDN_EUNSUPPORTED;
  if ((int64_t)p->n_q + p->n_k >= 1 << 16) return SGDN_EUNSUPPORTED;
  if (p->rows >= (1 << 26) - 3) return SGDN_EUNSUPPORTED;            // a wave a row, 2^32 threads a launch
  return SGDN_OK;
}

// Heads [rows, n, d]: given wherever there are any, aligned, and without overlap:
// heads inside of rows, or rows inside of heads.
bool bad_heads(const void* x, const sgdn_strides& s, int n, const sgdn_rope_shape* p) {
  if (n == 0) return false;
  if (x == nullptr || misaligned(x)) return true;
  const int64_t unit = p->dtype == SGDN_F32 ? 4 : 8, far = INT64_C(1) << 36;
  const bool rows = p->rows > 1, heads = n > 1;
  if (rows && (s.row < p->d || s.row > far || s.row % unit != 0)) return true;
  if (heads && (s.head < p->d || s.head > far || s.head % unit != 0)) return true;
  return rows && heads && s.row < (n - 1) * s.head + p->d && s.head < (p->rows - 1) * s.row + p->d;
}

int rope(const sgdn_rope_shape* p, const void* q, const void* k, bool norm, const void* wq, const void* wk,
         float w_offset, float eps, const int32_t* pos, int32_t pos_offset, const double* freqs,
         double magnitude, void* q_out, void* k_out, void* stream) {
  const int st = check_rope(p);
  if (st != SGDN_OK) return st;
  if (!isfinite((float)magnitude)) return SGDN_EINVAL;
  if (norm && (!known(p->w_dtype) || !isfinite(w_offset) || !(eps >= 0.f) || !isfinite(eps))) return SGDN_EINVAL;
  if (p->rows == 0 || p->n_q + p->n_k == 0) return SGDN_OK;
  if (!pos || (p->rot > 0 && !freqs) || misaligned(wq) || misaligned(wk)) return SGDN_EINVAL;
  if (reinterpret_cast<uintptr_t>(freqs) & 7) return SGDN_EINVAL;
  if (bad_heads(q, p->q, p->n_q, p) || bad_heads(k, p->k, p->n_k, p) || bad_heads(q_out, p->q_out, p->n_q, p) ||
      bad_heads(k_out, p->k_out, p->n_k, p))
    return SGDN_EINVAL;
  // in place: the same rows and heads
  auto moved = [p](const void* in, const void* out, int n, const sgdn_strides& i, const sgdn_strides& o) {
    return n > 0 && in == out && ((p->rows > 1 && i.row != o.row) || (n > 1 && i.head != o.head));
  };
  if (moved(q, q_out, p->n_q, p->q, p->q_out) || moved(k, k_out, p->n_k, p->k, p->k_out)) return SGDN_EINVAL;
  RopeArgs a;
  // strides of a single row or head: no distance, and no overflow either
  auto side = [p](const void* in, void* out, int n, const sgdn_strides& i, const sgdn_strides& o) {
    const int64_t rows = p->rows > 1, heads = n > 1;
    return HeadsArg{in, out, rows * i.row, heads * i.head, rows * o.row, heads * o.head};
  };
  a.q = side(q, q_out, p->n_q, p->q, p->q_out);
  a.k = side(k, k_out, p->n_k, p->k, p->k_out);
  a.R = p->rows; a.Hq = p->n_q; a.Hk = p->n_k; a.D = p->d; a.rot = p->rot;
  a.pos = pos; a.pos_offset = pos_offset; a.freqs = freqs; a.magnitude = (float)magnitude;
  a.wq = wq; a.wk = wk; a.w_offset = w_offset; a.eps = eps;
  a.slices = rope_slices(p->rows, p->n_q, p->n_k, p->d, p->dtype);
  return launch_rope(a, p->dtype, p->w_dtype, norm, p->layout == SGDN_ROPE_INTERLEAVED, static_cast<hipStream_t>(stream)) == hipSuccess
             ? SGDN_OK : SGDN_EHIP;
}

struct ChunkPlan { int cap, TR, GT, MT, S; size_t off_tiles, off_start, off_o, off_ml, total; };

// False where the end of a block of keys would pass 32 bits.
bool chunk_plan(const sgdn_paged* p, ChunkPlan* pl) {
  const int cols = chunk_columns(p->dtype), G = p->n_q / p->n_kv;
  pl->GT = G < cols ? G : cols;
  pl->MT = (G + pl->GT - 1) / pl->GT;
  pl->TR = cols / pl->GT;
  // each request has one tile that is not full, and so have the rows of none (in
  // front and behind); rows < 2^28, so that there are under 2^29 + 2
  const int64_t cap = ((int64_t)p->rows + pl->TR - 1) / pl->TR + (p->batch < p->rows ? p->batch : p->rows) + 2;
  const int64_t heads = (int64_t)p->n_kv * pl->MT, groups = chunk_groups(p->dtype, p->d);
  if (longest(p) > INT32_MAX - 127) return false;
  pl->cap = (int)cap;
  pl->S = (int)(groups > heads ? groups / heads : 1);
  const size_t parts = 2 * (size_t)pl->S * heads * cols;
  pl->off_tiles = 256;
  pl->off_start = pl->off_tiles + align256((size_t)cap * sizeof(ChunkTile));
  pl->off_o = pl->off_start + align256((size_t)pl->S * sizeof(int32_t));
  pl->off_ml = pl->off_o + (pl->S > 1 ? align256(parts * p->d * sizeof(float)) : 0);
  pl->total = pl->off_ml + (pl->S > 1 ? align256(parts * 2 * sizeof(float)) : 0);
  return true;
}

}  // namespace

extern "C" {

int sgdn_rope_freqs(int32_t rot, int32_t scaling, double base, double factor, double original,
                    double low, double high, double* freqs, double* magnitude) {
  if (rot < 2 || rot > 256 || rot % 2 != 0 || !freqs || !magnitude) return SGDN_EINVAL;
  if (scaling < SGDN_ROPE_PLAIN || scaling > SGDN_ROPE_BY_TURNS) return SGDN_EINVAL;
  if (!(base > 1.0) || !isfinite(base)) return SGDN_EINVAL;
  if (scaling != SGDN_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return SGDN_EINVAL;
  if (scaling == SGDN_ROPE_BASE && rot < 4) return SGDN_EINVAL;
  const double two_pi = 6.283185307179586476925;
  const bool ramped = scaling == SGDN_ROPE_BY_PAIR || scaling == SGDN_ROPE_BY_TURNS;
  if (ramped && (!(original > 0.0) || !isfinite(original) || !(low > 0.0) || !(high > low) || !isfinite(high)))
    return SGDN_EINVAL;
  double a = 0.0, b = 0.0;
  if (scaling == SGDN_ROPE_BY_PAIR) {
    a = fmax(floor(rot * log(original / (high * two_pi)) / (2.0 * log(base))), 0.0);
    b = fmin(ceil(rot * log(original / (low * two_pi)) / (2.0 * log(base))), rot - 1.0);
    if (a == b) b += 0.001;
  }
  if (scaling == SGDN_ROPE_BASE) base *= pow(factor, rot / (rot - 2.0));
  *magnitude = scaling == SGDN_ROPE_BY_PAIR && factor > 1.0 ? 1.0 + 0.1 * log(factor) : 1.0;
  for (int i = 0; i < rot / 2; ++i) {
    const double f = pow(base, -2.0 * i / rot);
    double keep = 1.0;                     // the part that is not slowed
    if (scaling == SGDN_ROPE_LINEAR) keep = 0.0;
    if (scaling == SGDN_ROPE_BY_PAIR) keep = 1.0 - fmin(fmax((i - a) / (b - a), 0.0), 1.0);
    if (scaling == SGDN_ROPE_BY_TURNS) keep = fmin(fmax((f * original / two_pi - low) / (high - low), 0.0), 1.0);
    freqs[i] = keep == 1.0 ? f : f * keep + f * (1.0 - keep) / factor;
  }
  return SGDN_OK;
}

int sgdn_rope(const sgdn_rope_shape* p, const void* q, const void* k, const int32_t* pos,
              int32_t pos_offset, const double* freqs, double magnitude, void* q_out, void* k_out,
              void* stream) {
  return rope(p, q, k, false, nullptr, nullptr, 0.f, 0.f, pos, pos_offset, freqs, magnitude, q_out, k_out, stream);
}

int sgdn_norm_rope(const sgdn_rope_shape* p, const void* q, const void* k, const void* wq,
                   const void* wk, float w_offset, float eps, const int32_t* pos,
                   int32_t pos_offset, const double* freqs, double magnitude, void* q_out,
                   void* k_out, void* stream) {
  return rope(p, q, k, true, wq, wk, w_offset, eps, pos, pos_offset, freqs, magnitude, q_out, k_out, stream);
}

size_t sgdn_paged_chunk_workspace_bytes(const sgdn_paged* p) {
  ChunkPlan pl;
  return check_read(p) == SGDN_OK && chunk_plan(p, &pl) ? pl.total : 0;
}

int sgdn_paged_attend_chunk(const sgdn_paged* p, const void* q, int64_t ldq, const void* k_cache,
                            const void* v_cache, const int32_t* table, const int32_t* cu,
                            const int32_t* lens, float scale, void* o, float* lse, void* ws,
                            size_t ws_bytes, void* stream) {
  const int st = check_read(p);
  if (st != SGDN_OK) return st;
  if (!known(p->o_dtype)) return SGDN_EINVAL;
  if (!isfinite(scale * 1.4426950408889634f)) return SGDN_EINVAL;
  ChunkPlan pl;
  if (!chunk_plan(p, &pl)) return SGDN_EUNSUPPORTED;
  if (p->rows == 0) return SGDN_OK;
  if (!q || !k_cache || !v_cache || !table || !cu || !lens || !o || !ws) return SGDN_EINVAL;
  if (misaligned(q) || misaligned(k_cache) || misaligned(v_cache) || misaligned(o) || misaligned(ws))
    return SGDN_EINVAL;
  if (bad_stride(ldq, (int64_t)p->n_q * p->d, p->dtype)) return SGDN_EINVAL;
  if (ws_bytes < pl.total) return SGDN_EWORKSPACE;
  ChunkArgs a;
  a.q = q; a.ldq = ldq; a.kc = k_cache; a.vc = v_cache;
  a.table = table; a.cu = cu; a.lens = lens; a.o = o; a.lse = lse;
  char* w = static_cast<char*>(ws);
  a.head = reinterpret_cast<ChunkHead*>(w);
  a.tiles = reinterpret_cast<ChunkTile*>(w + pl.off_tiles);
  a.start = reinterpret_cast<int32_t*>(w + pl.off_start);
  a.part_o = reinterpret_cast<float*>(w + pl.off_o);
  a.part_ml = reinterpret_cast<float*>(w + pl.off_ml);
  a.R = p->rows; a.B = p->batch; a.Hq = p->n_q; a.Hkv = p->n_kv; a.G = p->n_q / p->n_kv;
  a.lp = log2_page(p->page); a.n_pages = p->n_pages; a.W = p->width; a.max_len = longest(p);
  a.TR = pl.TR; a.GT = pl.GT; a.MT = pl.MT; a.cap = pl.cap; a.S = pl.S;
  a.balance = chunk_balance(p->dtype);
  a.scale = scale * 1.4426950408889634f;
  return launch_chunk(a, p->dtype, p->o_dtype, p->d, static_cast<hipStream_t>(stream)) == hipSuccess
             ? SGDN_OK : SGDN_EHIP;
}

}  // extern "C"
