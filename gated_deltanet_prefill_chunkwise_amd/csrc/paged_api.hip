// C ABI of the paged attention operators (declared in include/sgdn_attn.h):
// argument validation, workspace carve-up and launches.  Nothing here
// allocates device memory or synchronises.
#include <math.h>

#include "../../include/sgdn_attn.h"
#include "paged.h"

namespace {

using namespace sgdn;

constexpr size_t NO_WORKSPACE = 256;   // answer of sgdn_paged_workspace_bytes where none is used
constexpr int MAX_LIST = 4096;     // blocks of a list
constexpr int MAX_NB = 16384;      // blocks of a row that are ranked
constexpr int MAX_COUNT = 0x7fffffff - 1024;   // requests, rows of a plan: counted in steps of up to 1024

int log2_page(int page) {
  switch (page) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    default: return -1;
  }
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// A row stride: at least the row, and a multiple of 16 bytes.
bool bad_stride(int64_t ld, int64_t row, int dtype) {
  const int64_t esz = dtype == SGDN_F32 ? 4 : 2;
  return ld < row || (ld * esz) % 16 != 0 || ld > (INT64_C(1) << 40);
}

// The fields every call uses.
int check_shape(const sgdn_paged* p) {
  if (p == nullptr) return SGDN_EINVAL;
  if (p->rows < 0 || p->n_q < 1 || p->n_kv < 1 || p->d < 1 || p->page < 1 || p->n_pages < 1)
    return SGDN_EINVAL;
  if (p->dtype != SGDN_F32 && p->dtype != SGDN_BF16 && p->dtype != SGDN_F16) return SGDN_EINVAL;
  if (p->d != 64 && p->d != 128 && p->d != 256) return SGDN_EUNSUPPORTED;
  if (log2_page(p->page) < 0) return SGDN_EUNSUPPORTED;
  if (p->n_q % p->n_kv != 0) return SGDN_EUNSUPPORTED;
  if (p->n_kv > 65535) return SGDN_EUNSUPPORTED;                     // a grid dimension
  if ((int64_t)p->rows * p->n_q >= (INT64_C(1) << 28)) return SGDN_EUNSUPPORTED;
  if ((int64_t)p->n_pages * p->page >= (INT64_C(1) << 31)) return SGDN_EUNSUPPORTED;
  return SGDN_OK;
}

// ... and those of the calls that read a block table.
int check_read(const sgdn_paged* p) {
  const int st = check_shape(p);
  if (st != SGDN_OK) return st;
  if (p->batch < 1 || p->width < 1 || p->max_len < 0) return SGDN_EINVAL;
  if ((int64_t)p->width * p->page >= (INT64_C(1) << 31)) return SGDN_EUNSUPPORTED;
  if (p->max_len > p->width * p->page) return SGDN_EINVAL;
  return SGDN_OK;
}

// A launch holds fewer than 2^32 threads: `groups` workgroups, in eighths of
// the chip, of `threads`.
bool too_many(int64_t groups, int threads) { return (groups + 7) / 8 * 8 * threads >= (INT64_C(1) << 32); }

// Rows, heads and head tiles of the attention: a workgroup of 256 each.
bool too_many_units(const sgdn_paged* p) {
  return too_many((int64_t)p->rows * p->n_kv * ((p->n_q / p->n_kv + 15) / 16), 256);
}

int longest(const sgdn_paged* p) { return p->max_len > 0 ? p->max_len : p->width * p->page; }

// Rows and heads of the choice: a workgroup of up to 1024 each.
bool too_many_picks(const sgdn_paged* p) { return too_many((int64_t)p->rows * p->n_kv, 1024); }

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct AttendPlan { int S, MT, TQ; size_t off_ml, total; };

AttendPlan attend_plan(const sgdn_paged* p, int n_blocks, bool has_req) {
  AttendPlan pl;
  const int G = p->n_q / p->n_kv;
  pl.MT = (G + 15) / 16;
  const int64_t keys = n_blocks > 0 ? (int64_t)n_blocks * p->page : longest(p);
  pl.S = p->rows > 0 ? paged_splits((long long)p->rows * p->n_kv * pl.MT, (int)((keys + 31) / 32),
                                     p->d * (p->dtype == SGDN_F32 ? 4 : 2)) : 1;
  pl.off_ml = pl.total = 0;
  if (pl.S > 1) {
    const size_t parts = (size_t)p->rows * p->n_q * pl.S;
    pl.off_ml = align256(parts * p->d * sizeof(float));
    pl.total = pl.off_ml + align256(parts * 2 * sizeof(float));
  }
  pl.TQ = 0;
  if (n_blocks > 0 && pl.S == 1 && p->rows > 0)
    pl.TQ = paged_tile_rows(p->rows, p->batch, G, p->n_kv, p->d, has_req, p->dtype, log2_page(p->page), longest(p), n_blocks);
  if (pl.TQ > 0)
    pl.total = NO_WORKSPACE + align256((size_t)((p->rows + pl.TQ - 1) / pl.TQ) * p->n_kv * sizeof(int32_t));
  if (pl.total == 0) pl.total = NO_WORKSPACE;
  return pl;
}

size_t select_bytes(const sgdn_paged* p, int n_blocks) {
  const int nb = (longest(p) + p->page - 1) / p->page;
  if (nb <= n_blocks || p->rows == 0) return NO_WORKSPACE;
  return NO_WORKSPACE + align256((size_t)p->rows * p->n_kv * nb * sizeof(float));
}

int attend(const sgdn_paged* p, const void* q, int64_t ldq, const void* k_cache, const void* v_cache,
           const int32_t* table, const int32_t* row_req, const int32_t* row_len,
           const int32_t* blocks, int n_blocks, float scale, void* o, float* lse, void* ws,
           size_t ws_bytes, void* stream) {
  const int st = check_read(p);
  if (st != SGDN_OK) return st;
  if (p->o_dtype != SGDN_F32 && p->o_dtype != SGDN_BF16 && p->o_dtype != SGDN_F16) return SGDN_EINVAL;
  if (!isfinite(scale * 1.4426950408889634f)) return SGDN_EINVAL;
  if (too_many_units(p)) return SGDN_EUNSUPPORTED;
  if (p->rows == 0) return SGDN_OK;
  if (!q || !k_cache || !v_cache || !table || !row_len || !o) return SGDN_EINVAL;
  if (row_req == nullptr && p->rows > p->batch) return SGDN_EINVAL;
  if (misaligned(q) || misaligned(k_cache) || misaligned(v_cache) || misaligned(o) || misaligned(ws))
    return SGDN_EINVAL;
  if (bad_stride(ldq, (int64_t)p->n_q * p->d, p->dtype)) return SGDN_EINVAL;
  const AttendPlan pl = attend_plan(p, n_blocks, row_req != nullptr);
  if (pl.total > NO_WORKSPACE && !ws) return SGDN_EINVAL;
  if (pl.total > NO_WORKSPACE && ws_bytes < pl.total) return SGDN_EWORKSPACE;
  PageAttendArgs a;
  a.q = q; a.ldq = ldq; a.kc = k_cache; a.vc = v_cache;
  a.table = table; a.row_req = row_req; a.row_len = row_len; a.blocks = blocks;
  a.o = o; a.lse = lse;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + pl.off_ml);
  a.R = p->rows; a.B = p->batch; a.Hq = p->n_q; a.Hkv = p->n_kv; a.G = p->n_q / p->n_kv; a.MT = pl.MT;
  a.lp = log2_page(p->page); a.n_pages = p->n_pages; a.W = p->width; a.max_len = longest(p);
  a.n_blocks = n_blocks; a.S = pl.S;
  a.scale = scale * 1.4426950408889634f;
  a.TQ = pl.TQ;
  a.done = pl.TQ > 0 ? static_cast<int32_t*>(ws) : nullptr;
  if (pl.TQ > 0 && launch_paged_tiles(a, p->dtype, p->o_dtype, p->d, static_cast<hipStream_t>(stream)) != hipSuccess)
    return SGDN_EHIP;
  return launch_paged_attend(a, p->dtype, p->o_dtype, p->d, static_cast<hipStream_t>(stream)) == hipSuccess
             ? SGDN_OK : SGDN_EHIP;
}

}  // namespace

extern "C" {

int sgdn_paged_release(int32_t batch, int32_t page, int32_t width, int32_t n_free,
                       const int32_t* lens, const uint8_t* done, const int32_t* table,
                       int32_t* free_list, const int64_t* free_pos, int32_t* lens_out,
                       int64_t* free_pos_out, void* stream) {
  if (batch < 1 || page < 1 || width < 1 || n_free < 1) return SGDN_EINVAL;
  if (log2_page(page) < 0 || (int64_t)width * page >= (INT64_C(1) << 31)) return SGDN_EUNSUPPORTED;
  if (batch > MAX_COUNT) return SGDN_EUNSUPPORTED;
  if (!lens || !done || !table || !free_list || !free_pos || !lens_out || !free_pos_out)
    return SGDN_EINVAL;
  const ReleaseArgs a{batch, page, width, n_free, lens, done, table, free_list, free_pos, lens_out, free_pos_out};
  return launch_paged_release(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SGDN_OK : SGDN_EHIP;
}

int sgdn_paged_plan(int32_t batch, int32_t page, int32_t width, int32_t rows, int32_t n_free,
                    const int32_t* lens, const int32_t* add, int32_t* table,
                    const int32_t* free_list, const int64_t* free_pos, int32_t* lens_out,
                    int64_t* free_pos_out, int32_t* cu, int32_t* page_cu, int32_t* slot,
                    int32_t* row_req, int32_t* row_len, int32_t* status, void* stream) {
  if (batch < 1 || page < 1 || width < 1 || rows < 0 || n_free < 1) return SGDN_EINVAL;
  if (log2_page(page) < 0 || (int64_t)width * page >= (INT64_C(1) << 31)) return SGDN_EUNSUPPORTED;
  if (batch > MAX_COUNT || rows > MAX_COUNT) return SGDN_EUNSUPPORTED;
  if (!lens || !add || !table || !free_list || !free_pos || !lens_out || !free_pos_out || !cu ||
      !page_cu || !status)
    return SGDN_EINVAL;
  if (rows > 0 && (!slot || !row_req || !row_len)) return SGDN_EINVAL;
  const PagePlanArgs a{batch, page, width, rows, n_free, lens, add, table, free_list, free_pos,
                       lens_out, free_pos_out, cu, page_cu, slot, row_req, row_len, status};
  return launch_paged_plan(a, static_cast<hipStream_t>(stream)) == hipSuccess ? SGDN_OK : SGDN_EHIP;
}

int sgdn_paged_write(const sgdn_paged* p, const void* k, const void* v, int64_t ldk, int64_t ldv,
                     const int32_t* slot, void* k_cache, void* v_cache, int8_t* codes,
                     float* scale, void* stream) {
  const int st = check_shape(p);
  if (st != SGDN_OK) return st;
  if (((int64_t)p->rows + 15) / 16 * 256 >= (INT64_C(1) << 32)) return SGDN_EUNSUPPORTED;   // threads: 16 rows a workgroup
  if ((codes == nullptr) != (scale == nullptr)) return SGDN_EINVAL;
  if (p->rows == 0) return SGDN_OK;
  if (!k || !v || !slot || !k_cache || !v_cache) return SGDN_EINVAL;
  if (misaligned(k) || misaligned(v) || misaligned(k_cache) || misaligned(v_cache) || misaligned(codes))
    return SGDN_EINVAL;
  const int64_t row = (int64_t)p->n_kv * p->d;
  if (bad_stride(ldk, row, p->dtype) || bad_stride(ldv, row, p->dtype)) return SGDN_EINVAL;
  const PageWriteArgs a{k, v, ldk, ldv, slot, k_cache, v_cache, codes, scale,
                        p->rows, p->n_kv, p->n_pages, log2_page(p->page)};
  return launch_paged_write(a, p->dtype, p->d, static_cast<hipStream_t>(stream)) == hipSuccess ? SGDN_OK : SGDN_EHIP;
}

size_t sgdn_paged_workspace_bytes(const sgdn_paged* p, int32_t n_blocks, int32_t select) {
  if (check_read(p) != SGDN_OK || n_blocks < 0 || n_blocks > MAX_LIST) return 0;
  if (select == 0) return too_many_units(p) ? 0 : attend_plan(p, n_blocks, true).total;   // without row_req no more
  if (n_blocks < 1 || (longest(p) + p->page - 1) / p->page > MAX_NB || too_many_picks(p)) return 0;
  return select_bytes(p, n_blocks);
}

int sgdn_paged_attend(const sgdn_paged* p, const void* q, int64_t ldq, const void* k_cache,
                      const void* v_cache, const int32_t* table, const int32_t* row_req,
                      const int32_t* row_len, float scale, void* o, float* lse, void* ws,
                      size_t ws_bytes, void* stream) {
  return attend(p, q, ldq, k_cache, v_cache, table, row_req, row_len, nullptr, 0, scale, o, lse, ws,
                ws_bytes, stream);
}

int sgdn_paged_attend_sparse(const sgdn_paged* p, const void* q, int64_t ldq, const void* k_cache,
                             const void* v_cache, const int32_t* table, const int32_t* row_req,
                             const int32_t* row_len, const int32_t* blocks, int32_t n_blocks,
                             float scale, void* o, float* lse, void* ws, size_t ws_bytes,
                             void* stream) {
  if (n_blocks < 1) return SGDN_EINVAL;
  if (n_blocks > MAX_LIST) return SGDN_EUNSUPPORTED;
  if (p != nullptr && p->rows > 0 && blocks == nullptr) return SGDN_EINVAL;
  return attend(p, q, ldq, k_cache, v_cache, table, row_req, row_len, blocks, n_blocks, scale, o, lse,
                ws, ws_bytes, stream);
}

int sgdn_paged_select(const sgdn_paged* p, const void* q, int64_t ldq, const int8_t* codes,
                      const float* scale, const int32_t* table, const int32_t* row_req,
                      const int32_t* row_len, int32_t n_blocks, int32_t n_sink, int32_t n_local,
                      int32_t* blocks, void* ws, size_t ws_bytes, void* stream) {
  const int st = check_read(p);
  if (st != SGDN_OK) return st;
  if (n_blocks < 1 || n_sink < 0 || n_local < 1) return SGDN_EINVAL;
  if (n_blocks > MAX_LIST) return SGDN_EUNSUPPORTED;
  if ((int64_t)n_sink + n_local > n_blocks) return SGDN_EINVAL;
  const int nb = (longest(p) + p->page - 1) / p->page;
  if (nb > MAX_NB || too_many_picks(p)) return SGDN_EUNSUPPORTED;
  if (p->rows == 0) return SGDN_OK;
  if (!q || !codes || !scale || !table || !row_len || !blocks) return SGDN_EINVAL;
  if (row_req == nullptr && p->rows > p->batch) return SGDN_EINVAL;
  if (misaligned(q) || misaligned(codes) || misaligned(ws)) return SGDN_EINVAL;
  if (bad_stride(ldq, (int64_t)p->n_q * p->d, p->dtype)) return SGDN_EINVAL;
  const size_t need = select_bytes(p, n_blocks);
  if (need > NO_WORKSPACE && !ws) return SGDN_EINVAL;
  if (need > NO_WORKSPACE && ws_bytes < need) return SGDN_EWORKSPACE;
  const PageSelectArgs a{q, ldq, codes, scale, table, row_req, row_len, blocks, static_cast<float*>(ws),
                         p->rows, p->batch, p->n_q, p->n_kv, p->n_q / p->n_kv,
                         log2_page(p->page), p->n_pages, p->width, longest(p), nb,
                         n_blocks, n_sink, n_local};
  return launch_paged_select(a, p->dtype, p->d, static_cast<hipStream_t>(stream)) == hipSuccess ? SGDN_OK : SGDN_EHIP;
}

}  // extern "C"
