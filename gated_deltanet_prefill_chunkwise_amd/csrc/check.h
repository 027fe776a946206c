// Argument checks that the C entry points of the paged cache share.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/sgdn_attn.h"

namespace sgdn {

inline int log2_page(int page) {
  switch (page) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    default: return -1;
  }
}

inline bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// A row stride: at least the row, and a multiple of 16 bytes.
inline bool bad_stride(int64_t ld, int64_t row, int dtype) {
  const int64_t esz = dtype == SGDN_F32 ? 4 : 2;
  return ld < row || (ld * esz) % 16 != 0 || ld > (INT64_C(1) << 40);
}

// The fields every call uses.
inline int check_shape(const sgdn_paged* p) {
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
inline int check_read(const sgdn_paged* p) {
  const int st = check_shape(p);
  if (st != SGDN_OK) return st;
  if (p->batch < 1 || p->width < 1 || p->max_len < 0) return SGDN_EINVAL;
  if ((int64_t)p->width * p->page >= (INT64_C(1) << 31)) return SGDN_EUNSUPPORTED;
  if (p->max_len > p->width * p->page) return SGDN_EINVAL;
  return SGDN_OK;
}

// A launch holds fewer than 2^32 threads: `groups` workgroups, in eighths of
// the chip, of `threads`.
inline bool too_many(int64_t groups, int threads) { return (groups + 7) / 8 * 8 * threads >= (INT64_C(1) << 32); }

inline int longest(const sgdn_paged* p) { return p->max_len > 0 ? p->max_len : p->width * p->page; }

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace sgdn
