// Launch interfaces of the paged attention kernels (internal to libsgdn.so).
// Notation as in include/sgdn_attn.h: P tokens per page, W pages per table
// row, R rows (new tokens), Hq query heads in groups of G over Hkv heads.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sgdn {

struct ReleaseArgs {
  int B, P, W, F;
  const int32_t* lens;
  const uint8_t* done;
  const int32_t* table;
  int32_t* ring;
  const int64_t* pos;
  int32_t* lens_out;
  int64_t* pos_out;
};

struct PagePlanArgs {
  int B, P, W, R, F;
  const int32_t* lens;
  const int32_t* add;
  int32_t* table;
  const int32_t* ring;
  const int64_t* pos;
  int32_t* lens_out;
  int64_t* pos_out;
  int32_t* cu;
  int32_t* page_cu;
  int32_t* slot;
  int32_t* row_req;
  int32_t* row_len;
  int32_t* status;
};

struct PageWriteArgs {
  const void* k;
  const void* v;
  int64_t ldk, ldv;
  const int32_t* slot;
  void* kc;
  void* vc;
  int8_t* codes;      // NULL: no summaries
  float* scale;
  int R, Hkv, n_pages, lp;   // lp = log2 P
};

struct PageAttendArgs {
  const void* q;
  int64_t ldq;
  const void* kc;
  const void* vc;
  const int32_t* table;
  const int32_t* row_req;    // NULL: row r is request r
  const int32_t* row_len;
  const int32_t* blocks;     // NULL: every block
  void* o;
  float* lse;                // NULL: not wanted
  float* part_o;             // [R][Hq][S][D] unnormalised outputs of the splits (S > 1)
  float* part_ml;            // [R][Hq][S][2] their softmax reference and sum
  int R, B, Hq, Hkv, G, MT;  // MT = ceil(G / 16) head tiles of a group
  int lp, n_pages, W, max_len, n_blocks, S;
  float scale;               // of the scores, times log2(e)
  int32_t* done;             // [tiles][Hkv]: 1 where the tile kernel has made a tile's rows; NULL: no tiles
  int TQ;                    // rows of a tile
};

struct PageSelectArgs {
  const void* q;
  int64_t ldq;
  const int8_t* codes;
  const float* scale;
  const int32_t* table;
  const int32_t* row_req;
  const int32_t* row_len;
  int32_t* blocks;
  float* score;              // [R][Hkv][NB]
  int R, B, Hq, Hkv, G;
  int lp, n_pages, W, max_len, NB, K, n_sink, n_local;
};

// dtype: the boundary's sgdn_dtype values (0 fp32, 1 bf16, 2 fp16)
hipError_t launch_paged_release(const ReleaseArgs& a, hipStream_t s);
hipError_t launch_paged_plan(const PagePlanArgs& a, hipStream_t s);
hipError_t launch_paged_write(const PageWriteArgs& a, int dtype, int d, hipStream_t s);
// S of PageAttendArgs: `units` (row, head, head tile), `tiles` of 32 keys, bytes of a key row
int paged_splits(long long units, int tiles, int row_bytes);
hipError_t launch_paged_attend(const PageAttendArgs& a, int dtype, int o_dtype, int d, hipStream_t s);
// Rows of a tile of launch_paged_tiles, 0 where it is not used.
int paged_tile_rows(int R, int B, int G, int Hkv, int d, bool has_req, int dtype, int lp, int max_len, int n_blocks);
hipError_t launch_paged_tiles(const PageAttendArgs& a, int dtype, int o_dtype, int d, hipStream_t s);
hipError_t launch_paged_select(const PageSelectArgs& a, int dtype, int d, hipStream_t s);

}  // namespace sgdn
