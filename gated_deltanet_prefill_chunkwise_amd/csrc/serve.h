// Launch interfaces of the kernels around the paged cache (internal to
// libsgdn.so).  Notation as in include/sgdn_serve.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sgdn {

struct HeadsArg { const void* in; void* out; int64_t in_row, in_head, out_row, out_head; };

struct RopeArgs {
  HeadsArg q, k;
  int R, Hq, Hk, D, rot;
  const int32_t* pos;
  int pos_offset;
  const double* freqs;
  float magnitude;
  const void* wq;            // NULL: zeros
  const void* wk;
  float w_offset, eps;
  int slices;                // of a row's heads, a wave each
};

// A tile of the chunk attention: rows row0 .. row0 + rows - 1 of request req
// (-1: of none).  Row r sees ahead + r + 1 tokens, the last row `longest`.  The
// tiles' costs (CHUNK_TILE units and one for each 64 keys) stand in a row; `at` is
// where this one's begin.
struct ChunkTile { int32_t row0, rows, req, longest; int64_t at, ahead; };

// What the plan finds: tiles, and the units of cost that a slot takes.
struct ChunkHead { int64_t share; int32_t tiles; int32_t pad; };

struct ChunkArgs {
  const void* q;
  int64_t ldq;
  const void* kc;
  const void* vc;
  const int32_t* table;
  const int32_t* cu;
  const int32_t* lens;
  void* o;
  float* lse;                // NULL: not wanted
  ChunkHead* head;           // [1]
  ChunkTile* tiles;          // [cap]
  int32_t* start;            // [S] the tile that a slot's first unit of cost lies in
  float* part_o;             // [2 S][heads][columns][D] unnormalised outputs of parts of tiles
  float* part_ml;            // [2 S][heads][columns][2] their softmax reference and sum (-1: nothing seen)
  int R, B, Hq, Hkv, G, lp, n_pages, W, max_len;
  int TR, GT, MT;            // rows of a tile, query heads of one, head tiles of a group
  int cap;                   // tiles at most
  int S;                     // slots: workgroups of each head tile
  float balance;             // a share's square at least, of the longest tile's units
  float scale;               // of the scores, times log2(e)
};

// dtype: the boundary's sgdn_dtype values (0 fp32, 1 bf16, 2 fp16)
int rope_slices(int R, int Hq, int Hk, int d, int dtype);
hipError_t launch_rope(const RopeArgs& a, int dtype, int w_dtype, bool norm, bool interleaved, hipStream_t s);

// Columns ((row, query head) pairs of one key/value head) of a tile, and the
// workgroups that fill the chip.
int chunk_columns(int dtype);
int chunk_groups(int dtype, int d);
float chunk_balance(int dtype);
hipError_t launch_chunk(const ChunkArgs& a, int dtype, int o_dtype, int d, hipStream_t s);

}  // namespace sgdn
