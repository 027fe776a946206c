// What the kernels of the chunk attention share.
#pragma once

#include "common.h"
#include "serve.h"

namespace sgdn {

constexpr int CHUNK_KEYS = 64;         // keys of a block
// What blocks and tiles cost, in eighths of a block of a full tile of 16-bit
// columns.  A single row's blocks are bound by memory (1960 to 2280 clocks beside
// full tiles, which take 3240; prompts of 8192 rows and steps of prompts and
// single rows, 32/8 heads of 128), a tile's beginning and end by latency.
constexpr int CHUNK_COST = 8, CHUNK_COST_SINGLE = 5, CHUNK_TILE = 4 * CHUNK_COST;
constexpr int CHUNK16_COLS = 128;      // columns of a tile, 16-bit types

__device__ __forceinline__ int chunk_blocks(int longest) { return (int)(((int64_t)longest + CHUNK_KEYS - 1) / CHUNK_KEYS); }

// Tokens that row r sees.
__device__ __forceinline__ int chunk_sees(const ChunkArgs& a, const ChunkTile& t, int r) {
  return (int)min(max(t.ahead + r + 1, (int64_t)0), (int64_t)a.max_len);
}

__device__ __forceinline__ int chunk_cost(const ChunkArgs& a, int rows) { return rows == 1 ? a.single : CHUNK_COST; }
__device__ __forceinline__ int64_t chunk_cost_all(const ChunkArgs& a, const ChunkTile& t) {
  return CHUNK_TILE + (int64_t)chunk_blocks(t.longest) * chunk_cost(a, t.rows);
}

// The share of a slot (units of cost begin .. end - 1) of tile t: blocks b0 ..
// b1 - 1, those whose first unit lies in it.  Block j begins at unit t.at +
// CHUNK_TILE + j times its cost.
struct ChunkPart { int b0, b1; bool whole, first; };

__device__ __forceinline__ ChunkPart chunk_part(const ChunkArgs& a, const ChunkTile& t, int64_t begin, int64_t end) {
  const int n = chunk_blocks(t.longest), cost = chunk_cost(a, t.rows);
  auto block = [&](int64_t unit) {     // the first that begins there or later
    const int64_t x = unit - t.at - CHUNK_TILE;
    return x <= 0 ? 0 : (int)min((x + cost - 1) / cost, (int64_t)n);
  };
  ChunkPart p;
  p.b0 = block(begin);
  p.b1 = block(end);
  p.first = begin <= t.at;             // holds the tile's first unit
  p.whole = p.first && end >= t.at + chunk_cost_all(a, t);
  return p;
}

hipError_t launch_chunk16(const ChunkArgs& a, int dtype, int o_dtype, int d, hipStream_t s);

}  // namespace sgdn
