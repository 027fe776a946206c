// What the kernels of the chunk attention share.
#pragma once

#include "common.h"
#include "serve.h"

namespace sgdn {

constexpr int CHUNK_KEYS = 64;         // keys of a unit of cost
constexpr int CHUNK_TILE = 4;          // units that a tile costs beside its keys
constexpr int CHUNK16_COLS = 128;      // columns of a tile, 16-bit types

__device__ __forceinline__ int chunk_blocks(int longest) { return (int)(((int64_t)longest + CHUNK_KEYS - 1) / CHUNK_KEYS); }

// Tokens that row r sees.
__device__ __forceinline__ int chunk_sees(const ChunkArgs& a, const ChunkTile& t, int r) {
  return (int)min(max(t.ahead + r + 1, (int64_t)0), (int64_t)a.max_len);
}

// The share of a slot (units of cost begin .. end - 1) of tile t: blocks b0 ..
// b1 - 1.  Block j is unit t.at + CHUNK_TILE + j.
struct ChunkPart { int b0, b1; bool whole, first; };

__device__ __forceinline__ ChunkPart chunk_part(const ChunkTile& t, int64_t begin, int64_t end) {
  const int n = chunk_blocks(t.longest);
  const int64_t lo = begin - t.at - CHUNK_TILE, hi = end - t.at - CHUNK_TILE;
  ChunkPart p;
  p.b0 = (int)min(max(lo, (int64_t)0), (int64_t)n);
  p.b1 = (int)min(max(hi, (int64_t)0), (int64_t)n);
  p.first = begin <= t.at;             // holds the tile's first unit
  p.whole = p.first && hi >= n;
  return p;
}

hipError_t launch_chunk16(const ChunkArgs& a, int dtype, int o_dtype, int d, hipStream_t s);

}  // namespace sgdn
