// Which kernels a call of the chunk attention launches, by its sizes (host).
// B and cap are large where their sizes are: up to 2^31 - 1 and 2^29 + 1.
#pragma once

#include <stdint.h>

namespace sgdn {

constexpr int CHUNK_SMALL_PLAN = 256;  // threads of the plan of small calls

// All requests (with the rows of none in front and behind) and tiles are a
// thread's each.
inline bool chunk_small(int B, int cap) { return (int64_t)B + 2 <= CHUNK_SMALL_PLAN && cap <= CHUNK_SMALL_PLAN; }

// Sets of waves in the join only where tiles have many parts: elsewhere nearly
// all workgroups have nothing to do, and larger ones take longer to say so.  (8
// rows over 100000 tokens, 8 / 1 heads of 128, 112 parts: 61 us, 70 with one set;
// 8 prompts of up to 2048 tokens, 16 / 16 heads of 64, up to 2: 98 us with four
// sets, 89 with one, weights then in one part.)  cap bounds the tiles from the
// sizes alone: a step of fixed size whose table has 64 requests, one of them live,
// takes the one set (those 8 rows with 120 behind them 70 us, 61 in a table of
// one request).
inline bool chunk_many_parts(int S, int cap) { return S > 8 * ((int64_t)cap - 2); }

}  // namespace sgdn
