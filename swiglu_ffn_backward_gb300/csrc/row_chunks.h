// Chunks of rows whose column sums are taken together, in the backward of the norms between blocks: the plan, and the rows
// of a chunk (host arithmetic, and the same on the device).
#pragma once

#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#ifdef __CUDACC__
#define SWG_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SWG_HOST_DEVICE inline
#endif

namespace swg {

struct BnChunks {
  int64_t segment;      // rows of a gate row, or all
  int64_t rows;         // of a chunk, at most
  int64_t apart;        // distance of a chunk's rows
  int64_t phases;       // runs of such rows in a segment: apart, or as many as it has rows
  int64_t per_segment;  // chunks
  int64_t chunks;
};

// Rows first, first + apart, ... below end of segment `segment`. A chunk may have none (first >= end), and its first row
// then lies in another segment, or behind the last row of all. The gate row of a chunk is its segment.
template <typename Int>
struct ChunkRows {
  Int segment, first, end;
};
// chunk c of all: chunk i of a segment has the rows (i % phases) + apart (i / phases rows + 0, 1, ...) of it. kApart: the
// plan's apart is not 1. Int: 32 bits hold every row and chunk.
template <bool kApart, typename Int>
SWG_HOST_DEVICE ChunkRows<Int> chunk_rows(const BnChunks& k, Int c) {
  const Int per = static_cast<Int>(k.per_segment), segment = static_cast<Int>(k.segment);
  const Int phases = kApart ? static_cast<Int>(k.phases) : 1;
  ChunkRows<Int> w;
  w.segment = c / per;
  const Int in = c - w.segment * per, block = kApart ? in / phases : in, phase = in - block * phases;
  const Int rows = static_cast<Int>(k.rows) * (kApart ? static_cast<Int>(k.apart) : 1), last = (w.segment + 1) * segment;
  w.first = w.segment * segment + phase + block * rows;
  w.end = w.first + rows < last ? w.first + rows : last;
  return w;
}

// Chunks of one gate row where the gate has fewer rows than M, of at most 128 rows (like terms are rounded the same way,
// and a longer chain drifts), and such that `units` groups that take them in turn have nearly equal work: rows, and for
// each chunk the writing of its sums, about one row's. Segments of fewer rows than `apart` have one chunk a row.
constexpr int64_t kMostRows = 128;
inline BnChunks chunks_of(int64_t M, int64_t rows_per_gate, int64_t units, int64_t apart) {
  BnChunks k;
  k.segment = rows_per_gate > 1 ? rows_per_gate : M;
  k.apart = apart;
  k.phases = std::min(apart, k.segment);
  const int64_t phases = M / k.segment * k.phases, rows = (k.segment + apart - 1) / apart;  // of a phase, at most
  const int64_t least = (rows + kMostRows - 1) / kMostRows;
  int64_t best = INT64_MAX;
  // one or two chunks a group, or as few as may be
  for (const int64_t n : {least, units / phases, (units + phases - 1) / phases, 2 * units / phases}) {
    const int64_t m = std::min(rows, std::max(least, n));
    const int64_t per = (rows + m - 1) / m, of = (rows + per - 1) / per, chunks = phases * of;
    const int64_t cost = (chunks + units - 1) / units * (per + 1);
    if (cost < best) {
      best = cost;
      k.rows = per;
      k.per_segment = k.phases * of;
      k.chunks = chunks;
    }
  }
  return k;
}

}  // namespace swg
