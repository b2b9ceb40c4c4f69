// Shapes of the residual norm's blocks (host, plain integers): threads of a row,
// rows of a block, the ring of row groups, and the backward pass's chunks.
#pragma once

#include <algorithm>
#include <initializer_list>

namespace wam {

constexpr int kRowThreads = 224;  // row threads of a block when a row needs fewer (256 with the producer)
constexpr int kMaxStages = 8;
// Ring of a block (several blocks an SM) when two stages fit it, else what a
// block can have.  Two stages of the backward pass's four fp32 matrices are
// 57600 bytes at 1792 elements a group, the most of a block of 224 row threads
// (56 KB missed them, and one block an SM ran where grad_chunks plans for two:
// 65536 x 256 with its sums 120 us, 81 us so).
constexpr int kRing = 57 * 1024;
constexpr int kSmem = 224 * 1024;
constexpr int kStaticSmem = 3 * 1024;  // at most: barriers, sums and what the driver keeps of a block
constexpr int kSmemOfSm = 227 * 1024;

// Threads that share a row: NV elements each; a power of two below a warp,
// whole warps above.
inline int row_threads(int D, int nv) {
  const int t = (D + nv - 1) / nv;
  if (t > 32) return (t + 31) / 32 * 32;
  int p = 1;
  while (p < t) p *= 2;
  return p;
}
inline int rows_at_once(int tpr) { return tpr >= kRowThreads ? 1 : kRowThreads / tpr; }
inline int elems(int D) { return D > 7680 ? 24 : D > 3840 ? 16 : 8; }  // (blocks of at most 512, 512, 384 threads)

// The ring's shape: `rows` rows of up to four matrices a stage.
struct Ring {
  int stages, stage_bytes;
  int off[4];  // of each matrix in a stage
};
inline Ring ring_of(int D, int rows, int reserved, std::initializer_list<int> sizes) {
  Ring r{};
  int at = 0, i = 0;
  for (int e : sizes) {
    r.off[i++] = at;
    at += (rows * D * e + 15) / 16 * 16 + 16;  // (a span that starts inside a granule takes one more)
  }
  r.stage_bytes = (at + 127) / 128 * 128;
  const int budget = 2 * r.stage_bytes <= kRing ? kRing : kSmem - reserved;
  r.stages = std::max(1, std::min(kMaxStages, budget / r.stage_bytes));
  return r;
}
// Bytes behind the ring: n vectors of a sample's coefficients, where they are not in registers.
inline int coef_bytes(int D, int n) { return elems(D) == 8 ? 0 : n * ((D + 7) / 8 * 8) * 4; }
// Shared memory of a backward block: the ring and the coefficients, or the
// column sums of its row lanes, which are joined there at the end.
inline int grad_smem(const Ring& ring, int D) {
  const int nv = elems(D), tpr = row_threads(D, nv), R = rows_at_once(tpr);
  return std::max(ring.stages * ring.stage_bytes + coef_bytes(D, 2), R > 1 ? R * 3 * tpr * nv * 4 : 0);
}

// Backward blocks that an SM runs at once: two (by registers), one of more than 256 threads.
inline int grad_blocks_per_sm(int D) {
  const int tpr = row_threads(D, elems(D));
  return tpr * rows_at_once(tpr) <= kRowThreads ? 2 : 1;
}
// Chunks of rows per sample: as many blocks as run at once, each of at least
// four passes of its row lanes.
inline int grad_chunks(int M, int D, int rpg) {
  const int rows = rows_at_once(row_threads(D, elems(D))), blocks = 148 * grad_blocks_per_sm(D);
  const int groups = (M + rpg - 1) / rpg;
  const int most = (std::min(rpg, M) + 4 * rows - 1) / (4 * rows);
  return std::max(1, std::min(most, (blocks + groups - 1) / groups));
}

}  // namespace wam
