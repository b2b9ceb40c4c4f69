// How a feed-forward product is cut (host and device, plain integers): its
// columns into tiles, its reduction into pieces that are tiles of their own, into
// the stages of the operand ring, and into the segments of an accumulator.
// Every warp of a CTA counts stages and segments by these functions, and by
// nothing else.
#pragma once

#ifdef __CUDACC__
#define WAM_HD __host__ __device__ __forceinline__
#else
#define WAM_HD inline
#endif

namespace wam {

// Shares of the two gradients' reductions.  A gradient with few tiles and a
// long reduction (the weights' of a narrow layer over many rows, the input's
// of few rows through a wide one) would keep a few SMs busy after the rest are
// done: its reduction is cut so that no tile takes longer than an SM's part
// of all the work, at least `least` k-blocks each, and the pieces (fp32, in the
// workspace) are added by a kernel after it.  linear 5128 rows, 271 x 74 fp32, in a
// graph: 132 us whole, 37 us in pieces.
struct Pieces {
  int dx, dw;
};
inline Pieces pieces_for(bool f32, int M, int N, int K, int sides) {
  constexpr int kSms = 148;
  const int bn = f32 ? 64 : 128, least = f32 ? 4 : 12;
  const double over = f32 ? 5 : 6;  // a tile's fixed part, in k-blocks
  const double cols = (K + bn - 1) / bn;
  const double tx = (M + 127) / 128 * cols, tw = sides * ((N + 127) / 128 * cols);
  const int kx = sides * ((N + 63) / 64), kw = (M + 63) / 64;
  const double share = (tx * (kx + over) + tw * (kw + over)) / kSms;
  auto cut = [&](int kb, double elements) {
    const double t = share > least ? share : least;
    if (kb < 1.5 * t) return 1;
    int p = (int)(kb / t + 0.999);
    if (p > 16) p = 16;
    while (p > 1 && p * elements * 4 > 32e6) --p;  // (the pieces stay in L2)
    return p;
  };
  return {cut(kx, (double)M * K), cut(kw, (double)sides * N * K)};
}
// Accumulator columns of the tiles of a product with N output columns (gated: of
// g and of u each) whose plan asks for bn: no more than N needs.  They come in
// steps of 32, which a box of a matrix with the reduction innermost can have;
// of 64, the box of a reduction-outermost one (b_mn), the halves of a gated tile
// and the widths that the loaders of fp32 operands are made for; of 128 to a
// pair, in halves.
inline int tile_columns(int bn, int N, bool gated, bool b_mn, bool pair, bool f32) {
  const int step = pair ? 128 : b_mn || gated || f32 ? 64 : 32;
  const int n = gated ? 2 * ((N + 31) / 32 * 32) : N, cols = (n + step - 1) / step * step;
  return cols < bn ? cols : bn;
}
// First k-block of share i of n (at most 16) of a reduction of kb k-blocks (at
// most 2^19: two pairs of the longest one).
WAM_HD int share_begin(int kb, int i, int n) { return (int)((unsigned)kb * (unsigned)i / (unsigned)n); }

// Longest chain of k-blocks in one accumulator where the output is fp32: 896
// products, about 9e-7 of the result in truncated additions (1536: 1.2e-6, 6144: 3e-6).
constexpr int kChain = 14;
constexpr int kChainF32 = 12;  // fp32 operands: 768, 7e-7 at any length of the reduction

// k-blocks of the stage that starts at block kb of a part that ends at hi: at
// most subs, and never of both operand pairs (the second starts at kb0).
WAM_HD int stage_blocks(int kb, int hi, int kb0, int subs) {
  const int end = kb < kb0 && kb0 < hi ? kb0 : hi;
  return end - kb < subs ? end - kb : subs;
}
// Stages of the k-blocks [lo, hi), one or two k-blocks each: a part that crosses
// from one operand pair to the other may have a short stage before the seam.
WAM_HD int stages_of(int lo, int hi, int kb0, int subs) {
  const int seam = lo < kb0 && kb0 < hi ? kb0 : hi;
  return ((seam - lo + subs - 1) >> (subs - 1)) + ((hi - seam + subs - 1) >> (subs - 1));
}
// Accumulator segments of a part of n k-blocks whose chains are at most
// `chain` long (0: any length; a seam in the part may make them a stage longer).
WAM_HD int segments_for(int n, int chain) { return chain ? (n + chain - 1) / chain : 1; }
// The segments of the k-blocks [lo, hi): whole stages, `per` each but the last.
struct Segments {
  int per, count;
};
WAM_HD Segments segments_of(int lo, int hi, int kb0, int subs, int chain) {
  const int stages = stages_of(lo, hi, kb0, subs);
  const int n = segments_for(hi - lo, chain);
  if (n <= 1) return {stages, 1};
  Segments s;
  s.per = (stages + n - 1) / n;
  s.count = (stages + s.per - 1) / s.per;
  return s;
}

}  // namespace wam
