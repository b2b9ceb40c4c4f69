// Replays, on the host, how the warps of a feed-forward product walk one part
// [lo, hi) of a reduction: the producer fills stages pair by pair, the MMA
// warp closes accumulator segments, the epilogue waits for as many as it has
// counted.  Returns 0, or the number of the first disagreement.
#include <algorithm>

#include "op_reduction.h"

using namespace wam;

extern "C" int replay_part(int lo, int hi, int kb0, int subs, int chain, int most) {
  const Segments sg = segments_of(lo, hi, kb0, subs, chain, most);
  if (sg.per < 1 || sg.count < 1 || sg.count > std::max(1, segments_for(hi - lo, chain))) return 1;
  if (most && sg.count > most) return 2;
  // the producer's stages, one operand pair after the other
  int starts[2048], n = 0;
  for (int q = 0; q < 2; ++q) {
    const int end = q ? hi : std::min(hi, kb0);
    for (int kb = q ? std::max(lo, kb0) : lo; kb < end;) {
      if (n == 2048) return 3;
      starts[n++] = kb;
      kb += stage_blocks(kb, end, end, subs);
    }
  }
  if (n != stages_of(lo, hi, kb0, subs)) return 4;
  // the MMA warp
  int st = 0, in = 0, closed = 0, blocks = 0;
  for (int kb = lo; kb < hi;) {
    if (st == n || starts[st] != kb) return 5;
    const int ns = stage_blocks(kb, hi, kb0, subs);
    if (ns < 1 || ns > subs || (kb < kb0 && kb + ns > kb0)) return 6;
    kb += ns, ++st, ++in, blocks += ns;
    if (in == sg.per || kb >= hi) {
      if (chain && !most && blocks > (chain + subs - 1) / subs * subs + subs) return 7;  // (a seam may add one stage)
      ++closed, in = blocks = 0;
    }
  }
  if (st != n) return 8;
  return closed == sg.count ? 0 : 9;
}
// Every piece of a backward pass's two reductions, at one and two k-blocks a stage.
extern "C" int replay_backward(int f32, int M, int N, int K, int sides) {
  const Pieces c = pieces_for(f32, M, N, K, sides);
  const int kx = (N + 63) / 64, kw = (M + 63) / 64;
  for (int subs = 1; subs <= (f32 ? 1 : 2); ++subs)
    for (int chain : {0, f32 ? kChainF32 : kChain}) {
      for (int i = 0; i < c.dx; ++i)
        if (int e = replay_part(share_begin(sides * kx, i, c.dx), share_begin(sides * kx, i + 1, c.dx), kx, subs, chain, f32 ? 7 : 0))
          return 100 + e;
      for (int i = 0; i < c.dw; ++i)
        if (int e = replay_part(share_begin(kw, i, c.dw), share_begin(kw, i + 1, c.dw), kw, subs, chain, f32 ? 7 : 0)) return 200 + e;
    }
  return 0;
}
extern "C" int pieces_dx(int f32, int M, int N, int K, int sides) { return pieces_for(f32, M, N, K, sides).dx; }
extern "C" int columns(int bn, int N, int gated, int b_mn, int pair, int f32) { return tile_columns(bn, N, gated, b_mn, pair, f32); }
