// Replays, on the host, how the warps of a feed-forward product walk one part
// [lo, hi) of a reduction: the producer fills stages pair by pair, the MMA
// warp closes accumulator segments, the epilogue waits for as many as it has
// counted.  Returns 0, or the number of the first disagreement.
#include <algorithm>

#include "op_reduction.h"
#include "row_plan.h"

using namespace wam;

extern "C" int replay_part(int lo, int hi, int kb0, int subs, int chain, int nseg) {  // nseg: fp32 operands, segments a round (else 0)
  const Segments sg = segments_of(lo, hi, kb0, subs, chain);
  if (sg.per < 1 || sg.count < 1 || sg.count > std::max(1, segments_for(hi - lo, chain))) return 1;
  const int fills = nseg ? (sg.count + nseg - 1) / nseg : sg.count;
  // the producer's stages, one operand pair after the other (fp32: round after round)
  int starts[4096], n = 0;
  if (nseg) {
    for (int k = 0; k < fills; ++k)
      for (int kb = lo + k * nseg * sg.per; kb < std::min(hi, lo + (k + 1) * nseg * sg.per); ++kb) {
        if (n == 4096) return 3;
        starts[n++] = kb;
      }
  } else {
    for (int q = 0; q < 2; ++q) {
      const int end = q ? hi : std::min(hi, kb0);
      for (int kb = q ? std::max(lo, kb0) : lo; kb < end;) {
        if (n == 4096) return 3;
        starts[n++] = kb;
        kb += stage_blocks(kb, end, end, subs);
      }
    }
  }
  if (n != stages_of(lo, hi, kb0, subs)) return 4;
  // the MMA warp
  int st = 0, in = 0, slot = 0, closed = 0, blocks = 0;
  for (int kb = lo; kb < hi;) {
    if (st == n || starts[st] != kb) return 5;
    if (nseg && in == 0 && slot == 0 && kb != lo + closed * nseg * sg.per) return 2;
    const int ns = stage_blocks(kb, hi, kb0, subs);
    if (ns < 1 || ns > subs || (kb < kb0 && kb + ns > kb0)) return 6;
    kb += ns, ++st, ++in, blocks += ns;
    if (chain && blocks > (chain + subs - 1) / subs * subs + (lo < kb0 && kb0 < hi ? subs : 0)) return 7;  // (a seam may add a stage)
    bool last = kb >= hi;
    if (in == sg.per) in = blocks = 0, last |= !nseg || ++slot == nseg;
    if (last) ++closed, in = blocks = slot = 0;
  }
  if (st != n) return 8;
  return closed == fills ? 0 : 9;
}
// Every piece of a backward pass's two reductions, at one and two k-blocks a stage.
extern "C" int replay_backward(int f32, int M, int N, int K, int sides) {
  const Pieces c = pieces_for(f32, M, N, K, sides);
  const int kx = (N + 63) / 64, kw = (M + 63) / 64;
  for (int subs = 1; subs <= (f32 ? 1 : 2); ++subs)
    for (int chain : {0, f32 ? kChainF32 : kChain}) {
      for (int i = 0; i < c.dx; ++i)
        if (int e = replay_part(share_begin(sides * kx, i, c.dx), share_begin(sides * kx, i + 1, c.dx), kx, subs, chain, f32 ? 6 : 0))
          return 100 + e;
      for (int i = 0; i < c.dw; ++i)
        if (int e = replay_part(share_begin(kw, i, c.dw), share_begin(kw, i + 1, c.dw), kw, subs, chain, f32 ? 6 : 0)) return 200 + e;
    }
  return 0;
}
extern "C" int pieces_dx(int f32, int M, int N, int K, int sides) { return pieces_for(f32, M, N, K, sides).dx; }
extern "C" int columns(int bn, int N, int gated, int b_mn, int pair, int f32) { return tile_columns(bn, N, gated, b_mn, pair, f32); }
extern "C" int longest_chain(int n, int subs, int chain) { return std::min(n, segments_of(0, n, n, subs, chain).per * subs); }
// A backward norm block of D columns (element sizes of the stream and of the rest): bytes, and the stages of its ring.
extern "C" int grad_block(int D, int stream, int rest, int* stages, int* planned) {
  const int R = rows_at_once(row_threads(D, elems(D)));
  const Ring r = ring_of(D, R, coef_bytes(D, 2), {stream, rest, rest, stream});
  *stages = r.stages;
  *planned = grad_blocks_per_sm(D);
  return grad_smem(r, D) + kStaticSmem;
}
