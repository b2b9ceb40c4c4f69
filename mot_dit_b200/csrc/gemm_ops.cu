// tcgen05 products of the feed-forward operators, both directions (sm_100a).
//
//   C[m, n] = sum_k A[m, k] B[n, k], bf16 operands, fp32 accumulators.
//
// One kernel serves the forward product (A = x, B = W, both stored with the
// reduction innermost), the input gradient (A = dz, B = W stored with the
// reduction outermost) and the weight gradient (A = dz, B = x, both with the
// reduction outermost).  Nothing is transposed in memory: the tensor core
// reads either order from shared memory (the descriptor's major-ness bit), and
// a TMA box of 64 elements x 64 rows lands in the 128-byte-swizzled layout it
// wants for each.  A launch takes a list of products, so that both gradients
// of a layer share one grid and their last waves overlap.  A product may sum
// over two operand pairs (the two halves of a gated layer's input gradient),
// or have two B operands (gate and up): their columns sit side by side in the
// accumulator, and the epilogue forms act(g) u without g or u leaving the chip.
//
// Forms (launch_op_gemm chooses, with the measured costs):
//  - CTA pairs (CG = 2): two CTAs share each 256 x 256 MMA tile (the 2-SM
//    form), persistent, accumulators double-buffered in tensor memory so that
//    one tile's epilogue runs under the next one's MMAs;
//  - single CTAs (CG = 1): 128 x bn tiles, the same way;
//  - cluster split: few tiles and a long reduction.  The CTAs of a cluster
//    take one k-range each of one tile; each leaves its fp32 partial tile in
//    its (then idle) operand ring, and after one cluster barrier each CTA sums
//    and finishes its share of the rows, reading the partials of the others
//    through distributed shared memory in rank (= k) order.  No workspace, no
//    counters, a fixed order of addition.
//  - MANUAL: operands that TMA cannot address (rows that do not start on
//    16-byte boundaries) are brought in by four loader warps that write the
//    same swizzled layout; the rest of the kernel does not change.
//
// Warp roles: warp 0 TMA producer, warp 1 TMEM owner and MMA issuer, warps
// 2..5 epilogue (warp w reads TMEM lanes 32 (w % 4) ..), MANUAL: warps 6..9
// loaders.  No load is multicast.  Every wait is bounded (op_gemm_status).
#include <algorithm>
#include <atomic>

#include "cluster.cuh"
#include "kernels.h"
#include "op_epilogue.cuh"

namespace wam {
namespace {

constexpr int BM = 128;
constexpr int BK = 64;
constexpr int kABytes = BM * BK * 2;
constexpr int kStg = 32 * 64 * 4;  // staging of one epilogue warp: 32 rows x 64 fp32
constexpr int kBarBytes = 512;
constexpr int kSmemMax = 232448;
constexpr int kMaxStages = 12;
constexpr int kRaster = 8;  // row tiles that are walked together (operands shared through L2)

__device__ unsigned g_op_status;

struct ProductK {
  CUtensorMap ma[2], mb[2];
  OpMat a[2], b[2];
  int M, N;           // N: columns of the output (gated: of g and of u each)
  int kb0, kb;        // k-blocks of the first operand pair, of all pairs
  int bn;             // accumulator columns of a tile (gated: g and u halves)
  int tiles_m, tiles_n, tile0;
  int a_mn, b_mn, gated;
  OpEpi e;
};
struct GemmArgs {
  ProductK p[kOpProducts];
  OpColSum sums[2];
  int np, n_sums, tiles;
  int stages, stage_bytes;
  int split;    // CTAs of a cluster that share one tile's reduction (1: persistent)
  int nbuf, nseg;  // accumulator buffers, and segments of each
  int tm_cols;  // tensor-memory columns to allocate
};

struct Tile {
  int p, m, n;  // product, row tile, column tile
};
__device__ __forceinline__ Tile tile_at(const GemmArgs& g, int t) {
  Tile r;
  r.p = 0;
  while (r.p + 1 < g.np && t >= g.p[r.p + 1].tile0) ++r.p;
  const ProductK& P = g.p[r.p];
  const int l = t - P.tile0, per = kRaster * P.tiles_n, grp = l / per, in = l - grp * per;
  const int gm = min(kRaster, P.tiles_m - grp * kRaster);
  r.m = grp * kRaster + in % gm;
  r.n = in / gm;
  return r;
}

__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, bool mn) {
  // K-major: rows of 64 reduction elements, 8-row groups 1024 B apart.
  // MN-major: rows of 64 output elements, one row per reduction index; 8-row
  // groups 1024 B apart along the reduction (stride offset), blocks of 64
  // output elements 8192 B apart (leading offset).
  uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>(mn ? (8192 >> 4) : 1) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// Byte offset of 16-byte chunk q (0..15) of staging row r: rows of 256 bytes,
// chunks permuted so that neither the row-per-lane writes nor the eight-
// lanes-per-row reads meet a bank twice (gated: chunk q and q + 8 are read
// by one lane; else chunks 2 c and 2 c + 1).
__device__ __forceinline__ int stg_off(int r, int q, bool gated) {
  const int pos = gated ? (((q & 7) ^ (r & 7)) | (q & 8)) : (((q >> 1) ^ (r & 7)) | ((q & 1) << 3));
  return r * 256 + pos * 16;
}

// 64 staged columns of 32 rows -> the output.  Eight lanes share a row, eight
// (gated: four and four) columns each.
template <bool GATED>
__device__ __forceinline__ void finish_vec(const OpEpi& e, const uint8_t* stg, int lane, int m0, int M, int n0, int N) {
  constexpr int E = GATED ? 4 : 8;
  const int cg = lane & 7, n = n0 + cg * E;
  if (n >= N) return;
  float b[E], b2[E];
  epi_bias<E>(e.bias, n, b);
  if (GATED) epi_bias<E>(e.bias2, n, b2);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    float r[4][E];
    if (!GATED && e.res) {
      load_batch<E, 4>(e.res, e.out_f32, [&](int i) {
        const int m = m0 + (4 * h + i) * 4 + (lane >> 3);
        return m < M ? (long long)m * e.ld + n : -1ll;
      }, r);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rr = (4 * h + i) * 4 + (lane >> 3), m = m0 + rr;
      const int q0 = GATED ? cg : 2 * cg, q1 = GATED ? cg + 8 : 2 * cg + 1;
      const float4 x = *reinterpret_cast<const float4*>(stg + stg_off(rr, q0, GATED));
      const float4 y = *reinterpret_cast<const float4*>(stg + stg_off(rr, q1, GATED));
      if (m >= M) continue;
      const size_t at = (size_t)m * e.ld + n;
      if constexpr (GATED) {
        float g[4] = {x.x, x.y, x.z, x.w}, u[4] = {y.x, y.y, y.z, y.w};
        epi_gated<false, 4>(e, at, g, u, b, b2);
      } else {
        float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        epi_linear<false, 8>(e, at, v, b, r[i]);
      }
    }
  }
}
// The same for outputs whose rows are not 16-byte aligned: a row at a time,
// lanes on consecutive columns.
template <bool GATED>
__device__ __forceinline__ void finish_any(const OpEpi& e, const uint8_t* stg, int lane, int m0, int M, int n0, int N) {
  const int rows = min(32, M - m0);
#pragma unroll 1
  for (int h = 0; h < (GATED ? 1 : 2); ++h) {
    const int c = 32 * h + lane, n = n0 + c;
    if (n >= N) continue;
    float b[1], b2[1];
    epi_bias<1>(e.bias, n, b);
    if (GATED) epi_bias<1>(e.bias2, n, b2);
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 8) {
      float res[8][1];
      if (!GATED && e.res)
        load_batch<1, 8>(e.res, e.out_f32,
                         [&](int i) { return r0 + i < rows ? (long long)(m0 + r0 + i) * e.ld + n : -1ll; }, res);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + i;
        if (r >= rows) continue;
        float v[1] = {*reinterpret_cast<const float*>(stg + stg_off(r, c >> 2, GATED) + (c & 3) * 4)};
        const size_t at = (size_t)(m0 + r) * e.ld + n;
        if constexpr (GATED) {
          float u[1] = {*reinterpret_cast<const float*>(stg + stg_off(r, (c >> 2) + 8, GATED) + (c & 3) * 4)};
          epi_gated<false, 1>(e, at, v, u, b, b2);
        } else {
          epi_linear<false, 1>(e, at, v, b, res[i]);
        }
      }
    }
  }
}

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int CG, bool MANUAL>
__global__ void __launch_bounds__(MANUAL ? 320 : 192, 1) op_gemm_kernel(const __grid_constant__ GemmArgs g) {
  static_assert(CG == 1 || !MANUAL, "the loader warps serve single CTAs");
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {  // the swizzle is a function of the address bits
    if (threadIdx.x == 0) atomicOr(&g_op_status, kStatusTimeoutDrain);
    return;
  }
  const int stages = g.stages, sbytes = g.stage_bytes;
  uint8_t* sStg = smem + (size_t)stages * sbytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sStg + 4 * kStg);
  uint64_t* empty = full + kMaxStages;
  uint64_t* accf = empty + kMaxStages;
  uint64_t* acce = accf + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  unsigned* status = &g_op_status;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = g.split;
  const uint32_t rank = (CG == 2 || S > 1) ? cluster_rank() : 0u;
  const int unit = CG == 2 ? (int)(blockIdx.x >> 1) : (int)blockIdx.x / S;
  const int units = CG == 2 ? (int)(gridDim.x >> 1) : (int)gridDim.x / S;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], MANUAL ? 4 : 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], CG == 2 && rank == 0 ? 8 : 4);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0 && !MANUAL) {
    for (int p = 0; p < g.np; ++p) {
      prefetch_tensormap(&g.p[p].ma[0]);
      prefetch_tensormap(&g.p[p].mb[0]);
    }
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(tmem_slot, g.tm_cols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, g.tm_cols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();  // the peer's barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Accumulator buffers, nseg segments each: a segment takes up to seg_blocks
  // k-blocks, and the epilogue adds them (the tensor core's additions truncate,
  // which a long chain would show in an fp32 output).
  const int nbuf = g.nbuf, nseg = g.nseg, buf_cols = g.tm_cols / nbuf;
  auto seg_blocks = [&](int n_kb) { return (n_kb + nseg - 1) / nseg; };
  pdl_trigger();

  // k-blocks of this CTA's part of a tile
  auto k_lo = [&](const ProductK& P) { return S > 1 ? (int)((long long)P.kb * rank / S) : 0; };
  auto k_hi = [&](const ProductK& P) { return S > 1 ? (int)((long long)P.kb * (rank + 1) / S) : P.kb; };

  if (warp == 0) {
    if (!MANUAL && lane == 0) {
      const bool peer = CG == 2 && rank == 1;
      int it = 0, st = 0;  // loads issued; stage and its phase
      uint32_t phase = 0;
      bool ok = true;
      pdl_wait();
      for (int t = unit; t < g.tiles && ok; t += units) {
        const Tile tl = tile_at(g, t);
        const ProductK& P = g.p[tl.p];
        // (everything that the loop needs, in registers: an indexed parameter
        // read per k-block would be the loop's critical path)
        const int m0 = (tl.m * CG + (CG == 2 ? (int)rank : 0)) * BM;
        const int brows = P.bn / CG;
        const bool gated = P.gated, amn = P.a_mn, bmn = P.b_mn;
        const int n0 = gated ? tl.n * (P.bn / 2) : tl.n * P.bn + (CG == 2 ? (int)rank * brows : 0);
        const uint32_t bytes = (uint32_t)(kABytes + brows * BK * 2) * CG;
        const int lo = k_lo(P), hi = k_hi(P), kb0 = P.kb0;
        for (int q = 0; q < 2 && ok; ++q) {  // operand pairs
          const CUtensorMap* ma = &P.ma[q];
          const CUtensorMap* mb = gated && CG == 2 ? &P.mb[rank] : &P.mb[q];
          const CUtensorMap* mb1 = &P.mb[1];
          const int end = q ? hi : min(hi, kb0);
          for (int kb = q ? max(lo, kb0) : lo; kb < end; ++kb, ++it) {
            if (it >= stages && !mbar_wait(&empty[st], phase ^ 1, status, kStatusTimeoutTmaEmpty, abort_flag)) {
              ok = false;
              break;
            }
            if (!peer) mbar_arrive_expect_tx(&full[st], bytes);
            const int kk = (q ? kb - kb0 : kb) * BK;
            uint8_t* sa = smem + (size_t)st * sbytes;
            uint8_t* sb = sa + kABytes;
            const uint32_t bar = peer ? cluster_addr(&full[st], 0) : smem_u32(&full[st]);
            auto load = [&](const CUtensorMap* map, uint8_t* dst, int x, int y) {
              if (CG == 2 && peer)
                tma_load_3d_pair(dst, map, bar, x, y, 0);
              else
                tma_load_3d(dst, map, &full[st], x, y, 0);
            };
            if (amn) {
              load(ma, sa, m0, kk);
              load(ma, sa + 8192, m0 + 64, kk);
            } else {
              load(ma, sa, kk, m0);
            }
            if (bmn) {
              for (int j = 0; j < brows; j += 64) load(mb, sb + j * 128, n0 + j, kk);
            } else {
              load(mb, sb, kk, n0);  // gated: g's rows, then u's (a pair: one CTA each)
              if (CG == 1 && gated) load(mb1, sb + brows / 2 * 128, kk, n0);
            }
            if (++st == stages) st = 0, phase ^= 1;
          }
        }
      }
      // never leave with copies into the shared memory in flight, nor (pairs)
      // with MMAs still reading it
      if (!peer)
        for (int i = max(0, it - stages); i < it; ++i)
          mbar_wait(&full[i % stages], (i / stages) & 1, status, kStatusTimeoutDrain, nullptr);
      if (CG == 2) {
        volatile int gave_up = 0;
        for (int i = max(0, it - stages); i < it; ++i)
          mbar_wait(&empty[i % stages], (i / stages) & 1, status, kStatusTimeoutDrain, &gave_up);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank * (CG - 1) == 0) {
      int st = 0, buf = 0, lt = 0;
      uint32_t phase = 0, bphase = 0;
      bool ok = true;
      for (int t = unit; t < g.tiles && ok; t += units, ++lt) {
        const ProductK& P = g.p[tile_at(g, t).p];
        if (lt >= nbuf && !mbar_wait(&acce[buf], bphase ^ 1, status, kStatusTimeoutAccum, abort_flag)) break;
        tc_fence_after();
        const bool amn = P.a_mn, bmn = P.b_mn;
        const uint32_t bn = P.bn;
        const uint32_t idesc = idesc_bf16_f32(BM * CG, bn) | (amn ? 1u << 15 : 0u) | (bmn ? 1u << 16 : 0u);
        const uint64_t sa = amn ? 2048 >> 4 : 32 >> 4, sb = bmn ? 2048 >> 4 : 32 >> 4;  // descriptor step per K = 16
        const uint64_t da0 = smem_desc(0, amn), db0 = smem_desc(0, bmn);
        const int n_kb = k_hi(P) - k_lo(P), seg = seg_blocks(n_kb);
        uint32_t d = tmem + buf * buf_cols;
        for (int kb = 0, in = 0; kb < n_kb; ++kb) {
          if (!mbar_wait(&full[st], phase, status, kStatusTimeoutTmaFull, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem) + (uint32_t)(st * sbytes);
          // (the address field is 14 bits: in a cluster, shared addresses carry the CTA's rank above them)
          const uint64_t da = da0 | (a0 >> 4 & 0x3FFF), db = db0 | ((a0 + kABytes) >> 4 & 0x3FFF);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k) {
            const uint32_t acc = (in > 0 || k > 0) ? 1u : 0u;
            if constexpr (CG == 2)
              tc_mma_bf16_pair(d, da + k * sa, db + k * sb, idesc, acc);
            else
              tc_mma_bf16(d, da + k * sa, db + k * sb, idesc, acc);
          }
          if constexpr (CG == 2) {
            tc_commit_pair(smem_u32(&empty[st]));
            tc_commit_pair(cluster_addr(&empty[st], 1));
          } else {
            tc_commit(&empty[st]);
          }
          if (++st == stages) st = 0, phase ^= 1;
          if (++in == seg) in = 0, d += bn;
        }
        if constexpr (CG == 2) {
          tc_commit_pair(smem_u32(&accf[buf]));
          tc_commit_pair(cluster_addr(&accf[buf], 1));
        } else {
          tc_commit(&accf[buf]);
        }
        if (++buf == nbuf) buf = 0, bphase ^= 1;
      }
    }
    __syncwarp();
  } else if (warp < 6) {
    // ------------------------------------------------------------ epilogue
    pdl_wait();
    const int quad = warp & 3, te = threadIdx.x - 64;
    for (int i = 0; i < g.n_sums; ++i) {
      const OpColSum cs = g.sums[i];
      for (int c = blockIdx.x * 128 + te; c < cs.cols; c += gridDim.x * 128) {
        float a = 0.f;
#pragma unroll 16
        for (int r = 0; r < cs.rows; ++r) a += cs.part[(size_t)r * cs.cols + c];
        cs.out[c] = a;
      }
    }
    uint8_t* stg = sStg + quad * kStg;
    int buf = 0;
    uint32_t bphase = 0;
    for (int t = unit; t < g.tiles; t += units) {
      const Tile tl = tile_at(g, t);
      const ProductK& P = g.p[tl.p];
      const OpEpi e = P.e;
      const int bn = P.bn, pM = P.M, pN = P.N;
      const bool gated = P.gated;
      const int m0 = (tl.m * CG + (CG == 2 ? (int)rank : 0)) * BM;
      const int n0 = tl.n * (gated ? bn / 2 : bn);
      const int n_kb = k_hi(P) - k_lo(P), sg = seg_blocks(n_kb), segs = (n_kb + sg - 1) / sg;
      const bool ok = mbar_wait(&accf[buf], bphase, status, kStatusTimeoutAccum, abort_flag);
      tc_fence_after();
      if (!ok) *abort_flag = 1;
      epi_sync();  // one decision for all four warps
      if (*abort_flag) break;
      const uint32_t t_row = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * buf_cols;
      const int mw = m0 + quad * 32;
      // 32 accumulator columns, the segments added
      auto acc32 = [&](int c, float (&v)[32]) {
        tmem_ld32(t_row + c, v);
#pragma unroll 1
        for (int k = 1; k < segs; ++k) {
          float w[32];
          tmem_ld32(t_row + k * bn + c, w);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] += w[i];
        }
      };
      if (S > 1) {
        // leave the partial tile in the idle operand ring, chunk q of row r at q ^ (r & 7)
        if (mw < pM) {
          const int r = quad * 32 + lane;
          uint8_t* row = smem + (size_t)r * bn * 4;
          for (int c = 0; c < bn; c += 32) {
            float v[32];
            acc32(c, v);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<float4*>(row + ((((c >> 2) + q) ^ (r & 7)) << 4)) =
                  make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          }
        }
        break;  // one tile per cluster; the rest after the cluster barrier
      }
      const int step = gated ? 32 : 64, width = gated ? bn / 2 : bn;
      for (int c = 0; c < width; c += step) {
        float v[32];
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          acc32(gated ? c + h * (bn / 2) : c + 32 * h, v);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(stg + stg_off(lane, 8 * h + q, gated)) =
                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
        if (c + step >= width) tc_fence_before();
        __syncwarp();
        if (c + step >= width && lane == 0) {  // this warp's reads of the accumulator are done
          if (CG == 2 && rank == 1)
            mbar_arrive_cluster(cluster_addr(&acce[buf], 0));
          else
            mbar_arrive(&acce[buf]);
        }
        if (mw < pM) {
          if (gated) {
            if (e.vec)
              finish_vec<true>(e, stg, lane, mw, pM, n0 + c, pN);
            else
              finish_any<true>(e, stg, lane, mw, pM, n0 + c, pN);
          } else {
            if (e.vec)
              finish_vec<false>(e, stg, lane, mw, pM, n0 + c, pN);
            else
              finish_any<false>(e, stg, lane, mw, pM, n0 + c, pN);
          }
        }
        __syncwarp();
      }
      if (++buf == nbuf) buf = 0, bphase ^= 1;
    }
  } else if (MANUAL) {
    // ------------------------------------------------------------- loaders
    pdl_wait();
    const int tl_ = threadIdx.x - 192;
    int it = 0, s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = unit; t < g.tiles && ok; t += units) {
      const Tile tl = tile_at(g, t);
      const ProductK& P = g.p[tl.p];
      const int m0 = tl.m * BM, n0 = tl.n * (P.gated ? P.bn / 2 : P.bn);
      const int hi = k_hi(P);
      for (int kb = k_lo(P); kb < hi; ++kb, ++it) {
        // (one answer for the whole warp)
        if (it >= stages && !__all_sync(0xffffffffu, mbar_wait(&empty[s], phase ^ 1, status,
                                                               kStatusTimeoutTmaEmpty, abort_flag))) {
          ok = false;
          break;
        }
        const int q = kb >= P.kb0 ? 1 : 0, kk = (kb - (q ? P.kb0 : 0)) * BK;
        uint8_t* st = smem + (size_t)s * sbytes;
        // `rows` rows of 128 bytes at st + off, in batches of four chunks a thread
        auto bring = [&](const OpMat& mt, int off, int rows, int row0, int col0) {
          for (int i0 = tl_; i0 < rows * 8; i0 += 512) {
            uint4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int i = i0 + u * 128;
              if (i < rows * 8) v[u] = fetch8(mt, row0 + (i >> 3), col0 + (i & 7) * 8);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int i = i0 + u * 128, r = i >> 3;
              if (i < rows * 8) *reinterpret_cast<uint4*>(st + off + r * 128 + (((i & 7) ^ (r & 7)) << 4)) = v[u];
            }
          }
        };
        if (P.a_mn) {
          bring(P.a[q], 0, 64, kk, m0);
          bring(P.a[q], 8192, 64, kk, m0 + 64);
        } else {
          bring(P.a[q], 0, BM, m0, kk);
        }
        if (P.gated) {
          bring(P.b[0], kABytes, P.bn / 2, n0, kk);
          bring(P.b[1], kABytes + P.bn / 2 * 128, P.bn / 2, n0, kk);
        } else if (P.b_mn) {
          for (int j = 0; j < P.bn; j += 64) bring(P.b[q], kABytes + j * 128, 64, kk, n0 + j);
        } else {
          bring(P.b[q], kABytes, P.bn, n0, kk);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        if (++s == stages) s = 0, phase ^= 1;
      }
    }
  }

  if (S > 1) {  // (uniform over the cluster, reached on every path)
    __syncwarp();
    cluster_sync();  // every partial tile is in place
    if (warp >= 2 && warp < 6 && !*abort_flag) {
      const Tile tl = tile_at(g, unit);
      const ProductK& P = g.p[tl.p];
      const int m0 = tl.m * BM, n0 = tl.n * (P.gated ? P.bn / 2 : P.bn);
      const int valid = min(BM, P.M - m0);
      const int r_lo = valid * (int)rank / S, r_hi = valid * ((int)rank + 1) / S;
      uint32_t base[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) base[s] = s < S ? mapa_u32(smem_u32(smem), s) : 0u;
      const int te = threadIdx.x - 64;
      const OpEpi e = P.e;
      if (P.gated) {
        if (e.vec)
          finish_split<false, true, 4>(e, P.bn, P.N, base, S, te, 128, r_lo, r_hi, m0, n0);
        else
          finish_split<false, true, 1>(e, P.bn, P.N, base, S, te, 128, r_lo, r_hi, m0, n0);
      } else {
        if (e.vec)
          finish_split<false, false, 8>(e, P.bn, P.N, base, S, te, 128, r_lo, r_hi, m0, n0);
        else
          finish_split<false, false, 1>(e, P.bn, P.N, base, S, te, 128, r_lo, r_hi, m0, n0);
      }
    }
  }

  // ------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) {  // the last commits have arrived before the tensor memory is freed
      int n = 0;
      for (int t = unit; t < g.tiles; t += units) ++n;
      for (int l = max(0, n - nbuf); l < n; ++l)
        mbar_wait(&accf[l % nbuf], (l / nbuf) & 1, status, kStatusTimeoutDrain, nullptr);
    }
    __syncwarp();
  }
  if (CG == 2 || S > 1) cluster_sync();  // no CTA leaves while another may read its shared memory
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2)
      tmem_dealloc_pair(tmem, g.tm_cols);
    else
      tmem_dealloc(tmem, g.tm_cols);
  }
}

// ------------------------------------------------------------------- host --
struct Device {
  std::atomic<int> ready{0};
  int sms = 148, pairs = 74;
};
Device g_dev[64];

cudaError_t device_info(Device** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  Device& d = g_dev[dev];
  if (!d.ready.load(std::memory_order_acquire)) {  // (idempotent: two threads may both do it)
    int sms = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(op_gemm_kernel<1, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(op_gemm_kernel<2, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(op_gemm_kernel<1, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax)) != cudaSuccess)
      return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms);
    cfg.blockDim = dim3(192);
    cfg.dynamicSmemBytes = kSmemMax;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int pairs = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&pairs, op_gemm_kernel<2, false>, &cfg)) != cudaSuccess) return e;
    d.sms = sms;
    d.pairs = std::max(1, std::min(pairs, sms / 2));
    d.ready.store(1, std::memory_order_release);
  }
  *out = &d;
  return cudaSuccess;
}

struct Plan {
  int cg, bn, split;
  int seg;  // accumulator segments
};
// Longest chain of k-blocks in one accumulator when the output is fp32: 1536
// products, about 8e-7 of the result in truncated additions (6144: 3e-6).
constexpr int kChain = 24;

int ceil_div(int a, int b) { return (a + b - 1) / b; }
// Accumulator columns of product p's tiles under plan width bn.
int tile_cols(const OpProduct& p, const Plan& pl) {
  const int q = pl.cg == 2 ? 128 : 64;  // (MN-major halves of a pair are whole 64-column boxes)
  const int n = p.gated ? 2 * ceil_div(p.N, 32) * 32 : p.N;
  return std::min(pl.bn, ceil_div(n, q) * q);
}
int k_blocks(const OpProduct& p) { return std::max(1, p.pairs) * ceil_div(p.K, BK); }

// Estimated clocks of a plan: the busiest CTA (pair)'s k-blocks at the
// measured cost of one, plus the parts that nothing overlaps.
double plan_cost(const OpProduct* p, int n, const Plan& pl, const Device& d) {
  const double per = pl.cg == 2 ? (pl.bn == 256 ? 560 : 320) : pl.bn == 256 ? 580 : pl.bn == 128 ? 380 : 270;
  const int units = pl.cg == 2 ? d.pairs : d.sms;
  if (pl.split > 1) {
    const OpProduct& q = p[0];
    const int bn = tile_cols(q, pl), tn = ceil_div(q.gated ? 2 * q.N : q.N, bn), tm = ceil_div(q.M, BM);
    const int waves = ceil_div(tm * tn * pl.split, units);
    return waves * (ceil_div(k_blocks(q), pl.split) * per + 4500.0 + 6.0 * bn);
  }
  double load[160];
  for (int u = 0; u < units && u < 160; ++u) load[u] = 0;
  long long pos = 0;
  for (int i = 0; i < n; ++i) {
    const int bn = tile_cols(p[i], pl);
    const long long tiles = (long long)ceil_div(p[i].M, BM * pl.cg) * ceil_div(p[i].gated ? 2 * p[i].N : p[i].N, bn);
    const double c = k_blocks(p[i]) * per + 300;
    const long long all = tiles / units;
    for (int u = 0; u < units && u < 160; ++u) {
      const int off = (int)((u - pos % units + units) % units);
      load[u] += (all + (off < tiles % units ? 1 : 0)) * c;
    }
    pos += tiles;
  }
  double worst = 0;
  for (int u = 0; u < units && u < 160; ++u) worst = std::max(worst, load[u]);
  return worst + 2500.0 + 12.0 * pl.bn;
}

Plan choose(const OpProduct* p, int n, bool manual, const Device& d) {
  Plan best{1, 128, 1, 1};
  double bc = 1e30;
  int chain = 0;  // longest reduction that ends in fp32
  for (int i = 0; i < n; ++i)
    if (p[i].e.out_f32) chain = std::max(chain, k_blocks(p[i]));
  auto consider = [&](Plan pl) {
    pl.seg = std::max(1, ceil_div(ceil_div(chain, pl.split), kChain));
    if (pl.seg > 512 / pl.bn) {  // no tensor memory for so many: the narrowest tile takes what there is
      if (pl.bn > 64) return;
      pl.seg = 512 / pl.bn;
    }
    const double c = plan_cost(p, n, pl, d);
    if (c < bc) bc = c, best = pl;
  };
  for (int bn : {256, 128, 64}) {
    consider(Plan{1, bn, 1, 1});
    if (n == 1)
      for (int s = 2; s <= 8; ++s)
        if (k_blocks(p[0]) >= 2 * s) consider(Plan{1, bn, s, 1});
  }
  if (!manual) {
    consider(Plan{2, 256, 1, 1});
    consider(Plan{2, 128, 1, 1});
  }
  return best;
}

bool tma_ok(const OpMat& m) { return (reinterpret_cast<uintptr_t>(m.p) & 15) == 0 && m.ld % 8 == 0; }

}  // namespace

cudaError_t op_gemm_status(unsigned* bits) {
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return e;
  if ((e = cudaMemcpyFromSymbol(bits, g_op_status, 4)) != cudaSuccess) return e;
  const unsigned zero = 0;
  return *bits ? cudaMemcpyToSymbol(g_op_status, &zero, 4) : cudaSuccess;
}

cudaError_t launch_op_gemm(const OpProduct* p, int n, const OpColSum* sums, int n_sums, cudaStream_t s) {
  if (n < 1 || n > kOpProducts || n_sums < 0 || n_sums > 2) return cudaErrorInvalidValue;
  Device* d = nullptr;
  cudaError_t err = device_info(&d);
  if (err != cudaSuccess) return err;
  bool manual = false;
  for (int i = 0; i < n; ++i) {
    const int na = p[i].pairs == 2 ? 2 : 1, nb = (p[i].pairs == 2 || p[i].gated) ? 2 : 1;
    for (int k = 0; k < na; ++k) manual |= !tma_ok(p[i].a[k]);
    for (int k = 0; k < nb; ++k) manual |= !tma_ok(p[i].b[k]);
  }
  const Plan pl = choose(p, n, manual, *d);
  GemmArgs g;
  g.np = n;
  g.n_sums = n_sums;
  for (int i = 0; i < n_sums; ++i) g.sums[i] = sums[i];
  int tiles = 0, bmax = 0;
  for (int i = 0; i < n; ++i) {
    const OpProduct& q = p[i];
    ProductK& k = g.p[i];
    k.M = q.M;
    k.N = q.N;
    k.kb = k_blocks(q);
    k.kb0 = ceil_div(q.K, BK);
    k.bn = tile_cols(q, pl);
    k.tiles_m = ceil_div(q.M, BM * pl.cg);
    k.tiles_n = ceil_div(q.N, q.gated ? k.bn / 2 : k.bn);
    k.tile0 = tiles;
    tiles += k.tiles_m * k.tiles_n;
    k.a_mn = q.a_mn;
    k.b_mn = q.b_mn;
    k.gated = q.gated;
    k.e = q.e;
    bmax = std::max(bmax, k.bn);
    for (int j = 0; j < 2; ++j) {
      const OpMat& ma = q.a[q.pairs == 2 ? j : 0];
      const OpMat& mb = q.b[(q.pairs == 2 || q.gated) ? j : 0];
      k.a[j] = ma;
      k.b[j] = mb;
      if (manual) continue;
      const int boxb = q.b_mn ? 64 : q.gated ? k.bn / 2 : k.bn / pl.cg;
      if (!make_tmap_rows(&k.ma[j], ma.p, ma.inner, ma.outer, ma.ld, q.a_mn ? 64 : BM) ||
          !make_tmap_rows(&k.mb[j], mb.p, mb.inner, mb.outer, mb.ld, boxb))
        return cudaErrorInvalidValue;
    }
  }
  g.tiles = tiles;
  g.split = pl.split;
  g.stage_bytes = kABytes + bmax / pl.cg * BK * 2;
  g.stages = std::min(kMaxStages, (kSmemMax - kBarBytes - 4 * kStg) / g.stage_bytes);
  g.nseg = pl.seg;
  g.nbuf = pl.split == 1 && 2 * pl.seg * bmax <= 512 ? 2 : 1;
  g.tm_cols = 32;
  while (g.tm_cols < g.nbuf * pl.seg * bmax) g.tm_cols *= 2;
  const size_t smem = (size_t)g.stages * g.stage_bytes + 4 * kStg + kBarBytes;

  const int cluster = pl.cg == 2 ? 2 : pl.split;
  const int units = pl.split > 1 ? tiles : std::min(tiles, pl.cg == 2 ? d->pairs : d->sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units * cluster);
  cfg.blockDim = dim3(manual ? 320 : 192);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  int na = 0;
  if (cluster > 1) {
    at[na].id = cudaLaunchAttributeClusterDimension;
    at[na].val.clusterDim.x = cluster;
    at[na].val.clusterDim.y = at[na].val.clusterDim.z = 1;
    ++na;
  }
  if (pdl_enabled()) {
    at[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  cfg.attrs = at;
  cfg.numAttrs = na;
  if (pl.cg == 2) return cudaLaunchKernelEx(&cfg, op_gemm_kernel<2, false>, g);
  if (manual) return cudaLaunchKernelEx(&cfg, op_gemm_kernel<1, true>, g);
  return cudaLaunchKernelEx(&cfg, op_gemm_kernel<1, false>, g);
}

}  // namespace wam
