// tcgen05 products of the feed-forward operators, both directions (sm_100a).
//
//   C[m, n] = sum_k A[m, k] B[n, k], bf16 or fp32 operands, fp32 accumulators.
//
// One kernel serves the forward product (A = x, B = W, both stored with the
// reduction innermost), the input gradient (A = dz, B = W stored with the
// reduction outermost) and the weight gradient (A = dz, B = x, both with the
// reduction outermost).  Nothing is transposed in memory: the tensor core
// reads either order from shared memory (the descriptor's major-ness bit), and
// a TMA box of 64 elements a row lands in the 128-byte-swizzled layout that it
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
//  - kManual: bf16 operands that TMA cannot address (rows that do not start on
//    16-byte boundaries) are brought in by four loader warps that write the
//    same swizzled layout; the rest of the kernel does not change;
//  - kF32: fp32 operands are split into three bf16 parts by the warps that load
//    them (the epilogue's), and six part products are summed.
//
// Bound by the tensor pipe and the power cap where tiles are many (8448 x 6144 x
// 1536 gated: pipe busy 76% of the cycles at 1.69 GHz, 1.55 PFLOP/s; 4224 x
// 4096 x 1536 gated backward 1.45 PFLOP/s), by start, tail and whole waves where
// they are few (1088 x 1536 x 6144: 26.6 us in a graph, 144 tiles in one wave).
//
// Warp roles: warp 0 TMA producer, warp 1 TMEM owner and MMA issuer, warps
// 2..9 epilogue (warp w reads TMEM lanes 32 (w % 4) ..), kManual: warps 10..13
// loaders.  No load is multicast.  Every wait is bounded (op_gemm_status).
#include <algorithm>
#include <atomic>
#include <mutex>

#include "cluster.cuh"
#include "kernels.h"
#include "op_epilogue.cuh"
#include "op_reduction.h"

namespace wam {
namespace {

constexpr int BM = 128;
constexpr int BK = 64;
constexpr int kABytes = BM * BK * 2;
constexpr int kEpiWarps = 8;       // two per 32-row quarter of the tile, on alternate 32-column chunks
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kLoaders = 128;      // loader threads of kManual
// How operands come in: by TMA; by loader warps (bf16 at any alignment); by
// the epilogue warps, fp32 in three bf16 parts.
enum : int { kTma = 0, kManual = 1, kF32 = 2 };
constexpr int kStg = 32 * 32 * 4;  // staging of one epilogue warp: 32 rows x 32 fp32
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
  int pieces;         // shares of the reduction, each a tile of its own with its own output
  int chain;          // longest accumulator segment in k-blocks (0: one segment)
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
  int subs;  // k-blocks of a full stage
  int split;    // CTAs of a cluster that share one tile's reduction (1: persistent)
  int nbuf, buf_cols;  // accumulator buffers
  int nseg;            // fp32 operands: segment accumulators of the buffer (a round)
  int tm_cols;  // tensor-memory columns to allocate
};

struct Tile {
  int p, m, n;  // product, row tile, column tile
  int piece;
};
__device__ __forceinline__ Tile tile_at(const GemmArgs& g, int t) {
  Tile r;
  r.p = 0;
  while (r.p + 1 < g.np && t >= g.p[r.p + 1].tile0) ++r.p;
  const ProductK& P = g.p[r.p];
  int l = t - P.tile0;
  r.piece = 0;
  if (P.pieces > 1) {
    const int plane = P.tiles_m * P.tiles_n;
    r.piece = l / plane;
    l -= r.piece * plane;
  }
  const int per = kRaster * P.tiles_n, grp = l / per, in = l - grp * per;
  const int gm = min(kRaster, P.tiles_m - grp * kRaster);
  r.m = grp * kRaster + in % gm;
  r.n = in / gm;
  return r;
}

// Arrive on the barrier at this offset in both CTAs of the pair once every
// pair MMA issued so far by this thread completes.
__device__ __forceinline__ void tc_commit_both(uint32_t addr) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(addr),
      "h"((unsigned short)3)
      : "memory");
}

// 32 lanes x 32 consecutive columns to tensor memory.
__device__ __forceinline__ void tmem_st32f(uint32_t taddr, const float (&v)[32]) {
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// One thread of a converged warp.  (The compiler recognises the election and
// issues the thread's TMA and MMA instructions without guarding against
// several active lanes: a k-block of a 128 x 256 tile takes 0.278 us, the
// tensor rate, and 0.34 us under a lane test.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, bool mn, int subs) {
  // K-major: rows of 64 reduction elements, 8-row groups 1024 B apart.
  // MN-major: rows of 64 output elements, one row per reduction index; 8-row
  // groups 1024 B apart along the reduction (stride offset), blocks of 64
  // output elements a stage's 64 subs rows apart (leading offset).
  uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>(mn ? (subs * 8192) >> 4 : 1) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// ---- output of one warp: 32 rows (one per lane) x 32 columns, through the
// warp's staging so that global accesses run along rows.  Staging rows are 64
// (bf16) or 128 (fp32) bytes, their 16-byte chunks permuted so that neither
// the row-per-lane writes nor the chunk-per-lane reads meet a bank twice.
__device__ __forceinline__ uint4* stg16(uint8_t* stg, int r, int q) {
  return reinterpret_cast<uint4*>(stg + r * 64 + ((q ^ ((r >> 1) & 3)) << 4));
}
__device__ __forceinline__ float4* stg32(uint8_t* stg, int r, int q) {
  return reinterpret_cast<float4*>(stg + r * 128 + ((q ^ (r & 7)) << 4));
}
struct Window {
  int m0, M, n0, N, ld;
  int vec;
};
__device__ __forceinline__ void out_bf16(const float (&v)[32], void* out, const Window& w, uint8_t* stg, int lane) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *stg16(stg, lane, q) = make_uint4(pack_bf16(v[8 * q], v[8 * q + 1]), pack_bf16(v[8 * q + 2], v[8 * q + 3]),
                                      pack_bf16(v[8 * q + 4], v[8 * q + 5]), pack_bf16(v[8 * q + 6], v[8 * q + 7]));
  __syncwarp();
  __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(out);
  if (w.vec) {
    const int q = lane & 3, n = w.n0 + 8 * q;
    __nv_bfloat16* p = o + (size_t)(w.m0 + (lane >> 2)) * w.ld + n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      const uint4 x = *stg16(stg, r, q);
      if (w.m0 + r < w.M && n < w.N) *reinterpret_cast<uint4*>(p + (size_t)(8 * i) * w.ld) = x;
    }
  } else {
    const int n = w.n0 + lane, rows = min(32, w.M - w.m0);
    unsigned short* p = reinterpret_cast<unsigned short*>(o) + (size_t)w.m0 * w.ld + n;
    if (n < w.N) {
#pragma unroll 8
      for (int r = 0; r < rows; ++r, p += w.ld) *p = reinterpret_cast<const unsigned short*>(stg16(stg, r, lane >> 3))[lane & 7];
    }
  }
  __syncwarp();
}
// The residual's elements that this lane will add (requested before the
// accumulator is read): four of each of eight rows, unconverted.
struct ResidualVec {
  uint4 r[8];
  template <typename T>
  __device__ __forceinline__ void load(const void* res, const Window& w, int lane) {
    const int n = w.n0 + 4 * (lane & 7);
    const T* p = reinterpret_cast<const T*>(res) + (size_t)(w.m0 + (lane >> 3)) * w.ld + n;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (w.m0 + 4 * i + (lane >> 3) >= w.M || n >= w.N) continue;
      if constexpr (sizeof(T) == 4) {
        r[i] = *reinterpret_cast<const uint4*>(p + (size_t)(4 * i) * w.ld);
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(p + (size_t)(4 * i) * w.ld);
        r[i].x = x.x, r[i].y = x.y;
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void get(int i, float (&z)[4]) const {
    if constexpr (sizeof(T) == 4) {
      z[0] = __uint_as_float(r[i].x), z[1] = __uint_as_float(r[i].y), z[2] = __uint_as_float(r[i].z), z[3] = __uint_as_float(r[i].w);
    } else {
      z[0] = bf16_lo(r[i].x), z[1] = bf16_hi(r[i].x), z[2] = bf16_lo(r[i].y), z[3] = bf16_hi(r[i].y);
    }
  }
};
// v (+ residual) as T.
template <typename T>
__device__ __forceinline__ void out_stream(const float (&v)[32], void* out, const void* res, const ResidualVec& rv,
                                           const Window& w, uint8_t* stg, int lane) {
#pragma unroll
  for (int q = 0; q < 8; ++q) *stg32(stg, lane, q) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  __syncwarp();
  T* o = reinterpret_cast<T*>(out);
  if (w.vec) {
    const int q = lane & 7, n = w.n0 + 4 * q;
    T* p = o + (size_t)(w.m0 + (lane >> 3)) * w.ld + n;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      const float4 x = *stg32(stg, r, q);
      float y[4] = {x.x, x.y, x.z, x.w};
      if (w.m0 + r < w.M && n < w.N) {
        if (res) {
          float z[4];
          rv.get<T>(i, z);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] += z[j];
        }
        store_to<4>(p + (size_t)(4 * i) * w.ld, y);
      }
    }
  } else {
    const int n = w.n0 + lane, rows = min(32, w.M - w.m0);
    T* p = o + (size_t)w.m0 * w.ld + n;
    const T* pr = reinterpret_cast<const T*>(res) + (size_t)w.m0 * w.ld + n;
    if (n < w.N) {
      for (int r0 = 0; r0 < rows; r0 += 8) {
        Raw<T, 1> z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          z[i].zero();
          if (res && r0 + i < rows) z[i].load(pr + (size_t)(r0 + i) * w.ld);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float y[1];
          z[i].get(y);
          y[0] += reinterpret_cast<const float*>(stg32(stg, r0 + i, lane >> 2))[lane & 3];
          if (r0 + i < rows) store_to<1>(p + (size_t)(r0 + i) * w.ld, y);
        }
      }
    }
  }
  __syncwarp();
}
// In the operands' type, no residual.
template <bool F32>
__device__ __forceinline__ void out_same(const float (&v)[32], void* out, const Window& w, uint8_t* stg, int lane) {
  if constexpr (F32) {
    const ResidualVec none{};
    out_stream<float>(v, out, nullptr, none, w, stg, lane);
  } else {
    out_bf16(v, out, w, stg, lane);
  }
}
// Adds bias[n0 ..] to 32 columns (all lanes read the same words).
__device__ __forceinline__ void add_bias(float (&v)[32], const float* bias, int n0, int N, int vec) {
  if (!bias) return;
  if (vec && n0 + 32 <= N) {
    float4 b[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) b[q] = __ldg(reinterpret_cast<const float4*>(bias + n0) + q);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[4 * q] += b[q].x, v[4 * q + 1] += b[q].y, v[4 * q + 2] += b[q].z, v[4 * q + 3] += b[q].w;
  } else {
    float b[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) b[j] = n0 + j < N ? __ldg(bias + n0 + j) : 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += b[j];
  }
}

// Whether any thread of the epilogue warps says so (and a barrier of them).
__device__ __forceinline__ bool epi_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "n"(32 * kEpiWarps)
      : "memory");
  return r != 0;
}

// ---- fp32 operands as bf16 parts: x = hi + mid + lo, each the nearest bf16 of
// what the ones before leave, exact from 2^-110 in magnitude (3 x 8 bits; below,
// the last bits of lo would be under bf16's smallest).  Six of the nine products are
// taken; the other three together reach 2^-24 of the exact one (mid is up to
// 2^-8 of the operand, lo 2^-17).  What rounds to an infinite hi has no other
// parts (an infinity times a zero part still makes NaN of an infinite
// operand's row or column).
struct Feed {
  int it = 0, st = 0;
  uint32_t phase = 0;
};
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf16(x, y);
  float a = x - bf16_lo(hi), b = y - bf16_hi(hi);
  a = fabsf(a) <= 3.4e38f ? a : 0.f;
  b = fabsf(b) <= 3.4e38f ? b : 0.f;
  mid = pack_bf16(a, b);
  lo = pack_bf16(a - bf16_lo(mid), b - bf16_hi(mid));
}
// Eight elements [col, col + 8) of a row, zero outside the matrix.  VEC: rows
// start on 16 bytes and hold whole vectors (nothing here may touch what is loaded:
// it would wait for the load).
template <bool VEC>
__device__ __forceinline__ void fetch8_f32(const OpMat& m, int row, int col, float4& x, float4& y) {
  x = y = make_float4(0.f, 0.f, 0.f, 0.f);
  if (row >= m.outer || col >= m.inner) return;
  const float* p = reinterpret_cast<const float*>(m.p) + (size_t)row * m.ld + col;
  if constexpr (VEC) {
    const int n = m.inner - col;
    x = reinterpret_cast<const float4*>(p)[0];
    if (n > 4) y = reinterpret_cast<const float4*>(p)[1];
  } else {
    const int n = m.inner - col;
    x.x = p[0];
    if (n > 1) x.y = p[1];
    if (n > 2) x.z = p[2];
    if (n > 3) x.w = p[3];
    if (n > 4) y.x = p[4];
    if (n > 5) y.y = p[5];
    if (n > 6) y.z = p[6];
    if (n > 7) y.w = p[7];
  }
}
__device__ __forceinline__ bool vec_f32(const OpMat& m) {
  return ((reinterpret_cast<uintptr_t>(m.p) & 15) | (m.ld & 3) | (m.inner & 3)) == 0;
}
// k-blocks [lo, hi) of a 128 x BN tile: 256 threads, 16-byte chunks of the
// swizzled tiles; the next block's elements are requested as soon as the
// present ones are on their way to shared memory.  (VA, VB: fetch8_f32's VEC of either operand;
// parameters, so that the loop holds one kind of load: its instructions have to stay in the cache.)
template <int BN, bool VA, bool VB>
__device__ __forceinline__ void feed_f32(const ProductK& P, int m0, int n0, int lo, int hi, int te, uint8_t* smem, int sbytes,
                                         int stages, uint64_t* full, uint64_t* empty, Feed& f, unsigned* status,
                                         volatile int* abort) {
  constexpr int NA = 4, NB = BN / 32, PB = BN * BK * 2;
  const bool amn = P.a_mn, bmn = P.b_mn, gated = P.gated;
  const int kb0 = P.kb0;
  float4 v[NA + NB][2];
  auto load = [&](int kb) {
    const int q = kb >= kb0 ? 1 : 0, kk = (kb - (q ? kb0 : 0)) * BK;
    const OpMat A = P.a[q], B0 = P.b[gated ? 0 : q], B1 = P.b[gated ? 1 : q];
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int c = te + i * 256, r = c >> 3, k = (c & 7) * 8;
      if (amn)
        fetch8_f32<VA>(A, kk + (r & 63), m0 + (r >> 6) * 64 + k, v[i][0], v[i][1]);
      else
        fetch8_f32<VA>(A, m0 + r, kk + k, v[i][0], v[i][1]);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int c = te + i * 256, r = c >> 3, k = (c & 7) * 8;
      if (bmn)
        fetch8_f32<VB>(B0, kk + (r & 63), n0 + (r >> 6) * 64 + k, v[NA + i][0], v[NA + i][1]);
      else if (gated)
        fetch8_f32<VB>(r < BN / 2 ? B0 : B1, n0 + r % (BN / 2), kk + k, v[NA + i][0], v[NA + i][1]);
      else
        fetch8_f32<VB>(B0, n0 + r, kk + k, v[NA + i][0], v[NA + i][1]);
    }
  };
  load(lo);
  for (int kb = lo; kb < hi; ++kb, ++f.it) {
    if (f.it >= stages && !__all_sync(0xffffffffu, mbar_wait(&empty[f.st], f.phase ^ 1, status, kStatusTimeoutTmaEmpty, abort)))
      return;
    uint8_t* st = smem + (size_t)f.st * sbytes;
#pragma unroll
    for (int i = 0; i < NA + NB; ++i) {
      const int c = te + (i < NA ? i : i - NA) * 256, r = c >> 3;
      uint8_t* d = st + (i < NA ? 0 : 3 * kABytes) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
      const int plane = i < NA ? kABytes : PB;
      const float4 x = v[i][0], y = v[i][1];
      uint4 h, m, l;
      split2(x.x, x.y, h.x, m.x, l.x);
      split2(x.z, x.w, h.y, m.y, l.y);
      split2(y.x, y.y, h.z, m.z, l.z);
      split2(y.z, y.w, h.w, m.w, l.w);
      *reinterpret_cast<uint4*>(d) = h;
      *reinterpret_cast<uint4*>(d + plane) = m;
      *reinterpret_cast<uint4*>(d + 2 * plane) = l;
    }
    if (kb + 1 < hi) load(kb + 1);
    fence_proxy_async_smem();
    __syncwarp();
    if ((te & 31) == 0) mbar_arrive(&full[f.st]);
    if (++f.st == stages) f.st = 0, f.phase ^= 1;
  }
}


template <int CG, int MODE>
__global__ void __launch_bounds__(MODE == kManual ? kThreads + kLoaders : kThreads, 1) op_gemm_kernel(const __grid_constant__ GemmArgs g) {
  constexpr bool F32 = MODE == kF32, TMA = MODE == kTma;
  static_assert(CG == 1 || TMA, "loads by threads serve single CTAs");
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {  // the swizzle is a function of the address bits
    if (threadIdx.x == 0) atomicOr(&g_op_status, kStatusTimeoutDrain);
    return;
  }
  const int stages = g.stages, sbytes = g.stage_bytes;
  uint8_t* sStg = smem + (size_t)stages * sbytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sStg + kEpiWarps * kStg);
  uint64_t* empty = full + kMaxStages;
  uint64_t* accf = empty + kMaxStages;
  uint64_t* acce = accf + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  unsigned* status = &g_op_status;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int S = g.split;
  const uint32_t rank = (CG == 2 || S > 1) ? cluster_rank() : 0u;
  const int unit = CG == 2 ? (int)(blockIdx.x >> 1) : (int)blockIdx.x / S;
  const int units = CG == 2 ? (int)(gridDim.x >> 1) : (int)gridDim.x / S;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], TMA ? 1 : MODE == kManual ? kLoaders / 32 : kEpiWarps);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], CG == 2 && rank == 0 ? 2 * kEpiWarps : kEpiWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0 && TMA) {
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
  // Accumulator buffers.  Where the output is fp32 a tile's reduction goes through
  // segments (the tensor core's additions truncate, which a long chain would
  // show): each fills a buffer of its own, and the epilogue warps add them up
  // while the next one runs.  fp32 operands: up to nseg segments, and the small
  // products, lie side by side in one; a longer reduction takes several such
  // rounds, added up the same way.
  const int nbuf = g.nbuf, nseg = g.nseg, buf_cols = g.buf_cols;
  pdl_trigger();

  // k-blocks of this CTA's part of a tile
  auto k_lo = [&](const ProductK& P, int piece) {
    return S > 1 ? share_begin(P.kb, rank, S) : share_begin(P.kb, piece, P.pieces);
  };
  auto k_hi = [&](const ProductK& P, int piece) {
    return S > 1 ? share_begin(P.kb, rank + 1, S) : share_begin(P.kb, piece + 1, P.pieces);
  };
  auto segments = [&](const ProductK& P, int lo, int hi) {
    return segments_of(lo, hi, P.kb0, g.subs, P.chain);
  };

  if (warp == 0) {
    if (TMA && elect_one()) {
      const bool peer = CG == 2 && rank == 1;
      int it = 0, st = 0;  // stages filled; the next one and its phase
      uint32_t phase = 0;
      // a pair's stage completes on rank 0's barrier, for both CTAs' bytes
      const uint32_t full0 = CG == 2 ? cluster_addr(full, 0) : 0u;
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
        const int bbytes = brows * BK * 2, subs = g.subs;
        const int lo = k_lo(P, tl.piece), hi = k_hi(P, tl.piece), kb0 = P.kb0;
        for (int q = 0; q < 2 && ok; ++q) {  // operand pairs
          const CUtensorMap* ma = &P.ma[q];
          const CUtensorMap* mb = gated && CG == 2 ? &P.mb[rank] : &P.mb[q];
          const CUtensorMap* mb1 = &P.mb[1];
          const int end = q ? hi : min(hi, kb0);
          for (int kb = q ? max(lo, kb0) : lo; kb < end; ++it) {
            if (it >= stages && !mbar_wait(&empty[st], phase ^ 1, status, kStatusTimeoutTmaEmpty, abort_flag)) {
              ok = false;
              break;
            }
            const int ns = stage_blocks(kb, end, end, subs);
            // (a reduction-outermost box brings the rows of a whole stage)
            if (!peer)
              mbar_arrive_expect_tx(&full[st], (uint32_t)(kABytes * (amn ? subs : ns) + bbytes * (bmn ? subs : ns)) * CG);
            uint8_t* sa = smem + (size_t)st * sbytes;
            uint8_t* sb = sa + subs * kABytes;
            const uint32_t bar = full0 + 8 * st;
            auto load = [&](const CUtensorMap* map, uint8_t* dst, int x, int y) {
              if (CG == 2)
                tma_load_3d_pair(dst, map, bar, x, y, 0);
              else
                tma_load_3d(dst, map, &full[st], x, y, 0);
            };
            const int k0 = (q ? kb - kb0 : kb) * BK;
            if (amn) {
              load(ma, sa, m0, k0);
              load(ma, sa + subs * 8192, m0 + 64, k0);
            } else {
              for (int i = 0; i < ns; ++i) load(ma, sa + i * kABytes, k0 + i * BK, m0);
            }
            if (bmn) {
              for (int j = 0; j < brows; j += 64) load(mb, sb + subs * j * 128, n0 + j, k0);
            } else {
              for (int i = 0; i < ns; ++i) {
                load(mb, sb + i * bbytes, k0 + i * BK, n0);  // gated: g's rows, then u's (a pair: one CTA each)
                if (CG == 1 && gated) load(mb1, sb + i * bbytes + bbytes / 2, k0 + i * BK, n0);
              }
            }
            kb += ns;
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
    if (rank * (CG - 1) == 0 && elect_one()) {
      const int subs = g.subs;
      const uint32_t smem0 = smem_u32(smem);
      int st = 0, buf = 0, lt = 0;
      uint32_t phase = 0, bphase = 0;
      bool ok = true;
      for (int t = unit; t < g.tiles && ok; t += units) {  // lt: buffers filled
        const Tile tl = tile_at(g, t);
        const ProductK& P = g.p[tl.p];
        if (lt >= nbuf && !mbar_wait(&acce[buf], bphase ^ 1, status, kStatusTimeoutAccum, abort_flag)) break;
        tc_fence_after();
        const bool amn = P.a_mn, bmn = P.b_mn;
        const uint32_t bn = P.bn;
        const uint32_t idesc = idesc_bf16_f32(BM * CG, bn) | (amn ? 1u << 15 : 0u) | (bmn ? 1u << 16 : 0u);
        const uint64_t sa = amn ? 2048 >> 4 : 32 >> 4, sb = bmn ? 2048 >> 4 : 32 >> 4;  // descriptor step per K = 16
        const uint64_t da0 = smem_desc(0, amn, subs), db0 = smem_desc(0, bmn, subs);
        // bytes from one k-block of a stage to the next
        const uint32_t a_sub = amn ? 8192 : kABytes, b_sub = bmn ? 8192 : bn / CG * BK * 2;
        const int lo = k_lo(P, tl.piece), hi = k_hi(P, tl.piece), kb0 = P.kb0, per = segments(P, lo, hi).per;
        uint32_t d = tmem + buf * buf_cols;
        int in = 0, segst = 0;  // k-blocks and stages in the present segment
        int slot = 0;           // fp32 operands: the segment's place in its round
        for (int kb = lo; kb < hi;) {
          if (kb > lo && in == 0 && slot == 0) {  // the next segment's (round's) buffer is drained
            if (lt >= nbuf && !mbar_wait(&acce[buf], bphase ^ 1, status, kStatusTimeoutAccum, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            d = tmem + buf * buf_cols;
          }
          if (!mbar_wait(&full[st], phase, status, kStatusTimeoutTmaFull, abort_flag)) {
            ok = false;
            break;
          }
          if constexpr (F32) {
            // parts: A hi, mid, lo, then B's.  hi hi goes to the segment's
            // accumulator, the five smaller products to the last one, whose
            // truncations are 2^-8 of the others'.
            const uint32_t a0 = smem0 + (uint32_t)(st * sbytes), pb = bn * BK * 2;
            const uint32_t dx = tmem + nseg * bn;
            auto mma = [&](int i, int j, uint32_t to, uint32_t acc0) {
              const uint64_t da = da0 | ((a0 + i * kABytes) >> 4 & 0x3FFF);
              const uint64_t db = db0 | ((a0 + 3 * kABytes + j * pb) >> 4 & 0x3FFF);
#pragma unroll
              for (int k = 0; k < BK / 16; ++k) tc_mma_bf16(to, da + k * sa, db + k * sb, idesc, k > 0 ? 1u : acc0);
            };
            mma(0, 0, d, in > 0);
            mma(0, 2, dx, in > 0 || slot > 0);
            mma(2, 0, dx, 1);
            mma(1, 1, dx, 1);
            mma(0, 1, dx, 1);
            mma(1, 0, dx, 1);
            ++in, ++kb;
          } else {
            const int ns = stage_blocks(kb, hi, kb0, subs);
            uint32_t a0 = smem0 + (uint32_t)(st * sbytes), b0 = a0 + subs * kABytes;
            for (int i = 0; i < ns; ++i, ++kb, a0 += a_sub, b0 += b_sub) {
              // (the address field is 14 bits: in a cluster, shared addresses carry the CTA's rank above them)
              const uint64_t da = da0 | (a0 >> 4 & 0x3FFF), db = db0 | (b0 >> 4 & 0x3FFF);
#pragma unroll
              for (int k = 0; k < BK / 16; ++k) {
                const uint32_t acc = (in > 0 || k > 0) ? 1u : 0u;
                if constexpr (CG == 2)
                  tc_mma_bf16_pair(d, da + k * sa, db + k * sb, idesc, acc);
                else
                  tc_mma_bf16(d, da + k * sa, db + k * sb, idesc, acc);
              }
              ++in;
            }
          }
          ++segst;
          if constexpr (CG == 2)
            tc_commit_both(smem_u32(&empty[st]));
          else
            tc_commit(&empty[st]);
          if (++st == stages) st = 0, phase ^= 1;
          bool last = kb >= hi;  // of the buffer
          if (segst == per) {
            in = segst = 0;
            if constexpr (F32) {
              d += bn;
              last |= ++slot == nseg;
            } else {
              last = true;
            }
          }
          if (last) {
            if constexpr (CG == 2)
              tc_commit_both(smem_u32(&accf[buf]));
            else
              tc_commit(&accf[buf]);
            if (++buf == nbuf) buf = 0, bphase ^= 1;
            ++lt;
            in = segst = slot = 0;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp < 2 + kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    pdl_wait();
    const int quad = warp & 3, half = (warp - 2) >> 2, te = threadIdx.x - 64;
    for (int i = 0; i < g.n_sums; ++i) {
      const OpColSum cs = g.sums[i];
      for (int c = blockIdx.x * 256 + te; c < cs.cols; c += gridDim.x * 256) {
        float a = 0.f;
#pragma unroll 16
        for (int r = 0; r < cs.rows; ++r) a += cs.part[(size_t)r * cs.cols + c];
        cs.out[c] = a;
      }
    }
    uint8_t* stg = sStg + (warp - 2) * kStg;
    int buf = 0;
    uint32_t bphase = 0;
    Feed feed;
    for (int t = unit; t < g.tiles; t += units) {
      const Tile tl = tile_at(g, t);
      const ProductK& P = g.p[tl.p];
      OpEpi e = P.e;
      if (tl.piece) e.out = reinterpret_cast<float*>(e.out) + (size_t)tl.piece * P.M * e.ld;
      const int bn = P.bn, pM = P.M, pN = P.N;
      const bool gated = P.gated;
      const int m0 = (tl.m * CG + (CG == 2 ? (int)rank : 0)) * BM;
      const int n0 = tl.n * (gated ? bn / 2 : bn);
      const int k_first = k_lo(P, tl.piece), k_end = k_hi(P, tl.piece);
      const Segments sg = segments(P, k_first, k_end);
      const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
      const int mw = m0 + quad * 32;
      auto ready = [&] {  // the present buffer is complete (one decision for all warps)
        const bool ok = mbar_wait(&accf[buf], bphase, status, kStatusTimeoutAccum, abort_flag);
        const bool stop = epi_any(!ok || *abort_flag);
        if (stop) *abort_flag = 1;
        // (behind the barrier too: a gated tile of 64 columns has its u from sums that the quarter's other warp wrote)
        tc_fence_after();
        return !stop;
      };
      auto drained = [&] {  // this warp's reads of the accumulator are done
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2 && rank == 1)
            mbar_arrive_cluster(cluster_addr(&acce[buf], 0));
          else
            mbar_arrive(&acce[buf]);
        }
      };
      // all but the last segment (fp32 operands: round): summed in tensor memory,
      // behind the buffers (in registers the sums took those of the rest of the
      // epilogue)
      const uint32_t t_sum = t_lane + (F32 ? (nseg + 1) * bn : nbuf * buf_cols);
      const int fills = F32 ? (sg.count + nseg - 1) / nseg : sg.count;  // of a buffer
      int held = 1;  // segments in the present buffer
      // 32 columns of the present buffer, with those of the buffers before
      auto acc32 = [&](int c, bool before, float (&v)[32]) {
        const uint32_t t_row = t_lane + buf * buf_cols;
        float w[32];
        tmem_ld32(t_row + c, v);
        if constexpr (F32) {
#pragma unroll 1
          for (int k = 0; k < held; ++k) {  // the small products, the other segments
            tmem_ld32(t_row + (k ? k : nseg) * bn + c, w);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += w[i];
          }
        }
        if (before) {
          tmem_ld32(t_sum + c, w);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] += w[i];
        }
      };
      bool stop = false;
      for (int k = 0;; ++k) {
        if constexpr (F32) {  // these warps bring the operands in first
          held = min(nseg, sg.count - k * nseg);
          const bool va = vec_f32(P.a[0]) && vec_f32(P.a[1]), vb = vec_f32(P.b[0]) && vec_f32(P.b[1]);
          const int lo = k_first + k * nseg * sg.per, hi = min(k_end, lo + nseg * sg.per);
#define WAM_FEED(BN, VA, VB) \
  feed_f32<BN, VA, VB>(P, m0, n0, lo, hi, te, smem, sbytes, stages, full, empty, feed, status, abort_flag)
          if (bn == 128) {
            if (va)
              vb ? WAM_FEED(128, true, true) : WAM_FEED(128, true, false);
            else
              vb ? WAM_FEED(128, false, true) : WAM_FEED(128, false, false);
          } else {
            if (va)
              vb ? WAM_FEED(64, true, true) : WAM_FEED(64, true, false);
            else
              vb ? WAM_FEED(64, false, true) : WAM_FEED(64, false, false);
          }
#undef WAM_FEED
        }
        stop = !ready();
        if (stop || k + 1 == fills) break;
#pragma unroll 1
        for (int c = 32 * half; c < bn; c += 64) {
          float w[32];
          acc32(c, k > 0, w);
          tmem_st32f(t_sum + c, w);
        }
        drained();
        if (++buf == nbuf) buf = 0, bphase ^= 1;
      }
      if (stop) break;
      const uint32_t t_row = t_lane + buf * buf_cols;
      if (S > 1) {
        // leave the partial tile in the idle operand ring, chunk q of row r at q ^ (r & 7)
        if (mw < pM) {
          const int r = quad * 32 + lane;
          uint8_t* row = smem + (size_t)r * bn * 4;
          for (int c = 32 * half; c < bn; c += 64) {
            float v[32];
            acc32(c, fills > 1, v);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<float4*>(row + ((((c >> 2) + q) ^ (r & 7)) << 4)) =
                  make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          }
        }
        break;  // one tile per cluster; the rest after the cluster barrier
      }
      // 32 output columns at a time: everything but the residual in registers
      // (a row per lane), then through the staging
      const int width = gated ? bn / 2 : bn;
      if (32 * half >= width) drained();  // (a 32-column tile: nothing for the second half)
      for (int c = 32 * half; c < width; c += 64) {
        Window w{mw, pM, n0 + c, pN, e.ld, e.vec};
        const bool live = mw < pM && n0 + c < pN;
        float v[32];
        if (gated) {
          float u[32];
          if constexpr (F32) {
            acc32(c, fills > 1, v);
            acc32(bn / 2 + c, fills > 1, u);
          } else {  // (its output is never fp32: one segment)
            tmem_ld32(t_row + c, v);
            tmem_ld32(t_row + bn / 2 + c, u);
          }
          if (c + 64 >= width) drained();
          if (!live) continue;
          add_bias(v, e.bias, w.n0, pN, e.vec);
          add_bias(u, e.bias2, w.n0, pN, e.vec);
          if (e.z) {
            out_same<F32>(v, e.z, w, stg, lane);
            out_same<F32>(u, e.z2, w, stg, lane);
          }
          act_apply<!F32, 32>(e.act, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] *= u[j];
          out_same<F32>(v, e.out, w, stg, lane);
        } else {
          ResidualVec rv;
          if (e.res && live && e.vec) {
            if (F32 || e.out_f32)
              rv.load<float>(e.res, w, lane);
            else
              rv.load<__nv_bfloat16>(e.res, w, lane);
          }
          acc32(c, fills > 1, v);
          if (c + 64 >= width) drained();
          if (!live) continue;
          add_bias(v, e.bias, w.n0, pN, e.vec);
          if (e.z) out_same<F32>(v, e.z, w, stg, lane);
          act_apply<!F32, 32>(e.act, v);
          if (F32 || e.out_f32)
            out_stream<float>(v, e.out, e.res, rv, w, stg, lane);
          else if (e.res)
            out_stream<__nv_bfloat16>(v, e.out, e.res, rv, w, stg, lane);
          else
            out_bf16(v, e.out, w, stg, lane);
        }
      }
      if (++buf == nbuf) buf = 0, bphase ^= 1;
    }
  } else if (MODE == kManual) {
    // ------------------------------------------------------------- loaders
    pdl_wait();
    const int tl_ = threadIdx.x - kThreads;
    int it = 0, s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = unit; t < g.tiles && ok; t += units) {
      const Tile tl = tile_at(g, t);
      const ProductK& P = g.p[tl.p];
      const int m0 = tl.m * BM, n0 = tl.n * (P.gated ? P.bn / 2 : P.bn);
      const int hi = k_hi(P, tl.piece);
      for (int kb = k_lo(P, tl.piece); kb < hi; ++kb, ++it) {
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
    if (warp >= 2 && warp < 2 + kEpiWarps && !*abort_flag) {
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
          finish_split<F32, true, 4>(e, P.bn, P.N, base, S, te, 32 * kEpiWarps, r_lo, r_hi, m0, n0);
        else
          finish_split<F32, true, 1>(e, P.bn, P.N, base, S, te, 32 * kEpiWarps, r_lo, r_hi, m0, n0);
      } else {
        if (e.vec)
          finish_split<F32, false, 8>(e, P.bn, P.N, base, S, te, 32 * kEpiWarps, r_lo, r_hi, m0, n0);
        else
          finish_split<F32, false, 1>(e, P.bn, P.N, base, S, te, 32 * kEpiWarps, r_lo, r_hi, m0, n0);
      }
    }
  }

  // ------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  // The epilogue has seen the last commit of every buffer.  After a wait that
  // gave up it may not have: then the commits are waited for (again with a limit)
  // before the tensor memory is freed.
  if (warp == 1) {
    if (lane == 0 && *abort_flag) {
      int n = 0;
      for (int t = unit; t < g.tiles; t += units) {
        const Tile tl = tile_at(g, t);
        const ProductK& P = g.p[tl.p];
        const int segs = segments(P, k_lo(P, tl.piece), k_hi(P, tl.piece)).count;
        n += F32 ? (segs + nseg - 1) / nseg : segs;
      }
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
  std::mutex fill;
  int sms = 148;
  int clusters[9];  // clusters of n CTAs (one per SM) that run at once
};
Device g_dev[kMaxDevices];

cudaError_t device_info(Device** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  Device& d = g_dev[dev];
  std::unique_lock<std::mutex> lock(d.fill, std::defer_lock);
  if (!d.ready.load(std::memory_order_acquire)) lock.lock();
  if (lock.owns_lock() && !d.ready.load(std::memory_order_relaxed)) {
    int sms = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(op_gemm_kernel<1, kTma>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(op_gemm_kernel<2, kTma>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(op_gemm_kernel<1, kManual>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(op_gemm_kernel<1, kF32>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax)) != cudaSuccess)
      return e;
    for (int n = 1; n <= 8; ++n) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(sms / n * n);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = kSmemMax;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = n;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int c = 0;
      e = n == 2 ? cudaOccupancyMaxActiveClusters(&c, op_gemm_kernel<2, kTma>, &cfg)
                 : cudaOccupancyMaxActiveClusters(&c, op_gemm_kernel<1, kTma>, &cfg);
      if (e != cudaSuccess) return e;
      d.clusters[n] = std::max(1, std::min(c, sms / n));
    }
    d.sms = sms;
    d.ready.store(1, std::memory_order_release);
  }
  *out = &d;
  return cudaSuccess;
}

struct Plan {
  int cg, bn, split;
  int seg;  // accumulator segments (the most of any product)
  int sum = 0;  // fp32 operands: the segments come in rounds of seg, which are added up
};

int ceil_div(int a, int b) { return (a + b - 1) / b; }
// Accumulator columns of product p's tiles under plan width bn.
int tile_cols(const OpProduct& p, const Plan& pl, int mode) {
  return tile_columns(pl.bn, p.N, p.gated, p.b_mn, pl.cg == 2, mode == kF32);
}
int pieces_of(const OpProduct& p) { return std::max(1, p.pieces); }
// k-blocks of one of its tiles (the longest piece's)
int k_blocks(const OpProduct& p) { return ceil_div(std::max(1, p.pairs) * ceil_div(p.K, BK), pieces_of(p)); }

// Estimated ns of a plan, from measured parts: one k-block of a tile (all SMs
// busy, operands from L2), what follows a tile's last MMA, and the launch.
double plan_cost(const OpProduct* p, int n, const Plan& pl, const Device& d, int mode) {
  // a k-block: the tensor core and its operands, or the issue of its loads (115 ns each)
  auto per = [&](const OpProduct& q) {
    if (mode == kF32) return pl.bn == 128 ? 950.0 : 700.0;
    const double base = pl.cg == 2 ? 170 + 0.78 * pl.bn : pl.bn <= 128 ? 110 + 1.1 * pl.bn : 90 + 1.25 * pl.bn;
    const double subs = pl.bn / pl.cg <= 128 ? 2 : 1;
    const double loads = (q.a_mn ? 2 / subs : 1) + (q.b_mn ? pl.bn / pl.cg / 64 / subs : q.gated && pl.cg == 1 ? 2 : 1);
    return std::max(base, 115 * loads);
  };
  const double tail = 11.0 * pl.bn + 600 + (pl.cg == 2 ? 1000 : 0);
  if (pl.split > 1) {
    const OpProduct& q = p[0];
    const int bn = tile_cols(q, pl, mode), tn = ceil_div(q.gated ? 2 * q.N : q.N, bn), tm = ceil_div(q.M, BM);
    const int waves = ceil_div(tm * tn, d.clusters[pl.split]);
    return waves * (ceil_div(k_blocks(q), pl.split) * per(q) + tail + 2500);
  }
  const int units = pl.cg == 2 ? d.clusters[2] : d.sms;
  const bool bare = mode == kF32;  // one accumulator buffer: every tile's epilogue stands alone
  const double extra = bare ? tail : 150;
  if (n == 1) {
    const int bn = tile_cols(p[0], pl, mode), cols = p[0].gated ? 2 * p[0].N : p[0].N;
    const long long tiles = (long long)ceil_div(p[0].M, BM * pl.cg) * ceil_div(cols, bn) * pieces_of(p[0]);
    return (double)((tiles + units - 1) / units) * (k_blocks(p[0]) * per(p[0]) + extra) + tail;
  }
  // several products: the busiest unit's tiles
  double worst = 0;
  int first[kOpProducts];
  long long whole[kOpProducts], rest[kOpProducts], pos = 0;
  double c[kOpProducts];
  for (int i = 0; i < n; ++i) {
    const long long tiles = (long long)ceil_div(p[i].M, BM * pl.cg) *
                            ceil_div(p[i].gated ? 2 * p[i].N : p[i].N, tile_cols(p[i], pl, mode)) * pieces_of(p[i]);
    c[i] = k_blocks(p[i]) * per(p[i]) + extra;
    first[i] = (int)(pos % units);
    whole[i] = tiles / units;
    rest[i] = tiles % units;
    pos += tiles;
  }
  for (int u = 0; u < units; ++u) {
    double load = 0;
    for (int i = 0; i < n; ++i) {
      int off = u - first[i];
      if (off < 0) off += units;
      load += (whole[i] + (off < rest[i])) * c[i];
    }
    worst = std::max(worst, load);
  }
  return worst + tail;
}

Plan choose(const OpProduct* p, int n, int mode, const Device& d) {
  Plan best{1, 128, 1, 1};
  double bc = 1e30;
  int chain = 0;  // longest reduction that ends in fp32
  for (int i = 0; i < n; ++i)
    if (mode == kF32 || p[i].e.out_f32) chain = std::max(chain, k_blocks(p[i]));
  auto consider = [&](Plan pl) {
    pl.seg = std::max(1, segments_for(ceil_div(chain, pl.split), mode == kF32 ? kChainF32 : kChain));
    if (mode != kF32) {
      if (pl.seg > 1 && pl.bn > 160) return;  // (two buffers and the sums: no tensor memory for wider tiles)
    } else if (pl.seg > 512 / pl.bn - 1) {  // no tensor memory for so many: rounds, on the narrowest tile
      if (pl.bn > 64) return;
      pl.seg = 512 / pl.bn - 2;
      pl.sum = 1;
    }
    const double c = plan_cost(p, n, pl, d, mode);
    if (c < bc) bc = c, best = pl;
  };
  // Widths between the powers of two fill the SMs more evenly (1088 x 1536: 144
  // tiles of 96 columns, 26.6 us; 108 of 128, 27.9 us; both in a graph).  A
  // reduction-outermost operand takes a load per 64 columns, and they lose there
  // (2049 x 4111 x 1544 backward: 192 wide 103 us, 256 wide 94, pairs 77 us).
  const bool narrow = n == 1 && !p[0].gated && !p[0].b_mn;
  for (int bn = mode == kF32 ? 128 : 256; bn >= 64; bn -= 32) {  // (fp32: six parts of a wider tile leave no second stage)
    if ((bn & (bn - 1)) && (!narrow || mode == kF32)) continue;
    consider(Plan{1, bn, 1, 1});
    if (n > 1 || pieces_of(p[0]) > 1) continue;
    const int cols = tile_cols(p[0], Plan{1, bn, 1, 1}, mode);
    const long long tiles = (long long)ceil_div(p[0].M, BM) * ceil_div(p[0].gated ? 2 * p[0].N : p[0].N, cols);
    for (int s = 2; s <= 8; ++s)
      if (tiles <= d.clusters[s] && k_blocks(p[0]) >= 2 * s) consider(Plan{1, bn, s, 1});
  }
  if (mode == kTma) {
    consider(Plan{2, 256, 1, 1});
    if (narrow) consider(Plan{2, 192, 1, 1});  // (halves of 96 columns)
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

cudaError_t launch_op_gemm(const OpProduct* p, int n, bool f32, const OpColSum* sums, int n_sums, cudaStream_t s) {
  if (n < 1 || n > kOpProducts || n_sums < 0 || n_sums > 2) return cudaErrorInvalidValue;
  Device* d = nullptr;
  cudaError_t err = device_info(&d);
  if (err != cudaSuccess) return err;
  int mode = f32 ? kF32 : kTma;
  for (int i = 0; i < n; ++i) {
    const int na = p[i].pairs == 2 ? 2 : 1, nb = (p[i].pairs == 2 || p[i].gated) ? 2 : 1;
    for (int k = 0; k < na; ++k) if (!f32 && !tma_ok(p[i].a[k])) mode = kManual;
    for (int k = 0; k < nb; ++k) if (!f32 && !tma_ok(p[i].b[k])) mode = kManual;
  }
  const Plan pl = choose(p, n, mode, *d);
  GemmArgs g;
  int bmax = 0;
  for (int i = 0; i < n; ++i) bmax = std::max(bmax, tile_cols(p[i], pl, mode));
  const int sub_bytes = (kABytes + bmax / pl.cg * BK * 2) * (f32 ? 3 : 1), room = kSmemMax - kBarBytes - kEpiWarps * kStg;
  g.subs = mode == kTma && 6 * sub_bytes <= room ? 2 : 1;
  g.stage_bytes = g.subs * sub_bytes;
  g.stages = std::min(kMaxStages, room / g.stage_bytes);
  g.np = n;
  g.n_sums = n_sums;
  for (int i = 0; i < n_sums; ++i) g.sums[i] = sums[i];
  int tiles = 0;
  for (int i = 0; i < n; ++i) {
    const OpProduct& q = p[i];
    ProductK& k = g.p[i];
    k.M = q.M;
    k.N = q.N;
    k.kb = std::max(1, q.pairs) * ceil_div(q.K, BK);
    k.kb0 = ceil_div(q.K, BK);
    k.bn = tile_cols(q, pl, mode);
    k.tiles_m = ceil_div(q.M, BM * pl.cg);
    k.tiles_n = ceil_div(q.N, q.gated ? k.bn / 2 : k.bn);
    k.tile0 = tiles;
    k.pieces = std::max(1, q.pieces);
    k.chain = mode == kF32 ? kChainF32 : q.e.out_f32 ? kChain : 0;
    tiles += k.tiles_m * k.tiles_n * k.pieces;
    k.a_mn = q.a_mn;
    k.b_mn = q.b_mn;
    k.gated = q.gated;
    k.e = q.e;
    for (int j = 0; j < 2; ++j) {
      const OpMat& ma = q.a[q.pairs == 2 ? j : 0];
      const OpMat& mb = q.b[(q.pairs == 2 || q.gated) ? j : 0];
      k.a[j] = ma;
      k.b[j] = mb;
      if (mode != kTma) continue;
      const int boxb = q.b_mn ? 64 * g.subs : q.gated ? k.bn / 2 : k.bn / pl.cg;
      if (!make_tmap_rows(&k.ma[j], ma.p, ma.inner, ma.outer, ma.ld, q.a_mn ? 64 * g.subs : BM) ||
          !make_tmap_rows(&k.mb[j], mb.p, mb.inner, mb.outer, mb.ld, boxb))
        return cudaErrorInvalidValue;
    }
  }
  g.tiles = tiles;
  g.split = pl.split;
  g.nseg = pl.seg;
  g.nbuf = f32 ? 1 : 2;
  g.tm_cols = 32;
  g.buf_cols = bmax;
  while (g.tm_cols < (f32 ? pl.seg + 1 + pl.sum : pl.seg > 1 ? 3 : 2) * bmax) g.tm_cols *= 2;
  const size_t smem = (size_t)g.stages * g.stage_bytes + kEpiWarps * kStg + kBarBytes;

  const int cluster = pl.cg == 2 ? 2 : pl.split;
  const int units = pl.split > 1 ? tiles : std::min(tiles, pl.cg == 2 ? d->clusters[2] : d->sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units * cluster);
  cfg.blockDim = dim3(mode == kManual ? kThreads + kLoaders : kThreads);
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
  if (pl.cg == 2) return cudaLaunchKernelEx(&cfg, op_gemm_kernel<2, kTma>, g);
  if (mode == kManual) return cudaLaunchKernelEx(&cfg, op_gemm_kernel<1, kManual>, g);
  if (mode == kF32) return cudaLaunchKernelEx(&cfg, op_gemm_kernel<1, kF32>, g);
  return cudaLaunchKernelEx(&cfg, op_gemm_kernel<1, kTma>, g);
}

}  // namespace wam
