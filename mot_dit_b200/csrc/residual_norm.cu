// Gated residual with the norms on either side of it, both directions (sm_100a):
//   p = y or post_gain rms(y),  s = alpha x + gate p,
//   h = rms(s) gain (1 + scale) + shift,   rms(v) = v / sqrt(mean(v^2) + 1e-6).
// With n = s r, r = 1 / sqrt(mean(s^2) + eps), dn = dh gain (1 + scale):
//   dv = ds + r (dn - n mean(dn n)),  dx = alpha dv,  dp = gate dv,
//   dy = dp, or with q = y r_y: r_y (dp post_gain - q mean(dp post_gain q)),
// and the parameter gradients are column sums of dh n, dh and dv q.
//
// Bound by memory: forward 4, backward 6 row passes, each element read or
// written once (16896 x 1536, 1.965 GHz: 54.5 us, 0.87 of the copy rate; backward
// 84.6 us, 0.84; rows of 1537, which have no vector accesses, are bound by issue:
// 84 and 109 us).  A producer warp keeps a ring of row groups filled with
// asynchronous bulk copies (rows are contiguous, so a group is one span per
// matrix, widened to 16-byte granules: the ring takes any row length and
// alignment, and costs the row threads no registers).  A row's threads hold
// NV columns each; the column vectors of the block's sample stay in their
// registers.  The backward pass needs the mean of dp post_gain q, which depends
// on dv and so on the first means; it is expanded by linearity into three more
// sums of the same round, so that a row costs one block barrier: sum dv w y =
// sum w y ds + r sum w y dn - r^3 mean(dn s) sum w y s, w = gate post_gain.
// Column sums stay in registers over a block's rows (all of one sample), go to
// a partial array once, and a second kernel adds the partials in order: no
// atomics, the same bits every time.
#include <algorithm>
#include <type_traits>

#include "cluster.cuh"
#include "kernels.h"
#include "op_epilogue.cuh"
#include "row_plan.h"

namespace wam {
namespace {

constexpr float kEps = 1e-6f;

__device__ unsigned g_norm_status;

// Element j of thread t: groups of E consecutive elements, a row's threads
// side by side (E = 8 where 16-byte accesses may be used, else 1).
template <int E>
__device__ __forceinline__ int elem(int t, int tpr, int j) {
  return (t + (j / E) * tpr) * E + j % E;
}
// Elements [8 k, 8 k + 8) of this thread's columns of a row in shared memory
// (zero past its end).
template <int E, typename T>
__device__ __forceinline__ void row_get(const T* p, int D, int t, int tpr, int k, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += E) {
    const int i = elem<E>(t, tpr, 8 * k + j);
    Raw<T, E> r;
    r.zero();
    if (i < D) r.load(p + i);
    r.get(v + j);
  }
}
template <int E, typename T>
__device__ __forceinline__ void row_store(T* p, int D, int t, int tpr, int k, const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += E) {
    const int i = elem<E>(t, tpr, 8 * k + j);
    if (i < D) store_to<E>(p + i, v + j);
  }
}
// Elements [8 k, 8 k + 8) of this thread's columns of a vector (fill without one).
template <int E>
__device__ __forceinline__ void vec_get(const float* p, float fill, int D, int t, int tpr, int k, float (&v)[8]) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fill;
  } else if (E == 8 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    row_get<E>(p, D, t, tpr, k, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = elem<E>(t, tpr, 8 * k + j);
      v[j] = i < D ? p[i] : 0.f;
    }
  }
}
// The coefficients of this thread's columns: gain (1 + scale), shift, gate
// post_gain.  Eight columns: registers; more: shared memory behind the ring,
// where each thread keeps its own (no barrier).
template <int E, int NV>
struct Coef {
  float r[NV == 8 ? 3 : 1][8];
  float* s;
  int D, t, tpr;
  __device__ __forceinline__ Coef(uint8_t* smem, int D_, int t_, int tpr_)
      : s(reinterpret_cast<float*>(smem)), D(D_), t(t_), tpr(tpr_) {}
  __device__ __forceinline__ void put(int which, int k, const float (&v)[8]) {
    if constexpr (NV == 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[which][j] = v[j];
    } else {
      row_store<E>(s + which * ((D + 7) / 8 * 8), D, t, tpr, k, v);
    }
  }
  __device__ __forceinline__ void get(int which, int k, float (&v)[8]) const {
    if constexpr (NV == 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = r[which][j];
    } else {
      row_get<E>(s + which * ((D + 7) / 8 * 8), D, t, tpr, k, v);
    }
  }
  __device__ __forceinline__ void mul(int k, float (&v)[8]) const { get(0, k, v); }
  __device__ __forceinline__ void w(int k, float (&v)[8]) const { get(1, k, v); }
  __device__ __forceinline__ void add(int k, float (&v)[8]) const { get(2, k, v); }
  // Sample grp's coefficients (shift only where the forward's rows are formed).
  __device__ __forceinline__ void set(const ResNorm& a, int grp) {
    const size_t o = (size_t)grp * a.ld_mod;
#pragma unroll
    for (int k = 0; k < NV / 8; ++k) {
      float x[8], y[8];
      vec_get<E>(a.gain, 1.f, D, t, tpr, k, x);
      vec_get<E>(a.scale ? a.scale + o : nullptr, 0.f, D, t, tpr, k, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= 1.f + y[j];
      put(0, k, x);
      vec_get<E>(a.gate ? a.gate + o : nullptr, 1.f, D, t, tpr, k, x);
      vec_get<E>(a.post ? a.post_gain : nullptr, 1.f, D, t, tpr, k, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= y[j];
      put(1, k, x);
      if (!a.s) continue;
      vec_get<E>(a.shift ? a.shift + o : nullptr, 0.f, D, t, tpr, k, x);
      put(2, k, x);
    }
  }
};

// Two fp32 operations an instruction (the rows without vector accesses are
// bound by issue).
__device__ __forceinline__ unsigned long long bits2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split2f(unsigned long long v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
using f2 = unsigned long long;
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Barrier of the block's n row threads (the producer warp is not among them).
__device__ __forceinline__ void row_bar(int n) { asm volatile("bar.sync 1, %0;" ::"r"(n) : "memory"); }

// Sums of K (1 or 6) values over the threads of each row.  Within a warp the
// six are reduced together: each exchange halves what a lane carries (8, 4, 2,
// 1 values), so that it takes 9 shuffles and not 30.  Across warps: one
// barrier of the n row threads; `sh` holds [2][rows][warps][8], the halves taken in turn.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int t, int tpr, int ry, int rows, float* sh, int& phase, int n) {
  constexpr unsigned all = 0xffffffffu;
  if (tpr <= 32) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      for (int o = tpr / 2; o > 0; o >>= 1) v[k] += __shfl_xor_sync(all, v[k], o);
    return;
  }
  const int lane = t & 31, warp = t >> 5, warps = tpr >> 5;
  float* b = sh + (phase * rows + ry) * warps * 8;
  phase ^= 1;
  if constexpr (K == 1) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[0] += __shfl_xor_sync(all, v[0], o);
    if (lane == 0) b[warp * 8] = v[0];
    row_bar(n);
    float a = lane < warps ? b[lane * 8] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a += __shfl_xor_sync(all, a, o);
    v[0] = __shfl_sync(all, a, 0);
  } else {
    static_assert(K == 6, "1 or 6 values");
    float x[4], y[2], z;
    const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // lanes 16..31 keep values 4..7 (6, 7: none)
      const float lo = v[k], hi = k < 2 ? v[4 + k] : 0.f;
      x[k] = (h16 ? hi : lo) + __shfl_xor_sync(all, h16 ? lo : hi, 16);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) y[k] = (h8 ? x[2 + k] : x[k]) + __shfl_xor_sync(all, h8 ? x[k] : x[2 + k], 8);
    z = (h4 ? y[1] : y[0]) + __shfl_xor_sync(all, h4 ? y[0] : y[1], 4);
    z += __shfl_xor_sync(all, z, 2);
    z += __shfl_xor_sync(all, z, 1);
    if ((lane & 3) == 0) b[warp * 8 + (lane >> 2)] = z;  // lane bits 4, 3, 2 = the value's number
    row_bar(n);
    // lane: value lane % 8 of warps lane / 8, + 4, ...
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((lane >> 3) + 4 * i < warps) a += b[((lane >> 3) + 4 * i) * 8 + (lane & 7)];
    a += __shfl_xor_sync(all, a, 8);
    a += __shfl_xor_sync(all, a, 16);
#pragma unroll
    for (int k = 0; k < 6; ++k) v[k] = __shfl_sync(all, a, k);
  }
}

// ------------------------------------------------------------- the ring ----
struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  int abort;
};
__device__ __forceinline__ void bars_init(Bars& b, int stages, int warps) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&b.full[s], 1);
      mbar_init(&b.empty[s], warps);
    }
    b.abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
}
// Bytes [off, off + len) of a buffer of `total` bytes, as the 16-byte granules
// that hold them.  A granule that reaches past either end of the buffer is
// not read: its elements are copied one by one (`head` / `tail`).
struct Span {
  uintptr_t lo, hi;           // granules for the bulk copy
  uintptr_t head, head_end;   // bytes to copy singly
  uintptr_t tail, tail_end;
  uintptr_t at;               // the granule that lands at the stage's start
};
__device__ __forceinline__ Span span_of(const void* base, size_t total, size_t off, uint32_t len) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(base), a = b + off, e = a + len;
  Span s;
  s.at = s.lo = a & ~(uintptr_t)15;
  s.hi = (e + 15) & ~(uintptr_t)15;
  s.head = s.head_end = s.tail = s.tail_end = 0;
  if (s.lo < b) {
    s.lo += 16;
    s.head = a;
    s.head_end = s.lo < e ? s.lo : e;
  }
  if (s.hi > b + total && s.hi > s.lo) {
    s.hi -= 16;
    s.tail = s.hi > a ? s.hi : a;
    s.tail_end = e;
  }
  if (s.hi < s.lo) s.hi = s.lo;
  return s;
}
__device__ __forceinline__ void copy_ends(uint8_t* dst, const Span& s) {
  for (uintptr_t q = s.head; q < s.head_end; q += 2)
    *reinterpret_cast<unsigned short*>(dst + (q - s.at)) = *reinterpret_cast<const unsigned short*>(q);
  for (uintptr_t q = s.tail; q < s.tail_end; q += 2)
    *reinterpret_cast<unsigned short*>(dst + (q - s.at)) = *reinterpret_cast<const unsigned short*>(q);
}
// The producer warp: rows [lo, hi) of N matrices, R at a time; lane i deals
// with matrix i (one lane alone, with its 64-bit addresses, took longer than
// the rows' arithmetic).
template <int N>
__device__ __forceinline__ void produce(const void* base, int size, const Ring& ring, int M, int D, int lo, int hi, int R,
                                        uint8_t* smem, Bars& b) {
  const int lane = threadIdx.x & 31;
  const bool mine = lane < N && base;
  uint8_t* dst = smem + ring.off[lane < N ? lane : 0];
  const size_t total = (size_t)M * D * size, row = (size_t)D * size;
  int st = 0, it = 0;
  uint32_t phase = 0;
  for (int m = lo; m < hi; m += R, ++it) {
    if (it >= ring.stages && !__all_sync(0xffffffffu, mbar_wait(&b.empty[st], phase ^ 1, &g_norm_status,
                                                                kStatusTimeoutTmaEmpty, (volatile int*)&b.abort)))
      break;
    uint8_t* d = dst + (size_t)st * ring.stage_bytes;
    Span s{};
    if (mine) {
      s = span_of(base, total, m * row, (uint32_t)(min(R, hi - m) * row));
      copy_ends(d, s);
    }
    uint32_t bytes = (uint32_t)(s.hi - s.lo);
#pragma unroll
    for (int o = 1; o < N; o <<= 1) bytes += __shfl_xor_sync(0xffffffffu, bytes, o);
    __syncwarp();  // every lane's single elements are in place before the arrival that publishes them
    if (lane == 0) mbar_arrive_expect_tx(&b.full[st], bytes);
    __syncwarp();
    if (mine && s.hi > s.lo) bulk_load(d + (s.lo - s.at), reinterpret_cast<const void*>(s.lo), (uint32_t)(s.hi - s.lo), &b.full[st]);
    if (++st == ring.stages) st = 0, phase ^= 1;
  }
  // never leave with copies in flight
  if (lane == 0)
    for (int i = max(0, it - ring.stages); i < it; ++i)
      mbar_wait(&b.full[i % ring.stages], (i / ring.stages) & 1, &g_norm_status, kStatusTimeoutDrain, nullptr);
}
// Row `ry` of the group that starts at row m, in a stage.
template <typename T>
__device__ __forceinline__ const T* staged(const uint8_t* stage, int off, const void* base, int m, int D, int ry) {
  const uint32_t in = (uint32_t)((reinterpret_cast<uintptr_t>(base) + (size_t)m * D * sizeof(T)) & 15);
  return reinterpret_cast<const T*>(stage + off + in) + (size_t)ry * D;
}

// Block: n = tpr x R row threads and a producer warp; its rows are
// [M b / grid, M (b + 1) / grid).  RT / CT: the stream's and the compute type.
template <int E, int NV, bool SMALL, typename RT, typename CT>
__global__ void __launch_bounds__(SMALL ? 256 : NV == 24 ? 384 : 512, SMALL ? (E == 8 ? 3 : 2) : 1) res_norm_kernel(const ResNorm a, const Ring ring, int tpr, int R) {
  constexpr bool KEEP = NV == 8 || E == 8;  // the row in registers, else read from the ring for each pass
  constexpr int NK = KEEP ? NV / 8 : 1, kUnroll = KEEP ? NV / 8 : 1;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float sh[2 * 16 * 8];  // [2][rows][warps][8]: at most 16 warps in all
  __shared__ Bars bars;
  const int n = tpr * R, D = a.D;
  const int lo = (int)((long long)a.M * blockIdx.x / gridDim.x), hi = (int)((long long)a.M * (blockIdx.x + 1) / gridDim.x);
  bars_init(bars, ring.stages, n / 32);
  pdl_trigger();
  pdl_wait();
  if ((int)threadIdx.x >= n) {
    const bool first = threadIdx.x % 32 == 0;
    produce<2>(first ? a.x : a.y, first ? sizeof(RT) : sizeof(CT), ring, a.M, D, lo, hi, R, smem, bars);
    return;
  }
  const int ry = threadIdx.x / tpr, t = threadIdx.x - ry * tpr;
  int phase = 0, st = 0, next = lo + ry;  // (next: first row that needs other coefficients)
  uint32_t full_phase = 0;
  const float inv = 1.f / (float)D;
  Coef<E, NV> cf(smem + ring.stages * ring.stage_bytes, D, t, tpr);
  for (int m0 = lo; m0 < hi; m0 += R) {
    const int m = m0 + ry;
    const bool live = m < hi;  // (dead row lanes keep the barriers company)
    if (live && m >= next) {
      const int g = m / a.rows_per_group;
      cf.set(a, g);
      next = (g + 1) * a.rows_per_group;
    }
    // (a wait that gives up is reported; the rows go on, so that every barrier is met)
    mbar_wait(&bars.full[st], full_phase, &g_norm_status, kStatusTimeoutTmaFull, (volatile int*)&bars.abort);
    const uint8_t* stage = smem + (size_t)st * ring.stage_bytes;
    const RT* px = staged<RT>(stage, ring.off[0], a.x, m0, D, ry);
    const CT* py = staged<CT>(stage, ring.off[1], a.y, m0, D, ry);
    auto done = [&] {
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&bars.empty[st]);
      if (++st == ring.stages) st = 0, full_phase ^= 1;
    };
    const int Dl = live ? D : 0;
    float vv[NK][8], qq[NK][8];
    if (KEEP) {
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        row_get<E>(px, Dl, t, tpr, k, vv[k]);
        row_get<E>(py, Dl, t, tpr, k, qq[k]);
      }
      done();
    }
    float s1[1] = {0.f};
    float rp = 1.f;
    if (a.post) {
#pragma unroll kUnroll
      for (int k = 0; k < NV / 8; ++k) {
        float(&q)[8] = qq[KEEP ? k : 0];
        if (!KEEP) row_get<E>(py, Dl, t, tpr, k, q);
#pragma unroll
        for (int j = 0; j < 8; ++j) s1[0] += q[j] * q[j];
      }
      row_sum<1>(s1, t, tpr, ry, R, sh, phase, n);
      rp = rsqrtf(s1[0] * inv + kEps);
    }
    s1[0] = 0.f;
    auto stream = [&](int k) {  // v = alpha x + w (y r_y)
      float w[8], (&v)[8] = vv[KEEP ? k : 0], (&q)[8] = qq[KEEP ? k : 0];
      cf.w(k, w);
      if (!KEEP) {
        row_get<E>(px, Dl, t, tpr, k, v);
        row_get<E>(py, Dl, t, tpr, k, q);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = a.alpha * v[j] + w[j] * (q[j] * rp);
    };
#pragma unroll kUnroll
    for (int k = 0; k < NV / 8; ++k) {
      stream(k);
      const float(&v)[8] = vv[KEEP ? k : 0];
#pragma unroll
      for (int j = 0; j < 8; ++j) s1[0] += v[j] * v[j];
    }
    row_sum<1>(s1, t, tpr, ry, R, sh, phase, n);
    const float r = rsqrtf(s1[0] * inv + kEps);
#pragma unroll kUnroll
    for (int k = 0; k < NV / 8; ++k) {
      if (!KEEP) stream(k);
      if (!live) continue;
      float mul[8], add[8], (&v)[8] = vv[KEEP ? k : 0];
      cf.mul(k, mul);
      cf.add(k, add);
      row_store<E>(reinterpret_cast<RT*>(a.s) + (size_t)m * D, D, t, tpr, k, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * r * mul[j] + add[j];
      row_store<E>(reinterpret_cast<CT*>(a.h) + (size_t)m * D, D, t, tpr, k, v);
    }
    if (!KEEP) done();
  }
}

// Block: chunk blockIdx.x % chunks of the rows of sample blockIdx.x / chunks;
// n = tpr x R row threads and a producer warp.  Wide rows (NV > 8) are read from
// the ring twice, eight columns at a time, for their sums and for their
// gradients: the registers hold column sums instead.
template <int E, int NV, typename RT, typename CT>
__global__ void __launch_bounds__(NV == 24 ? 384 : 512) res_norm_grad_kernel(const ResNormGrad a, const Ring ring, int chunks, int tpr, int R) {
  constexpr bool KEEP = NV == 8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float sh[2 * 16 * 8];
  __shared__ Bars bars;
  const ResNorm& f = a.f;
  const int n = tpr * R, D = f.D;
  const int grp = blockIdx.x / chunks, ck = blockIdx.x % chunks, g_lo = grp * f.rows_per_group;
  const int g_n = min(f.rows_per_group, f.M - g_lo);
  const int lo = g_lo + (int)((long long)g_n * ck / chunks), hi = g_lo + (int)((long long)g_n * (ck + 1) / chunks);
  bars_init(bars, ring.stages, n / 32);
  pdl_trigger();
  pdl_wait();
  if ((int)threadIdx.x >= n) {
    const int i = threadIdx.x % 32;
    produce<4>(i == 0 ? f.x : i == 1 ? f.y : i == 2 ? a.dh : a.ds, i == 1 || i == 2 ? sizeof(CT) : sizeof(RT), ring, f.M, D, lo,
               hi, R, smem, bars);
    return;
  }
  const int ry = threadIdx.x / tpr, t = threadIdx.x - ry * tpr;
  int phase = 0, st = 0;
  uint32_t full_phase = 0;
  Coef<E, NV> cf(smem + ring.stages * ring.stage_bytes, D, t, tpr);
  cf.set(f, grp);
  f2 sa[NV / 2], sb[NV / 2], sq[NV / 2];
#pragma unroll
  for (int j = 0; j < NV / 2; ++j) sa[j] = sb[j] = sq[j] = bits2(0.f, 0.f);
  const float inv = 1.f / (float)D;
  for (int m0 = lo; m0 < hi; m0 += R) {
    const int m = m0 + ry;
    const bool live = m < hi;
    const int Dl = live ? D : 0;  // (a row lane past the chunk's end adds nothing)
    mbar_wait(&bars.full[st], full_phase, &g_norm_status, kStatusTimeoutTmaFull, (volatile int*)&bars.abort);
    const uint8_t* stage = smem + (size_t)st * ring.stage_bytes;
    const RT* ps = staged<RT>(stage, ring.off[0], f.x, m0, D, ry);
    const CT* py = staged<CT>(stage, ring.off[1], f.y, m0, D, ry);
    const CT* ph = staged<CT>(stage, ring.off[2], a.dh, m0, D, ry);
    const RT* pd = staged<RT>(stage, ring.off[3], a.ds, m0, D, ry);
    const int Dd = a.ds ? Dl : 0;
    f2 v2[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) v2[i] = bits2(0.f, 0.f);
    f2 s[4], y[4], dh[4], dv[4], mul[4], w[4];
    auto pack = [](const float(&f)[8], f2(&o)[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = bits2(f[2 * j], f[2 * j + 1]);
    };
    auto get = [&](int k) {
      float f[8];
      // (else each element's index and bounds test stays live over the rows, and
      // spills: 6000 x 4001, bf16 with an fp32 stream, 258 us; 224 us so)
      if (E == 1 && !KEEP) asm volatile("" : "+r"(cf.t));
      row_get<E>(ps, Dl, cf.t, tpr, k, f), pack(f, s);
      row_get<E>(ph, Dl, cf.t, tpr, k, f), pack(f, dh);
      row_get<E>(py, Dl, cf.t, tpr, k, f), pack(f, y);
      row_get<E>(pd, Dd, cf.t, tpr, k, f), pack(f, dv);
      cf.mul(k, f), pack(f, mul);
      cf.w(k, f), pack(f, w);
    };
    auto done = [&] {
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&bars.empty[st]);
      if (++st == ring.stages) st = 0, full_phase ^= 1;
    };
#pragma unroll 1
    for (int k = 0; k < NV / 8; ++k) {
      get(k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 dn = mul2(dh[j], mul[j]), wy = mul2(w[j], y[j]);
        v2[0] = fma2(s[j], s[j], v2[0]);
        v2[1] = fma2(dn, s[j], v2[1]);
        v2[2] = fma2(y[j], y[j], v2[2]);
        v2[3] = fma2(wy, dv[j], v2[3]);
        v2[4] = fma2(wy, dn, v2[4]);
        v2[5] = fma2(wy, s[j], v2[5]);
      }
    }
    float v[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      float a0, a1;
      split2f(v2[i], a0, a1);
      v[i] = a0 + a1;
    }
    if (KEEP) done();
    row_sum<6>(v, t, tpr, ry, R, sh, phase, n);
    const float r = rsqrtf(v[0] * inv + kEps);
    const float c = r * (r * (r * (v[1] * inv)));  // (r^3 alone leaves fp32's range at rows of 1e12, and r_y^2 / D at 1e17)
    const float rp = f.post ? rsqrtf(v[2] * inv + kEps) : 1.f;
    const float cy = f.post ? rp * (rp * (inv * (v[3] + r * v[4] - c * v[5]))) : 0.f;
    const f2 r2 = bits2(r, r), nc2 = bits2(-c, -c), rp2 = bits2(rp, rp), ncy2 = bits2(-cy, -cy), al2 = bits2(f.alpha, f.alpha);
#pragma unroll
    for (int k = 0; k < NV / 8; ++k) {
      if (!KEEP) get(k);
      float o0[8], o1[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 g = fma2(nc2, s[j], fma2(r2, mul2(dh[j], mul[j]), dv[j]));  // dv
        const int i = 4 * k + j;
        sa[i] = fma2(mul2(dh[j], s[j]), r2, sa[i]);
        sb[i] = add2(sb[i], dh[j]);
        sq[i] = fma2(g, mul2(y[j], rp2), sq[i]);
        split2f(mul2(rp2, fma2(ncy2, y[j], mul2(g, w[j]))), o1[2 * j], o1[2 * j + 1]);  // (rp = 1, cy = 0 without the norm)
        split2f(mul2(al2, g), o0[2 * j], o0[2 * j + 1]);
      }
      if (live) {
        row_store<E>(reinterpret_cast<RT*>(a.dx) + (size_t)m * D, D, cf.t, tpr, k, o0);
        row_store<E>(reinterpret_cast<CT*>(a.dy) + (size_t)m * D, D, cf.t, tpr, k, o1);
      }
    }
    if (!KEEP) done();
  }
  if (!a.part) return;
  float* part = a.part + (size_t)blockIdx.x * 3 * D;
  float fa[NV], fb[NV], fq[NV];
#pragma unroll
  for (int j = 0; j < NV / 2; ++j) {
    split2f(sa[j], fa[2 * j], fa[2 * j + 1]);
    split2f(sb[j], fb[2 * j], fb[2 * j + 1]);
    split2f(sq[j], fq[2 * j], fq[2 * j + 1]);
  }
  if (R == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = elem<E>(t, tpr, j);
      if (i < D) part[i] = fa[j], part[D + i] = fb[j], part[2 * D + i] = fq[j];
    }
    return;
  }
  // the row lanes' sums joined in the ring, which is idle: every row thread is
  // past its last stage, and so every copy has landed
  float* dyn = reinterpret_cast<float*>(smem);
  const int W = tpr * NV;
  row_bar(n);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float* d = dyn + (size_t)ry * 3 * W + elem<E>(t, tpr, j);
    d[0] = fa[j], d[W] = fb[j], d[2 * W] = fq[j];
  }
  row_bar(n);
  for (int i = threadIdx.x; i < 3 * D; i += n) {
    const int k = i / D, c = i % D;
    float x = 0.f;
    for (int r = 0; r < R; ++r) x += dyn[(size_t)r * 3 * W + k * W + c];
    part[i] = x;
  }
}

// Column sums from the partials: 32 columns x 32 lanes.  Fewer samples than
// lanes: 32 / groups lanes share each sample's chunks; more: each lane takes
// whole samples.
__global__ void __launch_bounds__(1024) res_norm_sum_kernel(const ResNormGrad a, int groups, int chunks) {
  __shared__ float sh[3][32][33];
  const ResNorm& f = a.f;
  const int tx = threadIdx.x, ty = threadIdx.y, D = f.D, d = blockIdx.x * 32 + tx;
  pdl_trigger();
  pdl_wait();
  const bool in = d < D;
  const float gain = in && f.gain ? f.gain[d] : 1.f, pg = in && f.post && f.post_gain ? f.post_gain[d] : 1.f;
  float tg = 0.f, tp = 0.f;  // dgain, dpost_gain
  auto emit = [&](int g, float A, float B, float Q) {
    const size_t o = (size_t)g * D + d, mo = (size_t)g * f.ld_mod + d;
    if (a.dscale) a.dscale[o] = gain * A;
    if (a.dshift) a.dshift[o] = B;
    if (a.dgate) a.dgate[o] = pg * Q;
    tg += (f.scale ? 1.f + f.scale[mo] : 1.f) * A;
    tp += (f.gate ? f.gate[mo] : 1.f) * Q;
  };
  const int lpg = groups < 32 ? 32 / groups : 1, sub = ty % lpg, used = groups < 32 ? groups * lpg : 32;
  float A = 0.f, B = 0.f, Q = 0.f;
  for (int g = ty / lpg; g < groups && ty < used; g += used / lpg) {
    A = B = Q = 0.f;
    if (in) {
      const float* p = a.part + ((size_t)g * chunks + sub) * 3 * D + d;
#pragma unroll 8
      for (int c = sub; c < chunks; c += lpg, p += (size_t)lpg * 3 * D) A += p[0], B += p[D], Q += p[2 * D];
      if (lpg == 1) emit(g, A, B, Q);
    }
  }
  if (lpg > 1) {
    sh[0][ty][tx] = A, sh[1][ty][tx] = B, sh[2][ty][tx] = Q;
    __syncthreads();
    if (ty < groups && in) {
      A = B = Q = 0.f;
      for (int l = ty * lpg; l < (ty + 1) * lpg; ++l) A += sh[0][l][tx], B += sh[1][l][tx], Q += sh[2][l][tx];
      emit(ty, A, B, Q);
    }
    __syncthreads();
  }
  sh[0][ty][tx] = tg;
  sh[1][ty][tx] = tp;
  __syncthreads();
  if (ty < 2 && in) {
    float x = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) x += sh[ty][r][tx];
    float* out = ty == 0 ? a.dgain : a.dpost_gain;
    if (out) out[d] = x;
  }
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int E, int NV, typename RT, typename CT>
cudaError_t run_fwd(const ResNorm& a, cudaStream_t s) {
  const int tpr = row_threads(a.D, NV), R = rows_at_once(tpr), threads = tpr * R + 32;
  const int coef = coef_bytes(a.D, 3);
  const Ring ring = ring_of(a.D, R, coef, {(int)sizeof(RT), (int)sizeof(CT)});
  const int smem = ring.stages * ring.stage_bytes + coef;
  auto* kernel = NV == 8 && threads <= 256 ? res_norm_kernel<E, NV, NV == 8, RT, CT> : res_norm_kernel<E, NV, false, RT, CT>;
  static std::atomic<bool> done[2][kMaxDevices];
  const cudaError_t e = allow_smem(kernel, kSmem, done[NV == 8 && threads <= 256]);
  if (e != cudaSuccess) return e;
  const int sms = current_sms();
  if (!sms) return cudaErrorNoDevice;
  // as many blocks as run at once: by registers (see the launch bounds) and by shared memory
  const int per = std::min(threads > 256 ? 1 : NV == 8 ? (E == 8 ? 3 : 2) : 1, kSmemOfSm / (smem + kStaticSmem));
  const int grid = std::max(1, std::min((a.M + R - 1) / R, sms * std::max(1, per)));
  return launch_k(kernel, dim3(grid), dim3(threads), smem, s, a, ring, tpr, R);
}
template <int E, int NV, typename RT, typename CT>
cudaError_t run_bwd(const ResNormGrad& a, int chunks, int groups, cudaStream_t s) {
  const int tpr = row_threads(a.f.D, NV), R = rows_at_once(tpr), threads = tpr * R + 32;
  const Ring ring = ring_of(a.f.D, R, coef_bytes(a.f.D, 2), {(int)sizeof(RT), (int)sizeof(CT), (int)sizeof(CT), (int)sizeof(RT)});
  const int smem = grad_smem(ring, a.f.D);
  auto* kernel = res_norm_grad_kernel<E, NV, RT, CT>;
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = allow_smem(kernel, kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_k(kernel, dim3((unsigned)chunks * groups), dim3(threads), smem, s, a, ring, chunks, tpr, R);
}
// f(E, NV, RT, CT) for a call's alignment, width and types.
template <typename F>
cudaError_t by_form(bool vec, int D, bool res_f32, bool f32, F f) {
  auto types = [&](auto e, auto nv) {
    if (f32) return f(e, nv, float{}, float{});
    return res_f32 ? f(e, nv, float{}, __nv_bfloat16{}) : f(e, nv, __nv_bfloat16{}, __nv_bfloat16{});
  };
  using std::integral_constant;
  auto widths = [&](auto e) {
    switch (elems(D)) {
      case 8: return types(e, integral_constant<int, 8>{});
      case 16: return types(e, integral_constant<int, 16>{});
      default: return types(e, integral_constant<int, 24>{});
    }
  };
  return vec ? widths(integral_constant<int, 8>{}) : widths(integral_constant<int, 1>{});
}

}  // namespace

cudaError_t launch_res_norm(const ResNorm& a, cudaStream_t s) {
  const bool v = a.D % 8 == 0 && aligned(a.x) && aligned(a.y) && aligned(a.s) && aligned(a.h);
  return by_form(v, a.D, a.res_f32, a.f32, [&](auto e, auto nv, auto rt, auto ct) {
    return run_fwd<decltype(e)::value, decltype(nv)::value, decltype(rt), decltype(ct)>(a, s);
  });
}

size_t res_norm_part_floats(int M, int D, int rpg) {
  const size_t groups = (M + rpg - 1) / rpg;
  return groups * grad_chunks(M, D, rpg) * 3 * (size_t)D;
}

cudaError_t launch_res_norm_grad(const ResNormGrad& a, cudaStream_t s) {
  const ResNorm& f = a.f;
  const int groups = (f.M + f.rows_per_group - 1) / f.rows_per_group, chunks = grad_chunks(f.M, f.D, f.rows_per_group);
  const bool v = f.D % 8 == 0 && aligned(f.x) && aligned(f.y) && aligned(a.ds) && aligned(a.dh) && aligned(a.dx) && aligned(a.dy);
  const cudaError_t e = by_form(v, f.D, f.res_f32, f.f32, [&](auto e_, auto nv, auto rt, auto ct) {
    return run_bwd<decltype(e_)::value, decltype(nv)::value, decltype(rt), decltype(ct)>(a, chunks, groups, s);
  });
  if (e != cudaSuccess || !a.part) return e;
  return launch_k(res_norm_sum_kernel, dim3((f.D + 31) / 32), dim3(32, 32), 0, s, a, groups, chunks);
}

cudaError_t res_norm_status(unsigned* bits) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_norm_status, 4);
  if (e != cudaSuccess || !*bits) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbol(g_norm_status, &zero, 4);
}

}  // namespace wam
