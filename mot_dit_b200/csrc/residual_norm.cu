// Gated residual with the norms on either side of it, both directions (sm_100a):
//   p = y or post_gain rms(y),  s = alpha x + gate p,
//   h = rms(s) gain (1 + scale) + shift,   rms(v) = v / sqrt(mean(v^2) + 1e-6).
// With n = s r, r = 1 / sqrt(mean(s^2) + eps), dn = dh gain (1 + scale):
//   dv = ds + r (dn - n mean(dn n)),  dx = alpha dv,  dp = gate dv,
//   dy = dp, or with q = y r_y: r_y (dp post_gain - q mean(dp post_gain q)),
// and the parameter gradients are column sums of dh n, dh and dv q.
//
// Bound by memory: forward 4, backward 6 row passes, each element read or
// written once.  Eight elements of a row sit in one thread's registers (a row
// is shared by D / 8 threads of a block, narrow rows by part of a warp), the
// column vectors of the block's sample stay there too, and the next row is
// requested before the present one is reduced.  The backward pass needs the
// mean of dp post_gain q, which depends on dv and so on the first means; it is
// expanded by linearity into three more sums of the same round, so that a row
// costs one block barrier: sum dv w y = sum w y ds + r sum w y dn - r^3 mean(dn s)
// sum w y s, w = gate post_gain.  Column sums stay in registers over a block's
// rows (all of one sample), go to a partial array once, and a second kernel
// adds the partials in order: no atomics, the same bits every time.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "op_epilogue.cuh"

namespace wam {
namespace {

constexpr float kEps = 1e-6f;
constexpr int kRowThreads = 256;  // threads of a block when a row needs fewer

// Threads that share a row: NV elements each; a power of two below a warp,
// whole warps above.
int row_threads(int D, int nv) {
  const int t = (D + nv - 1) / nv;
  if (t > 32) return (t + 31) / 32 * 32;
  int p = 1;
  while (p < t) p *= 2;
  return p;
}
int rows_at_once(int tpr) { return tpr >= kRowThreads ? 1 : kRowThreads / tpr; }
int elems(int D) { return D > 4096 ? 16 : 8; }

// Element j of thread t: groups of E consecutive elements, a row's threads
// side by side.
template <int E>
__device__ __forceinline__ int elem(int t, int tpr, int j) {
  return (t + (j / E) * tpr) * E + j % E;
}
// A row's elements of this thread, unconverted (zero past the row's end).
// E = 8: 16-byte accesses.
template <int E, int NV, typename T>
struct Row {
  Raw<T, E> r[NV / E];
  __device__ __forceinline__ void load(const T* p, int D, int t, int tpr) {
#pragma unroll
    for (int k = 0; k < NV / E; ++k) {
      const int i = elem<E>(t, tpr, E * k);
      if (i < D)
        r[k].load(p + i);
      else
        r[k].zero();
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < NV / E; ++k) r[k].zero();
  }
  __device__ __forceinline__ void get(float (&v)[NV], int, int, int) const {
#pragma unroll
    for (int k = 0; k < NV / E; ++k) r[k].get(v + E * k);
  }
};
// E = 2, any alignment.  fp32: single words.
template <int NV>
struct Row<2, NV, float> {
  float v_[NV];
  __device__ __forceinline__ void load(const float* p, int D, int t, int tpr) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = elem<2>(t, tpr, j);
      v_[j] = i < D ? p[i] : 0.f;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < NV; ++j) v_[j] = 0.f;
  }
  __device__ __forceinline__ void get(float (&v)[NV], int, int, int) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = v_[j];
  }
};
// bf16 pairs (2 k, 2 k + 1), in 4-byte words whatever the row's alignment.  A
// row that starts on a word holds its pairs in one word each.  One that
// starts two bytes past a word (`odd`) has pair k in the words k (its upper
// half) and k + 1 (its lower half): a thread loads word k and takes the next
// thread's from the neighbouring lane; where there is none (the last lane of
// the warp or of the row, the row's last word) the element is loaded by
// itself, and so is element 0 (word 0 reaches back before the row).
template <int NV>
struct Row<2, NV, __nv_bfloat16> {
  uint32_t w[NV / 2];
  unsigned short x[NV / 2];
  bool odd;
  __device__ __forceinline__ static bool edge(int t, int tpr, int k, int D) {
    return (threadIdx.x + threadIdx.y * blockDim.x) % 32 == 31 || t == tpr - 1 || 2 * k + 2 >= D;
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int D, int t, int tpr) {
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
    odd = (reinterpret_cast<uintptr_t>(p) & 2) != 0;
    if (!odd) {
#pragma unroll
      for (int j = 0; j < NV / 2; ++j) {
        const int i = 2 * (t + j * tpr);
        w[j] = 0;
        if (i + 1 < D)
          w[j] = *reinterpret_cast<const uint32_t*>(q + i);
        else if (i < D)
          w[j] = q[i];
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV / 2; ++j) {
        const int k = t + j * tpr, i = 2 * k;
        w[j] = 0;
        x[j] = 0;
        if (i < D) {
          if (k == 0)
            w[j] = (uint32_t)q[0] << 16;
          else
            w[j] = *reinterpret_cast<const uint32_t*>(q + i - 1);
          if (i + 1 < D && edge(t, tpr, k, D)) x[j] = q[i + 1];
        }
      }
    }
  }
  __device__ __forceinline__ void zero() {
    odd = false;
#pragma unroll
    for (int j = 0; j < NV / 2; ++j) w[j] = 0, x[j] = 0;
  }
  // (every lane of the warp takes part: rows of one warp may differ in `odd`)
  __device__ __forceinline__ void get(float (&v)[NV], int t, int tpr, int D) const {
#pragma unroll
    for (int j = 0; j < NV / 2; ++j) {
      const uint32_t next = __shfl_down_sync(0xffffffffu, w[j], 1);
      const uint32_t hi = edge(t, tpr, t + j * tpr, D) ? (uint32_t)x[j] << 16 : next << 16;
      v[2 * j] = __uint_as_float(odd ? w[j] & 0xffff0000u : w[j] << 16);
      v[2 * j + 1] = __uint_as_float(odd ? hi : w[j] & 0xffff0000u);
    }
  }
};
// Stores the row if it is live (every lane takes part).
template <int E, int NV, typename T>
__device__ __forceinline__ void row_store(T* p, bool live, int D, int t, int tpr, const float (&v)[NV]) {
  if constexpr (E == 8) {
    if (!live) return;
#pragma unroll
    for (int k = 0; k < NV / E; ++k) {
      const int i = elem<E>(t, tpr, E * k);
      if (i < D) store_to<E>(p + i, v + E * k);
    }
  } else if constexpr (sizeof(T) == 4) {
    if (!live) return;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = elem<2>(t, tpr, j);
      if (i < D) p[i] = v[j];
    }
  } else {
    // A row two bytes past a word: its word k joins the pair below (from the
    // lane before) and mine; the halves at a warp's or the row's ends alone.
    unsigned short* q = reinterpret_cast<unsigned short*>(p);
    const bool odd = (reinterpret_cast<uintptr_t>(p) & 2) != 0;
#pragma unroll
    for (int j = 0; j < NV / 2; ++j) {
      const int k = t + j * tpr, i = 2 * k;
      const uint32_t w = pack_bf16(v[2 * j], v[2 * j + 1]);
      const uint32_t before = __shfl_up_sync(0xffffffffu, w, 1);
      if (!live || i >= D) continue;
      if (!odd) {
        if (i + 1 < D)
          *reinterpret_cast<uint32_t*>(q + i) = w;
        else
          q[i] = (unsigned short)w;
      } else {
        if ((threadIdx.x + threadIdx.y * blockDim.x) % 32 == 0 || t == 0)
          q[i] = (unsigned short)w;
        else
          *reinterpret_cast<uint32_t*>(q + i - 1) = before >> 16 | w << 16;
        if (i + 1 < D && Row<2, NV, T>::edge(t, tpr, k, D)) q[i + 1] = (unsigned short)(w >> 16);
      }
    }
  }
}

// A column vector's elements of this thread (fill without one).
template <int E, int NV>
__device__ __forceinline__ void vec_load(const float* p, float fill, int D, int t, int tpr, float (&v)[NV]) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = fill;
    return;
  }
  if (E == 8 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    Row<8, NV, float> r;
    r.load(p, D, t, tpr);
    r.get(v, t, tpr, D);
    return;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = elem<E>(t, tpr, j);
    v[j] = i < D ? p[i] : 0.f;
  }
}

// Sums of K (1 or 6) values over the threads of each row.  Within a warp the
// six are reduced together: each exchange halves what a lane carries (8, 4, 2,
// 1 values), so that it takes 9 shuffles and not 30.  Across warps: one
// barrier; `sh` holds [2][rows][warps][8], the halves taken in turn.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int t, int tpr, int ry, int rows, float* sh, int& phase) {
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
    __syncthreads();
    float a = 0.f;
    for (int i = 0; i < warps; ++i) a += b[i * 8];
    v[0] = a;
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
    __syncthreads();
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < warps; ++i) {
      const float4 p = *reinterpret_cast<const float4*>(b + i * 8);
      const float2 q = *reinterpret_cast<const float2*>(b + i * 8 + 4);
      s[0] += p.x, s[1] += p.y, s[2] += p.z, s[3] += p.w, s[4] += q.x, s[5] += q.y;
    }
#pragma unroll
    for (int k = 0; k < 6; ++k) v[k] = s[k];
  }
}

// The coefficients of this thread's columns in sample grp: gain (1 + scale),
// shift, and gate post_gain.
template <int E, int NV>
__device__ __forceinline__ void coef(const ResNorm& a, int grp, int t, int tpr, float (&mul)[NV], float (&add)[NV],
                                     float (&w)[NV]) {
  const size_t o = (size_t)grp * a.ld_mod;
  float x[NV];
  vec_load<E, NV>(a.gain, 1.f, a.D, t, tpr, mul);
  vec_load<E, NV>(a.scale ? a.scale + o : nullptr, 0.f, a.D, t, tpr, x);
#pragma unroll
  for (int j = 0; j < NV; ++j) mul[j] *= 1.f + x[j];
  vec_load<E, NV>(a.shift ? a.shift + o : nullptr, 0.f, a.D, t, tpr, add);
  vec_load<E, NV>(a.gate ? a.gate + o : nullptr, 1.f, a.D, t, tpr, w);
  vec_load<E, NV>(a.post ? a.post_gain : nullptr, 1.f, a.D, t, tpr, x);
#pragma unroll
  for (int j = 0; j < NV; ++j) w[j] *= x[j];
}

// Block: (tpr, rows); its rows are [M b / grid, M (b + 1) / grid).  RT / CT:
// the stream's and the compute type.
template <int E, int NV, typename RT, typename CT>
__global__ void __launch_bounds__(512) res_norm_kernel(const ResNorm a) {
  __shared__ __align__(16) float sh[2 * 16 * 8];  // [2][rows][warps][8]: at most 16 warps in all
  const int t = threadIdx.x, tpr = blockDim.x, ry = threadIdx.y, R = blockDim.y, D = a.D;
  const int lo = (int)((long long)a.M * blockIdx.x / gridDim.x), hi = (int)((long long)a.M * (blockIdx.x + 1) / gridDim.x);
  const RT* px = reinterpret_cast<const RT*>(a.x);
  const CT* py = reinterpret_cast<const CT*>(a.y);
  pdl_trigger();
  pdl_wait();
  int phase = 0, grp = -1;
  float mul[NV], add[NV], w[NV];
  Row<E, NV, RT> rx;
  Row<E, NV, CT> ryy;
  auto load = [&](int m) {
    if (m < hi) {
      rx.load(px + (size_t)m * D, D, t, tpr);
      ryy.load(py + (size_t)m * D, D, t, tpr);
    }
  };
  rx.zero();
  ryy.zero();
  load(lo + ry);
  for (int m0 = lo; m0 < hi; m0 += R) {
    const int m = m0 + ry;
    const bool live = m < hi;  // (dead row lanes keep the barriers company)
    const int gr = (live ? m : hi - 1) / a.rows_per_group;
    if (gr != grp) coef<E, NV>(a, gr, t, tpr, mul, add, w);
    grp = gr;
    float v[NV], q[NV];
    rx.get(v, t, tpr, D);
    ryy.get(q, t, tpr, D);
    load(m + R);
    float s1[1] = {0.f};
    float rp = 1.f;
    if (a.post) {
#pragma unroll
      for (int j = 0; j < NV; ++j) s1[0] += q[j] * q[j];
      row_sum<1>(s1, t, tpr, ry, R, sh, phase);
      rp = 1.f / sqrtf(s1[0] / (float)D + kEps);
    }
    s1[0] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      v[j] = a.alpha * v[j] + w[j] * (q[j] * rp);
      s1[0] += v[j] * v[j];
    }
    row_sum<1>(s1, t, tpr, ry, R, sh, phase);
    const float r = 1.f / sqrtf(s1[0] / (float)D + kEps);
    row_store<E, NV>(reinterpret_cast<RT*>(a.s) + (size_t)m * D, live, D, t, tpr, v);
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = v[j] * r * mul[j] + add[j];
    row_store<E, NV>(reinterpret_cast<CT*>(a.h) + (size_t)m * D, live, D, t, tpr, v);
  }
}

// Block: chunk blockIdx.x % chunks of the rows of sample blockIdx.x / chunks.  AHEAD: the next
// row is requested early (the widest rows have no registers for it).
template <int E, int NV, bool AHEAD, typename RT, typename CT>
__global__ void __launch_bounds__(512) res_norm_grad_kernel(const ResNormGrad a, int chunks) {
  extern __shared__ float dyn[];    // [rows][3][tpr NV] column sums of the row lanes (rows > 1)
  __shared__ __align__(16) float sh[2 * 16 * 8];
  const ResNorm& f = a.f;
  const int t = threadIdx.x, tpr = blockDim.x, ry = threadIdx.y, R = blockDim.y, D = f.D;
  const int grp = blockIdx.x / chunks, ck = blockIdx.x % chunks, g_lo = grp * f.rows_per_group, g_n = min(f.rows_per_group, f.M - g_lo);
  const int lo = g_lo + (int)((long long)g_n * ck / chunks), hi = g_lo + (int)((long long)g_n * (ck + 1) / chunks);
  pdl_trigger();
  pdl_wait();
  int phase = 0;
  float mul[NV], w[NV];
  {
    float unused[NV];
    coef<E, NV>(f, grp, t, tpr, mul, unused, w);
  }
  float sa[NV], sb[NV], sq[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) sa[j] = sb[j] = sq[j] = 0.f;
  Row<E, NV, RT> xs, xd;
  Row<E, NV, CT> xy, xh;
  auto load = [&](int m) {
    if (m < hi) {
      const size_t o = (size_t)m * D;
      xs.load(reinterpret_cast<const RT*>(f.x) + o, D, t, tpr);
      xy.load(reinterpret_cast<const CT*>(f.y) + o, D, t, tpr);
      xh.load(reinterpret_cast<const CT*>(a.dh) + o, D, t, tpr);
      if (a.ds) xd.load(reinterpret_cast<const RT*>(a.ds) + o, D, t, tpr);
    } else {  // (a row lane past the chunk's end: adds nothing)
      xs.zero(), xy.zero(), xh.zero(), xd.zero();
    }
  };
  xd.zero();
  if (AHEAD) load(lo + ry);
  const float inv = 1.f / (float)D;
  for (int m0 = lo; m0 < hi; m0 += R) {
    const int m = m0 + ry;
    const bool live = m < hi;
    if (!AHEAD) load(m);
    float s[NV], y[NV], ds[NV], dh[NV];
    xs.get(s, t, tpr, D), xy.get(y, t, tpr, D), xd.get(ds, t, tpr, D), xh.get(dh, t, tpr, D);
    if (AHEAD) load(m + R);
    float v[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float dn = dh[j] * mul[j];
      v[0] += s[j] * s[j];
      v[1] += dn * s[j];
      if (f.post) {
        const float wy = w[j] * y[j];
        v[2] += y[j] * y[j];
        v[3] += wy * ds[j];
        v[4] += wy * dn;
        v[5] += wy * s[j];
      }
    }
    row_sum<6>(v, t, tpr, ry, R, sh, phase);
    const float r = 1.f / sqrtf(v[0] * inv + kEps);
    const float c = r * r * r * (v[1] * inv);
    const float rp = f.post ? 1.f / sqrtf(v[2] * inv + kEps) : 1.f;
    const float cy = f.post ? rp * rp * inv * (v[3] + r * v[4] - c * v[5]) : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float dv = ds[j] + r * dh[j] * mul[j] - s[j] * c;
      const float q = y[j] * rp;
      sa[j] += dh[j] * s[j] * r;
      sb[j] += dh[j];
      sq[j] += dv * q;
      ds[j] = f.alpha * dv;
      dh[j] = f.post ? rp * (dv * w[j] - y[j] * cy) : dv * w[j];
    }
    row_store<E, NV>(reinterpret_cast<RT*>(a.dx) + (size_t)m * D, live, D, t, tpr, ds);
    row_store<E, NV>(reinterpret_cast<CT*>(a.dy) + (size_t)m * D, live, D, t, tpr, dh);
  }
  if (!a.part) return;
  float* part = a.part + (size_t)blockIdx.x * 3 * D;
  if (R == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = elem<E>(t, tpr, j);
      if (i < D) part[i] = sa[j], part[D + i] = sb[j], part[2 * D + i] = sq[j];
    }
    return;
  }
  const int W = tpr * NV;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = elem<E>(t, tpr, j);
    float* d = dyn + (size_t)ry * 3 * W + i;
    d[0] = sa[j], d[W] = sb[j], d[2 * W] = sq[j];
  }
  __syncthreads();
  for (int i = ry * tpr + t; i < 3 * D; i += R * tpr) {
    const int k = i / D, c = i % D;
    float x = 0.f;
    for (int r = 0; r < R; ++r) x += dyn[(size_t)r * 3 * W + k * W + c];
    part[i] = x;
  }
}

// Column sums from the partials: 32 columns x 32 lanes.  Few samples: the
// lanes share each sample's chunks; many: each lane takes whole samples.
__global__ void __launch_bounds__(1024) res_norm_sum_kernel(const ResNormGrad a, int groups, int chunks) {
  __shared__ float sh[2][32][33];
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
  if (groups >= 32) {
    if (in)
      for (int g = ty; g < groups; g += 32) {
        float A = 0.f, B = 0.f, Q = 0.f;
        const float* p = a.part + (size_t)g * chunks * 3 * D + d;
        for (int c = 0; c < chunks; ++c, p += (size_t)3 * D) A += p[0], B += p[D], Q += p[2 * D];
        emit(g, A, B, Q);
      }
  } else {
    for (int g = 0; g < groups; ++g) {
      float v[3] = {0.f, 0.f, 0.f};
      if (in) {
        const float* p = a.part + ((size_t)g * chunks + ty) * 3 * D + d;
        for (int c = ty; c < chunks; c += 32, p += (size_t)32 * 3 * D) v[0] += p[0], v[1] += p[D], v[2] += p[2 * D];
      }
      float sum[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        __syncthreads();
        sh[0][ty][tx] = v[k];
        __syncthreads();
        float x = sh[0][tx][ty];  // lane tx of column ty
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (tx == 0) sh[1][0][ty] = x;
        __syncthreads();
        sum[k] = sh[1][0][tx];
      }
      if (ty == 0 && in) emit(g, sum[0], sum[1], sum[2]);
    }
    if (ty == 0 && in) {
      if (a.dgain) a.dgain[d] = tg;
      if (a.dpost_gain) a.dpost_gain[d] = tp;
    }
    return;
  }
  sh[0][ty][tx] = tg;
  sh[1][ty][tx] = tp;
  __syncthreads();
  if (ty < 2) {
    float x = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) x += sh[ty][r][tx];
    float* out = ty == 0 ? a.dgain : a.dpost_gain;
    if (in && out) out[d] = x;
  }
}

// Chunks of rows per sample: about three blocks an SM in all, each of at least
// four passes of its row lanes.
int grad_chunks(int M, int D, int rpg) {
  const int rows = rows_at_once(row_threads(D, elems(D)));
  const int groups = (M + rpg - 1) / rpg;
  const int most = (std::min(rpg, M) + 4 * rows - 1) / (4 * rows);
  return std::max(1, std::min(most, (444 + groups - 1) / groups));
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int E, int NV, typename RT, typename CT>
cudaError_t run_fwd(const ResNorm& a, cudaStream_t s) {
  const int tpr = row_threads(a.D, NV), R = rows_at_once(tpr);
  int dev = 0, sms = 148, per = 1;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
      (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, res_norm_kernel<E, NV, RT, CT>, tpr * R, 0)) != cudaSuccess)
    return e;
  const int grid = std::max(1, std::min((a.M + R - 1) / R, sms * std::max(1, per)));
  return launch_k(res_norm_kernel<E, NV, RT, CT>, dim3(grid), dim3(tpr, R), 0, s, a);
}
template <int E, int NV, typename RT, typename CT>
cudaError_t run_bwd(const ResNormGrad& a, int chunks, int groups, cudaStream_t s) {
  const int tpr = row_threads(a.f.D, NV), R = rows_at_once(tpr);
  const size_t smem = R > 1 && a.part ? (size_t)R * 3 * tpr * NV * 4 : 0;
  return launch_k(res_norm_grad_kernel<E, NV, NV == 8, RT, CT>, dim3((unsigned)chunks * groups), dim3(tpr, R), smem, s, a,
                  chunks);
}
// f(E, NV, RT, CT) for a call's alignment, width and types.
template <typename F>
cudaError_t by_form(bool vec, int D, bool res_f32, bool f32, F f) {
  auto types = [&](auto e, auto nv) {
    if (f32) return f(e, nv, float{}, float{});
    return res_f32 ? f(e, nv, float{}, __nv_bfloat16{}) : f(e, nv, __nv_bfloat16{}, __nv_bfloat16{});
  };
  using std::integral_constant;
  if (elems(D) == 8)
    return vec ? types(integral_constant<int, 8>{}, integral_constant<int, 8>{})
               : types(integral_constant<int, 2>{}, integral_constant<int, 8>{});
  return vec ? types(integral_constant<int, 8>{}, integral_constant<int, 16>{})
             : types(integral_constant<int, 2>{}, integral_constant<int, 16>{});
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

}  // namespace wam
