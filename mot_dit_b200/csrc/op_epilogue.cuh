// Activations with their derivatives, and the fused epilogue of the
// feed-forward products: bias, activation, gate product, residual and the
// saved pre-activations.  Shared by the products of many rows and of few, and by
// the activation gradients.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace wam {

// exp(x): the hardware form in the bf16 kernels (2 ulp and |x| 2^-24 of
// relative error, far below a bf16 step), the full one in fp32.
template <bool FAST>
__device__ __forceinline__ float exp_(float x) {
  return FAST ? __expf(x) : expf(x);
}
template <bool FAST>
__device__ __forceinline__ float div_(float a, float b) {
  return FAST ? __fdividef(a, b) : a / b;
}

constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// act(v[j]) for E values, the kind decided once.  A NaN stays one.
template <bool FAST, int E>
__device__ __forceinline__ void act_apply(int act, float (&v)[E]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = v[j] < 0.f ? 0.f : v[j];
      break;
    case kActSilu:
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = div_<FAST>(v[j], 1.f + exp_<FAST>(-v[j]));
      break;
    case kActGeluTanh:  // 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))
#pragma unroll
      for (int j = 0; j < E; ++j)
        v[j] = div_<FAST>(v[j], 1.f + exp_<FAST>(-kGelu2C * (v[j] + kGeluA * v[j] * v[j] * v[j])));
      break;
    case kActGeluErf:
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = 0.5f * v[j] * (1.f + erff(v[j] * kSqrtHalf));
      break;
    case kActSigmoid:
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = div_<FAST>(1.f, 1.f + exp_<FAST>(-v[j]));
      break;
    default:
      break;
  }
}

// act(z) and act'(z).  The terms that vanish for large |z| take z clamped
// where they are below any rounding, so that an infinite pre-activation has
// the limit's derivative and not inf * 0.
template <bool FAST>
__device__ __forceinline__ void act_and_grad(int act, float z, float& a, float& d) {
  switch (act) {
    case kActRelu:
      a = z < 0.f ? 0.f : z;
      d = z > 0.f ? 1.f : 0.f;
      break;
    case kActSilu: {
      const float p = div_<FAST>(1.f, 1.f + exp_<FAST>(-z));
      const float zc = fminf(fmaxf(z, -100.f), 100.f);
      a = z * p;
      d = p * (1.f + zc * (1.f - p));
      break;
    }
    case kActGeluTanh: {
      const float p = div_<FAST>(1.f, 1.f + exp_<FAST>(-kGelu2C * (z + kGeluA * z * z * z)));
      const float zc = fminf(fmaxf(z, -30.f), 30.f);
      a = z * p;
      d = p + kGelu2C * zc * p * (1.f - p) * (1.f + 3.f * kGeluA * zc * zc);
      break;
    }
    case kActGeluErf: {
      const float p = 0.5f * (1.f + erff(z * kSqrtHalf));
      const float zc = fminf(fmaxf(z, -30.f), 30.f);
      a = z * p;
      d = p + zc * exp_<FAST>(-0.5f * zc * zc) * kInvSqrt2Pi;
      break;
    }
    case kActSigmoid: {
      const float p = div_<FAST>(1.f, 1.f + exp_<FAST>(-z));
      a = p;
      d = p * (1.f - p);
      break;
    }
    default:
      a = z;
      d = 1.f;
  }
}

// ---------------------------------------------- E consecutive elements -----
// 16-byte (bf16, E = 4: 8-byte) accesses when E > 1, which the caller's
// alignment flag guarantees.  Raw<T, E> holds loaded elements unconverted, so
// that a batch of loads is in flight before the first is waited for (a
// conversion, or a branch on the type, between two loads would wait for each).
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <typename T, int E>
struct Raw;
template <>
struct Raw<float, 1> {
  float v;
  __device__ __forceinline__ void zero() { v = 0.f; }
  __device__ __forceinline__ void load(const float* p) { v = *p; }
  __device__ __forceinline__ void get(float* o) const { o[0] = v; }
};
template <>
struct Raw<__nv_bfloat16, 1> {
  unsigned short v;
  __device__ __forceinline__ void zero() { v = 0; }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const unsigned short*>(p); }
  __device__ __forceinline__ void get(float* o) const { o[0] = __uint_as_float((uint32_t)v << 16); }
};
template <int E>
struct Raw<float, E> {
  float4 v[E / 4];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) v[i] = reinterpret_cast<const float4*>(p)[i];
  }
  __device__ __forceinline__ void get(float* o) const {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) o[4 * i] = v[i].x, o[4 * i + 1] = v[i].y, o[4 * i + 2] = v[i].z, o[4 * i + 3] = v[i].w;
  }
};
template <>
struct Raw<__nv_bfloat16, 4> {
  uint2 v;
  __device__ __forceinline__ void zero() { v = make_uint2(0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float* o) const {
    o[0] = bf16_lo(v.x), o[1] = bf16_hi(v.x), o[2] = bf16_lo(v.y), o[3] = bf16_hi(v.y);
  }
};
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* o) const {
    o[0] = bf16_lo(v.x), o[1] = bf16_hi(v.x), o[2] = bf16_lo(v.y), o[3] = bf16_hi(v.y);
    o[4] = bf16_lo(v.z), o[5] = bf16_hi(v.z), o[6] = bf16_lo(v.w), o[7] = bf16_hi(v.w);
  }
};

template <int E>
__device__ __forceinline__ void load_f32(const float* p, float (&v)[E]) {
  Raw<float, E> r;
  r.load(p);
  r.get(v);
}
template <int E>
__device__ __forceinline__ void load_any(const void* p, bool f32, size_t i, float (&v)[E]) {
  if (f32) {
    load_f32<E>(reinterpret_cast<const float*>(p) + i, v);
  } else {
    Raw<__nv_bfloat16, E> r;
    r.load(reinterpret_cast<const __nv_bfloat16*>(p) + i);
    r.get(v);
  }
}
template <int E>
__device__ __forceinline__ void store_to(float* d, const float* v) {
  if constexpr (E == 1) {
    *d = v[0];
  } else {
#pragma unroll
    for (int k = 0; k < E / 4; ++k)
      reinterpret_cast<float4*>(d)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  }
}
template <int E>
__device__ __forceinline__ void store_to(__nv_bfloat16* d, const float* v) {
  if constexpr (E == 1)
    *d = __float2bfloat16_rn(v[0]);
  else if constexpr (E == 4)
    *reinterpret_cast<uint2*>(d) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  else
    *reinterpret_cast<uint4*>(d) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
template <int E>
__device__ __forceinline__ void store_any(void* p, bool f32, size_t i, const float (&v)[E]) {
  if (f32)
    store_to<E>(reinterpret_cast<float*>(p) + i, v);
  else
    store_to<E>(reinterpret_cast<__nv_bfloat16*>(p) + i, v);
}

// Eight elements [col, col + 8) of a row, zero outside the matrix, from any
// 2-byte-aligned address.
__device__ __forceinline__ uint4 fetch8(const OpMat& mt, int row, int col) {
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  if (row >= mt.outer || col >= mt.inner) return r;
  const size_t i = (size_t)row * mt.ld + col;
  const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(mt.p) + i;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (col + 8 <= mt.inner) {
    if ((a & 15) == 0) return *reinterpret_cast<const uint4*>(p);
    if ((a & 3) == 0) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // off by two bytes: the five words around it, when both ends lie inside
    if (i > 0 && i + 8 < (size_t)(mt.outer - 1) * mt.ld + mt.inner) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(a - 2);
      const uint32_t w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3], w4 = w[4];
      return make_uint4(__funnelshift_r(w0, w1, 16), __funnelshift_r(w1, w2, 16), __funnelshift_r(w2, w3, 16),
                        __funnelshift_r(w3, w4, 16));
    }
  }
  const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
  unsigned short h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = col + j < mt.inner ? q[j] : (unsigned short)0;
  r.x = h[0] | (uint32_t)h[1] << 16;
  r.y = h[2] | (uint32_t)h[3] << 16;
  r.z = h[4] | (uint32_t)h[5] << 16;
  r.w = h[6] | (uint32_t)h[7] << 16;
  return r;
}

// Bias of columns [n, n + E) (zero without one).
template <int E>
__device__ __forceinline__ void epi_bias(const float* bias, int n, float (&b)[E]) {
  if (bias) {
    load_f32<E>(bias + n, b);
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) b[j] = 0.f;
  }
}
// y[m, n..] = act(v + b) + r, z[m, n..] = v + b; i: the element's index.
template <bool F32, int E>
__device__ __forceinline__ void epi_linear(const OpEpi& e, size_t i, float (&v)[E], const float (&b)[E],
                                           const float (&r)[E]) {
#pragma unroll
  for (int j = 0; j < E; ++j) v[j] += b[j];
  if (e.z) store_any<E>(e.z, F32, i, v);
  act_apply<!F32, E>(e.act, v);
  if (e.res) {
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] += r[j];
  }
  store_any<E>(e.out, F32 || e.out_f32, i, v);
}
// a[m, n..] = act(g + bg) (u + bu); the pre-activations saved if asked for.
template <bool F32, int E>
__device__ __forceinline__ void epi_gated(const OpEpi& e, size_t i, float (&g)[E], float (&u)[E],
                                          const float (&bg)[E], const float (&bu)[E]) {
#pragma unroll
  for (int j = 0; j < E; ++j) {
    g[j] += bg[j];
    u[j] += bu[j];
  }
  if (e.z) {
    store_any<E>(e.z, F32, i, g);
    store_any<E>(e.z2, F32, i, u);
  }
  act_apply<!F32, E>(e.act, g);
#pragma unroll
  for (int j = 0; j < E; ++j) g[j] *= u[j];
  store_any<E>(e.out, F32, i, g);
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t mapa_u32(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}

// Rows [r_lo, r_hi) of a tile whose S fp32 partials ([row][bn], 16-byte chunk q
// of row r at q ^ (r & 7)) lie at the cluster addresses base[]: summed in rank
// order and finished by nthr threads.
template <bool F32, bool GATED, int E>
__device__ __forceinline__ void finish_split(const OpEpi& e, int bn, int N, const uint32_t (&base)[8], int S, int te,
                                             int nthr, int r_lo, int r_hi, int m0, int n0) {
  const int half = bn / 2, cols = GATED ? half : bn;
  const int groups = cols / E, items = (r_hi - r_lo) * groups;
  for (int it = te; it < items; it += nthr) {
    const int r = r_lo + it / groups, c = (it % groups) * E, n = n0 + c, m = m0 + r;
    if (n >= N) continue;
    const size_t at = (size_t)m * e.ld + n;
    float res[E];
    if (!GATED && e.res) load_any<E>(e.res, F32 || e.out_f32, at, res);
    float v[E], u[E];
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = u[j] = 0.f;
    for (int s = 0; s < S; ++s) {
      const uint32_t row = base[s] + r * bn * 4;
      if constexpr (E == 1) {
        float x;
        const int q = c >> 2;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(row + ((q ^ (r & 7)) << 4) + (c & 3) * 4) : "memory");
        v[0] += x;
        if (GATED) {
          const int q2 = (c + half) >> 2;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(row + ((q2 ^ (r & 7)) << 4) + (c & 3) * 4) : "memory");
          u[0] += x;
        }
      } else {
#pragma unroll
        for (int k = 0; k < E / 4; ++k) {
          const int q = (c >> 2) + k;
          const float4 x = ld_cluster4(row + ((q ^ (r & 7)) << 4));
          v[4 * k] += x.x, v[4 * k + 1] += x.y, v[4 * k + 2] += x.z, v[4 * k + 3] += x.w;
          if (GATED) {
            const int q2 = ((c + half) >> 2) + k;
            const float4 y = ld_cluster4(row + ((q2 ^ (r & 7)) << 4));
            u[4 * k] += y.x, u[4 * k + 1] += y.y, u[4 * k + 2] += y.z, u[4 * k + 3] += y.w;
          }
        }
      }
    }
    float b[E], b2[E];
    epi_bias<E>(e.bias, n, b);
    if constexpr (GATED) {
      epi_bias<E>(e.bias2, n, b2);
      epi_gated<F32, E>(e, at, v, u, b, b2);
    } else {
      epi_linear<F32, E>(e, at, v, b, res);
    }
  }
}

}  // namespace wam
