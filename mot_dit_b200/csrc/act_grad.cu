// Gradients through the activation of a linear layer and of a gated layer, and
// the column sums that are the bias gradients (sm_100a).
//
// One pass over the saved pre-activations and the incoming gradient: the
// product's operand dz (dg, du) is written once in the compute type, its
// column sums are taken in fp32 before that rounding.  Bound by memory:
// linear 3, gated 5 elements of traffic per output element (8448 x 4096 gated
// bf16: 346 MB, 53 us at the copy rate).  A block owns 32 E
// columns and one chunk of rows; eight row lanes keep their sums in registers
// and join them in shared memory, in a fixed order, and the chunks are
// added (in order) by the product that follows.
#include <algorithm>

#include "kernels.h"
#include "op_epilogue.cuh"

namespace wam {
namespace {

constexpr int kRows = 8;    // row lanes of a block
constexpr int kBlocksPerSm = 4;

// T: the compute type, DY: the incoming gradient's.  ANY: bf16 rows that do not
// start on 16 bytes, eight elements at a time all the same (the written rows
// are the workspace's, which do).
template <int E, bool GATED, typename T, typename DY, bool ANY>
__global__ void __launch_bounds__(32 * kRows, kBlocksPerSm) act_grad_kernel(const ActGrad a) {
  constexpr bool F32 = sizeof(T) == 4;
  // rows a thread has in flight (gated 8448 x 4096: 69 us with one, 82 with two
  // and 76 at three blocks an SM; linear 48 us with two, 51 with one)
  constexpr int kAhead = E == 1 ? 8 : E == 4 ? 4 : GATED ? 1 : 2;
  __shared__ float sh[GATED ? 2 : 1][kRows][32 * E];
  const int tx = threadIdx.x, ty = threadIdx.y;
  const int n = (blockIdx.x * 32 + tx) * E, chunk = blockIdx.y;
  const int lo = (int)((long long)a.M * chunk / a.chunks), hi = (int)((long long)a.M * (chunk + 1) / a.chunks);
  const DY* dy = reinterpret_cast<const DY*>(a.dy);
  const T* pz = reinterpret_cast<const T*>(a.z);
  const T* pu = reinterpret_cast<const T*>(a.u);
  pdl_trigger();
  pdl_wait();
  float s0[E], s1[E];
#pragma unroll
  for (int j = 0; j < E; ++j) s0[j] = s1[j] = 0.f;
  if (n < a.N) {
    for (int r0 = lo + ty; r0 < hi; r0 += kRows * kAhead) {
      Raw<DY, E> rd[kAhead];
      Raw<T, E> rz[kAhead], ru[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int r = r0 + i * kRows;
        if (r < hi) {
          const size_t at = (size_t)r * a.N + n;
          if constexpr (ANY) {
            rd[i].v = fetch8(OpMat{a.dy, a.N, a.N, a.M}, r, n);
            if (pz) rz[i].v = fetch8(OpMat{a.z, a.N, a.N, a.M}, r, n);
            if (GATED) ru[i].v = fetch8(OpMat{a.u, a.N, a.N, a.M}, r, n);
          } else {
            rd[i].load(dy + at);
            if (pz) rz[i].load(pz + at);
            if (GATED) ru[i].load(pu + at);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int r = r0 + i * kRows;
        if (r >= hi) break;
        const size_t at = (size_t)r * a.ld_dz + n;
        float d[E], z[E], u[E], o0[E], o1[E];
        rd[i].get(d);
        if (pz) rz[i].get(z);
        if (GATED) ru[i].get(u);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          float act = 0.f, der = 1.f;
          if (pz) act_and_grad<!F32>(a.act, z[j], act, der);
          if (GATED) {
            o0[j] = d[j] * u[j] * der;
            o1[j] = d[j] * act;
            s1[j] += o1[j];
          } else {
            o0[j] = d[j] * der;
          }
          s0[j] += o0[j];
        }
        if (a.dz) store_to<E>(reinterpret_cast<T*>(a.dz) + at, o0);
        if (GATED) store_to<E>(reinterpret_cast<T*>(a.du) + at, o1);
      }
    }
  }
  // fp32 rows that end inside a vector: the rest of it is zero (the product
  // takes it as part of the row)
  if (E == 1 && F32 && a.dz && n >= a.N && n < (a.N + 3) / 4 * 4)
    for (int r = lo + ty; r < hi; r += kRows) {
      reinterpret_cast<float*>(a.dz)[(size_t)r * a.ld_dz + n] = 0.f;
      if (GATED) reinterpret_cast<float*>(a.du)[(size_t)r * a.ld_dz + n] = 0.f;
    }
  if (!a.part) return;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    sh[0][ty][j * 32 + tx] = s0[j];
    if (GATED) sh[GATED ? 1 : 0][ty][j * 32 + tx] = s1[j];
  }
  __syncthreads();
  for (int i = ty * 32 + tx; i < 32 * E; i += 32 * kRows) {
    const int c = (blockIdx.x * 32 + i % 32) * E + i / 32;
    if (c >= a.N) continue;
#pragma unroll
    for (int k = 0; k < (GATED ? 2 : 1); ++k) {
      float v = 0.f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) v += sh[k][r][i];
      a.part[((size_t)k * a.chunks + chunk) * a.N + c] = v;
    }
  }
}

template <int E, bool GATED, typename T, typename DY, bool ANY = false>
cudaError_t run(const ActGrad& a, cudaStream_t s) {
  const dim3 grid(((a.dz && E == 1 ? (a.N + 3) / 4 * 4 : a.N) + 32 * E - 1) / (32 * E), a.chunks);
  return launch_k(act_grad_kernel<E, GATED, T, DY, ANY>, grid, dim3(32, kRows), 0, s, a);
}
template <int E, typename T>
cudaError_t run_types(const ActGrad& a, cudaStream_t s) {
  if (a.u) return run<E, true, T, T>(a, s);
  return a.dy_f32 ? run<E, false, T, float>(a, s) : run<E, false, T, T>(a, s);
}

__global__ void __launch_bounds__(256) repack_kernel(const OpMat src, __nv_bfloat16* __restrict__ dst, int ld) {
  pdl_trigger();
  pdl_wait();
  const size_t per = ld / 8, n = per * src.outer;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
    const int r = (int)(i / per), c = (int)(i % per) * 8;
    *reinterpret_cast<uint4*>(dst + (size_t)r * ld + c) = fetch8(src, r, c);
  }
}

struct PartSums {
  OpPartSum s[kOpProducts];
};
__global__ void __launch_bounds__(256) part_sum_kernel(const PartSums a) {
  pdl_trigger();
  pdl_wait();
  const OpPartSum& s = a.s[blockIdx.y];
  const bool vec = s.n % 4 == 0 && (reinterpret_cast<uintptr_t>(s.out) & 15) == 0;
  const int e = vec ? 4 : 1;
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * e; i < s.n; i += (size_t)gridDim.x * 256 * e) {
    if (vec) {
      float4 v = *reinterpret_cast<const float4*>(s.part + i);
#pragma unroll 4
      for (int p = 1; p < s.pieces; ++p) {
        const float4 x = *reinterpret_cast<const float4*>(s.part + p * s.n + i);
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
      }
      const float o[4] = {v.x, v.y, v.z, v.w};
      store_any<4>(s.out, s.f32, i, o);
    } else {
      float o[1] = {0.f};
#pragma unroll 4
      for (int p = 0; p < s.pieces; ++p) o[0] += s.part[p * s.n + i];
      store_any<1>(s.out, s.f32, i, o);
    }
  }
}
__global__ void __launch_bounds__(128) col_sum_kernel(const OpColSum a, const OpColSum b) {
  pdl_trigger();
  pdl_wait();
  const OpColSum& c = blockIdx.y ? b : a;
  const int i = blockIdx.x * 128 + threadIdx.x;
  if (i >= c.cols) return;
  float v = 0.f;
#pragma unroll 16
  for (int r = 0; r < c.rows; ++r) v += c.part[(size_t)r * c.cols + i];
  c.out[i] = v;
}

}  // namespace

cudaError_t launch_part_sums(const OpPartSum* sums, int n, cudaStream_t s) {
  PartSums a{};
  size_t most = 0;
  for (int i = 0; i < n; ++i) {
    a.s[i] = sums[i];
    most = std::max(most, sums[i].n);
  }
  return launch_k(part_sum_kernel, dim3((unsigned)std::min<size_t>((most + 1023) / 1024, 148 * 8), n), dim3(256), 0, s, a);
}

cudaError_t launch_col_sum(const OpColSum* sums, int n, cudaStream_t s) {
  return launch_k(col_sum_kernel, dim3((sums[0].cols + 127) / 128, n), dim3(128), 0, s, sums[0], sums[n - 1]);
}

// Two full waves of blocks at four an SM, chunks of at least 16 rows, and no
// more than 128 (their sums are added one after another).
int act_grad_chunks(int M, int N, bool f32) {
  const int e = f32 ? (N % 4 ? 1 : 4) : 8, cols = (N + 32 * e - 1) / (32 * e);
  return std::max(1, std::min({1184 / cols, (M + 15) / 16, 128}));
}

cudaError_t launch_act_grad(const ActGrad& a, cudaStream_t s) {
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool ptrs = al(a.dy) && al(a.z) && al(a.u) && al(a.dz) && al(a.du);
  if (a.f32)
    return ptrs && a.N % 4 == 0 && a.ld_dz % 4 == 0 ? run_types<4, float>(a, s) : run_types<1, float>(a, s);
  using H = __nv_bfloat16;
  if (ptrs && a.N % 8 == 0 && a.ld_dz % 8 == 0) return run_types<8, H>(a, s);
  if (a.dy_f32) return run<1, false, H, float>(a, s);
  return a.u ? run<8, true, H, H, true>(a, s) : run<8, false, H, H, true>(a, s);
}

cudaError_t launch_repack(const void* src, void* dst, int rows, int cols, int ld, cudaStream_t s) {
  const OpMat m{src, cols, cols, rows};
  const size_t n = (size_t)rows * (ld / 8);
  return launch_k(repack_kernel, dim3((unsigned)std::min<size_t>((n + 255) / 256, 148 * 8)), dim3(256), 0, s, m,
                  reinterpret_cast<__nv_bfloat16*>(dst), ld);
}

}  // namespace wam
