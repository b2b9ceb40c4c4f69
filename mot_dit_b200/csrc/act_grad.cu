// Gradients through the activation of a linear layer and of a gated layer, and
// the column sums that are the bias gradients (sm_100a).
//
// One pass over the saved pre-activations and the incoming gradient: the
// product's operand dz (dg, du) is written once in the compute type, its
// column sums are taken in fp32 before that rounding.  Bound by memory:
// linear 3, gated 5 elements of traffic per output element.  A block owns 32 E
// columns and one chunk of rows; eight row lanes keep their sums in registers
// and join them in shared memory, in a fixed order, and the chunks are
// added (in order) by the product that follows.
#include <algorithm>

#include "kernels.h"
#include "op_epilogue.cuh"

namespace wam {
namespace {

constexpr int kRows = 8;    // row lanes of a block
constexpr int kAhead = 4;   // rows a thread has in flight

template <int E, bool GATED, bool F32>
__global__ void __launch_bounds__(32 * kRows) act_grad_kernel(const ActGrad a) {
  __shared__ float sh[GATED ? 2 : 1][kRows][32 * E];
  const int tx = threadIdx.x, ty = threadIdx.y;
  const int n = (blockIdx.x * 32 + tx) * E, chunk = blockIdx.y;
  const int lo = (int)((long long)a.M * chunk / a.chunks), hi = (int)((long long)a.M * (chunk + 1) / a.chunks);
  pdl_trigger();
  pdl_wait();
  float s0[E], s1[E];
#pragma unroll
  for (int j = 0; j < E; ++j) s0[j] = s1[j] = 0.f;
  if (n < a.N) {
    for (int r0 = lo + ty; r0 < hi; r0 += kRows * kAhead) {
      float d[kAhead][E], z[kAhead][E], u[kAhead][E];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int r = r0 + i * kRows;
        if (r >= hi) break;
        const size_t at = (size_t)r * a.N + n;
        load_any<E>(a.dy, F32 || a.dy_f32, at, d[i]);
        if (a.z) load_any<E>(a.z, F32, at, z[i]);
        if (GATED) load_any<E>(a.u, F32, at, u[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int r = r0 + i * kRows;
        if (r >= hi) break;
        const size_t at = (size_t)r * a.ld_dz + n;
        float o0[E], o1[E];
#pragma unroll
        for (int j = 0; j < E; ++j) {
          float act = 0.f, der = 1.f;
          if (a.z) act_and_grad<!F32>(a.act, z[i][j], act, der);
          if (GATED) {
            o0[j] = d[i][j] * u[i][j] * der;
            o1[j] = d[i][j] * act;
            s1[j] += o1[j];
          } else {
            o0[j] = d[i][j] * der;
          }
          s0[j] += o0[j];
        }
        if (a.dz) store_any<E>(a.dz, F32, at, o0);
        if (GATED) store_any<E>(a.du, F32, at, o1);
      }
    }
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

template <int E, bool GATED, bool F32>
cudaError_t run(const ActGrad& a, cudaStream_t s) {
  const dim3 grid((a.N + 32 * E - 1) / (32 * E), a.chunks);
  return launch_k(act_grad_kernel<E, GATED, F32>, grid, dim3(32, kRows), 0, s, a);
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

cudaError_t launch_col_sum(const OpColSum* sums, int n, cudaStream_t s) {
  return launch_k(col_sum_kernel, dim3((sums[0].cols + 127) / 128, n), dim3(128), 0, s, sums[0], sums[n - 1]);
}

// At most 64 chunks (the partial sums stay small against the matrices), each
// of at least 16 rows.
int act_grad_chunks(int M) { return std::max(1, std::min(64, (M + 15) / 16)); }

cudaError_t launch_act_grad(const ActGrad& a, cudaStream_t s) {
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool ptrs = al(a.dy) && al(a.z) && al(a.u) && al(a.dz) && al(a.du);
  const bool gated = a.u != nullptr;
  if (a.f32) {
    const bool v = ptrs && a.N % 4 == 0 && a.ld_dz % 4 == 0;
    return gated ? (v ? run<4, true, true>(a, s) : run<1, true, true>(a, s))
                 : (v ? run<4, false, true>(a, s) : run<1, false, true>(a, s));
  }
  const bool v = ptrs && a.N % 8 == 0 && a.ld_dz % 8 == 0;
  return gated ? (v ? run<8, true, false>(a, s) : run<1, true, false>(a, s))
               : (v ? run<8, false, false>(a, s) : run<1, false, false>(a, s));
}

cudaError_t launch_repack(const void* src, void* dst, int rows, int cols, int ld, cudaStream_t s) {
  const OpMat m{src, cols, cols, rows};
  const size_t n = (size_t)rows * (ld / 8);
  return launch_k(repack_kernel, dim3((unsigned)std::min<size_t>((n + 255) / 256, 148 * 8)), dim3(256), 0, s, m,
                  reinterpret_cast<__nv_bfloat16*>(dst), ld);
}

}  // namespace wam
