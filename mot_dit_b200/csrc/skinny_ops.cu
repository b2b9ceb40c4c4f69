// Forward products of a few tokens (sm_100a): y = act(x W^T + b) + r and the
// gated a = act(x Wg^T + bg) (x Wu^T + bu) for M <= 16 rows of x.
//
// The weights are read once and everything else is small, so the kernel is
// bound by memory and by latency; it has no tiles to set up.  A block owns
// 8 NT features; its warps take the 32-element k-blocks in turn and each lane
// loads 16 bytes of a weight row (a warp: 8 rows x 64 bytes) straight into
// registers, several blocks ahead.  bf16: the same 16 bytes are the B operand
// of two 16 x 8 x 16 matrix instructions with the tokens as the 16 rows of A:
// lane q of a row holds k = 8 q .. 8 q + 7 of the block, and as long as x is
// loaded by the same pattern the order in which the instruction sees k does not
// matter.  The warps' sums meet in shared memory, in warp order.  With too few
// feature groups for the SMs a cluster of blocks shares a group, each block a
// share of the k-blocks, and its first block adds the others' sums.  fp32: one
// lane takes 4 elements of 8 rows' dot products with up to eight tokens.
#include <algorithm>

#include "cluster.cuh"
#include "kernels.h"
#include "op_epilogue.cuh"

namespace wam {
namespace {

constexpr int kWarps = 8;
constexpr int kAhead = 3;   // k-blocks of a warp in flight: 6144 x 1536 one token 6.3 us (2: 6.65, 4: 7.25)
constexpr int kPerSm = 3;   // blocks an SM (2: 9.4 us, 4: 6.65)

struct Skinny {
  OpMat x, w[2];
  int M, N, K, vec;  // vec: every row starts on 16 bytes
  OpEpi e;
};

__device__ __forceinline__ uint4 chunk8(const OpMat& m, int r, int c, bool vec) {
  if (!vec) return fetch8(m, r, c);
  if (r >= m.outer || c >= m.inner) return make_uint4(0u, 0u, 0u, 0u);
  return *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(m.p) + (size_t)r * m.ld + c);
}

// One output element from its sum(s).
template <bool F32, bool GATED>
__device__ __forceinline__ void finish_one(const OpEpi& e, int m, int n, float v0, float v1) {
  const size_t at = (size_t)m * e.ld + n;
  float v[1] = {v0}, b[1], r[1] = {0.f};
  epi_bias<1>(e.bias, n, b);
  if constexpr (GATED) {
    float u[1] = {v1}, b2[1];
    epi_bias<1>(e.bias2, n, b2);
    epi_gated<F32, 1>(e, at, v, u, b, b2);
  } else {
    if (e.res) load_any<1>(e.res, F32 || e.out_f32, at, r);
    epi_linear<F32, 1>(e, at, v, b, r);
  }
}

template <int NT, bool GATED>
__global__ void __launch_bounds__(32 * kWarps, kPerSm) skinny_bf16_kernel(const __grid_constant__ Skinny p, int ks) {
  constexpr int S = GATED ? 2 : 1, U = S * NT == 4 ? 2 : kAhead;  // k-blocks in flight (four weight rows: registers for two)
  __shared__ float red[kWarps][S * NT][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = (lane & 3) * 8;
  const int n0 = blockIdx.x / ks * 8 * NT, KB = (p.K + 31) / 32;
  const uint32_t rank = ks > 1 ? cluster_rank() : 0u;
  const int first = rank * kWarps + warp, step = ks * kWarps;
  const bool vec = p.vec;
  pdl_trigger();
  pdl_wait();
  float acc[S * NT][4];
#pragma unroll
  for (int i = 0; i < S * NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  for (int kb = first; kb < KB; kb += step * U) {
    uint4 w[U][S * NT], x[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (kb + u * step) * 32 + q;  // (past K: zero)
#pragma unroll
      for (int i = 0; i < S * NT; ++i) w[u][i] = chunk8(p.w[i / NT], n0 + (i % NT) * 8 + r, k, vec);
#pragma unroll
      for (int j = 0; j < 2; ++j) x[u][j] = chunk8(p.x, j * 8 + r, k, vec);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < S * NT; ++i) {
        const uint4 a = x[u][0], b = x[u][1];
        mma_bf16_16816(acc[i], a.x, b.x, a.y, b.y, w[u][i].x, w[u][i].y);
        mma_bf16_16816(acc[i], a.z, b.z, a.w, b.w, w[u][i].z, w[u][i].w);
      }
  }
#pragma unroll
  for (int i = 0; i < S * NT; ++i) {
    float* d = &red[warp][i][r * 8 + (lane & 3) * 2];
    *reinterpret_cast<float2*>(d) = make_float2(acc[i][0], acc[i][1]);
    *reinterpret_cast<float2*>(d + 64) = make_float2(acc[i][2], acc[i][3]);
  }
  __syncthreads();
  if (ks > 1) cluster_sync();  // every block's sums are in place
  if (rank == 0) {
    for (int i = threadIdx.x; i < p.M * 8 * NT; i += 32 * kWarps) {
      const int m = i / (8 * NT), c = i % (8 * NT), n = n0 + c;
      if (n >= p.N) continue;
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int tile = s * NT + c / 8, at = m * 8 + c % 8;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) v[s] += red[k][tile][at];
        for (int r = 1; r < ks; ++r) {
          const uint32_t base = mapa_u32(smem_u32(&red[0][tile][at]), r);
          float x[kWarps];
#pragma unroll
          for (int k = 0; k < kWarps; ++k)
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(x[k])
                         : "r"(base + k * (uint32_t)sizeof(red[0]))
                         : "memory");
#pragma unroll
          for (int k = 0; k < kWarps; ++k) v[s] += x[k];
        }
      }
      finish_one<false, GATED>(p.e, m, n, v[0], v[1]);
    }
  }
  if (ks > 1) cluster_sync();  // no block leaves while the first may read its sums
}

// fp32: each warp the same features, a share of k; up to MT tokens.
template <int WARPS, int NT, int MT, bool GATED>
__global__ void __launch_bounds__(32 * WARPS) skinny_f32_kernel(const __grid_constant__ Skinny p) {
  constexpr int S = GATED ? 2 : 1;
  __shared__ float red[WARPS][S * NT][MT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * NT, steps = (p.K + 127) / 128;
  pdl_trigger();
  pdl_wait();
  auto fetch = [&](const OpMat& m, int r, int c) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r >= m.outer || c >= m.inner) return v;
    const float* s = reinterpret_cast<const float*>(m.p) + (size_t)r * m.ld + c;
    if (p.vec) return *reinterpret_cast<const float4*>(s);  // (K a multiple of 4)
    v.x = s[0];
    if (c + 1 < m.inner) v.y = s[1];
    if (c + 2 < m.inner) v.z = s[2];
    if (c + 3 < m.inner) v.w = s[3];
    return v;
  };
  float acc[S * NT][MT];
#pragma unroll
  for (int i = 0; i < S * NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = 0.f;
#pragma unroll 2
  for (int st = warp; st < steps; st += WARPS) {
    const int k = st * 128 + lane * 4;
    float4 w[S * NT], x[MT];
#pragma unroll
    for (int i = 0; i < S * NT; ++i) w[i] = fetch(p.w[i / NT], n0 + i % NT, k);
#pragma unroll
    for (int j = 0; j < MT; ++j) x[j] = fetch(p.x, j, k);
#pragma unroll
    for (int i = 0; i < S * NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j)
        acc[i][j] += w[i].x * x[j].x + w[i].y * x[j].y + w[i].z * x[j].z + w[i].w * x[j].w;
  }
#pragma unroll
  for (int i = 0; i < S * NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[i][j] += __shfl_xor_sync(0xffffffffu, acc[i][j], o);
      if (lane == 0) red[warp][i][j] = acc[i][j];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < p.M * NT; i += 32 * WARPS) {
    const int m = i / NT, c = i % NT, n = n0 + c;
    if (n >= p.N) continue;
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int k = 0; k < WARPS; ++k) v[s] += red[k][s * NT + c][m];
    finish_one<true, GATED>(p.e, m, n, v[0], v[1]);
  }
}

template <int NT, bool GATED>
cudaError_t run_bf16(const Skinny& k, cudaStream_t s) {
  const int groups = (k.N + 8 * NT - 1) / (8 * NT), KB = (k.K + 31) / 32, sms = current_sms();
  // share a group's k-blocks while all blocks still run at once (1536 x 6144:
  // 8.1 us in pairs, 12.8 alone; 4096 x 4096: 15 us in pairs that do not, 10 alone)
  int ks = 1;
  while (ks < 4 && groups * ks * 2 <= kPerSm * sms && KB >= 4 * ks * kWarps) ks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(groups * ks);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  int na = 0;
  if (ks > 1) {
    at[na].id = cudaLaunchAttributeClusterDimension;
    at[na].val.clusterDim.x = ks;
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
  return cudaLaunchKernelEx(&cfg, skinny_bf16_kernel<NT, GATED>, k, ks);
}
template <int NT, int MT, bool GATED>
cudaError_t run_f32(const Skinny& k, cudaStream_t s) {
  return launch_k(skinny_f32_kernel<8, NT, MT, GATED>, dim3((k.N + NT - 1) / NT), dim3(256), 0, s, k);
}

}  // namespace

bool op_skinny_takes(const OpProduct& p, bool f32) {
  return !p.a_mn && !p.b_mn && p.pairs <= 1 && p.M <= (f32 ? 8 : 16);
}

cudaError_t launch_op_skinny(const OpProduct& p, bool f32, cudaStream_t s) {
  Skinny k;
  k.x = p.a[0];
  k.w[0] = p.b[0];
  k.w[1] = p.b[p.gated ? 1 : 0];
  k.M = p.M;
  k.N = p.N;
  k.K = p.K;
  k.e = p.e;
  const int unit = f32 ? 4 : 8;
  k.vec = p.K % unit == 0;
  for (const OpMat* m : {&k.x, &k.w[0], &k.w[1]})
    k.vec &= m->ld % unit == 0 && (reinterpret_cast<uintptr_t>(m->p) & 15) == 0;
  if (f32) {
    if (p.gated) return p.M <= 2 ? run_f32<4, 2, true>(k, s) : run_f32<2, 8, true>(k, s);
    return p.M <= 2 ? run_f32<4, 2, false>(k, s) : run_f32<4, 8, false>(k, s);
  }
  // Two feature groups a block halve the reads of x; one, when there are too
  // few blocks for the SMs otherwise.
  const bool two = p.N >= 16 * 148;
  if (p.gated) return two ? run_bf16<2, true>(k, s) : run_bf16<1, true>(k, s);
  return two ? run_bf16<2, false>(k, s) : run_bf16<1, false>(k, s);
}

}  // namespace wam
