// fp32 products of the feed-forward operators, both directions (the debug
// precision): C[m, n] = sum_k A[m, k] B[n, k] with every product and sum in fp32.
//
// T x T output tiles (T = 128 or 64), 256 threads, (T / 16)^2 sums a thread in
// registers, added two at a time (fma.rn.f32x2).  Operands pass through a
// double-buffered shared tile of 16 reduction indices stored [k][m], whichever
// of their two dimensions is contiguous in memory.  Tiles with a long
// reduction are shared by the CTAs of a cluster, one k-range each; the partial
// tiles are summed in rank (= k) order through distributed shared memory.  In
// a list of products each is split or not by its own length (the CTAs of a
// cluster then take a tile each).
// Bound by the fp32 pipes (2 T^2 / (2 T) flop per shared-memory word).
#include <algorithm>

#include "cluster.cuh"
#include "kernels.h"
#include "op_epilogue.cuh"

namespace wam {
namespace {

constexpr int KT = 16;

struct ProductF {
  OpMat a[2], b[2];
  int M, N, K;   // K: one pair's reduction
  int pairs;
  int tiles_m, tiles, cta0;  // cta0: first CTA, a whole number of clusters
  int split;                 // CTAs that share a tile (1, or the cluster)
  int a_mn, b_mn, gated, avec, bvec;
  OpEpi e;
};
struct ArgsF {
  ProductF p[kOpProducts];
  OpColSum sums[2];
  int np, n_sums;
};

__device__ __forceinline__ void fma2(float2& c, float2 a, float2 b) {
  unsigned long long &cc = reinterpret_cast<unsigned long long&>(c);
  asm("fma.rn.f32x2 %0, %1, %2, %0;"
      : "+l"(cc)
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
}

// Elements [c, c + 4) of row r, zero outside [0, rows) x [0, cols).
__device__ __forceinline__ float4 fetch4(const OpMat& m, int r, int c, bool vec) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r >= m.outer || c >= m.inner) return v;
  const float* p = reinterpret_cast<const float*>(m.p) + (size_t)r * m.ld + c;
  if (vec && c + 4 <= m.inner) return *reinterpret_cast<const float4*>(p);
  v.x = p[0];
  if (c + 1 < m.inner) v.y = p[1];
  if (c + 2 < m.inner) v.z = p[2];
  if (c + 3 < m.inner) v.w = p[3];
  return v;
}

template <int T>
__global__ void __launch_bounds__(256, T == 128 ? 2 : 4) op_gemm_f32_kernel(const __grid_constant__ ArgsF g) {
  constexpr int R = T / 16;        // sums per thread and dimension
  constexpr int L = T + 4;         // shared row of one k
  constexpr int F = T * KT / 1024; // float4 per thread, operand and step
  extern __shared__ __align__(16) float sh[];
  float* sA = sh;                  // [2][KT][L]
  float* sB = sh + 2 * KT * L;
  const int tid = threadIdx.x;
  int pi = 0;
  while (pi + 1 < g.np && (int)blockIdx.x >= g.p[pi + 1].cta0) ++pi;
  const ProductF& P = g.p[pi];
  const int S = P.split;
  const uint32_t rank = S > 1 ? cluster_rank() : 0u;
  const int l = ((int)blockIdx.x - P.cta0) / S, tm = l % P.tiles_m, tn = l / P.tiles_m;
  const bool idle = l >= P.tiles;  // (fills up a cluster of unsplit tiles)
  const int m0 = tm * T, width = P.gated ? T / 2 : T, n0 = tn * width;
  pdl_trigger();
  pdl_wait();
  for (int i = 0; i < g.n_sums; ++i) {
    const OpColSum cs = g.sums[i];
    for (int c = blockIdx.x * 256 + tid; c < cs.cols; c += gridDim.x * 256) {
      float a = 0.f;
#pragma unroll 16
      for (int r = 0; r < cs.rows; ++r) a += cs.part[(size_t)r * cs.cols + c];
      cs.out[c] = a;
    }
  }
  if (idle) return;

  const int steps = (P.K + KT - 1) / KT, all = steps * P.pairs;
  const int s_lo = (int)((long long)all * rank / S), s_hi = (int)((long long)all * (rank + 1) / S);
  float4 ra[F], rb[F];
  auto fetch = [&](int st) {
    const int q = st >= steps ? 1 : 0, k0 = (st - q * steps) * KT;
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const int f = tid + i * 256;
      if (P.a_mn)
        ra[i] = fetch4(P.a[q], k0 + f / (T / 4), m0 + f % (T / 4) * 4, P.avec);
      else
        ra[i] = fetch4(P.a[q], m0 + f / 4, k0 + f % 4 * 4, P.avec);
      if (P.b_mn) {
        rb[i] = fetch4(P.b[q], k0 + f / (T / 4), n0 + f % (T / 4) * 4, P.bvec);
      } else {
        const int r = f / 4, side = P.gated ? r / (T / 2) : q;
        rb[i] = fetch4(P.b[side], n0 + (P.gated ? r % (T / 2) : r), k0 + f % 4 * 4, P.bvec);
      }
    }
  };
  auto put = [&](float* dst, const float4& v, int f, bool mn) {
    if (mn) {
      *reinterpret_cast<float4*>(dst + f / (T / 4) * L + f % (T / 4) * 4) = v;
    } else {
      float* d = dst + f % 4 * 4 * L + f / 4;
      d[0] = v.x, d[L] = v.y, d[2 * L] = v.z, d[3 * L] = v.w;
    }
  };
  float2 acc[R][R / 2];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < R / 2; ++j) acc[i][j] = make_float2(0.f, 0.f);
  const int tx = tid & 15, ty = tid >> 4;
  if (s_lo < s_hi) fetch(s_lo);
  for (int st = s_lo; st < s_hi; ++st) {
    float* a = sA + (st & 1) * KT * L;
    float* b = sB + (st & 1) * KT * L;
#pragma unroll
    for (int i = 0; i < F; ++i) {
      put(a, ra[i], tid + i * 256, P.a_mn);
      put(b, rb[i], tid + i * 256, P.b_mn);
    }
    __syncthreads();
    if (st + 1 < s_hi) fetch(st + 1);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      float av[R];
      float2 bv[R / 2];
#pragma unroll
      for (int h = 0; h < R / 4; ++h) {
        const float4 x = *reinterpret_cast<const float4*>(a + k * L + h * 64 + ty * 4);
        const float4 y = *reinterpret_cast<const float4*>(b + k * L + h * 64 + tx * 4);
        av[4 * h] = x.x, av[4 * h + 1] = x.y, av[4 * h + 2] = x.z, av[4 * h + 3] = x.w;
        bv[2 * h] = make_float2(y.x, y.y), bv[2 * h + 1] = make_float2(y.z, y.w);
      }
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < R / 2; ++j) fma2(acc[i][j], make_float2(av[i], av[i]), bv[j]);
    }
  }
  // partial tile -> shared memory ([row][T], 16-byte chunk q of row r at q ^ (r & 7))
  __syncthreads();
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = (i / 4) * 64 + ty * 4 + (i & 3);
#pragma unroll
    for (int h = 0; h < R / 4; ++h) {
      const int q = h * 16 + tx;
      *reinterpret_cast<float4*>(sh + r * T + ((q ^ (r & 7)) << 2)) =
          make_float4(acc[i][2 * h].x, acc[i][2 * h].y, acc[i][2 * h + 1].x, acc[i][2 * h + 1].y);
    }
  }
  __syncthreads();
  if (S > 1) cluster_sync();
  uint32_t base[8];
#pragma unroll
  for (int s = 0; s < 8; ++s)
    base[s] = S > 1 ? (s < S ? mapa_u32(smem_u32(sh), s) : 0u) : smem_u32(sh);
  const int valid = min(T, P.M - m0);
  const int r_lo = valid * (int)rank / S, r_hi = valid * ((int)rank + 1) / S;
  if (P.gated) {
    if (P.e.vec)
      finish_split<true, true, 4>(P.e, T, P.N, base, S, tid, 256, r_lo, r_hi, m0, n0);
    else
      finish_split<true, true, 1>(P.e, T, P.N, base, S, tid, 256, r_lo, r_hi, m0, n0);
  } else {
    if (P.e.vec)
      finish_split<true, false, 4>(P.e, T, P.N, base, S, tid, 256, r_lo, r_hi, m0, n0);
    else
      finish_split<true, false, 1>(P.e, T, P.N, base, S, tid, 256, r_lo, r_hi, m0, n0);
  }
  if (S > 1) cluster_sync();  // no CTA leaves while another may read its shared memory
}

template <int T>
constexpr int smem_f32() {
  return std::max(4 * KT * (T + 4), T * T) * 4;
}

template <int T>
cudaError_t launch_t(ArgsF& g, const OpProduct* p, int n, int sms, cudaStream_t s) {
  long long tiles[kOpProducts], all = 0;
  int steps[kOpProducts] = {}, least = 1 << 30;
  for (int i = 0; i < n; ++i) {
    ProductF& k = g.p[i];
    k.tiles_m = (p[i].M + T - 1) / T;
    k.tiles = k.tiles_m * (int)((p[i].gated ? 2ll * p[i].N + T - 1 : p[i].N + T - 1) / T);
    tiles[i] = k.tiles;
    all += tiles[i];
    steps[i] = k.pairs * ((p[i].K + KT - 1) / KT);
    least = std::min(least, steps[i]);
  }
  // Cluster: until every SM has four blocks, or the longest reduction is as
  // short as the others; a share keeps eight steps.
  int S = 1;
  if (T == 64) {
    const int longest = *std::max_element(steps, steps + n);
    while (S < 8 && longest >= 16 * S && (all * S < 4 * sms || longest > 2 * S * least)) S *= 2;
  }
  int cta = 0;
  for (int i = 0; i < n; ++i) {
    ProductF& k = g.p[i];
    k.split = S > 1 && steps[i] >= 8 * S && (all < 2 * sms || steps[i] >= 2 * least) ? S : 1;
    k.cta0 = cta;
    cta += (k.tiles * k.split + S - 1) / S * S;
  }
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = allow_smem(op_gemm_f32_kernel<T>, smem_f32<T>(), done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cta);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem_f32<T>();
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  int na = 0;
  if (S > 1) {
    at[na].id = cudaLaunchAttributeClusterDimension;
    at[na].val.clusterDim.x = S;
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
  return cudaLaunchKernelEx(&cfg, op_gemm_f32_kernel<T>, g);
}

}  // namespace

cudaError_t launch_op_gemm_f32(const OpProduct* p, int n, const OpColSum* sums, int n_sums, cudaStream_t s) {
  if (n < 1 || n > kOpProducts || n_sums < 0 || n_sums > 2) return cudaErrorInvalidValue;
  const int sms = current_sms();
  if (!sms) return cudaErrorNoDevice;
  ArgsF g;
  g.np = n;
  g.n_sums = n_sums;
  for (int i = 0; i < n_sums; ++i) g.sums[i] = sums[i];
  auto vec = [](const OpMat& m) { return (reinterpret_cast<uintptr_t>(m.p) & 15) == 0 && m.ld % 4 == 0; };
  long long t128 = 0, t64 = 0;
  for (int i = 0; i < n; ++i) {
    const OpProduct& q = p[i];
    ProductF& k = g.p[i];
    k.M = q.M;
    k.N = q.N;
    k.K = q.K;
    k.pairs = q.pairs == 2 ? 2 : 1;
    k.a_mn = q.a_mn;
    k.b_mn = q.b_mn;
    k.gated = q.gated;
    k.e = q.e;
    k.avec = k.bvec = 1;
    for (int j = 0; j < 2; ++j) {
      k.a[j] = q.a[k.pairs == 2 ? j : 0];
      k.b[j] = q.b[(k.pairs == 2 || q.gated) ? j : 0];
      k.avec &= vec(k.a[j]);
      k.bvec &= vec(k.b[j]);
    }
    const long long cols = q.gated ? 2ll * q.N : q.N;
    t128 += ((q.M + 127ll) / 128) * ((cols + 127) / 128);
    t64 += ((q.M + 63ll) / 64) * ((cols + 63) / 64);
  }
  // A 128-wide tile does a quarter of the shared-memory traffic of four
  // 64-wide ones but needs two for every SM, in whole rounds.
  const double w128 = (double)((t128 + 2 * sms - 1) / (2 * sms)) * 8, w64 = (double)((t64 + 4 * sms - 1) / (4 * sms)) * 4 * 1.3;
  return t128 >= sms && w128 <= w64 ? launch_t<128>(g, p, n, sms, s) : launch_t<64>(g, p, n, sms, s);
}

}  // namespace wam
