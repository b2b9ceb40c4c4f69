// C ABI of the feed-forward and residual-norm operators (include/wam.h):
// argument checks, workspace layout and the launches of each direction.
#include <initializer_list>
#include <utility>

#include "kernels.h"
#include "op_reduction.h"
#include "wam.h"

using namespace wam;

namespace {

constexpr int kMaxDim = 1 << 24;  // rows, features (the tiles and chunks of what fits a device stay within 32 bits)

wam_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return WAM_OK;
  (void)cudaGetLastError();  // what failed is reported here, not by the caller's next call
  if (e == cudaErrorMemoryAllocation) return WAM_ERR_OOM;
  return WAM_ERR_CUDA;
}
size_t up(size_t n) { return (n + 255) / 256 * 256; }
int up8(int n) { return (n + 7) / 8 * 8; }
size_t esize(int dtype) { return dtype == WAM_FP32 ? 4 : 2; }
bool is_type(int t) { return t == WAM_FP32 || t == WAM_BF16; }
bool is_dim(int n) { return n >= 1 && n <= kMaxDim; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Zeroes the outputs of a call without rows.
wam_status zero(std::initializer_list<std::pair<void*, size_t>> outs, cudaStream_t s) {
  for (const auto& o : outs) {
    const cudaError_t e = o.first ? cudaMemsetAsync(o.first, 0, o.second, s) : cudaSuccess;
    if (e != cudaSuccess) return status_of(e);
  }
  return WAM_OK;
}

// A buffer of a call; an empty or null one overlaps nothing.
struct Span {
  const void* p;
  size_t bytes;
  bool empty() const { return !p || !bytes; }
  bool meets(const Span& o) const {
    if (empty() || o.empty()) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
    return a < b + o.bytes && b < a + bytes;
  }
  bool same(const Span& o) const { return p == o.p && bytes == o.bytes; }
};
// Every output apart from every input and every other output.
bool apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto a = outs.begin(); a != outs.end(); ++a) {
    for (auto b = a + 1; b != outs.end(); ++b)
      if (a->meets(*b)) return false;
    for (const Span& i : ins)
      if (a->meets(i)) return false;
  }
  return true;
}

OpEpi epilogue(void* out, int ld, bool out_f32) {
  OpEpi e{};
  e.out = out;
  e.ld = ld;
  e.out_f32 = out_f32;
  return e;
}
void set_vec(OpEpi& e) {
  e.vec = e.ld % 8 == 0 && aligned(e.out, 16) && aligned(e.bias, 16) && aligned(e.bias2, 16) && aligned(e.res, 16) &&
          aligned(e.z, 16) && aligned(e.z2, 16);
}
cudaError_t products(int dtype, const OpProduct* p, int n, const OpColSum* sums, int n_sums, cudaStream_t s) {
  if (n == 1 && n_sums == 0 && op_skinny_takes(p[0], dtype == WAM_FP32)) return launch_op_skinny(p[0], dtype == WAM_FP32, s);
  return launch_op_gemm(p, n, dtype == WAM_FP32, sums, n_sums, s);
}

// Workspace of a backward pass, in order: the activation's gradients (one or
// two [M, N8] matrices of the compute type), the bias gradients' partial sums,
// on the bf16 path when K is not a multiple of 8 copies of x and of the
// weights with padded rows (the tensor-core loads start on 16 bytes), and the
// pieces of the gradients' reductions.
struct BwdLayout {
  size_t dz, part, x, w, px, pw, total;
  int ldn, ldk;
  Pieces cut;
};
BwdLayout bwd_layout(int dtype, int M, int N, int K, int sides, bool need_dz) {
  BwdLayout l{};
  l.ldn = up8(N);
  l.ldk = up8(K);
  size_t at = 0;
  l.dz = at;
  if (need_dz) at += sides * up((size_t)M * l.ldn * esize(dtype));
  l.part = at;
  at += up((size_t)sides * act_grad_chunks(M, N, dtype == WAM_FP32) * N * 4);
  l.x = at;
  if (dtype == WAM_BF16 && K % 8) at += up((size_t)M * l.ldk * 2);
  l.w = at;
  if (dtype == WAM_BF16 && K % 8) at += sides * up((size_t)N * l.ldk * 2);
  l.cut = pieces_for(dtype == WAM_FP32, M, N, K, sides);
  l.px = at;
  if (l.cut.dx > 1) at += up((size_t)l.cut.dx * M * K * 4);
  l.pw = at;
  if (l.cut.dw > 1) at += sides * up((size_t)l.cut.dw * N * K * 4);
  l.total = at;
  return l;
}
// A gradient's epilogue: the output itself, or its pieces and the sum of them.
void gradient_out(OpProduct& q, void* out, int pieces, char* part, bool f32, OpPartSum* sums, int* n_sums) {
  q.pieces = pieces;
  if (pieces > 1) {
    q.e = epilogue(part, q.N, true);
    sums[(*n_sums)++] = {reinterpret_cast<const float*>(part), out, (size_t)q.M * q.N, pieces, f32};
  } else {
    q.e = epilogue(out, q.N, f32);
  }
  set_vec(q.e);
}

// The incoming gradient is the product's operand as it stands.
bool direct(int dtype, int N, int act, int dy_dtype) {
  return act == kActNone && dy_dtype == dtype && (dtype == WAM_FP32 || N % 8 == 0);
}

}  // namespace

extern "C" {

wam_status wam_ops_check_status(void) {
  unsigned gemm = 0, norm = 0;
  cudaError_t e = op_gemm_status(&gemm);
  if (e == cudaSuccess) e = res_norm_status(&norm);
  if (e != cudaSuccess) return status_of(e);
  return gemm | norm ? WAM_ERR_TIMEOUT : WAM_OK;
}

// ------------------------------------------------------------------ linear --
wam_status wam_op_linear_act(int dtype, int out_dtype, const void* x, const void* w, const float* bias,
                             const void* residual, void* y, void* z, int M, int N, int K, int act, void* stream) {
  if (!is_type(dtype) || !is_type(out_dtype) || (dtype == WAM_FP32 && out_dtype != WAM_FP32) || act < 0 ||
      act >= kActKinds || M < 0 || M > kMaxDim || !is_dim(N) || !is_dim(K))
    return WAM_ERR_INVALID_ARG;
  if (M == 0) return WAM_OK;
  const size_t e = esize(dtype), o = esize(out_dtype);
  if (!x || !w || !y || !aligned(x, e) || !aligned(w, e) || !aligned(y, o) || !aligned(z, e) || !aligned(residual, o) ||
      !aligned(bias, 4))
    return WAM_ERR_INVALID_ARG;
  const size_t mn = (size_t)M * N;
  const Span sy{y, mn * o}, sz{z, mn * e}, sx{x, (size_t)M * K * e}, sw{w, (size_t)N * K * e}, sb{bias, (size_t)N * 4},
      sr{residual, mn * o};
  if (!apart({sy, sz}, {sx, sw, sb, sr.same(sy) ? Span{} : sr})) return WAM_ERR_INVALID_ARG;
  OpProduct p{};
  p.a[0] = {x, K, K, M};
  p.b[0] = {w, K, K, N};
  p.pairs = 1;
  p.M = M;
  p.N = N;
  p.K = K;
  p.e = epilogue(y, N, out_dtype == WAM_FP32);
  p.e.bias = bias;
  p.e.res = residual;
  p.e.z = z;
  p.e.act = act;
  set_vec(p.e);
  return status_of(products(dtype, &p, 1, nullptr, 0, (cudaStream_t)stream));
}

wam_status wam_op_linear_act_workspace(int dtype, int M, int N, int K, int act, int dy_dtype, size_t* nbytes) {
  if (!is_type(dtype) || !is_type(dy_dtype) || (dtype == WAM_FP32 && dy_dtype != WAM_FP32) || act < 0 ||
      act >= kActKinds || M < 0 || M > kMaxDim || !is_dim(N) || !is_dim(K) || !nbytes)
    return WAM_ERR_INVALID_ARG;
  *nbytes = bwd_layout(dtype, M, N, K, 1, !direct(dtype, N, act, dy_dtype)).total;
  return WAM_OK;
}

wam_status wam_op_linear_act_backward(int dtype, int dy_dtype, const void* x, const void* w, const void* z,
                                      const void* dy, void* dx, void* dw, float* db, int M, int N, int K, int act,
                                      void* workspace, size_t nbytes, void* stream) {
  size_t need = 0;
  if (wam_op_linear_act_workspace(dtype, M, N, K, act, dy_dtype, &need) != WAM_OK) return WAM_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const size_t e = esize(dtype), o = esize(dy_dtype);
  if ((!dx && !dw && !db) || !aligned(dx, e) || !aligned(dw, e) || !aligned(db, 4)) return WAM_ERR_INVALID_ARG;
  if (M == 0) return zero({{dw, (size_t)N * K * e}, {db, (size_t)N * 4}}, s);  // no rows: the sums over them are zero
  if ((dw && !x) || (dx && !w) || !dy || (act != kActNone && !z) || !aligned(x, e) || !aligned(w, e) || !aligned(z, e) ||
      !aligned(dy, o) || nbytes < need || (need && (!workspace || !aligned(workspace, 256))))
    return WAM_ERR_INVALID_ARG;
  const size_t mn = (size_t)M * N, mk = (size_t)M * K, nk = (size_t)N * K;
  if (!apart({{dx, mk * e}, {dw, nk * e}, {db, (size_t)N * 4}, {workspace, need}},
             {{x, mk * e}, {w, nk * e}, {z, mn * e}, {dy, mn * o}}))
    return WAM_ERR_INVALID_ARG;
  const bool as_is = direct(dtype, N, act, dy_dtype);
  const BwdLayout l = bwd_layout(dtype, M, N, K, 1, !as_is);
  char* ws = reinterpret_cast<char*>(workspace);
  cudaError_t err;
  const int chunks = act_grad_chunks(M, N, dtype == WAM_FP32);
  float* part = db ? reinterpret_cast<float*>(ws + l.part) : nullptr;
  if (db || !as_is) {
    ActGrad a{};
    a.dy = dy;
    a.z = act == kActNone ? nullptr : z;
    a.dz = as_is ? nullptr : ws + l.dz;
    a.part = part;
    a.M = M;
    a.N = N;
    a.ld_dz = as_is ? N : l.ldn;
    a.act = act;
    a.f32 = dtype == WAM_FP32;
    a.dy_f32 = dy_dtype == WAM_FP32;
    a.chunks = chunks;
    if ((err = launch_act_grad(a, s)) != cudaSuccess) return status_of(err);
  }
  const bool pad = dtype == WAM_BF16 && K % 8;
  const int ldk = pad ? l.ldk : K;
  if (pad && dw) {
    if ((err = launch_repack(x, ws + l.x, M, K, ldk, s)) != cudaSuccess) return status_of(err);
    x = ws + l.x;
  }
  if (pad && dx) {
    if ((err = launch_repack(w, ws + l.w, N, K, ldk, s)) != cudaSuccess) return status_of(err);
    w = ws + l.w;
  }
  const int in = dtype == WAM_FP32 ? (N + 3) / 4 * 4 : N;  // (fp32: whole vectors, zero past N)
  const OpMat dz = as_is ? OpMat{dy, N, N, M} : OpMat{ws + l.dz, l.ldn, in, M};
  OpProduct p[2] = {};
  OpPartSum ps[2];
  int n = 0, n_ps = 0;
  auto add_dx = [&] {  // dx = dz W
    OpProduct& q = p[n++];
    q.a[0] = dz;
    q.b[0] = {w, ldk, K, N};
    q.pairs = 1;
    q.M = M;
    q.N = K;
    q.K = N;
    q.b_mn = 1;
    gradient_out(q, dx, l.cut.dx, ws + l.px, dtype == WAM_FP32, ps, &n_ps);
  };
  auto add_dw = [&] {  // dW = dz^T x
    OpProduct& q = p[n++];
    q.a[0] = dz;
    q.b[0] = {x, ldk, K, M};
    q.pairs = 1;
    q.M = N;
    q.N = K;
    q.K = M;
    q.a_mn = q.b_mn = 1;
    gradient_out(q, dw, l.cut.dw, ws + l.pw, dtype == WAM_FP32, ps, &n_ps);
  };
  // the longer tiles first: the last wave is made of the shorter ones
  const bool dx_first = (double)N / l.cut.dx >= (double)M / l.cut.dw;
  if (dx && dx_first) add_dx();
  if (dw) add_dw();
  if (dx && !dx_first) add_dx();
  const OpColSum cs{part, db, chunks, N};
  if (n == 0) return status_of(launch_col_sum(&cs, 1, s));
  err = products(dtype, p, n, &cs, db ? 1 : 0, s);
  if (err == cudaSuccess && n_ps) err = launch_part_sums(ps, n_ps, s);
  return status_of(err);
}

// ------------------------------------------------------------------- gated --
wam_status wam_op_gated(int dtype, const void* x, const void* wg, const void* wu, const float* bias_g,
                        const float* bias_u, void* a, void* g, void* u, int M, int F, int K, int act, void* stream) {
  if (!is_type(dtype) || act < 0 || act >= kActKinds || M < 0 || M > kMaxDim || !is_dim(F) || !is_dim(K) || !g != !u)
    return WAM_ERR_INVALID_ARG;
  if (M == 0) return WAM_OK;
  const size_t e = esize(dtype);
  if (!x || !wg || !wu || !a || !aligned(x, e) || !aligned(wg, e) || !aligned(wu, e) || !aligned(a, e) || !aligned(g, e) ||
      !aligned(u, e) || !aligned(bias_g, 4) || !aligned(bias_u, 4))
    return WAM_ERR_INVALID_ARG;
  const size_t mf = (size_t)M * F * e, fk = (size_t)F * K * e;
  if (!apart({{a, mf}, {g, mf}, {u, mf}},
             {{x, (size_t)M * K * e}, {wg, fk}, {wu, fk}, {bias_g, (size_t)F * 4}, {bias_u, (size_t)F * 4}}))
    return WAM_ERR_INVALID_ARG;
  OpProduct p{};
  p.a[0] = {x, K, K, M};
  p.b[0] = {wg, K, K, F};
  p.b[1] = {wu, K, K, F};
  p.pairs = 1;
  p.gated = 1;
  p.M = M;
  p.N = F;
  p.K = K;
  p.e = epilogue(a, F, dtype == WAM_FP32);
  p.e.bias = bias_g;
  p.e.bias2 = bias_u;
  p.e.z = g;
  p.e.z2 = u;
  p.e.act = act;
  set_vec(p.e);
  return status_of(products(dtype, &p, 1, nullptr, 0, (cudaStream_t)stream));
}

wam_status wam_op_gated_workspace(int dtype, int M, int F, int K, size_t* nbytes) {
  if (!is_type(dtype) || M < 0 || M > kMaxDim || !is_dim(F) || !is_dim(K) || !nbytes) return WAM_ERR_INVALID_ARG;
  *nbytes = bwd_layout(dtype, M, F, K, 2, true).total;
  return WAM_OK;
}

wam_status wam_op_gated_backward(int dtype, const void* x, const void* wg, const void* wu, const void* g, const void* u,
                                 const void* da, void* dx, void* dwg, void* dwu, float* dbias_g, float* dbias_u, int M,
                                 int F, int K, int act, void* workspace, size_t nbytes, void* stream) {
  size_t need = 0;
  if (wam_op_gated_workspace(dtype, M, F, K, &need) != WAM_OK || act < 0 || act >= kActKinds) return WAM_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const size_t e = esize(dtype);
  if ((!dx && !dwg && !dbias_g) || !dwg != !dwu || !dbias_g != !dbias_u || !aligned(dx, e) || !aligned(dwg, e) ||
      !aligned(dwu, e) || !aligned(dbias_g, 4) || !aligned(dbias_u, 4))
    return WAM_ERR_INVALID_ARG;
  const size_t mf = (size_t)M * F, mk = (size_t)M * K, fk = (size_t)F * K;
  if (M == 0) return zero({{dwg, fk * e}, {dwu, fk * e}, {dbias_g, (size_t)F * 4}, {dbias_u, (size_t)F * 4}}, s);
  if ((dwg && !x) || (dx && (!wg || !wu)) || !g || !u || !da || !aligned(x, e) || !aligned(wg, e) || !aligned(wu, e) ||
      !aligned(g, e) || !aligned(u, e) || !aligned(da, e) || nbytes < need || !workspace || !aligned(workspace, 256))
    return WAM_ERR_INVALID_ARG;
  if (!apart({{dx, mk * e}, {dwg, fk * e}, {dwu, fk * e}, {dbias_g, (size_t)F * 4}, {dbias_u, (size_t)F * 4}, {workspace, need}},
             {{x, mk * e}, {wg, fk * e}, {wu, fk * e}, {g, mf * e}, {u, mf * e}, {da, mf * e}}))
    return WAM_ERR_INVALID_ARG;
  const BwdLayout l = bwd_layout(dtype, M, F, K, 2, true);
  char* ws = reinterpret_cast<char*>(workspace);
  char* dg = ws + l.dz;
  char* du = dg + up((size_t)M * l.ldn * e);
  const int chunks = act_grad_chunks(M, F, dtype == WAM_FP32);
  float* part = dbias_g ? reinterpret_cast<float*>(ws + l.part) : nullptr;
  ActGrad a{};
  a.dy = da;
  a.z = g;
  a.u = u;
  a.dz = dg;
  a.du = du;
  a.part = part;
  a.M = M;
  a.N = F;
  a.ld_dz = l.ldn;
  a.act = act;
  a.f32 = a.dy_f32 = dtype == WAM_FP32;
  a.chunks = chunks;
  cudaError_t err = launch_act_grad(a, s);
  if (err != cudaSuccess) return status_of(err);
  const bool pad = dtype == WAM_BF16 && K % 8;
  const int ldk = pad ? l.ldk : K;
  if (pad && dwg) {
    if ((err = launch_repack(x, ws + l.x, M, K, ldk, s)) != cudaSuccess) return status_of(err);
    x = ws + l.x;
  }
  if (pad && dx) {
    char* g8 = ws + l.w;
    char* u8 = g8 + up((size_t)F * l.ldk * 2);
    if ((err = launch_repack(wg, g8, F, K, ldk, s)) != cudaSuccess ||
        (err = launch_repack(wu, u8, F, K, ldk, s)) != cudaSuccess)
      return status_of(err);
    wg = g8;
    wu = u8;
  }
  const int in = dtype == WAM_FP32 ? (F + 3) / 4 * 4 : F;  // (fp32: whole vectors, zero past F)
  OpProduct p[3] = {};
  OpPartSum ps[3];
  int n = 0, n_ps = 0;
  auto add_dx = [&] {  // dx = dg Wg + du Wu
    OpProduct& q = p[n++];
    q.a[0] = {dg, l.ldn, in, M};
    q.a[1] = {du, l.ldn, in, M};
    q.b[0] = {wg, ldk, K, F};
    q.b[1] = {wu, ldk, K, F};
    q.pairs = 2;
    q.M = M;
    q.N = K;
    q.K = F;
    q.b_mn = 1;
    gradient_out(q, dx, l.cut.dx, ws + l.px, dtype == WAM_FP32, ps, &n_ps);
  };
  const size_t piece_w = up((size_t)l.cut.dw * F * K * 4);
  auto add_dw = [&](const void* d, void* out, int side) {
    OpProduct& q = p[n++];
    q.a[0] = {d, l.ldn, in, M};
    q.b[0] = {x, ldk, K, M};
    q.pairs = 1;
    q.M = F;
    q.N = K;
    q.K = M;
    q.a_mn = q.b_mn = 1;
    gradient_out(q, out, l.cut.dw, ws + l.pw + side * piece_w, dtype == WAM_FP32, ps, &n_ps);
  };
  const bool dx_first = 2.0 * F / l.cut.dx >= (double)M / l.cut.dw;
  if (dx && dx_first) add_dx();
  if (dwg) {
    add_dw(dg, dwg, 0);
    add_dw(du, dwu, 1);
  }
  if (dx && !dx_first) add_dx();
  const OpColSum cs[2] = {{part, dbias_g, chunks, F}, {part ? part + (size_t)chunks * F : nullptr, dbias_u, chunks, F}};
  if (n == 0) return status_of(launch_col_sum(cs, 2, s));
  err = products(dtype, p, n, cs, dbias_g ? 2 : 0, s);
  if (err == cudaSuccess && n_ps) err = launch_part_sums(ps, n_ps, s);
  return status_of(err);
}

// ----------------------------------------------------------- residual norm --
wam_status wam_op_residual_norm(int dtype, int res_dtype, const void* x, const void* y, void* s, void* h, int M, int D,
                                float alpha, int post_norm, const float* post_gain, const float* gate,
                                const float* gain, const float* scale, const float* shift, int rows_per_group,
                                int ld_mod, void* stream) {
  if (!is_type(dtype) || !is_type(res_dtype) || (dtype == WAM_FP32 && res_dtype != WAM_FP32) || M < 0 || M > kMaxDim ||
      D < 1 || D > kResNormMax || rows_per_group < 0 || (!post_norm && post_gain))
    return WAM_ERR_INVALID_ARG;
  if (M == 0) return WAM_OK;
  const int rpg = rows_per_group == 0 || rows_per_group > M ? M : rows_per_group;
  const int groups = (M + rpg - 1) / rpg;
  const size_t e = esize(dtype), r = esize(res_dtype), n = (size_t)M * D;
  if (!x || !y || !s || !h || ((gate || scale || shift) && groups > 1 && ld_mod < D) || !aligned(x, r) || !aligned(s, r) ||
      !aligned(y, e) || !aligned(h, e) || !aligned(post_gain, 4) || !aligned(gate, 4) || !aligned(gain, 4) ||
      !aligned(scale, 4) || !aligned(shift, 4))
    return WAM_ERR_INVALID_ARG;
  const size_t table = ((size_t)(groups - 1) * ld_mod + D) * 4, vec = (size_t)D * 4;
  const Span sx{x, n * r}, ss{s, n * r}, sy{y, n * e}, sh{h, n * e};
  if (!apart({ss, sh}, {ss.same(sx) ? Span{} : sx, sh.same(sy) ? Span{} : sy, {post_gain, vec}, {gain, vec}, {gate, table},
                        {scale, table}, {shift, table}}))
    return WAM_ERR_INVALID_ARG;
  ResNorm a{x, y, s, h, post_gain, gate, gain, scale, shift, alpha, M, D, post_norm != 0, rpg, ld_mod, dtype == WAM_FP32,
            res_dtype == WAM_FP32};
  return status_of(launch_res_norm(a, (cudaStream_t)stream));
}

wam_status wam_op_residual_norm_workspace(int M, int D, int rows_per_group, size_t* nbytes) {
  if (M < 0 || M > kMaxDim || D < 1 || D > kResNormMax || rows_per_group < 0 || !nbytes) return WAM_ERR_INVALID_ARG;
  *nbytes = M == 0 ? 0 : res_norm_part_floats(M, D, rows_per_group == 0 || rows_per_group > M ? M : rows_per_group) * 4;
  return WAM_OK;
}

wam_status wam_op_residual_norm_backward(int dtype, int res_dtype, const void* s_in, const void* y, const void* ds,
                                         const void* dh, void* dx, void* dy, int M, int D, float alpha, int post_norm,
                                         const float* post_gain, const float* gate, const float* gain,
                                         const float* scale, int rows_per_group, int ld_mod, float* dpost_gain,
                                         float* dgate, float* dgain, float* dscale, float* dshift, void* workspace,
                                         size_t nbytes, void* stream) {
  size_t need = 0;
  if (!is_type(dtype) || !is_type(res_dtype) || (dtype == WAM_FP32 && res_dtype != WAM_FP32) ||
      (!post_norm && (post_gain || dpost_gain)) || wam_op_residual_norm_workspace(M, D, rows_per_group, &need) != WAM_OK)
    return WAM_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const size_t vec = (size_t)D * 4;
  // no rows, no samples: the vectors' gradients are zero, the tables' empty
  if (M == 0) return zero({{dpost_gain, vec}, {dgain, vec}}, st);
  const int rpg = rows_per_group == 0 || rows_per_group > M ? M : rows_per_group;
  const int groups = (M + rpg - 1) / rpg;
  const size_t e = esize(dtype), r = esize(res_dtype), n = (size_t)M * D;
  const bool sums = dpost_gain || dgate || dgain || dscale || dshift;
  if (!s_in || !y || !dh || !dx || !dy || ((gate || scale) && groups > 1 && ld_mod < D) || !aligned(s_in, r) ||
      !aligned(ds, r) || !aligned(dx, r) || !aligned(y, e) || !aligned(dh, e) || !aligned(dy, e) || !aligned(post_gain, 4) ||
      !aligned(gate, 4) || !aligned(gain, 4) || !aligned(scale, 4) || !aligned(dpost_gain, 4) || !aligned(dgate, 4) ||
      !aligned(dgain, 4) || !aligned(dscale, 4) || !aligned(dshift, 4) ||
      (sums && (!workspace || !aligned(workspace, 256) || nbytes < need)))
    return WAM_ERR_INVALID_ARG;
  const size_t table = ((size_t)(groups - 1) * ld_mod + D) * 4, grads = groups * vec;
  const Span ss{s_in, n * r}, sy{y, n * e}, sds{ds, n * r}, sdh{dh, n * e}, sdx{dx, n * r}, sdy{dy, n * e};
  auto unless = [](const Span& in, const Span& out) { return in.same(out) ? Span{} : in; };
  const Span t1{post_gain, vec}, t2{gate, table}, t3{gain, vec}, t4{scale, table};
  if (!apart({sdx}, {unless(ss, sdx), unless(sds, sdx), sy, sdh, t1, t2, t3, t4}) ||
      !apart({sdy}, {ss, sds, unless(sy, sdy), unless(sdh, sdy), t1, t2, t3, t4}) ||
      !apart({sdx, sdy, {dpost_gain, vec}, {dgate, grads}, {dgain, vec}, {dscale, grads}, {dshift, grads},
              {sums ? workspace : nullptr, need}}, {}) ||
      !apart({{dpost_gain, vec}, {dgate, grads}, {dgain, vec}, {dscale, grads}, {dshift, grads},
              {sums ? workspace : nullptr, need}}, {ss, sy, sds, sdh, t1, t2, t3, t4}))
    return WAM_ERR_INVALID_ARG;
  ResNormGrad a{};
  a.f = {s_in, y, nullptr, nullptr, post_gain, gate, gain, scale, nullptr, alpha, M, D, post_norm != 0, rpg, ld_mod,
         dtype == WAM_FP32, res_dtype == WAM_FP32};
  a.ds = ds;
  a.dh = dh;
  a.dx = dx;
  a.dy = dy;
  a.dpost_gain = dpost_gain;
  a.dgate = dgate;
  a.dgain = dgain;
  a.dscale = dscale;
  a.dshift = dshift;
  a.part = sums ? reinterpret_cast<float*>(workspace) : nullptr;
  return status_of(launch_res_norm_grad(a, st));
}

}  // extern "C"
