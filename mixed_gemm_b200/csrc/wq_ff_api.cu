// C ABI of the feed-forward operators (include/wq.h): argument checks and
// dispatch.  Every check runs on the host before anything is launched.
#include <math.h>

#include "wq_act_fn.cuh"
#include "wq_ff.cuh"
#include "wq_internal.cuh"

namespace wq {
namespace {

constexpr int64_t kMaxRows = 1LL << 24, kMaxCols = 1LL << 24;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

struct Span {
  const void* p;
  int64_t bytes;
};
bool meet(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}
// every output apart from every input and from every other output, and all of
// them 16-byte aligned
template <int NI, int NO>
int check_buffers(const Span (&in)[NI], const Span (&out)[NO]) {
  for (int i = 0; i < NI; ++i)
    if (!aligned(in[i].p, 16)) return WQ_ERR_ALIGNMENT;
  for (int o = 0; o < NO; ++o) {
    if (!aligned(out[o].p, 16)) return WQ_ERR_ALIGNMENT;
    for (int i = 0; i < NI; ++i)
      if (meet(out[o], in[i])) return WQ_ERR_INVALID_ARG;
    for (int q = 0; q < o; ++q)
      if (meet(out[o], out[q])) return WQ_ERR_INVALID_ARG;
  }
  return WQ_OK;
}

int status(cudaError_t e) {
  return e == cudaSuccess ? WQ_OK : e == cudaErrorNotSupported ? WQ_ERR_UNSUPPORTED : WQ_ERR_CUDA;
}

// Which kernel takes M tokens and a weight of `rows` rows (gated: both).  FEW streams
// the weight once into registers and reads all tokens once per 16 weight rows; THIN
// (at most 128 tokens) runs tcgen05 with the weight as the 128-row operand; PAIR with the
// tokens as rows of 256 x 256 tiles.  Measured (weights past L2), us, FEW / THIN / PAIR:
//                        8 tokens             16                   32                  128
//   INT8 2048 x 2048      2.8 / 5.2 / 7.5      3.0 / 5.0 / 6.7      3.9 / 4.9 / 6.7     - / 6.4 / 5.9
//   INT8 4096 x 4096      5.1 / 7.2 / 13.6     5.7 / 7.1 / 13.7     7.5 / 7.4 / 9.6     - / 9.8 / 9.8
//   INT8 8192 x 8192     13.6 / 14.7 / 27.0   15.4 / 15.0 / 18.0   22.0 / 15.2 / 18.4   - / 16.9 / 19.7
//   INT8 28672 x 8192    40.2 / 39.7 / 57.6   50.0 / 39.6 / 49.6   69.5 / 40.0 / 50.0   - / 44.2 / 56.5
//   gated 4096 x 4096    13.6 / 15.6 / 30.3   16.4 / 15.8 / 19.9   21.3 / 16.2 / 20.0
//   gated 28672 x 8192    143 / 141 / 190      163 / 142 / 191      233 / 142 / 192     - / 157 / 200
// (one token: 13.1 / 14.5 and 38.4 / 41.2 for the larger two INT8 ones.)  Deep layers of few
// rows are the exception: 500 x 16384 takes 7.5 / 7.1 with 8 tokens, 10 / 7.2 with 16 and
// 16 / 7.3 with 32, where THIN splits k.
enum Path { FEW, THIN, PAIR };
Path path_for(int64_t M, int64_t rows) {
  if (M <= 8 || (M <= 16 && rows <= 6144) || (M <= 32 && rows <= 2048)) return FEW;
  return M <= 128 ? THIN : PAIR;
}

int check_gated(int64_t M, int64_t F, int64_t K, int act) {
  if (M < 0 || M > kMaxRows || F <= 0 || K <= 0 || F > kMaxCols || K > kMaxCols || F % 8 || K % 8)
    return WQ_ERR_INVALID_ARG;
  if (F * K > (1LL << 40) || act < ACT_SILU || act > ACT_RELU) return WQ_ERR_INVALID_ARG;
  return WQ_OK;
}

int check_norm(int64_t M, int64_t D, int64_t per) {
  if (M < 0 || M > kMaxRows || D <= 0 || D > 16384 || D % 8 || per < 1) return WQ_ERR_INVALID_ARG;
  return WQ_OK;
}

}  // namespace
}  // namespace wq

using namespace wq;

extern "C" {

int wq_matmul_i8(const void* xq, const void* sx, const void* w, const void* sw, const void* bias,
                 int64_t M, int64_t N, int64_t K, int out_f32, void* out, void* stream) {
  if (M < 0 || M > kMaxRows || N <= 0 || N > kMaxCols || K <= 0 || K > 131056 || K % 16)
    return WQ_ERR_INVALID_ARG;
  if (M == 0) return WQ_OK;
  if (!xq || !sx || !w || !sw || !out) return WQ_ERR_INVALID_ARG;
  const Span in[] = {{xq, M * K}, {w, N * K}};
  const Span outs[] = {{out, M * N * (out_f32 ? 4 : 2)}};
  int st = check_buffers(in, outs);
  if (st) return st;
  if (!aligned(sx, 4) || !aligned(sw, 4) || !aligned(bias, 2)) return WQ_ERR_ALIGNMENT;
  if (meet(outs[0], {sx, M * 4}) || meet(outs[0], {sw, N * 4}) || meet(outs[0], {bias, N * 2}))
    return WQ_ERR_INVALID_ARG;
  I8Args a;
  a.xq = xq;
  a.sx = (const float*)sx;
  a.w = w;
  a.sw = (const float*)sw;
  a.bias = bias;
  a.M = M;
  a.N = N;
  a.K = K;
  a.f32 = out_f32 != 0;
  a.out = out;
  a.stream = (cudaStream_t)stream;
  const Path path = path_for(M, N);
  return status(path == FEW ? launch_i8_few(a) : path == THIN ? launch_i8_thin(a) : launch_i8_pair(a));
}

int wq_gated_ff(const void* x, const void* w_gate, const void* w_up, const void* b_gate,
                const void* b_up, int64_t M, int64_t F, int64_t K, int act, void* h, void* g,
                void* u, void* stream) {
  int st = check_gated(M, F, K, act);
  if (st) return st;
  if (M == 0) return WQ_OK;
  if (!x || !w_gate || !w_up || !h || !g != !u) return WQ_ERR_INVALID_ARG;
  const Span in[] = {{x, M * K * 2}, {w_gate, F * K * 2}, {w_up, F * K * 2}};
  const Span outs[] = {{h, M * F * 2}, {g, M * F * 2}, {u, M * F * 2}};
  if ((st = check_buffers(in, outs)) != WQ_OK) return st;
  if (!aligned(b_gate, 2) || !aligned(b_up, 2)) return WQ_ERR_ALIGNMENT;
  for (const Span& o : outs)
    if (meet(o, {b_gate, F * 2}) || meet(o, {b_up, F * 2})) return WQ_ERR_INVALID_ARG;
  GatedArgs a;
  a.x = x;
  a.wg = w_gate;
  a.wu = w_up;
  a.bg = b_gate;
  a.bu = b_up;
  a.M = M;
  a.F = F;
  a.K = K;
  a.act = act;
  a.h = h;
  a.g = g;
  a.u = u;
  a.stream = (cudaStream_t)stream;
  const Path path = path_for(M, 2 * F);
  return status(path == FEW    ? launch_gated_few(a)
                : path == THIN ? launch_gated_thin(a)
                               : launch_gated_pair(a));
}

int wq_gated_ff_backward_workspace_size(int64_t M, int64_t F, int64_t K, int need_bias,
                                        size_t* bytes) {
  if (!bytes || check_gated(M, F, K, ACT_SILU)) return WQ_ERR_INVALID_ARG;
  // dg and du; the bias sums' parts; the products' partial sums
  *bytes = M == 0 ? 0
                  : (size_t)(2 * M * F * 2 + (need_bias ? (int64_t)gated_chunks(M, F) * 2 * F * 4 : 0)) +
                        gated_grad_bytes(M, F, K);
  return WQ_OK;
}

int wq_gated_ff_backward(const void* dh, const void* x, const void* w_gate, const void* w_up,
                         const void* g, const void* u, int64_t M, int64_t F, int64_t K, int act,
                         void* workspace, size_t workspace_bytes, void* dx, void* dw_gate,
                         void* dw_up, void* db_gate, void* db_up, void* stream) {
  int st = check_gated(M, F, K, act);
  if (st) return st;
  if (!dw_gate != !dw_up || !db_gate != !db_up) return WQ_ERR_INVALID_ARG;
  const cudaStream_t s = (cudaStream_t)stream;
  const Span outs[] = {{dx, M * K * 2},   {dw_gate, F * K * 2}, {dw_up, F * K * 2},
                       {db_gate, F * 2},  {db_up, F * 2},       {workspace, (int64_t)workspace_bytes}};
  if (M == 0) {  // sums over no tokens
    const Span none[] = {{nullptr, 0}};
    if ((st = check_buffers(none, outs)) != WQ_OK) return st;
    for (int i = 1; i <= 4; ++i)
      if (outs[i].p) {
        const cudaError_t e = cudaMemsetAsync(const_cast<void*>(outs[i].p), 0, outs[i].bytes, s);
        if (e != cudaSuccess) return status(e);
      }
    return WQ_OK;
  }
  if (!dx && !dw_gate && !db_gate) return WQ_ERR_INVALID_ARG;
  if (!dh || !g || !u || !workspace || (dw_gate && !x) || (dx && (!w_gate || !w_up)))
    return WQ_ERR_INVALID_ARG;
  size_t need = 0;
  wq_gated_ff_backward_workspace_size(M, F, K, db_gate != nullptr, &need);
  if (workspace_bytes < need) return WQ_ERR_INVALID_ARG;
  const Span in[] = {{dh, M * F * 2}, {g, M * F * 2},      {u, M * F * 2},
                     {x, M * K * 2},  {w_gate, F * K * 2}, {w_up, F * K * 2}};
  if ((st = check_buffers(in, outs)) != WQ_OK) return st;
  uint16_t* dg = (uint16_t*)workspace;
  uint16_t* du = dg + M * F;
  float* partial = (float*)(du + M * F);
  void* parts = partial + (db_gate ? (int64_t)gated_chunks(M, F) * 2 * F : 0);
  cudaError_t e = launch_gated_dact(dh, g, u, M, F, act, dg, du, partial, db_gate, db_up, s);
  if (e == cudaSuccess && dx) e = launch_gated_dx(dg, du, w_gate, w_up, M, F, K, parts, dx, s);
  if (e == cudaSuccess && dw_gate) e = launch_gated_dw(dg, du, x, M, F, K, parts, dw_gate, dw_up, s);
  return status(e);
}

int wq_residual_norm(const void* x, const void* y, const void* gate, const void* w_post,
                     const void* w_pre, int64_t M, int64_t D, int64_t rows_per_gate, double scale,
                     double eps, void* r, void* h, void* hq, void* hs, void* rstd_post,
                     void* rstd_pre, void* stream) {
  int st = check_norm(M, D, rows_per_gate);
  if (st) return st;
  // (below 1e-30 the root of eps alone would leave fp32)
  if (!(eps >= 1e-30) || isinf(eps) || !isfinite(scale)) return WQ_ERR_INVALID_ARG;
  if (M == 0) return WQ_OK;  // (no rows: the tensors' addresses say nothing)
  if (rows_per_gate > M) rows_per_gate = M;
  if (!y && (r || gate || w_post)) return WQ_ERR_INVALID_ARG;
  if (!w_pre != !(h || hq) || !hq != !hs) return WQ_ERR_INVALID_ARG;
  if (!y && !w_pre) return WQ_ERR_INVALID_ARG;
  if ((rstd_post && !w_post) || (rstd_pre && !w_pre)) return WQ_ERR_INVALID_ARG;
  if (!x || (y && !r)) return WQ_ERR_INVALID_ARG;
  const int64_t b = M * D * 2, G = (M + rows_per_gate - 1) / rows_per_gate;
  // r may be x itself: a block reads its row before it writes it
  const Span in[] = {{r == x ? nullptr : x, b}, {y, b},          {gate, G * D * 2},
                     {w_post, D * 2},           {w_pre, D * 2}};
  const Span outs[] = {{r, b}, {h, b}, {hq, M * D}};
  if ((st = check_buffers(in, outs)) != WQ_OK) return st;
  if (!aligned(x, 16)) return WQ_ERR_ALIGNMENT;
  const Span vecs[] = {{hs, M * 4}, {rstd_post, M * 4}, {rstd_pre, M * 4}};
  for (int i = 0; i < 3; ++i) {
    if (!aligned(vecs[i].p, 4)) return WQ_ERR_ALIGNMENT;
    for (const Span& o : in)
      if (meet(vecs[i], o)) return WQ_ERR_INVALID_ARG;
    for (const Span& o : outs)
      if (meet(vecs[i], o)) return WQ_ERR_INVALID_ARG;
    if (meet(vecs[i], {x, b})) return WQ_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (meet(vecs[i], vecs[j])) return WQ_ERR_INVALID_ARG;
  }
  NormArgs a;
  a.x = x;
  a.y = y;
  a.gate = gate;
  a.wpost = w_post;
  a.wpre = w_pre;
  a.M = M;
  a.D = D;
  a.per = rows_per_gate;
  a.scale = scale;
  a.eps = eps;
  a.r = r;
  a.h = h;
  a.hq = hq;
  a.hs = (float*)hs;
  a.rpost = (float*)rstd_post;
  a.rpre = (float*)rstd_pre;
  a.stream = (cudaStream_t)stream;
  return status(launch_residual_norm(a));
}

int wq_residual_norm_backward_workspace_size(int64_t M, int64_t D, size_t* bytes) {
  if (!bytes || check_norm(M, D, 1)) return WQ_ERR_INVALID_ARG;
  int64_t rows = 0, ctas = 0;
  if (M > 0) norm_bwd_grid(M, D, &rows, &ctas);
  *bytes = (size_t)(ctas * 4 * D * 4);
  return WQ_OK;
}

int wq_residual_norm_backward(const void* dr, const void* dh, const void* x, const void* y,
                              const void* gate, const void* w_post, const void* w_pre,
                              const void* rstd_post, const void* rstd_pre, int64_t M, int64_t D,
                              int64_t rows_per_gate, double scale, void* workspace,
                              size_t workspace_bytes, void* dx, void* dy, void* dgate,
                              void* dw_post, void* dw_pre, void* stream) {
  int st = check_norm(M, D, rows_per_gate);
  if (st) return st;
  if (!isfinite(scale)) return WQ_ERR_INVALID_ARG;
  const int64_t b = M * D * 2;
  if (M == 0) {  // sums over no tokens (the tensors' addresses say nothing)
    const Span none[] = {{nullptr, 0}};
    const Span weights[] = {{dw_post, D * 2}, {dw_pre, D * 2}};
    if ((st = check_buffers(none, weights)) != WQ_OK) return st;
    for (const Span& w : weights)
      if (w.p) {
        const cudaError_t e =
            cudaMemsetAsync(const_cast<void*>(w.p), 0, w.bytes, (cudaStream_t)stream);
        if (e != cudaSuccess) return status(e);
      }
    return WQ_OK;
  }
  if (rows_per_gate > M) rows_per_gate = M;
  if (!y && (gate || w_post || dy || !w_pre)) return WQ_ERR_INVALID_ARG;
  if ((dgate && !gate) || (dw_post && !w_post) || (dw_pre && !w_pre)) return WQ_ERR_INVALID_ARG;
  const int64_t G = (M + rows_per_gate - 1) / rows_per_gate;
  const Span outs[] = {{dx, b},          {dy, b},         {dgate, G * D * 2},
                       {dw_post, D * 2}, {dw_pre, D * 2}, {workspace, (int64_t)workspace_bytes}};
  if (!x || !dx || !workspace || (y && !dy)) return WQ_ERR_INVALID_ARG;
  if (!w_pre != !dh || !w_pre != !rstd_pre || !w_post != !rstd_post) return WQ_ERR_INVALID_ARG;
  if (!dr && !dh) return WQ_ERR_INVALID_ARG;
  size_t need = 0;
  wq_residual_norm_backward_workspace_size(M, D, &need);
  if (workspace_bytes < need) return WQ_ERR_INVALID_ARG;
  const Span in[] = {{dr, b}, {dh, b}, {x, b}, {y, b}, {gate, G * D * 2}, {w_post, D * 2},
                     {w_pre, D * 2}};
  if ((st = check_buffers(in, outs)) != WQ_OK) return st;
  for (const void* v : {rstd_post, rstd_pre}) {
    if (!aligned(v, 4)) return WQ_ERR_ALIGNMENT;
    for (const Span& o : outs)
      if (meet(o, {v, M * 4})) return WQ_ERR_INVALID_ARG;
  }
  NormBwdArgs a;
  a.dr = dr;
  a.dh = dh;
  a.x = x;
  a.y = y;
  a.gate = gate;
  a.wpost = w_post;
  a.wpre = w_pre;
  a.rpost = (const float*)rstd_post;
  a.rpre = (const float*)rstd_pre;
  a.M = M;
  a.D = D;
  a.per = rows_per_gate;
  a.scale = scale;
  a.partial = (float*)workspace;
  a.dx = dx;
  a.dy = dy;
  a.dgate = dgate;
  a.dwpost = dw_post;
  a.dwpre = dw_pre;
  a.stream = (cudaStream_t)stream;
  return status(launch_residual_norm_bwd(a));
}

}  // extern "C"
