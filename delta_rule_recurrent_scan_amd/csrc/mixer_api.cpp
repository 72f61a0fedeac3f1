// C ABI of the operators around the recurrences: host-side validation,
// workspace sizing and launches of the short convolution, the selective scan,
// the gated head norm and the residual norm. Contract in include/osdn.h.
#include <hip/hip_runtime.h>

#include "api_common.hpp"
#include "mixer.hpp"

using namespace osdn_api;

namespace {

int status(int rc) {
  if (rc == -1) return OSDN_ERR_UNSUPPORTED;
  return rc == 0 ? OSDN_OK : OSDN_ERR_HIP;
}

// Channels, rows and tokens that the kernels index with 32 bits.
constexpr int kMaxTokens = 1 << 30;
bool width_ok(long long c) { return c <= (1 << 28); }

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws && bytes >= need && ((uintptr_t)ws & 255) == 0);
}

// Bytes that B x T rows of C elements with these strides span.
size_t span(int B, int T, long long C, long long bs, long long ts, size_t es) {
  if (B == 0 || T == 0 || C == 0) return 0;
  return ((size_t)(B - 1) * bs + (size_t)(T - 1) * ts + C) * es;
}

// Sizes of a convolution call; OSDN_OK or the status to return.
int conv_dims(int B, int T, int H, int D, int W, int dtype, long long xbs, long long xts,
              int l2norm) {
  if (B < 0 || T < 0 || H < 0 || D < 1 || T > kMaxTokens || xbs < 0 || xts < 0)
    return OSDN_ERR_BAD_DIMS;
  if (!width_ok((long long)H * D)) return OSDN_ERR_BAD_DIMS;
  if (W < 2 || W > 4 || !dtype_ok(dtype) || (l2norm && !dim_ok(D))) return OSDN_ERR_UNSUPPORTED;
  return OSDN_OK;
}

osdn::ConvArgs conv_args(int B, int T, int H, int D, int W, int dtype, const void* x,
                         long long xbs, long long xts, const float* weight, const float* bias,
                         const void* state0, const int* lengths, int act, int l2, float eps,
                         void* y, void* stateT, int whole) {
  osdn::ConvArgs a{};
  a.B = B; a.T = T; a.H = H; a.D = D; a.W = W;
  a.bf16 = dtype == OSDN_BF16;
  a.x = x; a.xbs = xbs; a.xts = xts;
  a.weight = weight; a.bias = bias; a.state0 = state0; a.lengths = lengths;
  a.act = act; a.l2 = l2; a.eps = eps;
  a.y = y; a.stateT = stateT; a.whole = whole;
  return a;
}

int conv_call(const osdn::ConvArgs& a, int in_place, hipStream_t s) {
  const size_t es = a.bf16 ? 2 : 4, C = (size_t)a.H * a.D, rows = (size_t)a.B * a.T;
  const size_t st = (size_t)a.B * (a.W - 1) * C * es;
  if (a.B == 0 || C == 0) return OSDN_OK;
  if (!a.weight || (rows > 0 && (!a.x || !a.y))) return OSDN_ERR_NULL_ARG;
  const Range ins[] = {rng(a.x, span(a.B, a.T, C, a.xbs, a.xts, es)),
                       rng(a.weight, C * a.W * 4), rng(a.bias, C * 4), rng(a.state0, st),
                       rng(a.lengths, (size_t)a.B * 4)};
  const Range outs[] = {rng(a.y, rows * C * es), rng(a.stateT, st)};
  const int allowed[][2] = {{1, 3}};
  if (!aliasing_ok(outs, ins, allowed, in_place ? 1 : 0)) return OSDN_ERR_ALIASING;
  if (a.T == 0 && (!a.stateT || a.stateT == a.state0)) return OSDN_OK;
  return status(osdn::launch_short_conv(a, s));
}

int gate_dims(int B, int H, int T, int D, int dtype, const void* z, long long zbs,
              long long zts) {
  if (B < 0 || H < 0 || T < 0 || (z && (zbs < 0 || zts < 0))) return OSDN_ERR_BAD_DIMS;
  if (!dim_ok(D) || !dtype_ok(dtype)) return OSDN_ERR_UNSUPPORTED;
  return width_ok((long long)H * D) ? OSDN_OK : OSDN_ERR_BAD_DIMS;
}

int res_dims(long long R, int C, int dtype, int res_dtype) {
  if (R < 0 || C < 0 || R > (1LL << 31)) return OSDN_ERR_BAD_DIMS;
  if (!dtype_ok(dtype) || !dtype_ok(res_dtype) || (dtype == OSDN_F32 && res_dtype == OSDN_BF16) ||
      C > OSDN_RESIDUAL_NORM_MAX_WIDTH)
    return OSDN_ERR_UNSUPPORTED;
  return OSDN_OK;
}

int ssm_dims(int B, int H, int G, int T, int P, int N, int dtype) {
  if (B < 0 || H < 0 || G < 0 || T < 0 || (H > 0 && (G == 0 || H % G != 0)) ||
      (long long)B * H > (1LL << 28) || T > kMaxTokens)
    return OSDN_ERR_BAD_DIMS;
  if (!dim_ok(P) || !dim_ok(N) || !dtype_ok(dtype)) return OSDN_ERR_UNSUPPORTED;
  return OSDN_OK;
}

osdn::SsmArgs ssm_args(int B, int H, int G, int T, int P, int N, int dtype, const void* x,
                       const float* dt, const float* A, const void* Bm, const void* Cm,
                       const float* D, const float* dt_bias, int softplus, const float* S0,
                       const int* lengths, void* y, float* ST, void* ws) {
  osdn::SsmArgs a{};
  a.B = B; a.H = H; a.G = G; a.T = T; a.P = P; a.N = N;
  a.bf16 = dtype == OSDN_BF16;
  a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.D = D; a.dt_bias = dt_bias;
  a.softplus = softplus; a.S0 = S0; a.lengths = lengths; a.y = y; a.ST = ST; a.ws = ws;
  return a;
}

}  // namespace

extern "C" {

// --- short convolution ------------------------------------------------------

int short_conv_forward(int B, int T, int H, int D, int W, int dtype, const void* x,
                       long long x_batch_stride, long long x_token_stride, const float* weight,
                       const float* bias, const void* state0, const int* lengths,
                       int activation, int l2norm, float eps, void* y, void* state_T,
                       void* stream) {
  const int rc = conv_dims(B, T, H, D, W, dtype, x_batch_stride, x_token_stride, l2norm);
  if (rc != OSDN_OK) return rc;
  return conv_call(conv_args(B, T, H, D, W, dtype, x, x_batch_stride, x_token_stride, weight,
                             bias, state0, lengths, activation, l2norm, eps, y, state_T, 0),
                   0, (hipStream_t)stream);
}

int short_conv_decode(int B, int T, int H, int D, int W, int dtype, const void* x,
                      long long x_batch_stride, long long x_token_stride, const float* weight,
                      const float* bias, const void* state, int activation, int l2norm,
                      float eps, void* y, void* state_out, void* stream) {
  const int rc = conv_dims(B, T, H, D, W, dtype, x_batch_stride, x_token_stride, l2norm);
  if (rc != OSDN_OK) return rc;
  if ((size_t)B * H > 0 && (!state || !state_out)) return OSDN_ERR_NULL_ARG;
  return conv_call(conv_args(B, T, H, D, W, dtype, x, x_batch_stride, x_token_stride, weight,
                             bias, state, nullptr, activation, l2norm, eps, y, state_out, 1),
                   1, (hipStream_t)stream);
}

size_t short_conv_backward_workspace_bytes(int B, int T, int H, int D, int W) {
  if (conv_dims(B, T, H, D, W, OSDN_F32, 0, 0, 0) != OSDN_OK) return 0;
  return round256(osdn::short_conv_backward_ws(B, T, H, D, W));
}

int short_conv_backward(int B, int T, int H, int D, int W, int dtype, int dy_dtype,
                        const void* x, long long x_batch_stride, long long x_token_stride,
                        const float* weight, const float* bias, const void* state0,
                        const int* lengths, int activation, int l2norm, float eps,
                        const void* dy, const void* dstate_T, void* dx, void* dstate0,
                        float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                        void* stream) {
  const int rc = conv_dims(B, T, H, D, W, dtype, x_batch_stride, x_token_stride, l2norm);
  if (rc != OSDN_OK) return rc;
  if (!dtype_ok(dy_dtype) || (dtype == OSDN_F32 && dy_dtype == OSDN_BF16))
    return OSDN_ERR_UNSUPPORTED;
  const size_t C = (size_t)H * D, rows = (size_t)B * T, es = elem(dtype);
  if (C == 0) return OSDN_OK;
  if (!weight || !dweight || (rows > 0 && (!x || !dy || !dx))) return OSDN_ERR_NULL_ARG;
  const size_t need = short_conv_backward_workspace_bytes(B, T, H, D, W);
  if (!workspace_ok(workspace, workspace_bytes, need)) return OSDN_ERR_WORKSPACE;
  const size_t st = (size_t)B * (W - 1) * C * es;
  const Range ins[] = {rng(x, span(B, T, C, x_batch_stride, x_token_stride, es)),
                       rng(weight, C * W * 4), rng(bias, C * 4), rng(state0, st),
                       rng(lengths, (size_t)B * 4), rng(dy, rows * C * elem(dy_dtype)),
                       rng(dstate_T, st)};
  const Range outs[] = {rng(dx, rows * C * es), rng(dstate0, st), rng(dweight, C * W * 4),
                        rng(dbias, C * 4), rng(workspace, need)};
  if (!aliasing_ok(outs, ins, nullptr, 0)) return OSDN_ERR_ALIASING;
  osdn::ConvBackwardArgs a{};
  a.f = conv_args(B, T, H, D, W, dtype, x, x_batch_stride, x_token_stride, weight, bias, state0,
                  lengths, activation, l2norm, eps, nullptr, nullptr, 0);
  a.dy_bf16 = dy_dtype == OSDN_BF16;
  a.dy = dy; a.dstateT = dstate_T; a.dx = dx; a.dstate0 = dstate0;
  a.dweight = dweight; a.dbias = dbias; a.ws = workspace;
  return status(osdn::launch_short_conv_backward(a, (hipStream_t)stream));
}

// --- gated head norm ----------------------------------------------------------

int gated_norm_forward(int B, int H, int T, int D, int dtype, const void* x, const void* z,
                       long long z_batch_stride, long long z_token_stride, const float* weight,
                       int weight_per_head, float eps, int gate_first, void* y, void* stream) {
  const int rc = gate_dims(B, H, T, D, dtype, z, z_batch_stride, z_token_stride);
  if (rc != OSDN_OK) return rc;
  const size_t n = (size_t)B * H * T * D, es = elem(dtype), C = (size_t)H * D;
  if (n == 0) return OSDN_OK;
  if (!x || !weight || !y) return OSDN_ERR_NULL_ARG;
  if (!aligned16(x) || !aligned16(y)) return OSDN_ERR_MISALIGNED;
  const Range ins[] = {rng(x, n * es),
                       rng(z, z ? span(B, T, C, z_batch_stride, z_token_stride, es) : 0),
                       rng(weight, (weight_per_head ? C : D) * 4)};
  const Range outs[] = {rng(y, n * es)};
  if (!aliasing_ok(outs, ins, nullptr, 0)) return OSDN_ERR_ALIASING;
  osdn::GatedNormArgs a{};
  a.B = B; a.H = H; a.T = T; a.D = D; a.bf16 = dtype == OSDN_BF16;
  a.x = x; a.z = z; a.zbs = z_batch_stride; a.zts = z_token_stride; a.weight = weight;
  a.per_head = weight_per_head; a.gate_first = gate_first; a.eps = eps; a.y = y;
  return status(osdn::launch_gated_norm(a, (hipStream_t)stream));
}

size_t gated_norm_backward_workspace_bytes(int B, int H, int T, int D) {
  if (gate_dims(B, H, T, D, OSDN_F32, nullptr, 0, 0) != OSDN_OK) return 0;
  return round256(osdn::gated_norm_backward_ws(B, H, T, D));
}

int gated_norm_backward(int B, int H, int T, int D, int dtype, const void* x, const void* z,
                        long long z_batch_stride, long long z_token_stride, const float* weight,
                        int weight_per_head, float eps, int gate_first, const void* dy, void* dx,
                        void* dz, float* dweight, void* workspace, size_t workspace_bytes,
                        void* stream) {
  const int rc = gate_dims(B, H, T, D, dtype, z, z_batch_stride, z_token_stride);
  if (rc != OSDN_OK) return rc;
  const size_t n = (size_t)B * H * T * D, es = elem(dtype), C = (size_t)H * D;
  if (H == 0 && weight_per_head) return OSDN_OK;
  if (!dweight || (n > 0 && (!x || !weight || !dy || !dx || (z && !dz))))
    return OSDN_ERR_NULL_ARG;
  if (!aligned16(x) || !aligned16(dy) || !aligned16(dx) || !aligned16(dz))
    return OSDN_ERR_MISALIGNED;
  const size_t need = gated_norm_backward_workspace_bytes(B, H, T, D);
  if (!workspace_ok(workspace, workspace_bytes, need)) return OSDN_ERR_WORKSPACE;
  const size_t nw = (weight_per_head ? C : D) * 4;
  const Range ins[] = {rng(x, n * es),
                       rng(z, z ? span(B, T, C, z_batch_stride, z_token_stride, es) : 0),
                       rng(weight, nw), rng(dy, n * es)};
  const Range outs[] = {rng(dx, n * es), rng(dz, z ? n * es : 0), rng(dweight, nw),
                        rng(workspace, need)};
  if (!aliasing_ok(outs, ins, nullptr, 0)) return OSDN_ERR_ALIASING;
  osdn::GatedNormArgs a{};
  a.B = B; a.H = H; a.T = T; a.D = D; a.bf16 = dtype == OSDN_BF16;
  a.x = x; a.z = z; a.zbs = z_batch_stride; a.zts = z_token_stride; a.weight = weight;
  a.per_head = weight_per_head; a.gate_first = gate_first; a.eps = eps;
  a.dy = dy; a.dx = dx; a.dz = dz; a.dweight = dweight; a.ws = workspace;
  return status(osdn::launch_gated_norm_backward(a, (hipStream_t)stream));
}

// --- residual norm -------------------------------------------------------------

int residual_norm_forward(long long R, int C, int dtype, int res_dtype, const void* x,
                          const void* residual, float scale, const float* weight, float eps,
                          void* y, void* h, void* stream) {
  const int rc = res_dims(R, C, dtype, res_dtype);
  if (rc != OSDN_OK) return rc;
  const size_t n = (size_t)R * C;
  if (n == 0) return OSDN_OK;
  if (!x || !weight || !y) return OSDN_ERR_NULL_ARG;
  const Range ins[] = {rng(x, n * elem(dtype)), rng(residual, n * elem(res_dtype)),
                       rng(weight, (size_t)C * 4)};
  const Range outs[] = {rng(y, n * elem(dtype)), rng(h, n * elem(res_dtype))};
  const int allowed[][2] = {{1, 1}};  // h == residual
  if (!aliasing_ok(outs, ins, allowed, 1)) return OSDN_ERR_ALIASING;
  osdn::ResidualNormArgs a{};
  a.R = R; a.C = C; a.bf16 = dtype == OSDN_BF16; a.res_bf16 = res_dtype == OSDN_BF16;
  a.x = x; a.residual = residual; a.scale = scale; a.weight = weight; a.eps = eps;
  a.y = y; a.h = h;
  return status(osdn::launch_residual_norm(a, (hipStream_t)stream));
}

size_t residual_norm_backward_workspace_bytes(long long R, int C) {
  if (res_dims(R, C, OSDN_F32, OSDN_F32) != OSDN_OK || C == 0) return 0;
  return round256(osdn::residual_norm_backward_ws(R, C));
}

int residual_norm_backward(long long R, int C, int dtype, int res_dtype, const void* dy,
                           const void* h, const void* dh, float scale, const float* weight,
                           float eps, void* dx, void* dresidual, float* dweight,
                           void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = res_dims(R, C, dtype, res_dtype);
  if (rc != OSDN_OK) return rc;
  if (C == 0) return OSDN_OK;
  const size_t n = (size_t)R * C;
  if (!dweight || (n > 0 && (!dy || !h || !weight || !dx))) return OSDN_ERR_NULL_ARG;
  const size_t need = residual_norm_backward_workspace_bytes(R, C);
  if (!workspace_ok(workspace, workspace_bytes, need)) return OSDN_ERR_WORKSPACE;
  const Range ins[] = {rng(dy, n * elem(dtype)), rng(h, n * elem(res_dtype)),
                       rng(dh, n * elem(res_dtype)), rng(weight, (size_t)C * 4)};
  const Range outs[] = {rng(dx, n * elem(dtype)), rng(dresidual, n * elem(res_dtype)),
                        rng(dweight, (size_t)C * 4), rng(workspace, need)};
  if (!aliasing_ok(outs, ins, nullptr, 0)) return OSDN_ERR_ALIASING;
  osdn::ResidualNormArgs a{};
  a.R = R; a.C = C; a.bf16 = dtype == OSDN_BF16; a.res_bf16 = res_dtype == OSDN_BF16;
  a.scale = scale; a.weight = weight; a.eps = eps; a.h = const_cast<void*>(h);
  a.dy = dy; a.dh = dh; a.dx = dx; a.dres = dresidual; a.dweight = dweight; a.ws = workspace;
  return status(osdn::launch_residual_norm_backward(a, (hipStream_t)stream));
}

// --- selective scan --------------------------------------------------------------

size_t ssm_forward_workspace_bytes(int B, int H, int G, int T, int P, int N, int dtype) {
  if (ssm_dims(B, H, G, T, P, N, dtype) != OSDN_OK) return 0;
  return round256(osdn::ssm_forward_ws(B, H, T, P, N, dtype == OSDN_BF16));
}

int ssm_forward(int B, int H, int G, int T, int P, int N, int dtype, const void* x,
                const float* dt, const float* A, const void* Bm, const void* Cm, const float* D,
                const float* dt_bias, int softplus, const float* S0, const int* lengths, void* y,
                float* S_T, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = ssm_dims(B, H, G, T, P, N, dtype);
  if (rc != OSDN_OK) return rc;
  const size_t BH = (size_t)B * H, es = elem(dtype), st = BH * P * N * 4;
  if (BH == 0) return OSDN_OK;
  if (!A || (T > 0 && (!x || !dt || !Bm || !Cm || !y))) return OSDN_ERR_NULL_ARG;
  const size_t need = ssm_forward_workspace_bytes(B, H, G, T, P, N, dtype);
  if (!workspace_ok(workspace, workspace_bytes, need)) return OSDN_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(Bm) || !aligned16(Cm) || !aligned16(y) || !aligned16(S0) ||
      !aligned16(S_T))
    return OSDN_ERR_MISALIGNED;
  const size_t tx = BH * T * P * es, tg = (size_t)B * G * T * N * es;
  const Range ins[] = {rng(x, tx), rng(dt, BH * T * 4), rng(A, (size_t)H * 4), rng(Bm, tg),
                       rng(Cm, tg), rng(D, (size_t)H * 4), rng(dt_bias, (size_t)H * 4),
                       rng(S0, st), rng(lengths, (size_t)B * 4)};
  const Range outs[] = {rng(y, tx), rng(S_T, st), rng(workspace, need)};
  const int allowed[][2] = {{1, 7}};  // S_T == S0
  if (!aliasing_ok(outs, ins, allowed, 1)) return OSDN_ERR_ALIASING;
  return status(osdn::launch_ssm_forward(
      ssm_args(B, H, G, T, P, N, dtype, x, dt, A, Bm, Cm, D, dt_bias, softplus, S0, lengths, y,
               S_T, workspace),
      (hipStream_t)stream));
}

int ssm_decode(int B, int H, int G, int T, int P, int N, int dtype, const void* x,
               const float* dt, const float* A, const void* Bm, const void* Cm, const float* D,
               const float* dt_bias, int softplus, const float* S, void* y, float* S_out,
               void* stream) {
  const int rc = ssm_dims(B, H, G, T, P, N, dtype);
  if (rc != OSDN_OK) return rc;
  const size_t BH = (size_t)B * H, es = elem(dtype), st = BH * P * N * 4;
  if (BH == 0) return OSDN_OK;
  if (!A || !S || !S_out || (T > 0 && (!x || !dt || !Bm || !Cm || !y))) return OSDN_ERR_NULL_ARG;
  if (!aligned16(x) || !aligned16(Bm) || !aligned16(Cm) || !aligned16(y) || !aligned16(S) ||
      !aligned16(S_out))
    return OSDN_ERR_MISALIGNED;
  const size_t tx = BH * T * P * es, tg = (size_t)B * G * T * N * es;
  const Range ins[] = {rng(x, tx), rng(dt, BH * T * 4), rng(A, (size_t)H * 4), rng(Bm, tg),
                       rng(Cm, tg), rng(D, (size_t)H * 4), rng(dt_bias, (size_t)H * 4),
                       rng(S, st)};
  const Range outs[] = {rng(y, tx), rng(S_out, st)};
  const int allowed[][2] = {{1, 7}};  // S_out == S
  if (!aliasing_ok(outs, ins, allowed, 1)) return OSDN_ERR_ALIASING;
  if (T == 0 && S_out == S) return OSDN_OK;
  return status(osdn::launch_ssm_decode(
      ssm_args(B, H, G, T, P, N, dtype, x, dt, A, Bm, Cm, D, dt_bias, softplus, S, nullptr, y,
               S_out, nullptr),
      (hipStream_t)stream));
}

size_t ssm_backward_workspace_bytes(int B, int H, int G, int T, int P, int N, int dtype) {
  if (ssm_dims(B, H, G, T, P, N, dtype) != OSDN_OK) return 0;
  return round256(osdn::ssm_backward_ws(B, H, G, T, P, N, dtype == OSDN_BF16));
}

int ssm_backward(int B, int H, int G, int T, int P, int N, int dtype, const void* x,
                 const float* dt, const float* A, const void* Bm, const void* Cm, const float* D,
                 const float* dt_bias, int softplus, const float* S0, const int* lengths,
                 const void* dy, const float* dS_T, void* dx, float* ddt, float* dA, void* dB,
                 void* dC, float* dD, float* ddt_bias, float* dS0, void* workspace,
                 size_t workspace_bytes, void* stream) {
  const int rc = ssm_dims(B, H, G, T, P, N, dtype);
  if (rc != OSDN_OK) return rc;
  const size_t BH = (size_t)B * H, es = elem(dtype), st = BH * P * N * 4;
  if (H == 0) return OSDN_OK;
  if (!A || !dA ||
      (BH * T > 0 && (!x || !dt || !Bm || !Cm || !dy || !dx || !ddt || !dB || !dC)))
    return OSDN_ERR_NULL_ARG;
  const size_t need = ssm_backward_workspace_bytes(B, H, G, T, P, N, dtype);
  if (!workspace_ok(workspace, workspace_bytes, need)) return OSDN_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(Bm) || !aligned16(Cm) || !aligned16(dy) || !aligned16(dx) ||
      !aligned16(dB) || !aligned16(dC) || !aligned16(S0) || !aligned16(dS_T) || !aligned16(dS0))
    return OSDN_ERR_MISALIGNED;
  const size_t tx = BH * T * P * es, tg = (size_t)B * G * T * N * es, hb = (size_t)H * 4;
  const Range ins[] = {rng(x, tx), rng(dt, BH * T * 4), rng(A, hb), rng(Bm, tg), rng(Cm, tg),
                       rng(D, hb), rng(dt_bias, hb), rng(S0, st), rng(lengths, (size_t)B * 4),
                       rng(dy, tx), rng(dS_T, st)};
  const Range outs[] = {rng(dx, tx), rng(ddt, BH * T * 4), rng(dA, hb), rng(dB, tg), rng(dC, tg),
                        rng(dD, hb), rng(ddt_bias, hb), rng(dS0, st), rng(workspace, need)};
  if (!aliasing_ok(outs, ins, nullptr, 0)) return OSDN_ERR_ALIASING;
  osdn::SsmArgs a = ssm_args(B, H, G, T, P, N, dtype, x, dt, A, Bm, Cm, D, dt_bias, softplus, S0,
                             lengths, nullptr, nullptr, workspace);
  a.dy = dy; a.dST = dS_T; a.dx = dx; a.dB = dB; a.dC = dC;
  a.ddt = ddt; a.dA = dA; a.dD = dD; a.dbias = ddt_bias; a.dS0 = dS0;
  return status(osdn::launch_ssm_backward(a, (hipStream_t)stream));
}

}  // extern "C"
