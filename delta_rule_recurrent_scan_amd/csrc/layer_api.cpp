// C ABI of the operators that complete a block: host-side validation, workspace
// sizing and launches of the gated linear recurrence, the rotary norm of queries
// and keys and the gated feed-forward product. Contract in include/osdn.h.
#include <hip/hip_runtime.h>

#include "api_common.hpp"
#include "layer.hpp"

using namespace osdn_api;

namespace {

typedef long long ll;

int status(int rc) {
  if (rc == -1) return OSDN_ERR_UNSUPPORTED;
  return rc == 0 ? OSDN_OK : OSDN_ERR_HIP;
}

constexpr int kMaxTokens = 1 << 30;

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws && bytes >= need && ((uintptr_t)ws & 255) == 0);
}

// Bytes that B x T rows of C elements with these strides span.
size_t span(ll B, ll T, ll C, ll bs, ll ts, size_t es) {
  if (B == 0 || T == 0 || C == 0) return 0;
  return ((size_t)(B - 1) * bs + (size_t)(T - 1) * ts + C) * es;
}

// --- gated linear recurrence ---------------------------------------------------

int glr_dims(int B, int T, int C, int dtype, const ll (&strides)[6], bool gate) {
  if (B < 0 || T < 0 || C < 0 || T > kMaxTokens) return OSDN_ERR_BAD_DIMS;
  for (int k = 0; k < (gate ? 6 : 4); ++k)
    if (strides[k] < 0) return OSDN_ERR_BAD_DIMS;
  if (!dtype_ok(dtype) || C > osdn::kGlrMaxStride) return OSDN_ERR_UNSUPPORTED;
  for (int k = 1; k < (gate ? 6 : 4); k += 2)
    if (strides[k] > osdn::kGlrMaxStride) return OSDN_ERR_UNSUPPORTED;
  return OSDN_OK;
}

osdn::GlrArgs glr_args(int B, int T, int C, int dtype, const void* x, const void* r,
                       const void* i, const ll (&st)[6], const float* A, const float* h0,
                       const int* lengths, int normalize) {
  osdn::GlrArgs a{};
  a.B = B; a.T = T; a.C = C; a.bf16 = dtype == OSDN_BF16;
  a.x = x; a.r = r; a.i = i;
  a.xbs = st[0]; a.xts = st[1]; a.rbs = st[2]; a.rts = st[3];
  a.ibs = i ? st[4] : 0; a.its = i ? st[5] : 0;
  a.A = A; a.h0 = h0; a.lengths = lengths; a.normalize = normalize;
  return a;
}

size_t state_bytes(int B, int T, int C) {
  return (size_t)B * ((T + OSDN_GLR_INTERVAL - 1) / OSDN_GLR_INTERVAL) * C * 4;
}

// --- rotary norm -----------------------------------------------------------------

int qk_dims(int B, int T, int Hq, int Hk, int D, int rot, int dtype, ll qbs, ll qts, ll kbs,
            ll kts, int norm) {
  if (B < 0 || T < 0 || Hq < 0 || Hk < 0 || rot < 0 || T > kMaxTokens || qbs < 0 || qts < 0 ||
      kbs < 0 || kts < 0 || (ll)Hq * D > (1 << 28) || (ll)Hk * D > (1 << 28))
    return OSDN_ERR_BAD_DIMS;
  if (!dim_ok(D) || !dtype_ok(dtype) || rot > D || rot % 16 != 0 || norm < OSDN_NORM_NONE ||
      norm > OSDN_NORM_L2)
    return OSDN_ERR_UNSUPPORTED;
  return OSDN_OK;
}

osdn::QkArgs qk_args(int B, int T, int Hq, int Hk, int D, int rot, int dtype, const void* q,
                     ll qbs, ll qts, const void* k, ll kbs, ll kts, const float* wq,
                     const float* wk, int norm, float eps, const float* inv_freq,
                     int interleaved, const int* positions, const int* lengths) {
  osdn::QkArgs a{};
  a.B = B; a.T = T; a.Hq = Hq; a.Hk = Hk; a.D = D; a.rot = rot; a.bf16 = dtype == OSDN_BF16;
  a.q = q; a.k = k; a.qbs = qbs; a.qts = qts; a.kbs = kbs; a.kts = kts;
  a.wq = wq; a.wk = wk; a.norm = norm; a.eps = eps; a.inv_freq = inv_freq;
  a.interleaved = interleaved; a.positions = positions; a.lengths = lengths;
  return a;
}

// --- gated feed-forward ------------------------------------------------------------

constexpr ll kFfnMax = 1LL << 21;

int ffn_dims(ll R, int C, int F, int dtype, ll xs, int act) {
  if (R < 0 || C < 0 || F < 0 || xs < 0 || R > (1LL << 31)) return OSDN_ERR_BAD_DIMS;
  if (!dtype_ok(dtype) || act < OSDN_ACT_SILU || act > OSDN_ACT_GELU_TANH || C > kFfnMax ||
      F > kFfnMax || xs > kFfnMax)
    return OSDN_ERR_UNSUPPORTED;
  return OSDN_OK;
}

// Where rows of C are whole eights the weights are read where they lie.
bool weights_ok(int C, const void* g, const void* u) {
  return C % 8 != 0 || (aligned16(g) && aligned16(u));
}

}  // namespace

extern "C" {

size_t glr_forward_workspace_bytes(int B, int T, int C) {
  if (glr_dims(B, T, C, OSDN_F32, {0, 0, 0, 0, 0, 0}, false) != OSDN_OK) return 0;
  return round256(osdn::glr_forward_ws(B, T, C));
}

int glr_forward(int B, int T, int C, int dtype, const void* x, ll x_batch_stride,
                ll x_token_stride, const void* r, ll r_batch_stride, ll r_token_stride,
                const void* i, ll i_batch_stride, ll i_token_stride, const float* A,
                const float* h0, const int* lengths, int normalize, void* y, float* h_T,
                float* states, void* workspace, size_t workspace_bytes, void* stream) {
  const ll st[6] = {x_batch_stride, x_token_stride, r_batch_stride,
                    r_token_stride, i_batch_stride, i_token_stride};
  const int rc = glr_dims(B, T, C, dtype, st, i != nullptr);
  if (rc != OSDN_OK) return rc;
  const size_t es = elem(dtype), n = (size_t)B * T * C, col = (size_t)B * C * 4;
  if (col == 0) return OSDN_OK;
  if (!A || (n > 0 && (!x || !r))) return OSDN_ERR_NULL_ARG;
  const size_t need = glr_forward_workspace_bytes(B, T, C);
  if (!workspace_ok(workspace, workspace_bytes, need)) return OSDN_ERR_WORKSPACE;
  const Range ins[] = {rng(x, span(B, T, C, st[0], st[1], es)),
                       rng(r, span(B, T, C, st[2], st[3], es)),
                       rng(i, i ? span(B, T, C, st[4], st[5], es) : 0), rng(A, (size_t)C * 4),
                       rng(h0, col), rng(lengths, (size_t)B * 4)};
  const Range outs[] = {rng(y, n * es), rng(h_T, col), rng(states, state_bytes(B, T, C)),
                        rng(workspace, need)};
  if (!aliasing_ok(outs, ins, nullptr, 0)) return OSDN_ERR_ALIASING;
  osdn::GlrArgs a = glr_args(B, T, C, dtype, x, r, i, st, A, h0, lengths, normalize);
  a.y = y; a.hT = h_T; a.states = states; a.ws = workspace;
  return status(osdn::launch_glr_forward(a, (hipStream_t)stream));
}

int glr_decode(int B, int T, int C, int dtype, const void* x, ll x_batch_stride,
               ll x_token_stride, const void* r, ll r_batch_stride, ll r_token_stride,
               const void* i, ll i_batch_stride, ll i_token_stride, const float* A,
               const float* h, int normalize, void* y, float* h_out, void* stream) {
  const ll st[6] = {x_batch_stride, x_token_stride, r_batch_stride,
                    r_token_stride, i_batch_stride, i_token_stride};
  const int rc = glr_dims(B, T, C, dtype, st, i != nullptr);
  if (rc != OSDN_OK) return rc;
  const size_t es = elem(dtype), n = (size_t)B * T * C, col = (size_t)B * C * 4;
  if (col == 0) return OSDN_OK;
  if (!A || !h || !h_out || (n > 0 && (!x || !r || !y))) return OSDN_ERR_NULL_ARG;
  const Range ins[] = {rng(x, span(B, T, C, st[0], st[1], es)),
                       rng(r, span(B, T, C, st[2], st[3], es)),
                       rng(i, i ? span(B, T, C, st[4], st[5], es) : 0), rng(A, (size_t)C * 4),
                       rng(h, col)};
  const Range outs[] = {rng(y, n * es), rng(h_out, col)};
  const int allowed[][2] = {{1, 4}};  // h_out == h
  if (!aliasing_ok(outs, ins, allowed, 1)) return OSDN_ERR_ALIASING;
  if (T == 0 && h_out == h) return OSDN_OK;
  osdn::GlrArgs a = glr_args(B, T, C, dtype, x, r, i, st, A, h, nullptr, normalize);
  a.y = y; a.hT = h_out;
  return status(osdn::launch_glr_decode(a, (hipStream_t)stream));
}

size_t glr_backward_workspace_bytes(int B, int T, int C, int have_states) {
  if (glr_dims(B, T, C, OSDN_F32, {0, 0, 0, 0, 0, 0}, false) != OSDN_OK) return 0;
  return round256(osdn::glr_backward_ws(B, T, C, have_states));
}

int glr_backward(int B, int T, int C, int dtype, const void* x, ll x_batch_stride,
                 ll x_token_stride, const void* r, ll r_batch_stride, ll r_token_stride,
                 const void* i, ll i_batch_stride, ll i_token_stride, const float* A,
                 const float* h0, const int* lengths, int normalize, const float* states,
                 const void* dy, const float* dh_T, void* dx, void* dr, void* di, float* dA,
                 float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
  const ll st[6] = {x_batch_stride, x_token_stride, r_batch_stride,
                    r_token_stride, i_batch_stride, i_token_stride};
  const int rc = glr_dims(B, T, C, dtype, st, i != nullptr);
  if (rc != OSDN_OK) return rc;
  const size_t es = elem(dtype), n = (size_t)B * T * C, col = (size_t)B * C * 4;
  if (C == 0) return OSDN_OK;
  if (!A || !dA || (n > 0 && (!x || !r || !dy || !dx || !dr || (i && !di))))
    return OSDN_ERR_NULL_ARG;
  const size_t need = glr_backward_workspace_bytes(B, T, C, states != nullptr);
  if (!workspace_ok(workspace, workspace_bytes, need)) return OSDN_ERR_WORKSPACE;
  const Range ins[] = {rng(x, span(B, T, C, st[0], st[1], es)),
                       rng(r, span(B, T, C, st[2], st[3], es)),
                       rng(i, i ? span(B, T, C, st[4], st[5], es) : 0),
                       rng(A, (size_t)C * 4),
                       rng(h0, col),
                       rng(lengths, (size_t)B * 4),
                       rng(states, state_bytes(B, T, C)),
                       rng(dy, n * es),
                       rng(dh_T, col)};
  const Range outs[] = {rng(dx, n * es), rng(dr, n * es),       rng(di, i ? n * es : 0),
                        rng(dA, (size_t)C * 4), rng(dh0, col), rng(workspace, need)};
  if (!aliasing_ok(outs, ins, nullptr, 0)) return OSDN_ERR_ALIASING;
  osdn::GlrArgs a = glr_args(B, T, C, dtype, x, r, i, st, A, h0, lengths, normalize);
  a.states = const_cast<float*>(states); a.ws = workspace; a.dy = dy; a.dhT = dh_T;
  a.dx = dx; a.dr = dr; a.di = di; a.dA = dA; a.dh0 = dh0;
  return status(osdn::launch_glr_backward(a, (hipStream_t)stream));
}

int qk_rotary_forward(int B, int T, int Hq, int Hk, int D, int rot, int dtype, const void* q,
                      ll q_batch_stride, ll q_token_stride, const void* k, ll k_batch_stride,
                      ll k_token_stride, const float* q_weight, const float* k_weight, int norm,
                      float eps, const float* inv_freq, int interleaved, const int* positions,
                      const int* lengths, void* q_out, void* k_out, void* stream) {
  const int rc = qk_dims(B, T, Hq, Hk, D, rot, dtype, q_batch_stride, q_token_stride,
                         k_batch_stride, k_token_stride, norm);
  if (rc != OSDN_OK) return rc;
  const size_t tokens = (size_t)B * T, es = elem(dtype), cq = (size_t)Hq * D, ck = (size_t)Hk * D;
  if (tokens * (cq + ck) == 0) return OSDN_OK;
  if ((cq && (!q || !q_out)) || (ck && (!k || !k_out)) || (rot && !inv_freq))
    return OSDN_ERR_NULL_ARG;
  if (!aligned16(q_out) || !aligned16(k_out)) return OSDN_ERR_MISALIGNED;
  const Range ins[] = {rng(q, span(B, T, cq, q_batch_stride, q_token_stride, es)),
                       rng(k, span(B, T, ck, k_batch_stride, k_token_stride, es)),
                       rng(q_weight, (size_t)D * 4), rng(k_weight, (size_t)D * 4),
                       rng(inv_freq, (size_t)rot * 2), rng(positions, tokens * 4),
                       rng(lengths, (size_t)B * 4)};
  const Range outs[] = {rng(q_out, tokens * cq * es), rng(k_out, tokens * ck * es)};
  if (!aliasing_ok(outs, ins, nullptr, 0)) return OSDN_ERR_ALIASING;
  osdn::QkArgs a = qk_args(B, T, Hq, Hk, D, rot, dtype, q, q_batch_stride, q_token_stride, k,
                           k_batch_stride, k_token_stride, q_weight, k_weight, norm, eps,
                           inv_freq, interleaved, positions, lengths);
  a.yq = q_out; a.yk = k_out;
  return status(osdn::launch_qk_rotary(a, (hipStream_t)stream));
}

size_t qk_rotary_backward_workspace_bytes(int B, int T, int D) {
  if (qk_dims(B, T, 0, 0, D, 0, OSDN_F32, 0, 0, 0, 0, 0) != OSDN_OK) return 0;
  return round256(osdn::qk_rotary_backward_ws(B, T, D));
}

int qk_rotary_backward(int B, int T, int Hq, int Hk, int D, int rot, int dtype, int dy_dtype,
                       const void* q, ll q_batch_stride, ll q_token_stride, const void* k,
                       ll k_batch_stride, ll k_token_stride, const float* q_weight,
                       const float* k_weight, int norm, float eps, const float* inv_freq,
                       int interleaved, const int* positions, const int* lengths,
                       const void* dq_out, const void* dk_out, void* dq, void* dk,
                       float* dq_weight, float* dk_weight, void* workspace,
                       size_t workspace_bytes, void* stream) {
  const int rc = qk_dims(B, T, Hq, Hk, D, rot, dtype, q_batch_stride, q_token_stride,
                         k_batch_stride, k_token_stride, norm);
  if (rc != OSDN_OK) return rc;
  if (!dtype_ok(dy_dtype) || (dtype == OSDN_F32 && dy_dtype == OSDN_BF16))
    return OSDN_ERR_UNSUPPORTED;
  const size_t tokens = (size_t)B * T, es = elem(dtype), ey = elem(dy_dtype),
               cq = (size_t)Hq * D, ck = (size_t)Hk * D;
  if (tokens > 0 && ((cq && (!q || !dq_out || !dq)) || (ck && (!k || !dk_out || !dk)) ||
                     (rot && !inv_freq)))
    return OSDN_ERR_NULL_ARG;
  if (!aligned16(dq_out) || !aligned16(dk_out) || !aligned16(dq) || !aligned16(dk))
    return OSDN_ERR_MISALIGNED;
  const size_t need = qk_rotary_backward_workspace_bytes(B, T, D);
  if (!workspace_ok(workspace, workspace_bytes, need)) return OSDN_ERR_WORKSPACE;
  const Range ins[] = {rng(q, span(B, T, cq, q_batch_stride, q_token_stride, es)),
                       rng(k, span(B, T, ck, k_batch_stride, k_token_stride, es)),
                       rng(q_weight, (size_t)D * 4), rng(k_weight, (size_t)D * 4),
                       rng(inv_freq, (size_t)rot * 2), rng(positions, tokens * 4),
                       rng(lengths, (size_t)B * 4), rng(dq_out, tokens * cq * ey),
                       rng(dk_out, tokens * ck * ey)};
  const Range outs[] = {rng(dq, tokens * cq * es), rng(dk, tokens * ck * es),
                        rng(dq_weight, (size_t)D * 4), rng(dk_weight, (size_t)D * 4),
                        rng(workspace, need)};
  if (!aliasing_ok(outs, ins, nullptr, 0)) return OSDN_ERR_ALIASING;
  osdn::QkArgs a = qk_args(B, T, Hq, Hk, D, rot, dtype, q, q_batch_stride, q_token_stride, k,
                           k_batch_stride, k_token_stride, q_weight, k_weight, norm, eps,
                           inv_freq, interleaved, positions, lengths);
  a.dy_bf16 = dy_dtype == OSDN_BF16;
  a.dyq = dq_out; a.dyk = dk_out; a.dq = dq; a.dk = dk;
  a.dwq = dq_weight; a.dwk = dk_weight; a.ws = workspace;
  return status(osdn::launch_qk_rotary_backward(a, (hipStream_t)stream));
}

size_t gated_ffn_forward_workspace_bytes(ll R, int C, int F, int dtype) {
  if (ffn_dims(R, C, F, dtype, 0, 0) != OSDN_OK) return 0;
  return round256(osdn::ffn_forward_ws(R, C, F, dtype == OSDN_BF16));
}

int gated_ffn_forward(ll R, int C, int F, int dtype, const void* x, ll x_row_stride,
                      const void* w_gate, const void* w_up, int activation, void* h, void* gate,
                      void* up, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = ffn_dims(R, C, F, dtype, x_row_stride, activation);
  if (rc != OSDN_OK) return rc;
  const size_t es = elem(dtype), n = (size_t)R * F, nw = (size_t)F * C;
  if (n == 0) return OSDN_OK;
  if (!h || (C > 0 && (!x || !w_gate || !w_up)) || (gate == nullptr) != (up == nullptr))
    return OSDN_ERR_NULL_ARG;
  if (!weights_ok(C, w_gate, w_up)) return OSDN_ERR_MISALIGNED;
  const size_t need = gated_ffn_forward_workspace_bytes(R, C, F, dtype);
  if (!workspace_ok(workspace, workspace_bytes, need)) return OSDN_ERR_WORKSPACE;
  const Range ins[] = {rng(x, span(1, R, C, 0, x_row_stride, es)), rng(w_gate, nw * es),
                       rng(w_up, nw * es)};
  const Range outs[] = {rng(h, n * es), rng(gate, n * es), rng(up, n * es),
                        rng(workspace, need)};
  if (!aliasing_ok(outs, ins, nullptr, 0)) return OSDN_ERR_ALIASING;
  osdn::FfnArgs a{};
  a.R = R; a.C = C; a.F = F; a.bf16 = dtype == OSDN_BF16; a.x = x; a.xs = x_row_stride;
  a.wg = w_gate; a.wu = w_up; a.act = activation; a.h = h; a.gate = gate; a.up = up;
  a.ws = workspace;
  return status(osdn::launch_ffn_forward(a, (hipStream_t)stream));
}

size_t gated_ffn_backward_workspace_bytes(ll R, int C, int F, int dtype) {
  if (ffn_dims(R, C, F, dtype, 0, 0) != OSDN_OK) return 0;
  return round256(osdn::ffn_backward_ws(R, C, F, dtype == OSDN_BF16));
}

int gated_ffn_backward(ll R, int C, int F, int dtype, const void* x, ll x_row_stride,
                       const void* w_gate, const void* w_up, const void* gate, const void* up,
                       int activation, const void* dh, void* dx, void* dw_gate, void* dw_up,
                       void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = ffn_dims(R, C, F, dtype, x_row_stride, activation);
  if (rc != OSDN_OK) return rc;
  const size_t es = elem(dtype), n = (size_t)R * F, nw = (size_t)F * C, nx = (size_t)R * C;
  if (C == 0) return OSDN_OK;
  if ((nx > 0 && (!x || !dx)) || (nw > 0 && (!w_gate || !w_up || !dw_gate || !dw_up)) ||
      (n > 0 && (!gate || !up || !dh)))
    return OSDN_ERR_NULL_ARG;
  if (!weights_ok(C, w_gate, w_up)) return OSDN_ERR_MISALIGNED;
  const size_t need = gated_ffn_backward_workspace_bytes(R, C, F, dtype);
  if (!workspace_ok(workspace, workspace_bytes, need)) return OSDN_ERR_WORKSPACE;
  const Range ins[] = {rng(x, span(1, R, C, 0, x_row_stride, es)), rng(w_gate, nw * es),
                       rng(w_up, nw * es), rng(gate, n * es), rng(up, n * es), rng(dh, n * es)};
  const Range outs[] = {rng(dx, nx * es), rng(dw_gate, nw * es), rng(dw_up, nw * es),
                        rng(workspace, need)};
  if (!aliasing_ok(outs, ins, nullptr, 0)) return OSDN_ERR_ALIASING;
  osdn::FfnArgs a{};
  a.R = R; a.C = C; a.F = F; a.bf16 = dtype == OSDN_BF16; a.x = x; a.xs = x_row_stride;
  a.wg = w_gate; a.wu = w_up; a.act = activation;
  a.gate = const_cast<void*>(gate); a.up = const_cast<void*>(up);
  a.dh = dh; a.dx = dx; a.dwg = dw_gate; a.dwu = dw_up; a.ws = workspace;
  return status(osdn::launch_ffn_backward(a, (hipStream_t)stream));
}

}  // extern "C"
