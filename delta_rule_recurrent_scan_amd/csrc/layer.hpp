// Host-side argument bundles of the operators that complete a block: the gated
// linear recurrence, the rotary norm of queries and keys and the gated
// feed-forward product. Pointers are device pointers owned by the caller;
// every launcher returns a hipError_t-compatible code (0 = success) or -1 when
// the sizes have no kernel instance.
#pragma once

#include "mixer.hpp"

namespace osdn {

// Tokens between the states that the recurrence's forward leaves.
constexpr int kGlrInterval = 16;
// Row strides (elements) up to which a tile of rows is addressed by 32-bit
// byte offsets.
constexpr long long kGlrMaxStride = 1LL << 22;

struct GlrArgs {
  int B, T, C;
  int bf16;
  const void *x, *r, *i;        // [B,T,C] rows; i may be null (no input gate)
  long long xbs, xts, rbs, rts, ibs, its;  // strides in elements
  const float* A;               // [C], <= 0
  const float* h0;              // [B,C] or null (zeros)
  const int* lengths;           // [B] or null (T each)
  int normalize;
  void* y;                      // [B,T,C] or null
  float* hT;                    // [B,C] or null
  float* states;                // [B,ceil(T/16),C] or null (forward: out, backward: in)
  void* ws;
  // backward
  const void* dy;               // [B,T,C]
  const float* dhT;             // [B,C] or null (zeros)
  void *dx, *dr, *di;           // [B,T,C]
  float *dA, *dh0;              // [C], [B,C] (dh0 may be null)
};

struct QkArgs {
  int B, T, Hq, Hk, D, rot;
  int bf16;
  const void *q, *k;            // [B,T,Hq*D], [B,T,Hk*D] rows
  long long qbs, qts, kbs, kts;
  const float *wq, *wk;         // [D] or null (ones)
  int norm;                     // 0 none, 1 rms, 2 l2
  float eps;
  const float* inv_freq;        // [rot / 2]
  int interleaved;
  const int* positions;         // [B,T] or null (0 .. T - 1)
  const int* lengths;           // [B] or null (T each)
  void *yq, *yk;                // [B,Hq,T,D], [B,Hk,T,D]
  // backward
  int dy_bf16;
  const void *dyq, *dyk;        // [B,Hq,T,D], [B,Hk,T,D]
  void *dq, *dk;                // [B,T,Hq*D], [B,T,Hk*D] contiguous
  float *dwq, *dwk;             // [D] or null
  void* ws;
};

int launch_qk_rotary(const QkArgs& a, hipStream_t s);
size_t qk_rotary_backward_ws(int B, int T, int D);
int launch_qk_rotary_backward(const QkArgs& a, hipStream_t s);

struct FfnArgs {
  long long R;
  int C, F;
  int bf16;
  const void* x;                // [R,C] rows
  long long xs;                 // their stride in elements
  const void *wg, *wu;          // [F,C]
  int act;                      // OSDN_ACT_*
  void *h, *gate, *up;          // [R,F]; gate and up: out (may be null) or, backward, in
  void* ws;
  // backward
  const void* dh;               // [R,F]
  void *dx, *dwg, *dwu;         // [R,C], [F,C], [F,C]
  // operands of the tiled products: rows of Cp and Fp elements, multiples of 8 (x and the
  // weights copied to ws with zeros behind C where theirs are not), dg, du [R,Fp] in ws
  int Cp, Fp;
  void *dg, *du;
  float* parts;
};

size_t ffn_forward_ws(long long R, int C, int F, int bf16);
int launch_ffn_forward(const FfnArgs& a, hipStream_t s);
size_t ffn_backward_ws(long long R, int C, int F, int bf16);
int launch_ffn_backward(const FfnArgs& a, hipStream_t s);

size_t glr_forward_ws(int B, int T, int C);
int launch_glr_forward(const GlrArgs& a, hipStream_t s);
int launch_glr_decode(const GlrArgs& a, hipStream_t s);
size_t glr_backward_ws(int B, int T, int C, int have_states);
int launch_glr_backward(const GlrArgs& a, hipStream_t s);

}  // namespace osdn
