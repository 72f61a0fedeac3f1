// Host-side argument bundles of the operators around the recurrences: the
// short causal convolution, the gated head norm, the residual norm and the
// selective state space scan. Pointers are device pointers owned by the
// caller; every launcher returns a hipError_t-compatible code (0 = success)
// or -1 when the sizes have no kernel instance.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace osdn {

// Channels are handled in groups of 8 per thread (16 bytes of bf16); a
// workgroup of 256 threads covers `cx` groups (a power of two, at most 64)
// times 256 / cx rows.
constexpr int kRowThreads = 256;

// A launch holds fewer than 2^32 threads; a call that needs more is refused.
inline bool grid_ok(long long blocks, int threads) {
  return blocks < (1LL << 32) / threads;
}

// The column sum below: 32 columns a workgroup of 1024 threads.
inline bool column_sum_ok(long long cols) { return grid_ok((cols + 31) / 32, 1024); }

inline int row_cx(long long ngroups) {
  int cx = 1;
  while (cx < 64 && cx < ngroups) cx *= 2;
  return cx;
}

struct ConvArgs {
  int B, T, H, D, W;
  int bf16;
  const void* x;              // [B,T,C] rows of C = H*D channels
  long long xbs, xts;         // strides of x in elements
  const float* weight;        // [C,W]
  const float* bias;          // [C] or null
  const void* state0;         // [B,W-1,C] or null (zeros)
  const int* lengths;         // [B] or null (T each)
  int act, l2;
  float eps;
  void* y;                    // [B,H,T,D]
  void* stateT;               // [B,W-1,C] or null
  int whole;                  // one thread walks all T tokens of a channel
};

struct ConvBackwardArgs {
  ConvArgs f;                 // y, stateT, whole unused
  int dy_bf16;
  const void* dy;             // [B,H,T,D]
  const void* dstateT;        // [B,W-1,C] or null (zeros)
  void* dx;                   // [B,T,C] contiguous
  void* dstate0;              // [B,W-1,C] or null
  float* dweight;             // [C,W]
  float* dbias;               // [C] or null
  void* ws;
};

struct GatedNormArgs {
  int B, H, T, D;
  int bf16;
  const void* x;              // [B,H,T,D]
  const void* z;              // [B,T,H*D] rows, or null (no gate)
  long long zbs, zts;
  const float* weight;        // [D], or [H,D] when per_head
  int per_head, gate_first;
  float eps;
  void* y;                    // [B,T,H*D]
  // backward
  const void* dy;             // [B,T,H*D]
  void* dx;                   // [B,H,T,D]
  void* dz;                   // [B,T,H*D] or null without a gate
  float* dweight;
  void* ws;
};

struct ResidualNormArgs {
  long long R;
  int C;
  int bf16, res_bf16;
  const void* x;              // [R,C]
  const void* residual;       // [R,C] or null
  float scale;
  const float* weight;        // [C]
  float eps;
  void* y;                    // [R,C]
  void* h;                    // [R,C] residual dtype (forward: out, may be null; backward: in)
  // backward
  const void* dy;             // [R,C]
  const void* dh;             // [R,C] or null
  void* dx;                   // [R,C]
  void* dres;                 // [R,C] or null
  float* dweight;             // [C]
  void* ws;
};

// Inputs and outputs of the selective scan; G groups of H / G heads share
// Bm and Cm.
struct SsmArgs {
  int B, H, G, T, P, N;
  int bf16;
  const void* x;              // [B,H,T,P]
  const float* dt;            // [B,H,T]
  const float* A;             // [H]
  const void *Bm, *Cm;        // [B,G,T,N]
  const float* D;             // [H] or null (zeros)
  const float* dt_bias;       // [H] or null (zeros)
  int softplus;
  const float* S0;            // [B,H,P,N] or null (zeros)
  const int* lengths;         // [B] or null
  void* y;                    // [B,H,T,P]
  float* ST;                  // [B,H,P,N] or null
  void* ws;
  // backward
  const void* dy;             // [B,H,T,P]
  const float* dST;           // [B,H,P,N] or null (zeros)
  void *dx, *dB, *dC;         // dtype
  float *ddt, *dA, *dD, *dbias, *dS0;  // dD, dbias, dS0 may be null
};

int launch_short_conv(const ConvArgs& a, hipStream_t s);
size_t short_conv_backward_ws(int B, int T, int H, int D, int W);
int launch_short_conv_backward(const ConvBackwardArgs& a, hipStream_t s);
int launch_gated_norm(const GatedNormArgs& a, hipStream_t s);
size_t gated_norm_backward_ws(int B, int H, int T, int D);
int launch_gated_norm_backward(const GatedNormArgs& a, hipStream_t s);
int launch_residual_norm(const ResidualNormArgs& a, hipStream_t s);
size_t residual_norm_backward_ws(long long R, int C);
int launch_residual_norm_backward(const ResidualNormArgs& a, hipStream_t s);
int launch_ssm_decode(const SsmArgs& a, hipStream_t s);
int launch_ssm_forward(const SsmArgs& a, hipStream_t s);
size_t ssm_forward_ws(int B, int H, int T, int P, int N, int bf16);
int launch_ssm_backward(const SsmArgs& a, hipStream_t s);
size_t ssm_backward_ws(int B, int H, int G, int T, int P, int N, int bf16);

// Column sums of fp32 partials [rows][cols]; column j goes to
// out0[(j % c) * w + j / c] while j / c < w, then to out1[j % c] and out2[j %
// c] (null: dropped). Parameter gradients are summed this way, in 64 bits and a fixed
// order, so that a call gives the same bits every time.
int launch_column_sum(const float* in, int rows, int cols, int c, int w,
                      float* out0, float* out1, float* out2, hipStream_t s);

}  // namespace osdn
