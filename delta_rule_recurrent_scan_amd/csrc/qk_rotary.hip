// Norm and rotation of queries and keys, from the token rows of a projection to
// the heads that the recurrences read. Per token (position p) and head:
//   n = x r,  r = 1 / sqrt(mean_D x^2 + eps)  (rms),  1 / sqrt(sum x^2 + eps)  (l2), 1
//   v = n * weight
//   (y_a, y_b) = (v_a cos - v_b sin, v_b cos + v_a sin),  angle p inv_freq_j
// for the rot / 2 pairs j: channels (j, j + rot / 2), or (2 j, 2 j + 1) when
// interleaved; channels from rot on pass through. Backward: the adjoint turned
// back, e, then dweight = sum e n and, with f = e * weight,
//   dx = r (f - n mean(n f))   (l2: sum; none: dx = f).
//
// Bound by HBM: every row is read and written once, 8 channels a lane, a head
// being 4, 8 or 16 adjacent lanes. A workgroup takes a few tokens with all their
// heads, so that an angle is worked out once for all heads: in turns and in 64
// bits (a position of 2^31 keeps 29 bits of its turn), its cosine and sine in 32,
// left in LDS. Weight gradients stay in registers while a workgroup walks its
// tokens and leave as one partial row each, summed in a fixed order.
#include "launch.hpp"
#include "layer.hpp"
#include "row_common.hpp"

namespace osdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;     // tokens of a workgroup's tile
constexpr int kMaxPairs = 64;     // D / 2 at most

struct Turns {
  float2 cs[kMaxTokens * kMaxPairs];   // [token][pair] (cos, sin)
  int b[kMaxTokens], t[kMaxTokens], on[kMaxTokens];
};

// The tile's tokens with their cosines and sines; the caller's barrier follows.
__device__ __forceinline__ void fill_turns(const QkArgs& a, Turns& s, long long tok, int nt) {
  const unsigned np = a.rot / 2;
  if ((int)threadIdx.x < nt) {
    const long long at = tok + threadIdx.x;
    const int b = (int)(at / a.T), t = (int)(at % a.T);
    s.b[threadIdx.x] = b;
    s.t[threadIdx.x] = t;
    s.on[threadIdx.x] = !a.lengths || t < a.lengths[b];
  }
  for (unsigned e = threadIdx.x; e < nt * np; e += kThreads) {
    const unsigned i = e / np, j = e % np;
    const long long at = tok + i;
    const double p = a.positions ? (double)a.positions[at] : (double)(at % a.T);
    double turn = p * (double)a.inv_freq[j] * 0.15915494309189533577;
    turn -= rint(turn);
    float sn, cs;
    sincospif(2.f * (float)turn, &sn, &cs);
    s.cs[i * np + j] = float2{cs, sn};
  }
}

// The rotation of a lane's channels d .. d + 7 of a head (L lanes); sign -1
// turns back. Every lane of the head calls it.
template <int L>
__device__ __forceinline__ void turn(float (&v)[8], const float2* cs, int d, int rot,
                                     int interleaved, float sign) {
  if (rot == 0) return;
  if (interleaved) {
    if (d < rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 w = cs[d / 2 + i];
        const float x = v[2 * i], y = v[2 * i + 1], s = w.y * sign;
        v[2 * i] = x * w.x - y * s;
        v[2 * i + 1] = y * w.x + x * s;
      }
    }
    return;
  }
  // the other member of a pair is rot / 2 channels away, rot / 16 lanes
  const int hr = rot / 16, l = d / 8, lane = threadIdx.x & 63;
  const int other = l < hr ? lane + hr : l < 2 * hr ? lane - hr : lane;
  const float s = l < hr ? -sign : sign;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float o = __shfl(v[i], other, 64);
    if (l < 2 * hr) {
      const float2 w = cs[(l < hr ? d : d - rot / 2) + i];
      v[i] = v[i] * w.x + o * (w.y * s);
    }
  }
}

template <int L>
__device__ __forceinline__ float root(const QkArgs& a, float ss) {
  const float m = group_sum<L>(ss);
  return a.norm == 0 ? 1.f : rsqrtf((a.norm == 1 ? m / (8 * L) : m) + a.eps);
}

// One input (queries or keys): H heads of every token of the tile.
template <typename Tin, int L, bool ALN>
__device__ __forceinline__ void forward_rows(const QkArgs& a, const Turns& s, long long tok, int nt,
                                             int H, const Tin* x, long long bs, long long ts,
                                             const float* weight, Tin* y) {
  constexpr int D = 8 * L, per = kThreads / L;
  const int d = (threadIdx.x % L) * 8, np = a.rot / 2;
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = weight ? weight[d + i] : 1.f;
  for (unsigned e = threadIdx.x / L; e < (unsigned)(nt * H); e += per) {
    const unsigned i = e / (unsigned)H, h = e % (unsigned)H;
    const long long b = s.b[i], t = s.t[i];
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
    if (s.on[i]) load_v<ALN, 8>(x + b * bs + t * ts + h * D + d, 8, v);
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) ss += v[k] * v[k];
    const float r = root<L>(a, ss);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= r * w[k];
    turn<L>(v, s.cs + i * np, d, a.rot, a.interleaved, 1.f);
    store_v<true, 8>(y + ((b * H + h) * (long long)a.T + t) * D + d, 8, v);
  }
}

template <typename Tin, int L, bool ALN>
__global__ __launch_bounds__(kThreads) void qk_rotary_kernel(QkArgs a, int per) {
  __shared__ Turns s;
  const long long tok = blockIdx.x * (long long)per, tokens = (long long)a.B * a.T;
  const int nt = (int)min((long long)per, tokens - tok);
  fill_turns(a, s, tok, nt);
  __syncthreads();
  forward_rows<Tin, L, ALN>(a, s, tok, nt, a.Hq, (const Tin*)a.q, a.qbs, a.qts, a.wq, (Tin*)a.yq);
  forward_rows<Tin, L, ALN>(a, s, tok, nt, a.Hk, (const Tin*)a.k, a.kbs, a.kts, a.wk, (Tin*)a.yk);
}

template <typename Tin, typename Tdy, int L, bool ALN>
__device__ __forceinline__ void backward_rows(const QkArgs& a, const Turns& s, long long tok,
                                              int nt, int H, const Tin* x, long long bs,
                                              long long ts, const float* weight, const Tdy* dy,
                                              Tin* dx, float (&dw)[8]) {
  constexpr int D = 8 * L, per = kThreads / L;
  const int d = (threadIdx.x % L) * 8, np = a.rot / 2;
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = weight ? weight[d + i] : 1.f;
  for (unsigned e = threadIdx.x / L; e < (unsigned)(nt * H); e += per) {
    const unsigned i = e / (unsigned)H, h = e % (unsigned)H;
    const long long b = s.b[i], t = s.t[i];
    float v[8], g[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = g[k] = 0.f;
    if (s.on[i]) {
      load_v<ALN, 8>(x + b * bs + t * ts + h * D + d, 8, v);
      load_v<true, 8>(dy + ((b * H + h) * (long long)a.T + t) * D + d, 8, g);
    }
    turn<L>(g, s.cs + i * np, d, a.rot, a.interleaved, -1.f);
    float ss = 0.f, q = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      ss += v[k] * v[k];
      q += v[k] * g[k] * w[k];
    }
    const float r = root<L>(a, ss);
    // n (n . f): r^2 x (x . f), over D for the mean
    const float m = a.norm == 0 ? 0.f : group_sum<L>(q) * r * r * (a.norm == 1 ? 1.f / D : 1.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      dw[k] += g[k] * v[k] * r;
      v[k] = r * (g[k] * w[k] - v[k] * m);
    }
    store_v<true, 8>(dx + (tok + i) * ((long long)H * D) + h * D + d, 8, v);
  }
}

// parts: [gridDim.x][2 D], the workgroups' sums of dweight (queries, keys).
template <typename Tin, typename Tdy, int L, bool ALN>
__global__ __launch_bounds__(kThreads) void qk_rotary_bwd_kernel(QkArgs a, int per) {
  __shared__ Turns s;
  __shared__ float red[kThreads * 9];
  constexpr int D = 8 * L;
  const long long tokens = (long long)a.B * a.T;
  float dwq[8] = {}, dwk[8] = {};
  for (long long tok = blockIdx.x * (long long)per; tok < tokens;
       tok += (long long)gridDim.x * per) {
    const int nt = (int)min((long long)per, tokens - tok);
    __syncthreads();   // the last tile's turns are read
    fill_turns(a, s, tok, nt);
    __syncthreads();
    backward_rows<Tin, Tdy, L, ALN>(a, s, tok, nt, a.Hq, (const Tin*)a.q, a.qbs, a.qts, a.wq,
                                    (const Tdy*)a.dyq, (Tin*)a.dq, dwq);
    backward_rows<Tin, Tdy, L, ALN>(a, s, tok, nt, a.Hk, (const Tin*)a.k, a.kbs, a.kts, a.wk,
                                    (const Tdy*)a.dyk, (Tin*)a.dk, dwk);
  }
  float* part = (float*)a.ws + (size_t)blockIdx.x * 2 * D;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) red[threadIdx.x * 9 + i] = which ? dwk[i] : dwq[i];
    __syncthreads();
    if (threadIdx.x < D) {
      float sum = 0.f;
      for (int r = threadIdx.x / 8; r < kThreads; r += L) sum += red[r * 9 + threadIdx.x % 8];
      part[which * D + threadIdx.x] = sum;
    }
  }
}

// Tokens a workgroup: as many as leave four workgroups a CU, up to eight.
int tile_tokens(long long tokens) {
  int per = kMaxTokens;
  while (per > 1 && tokens / per < 1024) per /= 2;
  return per;
}

// Workgroups of the backward, each a partial row: four a CU at most.
int bwd_blocks(long long tokens) {
  const int per = tile_tokens(tokens);
  const long long need = (tokens + per - 1) / per;
  return (int)(need < 1024 ? need : 1024);
}

template <typename Tin, int L, bool ALN>
int run_forward(const QkArgs& a, hipStream_t s) {
  const long long tokens = (long long)a.B * a.T;
  const int per = tile_tokens(tokens);
  const long long wgs = (tokens + per - 1) / per;
  if (!grid_ok(wgs, kThreads)) return -1;
  const int tk = ktimer_before(s, "qk_rotary");
  hipLaunchKernelGGL((qk_rotary_kernel<Tin, L, ALN>), dim3((unsigned)wgs), dim3(kThreads), 0, s, a,
                     per);
  ktimer_after(s, tk);
  return (int)hipGetLastError();
}

template <typename Tin, typename Tdy, int L, bool ALN>
int run_backward(const QkArgs& a, hipStream_t s) {
  const long long tokens = (long long)a.B * a.T;
  const int nb = bwd_blocks(tokens);
  if (nb > 0) {
    const int tk = ktimer_before(s, "qk_rotary_bwd");
    hipLaunchKernelGGL((qk_rotary_bwd_kernel<Tin, Tdy, L, ALN>), dim3(nb), dim3(kThreads), 0, s, a,
                       tile_tokens(tokens));
    ktimer_after(s, tk);
    const int rc = (int)hipGetLastError();
    if (rc) return rc;
  }
  const int D = 8 * L;
  const float* parts = (const float*)a.ws;
  if (!a.dwq && !a.dwk) return 0;
  return launch_column_sum(parts, nb, 2 * D, D, 0, nullptr, a.dwq, a.dwk, s);
}

enum Call { kForward, kBackward };

template <Call CALL, typename Tin, int L, bool ALN>
int run_dy(const QkArgs& a, hipStream_t s) {
  if constexpr (CALL == kForward) return run_forward<Tin, L, ALN>(a, s);
  return a.dy_bf16 == (sizeof(Tin) == 2) ? run_backward<Tin, Tin, L, ALN>(a, s)
                                         : run_backward<Tin, float, L, ALN>(a, s);
}

template <Call CALL, typename Tin, int L>
int run_l(const QkArgs& a, hipStream_t s) {
  const size_t es = sizeof(Tin);
  const size_t bits = (size_t)a.q | (size_t)a.k | (size_t)(a.qbs * es) | (size_t)(a.qts * es) |
                      (size_t)(a.kbs * es) | (size_t)(a.kts * es);
  return (bits & 15) == 0 ? run_dy<CALL, Tin, L, true>(a, s) : run_dy<CALL, Tin, L, false>(a, s);
}

template <Call CALL, typename Tin>
int run_d(const QkArgs& a, hipStream_t s) {
  switch (a.D) {
    case 32: return run_l<CALL, Tin, 4>(a, s);
    case 64: return run_l<CALL, Tin, 8>(a, s);
    case 128: return run_l<CALL, Tin, 16>(a, s);
  }
  return -1;
}

}  // namespace

int launch_qk_rotary(const QkArgs& a, hipStream_t s) {
  return a.bf16 ? run_d<kForward, __bf16>(a, s) : run_d<kForward, float>(a, s);
}

size_t qk_rotary_backward_ws(int B, int T, int D) {
  return (size_t)bwd_blocks((long long)B * T) * 2 * D * sizeof(float);
}

int launch_qk_rotary_backward(const QkArgs& a, hipStream_t s) {
  return a.bf16 ? run_d<kBackward, __bf16>(a, s) : run_d<kBackward, float>(a, s);
}

}  // namespace osdn
