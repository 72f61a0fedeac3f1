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
// being 4, 8 or 16 adjacent lanes (16384 tokens of 32 heads of 128 bf16: 56 us for 269 MB,
// 4.8 TB/s; backward of 20 heads with fp32 adjoints 66 us for 336 MB, 5.1 TB/s, and 5 us
// of column sum). A workgroup takes a few tokens with all their
// heads, so that an angle is worked out once for all heads: in turns and in 64 bits,
// with what the product and 1 / (2 pi) lose to them (2^31 at a frequency of one is 2^28
// turns, of which 24 bits behind the point would be left), its cosine and sine in 32, left
// in LDS. Weight gradients stay in registers while a workgroup walks its
// tokens and leave as one partial row each, summed in a fixed order.
#include "launch.hpp"
#include "layer.hpp"
#include "row_common.hpp"

namespace osdn {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;         // rows that a lane has on their way

struct Turns {
  float2 cs[kThreads * 4];        // [token][pair] (cos, sin), 4 L pairs at most
};

// Turns of the angle p f, less whole ones.
__device__ __forceinline__ double turns(double p, double f) {
  constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;   // 1 / (2 pi)
  const double w = p * f, t = w * hi;
  const double rest = fma(w, lo, fma(p, f, -w) * hi);
  const double turn = fma(w, hi, -rint(t)) + rest;
  return turn - rint(turn);
}

// The cosines and sines of the tile's tokens; the caller's barrier follows.
__device__ __forceinline__ void fill_turns(const QkArgs& a, Turns& s, long long tok, int nt) {
  const unsigned np = a.rot / 2;
  for (unsigned e = threadIdx.x; e < nt * np; e += kThreads) {
    const unsigned i = e / np, j = e % np;
    const long long at = tok + i;
    const double p = a.positions ? (double)a.positions[at] : (double)(at % a.T);
    const double turn = turns(p, (double)a.inv_freq[j]);
    float sn, cs;
    sincospif(2.f * (float)turn, &sn, &cs);
    s.cs[i * np + j] = float2{cs, sn};
  }
}

// A lane's place in a tile: 8 channels from d on of one token, and the heads first,
// first + step, ... of it. Neighbouring rows of lanes take neighbouring tokens, whose
// rows lie side by side in the heads.
struct Place {
  bool in, on;           // the token exists; it lies inside its sequence
  int d, first, step;
  long long b, t;
  int partner;           // the lane that holds the other members of its pairs
  bool turned;
};
template <int L>
__device__ __forceinline__ Place place(const QkArgs& a, long long tok, int per, long long tokens) {
  Place p;
  const int row = threadIdx.x / L, l = threadIdx.x % L, lane = threadIdx.x & 63;
  const long long at = tok + row % per;
  p.in = at < tokens;
  p.b = p.in ? at / a.T : 0;
  p.t = p.in ? at % a.T : 0;
  p.on = p.in && (!a.lengths || p.t < a.lengths[p.b]);
  p.d = 8 * l;
  p.first = row / per;
  p.step = kThreads / L / per;    // (per is a power of two up to kThreads / L)
  p.turned = p.d < a.rot;
  // (rot / 2 channels away are rot / 16 lanes)
  const int hr = a.rot / 16;
  p.partner = a.interleaved || !p.turned ? lane : l < hr ? lane + hr : lane - hr;
  return p;
}

// A lane's part of the rotation, y_i = v_i c_i + w_i s_i with w the other members of the
// pairs; turning back, s changes its sign.
struct Rotation {
  float c[8], s[8];
};
__device__ __forceinline__ void rotation(const QkArgs& a, const Turns& t, const Place& p, int token,
                                         Rotation& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r.c[i] = 1.f;
    r.s[i] = 0.f;
  }
  if (!p.turned) return;
  const int np = a.rot / 2, half = p.d < np ? 0 : np;
  const float2* cs = t.cs + token * np;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 w = cs[a.interleaved ? p.d / 2 + i / 2 : p.d - half + i];
    r.c[i] = w.x;
    r.s[i] = (a.interleaved ? i % 2 == 0 : half == 0) ? -w.y : w.y;
  }
}

// The other members of a lane's pairs, as they lie in memory.
template <typename T>
__device__ __forceinline__ void others(const Raw<T, 8>& x, const QkArgs& a, const Place& p,
                                       float (&o)[8]) {
  if (a.interleaved) {
    float v[8];
    x.widen(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v[i ^ 1];
    return;
  }
  Raw<T, 8> y;
#pragma unroll
  for (int i = 0; i < Raw<T, 8>::W; ++i) y.u[i] = __shfl(x.u[i], p.partner, 64);
  y.widen(o);
}

template <int L>
__device__ __forceinline__ float root(const QkArgs& a, float ss) {
  const float m = group_sum<L>(ss), s = (a.norm == 1 ? m / (8 * L) : m) + a.eps;
  // (rows of zeros, those behind a sequence too, keep their zeros with eps = 0)
  return a.norm == 0 ? 1.f : s == 0.f ? 0.f : rsqrtf(s);
}

// One input (queries or keys): H heads of the lane's token. The weights of both members
// of a pair are multiplied into the rotation, which all heads share.
template <typename Tin, int L, bool ALN>
__device__ __forceinline__ void forward_rows(const QkArgs& a, const Place& p, const Rotation& r,
                                             int H, const Tin* x, long long bs, long long ts,
                                             const float* weight, Tin* y) {
  constexpr int D = 8 * L;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int o = a.interleaved ? p.d + (i ^ 1) : 8 * (p.partner % L) + i;
    c[i] = r.c[i] * (weight ? weight[p.d + i] : 1.f);
    s[i] = r.s[i] * (weight ? weight[o] : 1.f);
  }
  if (!p.in) return;
  x += p.b * bs + p.t * ts + p.d;
  y += (p.b * H * a.T + p.t) * D + p.d;
  const long long hs = (long long)a.T * D;
  for (int h = p.first; h < H; h += kBatch * p.step) {
    Raw<Tin, 8> v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      v[k].zero();
      if (p.on && h + k * p.step < H) v[k].template load<ALN>(x + (h + k * p.step) * D, 8);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (h + k * p.step >= H) break;      // (a head's lanes leave together)
      float w[8], o[8], ss = 0.f;
      v[k].widen(w);
      others(v[k], a, p, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(w[i], w[i], ss);
      const float n = root<L>(a, ss);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = w[i] * c[i];
        w[i] = (p.turned ? fmaf(o[i], s[i], t) : t) * n;
      }
      store_v<true, 8>(y + (h + k * p.step) * hs, 8, w);
    }
  }
}

template <typename Tin, int L, bool ALN>
__global__ __launch_bounds__(kThreads) void qk_rotary_kernel(QkArgs a, int per) {
  __shared__ Turns s;
  const long long tok = blockIdx.x * (long long)per, tokens = (long long)a.B * a.T;
  fill_turns(a, s, tok, (int)min((long long)per, tokens - tok));
  __syncthreads();
  const Place p = place<L>(a, tok, per, tokens);
  Rotation r;
  rotation(a, s, p, threadIdx.x / L % per, r);
  forward_rows<Tin, L, ALN>(a, p, r, a.Hq, (const Tin*)a.q, a.qbs, a.qts, a.wq, (Tin*)a.yq);
  forward_rows<Tin, L, ALN>(a, p, r, a.Hk, (const Tin*)a.k, a.kbs, a.kts, a.wk, (Tin*)a.yk);
}

template <typename Tin, typename Tdy, int L, bool ALN>
__device__ __forceinline__ void backward_rows(const QkArgs& a, const Place& p, const Rotation& r,
                                              int H, const Tin* x, long long bs, long long ts,
                                              const float* weight, const Tdy* dy, Tin* dx,
                                              float (&dw)[8]) {
  constexpr int D = 8 * L, B = kBatch;
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = weight ? weight[p.d + i] : 1.f;
  if (!p.in) return;
  x += p.b * bs + p.t * ts + p.d;
  dx += (p.b * a.T + p.t) * ((long long)H * D) + p.d;
  dy += (p.b * H * a.T + p.t) * D + p.d;
  const long long hs = (long long)a.T * D;
  for (int h = p.first; h < H; h += B * p.step) {
    Raw<Tin, 8> xs[B];
    Raw<Tdy, 8> gs[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      xs[k].zero();
      gs[k].zero();
      if (p.on && h + k * p.step < H) {
        xs[k].template load<ALN>(x + (h + k * p.step) * D, 8);
        gs[k].template load<true>(dy + (h + k * p.step) * hs, 8);
      }
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
      if (h + k * p.step >= H) break;
      float v[8], e[8], o[8], ss = 0.f, q = 0.f;
      xs[k].widen(v);
      gs[k].widen(e);
      others(gs[k], a, p, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = e[i] * r.c[i];
        e[i] = p.turned ? fmaf(-o[i], r.s[i], t) : t;
        ss = fmaf(v[i], v[i], ss);
        q = fmaf(v[i], e[i] * w[i], q);
      }
      const float n = root<L>(a, ss);
      // n (n . f): n^2 x (x . f), over D for the mean
      const float m = a.norm == 0 ? 0.f : group_sum<L>(q) * n * n * (a.norm == 1 ? 1.f / D : 1.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw[i] = fmaf(e[i] * v[i], n, dw[i]);
        v[i] = n * (e[i] * w[i] - v[i] * m);
      }
      store_v<true, 8>(dx + (h + k * p.step) * D, 8, v);
    }
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
    __syncthreads();   // the last tile's turns are read
    fill_turns(a, s, tok, (int)min((long long)per, tokens - tok));
    __syncthreads();
    const Place p = place<L>(a, tok, per, tokens);
    Rotation r;
    rotation(a, s, p, threadIdx.x / L % per, r);
    backward_rows<Tin, Tdy, L, ALN>(a, p, r, a.Hq, (const Tin*)a.q, a.qbs, a.qts, a.wq,
                                    (const Tdy*)a.dyq, (Tin*)a.dq, dwq);
    backward_rows<Tin, Tdy, L, ALN>(a, p, r, a.Hk, (const Tin*)a.k, a.kbs, a.kts, a.wk,
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

// Tokens a workgroup: as many as leave four workgroups a CU. All its rows of lanes on
// tokens of their own give the longest runs of memory: 16384 tokens of 32 heads of 128
// take 57 us at 16 tokens a tile and 62 at 8.
int tile_tokens(long long tokens, int L) {
  int per = kThreads / L;
  while (per > 1 && tokens / per < 1024) per /= 2;
  return per;
}

// Workgroups of the backward, each a partial row: the three a CU that its registers
// leave room for (16384 tokens of 20 heads: 73 us; with 1024 77 us, with 512 75 us).
int bwd_blocks(long long tokens, int L) {
  const int per = tile_tokens(tokens, L);
  const long long need = (tokens + per - 1) / per;
  return (int)(need < 768 ? need : 768);
}

template <typename Tin, int L, bool ALN>
int run_forward(const QkArgs& a, hipStream_t s) {
  const long long tokens = (long long)a.B * a.T;
  const int per = tile_tokens(tokens, L);
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
  const int nb = bwd_blocks(tokens, L);
  if (nb > 0) {
    const int tk = ktimer_before(s, "qk_rotary_bwd");
    hipLaunchKernelGGL((qk_rotary_bwd_kernel<Tin, Tdy, L, ALN>), dim3(nb), dim3(kThreads), 0, s, a,
                       tile_tokens(tokens, L));
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
  return (size_t)bwd_blocks((long long)B * T, D / 8) * 2 * D * sizeof(float);
}

int launch_qk_rotary_backward(const QkArgs& a, hipStream_t s) {
  return a.bf16 ? run_d<kBackward, __bf16>(a, s) : run_d<kBackward, float>(a, s);
}

}  // namespace osdn
