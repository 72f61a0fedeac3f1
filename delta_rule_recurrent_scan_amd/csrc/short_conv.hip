// Short causal depthwise convolution with SiLU and, per head, an L2 row norm:
//   u_t = bias + sum_k weight[:, k] * x_{t - W + 1 + k}
//   v   = u * sigmoid(u)                               (activation)
//   y   = v * rsqrt(sum_head v^2 + eps)                (l2norm)
// from token rows x [B,T,C] (any row stride: a slice of a wider projection)
// to the heads [B,H,T,D] that the recurrences read, with the last W - 1
// inputs carried as a state.
//
// Bound by HBM: x is read once and y written once (2 x 2 bytes an element in
// bf16), some 15 VALU operations an element beside it. A thread owns 8
// consecutive channels and walks a segment of tokens with the last W - 1
// inputs and the weights in registers, so a wave moves 1 KB contiguous pieces
// of a row; a segment re-reads W - 1 rows of its predecessor (from L2). A
// head of 32, 64 or 128 channels is 4, 8 or 16 adjacent lanes, and its norm a
// DPP sum: no LDS. B 4, T 4096, 4096 channels of bf16 with the norm, 268 MB: 63
// us, 4.3 TB/s, where a copy of 256 MiB reaches 5.4 TB/s. Rows are fetched raw,
// eight in flight, and addressed by pointers that advance: widened at once, with an
// address formed a token, they took 84 us. A single token takes 4 to 8 us whether one
// sequence or 128, 256 channels or 2048: loads of weights, state and row in turn.
//
// Backward, with dv = r (dy - v r^2 <v, dy>) for the norm (r = rsqrt(..)),
// du = dv * sigmoid(u) (1 + u (1 - sigmoid(u))) and the inputs with their
// state as rows 0 .. T + W - 2:
//   dfull_r = sum_k weight[:, k] du_{r - k},  dweight_k = sum_t du_t full_{t+k}
// A thread recomputes u while it walks, keeps the W rows still open in
// registers and emits a row when its last term is in; weight gradients stay
// in registers over the segment, are added over the workgroup's segments in
// LDS, and leave as one partial a workgroup (summed in a fixed order by
// column_sum). 8 padded sequences of up to 2048 tokens, 2048 channels of bf16, at
// most 201 MB: 41 us; with 8 channels a thread and rows widened at once it was 82
// us (the open rows, the inputs and the weights leave room for few waves).
#include "launch.hpp"
#include "mixer.hpp"
#include "row_common.hpp"

namespace osdn {
namespace {

// Channels of a thread and tokens it fetches ahead.
constexpr int kFwdV = 8, kFwdBatch = 8, kBwdV = 4, kBwdBatch = 4;

template <typename T, int V>
struct ConvIn {
  const T* x;
  long long xts;
  const T* st;  // state rows of this batch entry, or null
  int C, W, c, nv;
  // row t of the inputs, t < 0 reading the state before them
  template <bool ALN>
  __device__ __forceinline__ void row(int t, float (&v)[V]) const {
    if (t >= 0) {
      load_v<ALN, V>(x + t * xts + c, nv, v);
    } else if (st) {
      load_v<ALN, V>(st + (size_t)(W - 1 + t) * C + c, nv, v);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = 0.f;
    }
  }
};

template <int W, int V>
__device__ __forceinline__ void load_weights(const float* weight, const float* bias, int c,
                                             int nv, float (&w)[W][V], float (&bi)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool ok = i < nv;
    bi[i] = ok && bias ? bias[c + i] : 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][i] = ok ? weight[(size_t)(c + i) * W + k] : 0.f;
  }
}

// A thread's channels in the heads [B,H,T,D]: one pointer that advances by D a
// token where its channels lie in one head, else an address an element.
template <typename T, int V, bool ALN>
struct Heads {
  T* p;  // channel c of token 0 (ALN)
  T* y;
  long long bh0;
  int Tn, D, c, nv;
  __device__ __forceinline__ Heads(T* base, long long bh, int T_, int D_, int c_, int nv_)
      : y(base), bh0(bh), Tn(T_), D(D_), c(c_), nv(nv_) {
    p = base + (bh + c_ / D_) * T_ * (long long)D_ + c_ % D_;
  }
  __device__ __forceinline__ T* at(int t, int i) const {
    return y + ((bh0 + (c + i) / D) * Tn + t) * (long long)D + (c + i) % D;
  }
  __device__ __forceinline__ void store(int t, const float (&v)[V]) const {
    if constexpr (ALN) {
      store_v<true, V>(p + t * (long long)D, V, v);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < nv) *at(t, i) = from_f32<T>(v[i]);
    }
  }
  __device__ __forceinline__ void load(int t, Raw<T, V>& r) const {
    if constexpr (ALN) {
      r.template load<true>(p + t * (long long)D, V);
    } else {
      float v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = i < nv ? to_f32(*at(t, i)) : 0.f;
      r.narrow(v);
    }
  }
};

template <typename Tin, int W, bool ALN>
__global__ __launch_bounds__(kRowThreads) void conv_kernel(ConvArgs a, int cx, int seg,
                                                           int nseg) {
  constexpr int V = kFwdV, NB = kFwdBatch;
  const int C = a.H * a.D, ng = (C + V - 1) / V;
  const int ncb = (ng + cx - 1) / cx, cb = blockIdx.x % ncb, rb = blockIdx.x / ncb;
  const int cg = cb * cx + (threadIdx.x & (cx - 1));
  const long long by = rb * (long long)(kRowThreads / cx) + threadIdx.x / cx;
  const int sg = (int)(by % nseg);
  const long long b = by / nseg;
  if (cg >= ng || b >= a.B) return;  // a head's lanes leave together
  const int c = cg * V, nv = C - c;
  int n = a.lengths ? a.lengths[b] : a.T;
  n = n < 0 ? 0 : n > a.T ? a.T : n;
  ConvIn<Tin, V> in{(const Tin*)a.x + b * a.xbs, a.xts,
                    a.state0 ? (const Tin*)a.state0 + b * (W - 1) * C : nullptr, C, W, c, nv};
  float w[W][V], bi[V];
  load_weights<W, V>(a.weight, a.bias, c, nv, w, bi);

  const int t0 = sg * seg, t1 = min(t0 + seg, a.T), tn = min(t1, n);
  const int L = a.D / V;  // lanes of a head (l2 only)
  const Heads<Tin, V, ALN> y((Tin*)a.y, b * a.H, a.T, a.D, c, nv);
  // h[0 .. W - 2]: the inputs before the batch; h[W - 1 + j]: the batch's
  float h[W - 1 + NB][V];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) in.template row<ALN>(t0 - (W - 1) + k, h[k]);
  auto token = [&](int t, int j) {
    float u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      u[i] = bi[i];
#pragma unroll
      for (int k = 0; k < W; ++k) u[i] += w[k][i] * h[j + k][i];
    }
    if (a.act) {
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] *= sigmoid_f(u[i]);
    }
    if (a.l2) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) s += u[i] * u[i];
      const float r = rsqrtf(head_sum(s, L) + a.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] *= r;
    }
    y.store(t, u);
  };
  int t = t0;
  const Tin* xp = in.x + t0 * in.xts + c;
  for (; t + NB <= tn; t += NB) {
    Raw<Tin, V> f[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j, xp += in.xts) f[j].template load<ALN>(xp, nv);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      f[j].widen(h[W - 1 + j]);
      token(t + j, j);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) h[k][i] = h[NB + k][i];
  }
  for (; t < tn; ++t, xp += in.xts) {
    load_v<ALN, V>(xp, nv, h[W - 1]);
    token(t, 0);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) h[k][i] = h[k + 1][i];
  }
  const float zero[V] = {};
  for (; t < t1; ++t) y.store(t, zero);

  if (sg == 0 && a.stateT) {
    // all rows read before any is written: state_T may be state0
    float f[W][V];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) in.template row<ALN>(n - (W - 1) + k, f[k]);
    Tin* st = (Tin*)a.stateT + b * (W - 1) * C + c;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_v<ALN, V>(st + (size_t)k * C, nv, f[k]);
  }
}

template <typename Tin, typename Tdy, int W, bool ALN>
__global__ __launch_bounds__(kRowThreads) void conv_bwd_kernel(ConvBackwardArgs p, int cx,
                                                               int seg, int nseg) {
  constexpr int V = kBwdV, NB = kBwdBatch;
  const ConvArgs& a = p.f;
  const int C = a.H * a.D, ng = (C + V - 1) / V;
  const int lx = threadIdx.x & (cx - 1), ly = threadIdx.x / cx;
  const int ncb = (ng + cx - 1) / cx, cb = blockIdx.x % ncb, rb = blockIdx.x / ncb;
  const int cg = cb * cx + lx;
  const long long by = rb * (long long)(kRowThreads / cx) + ly;
  const int sg = (int)(by % nseg);
  const long long b = by / nseg;
  const bool on = cg < ng && b < a.B;
  const int c = cg * V, nv = C - c;
  float dw[W + 1][V] = {};  // weight gradients, then the bias'
  if (on) {
    int n = a.lengths ? a.lengths[b] : a.T;
    n = n < 0 ? 0 : n > a.T ? a.T : n;
    ConvIn<Tin, V> in{(const Tin*)a.x + b * a.xbs, a.xts,
                      a.state0 ? (const Tin*)a.state0 + b * (W - 1) * C : nullptr, C, W, c, nv};
    float w[W][V], bi[V];
    load_weights<W, V>(a.weight, a.bias, c, nv, w, bi);
    const int L = a.D / V;
    // rows [r0, r1) of the T + W - 1 of the inputs with their state
    const int rows = a.T + W - 1;
    const int r0 = sg * seg, r1 = min(r0 + seg, rows);
    const Tin* dst = p.dstateT ? (const Tin*)p.dstateT + b * (W - 1) * C + c : nullptr;
    const Heads<Tdy, V, ALN> dyh((Tdy*)const_cast<void*>(p.dy), b * a.H, a.T, a.D, c, nv);
    Tin* dx = (Tin*)p.dx + (b * a.T - (W - 1)) * (long long)C + c;  // row t of them
    // h[0 .. W - 2]: the inputs before the batch; acc[k]: open row t + k
    float h[W - 1 + NB][V], acc[W][V] = {};
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int t = r0 - 2 * (W - 1) + k;
      if (t >= -(W - 1) && t < n) {
        in.template row<ALN>(t, h[k]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) h[k][i] = 0.f;
      }
    }
    // du_t of a token inside the sequence enters rows t .. t + W - 1
    auto inside = [&](int j, const float (&dy)[V], bool mine) {
      float u[V], d[V], sl[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        u[i] = bi[i];
#pragma unroll
        for (int k = 0; k < W; ++k) u[i] += w[k][i] * h[j + k][i];
        d[i] = dy[i];
        sl[i] = 1.f;
      }
      if (a.act) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float sgm = sigmoid_f(u[i]);
          sl[i] = sgm * (1.f + u[i] * (1.f - sgm));
          u[i] *= sgm;
        }
      }
      if (a.l2) {
        float s = 0.f, q = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s += u[i] * u[i];
          q += u[i] * d[i];
        }
        const float r = rsqrtf(head_sum(s, L) + a.eps);
        q = head_sum(q, L) * r * r;
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = r * (d[i] - u[i] * q);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        d[i] *= sl[i];
#pragma unroll
        for (int k = 0; k < W; ++k) acc[k][i] += w[k][i] * d[i];
        if (mine) {  // earlier tokens: a predecessor's sums
#pragma unroll
          for (int k = 0; k < W; ++k) dw[k][i] += d[i] * h[j + k][i];
          dw[W][i] += d[i];
        }
      }
    };
    auto close = [&]() {  // row t leaves the open ones
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[k][i] = acc[k + 1][i];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[W - 1][i] = 0.f;
    };
    // one token anywhere: before the sequence, in it or behind it
    auto any = [&](int t) {
      float dy[V];
      if (t >= -(W - 1) && t < n) {
        in.template row<ALN>(t, h[W - 1]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) h[W - 1][i] = 0.f;
      }
      if (t >= 0 && t < n) {
        Raw<Tdy, V> r;
        dyh.load(t, r);
        r.widen(dy);
        inside(0, dy, t >= r0);
      }
      if (t >= r0) {
        if (dst && t >= n && t < n + W - 1) {
          float f[V];
          load_v<ALN, V>(dst + (size_t)(t - n) * C, nv, f);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[0][i] += f[i];
        }
        if (t >= W - 1) {
          store_v<ALN, V>(dx + t * (long long)C, nv, acc[0]);
        } else if (p.dstate0) {
          store_v<ALN, V>((Tin*)p.dstate0 + (b * (W - 1) + t) * (long long)C + c, nv, acc[0]);
        }
      }
      close();
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) h[k][i] = h[k + 1][i];
    };
    int t = r0 - (W - 1);
    for (; t < max(r0, W - 1) && t < r1; ++t) any(t);
    // whole batches inside the sequence, every row an output row
    const Tin* xp = in.x + t * in.xts + c;
    for (; t + NB <= min(r1, n); t += NB) {
      Raw<Tin, V> f[NB];
      Raw<Tdy, V> e[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j, xp += in.xts) {
        f[j].template load<ALN>(xp, nv);
        dyh.load(t + j, e[j]);
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        float dy[V];
        f[j].widen(h[W - 1 + j]);
        e[j].widen(dy);
        inside(j, dy, true);
        store_v<ALN, V>(dx + (t + j) * (long long)C, nv, acc[0]);
        close();
      }
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) h[k][i] = h[NB + k][i];
    }
    for (; t < r1; ++t) any(t);
  }
  // the workgroup's segments added: one partial row [W + 1][C] a workgroup
  __shared__ float red[kRowThreads * (V + 1)];  // V + 1: adjacent threads on other banks
  float* part = (float*)p.ws + (size_t)rb * (W + 1) * C;
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) red[threadIdx.x * (V + 1) + i] = dw[k][i];
    __syncthreads();
    for (int e = threadIdx.x; e < cx * V; e += kRowThreads) {
      const int col = (cb * cx + e / V) * V + e % V;
      if (col >= C) continue;
      float s = 0.f;
      for (int r = 0; r < kRowThreads / cx; ++r) s += red[(r * cx + e / V) * (V + 1) + e % V];
      part[(size_t)k * C + col] = s;
    }
  }
}

// 32 columns and 32 row lanes a workgroup; a lane adds every 32nd row, eight
// in flight, then the lanes are added in LDS. In 64 bits, rounded once: the kernel
// waits for its rows, not for its sums.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ in, int rows,
                                                          int cols, int c, int w, float* out0,
                                                          float* out1, float* out2) {
  __shared__ double red[32][33];
  const int x = threadIdx.x & 31, r0 = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + x;
  double s[8] = {};
  if (j < cols) {
    const float* p = in + j;
    int r = r0;
    for (; r + 7 * 32 < rows; r += 8 * 32)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += p[(size_t)(r + 32 * i) * cols];
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (r + 32 * i < rows) s[i] += p[(size_t)(r + 32 * i) * cols];
  }
  red[r0][x] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  __syncthreads();
#pragma unroll
  for (int m = 16; m > 0; m /= 2) {
    if (r0 < m) red[r0][x] += red[r0 + m][x];
    __syncthreads();
  }
  if (r0 == 0 && j < cols) {
    const int k = j / c, ch = j % c;
    if (k < w) {
      out0[(size_t)ch * w + k] = (float)red[0][x];
    } else if (float* o = k == w ? out1 : out2) {
      o[ch] = (float)red[0][x];
    }
  }
}

// Tokens a thread walks: long enough that the W - 1 re-read rows are a small
// part, short enough that some 16 waves a CU are in flight. `per` = threads a
// segment length of one token would give.
int pick_seg(double per, int T, int least, int most) {
  int seg = most;
  while (seg > least && per / seg < 256.0 * 16 * 64) seg /= 2;
  return seg < T ? seg : (T > 0 ? T : 1);
}

template <typename Tin, int W>
int run_conv(const ConvArgs& a, hipStream_t s) {
  const int C = a.H * a.D, ng = (C + kFwdV - 1) / kFwdV, cx = row_cx(ng);
  const int seg = a.whole ? (a.T > 0 ? a.T : 1)
                          : pick_seg((double)a.B * a.T * ng, a.T, 8, 32);
  const int nseg = a.T > 0 ? (a.T + seg - 1) / seg : 1;
  const long long rows = (long long)a.B * nseg;
  const int per = kRowThreads / cx;
  const long long wgs = (ng + cx - 1) / cx * ((rows + per - 1) / per);
  if (!grid_ok(wgs, kRowThreads)) return -1;
  const dim3 grid((unsigned)wgs);
  // Rows of 16-byte pieces, or element by element where any tensor's rows start
  // elsewhere or heads end inside a thread's 8 channels: B 4, T 4096, 4096 channels of
  // bf16 (fp32) in 59 (119) us aligned, 120 (226) us with rows of 4101, 209 (282) us
  // with heads of 20; the backward of 8 x 2048 x 2048 in 52 (88), 106 (110) and 116 (123) us.
  const size_t m = 16 - 1, es = sizeof(Tin);
  const bool aln = a.D % 8 == 0 && ((size_t)a.x & m) == 0 && ((size_t)a.y & m) == 0 &&
                   ((size_t)a.state0 & m) == 0 && ((size_t)a.stateT & m) == 0 &&
                   (a.xbs * es & m) == 0 && (a.xts * es & m) == 0;
  const int tk = ktimer_before(s, "short_conv");
  if (aln) {
    hipLaunchKernelGGL((conv_kernel<Tin, W, true>), grid, dim3(kRowThreads), 0, s, a, cx, seg,
                       nseg);
  } else {
    hipLaunchKernelGGL((conv_kernel<Tin, W, false>), grid, dim3(kRowThreads), 0, s, a, cx, seg,
                       nseg);
  }
  ktimer_after(s, tk);
  return (int)hipGetLastError();
}

// Rows a thread of the backward walks: 32, or fewer where that would leave CUs
// without two workgroups (a segment recomputes W - 1 tokens of its predecessor).
// B 4, T 4096, bf16: 256 channels 17 us at 32 rows, 13 us at the 8 taken; 512
// channels 21.5 and 18.5 us; 2048 channels (over 1000 workgroups at 32 rows) 50 us.
constexpr int kConvBwdSeg = 32, kConvBwdLeast = 8, kConvBwdGroups = 512;

struct BwdGrid {
  int cx, seg, nseg, per, parts;
};
BwdGrid bwd_grid(int B, int T, int C, int W) {
  BwdGrid g;
  g.cx = row_cx((C + kBwdV - 1) / kBwdV);
  g.per = kRowThreads / g.cx;
  const double rows = (double)B * (T + W - 1) / g.per, cols = (C + kBwdV * g.cx - 1) / (kBwdV * g.cx);
  g.seg = kConvBwdSeg;
  while (g.seg > kConvBwdLeast && rows * cols / g.seg < kConvBwdGroups) g.seg /= 2;
  g.nseg = (T + W - 1 + g.seg - 1) / g.seg;
  g.parts = (int)(((long long)B * g.nseg + g.per - 1) / g.per);
  return g;
}

template <typename Tin, typename Tdy, int W>
int run_conv_bwd(const ConvBackwardArgs& p, hipStream_t s) {
  const ConvArgs& a = p.f;
  const int C = a.H * a.D, ng = (C + kBwdV - 1) / kBwdV;
  const BwdGrid g = bwd_grid(a.B, a.T, C, W);
  const long long wgs = (ng + g.cx - 1) / g.cx * (long long)g.parts;
  if (!grid_ok(wgs, kRowThreads) || !column_sum_ok((W + 1ll) * C)) return -1;
  const dim3 grid((unsigned)wgs);
  const size_t m = 16 - 1, es = sizeof(Tin);
  const bool aln = a.D % 8 == 0 && ((size_t)a.x & m) == 0 && ((size_t)p.dy & m) == 0 &&
                   ((size_t)a.state0 & m) == 0 && ((size_t)p.dstateT & m) == 0 &&
                   ((size_t)p.dx & m) == 0 && ((size_t)p.dstate0 & m) == 0 &&
                   (a.xbs * es & m) == 0 && (a.xts * es & m) == 0;
  const int tk = ktimer_before(s, "short_conv_bwd");
  if (g.parts == 0) {
    // an empty batch: the sums below are zeros
  } else if (aln) {
    hipLaunchKernelGGL((conv_bwd_kernel<Tin, Tdy, W, true>), grid, dim3(kRowThreads), 0, s, p,
                       g.cx, g.seg, g.nseg);
  } else {
    hipLaunchKernelGGL((conv_bwd_kernel<Tin, Tdy, W, false>), grid, dim3(kRowThreads), 0, s, p,
                       g.cx, g.seg, g.nseg);
  }
  ktimer_after(s, tk);
  const int rc = (int)hipGetLastError();
  if (rc) return rc;
  return launch_column_sum((const float*)p.ws, g.parts, (W + 1) * C, C, W, p.dweight, p.dbias,
                           nullptr, s);
}

template <typename Tin>
int run_conv_w(const ConvArgs& a, hipStream_t s) {
  switch (a.W) {
    case 2: return run_conv<Tin, 2>(a, s);
    case 3: return run_conv<Tin, 3>(a, s);
    case 4: return run_conv<Tin, 4>(a, s);
  }
  return -1;
}

template <typename Tin, typename Tdy>
int run_conv_bwd_w(const ConvBackwardArgs& a, hipStream_t s) {
  switch (a.f.W) {
    case 2: return run_conv_bwd<Tin, Tdy, 2>(a, s);
    case 3: return run_conv_bwd<Tin, Tdy, 3>(a, s);
    case 4: return run_conv_bwd<Tin, Tdy, 4>(a, s);
  }
  return -1;
}

}  // namespace

int launch_column_sum(const float* in, int rows, int cols, int c, int w, float* out0,
                      float* out1, float* out2, hipStream_t s) {
  const int tk = ktimer_before(s, "column_sum");
  hipLaunchKernelGGL(column_sum_kernel, dim3((cols + 31) / 32), dim3(1024), 0, s, in, rows, cols,
                     c, w, out0, out1, out2);
  ktimer_after(s, tk);
  return (int)hipGetLastError();
}

int launch_short_conv(const ConvArgs& a, hipStream_t s) {
  return a.bf16 ? run_conv_w<__bf16>(a, s) : run_conv_w<float>(a, s);
}

size_t short_conv_backward_ws(int B, int T, int H, int D, int W) {
  if (B == 0 || H == 0 || D == 0) return 0;
  return (size_t)bwd_grid(B, T, H * D, W).parts * (W + 1) * H * D * sizeof(float);
}

int launch_short_conv_backward(const ConvBackwardArgs& a, hipStream_t s) {
  if (a.f.bf16)
    return a.dy_bf16 ? run_conv_bwd_w<__bf16, __bf16>(a, s) : run_conv_bwd_w<__bf16, float>(a, s);
  return a.dy_bf16 ? -1 : run_conv_bwd_w<float, float>(a, s);
}

}  // namespace osdn
