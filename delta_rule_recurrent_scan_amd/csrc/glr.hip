// Gated linear recurrence, one decay per channel and token:
//   rho = sigmoid(r),  la = A rho,  a = exp(la),  m = sqrt(1 - a^2) (or 1)
//   h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t,     y_t = h_t
// and its adjoint. With g_t = dy_t + a_{t+1} g_{t+1}:
//   dx = g m sigmoid(i),  di = g m x sigmoid'(i)
//   dla = g (a h_{t-1} - (a^2 / m) sigmoid(i) x),  dr = dla la (1 - rho),
//   dA = sum dla rho.
// What g is multiplied by in each of them is formed as soon as a token's gates are there.
//
// A workgroup walks the tokens of one sequence (or a segment of it) for 64
// channels, a tile of 128 or 256 tokens at a time: a thread holds 8 or 16
// tokens of 2 channels, a wave two threads for each pair of channels, a tile eight
// waves. Every thread runs its own tokens from zero, the ends are joined over the waves
// through LDS with one barrier a tile, and a second run over the registers from the
// joined state gives the results: every input is read once and every output
// written once. Where the sequences and channels alone leave CUs idle the
// tokens are cut into segments, whose sums a first launch forms.
//
// The forward is bound by HBM, with the vector units close behind (some 45 instructions an
// element): 4 x 4096 x 4096 bf16 with an input gate and the states 105 us for 554 MB (5.3
// TB/s). The backward in bf16 is bound by both (some 70 instructions an element,
// seven of them of a quarter rate): 204 us for 957 MB (4.7 TB/s), where fp32 with its half
// as many elements a byte reaches 5.9 TB/s: 1 x 9001 x 1536 in segments, the states alone,
// 60 us for 336 MB and the backward from them 85 us for 497 MB. Short calls are their
// launches: 11 us of host and 4 us of kernel for a token of 128 x 4096 channels.
//
// Decays lie close to one and act over thousands of tokens. A product of
// rounded decays would be off by their common rounding times the number of
// tokens, so what carries a state from thread to thread is the exponential of
// a sum of the logarithms; only inside a thread are the decays themselves used.
// 1 - a^2 comes from a series where it is small.
#include <type_traits>

#include "launch.hpp"
#include "layer.hpp"
#include "row_common.hpp"

namespace osdn {
namespace {

constexpr int kThreads = 512, kWaves = 8;
constexpr int kCols = 64;                  // channels a workgroup
// K tokens a thread, 16 K a tile.
template <int K>
constexpr int kTile = 2 * kWaves * K;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// Two channels of one token as they lie in memory. The base is the same in
// all lanes and the byte offset 32 bits. VEC: one access, of any alignment (global memory
// takes them all: rows of 4096 bf16 channels 4097 apart 209 -> 140 us, their backward 370
// -> 238). With an odd number of channels by element: a pair that begins on an odd element
// gained nothing in the forward and lost in the backward.
typedef unsigned __attribute__((aligned(2))) any_u32;
typedef __attribute__((ext_vector_type(2), aligned(4))) float any_f32x2;
template <typename T, bool VEC>
struct Pair;
template <>
struct Pair<__bf16, true> {
  unsigned u;
  __device__ __forceinline__ void load(const char* base, unsigned o0, unsigned o1) {
    u = *(const any_u32*)(base + o0);
  }
  __device__ __forceinline__ float get(int j) const { return j ? high_bf16(u) : low_bf16(u); }
  __device__ __forceinline__ void shut() { u = 0xff80ff80u; }   // -inf
  __device__ __forceinline__ void zero() { u = 0u; }
};
// (joined to one register each element would be waited for where it is loaded)
template <>
struct Pair<__bf16, false> {
  unsigned u[2];
  __device__ __forceinline__ void load(const char* base, unsigned o0, unsigned o1) {
    u[0] = *(const unsigned short*)(base + o0);
    u[1] = *(const unsigned short*)(base + o1);
  }
  __device__ __forceinline__ float get(int j) const { return low_bf16(u[j]); }
  __device__ __forceinline__ void shut() { u[0] = u[1] = 0xff80u; }
  __device__ __forceinline__ void zero() { u[0] = u[1] = 0u; }
};
template <bool VEC>
struct Pair<float, VEC> {
  float v[2];
  __device__ __forceinline__ void load(const char* base, unsigned o0, unsigned o1) {
    if constexpr (VEC) {
      const any_f32x2 t = *(const any_f32x2*)(base + o0);
      v[0] = t[0]; v[1] = t[1];
    } else {
      v[0] = *(const float*)(base + o0);
      v[1] = *(const float*)(base + o1);
    }
  }
  __device__ __forceinline__ float get(int j) const { return v[j]; }
  __device__ __forceinline__ void shut() { v[0] = v[1] = -__builtin_inff(); }
  __device__ __forceinline__ void zero() { v[0] = v[1] = 0.f; }
};

// (past the caches, which the rows read ahead need: 2 % of a prompt's time)
template <bool ALN, typename T>
__device__ __forceinline__ void store_pair(T* p, float v0, float v1, int n) {
  if constexpr (ALN) {
    if (n <= 0) return;
    if constexpr (sizeof(T) == 2) {
      __builtin_nontemporal_store(pack_bf16(v0, v1), (unsigned*)p);
    } else {
      typedef __attribute__((ext_vector_type(2))) float f32x2;
      __builtin_nontemporal_store(f32x2{v0, v1}, (f32x2*)p);
    }
  } else {
    if (n > 0) p[0] = from_f32<T>(v0);
    if (n > 1) p[1] = from_f32<T>(v1);
  }
}

// A thread's place: the seg-th run of tokens of the tile and channels c, c + 1.
struct Place {
  int seg, c, n;        // n: how many of the two channels exist
  int c0, c1;           // the channels it reads (the last ones where there are none)
};
template <bool ALN>
__device__ __forceinline__ Place place(int cb, int C) {
  Place p;
  const int lane = threadIdx.x & 63;
  p.seg = 2 * wave_id() + (lane >> 5);
  p.c = cb * kCols + 2 * (lane & 31);
  p.n = C - p.c;
  p.c0 = min(p.c, ALN ? C - 2 : C - 1);
  p.c1 = min(p.c + 1, C - 1);
  return p;
}

// One input's rows of a tile.
template <typename Tin, bool ALN, int K>
struct Rows {
  Pair<Tin, ALN> v[K];
  // Token k of the thread's in the tile's rows at p with stride ts; tokens from n on read
  // token n - 1 (WHOLE: there are none).
  template <bool WHOLE>
  __device__ __forceinline__ void load(int k, const Tin* p, long long ts, int tile, int n,
                                       const Place& pl) {
    const char* base = (const char*)(p + (long long)tile * ts);
    const unsigned row = (unsigned)ts * (unsigned)sizeof(Tin);
    const unsigned b0 = pl.c0 * (unsigned)sizeof(Tin), b1 = pl.c1 * (unsigned)sizeof(Tin);
    if constexpr (WHOLE) {
      const unsigned o = row * (unsigned)(pl.seg * K);
      v[k].load(base + (size_t)row * k, o + b0, o + b1);
    } else {
      const unsigned o = row * (unsigned)min(pl.seg * K + k, n - 1 - tile);
      v[k].load(base, o + b0, o + b1);
    }
  }
};

// (1 - 4^w) / w for w in (-1/4, 0]: the polynomial of degree 4 through the Chebyshev
// nodes of that range (1.4e-8 off, 1.3e-7 with its roundings).
__device__ __forceinline__ float square_slope(float w) {
  float p = fmaf(-0.03698064014f, w, -0.15267968178f);
  p = fmaf(p, w, -0.44392627478f);
  p = fmaf(p, w, -0.96090275049f);
  return fmaf(p, w, -1.38629436493f);
}

// 1 - 4^w for w <= 0 with e = 2^w: from -1/4 on, where the difference would lose
// digits, from the polynomial.
__device__ __forceinline__ float one_minus_square(float w, float e) {
  const float p = square_slope(w);     // (a branch around it costs more)
  return w > -0.25f ? w * p : fmaf(-e, e, 1.f);
}

// sigmoid(x) and 1 - sigmoid(x) = exp(-x) sigmoid(x): from the rounded sigmoid the
// difference has no digits left at an open gate (off by 5e-4 at 10, 17 % at 15). Where
// exp(-x) is infinite the product is NaN, which the minimum drops.
__device__ __forceinline__ float sigmoid_and_rest(float x, float& rest) {
  const float e = __builtin_amdgcn_exp2f(-kLog2e * x), s = __builtin_amdgcn_rcpf(1.f + e);
  rest = fminf(e * s, 1.f);
  return s;
}

// The smaller of sigmoid(x) and the rest with x's sign: both in one register, as the
// larger is one less it.
__device__ __forceinline__ float lesser(float s, float rest, float x) {
  float v = copysignf(fminf(s, rest), x);
  asm("" : "+v"(v));     // (else its size and its sign are kept apart)
  return v;
}

// Decay and input factor of one token and channel: rho = sigmoid(r), A2 = A log2(e).
template <bool NORM>
__device__ __forceinline__ void factors(float rho, float A2, float& l2, float& a, float& m) {
  l2 = A2 * rho;
  a = __builtin_amdgcn_exp2f(l2);
  m = NORM ? __builtin_amdgcn_sqrtf(one_minus_square(l2, a)) : 1.f;
}

// The value of lane l ^ 32.
__device__ __forceinline__ float other_half(float x) {
  const unsigned u = __float_as_uint(x);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const unsigned lo = s[0], hi = s[1];
  return __uint_as_float((threadIdx.x & 32) ? lo : hi);
}

// Joins the threads' ends over a tile. A run of tokens maps the state c that
// enters it to exp2(L) c + H; in front of a thread's tokens stand the other half
// of its wave and the waves before (FWD: 0 .. 7 in turn, else 7 .. 0). Returns
// the state that enters this thread's tokens in `in` and carries the tile's.
//
// The carried state is updated as c + (H - (1 - exp2(L)) c) where exp2(L) is between 0.7
// and one: the factor's distance from one keeps its digits, so that steps of long
// memory do not add up the factors' roundings. Below (and above one, where A is positive)
// it is exp2(L) c + H: from the distance a small factor would lose its digits, and H what
// c outweighs. What is passed on is exp2(L) - 1, told by its sign bit (zero's too), or
// exp2(L).
template <bool FWD>
__device__ __forceinline__ void join(const float (&L)[2], const float (&H)[2], float (&carry)[2],
                                     float (&in)[2], float4* buf) {
  const int lane = threadIdx.x & 63, w = wave_id();
  const bool first = FWD ? lane < 32 : lane >= 32;
  float p[2], po[2], Ho[2], Q[2], E[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    // (n: minus half the logarithm; as a number it is under 1/4 only if it is positive)
    const float n = -0.5f * (L[j] + other_half(L[j]));
    const bool near = __float_as_uint(n) < __float_as_uint(0.25f);
    p[j] = __builtin_amdgcn_exp2f(L[j]);
    po[j] = other_half(p[j]);
    Ho[j] = other_half(H[j]);
    const float q = n * square_slope(-n);
    Q[j] = near ? q : p[j] * po[j];
    E[j] = fmaf(p[j], Ho[j], H[j]);
  }
  if (!first) buf[w * 32 + (lane & 31)] = float4{Q[0], E[0], Q[1], E[1]};
  __syncthreads();
  float c0 = carry[0], c1 = carry[1], m0 = c0, m1 = c1;
#pragma unroll
  for (int q = 0; q < kWaves; ++q) {
    const int v = FWD ? q : kWaves - 1 - q;
    const float4 t = buf[v * 32 + (lane & 31)];
    if (v == w) {
      m0 = c0;
      m1 = c1;
    }
    c0 = fmaf(t.x, c0, t.y) + (__float_as_int(t.x) < 0 ? c0 : 0.f);
    c1 = fmaf(t.z, c1, t.w) + (__float_as_int(t.z) < 0 ? c1 : 0.f);
  }
  carry[0] = c0;
  carry[1] = c1;
  in[0] = first ? m0 : fmaf(po[0], m0, Ho[0]);
  in[1] = first ? m1 : fmaf(po[1], m1, Ho[1]);
}

// All 64 channels of a block exist.
__device__ __forceinline__ bool whole_columns(int cb, int C) { return (cb + 1) * kCols <= C; }

// Keeps the two forms of a tile's loads apart: joined behind the branch they would take
// their addresses in 64 bits a lane.
template <bool WHOLE>
__device__ __forceinline__ void apart() {
  if constexpr (WHOLE) asm volatile("; whole tile");
}

__device__ __forceinline__ int seq_len(const GlrArgs& a, int b) {
  return a.lengths ? max(0, min(a.lengths[b], a.T)) : a.T;
}

// A segment's map, (L, H) of each channel: [B][S][2][C].
__device__ __forceinline__ float* seg_map(float* ws, int b, int S, int q, int C) {
  return ws + ((size_t)b * S + q) * 2 * C;
}

// The state that enters segment q: h0 (or dh_T) through the segments before
// it (FWD) or behind it.
template <bool FWD>
__device__ __forceinline__ void enter(const float* start, const float* ws, int b, int S, int q,
                                      int C, const Place& pl, float (&c)[2]) {
  c[0] = start ? start[(size_t)b * C + pl.c0] : 0.f;
  c[1] = start ? start[(size_t)b * C + pl.c1] : 0.f;
  for (int j = FWD ? 0 : S - 1; FWD ? j < q : j > q; j += FWD ? 1 : -1) {
    const float* m = ws + ((size_t)b * S + j) * 2 * C;
    c[0] = fmaf(__builtin_amdgcn_exp2f(m[pl.c0]), c[0], m[C + pl.c0]);
    c[1] = fmaf(__builtin_amdgcn_exp2f(m[pl.c1]), c[1], m[C + pl.c1]);
  }
}

// Tokens of segment q of S of a sequence of n, whole tiles.
__device__ __forceinline__ void seg_range(int n, int S, int q, int tile, int& t0, int& t1) {
  const int tiles = (n + tile - 1) / tile, per = (tiles + S - 1) / S;
  t0 = min(n, q * per * tile);
  t1 = min(n, (q + 1) * per * tile);
}

// ---------------------------------------------------------------------------
// Forward. PART: only the segments' maps (the first launch).
// ---------------------------------------------------------------------------

template <typename Tin, int K, bool ALN, bool GATE, bool NORM, bool PART>
__global__ __launch_bounds__(kThreads) void glr_kernel(GlrArgs a, int ncb, int S) {
  constexpr int TILE = kTile<K>;
  __shared__ float4 buf[2][kWaves * 32];
  const int cb = blockIdx.x % ncb, bq = blockIdx.x / ncb;
  const int nq = PART ? S - 1 : S, q = bq % nq, b = bq / nq;
  const Place pl = place<ALN>(cb, a.C);
  const int n = seq_len(a, b);
  int t0, t1;
  seg_range(n, S, q, TILE, t0, t1);
  const Tin* x = (const Tin*)a.x + b * a.xbs;
  const Tin* r = (const Tin*)a.r + b * a.rbs;
  const Tin* gi = GATE ? (const Tin*)a.i + b * a.ibs : nullptr;
  const float A2[2] = {a.A[pl.c0] * kLog2e, a.A[pl.c1] * kLog2e};
  float carry[2] = {0.f, 0.f}, Ltot[2] = {0.f, 0.f};
  if constexpr (!PART) enter<true>(a.h0, (const float*)a.ws, b, S, q, a.C, pl, carry);

  Rows<Tin, ALN, K> rx, rr, ri;
  auto fetch = [&](auto whole, int k, int tile) {
    rr.template load<whole()>(k, r, a.rts, tile, n, pl);
    rx.template load<whole()>(k, x, a.xts, tile, n, pl);
    if constexpr (GATE) ri.template load<whole()>(k, gi, a.its, tile, n, pl);
  };
  if (t0 < t1) {
#pragma unroll
    for (int k = 0; k < K; ++k) fetch(std::false_type(), k, t0);
  }
  int par = 0;
  for (int tile = t0; tile < t1; tile += TILE, par ^= 1) {
    float dec[K][2], in[K][2], L[2] = {0.f, 0.f}, H[2] = {0.f, 0.f};
    const int t = tile + pl.seg * K;
    if (tile + TILE > n) {
      // tokens behind the end: a closed gate keeps the state, and nothing comes in
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (t + k >= n) {
          rr.v[k].shut();
          rx.v[k].zero();
        }
    }
    // A token's registers take the same one of the next tile as soon as it is worked
    // off: its 100 KB a CU take nearly as long as the work.
    const int next = min(tile + TILE, t1 - 1) / TILE * TILE;
    auto tokens = [&](auto whole) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float l2, m;
          factors<NORM>(sigmoid_f(rr.v[k].get(j)), A2[j], l2, dec[k][j], m);
          float u = rx.v[k].get(j);
          if constexpr (GATE) u *= sigmoid_f(ri.v[k].get(j));
          in[k][j] = m * u;
          L[j] += l2;
          H[j] = fmaf(dec[k][j], H[j], in[k][j]);
        }
        fetch(whole, k, next);
        if (k % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      }
      apart<whole()>();
    };
    if (next + TILE <= n) {
      tokens(std::true_type());
    } else {
      tokens(std::false_type());
    }
    float h[2];
    join<true>(L, H, carry, h, buf[par]);
    if constexpr (PART) {
      Ltot[0] += L[0];
      Ltot[1] += L[1];
    } else {
      if (a.states && t % kGlrInterval == 0 && t < a.T) {
        float* st = a.states + ((size_t)b * ((a.T + kGlrInterval - 1) / kGlrInterval) +
                                t / kGlrInterval) * a.C + pl.c;
        store_pair<ALN>(st, h[0], h[1], pl.n);
      }
      if (a.y) {
        // rows of the tile from one base, 32-bit offsets
        char* y = (char*)((Tin*)a.y + ((size_t)b * a.T + tile) * a.C);
        const unsigned row = (unsigned)a.C * (unsigned)sizeof(Tin);
        const unsigned o = row * (unsigned)(pl.seg * K) + pl.c * (unsigned)sizeof(Tin);
        auto tokens = [&](bool whole) {
#pragma unroll
          for (int k = 0; k < K; ++k) {
            h[0] = fmaf(dec[k][0], h[0], in[k][0]);
            h[1] = fmaf(dec[k][1], h[1], in[k][1]);
            if (whole || t + k < n)
              store_pair<ALN>((Tin*)(y + (size_t)row * k + o), h[0], h[1], whole ? 2 : pl.n);
          }
        };
        if (tile + TILE <= n && whole_columns(cb, a.C)) {
          tokens(true);
        } else {
          tokens(false);
        }
      }
    }
  }
  if constexpr (PART) {
    // the threads' logarithms added over the 16 of a channel
    __syncthreads();
    float* red = (float*)buf;
    red[pl.seg * kCols + 2 * (threadIdx.x & 31)] = Ltot[0];
    red[pl.seg * kCols + 2 * (threadIdx.x & 31) + 1] = Ltot[1];
    __syncthreads();
    if (threadIdx.x < 32 && pl.n > 0) {
      float* m = seg_map((float*)a.ws, b, S, q, a.C);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (j >= pl.n) continue;
        float s = 0.f;
        for (int w = 0; w < 2 * kWaves; ++w) s += red[w * kCols + 2 * threadIdx.x + j];
        m[pl.c + j] = s;
        m[a.C + pl.c + j] = carry[j];
      }
    }
  } else {
    // the last segment leaves the state, the rows behind the sequence and
    // their states
    if (q == S - 1) {
      if (a.hT && threadIdx.x < 32)
        store_pair<ALN>(a.hT + (size_t)b * a.C + pl.c, carry[0], carry[1], pl.n);
      const int ns = (a.T + kGlrInterval - 1) / kGlrInterval;
      const int s0 = (n + TILE - 1) / TILE * (TILE / kGlrInterval);
      if (a.states)
        for (int t = s0 + pl.seg; t < ns; t += 2 * kWaves)
          store_pair<ALN>(a.states + ((size_t)b * ns + t) * a.C + pl.c, carry[0], carry[1], pl.n);
      if (a.y)
        for (int t = n + pl.seg; t < a.T; t += 2 * kWaves)
          store_pair<ALN>((Tin*)a.y + ((size_t)b * a.T + t) * a.C + pl.c, 0.f, 0.f, pl.n);
    }
  }
}

// ---------------------------------------------------------------------------
// Single tokens: two channels a thread, tokens in turn.
// ---------------------------------------------------------------------------

template <typename Tin, bool ALN, bool GATE, bool NORM>
__global__ __launch_bounds__(256) void glr_decode_kernel(GlrArgs a) {
  const int np = (a.C + 1) / 2;
  const long long at = blockIdx.x * 256LL + threadIdx.x;
  if (at >= (long long)a.B * np) return;
  const int b = (int)(at / np), c = (int)(at % np) * 2, n = a.C - c;
  const int c1 = min(c + 1, a.C - 1);
  const float A2[2] = {a.A[c] * kLog2e, a.A[c1] * kLog2e};
  float h[2] = {a.h0[(size_t)b * a.C + c], a.h0[(size_t)b * a.C + c1]};
  for (int t = 0; t < a.T; ++t) {
    Pair<Tin, ALN> x, r, g;
    const unsigned o = (unsigned)(c1 - c) * (unsigned)sizeof(Tin);
    x.load((const char*)((const Tin*)a.x + b * a.xbs + t * a.xts + c), 0, o);
    r.load((const char*)((const Tin*)a.r + b * a.rbs + t * a.rts + c), 0, o);
    if constexpr (GATE)
      g.load((const char*)((const Tin*)a.i + b * a.ibs + t * a.its + c), 0, o);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float l2, d, m, u = x.get(j);
      factors<NORM>(sigmoid_f(r.get(j)), A2[j], l2, d, m);
      if constexpr (GATE) u *= sigmoid_f(g.get(j));
      h[j] = fmaf(d, h[j], m * u);
    }
    store_pair<ALN>((Tin*)a.y + ((size_t)b * a.T + t) * a.C + c, h[0], h[1], n);
  }
  store_pair<ALN>(a.hT + (size_t)b * a.C + c, h[0], h[1], n);
}

// ---------------------------------------------------------------------------
// Backward: tiles from the last to the first. What passes from token t to t - 1
// is c_t = a_t g_t = a_t (dy_t + c_{t+1}).
// ---------------------------------------------------------------------------

constexpr int kBK = 8;   // tokens a thread

template <typename Tin, bool ALN>
__global__ __launch_bounds__(kThreads) void glr_bwd_part_kernel(GlrArgs a, int ncb, int S) {
  constexpr int K = kBK, TILE = kTile<K>;
  __shared__ float4 buf[2][kWaves * 32];
  const int cb = blockIdx.x % ncb, bq = blockIdx.x / ncb;
  const int q = 1 + bq % (S - 1), b = bq / (S - 1);
  const Place pl = place<ALN>(cb, a.C);
  const int n = seq_len(a, b);
  int t0, t1;
  seg_range(n, S, q, TILE, t0, t1);
  const Tin* r = (const Tin*)a.r + b * a.rbs;
  const Tin* dy = (const Tin*)a.dy + (size_t)b * a.T * a.C;
  const float A2[2] = {a.A[pl.c0] * kLog2e, a.A[pl.c1] * kLog2e};
  float carry[2] = {0.f, 0.f}, Ltot[2] = {0.f, 0.f};
  Rows<Tin, ALN, K> rr, rd;
  auto fetch = [&](auto whole, int k, int tile) {
    rr.template load<whole()>(k, r, a.rts, tile, n, pl);
    rd.template load<whole()>(k, dy, a.C, tile, n, pl);
  };
  const int last = t0 < t1 ? (t1 - 1) / TILE * TILE : -1;
  if (t0 < t1) {
#pragma unroll
    for (int k = 0; k < K; ++k) fetch(std::false_type(), k, last);
  }
  int par = 0;
  for (int tile = last; tile >= t0; tile -= TILE, par ^= 1) {
    float L[2] = {0.f, 0.f}, H[2] = {0.f, 0.f};
    const int t = tile + pl.seg * K;
    if (tile + TILE > n) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (t + k >= n) {
          rr.v[k].shut();
          rd.v[k].zero();
        }
    }
    const int next = max(tile - TILE, t0);
    auto tokens = [&](auto whole) {
#pragma unroll
      for (int k = K - 1; k >= 0; --k) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float l2 = A2[j] * sigmoid_f(rr.v[k].get(j));
          L[j] += l2;
          H[j] = __builtin_amdgcn_exp2f(l2) * (H[j] + rd.v[k].get(j));
        }
        fetch(whole, k, next);
      }
      apart<whole()>();
    };
    if (next + TILE <= n) {
      tokens(std::true_type());
    } else {
      tokens(std::false_type());
    }
    float in[2];
    join<false>(L, H, carry, in, buf[par]);
    Ltot[0] += L[0];
    Ltot[1] += L[1];
  }
  __syncthreads();
  float* red = (float*)buf;
  red[pl.seg * kCols + 2 * (threadIdx.x & 31)] = Ltot[0];
  red[pl.seg * kCols + 2 * (threadIdx.x & 31) + 1] = Ltot[1];
  __syncthreads();
  if (threadIdx.x < 32 && pl.n > 0) {
    float* m = seg_map((float*)a.ws, b, S, q, a.C);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (j >= pl.n) continue;
      float s = 0.f;
      for (int w = 0; w < 2 * kWaves; ++w) s += red[w * kCols + 2 * threadIdx.x + j];
      m[pl.c + j] = s;
      m[a.C + pl.c + j] = carry[j];
    }
  }
}

// parts: [B * S][C], the segments' parts of dA.
template <typename Tin, bool ALN, bool GATE, bool NORM>
__global__ __launch_bounds__(kThreads) void glr_bwd_kernel(GlrArgs a, int ncb, int S,
                                                           float* parts) {
  constexpr int K = kBK, TILE = kTile<K>;
  // fp32 rows and pairs by element take twice the registers of paired bf16 ones: rho and
  // its slope are then kept in one (4 x 4096 x 4095 fp32 564 -> 551 us, as separate ones
  // with what spills 572).
  constexpr bool TIGHT = !ALN || sizeof(Tin) == 4;
  __shared__ float4 buf[2][kWaves * 32];
  __shared__ double red[2 * kWaves][kCols];
  const int cb = blockIdx.x % ncb, bq = blockIdx.x / ncb, q = bq % S, b = bq / S;
  const Place pl = place<ALN>(cb, a.C);
  const int n = seq_len(a, b), ns = (a.T + kGlrInterval - 1) / kGlrInterval;
  int t0, t1;
  seg_range(n, S, q, TILE, t0, t1);
  const Tin* x = (const Tin*)a.x + b * a.xbs;
  const Tin* r = (const Tin*)a.r + b * a.rbs;
  const Tin* gi = GATE ? (const Tin*)a.i + b * a.ibs : nullptr;
  const Tin* dy = (const Tin*)a.dy + (size_t)b * a.T * a.C;
  const float A2[2] = {a.A[pl.c0] * kLog2e, a.A[pl.c1] * kLog2e};
  float carry[2];
  enter<false>(a.dhT, (const float*)a.ws, b, S, q, a.C, pl, carry);
  double dA[2] = {0.0, 0.0};
  const bool low = (threadIdx.x & 63) < 32;

  Rows<Tin, ALN, K> rx, rr, ri, rd;
  float s0 = 0.f, s1 = 0.f;
  auto fetch = [&](auto whole, int k, int tile) {
    rr.template load<whole()>(k, r, a.rts, tile, n, pl);
    rx.template load<whole()>(k, x, a.xts, tile, n, pl);
    if constexpr (GATE) ri.template load<whole()>(k, gi, a.its, tile, n, pl);
  };
  auto fetch_dy = [&](auto whole, int k, int tile) {
    rd.template load<whole()>(k, dy, a.C, tile, n, pl);
  };
  auto fetch_state = [&](int tile) {
    const int si = min((tile + pl.seg * K) / kGlrInterval, ns - 1);
    const float* st = a.states + ((size_t)b * ns + si) * a.C;
    s0 = st[pl.c0];
    s1 = st[pl.c1];
  };
  const int last = t0 < t1 ? (t1 - 1) / TILE * TILE : -1;
  if (t0 < t1) {
    fetch_state(last);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      fetch(std::false_type(), k, last);
      fetch_dy(std::false_type(), k, last);
    }
  }
  int par = 0;
  for (int tile = last; tile >= t0; tile -= TILE, par ^= 1) {
    const int t = tile + pl.seg * K;
    if (tile + TILE > n) {
      // (as in the forward, and no adjoint)
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (t + k >= n) {
          rr.v[k].shut();
          rx.v[k].zero();
          rd.v[k].zero();
        }
    }
    // What the results take from a token, with g the adjoint of its state: the factors
    // of dx (sx), di (si), dr (slope) and dA (rho), and bw: the state before it less what
    // reaches log a through m, by which dla = a g bw.
    float rho[K][2], slope[K][2], dec[K][2], in[K][2], sx[K][2], si[K][2], bw[K][2], kept[K][2];
    float L[2] = {0.f, 0.f}, H[2] = {0.f, 0.f}, st[2] = {s0, s1};
    const int next = max(tile - TILE, t0);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float l2, m, rest, u = rx.v[k].get(j);
        rho[k][j] = sigmoid_and_rest(rr.v[k].get(j), rest);
        slope[k][j] = rho[k][j] * rest;
        if constexpr (TIGHT) kept[k][j] = lesser(rho[k][j], rest, rr.v[k].get(j));
        L[j] += rho[k][j];
        factors<NORM>(rho[k][j], A2[j], l2, dec[k][j], m);
        sx[k][j] = m;
        if constexpr (GATE) {
          const float sg = sigmoid_and_rest(ri.v[k].get(j), rest);
          u *= sg;
          sx[k][j] *= sg;
          si[k][j] = m * u * rest;
        }
        in[k][j] = m * u;
        // (where a is one no gradient passes through m)
        bw[k][j] = NORM && m > 0.f ? dec[k][j] * u * __builtin_amdgcn_rcpf(m) : 0.f;
      }
    // (token by token as in the forward the registers run out)
    fetch_state(next);
    if (next + TILE <= n) {
#pragma unroll
      for (int k = 0; k < K; ++k) fetch(std::true_type(), k, next);
      apart<true>();
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) fetch(std::false_type(), k, next);
    }
    float F[2] = {low ? st[0] : 0.f, low ? st[1] : 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) F[j] = fmaf(dec[k][j], F[j], in[k][j]);
    L[0] *= A2[0];
    L[1] *= A2[1];
#pragma unroll
    for (int k = K - 1; k >= 0; --k)
#pragma unroll
      for (int j = 0; j < 2; ++j) H[j] = dec[k][j] * (H[j] + rd.v[k].get(j));
    // the state before the second half's tokens is the first half's end
    const float f0 = other_half(F[0]), f1 = other_half(F[1]);
    float h[2] = {low ? st[0] : f0, low ? st[1] : f1};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        bw[k][j] = h[j] - bw[k][j];
        h[j] = fmaf(dec[k][j], h[j], in[k][j]);
      }
    float c[2], sA[2] = {0.f, 0.f};
    join<false>(L, H, carry, c, buf[par]);
    const size_t base = ((size_t)b * a.T + tile) * a.C;
    const unsigned row = (unsigned)a.C * (unsigned)sizeof(Tin);
    const unsigned o = row * (unsigned)(pl.seg * K) + pl.c * (unsigned)sizeof(Tin);
    char *px = (char*)((Tin*)a.dx + base), *pr = (char*)((Tin*)a.dr + base),
         *pi = GATE ? (char*)((Tin*)a.di + base) : nullptr;
    auto tokens = [&](bool whole) {
#pragma unroll
      for (int k = K - 1; k >= 0; --k) {
        float ox[2], orr[2], oi[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float g = rd.v[k].get(j) + c[j];
          c[j] = dec[k][j] * g;
          ox[j] = g * sx[k][j];
          if constexpr (GATE) oi[j] = g * si[k][j];
          const float dla = c[j] * bw[k][j];
          float p = rho[k][j], s = slope[k][j];
          if constexpr (TIGHT) {
            const float lo = fabsf(kept[k][j]), hi = 1.f - lo;
            p = __float_as_int(kept[k][j]) >= 0 ? hi : lo;
            s = lo * hi;
          }
          orr[j] = dla * (kLn2 * A2[j]) * s;
          sA[j] = fmaf(dla, p, sA[j]);
        }
        if (whole || t + k < n) {
          const int nc = whole ? 2 : pl.n;
          store_pair<ALN>((Tin*)(px + (size_t)row * k + o), ox[0], ox[1], nc);
          store_pair<ALN>((Tin*)(pr + (size_t)row * k + o), orr[0], orr[1], nc);
          if constexpr (GATE) store_pair<ALN>((Tin*)(pi + (size_t)row * k + o), oi[0], oi[1], nc);
        }
      }
    };
    if (tile + TILE <= n && whole_columns(cb, a.C)) {
      tokens(true);
    } else {
      tokens(false);
    }
    // (behind the results: with the other rows dy's would take registers of their own
    // while the tokens' factors are formed, 4 x 4096 x 4096 bf16 225 us for 238)
    if (next + TILE <= n) {
#pragma unroll
      for (int k = 0; k < K; ++k) fetch_dy(std::true_type(), k, next);
      apart<true>();
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) fetch_dy(std::false_type(), k, next);
    }
    dA[0] += (double)sA[0];
    dA[1] += (double)sA[1];
  }
  const int lc = 2 * (threadIdx.x & 31);
  red[pl.seg][lc] = dA[0];
  red[pl.seg][lc + 1] = dA[1];
  __syncthreads();
  if (threadIdx.x < kCols && cb * kCols + (int)threadIdx.x < a.C) {
    double s = 0.0;
    for (int w = 0; w < 2 * kWaves; ++w) s += red[w][threadIdx.x];
    parts[((size_t)b * S + q) * a.C + cb * kCols + threadIdx.x] = (float)s;
  }
  if (q == 0 && a.dh0 && threadIdx.x < 32)
    store_pair<ALN>(a.dh0 + (size_t)b * a.C + pl.c, carry[0], carry[1], pl.n);
  if (q == S - 1)
    for (int t = n + pl.seg; t < a.T; t += 2 * kWaves) {
      const size_t at = ((size_t)b * a.T + t) * a.C + pl.c;
      store_pair<ALN>((Tin*)a.dx + at, 0.f, 0.f, pl.n);
      store_pair<ALN>((Tin*)a.dr + at, 0.f, 0.f, pl.n);
      if constexpr (GATE) store_pair<ALN>((Tin*)a.di + at, 0.f, 0.f, pl.n);
    }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

int col_blocks(int C) { return (C + kCols - 1) / kCols; }

// Tokens a thread of the forward: 16 halve the joins, and in bf16 their registers leave
// room for the tile ahead. Short sequences would leave waves of a tile empty.
bool long_runs(int T, int bf16) { return bf16 && T >= 512; }

// Segments of a sequence: one while the sequences and channels alone give more than half
// the CUs a workgroup (2 x 8192 x 5120, 160 of them: 187 us, backward 348, and 275 and 402
// in two segments, whose maps cost most of the inputs again); otherwise as many as give
// each CU one (1 x 8192 x 2048: 64 us with two a CU, 55 with one), of 128 tokens at least.
// They are dealt whole tiles, so that the last ones may get none: of the 5 of 1000 tokens
// of 128 a tile 4 work, of the 16 of 2048 tokens of 256 a tile 8.
int segments(int B, int T, int C) {
  const long long wgs = (long long)B * col_blocks(C);
  if (wgs == 0) return 1;
  long long S = 256 / wgs;
  if (S > T / 128) S = T / 128;
  return S < 2 ? 1 : (int)S;
}

size_t map_bytes(int B, int T, int C) {
  const int S = segments(B, T, C);
  return S > 1 ? ((size_t)B * S * 2 * C * sizeof(float) + 255) / 256 * 256 : 0;
}

bool even(const void* p, size_t es) { return ((size_t)p & (2 * es - 1)) == 0; }

template <typename Tin, int K, bool ALN, bool GATE, bool NORM>
int run_walk(const GlrArgs& a, hipStream_t s) {
  const int ncb = col_blocks(a.C), S = segments(a.B, a.T, a.C);
  if (!grid_ok((long long)ncb * a.B * S, kThreads)) return -1;
  if (S > 1) {
    const int tk = ktimer_before(s, "glr_part");
    hipLaunchKernelGGL((glr_kernel<Tin, K, ALN, GATE, NORM, true>),
                       dim3((unsigned)ncb * a.B * (S - 1)), dim3(kThreads), 0, s, a, ncb, S);
    ktimer_after(s, tk);
    const int rc = (int)hipGetLastError();
    if (rc) return rc;
  }
  const int tk = ktimer_before(s, "glr");
  hipLaunchKernelGGL((glr_kernel<Tin, K, ALN, GATE, NORM, false>), dim3((unsigned)ncb * a.B * S),
                     dim3(kThreads), 0, s, a, ncb, S);
  ktimer_after(s, tk);
  return (int)hipGetLastError();
}

template <typename Tin, bool ALN, bool GATE, bool NORM>
int run_forward(const GlrArgs& a, hipStream_t s) {
  if constexpr (sizeof(Tin) == 2 && ALN)
    if (long_runs(a.T, a.bf16)) return run_walk<Tin, 16, ALN, GATE, NORM>(a, s);
  return run_walk<Tin, 8, ALN, GATE, NORM>(a, s);
}

template <typename Tin, bool ALN, bool GATE, bool NORM>
int run_decode(const GlrArgs& a, hipStream_t s) {
  const long long wgs = ((long long)a.B * ((a.C + 1) / 2) + 255) / 256;
  if (!grid_ok(wgs, 256)) return -1;
  const int tk = ktimer_before(s, "glr_decode");
  hipLaunchKernelGGL((glr_decode_kernel<Tin, ALN, GATE, NORM>), dim3((unsigned)wgs), dim3(256), 0,
                     s, a);
  ktimer_after(s, tk);
  return (int)hipGetLastError();
}

template <typename Tin, bool ALN, bool GATE, bool NORM>
int run_backward(const GlrArgs& a0, hipStream_t s) {
  GlrArgs a = a0;
  const int ncb = col_blocks(a.C), S = segments(a.B, a.T, a.C);
  if (!grid_ok((long long)ncb * a.B * S, kThreads) || !column_sum_ok(a.C)) return -1;
  const size_t maps = map_bytes(a.B, a.T, a.C);
  float* parts = (float*)((char*)a.ws + maps);
  if (!a.states && a.T > 0 && a.B > 0) {
    // the states that a forward would have left, behind the partial sums
    a.states = parts + ((size_t)a.B * S * a.C + 63) / 64 * 64;
    GlrArgs f = a;
    f.y = nullptr;
    f.hT = nullptr;
    const int rc = run_forward<Tin, ALN, GATE, NORM>(f, s);
    if (rc) return rc;
  }
  if (S > 1) {
    const int tk = ktimer_before(s, "glr_bwd_part");
    hipLaunchKernelGGL((glr_bwd_part_kernel<Tin, ALN>), dim3((unsigned)ncb * a.B * (S - 1)),
                       dim3(kThreads), 0, s, a, ncb, S);
    ktimer_after(s, tk);
    const int rc = (int)hipGetLastError();
    if (rc) return rc;
  }
  if (a.B > 0) {
    const int tk = ktimer_before(s, "glr_bwd");
    hipLaunchKernelGGL((glr_bwd_kernel<Tin, ALN, GATE, NORM>), dim3((unsigned)ncb * a.B * S),
                       dim3(kThreads), 0, s, a, ncb, S, parts);
    ktimer_after(s, tk);
    const int rc = (int)hipGetLastError();
    if (rc) return rc;
  }
  return launch_column_sum(parts, a.B * S, a.C, a.C, 1, a.dA, nullptr, nullptr, s);
}

// What one launch is instantiated on.
enum Call { kForward, kDecode, kBackward };

template <Call CALL, typename Tin, bool ALN, bool GATE>
int run_norm(const GlrArgs& a, hipStream_t s) {
  if constexpr (CALL == kForward)
    return a.normalize ? run_forward<Tin, ALN, GATE, true>(a, s)
                       : run_forward<Tin, ALN, GATE, false>(a, s);
  if constexpr (CALL == kDecode)
    return a.normalize ? run_decode<Tin, ALN, GATE, true>(a, s)
                       : run_decode<Tin, ALN, GATE, false>(a, s);
  return a.normalize ? run_backward<Tin, ALN, GATE, true>(a, s)
                     : run_backward<Tin, ALN, GATE, false>(a, s);
}

template <Call CALL, typename Tin>
int run_t(const GlrArgs& a, hipStream_t s) {
  const size_t es = sizeof(Tin);
  // every pair of channels exists and is stored where a pair may start (inputs are read at
  // any alignment)
  const bool aln = a.C % 2 == 0 && even(a.y, es) && even(a.dx, es) && even(a.dr, es) &&
                   even(a.di, es) && even(a.hT, 4) && even(a.states, 4) && even(a.dh0, 4);
  if (aln) return a.i ? run_norm<CALL, Tin, true, true>(a, s) : run_norm<CALL, Tin, true, false>(a, s);
  return a.i ? run_norm<CALL, Tin, false, true>(a, s) : run_norm<CALL, Tin, false, false>(a, s);
}

}  // namespace

size_t glr_forward_ws(int B, int T, int C) { return map_bytes(B, T, C); }

int launch_glr_forward(const GlrArgs& a, hipStream_t s) {
  return a.bf16 ? run_t<kForward, __bf16>(a, s) : run_t<kForward, float>(a, s);
}

int launch_glr_decode(const GlrArgs& a, hipStream_t s) {
  return a.bf16 ? run_t<kDecode, __bf16>(a, s) : run_t<kDecode, float>(a, s);
}

size_t glr_backward_ws(int B, int T, int C, int have_states) {
  const size_t parts = ((size_t)B * segments(B, T, C) * C + 63) / 64 * 64 * sizeof(float);
  const size_t st = have_states ? 0
                                : (size_t)B * ((T + kGlrInterval - 1) / kGlrInterval) * C * sizeof(float);
  return map_bytes(B, T, C) + parts + st;
}

int launch_glr_backward(const GlrArgs& a, hipStream_t s) {
  return a.bf16 ? run_t<kBackward, __bf16>(a, s) : run_t<kBackward, float>(a, s);
}

}  // namespace osdn
