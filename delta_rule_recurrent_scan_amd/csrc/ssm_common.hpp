// Device helpers shared by the selective-scan kernels.
#pragma once

#include "device_common.hpp"

namespace osdn {

// The step size of a token: softplus(raw + bias) (or raw + bias itself).
// softplus(v) = max(v, 0) + log1p(e^-|v|), exact at both ends.
__device__ __forceinline__ float ssm_step(float raw, float bias, int softplus) {
  const float v = raw + bias;
  return softplus ? fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))) : v;
}
// d softplus / dv = 1 / (1 + e^-v).
__device__ __forceinline__ float ssm_step_slope(float raw, float bias, int softplus) {
  return softplus ? 1.f / (1.f + expf(-(raw + bias))) : 1.f;
}

// Tokens of batch entry b (lengths null: all T), clamped to [0, T].
__device__ __forceinline__ int ssm_length(const int* lengths, int b, int T) {
  if (!lengths) return T;
  const int n = lengths[b];
  return n < 0 ? 0 : n > T ? T : n;
}

// Inclusive prefix and suffix sums over each row of 16 lanes, and the suffix
// without the lane itself.
__device__ __forceinline__ float row16_prefix(float x) {
  x += dpp_f<0x111>(x);  // row_shr:1, :2, :4, :8 (zeros from outside the row)
  x += dpp_f<0x112>(x);
  x += dpp_f<0x114>(x);
  x += dpp_f<0x118>(x);
  return x;
}
__device__ __forceinline__ float row16_suffix(float x) {
  x += dpp_f<0x101>(x);  // row_shl:1, :2, :4, :8
  x += dpp_f<0x102>(x);
  x += dpp_f<0x104>(x);
  x += dpp_f<0x108>(x);
  return x;
}
__device__ __forceinline__ float row16_suffix_after(float x) {
  return dpp_f<0x101>(row16_suffix(x));
}

// The decays of one chunk of Q tokens. With l = dt A a token, the factor from
// token j to a later token i, exp(l_{j+1} + .. + l_i), is formed from sums
// that all run forward from one point: `up` inside i's block of 16, `dn`
// behind j inside its block, and whole blocks between. No difference of two
// long sums is taken, so a strong decay early in the chunk costs later pairs
// no precision; inside one block the difference is of sums over 16 tokens.
template <int Q>
struct ChunkDecay {
  float dt[Q];    // step
  float up[Q];    // log: block start .. token, inclusive
  float eup[Q];   // exp(up)
  float edn[Q];   // exp(log: after token .. block end)
  float ent[Q];   // chunk entry .. token
  float ext[Q];   // after token .. chunk exit
  float gap[16];  // [a][b], a > b: exp over the blocks strictly between
  float total;    // whole chunk
  float logtot;

  // By one whole wave; lane t (< Q) passes its token's step and log decay.
  __device__ __forceinline__ void fill(float step, float l) {
    constexpr int NB = Q / 16;
    const int t = threadIdx.x & 63;
    const float u = row16_prefix(l), d = row16_suffix_after(l);
    float bs[NB], pre[NB + 1];
    pre[0] = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      bs[b] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(u), 16 * b + 15));
      pre[b + 1] = pre[b] + bs[b];
    }
    float before = 0.f, after = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b < t / 16) before += bs[b];
      if (b > t / 16) after += bs[b];
    }
    if (t < Q) {
      dt[t] = step;
      up[t] = u;
      eup[t] = __expf(u);
      edn[t] = __expf(d);
      ent[t] = __expf(before + u);
      ext[t] = __expf(d + after);
    }
    if (t < NB * NB) {
      const int x = t / NB, y = t % NB;
      float g = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        if (b > y && b < x) g += bs[b];
      gap[x * 4 + y] = __expf(g);
    }
    if (t == 0) {
      total = __expf(pre[NB]);
      logtot = pre[NB];
    }
  }
};

// Decays of one tile of pairs in accumulator layout: lane l holds the factors
// from the tokens j = 16 jt + 4 (l / 16) + r to i = 16 it + l % 16, zero where
// j > i.
template <int Q>
__device__ __forceinline__ f32x4 pair_decay(const ChunkDecay<Q>& d, int it, int jt) {
  f32x4 f = {0.f, 0.f, 0.f, 0.f};
  const int i = it * 16 + acc_col(), j = jt * 16 + acc_row(0);
  if (jt < it) {
    const float g = d.eup[i] * d.gap[it * 4 + jt];
    const f32x4 e = *reinterpret_cast<const f32x4*>(d.edn + j);
#pragma unroll
    for (int r = 0; r < 4; ++r) f[r] = g * e[r];
  } else if (jt == it) {
    const f32x4 u = *reinterpret_cast<const f32x4*>(d.up + j);
    const float v = d.up[i];
#pragma unroll
    for (int r = 0; r < 4; ++r) f[r] = j + r <= i ? __expf(v - u[r]) : 0.f;
  }
  return f;
}

// The steps of the tile's tokens j.
template <int Q>
__device__ __forceinline__ f32x4 tile_steps(const ChunkDecay<Q>& d, int jt) {
  return *reinterpret_cast<const f32x4*>(d.dt + jt * 16 + acc_row(0));
}

// Inclusive sum of lanes l .. 63, and exclusive sum of lanes 0 .. l - 1.
__device__ __forceinline__ float wave_suffix_sum(float x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const float y = __shfl_down(x, d, 64);
    if (lane + d < 64) x += y;
  }
  return x;
}
__device__ __forceinline__ float wave_prefix_before(float x) {
  const float y = __shfl_up(wave_prefix_sum(x), 1, 64);
  return (threadIdx.x & 63) ? y : 0.f;
}

// acc += A * B^T over the first kmax (a multiple of 16) of the K indices.
template <int KEXT>
__device__ __forceinline__ void mma_upto(f32x4& acc, const Frag<KEXT, __bf16>& a,
                                         const Frag<KEXT, __bf16>& b, int kmax) {
#pragma unroll
  for (int i = 0; i < KEXT / 32; ++i)
    if (32 * i < kmax) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], acc, 0, 0, 0);
}
template <int KEXT>
__device__ __forceinline__ void mma_upto(f32x4& acc, const Frag<KEXT, float>& a,
                                         const Frag<KEXT, float>& b, int kmax) {
#pragma unroll
  for (int i = 0; i < KEXT / 4; ++i)
    if (4 * i < kmax) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], acc, 0, 0, 0);
}

// A fragment (row = lane % 16) in permuted k order from the accumulator tiles
// of that k range.
template <int KEXT>
__device__ __forceinline__ void frag_from_acc(Frag<KEXT, __bf16>& f, const f32x4 (&t)[KEXT / 16]) {
#pragma unroll
  for (int i = 0; i < KEXT / 32; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f.v[i][e] = (__bf16)t[2 * i][e];
      f.v[i][4 + e] = (__bf16)t[2 * i + 1][e];
    }
}
template <int KEXT>
__device__ __forceinline__ void frag_from_acc(Frag<KEXT, float>& f, const f32x4 (&t)[KEXT / 16]) {
#pragma unroll
  for (int b = 0; b < KEXT / 16; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[4 * b + e] = t[b][e];
}

// An fp32 operand as bf16 fragments that add up to it: the rounded value, what
// its rounding lost, and what that one's lost (24 bits in all, an error of
// some 6e-8). Used where a product's sum leaves in fp32 (states, step and
// parameter gradients); one rounding would leave 2e-3 there. fp32 operands
// are one fragment.
template <int KEXT, typename Tin>
struct Parts {
  static constexpr int M = sizeof(Tin) == 2 ? 3 : 1;
  Frag<KEXT, Tin> f[M];
};

__device__ __forceinline__ void split3(float p, __bf16& a, __bf16& b, __bf16& c) {
  a = (__bf16)p;
  p -= (float)a;
  b = (__bf16)p;
  c = (__bf16)(p - (float)b);
}

// x scaled by w[k] (natural k order, w in LDS).
template <int KEXT>
__device__ __forceinline__ void scale_parts(const Frag<KEXT, __bf16>& x, const float* w,
                                            Parts<KEXT, __bf16>& o) {
  const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int i = 0; i < KEXT / 32; ++i) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(w + 32 * i + 8 * g);
    const f32x4 b = *reinterpret_cast<const f32x4*>(w + 32 * i + 8 * g + 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      __bf16 p0, p1, p2;
      split3((float)x.v[i][e] * (e < 4 ? a[e & 3] : b[e & 3]), p0, p1, p2);
      o.f[0].v[i][e] = p0;
      o.f[1].v[i][e] = p1;
      o.f[2].v[i][e] = p2;
    }
  }
}
template <int KEXT>
__device__ __forceinline__ void scale_parts(const Frag<KEXT, float>& x, const float* w,
                                            Parts<KEXT, float>& o) {
  const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int i = 0; i < KEXT / 4; ++i) o.f[0].v[i] = x.v[i] * w[4 * i + g];
}

// Accumulator tiles of a k range as a split operand (permuted k order).
template <int KEXT>
__device__ __forceinline__ void parts_from_acc(Parts<KEXT, __bf16>& o,
                                               const f32x4 (&t)[KEXT / 16]) {
#pragma unroll
  for (int i = 0; i < KEXT / 32; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      __bf16 p0, p1, p2;
      split3(t[2 * i + e / 4][e & 3], p0, p1, p2);
      o.f[0].v[i][e] = p0;
      o.f[1].v[i][e] = p1;
      o.f[2].v[i][e] = p2;
    }
}
template <int KEXT>
__device__ __forceinline__ void parts_from_acc(Parts<KEXT, float>& o,
                                               const f32x4 (&t)[KEXT / 16]) {
  frag_from_acc<KEXT>(o.f[0], t);
}

// acc += A B^T with one operand in parts, smallest part first.
template <int KEXT, typename Tin>
__device__ __forceinline__ void mma_parts(f32x4& acc, const Parts<KEXT, Tin>& a,
                                          const Frag<KEXT, Tin>& b) {
#pragma unroll
  for (int m = Parts<KEXT, Tin>::M - 1; m >= 0; --m) mma(acc, a.f[m], b);
}
template <int KEXT, typename Tin>
__device__ __forceinline__ void mma_parts(f32x4& acc, const Frag<KEXT, Tin>& a,
                                          const Parts<KEXT, Tin>& b) {
#pragma unroll
  for (int m = Parts<KEXT, Tin>::M - 1; m >= 0; --m) mma(acc, a, b.f[m]);
}

// Four consecutive values of a row in LDS or global memory, widened / rounded.
__device__ __forceinline__ f32x4 load4(const __bf16* p) {
  const bf16x4 b = *reinterpret_cast<const bf16x4*>(p);
  return f32x4{(float)b[0], (float)b[1], (float)b[2], (float)b[3]};
}
__device__ __forceinline__ f32x4 load4(const float* p) {
  return *reinterpret_cast<const f32x4*>(p);
}
__device__ __forceinline__ void store4(__bf16* p, const f32x4& a) {
  bf16x4 b;
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = (__bf16)a[e];
  *reinterpret_cast<bf16x4*>(p) = b;
}
__device__ __forceinline__ void store4(float* p, const f32x4& a) {
  *reinterpret_cast<f32x4*>(p) = a;
}

// Staging of a Q x D tile of token rows through registers into LDS by NT
// threads: fetch() issues the loads (rows from `valid` on are zeros), put()
// writes them with row stride ld.
template <int Q, int D, typename Tin, int NT>
struct Stage {
  static constexpr int VE = 16 / sizeof(Tin), PER = D / VE, NV = Q * PER / NT;
  static_assert(Q * PER % NT == 0, "tile divides over the threads");
  uint4 v[NV];
  __device__ __forceinline__ void fetch(const Tin* src, int valid) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = i * NT + threadIdx.x, row = e / PER, col = e % PER * VE;
      v[i] = row < valid ? *reinterpret_cast<const uint4*>(src + (size_t)row * D + col)
                         : uint4{0u, 0u, 0u, 0u};
    }
  }
  __device__ __forceinline__ void put(Tin* dst, int ld) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = i * NT + threadIdx.x, row = e / PER, col = e % PER * VE;
      *reinterpret_cast<uint4*>(dst + row * ld + col) = v[i];
    }
  }
};

}  // namespace osdn
