// Device helpers shared by the selective-scan kernels.
#pragma once

#include "device_common.hpp"

namespace osdn {

// The step size of a token, softplus(raw + bias) (or raw + bias itself), and
// its slope by raw. softplus(v) = max(v, 0) + log1p(e), e = exp(-|v|), from the
// hardware's exp2 and log2 (one unit each): the argument's rounding is put
// back into e, and log1p(e) = log(1 + e) e / ((1 + e) - 1) makes up for the
// rounding of 1 + e. slope = 1 / (1 + exp(-v)).
__device__ __forceinline__ float ssm_step(float raw, float bias, int softplus, float& slope) {
  const float v = raw + bias;
  slope = 1.f;
  if (!softplus) return v;
  const float x = -fabsf(v), t = x * 1.44269504f;
  const float lost = fmaf(x, 1.44269504f, -t) + x * 1.92596299e-8f;  // of x log2(e)
  float e = __builtin_amdgcn_exp2f(t);
  e = fmaf(e, lost * 0.693147181f, e);
  const float w = 1.f + e, d = w - 1.f;
  const float l = d > 0.f ? __builtin_amdgcn_logf(w) * 0.693147181f * (e / d) : e;
  slope = (v >= 0.f ? 1.f : e) / w;
  return fmaxf(v, 0.f) + l;
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
template <int Q, bool Grad = false>
struct ChunkDecay {
  float dt[Q];    // step
  float up[Q];    // log: block start .. token, inclusive
  float eup[Q];   // exp(up)
  float edn[Q];   // exp(log: after token .. block end)
  float ent[Q];   // chunk entry .. token
  float wx[Q];    // after token .. chunk exit, times dt
  float ext[Grad ? Q : 4];    // the same without dt
  float slope[Grad ? Q : 4];  // of the step by its raw value
  float gap[16];  // [a][b], a > b: exp over the blocks strictly between
  float total;    // whole chunk
  float logtot;

  // By one whole wave; lane t (< Q) passes its token's step, log decay and
  // slope.
  __device__ __forceinline__ void fill(float step, float l, float sl) {
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
      const float x = __expf(d + after);
      wx[t] = x * step;
      if constexpr (Grad) {
        ext[t] = x;
        slope[t] = sl;
      }
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
template <int Q, bool G>
__device__ __forceinline__ f32x4 pair_decay(const ChunkDecay<Q, G>& d, int it, int jt) {
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
template <int Q, bool G>
__device__ __forceinline__ f32x4 tile_steps(const ChunkDecay<Q, G>& d, int jt) {
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
  for (int i = 0; i < KEXT / 32; ++i) {
    const f32x4 &a = t[2 * i], &b = t[2 * i + 1];
    const u32x4 q = {pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(b[0], b[1]),
                     pack_bf16(b[2], b[3])};
    f.v[i] = __builtin_bit_cast(bf16x8, q);
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

__device__ __forceinline__ void split3(float x, float y, unsigned& a, unsigned& b, unsigned& c) {
  a = pack_bf16(x, y);
  x -= low_bf16(a);
  y -= high_bf16(a);
  b = pack_bf16(x, y);
  c = pack_bf16(x - low_bf16(b), y - high_bf16(b));
}

// x scaled by w[k] (natural k order, w in LDS).
template <int KEXT>
__device__ __forceinline__ void scale_parts(const Frag<KEXT, __bf16>& x, const float* w,
                                            Parts<KEXT, __bf16>& o) {
  const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int i = 0; i < KEXT / 32; ++i) {
    const f32x4 f[2] = {*reinterpret_cast<const f32x4*>(w + 32 * i + 8 * g),
                        *reinterpret_cast<const f32x4*>(w + 32 * i + 8 * g + 4)};
    const u32x4 u = __builtin_bit_cast(u32x4, x.v[i]);
    u32x4 q[3];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      unsigned p0, p1, p2;
      split3(low_bf16(u[e]) * f[e / 2][2 * (e & 1)], high_bf16(u[e]) * f[e / 2][2 * (e & 1) + 1],
             p0, p1, p2);
      q[0][e] = p0;
      q[1][e] = p1;
      q[2][e] = p2;
    }
#pragma unroll
    for (int m = 0; m < 3; ++m) o.f[m].v[i] = __builtin_bit_cast(bf16x8, q[m]);
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
  for (int i = 0; i < KEXT / 32; ++i) {
    u32x4 q[3];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      unsigned p0, p1, p2;
      split3(t[2 * i + e / 2][2 * (e & 1)], t[2 * i + e / 2][2 * (e & 1) + 1], p0, p1, p2);
      q[0][e] = p0;
      q[1][e] = p1;
      q[2][e] = p2;
    }
#pragma unroll
    for (int m = 0; m < 3; ++m) o.f[m].v[i] = __builtin_bit_cast(bf16x8, q[m]);
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
  *reinterpret_cast<uint2*>(p) = uint2{pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3])};
}
__device__ __forceinline__ void store4(float* p, const f32x4& a) {
  *reinterpret_cast<f32x4*>(p) = a;
}

// A buffer descriptor over `bytes` from p (both wave-uniform): reads past the
// end return zeros and writes past it are dropped, by the hardware's range
// check, so that the last tile of a sequence takes the same instructions as
// the others; and a 32-bit offset a lane is the whole address, where a 64-bit
// pointer a lane would cost the registers that the tiles need.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer make_buffer(const void* p, long long bytes) {
  const int n = bytes < 0 ? 0 : bytes > 0x7fffffff ? 0x7fffffff : (int)bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, n, 0x00027000);
}
__device__ __forceinline__ uint4 buffer_load16(Buffer r, unsigned off) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ float buffer_load_f32(Buffer r, unsigned off) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}
// Four consecutive values, rounded, to element `at`.
__device__ __forceinline__ void buffer_store4(Buffer r, unsigned at, const f32x4& a, __bf16) {
  typedef __attribute__((ext_vector_type(2))) unsigned u32x2;
  __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3])}, r,
                                        at * 2, 0, 0);
}
__device__ __forceinline__ void buffer_store4(Buffer r, unsigned at, const f32x4& a, float) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, a), r, at * 4, 0, 0);
}

// Staging of a Q x D tile of token rows through registers into LDS by NT
// threads, of rows STRIDE apart in memory and LD in LDS: fetch() issues the
// loads (rows from `valid` on are zeros), put() writes them.
template <int Q, int D, typename Tin, int NT, int LD, int STRIDE = D>
struct Stage {
  static constexpr int VE = 16 / sizeof(Tin), PER = D / VE, RP = NT / PER;
  static constexpr int NV = (Q + RP - 1) / RP;
  static_assert(NT % PER == 0, "threads cover whole rows");
  uint4 v[NV];
  __device__ __forceinline__ static int row0() { return threadIdx.x / PER; }
  __device__ __forceinline__ void fetch(const Tin* src, int valid) {
    const Buffer r = make_buffer(src, (long long)min(valid, Q) * STRIDE * (int)sizeof(Tin) -
                                          (STRIDE - D) * (int)sizeof(Tin));
    const unsigned off =
        (unsigned)(row0() * STRIDE + threadIdx.x % PER * VE) * (unsigned)sizeof(Tin);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      v[i] = buffer_load16(r, off + i * (unsigned)(RP * STRIDE * sizeof(Tin)));
  }
  __device__ __forceinline__ void put(Tin* dst) const {
    Tin* d = dst + row0() * LD + threadIdx.x % PER * VE;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (Q % RP == 0 || row0() + i * RP < Q)
        *reinterpret_cast<uint4*>(d + i * RP * LD) = v[i];
  }
};

}  // namespace osdn
