// Device helpers shared by the selective-scan kernels.
#pragma once

#include "device_common.hpp"
#include "launch.hpp"
#include "mixer.hpp"
#include "pack_common.hpp"

namespace osdn {

// The step size of a token, softplus(raw + bias) (or raw + bias itself), and
// its slope by raw. softplus(v) = max(v, 0) + log1p(e), e = exp(-|v|), from the
// hardware's exp2 and log2 (one unit each): the argument's rounding is put
// back into e, and log1p(e) = log(1 + e) e / ((1 + e) - 1) makes up for the
// rounding of 1 + e. slope = 1 / (1 + exp(-v)). Behind |v| = 128 e is zero in
// fp32; the argument stops there, so that its product with log2(e) and what that
// lost are numbers also for infinite v and at the ends of the range, where they
// would be inf - inf: a raw step of -inf or of the lowest value is a step of zero
// with a slope of zero. A NaN compares false and stays.
__device__ __forceinline__ float ssm_step(float raw, float bias, int softplus, float& slope) {
  const float v = raw + bias;
  slope = 1.f;
  if (!softplus) return v;
  const float m = -fabsf(v), x = m < -128.f ? -128.f : m, t = x * 1.44269504f;
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

// A log decay as an fp32 sum and what its roundings lost. Sums of a few
// tens would otherwise carry an error of 2^-24 of themselves, absolute, into
// the exponent: 1e-6 relative on the decays, and the same one for every token
// behind, which adds up in the gradients of A and of the step's bias.
struct Log2f {
  float hi, lo;
};
__device__ __forceinline__ Log2f add(Log2f a, Log2f b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  return {s, ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo)};
}
// exp of it, the rounding of x log2(e) put back as well (into numbers: a factor
// past fp32's range is inf, where inf times what was lost would be NaN).
__device__ __forceinline__ float exp_of(float hi, float lo) {
  const float t = hi * 1.44269504f;
  const float lost = fmaf(hi, 1.44269504f, -t) + hi * 1.92596299e-8f;
  const float e = __builtin_amdgcn_exp2f(t);
  const float r = fmaf(e, fmaf(lost, 0.693147181f, lo), e);
  return e == INFINITY ? e : r;
}
__device__ __forceinline__ float exp_of(Log2f x) { return exp_of(x.hi, x.lo); }

template <int CTRL>
__device__ __forceinline__ Log2f dpp_l(Log2f x) {
  return {dpp_f<CTRL>(x.hi), dpp_f<CTRL>(x.lo)};
}
// Inclusive prefix sums over each row of 16 lanes, and the sums of the lanes
// behind each one (zeros come in from outside the row).
__device__ __forceinline__ Log2f row16_prefix(Log2f x) {
  x = add(x, dpp_l<0x111>(x));  // row_shr:1, :2, :4, :8
  x = add(x, dpp_l<0x112>(x));
  x = add(x, dpp_l<0x114>(x));
  x = add(x, dpp_l<0x118>(x));
  return x;
}
__device__ __forceinline__ Log2f row16_suffix_after(Log2f x) {
  x = add(x, dpp_l<0x101>(x));  // row_shl:1, :2, :4, :8
  x = add(x, dpp_l<0x102>(x));
  x = add(x, dpp_l<0x104>(x));
  x = add(x, dpp_l<0x108>(x));
  return dpp_l<0x101>(x);
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
  float ul[Q];    // what `up` lost to rounding
  float eup[Q];   // exp(up)
  float edn[Q];   // exp(log: after token .. block end)
  float ent[Q];   // chunk entry .. token
  float wx[Q];    // after token .. chunk exit, times dt
  float ext[Q];   // the same without dt
  float slope[Q]; // of the step by its raw value
  float gap[16];  // [a][b], a > b: exp over the blocks strictly between
  float total;    // whole chunk
  float logtot;
  float pad[2];

  // By one whole wave; lane t (< Q) passes its token's step, the step's slope
  // and A.
  __device__ __forceinline__ void fill(float step, float sl, float A) {
    constexpr int NB = Q / 16;
    const int t = threadIdx.x & 63;
    // below -256 a decay is zero whatever it is (and stays it over any growth that
    // fp32 holds); cut there, so that the sums' rounding errors are numbers, and
    // small enough to enter the exponential to first order: behind 15 tokens of -1e4
    // a pair's factor was off by 3e-5
    const float p = step * A;
    const Log2f l = p < -256.f ? Log2f{-256.f, 0.f} : Log2f{p, fmaf(step, A, -p)};
    const Log2f u = row16_prefix(l), d = row16_suffix_after(l);
    Log2f bs[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      bs[b].hi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(u.hi), 16 * b + 15));
      bs[b].lo = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(u.lo), 16 * b + 15));
    }
    Log2f before = {0.f, 0.f}, after = before, all = before, between = before;
    const int x = t / NB, y = t % NB;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const Log2f zero = {0.f, 0.f};
      before = add(before, b < t / 16 ? bs[b] : zero);
      after = add(after, b > t / 16 ? bs[b] : zero);
      between = add(between, b > y && b < x ? bs[b] : zero);
      all = add(all, bs[b]);
    }
    if (t < Q) {
      dt[t] = step;
      up[t] = u.hi;
      ul[t] = u.lo;
      eup[t] = exp_of(u);
      edn[t] = exp_of(d);
      ent[t] = exp_of(add(before, u));
      const float e = exp_of(add(d, after));
      wx[t] = e * step;
      ext[t] = e;
      slope[t] = sl;
    }
    if (t < NB * NB) gap[x * 4 + y] = exp_of(between);
    if (t == 0) {
      total = exp_of(all);
      logtot = all.hi;
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
    const f32x4 ul = *reinterpret_cast<const f32x4*>(d.ul + j);
    const float v = d.up[i], vl = d.ul[i];
#pragma unroll
    for (int r = 0; r < 4; ++r) f[r] = j + r <= i ? exp_of(v - u[r], vl - ul[r]) : 0.f;
  }
  return f;
}

// The steps of the tile's tokens j.
template <int Q>
__device__ __forceinline__ f32x4 tile_steps(const ChunkDecay<Q>& d, int jt) {
  return *reinterpret_cast<const f32x4*>(d.dt + jt * 16 + acc_row(0));
}

// row16_sum in 64 bits.
template <int CTRL>
__device__ __forceinline__ double dpp_d(double x) {
  const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
  const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)u, CTRL, 0xf, 0xf, false);
  const unsigned hi =
      __builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), CTRL, 0xf, 0xf, false);
  return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
__device__ __forceinline__ double row16_sum(double x) {
  x += dpp_d<0xB1>(x);
  x += dpp_d<0x4E>(x);
  x += dpp_d<0x141>(x);
  x += dpp_d<0x140>(x);
  return x;
}

__device__ __forceinline__ double wave_sum(double x) {
  x = row16_sum(x);
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}

// Inclusive sum of lanes l .. 63, and exclusive sum of lanes 0 .. l - 1. In 64
// bits: what the sums take in cancels in part (a chunk's pairs enter a token's
// decay gradient as the difference of two running sums).
__device__ __forceinline__ double wave_suffix_sum(double x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double y = __shfl_down(x, d, 64);
    if (lane + d < 64) x += y;
  }
  return x;
}
__device__ __forceinline__ double wave_prefix_before(double x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  const double y = __shfl_up(x, 1, 64);
  return lane ? y : 0.;
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

// Values that are inf or NaN. The test of a whole fragment is the largest exponent
// of the wave's elements, two operations a register, and the same for every lane.
__device__ __forceinline__ bool strange(__bf16 x) {
  return (__builtin_bit_cast(unsigned short, x) & 0x7f80) == 0x7f80;
}
__device__ __forceinline__ bool strange(float x) {
  return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u;
}
template <int KEXT>
__device__ __forceinline__ bool any_strange(const Frag<KEXT, __bf16>& f) {
  typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < KEXT / 32; ++i) {
    const u32x4 u = __builtin_bit_cast(u32x4, f.v[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, u[e] & 0x7fff7fffu));
  }
  return __ballot(max(m[0], m[1]) >= 0x7f80) != 0;
}
template <int KEXT>
__device__ __forceinline__ bool any_strange(const Frag<KEXT, float>& f) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < KEXT / 4; ++i) m = max(m, __float_as_uint(f.v[i]) & 0x7fffffffu);
  return __ballot(m >= 0x7f800000u) != 0;
}
template <int KEXT>
__device__ __forceinline__ void drop_strange(Frag<KEXT, __bf16>& f) {
#pragma unroll
  for (int i = 0; i < KEXT / 32; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (strange(f.v[i][e])) f.v[i][e] = (__bf16)0.f;
}
template <int KEXT>
__device__ __forceinline__ void drop_strange(Frag<KEXT, float>& f) {
#pragma unroll
  for (int i = 0; i < KEXT / 4; ++i)
    if (strange(f.v[i])) f.v[i] = 0.f;
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

// The same in two parts, the rounded values and what their rounding lost (16
// bits in all), `part` elements apart; fp32 is one part.
template <typename Tin>
constexpr int two_parts() { return sizeof(Tin) == 2 ? 2 : 1; }
// What rounding to the type loses.
__device__ __forceinline__ f32x4 rounding_rest(const f32x4& a, __bf16) {
  const unsigned x = pack_bf16(a[0], a[1]), y = pack_bf16(a[2], a[3]);
  return f32x4{a[0] - low_bf16(x), a[1] - high_bf16(x), a[2] - low_bf16(y), a[3] - high_bf16(y)};
}
__device__ __forceinline__ f32x4 rounding_rest(const f32x4&, float) {
  return f32x4{0.f, 0.f, 0.f, 0.f};
}
__device__ __forceinline__ void store4_two(__bf16* p, int part, const f32x4& a) {
  const uint2 hi = {pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3])};
  *reinterpret_cast<uint2*>(p) = hi;
  *reinterpret_cast<uint2*>(p + part) =
      uint2{pack_bf16(a[0] - low_bf16(hi.x), a[1] - high_bf16(hi.x)),
            pack_bf16(a[2] - low_bf16(hi.y), a[3] - high_bf16(hi.y))};
}
__device__ __forceinline__ void store4_two(float* p, int, const f32x4& a) { store4(p, a); }

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

// The decays of a chunk, formed once a call (ssm_decay), on their way through
// registers into LDS.
template <int Q, int NT>
struct StageDecay {
  static constexpr int N16 = sizeof(ChunkDecay<Q>) / 16, NV = (N16 + NT - 1) / NT;
  static_assert(sizeof(ChunkDecay<Q>) % 16 == 0, "whole 16-byte pieces");
  uint4 v[NV];
  __device__ __forceinline__ void fetch(const ChunkDecay<Q>* src) {
    const Buffer r = make_buffer(src, sizeof(*src));
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = buffer_load16(r, (threadIdx.x + i * NT) * 16);
  }
  __device__ __forceinline__ void put(ChunkDecay<Q>& dst) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (threadIdx.x + i * NT < N16) reinterpret_cast<uint4*>(&dst)[threadIdx.x + i * NT] = v[i];
  }
};

namespace {  // each source has its own kernel

// One wave a chunk of a (batch, head): bh = id / nch, chunk = id % nch.
template <int Q>
__global__ __launch_bounds__(256) void ssm_decay_kernel(SsmArgs a, int nch, long long n,
                                                        ChunkDecay<Q>* out) {
  const long long id = blockIdx.x * 4ll + wave_id();
  if (id >= n) return;
  const int lane = threadIdx.x & 63, c = (int)(id % nch);
  const long long bh = id / nch;
  const int h = (int)(bh % a.H), t = c * Q + lane;
  float sl = 0.f, st = 0.f;
  if (lane < Q && t < ssm_length(a.lengths, (int)(bh / a.H), a.T))
    st = ssm_step(a.dt[bh * a.T + t], a.dt_bias ? a.dt_bias[h] : 0.f, a.softplus, sl);
  out[id].fill(st, sl, a.A[h]);
}

// Bytes of the decays of a call, a multiple of 256.
template <int Q>
size_t decay_bytes(int B, int H, int T) {
  return ((size_t)B * H * ((T + Q - 1) / Q) * sizeof(ChunkDecay<Q>) + 255) / 256 * 256;
}

template <int Q>
void launch_decay(const SsmArgs& a, ChunkDecay<Q>* out, hipStream_t s) {
  const int nch = (a.T + Q - 1) / Q;
  const long long n = (long long)a.B * a.H * nch;
  if (n == 0) return;
  const int tk = ktimer_before(s, "ssm_decay");
  hipLaunchKernelGGL((ssm_decay_kernel<Q>), dim3((unsigned)((n + 3) / 4)), dim3(256), 0, s, a,
                     nch, n, out);
  ktimer_after(s, tk);
}

}  // namespace

}  // namespace osdn
