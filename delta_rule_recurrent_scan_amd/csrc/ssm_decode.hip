// Selective scan, single tokens: T tokens (usually 1) through
//   S <- exp(dt A) S + (dt x) B^T,   y = S C + D x
// with the P x N fp32 state of a (batch, head) in the registers of one
// workgroup, read once and written once. Bound by streaming that state (two
// 64 KB passes at 128 x 128 against under 1 KB of token data): a row is spread
// over 16 lanes in 16-byte pieces, so a load instruction of a lane group covers
// 256 contiguous bytes, and the readout's row sums are row-of-16 DPP sums with
// no barrier. The state may be written over itself: every element is read
// and written by the same thread. 2048 states of 128 x 128, 270 MB: 41 us
// when the same states move on call after call (part of them is still in the
// memory-side cache), 51 us with other states each call, 5.3 TB/s, which is what
// a copy of that size reaches.
#include "launch.hpp"
#include "mixer.hpp"
#include "row_state.hpp"
#include "ssm_common.hpp"

namespace osdn {
namespace {

template <int P, int N, typename Tin>
__global__ __launch_bounds__(kDecThreads) void ssm_decode_kernel(SsmArgs a) {
  constexpr int NC = N / 16, NR = P / 16;
  const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H;
  const int cl = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const float* S0 = a.S0 + (size_t)bh * P * N;
  float s[NR][NC];
#pragma unroll
  for (int i = 0; i < NR; ++i) load_cols<N, float>(S0 + (size_t)(rg + 16 * i) * N, cl, s[i]);
  const float A = a.A[h], D = a.D ? a.D[h] : 0.f, bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  const size_t th = (size_t)bh * a.T;
  const size_t tg = ((size_t)b * a.G + h / (a.H / a.G)) * a.T;
  for (int t = 0; t < a.T; ++t) {
    float Bv[NC], Cv[NC];
    load_cols<N, Tin>((const Tin*)a.Bm + (tg + t) * N, cl, Bv);
    load_cols<N, Tin>((const Tin*)a.Cm + (tg + t) * N, cl, Cv);
    float slope;
    const float dt = ssm_step(a.dt[th + t], bias, a.softplus, slope);
    const float al = expf(dt * A);
    float x[NR], y[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      x[i] = to_f32(((const Tin*)a.x)[(th + t) * P + rg + 16 * i]);
      float acc = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        s[i][j] = al * s[i][j] + dt * x[i] * Bv[j];
        acc += s[i][j] * Cv[j];
      }
      y[i] = acc;
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) y[i] = row16_sum(y[i]) + D * x[i];
#pragma unroll
    for (int i = 0; i < NR; ++i)
      if (cl == (i & 15)) ((Tin*)a.y)[(th + t) * P + rg + 16 * i] = from_f32<Tin>(y[i]);
  }
  float* ST = a.ST + (size_t)bh * P * N;
#pragma unroll
  for (int i = 0; i < NR; ++i) store_cols<N>(ST + (size_t)(rg + 16 * i) * N, cl, s[i]);
}

template <int P, int N>
int run_decode(const SsmArgs& a, hipStream_t s) {
  if (!grid_ok((long long)a.B * a.H, kDecThreads)) return -1;
  const int tk = ktimer_before(s, "ssm_decode");
  if (a.bf16) {
    hipLaunchKernelGGL((ssm_decode_kernel<P, N, __bf16>), dim3(a.B * a.H), dim3(kDecThreads), 0,
                       s, a);
  } else {
    hipLaunchKernelGGL((ssm_decode_kernel<P, N, float>), dim3(a.B * a.H), dim3(kDecThreads), 0,
                       s, a);
  }
  ktimer_after(s, tk);
  return (int)hipGetLastError();
}

template <int P>
int run_decode_n(const SsmArgs& a, hipStream_t s) {
  switch (a.N) {
    case 32: return run_decode<P, 32>(a, s);
    case 64: return run_decode<P, 64>(a, s);
    case 128: return run_decode<P, 128>(a, s);
  }
  return -1;
}

}  // namespace

int launch_ssm_decode(const SsmArgs& a, hipStream_t s) {
  switch (a.P) {
    case 32: return run_decode_n<32>(a, s);
    case 64: return run_decode_n<64>(a, s);
    case 128: return run_decode_n<128>(a, s);
  }
  return -1;
}

}  // namespace osdn
