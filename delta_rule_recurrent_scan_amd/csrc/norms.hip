// Norms around a block.
//
// Gated head norm: from the heads [B,H,T,D] a recurrence leaves to the token
// rows [B,T,H*D] of the output projection, with the gate z of the same rows:
//   gate after:  y = x * rsqrt(mean_head x^2 + eps) * weight * silu(z)
//   gate first:  v = x * silu(z),  y = v * rsqrt(mean_head v^2 + eps) * weight
// Residual norm: h = residual + scale * x,  y = h * rsqrt(mean h^2 + eps) *
// weight, with h kept for the next block (y is formed from the 32-bit h, the
// stored one is rounded to the residual's type).
//
// All are bound by HBM: every input is read and every output written once,
// 16 bytes a lane, with the sums in 32 bits. A head is 4, 8 or 16 adjacent
// lanes; a row of the residual norm is one wave (up to 1536 elements, no
// barrier) or four, held in registers between the sum and the scaling. In bf16,
// where a copy of 256 MiB reaches 5.4 TB/s: gated norm of 16384 rows of 16 heads of
// 128, 201 MB, 36 to 38 us (5.3 to 5.6 TB/s); residual norm of 16384 rows of 2048 on a 32-bit
// stream, 403 MB, 68 to 72 us (5.6 to 5.9 TB/s).
//
// Backward of n = v r, y = n * weight (r the reciprocal root):
//   dn = dy * weight,  dv = r (dn - n mean(n dn)),  dweight = sum dy n
// Weight gradients stay in registers while a workgroup walks its rows, are
// added over its row lanes in LDS and leave as one partial a workgroup,
// summed in a fixed order by column_sum. Gated: 16384 rows of 8 heads of 64, 84 MB,
// 16 to 19 us and 2 to 4 us for the sum; residual: 4097 rows of 1021, 42 MB, 11 to 14
// us and 3 to 5 us (with a partial a wave and unaligned rows element by element it was
// 69 us: they take the same wide accesses as aligned ones now).
#include "launch.hpp"
#include "mixer.hpp"
#include "row_common.hpp"

namespace osdn {
namespace {

// ---------------------------------------------------------------------------
// Gated head norm
// ---------------------------------------------------------------------------

// A thread takes 8 channels of one row: of 201 MB of bf16, in turn, 1 row a thread
// takes 37 us, 2 take 39 and 4 take 43 (fewer workgroups, each longer).
template <typename Tin, bool ZALN>
__global__ __launch_bounds__(kRowThreads) void gated_norm_kernel(GatedNormArgs a, int cx) {
  const int D = a.D, C = a.H * D, ng = C / 8, L = D / 8;
  const int ncb = (ng + cx - 1) / cx, per = kRowThreads / cx;
  const int cg = (int)(blockIdx.x % ncb) * cx + (threadIdx.x & (cx - 1));
  const long long row = (blockIdx.x / ncb) * (long long)per + threadIdx.x / cx;
  if (cg >= ng || row >= (long long)a.B * a.T) return;  // a head's lanes leave together
  const int c = cg * 8, h = c / D, d = c % D;
  const long long b = row / a.T, t = row % a.T;
  float w[8], x[8], g[8];
  load_v<true, 8>((const Tin*)a.x + ((b * a.H + h) * a.T + t) * D + d, 8, x);
  if (a.z) load_v<ZALN, 8>((const Tin*)a.z + b * a.zbs + t * a.zts + c, 8, g);
  load_v<false, 8>(a.weight + (a.per_head ? c : d), 8, w);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    g[i] = a.z ? g[i] * sigmoid_f(g[i]) : 1.f;
    if (a.gate_first) x[i] *= g[i];
    s += x[i] * x[i];
  }
  const float r = rsqrtf(head_sum(s, L) / D + a.eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i] * (a.gate_first ? 1.f : g[i]);
  store_v<true, 8>((Tin*)a.y + row * C + c, 8, x);
}

template <typename Tin, bool ZALN>
__global__ __launch_bounds__(kRowThreads) void gated_norm_bwd_kernel(GatedNormArgs a, int cx,
                                                                     int nrb) {
  const int D = a.D, C = a.H * D, ng = C / 8, L = D / 8;
  const int ncb = (ng + cx - 1) / cx, per = kRowThreads / cx;
  const int cb = blockIdx.x % ncb, rb = blockIdx.x / ncb;
  const int cg = cb * cx + (threadIdx.x & (cx - 1));
  const long long rows = (long long)a.B * a.T;
  const int c = cg * 8, h = c / D, d = c % D;
  float dw[8] = {};
  if (cg < ng) {
    float w[8];
    load_v<false, 8>(a.weight + (a.per_head ? c : d), 8, w);
    const Tin* z = (const Tin*)a.z;
    // one row at a time: two in flight take a quarter longer (fewer waves a SIMD)
    for (long long row = rb * (long long)per + threadIdx.x / cx; row < rows;
         row += (long long)nrb * per) {
      const long long b = row / a.T, t = row % a.T;
      const size_t at = ((b * a.H + h) * a.T + t) * D + d;
      float x[8], g[8], e[8];
      load_v<true, 8>((const Tin*)a.x + at, 8, x);
      if (z) load_v<ZALN, 8>(z + b * a.zbs + t * a.zts + c, 8, g);
      load_v<true, 8>((const Tin*)a.dy + row * C + c, 8, e);
      float gate[8], sl[8], v[8], s = 0.f, q = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float sg = z ? sigmoid_f(g[i]) : 1.f;
        gate[i] = z ? g[i] * sg : 1.f;
        sl[i] = z ? sg * (1.f + g[i] * (1.f - sg)) : 0.f;
        v[i] = a.gate_first ? x[i] * gate[i] : x[i];
        const float up = a.gate_first ? e[i] : e[i] * gate[i];
        s += v[i] * v[i];
        q += v[i] * up * w[i];
      }
      const float r = rsqrtf(head_sum(s, L) / D + a.eps);
      const float m = head_sum(q, L) / D * r * r * r;
      float dx[8], dz[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = v[i] * r;
        const float up = a.gate_first ? e[i] : e[i] * gate[i];
        dw[i] += up * n;
        const float dv = r * up * w[i] - v[i] * m;
        dx[i] = a.gate_first ? dv * gate[i] : dv;
        dz[i] = (a.gate_first ? dv * x[i] : e[i] * n * w[i]) * sl[i];
      }
      store_v<true, 8>((Tin*)a.dx + at, 8, dx);
      if (z) store_v<true, 8>((Tin*)a.dz + row * C + c, 8, dz);
    }
  }
  // the workgroup's rows added, and its heads where they share the weight
  __shared__ float red[kRowThreads * 9];
#pragma unroll
  for (int i = 0; i < 8; ++i) red[threadIdx.x * 9 + i] = dw[i];
  __syncthreads();
  const int cols = a.per_head ? cx * 8 : D;
  for (int e = threadIdx.x; e < cols; e += kRowThreads) {
    const int col = cb * cx * 8 + e;
    if (a.per_head && col >= C) continue;
    float s = 0.f;
    for (int r = 0; r < per; ++r)
      for (int k = e / 8; k < cx; k += cols / 8) s += red[(r * cx + k) * 9 + e % 8];
    if (a.per_head) {
      ((float*)a.ws)[(size_t)rb * C + col] = s;
    } else {
      ((float*)a.ws)[(size_t)blockIdx.x * D + e] = s;
    }
  }
}

bool z_aligned(const GatedNormArgs& a) {
  const size_t es = a.bf16 ? 2 : 4;
  return ((size_t)a.z & 15) == 0 && (a.zbs * es & 15) == 0 && (a.zts * es & 15) == 0;
}

template <typename Tin>
int run_gated(const GatedNormArgs& a, hipStream_t s) {
  const int ng = a.H * a.D / 8, cx = row_cx(ng), per = kRowThreads / cx;
  const long long rows = (long long)a.B * a.T;
  const long long wgs = (ng + cx - 1) / cx * ((rows + per - 1) / per);
  if (!grid_ok(wgs, kRowThreads)) return -1;
  const dim3 grid((unsigned)wgs);
  const int tk = ktimer_before(s, "gated_norm");
  if (z_aligned(a)) {
    hipLaunchKernelGGL((gated_norm_kernel<Tin, true>), grid, dim3(kRowThreads), 0, s, a, cx);
  } else {
    hipLaunchKernelGGL((gated_norm_kernel<Tin, false>), grid, dim3(kRowThreads), 0, s, a, cx);
  }
  ktimer_after(s, tk);
  return (int)hipGetLastError();
}

// Row blocks of the backward: about 1024 workgroups in all (4 a CU), each
// with one partial row of the weight gradient.
int gate_row_blocks(int B, int H, int T, int D) {
  if (H == 0) return 0;
  const int ng = H * D / 8, cx = row_cx(ng), per = kRowThreads / cx;
  const long long rows = (long long)B * T, ncb = (ng + cx - 1) / cx;
  long long most = 1024 / ncb, need = (rows + per - 1) / per;
  if (most < 1) most = 1;
  return (int)(need < most ? need : most);
}

template <typename Tin>
int run_gated_bwd(const GatedNormArgs& a, hipStream_t s) {
  const int ng = a.H * a.D / 8, cx = row_cx(ng);
  const int nrb = gate_row_blocks(a.B, a.H, a.T, a.D);
  if (!column_sum_ok(a.per_head ? (long long)a.H * a.D : a.D)) return -1;
  const dim3 grid((unsigned)((ng + cx - 1) / cx * nrb));
  const int tk = ktimer_before(s, "gated_norm_bwd");
  if (nrb == 0) {
    // no rows: the sums below are zeros
  } else if (z_aligned(a)) {
    hipLaunchKernelGGL((gated_norm_bwd_kernel<Tin, true>), grid, dim3(kRowThreads), 0, s, a, cx,
                       nrb);
  } else {
    hipLaunchKernelGGL((gated_norm_bwd_kernel<Tin, false>), grid, dim3(kRowThreads), 0, s, a,
                       cx, nrb);
  }
  ktimer_after(s, tk);
  const int rc = (int)hipGetLastError();
  if (rc) return rc;
  if (a.per_head)
    return launch_column_sum((const float*)a.ws, nrb, a.H * a.D, a.H * a.D, 1, a.dweight,
                             nullptr, nullptr, s);
  return launch_column_sum((const float*)a.ws, (int)grid.x, a.D, a.D, 1, a.dweight, nullptr,
                           nullptr, s);
}

// ---------------------------------------------------------------------------
// Residual norm: WPR waves a row, each lane NV vectors of 8 elements.
// ---------------------------------------------------------------------------

// Sum over the WPR waves of a row (every wave of the workgroup calls it).
template <int WPR>
__device__ __forceinline__ float row_total(float s, float* red) {
  s = wave_sum(s);
  if constexpr (WPR > 1) {
    const int w = wave_id();
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[w] = s;
    __syncthreads();
    s = 0.f;
    const int w0 = w / WPR * WPR;
#pragma unroll
    for (int i = 0; i < WPR; ++i) s += red[w0 + i];
  }
  return s;
}

constexpr int kResThreads = 256, kResWaves = kResThreads / 64;

template <typename Tin, typename Tr, bool ALN, int NV, int WPR>
__global__ __launch_bounds__(kResThreads) void residual_norm_kernel(ResidualNormArgs a) {
  constexpr int RPW = kResWaves / WPR;  // rows of a workgroup
  __shared__ float red[kResWaves];
  const long long row = blockIdx.x * (long long)RPW + threadIdx.x / (64 * WPR);
  const int l = threadIdx.x % (64 * WPR);
  const bool on = row < a.R;
  const size_t base = (size_t)(on ? row : 0) * a.C;
  float h[NV][8], s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * 64 * WPR + l) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[j][i] = 0.f;
    if (!on || c >= a.C) continue;
    float x[8];
    load_v<ALN, 8>((const Tin*)a.x + base + c, a.C - c, x);
    if (a.residual) load_v<ALN, 8>((const Tr*)a.residual + base + c, a.C - c, h[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[j][i] += a.scale * x[i];
      s += h[j][i] * h[j][i];
    }
  }
  const float r = rsqrtf(row_total<WPR>(s, red) / a.C + a.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * 64 * WPR + l) * 8;
    if (!on || c >= a.C) continue;
    float w[8];
    load_v<ALN, 8>(a.weight + c, a.C - c, w);
    if (a.h) store_v<ALN, 8>((Tr*)a.h + base + c, a.C - c, h[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[j][i] *= r * w[i];
    store_v<ALN, 8>((Tin*)a.y + base + c, a.C - c, h[j]);
  }
}

template <typename Tin, typename Tr, bool ALN, int NV, int WPR>
__global__ __launch_bounds__(kResThreads) void residual_norm_bwd_kernel(ResidualNormArgs a) {
  constexpr int RPW = kResWaves / WPR;
  __shared__ float red[kResWaves];
  __shared__ float wred[RPW > 1 ? NV * 64 * 9 : 1];
  const int l = threadIdx.x % (64 * WPR);
  float dw[NV][8] = {};
  const long long step = (long long)gridDim.x * RPW;
  // rows of one workgroup run in step (the barriers of row_total)
  for (long long first = blockIdx.x * (long long)RPW; first < a.R; first += step) {
    const long long row = first + threadIdx.x / (64 * WPR);
    const bool on = row < a.R;
    const size_t base = (size_t)(on ? row : 0) * a.C;
    float h[NV][8], e[NV][8], s = 0.f, q = 0.f;
    Raw<Tr, 8> g[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * 64 * WPR + l) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = e[j][i] = 0.f;
      g[j].zero();
      if (!on || c >= a.C) continue;
      load_v<ALN, 8>((const Tr*)a.h + base + c, a.C - c, h[j]);
      load_v<ALN, 8>((const Tin*)a.dy + base + c, a.C - c, e[j]);
      if (a.dh) g[j].template load<ALN>((const Tr*)a.dh + base + c, a.C - c);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * 64 * WPR + l) * 8;
      if (!on || c >= a.C) continue;
      float w[8];
      load_v<ALN, 8>(a.weight + c, a.C - c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s += h[j][i] * h[j][i];
        q += h[j][i] * e[j][i] * w[i];
      }
    }
    const float r = rsqrtf(row_total<WPR>(s, red) / a.C + a.eps);
    const float m = row_total<WPR>(q, red) / a.C * r * r * r;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * 64 * WPR + l) * 8;
      if (!on || c >= a.C) continue;
      float w[8], gv[8];
      load_v<ALN, 8>(a.weight + c, a.C - c, w);
      g[j].widen(gv);
      float dx[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw[j][i] += e[j][i] * h[j][i] * r;
        gv[i] += r * e[j][i] * w[i] - h[j][i] * m;
        dx[i] = a.scale * gv[i];
      }
      store_v<ALN, 8>((Tin*)a.dx + base + c, a.C - c, dx);
      if (a.dres) store_v<ALN, 8>((Tr*)a.dres + base + c, a.C - c, gv);
    }
  }
  // the workgroup's rows added, one wave after the other: one partial each
  if constexpr (RPW > 1) {
    for (int r = RPW - 1; r >= 0; --r) {
      if (wave_id() == r) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float* p = wred + (j * 64 + l) * 9 + i;
            if (r < RPW - 1) dw[j][i] += *p;
            if (r > 0) *p = dw[j][i];
          }
      }
      __syncthreads();
    }
    if (wave_id() != 0) return;
  }
  float* part = (float*)a.ws + (size_t)blockIdx.x * a.C;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * 64 * WPR + l) * 8;
    if (c < a.C) store_v<ALN, 8>(part + c, a.C - c, dw[j]);
  }
}

// Waves and vectors a row. One wave (no barrier) while a row is 3 vectors a lane;
// above, the four waves of a workgroup, which leave fewer registers a lane and more
// rows in flight. bf16 on fp32: 16384 rows of 2048, 79 us at 4 vectors of one wave
// and 69 us at 1 of four, backward 84 and 74 us; of 4096, 164 and 143 us (8 against
// 2 vectors), backward 211 and 172 us; 4097 rows of 1501, where a quarter of the
// four waves' lanes is idle, 11 and 12 us.
constexpr int kMaxWidth = kResWaves * 64 * 8 * 8;  // 16384
struct Shape {
  int nv, wpr;
};
Shape row_shape(int C) {
  for (int nv = 1; nv <= 3; ++nv)
    if (64 * 8 * nv >= C) return Shape{nv, 1};
  for (int nv = 1; nv <= 4; nv *= 2)
    if (64 * 8 * kResWaves * nv >= C) return Shape{nv, kResWaves};
  return Shape{8, kResWaves};
}

// Workgroups of the backward, each a partial row of the weight gradient: four a
// CU for rows of one wave, two for the wider ones, whose partials cost more. With
// the column sum: 4097 rows of 1021 bf16 14 us with 1024 partials and 16 with 512;
// 65536 of 512 75 and 79; 16384 of 2048 on fp32 79 and 76; of 8192 338 and 328.
int res_blocks(long long R, int wpr) {
  const int rpw = kResWaves / wpr;
  const long long need = (R + rpw - 1) / rpw;
  const long long most = wpr == 1 ? 1024 : 512;
  return (int)(need < most ? need : most);
}

template <typename Tin, typename Tr, bool ALN, int NV, int WPR>
int run_res(const ResidualNormArgs& a, int bwd, hipStream_t s) {
  if (!bwd) {
    const int rpw = kResWaves / WPR;
    if (!grid_ok((a.R + rpw - 1) / rpw, kResThreads)) return -1;
    const int tk = ktimer_before(s, "residual_norm");
    hipLaunchKernelGGL((residual_norm_kernel<Tin, Tr, ALN, NV, WPR>),
                       dim3((unsigned)((a.R + rpw - 1) / rpw)), dim3(kResThreads), 0, s, a);
    ktimer_after(s, tk);
    return (int)hipGetLastError();
  }
  const int nb = res_blocks(a.R, WPR);
  if (nb) {
    const int tk = ktimer_before(s, "residual_norm_bwd");
    hipLaunchKernelGGL((residual_norm_bwd_kernel<Tin, Tr, ALN, NV, WPR>), dim3(nb),
                       dim3(kResThreads), 0, s, a);
    ktimer_after(s, tk);
    const int rc = (int)hipGetLastError();
    if (rc) return rc;
  }
  return launch_column_sum((const float*)a.ws, nb, a.C, a.C, 1, a.dweight, nullptr, nullptr, s);
}

template <typename Tin, typename Tr, bool ALN>
int run_res_n(const ResidualNormArgs& a, int bwd, hipStream_t s) {
  const Shape p = row_shape(a.C);
  switch (p.nv + (p.wpr == 1 ? 0 : 10)) {
    case 1: return run_res<Tin, Tr, ALN, 1, 1>(a, bwd, s);
    case 2: return run_res<Tin, Tr, ALN, 2, 1>(a, bwd, s);
    case 3: return run_res<Tin, Tr, ALN, 3, 1>(a, bwd, s);
    case 11: return run_res<Tin, Tr, ALN, 1, kResWaves>(a, bwd, s);
    case 12: return run_res<Tin, Tr, ALN, 2, kResWaves>(a, bwd, s);
    case 14: return run_res<Tin, Tr, ALN, 4, kResWaves>(a, bwd, s);
    case 18: return run_res<Tin, Tr, ALN, 8, kResWaves>(a, bwd, s);
  }
  return -1;
}

template <typename Tin, typename Tr>
int run_res_t(const ResidualNormArgs& a, bool aln, int bwd, hipStream_t s) {
  return aln ? run_res_n<Tin, Tr, true>(a, bwd, s) : run_res_n<Tin, Tr, false>(a, bwd, s);
}

int run_res_any(const ResidualNormArgs& a, bool aln, int bwd, hipStream_t s) {
  if (a.bf16)
    return a.res_bf16 ? run_res_t<__bf16, __bf16>(a, aln, bwd, s)
                      : run_res_t<__bf16, float>(a, aln, bwd, s);
  return a.res_bf16 ? -1 : run_res_t<float, float>(a, aln, bwd, s);
}

bool al(const void* p) { return ((size_t)p & 15) == 0; }

}  // namespace

int launch_gated_norm(const GatedNormArgs& a, hipStream_t s) {
  return a.bf16 ? run_gated<__bf16>(a, s) : run_gated<float>(a, s);
}

size_t gated_norm_backward_ws(int B, int H, int T, int D) {
  if (H == 0) return 0;
  return (size_t)gate_row_blocks(B, H, T, D) * H * D * sizeof(float);
}

int launch_gated_norm_backward(const GatedNormArgs& a, hipStream_t s) {
  return a.bf16 ? run_gated_bwd<__bf16>(a, s) : run_gated_bwd<float>(a, s);
}

int launch_residual_norm(const ResidualNormArgs& a, hipStream_t s) {
  if (a.C > kMaxWidth) return -1;
  const bool aln = a.C % 8 == 0 && al(a.x) && al(a.residual) && al(a.weight) && al(a.y) && al(a.h);
  return run_res_any(a, aln, 0, s);
}

size_t residual_norm_backward_ws(long long R, int C) {
  if (C > kMaxWidth) return 0;
  return (size_t)res_blocks(R, row_shape(C).wpr) * C * sizeof(float);
}

int launch_residual_norm_backward(const ResidualNormArgs& a, hipStream_t s) {
  if (a.C > kMaxWidth) return -1;
  const bool aln = a.C % 8 == 0 && al(a.dy) && al(a.h) && al(a.weight) && al(a.dh) && al(a.dx) &&
                   al(a.dres) && al(a.ws);
  return run_res_any(a, aln, 1, s);
}

}  // namespace osdn
