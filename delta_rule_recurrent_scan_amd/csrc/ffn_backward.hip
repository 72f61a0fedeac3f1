// Gated feed-forward product, backward, from the stored g and u:
//   dg = dh u act'(g),  du = dh act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
// A first kernel forms dg and du (5 elements moved for one of dh, bound by HBM) in
// the operands' type, the two products are tiles on the matrix units: dx over both
// halves of 2 F, the weights' gradients over the rows. dg and du are rounded once
// in bf16 (2^-9 of each term, as the results' own rounding is): held in two parts
// they would double the matrix work. Products whose tiles do not fill the card are
// split over k and added in a fixed order in 32 bits.
#include "ffn_common.hpp"
#include "launch.hpp"

namespace osdn {
namespace ffn {
namespace {

template <typename T>
__global__ __launch_bounds__(256) void ffn_grad_kernel(FfnArgs a, long long n, T* dg, T* du) {
  const long long at = (blockIdx.x * 256LL + threadIdx.x) * 8;
  if (at >= n) return;
  const int m = (int)min(8LL, n - at);
  float g[8], u[8], d[8];
  load_v<false, 8>((const T*)a.gate + at, m, g);
  load_v<false, 8>((const T*)a.up + at, m, u);
  load_v<false, 8>((const T*)a.dh + at, m, d);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f, s;
    activated(g[i], a.act, f, s);
    g[i] = d[i] * u[i] * s;
    u[i] = d[i] * f;
  }
  store_v<false, 8>(dg + at, m, g);
  store_v<false, 8>(du + at, m, u);
}

// dx: rows of dg and du (K-major over f) by the weights' columns (f along k). Tiles of
// k: the whole ones of dg, those of du, then the two ends.
template <typename T, class S>
struct InputSrc {
  typedef Stage<T, S::BM, true, S::NT> SA;
  typedef Stage<T, S::BN, false, S::NT> StageB;
  const T *dg, *du, *wg, *wu;
  int C, F, rows, cols, full;
  unsigned oa[SA::PER], ob[StageB::PER];
  uint4 va[SA::PER], vb[StageB::PER];
  __device__ __forceinline__ int place(int t, bool& second) const {
    const int half = full / 2;
    second = t < full ? t >= half : t > full;
    return (t < full ? t - (second ? half : 0) : half) * kTileK<T>;
  }
  __device__ __forceinline__ void direct_a(int t, char* a) const {
    bool second;
    const int k = place(t, second);
    SA::direct(a, (second ? du : dg) + k, oa);
  }
  __device__ __forceinline__ void direct_b(int t, char* b) const {
    bool second;
    const int k = place(t, second);
    StageB::direct(b, (second ? wu : wg) + (long long)k * C, ob);
  }
  __device__ __forceinline__ void fetch(int t) {
    bool second;
    const int k = place(t, second);
    SA::fetch(va, (second ? du : dg) + k, F, rows, F - k);
    StageB::fetch(vb, (second ? wu : wg) + (long long)k * C, C, cols, F - k);
  }
  __device__ __forceinline__ void put(char* a, char* b) const {
    SA::put(a, va);
    StageB::put(b, vb);
  }
  __device__ __forceinline__ uint4 fragb(const char* lb, int j, int step) const {
    return StageB::frag(lb, wave_id() % S::WN * (S::BN / S::WN) + 16 * j, step);
  }
};

// A weight's gradient: columns of dg or du by columns of x, rows along k.
template <typename T, class S>
struct WeightSrc {
  typedef Stage<T, S::BM, false, S::NT> SA;
  typedef Stage<T, S::BN, false, S::NT> StageB;
  const T *d, *x;
  long long R, xs;
  int F, rows, cols, full;
  unsigned oa[SA::PER], ob[StageB::PER];
  uint4 va[SA::PER], vb[StageB::PER];
  __device__ __forceinline__ void direct_a(int t, char* a) const {
    SA::direct(a, d + (long long)t * kTileK<T> * F, oa);
  }
  __device__ __forceinline__ void direct_b(int t, char* b) const {
    StageB::direct(b, x + (long long)t * kTileK<T> * xs, ob);
  }
  __device__ __forceinline__ void fetch(int t) {
    const long long k = (long long)t * kTileK<T>;
    const int nk = (int)min(R - k, (long long)kTileK<T>);
    SA::fetch(va, d + k * F, F, rows, nk);
    StageB::fetch(vb, x + k * xs, xs, cols, nk);
  }
  __device__ __forceinline__ void put(char* a, char* b) const {
    SA::put(a, va);
    StageB::put(b, vb);
  }
  __device__ __forceinline__ uint4 fragb(const char* lb, int j, int step) const {
    return StageB::frag(lb, wave_id() % S::WN * (S::BN / S::WN) + 16 * j, step);
  }
};

// A wave's tiles to rows of N columns from (m0, n0), as T or as fp32 parts.
template <typename T, class S>
__device__ __forceinline__ void store_tile(const f32x4 (&acc)[S::TM][S::TN], T* out, long long m0,
                                           long long M, int n0, int N, bool vec) {
  const int l = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  const int wm = wave_id() / S::WN * (S::BM / S::WM), wn = wave_id() % S::WN * (S::BN / S::WN);
#pragma unroll
  for (int i = 0; i < S::TM; ++i) {
    const long long m = m0 + wm + 16 * i + l;
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < S::TN; ++j) {
      const int n = n0 + wn + 16 * j + 4 * g;
      store4(out + m * N + n, acc[i][j], N - n, vec);
    }
  }
}

template <typename T, class S, bool DIRECT>
__global__ __launch_bounds__(S::NT) void ffn_dx_kernel(FfnArgs a, const T* dg, const T* du,
                                                       float* parts, int tm, int tn, int splits,
                                                       int per, int vec) {
  const TileAt at = tile_at(tm, tn, splits);
  const long long m0 = (long long)at.m * S::BM;
  const int n0 = at.n * S::BN;
  InputSrc<T, S> src;
  src.C = a.C;
  src.F = a.F;
  src.full = 2 * (a.F / kTileK<T>);
  src.dg = dg + m0 * a.F;
  src.du = du + m0 * a.F;
  src.wg = (const T*)a.wg + n0;
  src.wu = (const T*)a.wu + n0;
  src.rows = (int)min((long long)S::BM, a.R - m0);
  src.cols = min(S::BN, a.C - n0);
  if constexpr (DIRECT) {
    decltype(src)::SA::offsets(src.oa, a.F, src.rows);
    decltype(src)::StageB::offsets(src.ob, a.C, src.cols);
  }
  f32x4 acc[S::TM][S::TN];
  const int t0 = at.split * per, nt = 2 * ((a.F + kTileK<T> - 1) / kTileK<T>);
  products<T, S, true, DIRECT>(acc, src, t0, min(t0 + per, nt));
  if (splits > 1) {
    store_tile<float, S>(acc, parts + (long long)at.split * a.R * a.C, m0, a.R, n0, a.C, vec);
  } else {
    store_tile<T, S>(acc, (T*)a.dx, m0, a.R, n0, a.C, vec);
  }
}

// Tiles of m: first those of the gate's gradient, then those of the other.
template <typename T, class S, bool DIRECT>
__global__ __launch_bounds__(S::NT) void ffn_dw_kernel(FfnArgs a, const T* dg, const T* du,
                                                       float* parts, int tm, int tn, int splits,
                                                       int per, int vec) {
  const TileAt at = tile_at(2 * tm, tn, splits);
  const bool second = at.m >= tm;
  const int m0 = (at.m - (second ? tm : 0)) * S::BM, n0 = at.n * S::BN;
  WeightSrc<T, S> src;
  src.F = a.F;
  src.R = a.R;
  src.xs = a.xs;
  src.full = (int)(a.R / kTileK<T>);
  src.d = (second ? du : dg) + m0;
  src.x = (const T*)a.x + n0;
  src.rows = min(S::BM, a.F - m0);
  src.cols = min(S::BN, a.C - n0);
  if constexpr (DIRECT) {
    decltype(src)::SA::offsets(src.oa, a.F, src.rows);
    decltype(src)::StageB::offsets(src.ob, a.xs, src.cols);
  }
  const int nt = (int)((a.R + kTileK<T> - 1) / kTileK<T>);
  f32x4 acc[S::TM][S::TN];
  const int t0 = at.split * per;
  products<T, S, false, DIRECT>(acc, src, t0, min(t0 + per, nt));
  if (splits > 1) {
    float* p = parts + ((long long)(second ? splits : 0) + at.split) * a.F * a.C;
    store_tile<float, S>(acc, p, m0, a.F, n0, a.C, vec);
  } else {
    store_tile<T, S>(acc, (T*)(second ? a.dwu : a.dwg), m0, a.F, n0, a.C, vec);
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

bool on16(const void* p) { return ((size_t)p & 15) == 0; }

int tiles_of(long long n, int bf16) {
  const int kt = bf16 ? kTileK<__bf16> : kTileK<float>;
  return (int)((n + kt - 1) / kt);
}
Cut dx_cut(long long R, int C, int F, int bf16) { return cut_of(R, C, 2 * tiles_of(F, bf16)); }
Cut dw_cut(long long R, int C, int F, int bf16) {
  return cut_of(2LL * F, C, tiles_of(R, bf16));
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }
size_t half_bytes(long long R, int F, int bf16) { return round256((size_t)R * F * (bf16 ? 2 : 4)); }

template <typename T, class S, bool DIRECT>
int run_dx(const FfnArgs& a, const T* dg, const T* du, float* parts, int splits, hipStream_t s) {
  const int nt = 2 * tiles_of(a.F, a.bf16), per = (nt + splits - 1) / splits;
  const long long tm = (a.R + S::BM - 1) / S::BM, tn = (a.C + S::BN - 1) / S::BN;
  if (!grid_ok(tm * tn * splits, S::NT)) return -1;
  const int vec = a.C % 4 == 0 && on16(a.dx);
  const int tk = ktimer_before(s, "ffn_dx");
  hipLaunchKernelGGL((ffn_dx_kernel<T, S, DIRECT>), dim3((unsigned)(tm * tn * splits)),
                     dim3(S::NT), 0, s, a, dg, du, parts, (int)tm, (int)tn, splits, per, vec);
  ktimer_after(s, tk);
  const int rc = (int)hipGetLastError();
  if (rc || splits == 1) return rc;
  return launch_ffn_sum(parts, splits, a.R * a.C, a.dx, a.bf16, s);
}

template <typename T, class S, bool DIRECT>
int run_dw(const FfnArgs& a, const T* dg, const T* du, float* parts, int splits, hipStream_t s) {
  const int nt = tiles_of(a.R, a.bf16), per = (nt + splits - 1) / splits;
  const long long tm = (a.F + S::BM - 1) / S::BM, tn = (a.C + S::BN - 1) / S::BN;
  if (!grid_ok(2 * tm * tn * splits, S::NT)) return -1;
  const int vec = a.C % 4 == 0 && on16(a.dwg) && on16(a.dwu);
  const int tk = ktimer_before(s, "ffn_dw");
  hipLaunchKernelGGL((ffn_dw_kernel<T, S, DIRECT>), dim3((unsigned)(2 * tm * tn * splits)),
                     dim3(S::NT), 0, s, a, dg, du, parts, (int)tm, (int)tn, splits, per, vec);
  ktimer_after(s, tk);
  int rc = (int)hipGetLastError();
  if (rc || splits == 1) return rc;
  const long long n = (long long)a.F * a.C;
  rc = launch_ffn_sum(parts, splits, n, a.dwg, a.bf16, s);
  return rc ? rc : launch_ffn_sum(parts + splits * n, splits, n, a.dwu, a.bf16, s);
}

template <typename T, class S>
int run_dx_s(const FfnArgs& a, const T* dg, const T* du, float* parts, int splits, hipStream_t s) {
  constexpr int U = kUnit<T>;
  const bool direct = on16(a.wg) && on16(a.wu) && a.C % U == 0 && a.F % U == 0;
  return direct ? run_dx<T, S, true>(a, dg, du, parts, splits, s)
                : run_dx<T, S, false>(a, dg, du, parts, splits, s);
}
template <typename T, class S>
int run_dw_s(const FfnArgs& a, const T* dg, const T* du, float* parts, int splits, hipStream_t s) {
  constexpr int U = kUnit<T>;
  const bool direct = on16(a.x) && a.xs % U == 0 && a.C % U == 0 && a.F % U == 0;
  return direct ? run_dw<T, S, true>(a, dg, du, parts, splits, s)
                : run_dw<T, S, false>(a, dg, du, parts, splits, s);
}

template <typename T>
int run(const FfnArgs& a, hipStream_t s) {
  const size_t half = half_bytes(a.R, a.F, a.bf16);
  T *dg = (T*)a.ws, *du = (T*)((char*)a.ws + half);
  float* parts = (float*)((char*)a.ws + 2 * half);
  const long long n = a.R * a.F;
  int rc = 0;
  if (n > 0) {
    const long long wgs = (n + 2047) / 2048;
    if (!grid_ok(wgs, 256)) return -1;
    const int tk = ktimer_before(s, "ffn_grad");
    hipLaunchKernelGGL((ffn_grad_kernel<T>), dim3((unsigned)wgs), dim3(256), 0, s, a, n, dg, du);
    ktimer_after(s, tk);
    rc = (int)hipGetLastError();
    if (rc) return rc;
  }
  if (a.R > 0) {
    const Cut c = dx_cut(a.R, a.C, a.F, a.bf16);
    rc = c.shape == 0   ? run_dx_s<T, Large>(a, dg, du, parts, c.splits, s)
         : c.shape == 1 ? run_dx_s<T, Middle>(a, dg, du, parts, c.splits, s)
                        : run_dx_s<T, Small>(a, dg, du, parts, c.splits, s);
    if (rc) return rc;
  }
  if (a.F == 0) return 0;
  const Cut c = dw_cut(a.R, a.C, a.F, a.bf16);
  return c.shape == 0   ? run_dw_s<T, Large>(a, dg, du, parts, c.splits, s)
         : c.shape == 1 ? run_dw_s<T, Middle>(a, dg, du, parts, c.splits, s)
                        : run_dw_s<T, Small>(a, dg, du, parts, c.splits, s);
}

}  // namespace
}  // namespace ffn

size_t ffn_backward_ws(long long R, int C, int F, int bf16) {
  const ffn::Cut x = ffn::dx_cut(R, C, F, bf16), w = ffn::dw_cut(R, C, F, bf16);
  const size_t px = x.splits > 1 ? (size_t)x.splits * R * C * sizeof(float) : 0;
  const size_t pw = w.splits > 1 ? (size_t)w.splits * 2 * F * C * sizeof(float) : 0;
  return 2 * ffn::half_bytes(R, F, bf16) + (px > pw ? px : pw);
}

int launch_ffn_backward(const FfnArgs& a, hipStream_t s) {
  return a.bf16 ? ffn::run<__bf16>(a, s) : ffn::run<float>(a, s);
}

}  // namespace osdn
