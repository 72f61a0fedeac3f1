// Gated feed-forward product, forward: g = x Wg^T, u = x Wu^T, h = act(g) u, in one
// kernel: a workgroup's tile holds the same columns of g and u, so that the
// activation and the product are taken from the accumulators in 32 bits and only
// h (and, where a backward pass is to follow, g and u) are rounded and stored.
//
// Bound by the matrix units where there are many rows; by the weights' bytes for a
// few (up to 64), which have a kernel of their own: 16 columns of both weights a
// workgroup, its eight waves taking tiles of k in turn straight from memory into
// registers, their sums joined in LDS.
#include "ffn_common.hpp"
#include "launch.hpp"

namespace osdn {
namespace ffn {
namespace {

// Rows of x by rows of both weights, all K-major.
template <typename T, class S>
struct ForwardSrc {
  typedef Stage<T, S::BM, true, S::NT> SA;
  typedef Stage<T, S::BN / 2, true, S::NT> StageB;
  static constexpr int HALF = S::BN / 2 * kRowBytes;
  const T *x, *wg, *wu;
  long long xs;
  int C, rows, cols, full;    // rows of x and of each weight from the tile on
  unsigned oa[SA::PER], ob[StageB::PER];
  uint4 va[SA::PER], vg[StageB::PER], vu[StageB::PER];

  __device__ __forceinline__ void direct_a(int t, char* a) const {
    SA::direct(a, x + t * kTileK<T>, oa);
  }
  __device__ __forceinline__ void direct_b(int t, char* b) const {
    const int k = t * kTileK<T>;
    StageB::direct(b, wg + k, ob);
    StageB::direct(b + HALF, wu + k, ob);
  }
  __device__ __forceinline__ void fetch(int t) {
    const int k = t * kTileK<T>;
    SA::fetch(va, x + k, xs, rows, C - k);
    StageB::fetch(vg, wg + k, C, cols, C - k);
    StageB::fetch(vu, wu + k, C, cols, C - k);
  }
  __device__ __forceinline__ void put(char* a, char* b) const {
    SA::put(a, va);
    StageB::put(b, vg);
    StageB::put(b + HALF, vu);
  }
  // gate columns, then up columns of the wave
  __device__ __forceinline__ uint4 fragb(const char* lb, int j, int step) const {
    constexpr int TH = S::TN / 2;
    const int w = wave_id() % S::WN * (16 * TH);
    return StageB::frag(j < TH ? lb : lb + HALF, w + 16 * (j % TH), step);
  }
};

template <typename T, class S, bool DIRECT>
__global__ __launch_bounds__(S::NT) void ffn_kernel(FfnArgs a, int tm, int tn, int splits, int per,
                                                    int vec) {
  constexpr int BF = S::BN / 2, TH = S::TN / 2;
  const TileAt at = tile_at(tm, tn, splits);
  const long long m0 = (long long)at.m * S::BM;
  const int f0 = at.n * BF;
  ForwardSrc<T, S> src;
  src.xs = a.xs;
  src.C = a.C;
  src.x = (const T*)a.x + m0 * a.xs;
  src.wg = (const T*)a.wg + (long long)f0 * a.C;
  src.wu = (const T*)a.wu + (long long)f0 * a.C;
  src.rows = (int)min((long long)S::BM, a.R - m0);
  src.cols = min(BF, a.F - f0);
  src.full = a.C / kTileK<T>;
  if constexpr (DIRECT) {
    decltype(src)::SA::offsets(src.oa, a.xs, src.rows);
    decltype(src)::StageB::offsets(src.ob, a.C, src.cols);
  }
  const int t0 = at.split * per, nt = (a.C + kTileK<T> - 1) / kTileK<T>;
  f32x4 acc[S::TM][S::TN];
  products<T, S, true, DIRECT>(acc, src, t0, min(t0 + per, nt));

  const int l = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  const int wm = wave_id() / S::WN * (S::BM / S::WM), wn = wave_id() % S::WN * (16 * TH);
#pragma unroll
  for (int i = 0; i < S::TM; ++i) {
    const long long m = m0 + wm + 16 * i + l;
    if (m >= a.R) continue;
#pragma unroll
    for (int j = 0; j < TH; ++j) {
      const int f = f0 + wn + 16 * j + 4 * g, n = a.F - f;
      const long long to = m * a.F + f;
      const f32x4 &x = acc[i][j], &u = acc[i][j + TH];
      if (splits > 1) {
        float* p = (float*)a.ws + (long long)at.split * 2 * a.R * a.F;
        store4(p + to, x, n, vec);
        store4(p + a.R * a.F + to, u, n, vec);
        continue;
      }
      f32x4 h;
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = activated(x[k], a.act) * u[k];
      store4((T*)a.h + to, h, n, vec);
      if (a.gate) {
        store4((T*)a.gate + to, x, n, vec);
        store4((T*)a.up + to, u, n, vec);
      }
    }
  }
}

// The activation over sums that were split: part [splits][2][R F].
template <typename T>
__global__ __launch_bounds__(256) void ffn_join_kernel(FfnArgs a, int splits) {
  const long long n = a.R * a.F, at = blockIdx.x * 256LL + threadIdx.x;
  if (at >= n) return;
  float g = 0.f, u = 0.f;
  for (int s = 0; s < splits; ++s) {
    g += ((const float*)a.ws)[(long long)s * 2 * n + at];
    u += ((const float*)a.ws)[((long long)s * 2 + 1) * n + at];
  }
  ((T*)a.h)[at] = from_f32<T>(activated(g, a.act) * u);
  if (a.gate) {
    ((T*)a.gate)[at] = from_f32<T>(g);
    ((T*)a.up)[at] = from_f32<T>(u);
  }
}

// ---------------------------------------------------------------------------
// Few rows: NR fragments of 16 rows.
// ---------------------------------------------------------------------------

constexpr int kRowsWaves = 8;

// The lane's unit of a row of k, elements behind nk as zeros.
template <typename T>
__device__ __forceinline__ uint4 row_unit(const T* p, int nk) {
  uint4 v = uint4{0u, 0u, 0u, 0u};
  if (nk >= kUnit<T>) {
    __builtin_memcpy(&v, p, 16);
  } else if (nk > 0) {
    T t[kUnit<T>];
#pragma unroll
    for (int i = 0; i < kUnit<T>; ++i) t[i] = i < nk ? p[i] : from_f32<T>(0.f);
    __builtin_memcpy(&v, t, 16);
  }
  return v;
}

template <typename T, int NR>
__global__ __launch_bounds__(64 * kRowsWaves) void ffn_rows_kernel(FfnArgs a) {
  __shared__ f32x4 red[kRowsWaves][2][NR][64];
  const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4, w = wave_id();
  const int f0 = blockIdx.x * 16, R = (int)a.R;
  const long long fr = (long long)min(f0 + l, a.F - 1) * a.C;
  const T *wg = (const T*)a.wg + fr, *wu = (const T*)a.wu + fr, *x[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) x[i] = (const T*)a.x + (long long)min(16 * i + l, R - 1) * a.xs;
  f32x4 acc[2][NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) acc[0][i] = acc[1][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int nt = a.C / kTileK<T>;
  auto take = [&](int k, int nk) {
    uint4 fg[2], fu[2], fx[NR][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int o = (4 * s + g) * kUnit<T>;
      fg[s] = row_unit(wg + k + o, nk - o);
      fu[s] = row_unit(wu + k + o, nk - o);
#pragma unroll
      for (int i = 0; i < NR; ++i) fx[i][s] = row_unit(x[i] + k + o, nk - o);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        mma(acc[0][i], fg[s], fx[i][s], T());
        mma(acc[1][i], fu[s], fx[i][s], T());
      }
  };
#pragma unroll 4
  for (int t = w; t < nt; t += kRowsWaves) take(t * kTileK<T>, kTileK<T>);
  if (nt * kTileK<T> < a.C && w == nt % kRowsWaves) take(nt * kTileK<T>, a.C - nt * kTileK<T>);
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    red[w][0][i][lane] = acc[0][i];
    red[w][1][i][lane] = acc[1][i];
  }
  __syncthreads();
  if (w >= NR) return;
  f32x4 x0 = red[0][0][w][lane], u0 = red[0][1][w][lane];
#pragma unroll
  for (int v = 1; v < kRowsWaves; ++v) {
    x0 += red[v][0][w][lane];
    u0 += red[v][1][w][lane];
  }
  const int m = 16 * w + l, f = f0 + 4 * g;
  if (m >= R) return;
  f32x4 h;
#pragma unroll
  for (int k = 0; k < 4; ++k) h[k] = activated(x0[k], a.act) * u0[k];
  const long long to = (long long)m * a.F + f;
  store4((T*)a.h + to, h, a.F - f, false);
  if (a.gate) {
    store4((T*)a.gate + to, x0, a.F - f, false);
    store4((T*)a.up + to, u0, a.F - f, false);
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

constexpr int kFewRows = 64;

bool on16(const void* p) { return ((size_t)p & 15) == 0; }

template <typename T, int NR>
int run_rows(const FfnArgs& a, hipStream_t s) {
  const int tk = ktimer_before(s, "ffn_rows");
  hipLaunchKernelGGL((ffn_rows_kernel<T, NR>), dim3((a.F + 15) / 16), dim3(64 * kRowsWaves), 0, s,
                     a);
  ktimer_after(s, tk);
  return (int)hipGetLastError();
}

template <typename T, class S, bool DIRECT>
int run_tiles(const FfnArgs& a, int splits, hipStream_t s) {
  const int nt = (a.C + kTileK<T> - 1) / kTileK<T>, per = (nt + splits - 1) / splits;
  const long long tm = (a.R + S::BM - 1) / S::BM, tn = (a.F + S::BN / 2 - 1) / (S::BN / 2);
  if (!grid_ok(tm * tn * splits, S::NT)) return -1;
  const int vec = a.F % 4 == 0 && on16(a.h) && on16(a.gate) && on16(a.up);
  int tk = ktimer_before(s, "ffn");
  hipLaunchKernelGGL((ffn_kernel<T, S, DIRECT>), dim3((unsigned)(tm * tn * splits)), dim3(S::NT), 0,
                     s, a, (int)tm, (int)tn, splits, per, vec);
  ktimer_after(s, tk);
  int rc = (int)hipGetLastError();
  if (rc || splits == 1) return rc;
  tk = ktimer_before(s, "ffn_join");
  hipLaunchKernelGGL((ffn_join_kernel<T>), dim3((unsigned)((a.R * a.F + 255) / 256)), dim3(256), 0,
                     s, a, splits);
  ktimer_after(s, tk);
  return (int)hipGetLastError();
}

template <typename T, class S>
int run_shape(const FfnArgs& a, int splits, hipStream_t s) {
  const size_t es = sizeof(T);
  const bool direct = on16(a.x) && on16(a.wg) && on16(a.wu) && a.xs * es % 16 == 0 &&
                      a.C * es % 16 == 0;
  return direct ? run_tiles<T, S, true>(a, splits, s) : run_tiles<T, S, false>(a, splits, s);
}

template <typename T>
int run(const FfnArgs& a, hipStream_t s) {
  if (a.R <= 16) return run_rows<T, 1>(a, s);
  if (a.R <= 32) return run_rows<T, 2>(a, s);
  if (a.R <= kFewRows) return run_rows<T, 4>(a, s);
  const Cut c = cut_of(a.R, 2LL * a.F, (a.C + kTileK<T> - 1) / kTileK<T>);
  switch (c.shape) {
    case 0: return run_shape<T, Large>(a, c.splits, s);
    case 1: return run_shape<T, Middle>(a, c.splits, s);
  }
  return run_shape<T, Small>(a, c.splits, s);
}

}  // namespace

// The share of a CU's rate that a shape reaches, and how many of its workgroups a
// CU holds.
Cut cut_of(long long M, long long N, int nt) {
  const int bm[] = {256, 128, 64}, at_once[] = {1, 2, 4};
  const double rate[] = {1.0, 0.7, 0.4};
  Cut best{2, 1};
  nt = nt < 1 ? 1 : nt;
  double least = 1e300;
  for (int k = 0; k < 3; ++k) {
    const double tiles = (double)((M + bm[k] - 1) / bm[k]) * (double)((N + bm[k] - 1) / bm[k]);
    for (int s = 1; s <= 16 && (s == 1 || nt / s >= 4); ++s) {
      const int per = (nt + s - 1) / s;
      if ((nt + per - 1) / per != s) continue;     // (no empty part)
      // rounds of the workgroups that are there at once, at a whole tile's cost each
      const double wgs = tiles * s, full = 256.0 * at_once[k];
      const double rounds = wgs <= 256 ? 1.0 / at_once[k] : (double)(long long)((wgs + full - 1) / full);
      double t = rounds * at_once[k] * ((double)bm[k] * bm[k] / 65536) / rate[k] * (per + 3);
      // the parts written and read, and the launch that adds them
      if (s > 1) t += 8 + (double)s * (double)M * (double)N * 8 / 5e6 / 1.0;
      if (t < least) {
        least = t;
        best = Cut{k, s};
      }
    }
  }
  return best;
}

namespace {

template <typename T>
__global__ __launch_bounds__(256) void ffn_sum_kernel(const float* part, int splits, long long n,
                                                      T* out) {
  const long long at = blockIdx.x * 256LL + threadIdx.x;
  if (at >= n) return;
  float v = 0.f;
  for (int s = 0; s < splits; ++s) v += part[s * n + at];
  out[at] = from_f32<T>(v);
}

}  // namespace

int launch_ffn_sum(const float* part, int splits, long long n, void* out, int bf16, hipStream_t s) {
  const int tk = ktimer_before(s, "ffn_sum");
  const dim3 grid((unsigned)((n + 255) / 256));
  if (bf16) {
    hipLaunchKernelGGL((ffn_sum_kernel<__bf16>), grid, dim3(256), 0, s, part, splits, n,
                       (__bf16*)out);
  } else {
    hipLaunchKernelGGL((ffn_sum_kernel<float>), grid, dim3(256), 0, s, part, splits, n,
                       (float*)out);
  }
  ktimer_after(s, tk);
  return (int)hipGetLastError();
}

}  // namespace ffn

size_t ffn_forward_ws(long long R, int C, int F, int bf16) {
  if (R <= ffn::kFewRows) return 0;
  const int kt = bf16 ? ffn::kTileK<__bf16> : ffn::kTileK<float>;
  const ffn::Cut c = ffn::cut_of(R, 2LL * F, (C + kt - 1) / kt);
  return c.splits > 1 ? (size_t)c.splits * 2 * R * F * sizeof(float) : 0;
}

int launch_ffn_forward(const FfnArgs& a, hipStream_t s) {
  return a.bf16 ? ffn::run<__bf16>(a, s) : ffn::run<float>(a, s);
}

}  // namespace osdn
