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

namespace osdn {
namespace ffn {
namespace {

// Rows of x by rows of both weights, all K-major. The wave's first half of column tiles
// is of the gate, the second of the other; two column tiles of 16 take their columns in
// turns of four, so that a lane's results are eight consecutive ones.
template <typename T, class S>
struct Forward {
  typedef Stage<T, S::BM, true, S::NT> StageA;
  typedef Stage<T, S::BN / 2, true, S::NT, true> StageB;
  static constexpr int BF = S::BN / 2, TH = S::TN / 2, HALF = BF * kRowBytes;
  static_assert(TH % 2 == 0, "column tiles in pairs");
  const T *x, *wg, *wu;
  long long m0;
  int f0, rows, cols, full, C;
  long long xs;
  unsigned oa[StageA::PER], ob[StageB::PER];
  uint4 va[StageA::PER], vg[StageB::PER], vu[StageB::PER];

  __device__ __forceinline__ void place(const FfnArgs& a, const Item& it) {
    m0 = (long long)it.m * S::BM;
    f0 = it.n * BF;
    xs = a.xs;
    C = a.C;
    x = (const T*)a.x + m0 * a.xs;
    wg = (const T*)a.wg + (long long)f0 * a.C;
    wu = (const T*)a.wu + (long long)f0 * a.C;
    rows = (int)min((long long)S::BM, a.R - m0);
    cols = min(BF, a.F - f0);
    full = a.C / kTileK<T>;
    StageA::offsets(oa, a.xs, rows);
    StageB::offsets(ob, a.C, cols);
  }
  __device__ __forceinline__ void direct_a(int t, char* a) const {
    StageA::direct(a, x + t * kTileK<T>, oa);
  }
  __device__ __forceinline__ void direct_b(int t, char* b) const {
    const int k = t * kTileK<T>;
    StageB::direct(b, wg + k, ob);
    StageB::direct(b + HALF, wu + k, ob);
  }
  __device__ __forceinline__ void fetch(int t) {
    const int k = t * kTileK<T>;
    StageA::fetch(va, x + k, xs, rows, C - k);
    StageB::fetch(vg, wg + k, C, cols, C - k);
    StageB::fetch(vu, wu + k, C, cols, C - k);
  }
  __device__ __forceinline__ void put(char* a, char* b) const {
    StageA::put(a, va);
    StageB::put(b, vg);
    StageB::put(b + HALF, vu);
  }
  // Column tile j: the first row of its run of fours within the wave's columns.
  __device__ __forceinline__ static int column(int wave, int j) {
    return wave % S::WN * (16 * TH) + 32 * (j / 2) + 4 * (j % 2);
  }
  __device__ __forceinline__ uint4 fragb(const char* lb, int j, int step) const {
    return StageB::frag(j < TH ? lb : lb + HALF, column(wave_id(), j % TH), step);
  }
  static __device__ __forceinline__ bool vectors(const FfnArgs& a) {
    constexpr int E = 8;
    return a.F % E == 0 && (((size_t)a.h | (size_t)a.gate | (size_t)a.up) & 15) == 0;
  }
  __device__ __forceinline__ void store_row(const FfnArgs& a, int i,
                                            const f32x4 (&row)[S::TN]) const {
    // (the branch around whole rows: one for every element costs as much as its work)
    switch (a.act) {
      case OSDN_ACT_SILU: return store_row<OSDN_ACT_SILU>(a, i, row);
      case OSDN_ACT_GELU: return store_row<OSDN_ACT_GELU>(a, i, row);
      default: return store_row<OSDN_ACT_GELU_TANH>(a, i, row);
    }
  }
  template <int ACT>
  __device__ __forceinline__ void store_row(const FfnArgs& a, int i,
                                            const f32x4 (&row)[S::TN]) const {
    const int thread = fresh_thread(), lane = thread & 63, wave = wave_of(thread);
    const long long m = m0 + wave / S::WN * (S::BM / S::WM) + 16 * i + (lane & 15);
    if (m >= a.R) return;
    const bool vec = vectors(a);
#pragma unroll
    for (int j = 0; j < TH; j += 2) {
      const int f = f0 + column(wave, j) + 8 * (lane >> 4);
      float x[8], u[8], h[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = row[j + k / 4][k % 4];
        u[k] = row[TH + j + k / 4][k % 4];
        h[k] = activated<ACT>(x[k]) * u[k];
      }
      const long long to = m * a.F + f;
      store8((T*)a.h + to, h, a.F - f, vec);
      if (a.gate) {
        store8((T*)a.gate + to, x, a.F - f, vec);
        store8((T*)a.up + to, u, a.F - f, vec);
      }
    }
  }
};

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

template <typename T, class S>
int run_shape(const FfnArgs& a, const Plan& p, hipStream_t s) {
  const size_t es = sizeof(T);
  const bool direct = on16(a.x) && on16(a.wg) && on16(a.wu) && a.xs * es % 16 == 0 &&
                      a.C * es % 16 == 0;
  return launch_products<T, S, Forward<T, S>>(a, p, direct, "ffn", "ffn_join", s);
}

bool forward_plan(Plan& p, long long R, int C, int F, int bf16) {
  return make_plan(p, 1, R, 2LL * F, C, bf16, C % (bf16 ? 8 : 4) == 0);
}

template <typename T>
int run(const FfnArgs& a, hipStream_t s) {
  if (a.R <= 16) return run_rows<T, 1>(a, s);
  if (a.R <= 32) return run_rows<T, 2>(a, s);
  if (a.R <= kFewRows) return run_rows<T, 4>(a, s);
  Plan p;
  if (!forward_plan(p, a.R, a.C, a.F, a.bf16)) return -1;
  FfnArgs b = a;
  b.parts = (float*)a.ws;
  switch (p.shape) {
    case 0: return run_shape<T, Large>(b, p, s);
    case 1: return run_shape<T, Middle>(b, p, s);
  }
  return run_shape<T, SmallPairs>(b, p, s);
}

}  // namespace

// What a tile of k costs a workgroup that has a CU to itself or shares it with as many
// as fit, in microseconds, by shape: bf16 is bound by operands from L2 and LDS, the more
// the smaller the tile; fp32 by the matrix units.
bool make_plan(Plan& best, int sets, long long M, long long N, long long K, int bf16,
               bool direct) {
  const int bm[] = {256, 128, 64}, kt = bf16 ? kTileK<__bf16> : kTileK<float>;
  const int at_once[] = {1, 2, 4};
  const double cost[2][3] = {{7.0, 1.75, 0.45}, {1.46, 0.5, 0.2}};
  const long long nt = K > 0 ? (K + kt - 1) / kt : 1;
  double least = 1e300;
  if (nt > (1 << 26)) return false;
  for (int k = direct ? 0 : 1; k < 3; ++k) {
    const long long tm = sets * ((M + bm[k] - 1) / bm[k]), tn = (N + bm[k] - 1) / bm[k];
    const long long tiles = tm * tn, full = 256 * at_once[k];
    if (!grid_ok(16 * tiles, 512)) continue;
    const long long whole = tiles / full * full, rest = tiles - whole;
    for (int s = 1; s <= 16 && (s == 1 || (rest > 0 && nt / s >= 4)); ++s) {
      const long long per = (nt + s - 1) / s;
      if ((nt + per - 1) / per != s) continue;     // (no empty part)
      // a round costs its tiles of k and the start and end of a tile; one of fewer
      // workgroups than CUs runs each of them alone
      const double each = bf16 ? 8 : 2, wgs = (double)(rest * s);
      const double last = wgs <= 256 ? (wgs > 0) : at_once[k] * (double)((rest * s + full - 1) / full);
      double t = cost[bf16][k] * (at_once[k] * (double)(whole / full) * (nt + each) +
                                  last * (per + each));
      // parts written and read, and the launch that adds them
      if (s > 1) t += 5 + wgs * bm[k] * bm[k] * 8 / 4e6;
      if (t < least) {
        least = t;
        best = Plan{k, (int)tm, (int)tn, (int)nt, (int)whole, s, (int)per};
      }
    }
  }
  return least < 1e300;
}

size_t parts_bytes(const Plan& p) {
  const int b[] = {256, 128, 64};
  return p.splits > 1 ? (size_t)p.rest() * p.splits * b[p.shape] * b[p.shape] * sizeof(float) : 0;
}

}  // namespace ffn

size_t ffn_forward_ws(long long R, int C, int F, int bf16) {
  if (R <= ffn::kFewRows) return 0;
  ffn::Plan p;
  return F > 0 && ffn::forward_plan(p, R, C, F, bf16) ? ffn::parts_bytes(p) : 0;
}

int launch_ffn_forward(const FfnArgs& a, hipStream_t s) {
  return a.bf16 ? ffn::run<__bf16>(a, s) : ffn::run<float>(a, s);
}

}  // namespace osdn
