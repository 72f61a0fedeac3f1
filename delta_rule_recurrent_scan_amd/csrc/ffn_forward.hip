// Gated feed-forward product, forward: g = x Wg^T, u = x Wu^T, h = act(g) u, in one
// kernel: a workgroup's tile holds the same columns of g and u, so that the
// activation and the product are taken from the accumulators in 32 bits and only
// h (and, where a backward pass is to follow, g and u) are rounded and stored.
//
// Bound by the matrix units where there are many rows: 8192 x 2048 x 5632 bf16 takes 360
// us with g and u kept (1050 TFLOP/s) and 317 without (1190): a tile's results are 3 x 64
// KB that its CU writes while it multiplies nothing. A few rows (up to 64) have a kernel
// of their own, which streams the weights: 16 columns of both a workgroup, its eight waves
// taking tiles of k in turn straight from memory into registers, their sums joined in LDS.
// 8 rows of the same weights take 13 us for 46 MB, where a copy's rate would be 9: the 352
// workgroups are alike, so that some of the 256 CUs stream two and some one.
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
    C = a.Cp;
    x = (const T*)a.x + m0 * a.xs;
    wg = (const T*)a.wg + (long long)f0 * C;
    wu = (const T*)a.wu + (long long)f0 * C;
    rows = (int)min((long long)S::BM, a.R - m0);
    cols = min(BF, a.F - f0);
    full = C / kTileK<T>;
    StageA::offsets(oa, a.xs, rows);
    StageB::offsets(ob, C, cols);
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

// Rows up to which the weights are streamed. Microseconds of a call among others, with
// weights from memory, by that kernel and by tiles:
//                        16 rows        32 rows        64 rows
//   bf16 1024 x 2816   5.6   10.4     6.4   10.7     8.8   10.8
//        2048 x 5632   16.5  26.8     21.0  27.2     26.0  27.2
//        4096 x 5632   29.4  24.4     37.3  25.3     47.4  26.2
//   fp32 1024 x 2816   8.4   18.1     10.6  18.1     19.5  18.4
//        2048 x 5632   28.3  38.1     36.5  38.7     66.8  38.8
// So it is the faster one up to 32 rows of up to 8 KB, and up to 64 of up to 4 KB; longer
// rows of more than 32 lose by it. (With eight fragments, 128 rows: 2048 x 5632 bf16 43 us
// and tiles 19, the weights in the caches.)
constexpr int kFewRows = 64;

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
  return launch_products<T, S, Forward<T, S>>(a, p, "ffn", "ffn_join", s);
}

bool forward_plan(Plan& p, long long R, int C, int F, int bf16) {
  return make_plan(p, kForwards, R, 2LL * F, whole_eights(C), bf16);
}

template <typename T>
__global__ __launch_bounds__(256) void ffn_pad_kernel(Pads p) {
  pad_group<T>(p, blockIdx.x * 256LL + threadIdx.x);
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
  const Pads pads = align_operands(b, (char*)a.ws + round256(parts_bytes(p)));
  const long long wgs = (pads.end[2] + 255) / 256;
  if (!grid_ok(wgs, 256)) return -1;
  if (wgs > 0) {
    const int tk = ktimer_before(s, "ffn_pad");
    hipLaunchKernelGGL((ffn_pad_kernel<T>), dim3((unsigned)wgs), dim3(256), 0, s, pads);
    ktimer_after(s, tk);
    const int rc = (int)hipGetLastError();
    if (rc) return rc;
  }
  if constexpr (sizeof(T) == 2)
    if (p.shape == 0) return run_shape<T, Large>(b, p, s);
  if (p.shape == 1) return run_shape<T, Middle>(b, p, s);
  return run_shape<T, SmallPairs>(b, p, s);
}

}  // namespace

// Microseconds of a tile of k, by shape: of one workgroup that has its CU to itself
// (bound by the way of its operands in bf16, by the matrix units in fp32), and the CU's
// share of each where as many as fit run at once. Measured with one, two and four
// workgroups a CU at 176 tiles of k (bf16) and 128 (fp32).
struct Cost {
  int bm, bn, at_once;
  double alone, share, each;       // each: start and end of a tile
};
// (large fp32 tiles gain nothing: the middle ones have the matrix units busy)
constexpr Cost kBf16[] = {{256, 256, 1, 1.46, 1.46, 8.0}, {128, 128, 2, 0.73, 0.575, 4.0},
                          {64, 64, 4, 0.45, 0.25, 1.0}, {64, 128, 2, 0.55, 0.4, 2.0}};
constexpr Cost kF32[] = {{0, 0, 0, 0, 0, 0}, {128, 128, 2, 2.5, 1.95, 4.0},
                         {64, 64, 4, 0.91, 0.64, 1.0}, {64, 128, 2, 1.2, 1.0, 2.0}};

// A second launch and its parts: written and read, each once.
constexpr double kJoin = 6.5;
double parts_time(long long parts, const Cost& c) { return (double)parts * c.bm * c.bn * 8 / 4e6; }

bool make_plan(Plan& best, Kind kind, long long M, long long N, long long K, int bf16,
               double* microseconds) {
  const int kt = bf16 ? kTileK<__bf16> : kTileK<float>;
  const long long nt = K > 0 ? (K + kt - 1) / kt : 1;
  double least = 1e300;
  if (nt > (1 << 26)) return false;
  for (int k = bf16 ? 0 : 1; k < 3; ++k) {
    const Cost& c = (bf16 ? kBf16 : kF32)[k == 2 && kind == kForwards ? 3 : k];
    const long long tm = (kind == kTwo ? 2 : 1) * ((M + c.bm - 1) / c.bm);
    const long long tn = (N + c.bn - 1) / c.bn, tiles = tm * tn, full = 256 * c.at_once;
    if (!grid_ok(16 * tiles, 512)) continue;
    // workgroups of `len` tiles of k each
    auto time = [&](long long wgs, long long len) {
      const long long a_cu = (wgs + 255) / 256, rem = a_cu % c.at_once;
      const double one = c.at_once * c.share * len + c.each;
      const double last = rem * c.share > c.alone ? rem * c.share : c.alone;
      return (double)(a_cu / c.at_once) * one + (rem ? last * len + c.each : 0.0);
    };
    const long long whole = tiles / full * full, rest = tiles - whole;
    for (int s = 1; s <= 16 && (s == 1 || (rest > 0 && nt / s >= 4)); ++s) {
      const long long per = (nt + s - 1) / s;
      if ((nt + per - 1) / per != s) continue;     // (no empty part)
      double t = time(whole, nt) + time(rest * s, per);
      if (s > 1) t += kJoin + parts_time(rest * s, c);
      if (t < least) {
        least = t;
        best = Plan{k, (int)tm, (int)tn, (int)nt, (int)whole, s, (int)per, c.bm * c.bn, 0};
      }
    }
  }
  if (microseconds) *microseconds = least;
  return least < 1e300;
}

// Two products that leave the card half empty each run side by side: all items of both on
// the card at once, none whole rounds. Its time is that of the longest item alone or of a
// CU's share of all the work, taken as even: items of two lengths dealt in turn are not
// (333 x 509 x 1366 fp32: 192 of 22 tiles of k and 352 of 11, of which the busiest CU has
// 44 and a CU on average 31.6; 44 at 0.64 are 28 of the launch's 30 us).
bool make_pair(Plan& p, Plan& q, const long long (&one)[3], const long long (&two)[3], int bf16,
               double microseconds) {
  const int kt = bf16 ? kTileK<__bf16> : kTileK<float>;
  double least = microseconds;
  const long long n1 = one[2] > 0 ? (one[2] + kt - 1) / kt : 1;
  const long long n2 = two[2] > 0 ? (two[2] + kt - 1) / kt : 1;
  // the parts that n tiles of k may be cut into, and their lengths
  struct Cuts {
    int n = 0, s[16];
    long long per[16];
    explicit Cuts(long long nt) {
      for (int k = 1; k <= 16 && (k == 1 || nt >= 4 * k); ++k) {
        const long long len = (nt + k - 1) / k;
        if (len * (k - 1) >= nt) continue;         // (an empty part)
        s[n] = k;
        per[n++] = len;
      }
    }
  };
  const Cuts u(n1), v(n2);
  for (int k = bf16 ? 0 : 1; k < 3; ++k) {
    const Cost& c = (bf16 ? kBf16 : kF32)[k];
    const long long m1 = (one[0] + c.bm - 1) / c.bm, c1 = (one[1] + c.bn - 1) / c.bn;
    const long long m2 = 2 * ((two[0] + c.bm - 1) / c.bm), c2 = (two[1] + c.bn - 1) / c.bn;
    const long long room = 256 * c.at_once;
    if (m1 * c1 + m2 * c2 > room || m1 * c1 == 0 || m2 * c2 == 0) continue;
    for (int i = 0; i < u.n; ++i)
      for (int j = 0; j < v.n; ++j) {
        const int s1 = u.s[i], s2 = v.s[j];
        const long long per1 = u.per[i], per2 = v.per[j];
        const long long w1 = m1 * c1 * s1, w2 = m2 * c2 * s2;
        if (w1 + w2 > room) break;                 // (more parts are more)
        const long long longest = per1 > per2 ? per1 : per2;
        const double all = c.share * (double)(w1 * per1 + w2 * per2) / 256;
        double t = (longest * c.alone > all ? longest * c.alone : all) + c.each;
        if (s1 > 1 || s2 > 1) t += kJoin;
        if (s1 > 1) t += parts_time(w1, c);
        if (s2 > 1) t += parts_time(w2, c);
        if (t < least) {
          least = t;
          const int area = c.bm * c.bn;
          p = Plan{k, (int)m1, (int)c1, (int)n1, 0, s1, (int)per1, area, 0};
          q = Plan{k, (int)m2, (int)c2, (int)n2, 0, s2, (int)per2, area, 0};
          q.parts_at = (long long)(parts_bytes(p) / sizeof(float));
        }
      }
  }
  return least < microseconds;
}

size_t parts_bytes(const Plan& p) {
  return p.splits > 1 ? (size_t)p.rest() * p.splits * p.area * sizeof(float) : 0;
}

size_t aligned_bytes(long long R, int C, int F, int bf16) {
  const size_t row = (size_t)whole_eights(C) * (bf16 ? 2 : 4);
  return round256(R * row) + (C % 8 ? 2 * round256(F * row) : 0);
}

Pads align_operands(FfnArgs& a, char* room) {
  const size_t es = a.bf16 ? 2 : 4;
  a.Cp = whole_eights(a.C);
  a.Fp = whole_eights(a.F);
  const bool px = a.R > 0 && a.C > 0 && (a.Cp != a.C || !on16(a.x) || a.xs * es % 16 != 0);
  const bool pw = a.Cp != a.C && a.F > 0;
  Pads p{};
  p.C = a.C;
  p.Cp = a.Cp;
  long long end = 0;
  auto take = [&](int k, const void*& in, long long ld, long long rows) {
    p.in[k] = in;
    p.out[k] = room;
    p.ld[k] = ld;
    end += rows * (a.Cp / 8);
    in = room;
    room += round256((size_t)rows * a.Cp * es);
  };
  if (px) {
    take(0, a.x, a.xs, a.R);
    a.xs = a.Cp;
  }
  p.end[0] = end;
  if (pw) take(1, a.wg, a.C, a.F);
  p.end[1] = end;
  if (pw) take(2, a.wu, a.C, a.F);
  p.end[2] = end;
  return p;
}

}  // namespace ffn

size_t ffn_forward_ws(long long R, int C, int F, int bf16) {
  if (R <= ffn::kFewRows) return 0;
  ffn::Plan p;
  if (F == 0 || !ffn::forward_plan(p, R, C, F, bf16)) return 0;
  return ffn::round256(ffn::parts_bytes(p)) + ffn::aligned_bytes(R, C, F, bf16);
}

int launch_ffn_forward(const FfnArgs& a, hipStream_t s) {
  return a.bf16 ? ffn::run<__bf16>(a, s) : ffn::run<float>(a, s);
}

}  // namespace osdn
