// Gated feed-forward product, backward, from the stored g and u:
//   dg = dh u act'(g),  du = dh act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
// A first kernel forms dg and du (5 elements moved for one of dh, bound by HBM: 76 us for
// 461 MB, 6.1 TB/s) in the operands' type, the two products are tiles on the matrix units:
// dx over both halves of 2 F (8192 x 2048 x 5632 bf16: 300 us, 1260 TFLOP/s), the weights'
// gradients over the rows (325 us and 16 of joining parts, 1110). dg and du are rounded
// once in bf16 (2^-9 of each term on average, as the results' own rounding is): held in
// two parts they would double the matrix work. Where both products leave the card half
// empty they run in one launch (333 x 509 x 1366 fp32: 18 + 8 + 21 us in turn, 32 + 6
// together).
#include "ffn_common.hpp"

namespace osdn {
namespace ffn {
namespace {

// dg and du in rows of Fp elements, zeros behind F; behind the first n workgroups the
// copies of operands off 16 bytes.
template <typename T>
__global__ __launch_bounds__(256) void ffn_grad_kernel(FfnArgs a, Pads p, unsigned n) {
  if (blockIdx.x >= n) return pad_group<T>(p, (blockIdx.x - n) * 256LL + threadIdx.x);
  const long long at = (blockIdx.x * 256LL + threadIdx.x) * 8;
  if (at >= a.R * a.Fp) return;
  long long from = at;
  int m = 8;
  if (a.Fp != a.F) {
    const long long r = at / a.Fp;
    const int f = (int)(at % a.Fp);
    from = r * a.F + f;
    m = min(8, a.F - f);
  }
  float g[8], u[8], d[8];
  load_v<false, 8>((const T*)a.gate + from, m, g);
  load_v<false, 8>((const T*)a.up + from, m, u);
  load_v<false, 8>((const T*)a.dh + from, m, d);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f, s;
    activated(g[i], a.act, f, s);
    g[i] = d[i] * u[i] * s;
    u[i] = d[i] * f;
  }
  store_v<true, 8>((T*)a.dg + at, 8, g);
  store_v<true, 8>((T*)a.du + at, 8, u);
}

// A wave's i-th 16 rows, from m0 on of M, to columns from n0 on of N.
template <typename T, class S>
__device__ __forceinline__ void store_columns(T* out, int i, long long m0, long long M, int n0,
                                              int N, const f32x4 (&row)[S::TN]) {
  const int thread = fresh_thread(), lane = thread & 63, wave = wave_of(thread);
  const long long m = m0 + wave / S::WN * (S::BM / S::WM) + 16 * i + (lane & 15);
  if (m >= M) return;
  const bool vec = N % 4 == 0 && ((size_t)out & 15) == 0;
#pragma unroll
  for (int j = 0; j < S::TN; ++j) {
    const int n = n0 + wave % S::WN * (S::BN / S::WN) + 16 * j + 4 * (lane >> 4);
    store4(out + m * N + n, row[j], N - n, vec);
  }
}

// dx: rows of dg and du (K-major over f) by the weights' columns (f along k). Tiles of
// k: the whole ones of dg, those of du, then the two ends.
template <typename T, class S>
struct Input {
  typedef Stage<T, S::BM, true, S::NT> StageA;
  typedef Stage<T, S::BN, false, S::NT> StageB;
  const T *dg, *du, *wg, *wu;
  long long m0;
  int n0, C, F, Fp, rows, cols, full;
  unsigned oa[StageA::PER], ob[StageB::PER];
  uint4 va[StageA::PER], vb[StageB::PER];

  __device__ __forceinline__ void place(const FfnArgs& a, const Item& it) {
    m0 = (long long)it.m * S::BM;
    n0 = it.n * S::BN;
    C = a.Cp;
    F = a.F;
    Fp = a.Fp;
    dg = (const T*)a.dg + m0 * Fp;
    du = (const T*)a.du + m0 * Fp;
    wg = (const T*)a.wg + n0;
    wu = (const T*)a.wu + n0;
    rows = (int)min((long long)S::BM, a.R - m0);
    cols = min(S::BN, C - n0);
    full = 2 * (a.F / kTileK<T>);
    StageA::offsets(oa, Fp, rows);
    StageB::offsets(ob, C, cols);
  }
  __device__ __forceinline__ int along(int t, bool& second) const {
    const int half = full / 2;
    second = t < full ? t >= half : t > full;
    return (t < full ? t - (second ? half : 0) : half) * kTileK<T>;
  }
  __device__ __forceinline__ void direct_a(int t, char* a) const {
    bool second;
    const int k = along(t, second);
    StageA::direct(a, (second ? du : dg) + k, oa);
  }
  __device__ __forceinline__ void direct_b(int t, char* b) const {
    bool second;
    const int k = along(t, second);
    StageB::direct(b, (second ? wu : wg) + (long long)k * C, ob);
  }
  __device__ __forceinline__ void fetch(int t) {
    bool second;
    const int k = along(t, second);
    StageA::fetch(va, (second ? du : dg) + k, Fp, rows, F - k);
    StageB::fetch(vb, (second ? wu : wg) + (long long)k * C, C, cols, F - k);
  }
  __device__ __forceinline__ void put(char* a, char* b) const {
    StageA::put(a, va);
    StageB::put(b, vb);
  }
  __device__ __forceinline__ uint4 fragb(const char* lb, int j, int step) const {
    return StageB::frag(lb, wave_id() % S::WN * (S::BN / S::WN) + 16 * j, step);
  }
  __device__ __forceinline__ void store_row(const FfnArgs& a, int i,
                                            const f32x4 (&row)[S::TN]) const {
    store_columns<T, S>((T*)a.dx, i, m0, a.R, n0, a.C, row);
  }
};

// The weights' gradients: columns of dg or du by columns of x, rows along k. Tiles of m:
// first those of the gate's gradient, then those of the other.
template <typename T, class S>
struct Weight {
  typedef Stage<T, S::BM, false, S::NT> StageA;
  typedef Stage<T, S::BN, false, S::NT> StageB;
  const T *d, *x;
  T* out;
  long long R, xs;
  int m0, n0, F, rows, cols, full;
  unsigned oa[StageA::PER], ob[StageB::PER];
  uint4 va[StageA::PER], vb[StageB::PER];

  __device__ __forceinline__ void place(const FfnArgs& a, const Item& it) {
    const int tm = (a.F + S::BM - 1) / S::BM;
    const bool second = it.m >= tm;
    m0 = (it.m - (second ? tm : 0)) * S::BM;
    n0 = it.n * S::BN;
    F = a.Fp;
    R = a.R;
    xs = a.xs;
    full = (int)(a.R / kTileK<T>);
    d = (const T*)(second ? a.du : a.dg) + m0;
    x = (const T*)a.x + n0;
    out = (T*)(second ? a.dwu : a.dwg);
    rows = min(S::BM, F - m0);
    cols = min(S::BN, a.Cp - n0);
    StageA::offsets(oa, F, rows);
    StageB::offsets(ob, a.xs, cols);
  }
  __device__ __forceinline__ void direct_a(int t, char* a) const {
    StageA::direct(a, d + (long long)t * kTileK<T> * F, oa);
  }
  __device__ __forceinline__ void direct_b(int t, char* b) const {
    StageB::direct(b, x + (long long)t * kTileK<T> * xs, ob);
  }
  __device__ __forceinline__ void fetch(int t) {
    const long long k = (long long)t * kTileK<T>;
    const int nk = (int)min(R - k, (long long)kTileK<T>);
    StageA::fetch(va, d + k * F, F, rows, nk);
    StageB::fetch(vb, x + k * xs, xs, cols, nk);
  }
  __device__ __forceinline__ void put(char* a, char* b) const {
    StageA::put(a, va);
    StageB::put(b, vb);
  }
  __device__ __forceinline__ uint4 fragb(const char* lb, int j, int step) const {
    return StageB::frag(lb, wave_id() % S::WN * (S::BN / S::WN) + 16 * j, step);
  }
  __device__ __forceinline__ void store_row(const FfnArgs& a, int i,
                                            const f32x4 (&row)[S::TN]) const {
    store_columns<T, S>(out, i, m0, a.F, n0, a.C, row);
  }
};

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

// How both products are cut. pair: in one launch.
struct Plans {
  Plan x, w;
  bool pair;
  size_t parts() const {
    const size_t px = parts_bytes(x), pw = parts_bytes(w);
    return pair ? px + pw : px > pw ? px : pw;
  }
};
bool make_plans(Plans& p, long long R, int C, int F, int bf16) {
  p = Plans{};
  const long long kt = bf16 ? kTileK<__bf16> : kTileK<float>;
  // (tiles of k of dx: whole ones of each half, then the ends)
  const long long x[3] = {R, C, 2 * ((F + kt - 1) / kt) * kt}, w[3] = {F, C, R};
  double tx = 0.0, tw = 0.0;
  if (C == 0) return true;
  if (R > 0 && !make_plan(p.x, kOne, x[0], x[1], x[2], bf16, &tx)) return false;
  if (F > 0 && !make_plan(p.w, kTwo, w[0], w[1], w[2], bf16, &tw)) return false;
  if (R > 0 && F > 0) p.pair = make_pair(p.x, p.w, x, w, bf16, tx + tw + kLaunch);
  return true;
}

size_t half_bytes(long long R, int F, int bf16) {
  return round256((size_t)R * whole_eights(F) * (bf16 ? 2 : 4));
}

enum What { kDx, kDw, kBoth };
template <typename T, class S>
int run_shape(const FfnArgs& a, const Plans& p, What what, hipStream_t s) {
  typedef Input<T, S> X;
  typedef Weight<T, S> W;
  if (what == kBoth)
    return launch_pair<T, S, X, W>(a, p.x, p.w, "ffn_dxdw", "ffn_dxdw_join", s);
  return what == kDx ? launch_products<T, S, X>(a, p.x, "ffn_dx", "ffn_dx_join", s)
                     : launch_products<T, S, W>(a, p.w, "ffn_dw", "ffn_dw_join", s);
}

template <typename T>
int run_plan(const FfnArgs& a, const Plans& p, What what, hipStream_t s) {
  const int shape = what == kDw ? p.w.shape : p.x.shape;
  if constexpr (sizeof(T) == 2)
    if (shape == 0) return run_shape<T, Large>(a, p, what, s);
  if (shape == 1) return run_shape<T, Middle>(a, p, what, s);
  return run_shape<T, Small>(a, p, what, s);
}

template <typename T>
int run(const FfnArgs& a0, hipStream_t s) {
  FfnArgs a = a0;
  const size_t half = half_bytes(a.R, a.F, a.bf16);
  a.dg = a.ws;
  a.du = (char*)a.ws + half;
  char* room = (char*)a.ws + 2 * half;
  Plans p;
  const long long wgs = (a.R * whole_eights(a.F) + 2047) / 2048;
  const Pads pads = align_operands(a, room);
  const long long copies = (pads.end[2] + 255) / 256;
  if (!make_plans(p, a.R, a.C, a.F, a.bf16) || !grid_ok(wgs + copies, 256)) return -1;
  a.parts = (float*)(room + aligned_bytes(a.R, a.C, a.F, a.bf16));
  int rc = 0;
  if (wgs + copies > 0) {
    const int tk = ktimer_before(s, "ffn_grad");
    hipLaunchKernelGGL((ffn_grad_kernel<T>), dim3((unsigned)(wgs + copies)), dim3(256), 0, s, a,
                       pads, (unsigned)wgs);
    ktimer_after(s, tk);
    rc = (int)hipGetLastError();
  }
  if (!rc && p.pair) return run_plan<T>(a, p, kBoth, s);
  if (!rc && a.R > 0) rc = run_plan<T>(a, p, kDx, s);
  if (!rc && a.F > 0) rc = run_plan<T>(a, p, kDw, s);
  return rc;
}

}  // namespace
}  // namespace ffn

size_t ffn_backward_ws(long long R, int C, int F, int bf16) {
  ffn::Plans p;
  const size_t parts = ffn::make_plans(p, R, C, F, bf16) ? p.parts() : 0;
  return 2 * ffn::half_bytes(R, F, bf16) + ffn::aligned_bytes(R, C, F, bf16) + parts;
}

int launch_ffn_backward(const FfnArgs& a, hipStream_t s) {
  return a.bf16 ? ffn::run<__bf16>(a, s) : ffn::run<float>(a, s);
}

}  // namespace osdn
