// Selective state space scan, prompts. Per (batch, head), with a_t =
// exp(dt_t A) and the head's group's keys B and queries C:
//   S_t = a_t S_{t-1} + dt_t x_t B_t^T        (P x N)
//   y_t = S_t C_t + D x_t
// in chunks of Q tokens: with L_ij = exp(sum of dt A over (j, i]),
//   y_i = sum_{j<=i} (C_i . B_j) L_ij dt_j x_j + L_i0 S_in C_i + D x_i
//   S_out = L_Q0 S_in + sum_j L_Qj dt_j x_j B_j^T
// as matrix products on MFMA.
//
// One workgroup walks a segment of the chunks of one (batch, head) with the
// state in accumulators: each wave owns 16 or 32 rows p of it (all N columns),
// so that the state never leaves registers between chunks; its tiles, read as
// (row p, k = n) fragments in accumulator order, are the operand of the
// readout without a trip through LDS, 32 columns at a time. Scores are formed once
// a chunk, each wave a share of the token rows, and pass through LDS. The next
// chunk's rows are in flight while one is worked on.
//
// A (batch, head) is cut into segments where B * H alone leaves CUs idle:
// a first pass forms each segment's own contribution to the state (keys and
// values only), a small kernel chains them, and the segments then run at once.
//
// Rounding (bf16 inputs): y is rounded to bf16 once, at the end, and its error is
// that rounding (1.66e-3 relative L2): the state and the scores enter it in two bf16
// parts (16 bits). With the state in one part y is off by 1.70e-3 over long prompts and
// by 2.0e-3 to 2.5e-3 where few tokens follow a state that came in, and the scan takes 7
// us less; with the scores in one part 2.1e-3 to 2.7e-3, 4 us less. The state's own update takes
// dt x L in three bf16 parts (24 bits), and is accumulated in fp32. fp32 inputs use
// fp32 MFMA throughout (Q = 32).
//
// Masked pairs are zeros that the products still take; what is not a number in x is
// taken out before and put back behind (3 us of the scan for finding none).
//
// What bounds it: at B 4, H 16, G 2, T 4096, 128 x 128 bf16 the products, with
// the state's update in three parts and formed twice (by the first pass and by
// the scan), are 73 GFLOP, 63 us at the 1150 TFLOP/s that a large matrix product
// reaches; the kernels take 131 to 134 us (decays 6, first pass 34, chain 10, scan 81
// to 84). The 156 MB of inputs and outputs alone would be 29 us. In the scan the matrix
// units, the VALU (splitting, decays) and LDS are each busy a third of the time,
// one after the other within a chunk, with two waves a SIMD to overlap them.
// Measured beside it, scores and state in one part (67 us): the update in one part
// instead of three 59 us, no readout 36, no update 49; 8 waves of one p tile each 94 us
// (LDS reads twice as often); row strides of 72 or 76 words instead of 68 no change.
#include "launch.hpp"
#include "mixer.hpp"
#include "ssm_common.hpp"

namespace osdn {
namespace {

// Waves of a workgroup, and 16-row tiles p a wave: two at P = 128, where every
// key and query fragment read from LDS then serves two products.
template <int P>
constexpr int scan_waves() { return P / 16 < 4 ? P / 16 : 4; }

template <typename Tin>
constexpr int scan_q() { return sizeof(Tin) == 2 ? 64 : 32; }

// Segments of the T tokens: `len` tokens each (a multiple of the chunk).
struct Segments {
  int n, len;
};

template <int P, int N, typename Tin, bool YOUT>
__global__ __launch_bounds__(64 * scan_waves<P>(), 2) void ssm_scan_kernel(
    SsmArgs a, int nseg, int seglen, const ChunkDecay<scan_q<Tin>()>* decay, float* seg_state,
    float* seg_log) {
  constexpr int Q = scan_q<Tin>(), NW = scan_waves<P>(), NT = 64 * NW, PT = P / 16 / NW;
  constexpr int QT = Q / 16, NTL = N / 16;
  constexpr int LN = N + 16 / sizeof(Tin), LP = P + 16 / sizeof(Tin);
  // scores: IM query tiles a wave, or JH waves a query tile
  constexpr int IM = NW < QT ? QT / NW : 1, JH = NW > QT ? NW / QT : 1, JM = (QT + JH - 1) / JH;
  __shared__ __attribute__((aligned(16))) Tin Bs[Q * LN];
  __shared__ __attribute__((aligned(16))) Tin Cs[YOUT ? Q * LN : 16];
  __shared__ __attribute__((aligned(16))) Tin Xs[Q * LP];
  constexpr int M2 = two_parts<Tin>();  // of the scores
  __shared__ __attribute__((aligned(16))) Tin Ms[YOUT ? M2 * Q * Q : 16];  // fragment order
  __shared__ __attribute__((aligned(16))) ChunkDecay<Q> dec;

  const int lane = threadIdx.x & 63, w = wave_id();
  const int nwg = YOUT ? nseg : nseg - 1;  // the last segment hands nothing on
  const int bh = blockIdx.x / nwg, sg = blockIdx.x % nwg;
  const int b = bh / a.H, h = bh % a.H;
  const int n = ssm_length(a.lengths, b, a.T);
  const float D = a.D ? a.D[h] : 0.f;
  const size_t th = (size_t)bh * a.T;
  const size_t tg = ((size_t)b * a.G + h / (a.H / a.G)) * a.T;
  const Tin* x = (const Tin*)a.x + th * P;
  const Tin* Bm = (const Tin*)a.Bm + tg * N;
  const Tin* Cm = (const Tin*)a.Cm + tg * N;
  Tin* y = (Tin*)a.y + th * P;
  const ChunkDecay<Q>* dc = decay + (size_t)bh * ((a.T + Q - 1) / Q);

  const int t0 = sg * seglen, t1 = min(t0 + seglen, a.T), tn = min(t1, n);

  // S[pt][nt]: rows n = 16 nt + 4 (l / 16) + e of column p = l % 16 of the
  // wave's p tile
  f32x4 S[PT][NTL];
  const int n0 = 4 * (lane >> 4);
  const size_t srow = (size_t)(w * PT * 16 + (lane & 15)) * N + n0;
  const float* in = !YOUT ? nullptr
                    : nseg > 1 ? seg_state + ((size_t)bh * nseg + sg) * P * N
                    : a.S0    ? a.S0 + (size_t)bh * P * N
                              : nullptr;
#pragma unroll
  for (int pt = 0; pt < PT; ++pt)
#pragma unroll
    for (int nt = 0; nt < NTL; ++nt)
      S[pt][nt] = in ? load4(in + srow + 16 * (pt * N + nt)) : f32x4{0.f, 0.f, 0.f, 0.f};
  float logsum = 0.f;

  Stage<Q, N, Tin, NT, LN> fb, fc;
  Stage<Q, P, Tin, NT, LP> fx;
  StageDecay<Q, NT> fd;
  auto fetch = [&](int t) {
    const int valid = tn - t;
    fb.fetch(Bm + (size_t)t * N, valid);
    if (YOUT) fc.fetch(Cm + (size_t)t * N, valid);
    fx.fetch(x + (size_t)t * P, valid);
    fd.fetch(dc + t / Q);
  };
  if (t0 < tn) fetch(t0);
  for (int t = t0; t < tn; t += Q) {
    const int valid = tn - t;
    __syncthreads();
    fb.put(Bs);
    if (YOUT) fc.put(Cs);
    fx.put(Xs);
    fd.put(dec);
    if (t + Q < tn) fetch(t + Q);
    __syncthreads();

    if constexpr (YOUT) {
      // scores: query tile it, key tiles up to the diagonal, shared by JH waves
#pragma unroll
      for (int q = 0; q < IM; ++q) {
        const int it = q * NW + w % QT, jh = NW > QT ? w / QT : 0;
        Frag<N, Tin> cf;
        cf.load(Cs + it * 16 * LN, LN);
#pragma unroll
        for (int m = 0; m < JM; ++m) {
          const int jt = jh + JH * m;
          if (jt >= QT) break;
          f32x4 s = {0.f, 0.f, 0.f, 0.f};
          if (jt <= it) {
            Frag<N, Tin> bf;
            bf.load(Bs + jt * 16 * LN, LN);
            mma(s, bf, cf);
            const f32x4 l = pair_decay(dec, it, jt), dj = tile_steps(dec, jt);
#pragma unroll
            for (int r = 0; r < 4; ++r) s[r] *= l[r] * dj[r];
            if (jt == it) {  // zeros ahead of the query whatever the key holds
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (acc_row(r) > acc_col()) s[r] = 0.f;
            }
          }
          Frag<Q, Tin>::store_acc_kblock(Ms + it * Frag<Q, Tin>::ELEMS, jt, s);
          if constexpr (M2 == 2)
            Frag<Q, Tin>::store_acc_kblock(Ms + Q * Q + it * Frag<Q, Tin>::ELEMS, jt,
                                           rounding_rest(s, Tin()));
        }
      }
      __syncthreads();
    }

    f32x4 acc[QT][PT];
    if constexpr (YOUT) {
      // S C of every query tile, a 32-wide block of n at a time: of the state's two
      // parts only a block's fragments are held
#pragma unroll
      for (int it = 0; it < QT; ++it)
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) acc[it][pt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < N / 32; ++i) {
        Frag<32, Tin> sf[PT][M2];
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) {
          const f32x4 s[2] = {S[pt][2 * i], S[pt][2 * i + 1]};
          frag_from_acc<32>(sf[pt][0], s);
          if constexpr (M2 == 2) {
            const f32x4 r[2] = {rounding_rest(s[0], Tin()), rounding_rest(s[1], Tin())};
            frag_from_acc<32>(sf[pt][1], r);
          }
        }
#pragma unroll
        for (int it = 0; it < QT; ++it) {
          Frag<32, Tin> cf;
          cf.load_perm(Cs + it * 16 * LN + 32 * i, LN);
#pragma unroll
          for (int m = M2 - 1; m >= 0; --m)
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) mma(acc[it][pt], sf[pt][m], cf);
        }
      }
    }
    Frag<Q, Tin> xf[PT];
#pragma unroll
    for (int pt = 0; pt < PT; ++pt) xf[pt].load_kmajor(Xs + (w * PT + pt) * 16, LP);
    if constexpr (YOUT) {
      // an inf or NaN of x would reach earlier tokens as its product with their
      // zero scores: it is left out of the products, and its channel made NaN from
      // its token on
      bool odd = false;
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) odd |= any_strange(xf[pt]);
      if (odd) {
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) drop_strange(xf[pt]);
      }
      const Buffer yb =
          make_buffer(y + (size_t)t * P, (long long)min(t1 - t, Q) * P * (int)sizeof(Tin));
#pragma unroll
      for (int it = 0; it < QT; ++it) {
        Frag<Q, Tin> mf[M2];
#pragma unroll
        for (int m = 0; m < M2; ++m) mf[m].load_global(Ms + m * Q * Q + it * Frag<Q, Tin>::ELEMS);
        const int ti = it * 16 + (lane & 15);
        const float ent = dec.ent[ti];
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) {
          f32x4& o = acc[it][pt];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] *= ent;
#pragma unroll
          for (int m = M2 - 1; m >= 0; --m) mma_upto<Q>(o, xf[pt], mf[m], 16 * (it + 1));
          const int p = (w * PT + pt) * 16 + n0;
          if (odd) {
#pragma unroll 1
            for (int j = 0; j <= ti; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (strange(Xs[j * LP + p + e])) o[e] = NAN;
          }
          const f32x4 xv = load4(Xs + ti * LP + p);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = ti < valid ? o[e] + D * xv[e] : 0.f;
          buffer_store4(yb, ti * P + p, o, Tin());
        }
      }
      if (odd) {  // the state takes them
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) xf[pt].load_kmajor(Xs + (w * PT + pt) * 16, LP);
      }
    }

    const float total = dec.total;
    logsum += dec.logtot;
    Parts<Q, Tin> xw[PT];
#pragma unroll
    for (int pt = 0; pt < PT; ++pt) scale_parts<Q>(xf[pt], dec.wx, xw[pt]);
#pragma unroll
    for (int nt = 0; nt < NTL; ++nt) {
      Frag<Q, Tin> bf;
      bf.load_kmajor(Bs + nt * 16, LN);
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) S[pt][nt][e] *= total;
        mma_parts(S[pt][nt], bf, xw[pt]);
      }
    }
  }

  if constexpr (YOUT) {
    // rows behind the sequence's last chunk
    const int from = tn > t0 ? t0 + (tn - t0 + Q - 1) / Q * Q : t0;
    constexpr int VE = 16 / sizeof(Tin);
    for (int e = threadIdx.x; e < max(t1 - from, 0) * (P / VE); e += NT)
      *reinterpret_cast<uint4*>(y + (size_t)from * P + (size_t)e * VE) = uint4{0u, 0u, 0u, 0u};
  }
  float* out = YOUT ? (a.ST && sg == nseg - 1 ? a.ST + (size_t)bh * P * N : nullptr)
                    : seg_state + ((size_t)bh * nseg + sg + 1) * P * N;
  if (out) {
#pragma unroll
    for (int pt = 0; pt < PT; ++pt)
#pragma unroll
      for (int nt = 0; nt < NTL; ++nt) store4(out + srow + 16 * (pt * N + nt), S[pt][nt]);
    if (!YOUT && threadIdx.x == 0) seg_log[(size_t)bh * (nseg - 1) + sg] = logsum;
  }
}

// The states entering the segments, in place: slot i + 1 holds segment i's
// contribution and becomes the state entering segment i + 1; slot 0 is S0 (a
// copy: the last segment's workgroup may write S_T over S0 before the first
// one's starts).
__global__ __launch_bounds__(256) void ssm_chain_kernel(int PN, int nseg, const float* S0,
                                                        float* state, const float* logd) {
  const int bh = blockIdx.y;
  const int e = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (e >= PN) return;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (S0) s = load4(S0 + (size_t)bh * PN + e);
  float* p = state + (size_t)bh * nseg * PN + e;
  store4(p, s);
  for (int i = 0; i + 1 < nseg; ++i) {
    p += PN;
    const float f = expf(logd[(size_t)bh * (nseg - 1) + i]);
    const f32x4 c = load4(p);
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = f * s[k] + c[k];
    store4(p, s);
  }
}

// Segments: enough to give every CU two workgroups' work (512 of them; 256 or
// 1024 are slower), none shorter than 2 chunks, and none at all if that makes
// fewer than 4: the first pass over all but the last segment and two trips of
// the states then cost more than the shorter walk gives. In 128 x 128 bf16: 192
// (batch, head) pairs of 1024 tokens 75 us whole, 95 us in 3 segments; 128 pairs
// of 2048 tokens 140 us whole, 100 us in 4; 8 pairs of 64 x 128, 512 tokens, 23 us
// in segments of 2 chunks, 29 us of 4.
Segments segments(int B, int H, int T, int Q) {
  const int nch = (T + Q - 1) / Q;
  const long long bh = (long long)B * H;
  long long want = bh > 0 ? (512 + bh - 1) / bh : 1;
  if (want > nch / 2) want = nch / 2;
  if (want < 4) want = 1;
  const int per = nch > 0 ? (int)((nch + want - 1) / want) : 1;
  Segments s;
  s.len = per * Q;
  s.n = nch > 0 ? (nch + per - 1) / per : 1;
  return s;
}

template <int P, int N, typename Tin>
int run_scan(const SsmArgs& a, hipStream_t s) {
  const int BH = a.B * a.H, PN = P * N;
  const Segments g = segments(a.B, a.H, a.T, scan_q<Tin>());
  constexpr int Q = scan_q<Tin>();
  constexpr int NT = 64 * scan_waves<P>();
  const long long chunks = (long long)BH * ((a.T + Q - 1) / Q);
  if (!grid_ok((chunks + 3) / 4, 256) || !grid_ok((long long)BH * g.n, NT)) return -1;
  ChunkDecay<Q>* dc = (ChunkDecay<Q>*)a.ws;
  launch_decay<Q>(a, dc, s);
  float* st = (float*)((char*)a.ws + decay_bytes<Q>(a.B, a.H, a.T));
  float* lg = st + (size_t)BH * g.n * PN;
  if (g.n > 1) {
    int tk = ktimer_before(s, "ssm_state");
    hipLaunchKernelGGL((ssm_scan_kernel<P, N, Tin, false>), dim3((unsigned)(BH * (g.n - 1))),
                       dim3(NT), 0, s, a, g.n, g.len, dc, st, lg);
    ktimer_after(s, tk);
    tk = ktimer_before(s, "ssm_chain");
    hipLaunchKernelGGL(ssm_chain_kernel, dim3((PN / 4 + 255) / 256, BH), dim3(256), 0, s, PN,
                       g.n, a.S0, st, lg);
    ktimer_after(s, tk);
  }
  const int tk = ktimer_before(s, "ssm_scan");
  hipLaunchKernelGGL((ssm_scan_kernel<P, N, Tin, true>), dim3((unsigned)(BH * g.n)),
                     dim3(NT), 0, s, a, g.n, g.len, dc, st, lg);
  ktimer_after(s, tk);
  return (int)hipGetLastError();
}

template <int P, int N>
int run_scan_t(const SsmArgs& a, hipStream_t s) {
  return a.bf16 ? run_scan<P, N, __bf16>(a, s) : run_scan<P, N, float>(a, s);
}

template <int P>
int run_scan_n(const SsmArgs& a, hipStream_t s) {
  switch (a.N) {
    case 32: return run_scan_t<P, 32>(a, s);
    case 64: return run_scan_t<P, 64>(a, s);
    case 128: return run_scan_t<P, 128>(a, s);
  }
  return -1;
}

}  // namespace

size_t ssm_forward_ws(int B, int H, int T, int P, int N, int bf16) {
  const Segments g = segments(B, H, T, bf16 ? scan_q<__bf16>() : scan_q<float>());
  const size_t d = bf16 ? decay_bytes<scan_q<__bf16>()>(B, H, T)
                        : decay_bytes<scan_q<float>()>(B, H, T);
  return d + (g.n > 1 ? (size_t)B * H * g.n * ((size_t)P * N + 1) * sizeof(float) : 0);
}

int launch_ssm_forward(const SsmArgs& a, hipStream_t s) {
  switch (a.P) {
    case 32: return run_scan_n<32>(a, s);
    case 64: return run_scan_n<64>(a, s);
    case 128: return run_scan_n<128>(a, s);
  }
  return -1;
}

}  // namespace osdn
