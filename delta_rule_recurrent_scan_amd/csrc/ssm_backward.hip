// Backward of the selective state space scan. With the state adjoint
//   dS_t = dy_t C_t^T + a_{t+1} dS_{t+1}        (P x N, from dS_T)
// the gradients of a (batch, head) are
//   dx_t = dt_t dS_t B_t + D dy_t
//   dB_t = dt_t dS_t^T x_t,  dC_t = S_t^T dy_t  (summed over the group's heads)
//   d dt_t = x_t . dS_t B_t + A g_t,  dA = sum dt_t g_t,  dD = sum dy . x
//   g_t = a_t <dS_t, S_{t-1}>                   (of the log decay dt_t A)
// and dS_0 = a_1 dS_1. In chunks of Q tokens, with L_ij the decay from token j
// to i, S the state entering the chunk and dS the adjoint leaving it:
//   K_ij = (C_i . B_j) L_ij dt_j,  Z_ij = (dy_i . x_j) L_ij dt_j      (j <= i)
//   dx_j = sum_i K_ij dy_i + L_Qj dt_j dS B_j + D dy_j
//   dC_i = sum_j Z_ij B_j + L_i0 S^T dy_i
//   dB_j = sum_i Z_ij C_i + L_Qj dt_j dS^T x_j
// g_t is the sum over every pair of a source before t (the entering state, a
// token j < t) and a use at or after it (a token i >= t, the leaving adjoint):
//   g_t = sum_{i>=t>j} (C_i . B_j) Z_ij + sum_{i>=t} w_i + sum_{j<t} u_j
//         + L_Q0 <dS, S>,   w_i = C_i . (L_i0 S^T dy_i),
//                           u_j = B_j . (L_Qj dt_j dS^T x_j)
// of which the last three are sums of one sign of index, and the first, a
// suffix sum of (row - column) sums, stays inside one chunk: nothing grows
// with the sequence and then cancels.
//
// Two kernels. The walk forms S at every chunk's entry and dS at every
// chunk's exit (both directions in one launch, a workgroup a segment of one
// (batch, head), the state in accumulators as in the forward) and writes them
// in fp32 in accumulator order, so that the second kernel's fragments are
// contiguous 16-byte loads. The chunk kernel then takes every chunk at once: a
// workgroup loops over heads of a group, with the group's scores C B^T held
// and dB, dC accumulated in registers, so the sum over heads costs no memory
// and no atomics. The wave's share is a token tile for the scores and dx, and
// tiles of state columns n for dB and dC.
//
// Rounding (bf16 inputs): dS enters dx, and K and Z their products, in two bf16 parts
// (16 bits; one part is 2e-3 of each head's terms, and more of the sums where the
// heads of a group cancel); S, dS and the walks' dt x L enter in three bf16 parts (24
// bits) wherever the result reaches an fp32 output. The errors of dx, dB and dC are
// the results' own rounding. dS in one part left dx 1.9e-3 to 2.0e-3 off where dS makes
// up most of it, and the chunk kernel took 116 us instead of 128: at 128 x 128 both
// parts fit into LDS for one half of P after the other, two barriers a head more.
//
// What bounds it: at B 4, H 16, G 2, T 2048, 128 x 128 bf16 the states are 268 MB,
// written by the walk (92 to 96 us; 4.7 TB/s with the rows it reads) and read by the
// chunk kernel (128 us: one workgroup a CU by its LDS, four barriers a head; LDS and
// VALU each busy two fifths of it, the matrix units a fifth; 44 % of the LDS cycles are
// bank conflicts, 33 % in the walk). The inputs and gradients alone are 123 MB, 23 us.
// Longer chunks would move fewer states, but a chunk's pairs and its rows of four
// tensors fill the LDS at 64. On the way here: states in whole rows of P and 64-bit
// lane addresses spilled registers, and every reload waits for all loads in flight
// (chunk kernel 338 us); a workgroup walking all P rows 106 us, slices of 32 rows 107
// us, of 64 rows 90 us.
#include "launch.hpp"
#include "mixer.hpp"
#include "ssm_common.hpp"

namespace osdn {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;  // of the chunk kernel

template <typename Tin>
constexpr int bwd_q() { return sizeof(Tin) == 2 ? 64 : 32; }

// Where an element of a state lies in accumulator order: tile (p / 16, n / 16)
// of 64 lanes x 4 values, lane (n % 16) + 16 * (p % 16 / 4), value p % 4.
__device__ __forceinline__ void state_elem(int e, int ntl, int& p, int& n) {
  const int tile = e / 256, lane = e % 256 / 4;
  p = tile / ntl * 16 + 4 * (lane / 16) + e % 4;
  n = tile % ntl * 16 + lane % 16;
}

// ---------------------------------------------------------------------------
// The walk. Streams 0 .. BH - 1 run forward (x, B, weights dt L_Qj, from S0),
// BH .. 2 BH - 1 in reverse (dy, C, weights L_i0, from dS_T). Segment k counts
// along the direction.
// ---------------------------------------------------------------------------
// Rows p of the state a workgroup walks (a slice of P: the rows do not meet),
// 16 a wave.
template <int P>
constexpr int walk_rows() { return P < 64 ? P : 64; }

template <int P, int N, typename Tin, bool WRITE>
__global__ __launch_bounds__(4 * walk_rows<P>(), 3) void ssm_walk_kernel(
    SsmArgs a, int nseg, int segch, const ChunkDecay<bwd_q<Tin>()>* decay, float* slots,
    float* slot_log, float* states) {
  constexpr int Q = bwd_q<Tin>(), SP = walk_rows<P>(), NW = SP / 16, NT = 64 * NW;
  constexpr int NTL = N / 16;
  constexpr int LN = N + 16 / sizeof(Tin), LP = SP + 16 / sizeof(Tin);
  __shared__ __attribute__((aligned(16))) Tin Ks[Q * LN];
  __shared__ __attribute__((aligned(16))) Tin Vs[Q * LP];
  __shared__ __attribute__((aligned(16))) ChunkDecay<Q> dec;

  const int lane = threadIdx.x & 63, w = wave_id();
  const int BH = a.B * a.H, nwg = WRITE ? nseg : nseg - 1;
  const int ps = blockIdx.x % (P / SP), id = blockIdx.x / (P / SP);
  const int stream = id / nwg, k = id % nwg;
  const bool rev = stream >= BH;
  const int bh = rev ? stream - BH : stream;
  const int b = bh / a.H, h = bh % a.H, sg = rev ? nseg - 1 - k : k;
  const int n = ssm_length(a.lengths, b, a.T), nch = (a.T + Q - 1) / Q;
  const size_t th = (size_t)bh * a.T;
  const size_t tg = ((size_t)b * a.G + h / (a.H / a.G)) * a.T;
  const Tin* val = (const Tin*)(rev ? a.dy : a.x) + th * P + ps * SP;
  const Tin* key = (const Tin*)(rev ? a.Cm : a.Bm) + tg * N;

  // S[nt]: rows p = 4 (l / 16) + e of the wave's p tile, column n = l % 16
  f32x4 S[NTL];
  const float* from = rev ? a.dST : a.S0;
  const int tile0 = (ps * NW + w) * NTL;
#pragma unroll
  for (int nt = 0; nt < NTL; ++nt) {
    const int at = ((tile0 + nt) * 64 + lane) * 4;
    if (!WRITE || (k == 0 && !from)) {
      S[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    } else if (k > 0) {
      S[nt] = load4(slots + ((size_t)stream * (nseg - 1) + k - 1) * P * N + at);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int p, c;
        state_elem(at + e, NTL, p, c);
        S[nt][e] = from[((size_t)bh * P + p) * N + c];
      }
    }
  }
  float logsum = 0.f;

  const int c0 = sg * segch, c1 = min(c0 + segch, nch);
  const int cn = min(c1, (n + Q - 1) / Q);  // chunks with tokens
  const int count = max(cn - c0, 0);
  auto chunk = [&](int i) { return rev ? cn - 1 - i : c0 + i; };
  // rows two chunks ahead: at one workgroup a CU nothing else hides a fetch
  Stage<Q, N, Tin, NT, LN> fk[2];
  Stage<Q, SP, Tin, NT, LP, P> fv[2];
  StageDecay<Q, NT> fd[2];
  auto fetch = [&](int i, auto& k, auto& v, auto& d) {
    const int t = chunk(i) * Q, valid = n - t;
    k.fetch(key + (size_t)t * N, valid);
    v.fetch(val + (size_t)t * P, valid);
    d.fetch(decay + (size_t)bh * nch + chunk(i));
  };
  auto step = [&](int i, auto& k, auto& v, auto& d) {
    __syncthreads();
    k.put(Ks);
    v.put(Vs);
    d.put(dec);
    if (i + 2 < count) fetch(i + 2, k, v, d);
    if constexpr (WRITE) {
      float* out = states + ((size_t)stream * nch + chunk(i)) * P * N;
#pragma unroll
      for (int nt = 0; nt < NTL; ++nt)
        store4(out + (tile0 + nt) * 256 + (unsigned)(lane * 4), S[nt]);
    }
    __syncthreads();
    const float total = dec.total;
    logsum += dec.logtot;
    Parts<Q, Tin> vw;
    {
      Frag<Q, Tin> vf;
      vf.load_kmajor(Vs + w * 16, LP);
      scale_parts<Q>(vf, rev ? dec.ent : dec.wx, vw);
    }
#pragma unroll
    for (int nt = 0; nt < NTL; ++nt) {
      Frag<Q, Tin> kf;
      kf.load_kmajor(Ks + nt * 16, LN);
#pragma unroll
      for (int e = 0; e < 4; ++e) S[nt][e] *= total;
      mma_parts(S[nt], vw, kf);
    }
  };
  if (count > 0) fetch(0, fk[0], fv[0], fd[0]);
  if (count > 1) fetch(1, fk[1], fv[1], fd[1]);
  for (int i = 0; i < count; i += 2) {
    step(i, fk[0], fv[0], fd[0]);
    if (i + 1 < count) step(i + 1, fk[1], fv[1], fd[1]);
  }

  if constexpr (!WRITE) {
    float* out = slots + ((size_t)stream * (nseg - 1) + k) * P * N;
#pragma unroll
    for (int nt = 0; nt < NTL; ++nt) store4(out + ((tile0 + nt) * 64 + lane) * 4, S[nt]);
    if (threadIdx.x == 0 && ps == 0) slot_log[(size_t)stream * (nseg - 1) + k] = logsum;
  } else if (rev && k == nseg - 1 && a.dS0) {
#pragma unroll
    for (int nt = 0; nt < NTL; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        int p, c;
        state_elem(((tile0 + nt) * 64 + lane) * 4 + e, NTL, p, c);
        a.dS0[((size_t)bh * P + p) * N + c] = S[nt][e];
      }
  }
}

// Segments' contributions (slot k: segment k's own) into the states entering
// segment k + 1, in place, along each stream.
__global__ __launch_bounds__(256) void ssm_walk_chain_kernel(int BH, int PN, int N, int nslots,
                                                             const float* S0, const float* dST,
                                                             float* slots, const float* logd) {
  const int stream = blockIdx.y, e = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (e >= PN) return;
  const bool rev = stream >= BH;
  const float* from = rev ? dST : S0;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (from) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int p, n;
      state_elem(e + i, N / 16, p, n);
      s[i] = from[(size_t)(rev ? stream - BH : stream) * PN + (size_t)p * N + n];
    }
  }
  for (int i = 0; i < nslots; ++i) {
    float* q = slots + ((size_t)stream * nslots + i) * PN + e;
    const float f = expf(logd[(size_t)stream * nslots + i]);
    const f32x4 c = load4(q);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = f * s[j] + c[j];
    store4(q, s);
  }
}

// ---------------------------------------------------------------------------
// The chunk kernel: workgroup (batch, group, chunk, part of the group's heads).
// ---------------------------------------------------------------------------
struct ChunkOut {
  const float* states;  // [2][BH][nch][P N], accumulator order
  float* sums;          // [B nch][3][H]: dA, dD, dbias of a chunk
  float *dBp, *dCp;     // [parts][B G T N] fp32 where the heads are split
  int parts, hper;      // head parts of a group, heads of a part
};

template <int P, int N, typename Tin>
__global__ __launch_bounds__(kThreads, 2) void ssm_bwd_chunk_kernel(
    SsmArgs a, ChunkOut o, const ChunkDecay<bwd_q<Tin>()>* decay) {
  constexpr int Q = bwd_q<Tin>(), QT = Q / 16, NTL = N / 16, PTL = P / 16;
  constexpr int PAD = 16 / sizeof(Tin), LN = N + PAD, LP = P + PAD, LQ = Q + PAD;
  // shares of the waves: state columns (n tile, token tiles tn, tn + TN, ..);
  // scores (query tile, key tiles jh, jh + JH, ..); dx (token tile, p tiles)
  constexpr int TN = kWaves / NTL, JH = kWaves / QT, TM = (QT + TN - 1) / TN,
                JM = (QT + JH - 1) / JH;
  __shared__ __attribute__((aligned(16))) Tin Bs[Q * LN];
  __shared__ __attribute__((aligned(16))) Tin Cs[Q * LN];
  __shared__ __attribute__((aligned(16))) Tin Xs[Q * LP];
  __shared__ __attribute__((aligned(16))) Tin Ys[Q * LP];
  constexpr int M2 = two_parts<Tin>(), QL = Q * LQ;
  __shared__ __attribute__((aligned(16))) Tin Ks[M2 * QL];
  __shared__ __attribute__((aligned(16))) Tin Zs[M2 * QL];
  // dS in its parts, over all of P or (128 x 128, where LDS has no room for both
  // parts of all of it) over one half after the other
  constexpr int NS = M2 == 2 && P * N >= 128 * 128 ? 2 : 1, PS = P / NS, LS = PS + PAD,
                DL = N * LS;
  __shared__ __attribute__((aligned(16))) Tin dSs[M2 * DL];
  __shared__ __attribute__((aligned(16))) ChunkDecay<Q> decs[2];
  // sums of a head, read while the next one is worked on
  struct Sums {
    double row[JH][Q], col[QT][Q];
    float diag[Q], w[NTL][Q], u[NTL][Q], dot[kWaves], dd[kWaves];
  };
  __shared__ Sums acc2[2];

  const int lane = threadIdx.x & 63, w = wave_id(), lc = lane & 15, g4 = 4 * (lane >> 4);
  const int nch = (a.T + Q - 1) / Q, Hg = a.H / a.G;
  int id = blockIdx.x;
  const int part = id % o.parts;
  id /= o.parts;
  const int c = id % nch;
  id /= nch;
  const int g = id % a.G, b = id / a.G;
  const int BH = a.B * a.H, t0 = c * Q;
  const int n = ssm_length(a.lengths, b, a.T), valid = n - t0, rows = min(Q, a.T - t0);
  const int h0 = g * Hg + part * o.hper, h1 = min(h0 + o.hper, (g + 1) * Hg);
  const size_t tg = ((size_t)b * a.G + g) * a.T + t0;
  const size_t GTN = (size_t)a.B * a.G * a.T * N;
  float* sums = o.sums + ((size_t)b * nch + c) * 3 * a.H;

  const int nt = w % NTL, tn = w / NTL, qi = w % QT, jh = w / QT;
  f32x4 dB[TM], dC[TM];  // token tiles tn + TN m
#pragma unroll
  for (int m = 0; m < TM; ++m) dB[m] = dC[m] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (valid > 0) {
    Stage<Q, P, Tin, kThreads, LP> fx, fy;
    StageDecay<Q, kThreads> fd;
    auto fetch = [&](int h) {
      const size_t bh = (size_t)b * a.H + h, th = bh * a.T + t0;
      fx.fetch((const Tin*)a.x + th * P, valid);
      fy.fetch((const Tin*)a.dy + th * P, valid);
    };
    auto fetch_decay = [&](int h) { fd.fetch(decay + ((size_t)b * a.H + h) * nch + c); };
    // the step's gradient of every token, from the sums of head h
    auto finish = [&](int h, int lane, int zero) {
      const Sums& z = acc2[((h - h0) & 1) + zero];
      const ChunkDecay<Q>& dec = decs[((h - h0) & 1) + zero];
      double R = 0., col = 0., wi = 0., uj = 0., own = 0., step = 0.;
      float slope = 0.f;
      if (lane < Q) {
#pragma unroll
        for (int q = 0; q < JH; ++q) R += z.row[q][lane];
#pragma unroll
        for (int q = 0; q < QT; ++q) col += z.col[q][lane];
#pragma unroll
        for (int q = 0; q < NTL; ++q) {
          wi += z.w[q][lane];
          uj += z.u[q][lane];
        }
        step = dec.dt[lane];
        slope = dec.slope[lane];
        own = z.diag[lane] + col + uj;
      }
      double dot = 0.;
      float dd = 0.f;
#pragma unroll
      for (int q = 0; q < kWaves; ++q) {
        if (q < NTL) dot += z.dot[q];
        dd += z.dd[q];
      }
      double gt = wave_suffix_sum(R - col * step + wi) + wave_prefix_before(uj * step) +
                  dec.total * dot;
      // nothing crosses a token whose decay is zero in fp32; the sums' rest of
      // 2^-53 would count where the step that empties the state is 1e20 or more
      if (step * a.A[h] < -104.) gt = 0.;
      const bool in = lane < Q && lane < valid;
      const float draw = in ? (float)((own + a.A[h] * gt) * slope) : 0.f;
      __builtin_amdgcn_raw_buffer_store_b32(
          __float_as_uint(draw),
          make_buffer(a.ddt + ((size_t)b * a.H + h) * a.T + t0, rows * 4), lane * 4, 0, 0);
      const float sa = (float)wave_sum(in ? step * gt : 0.), sb = wave_sum(draw);
      if (lane == 0) {
        sums[h] = sa;
        sums[a.H + h] = dd;
        sums[2 * a.H + h] = sb;
      }
    };
    {
      Stage<Q, N, Tin, kThreads, LN> fb, fc;
      fb.fetch((const Tin*)a.Bm + tg * N, valid);
      fc.fetch((const Tin*)a.Cm + tg * N, valid);
      fetch(h0);
      fetch_decay(h0);
      fb.put(Bs);
      fc.put(Cs);
    }
    __syncthreads();
    // scores of the wave's query tile: rows j = 4 (l / 16) + r, column i = l % 16
    f32x4 CB[JM];
    {
      Frag<N, Tin> cf;
      cf.load(Cs + qi * 16 * LN, LN);
#pragma unroll
      for (int m = 0; m < JM; ++m) {
        const int jt = jh + JH * m;
        CB[m] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (jt <= qi) {
          Frag<N, Tin> bf;
          bf.load(Bs + jt * 16 * LN, LN);
          mma(CB[m], bf, cf);
        }
      }
    }

    // the states of a head over the wave's columns n, in halves of P: the first
    // is in flight from the middle of the head before it, the second while the
    // scores are formed
    constexpr int NH = P >= 64 ? 2 : 1, PH = P / NH, PHL = PH / 16;
    static_assert(NS == 1 || NS == NH, "dS by the halves that are loaded");
    f32x4 sv[NH][PHL], dv[NH][PHL];
    auto load_states = [&](int h, int hf) {
      const float* sf = o.states + (((size_t)b * a.H + h) * nch + c) * P * N;
      const Buffer rf = make_buffer(sf, P * N * 4),
                   rr = make_buffer(sf + (size_t)BH * nch * P * N, P * N * 4);
#pragma unroll
      for (int pb = 0; pb < PHL; ++pb) {
        const unsigned at = (((hf * PHL + pb) * NTL + nt) * 64 + lane) * 16;
        sv[hf][pb] = __builtin_bit_cast(f32x4, buffer_load16(rf, at));
        dv[hf][pb] = __builtin_bit_cast(f32x4, buffer_load16(rr, at));
      }
    };
    load_states(h0, 0);
    for (int h = h0; h < h1; ++h) {
      const size_t bh = (size_t)b * a.H + h, th = bh * a.T + t0;
      const float D = a.D ? a.D[h] : 0.f;
      // an offset of zero that the compiler takes for new in every head: it
      // would otherwise keep some forty LDS addresses across the loop, spill
      // them, and wait for every load in flight to reload one
      int zero = 0, lane_now = threadIdx.x & 63;
      asm volatile("" : "+s"(zero), "+v"(lane_now));
      const int lane = lane_now, lc = lane & 15, g4 = 4 * (lane >> 4);
      Tin *bs = Bs + zero, *cs = Cs + zero, *xs = Xs + zero, *ys = Ys + zero, *ks = Ks + zero,
          *zs = Zs + zero, *ds = dSs + zero;
      const ChunkDecay<Q>& dec = decs[((h - h0) & 1) + zero];
      Sums& z = acc2[((h - h0) & 1) + zero];
      // the previous head's readers of these buffers are behind a barrier
      fx.put(xs);
      fy.put(ys);
      fd.put(decs[((h - h0) & 1) + zero]);
      if constexpr (NH > 1) load_states(h, 1);
      if (h + 1 < h1) fetch(h + 1);
      __syncthreads();

      // scores of dy and x, K and Z, and the pairs' sums (in 64 bits: a token's
      // decay gradient is the difference of rows' and columns' running sums)
      {
        Frag<P, Tin> yf;
        yf.load(ys + qi * 16 * LP, LP);
        double rsum = 0.;
        const int i = qi * 16 + lc;
#pragma unroll
        for (int m = 0; m < JM; ++m) {
          const int jt = jh + JH * m;
          f32x4 kk = {0.f, 0.f, 0.f, 0.f}, zz = {0.f, 0.f, 0.f, 0.f};
          if (jt >= QT) break;
          if (jt <= qi) {
            f32x4 s = {0.f, 0.f, 0.f, 0.f};
            Frag<P, Tin> xf;
            xf.load(xs + jt * 16 * LP, LP);
            mma(s, xf, yf);
            const f32x4 l = pair_decay(dec, qi, jt), dj = tile_steps(dec, jt);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int j = jt * 16 + g4 + r;
              const float zl = s[r] * l[r];
              kk[r] = CB[m][r] * l[r] * dj[r];
              zz[r] = zl * dj[r];
              float v = CB[m][r] * zl;  // the pair without its step
              if (j == i) {
                z.diag[j] = v;  // no decay between: not part of g
                v = 0.f;
              }
              rsum += (double)v * dj[r];
              const double sum = row16_sum((double)v);
              if (lc == 0) z.col[qi][j] = sum;
            }
          } else if (lc == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) z.col[qi][jt * 16 + g4 + r] = 0.f;
          }
          store4_two(ks + i * LQ + jt * 16 + g4, QL, kk);
          store4_two(zs + i * LQ + jt * 16 + g4, QL, zz);
        }
        rsum += __shfl_xor(rsum, 16, 64);
        rsum += __shfl_xor(rsum, 32, 64);
        if (lane < 16) z.row[jh][i] = rsum;
      }
      // what the entering state and the leaving adjoint give to dC and dB, and
      // <dS, S> as a tree over the lane's values (its error is shared by every
      // token of the chunk)
      f32x4 aw[TM], au[TM];
#pragma unroll
      for (int m = 0; m < TM; ++m) aw[m] = au[m] = f32x4{0.f, 0.f, 0.f, 0.f};
      float dot = 0.f;
#pragma unroll
      for (int hf = 0; hf < NH; ++hf) {
        if (tn == 0) {
          float d[PHL];
#pragma unroll
          for (int pb = 0; pb < PHL; ++pb) {
            const f32x4 &u = sv[hf][pb], &v = dv[hf][pb];
            if (NS == 1 || hf == 0)
              store4_two(ds + (nt * 16 + lc) * LS + (hf * PHL + pb) * 16 + g4, DL, v);
            d[pb] = (u[0] * v[0] + u[1] * v[1]) + (u[2] * v[2] + u[3] * v[3]);
          }
#pragma unroll
          for (int m = PHL / 2; m > 0; m /= 2)
#pragma unroll
            for (int pb = 0; pb < m; ++pb) d[pb] += d[pb + m];
          dot += d[0];
        }
        Parts<PH, Tin> sp, dp;
        parts_from_acc<PH>(sp, sv[hf]);
#pragma unroll
        for (int m = 0; m < TM; ++m) {
          const int it = tn + TN * m;
          if (it >= QT) break;
          Frag<PH, Tin> f;
          f.load_perm(ys + it * 16 * LP + hf * PH, LP);
          mma_parts(aw[m], sp, f);
        }
        __builtin_amdgcn_sched_barrier(0);
        parts_from_acc<PH>(dp, dv[hf]);
#pragma unroll
        for (int m = 0; m < TM; ++m) {
          const int it = tn + TN * m;
          if (it >= QT) break;
          Frag<PH, Tin> f;
          f.load_perm(xs + it * 16 * LP + hf * PH, LP);
          mma_parts(au[m], dp, f);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (tn == 0) {
        dot = wave_sum(dot);
        if (lane == 0) z.dot[w] = dot;
      }
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        const int it = tn + TN * m;
        if (it >= QT) break;
        const int i = it * 16 + lc;
        const f32x4 cv = load4(cs + i * LN + nt * 16 + g4), bv = load4(bs + i * LN + nt * 16 + g4);
        const float ent = dec.ent[i], ex = dec.ext[i], dti = dec.dt[i];
        float ws = 0.f, us = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w4 = aw[m][e] * ent, u4 = au[m][e] * ex;
          ws += w4 * cv[e];
          us += u4 * bv[e];
          dC[m][e] += w4;
          dB[m][e] += u4 * dti;
        }
        ws = add_swap32(add_swap16(ws));
        us = add_swap32(add_swap16(us));
        if (lane < 16) {
          z.w[nt][i] = ws;
          z.u[nt][i] = us;
        }
      }
      if (w == kWaves - QT && h > h0) finish(h - 1, lane, zero);  // the least of the scores
      __syncthreads();

      if (h + 1 < h1) {
        fetch_decay(h + 1);
        load_states(h + 1, 0);
      }
      // dB, dC from the chunk's own pairs, over the wave's columns n
      auto own_pairs = [&]() {
        Frag<Q, Tin> bT, cT;  // rows n, k = token
        bT.load_kmajor(bs + nt * 16, LN);
        cT.load_kmajor(cs + nt * 16, LN);
#pragma unroll
        for (int m = 0; m < TM; ++m) {
          const int it = tn + TN * m;
          if (it >= QT) break;
#pragma unroll
          for (int q = M2 - 1; q >= 0; --q) {
            Frag<Q, Tin> zf;
            zf.load(zs + q * QL + it * 16 * LQ, LQ);
            mma(dC[m], bT, zf);
            zf.load_kmajor(zs + q * QL + it * 16, LQ);  // rows j, k = i
            mma(dB[m], cT, zf);
          }
        }
      };

      // dx of token tile qi over the p of dS that lie in LDS, and its share of dD
      float dd = 0.f;
      auto inputs = [&](int s) {
        const int j = qi * 16 + lc;
        Frag<N, Tin> bf;
        bf.load(bs + qi * 16 * LN, LN);
        Frag<Q, Tin> kf[M2];  // rows j, k = i
#pragma unroll
        for (int m = 0; m < M2; ++m) kf[m].load_kmajor(ks + m * QL + qi * 16, LQ);
        const float f = dec.wx[j];
        const Buffer dxb =
            make_buffer((Tin*)a.dx + th * P, (long long)rows * P * (int)sizeof(Tin));
#pragma unroll
        for (int q = 0; q < (PTL / NS + JH - 1) / JH; ++q) {
          const int pl = q * JH + jh, pt = s * (PTL / NS) + pl;
          if (pl >= PTL / NS) break;
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int m = M2 - 1; m >= 0; --m) {
            Frag<N, Tin> df;
            df.load_kmajor(ds + m * DL + pl * 16, LS);  // rows p, k = n
            mma(acc, df, bf);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] *= f;
          Frag<Q, Tin> yT;
          yT.load_kmajor(ys + pt * 16, LP);  // rows p, k = i
#pragma unroll
          for (int m = M2 - 1; m >= 0; --m) mma(acc, yT, kf[m]);
          const f32x4 yv = load4(ys + j * LP + pt * 16 + g4);
          const f32x4 xv = load4(xs + j * LP + pt * 16 + g4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dd += yv[e] * xv[e];
            acc[e] = j < valid ? acc[e] + D * yv[e] : 0.f;
          }
          buffer_store4(dxb, j * P + pt * 16 + g4, acc, Tin());
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      if constexpr (NS == 1) {
        own_pairs();
        inputs(0);
      } else {
        inputs(0);
        __syncthreads();
        if (tn == 0) {
#pragma unroll
          for (int pb = 0; pb < PHL; ++pb)
            store4_two(ds + (nt * 16 + lc) * LS + pb * 16 + g4, DL, dv[1][pb]);
        }
        own_pairs();
        __syncthreads();
        inputs(1);
      }
      dd = wave_sum(dd);
      if (lane == 0) z.dd[w] = dd;
      __syncthreads();
    }
    if (w == 0) finish(h1 - 1, lane, 0);
  } else {
    // a chunk behind its sequence: zeros
    for (int h = h0; h < h1; ++h) {
      const size_t th = ((size_t)b * a.H + h) * a.T + t0;
      constexpr int VE = 16 / sizeof(Tin);
      for (int e = threadIdx.x; e < rows * (P / VE); e += kThreads)
        *reinterpret_cast<uint4*>((Tin*)a.dx + th * P + (size_t)e * VE) = uint4{0u, 0u, 0u, 0u};
      if (threadIdx.x < rows) a.ddt[th + threadIdx.x] = 0.f;
      if (threadIdx.x < 3) sums[threadIdx.x * a.H + h] = 0.f;
    }
  }

#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int it = tn + TN * m, t = it * 16 + lc;
    if (it >= QT || t >= rows) continue;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const f32x4 vb = t < valid ? dB[m] : zero, vc = t < valid ? dC[m] : zero;
    const size_t at = (tg + t) * N + nt * 16 + g4;
    if (o.parts == 1) {
      store4((Tin*)a.dB + at, vb);
      store4((Tin*)a.dC + at, vc);
    } else {
      store4(o.dBp + part * GTN + at, vb);
      store4(o.dCp + part * GTN + at, vc);
    }
  }
}

// dB, dC from the head parts' sums, in order.
template <typename Tin>
__global__ __launch_bounds__(256) void ssm_part_sum_kernel(size_t n4, int parts, const float* dBp,
                                                           const float* dCp, Tin* dB, Tin* dC) {
  const size_t e = blockIdx.x * (size_t)256 + threadIdx.x;
  if (e >= n4) return;
  f32x4 sb = {0.f, 0.f, 0.f, 0.f}, sc = sb;
  for (int p = 0; p < parts; ++p) {
    const f32x4 x = load4(dBp + (p * n4 + e) * 4), y = load4(dCp + (p * n4 + e) * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sb[i] += x[i];
      sc[i] += y[i];
    }
  }
  store4(dB + e * 4, sb);
  store4(dC + e * 4, sc);
}

struct Plan {
  int nch, nseg, segch, parts, hper;
  size_t states, slots, logs, sums, parts_at, total;  // offsets in floats
};

Plan make_plan(int B, int H, int G, int T, int P, int N, int Q) {
  Plan p{};
  const long long BH = (long long)B * H;
  p.nch = (T + Q - 1) / Q;
  // walks: a workgroup a CU over both directions, in segments of 4 chunks at least,
  // and none at all if that makes fewer than 4: a pass that writes no states and two
  // more launches then cost what the shorter walk gives. The whole backward in one walk
  // and in segments, bf16: 8 pairs of 64 x 128, 8 chunks 41 and 45 us, 12 chunks 48.5
  // and 48, 16 chunks 57 and 48, 48 chunks 120 and 62; of 32 x 32, 12 chunks 29 and 34,
  // 16 chunks 33 and 34, 24 chunks 39 and 35; 32 pairs of 64 x 128 (4 segments), 24
  // chunks 116 and 102; 64 pairs (2 segments), 16 chunks 86 and 89; 100 pairs (2), 16
  // chunks 112 and 122, 48 chunks 416 and 437.
  const long long streams = 2 * BH * (P < 64 ? 1 : P / 64);
  long long want = streams > 0 ? (256 + streams - 1) / streams : 1;
  if (want > p.nch / 4) want = p.nch / 4;
  if (want < 4) want = 1;
  p.segch = p.nch > 0 ? (int)((p.nch + want - 1) / want) : 1;
  p.nseg = p.nch > 0 ? (p.nch + p.segch - 1) / p.segch : 1;
  // chunks: heads of a group are split where the chunks alone leave CUs idle
  const int Hg = G > 0 ? H / G : 1;
  const long long wgs = (long long)B * G * p.nch;
  long long parts = wgs > 0 ? (256 + wgs - 1) / wgs : 1;
  if (parts > Hg) parts = Hg;
  p.hper = Hg > 0 ? (int)((Hg + parts - 1) / parts) : 1;
  p.parts = Hg > 0 ? (Hg + p.hper - 1) / p.hper : 1;
  const size_t PN = (size_t)P * N;
  p.states = 0;
  p.slots = p.states + 2 * BH * p.nch * PN;
  p.logs = p.slots + 2 * BH * (p.nseg - 1) * PN;
  p.sums = p.logs + (2 * BH * (p.nseg - 1) + 3) / 4 * 4;
  p.parts_at = p.sums + ((size_t)3 * B * p.nch * H + 3) / 4 * 4;
  p.total = p.parts_at + (p.parts > 1 ? (size_t)2 * p.parts * B * G * T * N : 0);
  return p;
}

template <int P, int N, typename Tin>
int run_bwd(const SsmArgs& a, hipStream_t s) {
  const int BH = a.B * a.H, PN = P * N;
  const Plan p = make_plan(a.B, a.H, a.G, a.T, P, N, bwd_q<Tin>());
  constexpr int NT = 4 * walk_rows<P>(), SL = P / walk_rows<P>(), Q = bwd_q<Tin>();
  float* ws = (float*)((char*)a.ws + decay_bytes<Q>(a.B, a.H, a.T));
  float *slots = ws + p.slots, *logs = ws + p.logs, *states = ws + p.states;
  ChunkDecay<Q>* decay = (ChunkDecay<Q>*)a.ws;
  const long long chunks = (long long)BH * p.nch, streams = 2ll * BH * SL;
  const long long wgs = (long long)a.B * a.G * p.nch * p.parts;
  if (!grid_ok((chunks + 3) / 4, 256) || !grid_ok(streams * p.nseg, NT) ||
      !grid_ok(wgs, kThreads) || !column_sum_ok(3ll * a.H))
    return -1;
  launch_decay<Q>(a, decay, s);
  if (BH == 0)  // an empty batch: zeros for the parameters
    return launch_column_sum(ws, 0, 3 * a.H, a.H, 1, a.dA, a.dD, a.dbias, s);
  int tk;
  if (p.nseg > 1) {
    tk = ktimer_before(s, "ssm_bwd_state");
    hipLaunchKernelGGL((ssm_walk_kernel<P, N, Tin, false>),
                       dim3((unsigned)(streams * (p.nseg - 1))), dim3(NT), 0, s, a, p.nseg,
                       p.segch, decay, slots, logs, states);
    ktimer_after(s, tk);
    tk = ktimer_before(s, "ssm_bwd_chain");
    hipLaunchKernelGGL(ssm_walk_chain_kernel, dim3((PN / 4 + 255) / 256, 2 * BH), dim3(256), 0, s,
                       BH, PN, N, p.nseg - 1, a.S0, a.dST, slots, logs);
    ktimer_after(s, tk);
  }
  tk = ktimer_before(s, "ssm_bwd_walk");
  hipLaunchKernelGGL((ssm_walk_kernel<P, N, Tin, true>), dim3((unsigned)(streams * p.nseg)),
                     dim3(NT), 0, s, a, p.nseg, p.segch, decay, slots, logs, states);
  ktimer_after(s, tk);
  int rc = (int)hipGetLastError();
  if (rc) return rc;
  if (p.nch > 0) {
    const size_t GTN = (size_t)a.B * a.G * a.T * N;
    const ChunkOut o{states, ws + p.sums, ws + p.parts_at,
                     ws + p.parts_at + (size_t)p.parts * GTN, p.parts, p.hper};
    tk = ktimer_before(s, "ssm_bwd");
    hipLaunchKernelGGL((ssm_bwd_chunk_kernel<P, N, Tin>),
                       dim3((unsigned)wgs), dim3(kThreads),
                       0, s, a, o, decay);
    ktimer_after(s, tk);
    if (p.parts > 1) {
      tk = ktimer_before(s, "ssm_bwd_parts");
      hipLaunchKernelGGL((ssm_part_sum_kernel<Tin>), dim3((unsigned)((GTN / 4 + 255) / 256)),
                         dim3(256), 0, s, GTN / 4, p.parts, o.dBp, o.dCp, (Tin*)a.dB,
                         (Tin*)a.dC);
      ktimer_after(s, tk);
    }
    rc = (int)hipGetLastError();
    if (rc) return rc;
  }
  return launch_column_sum(ws + p.sums, a.B * p.nch, 3 * a.H, a.H, 1, a.dA, a.dD, a.dbias, s);
}

template <int P, int N>
int run_bwd_t(const SsmArgs& a, hipStream_t s) {
  return a.bf16 ? run_bwd<P, N, __bf16>(a, s) : run_bwd<P, N, float>(a, s);
}

template <int P>
int run_bwd_n(const SsmArgs& a, hipStream_t s) {
  switch (a.N) {
    case 32: return run_bwd_t<P, 32>(a, s);
    case 64: return run_bwd_t<P, 64>(a, s);
    case 128: return run_bwd_t<P, 128>(a, s);
  }
  return -1;
}

}  // namespace

size_t ssm_backward_ws(int B, int H, int G, int T, int P, int N, int bf16) {
  return make_plan(B, H, G, T, P, N, bf16 ? bwd_q<__bf16>() : bwd_q<float>()).total *
             sizeof(float) +
         (bf16 ? decay_bytes<bwd_q<__bf16>()>(B, H, T) : decay_bytes<bwd_q<float>()>(B, H, T));
}

int launch_ssm_backward(const SsmArgs& a, hipStream_t s) {
  switch (a.P) {
    case 32: return run_bwd_n<32>(a, s);
    case 64: return run_bwd_n<64>(a, s);
    case 128: return run_bwd_n<128>(a, s);
  }
  return -1;
}

}  // namespace osdn
