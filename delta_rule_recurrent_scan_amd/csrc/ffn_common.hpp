// Tiled products of the gated feed-forward block: acc[m][n] = sum_k A[m,k] B[n,k],
// each operand lying in memory with k along its rows (K-major) or with m or n
// along them (MN-major).
//
// A workgroup forms a BM x BN tile. Tiles of 128 bytes of k (64 bf16, 32 fp32) go
// from global memory straight to LDS, 16 bytes a lane, into the one of two stages
// that is not being read; each wave feeds its matrix instructions from the other.
// LDS rows are swizzled in units of 16 bytes, so that the lanes that are served
// together lie on different banks: unit u of K-major row r at u ^ (r & 7), of
// MN-major row k at u ^ 2 f(k). MN-major bf16 is read by the LDS transpose load,
// which gives a lane the run of k that a K-major row would.
//
// Operands whose rows do not start on 16 bytes, and the last part of k, go through
// registers, with zeros behind the end of k. Rows behind m and n repeat the last
// one; their products are not stored.
#pragma once

#include "device_common.hpp"
#include "layer.hpp"
#include "pack_common.hpp"
#include "row_common.hpp"
#include "../../include/osdn.h"

namespace osdn {
namespace ffn {

constexpr int kRowBytes = 128;   // of a K-major LDS row: one tile of k
template <typename T>
constexpr int kUnit = 16 / (int)sizeof(T);       // elements of 16 bytes
template <typename T>
constexpr int kTileK = kRowBytes / (int)sizeof(T);

typedef __attribute__((address_space(3))) char lds_char;

// 16 bytes a lane from the buffer r at the lane's byte offset to LDS, 1 KB from `lds`
// on. The load writes no register; the compiler does not know of it (of the builtin's
// it would wait for all before every transpose load), so the waits are written out,
// wait_loads() below. Memory past the LDS address register takes one cycle to use it.
__device__ __forceinline__ void load_lds(u32x4 r, unsigned offset, unsigned lds) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %0, %1, 0 offen lds"
      :
      : "v"(offset), "s"(r), "s"(lds)
      : "m0", "memory");
}

// One 16-byte unit of each operand a lane: 32 of k for bf16, 16 for fp32.
__device__ __forceinline__ void mma(f32x4& acc, const uint4& a, const uint4& b, __bf16) {
  acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x4& acc, const uint4& a, const uint4& b, float) {
  const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], acc, 0, 0, 0);
}

// Swizzle of an MN-major row.
__device__ __forceinline__ int mn_swizzle(int k) { return ((k & 3) | ((k >> 3) & 1) << 2) << 1; }

// ROWS rows (m or n) of an operand, one tile of k, in LDS. NT threads stage it.
template <typename T, int ROWS, bool KMAJ, int NT>
struct Stage {
  static constexpr int BYTES = ROWS * kRowBytes;
  static constexpr int UNITS = BYTES / 16, PER = UNITS / NT;   // units a thread
  static constexpr int UPR = KMAJ ? 8 : ROWS / kUnit<T>;       // units an LDS row
  static_assert(UNITS % NT == 0 && NT % 64 == 0, "whole waves stage a tile");

  __device__ __forceinline__ static int swizzle(int row) {
    return KMAJ ? row & 7 : mn_swizzle(row) & (UPR - 1);
  }
  // LDS row and logical unit of the thread's j-th unit.
  __device__ __forceinline__ static void where(int j, int& row, int& u) {
    const int at = (wave_id() * PER + j) * 64 + (threadIdx.x & 63);
    row = at / UPR;
    u = (at % UPR) ^ swizzle(row);
  }
  // Byte offsets of the thread's units from the tile's first element; `rows` of
  // the operand exist from there on (a multiple of a unit when MN-major).
  __device__ __forceinline__ static void offsets(unsigned (&o)[PER], long long ld, int rows) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      int row, u;
      where(j, row, u);
      if constexpr (KMAJ) {
        o[j] = (unsigned)min(row, rows - 1) * (unsigned)ld * (unsigned)sizeof(T) + u * 16;
      } else {
        o[j] = (unsigned)row * (unsigned)ld * (unsigned)sizeof(T) +
               min(u * kUnit<T>, rows - kUnit<T>) * (unsigned)sizeof(T);
      }
    }
  }
  // A whole tile of k, global memory to LDS. p: its first element.
  __device__ __forceinline__ static void direct(char* lds, const T* p, const unsigned (&o)[PER]) {
    const u32x4 r = {(unsigned)(size_t)p, (unsigned)((size_t)p >> 32) & 0xffffu, ~0u, 0x00027000u};
#pragma unroll
    for (int j = 0; j < PER; ++j)
      load_lds(r, o[j], (unsigned)(size_t)(lds_char*)lds + (wave_id() * PER + j) * 1024);
  }
  // Any tile through registers: nk of k exist, `rows` rows.
  __device__ __forceinline__ static void fetch(uint4 (&v)[PER], const T* p, long long ld, int rows,
                                               int nk) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      int row, u;
      where(j, row, u);
      const int m = KMAJ ? row : u * kUnit<T>, k = KMAJ ? u * kUnit<T> : row;
      const int have = KMAJ ? (m < rows ? nk - k : 0) : (k < nk ? rows - m : 0);
      v[j] = uint4{0u, 0u, 0u, 0u};
      const T* q = p + (KMAJ ? (long long)m * ld + k : (long long)k * ld + m);
      if (have >= kUnit<T>) {
        __builtin_memcpy(&v[j], q, 16);
      } else if (have > 0) {
        T t[kUnit<T>];
#pragma unroll
        for (int i = 0; i < kUnit<T>; ++i) t[i] = i < have ? q[i] : from_f32<T>(0.f);
        __builtin_memcpy(&v[j], t, 16);
      }
    }
  }
  __device__ __forceinline__ static void put(char* lds, const uint4 (&v)[PER]) {
#pragma unroll
    for (int j = 0; j < PER; ++j)
      *(uint4*)(lds + ((wave_id() * PER + j) * 64 + (threadIdx.x & 63)) * 16) = v[j];
  }
  // The lane's unit of the 16 rows from `row0` on (a multiple of 16), step 0 or 1
  // of the tile: k = 8 (bf16) or 4 (fp32) times the lane's group and on.
  __device__ __forceinline__ static uint4 frag(const char* lds, int row0, int step) {
    const int lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
    if constexpr (KMAJ) {
      return *(const uint4*)(lds + (row0 + l) * kRowBytes + (((4 * step + g) ^ (l & 7)) << 4));
    } else if constexpr (sizeof(T) == 2) {
      typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
      const int k = 32 * step + 8 * g + (l >> 2);
      const int u = (row0 / 8 + ((l & 3) >> 1)) ^ swizzle(k);
      const char* q = lds + k * (ROWS * 2) + u * 16 + 8 * (l & 1);
      const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)q);
      const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(q + 4 * ROWS * 2));
      return __builtin_bit_cast(uint4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 16 * step + 4 * g + i, m = row0 + l;
        v[i] = *(const float*)(lds + k * (ROWS * 4) + ((m / 4) ^ swizzle(k)) * 16 + (m & 3) * 4);
      }
      return uint4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                   __float_as_uint(v[3])};
    }
  }
};

// A tile shape: BM x BN by WM x WN waves.
template <int BM_, int BN_, int WM_, int WN_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int NT = 64 * WM * WN;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;   // 16 x 16 tiles a wave
};
typedef Shape<256, 256, 2, 4> Large;
typedef Shape<128, 128, 2, 2> Middle;
typedef Shape<64, 64, 2, 2> Small;

// Where a workgroup's tile lies: runs of eight tiles of m for each of n, and
// consecutive ones on the same XCD (workgroups go to the eight in turn), so that
// the workgroups of an XCD share their operands' rows in its L2.
struct TileAt {
  int m, n, split;
};
__device__ __forceinline__ TileAt tile_at(int tm, int tn, int splits) {
  const int total = tm * tn * splits, id = blockIdx.x;
  const int x = id % 8, i = id / 8;
  const int at = x * (total / 8) + min(x, total % 8) + i;
  const int per = tm * tn, s = at / per, r = at % per;
  const int width = 8 * tn, g = r / width, m0 = g * 8, h = min(tm - m0, 8), w = r % width;
  return TileAt{m0 + w % h, w / h, s};
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The products of a wave over the tiles of k from t0 to t1, in the order of `src`:
// those of a whole tile's length, src.full of them, before the ends. src.direct_a(t, a)
// and src.direct_b(t, b) send a whole tile's operand to LDS, src.fetch(t) and
// src.put(a, b) take any through registers; src.fragb(b, j, step) is the wave's j-th 16
// columns.
//
// Whole tiles pass through five buffers in turn, A and B of one tile after the other:
// while tile t is used, t + 1 and A of t + 2 are on their way, and B of t + 2 and A of
// t + 3 follow as soon as every wave has read tile t, so that the memory pipes never
// run empty. A wave works off a tile in four parts (two steps of k, two halves of its
// rows) and fetches each part's operands while the one before is multiplied; the
// barrier stands before a tile's last part, whose operands are in registers.
template <typename T, class S, bool AK, bool DIRECT, class Src>
__device__ __forceinline__ void products(f32x4 (&acc)[S::TM][S::TN], Src& src, int t0, int t1) {
  constexpr int BUF = (S::BM > S::BN ? S::BM : S::BN) * kRowBytes;
  __shared__ __attribute__((aligned(1024))) char u0[BUF], u1[BUF], u2[BUF], u3[BUF], u4[BUF];
  typedef Stage<T, S::BM, AK, S::NT> SA;
  constexpr int NA = SA::PER, NB = S::BN * kRowBytes / 16 / S::NT, HM = S::TM / 2;
  const int wm = wave_id() / S::WN * (S::BM / S::WM);
#pragma unroll
  for (int i = 0; i < S::TM; ++i)
#pragma unroll
    for (int j = 0; j < S::TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto read_a = [&](uint4 (&f)[HM], const char* la, int step, int half) {
#pragma unroll
    for (int i = 0; i < HM; ++i) f[i] = SA::frag(la, wm + 16 * (half * HM + i), step);
  };
  auto read_b = [&](uint4 (&f)[S::TN], const char* lb, int step) {
#pragma unroll
    for (int j = 0; j < S::TN; ++j) f[j] = src.fragb(lb, j, step);
  };
  // (columns first: a lane then holds four consecutive n of one m)
  auto multiply = [&](const uint4 (&fa)[HM], const uint4 (&fb)[S::TN], int half) {
#pragma unroll
    for (int i = 0; i < HM; ++i)
#pragma unroll
      for (int j = 0; j < S::TN; ++j) mma(acc[half * HM + i][j], fb[j], fa[i], T());
  };

  if constexpr (DIRECT) {
    const int tf = min(t1, src.full);
    uint4 fa[2][HM], fb[2][S::TN];
    auto fence = [&]() {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    // tile t in buffers a, b; the next one's are an, bn
    auto tile = [&](int t, char* a, char* b, const char* an, const char* bn) {
      read_a(fa[1], a, 0, 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(fa[0], fb[0], 0);
      __builtin_amdgcn_sched_barrier(0);
      read_b(fb[1], b, 1);
      read_a(fa[0], a, 1, 0);
      __builtin_amdgcn_sched_barrier(0);
      multiply(fa[1], fb[0], 1);
      __builtin_amdgcn_sched_barrier(0);
      read_a(fa[1], a, 1, 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(fa[0], fb[1], 0);
      __builtin_amdgcn_sched_barrier(0);
      if (t + 1 < tf) {
        // the next tile has arrived, A of the one behind it may be on its way
        if (t + 2 < tf) {
          wait_loads<NA>();
        } else {
          wait_loads<0>();
        }
        fence();
        if (t + 2 < tf) src.direct_b(t + 2, a);
        if (t + 3 < tf) src.direct_a(t + 3, b);
        read_b(fb[0], bn, 0);
        read_a(fa[0], an, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      multiply(fa[1], fb[1], 1);
      __builtin_amdgcn_sched_barrier(0);
    };
    if (t0 < tf) {
      src.direct_a(t0, u0);
      src.direct_b(t0, u1);
      if (t0 + 1 < tf) {
        src.direct_a(t0 + 1, u2);
        src.direct_b(t0 + 1, u3);
      }
      if (t0 + 2 < tf) {
        src.direct_a(t0 + 2, u4);
        wait_loads<2 * NA + NB>();
      } else {
        wait_loads<0>();
      }
      fence();
      read_b(fb[0], u1, 0);
      read_a(fa[0], u0, 0, 0);
      for (int t = t0;;) {
        tile(t, u0, u1, u2, u3);
        if (++t >= tf) break;
        tile(t, u2, u3, u4, u0);
        if (++t >= tf) break;
        tile(t, u4, u0, u1, u2);
        if (++t >= tf) break;
        tile(t, u1, u2, u3, u4);
        if (++t >= tf) break;
        tile(t, u3, u4, u0, u1);
        if (++t >= tf) break;
      }
    }
    t0 = max(t0, tf);
  }
  // through registers, a tile ahead of the one that is being used
  if (t0 < t1) src.fetch(t0);
  for (int t = t0; t < t1; ++t) {
    __syncthreads();
    src.put(u0, u1);
    __syncthreads();
    if (t + 1 < t1) src.fetch(t + 1);
#pragma unroll
    for (int step = 0; step < 2; ++step) {
      uint4 fa[HM], fb[S::TN];
      read_b(fb, u1, step);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        read_a(fa, u0, step, half);
        multiply(fa, fb, half);
      }
    }
  }
}

// Four consecutive elements of a row, n of them inside; vec: rows start on 16 bytes
// and hold whole fours.
template <typename T>
__device__ __forceinline__ void store4(T* p, const f32x4& v, int n, bool vec) {
  if (vec) {
    if (n <= 0) return;
    if constexpr (sizeof(T) == 2) {
      *(uint2*)p = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
      *(f32x4*)p = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

// The activation of g, and its slope.
__device__ __forceinline__ float activated(float g, int act) {
  if (act == OSDN_ACT_SILU) return g * sigmoid_f(g);
  if (act == OSDN_ACT_GELU) return g * (0.5f * erfcf(-0.707106781186547524f * g));
  return g * sigmoid_f(1.59576912160573071f * fmaf(0.044715f * g * g, g, g));
}
__device__ __forceinline__ void activated(float g, int act, float& f, float& slope) {
  if (act == OSDN_ACT_SILU) {
    const float s = sigmoid_f(g);
    f = g * s;
    slope = s * fmaf(g, 1.f - s, 1.f);
  } else if (act == OSDN_ACT_GELU) {
    const float p = 0.5f * erfcf(-0.707106781186547524f * g);
    f = g * p;
    slope = fmaf(g * 0.398942280401432678f,
                 __builtin_amdgcn_exp2f(-0.721347520444481704f * g * g), p);
  } else {
    // 0.5 (1 + tanh z) = sigmoid(2 z), z = sqrt(2 / pi) (g + 0.044715 g^3)
    const float p = sigmoid_f(1.59576912160573071f * fmaf(0.044715f * g * g, g, g));
    f = g * p;
    slope = fmaf(g * p * (1.f - p), 1.59576912160573071f * fmaf(0.134145f * g, g, 1.f), p);
  }
}

// How a product of M x N (in tiles of k: nt) is cut: the shape (0 large, 1 middle, 2
// small) and the parts that its k is split into.
struct Cut {
  int shape, splits;
};
Cut cut_of(long long M, long long N, int nt);

// out[i] = the sum over the splits of part[s][i] of n elements, in order.
int launch_ffn_sum(const float* part, int splits, long long n, void* out, int bf16, hipStream_t s);

}  // namespace ffn
}  // namespace osdn
