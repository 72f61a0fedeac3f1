// Tiled products of the gated feed-forward block: acc[m][n] = sum_k A[m,k] B[n,k],
// each operand lying in memory with k along its rows (K-major) or with m or n
// along them (MN-major).
//
// A workgroup forms a BM x BN tile. Tiles of 128 bytes of k (64 bf16, 32 fp32) go
// from global memory straight to LDS, 16 bytes a lane, two tiles ahead of the one
// that is used, through five buffers in turn; each wave fetches the operands of its next
// matrix instructions while the last are worked off. A tile of k of 256 x 256 bf16 takes
// 1.46 us (1470 TFLOP/s); what a product loses against that is its start, its results'
// way to memory, and rounds of tiles that do not fill the card. Those are cut along k and
// added by a second launch, in a fixed order, where a model of these costs says that it
// pays (make_plan).
//
// LDS rows are swizzled in units of 16 bytes, so that the lanes that are served
// together lie on different banks: unit u of K-major row r at u ^ (r & 7), of
// MN-major row k at u ^ 2 f(k) (fp32: u ^ (k & 12)). MN-major bf16 is read by the LDS
// transpose load, which gives a lane the run of k that a K-major row would.
//
// The last part of k goes through registers, with zeros behind the end of k. Rows
// behind m and n repeat the last one; their products are not stored. All rows start on
// 16 bytes and hold whole eights of elements: operands that do not are first copied so
// (777 x 1021 x 2001 in bf16: with rows of any alignment through registers the products
// took 40 to 97 us, now 22 to 28).
#pragma once

#include "device_common.hpp"
#include "launch.hpp"
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

// The thread's number, worked out anew: what depends on it is not kept in registers
// over the products of an item, whose accumulators and operands take them all.
__device__ __forceinline__ int fresh_thread() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}
__device__ __forceinline__ int wave_of(int thread) {
  return __builtin_amdgcn_readfirstlane(thread >> 6);
}

// Swizzle of rows that are read in runs of four, eight apart.
__device__ __forceinline__ int runs_swizzle(int r) { return (r & 3) | ((r >> 3) & 1) << 2; }

// ROWS rows (m or n) of an operand, one tile of k, in LDS. NT threads stage it. RUNS
// (K-major): fragments take rows in runs of four, eight apart.
template <typename T, int ROWS, bool KMAJ, int NT, bool RUNS = false>
struct Stage {
  static constexpr int BYTES = ROWS * kRowBytes;
  static constexpr int UNITS = BYTES / 16, PER = UNITS / NT;   // units a thread
  static constexpr int UPR = KMAJ ? 8 : ROWS / kUnit<T>;       // units an LDS row
  static_assert(UNITS % NT == 0 && NT % 64 == 0, "whole waves stage a tile");

  __device__ __forceinline__ static int swizzle(int row) {
    if constexpr (KMAJ) return RUNS ? runs_swizzle(row) : row & 7;
    // (fp32: the four rows that a wave reads at once lie four apart, 64 bytes of each)
    return (sizeof(T) == 2 ? runs_swizzle(row) * 2 : row & 12) & (UPR - 1);
  }
  // LDS row and logical unit of a thread's j-th unit.
  __device__ __forceinline__ static void where(int thread, int j, int& row, int& u) {
    const int at = (wave_of(thread) * PER + j) * 64 + (thread & 63);
    row = at / UPR;
    u = (at % UPR) ^ swizzle(row);
  }
  // Byte offsets of the thread's units from the tile's first element; `rows` of
  // the operand exist from there on (a multiple of a unit when MN-major).
  __device__ __forceinline__ static void offsets(unsigned (&o)[PER], long long ld, int rows) {
    const int thread = fresh_thread();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      int row, u;
      where(thread, j, row, u);
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
    const int thread = fresh_thread();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      int row, u;
      where(thread, j, row, u);
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
      // RUNS: row0 is 8 h of a block of 32 rows' first, or 8 h + 4
      const int r = row0 + (RUNS ? 8 * (l >> 2) + (l & 3) : l);
      return *(const uint4*)(lds + r * kRowBytes + (((4 * step + g) ^ swizzle(r)) << 4));
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
typedef Shape<64, 128, 2, 2> SmallPairs;   // the forward's: column tiles in pairs

// How a product is cut: tm x tn tiles over nt tiles of k. The first `whole` tiles
// (full rounds of the workgroups that are on the card at once) are formed whole, the
// rest in `splits` parts of `per` tiles of k each, which a second launch adds.
struct Plan {
  int shape;                       // 0 large, 1 middle, 2 small
  int tm, tn, nt, whole, splits, per;
  int area;                        // elements of a tile
  long long parts_at;              // its parts' place in FfnArgs::parts
  __host__ __device__ int rest() const { return tm * tn - whole; }
  // Items of the rest that go before the whole tiles: the workgroups that begin with a
  // part store their results while the others multiply, and the other way about.
  __host__ __device__ int lead() const { return whole ? splits / 2 * rest() : 0; }
  __host__ __device__ int items() const { return whole + rest() * splits; }
};

struct Item {
  int m, n, split, t0, t1;
  int tile;                        // of the rest (-1: a whole tile)
};
// Consecutive numbers on one XCD (workgroups go to the eight in turn): number id of
// `total`.
__device__ __forceinline__ int on_xcd(int id, int total) {
  const int x = id % 8;
  return x * (total / 8) + min(x, total % 8) + id / 8;
}
// Tiles run over eight of m for each of n, so that the workgroups of an XCD share their
// operands' rows in its L2.
__device__ __forceinline__ void tile_place(const Plan& p, int r, int& m, int& n) {
  const int width = 8 * p.tn, m0 = r / width * 8, h = min(p.tm - m0, 8), w = r % width;
  m = m0 + w % h;
  n = w / h;
}
__device__ __forceinline__ Item item_at(const Plan& p, int id) {
  Item it;
  int r;
  const int lead = p.lead();
  if (id >= lead && id < lead + p.whole) {
    r = on_xcd(id - lead, p.whole);
    it.split = it.tile = -1;
    it.t0 = 0;
    it.t1 = p.nt;
  } else {
    const int rest = p.rest(), k = id < lead ? id : id - p.whole;
    const int j = id < lead ? on_xcd(k, lead) : lead + on_xcd(k - lead, rest * p.splits - lead);
    it.split = j / rest;
    it.tile = j % rest;
    r = p.whole + it.tile;
    it.t0 = it.split * p.per;
    it.t1 = min(p.nt, it.t0 + p.per);
  }
  tile_place(p, r, it.m, it.n);
  return it;
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// One item of a product. Op is the product:
//   place(a, item)       the operands' tile
//   direct_a(t, lds), direct_b  tile t of k of an operand to LDS, whole tiles (t < full)
//   fetch(t), put(a, b)  any tile through registers
//   fragb(lds, j, step)  the wave's j-th 16 columns
//   store_row(a, i, row) the wave's i-th 16 rows of results
//
// Whole tiles of k pass through five buffers in turn, A and B of one tile after the
// other: while tile t is used, t + 1 and A of t + 2 are on their way, and B of t + 2 and
// A of t + 3 follow as soon as every wave has read tile t, so that the memory pipes
// never run empty. A wave works off a tile in four parts (two steps of k, two halves of
// its rows) and fetches each part's operands while the one before is multiplied; the
// barrier stands before a tile's last part, whose operands are in registers.
//
// id: the item's number; u0 .. u4: the buffers.
template <class S>
constexpr int kBuffer = (S::BM > S::BN ? S::BM : S::BN) * kRowBytes;
template <typename T, class S, class Op>
__device__ __forceinline__ void products(const FfnArgs& a, const Plan& p, int id, char* u0,
                                         char* u1, char* u2, char* u3, char* u4) {
  typedef typename Op::StageA SA;
  constexpr int NA = SA::PER, NB = S::BN * kRowBytes / 16 / S::NT, HM = S::TM / 2;
  const int wm = wave_id() / S::WN * (S::BM / S::WM);

  f32x4 acc[S::TM][S::TN];
#pragma unroll
  for (int i = 0; i < S::TM; ++i)
#pragma unroll
    for (int j = 0; j < S::TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto read_a = [&](uint4 (&f)[HM], const char* la, int step, int half) {
#pragma unroll
    for (int i = 0; i < HM; ++i) f[i] = SA::frag(la, wm + 16 * (half * HM + i), step);
  };
  // (columns first: a lane then holds four consecutive n of one m)
  auto multiply = [&](const uint4 (&fa)[HM], const uint4 (&fb)[S::TN], int half) {
#pragma unroll
    for (int i = 0; i < HM; ++i)
#pragma unroll
      for (int j = 0; j < S::TN; ++j) mma(acc[half * HM + i][j], fb[j], fa[i], T());
  };

  const Item it = item_at(p, id);
  Op op;
  op.place(a, it);
  int t = it.t0;
  {
    const int tf = min(it.t1, op.full);
    uint4 fa[2][HM], fb[2][S::TN];
    auto read_b = [&](uint4 (&f)[S::TN], const char* lb, int step) {
#pragma unroll
      for (int j = 0; j < S::TN; ++j) f[j] = op.fragb(lb, j, step);
    };
    auto fence = [&]() {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    // tile t in buffers la, lb; the next one's are an, bn
    auto tile = [&](char* la, char* lb, const char* an, const char* bn) {
      read_a(fa[1], la, 0, 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(fa[0], fb[0], 0);
      __builtin_amdgcn_sched_barrier(0);
      read_b(fb[1], lb, 1);
      read_a(fa[0], la, 1, 0);
      __builtin_amdgcn_sched_barrier(0);
      multiply(fa[1], fb[0], 1);
      __builtin_amdgcn_sched_barrier(0);
      read_a(fa[1], la, 1, 1);
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
        if (t + 2 < tf) op.direct_b(t + 2, la);
        if (t + 3 < tf) op.direct_a(t + 3, lb);
        read_b(fb[0], bn, 0);
        read_a(fa[0], an, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      multiply(fa[1], fb[1], 1);
      __builtin_amdgcn_sched_barrier(0);
    };
    if (t < tf) {
      op.direct_a(t, u0);
      op.direct_b(t, u1);
      if (t + 1 < tf) {
        op.direct_a(t + 1, u2);
        op.direct_b(t + 1, u3);
      }
      if (t + 2 < tf) {
        op.direct_a(t + 2, u4);
        wait_loads<2 * NA + NB>();
      } else {
        wait_loads<0>();
      }
      fence();
      read_b(fb[0], u1, 0);
      read_a(fa[0], u0, 0, 0);
      for (;;) {
        tile(u0, u1, u2, u3);
        if (++t >= tf) break;
        tile(u2, u3, u4, u0);
        if (++t >= tf) break;
        tile(u4, u0, u1, u2);
        if (++t >= tf) break;
        tile(u1, u2, u3, u4);
        if (++t >= tf) break;
        tile(u3, u4, u0, u1);
        if (++t >= tf) break;
      }
    }
  }
  // through registers, a tile ahead of the one that is being used
  if (t < it.t1) op.fetch(t);
  for (; t < it.t1; ++t) {
    __syncthreads();
    op.put(u0, u1);
    __syncthreads();
    if (t + 1 < it.t1) op.fetch(t + 1);
#pragma unroll
    for (int step = 0; step < 2; ++step) {
      uint4 fa[HM], fb[S::TN];
#pragma unroll
      for (int j = 0; j < S::TN; ++j) fb[j] = op.fragb(u1, j, step);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        read_a(fa, u0, step, half);
        multiply(fa, fb, half);
      }
    }
  }

  if (p.splits > 1 && it.tile >= 0) {
    f32x4* part = (f32x4*)(a.parts + p.parts_at) +
                  (size_t)(it.tile * p.splits + it.split) * (S::BM * S::BN / 4) + fresh_thread();
#pragma unroll
    for (int i = 0; i < S::TM; ++i)
#pragma unroll
      for (int j = 0; j < S::TN; ++j) part[(i * S::TN + j) * S::NT] = acc[i][j];
  } else {
#pragma unroll
    for (int i = 0; i < S::TM; ++i) op.store_row(a, i, acc[i]);
  }
}

// The parts of one tile's i-th rows added in order, and stored.
template <class S, class Op>
__device__ __forceinline__ void join_parts(const FfnArgs& a, const Plan& p, int id) {
  const int tile = id / S::TM, i = id % S::TM;
  Item it;
  it.t0 = it.t1 = it.split = 0;
  it.tile = tile;
  tile_place(p, p.whole + tile, it.m, it.n);
  Op op;
  op.place(a, it);
  const f32x4* part = (const f32x4*)(a.parts + p.parts_at) +
                      (size_t)tile * p.splits * (S::BM * S::BN / 4) +
                      i * S::TN * S::NT + threadIdx.x;
  f32x4 row[S::TN];
#pragma unroll
  for (int j = 0; j < S::TN; ++j) row[j] = part[j * S::NT];
  for (int s = 1; s < p.splits; ++s) {
    part += S::BM * S::BN / 4;
#pragma unroll
    for (int j = 0; j < S::TN; ++j) row[j] += part[j * S::NT];
  }
  op.store_row(a, i, row);
}

template <typename T, class S, class Op>
__global__ __launch_bounds__(S::NT) void ffn_kernel(FfnArgs a, Plan p) {
  __shared__ __attribute__((aligned(1024))) char u0[kBuffer<S>], u1[kBuffer<S>], u2[kBuffer<S>],
      u3[kBuffer<S>], u4[kBuffer<S>];
  products<T, S, Op>(a, p, blockIdx.x, u0, u1, u2, u3, u4);
}
template <class S, class Op>
__global__ __launch_bounds__(S::NT) void ffn_join_kernel(FfnArgs a, Plan p) {
  join_parts<S, Op>(a, p, blockIdx.x);
}
// Two products in one launch, the items of the first before those of the second.
template <typename T, class S, class Op1, class Op2>
__global__ __launch_bounds__(S::NT) void ffn_pair_kernel(FfnArgs a, Plan p, Plan q) {
  __shared__ __attribute__((aligned(1024))) char u0[kBuffer<S>], u1[kBuffer<S>], u2[kBuffer<S>],
      u3[kBuffer<S>], u4[kBuffer<S>];
  const int n = p.items();
  if ((int)blockIdx.x < n) {
    products<T, S, Op1>(a, p, blockIdx.x, u0, u1, u2, u3, u4);
  } else {
    products<T, S, Op2>(a, q, blockIdx.x - n, u0, u1, u2, u3, u4);
  }
}
template <class S, class Op1, class Op2>
__global__ __launch_bounds__(S::NT) void ffn_pair_join_kernel(FfnArgs a, Plan p, Plan q, int n) {
  if ((int)blockIdx.x < n) {
    join_parts<S, Op1>(a, p, blockIdx.x);
  } else {
    join_parts<S, Op2>(a, q, blockIdx.x - n);
  }
}

template <typename T, class S, class Op>
int launch_products(const FfnArgs& a, const Plan& p, const char* name, const char* join_name,
                    hipStream_t s) {
  int tk = ktimer_before(s, name);
  hipLaunchKernelGGL((ffn_kernel<T, S, Op>), dim3(p.items()), dim3(S::NT), 0, s, a, p);
  ktimer_after(s, tk);
  const int rc = (int)hipGetLastError();
  if (rc || p.splits == 1) return rc;
  tk = ktimer_before(s, join_name);
  hipLaunchKernelGGL((ffn_join_kernel<S, Op>), dim3(p.rest() * S::TM), dim3(S::NT), 0, s, a, p);
  ktimer_after(s, tk);
  return (int)hipGetLastError();
}

template <typename T, class S, class Op1, class Op2>
int launch_pair(const FfnArgs& a, const Plan& p, const Plan& q, const char* name,
                const char* join_name, hipStream_t s) {
  int tk = ktimer_before(s, name);
  hipLaunchKernelGGL((ffn_pair_kernel<T, S, Op1, Op2>), dim3(p.items() + q.items()), dim3(S::NT),
                     0, s, a, p, q);
  ktimer_after(s, tk);
  const int rc = (int)hipGetLastError();
  const int n = p.splits > 1 ? p.rest() * S::TM : 0, m = q.splits > 1 ? q.rest() * S::TM : 0;
  if (rc || n + m == 0) return rc;
  tk = ktimer_before(s, join_name);
  hipLaunchKernelGGL((ffn_pair_join_kernel<S, Op1, Op2>), dim3(n + m), dim3(S::NT), 0, s, a, p, q,
                     n);
  ktimer_after(s, tk);
  return (int)hipGetLastError();
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

// Eight of them; vec: rows hold whole eights.
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8], int n, bool vec) {
  if (vec) {
    if (n > 0) store_v<true, 8>(p, 8, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

// The activation of g, and its slope.
template <int ACT>
__device__ __forceinline__ float activated(float g) {
  if constexpr (ACT == OSDN_ACT_SILU) return g * sigmoid_f(g);
  if constexpr (ACT == OSDN_ACT_GELU) return g * (0.5f * erfcf(-0.707106781186547524f * g));
  return g * sigmoid_f(1.59576912160573071f * fmaf(0.044715f * g * g, g, g));
}
__device__ __forceinline__ float activated(float g, int act) {
  return act == OSDN_ACT_SILU   ? activated<OSDN_ACT_SILU>(g)
         : act == OSDN_ACT_GELU ? activated<OSDN_ACT_GELU>(g)
                                : activated<OSDN_ACT_GELU_TANH>(g);
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
    // (p is 0 or 1 from |g| = 16 on; the factor of 1 - p would be infinite from 1e20 on)
    const float c = __builtin_amdgcn_fmed3f(g, -16.f, 16.f);
    slope = fmaf(c * p * (1.f - p), 1.59576912160573071f * fmaf(0.134145f * c, c, 1.f), p);
  }
}

// The plan of a product of M x N over K, of the two in the weights' gradients or of the
// forward's, and the bytes of its parts.
constexpr double kLaunch = 4.5;   // microseconds between two launches
enum Kind { kOne, kTwo, kForwards };
bool make_plan(Plan& p, Kind kind, long long M, long long N, long long K, int bf16,
               double* microseconds = nullptr);
// Plans of the products kOne and kTwo of these sizes in one launch, where that takes less
// time than `microseconds`.
bool make_pair(Plan& p, Plan& q, const long long (&one)[3], const long long (&two)[3], int bf16,
               double microseconds);
size_t parts_bytes(const Plan& p);

inline int whole_eights(int n) { return (n + 7) / 8 * 8; }
inline size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
inline bool on16(const void* p) { return ((size_t)p & 15) == 0; }

// Copies of up to three operands: rows of C elements to rows of Cp, zeros behind C.
struct Pads {
  const void* in[3];
  void* out[3];
  long long ld[3], end[3];    // end: of its groups of eight among all
  int C, Cp;
};
// The id-th group of eight.
template <typename T>
__device__ __forceinline__ void pad_group(const Pads& p, long long id) {
  if (id >= p.end[2]) return;
  const int k = id < p.end[0] ? 0 : id < p.end[1] ? 1 : 2;
  const long long at = id - (k ? p.end[k - 1] : 0);
  const unsigned per = p.Cp / 8;
  const long long r = at / per;
  const int c = (int)(at % per) * 8;
  float v[8];
  load_v<false, 8>((const T*)p.in[k] + r * p.ld[k] + c, p.C - c, v);
  store_v<true, 8>((T*)p.out[k] + r * p.Cp + c, 8, v);
}
// Bytes that copies of x and the weights may take, and those that are needed: a's pointers
// and strides are then the copies'. pads.end[2]: the groups to copy, none if 0.
size_t aligned_bytes(long long R, int C, int F, int bf16);
Pads align_operands(FfnArgs& a, char* room);

}  // namespace ffn
}  // namespace osdn
