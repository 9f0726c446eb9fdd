// attend_mma.cuh -- attention over the cache on tensor cores, for heads of 64 to 256.
//
// Everything is turned round: scores are S^T = K Q^T, tokens by rows, and the output O^T =
// V^T P^T, so that the 16 rows of an m16n8k16 are tokens and then elements, and the eight
// columns are the queries that share a head: one decoded token's four or eight queries leave
// no columns empty that cost anything.
//
// Codes go into the products exactly, as normal fp16: e4m3 as the fp16 of the same value, a
// 4-bit code c as c - 8 (or 16 (c - 8): its bits stay where they lie).  A product's sum is cut
// at a place that goes by its operands' exponents, and a subnormal's is -14 whatever its value:
// c * 2^-24, which needs no subtraction, leaves the sum six to ten bits less.  Less 8 (values' less
// 8 and less 7 in turn), codes are even about zero, and what is added up is no larger than the
// values are.  (8000 tokens in groups of 32, f32: 6.6e-7 off in norm; as subnormals 5.6e-5.)
// A sum is cut toward zero, so one that goes on through all tokens loses 2^-26 of itself at each
// product: 500 queries over 40000 tokens of 8 bits were 3.3e-5 off.  Products of 16 tokens are
// therefore added up outside, where sums are rounded: 8e-7, for 1 to 8% of the time.
// A group's scale s and middle m = l + 8 s come in 32 bits outside: for keys
//   S = sum over groups of s_g (q_g . c_g) + m_g (sum of q_g),
// for values P_g = P s_g meets the codes, and sum_t P_t m_tg is kept beside.  Queries are
// scaled to 2^14 by a power of two a row and taken in one piece of 11 bits (bf16) or two.
// P s_g is held at most 2^15: M, which exponents are taken against, is the largest of
// x + floor(log2 s), so what is rounded off is small beside the largest product.
//
// The order of the contraction's elements is free as long as both sides have the same one:
// a lane's share of a row is contiguous, read from shared memory as it lies.
//
// Measured, in a graph: 32 sequences of up to 8192 tokens, 8 heads of 128 with 4 queries each,
// 8 bits: 57 us for 251 MB; all of 8192: 100 us for 554 MB, 81% of the copy rate, with the
// join some 5 us of it.  Memory bounds it.  4 sequences of up to 65536 with 8 queries, 4 bits in
// groups of 32: 94 to 101 us for 273 MB: 60.6 M warp instructions, 62% of the issue slots, and
// waits for one another's results.  A warp a query, on the other units: 20197 and 147804 us.  A
// worker may have a single tile: with two at least one token's attention takes 10.1 us for 9.7,
// with eight 15.7.
#pragma once

#include "attend.cuh"

namespace lp {
namespace {  // what a launch asks the runtime once belongs to its own library

constexpr float kLift = 14.0f;    // the largest weight is near 2^14
constexpr int kLeastScale = -60;  // scales below 2^-60 count as 2^-60 in M

template <int BITS, int DIM, int BS, bool WIDE, int NR>
struct Shape {
  static constexpr int kBits = BITS, kDim = DIM, kBlock = BS, kNR = NR;
  static constexpr bool kWide = WIDE;
  static constexpr int kBlocks = DIM / BS;           // blocks of elements of one group each
  static constexpr int kSteps = BS / 16;             // contraction steps of a block
  static constexpr int kRow = DIM * BITS / 8;        // bytes of a head
  static constexpr int kKeyBytes = BS / 4 * BITS / 8;    // a lane's, of a block of a key
  static constexpr int kValues = BS / 8;             // a lane's elements, of a block of a value
  static constexpr int kValueBytes = kValues * BITS / 8;
  // of queries and of P s_g.  A piece has 11 bits, and bf16 queries no more than 8; one piece of
  // P rounds by an eighth of the step of a bf16 result: 1.68e-3 off in norm, where the result's
  // own rounding leaves 1.67e-3.  Two cost 9% of a step in 8 bits, some 20% in 4.
  static constexpr int kPieces = WIDE ? 2 : 1;
  static constexpr int kTile = kRow <= 128 ? 32 : 16;    // tokens
  static constexpr int kM = kTile / 16;
  static constexpr int kUnit = kRow % 16 == 0 ? 16 : 8;  // bytes copied at once
  static constexpr int kChunks = kRow / kUnit;
  static constexpr int kCodes = kTile * kRow;        // bytes of a tile's keys
  static constexpr int kParams = kTile * kBlocks * 4;
  static constexpr int kStage = 2 * (kCodes + kParams);
  static constexpr int kStages = 2;
  static constexpr int kRows = 8 * NR;
  // blocks of four warps on an SM: 168 registers a thread where that holds the sums, else 255
  // (a fourth block leaves 128, and the sums of 8 rows by 128 elements are spilled)
  static constexpr int kResident = NR == 1 && DIM <= 128 ? 3 : 2;
};

// Which 16 bytes of a row lie where: rows that are read together lie in different banks.
template <int ROW>
__device__ __forceinline__ int swizzle(int token) {
  if (ROW == 128 || ROW == 256) return token & 7;
  if (ROW == 64) return (token >> 1) & 3;
  return 0;
}
template <int ROW>
__device__ __forceinline__ int swizzled(int byte, int f) {
  if (ROW == 64 || ROW == 128 || ROW == 256) return ((byte >> 4) ^ f) << 4 | (byte & 15);
  return byte;
}

template <int N>
struct Bytes {  // N bytes out of shared memory, in words
  uint32_t w[N <= 4 ? 1 : N / 4];
};

template <int N, int ROW>
__device__ __forceinline__ Bytes<N> bytes_at(const char* row, int byte, int f) {
  Bytes<N> r;
  if constexpr (N == 32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + swizzled<ROW>(byte + 16 * i, f));
      r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
  } else {
    const char* p = row + swizzled<ROW>(byte, f);
    if constexpr (N == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
    } else if constexpr (N == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      r.w[0] = v.x, r.w[1] = v.y;
    } else if constexpr (N == 4) {
      r.w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
      r.w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
      r.w[0] = *reinterpret_cast<const uint8_t*>(p);
    }
  }
  return r;
}

__device__ __forceinline__ uint32_t e4m3_two(uint32_t two) {  // to fp16
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(two)));
  return h;
}

__device__ __forceinline__ uint32_t f16_two(float low, float high) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(high), "f"(low));
  return r;
}

// Two 4-bit codes less a middle, as fp16: c (bits 0 to 3 of each half) in the last places of 1024,
// or 16 c (bits 4 to 7), less 1024 and the middle.  Mask and places are one instruction where they
// are written as one (as two they take a tenth more at the long size below).
template <int MIDDLE = 8>
__device__ __forceinline__ uint32_t codes_low(uint32_t x) {
  uint32_t r;
  asm("{ .reg .b32 t; lop3.b32 t, %1, 0x000f000f, 0x64006400, 0xea; add.rn.f16x2 %0, t, %2; }"
      : "=r"(r) : "r"(x), "r"(0xe400e400u + 0x00010001u * MIDDLE));
  return r;
}
template <int MIDDLE = 8>
__device__ __forceinline__ uint32_t codes_high(uint32_t x) {
  uint32_t r;
  asm("{ .reg .b32 t; lop3.b32 t, %1, 0x00f000f0, 0x64006400, 0xea; add.rn.f16x2 %0, t, %2; }"
      : "=r"(r) : "r"(x), "r"(0xe400e400u + 0x00100010u * MIDDLE));
  return r;
}

// Of 4-bit params: a group's scale, and the value of its middle code.
__device__ __forceinline__ float scale_of(uint32_t held) { return __uint_as_float(held << 16); }
template <int MIDDLE = 8>
__device__ __forceinline__ float middle_of(uint32_t held) {
  return fmaf(float(MIDDLE), scale_of(held), __uint_as_float(held & 0xffff0000u));
}

// Whether what is held for a group stands for numbers.
template <int BITS>
__device__ __forceinline__ bool numbers(uint32_t held) {
  return fabsf(BITS == 8 ? __uint_as_float(held) : middle_of(held)) < INFINITY;
}

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// The first product of a sum.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.0f));
}

__device__ __forceinline__ void copy_async(uint32_t to, const char* from, int unit, int bytes) {
  if (unit == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
  else if (unit == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void copy_all(uint32_t to, const char* from, int unit) {
  if (unit == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}

__device__ __forceinline__ float power_of_two(int e) {  // e in [-126, 127]
  return __uint_as_float(uint32_t(e + 127) << 23);
}

// ------------------------------------------------------------------ the work's division

// A sequence's tiles of tokens: those that any of its rows sees.
struct Tiles {
  int first, count;  // tokens from first * kTile
};

template <int TILE>
__device__ __forceinline__ Tiles tiles_of(const AttendArgs& a, const Sequence& s) {
  Tiles t;
  const int end = s.rows > 0 ? s.tokens : 0;
  const int lo = s.rows > 0 ? min(seen(a, s, 0).lo, end) : 0;
  t.first = lo / TILE;
  t.count = (end + TILE - 1) / TILE - t.first;
  if (end <= lo) t.count = 0;
  return t;
}

struct Division {
  int64_t total;
  int workers;
  __device__ __forceinline__ int64_t start(int w) const { return w * total / workers; }
  // the worker that has tile i
  __device__ __forceinline__ int owner(int64_t i) const {
    return int(((i + 1) * workers - 1) / total);
  }
};

// All tiles: a warp together.
template <int TILE>
__device__ __forceinline__ Division divide(const AttendArgs& a) {
  const int lane = threadIdx.x & 31;
  int64_t all = 0;
  for (int i = lane; i < a.batch; i += 32) all += tiles_of<TILE>(a, sequence(a, i)).count;
#pragma unroll
  for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(kFullWarp, all, o);
  Division d;
  d.total = all * a.row_tiles;
  d.workers = int(min(int64_t(a.workers), max(int64_t(1), d.total)));
  return d;
}

// ------------------------------------------------------------------ queries

// A row tile's queries as the B operand of S^T: rows lane / 4, a lane's elements as
// bytes_at() gives a key's.
template <class T>
struct Queries {
  static constexpr int kLowSums = T::kBits == 4 ? T::kBlocks : 1;
  uint32_t q[T::kDim / 16][T::kNR][T::kPieces][2];
  float unit[T::kNR][2];  // of rows 2 (lane % 4) and the next: exponent = S * unit
  float low[T::kNR][2][kLowSums];  // 4 bits: sums of q over the blocks
  Seen see[T::kNR][2];

  __device__ __forceinline__ static int element(int step, int c, int e) {
    const int block = step / T::kSteps, i = step % T::kSteps;
    const int base = block * T::kBlock + c * (T::kBlock / 4);
    if (T::kBits == 8) return base + 4 * i + e;
    if (T::kBlock == 16) return base + (e & 1) * 2 + (e >> 1);  // (0, 2), (1, 3)
    return base + 8 * (i / 2) + 2 * (i & 1) + (e & 1) * 4 + (e >> 1);
  }

  __device__ __forceinline__ void load(const AttendArgs& a, int b, int h, int tile,
                                       const Sequence& s) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int rows = a.rows * a.shared;
#pragma unroll
    for (int n = 0; n < T::kNR; ++n) {
      const int i = tile * T::kRows + n * 8 + g;
      const int r = i / a.shared, j = i - r * a.shared;
      const bool there = i < rows && r < s.rows;
      const char* from = static_cast<const char*>(a.q.data) + b * a.q.batch_stride +
                         r * a.q.row_stride + (h * a.shared + j) * a.q.head_stride;
      float most = 0.0f;
      float x[T::kDim / 16][4];
      constexpr int kRun = T::kBlock / 4;  // a lane's elements of a block lie together
#pragma unroll
      for (int k = 0; k < T::kBlocks; ++k) {
        float run[kRun];
        const int first = k * T::kBlock + c * kRun;
        if (!there) {
#pragma unroll
          for (int e = 0; e < kRun; ++e) run[e] = 0.0f;
        } else if (!a.wide_q) {
#pragma unroll
          for (int e = 0; e < kRun; ++e) run[e] = load_as_float(from, first + e, a.dt);
        } else if (a.dt == LP_F32) {
#pragma unroll
          for (int e = 0; e < kRun; e += 2) {
            const float2 v = __ldg(reinterpret_cast<const float2*>(from + (first + e) * 4));
            run[e] = v.x, run[e + 1] = v.y;
          }
        } else {
          uint2 raw[kRun / 4];
#pragma unroll
          for (int e = 0; e < kRun / 4; ++e)
            raw[e] = __ldg(reinterpret_cast<const uint2*>(from + (first + 4 * e) * 2));
#pragma unroll
          for (int e = 0; e < kRun; ++e) {
            const uint32_t w = (e & 2) ? raw[e / 4].y : raw[e / 4].x;
            const uint32_t u = (e & 1) ? w >> 16 : w & 0xffffu;
            run[e] = a.dt == LP_BF16 ? __uint_as_float(u << 16) : Elt<LP_F16>::half_bits_to_float(u);
          }
        }
#pragma unroll
        for (int i = 0; i < T::kSteps; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[k * T::kSteps + i][e] = run[element(k * T::kSteps + i, 0, e) - k * T::kBlock];
#pragma unroll
        for (int e = 0; e < kRun; ++e) most = fmaxf(most, fabsf(run[e]));
      }
      most = fmaxf(most, __shfl_xor_sync(kFullWarp, most, 1));
      most = fmaxf(most, __shfl_xor_sync(kFullWarp, most, 2));
      // to [2^14, 2^15); in two steps, a factor can be beyond 2^127
      const int up = most > 0.0f && most <= 3.4028235e38f
                         ? 14 - (int(__float_as_uint(most) >> 23) - 127) : 0;
      const float f1 = power_of_two(up / 2), f2 = power_of_two(up - up / 2);
      const float mine = a.scale / f1 / f2;
      float sums[kLowSums] = {};
#pragma unroll
      for (int t = 0; t < T::kDim / 16; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[t][e] = x[t][e] * f1 * f2;
          if (T::kBits == 4) sums[t / T::kSteps] += x[t][e];
        }
        // codes whose bits lie four higher are 16 times what they are
        if (T::kBits == 4) x[t][2] *= 0.0625f, x[t][3] *= 0.0625f;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float y = x[t][2 * p], z = x[t][2 * p + 1];
          const uint32_t top = f16_two(y, z);
          q[t][n][0][p] = top;
          if (T::kWide)
            q[t][n][T::kPieces - 1][p] = f16_two(y - Elt<LP_F16>::half_bits_to_float(top & 0xffffu),
                                                 z - Elt<LP_F16>::half_bits_to_float(top >> 16));
        }
      }
      if (T::kBits == 4) {
#pragma unroll
        for (int k = 0; k < kLowSums; ++k) {
          sums[k] += __shfl_xor_sync(kFullWarp, sums[k], 1);
          sums[k] += __shfl_xor_sync(kFullWarp, sums[k], 2);
        }
      }
      // from the lanes of a row to those that have its column of S^T
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int from_lane = (2 * c + e) * 4;
        unit[n][e] = __shfl_sync(kFullWarp, mine, from_lane);
        if (T::kBits == 4) {
#pragma unroll
          for (int k = 0; k < kLowSums; ++k)
            low[n][e][k] = __shfl_sync(kFullWarp, sums[k], from_lane);
        }
        const int row = tile * T::kRows + n * 8 + 2 * c + e;
        see[n][e] = row < rows ? seen(a, s, row / a.shared) : Seen{0, 0};
      }
    }
  }
};

// ------------------------------------------------------------------ a tile's copies

template <class T>
struct Loader {
  char* smem;         // this warp's stages
  const char* codes[2];
  const char* params[2];
  int groups, gstep;  // of a head; blocks of a group
  int b;
  int32_t next;       // the block of this lane's token of the tile after

  __device__ __forceinline__ void init(const AttendArgs& a, char* at, int sequence, int h) {
    smem = at;
    b = sequence;
    groups = a.dim / a.group;
    gstep = T::kBlocks / groups;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      codes[p] = static_cast<const char*>(a.part[p].codes) + h * a.part[p].code_head_stride;
      params[p] = static_cast<const char*>(a.part[p].params) + h * a.part[p].param_head_stride;
    }
  }
  __device__ __forceinline__ void look(const AttendArgs& a, int tile) {
    const int t = tile * T::kTile + (threadIdx.x & (T::kTile - 1));
    next = t < a.most
               ? __ldg(a.blocks + int64_t(b) * a.blocks_stride + a.per_block.quot(uint32_t(t)))
               : -1;
  }
  // Keys and values lie alike: one place for both.  ALL: every token is there.
  template <int PARTS, bool ALL>
  __device__ __forceinline__ void copies(uint32_t base, uint32_t mine, uint32_t held) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < (T::kTile * T::kChunks + 31) / 32; ++k) {
      const int idx = k * 32 + lane;
      const int token = 32 % T::kChunks == 0 ? k * (32 / T::kChunks) + lane / T::kChunks
                                             : idx / T::kChunks;
      const int piece = 32 % T::kChunks == 0 ? lane % T::kChunks : idx - token * T::kChunks;
      const uint32_t row = __shfl_sync(kFullWarp, mine, token);
      if (T::kTile * T::kChunks % 32 != 0 && token >= T::kTile) continue;
      const int64_t at = int64_t(uint64_t(row) * T::kUnit) + piece * T::kUnit;
      const uint32_t to = base + token * T::kRow +
                          swizzled<T::kRow>(piece * T::kUnit, swizzle<T::kRow>(token));
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        if (ALL) copy_all(to + p * T::kCodes, codes[p] + at, T::kUnit);
        else copy_async(to + p * T::kCodes, codes[p] + at, T::kUnit,
                        (held >> token) & 1u ? T::kUnit : 0);
      }
    }
  }
  template <int PARTS>
  __device__ __forceinline__ void param_copy(const AttendArgs& a, uint32_t base, int p,
                                             const char* from, bool there) {
    const int lane = threadIdx.x & 31;
    if (T::kTile == 32 || (lane >> 4) == p || (PARTS == 1 && lane < 16)) {
      const uint32_t at = base + 2 * T::kCodes + p * T::kParams +
                          (lane & (T::kTile - 1)) * T::kBlocks * 4;
      if (T::kBlocks % 4 == 0 && a.wide_params) {
#pragma unroll
        for (int k = 0; k < T::kBlocks; k += 4)
          if (k < groups) copy_async(at + 4 * k, from + 4 * k, 16, there ? 16 : 0);
      } else {
#pragma unroll
        for (int k = 0; k < T::kBlocks; ++k)
          if (k < groups) copy_async(at + 4 * k, from + 4 * k, 4, there ? 4 : 0);
      }
    }
  }
  // Starts the copies of a tile whose blocks are looked up; which of its tokens are there.
  // PARTS: 2, or 1 for the keys alone.
  template <int PARTS>
  __device__ __forceinline__ uint32_t start(const AttendArgs& a, int tile, int end, int stage) {
    const int lane = threadIdx.x & 31;
    const int t = tile * T::kTile + (lane & (T::kTile - 1));
    const uint32_t i = a.per_block.quot(uint32_t(t));
    int64_t slot = int64_t(next) * a.block + (t - int64_t(i) * a.block);
    const bool there = t < end && slot >= 0 && slot < a.n_slots;
    if (!there) slot = 0;
    const uint32_t held = __ballot_sync(kFullWarp, there);
    const uint32_t base = uint32_t(__cvta_generic_to_shared(smem)) + stage * T::kStage;
    if (a.code_step != 0) {
      const uint32_t mine = uint32_t(slot) * a.code_step;
      if (held == kFullWarp) {
        copies<PARTS, true>(base, mine, held);
      } else {
        copies<PARTS, false>(base, mine, held);
      }
      const int64_t at = int64_t(uint64_t(uint32_t(slot) * a.param_step) * 4);
#pragma unroll
      for (int p = 0; p < PARTS; ++p) param_copy<PARTS>(a, base, p, params[p] + at, there);
    } else {
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        const lp_cache_part& part = a.part[p];
        const uint64_t mine = reinterpret_cast<uint64_t>(
            codes[p] + slot_place(a, slot, part.code_page_stride, part.code_slot_stride));
        const uint32_t to = base + p * T::kCodes;
#pragma unroll 1
        for (int idx = lane; idx < (T::kTile * T::kChunks + 31) / 32 * 32; idx += 32) {
          const int token = idx / T::kChunks, piece = idx - token * T::kChunks;
          const uint64_t row = __shfl_sync(kFullWarp, mine, token);
          if (token < T::kTile)
            copy_async(to + token * T::kRow +
                           swizzled<T::kRow>(piece * T::kUnit, swizzle<T::kRow>(token)),
                       reinterpret_cast<const char*>(row) + piece * T::kUnit, T::kUnit,
                       (held >> token) & 1u ? T::kUnit : 0);
        }
        param_copy<PARTS>(a, base, p,
                          params[p] + slot_place(a, slot, part.param_page_stride,
                                                 part.param_slot_stride), there);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return held;
  }
};

// ------------------------------------------------------------------ scores

// A token's params, of each block of elements.
template <class T>
struct BlockParams {
  uint32_t w[T::kBlocks];
};

template <class T>
__device__ __forceinline__ BlockParams<T> block_params(const char* at, int gstep) {
  BlockParams<T> r;
  if (T::kBlocks % 4 == 0 && gstep == 1) {
#pragma unroll
    for (int k = 0; k < T::kBlocks; k += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(at + 4 * k);
      r.w[k] = v.x, r.w[(k + 1) % T::kBlocks] = v.y;
      r.w[(k + 2) % T::kBlocks] = v.z, r.w[(k + 3) % T::kBlocks] = v.w;
    }
  } else {
    int group = 0, in = 0;
#pragma unroll
    for (int k = 0; k < T::kBlocks; ++k) {
      r.w[k] = *reinterpret_cast<const uint32_t*>(at + 4 * group);
      if (++in == gstep) in = 0, ++group;
    }
  }
  return r;
}

// S^T of a tile: tokens lane / 4 (and that + 8) of each sixteen, rows 2 (lane % 4) and the
// next of each eight.
template <class T>
__device__ __forceinline__ void scores(float (&s)[T::kM][T::kNR][4], const Queries<T>& q,
                                       const char* stage, int gstep) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int f = swizzle<T::kRow>(g);
#pragma unroll
  for (int m = 0; m < T::kM; ++m) {
    const char* row = stage + (m * 16 + g) * T::kRow;
    const char* held = stage + 2 * T::kCodes + (m * 16 + g) * T::kBlocks * 4;
    const auto p0 = block_params<T>(held, gstep);
    const auto p1 = block_params<T>(held + 8 * T::kBlocks * 4, gstep);
#pragma unroll
    for (int k = 0; k < T::kBlocks; ++k) {
      const int at = k * (T::kBlock * T::kBits / 8) + c * T::kKeyBytes;
      const auto x = bytes_at<T::kKeyBytes, T::kRow>(row, at, f);
      const auto y = bytes_at<T::kKeyBytes, T::kRow>(row + 8 * T::kRow, at, f);
      float acc[T::kNR][4] = {};
#pragma unroll
      for (int i = 0; i < T::kSteps; ++i) {
        uint32_t op[4];
        if (T::kBits == 8) {
          op[0] = e4m3_two(x.w[i]), op[1] = e4m3_two(y.w[i]);
          op[2] = e4m3_two(x.w[i] >> 16), op[3] = e4m3_two(y.w[i] >> 16);
        } else if (T::kBlock == 16) {
          const uint32_t u = __byte_perm(x.w[0], 0, 0x4140), v = __byte_perm(y.w[0], 0, 0x4140);
          op[0] = codes_low(u), op[1] = codes_low(v);
          op[2] = codes_high(u), op[3] = codes_high(v);
        } else {
          const uint32_t u = i & 1 ? x.w[i / 2] >> 8 : x.w[i / 2];
          const uint32_t v = i & 1 ? y.w[i / 2] >> 8 : y.w[i / 2];
          op[0] = codes_low(u), op[1] = codes_low(v);
          op[2] = codes_high(u), op[3] = codes_high(v);
        }
#pragma unroll
        for (int n = 0; n < T::kNR; ++n)
#pragma unroll
          for (int p = T::kPieces - 1; p >= 0; --p) mma(acc[n], op, q.q[k * T::kSteps + i][n][p]);
      }
      const uint32_t h0 = p0.w[k], h1 = p1.w[k];
#pragma unroll
      for (int n = 0; n < T::kNR; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t h = e < 2 ? h0 : h1;
          const float before = k == 0 ? 0.0f : s[m][n][e];
          if (T::kBits == 8) {
            s[m][n][e] = fmaf(acc[n][e], __uint_as_float(h), before);
          } else {
            const float lows = fmaf(middle_of(h), q.low[n][e & 1][k], before);
            s[m][n][e] = fmaf(acc[n][e], scale_of(h), lows);
          }
        }
    }
  }
}

// ------------------------------------------------------------------ a unit's sums

template <class T>
struct Sums {
  static constexpr int kLows = T::kBits == 4 ? T::kBlocks : 1;
  // O^T: elements k * kBlock + (lane / 4) * kValues + 2 v (entries 0, 1) and the next
  // (entries 2, 3), rows 2 (lane % 4) and the next
  float o[T::kBlocks][T::kValues / 2][T::kNR][4];
  float low[kLows][T::kNR][2];  // this lane's tokens' share
  float mass[T::kNR][2];        // of this lane's tokens
  float top[T::kNR][2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < T::kNR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mass[n][e] = 0.0f, top[n][e] = -INFINITY;
#pragma unroll
        for (int k = 0; k < kLows; ++k) low[k][n][e] = 0.0f;
      }
#pragma unroll
    for (int k = 0; k < T::kBlocks; ++k)
#pragma unroll
      for (int v = 0; v < T::kValues / 2; ++v)
#pragma unroll
        for (int n = 0; n < T::kNR; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[k][v][n][e] = 0.0f;
  }

  // NaN codes of values of tokens that some rows do not see: those that see them get NaN,
  // and the codes become 0, which adds nothing to the others.
  __device__ __forceinline__ void split_nan(const Queries<T>& q, char* values, int t0, uint32_t held);
  // The same for groups whose params are no numbers.
  __device__ __forceinline__ void split_params(const Queries<T>& q, char* params, int t0,
                                               uint32_t held, int gstep);

  __device__ __forceinline__ void add(const Queries<T>& q, char* stage, int t0, uint32_t held,
                                      int gstep, bool all_seen) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    float s[T::kM][T::kNR][4];
    scores<T>(s, q, stage, gstep);
    // params of this lane's tokens, and the largest scale of each as an exponent
    char* held_at = stage + 2 * T::kCodes + T::kParams;
    float large[T::kM][2];
    const auto look = [&] {
      uint32_t all = 0;
#pragma unroll
      for (int m = 0; m < T::kM; ++m)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const auto p = block_params<T>(held_at + (m * 16 + 8 * u + g) * T::kBlocks * 4, gstep);
          uint32_t most = T::kBits == 8 ? p.w[0] : p.w[0] << 16;
#pragma unroll
          for (int k = 1; k < T::kBlocks; ++k)
            most = max(most, T::kBits == 8 ? p.w[k] : p.w[k] << 16);
          large[m][u] = float(max(int((most >> 23) & 255u) - 127, kLeastScale));
          all = max(all, most);
        }
      return all < 0x7f800000u;
    };
    bool fine = look();
    if (T::kBits == 4 && !all_seen)
      for (int i = lane; i < T::kTile * T::kBlocks; i += 32)
        fine = fine && numbers<T::kBits>(reinterpret_cast<const uint32_t*>(held_at)[i]);
    // a weight of 0 does not take away an infinity; and an infinite scale is nobody's largest
    if (!__all_sync(kFullWarp, fine)) {
      split_params(q, held_at, t0, held, gstep);
      look();
    }
    float now[T::kNR][2];
#pragma unroll
    for (int n = 0; n < T::kNR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) now[n][e] = top[n][e];
#pragma unroll
    for (int m = 0; m < T::kM; ++m)
#pragma unroll
      for (int n = 0; n < T::kNR; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float& x = s[m][n][e];
          x *= q.unit[n][e & 1];
          if (!all_seen) {
            const int i = m * 16 + 8 * (e >> 1) + g;
            const Seen& v = q.see[n][e & 1];
            if (t0 + i < v.lo || t0 + i >= v.end || !((held >> i) & 1u)) x = -INFINITY;
          }
          now[n][e & 1] = fmaxf(now[n][e & 1], x + large[m][e >> 1]);
        }
    bool grew = false;
#pragma unroll
    for (int n = 0; n < T::kNR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o *= 2)
          now[n][e] = fmaxf(now[n][e], __shfl_xor_sync(kFullWarp, now[n][e], o));
        grew = grew || now[n][e] != top[n][e];
      }
    float from[T::kNR][2];
#pragma unroll
    for (int n = 0; n < T::kNR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) from[n][e] = now[n][e] == -INFINITY ? 0.0f : now[n][e];
    if (__any_sync(kFullWarp, grew)) {
#pragma unroll
      for (int n = 0; n < T::kNR; ++n) {
        const float f0 = ex2(top[n][0] - from[n][0]), f1 = ex2(top[n][1] - from[n][1]);
        top[n][0] = now[n][0], top[n][1] = now[n][1];
        mass[n][0] *= f0, mass[n][1] *= f1;
        if (T::kBits == 4) {
#pragma unroll
          for (int k = 0; k < kLows; ++k) low[k][n][0] *= f0, low[k][n][1] *= f1;
        }
#pragma unroll
        for (int k = 0; k < T::kBlocks; ++k)
#pragma unroll
          for (int v = 0; v < T::kValues / 2; ++v)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[k][v][n][e] *= e & 1 ? f1 : f0;
      }
    }
    float lifted[T::kNR][2];
#pragma unroll
    for (int n = 0; n < T::kNR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) lifted[n][e] = from[n][e] - kLift;
#pragma unroll
    for (int m = 0; m < T::kM; ++m)
#pragma unroll
      for (int n = 0; n < T::kNR; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[m][n][e] = ex2(s[m][n][e] - lifted[n][e & 1]);
          mass[n][e & 1] += s[m][n][e];
        }
    char* values = stage + T::kCodes;
    if (T::kBits == 8 && !all_seen) {
      bool bad = false;
      for (int i = lane * 4; i < T::kCodes; i += 128) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(values + i);
        bad = bad || (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
      }
      if (__any_sync(kFullWarp, bad)) split_nan(q, values, t0, held);
    }
    const int fa = swizzle<T::kRow>(2 * c), fb = swizzle<T::kRow>(2 * c + 1);
#pragma unroll
    for (int m = 0; m < T::kM; ++m) {
      const char* row = values + (m * 16 + 2 * c) * T::kRow;
      const auto p0 = block_params<T>(held_at + (m * 16 + g) * T::kBlocks * 4, gstep);
      const auto p1 = block_params<T>(held_at + (m * 16 + 8 + g) * T::kBlocks * 4, gstep);
#pragma unroll
      for (int k = 0; k < T::kBlocks; ++k) {
        // P s_g, rounded, as the B operand
        const uint32_t h0 = p0.w[k], h1 = p1.w[k];
        const float s0 = T::kBits == 8 ? __uint_as_float(h0) : scale_of(h0);
        const float s1 = T::kBits == 8 ? __uint_as_float(h1) : scale_of(h1);
        uint32_t p[T::kNR][T::kPieces][2];
#pragma unroll
        for (int n = 0; n < T::kNR; ++n) {
          const float* e = s[m][n];
          const float w0 = e[0] * s0, w1 = e[1] * s0, w2 = e[2] * s1, w3 = e[3] * s1;
          const uint32_t a = f16_two(w0, w1), b = f16_two(w2, w3);
          p[n][0][0] = transposed(a), p[n][0][1] = transposed(b);
          if (T::kWide) {
            p[n][T::kPieces - 1][0] =
                transposed(f16_two(w0 - Elt<LP_F16>::half_bits_to_float(a & 0xffffu),
                                   w1 - Elt<LP_F16>::half_bits_to_float(a >> 16)));
            p[n][T::kPieces - 1][1] =
                transposed(f16_two(w2 - Elt<LP_F16>::half_bits_to_float(b & 0xffffu),
                                   w3 - Elt<LP_F16>::half_bits_to_float(b >> 16)));
          }
          if (T::kBits == 4) {
            // (less 8 and less 7, in turn: codes' mean is between, and what all have in common
            // would grow with the tokens, where their sum does as the root)
            const float l0 = middle_of<8>(h0), l1 = middle_of<7>(h1);
            low[k % kLows][n][0] = fmaf(e[0], l0, fmaf(e[2], l1, low[k % kLows][n][0]));
            low[k % kLows][n][1] = fmaf(e[1], l0, fmaf(e[3], l1, low[k % kLows][n][1]));
          }
        }
        const int at = k * (T::kBlock * T::kBits / 8) + g * T::kValueBytes;
        const auto va = bytes_at<T::kValueBytes, T::kRow>(row, at, fa);
        const auto vb = bytes_at<T::kValueBytes, T::kRow>(row + T::kRow, at, fb);
        const auto vc = bytes_at<T::kValueBytes, T::kRow>(row + 8 * T::kRow, at, fa);
        const auto vd = bytes_at<T::kValueBytes, T::kRow>(row + 9 * T::kRow, at, fb);
#pragma unroll
        for (int v = 0; v < T::kValues / 2; ++v) {
          uint32_t op[4];
          if (T::kBits == 8) {
            const int sel = v & 1 ? 0x7362 : 0x5140;
            const uint32_t x = __byte_perm(va.w[v / 2], vb.w[v / 2], sel);
            const uint32_t y = __byte_perm(vc.w[v / 2], vd.w[v / 2], sel);
            op[0] = e4m3_two(x), op[1] = e4m3_two(x >> 16);
            op[2] = e4m3_two(y), op[3] = e4m3_two(y >> 16);
          } else {
            const int i = v & 3, sel = i | (4 + i) << 8;
            const uint32_t x = __byte_perm(va.w[v / 4], vb.w[v / 4], sel);
            const uint32_t y = __byte_perm(vc.w[v / 4], vd.w[v / 4], sel);
            op[0] = codes_low(x), op[1] = codes_high(x);
            op[2] = codes_low<7>(y), op[3] = codes_high<7>(y);
          }
#pragma unroll
          for (int n = 0; n < T::kNR; ++n) {  // (added outside, where a sum is rounded, not cut)
            float t[4];
            mma_first(t, op, p[n][T::kPieces - 1]);
            if (T::kWide) mma(t, op, p[n][0]);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[k][v][n][e] += t[e];
          }
        }
      }
    }
  }

  // Sums over the lanes that share a row; O^T as sums of weight times value.
  __device__ __forceinline__ void join() {
#pragma unroll
    for (int n = 0; n < T::kNR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) {
          mass[n][e] += __shfl_xor_sync(kFullWarp, mass[n][e], x);
          if (T::kBits == 4) {
#pragma unroll
            for (int k = 0; k < kLows; ++k)
              low[k][n][e] += __shfl_xor_sync(kFullWarp, low[k][n][e], x);
          }
        }
      }
    if (T::kBits == 4) {
#pragma unroll
      for (int k = 0; k < T::kBlocks; ++k)
#pragma unroll
        for (int v = 0; v < T::kValues / 2; ++v)
#pragma unroll
          for (int n = 0; n < T::kNR; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[k][v][n][e] = fmaf(o[k][v][n][e], e < 2 ? 1.0f : 0.0625f,
                                   low[k % kLows][n][e & 1]);
    }
  }
};

template <class T>
__device__ __forceinline__ void Sums<T>::split_nan(const Queries<T>& q, char* values, int t0,
                                                uint32_t held) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  for (int i = 0; i < T::kTile; ++i) {
    const char* row = values + i * T::kRow;
    const int f = swizzle<T::kRow>(i);
#pragma unroll
    for (int k = 0; k < T::kBlocks; ++k)
#pragma unroll
      for (int j = 0; j < T::kValues; ++j) {
        const int at = k * T::kBlock + g * T::kValues + j;
        if ((row[swizzled<T::kRow>(at, f)] & 0x7f) != 0x7f) continue;
#pragma unroll
        for (int n = 0; n < T::kNR; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const Seen& v = q.see[n][e];
            if (t0 + i >= v.lo && t0 + i < v.end && ((held >> i) & 1u))
              o[k][j / 2][n][2 * (j & 1) + e] = __uint_as_float(0x7fc00000u);
          }
      }
  }
  __syncwarp();
  for (int i = lane; i < T::kCodes; i += 32)
    if ((values[i] & 0x7f) == 0x7f) values[i] = 0;
  __syncwarp();
}

template <class T>
__device__ __forceinline__ void Sums<T>::split_params(const Queries<T>& q, char* params, int t0,
                                                      uint32_t held, int gstep) {
  const int lane = threadIdx.x & 31;
  for (int i = 0; i < T::kTile; ++i) {
    const auto p = block_params<T>(params + i * T::kBlocks * 4, gstep);
#pragma unroll
    for (int k = 0; k < T::kBlocks; ++k) {
      if (numbers<T::kBits>(p.w[k])) continue;
#pragma unroll
      for (int n = 0; n < T::kNR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const Seen& v = q.see[n][e];
          if (t0 + i < v.lo || t0 + i >= v.end || !((held >> i) & 1u)) continue;
#pragma unroll
          for (int j = 0; j < T::kValues / 2; ++j)
            o[k][j][n][e] = o[k][j][n][2 + e] = __uint_as_float(0x7fc00000u);
        }
    }
  }
  __syncwarp();
  for (int i = lane; i < T::kTile * T::kBlocks; i += 32) {
    uint32_t& w = reinterpret_cast<uint32_t*>(params)[i];  // (some are nobody's)
    if (!numbers<T::kBits>(w)) w = 0;
  }
  __syncwarp();
}

// ------------------------------------------------------------------ kernels

constexpr int kMostTeamWarps = 4;

// One worker's range of tiles, unit by unit.
template <class T>
__global__ void __launch_bounds__(kMostTeamWarps * 32, T::kResident)
    attend_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ __align__(128) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int in_team = warp % a.team;
  // neighbours have the same tokens' next heads: what lies together is read together
  const int index = blockIdx.x * (blockDim.x / 32 / a.team) + warp / a.team;
  const int worker = index / a.head_groups, group = index - worker * a.head_groups;
  // the calls before may still read what this one writes
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Division d = divide<T::kTile>(a);
  if (d.total == 0 || worker >= d.workers) return;
  const int64_t begin = d.start(worker), stop = d.start(worker + 1);
  const int units = a.row_tiles;
  int64_t base = 0;  // tiles before sequence b
  int b = 0;
  {  // the sequence that tile `begin` is of
    int64_t sum = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      const int64_t n = b0 + lane < a.batch
                            ? int64_t(tiles_of<T::kTile>(a, sequence(a, b0 + lane)).count) * units : 0;
      int64_t incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(kFullWarp, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t over = __ballot_sync(kFullWarp, sum + incl > begin);
      if (over != 0) {
        const int i = __ffs(over) - 1;
        b = b0 + i;
        base = sum + __shfl_sync(kFullWarp, incl - n, i);
        break;
      }
      sum += __shfl_sync(kFullWarp, incl, 31);
    }
  }
  for (int64_t at = begin; at < stop;) {
    const Sequence s = sequence(a, b);
    const Tiles tiles = tiles_of<T::kTile>(a, s);
    if (tiles.count == 0 || at >= base + int64_t(tiles.count) * units) {
      base += int64_t(tiles.count) * units;
      ++b;
      continue;
    }
    const int unit = int((at - base) / tiles.count);
    const int tile = int(at - base - int64_t(unit) * tiles.count);
    const int count = int(min(int64_t(tiles.count - tile), stop - at));
    const int rt = unit, h = group * a.team + in_team;
    // tiles that a row of this tile of rows sees
    const int r0 = rt * T::kRows / a.shared;
    const int r1 = min(rt * T::kRows + T::kRows - 1, a.rows * a.shared - 1) / a.shared;
    const Seen lowest = seen(a, s, min(r0, s.rows - 1)), highest = seen(a, s, min(r1, s.rows - 1));
    const int first = max(tiles.first + tile, r0 < s.rows ? lowest.lo / T::kTile : INT32_MAX);
    const int last = min(tiles.first + tile + count, (highest.end + T::kTile - 1) / T::kTile);
    // tokens that all of them see
    const int from = highest.lo, until = r1 < s.rows ? lowest.end : 0;

    Loader<T> load;
    load.init(a, smem + warp * (T::kStages * T::kStage), b, h);
    uint32_t held = 0;
    if (first < last) {
      load.look(a, first);
      held = load.template start<2>(a, first, highest.end, 0);
      if (first + 1 < last) load.look(a, first + 1);
    }
    Queries<T> q;
    q.load(a, b, h, rt, s);
    Sums<T> sums;
    sums.clear();
    for (int i = first; i < last; ++i) {
      uint32_t held_next = 0;
      const int stage = (i - first) & 1;
      if (i + 1 < last) {
        held_next = load.template start<2>(a, i + 1, highest.end, stage ^ 1);
        if (i + 2 < last) load.look(a, i + 2);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncwarp();
      const int t0 = i * T::kTile;
      const bool all_seen = t0 >= from && t0 + T::kTile <= until &&
                            (T::kTile == 32 ? held : held | 0xffff0000u) == kFullWarp;
      sums.add(q, load.smem + stage * T::kStage, t0, held, load.gstep, all_seen);
      __syncwarp();
      held = held_next;
    }
    sums.join();
    const bool whole = count == tiles.count;
    const int part = at == begin ? 0 : 1;
    if (tile == 0 && in_team == 0 && group == 0 && lane == 0)
      a.shares[int64_t(b) * a.row_tiles + rt] =
          make_int4(worker, whole ? worker : d.owner(at + tiles.count - 1), part, 0);
    const int64_t slot = ((int64_t(worker) * a.head_groups + group) * 2 + part) * a.team + in_team;
#pragma unroll
    for (int n = 0; n < T::kNR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = n * 8 + 2 * c + e;  // of the tile's rows
        const int row = rt * T::kRows + i;
        if (row >= a.rows * a.shared) continue;
        const int r = row / a.shared, j = h * a.shared + row - r * a.shared;
        const float mass = sums.mass[n][e];
        if (!whole) {
          float* to = a.sums + (slot * T::kRows + i) * T::kDim + g * T::kValues;
#pragma unroll
          for (int k = 0; k < T::kBlocks; ++k)
#pragma unroll
            for (int v = 0; v < T::kValues / 2; ++v)
              *reinterpret_cast<float2*>(to + k * T::kBlock + 2 * v) =
                  make_float2(sums.o[k][v][n][e], sums.o[k][v][n][2 + e]);
          if (g == 0) a.tops[slot * T::kRows + i] = make_float2(sums.top[n][e], mass);
          continue;
        }
        const float inv = mass == 0.0f ? 0.0f : 1.0f / mass;
        char* to = static_cast<char*>(a.out.data) + b * a.out.batch_stride +
                   r * a.out.row_stride + j * a.out.head_stride;
#pragma unroll
        for (int k = 0; k < T::kBlocks; ++k)
#pragma unroll
          for (int v = 0; v < T::kValues / 2; ++v) {
            const float x = mass == 0.0f ? 0.0f : sums.o[k][v][n][e] * inv;
            const float y = mass == 0.0f ? 0.0f : sums.o[k][v][n][2 + e] * inv;
            const int d0 = k * T::kBlock + g * T::kValues + 2 * v;
            store_float(to, d0, x, a.dt);
            store_float(to, d0 + 1, y, a.dt);
          }
        if (a.lse != nullptr && g == 0)
          a.lse[(int64_t(b) * a.rows + r) * (a.heads * a.shared) + j] =
              mass == 0.0f ? -INFINITY : sums.top[n][e] - kLift + log2f(mass);
      }
    at += count;
  }
}

// Joins what several workers have of a unit: a block a row of a head.  Rows of sequences
// without tiles become zeros.
constexpr int kJoinWarps = 8;
constexpr int kJoinHeld = kSms * kMostWarps;  // workers, at most

template <int TILE, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32)
    attend_join_kernel(const __grid_constant__ AttendArgs a) {
  __shared__ float acc[kJoinWarps][256], factors[kJoinHeld];
  __shared__ float most[kJoinWarps], masses[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_head = a.rows * a.shared;
  const int row = blockIdx.x % per_head;
  const int h = blockIdx.x / per_head % a.heads, b = blockIdx.x / per_head / a.heads;
  const int rt = row / ROWS;
  const int r = row / a.shared, j = h * a.shared + row - r * a.shared;
  char* to = static_cast<char*>(a.out.data) + b * a.out.batch_stride + r * a.out.row_stride +
             j * a.out.head_stride;
  float* lse = a.lse != nullptr ? a.lse + (int64_t(b) * a.rows + r) * (a.heads * a.shared) + j
                                : nullptr;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int4 share = a.shares[int64_t(b) * a.row_tiles + rt];  // of anything, without tiles
  if (tiles_of<TILE>(a, sequence(a, b)).count == 0) {
    for (int i = threadIdx.x; i < a.dim; i += blockDim.x) store_float(to, i, 0.0f, a.dt);
    if (lse != nullptr && threadIdx.x == 0) *lse = -INFINITY;
    return;
  }
  const int w0 = share.x, w1 = share.y, inside = share.z;
  if (w0 == w1) return;  // written whole
  const int n = w1 - w0 + 1;
  const auto slot = [&](int i) {
    return (((int64_t(w0 + i) * a.head_groups + h / a.team) * 2 + (i == 0 ? inside : 0)) * a.team +
            h % a.team) * ROWS + row % ROWS;
  };
  float top = -INFINITY;
  for (int i = threadIdx.x; i < n; i += blockDim.x) top = fmaxf(top, a.tops[slot(i)].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullWarp, top, o));
  if (lane == 0) most[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) top = fmaxf(top, most[i]);
  const float from = top == -INFINITY ? 0.0f : top;
  float mass = 0.0f;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const float2 t = a.tops[slot(i)];
    const float f = ex2(t.x - from);
    factors[i] = f;
    mass = fmaf(f, t.y, mass);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) mass += __shfl_xor_sync(kFullWarp, mass, o);
  if (lane == 0) masses[warp] = mass;
  __syncthreads();
  float sum[8] = {};  // elements lane * 2 + 64 i and the next
#pragma unroll 8
  for (int k = warp; k < n; k += kJoinWarps) {
    const float* p = a.sums + slot(k) * a.dim + lane * 2;
    const float f = factors[k];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (64 * i + lane * 2 < a.dim) {
        const float2 x = *reinterpret_cast<const float2*>(p + 64 * i);
        sum[2 * i] = fmaf(f, x.x, sum[2 * i]), sum[2 * i + 1] = fmaf(f, x.y, sum[2 * i + 1]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc[warp][lane * 2 + 64 * i] = sum[2 * i], acc[warp][lane * 2 + 64 * i + 1] = sum[2 * i + 1];
  __syncthreads();
  mass = 0.0f;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) mass += masses[i];
  for (int i = threadIdx.x; i < a.dim; i += blockDim.x) {
    float x = 0.0f;
#pragma unroll
    for (int k = 0; k < kJoinWarps; ++k) x += acc[k][i];
    store_float(to, i, mass == 0.0f ? 0.0f : x / mass, a.dt);
  }
  if (lse != nullptr && threadIdx.x == 0)
    *lse = mass == 0.0f ? -INFINITY : top - kLift + log2f(mass);
}

// weights[b, h, t] += the sum over a head's rows of 2^(x - lse): the scores once more, from
// the keys alone.  A tile belongs to one warp, whatever the rows: no sum has two writers.
template <class T>
__global__ void __launch_bounds__(kMostTeamWarps * 32, T::kResident)
    weights_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ __align__(128) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int in_team = warp % a.team;
  const int64_t worker = int64_t(blockIdx.x) * (blockDim.x / 32 / a.team) + warp / a.team;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int64_t total = 0;
  for (int b = lane; b < a.batch; b += 32) total += tiles_of<T::kTile>(a, sequence(a, b)).count;
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(kFullWarp, total, o);
  total *= a.head_groups;
  const int64_t begin = worker * total / a.workers, stop = (worker + 1) * total / a.workers;
  int64_t base = 0;
  int b = 0;
  for (int64_t at = begin; at < stop;) {
    const Sequence s = sequence(a, b);
    const Tiles tiles = tiles_of<T::kTile>(a, s);
    if (at >= base + int64_t(tiles.count) * a.head_groups) {
      base += int64_t(tiles.count) * a.head_groups;
      ++b;
      continue;
    }
    const int hg = int((at - base) / tiles.count);
    const int tile = int(at - base - int64_t(hg) * tiles.count);
    const int count = int(min(int64_t(tiles.count - tile), stop - at));
    const int h = hg * a.team + in_team;
    Loader<T> load;
    load.init(a, smem + warp * (T::kStages * T::kStage), b, h);
    Queries<T> q;
    float lse[T::kNR][2];
    int loaded = -1;
    load.look(a, tiles.first + tile);
    uint32_t held = load.template start<1>(a, tiles.first + tile, s.tokens, 0);
    for (int i = 0; i < count; ++i) {
      uint32_t held_next = 0;
      if (i + 1 < count) {
        load.look(a, tiles.first + tile + i + 1);
        held_next = load.template start<1>(a, tiles.first + tile + i + 1, s.tokens, (i + 1) & 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncwarp();
      const int t0 = (tiles.first + tile + i) * T::kTile;
      float sum[T::kM][2] = {};
      for (int rt = 0; rt < a.row_tiles; ++rt) {
        if (loaded != rt) {
          loaded = rt;
          q.load(a, b, h, rt, s);
#pragma unroll
          for (int n = 0; n < T::kNR; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int row = rt * T::kRows + n * 8 + 2 * c + e, r = row / a.shared;
              lse[n][e] = r < s.rows && row < a.rows * a.shared
                              ? a.lse[(int64_t(b) * a.rows + r) * (a.heads * a.shared) +
                                      h * a.shared + row - r * a.shared]
                              : -INFINITY;
            }
        }
        float x[T::kM][T::kNR][4];
        scores<T>(x, q, load.smem + (i & 1) * T::kStage, load.gstep);
#pragma unroll
        for (int m = 0; m < T::kM; ++m)
#pragma unroll
          for (int n = 0; n < T::kNR; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const Seen& v = q.see[n][e & 1];
              const int t = t0 + m * 16 + 8 * (e >> 1) + g;
              if (t >= v.lo && t < v.end && lse[n][e & 1] != -INFINITY)
                sum[m][e >> 1] += ex2(x[m][n][e] * q.unit[n][e & 1] - lse[n][e & 1]);
            }
      }
#pragma unroll
      for (int m = 0; m < T::kM; ++m)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float x = sum[m][u];
          x += __shfl_xor_sync(kFullWarp, x, 1);
          x += __shfl_xor_sync(kFullWarp, x, 2);
          const int k = m * 16 + 8 * u + g;
          if (c == 0 && ((held >> k) & 1u)) {
            float* w = a.weights + b * a.weights_batch + h * a.weights_head + t0 + k;
            *w += x;
          }
        }
      __syncwarp();
      held = held_next;
    }
    at += count;
  }
}

// ------------------------------------------------------------------ launches

inline cudaError_t launch_after(void (*kernel)(AttendArgs), dim3 grid, dim3 block, size_t smem,
                                cudaStream_t stream, const AttendArgs& a) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Blocks of `warps` warps on all SMs, as registers and shared memory allow, up to kMostWarps
// warps an SM; asked for once a device, with the setting of the shared memory that a launch
// may take.
template <class T>
cudaError_t prepare_kernel(void (*kernel)(AttendArgs), int warps, PerDevice<5>& known,
                           int* blocks) {
  std::atomic<int>* held = known.at(warps);
  if (held != nullptr && (*blocks = held->load(std::memory_order_acquire)) > 0) return cudaSuccess;
  // the largest that any call asks for, so that no order of calls makes it less
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kMostTeamWarps * T::kStages * T::kStage);
  if (e != cudaSuccess) return e;
  int n = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, warps * 32,
                                                    warps * T::kStages * T::kStage);
  if (e != cudaSuccess) return e;
  *blocks = kSms * max(1, min(n, kMostWarps / warps));
  if (held != nullptr) held->store(*blocks, std::memory_order_release);
  return cudaSuccess;
}

template <class T>
cudaError_t attend_with(AttendArgs a, cudaStream_t stream) {
  static PerDevice<5> known, known_weights;
  const int teams = a.team >= 3 ? 1 : 4 / a.team, warps = a.team * teams;
  const size_t smem = size_t(warps) * T::kStages * T::kStage;
  a.row_tiles = (a.rows * a.shared + T::kRows - 1) / T::kRows;
  int blocks = 0;
  cudaError_t e = cudaSuccess;
  if (!a.weights_only) {
    e = prepare_kernel<T>(attend_kernel<T>, warps, known, &blocks);
    if (e != cudaSuccess) return e;
    // every head group has the same number of workers
    if (blocks * teams < a.head_groups) blocks = (a.head_groups + teams - 1) / teams;
    a.workers = blocks * teams / a.head_groups;
    e = launch_after(attend_kernel<T>, dim3(blocks), dim3(warps * 32), smem, stream, a);
    if (e != cudaSuccess) return e;
    const int64_t rows = int64_t(a.batch) * a.heads * a.rows * a.shared;
    e = launch_after(attend_join_kernel<T::kTile, T::kRows>, dim3(unsigned(rows)),
                     dim3(kJoinWarps * 32), 0, stream, a);
  }
  if (e != cudaSuccess || a.weights == nullptr) return e;
  e = prepare_kernel<T>(weights_kernel<T>, warps, known_weights, &blocks);
  if (e != cudaSuccess) return e;
  a.workers = blocks * teams;
  return launch_after(weights_kernel<T>, dim3(blocks), dim3(warps * 32), smem, stream, a);
}

// The largest block of elements that a group holds whole, of those that there are kernels for.
template <int BITS, bool WIDE, int NR>
cudaError_t attend_mma(const AttendArgs& a, int block, cudaStream_t stream) {
#define LP_CASE(D, B) \
  if (a.dim == D && block == B) return attend_with<Shape<BITS, D, B, WIDE, NR>>(a, stream);
  LP_CASE(64, 64) LP_CASE(64, 32) LP_CASE(64, 16)
  LP_CASE(80, 16)
  LP_CASE(96, 32) LP_CASE(96, 16)
  LP_CASE(128, 128) LP_CASE(128, 32) LP_CASE(128, 16)
  LP_CASE(192, 64) LP_CASE(192, 32) LP_CASE(192, 16)
  LP_CASE(256, 128) LP_CASE(256, 32) LP_CASE(256, 16)
#undef LP_CASE
  return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace lp
