// attend_chunk.cu -- attention of many queries at once over a cache of 8 bits with one scale
// a head: a prompt's chunk over what the cache holds of it, on the 5th-generation tensor cores.
//
// A block has 2 x 128 queries of one head of the cache (its query heads side by side) and goes
// through the tokens in tiles of 128.  Codes become fp16 of the same value on their way to
// shared memory; the scales stay outside, as in attend_mma.cuh:
//   S = Q K^T   from shared memory, 128 x 128 in tensor memory
//   P = 2^(s_k S unit - R) s_v, fp16, over S's place in tensor memory (two pieces, for fp16)
//   O += P V    P from tensor memory, V from shared memory
// A tensor core cuts sums toward zero, 2^-26 of them at each product: 1.3e-4 over 65536 tokens, in
// two pieces.  Every kRun tiles O is added to what is kept outside (in L2), in 32 bits with
// rounding, and begins anew: 8e-6, 4 us each.
// R, which exponents are taken against, is the largest of x + floor(log2 s_v) some time ago: O
// is scaled only when that grew by more than 2^kSlack, so P stays below 2^(kLift + kSlack + 1) = 2^15.
//
// Four roles, by warps: the two 128s of queries take turns, so that one's products run while
// the other's exponentials do.
//   0-3, 4-7   a thread a query: exponents, P, the sums
//   8-11       codes to fp16, two tiles ahead
//   12         issues the products
// Measured: 1024 queries of 32 heads over 16384 tokens, in a graph: 528 us, 504 TFLOP/s, 26% of
// the tensor pipe; by m16n8k16 1447.  What bounds it is the softmax's way out of tensor memory
// and back: 6.0 thousand cycles of the 7.5 thousand that a tile takes (a pair's two loads, 128
// exponents, the stores); the products are 2.  One block an SM, of 13 warps with 128 registers;
// with the softmax over 16 warps 567 to 695 us, with registers moved to it 803, with 12 warps of
// 168 registers 584 to 642.  fp16 takes P in two pieces, 828 us; heads of 64 take 445.
// (One piece rounds P to 11 bits, an eighth of a bf16 result's step, which is 1.65e-3 off in norm
// by its own rounding alone and 1.66e-3 so.)
//
// Every wait is bounded, by tries and not by a clock, which goes on while the kernel is off the
// GPU.  Where one runs out all roles stop, the products that were begun end, and the block's
// queries that take part become NaN, their logs of sums too, and so the weights that they add.
#include <algorithm>

#include "attend.cuh"

namespace lp {
namespace {

constexpr int kTile = 128;     // tokens
constexpr int kThreads = 13 * 32;
constexpr float kLift = 8.0f;
constexpr float kSlack = 6.0f;
constexpr int kLeastScale = -60;
constexpr int kRun = 64;       // tiles that are added up in tensor memory
constexpr uint32_t kPatience = 1u << 21;  // tries of a wait, of 1.5 us: 3 s in all

struct alignas(1024) Shared {
  // each half of 64 elements: rows of 128 bytes, their 16-byte pieces permuted by row % 8
  char q[2][2 * kTile * 128];
  char k[2][2 * kTile * 128];
  char v[2][2 * kTile * 128];
  float scales[4][3][kTile];  // keys', values', and the values' as exponents
  uint32_t held[4][4];  // bits of the tile's tokens that are there
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_done[2], drained;
#ifdef LP_TEST_CHUNK_TIMEOUT
  uint64_t never;
#endif
  const char* rows[2][2][kTile];  // of codes: [buffer][keys, values][token]
  // what is no number in tokens that some queries do not see is taken out of the products, and
  // noted at the end for those that do: a bit a query, of each element and of all
  uint32_t nan[kTile][8], nan_all[8];
  uint32_t tmem;
  int failed, nan_hidden;
};

__device__ __forceinline__ uint32_t at(const void* p) {
  return uint32_t(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void bar_init(uint64_t* b, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(at(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(at(b)) : "memory");
}
// False where the wait runs out, or another's did.
__device__ __forceinline__ bool bar_wait(Shared& s, uint64_t* b, uint32_t phase,
                                         uint32_t tries = kPatience) {
  for (uint32_t i = 0; i < tries; ++i) {
    uint32_t done;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(done) : "r"(at(b)), "r"(phase) : "memory");
    if (done) return true;
    if ((i & 255u) == 255u && *static_cast<volatile int*>(&s.failed) != 0) return false;
  }
  *static_cast<volatile int*>(&s.failed) = 1;
  return false;
}

// Whether it holds for all of the 128 threads that meet here.
__device__ __forceinline__ bool all_of_128(bool x) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.and.pred q, 1, 128, p; "
      "selp.u32 %0, 1, 0, q; }" : "=r"(r) : "r"(uint32_t(x)) : "memory");
  return r != 0;
}

// Shared-memory operands: 128-byte swizzle; `leading` and `stride` in bytes.
__device__ __forceinline__ uint64_t operand(const void* p, uint32_t leading, uint32_t stride) {
  return uint64_t((at(p) & 0x3ffffu) >> 4) | uint64_t(leading >> 4) << 16 |
         uint64_t(stride >> 4) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}
// fp16 products into fp32; `turned`: B's contraction runs across its rows.
__host__ __device__ constexpr uint32_t instruction(int m, int n, bool turned) {
  return (1u << 4) | (turned ? 1u << 16 : 0u) | uint32_t(n / 8) << 17 | uint32_t(m / 16) << 24;
}
__device__ __forceinline__ void mma_shared(uint32_t d, uint64_t a, uint64_t b, uint32_t what,
                                           bool add) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a), "l"(b),
      "r"(what), "r"(uint32_t(add))
      : "memory");
}
__device__ __forceinline__ void mma_tensor(uint32_t d, uint32_t a, uint64_t b, uint32_t what,
                                           bool add) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a), "l"(b),
      "r"(what), "r"(uint32_t(add))
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(at(b))
               : "memory");
}

#define LP_R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), \
                    "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define LP_W8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), \
                    "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])

// 32 columns of this thread's row.
__device__ __forceinline__ void tensor_load(uint32_t (&x)[32], uint32_t from) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : LP_R8(x, 0), LP_R8(x, 8), LP_R8(x, 16), LP_R8(x, 24) : "r"(from));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tensor_store(uint32_t to, const uint32_t (&x)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::LP_W8(x, 0),
      LP_W8(x, 8), LP_W8(x, 16), LP_W8(x, 24), "r"(to)
      : "memory");
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  return uint64_t(__float_as_uint(a)) | uint64_t(__float_as_uint(b)) << 32;
}
__device__ __forceinline__ float lower(uint64_t v) { return __uint_as_float(uint32_t(v)); }
__device__ __forceinline__ float upper(uint64_t v) { return __uint_as_float(uint32_t(v >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t halves(float low, float high) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(high), "f"(low));
  return r;
}

// 16 codes as fp16, two pieces of a row.
__device__ __forceinline__ void put_codes(char* half, int row, int piece, const uint4& c) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * i]) : "h"(uint16_t(w[i])));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * i + 1]) : "h"(uint16_t(w[i] >> 16)));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<uint4*>(half + row * 128 + (((piece * 2 + i) ^ (row & 7)) << 4)) =
        make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
}

__device__ __forceinline__ bool has_nan(const uint4& c) {
  const auto one = [](uint32_t w) { return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0; };
  return one(c.x) || one(c.y) || one(c.z) || one(c.w);
}

// The block's queries [lo, hi) that see a token, in bits.
struct Seers {
  int lo, hi;
  __device__ __forceinline__ void note(uint32_t* bits) const {
    for (int i = 0; i < 8; ++i) {
      const int a = min(max(lo - 32 * i, 0), 32), b = min(max(hi - 32 * i, 0), 32);
      if (a < b) atomicOr(bits + i, uint32_t(((uint64_t(1) << b) - 1) ^ ((uint64_t(1) << a) - 1)));
    }
  }
};

__device__ __forceinline__ Seers seers_of(const AttendArgs& a, const Sequence& seq, int i0, int t) {
  // row r's end is the tokens less (rows - 1 - r), and its first the end less the window
  const int64_t first = int64_t(t) - seq.tokens + seq.rows;
  const int64_t rows = seq.rows;
  const int64_t last = (a.window > 0 ? min(rows, first + min(a.window, int64_t(1) << 31)) : rows) - 1;
  Seers s;
  s.lo = int(min(max(max(first, int64_t(0)) * a.shared - i0, int64_t(0)), int64_t(2 * kTile)));
  s.hi = int(min(max((last + 1) * a.shared - i0, int64_t(0)), int64_t(2 * kTile)));
  return s;
}

// 16 codes without NaN.
__device__ __forceinline__ uint4 without_nan(const uint4& c) {
  const auto one = [](uint32_t w) {
    return w & ~(((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu);
  };
  return make_uint4(one(c.x), one(c.y), one(c.z), one(c.w));
}

// Notes what a tile's tokens, of which some queries see not all, have of values that are no
// numbers: threads `index` of `count`.
__device__ __noinline__ void note_hidden(Shared& s, const AttendArgs& a, int b, int h, int i0,
                                         int tile, int end, int index, int count) {
  const Sequence seq = sequence(a, b);
  const lp_cache_part& p = a.part[1];
  const int pieces = a.dim / 16;
  for (int i = index; i < kTile * pieces; i += count) {
    const int t = tile * kTile + i / pieces, d = i % pieces * 16;
    const int64_t slot = t < end ? slot_of(a, b, t) : -1;
    if (slot < 0) continue;
    const Seers seers = seers_of(a, seq, i0, t);
    const float scale = *reinterpret_cast<const float*>(
        static_cast<const char*>(p.params) + h * p.param_head_stride +
        slot_place(a, slot, p.param_page_stride, p.param_slot_stride));
    if (d == 0 && !(fabsf(scale) < INFINITY)) seers.note(s.nan_all);
    const uint8_t* codes = static_cast<const uint8_t*>(p.codes) + h * p.code_head_stride +
                           slot_place(a, slot, p.code_page_stride, p.code_slot_stride) + d;
    for (int e = 0; e < 16; ++e)
      if ((codes[e] & 0x7f) == 0x7f) seers.note(s.nan[d + e]);
  }
}

// What is kept of this thread's row, a column every kTile floats.
template <int DIM>
__device__ __forceinline__ float* kept_at(const AttendArgs& a) {
  return a.kept + (int64_t(blockIdx.x) * 2 + (threadIdx.x >> 7)) * DIM * kTile +
         (threadIdx.x & (kTile - 1));
}

// Adds what tensor memory has of a row to what is kept of it.
template <int DIM>
__device__ __noinline__ void keep(uint32_t o_mine, float* kept, float factor, bool first) {
#pragma unroll 1
  for (int c = 0; c < DIM; c += 32) {
    uint32_t x[32];
    tensor_load(x, o_mine + c);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      float* at = kept + (c + e) * kTile;
      *at = first ? __uint_as_float(x[e]) : fmaf(*at, factor, __uint_as_float(x[e]));
    }
  }
}

// And the other way.
template <int DIM>
__device__ __noinline__ void add_kept(uint32_t o_mine, const float* kept, float factor) {
#pragma unroll 1
  for (int c = 0; c < DIM; c += 32) {
    uint32_t x[32];
    tensor_load(x, o_mine + c);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      x[e] = __float_as_uint(fmaf(kept[(c + e) * kTile], factor, __uint_as_float(x[e])));
    tensor_store(o_mine + c, x);
  }
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 16 columns, under way while the ones before are worked on.
__device__ __forceinline__ void tensor_load16(uint32_t (&x)[16], uint32_t from) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : LP_R8(x, 0), LP_R8(x, 8) : "r"(from));
}
// What was loaded is there; ties its registers to this place.
__device__ __forceinline__ void tensor_landed(uint32_t (&x)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int e = 0; e < 16; e += 8)
    asm volatile("" : "+r"(x[e]), "+r"(x[e + 1]), "+r"(x[e + 2]), "+r"(x[e + 3]), "+r"(x[e + 4]),
                      "+r"(x[e + 5]), "+r"(x[e + 6]), "+r"(x[e + 7]));
}

// One query's view of a tile.
struct Look {
  uint32_t s_mine;          // its row of S
  const float* scales;
  const uint32_t* held;
  uint64_t unit2;
  int lo, end;              // tokens that it sees, from the tile's first

  // bits of 16 columns from c
  __device__ __forceinline__ uint32_t bits(int c) const {
    const int a = min(max(lo - c, 0), 16), b = min(max(end - c, 0), 16);
    return (a >= b ? 0u : ((1u << b) - 1u) & ~((1u << a) - 1u)) & (held[c >> 5] >> (c & 31));
  }
};

// The largest of x + floor(log2 s_v), and of `now`.  ALL: the query sees every token.
template <bool ALL>
__device__ __forceinline__ float row_largest(const Look& w, float now) {
  uint32_t x[2][16];
  tensor_load16(x[0], w.s_mine);
#pragma unroll
  for (int c = 0; c < kTile; c += 16) {
    uint32_t(&y)[16] = x[(c >> 4) & 1];
    tensor_landed(y);
    if (c + 16 < kTile) tensor_load16(x[((c >> 4) + 1) & 1], w.s_mine + c + 16);
    const uint32_t bits = ALL ? 0u : w.bits(c);
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(w.scales + c + e);
      const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(w.scales + 2 * kTile + c + e);
      const uint64_t a = fma2(mul2(uint64_t(y[e]) | uint64_t(y[e + 1]) << 32, k.x), w.unit2, l.x);
      const uint64_t b = fma2(mul2(uint64_t(y[e + 2]) | uint64_t(y[e + 3]) << 32, k.y), w.unit2, l.y);
      if (ALL) {
        now = fmaxf(now, fmaxf(fmaxf(lower(a), upper(a)), fmaxf(lower(b), upper(b))));
      } else {
        now = fmaxf(now, bits & (1u << e) ? lower(a) : -INFINITY);
        now = fmaxf(now, bits & (2u << e) ? upper(a) : -INFINITY);
        now = fmaxf(now, bits & (4u << e) ? lower(b) : -INFINITY);
        now = fmaxf(now, bits & (8u << e) ? upper(b) : -INFINITY);
      }
    }
  }
  return now;
}

// P of 16 columns from c, whose S is y: eight words.
template <bool ALL, typename F>
__device__ __forceinline__ void weights16(const Look& w, int c, const uint32_t (&y)[16],
                                          uint64_t base2, F&& each) {
  const uint32_t bits = ALL ? 0u : w.bits(c);
#pragma unroll
  for (int e = 0; e < 16; e += 4) {
    const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(w.scales + c + e);
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(w.scales + kTile + c + e);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = e + 2 * u;
      const uint64_t z = fma2(mul2(uint64_t(y[i]) | uint64_t(y[i + 1]) << 32, u ? k.y : k.x),
                              w.unit2, base2);
      float e0 = ex2(lower(z)), e1 = ex2(upper(z));
      if (!ALL) {
        e0 = bits & (1u << i) ? e0 : 0.0f;
        e1 = bits & (2u << i) ? e1 : 0.0f;
      }
      const uint64_t ee = pair(e0, e1);
      each(i / 2, ee, mul2(ee, u ? v.y : v.x));
    }
  }
}

// P and its sum; *most: the largest of its even and odd columns, as fp16.
template <bool ALL>
__device__ __forceinline__ void row_weights(const Look& w, uint64_t base2, uint32_t (&p)[64],
                                            uint64_t* sum, uint32_t* most) {
  uint32_t x[2][16];
  uint64_t sums[2] = {0, 0};
  uint32_t top[2] = {0, 0};
  tensor_load16(x[0], w.s_mine);
#pragma unroll
  for (int c = 0; c < kTile; c += 16) {
    uint32_t(&y)[16] = x[(c >> 4) & 1];
    tensor_landed(y);
    if (c + 16 < kTile) tensor_load16(x[((c >> 4) + 1) & 1], w.s_mine + c + 16);
    weights16<ALL>(w, c, y, base2, [&](int i, uint64_t ee, uint64_t z) {
      sums[i & 1] = add2(sums[i & 1], ee);
      p[c / 2 + i] = halves(lower(z), upper(z));
      asm("max.f16x2 %0, %0, %1;" : "+r"(top[i & 1]) : "r"(p[c / 2 + i]));
    });
  }
  *sum = add2(sums[0], sums[1]);
  asm("max.f16x2 %0, %1, %2;" : "=r"(*most) : "r"(top[0]), "r"(top[1]));
}

// What fp16 left of P, over S from its end: a second piece.
template <bool ALL>
__device__ __forceinline__ void row_rest(const Look& w, uint64_t base2, const uint32_t (&p)[64]) {
#pragma unroll
  for (int c = kTile - 16; c >= 0; c -= 16) {
    uint32_t y[16], rest[8];
    tensor_load16(y, w.s_mine + c);
    tensor_landed(y);
    weights16<ALL>(w, c, y, base2, [&](int i, uint64_t, uint64_t z) {
      const uint32_t h = p[c / 2 + i];
      rest[i] = halves(lower(z) - Elt<LP_F16>::half_bits_to_float(h & 0xffffu),
                       upper(z) - Elt<LP_F16>::half_bits_to_float(h >> 16));
    });
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::LP_W8(rest, 0),
        "r"(w.s_mine + 64 + c / 2) : "memory");
  }
}

template <int DIM, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
    attend_chunk_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ char raw_shared[];
  Shared& s = *reinterpret_cast<Shared*>((reinterpret_cast<uintptr_t>(raw_shared) + 1023) &
                                         ~uintptr_t(1023));
  constexpr int kPieces = DIM / 16;      // 16 codes each
  constexpr uint32_t kHalf = kTile * 128;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per_head = a.rows * a.shared;
  const int pairs = (per_head + 2 * kTile - 1) / (2 * kTile);
  // the last rows see most: they begin first
  const int pr = pairs - 1 - int(blockIdx.x % pairs);
  const int h = blockIdx.x / pairs % a.heads, b = blockIdx.x / pairs / a.heads;
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(at(&s.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&s.k_full[i], 128), bar_init(&s.v_full[i], 128);
      bar_init(&s.k_empty[i], 1), bar_init(&s.v_empty[i], 1);
      bar_init(&s.s_full[i], 1), bar_init(&s.p_full[i], 128), bar_init(&s.o_done[i], 1);
    }
    bar_init(&s.drained, 1);
#ifdef LP_TEST_CHUNK_TIMEOUT
    bar_init(&s.never, 1);
#endif
    s.failed = s.nan_hidden = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Sequence seq = sequence(a, b);
  const int i0 = pr * 2 * kTile;  // of the rows and query heads of this head
  const int r0 = i0 / a.shared;
  const int r1 = min(min(i0 + 2 * kTile, per_head) - 1, max(0, seq.rows * a.shared - 1)) / a.shared;
  const bool any = r0 < seq.rows;
  const Seen low = seen(a, seq, any ? r0 : 0), high = seen(a, seq, any ? r1 : 0);
  // tiles that any row sees; tokens that all of them see
  const int first = any ? low.lo / kTile : 0;
  const int last = any ? max(first, (high.end + kTile - 1) / kTile) : 0;
  const int tiles = last - first;
  const int all_from = high.lo, all_until = low.end;

  // queries, scaled to 2^14 by a power of two a row
  float unit = 0.0f;
  int row = 0, r = 0, j = 0;
  bool there = false;
  if (warp < 8) {
    row = i0 + tid;
    r = row / a.shared, j = h * a.shared + row - r * a.shared;
    there = row < per_head && r < seq.rows;
    const char* from = static_cast<const char*>(a.q.data) + b * a.q.batch_stride +
                       r * a.q.row_stride + j * a.q.head_stride;
    char* to = s.q[warp >> 2];
    const int in = tid & 127;
    uint2 held[DIM / 4];  // four elements each, of 16 bits
#pragma unroll
    for (int c = 0; c < DIM / 4; ++c) {
      held[c] = make_uint2(0, 0);
      if (there && a.wide_q) {
        held[c] = __ldg(reinterpret_cast<const uint2*>(from) + c);
      } else if (there) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const uint16_t*>(from + (c * 4 + e) * 2);
        held[c] = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
      }
    }
    const auto value = [&](int d) {
      const uint32_t w = (d & 2) ? held[d / 4].y : held[d / 4].x;
      const uint32_t bits = (d & 1) ? w >> 16 : w & 0xffffu;
      return WIDE ? Elt<LP_F16>::half_bits_to_float(bits) : __uint_as_float(bits << 16);
    };
    float most = 0.0f;
#pragma unroll
    for (int d = 0; d < DIM; ++d) most = fmaxf(most, fabsf(value(d)));
    const int up = most > 0.0f && most <= 3.4028235e38f
                       ? 14 - (int(__float_as_uint(most) >> 23) - 127) : 0;
    const float f1 = __uint_as_float(uint32_t(up / 2 + 127) << 23);
    const float f2 = __uint_as_float(uint32_t(up - up / 2 + 127) << 23);
    unit = a.scale / f1 / f2;
#pragma unroll
    for (int c = 0; c < DIM / 8; ++c) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = halves(value(c * 8 + 2 * e) * f1 * f2, value(c * 8 + 2 * e + 1) * f1 * f2);
      *reinterpret_cast<uint4*>(to + (c >> 3) * kHalf + in * 128 + (((c & 7) ^ (in & 7)) << 4)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s.tmem;
  // columns: S (and P) of the two 128s, then O
  const uint32_t o_at = tmem + 256;

  float mass = 0.0f, ref = -INFINITY, kept_ref = -INFINITY;
  if (warp < 8) {
    // ---------------------------------------------------------------- a thread a query
    const int half = warp >> 2;
    const uint32_t lanes = uint32_t(warp & 3) << 21;  // 32 lanes, at bit 16
    const uint32_t s_mine = tmem + half * 128 + lanes, o_mine = o_at + half * DIM + lanes;
    const Seen v = there ? seen(a, seq, r) : Seen{0, 0};
    Look w;
    w.s_mine = s_mine;
    w.unit2 = pair(unit, unit);
    for (int run = 0; run < tiles; run += kRun) {
      if (run > 0) {  // O begins anew with the next product
        if (!__all_sync(kFullWarp, bar_wait(s, &s.s_full[half], run & 1))) goto stopped;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        keep<DIM>(o_mine, kept_at<DIM>(a), kept_ref == -INFINITY ? 0.0f : ex2(kept_ref - ref),
                  run == kRun);
        kept_ref = ref;
      }
      for (int t = run; t < min(tiles, run + kRun); ++t) {
        if (!__all_sync(kFullWarp, bar_wait(s, &s.s_full[half], t & 1))) goto stopped;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const int t0 = (first + t) * kTile, slot = t & 3;
        w.scales = s.scales[slot][0];
        w.held = s.held[slot];
        w.lo = v.lo - t0, w.end = v.end - t0;
        const bool all = t0 >= all_from && t0 + kTile <= all_until &&
                         (w.held[0] & w.held[1] & w.held[2] & w.held[3]) == ~0u;
        // P is taken against the reference that there is; only where something has outgrown it
        // (the first time, always) is the largest looked for, and the reference moved
        uint32_t p[64], most;
        uint64_t sum2, base2;
        bool look = __any_sync(kFullWarp, ref == -INFINITY);
        for (;;) {
          if (look) {
            const float now = all ? row_largest<true>(w, ref) : row_largest<false>(w, ref);
            const bool grow = now > ref + kSlack || (ref == -INFINITY && now > -INFINITY);
            const float f = grow ? (ref == -INFINITY ? 0.0f : ex2(ref - now)) : 1.0f;
            if (grow) ref = now, mass *= f;
            if (t > 0 && __any_sync(kFullWarp, grow)) {
#pragma unroll 1
              for (int c = 0; c < DIM; c += 32) {
                uint32_t x[32];
                tensor_load(x, o_mine + c);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                tensor_store(o_mine + c, x);
              }
            }
          }
          const float base = (ref == -INFINITY ? 0.0f : -ref) + kLift;
          base2 = pair(base, base);
          if (all) row_weights<true>(w, base2, p, &sum2, &most);
          else row_weights<false>(w, base2, p, &sum2, &most);
          // 2^15 and above
          const bool over = (most & 0xffffu) >= 0x7800u || (most >> 16) >= 0x7800u;
          if (look || !__any_sync(kFullWarp, over)) break;
          look = true;
        }
        mass += lower(sum2) + upper(sum2);
        if (WIDE) {
          if (all) row_rest<true>(w, base2, p);
          else row_rest<false>(w, base2, p);
        }
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = p[c + e];
          tensor_store(s_mine + c, x);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        bar_arrive(&s.p_full[half]);
      }
    }
  stopped:
    if (tiles > 0) bar_wait(s, &s.o_done[half], 0);
    __syncwarp();
  } else if (warp < 12) {
    // ------------------------------------------------------- codes on their way to the products
    const int in = tid - 256;  // its token, for what is done once a token
    const lp_cache_part &kp = a.part[0], &vp = a.part[1];
    const int piece = in % kPieces, line = in / kPieces;   // its 16 codes, of every kLines-th token
    constexpr int kLines = 128 / kPieces, kMine = kTile / kLines;
    float scale[2];
    // (rows that do not see a token have 0 * what it holds)
    const auto hides = [&](int t) {
      const int t0 = (first + t) * kTile;
      return !(t0 >= all_from && t0 + kTile <= all_until);
    };
    const auto look = [&](int t) {  // a tile's tokens: where they lie, and their scales
      const int token = (first + t) * kTile + in;
      const int64_t slot = t < tiles && token < high.end ? slot_of(a, b, token) : -1;
      const uint32_t held = __ballot_sync(kFullWarp, slot >= 0);
      if (t >= tiles) return;
      if (lane == 0) s.held[t & 3][in >> 5] = held;
      scale[0] = scale[1] = 0.0f;
      s.rows[t & 1][0][in] = s.rows[t & 1][1][in] = nullptr;
      if (slot >= 0) {
        s.rows[t & 1][0][in] = static_cast<const char*>(kp.codes) + h * kp.code_head_stride +
                               slot_place(a, slot, kp.code_page_stride, kp.code_slot_stride);
        s.rows[t & 1][1][in] = static_cast<const char*>(vp.codes) + h * vp.code_head_stride +
                               slot_place(a, slot, vp.code_page_stride, vp.code_slot_stride);
        scale[0] = *reinterpret_cast<const float*>(
            static_cast<const char*>(kp.params) + h * kp.param_head_stride +
            slot_place(a, slot, kp.param_page_stride, kp.param_slot_stride));
        scale[1] = *reinterpret_cast<const float*>(
            static_cast<const char*>(vp.params) + h * vp.param_head_stride +
            slot_place(a, slot, vp.param_page_stride, vp.param_slot_stride));
        if (!(fabsf(scale[1]) < INFINITY) && hides(t)) {
          *static_cast<volatile int*>(&s.nan_hidden) = 1;
          scale[1] = 0.0f;
        }
      }
    };
    const auto put_scales = [&](int t) {
      s.scales[t & 3][0][in] = scale[0];
      s.scales[t & 3][1][in] = scale[1];
      s.scales[t & 3][2][in] =
          float(max(int((__float_as_uint(scale[1]) >> 23) & 255u) - 127, kLeastScale));
    };
    uint4 codes[2][kMine];
    const auto fetch = [&](int t, int part) {
      if (t >= tiles) return;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const char* p = s.rows[t & 1][part][line + i * kLines];
        codes[part][i] = p != nullptr ? __ldg(reinterpret_cast<const uint4*>(p) + piece)
                                      : make_uint4(0, 0, 0, 0);
      }
    };
    look(0);
    all_of_128(true);
    fetch(0, 0);
    fetch(0, 1);
    for (int t = 0; t < tiles; ++t) {
      const int stage = t & 1;
      const uint32_t turn = ((t >> 1) & 1) ^ 1;  // the first turn of each stage does not wait
      // (a tile's scales are read until its P is there: four tiles have them apart)
      if (!all_of_128(bar_wait(s, &s.k_empty[stage], turn))) break;
#ifdef LP_TEST_CHUNK_TIMEOUT
      // test builds only: the first two blocks' loaders wait for what never comes, at their
      // first tile and their second, and so run out
      if (blockIdx.x == t && t < 2 &&
          !all_of_128(bar_wait(s, &s.never, 0, LP_TEST_CHUNK_TIMEOUT))) break;
#endif
      put_scales(t);
      char* k = s.k[stage];
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        put_codes(k + (piece >> 2) * kHalf, line + i * kLines, piece & 3, codes[0][i]);
      look(t + 1);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      bar_arrive(&s.k_full[stage]);
      // (the next tile's places are there, too)
      if (!all_of_128(bar_wait(s, &s.v_empty[stage], turn))) break;
      fetch(t + 1, 0);
      char* v = s.v[stage];
      bool bad = false;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        put_codes(v + (piece >> 2) * kHalf, line + i * kLines, piece & 3, codes[1][i]);
        bad = bad || has_nan(codes[1][i]);
      }
      if (bad && hides(t)) {
        *static_cast<volatile int*>(&s.nan_hidden) = 1;
#pragma unroll
        for (int i = 0; i < kMine; ++i)
          put_codes(v + (piece >> 2) * kHalf, line + i * kLines, piece & 3,
                    without_nan(codes[1][i]));
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      bar_arrive(&s.v_full[stage]);
      fetch(t + 1, 1);
    }
  } else if (lane == 0 && tiles > 0) {
    // ------------------------------------------------------------------- the products' issue
    constexpr uint32_t kScore = instruction(kTile, kTile, false);
    constexpr uint32_t kValue = instruction(kTile, DIM, true);
    // (places in an operand are added to its address, which counts 16 bytes)
    const uint64_t q_op[2] = {operand(s.q[0], 16, 1024), operand(s.q[1], 16, 1024)};
    const uint64_t k_op[2] = {operand(s.k[0], 16, 1024), operand(s.k[1], 16, 1024)};
    const uint64_t v_op[2] = {operand(s.v[0], kHalf, 1024), operand(s.v[1], kHalf, 1024)};
    const auto score = [&](int t, int half) {
      const uint64_t qo = half ? q_op[1] : q_op[0], ko = t & 1 ? k_op[1] : k_op[0];
#pragma unroll
      for (int i = 0; i < DIM / 16; ++i) {
        const uint32_t off = ((i >> 2) * kHalf + (i & 3) * 32) >> 4;
        mma_shared(tmem + half * 128, qo + off, ko + off, kScore, i > 0);
      }
      commit(&s.s_full[half]);
    };
    bool ok = bar_wait(s, &s.k_full[0], 0);
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (ok) score(0, 0), score(0, 1), commit(&s.k_empty[0]);
    for (int t = 0; ok && t < tiles; ++t) {
      for (int half = 0; ok && half < 2; ++half) {
        ok = bar_wait(s, &s.p_full[half], t & 1) &&
             (half == 1 || bar_wait(s, &s.v_full[t & 1], (t >> 1) & 1)) &&
             (half == 1 || t + 1 == tiles || bar_wait(s, &s.k_full[(t + 1) & 1], ((t + 1) >> 1) & 1));
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
        for (int piece = WIDE ? 1 : 0; piece >= 0; --piece)
#pragma unroll
          for (int i = 0; i < kTile / 16; ++i)
            mma_tensor(o_at + half * DIM, tmem + half * 128 + piece * 64 + i * 8,
                       (t & 1 ? v_op[1] : v_op[0]) + i * (2048 >> 4), kValue,
                       t % kRun != 0 || i > 0 || piece != (WIDE ? 1 : 0));
        if (t + 1 == tiles) commit(&s.o_done[half]);
        if (half == 1) commit(&s.v_empty[t & 1]);
        // S of the next tile goes where this one's P was: products run in their order
        if (t + 1 < tiles) score(t + 1, half);
        if (half == 1 && t + 1 < tiles) commit(&s.k_empty[(t + 1) & 1]);
      }
    }
    if (!ok) {  // tensor memory is given back only when nothing writes it any more
      commit(&s.drained);
      for (uint32_t i = 0; i < kPatience && !bar_wait(s, &s.drained, 0, 1); ++i) {
      }
    }
  }
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const bool failed = *static_cast<volatile int*>(&s.failed) != 0;
  const bool hidden = *static_cast<volatile int*>(&s.nan_hidden) != 0;
  if (warp < 8) {
    // ------------------------------------------------------------------------------- results
    char* to = static_cast<char*>(a.out.data) + b * a.out.batch_stride + r * a.out.row_stride +
               j * a.out.head_stride;
    const uint32_t o_mine = o_at + (warp >> 2) * DIM + (uint32_t(warp & 3) << 21);
    const bool none = tiles == 0 || !there || (mass == 0.0f && !failed);
    if (failed) mass = __uint_as_float(0x7fc00000u);  // whatever there is of it
    const float inv = 1.0f / mass;
    if (a.lse != nullptr && row < per_head)
      a.lse[(int64_t(b) * a.rows + r) * (a.heads * a.shared) + j] =
          none ? -INFINITY : ref - kLift + log2f(mass);
    if (tiles > kRun)
      add_kept<DIM>(o_mine, kept_at<DIM>(a),
                    kept_ref == -INFINITY ? 0.0f : ex2(kept_ref - ref));
#pragma unroll 1
    for (int c = 0; c < DIM; c += 32) {
      uint32_t x[32];
      __syncwarp();
      if (tiles > 0) {
        tensor_load(x, o_mine + c);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = 0;
      }
#pragma unroll
      for (int e = 0; e < 32; ++e)
        x[e] = none ? 0u : __float_as_uint(__uint_as_float(x[e]) * inv);
      if (row >= per_head) continue;
      if (a.wide_out) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          uint32_t w[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float y = __uint_as_float(x[e + 2 * u]), z = __uint_as_float(x[e + 2 * u + 1]);
            if (WIDE) w[u] = halves(y, z);
            else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[u]) : "f"(z), "f"(y));
          }
          *reinterpret_cast<uint2*>(to + (c + e) * 2) = make_uint2(w[0], w[1]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) store_float(to, c + e, __uint_as_float(x[e]), a.dt);
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  if (hidden) {  // for all of the block: rows that see what was taken out have it
    for (int i = tid; i < DIM * 8; i += kThreads) s.nan[i >> 3][i & 7] = 0;
    if (tid < 8) s.nan_all[tid] = 0;
    __syncthreads();
    for (int t = first; t < last; ++t)
      if (t * kTile < all_from || t * kTile + kTile > all_until)
        note_hidden(s, a, b, h, i0, t, high.end, tid, kThreads);
    __syncthreads();
    if (warp < 8 && there) {
      char* to = static_cast<char*>(a.out.data) + b * a.out.batch_stride + r * a.out.row_stride +
                 j * a.out.head_stride;
      for (int d = 0; d < DIM; ++d)
        if (((s.nan[d][warp] | s.nan_all[warp]) >> lane) & 1u)
          store_float(to, d, __uint_as_float(0x7fc00000u), a.dt);
    }
  }
}

template <int DIM, bool WIDE>
cudaError_t launch_chunk(const AttendArgs& a, cudaStream_t stream) {
  static PerDevice<1> allowed;
  const int smem = int(sizeof(Shared)) + 1024;
  const cudaError_t e = allow_shared(attend_chunk_kernel<DIM, WIDE>, smem, allowed);
  if (e != cudaSuccess) return e;
  const int64_t pairs = (int64_t(a.rows) * a.shared + 2 * kTile - 1) / (2 * kTile);
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(pairs * a.heads * a.batch));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_chunk_kernel<DIM, WIDE>, a);
}

}  // namespace

// Floats that the blocks keep of their rows, `rows` to a head of the cache; 0 where these are
// too few for the kernel.
int64_t chunk_kept(int64_t rows, int64_t heads, int64_t batch, int64_t dim) {
  // A block's time is that of its tokens, whoever else runs (528 us for 16384), the other kernel's
  // that of all queries: 407 us for 32 x 256 of them over 16384, 503 for 40 x 256; 127 us for
  // 16 x 256 over 8192, in half-filled blocks.  They meet near 43 x 256.
  const int64_t full = rows * heads * batch / (2 * kTile);
  if ((dim != 64 && dim != 128) || rows < kTile || full < 43) return 0;
  return (rows + 2 * kTile - 1) / (2 * kTile) * 2 * kTile * heads * batch * dim;
}

bool chunk_fits(const AttendArgs& a) {
  const int64_t floats = chunk_kept(int64_t(a.rows) * a.shared, a.heads, a.batch, a.dim);
  return a.bits == 8 && a.group == a.dim && a.dt != LP_F32 && floats > 0 &&
         floats / (2 * kTile * a.dim) <= INT32_MAX;
}

cudaError_t attend_chunk(const AttendArgs& a, cudaStream_t stream) {
  if (a.dim == 128)
    return a.dt == LP_BF16 ? launch_chunk<128, false>(a, stream) : launch_chunk<128, true>(a, stream);
  return a.dt == LP_BF16 ? launch_chunk<64, false>(a, stream) : launch_chunk<64, true>(a, stream);
}

}  // namespace lp
