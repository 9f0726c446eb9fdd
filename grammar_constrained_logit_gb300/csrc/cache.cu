// cache.cu -- keys and values quantised as they are written to a cache, and read back.
//
// A group is `group` consecutive elements of one token and head.  Over its finite
// elements (|x| <= the largest bf16):
//   8 bits  s = max(max|x| * fl(1/448), 2^-126)            (32-bit scale)
//           code = e4m3(x * fl(1/s)), round to nearest even, saturating; value = code * s
//   4 bits  lo, hi: the least and largest;  s = bf16(max((hi/2 - lo/2) * fl(1/7.5), 2^-126)),
//           l = bf16(lo);  code = rint(min(max((x - l) * fl(1/s), 0), 15));  value = l + code * s
// Every step is a 32-bit operation rounded to nearest, so which code a value gets does
// not depend on who computes it.  The 4-bit pair is held in 16 bits each, an eighth of a
// 32-element group's codes: codes are taken against the rounded pair, so the rounding
// costs range at the group's ends (2^-8 of lo), not accuracy between; bf16 rather than
// fp16 because no input overflows it.
//
// What bounds both is memory, if the instructions between are few: a thread keeps its
// place within the token and steps over tokens, so its addresses are worked out once;
// extrema are taken of 16-bit pairs; arithmetic goes two 32-bit values at a time; codes
// are rounded by adding 1.5 * 2^23 and read by placing them in a float's last bits.
// 32768 tokens of 2 x 8 x 128 bf16 written to 8 bits: 31.1 us, 95% of the measured copy
// rate; 131072 read back from 4 bits: 111 us, 94%.
#include <algorithm>

#include "common.cuh"

namespace lp {
namespace {

constexpr int kMaxParts = 8;
constexpr int kThreads = 256;
constexpr float kLargest = 3.3895313892515355e38f;
constexpr float kTiny = 1.1754943508222875e-38f;  // 2^-126

// n / d for n < 2^31: with 2^(l-1) < d <= 2^l, m = ceil(2^(31+l) / d) is below 2^32 and
// n m / 2^(31+l) exceeds n / d by less than n / 2^(31+l) < 1 / d.
struct Div {
  uint32_t d, m, shift;
  void set(uint32_t by) {
    d = by;
    uint32_t l = 0;
    while ((uint64_t(1) << l) < by) ++l;
    shift = 31 + l;
    m = uint32_t(((uint64_t(1) << shift) + by - 1) / by);
  }
  __device__ __forceinline__ uint32_t quot(uint32_t n) const {
    return uint32_t((uint64_t(n) * m) >> shift);
  }
};

struct CacheArgs {
  lp_cache_part part[kMaxParts];
  lp_heads x[kMaxParts];
  const int64_t* slots;
  int64_t n, n_slots, page;
  int heads, dim, group;
  Div per_page;  // where slots are below 2^31
  // of the vector kernels: a token has `per_token` items (groups to write, vectors to
  // read) and a block takes `tokens` tokens at a time, or one of `tiles` parts of a token
  Div per_token, per_head, tiles, per_group;
  int items, tokens;                // a block's items at a time; of how many tokens
  int lanes, reach, segments;       // write: lanes a group, the power of two from there, groups a warp
};

template <int DT>
__device__ __forceinline__ float load_float(const char* p) {
  return Elt<DT>::load1(p);
}

__device__ __forceinline__ uint32_t bf16_bits(float x) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
  return r;
}

template <int DT>
__device__ __forceinline__ uint32_t rounded_bits(float x) {
  if (DT == LP_F32) return __float_as_uint(x);
  if (DT == LP_BF16) return bf16_bits(x);
  uint16_t r;
  asm("cvt.rn.f16.f32 %0, %1;" : "=h"(r) : "f"(x));
  return r;
}

// e4m3 codes of two values: a in the low byte
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(code & 0xffu)));
  return Elt<LP_F16>::half_bits_to_float(h & 0xffffu);
}

struct Range {  // of a group's finite elements
  float lo = INFINITY, hi = -INFINITY;
  __device__ __forceinline__ void add(float x) {
    if (fabsf(x) <= kLargest) lo = fminf(lo, x), hi = fmaxf(hi, x);
  }
};

struct Scale {
  float inv, low;      // code = (x - low) * inv
  uint32_t held;       // what the cache holds
};

template <int BITS>
__device__ __forceinline__ Scale scale_of(Range r) {
  if (!(r.lo <= r.hi)) r.lo = r.hi = 0.0f;
  Scale s;
  if (BITS == 8) {
    const float most = fmaxf(-r.lo, r.hi);
    const float scale = fmaxf(__fmul_rn(most, float(1.0 / 448)), kTiny);
    s.inv = __frcp_rn(scale);
    s.low = 0.0f;
    s.held = __float_as_uint(scale);
  } else {
    const float d = __fsub_rn(__fmul_rn(r.hi, 0.5f), __fmul_rn(r.lo, 0.5f));
    const uint32_t scale = bf16_bits(fmaxf(__fmul_rn(d, float(1.0 / 7.5)), kTiny));
    const uint32_t low = bf16_bits(r.lo);
    s.inv = __frcp_rn(__uint_as_float(scale << 16));
    s.low = __uint_as_float(low << 16);
    s.held = scale | (low << 16);
  }
  return s;
}

__device__ __forceinline__ uint32_t code4(float x, const Scale& s) {
  const float y = __fmul_rn(__fsub_rn(x, s.low), s.inv);
  // NaN: 0.  The sum with 2^23 rounds to an integer, ties to even
  return __float_as_uint(__fadd_rn(fminf(fmaxf(y, 0.0f), 15.0f), 8388608.0f)) & 15u;
}

// Where a slot lies, from a part's base.
__device__ __forceinline__ int64_t place(const CacheArgs& a, int64_t slot, int64_t page_stride,
                                         int64_t slot_stride) {
  if (a.page >= a.n_slots) return slot * slot_stride;  // one page
  const int64_t p = a.n_slots <= INT32_MAX ? int64_t(a.per_page.quot(uint32_t(slot)))
                                           : slot / a.page;
  return p * page_stride + (slot - p * a.page) * slot_stride;
}

__device__ __forceinline__ int64_t code_place(const CacheArgs& a, const lp_cache_part& p,
                                              int64_t slot) {
  return place(a, slot, p.code_page_stride, p.code_slot_stride);
}

__device__ __forceinline__ int64_t param_place(const CacheArgs& a, const lp_cache_part& p,
                                               int64_t slot) {
  return place(a, slot, p.param_page_stride, p.param_slot_stride);
}

// One warp a group.
template <int DT, int BITS>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheArgs a) {
  constexpr int Bt = Elt<DT>::kBytes;
  const int lane = threadIdx.x & 31;
  const int groups = a.dim / a.group;
  const lp_cache_part& part = a.part[blockIdx.y];
  const lp_heads& xs = a.x[blockIdx.y];
  const int64_t total = a.n * a.heads * groups;
  for (int64_t i = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); i < total;
       i += int64_t(gridDim.x) * (kThreads / 32)) {
    const int g = int(i % groups), h = int(i / groups % a.heads);
    const int64_t t = i / groups / a.heads;
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.n_slots) continue;
    const char* x = static_cast<const char*>(xs.data) +
                    (t * xs.token_stride + h * xs.head_stride + int64_t(g) * a.group) * Bt;
    Range r;
    for (int e = lane; e < a.group; e += 32) r.add(load_float<DT>(x + e * Bt));
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      r.lo = fminf(r.lo, __shfl_xor_sync(kFullWarp, r.lo, o));
      r.hi = fmaxf(r.hi, __shfl_xor_sync(kFullWarp, r.hi, o));
    }
    const Scale s = scale_of<BITS>(r);
    uint8_t* codes = static_cast<uint8_t*>(part.codes) +
                     code_place(a, part, slot) + h * part.code_head_stride + int64_t(g) * a.group * BITS / 8;
    if (BITS == 8) {
      for (int e = lane; e < a.group; e += 32)
        codes[e] = uint8_t(e4m3_pair(__fmul_rn(load_float<DT>(x + e * Bt), s.inv), 0.0f));
    } else {
      for (int e = lane; e < a.group / 2; e += 32)
        codes[e] = uint8_t(code4(load_float<DT>(x + 2 * e * Bt), s) |
                           code4(load_float<DT>(x + (2 * e + 1) * Bt), s) << 4);
    }
    if (lane == 0)
      *reinterpret_cast<uint32_t*>(static_cast<char*>(part.params) +
                                   param_place(a, part, slot) + h * part.param_head_stride +
                                   int64_t(g) * 4) = s.held;
  }
}

// One thread a byte of codes' elements: one of 8 bits, two of 4.
template <int DT, int BITS>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheArgs a) {
  constexpr int Bt = Elt<DT>::kBytes, E = 8 / BITS;
  const lp_cache_part& part = a.part[blockIdx.y];
  const lp_heads& xs = a.x[blockIdx.y];
  const int bytes = a.dim / E;
  const int64_t total = a.n * a.heads * bytes;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kThreads) {
    const int c = int(i % bytes), h = int(i / bytes % a.heads);
    const int64_t t = i / bytes / a.heads;
    const int64_t slot = a.slots[t];
    char* x = static_cast<char*>(xs.data) +
              (t * xs.token_stride + h * xs.head_stride + int64_t(c) * E) * Bt;
    float v[2] = {0.0f, 0.0f};
    if (slot >= 0 && slot < a.n_slots) {
      const uint32_t code = *(static_cast<const uint8_t*>(part.codes) +
                              code_place(a, part, slot) + h * part.code_head_stride + c);
      const uint32_t held = *reinterpret_cast<const uint32_t*>(
          static_cast<const char*>(part.params) +
          param_place(a, part, slot) + h * part.param_head_stride + int64_t(c * E / a.group) * 4);
      if (BITS == 8) {
        v[0] = __fmul_rn(e4m3_value(code), __uint_as_float(held));
      } else {
        const float s = __uint_as_float(held << 16), low = __uint_as_float(held & 0xffff0000u);
        v[0] = __fmaf_rn(float(code & 15), s, low);  // the product is exact: one rounding
        v[1] = __fmaf_rn(float(code >> 4), s, low);
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) Elt<DT>::store1(x + e * Bt, rounded_bits<DT>(v[e]));
  }
}

// ---------------------------------------------------------------- vector kernels

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  return uint64_t(__float_as_uint(a)) | uint64_t(__float_as_uint(b)) << 32;
}
__device__ __forceinline__ float first(uint64_t v) { return __uint_as_float(uint32_t(v)); }
__device__ __forceinline__ float second(uint64_t v) { return __uint_as_float(uint32_t(v >> 32)); }

// Two 32-bit operations in one instruction, each rounded to nearest.
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

// Packed maximum and minimum of 16-bit pairs; in a maximum a NaN stays.
template <int DT>
__device__ __forceinline__ uint32_t max16(uint32_t a, uint32_t b) {
  uint32_t r;
  if (DT == LP_BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <int DT>
__device__ __forceinline__ uint32_t min16(uint32_t a, uint32_t b) {
  uint32_t r;
  if (DT == LP_BF16) asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int DT>
__device__ __forceinline__ uint64_t floats16(uint32_t w) {  // the two elements of a word
  if (DT == LP_BF16) return uint64_t(w << 16) | uint64_t(w & 0xffff0000u) << 32;
  return pack2(Elt<LP_F16>::half_bits_to_float(w & 0xffffu),
               Elt<LP_F16>::half_bits_to_float(w >> 16));
}

// E consecutive elements of an input.  Sixteen are 32 bytes (16-bit types) or twice that,
// and are loaded 32 bytes at once; eight, 16 bytes at once.
template <int DT, int E>
struct Vec {
  static constexpr int kWords = E * Elt<DT>::kBytes / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const char* p) {
    if (E == 16) {
#pragma unroll
      for (int i = 0; i < kWords; i += 8)
        asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]),
                       "=r"(w[i + 5]), "=r"(w[i + 6]), "=r"(w[i + 7])
                     : "l"(p + 4 * i));
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p + 4 * i));
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ uint64_t pair(int i) const {  // elements 2i and 2i + 1
    if (DT == LP_F32) return uint64_t(w[2 * i]) | uint64_t(w[2 * i + 1]) << 32;
    return floats16<DT>(w[i]);
  }
  // The finite range, for 8 bits as (-most, most).  An infinity or a NaN shows in the
  // result, and only then the elements are gone through one by one.  *fine: there is none.
  template <int BITS>
  __device__ __forceinline__ Range range(bool* fine) const {
    Range r;
    *fine = true;
    if (DT == LP_F32) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const float x = __uint_as_float(w[i]);
        if (BITS == 8) r.hi = max_nan(r.hi, fabsf(x));
        else r.lo = fminf(r.lo, x), r.hi = max_nan(r.hi, x);
      }
    } else {
      uint32_t hi = BITS == 8 ? w[0] & 0x7fff7fffu : w[0], lo = w[0];
#pragma unroll
      for (int i = 1; i < kWords; ++i) {
        hi = max16<DT>(hi, BITS == 8 ? w[i] & 0x7fff7fffu : w[i]);
        if (BITS == 4) lo = min16<DT>(lo, w[i]);
      }
      const uint64_t h = floats16<DT>(hi), l = floats16<DT>(lo);
      r.hi = max_nan(first(h), second(h));
      r.lo = fminf(first(l), second(l));
    }
    if (BITS == 8) r.lo = -r.hi;
    if (!(r.hi <= kLargest && r.lo >= -kLargest)) {
      *fine = false;
      r = Range();
#pragma unroll
      for (int i = 0; i < E / 2; ++i) r.add(first(pair(i))), r.add(second(pair(i)));
      if (BITS == 8) r.hi = fmaxf(-r.lo, r.hi), r.lo = -r.hi;
    }
    return r;
  }
};

// What a thread works on: item `idx` of token `t`, and of every `step`-th after it.
struct Work {
  int64_t t, step;
  int head, idx;
  bool there;
};

// item: this thread's among the block's
template <int U>
__device__ __forceinline__ Work work_of(const CacheArgs& a, uint32_t item) {
  Work w;
  uint32_t block = blockIdx.x, sub = 0, idx = item;
  if (a.tiles.d > 1) {
    block = a.tiles.quot(blockIdx.x);
    idx += (blockIdx.x - block * a.tiles.d) * a.items;
  } else {
    sub = a.per_token.quot(item);
    idx -= sub * a.per_token.d;
  }
  w.there = item < uint32_t(a.items) && idx < a.per_token.d;
  w.t = int64_t(block) * U * a.tokens + sub;
  w.step = a.tokens;
  w.head = 0;
  w.idx = int(idx);
  if (a.heads > 1) {
    w.head = int(a.per_head.quot(idx));
    w.idx -= w.head * int(a.per_head.d);
  }
  return w;
}

// A group on `lanes` neighbouring lanes, R vectors a lane, as many groups side by side in
// a warp as fit; U tokens of that at once.
template <int DT, int BITS, int E, int R, int U>
__global__ void __launch_bounds__(kThreads)
    cache_write_vec_kernel(const __grid_constant__ CacheArgs a) {
  constexpr int Bt = Elt<DT>::kBytes;
  const lp_cache_part& part = a.part[blockIdx.y];
  const lp_heads& xs = a.x[blockIdx.y];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seg = lane / a.lanes, at = lane - seg * a.lanes;
  const int units = a.group / E;
  const Work w = work_of<U>(a, seg < a.segments ? warp * a.segments + seg : UINT32_MAX >> 1);
  const char* x = static_cast<const char*>(xs.data) +
                  (w.t * xs.token_stride + w.head * xs.head_stride + int64_t(w.idx) * a.group) * Bt +
                  at * (E * Bt);

  Vec<DT, E> v[U][R];
  int64_t slot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    slot[u] = -1;
    if (w.there && w.t + u * w.step < a.n) {
      slot[u] = __ldg(a.slots + w.t + u * w.step);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (R == 1 || r * a.lanes + at < units) v[u][r].load(x + r * a.lanes * (E * Bt));
    }
    x += w.step * xs.token_stride * Bt;
  }
  uint8_t* codes0 = static_cast<uint8_t*>(part.codes) + w.head * part.code_head_stride +
                    int64_t(w.idx) * a.group * BITS / 8 + at * (E * BITS / 8);
  char* params0 = static_cast<char*>(part.params) + w.head * part.param_head_stride + w.idx * 4;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool live = slot[u] >= 0 && slot[u] < a.n_slots;
    Range range;
    bool fine = true;
    if (live) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (R == 1 || r * a.lanes + at < units) {
          bool f;
          const Range one = v[u][r].template range<BITS>(&f);
          range.lo = R == 1 ? one.lo : fminf(range.lo, one.lo);
          range.hi = R == 1 ? one.hi : fmaxf(range.hi, one.hi);
          fine = fine && f;
        }
    }
    for (int o = a.reach; o; o >>= 1) {
      const float hi = __shfl_down_sync(kFullWarp, range.hi, o);
      if (at + o < a.lanes) range.hi = fmaxf(range.hi, hi);
      if (BITS == 4) {
        const float lo = __shfl_down_sync(kFullWarp, range.lo, o);
        if (at + o < a.lanes) range.lo = fminf(range.lo, lo);
      }
    }
    if (a.lanes > 1) {
      range.hi = __shfl_sync(kFullWarp, range.hi, lane - at);
      if (BITS == 4) range.lo = __shfl_sync(kFullWarp, range.lo, lane - at);
    }
    if (BITS == 8) range.lo = -range.hi;
    if (!live) continue;
    const Scale s = scale_of<BITS>(range);
    uint8_t* codes = codes0 + code_place(a, part, slot[u]);
    const uint64_t inv = pack2(s.inv, s.inv), off = pack2(-s.low, -s.low);
    // Whether all of the lane's codes round to 0 .. 15 as they are: not where the pair's
    // rounding moved the range by half a step, nor with infinities and NaN
    const bool inside = fine && __fmul_rn(__fsub_rn(range.lo, s.low), s.inv) > -0.5f &&
                        __fmul_rn(__fsub_rn(range.hi, s.low), s.inv) < 15.5f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (R > 1 && r * a.lanes + at >= units) continue;
      uint8_t* c = codes + r * a.lanes * (E * BITS / 8);
      const Vec<DT, E>& x = v[u][r];
      uint32_t w[E * BITS / 32];
      if (BITS == 8) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
          const uint64_t p = mul2(x.pair(2 * i), inv), q = mul2(x.pair(2 * i + 1), inv);
          w[i] = e4m3_pair(first(p), second(p)) | e4m3_pair(first(q), second(q)) << 16;
        }
      } else {
        uint64_t y[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) y[i] = mul2(add2(x.pair(i), off), inv);
        if (!inside) {
#pragma unroll
          for (int i = 0; i < E / 2; ++i)  // NaN: 0
            y[i] = pack2(fminf(fmaxf(first(y[i]), 0.0f), 15.0f),
                         fminf(fmaxf(second(y[i]), 0.0f), 15.0f));
        }
#pragma unroll
        for (int i = 0; i < E / 8; ++i) {
          // The sum with 1.5 * 2^23 rounds to an integer, ties to even, in the last bits of a
          // word that is zero up to bit 21 otherwise; a pair's byte is one multiplication.
          uint32_t byte[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t z = add2(y[4 * i + j], pack2(12582912.0f, 12582912.0f));
            byte[j] = uint32_t(z >> 32) * 16u + uint32_t(z);
          }
          w[i] = __byte_perm(__byte_perm(byte[0], byte[1], 0x0040),
                             __byte_perm(byte[2], byte[3], 0x0040), 0x5410);
        }
      }
      constexpr int kOut = E * BITS / 32;
      if (kOut == 4) *reinterpret_cast<uint4*>(c) = make_uint4(w[0], w[1], w[2], w[kOut - 1]);
      else if (kOut == 2) *reinterpret_cast<uint2*>(c) = make_uint2(w[0], w[kOut - 1]);
      else *reinterpret_cast<uint32_t*>(c) = w[0];
    }
    if (at == 0)
      *reinterpret_cast<uint32_t*>(params0 + param_place(a, part, slot[u])) = s.held;
  }
}

// E elements a thread, of U tokens at once.
template <int DT, int BITS, int E, int U>
__global__ void __launch_bounds__(kThreads)
    cache_read_vec_kernel(const __grid_constant__ CacheArgs a) {
  constexpr int Bt = Elt<DT>::kBytes, kIn = E * BITS / 32;
  const lp_cache_part& part = a.part[blockIdx.y];
  const lp_heads& xs = a.x[blockIdx.y];
  const Work work = work_of<U>(a, threadIdx.x);
  if (!work.there) return;
  int64_t slot[U];
  uint32_t w[U][kIn], held[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    slot[u] = -1;
    if (work.t + u * work.step < a.n) slot[u] = __ldg(a.slots + work.t + u * work.step);
  }
  const uint8_t* codes = static_cast<const uint8_t*>(part.codes) +
                         work.head * part.code_head_stride + int64_t(work.idx) * (E * BITS / 8);
  const char* params = static_cast<const char*>(part.params) +
                       work.head * part.param_head_stride + a.per_group.quot(work.idx) * 4;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (slot[u] < 0 || slot[u] >= a.n_slots) {
      slot[u] = -1;
      continue;
    }
    const uint8_t* p = codes + code_place(a, part, slot[u]);
    if (kIn == 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      w[u][0] = v.x, w[u][1] = v.y, w[u][kIn - 2] = v.z, w[u][kIn - 1] = v.w;
    } else if (kIn == 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      w[u][0] = v.x, w[u][kIn - 1] = v.y;
    } else {
      w[u][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
    held[u] = __ldg(reinterpret_cast<const uint32_t*>(params + param_place(a, part, slot[u])));
  }
  char* x = static_cast<char*>(xs.data) +
            (work.t * xs.token_stride + work.head * xs.head_stride + int64_t(work.idx) * E) * Bt;
#pragma unroll
  for (int u = 0; u < U; ++u, x += work.step * xs.token_stride * Bt) {
    if (work.t + u * work.step >= a.n) return;
    uint64_t v[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) v[i] = 0;
    if (slot[u] >= 0) {
      if (BITS == 8) {
        const float s1 = __uint_as_float(held[u]);
        const uint64_t s = pack2(s1, s1);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          uint32_t two;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
              : "=r"(two) : "h"(uint16_t(w[u][i / 2] >> (16 * (i & 1)))));
          v[i] = mul2(floats16<LP_F16>(two), s);
        }
      } else {
        const float s1 = __uint_as_float(held[u] << 16);
        const float low1 = __uint_as_float(held[u] & 0xffff0000u);
        const uint64_t s = pack2(s1, s1), low = pack2(low1, low1);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          // A code whose lowest bit is bit b of a word is the last place of a float of
          // exponent 23 - b: with that float's leading bit it reads 2^(23-b) + code, and
          // less 2^(23-b) it is the code, exactly.
          constexpr uint32_t kOne = 127 + 23;
          const uint32_t x4 = (i & 3) < 2 ? w[u][i / 4] : w[u][i / 4] >> 16;
          const int b = 8 * (i & 1);
          const uint32_t m0 = (kOne - b) << 23, m1 = (kOne - b - 4) << 23;
          const uint64_t code =
              add2(uint64_t((x4 & (15u << b)) | m0) | uint64_t((x4 & (15u << (b + 4))) | m1) << 32,
                   pack2(-__uint_as_float(m0), -__uint_as_float(m1)));
          v[i] = fma2(code, s, low);  // the product is exact: one rounding
        }
      }
    }
    constexpr int kOut = E * Bt / 4;
    uint32_t o[kOut];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      if (DT == LP_F32) {
        o[(2 * i) % kOut] = uint32_t(v[i]), o[(2 * i + 1) % kOut] = uint32_t(v[i] >> 32);
      } else if (DT == LP_BF16) {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(second(v[i])), "f"(first(v[i])));
      } else {
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(second(v[i])), "f"(first(v[i])));
      }
    }
    if (E == 16) {
#pragma unroll
      for (int i = 0; i < kOut; i += 8)
        asm volatile("st.global.L1::no_allocate.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(o[i]),
                     "r"(o[i + 1]), "r"(o[i + 2]), "r"(o[i + 3]), "r"(o[i + 4]), "r"(o[i + 5]),
                     "r"(o[i + 6]), "r"(o[i + 7]), "l"(x + 4 * i)
                     : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < kOut; i += 4)
        __stcs(reinterpret_cast<uint4*>(x + 4 * i), make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]));
    }
  }
}

// Whether vectors of E elements fit the groups, and are aligned wherever they are touched.
template <int DT, int BITS>
bool vectors_of(int E, const CacheArgs& a, int n_parts) {
  if (a.dim % E || a.group % E) return false;
  uint64_t x = 0, codes = 0;
  for (int i = 0; i < n_parts; ++i) {
    x |= reinterpret_cast<uintptr_t>(a.x[i].data) |
         uint64_t(a.x[i].token_stride) * Elt<DT>::kBytes |
         uint64_t(a.x[i].head_stride) * Elt<DT>::kBytes;
    codes |= reinterpret_cast<uintptr_t>(a.part[i].codes) | uint64_t(a.part[i].code_page_stride) |
             uint64_t(a.part[i].code_slot_stride) | uint64_t(a.part[i].code_head_stride);
  }
  return x % (E == 16 ? 32 : 16) == 0 && codes % (E * BITS / 8) == 0;
}

// Fills in what the vector kernels go by, for a token of per_token items and blocks of
// per_block at a time; the grid.
dim3 plan_work(CacheArgs& a, int64_t per_token, int per_block, int U, int n_parts) {
  a.per_token.set(uint32_t(per_token));
  a.per_head.set(uint32_t(per_token / a.heads));
  const int64_t tiles = per_token > per_block ? (per_token + per_block - 1) / per_block : 1;
  a.tiles.set(uint32_t(tiles));
  a.tokens = tiles > 1 ? 1 : int(per_block / per_token);
  a.items = tiles > 1 ? per_block : a.tokens * int(per_token);
  const int64_t at_once = int64_t(U) * a.tokens;
  return dim3(unsigned((a.n + at_once - 1) / at_once * tiles), unsigned(n_parts));
}

template <int DT, int BITS, int E, int R, int U>
cudaError_t write_vec(CacheArgs a, int n_parts, cudaStream_t stream) {
  const int units = a.group / E;
  a.lanes = (units + R - 1) / R;
  a.segments = 32 / a.lanes;
  a.reach = 1;
  while (a.reach < a.lanes) a.reach *= 2;
  a.reach /= 2;
  const dim3 grid = plan_work(a, int64_t(a.heads) * (a.dim / a.group),
                              kThreads / 32 * a.segments, U, n_parts);
  return launch_kernel(cache_write_vec_kernel<DT, BITS, E, R, U>, grid, kThreads, 0, stream, a);
}

template <int DT, int BITS, int E, int U>
cudaError_t read_vec(CacheArgs a, int n_parts, cudaStream_t stream) {
  a.per_group.set(uint32_t(a.group / E));
  const dim3 grid = plan_work(a, int64_t(a.heads) * (a.dim / E), kThreads, U, n_parts);
  return launch_kernel(cache_read_vec_kernel<DT, BITS, E, U>, grid, kThreads, 0, stream, a);
}

template <int DT, int BITS>
cudaError_t launch_piece(const CacheArgs& a, bool write, int n_parts, cudaStream_t stream) {
  const bool indexed = int64_t(a.heads) * a.dim <= INT32_MAX;
  // Several tokens a thread keep as many loads in flight: 131072 tokens read from 4 bits in
  // 152 us with one, 125 with two, 111 with four, 115 with eight; 32-bit values, twice as
  // wide, are best with two (6001 x 2 x 5 x 80 written and read: 11.2 us, with four 12.7).
  // Few tokens, of which SMs would get no block, are rather spread (32 written: 2.3 us with
  // two a thread, 2.0 with one).
  constexpr int U = DT == LP_F32 ? 2 : 4;
  const bool few = a.n * a.heads * a.dim < 152 * kThreads * 16;
  if (indexed && vectors_of<DT, BITS>(16, a, n_parts) && !(write && a.group > 2 * 32 * 16)) {
    if (!write)
      return few ? read_vec<DT, BITS, 16, 1>(a, n_parts, stream)
                 : read_vec<DT, BITS, 16, U>(a, n_parts, stream);
    // Groups of more than one vector have two on a lane, of half the lanes: fewer steps to
    // their range, and its parameters are made by fewer threads.  32768 x 2 x 8 x 128 bf16:
    // 31.3 us written to 4 bits in groups of 32 and 31.1 to 8 in groups of 128, with one
    // vector a lane 35.6 and 33.4.  Two tokens at once for 4 bits (with one 33.3), one for 8
    // (31.9 in groups of 32, with two 32.7).  32-bit values are four loads as they are: 25.5
    // and 27.0 with two vectors (16384, 4 bits, groups of 32), 26.3 and 26.1 (8, of 128).
    constexpr int pair_tokens = BITS == 4 && DT != LP_F32 ? 2 : 1;
    if (a.group > 32 * 16 || (DT != LP_F32 && a.group > 16 && !few))
      return write_vec<DT, BITS, 16, 2, pair_tokens>(a, n_parts, stream);
    return few ? write_vec<DT, BITS, 16, 1, 1>(a, n_parts, stream)
               : write_vec<DT, BITS, 16, 1, U>(a, n_parts, stream);
  }
  if (indexed && vectors_of<DT, BITS>(8, a, n_parts) && !(write && a.group > 4 * 32 * 8)) {
    if (!write) return read_vec<DT, BITS, 8, 4>(a, n_parts, stream);
    // The same, four on a lane: 32768 x 2 x 8 x 72 fp16, one group a head, written to 8 bits
    // 23.3 us and in groups of 24 to 4 bits 26.6, with one vector a lane 33.8 and 40.4 (their
    // bytes take 17.1 and 14.9).  A group's parameters are made by its lanes: with a group a
    // lane, 128 in groups of 8 to 4 bits, 55 us for 29.8.
    if (a.group > 16) return write_vec<DT, BITS, 8, 4, 1>(a, n_parts, stream);
    return write_vec<DT, BITS, 8, 1, 4>(a, n_parts, stream);
  }
  // What no vector fits: odd widths, strides off their boundaries, groups of more than 1024.
  // Right for all of it and no more: an element or a byte a thread, places by division.
  // 32768 x 2 x 8 x 34 bf16 to 8 bits take 156 us (their bytes 8.2), 4096 x 2 x 4 x 2048 in
  // groups of 2048 82 (29.7); 131072 x 2 x 8 x 34 read from 4 bits 195 (27.7).
  if (write) {
    const int64_t warps = a.n * a.heads * (a.dim / a.group);
    const dim3 grid(unsigned(std::min<int64_t>((warps + 7) / 8, 152 * 64)), unsigned(n_parts));
    return launch_kernel(cache_write_kernel<DT, BITS>, grid, kThreads, 0, stream, a);
  }
  const int64_t threads = a.n * a.heads * (int64_t(a.dim) * BITS / 8);
  const dim3 grid(unsigned(std::min<int64_t>((threads + kThreads - 1) / kThreads, 152 * 64)),
                  unsigned(n_parts));
  return launch_kernel(cache_read_kernel<DT, BITS>, grid, kThreads, 0, stream, a);
}

template <int DT, int BITS>
cudaError_t launch(const CacheArgs& a0, bool write, int n_parts, cudaStream_t stream) {
  CacheArgs a = a0;
  // heads that follow one another everywhere are one long head
  bool flat = a.group <= a.dim && int64_t(a.heads) * a.dim <= INT32_MAX;
  for (int i = 0; i < n_parts; ++i)
    flat = flat && a.x[i].head_stride == a.dim &&
           a.part[i].code_head_stride == int64_t(a.dim) * BITS / 8 &&
           a.part[i].param_head_stride == int64_t(a.dim / a.group) * 4;
  if (flat) a.dim *= a.heads, a.heads = 1;
  // as many tokens a launch as 31-bit indices hold
  const int64_t most = std::max<int64_t>(1, INT32_MAX / (int64_t(a.heads) * a.dim));
  const int64_t n = a.n;
  for (int64_t t = 0; t < n; t += most) {
    a.n = std::min(most, n - t);
    a.slots = a0.slots + t;
    for (int i = 0; i < n_parts; ++i)
      a.x[i].data = static_cast<char*>(a0.x[i].data) + t * a0.x[i].token_stride * Elt<DT>::kBytes;
    const cudaError_t e = launch_piece<DT, BITS>(a, write, n_parts, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

lp_status run(const lp_cache_part* parts, const lp_heads* x, int64_t n_parts, int bits,
              lp_dtype dt, int64_t n_slots, int64_t page_size, int64_t heads, int64_t dim,
              int64_t group, const int64_t* slots, int64_t n, bool write, cudaStream_t stream) {
  if (dt != LP_F32 && dt != LP_F16 && dt != LP_BF16) return LP_ERR_UNSUPPORTED_DTYPE;
  if (n_parts < 0 || n_parts > kMaxParts || (bits != 8 && bits != 4) || n_slots < 0 ||
      page_size < 1 || heads < 0 || dim < 0 || group < 1 || dim % group != 0 ||
      (bits == 4 && group % 2 != 0) || n < 0)
    return LP_ERR_INVALID_ARGUMENT;
  // (a group's bytes are counted in 31 bits)
  if (heads > INT32_MAX || dim > INT32_MAX || group > (1 << 29)) return LP_ERR_TOO_LARGE;
  if (n_parts == 0 || n == 0 || heads == 0 || dim == 0) return LP_OK;
  if (heads > INT64_MAX / 4 / dim || n > INT64_MAX / 4 / (heads * dim)) return LP_ERR_TOO_LARGE;
  if (parts == nullptr || x == nullptr || slots == nullptr) return LP_ERR_INVALID_ARGUMENT;
  const int eb = dt == LP_F32 ? 4 : 2;
  for (int64_t i = 0; i < n_parts; ++i) {
    const lp_cache_part& p = parts[i];
    if (x[i].data == nullptr || reinterpret_cast<uintptr_t>(x[i].data) % eb != 0)
      return LP_ERR_INVALID_ARGUMENT;
    if (n_slots > 0 && (p.codes == nullptr || p.params == nullptr)) return LP_ERR_INVALID_ARGUMENT;
    if ((reinterpret_cast<uintptr_t>(p.params) | uint64_t(p.param_page_stride) |
         uint64_t(p.param_slot_stride) | uint64_t(p.param_head_stride)) % 4 != 0)
      return LP_ERR_INVALID_ARGUMENT;
  }
  CacheArgs a = {};
  for (int64_t i = 0; i < n_parts; ++i) a.part[i] = parts[i], a.x[i] = x[i];
  a.slots = slots;
  a.n = n;
  a.n_slots = n_slots;
  a.page = page_size;
  if (page_size < n_slots && n_slots <= INT32_MAX) a.per_page.set(uint32_t(page_size));
  a.heads = int(heads);
  a.dim = int(dim);
  a.group = int(group);
  const int np = int(n_parts);
  cudaError_t e;
  if (bits == 8)
    e = dt == LP_F32   ? launch<LP_F32, 8>(a, write, np, stream)
        : dt == LP_F16 ? launch<LP_F16, 8>(a, write, np, stream)
                       : launch<LP_BF16, 8>(a, write, np, stream);
  else
    e = dt == LP_F32   ? launch<LP_F32, 4>(a, write, np, stream)
        : dt == LP_F16 ? launch<LP_F16, 4>(a, write, np, stream)
                       : launch<LP_BF16, 4>(a, write, np, stream);
  return status_of(e);
}

}  // namespace
}  // namespace lp

extern "C" lp_status lp_cache_write(const lp_cache_part* parts, const lp_heads* x,
                                    int64_t n_parts, int32_t bits, lp_dtype dt, int64_t n_slots,
                                    int64_t page_size, int64_t heads, int64_t dim, int64_t group,
                                    const int64_t* slots, int64_t n, cudaStream_t stream) {
  return lp::run(parts, x, n_parts, bits, dt, n_slots, page_size, heads, dim, group, slots, n,
                 true, stream);
}

extern "C" lp_status lp_cache_read(const lp_cache_part* parts, const lp_heads* out,
                                   int64_t n_parts, int32_t bits, lp_dtype dt, int64_t n_slots,
                                   int64_t page_size, int64_t heads, int64_t dim, int64_t group,
                                   const int64_t* slots, int64_t n, cudaStream_t stream) {
  return lp::run(parts, out, n_parts, bits, dt, n_slots, page_size, heads, dim, group, slots, n,
                 false, stream);
}
