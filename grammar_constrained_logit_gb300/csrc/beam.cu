// beam.cu -- beam search's selection over beams and vocabulary, under the packed
// bitmask.
//
// For a live row r (score s_r above -inf, not finished) with kept tokens
// C_r = {v < vocab : bit set or row not masked, x_rv above -inf},
//   candidate (r, v):  s_r + ((x_rv - M_r) - log S_r),
//   M_r = max_{C_r} x,  S_r = sum_{C_r} exp(x - M_r).
// A finished row has one candidate, (pad, s_r).  A batch's n best candidates come
// out highest first, ties to the lowest (beam, token).
//
// Two kernels.
//
// The first reads the logits once, a chunk of 2 KB a warp (512 bytes where there would be
// few chunks to the n), and leaves (max, sum of exp(x - max)) of each: 8 bytes, so nothing
// of the size of the logits is written.  A chunk is a range of token indices, whatever the
// row's alignment, and its sum has a fixed order: two equal rows get equal scores to the
// last bit, and ties between them fall by index as stated.  What bounds it is memory, with
// the warps' own instructions (7.7 a token and lane, one of them the exponential) close
// behind: 128 x 8 rows of 202048 fp16 take 65 us, 6.3 TB/s, 93% of the measured copy rate.
//
// The second, one block (or a cluster of them) a batch entry, joins the chunks to M_r and
// S_r, takes the n-th largest chunk maximum's score as a lower bound T of the n-th best
// candidate, and reads again only the chunks whose maximum reaches T: about n of them,
// whatever the vocabulary.  It waits at each turn for what the last one found, some
// 10000 cycles in all: 5 us after the first kernel for a few rows, 8 with a full batch, 12
// with 4 x 64 beams to join.  Far more where the bound admits too much: 1 x 64 rows of
// 18000 bf16, n = 128, take 21 us, but 48 with one beam alive, whose 18 chunks are fewer
// than n and bound nothing.
#include <algorithm>

#include "common.cuh"

namespace lp {
namespace {

constexpr int kStreamThreads = 256;
constexpr int kVecs = 4;              // 16-byte groups a lane holds of a chunk, at most
constexpr int kFinishThreads = 512;   // of a block of the second kernel
constexpr int kFinishWarps = kFinishThreads / 32;
constexpr int kMaxSelect = 256;       // largest n_select and beams
constexpr int kBuf = 1024;            // candidates held at once (a power of two)
constexpr int kList = 2048;           // chunks gone through at once
constexpr int64_t kMostStaged = 128 * 1024;  // bytes of chunks' maxima held in shared memory
constexpr int kBufNew = kBuf - kMaxSelect;
constexpr int kSms = 152;

// Tokens of a chunk of N groups a lane: 512 f32 or 1024 of 16 bits with four; a quarter of
// that with one.
template <int DT, int N>
constexpr int kChunk = N * 32 * Elt<DT>::kPerVec;

struct BeamArgs {
  const char* logits;
  int64_t stride;  // bytes
  int64_t V;
  const uint32_t* bitmask;
  int64_t bm_stride;  // words
  const uint8_t* needs;
  const float* scores;
  const uint8_t* finished;
  int64_t pad;
  int rows, beams, n, chunks;
  int chunk_tokens;
  int step_rows, step_chunks;  // from a warp's chunk to its next
  int staged;      // a batch entry's chunks fit in shared memory
  int sum_bits;    // S <= V is held in units of 2^-sum_bits, within 63 bits
  float2* part;    // [rows, chunks]: (max, sum of exp(x - max)); of live rows only
  float* out_scores;
  int64_t* out_tokens;
  int32_t* out_parents;
};

struct Cand {
  uint64_t key;   // order-preserving bits of the score
  uint64_t flat;  // beam * 2^31 + token
};

__device__ __forceinline__ bool better(const Cand& a, const Cand& b) {
  return a.key > b.key || (a.key == b.key && a.flat < b.flat);
}

// Bytes sh .. sh+15 of the 32 bytes lo, hi.
__device__ __forceinline__ uint4 shifted(uint4 lo, uint4 hi, int sh) {
  if (sh & 8) lo = make_uint4(lo.z, lo.w, hi.x, hi.y), hi = make_uint4(hi.z, hi.w, 0, 0);
  if (sh & 4) lo = make_uint4(lo.y, lo.z, lo.w, hi.x), hi.x = hi.y;
  const int b = (sh & 3) * 8;
  return make_uint4(__funnelshift_r(lo.x, lo.y, b), __funnelshift_r(lo.y, lo.z, b),
                    __funnelshift_r(lo.z, lo.w, b), __funnelshift_r(lo.w, hi.x, b));
}

template <int DT>
__device__ __forceinline__ uint32_t neg_inf_word() {
  return DT == LP_F32 ? 0xff800000u : DT == LP_BF16 ? 0xff80ff80u : 0xfc00fc00u;
}

// Tokens j .. j+kPerVec-1 of a row whose address is sh bytes past a 16-byte boundary;
// tokens from V on come back as -inf.  Reads nothing outside the row's V tokens.
template <int DT>
__device__ __forceinline__ uint4 load_group(const char* __restrict__ row, int64_t j, int64_t V,
                                            int sh) {
  constexpr int E = Elt<DT>::kPerVec, Bt = Elt<DT>::kBytes;
  const char* p = row + j * Bt;
  if (sh == 0) {
    if (j + E <= V) return __ldg(reinterpret_cast<const uint4*>(p));
  } else if (j > 0 && j + 2 * E <= V) {
    const uint4* q = reinterpret_cast<const uint4*>(p - sh);
    return shifted(__ldg(q), __ldg(q + 1), sh);
  }
  // the row's first and last tokens: one at a time
  uint32_t w[4];
  const uint32_t none = neg_inf_word<DT>();
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = none;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (j + e < V) {
      const uint32_t b = Elt<DT>::bits1(p + e * Bt);
      if (Bt == 4) w[e] = b;
      else w[e / 2] = (e & 1) ? ((w[e / 2] & 0xffffu) | (b << 16)) : ((w[e / 2] & 0xffff0000u) | b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Keep bits of a group's tokens (bits of tokens from V on: clear).
template <int DT>
__device__ __forceinline__ uint32_t group_keep(const uint32_t* __restrict__ bm, int64_t j,
                                               int64_t V) {
  constexpr int E = Elt<DT>::kPerVec;
  if (j >= V) return 0u;
  uint32_t k = (1u << E) - 1u;
  if (V - j < E) k = (1u << int(V - j)) - 1u;
  if (bm != nullptr) {
    const uint32_t b = __ldg(reinterpret_cast<const uint8_t*>(bm) + (j >> 3));
    k &= E == 8 ? b : (b >> (j & 4));
  }
  return k;
}

// Keep bits of a lane's tokens in a chunk, a group's in E bits; clear from V on.
template <int DT, int N>
__device__ __forceinline__ uint32_t chunk_keep(const uint32_t* bm, int64_t j0, int64_t V,
                                               int lane) {
  constexpr int E = Elt<DT>::kPerVec;
  uint32_t keep = 0;
  if (unsigned(j0) + kChunk<DT, N> <= unsigned(V)) {
    if (bm == nullptr) return N * E == 32 ? 0xffffffffu : (1u << (N * E)) - 1u;
    const uint8_t* mask = reinterpret_cast<const uint8_t*>(bm) + (j0 + lane * E) / 8;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint32_t m = __ldg(mask + i * (4 * E));
      if (E == 4) m = m >> (lane & 1) * 4 & 15u;
      keep |= m << (i * E);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      keep |= group_keep<DT>(bm, j0 + (i * 32 + lane) * E, V) << (i * E);
  }
  return keep;
}

// What a group's words keep, by its keep bits: looked up instead of worked out for each
// word (5 instructions a group instead of 28 for 8 tokens).
template <int DT>
struct KeepTable {
  uint4 words[1 << Elt<DT>::kPerVec];
  __device__ __forceinline__ void fill() {  // by a block of at least as many threads
    const uint32_t k = threadIdx.x;
    if (k >= (1u << Elt<DT>::kPerVec)) return;
    words[k] = DT == LP_F32 ? make_uint4(k & 1 ? ~0u : 0u, k & 2 ? ~0u : 0u, k & 4 ? ~0u : 0u,
                                         k & 8 ? ~0u : 0u)
                            : make_uint4(keep_mask16(k, 0), keep_mask16(k, 1), keep_mask16(k, 2),
                                         keep_mask16(k, 3));
  }
  __device__ __forceinline__ uint4 kept(const uint4& v, uint32_t k) const {
    const uint4 m = words[k];
    const uint32_t none = neg_inf_word<DT>();
    return make_uint4((v.x & m.x) | (none & ~m.x), (v.y & m.y) | (none & ~m.y),
                      (v.z & m.z) | (none & ~m.z), (v.w & m.w) | (none & ~m.w));
  }
};

// A chunk's groups of this lane, masked tokens as -inf.  ALL: groups that the mask leaves
// out are loaded too, so that the loads do not wait for its bits.
template <int DT, int N, bool ALL>
__device__ __forceinline__ void load_chunk(uint4 (&v)[N], const char* row, uint32_t keep,
                                           bool masked, int64_t j0, int64_t V, int lane,
                                           const KeepTable<DT>* table = nullptr) {
  constexpr int E = Elt<DT>::kPerVec;
  constexpr uint32_t kAll = (1u << E) - 1u;
  const int sh = int(reinterpret_cast<uintptr_t>(row) & 15);
  const uint32_t none = neg_inf_word<DT>();
  // (V is below 2^31: 32-bit comparisons do)
  if (unsigned(j0) + kChunk<DT, N> + (sh ? E : 0) <= unsigned(V) && (sh == 0 || j0 > 0)) {
    // within the row: nothing to check token by token
    const uint4* p = reinterpret_cast<const uint4*>(row + (j0 + lane * E) * Elt<DT>::kBytes - sh);
    if (!masked) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[i] = sh == 0 ? __ldg(p + i * 32) : shifted(__ldg(p + i * 32), __ldg(p + i * 32 + 1), sh);
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!ALL) v[i] = make_uint4(none, none, none, none);
      if (ALL || (keep >> (i * E) & kAll))
        v[i] = sh == 0 ? __ldg(p + i * 32) : shifted(__ldg(p + i * 32), __ldg(p + i * 32 + 1), sh);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t j = j0 + (i * 32 + lane) * E;
      v[i] = make_uint4(none, none, none, none);
      if (ALL ? j < V : (keep >> (i * E) & kAll) != 0) v[i] = load_group<DT>(row, j, V, sh);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t k = keep >> (i * E) & kAll;
    if (table) v[i] = table->kept(v[i], k);
    else if (k != kAll) v[i] = Elt<DT>::blend(v[i], k, none);
  }
}

// Element `at` of a chunk's groups, a number known only at run time.
template <int DT>
__device__ __forceinline__ float element(const uint4 (&v)[kVecs], unsigned at) {
  constexpr unsigned E = Elt<DT>::kPerVec;
  const unsigned g = at / E, e = at % E;
  const uint4 lo = g & 1 ? v[1] : v[0], hi = g & 1 ? v[3] : v[2];
  const uint4 w = g & 2 ? hi : lo;
  if (DT == LP_F32) return __uint_as_float(e & 2 ? (e & 1 ? w.w : w.z) : (e & 1 ? w.y : w.x));
  const uint32_t pair = e & 4 ? (e & 2 ? w.w : w.z) : (e & 2 ? w.y : w.x);
  const uint32_t half = e & 1 ? pair >> 16 : pair & 0xffffu;
  return DT == LP_BF16 ? __uint_as_float(half << 16) : Elt<LP_F16>::half_bits_to_float(half);
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  return uint64_t(__float_as_uint(a)) | uint64_t(__float_as_uint(b)) << 32;
}
__device__ __forceinline__ float low_of(uint64_t v) { return __uint_as_float(uint32_t(v)); }
__device__ __forceinline__ float high_of(uint64_t v) { return __uint_as_float(uint32_t(v >> 32)); }

constexpr float kLog2e = 1.44269504f;

// The differences x - m of two neighbouring tokens, rounded once from the 16-bit value:
// the mixed-type addition needs no conversion, whose unit the exponentials want.
template <int DT>
__device__ __forceinline__ uint64_t differences(const uint4& v, int e, float m) {
  if (DT == LP_F32) return add2(pack2(Elt<DT>::get(v, e), Elt<DT>::get(v, e + 1)), pack2(-m, -m));
  const uint32_t w = word_of(v, e >> 1);
  const uint16_t a = uint16_t(w), b = uint16_t(w >> 16);
  float x, y;
  if (DT == LP_BF16) {
    asm("add.rn.f32.bf16 %0, %1, %2;" : "=f"(x) : "h"(a), "f"(-m));
    asm("add.rn.f32.bf16 %0, %1, %2;" : "=f"(y) : "h"(b), "f"(-m));
  } else {
    asm("add.rn.f32.f16 %0, %1, %2;" : "=f"(x) : "h"(a), "f"(-m));
    asm("add.rn.f32.f16 %0, %1, %2;" : "=f"(y) : "h"(b), "f"(-m));
  }
  return pack2(x, y);
}

// Sum over a lane's tokens of exp(x - m).  The difference comes first: it is exact near
// the maximum, where the sum comes from, however far from zero the logits are.  -inf
// gives 2^-inf = 0; a NaN, or m infinite, gives NaN, and the caller sums again with care.
template <int DT, int N>
__device__ __forceinline__ float sum_exp(const uint4 (&v)[N], float m) {
  const uint64_t scale = pack2(kLog2e, kLog2e);
  uint64_t s[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int e = 0; e < Elt<DT>::kPerVec; e += 2) {
      const uint64_t t = mul2(differences<DT>(v[i], e, m), scale);
      s[i & 1] = add2(s[i & 1], pack2(ex2(low_of(t)), ex2(high_of(t))));
    }
  }
  const uint64_t both = add2(s[0], s[1]);
  return low_of(both) + high_of(both);
}

// The same where there is a NaN, which is no candidate, or a maximum of +inf, whose
// tokens share all of the mass.
template <int DT, int N>
__device__ __forceinline__ float sum_exp_careful(const uint4 (&v)[N], float m) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < Elt<DT>::kPerVec; ++e) {
      const float x = Elt<DT>::get(v[i], e);
      if (x == m) s += 1.0f;
      else if (x > -INFINITY && m < INFINITY) s += ex2((x - m) * kLog2e);
    }
  return s;
}

__device__ __forceinline__ float warp_max(float m) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(m));
  return r;
}

// What a warp knows of a chunk before it reads its tokens.
template <int DT, int N>
struct At {
  int row, c;
  bool live, masked;
  uint32_t keep;

  // AT_ONCE: the loads do not wait for one another; the mask is read for nothing where the
  // row is dead or not masked.
  template <bool AT_ONCE>
  __device__ __forceinline__ void find(const BeamArgs& a, int lane) {
    const float s = __ldg(a.scores + row);
    const uint8_t fin = a.finished != nullptr ? __ldg(a.finished + row) : 0;
    const uint8_t need = a.needs != nullptr ? __ldg(a.needs + row) : 1;
    masked = a.bitmask != nullptr;
    if (!AT_ONCE) {
      masked = masked && need != 0;
      live = s > -INFINITY && fin == 0;
    }
    const int64_t j0 = int64_t(c) * kChunk<DT, N>;
    if (AT_ONCE || live)
      keep = chunk_keep<DT, N>(masked ? a.bitmask + int64_t(row) * a.bm_stride : nullptr, j0, a.V,
                               lane);
    if (AT_ONCE) {
      if (masked && need == 0) keep = chunk_keep<DT, N>(nullptr, j0, a.V, lane), masked = false;
      live = s > -INFINITY && fin == 0;
    }
  }
};

// EARLY: for problems of one chunk a warp, which only wait for memory: the tokens' loads
// wait neither for the row's state nor for its mask.  Loads overlap between warps, not
// within one.  A second chunk in registers (79 of them) took the blocks of an SM from 5 to
// 3 and 128 x 8 rows of 202048 fp16 from 76 to 88 us; the next chunk's state and mask
// asked for ahead took 24 x 5 rows of 65519 from 12.7 to 14.0 us; the next chunk copied
// into shared memory meanwhile took the former to 83 us, the latter to 13.5.  What bounds
// a warp is its own instructions, 7.7 a token.  None of these cases has a mask.
template <int DT, int N, bool EARLY>
__global__ void __launch_bounds__(kStreamThreads, EARLY ? 5 : 6) beam_stream_kernel(BeamArgs a) {
  __shared__ KeepTable<DT> table;
  table.fill();
  __syncthreads();
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int lane = threadIdx.x & 31;
  const unsigned total = unsigned(a.rows) * unsigned(a.chunks);
  const unsigned step = gridDim.x * (kStreamThreads / 32);
  unsigned w = blockIdx.x * (kStreamThreads / 32) + (threadIdx.x >> 5);
  At<DT, N> at;
  at.row = int(w / unsigned(a.chunks)), at.c = int(w % unsigned(a.chunks));
  for (; w < total; w += step) {
    const int row = at.row, c = at.c;
    at.template find<EARLY>(a, lane);
    uint4 v[N];
    if (EARLY || at.live)
      load_chunk<DT, N, EARLY>(v, a.logits + row * a.stride, at.keep, at.masked,
                               int64_t(c) * kChunk<DT, N>, a.V, lane, &table);
    if (!EARLY) {  // (a division is as much as 4 tokens)
      at.row += a.step_rows, at.c += a.step_chunks;
      if (at.c >= a.chunks) at.c -= a.chunks, ++at.row;
    }
    if (!at.live) continue;
    float m = VecMax<DT>::run(v[0], 0xffu);
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, VecMax<DT>::run(v[i], 0xffu));
    m = fmaxf(warp_max(m), -INFINITY);  // nothing but NaN: no candidate
    float sum = sum_exp<DT, N>(v, m);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullWarp, sum, o);
    if (!(sum < INFINITY)) {
      sum = 0.0f;
      if (m > -INFINITY) sum = sum_exp_careful<DT, N>(v, m);
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullWarp, sum, o);
    }
    if (lane == 0) a.part[w] = make_float2(m, sum);
  }
}

// Sorts m candidates at c (best first); c has room for the next power of two.
__device__ void sort_best_first(Cand* c, int m) {
  int p = 2;
  while (p < m) p <<= 1;
  for (int i = m + threadIdx.x; i < p; i += kFinishThreads) c[i] = Cand{0, ~0ull};
  __syncthreads();
  for (int k = 2; k <= p; k <<= 1) {
    for (int j = k >> 1; j; j >>= 1) {
      for (int t = threadIdx.x; t < p / 2; t += kFinishThreads) {
        const int lo = 2 * t - (t & (j - 1)), hi = lo + j;
        const Cand x = c[lo], y = c[hi];
        if (better(y, x) == ((lo & k) == 0)) c[lo] = y, c[hi] = x;
      }
      __syncthreads();
    }
  }
}

// A value held as two floats: hi is the value rounded, lo what that left.  Scores are
// summed in this form, which holds 48 bits and more: 64-bit arithmetic is 1/64 of the
// 32-bit rate here, and the few dozen operations a batch entry needs took 1000 cycles.
struct Two {
  float hi, lo;
};

__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return Two{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}

__device__ __forceinline__ uint64_t key_of(Two v) {
  if (!(fabsf(v.hi) < INFINITY)) v.lo = 0.0f;
  // as 64-bit arithmetic rounds it: lo to a multiple of 2^-52 of hi's leading bit, which
  // a lo of 2^-29 of that and more is already
  const uint32_t e = __float_as_uint(v.hi) & 0x7f800000u;
  if (e > (29u << 23)) {
    const float b = __uint_as_float(e - (29u << 23));
    if (fabsf(v.lo) < b) v.lo = __fsub_rn(__fadd_rn(v.lo, 1.5f * b), 1.5f * b);
  }
  return uint64_t(fkey(v.hi)) << 32 | fkey(v.lo);
}

__device__ __forceinline__ float key_score(uint64_t k) { return key_float(uint32_t(k >> 32)); }

constexpr uint64_t kNoScore = 0x007fffffull << 32 | 0xffffffffull;  // keys of -inf: none above

// The same for 32 < m <= kFinishThreads, one candidate a thread in registers: neighbours up
// to 16 places apart meet by shuffles, the others through c.  Returns this thread's, in order.
__device__ __forceinline__ Cand sorted_in_threads(Cand* c, int m) {
  const int t = threadIdx.x;
  Cand x = t < m ? c[t] : Cand{0, ~0ull};
  __syncthreads();
  int p = 2;
  while (p < m) p <<= 1;
  for (int k = 2; k <= p; k <<= 1) {
    for (int j = k >> 1; j; j >>= 1) {
      Cand y;
      if (j < 32) {
        if (t >= p) continue;  // (whole warps: p is at least 32 here)
        y.key = __shfl_xor_sync(kFullWarp, x.key, j);
        y.flat = __shfl_xor_sync(kFullWarp, x.flat, j);
      } else {
        if (t < p) c[t] = x;
        __syncthreads();
        if (t < p) y = c[t ^ j];
        __syncthreads();
        if (t >= p) continue;
      }
      const bool first = ((t & j) == 0) == ((t & k) == 0);  // the better one belongs here
      if (better(y, x) == first) x = y;
    }
  }
  return x;
}

// log of a whole number of units, to 2^-38: the number's leading 7 bits choose
// c near 1/m, a 10-bit number whose logarithm is tabled (the table-driven scheme of
// Tang, ACM TOMS 16(4), 1990); t = m c - 1 is below 2^-7 and its series is short.
struct LogEntry {
  float c, hi, lo;  // -log c = hi + lo
};
struct LogTable {
  LogEntry at[128];
};

constexpr double series_log(double x) {  // 2 artanh((x - 1) / (x + 1)), x in [1/2, 1]
  const double u = (x - 1.0) / (x + 1.0), uu = u * u;
  double term = u, sum = 0.0;
  for (int k = 1; k < 80; k += 2) {
    sum += term / k;
    term *= uu;
  }
  return 2.0 * sum;
}

constexpr LogTable make_log_table() {
  LogTable t{};
  for (int i = 0; i < 128; ++i) {
    const double c = double(int(1024.0 / (1.0 + (i + 0.5) / 128.0) + 0.5)) / 1024.0;
    const double v = -series_log(c);
    t.at[i].c = float(c);
    t.at[i].hi = float(v);
    t.at[i].lo = float(v - double(float(v)));
  }
  return t;
}

__device__ const LogTable kLogTable = make_log_table();

// log(S / 2^bits), S > 0.  Exactly 0 for a row of one token, which then scores as a
// finished beam would.
__device__ __forceinline__ Two log_units(unsigned long long S, int bits, const LogEntry* table) {
  if (S == 1ull << bits) return Two{0.0f, 0.0f};
  const int lz = __clzll(S);
  const unsigned long long f = S << lz;  // m = f / 2^63 in [1, 2)
  const LogEntry q = table[unsigned(f >> 56) & 127u];
  const float mh = float(unsigned(f >> 40)) * 0x1p-23f;
  const float ml = float(unsigned(f >> 16) & 0xffffffu) * 0x1p-47f;
  const float p = __fmul_rn(mh, q.c);
  const float th = __fsub_rn(p, 1.0f);  // exact: p is near 1
  const Two t = two_sum(th, __fmaf_rn(ml, q.c, __fmaf_rn(mh, q.c, -p)));
  // t - t^2/2 + t^3 (1/3 - t/4 + t^2/5 - t^3/6)
  const float sq = __fmul_rn(t.hi, t.hi);
  const float sq_lo = __fmaf_rn(2.0f * t.hi, t.lo, __fmaf_rn(t.hi, t.hi, -sq));
  const float rest = t.hi * sq *
      __fmaf_rn(t.hi, __fmaf_rn(t.hi, __fmaf_rn(t.hi, -1.0f / 6, 0.2f), -0.25f), 1.0f / 3);
  const float e = float(63 - lz - bits);
  // log 2 = 0x1.62e4p-1 (15 bits, so e times it is exact) + 0x1.7f7d1cp-20
  Two r = two_sum(e * 0x1.62e4p-1f, q.hi);
  float lo = __fadd_rn(r.lo, __fmaf_rn(e, 0x1.7f7d1cp-20f, q.lo));
  r = two_sum(r.hi, t.hi);
  lo = __fadd_rn(lo, __fadd_rn(r.lo, t.lo));
  r = two_sum(r.hi, -0.5f * sq);
  lo = __fadd_rn(lo, __fadd_rn(r.lo, __fmaf_rn(-0.5f, sq_lo, rest)));
  return two_sum(r.hi, lo);
}

enum { kOn, kAgain, kStretches };

struct FinishSmem {
  Cand buf[kBuf];             // what is new; the best so far joins behind it to be sorted
  Cand front[kMaxSelect];     // the best so far, sorted
  Two log_s[kMaxSelect];      // log S
  float score[kMaxSelect];
  float top[kMaxSelect];      // M; -inf: a beam without candidates
  uint8_t ended[kMaxSelect];  // finished: one candidate, its own score
  uint8_t masked[kMaxSelect];
  unsigned best[kFinishThreads];  // each thread's, which the bound is taken from
  LogEntry log_table[128];
  unsigned list[kList];       // chunks to go through
  int list_n, count, front_n, exact, overflow, next, raised;
  float T;
  Cand bound;                 // exact: candidates worse than this are out
};

// s + ((x - M) - log S)
__device__ __forceinline__ Two score_of(const FinishSmem& sm, int k, float x) {
  const float M = sm.top[k];
  if (!(M < INFINITY) && x != M) return Two{-INFINITY, 0.0f};  // +inf tokens share all
  const Two z = sm.log_s[k];
  Two d{0.0f, 0.0f};
  if (x != M) d = two_sum(x, -M);
  if (!(d.hi > -INFINITY)) return Two{-INFINITY, 0.0f};  // out of the 32-bit range
  Two e = two_sum(d.hi, -z.hi);
  e = two_sum(e.hi, __fadd_rn(e.lo, __fsub_rn(d.lo, z.lo)));
  Two f = two_sum(sm.score[k], e.hi);
  if (!(fabsf(f.hi) < INFINITY)) return Two{f.hi, 0.0f};
  return two_sum(f.hi, __fadd_rn(f.lo, e.lo));
}

// A logit of beam k below this cannot reach a score of T: 32-bit arithmetic, taken low by
// more than its rounding.
__device__ __forceinline__ float least_of(const FinishSmem& sm, int k, float T) {
  const float s = sm.score[k], M = sm.top[k], z = sm.log_s[k].hi;
  if (!(T > -INFINITY && s < INFINITY && M < INFINITY)) return -INFINITY;
  const float slack = 0x1p-20f * (fabsf(T) + fabsf(s) + fabsf(z) + fabsf(M)) + 0x1p-20f;
  const float x = (((T - s) + z) + M) - slack;
  return x < INFINITY ? x : -INFINITY;  // out of the 32-bit range: no bound
}

// Joins the first m new candidates with the best so far and makes the n-th best the
// bound.  keep: the n best become the best so far; else only the bound is taken.
__device__ __noinline__ void join(FinishSmem& sm, int m, int n, bool keep) {
  __syncthreads();
  const int front_n = sm.front_n;
  for (int t = threadIdx.x; t < front_n; t += kFinishThreads) sm.buf[m + t] = sm.front[t];
  __syncthreads();
  sort_best_first(sm.buf, m + front_n);
  const int have = min(m + front_n, n);
  if (keep)
    for (int t = threadIdx.x; t < have; t += kFinishThreads) sm.front[t] = sm.buf[t];
  if (threadIdx.x == 0) {
    if (have == n) sm.bound = sm.buf[n - 1], sm.exact = 1, sm.T = key_score(sm.bound.key);
    if (keep) sm.front_n = have;
    sm.count = 0;
  }
  __syncthreads();
}

// A lower bound of the score that a beam's chunk of maximum m holds.
__device__ __forceinline__ unsigned low_key(float s, float M, float z, float m) {
  const float d = m == M ? 0.0f : m - M;
  const float low = (s + (d - z)) - (0x1p-20f * (fabsf(s) + fabsf(d) + fabsf(z)) + 0x1p-20f);
  return fkey(low > -INFINITY ? low : s == INFINITY ? s : -INFINITY);
}

// One beam, by one warp: M and S from its chunks, the chunks' maxima staged.  Returns the
// lower bound of this lane's best chunk.
__device__ __forceinline__ unsigned beam_sums(FinishSmem& sm, const BeamArgs& a, int row0, int k,
                                              float* staged) {
  constexpr int kHeld = 8;  // chunks a lane keeps in registers; a longer row is read again
  const int lane = threadIdx.x & 31, C = a.chunks, row = row0 + k;
  const float2* p = a.part + int64_t(row) * C;
  // all of these are on their way at once; chunks of a dead row are garbage, not used
  float2 q[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    q[i] = lane + 32 * i < C ? p[lane + 32 * i] : make_float2(-INFINITY, 0.0f);
  const float s = __ldg(a.scores + row);
  const uint8_t fin = a.finished != nullptr ? __ldg(a.finished + row) : 0;
  const uint8_t need = a.needs != nullptr ? __ldg(a.needs + row) : 1;
  const bool alive = s > -INFINITY, ended = alive && fin != 0;
  float M = -INFINITY, mine = -INFINITY;
  Two z{0.0f, 0.0f};
  if (alive && !ended) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (staged && lane + 32 * i < C) staged[lane + 32 * i] = q[i].x;
      mine = fmaxf(mine, q[i].x);
    }
    for (int c = lane + 32 * kHeld; c < C; c += 32) {
      const float m = p[c].x;
      if (staged) staged[c] = m;
      mine = fmaxf(mine, m);
    }
    M = key_float(__reduce_max_sync(kFullWarp, fkey(mine)));
    // whole multiples of a unit: their sum is exact, whatever its order.  S is at least 1
    // and the unit 2^-40 (vocabularies up to 2^23), so what a term loses does not count
    const float unit = __uint_as_float(unsigned(127 + a.sum_bits) << 23);
    unsigned long long S = 0;
    auto term = [&](float2 v) {
      if (v.x > -INFINITY) S += __float2ull_rn((v.x == M ? v.y : v.y * expf(v.x - M)) * unit);
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (32 * i < C) term(q[i]);
    for (int c = lane + 32 * kHeld; c < C; c += 32) term(p[c]);
    // 64-bit lanes in limbs of 22 bits: 32 of them stay within 32 bits
    const unsigned l0 = __reduce_add_sync(kFullWarp, unsigned(S) & 0x3fffffu);
    const unsigned l1 = __reduce_add_sync(kFullWarp, unsigned(S >> 22) & 0x3fffffu);
    const unsigned l2 = __reduce_add_sync(kFullWarp, unsigned(S >> 44));
    S = l0 + ((unsigned long long)l1 << 22) + ((unsigned long long)l2 << 44);
    if (M > -INFINITY) z = log_units(S, a.sum_bits, sm.log_table);
  }
  if (lane == 0) {
    sm.score[k] = alive ? s : -INFINITY;
    sm.ended[k] = ended;
    sm.masked[k] = a.bitmask != nullptr && need != 0;
    sm.top[k] = ended ? 0.0f : M;
    sm.log_s[k] = z;
  }
  if (ended) return lane == 0 ? fkey(s) : 0;
  return mine > -INFINITY ? low_key(s, M, z.hi, mine) : 0;
}

// The n-th largest of the warp's keys, N a lane, taken low: measured from the largest, in
// steps of 1/64 of the distance (1/1024 at the least), as a bound need not be tight.  -inf
// when fewer than n are there.
__device__ __forceinline__ unsigned key_at(const unsigned* keys, int i) { return keys[i]; }
__device__ __forceinline__ unsigned key_at(const Cand* c, int i) { return unsigned(c[i].key >> 32); }

template <int N, typename K>
__device__ __forceinline__ float nth_largest(const K* keys, int n) {
  constexpr int kBase = (127 - 4) << 6;  // 2^-4, in steps of 2^-6 of a power of two
  const int lane = threadIdx.x & 31;
  unsigned mine[N], most = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) most = max(most, mine[i] = key_at(keys, i * 32 + lane));
  most = __reduce_max_sync(kFullWarp, most);
  const float top = key_float(most);
  int near[N];  // 2047 at the largest, 0 where there is none or it is 2^28 away
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float d = mine[i] == most ? 0.0f : top - key_float(mine[i]);
    const int q = int(__float_as_uint(d + 0x1p-4f) >> 17) - kBase;
    near[i] = mine[i] == 0 || !(d < 0x1p27f) ? 0 : max(0, 2047 - q);
  }
  int T = 0;
#pragma unroll 1  // the kernel runs through its code once: less of it is less to fetch
  for (int sh = 10; sh >= 0; sh -= 2) {
    unsigned there[4] = {0, 0, 0, 0};  // three counts of up to 512, ten bits each
#pragma unroll
    for (int i = 0; i < N; ++i) {
      there[i & 3] += near[i] >= (T | 1 << sh) ? 1u : 0u;
      there[i & 3] += near[i] >= (T | 2 << sh) ? 1u << 10 : 0u;
      there[i & 3] += near[i] >= (T | 3 << sh) ? 1u << 20 : 0u;
    }
    const unsigned all = __reduce_add_sync(kFullWarp, (there[0] + there[1]) + (there[2] + there[3]));
    const int c1 = all & 1023u, c2 = all >> 10 & 1023u, c3 = all >> 20;
    T |= (c3 >= n ? 3 : c2 >= n ? 2 : c1 >= n ? 1 : 0) << sh;
  }
  if (T == 0) return -INFINITY;
  if (!(top < INFINITY)) return top;
  const float d = __uint_as_float(unsigned(2047 - T + 1 + kBase) << 17) - 0x1p-4f;
  return top - (d + 0x1p-20f * (fabsf(top) + d));
}

// A cluster's blocks share one batch entry: each goes through its part of the chunks, the
// first holds what they find.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n"
               "barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// Only while that block is sure to run: the first one is left last, and nobody reads it
// behind the barrier that may be its last; what it has to say it writes to the others
// before that.
__device__ __forceinline__ FinishSmem* of_block(FinishSmem* p, int rank) {
  uint64_t r;
  asm("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<FinishSmem*>(r);
}

template <int DT, int R, int B>
__global__ void __launch_bounds__(kFinishThreads, B) beam_finish_kernel(BeamArgs a) {
  extern __shared__ __align__(16) char raw[];
  FinishSmem& sm = *reinterpret_cast<FinishSmem*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / R, rank = blockIdx.x % R, row0 = b * a.beams, C = a.chunks;
  FinishSmem& hub = R > 1 ? *of_block(&sm, 0) : sm;
  float* staged = a.staged ? reinterpret_cast<float*>(raw + sizeof(FinishSmem)) : nullptr;
  if (tid == 0) sm.count = 0, sm.front_n = 0, sm.list_n = 0, sm.exact = 0, sm.overflow = 0;
  for (int i = tid; i < 128; i += kFinishThreads) sm.log_table[i] = kLogTable.at[i];
  if (R > 1) cluster_sync();
  else __syncthreads();
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  unsigned best = 0;
  for (int k = warp; k < a.beams; k += kFinishWarps)
    best = max(best, beam_sums(sm, a, row0, k, staged ? staged + k * C : nullptr));

  // From here a turn takes 32 chunks a warp: of as many beams as there are warps, or of
  // fewer beams with several warps to each.
  auto chunk_max = [&](int k, int c) {
    return staged ? staged[k * C + c] : a.part[int64_t(row0 + k) * C + c].x;
  };
  const int per_turn = min(a.beams, kFinishWarps), share = kFinishWarps / per_turn;
  const int my_beam = warp % per_turn, my_share = warp / per_turn;
  const int c_first = my_share < share ? my_share * 32 + lane : INT32_MAX, c_step = share * 32;

  // A lower bound T of the n-th best score: the n-th largest of these lanes' bests, each a
  // candidate of its own.  With few lanes to the n, of one chunk a thread instead.
  const bool few = min(C, 32) * per_turn < 4 * a.n;
  if (few) {
    __syncthreads();
    best = 0;
    const unsigned total = unsigned(a.beams) * unsigned(C);
    for (unsigned i = tid; i < total; i += kFinishThreads) {
      const int k = int(i / unsigned(C)), c = int(i % unsigned(C));
      const float M = sm.top[k], s = sm.score[k];
      if (M == -INFINITY) continue;
      if (sm.ended[k]) {
        if (c == 0) best = max(best, fkey(s));
        continue;
      }
      const float m = chunk_max(k, c);
      if (m > -INFINITY) best = max(best, low_key(s, M, sm.log_s[k].hi, m));
    }
  }
  sm.best[tid] = best;
  __syncthreads();
  if (warp == 0) {
    constexpr int W = kFinishWarps;
    const int used = few ? W : a.beams;  // warps whose lanes have found something
    const float T = used * 4 <= W   ? nth_largest<W / 4>(sm.best, a.n)
                    : used * 2 <= W ? nth_largest<W / 2>(sm.best, a.n)
                                    : nth_largest<W>(sm.best, a.n);
    if (lane == 0) sm.T = T;
  }
  __syncthreads();

  // Chunks whose maximum reaches the bound are listed and gone through, all of them at
  // once; where the list overflows, again from the start in stretches that it holds.
  bool whole = true;
  int k0 = 0, turn = 0;
  const int turns = (C + c_step - 1) / c_step;
  for (;;) {
    if (whole) {
      for (int k = my_beam; k < a.beams; k += per_turn) {
        if (sm.top[k] == -INFINITY) continue;
        const bool ended = sm.ended[k];
        const float least = ended ? sm.T : least_of(sm, k, sm.T);
        for (int c = c_first; c < C; c += c_step) {
          if (R > 1 && c % R != rank) continue;
          const float m = ended ? (c ? -INFINITY : sm.score[k]) : chunk_max(k, c);
          if (m > -INFINITY && m >= least) {
            const int at = atomicAdd(&sm.list_n, 1);
            if (at < kList) sm.list[at] = unsigned(k) << 22 | unsigned(c);
            else hub.overflow = 1;
          }
        }
      }
      k0 = a.beams;
    } else {
      // of 32 neighbouring chunks each of R blocks has 32 / R
      for (int i = 0; i < kList * R / kFinishThreads && k0 < a.beams; ++i) {
        const int k = k0 + my_beam;
        const int64_t c = int64_t(c_first) + int64_t(turn) * c_step;
        if (k < a.beams && c < C && sm.top[k] > -INFINITY && (R == 1 || int(c) % R == rank)) {
          const bool ended = sm.ended[k];
          const float m = ended ? (c ? -INFINITY : sm.score[k]) : chunk_max(k, int(c));
          if (m > -INFINITY && m >= (ended ? sm.T : least_of(sm, k, sm.T)))
            sm.list[atomicAdd(&sm.list_n, 1)] = unsigned(k) << 22 | unsigned(c);
        }
        if (++turn == turns) turn = 0, k0 += per_turn;
      }
    }
    __syncthreads();
    const int n_list = min(sm.list_n, kList);
    for (;;) {
      const bool exact = sm.exact;
      for (int l = warp; l < n_list; l += kFinishWarps) {
        const unsigned id = sm.list[l];
        const int k = int(id >> 22), c = int(id & 0x3fffffu);
        const uint64_t flat0 = uint64_t(k) << 31;
        auto found = [&](const Cand& y) {
          if (exact && better(sm.bound, y)) return;
          const int at = atomicAdd(&hub.count, 1);
          if (at < kBufNew) hub.buf[at] = y;
        };
        if (sm.ended[k]) {
          if (lane == 0) found(Cand{key_of(Two{sm.score[k], 0.0f}), flat0});
          continue;
        }
        const float least = least_of(sm, k, sm.T);
        const char* row = a.logits + int64_t(row0 + k) * a.stride;
        const uint32_t* bm = sm.masked[k] ? a.bitmask + int64_t(row0 + k) * a.bm_stride : nullptr;
        // (a small chunk is the beginning of a large one that ends there)
        const int64_t j0 = int64_t(c) * a.chunk_tokens, end = min(a.V, j0 + a.chunk_tokens);
        uint4 v[kVecs];
        load_chunk<DT, kVecs, true>(v, row, chunk_keep<DT, kVecs>(bm, j0, end, lane),
                                    bm != nullptr, j0, end, lane);
        uint32_t hits = 0;
#pragma unroll
        for (int g = 0; g < kVecs; ++g) {
          if (!(VecMax<DT>::run(v[g], 0xffu) >= least)) continue;
#pragma unroll
          for (int e = 0; e < Elt<DT>::kPerVec; ++e) {
            const float x = Elt<DT>::get(v[g], e);
            if (x >= least && x > -INFINITY) hits |= 1u << (g * Elt<DT>::kPerVec + e);
          }
        }
        for (; hits; hits &= hits - 1) {
          const unsigned bit = __ffs(hits) - 1;
          const unsigned j = unsigned(j0) + lane * Elt<DT>::kPerVec +
                             bit / Elt<DT>::kPerVec * (32 * Elt<DT>::kPerVec) +
                             bit % Elt<DT>::kPerVec;
          found(Cand{key_of(score_of(sm, k, element<DT>(v, bit))), flat0 + j});
        }
      }
      if (R > 1) cluster_sync();
      else __syncthreads();
      // the first block looks at what there is, the others wait for what it says
      if (R == 1 || rank == 0) {
        const int count = sm.count;
        int next = kOn;
        if (sm.overflow) {
          next = kStretches;
          __syncthreads();  // everyone has seen it before it is taken back
        } else if (count > kBufNew) {
          // too many: what was seen raises the bound, and the list is gone through again.
          // By its score where that is above the last, else by the whole order (strictly,
          // as kBufNew > n and no two candidates are equal)
          next = kAgain;
          if (!exact) {
            if (warp == 0) {
              const float T = nth_largest<kFinishWarps>(sm.buf, a.n);
              if (lane == 0) sm.raised = T > sm.T, sm.T = fmaxf(T, sm.T);
            }
            __syncthreads();
          }
          if (exact || !sm.raised) join(sm, kBufNew, a.n, false);
          else if (tid == 0) sm.count = 0;
        } else if (k0 < a.beams) {
          join(sm, count, a.n, true);  // with chunks to come, the n best are kept
        }
        if (tid == 0) {
          sm.next = next;
          if (next == kStretches) sm.count = 0, sm.overflow = 0;
        }
      }
      if (R > 1) {
        if (rank == 0) {
          __syncthreads();
          if (tid > 0 && tid < R) {
            FinishSmem& other = *of_block(&sm, tid);
            other.next = sm.next, other.T = sm.T, other.exact = sm.exact, other.bound = sm.bound;
          }
        }
        cluster_sync();
      }
      __syncthreads();
      if (sm.next != kAgain) break;
    }
    if (sm.next == kStretches) whole = false, k0 = 0, turn = 0;
    if (k0 >= a.beams) break;
    __syncthreads();
    if (tid == 0) sm.list_n = 0;
    __syncthreads();
  }
  if (R > 1 && rank != 0) return;

  // the new ones and the best so far, in order
  const int count = sm.count, m = count + sm.front_n;
  if (sm.front_n > 0) {
    for (int t = tid; t < sm.front_n; t += kFinishThreads) sm.buf[count + t] = sm.front[t];
    __syncthreads();
  }
  auto put = [&](int at, const Cand& y) {
    const int64_t to = int64_t(b) * a.n + at;
    const bool is = y.key > kNoScore;  // a score of -inf, a sum that overflowed, is none
    const int parent = int(y.flat >> 31);
    a.out_scores[to] = is ? key_score(y.key) : -INFINITY;
    a.out_tokens[to] = !is ? -1 : sm.ended[parent] ? a.pad : int64_t(y.flat & 0x7fffffffu);
    a.out_parents[to] = is ? parent : -1;
  };
  if (m <= 32) {
    // the place of a candidate is the number of better ones
    const int mine = tid >> 5;  // a warp's worth of threads each
    for (int t = mine; t < m; t += kFinishWarps) {
      const Cand y = sm.buf[t];
      const int at = __popc(__ballot_sync(kFullWarp, lane < m && better(sm.buf[lane], y)));
      if (at < a.n && lane == 0) put(at, y);
    }
  } else if (m <= kFinishThreads) {
    const Cand y = sorted_in_threads(sm.buf, m);
    if (tid < min(m, a.n)) put(tid, y);
  } else {
    sort_best_first(sm.buf, m);
    for (int t = tid; t < min(m, a.n); t += kFinishThreads) put(t, sm.buf[t]);
  }
  for (int t = m + tid; t < a.n; t += kFinishThreads) put(t, Cand{0, 0});
}

template <typename K>
int resident_blocks(K kernel) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kStreamThreads, 0) != cudaSuccess) {
    (void)cudaGetLastError();
    n = 0;
  }
  return std::max(1, n) * kSms;
}

// Clusters of R blocks that run at once (a cluster lies within one group of SMs).
template <int DT, int R, int B>
int resident_clusters() {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = R;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(R);
  cfg.blockDim = dim3(kFinishThreads);
  cfg.dynamicSmemBytes = sizeof(FinishSmem);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, beam_finish_kernel<DT, R, B>, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    n = 0;
  }
  return n;
}

template <int DT, int R, int B>
cudaError_t finish_with(cudaLaunchConfig_t cfg, BeamArgs a, int64_t batch) {
  static_assert(sizeof(FinishSmem) <= 48 * 1024, "within the default limit");
  const int64_t staged = int64_t(a.beams) * a.chunks * 4;
  a.staged = staged <= kMostStaged;
  cfg.dynamicSmemBytes = sizeof(FinishSmem) + (a.staged ? size_t(staged) : 0);
  if (cfg.dynamicSmemBytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(beam_finish_kernel<DT, R, B>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               int(sizeof(FinishSmem) + kMostStaged));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attrs[2];
  attrs[0] = cfg.attrs[0];
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = R;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = R > 1 ? 2 : 1;
  cfg.gridDim = dim3(unsigned(batch * R));
  cfg.blockDim = dim3(kFinishThreads);
  return cudaLaunchKernelEx(&cfg, beam_finish_kernel<DT, R, B>, a);
}

template <int DT>
cudaError_t finish(const cudaLaunchConfig_t& cfg, const BeamArgs& a, int64_t batch) {
  // Many to find: a cluster of blocks goes through the chunks side by side, as long as all
  // clusters run at once.  4 x 64 rows of 32000 bf16, n = 128: 24 us with it, 39 without;
  // 4 x 16 rows of 4175, n = 32: 11.8 and 13.5; but 17 x 16 rows of 19473, n = 32, where 16
  // clusters run: 24 and 20.  With n up to 16 one block's 16 warps do; n stands for the
  // chunks that are read again, of which the first look at all of an entry's chunks is
  // apart: 15 x 16 rows of 155059 bf16 take 25.7 us in 15 blocks with n = 16, and 28.3 in
  // clusters with n = 32.  (72 registers a thread leave one block to an SM, whether or not
  // the chunks' maxima take up to 128 KB of its shared memory, so what is asked without
  // them holds with them.)
  static const int clusters = resident_clusters<DT, 8, 1>();
  if (a.n > 16 && batch <= clusters) return finish_with<DT, 8, 1>(cfg, a, batch);
  // One block an SM may take 80 registers a thread (8 x 4 rows of 128256 bf16: 9.2 us, with
  // 64 of them 10.3); with more blocks than SMs two have to fit (161 x 8 rows of 17976:
  // 26.6 us, else 32.5).
  if (batch > kSms) return finish_with<DT, 1, 2>(cfg, a, batch);
  return finish_with<DT, 1, 1>(cfg, a, batch);
}

template <int DT, int N>
cudaError_t stream_with(cudaLaunchConfig_t cfg, BeamArgs a) {
  static const int resident = resident_blocks(beam_stream_kernel<DT, N, false>);
  static const int resident_early = resident_blocks(beam_stream_kernel<DT, N, true>);
  const int64_t blocks = (int64_t(a.rows) * a.chunks + 7) / 8;
  cfg.blockDim = dim3(kStreamThreads);
  if (blocks <= resident_early) {
    cfg.gridDim = dim3(unsigned(blocks));
    return cudaLaunchKernelEx(&cfg, beam_stream_kernel<DT, N, true>, a);
  }
  const int64_t grid = std::min<int64_t>(blocks, resident);
  a.step_rows = int(grid * (kStreamThreads / 32) / a.chunks);
  a.step_chunks = int(grid * (kStreamThreads / 32) % a.chunks);
  cfg.gridDim = dim3(unsigned(grid));
  return cudaLaunchKernelEx(&cfg, beam_stream_kernel<DT, N, false>, a);
}

template <int DT>
cudaError_t launch(const BeamArgs& a, int64_t batch, cudaStream_t stream) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const cudaError_t e = a.chunk_tokens == kChunk<DT, kVecs> ? stream_with<DT, kVecs>(cfg, a)
                                                            : stream_with<DT, 1>(cfg, a);
  if (e != cudaSuccess) return e;
  return finish<DT>(cfg, a, batch);
}

// Tokens of the chunks of a call.  The bound is an n-th largest chunk maximum, so with few
// chunks to the n it admits too much: small ones then.
int64_t chunk_tokens(lp_dtype dt, int64_t beams, int64_t V, int64_t n) {
  const int64_t large = dt == LP_F32 ? kChunk<LP_F32, kVecs> : kChunk<LP_F16, kVecs>;
  return beams * ((V + large - 1) / large) < 8 * n ? large / kVecs : large;
}

// Rows of a call's workspace hold this many chunks at most, whatever its n.
int64_t most_chunks(lp_dtype dt, int64_t V) {
  const int64_t small = (dt == LP_F32 ? kChunk<LP_F32, kVecs> : kChunk<LP_F16, kVecs>) / kVecs;
  return std::max<int64_t>(1, V / small + (V % small != 0));
}

bool known(lp_dtype dt) { return dt == LP_F32 || dt == LP_F16 || dt == LP_BF16; }

}  // namespace
}  // namespace lp

extern "C" int64_t lp_beam_select_workspace_bytes(lp_dtype dt, int64_t rows, int64_t vocab_size) {
  if (!lp::known(dt) || rows < 0 || vocab_size < 0) return -1;
  const int64_t chunks = lp::most_chunks(dt, vocab_size);
  return rows > INT64_MAX / 8 / chunks ? -1 : rows * chunks * 8;
}

extern "C" lp_status lp_beam_select(const void* logits, lp_dtype dt, int64_t batch, int64_t beams,
                                    int64_t cols, int64_t logits_stride, const int32_t* bitmask,
                                    int64_t bitmask_rows, int64_t bitmask_words,
                                    int64_t bitmask_stride, int64_t vocab_size,
                                    const uint8_t* row_needs_mask, const float* scores,
                                    const uint8_t* finished, int64_t pad_id, int64_t n_select,
                                    float* out_scores, int64_t* out_tokens, int32_t* out_parents,
                                    void* workspace, int64_t workspace_bytes,
                                    cudaStream_t stream) {
  using namespace lp;
  if (!known(dt)) return LP_ERR_UNSUPPORTED_DTYPE;
  if (batch < 0 || beams < 1 || cols < 0 || logits_stride < cols || n_select < 0)
    return LP_ERR_INVALID_ARGUMENT;
  if (beams > kMaxSelect || n_select > kMaxSelect) return LP_ERR_TOO_LARGE;
  const int64_t eb = dt == LP_F32 ? 4 : 2;
  int64_t V = vocab_size;
  if (bitmask != nullptr) {
    if (bitmask_words < 0 || bitmask_words > INT64_MAX / 32 || bitmask_stride < bitmask_words)
      return LP_ERR_INVALID_ARGUMENT;
    if (V < 0) V = std::min(cols, bitmask_words * 32);
    if (V > bitmask_words * 32) return LP_ERR_INVALID_ARGUMENT;
  } else {
    if (row_needs_mask != nullptr) return LP_ERR_INVALID_ARGUMENT;
    if (V < 0) V = cols;
  }
  if (V > cols) return LP_ERR_INVALID_ARGUMENT;
  if (V > INT32_MAX - 64 || batch > (int64_t(1) << 27) / beams) return LP_ERR_TOO_LARGE;
  const int64_t rows = batch * beams;
  if (bitmask != nullptr && bitmask_rows < rows) return LP_ERR_INVALID_ARGUMENT;
  if (batch == 0 || n_select == 0) return LP_OK;
  if (scores == nullptr || out_scores == nullptr || out_tokens == nullptr ||
      out_parents == nullptr || (V > 0 && logits == nullptr) ||
      (V > 0 && reinterpret_cast<uintptr_t>(logits) % eb != 0) ||
      logits_stride > INT64_MAX / eb / rows)
    return LP_ERR_INVALID_ARGUMENT;
  const int64_t need = lp_beam_select_workspace_bytes(dt, rows, V);
  const int64_t tokens = chunk_tokens(dt, beams, V, n_select);
  const int64_t chunks = std::max<int64_t>(1, (V + tokens - 1) / tokens);
  if (rows > INT32_MAX / chunks) return LP_ERR_TOO_LARGE;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need ||
                   reinterpret_cast<uintptr_t>(workspace) % 8 != 0))
    return LP_ERR_INVALID_ARGUMENT;
  BeamArgs a = {};
  a.logits = static_cast<const char*>(logits);
  a.stride = logits_stride * eb;
  a.V = V;
  a.bitmask = reinterpret_cast<const uint32_t*>(bitmask);
  a.bm_stride = bitmask_stride;
  a.needs = row_needs_mask;
  a.scores = scores;
  a.finished = finished;
  a.pad = pad_id;
  a.rows = int(rows);
  a.beams = int(beams);
  a.n = int(n_select);
  a.chunks = int(chunks);
  a.chunk_tokens = int(tokens);
  a.sum_bits = 40;
  while (a.sum_bits > 32 && (V >> (63 - a.sum_bits)) > 0) --a.sum_bits;
  a.part = static_cast<float2*>(workspace);
  a.out_scores = out_scores;
  a.out_tokens = out_tokens;
  a.out_parents = out_parents;
  const cudaError_t e = dt == LP_F32   ? launch<LP_F32>(a, batch, stream)
                        : dt == LP_F16 ? launch<LP_F16>(a, batch, stream)
                                       : launch<LP_BF16>(a, batch, stream);
  return status_of(e);
}
