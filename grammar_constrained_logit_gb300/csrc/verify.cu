// verify.cu -- drafted tokens against the target's probabilities.
//
//   p_i(v) = exp((x_iv - M_i) / T) / S_i over the row's candidates,   q_i the draft's
//   draft i is accepted if u_i q_i < p_i at it; after n accepted ones
//   argmax_v log r_v + g_v says one token more, r = max(p_n - q_n, 0) after a refusal and
//   r = p_n else: with Gumbel noise g that is a draw from r / sum r.
//
// The first kernel reads every row once and leaves (largest, sum of exp((x - largest) / T)) of
// each of its runs; the second, a cluster of blocks a slot, joins those to (M, S), decides the
// slot's acceptances, and goes through the one row that says a token.
//
// log r + g is largest where r / t is, t = -log u > 0.  With m = 1 - u that ratio lies between
// r / (m / (1 - m)) and r / (m + m^2 / 2): a token whose upper bound is below a lower bound
// that its block has found is done with, without a logarithm.  Of the others a thread keeps
// its best, by the upper bound, and the second's bound; the best ones are then scored as
// defined.  Should a second one still reach the winner (once in some thousand slots), or
// nothing be left of p - q, the slot's first block goes through the row once more, token by
// token as defined.
//
// Measured, in a graph: 64 x 8 rows of 128256 bf16 with a tenth kept 66 us for 144 MB, 48 x 5 of
// 65519 fp16 27.6, 1 x 4 of 32000 f32 9.8.  The first kernel (33 us cold) is bound by instructions,
// 11.7 for each of a lane's tokens, 71% of the issue slots: four blocks an SM, that leave a lane
// 64 registers for what is under way (five: 71 us for the whole, six: 81).  The second (39 us
// cold) by the noise of the tokens that the bounds leave, four words for each four of which one
// is left (three blocks an SM: 80 us for the whole).
#include <algorithm>

#include "common.cuh"

namespace lp {
namespace {

constexpr int kStreamThreads = 256;
constexpr int kVecs = 4;                    // 16-byte vectors a lane has of a chunk
constexpr int kChunkVecs = kVecs * 32;
constexpr int kThreads = 256;               // of a block of the second kernel
constexpr int kWarps = kThreads / 32;
constexpr int kMostRows = 256;              // of a slot: a thread has a draft at most
constexpr int kMostCluster = 8;
constexpr int kSms = 152;
constexpr float kLog2e = 1.4426950408889634f;

struct VerifyArgs {
  const char* logits;
  int64_t stride;  // bytes
  int V;
  const uint32_t* bitmask;
  int64_t bm_stride;
  const uint8_t* needs;
  int rows, per_slot;
  const int64_t* drafts;
  const float* probs;
  int64_t probs_slot, probs_row;
  const float* uniforms;
  const float* temperature;
  float temperature_scalar;
  uint64_t seed, offset;
  const uint64_t* seeds;
  int64_t* out_tokens;
  int32_t* out_accepted;
  float2* part;  // [rows, runs]
  int runs, run; // of a row; vectors of one
  Div per_row;   // runs
};

__device__ __forceinline__ float heat_of(const VerifyArgs& a, int slot) {
  return a.temperature != nullptr ? __ldg(a.temperature + slot) : a.temperature_scalar;
}

__device__ __forceinline__ const uint32_t* mask_of(const VerifyArgs& a, int64_t row) {
  return a.bitmask != nullptr && (a.needs == nullptr || a.needs[row] != 0)
             ? a.bitmask + row * a.bm_stride
             : nullptr;
}

__device__ __forceinline__ bool kept(const uint32_t* mask, int v) {
  return mask == nullptr || ((__ldg(mask + (v >> 5)) >> (v & 31)) & 1u) != 0;
}

// x / T of a candidate relative to the row's largest; candidates at +inf share the mass.
__device__ __forceinline__ float relative(float x, float top) { return x == top ? 0.0f : x - top; }

// What a candidate's distance to the largest is multiplied by, as a power of two.  Not 0, with an
// infinite temperature: a candidate's distance stays finite and what is none keeps -inf.
__device__ __forceinline__ float rate_of(float heat) {
  return heat > 0.0f ? fmaxf(fminf(kLog2e / heat, 3e38f), 1.4012984643248171e-45f) : 3e38f;
}

__device__ __forceinline__ void best_of(float& x, int& v, float y, int w) {
  if (y > x || (y == x && w < v)) x = y, v = w;
}

// A row's 16-byte vectors: aligned ones, of which the first and the last may hold tokens
// that are not the row's.
template <int DT>
struct RowVecs {
  static constexpr int kPer = Elt<DT>::kPerVec;
  const char* at;
  const uint32_t* mask;
  int before, V;  // tokens of the first vector before the row

  __device__ __forceinline__ RowVecs(const VerifyArgs& a, int64_t row) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.logits) + row * a.stride;
    before = int(p & 15) / Elt<DT>::kBytes;
    at = reinterpret_cast<const char*>(p & ~uintptr_t(15));
    mask = mask_of(a, row);
    V = a.V;
  }
  __device__ __forceinline__ int count() const {
    return V == 0 ? 0 : int((uint32_t(before) + uint32_t(V) + kPer - 1) / kPer);
  }
  __device__ __forceinline__ int first_token(int q) const {
    return int(uint32_t(q) * kPer - uint32_t(before));
  }
  // What the mask has of a vector's tokens: asked for early, looked at late.
  __device__ __forceinline__ uint32_t mask_word(int q) const {
    if (mask == nullptr) return ~0u;
    const int j = first_token(q);
    // aligned rows: a vector's bits lie within a word
    return before == 0 ? __ldg(mask + (j >> 5)) : mask_bits(mask, max(j, 0), kPer - max(0, -j), V);
  }
  // Bits of the vector's tokens that are candidates, as far as the mask goes.
  __device__ __forceinline__ uint32_t bits(int q, uint32_t word) const {
    const int j = first_token(q), lo = max(0, -j), n = min(kPer, V - j);
    const uint32_t keep = ((1u << n) - 1u) & ~((1u << lo) - 1u);
    return keep & (mask == nullptr ? ~0u : before == 0 ? word >> (j & 31) : word << lo);
  }
};

__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  return uint64_t(__float_as_uint(a)) | uint64_t(__float_as_uint(b)) << 32;
}
__device__ __forceinline__ float low_of(uint64_t v) { return __uint_as_float(uint32_t(v)); }
__device__ __forceinline__ float high_of(uint64_t v) { return __uint_as_float(uint32_t(v >> 32)); }
__device__ __forceinline__ uint64_t add_pairs(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul_pairs(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Bytes of x by `sel`'s digits; 8 more than a byte's number is its highest bit, eight times.
__device__ __forceinline__ uint32_t bytes_by(uint32_t x, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(x), "r"(sel));
  return r;
}

// -inf in the places whose bit is clear.  Four bits times 0x10204080 are the highest bits of
// four bytes, and a byte permutation spreads those over two 16-bit places at a time.
template <int DT>
__device__ __forceinline__ uint4 only(const uint4& v, uint32_t keep) {
  if (DT == LP_F32) return Elt<DT>::blend(v, keep, 0xff800000u);
  const uint32_t fill = DT == LP_BF16 ? 0xff80ff80u : 0xfc00fc00u;
  const uint32_t lo = (keep & 15u) * 0x10204080u, hi = (keep >> 4) * 0x10204080u;
  uint4 r;
  uint32_t m;
  m = bytes_by(lo, 0x9988), r.x = (v.x & m) | (fill & ~m);
  m = bytes_by(lo, 0xbbaa), r.y = (v.y & m) | (fill & ~m);
  m = bytes_by(hi, 0x9988), r.z = (v.z & m) | (fill & ~m);
  m = bytes_by(hi, 0xbbaa), r.w = (v.w & m) | (fill & ~m);
  return r;
}

// (largest, sum) of vectors [q0, q1) with whatever is among the logits: NaN is no candidate,
// and candidates at +inf share the mass.
template <int DT>
__device__ __noinline__ float2 any_run(const RowVecs<DT> x, int q0, int q1, float rate) {
  const int lane = threadIdx.x & 31;
  float top = -INFINITY, sum = 0.0f;
  for (int q = q0 + lane; q < q1; q += 32) {
    const uint4 raw = only<DT>(__ldg(reinterpret_cast<const uint4*>(x.at) + q),
                               x.bits(q, x.mask_word(q)));
    top = fmaxf(top, VecMax<DT>::run(raw, (1u << RowVecs<DT>::kPer) - 1u));
  }
  top = key_float(__reduce_max_sync(kFullWarp, fkey(top)));
  for (int q = q0 + lane; q < q1; q += 32) {
    const uint4 raw = only<DT>(__ldg(reinterpret_cast<const uint4*>(x.at) + q),
                               x.bits(q, x.mask_word(q)));
#pragma unroll
    for (int e = 0; e < RowVecs<DT>::kPer; ++e) {
      const float y = Elt<DT>::get(raw, e);
      if (y > -INFINITY) sum += ex2(relative(y, top) * rate);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullWarp, sum, o);
  return make_float2(top, sum);
}

// A warp a run of a row's vectors: each lane its own largest and sum, joined at the end.  A
// vector's place in registers is loaded again as soon as it is used up.
template <int DT>
__global__ void __launch_bounds__(kStreamThreads, 4)
    verify_stream_kernel(const __grid_constant__ VerifyArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr float kLowest = -3.4028234663852886e38f;
  const int lane = threadIdx.x & 31;
  const uint32_t warp = blockIdx.x * (kStreamThreads / 32) + (threadIdx.x >> 5);
  const uint32_t row = a.per_row.quot(warp);
  if (row >= uint32_t(a.rows)) return;
  const int run = int(warp - row * a.per_row.d);
  const float rate = rate_of(heat_of(a, int(row) / a.per_slot));
  const RowVecs<DT> x(a, row);
  const int q0 = run * a.run, q1 = min(q0 + a.run, x.count());
  uint4 raw[kVecs];
  uint32_t word[kVecs];
  const auto fetch = [&](int u, int q) {
    raw[u] = make_uint4(0, 0, 0, 0);
    word[u] = 0;
    if (q < q1) {
      raw[u] = __ldg(reinterpret_cast<const uint4*>(x.at) + q);
      word[u] = x.mask_word(q);
    }
  };
#pragma unroll
  for (int u = 0; u < kVecs; ++u) fetch(u, q0 + u * 32 + lane);
  float top = kLowest;
  uint64_t sums = 0;
  const uint64_t by = pair_of(rate, rate);
  for (int q = q0 + lane; q - lane < q1; q += kChunkVecs) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int at = q + u * 32;
      // what is no candidate becomes -inf
      const uint4 v = only<DT>(raw[u], at < q1 ? x.bits(at, word[u]) : 0u);
      fetch(u, at + kChunkVecs);
      const float now = fmaxf(top, VecMax<DT>::run(v, (1u << RowVecs<DT>::kPer) - 1u));
      const float f = ex2((top - now) * rate);
      const uint64_t less = pair_of(-now, -now);
      sums = mul_pairs(sums, pair_of(f, f));
      top = now;
#pragma unroll
      for (int e = 0; e < RowVecs<DT>::kPer; e += 2) {
        const uint64_t t = mul_pairs(add_pairs(pair_of(Elt<DT>::get(v, e),
                                                       Elt<DT>::get(v, e + 1)), less), by);
        sums = add_pairs(sums, pair_of(ex2(low_of(t)), ex2(high_of(t))));
      }
    }
  }
  float sum = low_of(sums) + high_of(sums);
  const float all = key_float(__reduce_max_sync(kFullWarp, fkey(top)));
  sum *= ex2((top - all) * rate);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullWarp, sum, o);
  // the largest itself counts 1, so without a candidate there is 0
  float2 found = make_float2(sum == 0.0f ? -INFINITY : all, sum);
  if (!(sum < INFINITY)) found = any_run<DT>(x, q0, q1, rate);
  if (lane == 0) a.part[int64_t(row) * a.runs + run] = found;
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct Found {
  float score;  // as defined; of what r is measured in, less `shift`
  int token;
  float second;  // the largest upper bound of what was not scored
  int pad;
};

__device__ __forceinline__ Found join(Found f, const Found& g) {
  best_of(f.score, f.token, g.score, g.token);
  f.second = fmaxf(f.second, g.second);
  return f;
}

template <int DT>
__device__ __forceinline__ float logit_at(const char* x, int v) {
  return Elt<DT>::load1(x + int64_t(v) * Elt<DT>::kBytes);
}

// The row that says a token.
struct Row {
  const char* x;
  const uint32_t* mask;
  const float* q;  // what the draft's probabilities are, or NULL
  int64_t draft;   // NULL: all on this token, if there is one
  float top, sum, heat, rate, shift;
  uint2 key;
  uint32_t row, offset_lo, offset_hi;
};

// log r + g as defined, or -inf.
__device__ __forceinline__ float score_of(const Row& w, bool rest, float y, float d, uint32_t word) {
  if (!(y > -INFINITY)) return -INFINITY;
  if (!rest) return __fdiv_rn(y, w.heat) + gumbel_from_word(word);
  const float r = expf(__fdiv_rn(relative(y, w.top), w.heat)) / w.sum - d;
  return r > 0.0f ? logf(r) + gumbel_from_word(word) : -INFINITY;
}

template <int N>
struct Group {  // N tokens
  float y[N], d[N];
  uint32_t keep;
};

// The word of the mask that has tokens v0 .. v0 + 7, v0 a multiple of 8.
__device__ __forceinline__ uint32_t group_word(const Row& w, uint32_t v0, uint32_t V) {
  return w.mask != nullptr && v0 < V ? __ldg(w.mask + (v0 >> 5)) : ~0u;
}

// Tokens v0 .. v0 + 7.
template <int DT>
__device__ __forceinline__ void load_group(Group<8>& g, const Row& w, uint32_t word, uint32_t v0,
                                           uint32_t V, bool whole, bool whole_q) {
  const uint32_t m = v0 < V ? min(8u, V - v0) : 0u;
  g.keep = ((1u << m) - 1u) & (word >> (v0 & 31));
#pragma unroll
  for (int e = 0; e < 8; ++e) g.y[e] = -INFINITY, g.d[e] = 0.0f;
  if (g.keep == 0) return;
  if (whole && m == 8) {
    uint4 v[2];
    const uint4* p = reinterpret_cast<const uint4*>(w.x + int64_t(v0) * Elt<DT>::kBytes);
    v[0] = __ldg(p);
    if (DT == LP_F32) v[1] = __ldg(p + 1);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      g.y[e] = Elt<DT>::get(v[e / Elt<DT>::kPerVec], e % Elt<DT>::kPerVec);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < int(m)) g.y[e] = logit_at<DT>(w.x, int(v0) + e);
  }
  if (w.q == nullptr) return;
  if (whole_q && m == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(w.q + v0) + i);
      g.d[4 * i] = v.x, g.d[4 * i + 1] = v.y, g.d[4 * i + 2] = v.z, g.d[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < int(m)) g.d[e] = __ldg(w.q + v0 + e);
  }
}

__device__ __forceinline__ uint4 noise(const Row& w, uint32_t v) {
  return philox4x32_10(make_uint4(v >> 2, w.row, w.offset_lo, w.offset_hi), w.key);
}

// The best of a block's threads, in every thread; two barriers.
__device__ __forceinline__ Found block_best(Found f, Found* warps) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Found g;
    g.score = __shfl_xor_sync(kFullWarp, f.score, o);
    g.token = __shfl_xor_sync(kFullWarp, f.token, o);
    g.second = __shfl_xor_sync(kFullWarp, f.second, o);
    f = join(f, g);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = f;
  __syncthreads();
  f = warps[0];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) f = join(f, warps[i]);
  return f;
}

// The whole row as defined, by one block.
template <int DT>
__device__ __noinline__ Found every_token(Row w, bool rest, int V, Found* warps) {
  Found f = {-INFINITY, INT32_MAX, 0.0f, 0};
  for (int64_t v = threadIdx.x; v < V; v += kThreads) {
    if (!kept(w.mask, int(v))) continue;
    const float d = !rest ? 0.0f : w.q != nullptr ? w.q[v] : v == w.draft ? 1.0f : 0.0f;
    const float score = score_of(w, rest, logit_at<DT>(w.x, int(v)), d,
                                 word_of(noise(w, uint32_t(v)), int(v & 3)));
    if (score > -INFINITY) best_of(f.score, f.token, score, int(v));
  }
  return block_best(f, warps);
}

// A cluster of blocks a slot.
template <int DT>
__global__ void __launch_bounds__(kThreads, 4) verify_say_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ float tops[kMostRows], sums[kMostRows];
  __shared__ int firsts[kMostRows];  // greedy: the lowest-index largest
  __shared__ Found warps[kWarps];
  __shared__ alignas(16) Found founds[kMostCluster];
  __shared__ int count, there;
  __shared__ uint32_t reached;  // a lower bound of the block's best r / t
  const int blocks = int(cluster_size()), rank = int(cluster_rank());
  const int slot = blockIdx.x / blocks, R = a.per_slot, tid = threadIdx.x, lane = tid & 31;
  // (a block may write to another's shared memory once that one has begun: told here, waited
  // for below)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (tid == 0) count = there = R - 1, reached = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const float heat = heat_of(a, slot);
  const bool greedy = !(heat > 0.0f);
  const float rate = rate_of(heat);
  const int64_t* drafts = a.drafts + int64_t(slot) * (R - 1);
  // a thread's draft, its logit and its probability, under way while the rows are joined
  int64_t draft = -1;
  float draft_x = -INFINITY, draft_q = 1.0f, draft_u = 0.0f;
  if (tid < R - 1) {
    draft = drafts[tid];
    if (draft >= 0 && draft < a.V) {
      const int64_t row = int64_t(slot) * R + tid;
      if (kept(mask_of(a, row), int(draft)))
        draft_x = logit_at<DT>(a.logits + row * a.stride, int(draft));
      if (a.probs != nullptr) draft_q = a.probs[slot * a.probs_slot + tid * a.probs_row + draft];
      draft_u = a.uniforms[int64_t(slot) * (R - 1) + tid];
    }
  }
  for (int i = tid >> 5; i < R; i += kWarps) {
    const int64_t row = int64_t(slot) * R + i;
    const float2* part = a.part + row * a.runs;
    float top = -INFINITY, sum = 0.0f;
#pragma unroll 4
    for (int c = lane; c < a.runs; c += 32) {
      const float2 p = part[c];
      const float now = fmaxf(top, p.x);
      if (now > -INFINITY)
        sum = sum * ex2(relative(top, now) * rate) + p.y * ex2(relative(p.x, now) * rate);
      top = now;
    }
    const float all = key_float(__reduce_max_sync(kFullWarp, fkey(top)));
    sum = top > -INFINITY ? sum * ex2(relative(top, all) * rate) : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullWarp, sum, o);
    int first = INT32_MAX;
    if (greedy && all > -INFINITY) {  // in the first run that has it
      int chunk = INT32_MAX;
      for (int c = lane; c < a.runs; c += 32)
        if (chunk == INT32_MAX && part[c].x == all) chunk = c;
      chunk = __reduce_min_sync(kFullWarp, chunk);
      const RowVecs<DT> x(a, row);
      const int q0 = chunk * a.run, q1 = min(q0 + a.run, x.count());
      for (int q = q0 + lane; q < q1; q += 32) {
        const uint4 raw = __ldg(reinterpret_cast<const uint4*>(x.at) + q);
        const uint32_t keep = x.bits(q, x.mask_word(q));
#pragma unroll
        for (int e = RowVecs<DT>::kPer - 1; e >= 0; --e)
          if (((keep >> e) & 1u) && Elt<DT>::get(raw, e) == all)
            first = min(first, x.first_token(q) + e);
      }
      first = __reduce_min_sync(kFullWarp, first);
    }
    if (lane == 0) tops[i] = all, sums[i] = sum, firsts[i] = first;
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (tid < R - 1) {
    bool taken = false;
    if (draft < 0 || draft >= a.V) {
      atomicMin(&there, tid);
    } else if (greedy) {
      taken = draft == firsts[tid] && draft_u * draft_q < 1.0f;
    } else if (draft_x > -INFINITY) {
      // exp(d / T) with the quotient's rounding taken back: an acceptance hangs on p's last
      // places
      const float d = relative(draft_x, tops[tid]), quot = __fdiv_rn(d, heat);
      const float over = d > -INFINITY && quot > -INFINITY && heat < INFINITY
                             ? fmaf(-quot, heat, d) / heat : 0.0f;
      const float e = expf(quot), p = fmaf(e, over, e);
      taken = draft_u * draft_q * sums[tid] < p;
    }
    if (!taken) atomicMin(&count, tid);
  }
  __syncthreads();
  const int n = count;
  const int64_t row = int64_t(slot) * R + n;
  const float top = tops[n];
  const bool refused = n < there;
  int token = firsts[n];
  if (!greedy && top > -INFINITY) {
    Row w;
    w.x = a.logits + row * a.stride;
    w.mask = mask_of(a, row);
    w.q = refused && a.probs != nullptr ? a.probs + slot * a.probs_slot + n * a.probs_row : nullptr;
    w.draft = refused ? drafts[n] : -1;
    w.top = top, w.sum = sums[n], w.heat = heat, w.rate = rate;
    w.shift = refused ? 0.0f : __fdiv_rn(top, heat);
    const uint64_t seed = a.seeds != nullptr ? a.seeds[row] : a.seed;
    w.key = make_uint2(uint32_t(seed), uint32_t(seed >> 32));
    w.row = uint32_t(row), w.offset_lo = uint32_t(a.offset), w.offset_hi = uint32_t(a.offset >> 32);
    const bool whole = reinterpret_cast<uintptr_t>(w.x) % 16 == 0;
    const bool whole_q = w.q != nullptr && reinterpret_cast<uintptr_t>(w.q) % 16 == 0;
    const float by = (refused ? -log2f(w.sum) : 0.0f) + 2.9e-5f;  // and 1.00002 times that
    // what rounding in the score as defined may make up for; nothing is passed over where the
    // scores are so large that it is much, or where the largest is +inf
    const float slack = fmaxf(0.0f, 0.999f - fabsf(w.shift) * 1e-6f);
    const float keen = slack > 0.5f ? slack : 0.0f;

    float best = -1.0f, second = -1.0f, best_y = -INFINITY, best_d = 0.0f;
    uint32_t best_word = 0;
    int best_v = INT32_MAX;
    const uint32_t V = uint32_t(a.V), step = uint32_t(blocks) * kThreads * 8;
    uint32_t v0 = uint32_t(rank * kThreads + tid) * 8;
    Group<8> g;
    // logits and probabilities come one round ahead, the mask that says which of them two
    uint32_t word = group_word(w, v0, V), word_after = group_word(w, v0 + step, V);
    load_group<DT>(g, w, word, v0, V, whole, whole_q);
    while (v0 < V) {
      Group<8> next;
      word = word_after;
      word_after = group_word(w, v0 + 2 * step, V);
      load_group<DT>(next, w, word, v0 + step, V, whole, whole_q);
      const float bound = __uint_as_float(*static_cast<volatile uint32_t*>(&reached)) * keen;
      float r[8];
      uint32_t live = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (w.q == nullptr && int64_t(v0) + e == w.draft) g.d[e] = 1.0f;
        // p is within 1e-5 of itself: r is this, or less
        const float d = top < INFINITY ? g.y[e] - top : relative(g.y[e], top);
        r[e] = ex2(fmaf(d, rate, by)) - g.d[e];
        // (m is 2^-24 at least)
        live |= uint32_t(r[e] > 0.0f && r[e] >= bound * 5.9e-8f) << e;
      }
      live &= g.keep;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (((live >> (4 * half)) & 15u) == 0) continue;
        const uint4 words = noise(w, v0 + 4 * half);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * half + i;
          const uint32_t word = word_of(words, i);
          const float m = fmaf(float(~word >> 9), 1.1920928955078125e-07f, 5.9604644775390625e-08f);
          const float least = fmaf(m * 0.5f, m, m);  // t is this, or more
          if (!((live >> e) & 1u) || r[e] < bound * least) continue;
          const float s = __fdividef(r[e], least) * 1.00001f;
          second = fmaxf(second, fminf(s, best));
          if (s > best) {
            best = s, best_v = int(v0) + e, best_y = g.y[e], best_d = g.d[e], best_word = word;
            // t is m / (1 - m) at most, and r no less than p 1e-4 below
            const float low = fmaf(r[e] + g.d[e], -1e-4f, r[e]) * (1.0f - m) * 0.9999f;
            if (low > 0.0f && m < 1.0f)
              atomicMax(&reached, __float_as_uint(fminf(__fdividef(low, m), 1e30f)));
          }
        }
      }
      g = next;
      v0 += step;
    }
    Found f = {-INFINITY, INT32_MAX, second, 0};
    if (best_v != INT32_MAX) {
      f.score = score_of(w, refused, best_y, best_d, best_word);
      if (f.score > -INFINITY) f.token = best_v;
    }
    f = block_best(f, warps);
    if (tid == 0) {
      uint32_t at;
      asm("mapa.shared::cluster.u32 %0, %1, 0;"
          : "=r"(at) : "r"(uint32_t(__cvta_generic_to_shared(founds + rank))));
      asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                   "r"(__float_as_uint(f.score)), "r"(f.token), "r"(__float_as_uint(f.second)), "r"(0)
                   : "memory");
    }
    cluster_sync();
    if (rank != 0) return;
    f = founds[0];
    for (int i = 1; i < blocks; ++i) f = join(f, founds[i]);
    // whether something that was not scored reaches the best
    if (f.token != INT32_MAX && !(f.second < expf(f.score - w.shift) * keen))
      f = every_token<DT>(w, refused, a.V, warps);
    if (f.token == INT32_MAX) f = every_token<DT>(w, refused, a.V, warps);
    if (f.token == INT32_MAX) f = every_token<DT>(w, false, a.V, warps);
    token = f.token;
  }
  if (rank != 0) return;
  if (token == INT32_MAX) token = -1;
  for (int i = tid; i < R; i += kThreads)
    a.out_tokens[int64_t(slot) * R + i] = i < n ? drafts[i] : i == n ? token : -1;
  if (tid == 0) a.out_accepted[slot] = n;
}

template <int DT>
cudaError_t launch(VerifyArgs a, cudaStream_t stream) {
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kStreamThreads);
  // as many runs as there are warps on all SMs, of a chunk each at least
  const int64_t resident = int64_t(kSms) * 4 * (kStreamThreads / 32);
  const int64_t vecs = std::max<int64_t>(1, a.V / Elt<DT>::kPerVec + 2);
  const int64_t most = (vecs + kChunkVecs - 1) / kChunkVecs;
  const int64_t runs = std::max<int64_t>(1, std::min(most, resident / a.rows));
  a.run = int((vecs + runs - 1) / runs + 31) / 32 * 32;
  a.runs = int((vecs + a.run - 1) / a.run);
  a.per_row.set(uint32_t(a.runs));
  const int64_t warps = int64_t(a.rows) * a.runs;
  cfg.gridDim = dim3(unsigned((warps + kStreamThreads / 32 - 1) / (kStreamThreads / 32)));
  const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_stream_kernel<DT>, a);
  if (e != cudaSuccess) return e;
  const int64_t slots = a.rows / a.per_slot;
  // blocks to a slot: as many as have a round of tokens, and as all slots have room for
  int blocks = kMostCluster;
  while (blocks > 1 && (slots * blocks > kSms * 4 || blocks * kThreads * 8 >= 2 * a.V))
    blocks /= 2;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = unsigned(blocks);
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  cfg.blockDim = dim3(kThreads);
  cfg.gridDim = dim3(unsigned(slots * blocks));
  return cudaLaunchKernelEx(&cfg, verify_say_kernel<DT>, a);
}

// Runs of a row, at most: a chunk of vectors each.
int64_t chunks_of(lp_dtype dt, int64_t V) {
  const int64_t per = dt == LP_F32 ? 4 : 8;
  return (std::max<int64_t>(1, V / per + 2) + kChunkVecs - 1) / kChunkVecs;
}

}  // namespace
}  // namespace lp

extern "C" int64_t lp_verify_drafts_workspace_bytes(lp_dtype dt, int64_t rows,
                                                    int64_t vocab_size) {
  if ((dt != LP_F32 && dt != LP_F16 && dt != LP_BF16) || rows < 0 || vocab_size < 0 ||
      rows > (int64_t(1) << 27) || vocab_size > INT32_MAX - 64)
    return -1;
  return (rows * lp::chunks_of(dt, vocab_size) * 8 + 15) / 16 * 16;
}

extern "C" lp_status lp_verify_drafts(const void* logits, lp_dtype dt, int64_t B, int64_t cols,
                                      int64_t logits_stride, const int32_t* bitmask,
                                      int64_t bitmask_rows, int64_t bitmask_words,
                                      int64_t bitmask_stride, int64_t vocab_size,
                                      const uint8_t* row_needs_mask, int64_t rows_per_slot,
                                      const int64_t* drafts, const float* draft_probs,
                                      int64_t probs_slot_stride, int64_t probs_row_stride,
                                      const float* uniforms, const float* temperature,
                                      float temperature_scalar, uint64_t seed, uint64_t offset,
                                      const uint64_t* seeds, int64_t* out_tokens,
                                      int32_t* out_accepted, void* workspace,
                                      int64_t workspace_bytes, cudaStream_t stream) {
  using namespace lp;
  if (dt != LP_F32 && dt != LP_F16 && dt != LP_BF16) return LP_ERR_UNSUPPORTED_DTYPE;
  if (B < 0 || cols < 0 || logits_stride < cols || rows_per_slot < 1)
    return LP_ERR_INVALID_ARGUMENT;
  if (rows_per_slot > kMostRows) return LP_ERR_TOO_LARGE;
  if (B % rows_per_slot != 0) return LP_ERR_INVALID_ARGUMENT;
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
  if (V > INT32_MAX - 64 || B > (int64_t(1) << 27)) return LP_ERR_TOO_LARGE;
  if (bitmask != nullptr && bitmask_rows < B) return LP_ERR_INVALID_ARGUMENT;
  if (B == 0) return LP_OK;
  const int64_t eb = dt == LP_F32 ? 4 : 2;
  const bool drafted = rows_per_slot > 1;
  if (out_tokens == nullptr || out_accepted == nullptr ||
      (drafted && (drafts == nullptr || uniforms == nullptr)) ||
      (V > 0 && logits == nullptr) || reinterpret_cast<uintptr_t>(logits) % eb != 0 ||
      logits_stride > INT64_MAX / eb / B ||
      (reinterpret_cast<uintptr_t>(draft_probs) | reinterpret_cast<uintptr_t>(uniforms) |
       reinterpret_cast<uintptr_t>(temperature) | reinterpret_cast<uintptr_t>(out_accepted) |
       reinterpret_cast<uintptr_t>(bitmask)) % 4 != 0 ||
      (reinterpret_cast<uintptr_t>(drafts) | reinterpret_cast<uintptr_t>(seeds) |
       reinterpret_cast<uintptr_t>(out_tokens)) % 8 != 0)
    return LP_ERR_INVALID_ARGUMENT;
  const int64_t need = lp_verify_drafts_workspace_bytes(dt, B, V);
  // (warps are counted in 31 bits)
  if (B > INT32_MAX / chunks_of(dt, V)) return LP_ERR_TOO_LARGE;
  if (workspace == nullptr || workspace_bytes < need ||
      reinterpret_cast<uintptr_t>(workspace) % 16 != 0)
    return LP_ERR_INVALID_ARGUMENT;
  VerifyArgs a = {};
  a.logits = static_cast<const char*>(logits);
  a.stride = logits_stride * eb;
  a.V = int(V);
  a.bitmask = reinterpret_cast<const uint32_t*>(bitmask);
  a.bm_stride = bitmask_stride;
  a.needs = row_needs_mask;
  a.rows = int(B), a.per_slot = int(rows_per_slot);
  a.drafts = drafts;
  a.probs = draft_probs;
  a.probs_slot = probs_slot_stride, a.probs_row = probs_row_stride;
  a.uniforms = uniforms;
  a.temperature = temperature;
  a.temperature_scalar = temperature_scalar;
  a.seed = seed, a.offset = offset;
  a.seeds = seeds;
  a.out_tokens = out_tokens;
  a.out_accepted = out_accepted;
  a.part = static_cast<float2*>(workspace);
  const cudaError_t e = dt == LP_F32   ? launch<LP_F32>(a, stream)
                        : dt == LP_F16 ? launch<LP_F16>(a, stream)
                                       : launch<LP_BF16>(a, stream);
  return status_of(e);
}
