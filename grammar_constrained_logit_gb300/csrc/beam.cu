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
// Two kernels.  The first reads the logits once, a chunk of 2 KB a warp, and leaves
// (max, sum of exp(x - max)) of each chunk: 8 bytes for 2048, so nothing of the size
// of the logits is written.  A chunk is a range of token indices, whatever the row's
// alignment, and its sum has a fixed order: two equal rows get equal scores to the
// last bit, and ties between them fall by index as stated.  The second kernel, one
// block a batch, joins the chunks to M_r and S_r, takes the n-th largest chunk
// maximum's score as a lower bound T of the n-th best candidate, and reads again
// only the chunks whose maximum reaches T: about n of them, whatever the vocabulary.
#include <algorithm>

#include "common.cuh"

namespace lp {
namespace {

constexpr int kStreamThreads = 256;
constexpr int kVecs = 4;              // 16-byte groups a lane holds of a chunk
constexpr int kFinishThreads = 512;
constexpr int kFinishWarps = kFinishThreads / 32;
constexpr int kMaxSelect = 256;       // largest n_select and beams
constexpr int kBuf = 2048;            // candidates held at once (a power of two)
constexpr int kBufNew = kBuf - kMaxSelect;
constexpr int kSms = 152;

template <int DT>
constexpr int kChunk = kVecs * 32 * Elt<DT>::kPerVec;  // tokens: 512 f32, 1024 16-bit

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
  float2* part;  // [rows, chunks]: (max, sum of exp(x - max)); rows that are dead or finished: not written
  float* out_scores;
  int64_t* out_tokens;
  int32_t* out_parents;
};

struct Cand {
  uint64_t key;   // order-preserving bits of the score in 64 bits
  uint64_t flat;  // beam * 2^31 + token
};

__device__ __forceinline__ bool better(const Cand& a, const Cand& b) {
  return a.key > b.key || (a.key == b.key && a.flat < b.flat);
}

__device__ __forceinline__ uint64_t dkey(double x) {
  const uint64_t u = uint64_t(__double_as_longlong(x + 0.0));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

__device__ __forceinline__ double key_double(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
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

// A chunk's groups of this lane, masked tokens as -inf.
template <int DT>
__device__ __forceinline__ void load_chunk(uint4 (&v)[kVecs], const char* row, const uint32_t* bm,
                                           int64_t j0, int64_t V, int lane) {
  constexpr int E = Elt<DT>::kPerVec;
  const int sh = int(reinterpret_cast<uintptr_t>(row) & 15);
  uint32_t keep[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) keep[i] = group_keep<DT>(bm, j0 + (i * 32 + lane) * E, V);
  const uint32_t none = neg_inf_word<DT>();
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    v[i] = make_uint4(none, none, none, none);
    if (keep[i]) v[i] = load_group<DT>(row, j0 + (i * 32 + lane) * E, V, sh);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) v[i] = Elt<DT>::blend(v[i], keep[i], none);
}

__device__ __forceinline__ bool row_live(const BeamArgs& a, int row) {
  return __ldg(a.scores + row) > -INFINITY &&
         (a.finished == nullptr || __ldg(a.finished + row) == 0);
}

__device__ __forceinline__ const uint32_t* row_mask(const BeamArgs& a, int row) {
  if (a.bitmask == nullptr || (a.needs != nullptr && __ldg(a.needs + row) == 0)) return nullptr;
  return a.bitmask + int64_t(row) * a.bm_stride;
}

template <int DT>
__global__ void __launch_bounds__(kStreamThreads) beam_stream_kernel(BeamArgs a) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int lane = threadIdx.x & 31;
  const unsigned total = unsigned(a.rows) * unsigned(a.chunks);
  const unsigned step = gridDim.x * (kStreamThreads / 32);
  for (unsigned w = blockIdx.x * (kStreamThreads / 32) + (threadIdx.x >> 5); w < total;
       w += step) {
    const int row = int(w / unsigned(a.chunks)), c = int(w % unsigned(a.chunks));
    if (!row_live(a, row)) continue;
    uint4 v[kVecs];
    load_chunk<DT>(v, a.logits + row * a.stride, row_mask(a, row), int64_t(c) * kChunk<DT>, a.V,
                   lane);
    float m = VecMax<DT>::run(v[0], 0xffu);
#pragma unroll
    for (int i = 1; i < kVecs; ++i) m = fmaxf(m, VecMax<DT>::run(v[i], 0xffu));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullWarp, m, o));
    m = fmaxf(m, -INFINITY);  // nothing but NaN: no candidate
    float s[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      s[i] = 0.0f;
#pragma unroll
      for (int e = 0; e < Elt<DT>::kPerVec; ++e) {
        // the difference first: exact near the maximum, where the sum comes from; the
        // maximum with -200 turns masked tokens and NaN into 2^-200, which is 0
        const float x = Elt<DT>::get(v[i], e);
        const float t = fmaxf((x - m) * 1.44269504f, -200.0f);
        s[i] += m < INFINITY ? ex2(t) : float(x == m);  // +inf tokens share all of the mass
      }
    }
    float sum = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullWarp, sum, o);
    if (lane == 0) a.part[w] = make_float2(m, m > -INFINITY ? sum : 0.0f);
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

struct FinishSmem {
  Cand buf[kBuf];             // what is new; the best so far joins behind it to be sorted
  Cand front[kMaxSelect];     // the best so far, sorted
  double base_s[kMaxSelect];  // score, log S, max of each beam
  double log_s[kMaxSelect];
  float top[kMaxSelect];      // -inf: a beam without candidates
  float least[kMaxSelect];    // tokens below this logit are out
  uint8_t ended[kMaxSelect];  // finished: one candidate, its own score
  unsigned list[kFinishThreads];
  int list_n, count, front_n;
  Cand bound;                 // candidates worse than this are out
};

// Smallest float logit of a beam that can still reach the bound.  The slack covers the
// rounding of the scores' own 64-bit arithmetic.
__device__ void set_least(FinishSmem& sm, int beams) {
  const double T = key_double(sm.bound.key);
  for (int k = threadIdx.x; k < beams; k += kFinishThreads) {
    const double s = sm.base_s[k], M = sm.top[k], z = sm.log_s[k];
    float x = -INFINITY;
    if (T > -INFINITY && s < INFINITY && M < INFINITY) {
      const double at = ((T - s) + z) + M;
      const double slack = 0x1p-48 * (fabs(T) + fabs(s) + fabs(z) + fabs(M));
      x = __double2float_rd(at - slack);
    }
    sm.least[k] = x;
  }
}

// Joins the first m new candidates with the best so far and makes the n-th best the
// bound.  keep: the n best become the best so far; else only the bound is taken.
__device__ void join(FinishSmem& sm, int m, int n, int beams, bool keep) {
  __syncthreads();
  const int front_n = sm.front_n;
  for (int t = threadIdx.x; t < front_n; t += kFinishThreads) sm.buf[m + t] = sm.front[t];
  __syncthreads();
  sort_best_first(sm.buf, m + front_n);
  const int have = min(m + front_n, n);
  if (keep)
    for (int t = threadIdx.x; t < have; t += kFinishThreads) sm.front[t] = sm.buf[t];
  if (threadIdx.x == 0) {
    if (have == n) sm.bound = sm.buf[n - 1];
    if (keep) sm.front_n = have;
    sm.count = 0;
  }
  __syncthreads();
  set_least(sm, beams);
  __syncthreads();
}

template <int DT>
__global__ void __launch_bounds__(kFinishThreads) beam_finish_kernel(BeamArgs a) {
  extern __shared__ __align__(16) char raw[];
  FinishSmem& sm = *reinterpret_cast<FinishSmem*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x, row0 = b * a.beams, C = a.chunks;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  // M and log S of each beam
  for (int k = warp; k < a.beams; k += kFinishWarps) {
    const int row = row0 + k;
    const float s = __ldg(a.scores + row);
    const bool alive = s > -INFINITY;
    const bool ended = alive && a.finished != nullptr && __ldg(a.finished + row) != 0;
    float M = -INFINITY;
    double z = 0.0;
    if (alive && !ended) {
      const float2* p = a.part + int64_t(row) * C;
      for (int c = lane; c < C; c += 32) M = fmaxf(M, p[c].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullWarp, M, o));
      double S = 0.0;
      for (int c = lane; c < C; c += 32) {
        const float2 q = p[c];
        if (q.x > -INFINITY) S += double(q.x == M ? q.y : q.y * expf(q.x - M));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) S += __shfl_xor_sync(kFullWarp, S, o);
      z = M > -INFINITY ? log(S) : 0.0;
    }
    if (lane == 0) {
      sm.base_s[k] = double(s);
      sm.log_s[k] = z;
      sm.top[k] = ended ? 0.0f : M;
      sm.ended[k] = ended;
    }
  }
  if (tid == 0) sm.count = 0, sm.front_n = 0, sm.list_n = 0;
  __syncthreads();

  // A lower bound of the n-th best score: the n-th largest of the threads' best chunks.
  // Each is a candidate of its own, taken low by the rounding of its 32-bit arithmetic.
  const unsigned total = unsigned(a.beams) * unsigned(C);
  unsigned best = 0;
  for (unsigned i = tid; i < total; i += kFinishThreads) {
    const int k = int(i / unsigned(C)), c = int(i % unsigned(C));
    const float M = sm.top[k];
    if (M == -INFINITY) continue;
    const float s = float(sm.base_s[k]), z = float(sm.log_s[k]);
    float low;
    if (sm.ended[k]) {
      if (c) continue;
      low = s;
    } else {
      const float m = a.part[int64_t(row0 + k) * C + c].x;
      if (m == -INFINITY) continue;
      const float d = m == M ? 0.0f : m - M;
      low = (s + (d - z)) - 0x1p-20f * (fabsf(s) + fabsf(d) + fabsf(z));
      if (!(low > -INFINITY)) low = s == INFINITY ? s : -INFINITY;
    }
    best = max(best, fkey(low));
  }
  unsigned T = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const int there = __syncthreads_count(best >= (T | (1u << bit)));
    if (there >= a.n) T |= 1u << bit;
    if (there == a.n) break;
  }
  if (tid == 0) sm.bound = Cand{T ? dkey(double(key_float(T))) : 0, ~0ull};
  __syncthreads();
  if (T == 0 && tid == 0) sm.bound.key = dkey(-INFINITY);
  __syncthreads();
  set_least(sm, a.beams);
  __syncthreads();

  for (unsigned i0 = 0; i0 < total; i0 += kFinishThreads) {
    // the chunks of this stretch whose maximum reaches the bound
    const unsigned i = i0 + tid;
    bool in = false;
    if (i < total) {
      const int k = int(i / unsigned(C)), c = int(i % unsigned(C));
      if (sm.top[k] > -INFINITY) {
        if (sm.ended[k]) {
          in = c == 0 && dkey(sm.base_s[k]) >= sm.bound.key;
        } else {
          const float m = a.part[int64_t(row0 + k) * C + c].x;
          in = m > -INFINITY && m >= sm.least[k];
        }
      }
    }
    if (__syncthreads_or(in) == 0) continue;
    if (in) sm.list[atomicAdd(&sm.list_n, 1)] = i;
    __syncthreads();
    const int n_list = sm.list_n;
    for (int l0 = 0; l0 < n_list;) {
      const Cand bound = sm.bound;
      const int before = sm.count;
      __syncthreads();
      if (l0 + warp < n_list) {
        const unsigned id = sm.list[l0 + warp];
        const int k = int(id / unsigned(C)), c = int(id % unsigned(C));
        const double s = sm.base_s[k];
        const uint64_t flat0 = uint64_t(k) << 31;
        if (sm.ended[k]) {
          const Cand y{dkey(s), flat0};
          if (lane == 0 && !better(bound, y)) {
            const int at = atomicAdd(&sm.count, 1);
            if (at < kBufNew) sm.buf[at] = y;
          }
        } else {
          const float M = sm.top[k], least = sm.least[k];
          const double z = sm.log_s[k];
          uint4 v[kVecs];
          load_chunk<DT>(v, a.logits + int64_t(row0 + k) * a.stride, row_mask(a, row0 + k),
                         int64_t(c) * kChunk<DT>, a.V, lane);
#pragma unroll
          for (int g = 0; g < kVecs; ++g) {
#pragma unroll
            for (int e = 0; e < Elt<DT>::kPerVec; ++e) {
              const float x = Elt<DT>::get(v[g], e);
              if (x > -INFINITY && x >= least) {
                const double score = s + ((x == M ? 0.0 : double(x) - double(M)) - z);
                const int64_t j =
                    int64_t(c) * kChunk<DT> + (g * 32 + lane) * Elt<DT>::kPerVec + e;
                const Cand y{dkey(score), flat0 + uint64_t(j)};
                if (score > -INFINITY && !better(bound, y)) {
                  const int at = atomicAdd(&sm.count, 1);
                  if (at < kBufNew) sm.buf[at] = y;
                }
              }
            }
          }
        }
      }
      __syncthreads();
      const int count = sm.count;
      if (count <= kBufNew) {
        l0 += kFinishWarps;
        if (count > kBufNew / 2) join(sm, count, a.n, a.beams, true);
      } else if (before > 0) {
        // too many: settle what earlier turns left, and read this turn's chunks again
        join(sm, before, a.n, a.beams, true);
      } else {
        // too many from this turn alone: what was seen raises the bound (strictly, as
        // kBufNew > n and no two candidates are equal), and the turn is done again
        join(sm, kBufNew, a.n, a.beams, false);
      }
      __syncthreads();
    }
    if (tid == 0) sm.list_n = 0;
    __syncthreads();
  }
  join(sm, sm.count, a.n, a.beams, true);

  for (int t = tid; t < a.n; t += kFinishThreads) {
    float score = -INFINITY;
    int64_t token = -1;
    int parent = -1;
    if (t < sm.front_n) {
      const Cand y = sm.front[t];
      parent = int(y.flat >> 31);
      token = sm.ended[parent] ? a.pad : int64_t(y.flat & 0x7fffffffu);
      score = float(key_double(y.key));
    }
    a.out_scores[int64_t(b) * a.n + t] = score;
    a.out_tokens[int64_t(b) * a.n + t] = token;
    a.out_parents[int64_t(b) * a.n + t] = parent;
  }
}

template <int DT>
cudaError_t launch(const BeamArgs& a0, int64_t batch, cudaStream_t stream) {
  BeamArgs a = a0;
  static_assert(sizeof(FinishSmem) <= 48 * 1024, "within the default limit");
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const int64_t warps = int64_t(a.rows) * a.chunks;
  cfg.gridDim = dim3(unsigned(std::min<int64_t>((warps + 7) / 8, kSms * 8)));
  cfg.blockDim = dim3(kStreamThreads);
  cudaError_t e = cudaLaunchKernelEx(&cfg, beam_stream_kernel<DT>, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(unsigned(batch));
  cfg.blockDim = dim3(kFinishThreads);
  cfg.dynamicSmemBytes = sizeof(FinishSmem);
  return cudaLaunchKernelEx(&cfg, beam_finish_kernel<DT>, a);
}

int64_t chunk_tokens(lp_dtype dt) { return dt == LP_F32 ? kChunk<LP_F32> : kChunk<LP_F16>; }

bool known(lp_dtype dt) { return dt == LP_F32 || dt == LP_F16 || dt == LP_BF16; }

}  // namespace
}  // namespace lp

extern "C" int64_t lp_beam_select_workspace_bytes(lp_dtype dt, int64_t rows, int64_t vocab_size) {
  if (!lp::known(dt) || rows < 0 || vocab_size < 0) return -1;
  const int64_t T = lp::chunk_tokens(dt);
  const int64_t chunks = std::max<int64_t>(1, vocab_size / T + (vocab_size % T != 0));
  if (rows > INT64_MAX / 8 / chunks) return -1;
  return rows * chunks * 8;
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
  const int64_t chunks = std::max<int64_t>(1, (V + chunk_tokens(dt) - 1) / chunk_tokens(dt));
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
  a.part = static_cast<float2*>(workspace);
  a.out_scores = out_scores;
  a.out_tokens = out_tokens;
  a.out_parents = out_parents;
  const cudaError_t e = dt == LP_F32   ? launch<LP_F32>(a, batch, stream)
                        : dt == LP_F16 ? launch<LP_F16>(a, batch, stream)
                                       : launch<LP_BF16>(a, batch, stream);
  return e == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}
