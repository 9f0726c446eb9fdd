// verify.cu -- drafted tokens against the target's probabilities.
//
//   p_i(v) = exp((x_iv - M_i) / T) / S_i over the row's candidates,   q_i the draft's
//   draft i is accepted if u_i q_i < p_i at it; after n accepted ones
//   argmax_v log r_v + g_v says one token more, r = max(p_n - q_n, 0) after a refusal and
//   r = p_n else: with Gumbel noise g that is a draw from r / sum r.
//
// The first kernel reads every row once for (M, S) and its largest token; the second decides
// a slot's acceptances from them and goes through the one row that says a token.
#include <algorithm>

#include "common.cuh"

namespace lp {
namespace {

constexpr int kThreads = 512;
constexpr int kMostRows = 256;  // of a slot

struct RowStats {
  float top, sum;  // over the candidates; -inf and 0 where there is none
  int first;       // the lowest-index largest
  int pad;
};

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
  RowStats* stats;
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

// Whether (x, v) goes before (y, w): larger, or as large and lower.
__device__ __forceinline__ bool before(float x, int v, float y, int w) {
  return x > y || (x == y && v < w);
}

__device__ __forceinline__ void best_of(float& x, int& v, float y, int w) {
  if (before(y, w, x, v)) x = y, v = w;
}

// The block's best, in every thread; two barriers.
__device__ __forceinline__ void block_best(float& x, int& v, float* xs, int* vs) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float y = __shfl_xor_sync(kFullWarp, x, o);
    const int w = __shfl_xor_sync(kFullWarp, v, o);
    best_of(x, v, y, w);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) xs[threadIdx.x >> 5] = x, vs[threadIdx.x >> 5] = v;
  __syncthreads();
  x = xs[0], v = vs[0];
  for (int i = 1; i < kThreads / 32; ++i) best_of(x, v, xs[i], vs[i]);
}

// A block a row.
template <int DT>
__global__ void __launch_bounds__(kThreads) verify_stats_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ float xs[kThreads / 32];
  __shared__ int vs[kThreads / 32];
  const int64_t row = blockIdx.x;
  const char* x = a.logits + row * a.stride;
  const uint32_t* mask = mask_of(a, row);
  const float heat = heat_of(a, int(row / a.per_slot));
  float top = -INFINITY;
  int first = INT32_MAX;
  for (int v = threadIdx.x; v < a.V; v += kThreads)
    if (kept(mask, v)) {
      const float y = Elt<DT>::load1(x + int64_t(v) * Elt<DT>::kBytes);
      if (y > top) top = y, first = v;
    }
  block_best(top, first, xs, vs);
  float sum = 0.0f;
  if (top > -INFINITY && heat > 0.0f)
    for (int v = threadIdx.x; v < a.V; v += kThreads)
      if (kept(mask, v)) {
        const float y = Elt<DT>::load1(x + int64_t(v) * Elt<DT>::kBytes);
        if (y > -INFINITY) sum += expf(__fdiv_rn(relative(y, top), heat));
      }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullWarp, sum, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) xs[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 32; ++i) sum += xs[i];
    RowStats s;
    s.top = top, s.sum = sum, s.first = first, s.pad = 0;
    a.stats[row] = s;
  }
}

// A block a slot.
template <int DT>
__global__ void __launch_bounds__(kThreads) verify_say_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ float xs[kThreads / 32];
  __shared__ int vs[kThreads / 32];
  __shared__ int count, there;
  const int slot = blockIdx.x, R = a.per_slot, tid = threadIdx.x;
  const float heat = heat_of(a, slot);
  const bool greedy = !(heat > 0.0f);
  const int64_t* drafts = a.drafts + int64_t(slot) * (R - 1);
  if (tid == 0) count = there = R - 1;
  __syncthreads();
  for (int i = tid; i < R - 1; i += kThreads) {
    const int64_t v = drafts[i];
    bool taken = false;
    if (v < 0 || v >= a.V) {
      atomicMin(&there, i);
    } else {
      const int64_t row = int64_t(slot) * R + i;
      const RowStats s = a.stats[row];
      double p = 0.0;
      if (greedy) {
        p = v == s.first ? 1.0 : 0.0;
      } else if (kept(mask_of(a, row), int(v))) {
        const float x = Elt<DT>::load1(a.logits + row * a.stride + v * Elt<DT>::kBytes);
        if (x > -INFINITY) p = exp(double(relative(x, s.top)) / double(heat)) / double(s.sum);
      }
      const double q = a.probs != nullptr
                           ? double(a.probs[slot * a.probs_slot + i * a.probs_row + v]) : 1.0;
      taken = double(a.uniforms[int64_t(slot) * (R - 1) + i]) * q < p;
    }
    if (!taken) atomicMin(&count, i);
  }
  __syncthreads();
  const int n = count;
  const int64_t row = int64_t(slot) * R + n;
  const RowStats s = a.stats[row];
  const bool refused = n < there;
  int token = s.first;
  if (!greedy && s.top > -INFINITY) {
    const uint32_t* mask = mask_of(a, row);
    const char* x = a.logits + row * a.stride;
    const float* q = refused && a.probs != nullptr
                         ? a.probs + slot * a.probs_slot + n * a.probs_row : nullptr;
    const int64_t draft = refused ? drafts[n] : -1;
    const uint64_t seed = a.seeds != nullptr ? a.seeds[row] : a.seed;
    const uint2 key = make_uint2(uint32_t(seed), uint32_t(seed >> 32));
    for (int rest = refused; rest >= 0; --rest) {  // the second time where nothing was left
      float best = -INFINITY;
      token = INT32_MAX;
      for (int v4 = tid * 4; v4 < a.V; v4 += kThreads * 4) {
        const uint4 w = philox4x32_10(make_uint4(uint32_t(v4) >> 2, uint32_t(row),
                                                 uint32_t(a.offset), uint32_t(a.offset >> 32)), key);
        for (int e = 0; e < 4 && v4 + e < a.V; ++e) {
          const int v = v4 + e;
          if (!kept(mask, v)) continue;
          const float y = Elt<DT>::load1(x + int64_t(v) * Elt<DT>::kBytes);
          if (!(y > -INFINITY)) continue;
          float score;
          if (rest) {
            const float p = expf(__fdiv_rn(relative(y, s.top), heat)) / s.sum;
            const float r = p - (q != nullptr ? q[v] : v == draft ? 1.0f : 0.0f);
            if (!(r > 0.0f)) continue;
            score = logf(r);
          } else {
            score = __fdiv_rn(y, heat);
          }
          best_of(best, token, score + gumbel_from_word(word_of(w, e)), v);
        }
      }
      block_best(best, token, xs, vs);
      if (token != INT32_MAX) break;
    }
  }
  if (token == INT32_MAX) token = -1;
  for (int i = tid; i < R; i += kThreads)
    a.out_tokens[int64_t(slot) * R + i] = i < n ? drafts[i] : i == n ? token : -1;
  if (tid == 0) a.out_accepted[slot] = n;
}

template <int DT>
cudaError_t launch(const VerifyArgs& a, cudaStream_t stream) {
  cudaError_t e = launch_kernel(verify_stats_kernel<DT>, dim3(unsigned(a.rows)), dim3(kThreads), 0,
                                stream, a);
  if (e != cudaSuccess) return e;
  return launch_kernel(verify_say_kernel<DT>, dim3(unsigned(a.rows / a.per_slot)), dim3(kThreads),
                       0, stream, a);
}

}  // namespace
}  // namespace lp

extern "C" int64_t lp_verify_drafts_workspace_bytes(lp_dtype dt, int64_t rows,
                                                    int64_t vocab_size) {
  if ((dt != LP_F32 && dt != LP_F16 && dt != LP_BF16) || rows < 0 || vocab_size < 0 ||
      rows > (int64_t(1) << 27) || vocab_size > INT32_MAX - 64)
    return -1;
  return rows * int64_t(sizeof(lp::RowStats));
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
  a.stats = static_cast<RowStats*>(workspace);
  const cudaError_t e = dt == LP_F32   ? launch<LP_F32>(a, stream)
                        : dt == LP_F16 ? launch<LP_F16>(a, stream)
                                       : launch<LP_BF16>(a, stream);
  return status_of(e);
}
