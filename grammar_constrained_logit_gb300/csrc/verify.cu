// verify.cu -- drafted tokens against the target's probabilities.
//
//   p_i(v) = exp((x_iv - M_i) / T) / S_i over the row's candidates,   q_i the draft's
//   draft i is accepted if u_i q_i < p_i at it; after n accepted ones
//   argmax_v log r_v + g_v says one token more, r = max(p_n - q_n, 0) after a refusal and
//   r = p_n else: with Gumbel noise g that is a draw from r / sum r.
//
// The first kernel reads every row once and leaves (largest, sum of exp((x - largest) / T)) of
// each chunk of 2 KB; the second, a cluster of blocks a slot, joins those to (M, S), decides the
// slot's acceptances, and goes through the one row that says a token.
//
// There a token that cannot win is told by its noise word alone: log r + g > best means
// -log u < r exp(-best), and 1 - u <= -log u, so where 1 - u is not below that (with a margin
// for its roundings) neither logarithm is taken.
#include <algorithm>

#include "common.cuh"

namespace lp {
namespace {

constexpr int kStreamThreads = 256;
constexpr int kVecs = 4;                    // 16-byte vectors a lane has of a chunk
constexpr int kChunkVecs = kVecs * 32;
constexpr int kThreads = 512;               // of a block of the second kernel
constexpr int kWarps = kThreads / 32;
constexpr int kMostRows = 256;              // of a slot
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
  float2* part;  // [rows, chunks]
  int chunks;
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

// What a candidate's distance to the largest is multiplied by, as a power of two.
__device__ __forceinline__ float rate_of(float heat) {
  return fminf(kLog2e / heat, 3e38f);
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
  __device__ __forceinline__ int64_t count() const {
    return (int64_t(before) + V + kPer - 1) / kPer;
  }
  __device__ __forceinline__ int first_token(int64_t q) const { return int(q * kPer - before); }
  // Bits of the vector's tokens that are candidates, as far as the mask goes.
  __device__ __forceinline__ uint32_t bits(int64_t q) const {
    const int j = first_token(q), lo = max(0, -j), n = min(kPer, V - j);
    uint32_t keep = ((1u << n) - 1u) & ~((1u << lo) - 1u);
    if (mask != nullptr) keep &= mask_bits(mask, j + lo, kPer - lo, V) << lo;
    return keep;
  }
};

// A warp a chunk.
template <int DT>
__global__ void __launch_bounds__(kStreamThreads)
    verify_stream_kernel(const __grid_constant__ VerifyArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t total = int64_t(a.rows) * a.chunks;
  for (int64_t i = int64_t(blockIdx.x) * (kStreamThreads / 32) + (threadIdx.x >> 5); i < total;
       i += int64_t(gridDim.x) * (kStreamThreads / 32)) {
    const int64_t row = i / a.chunks;
    const int chunk = int(i - row * a.chunks);
    const RowVecs<DT> x(a, row);
    const int64_t vecs = x.count();
    uint4 raw[kVecs];
    uint32_t keep[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int64_t q = int64_t(chunk) * kChunkVecs + u * 32 + lane;
      keep[u] = 0;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (q < vecs) {
        raw[u] = __ldg(reinterpret_cast<const uint4*>(x.at) + q);
        keep[u] = x.bits(q);
      }
    }
    const float rate = rate_of(heat_of(a, int(row / a.per_slot)));
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) top = fmaxf(top, VecMax<DT>::run(raw[u], keep[u]));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullWarp, top, o));
    float sum = 0.0f;
    if (top > -INFINITY) {
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
#pragma unroll
        for (int e = 0; e < RowVecs<DT>::kPer; ++e) {
          const float y = Elt<DT>::get(raw[u], e);
          const float t = (top == INFINITY ? relative(y, top) : y - top) * rate;
          // NaN is no candidate: a maximum takes the other side
          sum += ex2((keep[u] >> e) & 1u ? fmaxf(t, -200.0f) : -200.0f);
        }
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullWarp, sum, o);
    }
    if (lane == 0) a.part[i] = make_float2(top, sum);
  }
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
  float score;
  int token;
};

// The best of all the cluster's threads, in every thread.
__device__ __forceinline__ Found cluster_best(Found f, Found* warps, Found* mine) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    best_of(f.score, f.token, __shfl_xor_sync(kFullWarp, f.score, o),
            __shfl_xor_sync(kFullWarp, f.token, o));
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = f;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kWarps; ++i) best_of(f.score, f.token, warps[i].score, warps[i].token);
    *mine = f;
  }
  cluster_sync();
  const uint32_t at = uint32_t(__cvta_generic_to_shared(mine));
  f.score = -INFINITY, f.token = INT32_MAX;
  for (uint32_t r = 0; r < cluster_size(); ++r) {
    uint32_t remote, s, t;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(r));
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(s), "=r"(t) : "r"(remote) : "memory");
    best_of(f.score, f.token, __uint_as_float(s), int(t));
  }
  cluster_sync();  // nobody leaves, or writes the next one, before all have read
  return f;
}

template <int DT>
__device__ __forceinline__ float logit_at(const char* x, int v) {
  return Elt<DT>::load1(x + int64_t(v) * Elt<DT>::kBytes);
}

// A cluster of blocks a slot.
template <int DT>
__global__ void __launch_bounds__(kThreads) verify_say_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ float tops[kMostRows], sums[kMostRows];
  __shared__ int firsts[kMostRows];  // greedy: the lowest-index largest
  __shared__ Found warps[kWarps];
  __shared__ alignas(8) Found mine;
  __shared__ int count, there;
  const int blocks = int(cluster_size()), rank = int(cluster_rank());
  const int slot = blockIdx.x / blocks, R = a.per_slot, tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) count = there = R - 1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const float heat = heat_of(a, slot);
  const bool greedy = !(heat > 0.0f);
  const float rate = rate_of(heat);
  const int64_t* drafts = a.drafts + int64_t(slot) * (R - 1);
  for (int i = tid >> 5; i < R; i += kWarps) {
    const int64_t row = int64_t(slot) * R + i;
    const float2* part = a.part + row * a.chunks;
    float top = -INFINITY, sum = 0.0f;
    for (int c = lane; c < a.chunks; c += 32) {
      const float2 p = part[c];
      const float now = fmaxf(top, p.x);
      if (now > -INFINITY)
        sum = sum * ex2(relative(top, now) * rate) + p.y * ex2(relative(p.x, now) * rate);
      top = now;
    }
    float all = top;
#pragma unroll
    for (int o = 16; o; o >>= 1) all = fmaxf(all, __shfl_xor_sync(kFullWarp, all, o));
    sum = top > -INFINITY ? sum * ex2(relative(top, all) * rate) : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullWarp, sum, o);
    int first = INT32_MAX;
    if (greedy && all > -INFINITY) {  // in the first chunk that has it
      int chunk = INT32_MAX;
      for (int c = lane; c < a.chunks; c += 32)
        if (chunk == INT32_MAX && part[c].x == all) chunk = c;
      chunk = __reduce_min_sync(kFullWarp, chunk);
      const RowVecs<DT> x(a, row);
      const int64_t vecs = x.count();
      for (int u = 0; u < kVecs; ++u) {
        const int64_t q = int64_t(chunk) * kChunkVecs + u * 32 + lane;
        if (q >= vecs) continue;
        const uint4 raw = __ldg(reinterpret_cast<const uint4*>(x.at) + q);
        const uint32_t keep = x.bits(q);
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
  for (int i = tid; i < R - 1; i += kThreads) {
    const int64_t v = drafts[i];
    bool taken = false;
    if (v < 0 || v >= a.V) {
      atomicMin(&there, i);
    } else {
      const int64_t row = int64_t(slot) * R + i;
      double p = 0.0;
      if (greedy) {
        p = v == firsts[i] ? 1.0 : 0.0;
      } else if (kept(mask_of(a, row), int(v))) {
        const float x = logit_at<DT>(a.logits + row * a.stride, int(v));
        if (x > -INFINITY) p = exp(double(relative(x, tops[i])) / double(heat)) / double(sums[i]);
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
  const float top = tops[n], sum = sums[n];
  const bool refused = n < there;
  int token = firsts[n];
  if (!greedy && top > -INFINITY) {
    const uint32_t* mask = mask_of(a, row);
    const char* x = a.logits + row * a.stride;
    const float* q = refused && a.probs != nullptr
                         ? a.probs + slot * a.probs_slot + n * a.probs_row : nullptr;
    const int64_t draft = refused ? drafts[n] : -1;
    const uint64_t seed = a.seeds != nullptr ? a.seeds[row] : a.seed;
    const uint2 key = make_uint2(uint32_t(seed), uint32_t(seed >> 32));
    const bool whole = (reinterpret_cast<uintptr_t>(x) % (4 * Elt<DT>::kBytes)) == 0;
    const bool whole_q = q != nullptr && reinterpret_cast<uintptr_t>(q) % 16 == 0;
    const float inv = 1.0f / sum;
    const float shift = __fdiv_rn(top, heat);
    for (int rest = refused; rest >= 0; --rest) {  // the second time where nothing was left
      Found f = {-INFINITY, INT32_MAX};
      float bound = 3e38f;  // exp(-best), of what r is measured in
      const int step = blocks * kThreads * 4;
      for (int v4 = (rank * kThreads + tid) * 4; v4 < a.V; v4 += step) {
        const int m = min(4, a.V - v4);
        uint32_t keep = (1u << m) - 1u;
        if (mask != nullptr) keep &= __ldg(mask + (v4 >> 5)) >> (v4 & 31);
        if (keep != 0) {
          float y[4], d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          if (whole && m == 4) {
            if (DT == LP_F32) {
              const float4 w = __ldg(reinterpret_cast<const float4*>(x) + v4 / 4);
              y[0] = w.x, y[1] = w.y, y[2] = w.z, y[3] = w.w;
            } else {
              const uint2 w = __ldg(reinterpret_cast<const uint2*>(x) + v4 / 4);
              const uint4 w4 = make_uint4(w.x, w.y, 0, 0);
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = Elt<DT>::get(w4, e);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = e < m ? logit_at<DT>(x, v4 + e) : -INFINITY;
          }
          if (rest && q != nullptr) {
            if (whole_q && m == 4) {
              const float4 w = __ldg(reinterpret_cast<const float4*>(q) + v4 / 4);
              d[0] = w.x, d[1] = w.y, d[2] = w.z, d[3] = w.w;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) d[e] = e < m ? __ldg(q + v4 + e) : 0.0f;
            }
          } else if (rest) {
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = v4 + e == draft ? 1.0f : 0.0f;
          }
          const uint4 w = philox4x32_10(make_uint4(uint32_t(v4) >> 2, uint32_t(row),
                                                   uint32_t(a.offset), uint32_t(a.offset >> 32)), key);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (!((keep >> e) & 1u) || !(y[e] > -INFINITY)) continue;
            const uint32_t word = word_of(w, e);
            const float p = ex2(relative(y[e], top) * rate) * (rest ? inv : 1.0f);
            const float missing = (float(~word >> 9) + 0.5f) * 1.1920928955078125e-07f;  // 1 - u
            // p is within 1e-5 of itself, whatever is left of p - d
            if (!(missing < fmaf(p, 1.00002f, -d[e]) * bound * 1.001f)) continue;
            float score;
            if (rest) {
              const float r = expf(__fdiv_rn(relative(y[e], top), heat)) / sum - d[e];
              if (!(r > 0.0f)) continue;
              score = logf(r);
            } else {
              score = __fdiv_rn(y[e], heat);
            }
            best_of(f.score, f.token, score + gumbel_from_word(word), v4 + e);
            if (fabsf(shift) < 1024.0f) bound = fminf(expf((rest ? 0.0f : shift) - f.score), 3e38f);
          }
        }
        // what the warp has found holds for all of its lanes
        bound = __uint_as_float(__reduce_min_sync(__activemask(), __float_as_uint(bound)));
      }
      f = cluster_best(f, warps, &mine);
      token = f.token;
      if (token != INT32_MAX) break;
    }
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
  const int64_t warps = int64_t(a.rows) * a.chunks;
  cfg.gridDim = dim3(unsigned(std::min<int64_t>((warps + 7) / 8, kSms * 64)));
  const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_stream_kernel<DT>, a);
  if (e != cudaSuccess) return e;
  const int64_t slots = a.rows / a.per_slot;
  // blocks to a slot: as many as have a round of tokens, and as all slots have room for
  int blocks = kMostCluster;
  while (blocks > 1 && (slots * blocks > kSms * 4 || blocks * kThreads * 4 >= 2 * a.V)) blocks /= 2;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = unsigned(blocks);
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  cfg.blockDim = dim3(kThreads);
  cfg.gridDim = dim3(unsigned(slots * blocks));
  return cudaLaunchKernelEx(&cfg, verify_say_kernel<DT>, a);
}

// Chunks of a row, wherever it starts.
int64_t chunks_of(lp_dtype dt, int64_t V) {
  const int64_t per = dt == LP_F32 ? 4 : 8;
  return std::max<int64_t>(1, (V + per - 1 + per * kChunkVecs - 1) / (per * kChunkVecs));
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
  a.chunks = int(chunks_of(dt, V));
  const cudaError_t e = dt == LP_F32   ? launch<LP_F32>(a, stream)
                        : dt == LP_F16 ? launch<LP_F16>(a, stream)
                                       : launch<LP_BF16>(a, stream);
  return status_of(e);
}
