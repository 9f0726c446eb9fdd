// evict.cu -- a cache's sequences cut to their tokens of most attention weight, in place.
//
// Of a head's n > keep tokens stay the first ones, the last ones and the K = keep - first -
// recent heaviest of those between.  The K-th largest weight is found digit by digit, eight
// bits of an order-preserving key at a time; what is above it stays, and of what equals it
// the lowest ones.  The j-th kept token, at s(j) >= j, moves to place j.  s(j) > j' for every
// j' < j: places written for earlier tokens hold no source of later ones, so a block that
// goes through them in order, and reads a batch before it writes it, needs no second copy.
#include <algorithm>

#include "common.cuh"

namespace lp {
namespace {

constexpr int kMaxParts = 8;
constexpr int kThreads = 1024;
constexpr int kMoveThreads = 512;
constexpr int kAtOnce = 4;  // pieces a thread holds

struct EvictArgs {
  lp_cache_part part[kMaxParts];
  int n_parts;
  int64_t n_slots, page;
  Div per_page;
  int heads;
  int code_bytes, param_bytes;  // of a head
  int code_unit, param_unit;    // bytes moved at once
  float* weights;
  int64_t weights_batch, weights_head;
  int batch;
  const int32_t* blocks;
  int64_t blocks_stride, block;
  int most;
  Div per_block;
  const int32_t* lengths;
  int keep, first, recent;
  int32_t* new_lengths;
  int32_t* source;  // [batch, heads, keep]: s(j)
};

__device__ __forceinline__ int64_t place(const EvictArgs& a, int64_t slot, int64_t page_stride,
                                         int64_t slot_stride) {
  if (a.page >= a.n_slots) return slot * slot_stride;
  const int64_t p = a.n_slots <= INT32_MAX ? int64_t(a.per_page.quot(uint32_t(slot)))
                                           : slot / a.page;
  return p * page_stride + (slot - p * a.page) * slot_stride;
}

__device__ __forceinline__ int64_t slot_of(const EvictArgs& a, int b, int t) {
  const uint32_t i = a.per_block.quot(uint32_t(t));
  const int64_t slot = int64_t(__ldg(a.blocks + int64_t(b) * a.blocks_stride + i)) * a.block +
                       (t - int64_t(i) * a.block);
  return slot >= 0 && slot < a.n_slots ? slot : -1;
}

// Keys in the order of the weights; 0 for NaN, which counts as the least.
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 0u : fkey(w); }

// The sum over the threads before this one, and *all over all; two barriers.
__device__ __forceinline__ int scan(int x, int* warps, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFullWarp, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i == warp) before = total;
    total += warps[i];
  }
  *all = total;
  return before + incl - x;
}

// Which tokens stay: a block a sequence and head.  Moves the weights.
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int counts[256], warps[kThreads / 32], digit, above;
  const int b = blockIdx.x / a.heads, h = blockIdx.x - b * a.heads, tid = threadIdx.x;
  const int n = min(max(__ldg(a.lengths + b), 0), a.most);
  const int left = min(n, a.keep);
  if (n <= a.keep || a.weights == nullptr) {
    if (h == 0 && tid == 0) a.new_lengths[b] = left;
    return;
  }
  float* w = a.weights + b * a.weights_batch + h * a.weights_head;
  int32_t* source = a.source + (int64_t(b) * a.heads + h) * a.keep;
  const int lo = a.first, hi = n - a.recent;
  int want = a.keep - a.first - a.recent;  // of [lo, hi)
  uint32_t key = 0;                        // of the want-th largest, as far as it is known
  for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) counts[i] = 0;
    __syncthreads();
    for (int t = lo + tid; t < hi; t += kThreads) {
      const uint32_t k = weight_key(w[t]);
      if (shift == 24 || (k >> (shift + 8)) == (key >> (shift + 8)))
        atomicAdd(&counts[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int over = 0, d = 255;
      while (d > 0 && over + counts[d] < want) over += counts[d--];
      digit = d, above = over;
    }
    __syncthreads();
    key |= uint32_t(digit) << shift;
    want -= above;
    __syncthreads();
  }
  // key: the smallest that stays; `want` of those equal to it do
  const bool none = a.keep == a.first + a.recent;
  int at = 0, equal = 0;
  for (int t0 = 0; t0 < n; t0 += kThreads) {
    const int t = t0 + tid;
    const float x = t < n ? w[t] : 0.0f;
    const uint32_t k = weight_key(x);
    const bool held = t < n && (t < lo || t >= hi);
    const bool middle = t < n && !held && !none;
    int all;
    const int rank = equal + scan(middle && k == key, warps, &all);
    equal += all;
    const bool stays = held || (middle && (k > key || (k == key && rank < want)));
    const int j = at + scan(stays, warps, &all);
    at += all;
    if (stays) source[j] = t, w[j] = x;
  }
  __syncthreads();
  for (int t = left + tid; t < n; t += kThreads) w[t] = 0.0f;
  if (h == 0 && tid == 0) a.new_lengths[b] = left;
}

struct alignas(16) Piece {
  uint32_t w[4];
};

__device__ __forceinline__ void load_piece(Piece& p, const char* from, int unit) {
  if (unit == 16) p = *reinterpret_cast<const Piece*>(from);
  else if (unit == 8) *reinterpret_cast<uint2*>(&p) = *reinterpret_cast<const uint2*>(from);
  else if (unit == 4) p.w[0] = *reinterpret_cast<const uint32_t*>(from);
  else if (unit == 2) p.w[0] = *reinterpret_cast<const uint16_t*>(from);
  else p.w[0] = *reinterpret_cast<const uint8_t*>(from);
}

__device__ __forceinline__ void store_piece(const Piece& p, char* to, int unit) {
  if (unit == 16) *reinterpret_cast<Piece*>(to) = p;
  else if (unit == 8) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(&p);
  else if (unit == 4) *reinterpret_cast<uint32_t*>(to) = p.w[0];
  else if (unit == 2) *reinterpret_cast<uint16_t*>(to) = uint16_t(p.w[0]);
  else *reinterpret_cast<uint8_t*>(to) = uint8_t(p.w[0]);
}

// Moves codes and params: a block a sequence and head.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  const int b = blockIdx.x / a.heads, h = blockIdx.x - b * a.heads;
  const int n = min(max(__ldg(a.lengths + b), 0), a.most);
  if (n <= a.keep) return;
  const int32_t* source = a.source + (int64_t(b) * a.heads + h) * a.keep;
  const int codes = a.code_bytes / a.code_unit, params = a.param_bytes / a.param_unit;
  const int per_part = codes + params, per_token = a.n_parts * per_part;
  const int64_t total = int64_t(a.keep) * per_token;
  for (int64_t i0 = 0; i0 < total; i0 += kMoveThreads * kAtOnce) {
    Piece held[kAtOnce];
    char* to[kAtOnce];
    int unit[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      to[u] = nullptr;
      unit[u] = 0;
      const int64_t i = i0 + u * kMoveThreads + threadIdx.x;
      if (i >= total) continue;
      const int j = int(i / per_token), piece = int(i - int64_t(j) * per_token);
      const int s = source[j];
      if (s == j) continue;
      const int64_t from_slot = slot_of(a, b, s), to_slot = slot_of(a, b, j);
      if (from_slot < 0 || to_slot < 0) continue;
      const lp_cache_part& p = a.part[piece / per_part];
      const int e = piece % per_part;
      const bool is_code = e < codes;
      const int64_t page_stride = is_code ? p.code_page_stride : p.param_page_stride;
      const int64_t slot_stride = is_code ? p.code_slot_stride : p.param_slot_stride;
      char* base = static_cast<char*>(is_code ? p.codes : p.params) +
                   h * (is_code ? p.code_head_stride : p.param_head_stride) +
                   (is_code ? e * a.code_unit : (e - codes) * a.param_unit);
      unit[u] = is_code ? a.code_unit : a.param_unit;
      to[u] = base + place(a, to_slot, page_stride, slot_stride);
      load_piece(held[u], base + place(a, from_slot, page_stride, slot_stride), unit[u]);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (to[u] != nullptr) store_piece(held[u], to[u], unit[u]);
    __syncthreads();
  }
}

bool fits(int64_t a, int64_t b, int64_t most) { return b == 0 || a <= most / b; }

// The widest unit that divides everything in `bits_of`.
int unit_of(uint64_t bits_of) {
  for (int u : {16, 8, 4, 2})
    if (bits_of % u == 0) return u;
  return 1;
}

}  // namespace
}  // namespace lp

extern "C" int64_t lp_cache_evict_workspace_bytes(int64_t batch, int64_t heads, int64_t keep) {
  using namespace lp;
  if (batch < 0 || heads < 0 || keep < 0 || keep > INT32_MAX || !fits(batch, heads, INT32_MAX))
    return -1;
  return (batch * heads * keep * 4 + 15) / 16 * 16;
}

extern "C" lp_status lp_cache_evict(const lp_cache_part* parts, int64_t n_parts, int32_t bits,
                                    int64_t n_slots, int64_t page_size, int64_t heads, int64_t dim,
                                    int64_t group, float* weights, int64_t weights_batch_stride,
                                    int64_t weights_head_stride, int64_t batch,
                                    const int32_t* blocks, int64_t blocks_stride,
                                    int64_t max_blocks, int64_t block_size, const int32_t* lengths,
                                    int64_t keep, int64_t first, int64_t recent,
                                    int32_t* new_lengths, void* workspace, int64_t workspace_bytes,
                                    cudaStream_t stream) {
  using namespace lp;
  if (n_parts < 0 || n_parts > kMaxParts || (bits != 8 && bits != 4) || n_slots < 0 ||
      page_size < 1 || heads < 0 || dim < 0 || group < 1 || dim % group != 0 ||
      (bits == 4 && group % 2 != 0) || batch < 0 || max_blocks < 0 || block_size < 1 ||
      blocks_stride < max_blocks || keep < 0 || first < 0 || recent < 0 || first > keep ||
      recent > keep - first)
    return LP_ERR_INVALID_ARGUMENT;
  if (heads > INT32_MAX || dim > (1 << 29) || !fits(block_size, max_blocks, 1 << 30) ||
      !fits(batch, heads, INT32_MAX) || batch > INT32_MAX)
    return LP_ERR_TOO_LARGE;
  if (batch == 0) return LP_OK;
  const int64_t most = max_blocks * block_size;
  // no sequence is longer than the blocks hold
  keep = std::min(keep, most), first = std::min(first, keep), recent = std::min(recent, keep - first);
  if (lengths == nullptr || new_lengths == nullptr || (most > 0 && blocks == nullptr) ||
      (most > 0 && heads > 0 && weights == nullptr) || (n_parts > 0 && parts == nullptr) ||
      (reinterpret_cast<uintptr_t>(blocks) | reinterpret_cast<uintptr_t>(lengths) |
       reinterpret_cast<uintptr_t>(new_lengths) | reinterpret_cast<uintptr_t>(weights)) % 4 != 0 ||
      (new_lengths < lengths + batch && lengths < new_lengths + batch))
    return LP_ERR_INVALID_ARGUMENT;
  EvictArgs a = {};
  uint64_t code_bits = uint64_t(dim) * bits / 8, param_bits = uint64_t(dim / group) * 4;
  a.code_bytes = int(code_bits), a.param_bytes = int(param_bits);
  for (int64_t i = 0; i < n_parts; ++i) {
    const lp_cache_part& p = parts[i];
    if (n_slots > 0 && dim > 0 && (p.codes == nullptr || p.params == nullptr))
      return LP_ERR_INVALID_ARGUMENT;
    if ((reinterpret_cast<uintptr_t>(p.params) | uint64_t(p.param_page_stride) |
         uint64_t(p.param_slot_stride) | uint64_t(p.param_head_stride)) % 4 != 0)
      return LP_ERR_INVALID_ARGUMENT;
    code_bits |= reinterpret_cast<uintptr_t>(p.codes) | uint64_t(p.code_page_stride) |
                 uint64_t(p.code_slot_stride) | uint64_t(p.code_head_stride);
    param_bits |= reinterpret_cast<uintptr_t>(p.params) | uint64_t(p.param_page_stride) |
                  uint64_t(p.param_slot_stride) | uint64_t(p.param_head_stride);
    a.part[i] = p;
  }
  const int64_t need = lp_cache_evict_workspace_bytes(batch, heads, keep);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need ||
                   reinterpret_cast<uintptr_t>(workspace) % 16 != 0))
    return LP_ERR_INVALID_ARGUMENT;
  a.n_parts = dim > 0 ? int(n_parts) : 0;
  a.n_slots = n_slots;
  a.page = page_size;
  if (page_size < n_slots && n_slots <= INT32_MAX) a.per_page.set(uint32_t(page_size));
  a.heads = std::max(1, int(heads));
  a.code_unit = unit_of(code_bits), a.param_unit = unit_of(param_bits);
  a.weights = heads > 0 ? weights : nullptr;
  a.weights_batch = weights_batch_stride, a.weights_head = weights_head_stride;
  a.batch = int(batch);
  a.blocks = blocks;
  a.blocks_stride = blocks_stride;
  a.block = block_size;
  a.most = int(most);
  a.per_block.set(uint32_t(std::min<int64_t>(block_size, INT32_MAX)));
  a.lengths = lengths;
  a.keep = int(keep), a.first = int(first), a.recent = int(recent);
  a.new_lengths = new_lengths;
  a.source = static_cast<int32_t*>(workspace);
  const dim3 grid(unsigned(batch * a.heads));
  cudaError_t e = launch_kernel(evict_select_kernel, grid, dim3(kThreads), 0, stream, a);
  if (e == cudaSuccess && a.n_parts > 0 && heads > 0 && n_slots > 0)
    e = launch_kernel(evict_move_kernel, grid, dim3(kMoveThreads), 0, stream, a);
  return status_of(e);
}
