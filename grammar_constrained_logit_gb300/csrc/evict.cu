// evict.cu -- a cache's sequences cut to their tokens of most attention weight, in place.
//
// Of a head's n > keep tokens stay the first ones, the last ones and the K = keep - first -
// recent heaviest of those between.  The K-th largest weight is found digit by digit of
// an order-preserving key, of 9, 8, 8 and 7 bits (four of 8 past a cluster's shared memory); what
// is above it stays, and of what equals it
// the lowest ones.  The j-th kept token, at s(j) >= j, moves to place j.
//
// s(j') > j for every j < j': what is written for a token is never the source of a later one,
// so loads may run ahead of stores as far as they like, and a store has to wait only for the
// loads of its own round and those before it.  A round is what the blocks of a cluster hold
// in shared memory; they meet at one barrier a round, with the next round's loads under way.
//
// Measured, in a graph, 8 heads of 128: 32 sequences of up to 4096 tokens to 2048 in 8 bits 68 us
// (17 the selection, 50 the moves; 113 MB), 4 of 65536 to 16384 in 4 bits 102 us (37 and 64), one
// of 640 to 512 11.5 us.  Selection: chains of barriers over a cluster.  Moves: instructions,
// 53% of the issue slots, for pieces of 16 bytes, and the rounds' barriers; with a thread's
// place worked out for each piece instead of once they took twice as long.
#include <algorithm>

#include "common.cuh"

namespace lp {
namespace {

constexpr int kMaxParts = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kCodeThreads = 224;        // of a block: the last warp moves params
constexpr int kRoundTokens = kMoveThreads;  // a thread looks one up
constexpr int kMostCluster = 8;
constexpr int kSms = 152;
constexpr int kBins = 512;
constexpr int kHeldTokens = 40 * 1024;  // weights that a block holds in shared memory
constexpr int kRoundBytes = 48 * 1024;  // of a round's tokens, at most; a block holds two

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
  int slice;        // tokens of a sequence to a block of the selection
  int round_tokens;
};

__device__ __forceinline__ int cluster_size() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return int(n);
}
__device__ __forceinline__ int cluster_rank() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(n));
  return int(n);
}
__device__ __forceinline__ void cluster_sync(int blocks) {
  if (blocks == 1) {
    __syncthreads();
    return;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Words of another block's shared memory, at the place of `p` in this one's.
__device__ __forceinline__ uint32_t remote_at(const void* p, int rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(at) : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(uint32_t(rank)));
  return at;
}
__device__ __forceinline__ int2 remote2(const void* p, int rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y) : "r"(remote_at(p, rank)) : "memory");
  return v;
}

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

// The sums over the warps before this one of each warp's (x, y), and over all: one barrier,
// and one before it.
__device__ __forceinline__ int2 warps_before(int2 x, int2* warps, int2* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) warps[warp] = x;
  __syncthreads();
  int2 v = lane < kWarps ? warps[lane] : make_int2(0, 0);
  int2 incl = v;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const int y = __shfl_up_sync(kFullWarp, incl.x, o), z = __shfl_up_sync(kFullWarp, incl.y, o);
    if (lane >= o) incl.x += y, incl.y += z;
  }
  *all = make_int2(__shfl_sync(kFullWarp, incl.x, kWarps - 1),
                   __shfl_sync(kFullWarp, incl.y, kWarps - 1));
  return make_int2(__shfl_sync(kFullWarp, incl.x - v.x, warp),
                   __shfl_sync(kFullWarp, incl.y - v.y, warp));
}

// Which tokens stay, and where the weights go: a cluster of blocks a sequence and head, each
// with a slice of the weights in shared memory.
__global__ void __launch_bounds__(kThreads, 2)
    evict_slices_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ float held[];
  __shared__ alignas(8) int bins[4][kBins];
  __shared__ int2 warps[kWarps];
  __shared__ alignas(8) int counts[2];
  __shared__ int found[2];
  const int blocks = cluster_size(), rank = cluster_rank(), tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x / blocks, b = unit / a.heads, h = unit - b * a.heads;
  for (int i = tid; i < 4 * kBins; i += kThreads) bins[0][i] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n = min(max(__ldg(a.lengths + b), 0), a.most);
  const int left = min(n, a.keep);
  if (n <= a.keep || a.weights == nullptr) {  // for all of the cluster
    if (h == 0 && rank == 0 && tid == 0) a.new_lengths[b] = left;
    return;
  }
  float* w = a.weights + b * a.weights_batch + h * a.weights_head;
  int32_t* source = a.source + (int64_t(b) * a.heads + h) * a.keep;
  const int lo = a.first, hi = n - a.recent;
  const int t0 = min(n, rank * a.slice), t1 = min(n, t0 + a.slice);  // this block's
#pragma unroll 4
  for (int i = tid; i < t1 - t0; i += kThreads) held[i] = w[t0 + i];
  __syncthreads();
  int want = a.keep - a.first - a.recent;  // of [lo, hi)
  const bool none = want == 0;
  uint32_t key = 0;  // of the want-th largest, as far as it is known
#pragma unroll
  for (int pass = 0; pass < 4; ++pass) {
    if (none) break;
    // 9, 8, 8 and 7 bits: the first are sign and exponent
    constexpr int kShift[4] = {23, 15, 7, 0}, kDigits[4] = {512, 256, 256, 128};
    const int shift = kShift[pass], digits = kDigits[pass];
#pragma unroll 4
    for (int i0 = warp * 32; i0 < t1 - t0; i0 += kThreads) {
      const int i = i0 + lane, t = t0 + i;
      const uint32_t k = i < t1 - t0 ? weight_key(held[i]) : 0u;
      const bool counts_here = i < t1 - t0 && t >= lo && t < hi &&
                               (pass == 0 || (k >> kShift[max(0, pass - 1)]) ==
                                                 (key >> kShift[max(0, pass - 1)]));
      const uint32_t digit = (k >> shift) & (digits - 1);
      if (pass == 0) {  // many of a warp's share an exponent: one addition for each
        const uint32_t same = __match_any_sync(kFullWarp, counts_here ? digit : kBins);
        if (counts_here && lane == __ffs(same) - 1) atomicAdd(&bins[pass][digit], __popc(same));
      } else if (counts_here) {
        atomicAdd(&bins[pass][digit], 1);
      }
    }
    cluster_sync(blocks);
    // this thread's two digits, the highest first, over all blocks
    const int low = digits - 2 * (tid + 1);
    int2 sum = make_int2(0, 0);
    if (low >= 0) {
      if (blocks == 1) {
        sum = *reinterpret_cast<const int2*>(&bins[pass][low]);
      } else {
        int2 v[kMostCluster];
#pragma unroll
        for (int r = 0; r < kMostCluster; ++r)
          v[r] = r < blocks ? remote2(&bins[pass][low], r) : make_int2(0, 0);
#pragma unroll
        for (int r = 0; r < kMostCluster; ++r) sum.x += v[r].x, sum.y += v[r].y;
      }
    }
    int incl = sum.x + sum.y;
    const int own = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFullWarp, incl, o);
      if (lane >= o) incl += y;
    }
    int2 all;
    const int before = warps_before(make_int2(__shfl_sync(kFullWarp, incl, 31), 0), warps, &all).x +
                       incl - own;
    if (before < want && want <= before + own) {
      const bool high = want <= before + sum.y;
      found[0] = high ? low + 1 : low;
      found[1] = high ? before : before + sum.y;
    }
    __syncthreads();
    key |= uint32_t(found[0]) << shift;
    want -= found[1];
  }
  // A warp's run of tokens, in order: what stays for sure, and what equals the key
  const int run = ((t1 - t0 + kThreads - 1) / kThreads) * 32;
  const int i0 = min(t1 - t0, warp * run), i1 = min(t1 - t0, i0 + run);
  const auto kind = [&](int i) {  // 0: goes, 1: equals the key, 2: stays
    if (i >= i1) return 0;
    const int t = t0 + i;
    if (t < lo || t >= hi) return 2;
    if (none) return 0;
    const uint32_t k = weight_key(held[i]);
    return k > key ? 2 : int(k == key);
  };
  int2 mine = make_int2(0, 0);
#pragma unroll 4
  for (int i = i0; i < i1; i += 32) {
    const int x = kind(i + lane);
    mine.x += __popc(__ballot_sync(kFullWarp, x == 2));
    mine.y += __popc(__ballot_sync(kFullWarp, x == 1));
  }
  int2 all;
  int2 at = warps_before(mine, warps, &all);
  if (tid == 0) counts[0] = all.x, counts[1] = all.y;
  cluster_sync(blocks);
  for (int r = 0; r < rank; ++r) {
    const int2 v = remote2(counts, r);
    at.x += v.x, at.y += v.y;
  }
  // every block has read its weights: they may be written
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
  for (int i = i0; i < i1; i += 32) {
    const int x = kind(i + lane);
    const uint32_t sure = __ballot_sync(kFullWarp, x == 2), equal = __ballot_sync(kFullWarp, x == 1);
    const int rank_equal = at.y + __popc(equal & below);
    if (x == 2 || (x == 1 && rank_equal < want)) {
      const int j = at.x + __popc(sure & below) + min(rank_equal, want);
      source[j] = t0 + i + lane;
      w[j] = held[i + lane];
    }
    at.x += __popc(sure), at.y += __popc(equal);
  }
  for (int t = max(t0, left) + tid; t < t1; t += kThreads) w[t] = 0.0f;
  if (h == 0 && rank == 0 && tid == 0) a.new_lengths[b] = left;
  cluster_sync(blocks);  // counts are read by others
}

// The same for sequences longer than a cluster's shared memory holds: a block each, going
// through the weights in order.
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

template <typename T>
__device__ __forceinline__ void copy_as(void* to, const void* from) {
  *static_cast<T*>(to) = *static_cast<const T*>(from);
}

__device__ __forceinline__ void copy_unit(void* to, const void* from, int unit) {
  if (unit == 16) copy_as<Piece>(to, from);
  else if (unit == 8) copy_as<uint2>(to, from);
  else if (unit == 4) copy_as<uint32_t>(to, from);
  else if (unit == 2) copy_as<uint16_t>(to, from);
  else copy_as<uint8_t>(to, from);
}

// Into shared memory: started, and waited for later, where the unit allows it.
__device__ __forceinline__ void fetch_unit(char* to, const char* from, int unit) {
  const uint32_t at = uint32_t(__cvta_generic_to_shared(to));
  if (unit == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else if (unit == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(from) : "memory");
  else if (unit == 4) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at), "l"(from) : "memory");
  else copy_unit(to, from, unit);
}

// Moves codes and params: a cluster of blocks a sequence and head, in rounds.  A thread has
// one piece of a token, of every `step`-th token: its strides and bases are worked out once,
// and what it fetches it stores itself.
__global__ void __launch_bounds__(kMoveThreads, 4)
    evict_move_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) char staged[];  // [2][round_tokens][pieces][16]
  __shared__ int64_t from_slots[3][kRoundTokens], to_slots[3][kRoundTokens];
  const int blocks = cluster_size(), rank = cluster_rank();
  const int owner = blockIdx.x / blocks, b = owner / a.heads, h = owner - b * a.heads;
  const int code_pieces = a.code_bytes / a.code_unit, param_pieces = a.param_bytes / a.param_unit;
  const int staged_bytes = a.n_parts * (code_pieces + param_pieces) * 16;  // of a token
  const bool is_code = threadIdx.x < kCodeThreads;
  const int unit = is_code ? a.code_unit : a.param_unit;
  const int per_part = is_code ? code_pieces : param_pieces, pieces = a.n_parts * per_part;
  const int at = is_code ? threadIdx.x : threadIdx.x - kCodeThreads;
  const int step = (is_code ? kCodeThreads : kMoveThreads - kCodeThreads) / pieces;
  const int first = at / pieces;
  int piece = at - first * pieces;
  char* stage = staged + (is_code ? piece : a.n_parts * code_pieces + piece) * 16;
  const int part = piece / per_part;
  piece -= part * per_part;
  const lp_cache_part& p = a.part[part];
  const int64_t page_stride = is_code ? p.code_page_stride : p.param_page_stride;
  const int64_t slot_stride = is_code ? p.code_slot_stride : p.param_slot_stride;
  char* base = static_cast<char*>(is_code ? p.codes : p.params) +
               h * (is_code ? p.code_head_stride : p.param_head_stride) + piece * unit;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n = min(max(__ldg(a.lengths + b), 0), a.most);
  if (n <= a.keep) return;  // for all of the cluster
  const int32_t* source = a.source + (int64_t(b) * a.heads + h) * a.keep;
  const int per_round = a.round_tokens * blocks;
  const int rounds = (a.keep + per_round - 1) / per_round;

  // A round's tokens are looked up two rounds ahead, in three steps that wait for one another
  // only where there is other work between: the source, its block, its slot.
  const auto place_of = [&](int round) {
    return (int64_t(round) * blocks + rank) * a.round_tokens + threadIdx.x;
  };
  const auto source_of = [&](int round) {
    const int64_t j = place_of(round);
    return threadIdx.x < a.round_tokens && round < rounds && j < a.keep ? source[j] : -1;
  };
  const auto block_id = [&](int t) {
    return t < 0 ? -1
                 : __ldg(a.blocks + int64_t(b) * a.blocks_stride + a.per_block.quot(uint32_t(t)));
  };
  const auto slot_in = [&](int id, int t) {
    const int64_t slot = int64_t(id) * a.block +
                         (t - int64_t(a.per_block.quot(uint32_t(t))) * a.block);
    return t >= 0 && slot >= 0 && slot < a.n_slots ? slot : int64_t(-1);
  };
  const auto put = [&](int round, int s, int from_id, int to_id) {
    if (threadIdx.x >= a.round_tokens || round >= rounds) return;
    const int j = s < 0 || place_of(round) == s ? -1 : int(place_of(round));
    const int64_t from = slot_in(from_id, j < 0 ? -1 : s), to = slot_in(to_id, j);
    from_slots[round % 3][threadIdx.x] = to < 0 ? -1 : from;
    to_slots[round % 3][threadIdx.x] = to;
  };
  const auto fetch = [&](int round) {
    if (round < rounds && first < step)
#pragma unroll 2
      for (int i = first; i < a.round_tokens; i += step) {
        const int64_t from = from_slots[round % 3][i];
        if (from >= 0)
          fetch_unit(stage + ((round & 1) * a.round_tokens + i) * staged_bytes,
                     base + place(a, from, page_stride, slot_stride), unit);
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const auto store = [&](int round) {
    if (first < step)
#pragma unroll 2
      for (int i = first; i < a.round_tokens; i += step)
        if (from_slots[round % 3][i] >= 0)
          copy_unit(base + place(a, to_slots[round % 3][i], page_stride, slot_stride),
                    stage + ((round & 1) * a.round_tokens + i) * staged_bytes, unit);
  };

  for (int round = 0; round < 2; ++round) {
    const int s = source_of(round);
    put(round, s, block_id(s), block_id(s < 0 ? -1 : int(place_of(round))));
  }
  __syncthreads();
  fetch(0);
  int ahead = source_of(2);
  for (int round = 0; round < rounds; ++round) {
    fetch(round + 1);
    const int from_id = block_id(ahead), to_id = block_id(ahead < 0 ? -1 : int(place_of(round + 2)));
    const int after = source_of(round + 3);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    if (blocks == 1) {
      __syncthreads();  // the sources are read, by all
    } else {
      // nothing was written that the others wait for: the loads are done, and that is all
      asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    store(round);
    put(round + 2, ahead, from_id, to_id);
    ahead = after;
    __syncthreads();  // the slots of two rounds from here are there
  }
}

// The same for tokens of more pieces than a round: a block a sequence and head.
__global__ void __launch_bounds__(kMoveThreads)
    evict_move_wide_kernel(const __grid_constant__ EvictArgs a) {
  const int b = blockIdx.x / a.heads, h = blockIdx.x - b * a.heads;
  const int n = min(max(__ldg(a.lengths + b), 0), a.most);
  if (n <= a.keep) return;
  const int32_t* source = a.source + (int64_t(b) * a.heads + h) * a.keep;
  const int codes = a.code_bytes / a.code_unit, params = a.param_bytes / a.param_unit;
  const int per_part = codes + params;
  const int64_t per_token = int64_t(a.n_parts) * per_part;
  const int64_t total = int64_t(a.keep) * per_token;
  for (int64_t i0 = 0; i0 < total; i0 += kMoveThreads) {
    Piece held;
    char* to = nullptr;
    int unit = 0;
    const int64_t i = i0 + threadIdx.x;
    if (i < total) {
      const int j = int(i / per_token);
      const int64_t piece = i - j * per_token;
      const int s = source[j];
      const int64_t from_slot = slot_of(a, b, s), to_slot = slot_of(a, b, j);
      if (s != j && from_slot >= 0 && to_slot >= 0) {
        const lp_cache_part& p = a.part[piece / per_part];
        const int e = int(piece % per_part);
        const bool is_code = e < codes;
        const int64_t page_stride = is_code ? p.code_page_stride : p.param_page_stride;
        const int64_t slot_stride = is_code ? p.code_slot_stride : p.param_slot_stride;
        char* base = static_cast<char*>(is_code ? p.codes : p.params) +
                     h * (is_code ? p.code_head_stride : p.param_head_stride) +
                     (is_code ? int64_t(e) * a.code_unit : int64_t(e - codes) * a.param_unit);
        unit = is_code ? a.code_unit : a.param_unit;
        to = base + place(a, to_slot, page_stride, slot_stride);
        copy_unit(&held, base + place(a, from_slot, page_stride, slot_stride), unit);
      }
    }
    __syncthreads();
    if (to != nullptr) copy_unit(to, &held, unit);
    __syncthreads();
  }
}

cudaError_t launch_cluster(void (*kernel)(EvictArgs), int64_t units, int blocks, int threads,
                           size_t smem, cudaStream_t stream, const EvictArgs& a) {
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = unsigned(blocks);
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(units * blocks));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch(EvictArgs a, cudaStream_t stream) {
  const int64_t units = int64_t(a.batch) * a.heads;
  cudaError_t e;
  if (a.most <= kMostCluster * kHeldTokens && units <= INT32_MAX / kMostCluster) {
    // as many blocks as there is room for on all SMs, and as have 2048 tokens each
    int blocks = (a.most + kHeldTokens - 1) / kHeldTokens;
    blocks = blocks > 4 ? 8 : blocks > 2 ? 4 : blocks > 1 ? 2 : 1;
    while (blocks < kMostCluster && units * blocks * 2 <= 2 * kSms && a.most > 2048 * blocks)
      blocks *= 2;
    a.slice = (a.most + blocks - 1) / blocks;
    const int smem = std::max(1, a.slice) * 4;
    static PerDevice<1> allowed;
    e = allow_shared(evict_slices_kernel, kHeldTokens * 4, allowed);
    if (e == cudaSuccess)
      e = launch_cluster(evict_slices_kernel, units, blocks, kThreads, smem, stream, a);
  } else {
    e = launch_kernel(evict_select_kernel, dim3(unsigned(units)), dim3(kThreads), 0, stream, a);
  }
  if (e != cudaSuccess || a.n_parts == 0 || a.weights == nullptr || a.n_slots == 0 || a.keep == 0)
    return e;
  const int64_t codes = int64_t(a.n_parts) * (a.code_bytes / a.code_unit);
  const int64_t params = int64_t(a.n_parts) * (a.param_bytes / a.param_unit);
  if (codes > kCodeThreads || params > kMoveThreads - kCodeThreads ||
      units > INT32_MAX / kMostCluster)
    return launch_kernel(evict_move_wide_kernel, dim3(unsigned(units)), dim3(kMoveThreads), 0,
                         stream, a);
  const int64_t pieces = codes + params;
  int blocks = 1;
  while (blocks < kMostCluster && units * blocks * 2 <= 8 * kSms && a.keep > 64 * blocks) blocks *= 2;
  // of a block's round, two at once: as much as leaves room for all blocks, four an SM
  const int64_t bytes = units * blocks <= 2 * kSms ? kRoundBytes : 20 * 1024;
  a.round_tokens = int(std::min<int64_t>({kRoundTokens, bytes / (pieces * 16), a.keep}));
  a.round_tokens = std::min(a.round_tokens, (a.keep + blocks - 1) / blocks);
  const size_t smem = size_t(2) * a.round_tokens * pieces * 16;
  static PerDevice<1> allowed;
  e = allow_shared(evict_move_kernel, 2 * kRoundBytes, allowed);
  if (e != cudaSuccess) return e;
  return launch_cluster(evict_move_kernel, units, blocks, kMoveThreads, smem, stream, a);
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
  // pages that follow one another are one
  bool linear = true;
  for (int i = 0; i < a.n_parts; ++i)
    linear = linear && a.part[i].code_page_stride == a.part[i].code_slot_stride * page_size &&
             a.part[i].param_page_stride == a.part[i].param_slot_stride * page_size;
  if (linear) a.page = std::max(page_size, n_slots);
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
  return status_of(launch(a, stream));
}
