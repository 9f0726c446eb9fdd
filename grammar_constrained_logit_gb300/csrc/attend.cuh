// attend.cuh -- what the kernels of attention over the cache share: their arguments, where a
// token's codes lie, and which tokens a row sees.
#pragma once

#include "common.cuh"

namespace lp {

constexpr int kSms = 152;
constexpr int kMostWarps = 16;  // resident on an SM, at most

struct AttendArgs {
  lp_cache_part part[2];  // keys, values
  int64_t n_slots, page;
  int heads, dim, group, bits;
  Div per_page;  // where slots are below 2^31
  lp_rows q, out;  // strides in bytes
  lp_dtype dt;
  int batch, rows, shared;  // shared: query heads to a head of the cache
  const int32_t* blocks;
  int64_t blocks_stride, block;
  int most;        // tokens of a sequence, at most
  Div per_block;
  Div per_group;
  const int32_t* lengths;
  const int32_t* n_rows;
  float scale;     // times log2(e): scores are exponents of two
  int64_t window;  // 0: none
  float* weights;
  int64_t weights_batch, weights_head;
  float* lse;      // [batch, rows, q_heads]: log2 of a row's sum; only with weights
  // of the tensor-core kernels: the work is cut into tiles of tokens, in the order (sequence,
  // tile of rows, tile of tokens).  `workers` workers take a range of them each: one team of
  // warps for every `team` heads, a warp a head
  int team, head_groups, row_tiles, workers;
  bool wide_params;   // 16-byte copies of params
  // a slot's place is slot * stride in both parts, and counted in copied units (codes) and
  // words (params) it is below 2^32: then these are the strides
  uint32_t code_step, param_step;
  float* sums;     // [workers, 2, team, tile's rows, dim]: of what a worker has of a unit
  float2* tops;    // [workers, 2, team, tile's rows]: (largest exponent, mass)
  int4* shares;    // [batch, row tiles]: a unit's first worker and last, whether the first one
                   // has it as its part 1
  float* kept;     // of the kernel of many rows: [blocks, 2, dim, 128]
  bool wide_q, wide_out;  // queries are loaded, results stored, 8 bytes at a time
  bool weights_only;      // the queries' sums are there
};

// What a sequence has: its tokens, and the queries that take part.
struct Sequence {
  int tokens, rows;
};

__device__ __forceinline__ Sequence sequence(const AttendArgs& a, int b) {
  Sequence s;
  s.tokens = min(max(__ldg(a.lengths + b), 0), a.most);
  s.rows = a.n_rows != nullptr ? min(max(__ldg(a.n_rows + b), 0), a.rows) : a.rows;
  return s;
}

// The tokens [lo, end) that row r sees.
struct Seen {
  int lo, end;
};

__device__ __forceinline__ Seen seen(const AttendArgs& a, const Sequence& s, int r) {
  Seen v;
  v.end = r < s.rows ? s.tokens - (s.rows - 1 - r) : 0;
  v.end = max(v.end, 0);
  v.lo = a.window > 0 && a.window < v.end ? v.end - int(a.window) : 0;
  return v;
}

// Token t's slot, or -1.
__device__ __forceinline__ int64_t slot_of(const AttendArgs& a, int b, int t) {
  const uint32_t i = a.per_block.quot(uint32_t(t));
  const int64_t slot = int64_t(__ldg(a.blocks + int64_t(b) * a.blocks_stride + i)) * a.block +
                       (t - int64_t(i) * a.block);
  return slot >= 0 && slot < a.n_slots ? slot : -1;
}

// Where a slot lies, from a part's base.
__device__ __forceinline__ int64_t slot_place(const AttendArgs& a, int64_t slot,
                                              int64_t page_stride, int64_t slot_stride) {
  if (a.page >= a.n_slots) return slot * slot_stride;  // one page
  const int64_t p = a.n_slots <= INT32_MAX ? int64_t(a.per_page.quot(uint32_t(slot)))
                                           : slot / a.page;
  return p * page_stride + (slot - p * a.page) * slot_stride;
}

__device__ __forceinline__ float load_as_float(const char* p, int64_t i, lp_dtype dt) {
  if (dt == LP_F32) return Elt<LP_F32>::load1(p + i * 4);
  return dt == LP_F16 ? Elt<LP_F16>::load1(p + i * 2) : Elt<LP_BF16>::load1(p + i * 2);
}

__device__ __forceinline__ void store_float(char* p, int64_t i, float x, lp_dtype dt) {
  if (dt == LP_F32) {
    *reinterpret_cast<float*>(p + i * 4) = x;
  } else {
    uint16_t h;
    if (dt == LP_BF16) asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
    else asm("cvt.rn.f16.f32 %0, %1;" : "=h"(h) : "f"(x));
    *reinterpret_cast<uint16_t*>(p + i * 2) = h;
  }
}

}  // namespace lp
