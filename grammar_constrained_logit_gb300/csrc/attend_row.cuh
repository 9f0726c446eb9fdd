// attend_row.cuh -- one query's attention by one warp, its lanes across the head: of any width,
// group, stride and alignment.
#pragma once

#include "attend.cuh"

namespace lp {

// The value of element d of a head's codes.
template <int BITS>
__device__ __forceinline__ float value_at(const AttendArgs& a, const uint8_t* codes,
                                          const char* params, int d) {
  const uint32_t held = *reinterpret_cast<const uint32_t*>(params + a.per_group.quot(uint32_t(d)) * 4);
  if (BITS == 8) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(codes[d])));
    return __fmul_rn(Elt<LP_F16>::half_bits_to_float(h & 0xffffu), __uint_as_float(held));
  }
  const uint32_t code = (codes[d >> 1] >> (4 * (d & 1))) & 15u;
  return __fmaf_rn(float(code), __uint_as_float(held << 16), __uint_as_float(held & 0xffff0000u));
}

__device__ __forceinline__ float value_at(const AttendArgs& a, const uint8_t* codes,
                                          const char* params, int d) {
  return a.bits == 8 ? value_at<8>(a, codes, params, d) : value_at<4>(a, codes, params, d);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(kFullWarp, x, o);
  return x;
}

struct Head {  // of one part, at one slot
  const uint8_t* codes;
  const char* params;
};

__device__ __forceinline__ Head head_at(const AttendArgs& a, int part, int64_t slot, int h) {
  const lp_cache_part& p = a.part[part];
  Head r;
  r.codes = static_cast<const uint8_t*>(p.codes) +
            slot_place(a, slot, p.code_page_stride, p.code_slot_stride) + h * p.code_head_stride;
  r.params = static_cast<const char*>(p.params) +
             slot_place(a, slot, p.param_page_stride, p.param_slot_stride) +
             h * p.param_head_stride;
  return r;
}

// q and sum: the warp's own, dim floats each.
__device__ __forceinline__ void attend_row(const AttendArgs& a, int b, int r, int j, float* q,
                                           float* sum) {
  const int lane = threadIdx.x & 31;
  const int h = j / a.shared;
  const Sequence s = sequence(a, b);
  const Seen v = seen(a, s, r);
  const char* from = static_cast<const char*>(a.q.data) + b * a.q.batch_stride +
                     r * a.q.row_stride + j * a.q.head_stride;
  char* to = static_cast<char*>(a.out.data) + b * a.out.batch_stride + r * a.out.row_stride +
             j * a.out.head_stride;
  for (int d = lane; d < a.dim; d += 32) q[d] = load_as_float(from, d, a.dt), sum[d] = 0.0f;
  float top = -INFINITY, mass = 0.0f;
  for (int t = v.lo; t < v.end; ++t) {
    const int64_t slot = slot_of(a, b, t);
    if (slot < 0) continue;
    const Head key = head_at(a, 0, slot, h);
    float x = 0.0f;
    for (int d = lane; d < a.dim; d += 32) x += q[d] * value_at(a, key.codes, key.params, d);
    x = warp_sum(x) * a.scale;
    const float now = fmaxf(top, x);
    const float ref = now == -INFINITY ? 0.0f : now;
    const float keep = exp2f(top - ref), e = exp2f(x - ref);
    top = now;
    mass = mass * keep + e;
    const Head value = head_at(a, 1, slot, h);
    for (int d = lane; d < a.dim; d += 32)
      sum[d] = sum[d] * keep + e * value_at(a, value.codes, value.params, d);
  }
  const float inv = mass == 0.0f ? 0.0f : 1.0f / mass;
  for (int d = lane; d < a.dim; d += 32)
    store_float(to, d, mass == 0.0f ? 0.0f : sum[d] * inv, a.dt);
  if (a.lse != nullptr && lane == 0)
    a.lse[(int64_t(b) * a.rows + r) * (a.heads * a.shared) + j] = mass == 0.0f ? -INFINITY : top + log2f(mass);
}

}  // namespace lp
