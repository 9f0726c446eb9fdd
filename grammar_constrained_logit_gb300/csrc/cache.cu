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
// costs range at the group's ends (2^-9 of lo), not accuracy between; bf16 rather than
// fp16 because no input overflows it.
#include <algorithm>

#include "common.cuh"

namespace lp {
namespace {

constexpr int kMaxParts = 8;
constexpr int kThreads = 256;
constexpr float kLargest = 3.3895313892515355e38f;
constexpr float kTiny = 1.1754943508222875e-38f;  // 2^-126

struct CacheArgs {
  lp_cache_part part[kMaxParts];
  lp_heads x[kMaxParts];
  const int64_t* slots;
  int64_t n, n_slots, page;
  int heads, dim, group;
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
  return __float2uint_rn(fminf(fmaxf(y, 0.0f), 15.0f));  // NaN: 0
}

// Where a slot's head lies, from a part's base.
__device__ __forceinline__ int64_t place(int64_t slot, int64_t page, int64_t page_stride,
                                         int64_t slot_stride, int64_t head, int64_t head_stride) {
  const int64_t p = slot / page;
  return p * page_stride + (slot - p * page) * slot_stride + head * head_stride;
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
                     place(slot, a.page, part.code_page_stride, part.code_slot_stride, h,
                           part.code_head_stride) + int64_t(g) * a.group * BITS / 8;
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
                                   place(slot, a.page, part.param_page_stride,
                                         part.param_slot_stride, h, part.param_head_stride) +
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
                              place(slot, a.page, part.code_page_stride, part.code_slot_stride, h,
                                    part.code_head_stride) + c);
      const uint32_t held = *reinterpret_cast<const uint32_t*>(
          static_cast<const char*>(part.params) +
          place(slot, a.page, part.param_page_stride, part.param_slot_stride, h,
                part.param_head_stride) + int64_t(c * E / a.group) * 4);
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

template <int DT, int BITS>
cudaError_t launch(const CacheArgs& a, bool write, int n_parts, cudaStream_t stream) {
  if (write) {
    const int64_t warps = a.n * a.heads * (a.dim / a.group);
    const dim3 grid(unsigned(std::min<int64_t>((warps + 7) / 8, 152 * 64)), unsigned(n_parts));
    cache_write_kernel<DT, BITS><<<grid, kThreads, 0, stream>>>(a);
  } else {
    const int64_t threads = a.n * a.heads * (int64_t(a.dim) * BITS / 8);
    const dim3 grid(unsigned(std::min<int64_t>((threads + kThreads - 1) / kThreads, 152 * 64)),
                    unsigned(n_parts));
    cache_read_kernel<DT, BITS><<<grid, kThreads, 0, stream>>>(a);
  }
  return cudaPeekAtLastError();
}

lp_status run(const lp_cache_part* parts, const lp_heads* x, int64_t n_parts, int bits,
              lp_dtype dt, int64_t n_slots, int64_t page_size, int64_t heads, int64_t dim,
              int64_t group, const int64_t* slots, int64_t n, bool write, cudaStream_t stream) {
  if (dt != LP_F32 && dt != LP_F16 && dt != LP_BF16) return LP_ERR_UNSUPPORTED_DTYPE;
  if (n_parts < 0 || n_parts > kMaxParts || (bits != 8 && bits != 4) || n_slots < 0 ||
      page_size < 1 || heads < 0 || dim < 0 || group < 1 || dim % group != 0 ||
      (bits == 4 && group % 2 != 0) || n < 0)
    return LP_ERR_INVALID_ARGUMENT;
  if (heads > INT32_MAX || dim > INT32_MAX) return LP_ERR_TOO_LARGE;
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
  return e == cudaSuccess ? LP_OK : LP_ERR_CUDA;
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
