// attend.cu -- attention over the quantised cache: the entry point, and the kernels for
// what the tensor-core ones do not take.
//
//   x_rt = scale q_r . k_t,   p = softmax over the tokens that row r sees,   out = sum p_t v_t
//   k, v = code * s  (8 bits),   l + code * s  (4 bits)
//
// One pass over the tokens: with M the largest score so far, sums of 2^(x - M) and of
// 2^(x - M) v are kept, and scaled by 2^(M - M') when M grows to M'.
#include <algorithm>
#include <cmath>

#include "attend.cuh"

namespace lp {

int64_t chunk_kept(int64_t rows, int64_t heads, int64_t batch, int64_t dim);
bool chunk_fits(const AttendArgs& a);
cudaError_t attend_chunk(const AttendArgs& a, cudaStream_t stream);
cudaError_t attend_8n1(const AttendArgs& a, int block, cudaStream_t stream);
cudaError_t attend_8n2(const AttendArgs& a, int block, cudaStream_t stream);
cudaError_t attend_8w1(const AttendArgs& a, int block, cudaStream_t stream);
cudaError_t attend_8w2(const AttendArgs& a, int block, cudaStream_t stream);
cudaError_t attend_4n1(const AttendArgs& a, int block, cudaStream_t stream);
cudaError_t attend_4n2(const AttendArgs& a, int block, cudaStream_t stream);
cudaError_t attend_4w1(const AttendArgs& a, int block, cudaStream_t stream);
cudaError_t attend_4w2(const AttendArgs& a, int block, cudaStream_t stream);

namespace {

constexpr int kWarps = 4;       // of a block of weights_any_kernel
constexpr int kMostAnyWarps = 16;
constexpr int kQueries = 4;     // of a block of attend_any_kernel
constexpr int kGroup = 2;       // tokens that a warp of it has at a time
constexpr int kMostDim = 1024;
constexpr int kAnyBytes = 96 * 1024;  // of shared memory of a block of attend_any_kernel

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

// Elements d0 .. d0 + 127 of kGroup heads, four to a lane; 0 behind the last (whose
// place loads the last again: no load waits for a choice).
template <int BITS>
__device__ __forceinline__ void unpack(const AttendArgs& a, const Head (&from)[kGroup], int d0,
                                       float (&to)[4][kGroup]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int d = d0 + 32 * e + lane;
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      const float x = value_at<BITS>(a, from[u].codes, from[u].params, min(d, a.dim - 1));
      to[e][u] = d < a.dim ? x : 0.0f;
    }
  }
}

// Any width, group, stride and alignment: a block has up to kQueries queries of one head of the
// cache, its warps kGroup tokens in turn, their lanes across the head: what a lane has unpacked
// meets all queries.  The warps' sums are joined at the end.
//   Bound by instructions: a lane has one element at a time, whatever the alignment.  8 x 32
// queries of 72 elements, four to a head, over 4096 tokens of 8 bits: 7893 us with a warp a
// query, 830 with a block a query, 416 so (the heads' codes read once: 6).
template <int BITS>
__global__ void __launch_bounds__(kMostAnyWarps * 32)
    attend_any_kernel(const __grid_constant__ AttendArgs a, const int tiles) {
  extern __shared__ float shared_floats[];
  __shared__ float tops[kMostAnyWarps][kQueries], masses[kMostAnyWarps][kQueries];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q_heads = a.heads * a.shared, per_head = a.rows * a.shared;
  float* q = shared_floats;                     // [kQueries][dim]
  float* sums = shared_floats + kQueries * a.dim;  // [warps][kQueries][dim]
  float* sum = sums + warp * kQueries * a.dim;
  const int64_t total = int64_t(a.batch) * a.heads * tiles;
  for (int64_t unit = blockIdx.x; unit < total; unit += gridDim.x) {
    const int tile = int(unit % tiles), h = int(unit / tiles % a.heads),
              b = int(unit / tiles / a.heads);
    const Sequence s = sequence(a, b);
    Seen v[kQueries];
    int lo = INT32_MAX, end = 0;
#pragma unroll
    for (int i = 0; i < kQueries; ++i) {
      const int row = tile * kQueries + i;
      v[i] = seen(a, s, row < per_head ? row / a.shared : a.rows);
      if (v[i].lo < v[i].end && a.n_slots > 0) lo = min(lo, v[i].lo), end = max(end, v[i].end);
    }
#pragma unroll
    for (int i = 0; i < kQueries; ++i) {
      const int row = tile * kQueries + i, r = row / a.shared;
      const char* from = static_cast<const char*>(a.q.data) + b * a.q.batch_stride +
                         r * a.q.row_stride + (h * a.shared + row - r * a.shared) * a.q.head_stride;
      for (int d = threadIdx.x; d < a.dim; d += blockDim.x)
        q[i * a.dim + d] = row < per_head ? load_as_float(from, d, a.dt) : 0.0f;
      for (int d = lane; d < a.dim; d += 32) sum[i * a.dim + d] = 0.0f;
    }
    __syncthreads();
    float top[kQueries], mass[kQueries];
#pragma unroll
    for (int i = 0; i < kQueries; ++i) top[i] = -INFINITY, mass[i] = 0.0f;
    for (int64_t t64 = int64_t(lo) + warp * kGroup; t64 < end; t64 += warps * kGroup) {
      const int t = int(t64);
      Head key[kGroup], value[kGroup];
      bool there[kGroup];
      float x[kQueries][kGroup];
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        const int64_t slot = t + u < end ? slot_of(a, b, t + u) : -1;
        there[u] = slot >= 0;
        // (where there is none any other is loaded, so that loads do not wait for a choice)
        key[u] = head_at(a, 0, there[u] ? slot : 0, h);
        value[u] = head_at(a, 1, there[u] ? slot : 0, h);
#pragma unroll
        for (int i = 0; i < kQueries; ++i) x[i][u] = 0.0f;
      }
      // 128 elements at once; keys' and values' first ones are under way together
      float k[4][kGroup], y[4][kGroup];
      unpack<BITS>(a, value, 0, y);
      for (int d0 = 0; d0 < a.dim; d0 += 128) {
        unpack<BITS>(a, key, d0, k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = d0 + 32 * e + lane;
#pragma unroll
          for (int i = 0; i < kQueries; ++i) {
            const float qd = d < a.dim ? q[i * a.dim + d] : 0.0f;
#pragma unroll
            for (int u = 0; u < kGroup; ++u) x[i][u] += qd * k[e][u];
          }
        }
      }
      float keep[kQueries];
      uint32_t live = 0;  // who sees what of the kGroup tokens
#pragma unroll
      for (int i = 0; i < kQueries; ++i) {
        float now = top[i];
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
          x[i][u] = warp_sum(x[i][u]) * a.scale;
          if (there[u] && t + u >= v[i].lo && t + u < v[i].end) {
            live |= 1u << (i * kGroup + u);
            now = fmaxf(now, x[i][u]);
          }
        }
        const float ref = now == -INFINITY ? 0.0f : now;
        keep[i] = exp2f(top[i] - ref);
        top[i] = now;
        mass[i] *= keep[i];
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
          x[i][u] = (live >> (i * kGroup + u)) & 1u ? exp2f(x[i][u] - ref) : 0.0f;
          mass[i] += x[i][u];
        }
      }
      for (int d0 = 0; d0 < a.dim; d0 += 128) {
        if (d0 > 0) unpack<BITS>(a, value, d0, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = d0 + 32 * e + lane;
          if (d >= a.dim) continue;
#pragma unroll
          for (int i = 0; i < kQueries; ++i) {
            float z = sum[i * a.dim + d] * keep[i];
#pragma unroll
            for (int u = 0; u < kGroup; ++u)  // (what is not seen may be no number)
              if ((live >> (i * kGroup + u)) & 1u) z += x[i][u] * y[e][u];
            sum[i * a.dim + d] = z;
          }
        }
      }
    }
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < kQueries; ++i) tops[warp][i] = top[i], masses[warp][i] = mass[i];
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < kQueries; ++i) {
      const int row = tile * kQueries + i, r = row / a.shared, j = h * a.shared + row - r * a.shared;
      if (row >= per_head) break;
      float most = -INFINITY, all = 0.0f;
      for (int w = 0; w < warps; ++w) most = fmaxf(most, tops[w][i]);
      const float ref = most == -INFINITY ? 0.0f : most;
      for (int w = 0; w < warps; ++w) all += masses[w][i] * exp2f(tops[w][i] - ref);
      const float inv = all == 0.0f ? 0.0f : 1.0f / all;
      char* to = static_cast<char*>(a.out.data) + b * a.out.batch_stride + r * a.out.row_stride +
                 j * a.out.head_stride;
      for (int d = threadIdx.x; d < a.dim; d += blockDim.x) {
        float y = 0.0f;
        for (int w = 0; w < warps; ++w)
          y += sums[(w * kQueries + i) * a.dim + d] * exp2f(tops[w][i] - ref);
        store_float(to, d, all == 0.0f ? 0.0f : y * inv, a.dt);
      }
      if (a.lse != nullptr && threadIdx.x == 0)
        a.lse[(int64_t(b) * a.rows + r) * q_heads + j] =
            all == 0.0f ? -INFINITY : ref + log2f(all);
    }
    __syncthreads();  // the sums are read
  }
}

// weights[b, h, t] += the sum of 2^(x - lse) over the rows and query heads of h: a warp a
// token and head, its rows one after another.
__global__ void __launch_bounds__(kWarps * 32) weights_any_kernel(const __grid_constant__ AttendArgs a) {
  const int lane = threadIdx.x & 31;
  const int q_heads = a.heads * a.shared;
  const int64_t total = int64_t(a.batch) * a.heads * a.most;
  for (int64_t i = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); i < total;
       i += int64_t(gridDim.x) * kWarps) {
    const int t = int(i % a.most), h = int(i / a.most % a.heads), b = int(i / a.most / a.heads);
    const Sequence s = sequence(a, b);
    if (t >= s.tokens) continue;
    const int64_t slot = slot_of(a, b, t);
    if (slot < 0) continue;
    const Head key = head_at(a, 0, slot, h);
    float sum = 0.0f;
    for (int r = 0; r < s.rows; ++r) {
      const Seen v = seen(a, s, r);
      if (t < v.lo || t >= v.end) continue;
      for (int j = h * a.shared; j < (h + 1) * a.shared; ++j) {
        const char* q = static_cast<const char*>(a.q.data) + b * a.q.batch_stride +
                        r * a.q.row_stride + j * a.q.head_stride;
        float x = 0.0f;
        for (int d = lane; d < a.dim; d += 32)
          x += load_as_float(q, d, a.dt) * value_at(a, key.codes, key.params, d);
        x = warp_sum(x) * a.scale;
        const float lse = a.lse[(int64_t(b) * a.rows + r) * q_heads + j];
        if (lse != -INFINITY) sum += exp2f(x - lse);
      }
    }
    if (lane == 0) {
      float* w = a.weights + b * a.weights_batch + h * a.weights_head + t;
      *w += sum;
    }
  }
}

cudaError_t attend_any(const AttendArgs& a, cudaStream_t stream) {
  const int tiles = (a.rows * a.shared + kQueries - 1) / kQueries;
  const int64_t units = int64_t(a.batch) * a.heads * tiles;
  // as many warps as it holds the sums of
  const int warps = std::min(kMostAnyWarps, kAnyBytes / 4 / a.dim / kQueries - 1);
  const int smem = (warps + 1) * kQueries * a.dim * 4;
  static PerDevice<1> allowed[2];
  void (*kernel)(AttendArgs, int) = a.bits == 8 ? attend_any_kernel<8> : attend_any_kernel<4>;
  cudaError_t e = allow_shared(kernel, kAnyBytes, allowed[a.bits == 8]);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kernel,
                                dim3(unsigned(std::min<int64_t>(units, kSms * 64))),
                                dim3(warps * 32), size_t(smem), stream, a, tiles);
  if (e != cudaSuccess || a.weights == nullptr || a.most == 0) return e;
  const int64_t tokens = int64_t(a.batch) * a.heads * a.most;
  const dim3 all(unsigned(std::min<int64_t>((tokens + kWarps - 1) / kWarps, kSms * 64)));
  return launch_kernel(weights_any_kernel, all, dim3(kWarps * 32), 0, stream, a);
}

// The tensor-core kernels: of the cache's bits, with queries and weights in one piece or two.
using Launch = cudaError_t (*)(const AttendArgs&, int, cudaStream_t);

// The blocks that groups are made of, for the widths that there are kernels for; 0: none.
int block_of(int dim, int group) {
  for (int most : {dim == 128 || dim == 256 ? 128 : dim == 64 || dim == 192 ? 64 : 32, 32, 16}) {
    if (dim != 64 && dim != 80 && dim != 96 && dim != 128 && dim != 192 && dim != 256) return 0;
    if (dim % most == 0 && group % most == 0) return most;
  }
  return 0;
}

bool aligned(const AttendArgs& a, int unit, bool params) {
  uint64_t x = 0;
  for (const lp_cache_part& p : a.part)
    x |= params ? reinterpret_cast<uintptr_t>(p.params) | uint64_t(p.param_page_stride) |
                      uint64_t(p.param_slot_stride) | uint64_t(p.param_head_stride)
                : reinterpret_cast<uintptr_t>(p.codes) | uint64_t(p.code_page_stride) |
                      uint64_t(p.code_slot_stride) | uint64_t(p.code_head_stride);
  return x % unit == 0;
}

// Columns of the products that a head's queries fill.  20 queries over 8192 tokens of 32
// sequences take 206 us in sixteens and 288 in eights, which go through the tokens more often;
// 15 over 1024, with little to go through, 33 and 30.
int rows_at_once(int64_t rows) { return rows <= 8 ? 8 : 16; }

bool fits(int64_t a, int64_t b, int64_t most) { return b == 0 || a <= most / b; }

}  // namespace
}  // namespace lp

extern "C" int64_t lp_cache_attend_workspace_bytes(int64_t batch, int64_t rows, int64_t q_heads,
                                                   int64_t heads, int64_t dim) {
  using namespace lp;
  if (batch < 0 || rows < 0 || q_heads < 0 || heads < 0 || dim < 0 || dim > kMostDim ||
      !fits(rows, q_heads, 1 << 24) || !fits(batch, rows * q_heads, INT32_MAX))
    return -1;
  // of each row its sum; who shares a unit; what the workers leave of the shared ones; and what
  // blocks of many rows keep
  const int64_t per_head = heads == 0 ? 0 : rows * (q_heads / heads);
  const int64_t left = int64_t(kSms) * kMostWarps * 2 * rows_at_once(per_head) * (dim * 4 + 8);
  return (batch * rows * q_heads * 4 + 15) / 16 * 16 + batch * ((per_head + 7) / 8) * 16 +
         (left + 15) / 16 * 16 + chunk_kept(per_head, heads, batch, dim) * 4;
}

extern "C" lp_status lp_cache_attend(const lp_cache_part* parts, int32_t bits, int64_t n_slots,
                                     int64_t page_size, int64_t heads, int64_t dim, int64_t group,
                                     const lp_rows* q, const lp_rows* out, lp_dtype dt,
                                     int64_t batch, int64_t rows, int64_t q_heads,
                                     const int32_t* blocks, int64_t blocks_stride,
                                     int64_t max_blocks, int64_t block_size,
                                     const int32_t* lengths, const int32_t* n_rows, float scale,
                                     int64_t window, float* weights, int64_t weights_batch_stride,
                                     int64_t weights_head_stride, void* workspace,
                                     int64_t workspace_bytes, cudaStream_t stream) {
  using namespace lp;
  if (dt != LP_F32 && dt != LP_F16 && dt != LP_BF16) return LP_ERR_UNSUPPORTED_DTYPE;
  if ((bits != 8 && bits != 4) || n_slots < 0 || page_size < 1 || heads < 0 || dim < 0 ||
      group < 1 || dim % group != 0 || (bits == 4 && group % 2 != 0) || batch < 0 || rows < 0 ||
      q_heads < 0 || (heads == 0 ? q_heads != 0 : q_heads % heads != 0) || max_blocks < 0 ||
      block_size < 1 || blocks_stride < max_blocks || window < 0 || !std::isfinite(scale))
    return LP_ERR_INVALID_ARGUMENT;
  if (dim > kMostDim || !fits(block_size, max_blocks, 1 << 30) ||
      !fits(rows, q_heads, 1 << 24) || !fits(batch, rows * q_heads, INT32_MAX) ||
      batch > INT32_MAX)
    return LP_ERR_TOO_LARGE;
  if (batch == 0 || rows == 0 || q_heads == 0 || dim == 0) return LP_OK;
  const int eb = dt == LP_F32 ? 4 : 2;
  if (parts == nullptr || q == nullptr || out == nullptr || q->data == nullptr ||
      out->data == nullptr || out->data == q->data || lengths == nullptr || (max_blocks > 0 && blocks == nullptr) ||
      (reinterpret_cast<uintptr_t>(q->data) | reinterpret_cast<uintptr_t>(out->data)) % eb != 0 ||
      (reinterpret_cast<uintptr_t>(blocks) | reinterpret_cast<uintptr_t>(lengths) |
       reinterpret_cast<uintptr_t>(n_rows) | reinterpret_cast<uintptr_t>(weights)) % 4 != 0)
    return LP_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < 2; ++i) {
    const lp_cache_part& p = parts[i];
    if (n_slots > 0 && (p.codes == nullptr || p.params == nullptr)) return LP_ERR_INVALID_ARGUMENT;
    if ((reinterpret_cast<uintptr_t>(p.params) | uint64_t(p.param_page_stride) |
         uint64_t(p.param_slot_stride) | uint64_t(p.param_head_stride)) % 4 != 0)
      return LP_ERR_INVALID_ARGUMENT;
  }
  const int64_t need = lp_cache_attend_workspace_bytes(batch, rows, q_heads, heads, dim);
  if (workspace == nullptr || workspace_bytes < need ||
      reinterpret_cast<uintptr_t>(workspace) % 16 != 0)
    return LP_ERR_INVALID_ARGUMENT;
  AttendArgs a = {};
  a.part[0] = parts[0], a.part[1] = parts[1];
  a.n_slots = n_slots;
  a.page = page_size;
  if (page_size < n_slots && n_slots <= INT32_MAX) a.per_page.set(uint32_t(page_size));
  a.heads = int(heads), a.dim = int(dim), a.group = int(group), a.bits = bits;
  a.q = *q, a.out = *out;
  for (lp_rows* r : {&a.q, &a.out}) r->batch_stride *= eb, r->row_stride *= eb, r->head_stride *= eb;
  a.dt = dt;
  a.batch = int(batch), a.rows = int(rows), a.shared = int(q_heads / heads);
  a.blocks = blocks;
  a.blocks_stride = blocks_stride;
  a.block = block_size;
  a.most = int(max_blocks * block_size);
  a.per_block.set(uint32_t(std::min<int64_t>(block_size, INT32_MAX)));
  a.lengths = lengths;
  a.n_rows = n_rows;
  a.per_group.set(uint32_t(group));
  a.scale = float(double(scale) * 1.4426950408889634);
  a.window = window;
  a.weights = weights;
  a.weights_batch = weights_batch_stride;
  a.weights_head = weights_head_stride;
  a.lse = weights != nullptr ? static_cast<float*>(workspace) : nullptr;
  const int block = block_of(a.dim, a.group);
  const int row = a.dim * bits / 8;
  if (block == 0 || n_slots == 0 || !aligned(a, row % 16 == 0 ? 16 : 8, false))
    return status_of(attend_any(a, stream));
  a.wide_params = a.dim / a.group % 4 == 0 && aligned(a, 16, true);
  {
    const lp_cache_part &k = parts[0], &v = parts[1];
    const bool one_page = page_size >= n_slots;
    const int64_t unit = row % 16 == 0 ? 16 : 8;
    const auto alike = [&](int64_t s, int64_t t, int64_t sp, int64_t tp, int64_t size) {
      return s == t && s > 0 && (one_page || (sp == tp && sp == s * page_size)) &&
             s / size <= INT64_MAX / n_slots && s / size * n_slots <= UINT32_MAX;
    };
    if (alike(k.code_slot_stride, v.code_slot_stride, k.code_page_stride, v.code_page_stride, unit) &&
        alike(k.param_slot_stride, v.param_slot_stride, k.param_page_stride, v.param_page_stride, 4)) {
      a.code_step = uint32_t(k.code_slot_stride / unit);
      a.param_step = uint32_t(k.param_slot_stride / 4);
    }
  }
  // heads side by side read a token's codes, which lie side by side, and its table together
  a.team = 4;
  while (a.heads % a.team != 0) --a.team;
  a.head_groups = a.heads / a.team;
  const int at_once = rows_at_once(int64_t(a.rows) * a.shared);
  char* left = static_cast<char*>(workspace) + (batch * rows * q_heads * 4 + 15) / 16 * 16;
  a.shares = reinterpret_cast<int4*>(left);
  left += batch * ((rows * (q_heads / heads) + 7) / 8) * 16;
  const int64_t held = int64_t(kSms) * kMostWarps * 2 * at_once;
  a.wide_q = (reinterpret_cast<uintptr_t>(q->data) | uint64_t(a.q.batch_stride) |
              uint64_t(a.q.row_stride) | uint64_t(a.q.head_stride)) % 8 == 0;
  a.sums = reinterpret_cast<float*>(left);
  a.tops = reinterpret_cast<float2*>(left + held * a.dim * 4);
  a.kept = reinterpret_cast<float*>(left + held * (a.dim * 4 + 8));  // (a multiple of 16)
  static const Launch launches[2][2][2] = {{{attend_8n1, attend_8n2}, {attend_8w1, attend_8w2}},
                                           {{attend_4n1, attend_4n2}, {attend_4w1, attend_4w2}}};
  a.wide_out = (reinterpret_cast<uintptr_t>(out->data) | uint64_t(a.out.batch_stride) |
                uint64_t(a.out.row_stride) | uint64_t(a.out.head_stride)) % 8 == 0;
  if (chunk_fits(a)) {
    const cudaError_t e = attend_chunk(a, stream);
    if (e != cudaSuccess || weights == nullptr) return status_of(e);
    a.weights_only = true;
  }
  return status_of(launches[bits == 4][dt != LP_BF16][at_once == 16](a, block, stream));
}
