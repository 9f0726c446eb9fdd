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
#include "attend_row.cuh"

namespace lp {

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
constexpr int kGroup = 4;       // tokens that a warp of attend_any_kernel has at a time
constexpr int kMostDim = 1024;

// Any width, group, stride and alignment: a block a query, its warps with kGroup
// tokens in turn, whose trips to memory run side by side, their lanes
// across the head; the warps' sums are joined at the end.
//   What a lane loads is one byte, so it is the trips that bound it: 8 x 32 queries of 72
// elements over 4096 tokens took 7893 us with a warp a query and a token at a time.
__global__ void __launch_bounds__(kMostAnyWarps * 32)
    attend_any_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ float shared_floats[];
  __shared__ float tops[kMostAnyWarps], masses[kMostAnyWarps];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* q = shared_floats;
  float* sums = shared_floats + a.dim;
  float* sum = sums + warp * a.dim;
  const int q_heads = a.heads * a.shared;
  const int64_t total = int64_t(a.batch) * a.rows * q_heads;
  for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
    const int j = int(i % q_heads), r = int(i / q_heads % a.rows), b = int(i / q_heads / a.rows);
    const int h = j / a.shared;
    const Seen v = seen(a, sequence(a, b), r);
    const char* from = static_cast<const char*>(a.q.data) + b * a.q.batch_stride +
                       r * a.q.row_stride + j * a.q.head_stride;
    for (int d = threadIdx.x; d < a.dim; d += blockDim.x) q[d] = load_as_float(from, d, a.dt);
    for (int d = lane; d < a.dim; d += 32) sum[d] = 0.0f;
    __syncthreads();
    float top = -INFINITY, mass = 0.0f;
    for (int t = v.lo + warp * kGroup; t < v.end; t += warps * kGroup) {
      Head key[kGroup], value[kGroup];
      bool there[kGroup];
      float x[kGroup];
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        const int64_t slot = t + u < v.end ? slot_of(a, b, t + u) : -1;
        there[u] = slot >= 0;
        x[u] = 0.0f;
        if (there[u]) key[u] = head_at(a, 0, slot, h), value[u] = head_at(a, 1, slot, h);
      }
      for (int d = lane; d < a.dim; d += 32) {
        const float qd = q[d];
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
          if (there[u]) x[u] += qd * value_at(a, key[u].codes, key[u].params, d);
      }
      float now = top;
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        x[u] = warp_sum(x[u]) * a.scale;
        if (there[u]) now = fmaxf(now, x[u]);
      }
      const float ref = now == -INFINITY ? 0.0f : now;
      const float keep = exp2f(top - ref);
      top = now;
      mass *= keep;
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        x[u] = there[u] ? exp2f(x[u] - ref) : 0.0f;
        mass += x[u];
      }
      for (int d = lane; d < a.dim; d += 32) {
        float y = sum[d] * keep;
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
          if (there[u]) y += x[u] * value_at(a, value[u].codes, value[u].params, d);
        sum[d] = y;
      }
    }
    if (lane == 0) tops[warp] = top, masses[warp] = mass;
    __syncthreads();
    float most = -INFINITY, all = 0.0f;
    for (int w = 0; w < warps; ++w) most = fmaxf(most, tops[w]);
    const float ref = most == -INFINITY ? 0.0f : most;
    for (int w = 0; w < warps; ++w) all += masses[w] * exp2f(tops[w] - ref);
    const float inv = all == 0.0f ? 0.0f : 1.0f / all;
    char* to = static_cast<char*>(a.out.data) + b * a.out.batch_stride + r * a.out.row_stride +
               j * a.out.head_stride;
    for (int d = threadIdx.x; d < a.dim; d += blockDim.x) {
      float y = 0.0f;
      for (int w = 0; w < warps; ++w) y += sums[w * a.dim + d] * exp2f(tops[w] - ref);
      store_float(to, d, all == 0.0f ? 0.0f : y * inv, a.dt);
    }
    if (a.lse != nullptr && threadIdx.x == 0)
      a.lse[(int64_t(b) * a.rows + r) * q_heads + j] = all == 0.0f ? -INFINITY : ref + log2f(all);
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
  const int64_t queries = int64_t(a.batch) * a.rows * a.heads * a.shared;
  const int warps = a.dim <= 512 ? kMostAnyWarps : kMostAnyWarps / 2;  // 48 KB hold their sums
  cudaError_t e = launch_kernel(attend_any_kernel,
                                dim3(unsigned(std::min<int64_t>(queries, kSms * 64))),
                                dim3(warps * 32), size_t(warps + 1) * a.dim * 4, stream, a);
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
  // of each row its sum; who shares a unit; and what the workers leave of the shared ones
  const int64_t per_head = heads == 0 ? 0 : rows * (q_heads / heads);
  const int64_t left = int64_t(kSms) * kMostWarps * 2 * rows_at_once(per_head) * (dim * 4 + 8);
  return (batch * rows * q_heads * 4 + 15) / 16 * 16 + batch * ((per_head + 7) / 8) * 16 +
         (left + 15) / 16 * 16;
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
  a.team = 4;
  while (a.heads % a.team != 0) --a.team;
  a.head_groups = a.heads / a.team;
  a.min_tiles = 2;
  const int at_once = rows_at_once(int64_t(a.rows) * a.shared);
  char* left = static_cast<char*>(workspace) + (batch * rows * q_heads * 4 + 15) / 16 * 16;
  a.shares = reinterpret_cast<int4*>(left);
  left += batch * ((rows * (q_heads / heads) + 7) / 8) * 16;
  const int64_t held = int64_t(kSms) * kMostWarps * 2 * at_once;
  a.wide_q = (reinterpret_cast<uintptr_t>(q->data) | uint64_t(a.q.batch_stride) |
              uint64_t(a.q.row_stride) | uint64_t(a.q.head_stride)) % 8 == 0;
  a.sums = reinterpret_cast<float*>(left);
  a.tops = reinterpret_cast<float2*>(left + held * a.dim * 4);
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
