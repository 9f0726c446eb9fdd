// reorder.cu -- the states of a beam search follow their beams, in place, many
// tensors in one launch:
//
//   state[.., b*K + k, ..] = old state[.., b*K + parents[b, k], ..]
//
// A thread owns one column (16 bytes at one place of the row) of all K rows of a batch
// entry: it reads the distinct rows that others take, then writes the rows that change,
// so no second buffer and no barrier is needed, a row that keeps its place is not
// written, and one that nobody else takes is not read.  What bounds it is memory:
// (distinct sources + rows that change) x the row's bytes.
#include <algorithm>

#include "common.cuh"

namespace lp {
namespace {

constexpr int kMaxBeams = 256;
constexpr int kLaunchStates = 64;  // states of one launch (its parameters: 5 KB)
constexpr int kSegBytes = 32768;   // of a row, a block

struct State {
  char* data;
  int64_t row_stride, run, token;   // bytes; token: 0: none, -1: outer[0] is the tokens' axis
  int64_t outer_stride[3];          // bytes
  int outer[3];
  int width;                        // bytes of an access: the alignment of base and strides
};

struct ReorderArgs {
  State st[kLaunchStates];
  unsigned first[kLaunchStates + 1];  // first block of each state
  int n;
  int64_t batch;
  int beams;
  const int32_t* parents;
  const int32_t* start;
  const int32_t* stop;
};

template <int W> struct Word;
template <> struct Word<16> { using T = uint4; };
template <> struct Word<8> { using T = uint2; };
template <> struct Word<4> { using T = uint32_t; };
template <> struct Word<2> { using T = uint16_t; };
template <> struct Word<1> { using T = uint8_t; };

struct Plan {                   // of one batch entry
  uint8_t source[kMaxBeams];    // the distinct rows to read
  uint8_t dest[kMaxBeams];      // the rows to write, and what each takes
  uint8_t slot[kMaxBeams];
  int sources, dests;
};

// Bytes [lo, hi) of the rows at p, W at a time; room: one 16-byte slot a thread and source.
template <int W>
__device__ void move_columns(char* p, int64_t row_stride, int64_t lo, int64_t hi, const Plan& plan,
                             uint4* room) {
  using T = typename Word<W>::T;
  for (int64_t at = lo + int64_t(threadIdx.x) * W; at < hi; at += int64_t(blockDim.x) * W) {
    for (int i = 0; i < plan.sources; ++i)
      *reinterpret_cast<T*>(room + i * blockDim.x + threadIdx.x) =
          *reinterpret_cast<const T*>(p + plan.source[i] * row_stride + at);
    for (int i = 0; i < plan.dests; ++i)
      *reinterpret_cast<T*>(p + plan.dest[i] * row_stride + at) =
          *reinterpret_cast<const T*>(room + plan.slot[i] * blockDim.x + threadIdx.x);
  }
}

__global__ void reorder_kernel(const __grid_constant__ ReorderArgs a) {
  extern __shared__ __align__(16) char raw[];
  uint4* room = reinterpret_cast<uint4*>(raw);
  __shared__ Plan plan;
  __shared__ uint32_t taken[kMaxBeams / 32], moved[kMaxBeams / 32];

  int s = 0;
  while (blockIdx.x >= a.first[s + 1]) ++s;
  const State& st = a.st[s];
  unsigned id = blockIdx.x - a.first[s];
  const unsigned segs = unsigned((st.run + kSegBytes - 1) / kSegBytes);
  const int64_t seg = id % segs;
  id /= segs;
  const int64_t b = id % unsigned(a.batch);
  id /= unsigned(a.batch);
  char* p = st.data + b * a.beams * st.row_stride;
  int64_t at0 = 0;  // place on the first outer axis
#pragma unroll
  for (int d = 2; d >= 0; --d) {
    at0 = int64_t(id % unsigned(st.outer[d]));
    p += at0 * st.outer_stride[d];
    id /= unsigned(st.outer[d]);
  }

  // the bytes of this block: its segment within the batch entry's range
  int64_t lo = 0, hi = st.run;
  if (st.token > 0) {
    const int64_t tokens = st.run / st.token;
    if (a.start) lo = min(max(int64_t(a.start[b]), int64_t(0)), tokens) * st.token;
    if (a.stop) hi = min(max(int64_t(a.stop[b]), int64_t(0)), tokens) * st.token;
  } else if (st.token < 0) {
    if ((a.start && at0 < a.start[b]) || (a.stop && at0 >= a.stop[b])) return;
  }
  lo = max(lo, seg * kSegBytes);
  hi = min(hi, (seg + 1) * kSegBytes);
  if (lo >= hi) return;

  // which rows are read, which are written
  if (threadIdx.x < kMaxBeams / 32) taken[threadIdx.x] = 0;
  __syncthreads();
  const int32_t* parents = a.parents + b * a.beams;
  for (int k0 = 0; k0 < a.beams; k0 += blockDim.x) {
    const int k = k0 + threadIdx.x;
    const int from = k < a.beams ? parents[k] : -1;
    const bool moves = from >= 0 && from < a.beams && from != k;
    const uint32_t all = __ballot_sync(kFullWarp, moves);
    if (k < kMaxBeams && (k & 31) == 0) moved[k >> 5] = all;
    if (moves) atomicOr(&taken[from >> 5], 1u << (from & 31));
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int n_src = 0, n_dst = 0;
    for (int w = 0; w * 32 < a.beams; ++w) {
      const uint32_t below = (1u << threadIdx.x) - 1u;
      if (taken[w] >> threadIdx.x & 1u)
        plan.source[n_src + __popc(taken[w] & below)] = uint8_t(w * 32 + threadIdx.x);
      if (moved[w] >> threadIdx.x & 1u) {
        const int k = w * 32 + threadIdx.x, from = parents[k];
        int slot = __popc(taken[from >> 5] & ((1u << (from & 31)) - 1u));
        for (int u = 0; u < (from >> 5); ++u) slot += __popc(taken[u]);
        const int at = n_dst + __popc(moved[w] & below);
        plan.dest[at] = uint8_t(k);
        plan.slot[at] = uint8_t(slot);
      }
      n_src += __popc(taken[w]);
      n_dst += __popc(moved[w]);
    }
    if (threadIdx.x == 0) plan.sources = n_src, plan.dests = n_dst;
  }
  __syncthreads();
  if (plan.dests == 0) return;

  switch (st.width) {
    case 16: {
      // the range may begin and end inside a 16-byte word: those bytes one by one
      const int64_t up = (lo + 15) & ~int64_t(15), down = hi & ~int64_t(15);
      if (up >= down) {
        move_columns<1>(p, st.row_stride, lo, hi, plan, room);
      } else {
        move_columns<16>(p, st.row_stride, up, down, plan, room);
        move_columns<1>(p, st.row_stride, lo, up, plan, room);
        move_columns<1>(p, st.row_stride, down, hi, plan, room);
      }
      break;
    }
    case 8: move_columns<8>(p, st.row_stride, lo, hi, plan, room); break;
    case 4: move_columns<4>(p, st.row_stride, lo, hi, plan, room); break;
    case 2: move_columns<2>(p, st.row_stride, lo, hi, plan, room); break;
    default: move_columns<1>(p, st.row_stride, lo, hi, plan, room); break;
  }
}

}  // namespace
}  // namespace lp

extern "C" lp_status lp_reorder_states(const lp_state* states, int64_t n_states, int64_t batch,
                                       int64_t beams, const int32_t* parents, const int32_t* start,
                                       const int32_t* stop, cudaStream_t stream) {
  using namespace lp;
  if (n_states < 0 || batch < 0 || beams < 1 || (n_states > 0 && states == nullptr))
    return LP_ERR_INVALID_ARGUMENT;
  if (beams > kMaxBeams || batch > (int64_t(1) << 27) / beams) return LP_ERR_TOO_LARGE;
  for (int64_t i = 0; i < n_states; ++i) {
    const lp_state& s = states[i];
    if (s.run_bytes < 0 || s.token_bytes < -1 || s.outer[0] < 0 || s.outer[1] < 0 ||
        s.outer[2] < 0 || (s.token_bytes > 0 && s.run_bytes % s.token_bytes != 0))
      return LP_ERR_INVALID_ARGUMENT;
    const bool some = batch > 0 && s.run_bytes > 0 && s.outer[0] > 0 && s.outer[1] > 0 &&
                      s.outer[2] > 0;
    if (some && (s.data == nullptr || (s.row_stride < s.run_bytes && s.row_stride > -s.run_bytes &&
                                       batch * beams > 1)))
      return LP_ERR_INVALID_ARGUMENT;
    if (s.outer[0] > INT32_MAX || s.outer[1] > INT32_MAX || s.outer[2] > INT32_MAX)
      return LP_ERR_TOO_LARGE;
  }
  if (batch > 0 && n_states > 0 && parents == nullptr) return LP_ERR_INVALID_ARGUMENT;

  // what all blocks need: as many blocks as the largest launches allow, checked first
  auto blocks_of = [&](const lp_state& s) -> int64_t {
    const int64_t segs = s.run_bytes / kSegBytes + (s.run_bytes % kSegBytes != 0);
    int64_t n = batch;
    for (int64_t f : {segs, s.outer[0], s.outer[1], s.outer[2]}) {
      if (f == 0) return 0;
      if (n > INT32_MAX / f) return -1;
      n *= f;
    }
    return n;
  };
  for (int64_t i = 0; i < n_states; ++i)
    if (blocks_of(states[i]) < 0) return LP_ERR_TOO_LARGE;

  const int threads = int(std::max<int64_t>(32, std::min<int64_t>(256, (98304 / 16 / beams) & ~31)));
  const size_t smem = size_t(threads) * 16 * size_t(beams);
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(reorder_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kMaxBeams * 32 * 16) != cudaSuccess)
    return LP_ERR_CUDA;
  ReorderArgs a = {};
  a.batch = batch;
  a.beams = int(beams);
  a.parents = parents;
  a.start = start;
  a.stop = stop;
  for (int64_t i = 0; i < n_states;) {
    a.n = 0;
    for (; i < n_states && a.n < kLaunchStates; ++i) {
      const lp_state& s = states[i];
      const int64_t n = blocks_of(s);
      if (n == 0) continue;
      if (a.n > 0 && int64_t(a.first[a.n]) + n > INT32_MAX) break;
      State& t = a.st[a.n];
      t.data = static_cast<char*>(s.data);
      t.row_stride = s.row_stride;
      t.run = s.run_bytes;
      t.token = s.token_bytes;
      uint64_t bits = reinterpret_cast<uint64_t>(s.data) | uint64_t(s.row_stride) | 16;
      for (int d = 0; d < 3; ++d) {
        t.outer[d] = int(s.outer[d]);
        t.outer_stride[d] = s.outer_stride[d];
        if (s.outer[d] > 1) bits |= uint64_t(s.outer_stride[d]);
      }
      // 16-byte words can begin and end a range anywhere; narrower ones are whole in it
      if (bits % 16 != 0) bits |= uint64_t(s.run_bytes) | uint64_t(std::max<int64_t>(0, s.token_bytes));
      t.width = int(bits & (~bits + 1));
      a.first[a.n + 1] = a.first[a.n] + unsigned(n);
      ++a.n;
    }
    if (a.n == 0) break;
    reorder_kernel<<<a.first[a.n], threads, smem, stream>>>(a);
    if (cudaPeekAtLastError() != cudaSuccess) return LP_ERR_CUDA;
  }
  return LP_OK;
}
