// reorder.cu -- the states of a beam search follow their beams, in place, many
// tensors in one launch:
//
//   state[.., b*K + k, ..] = old state[.., b*K + parents[b, k], ..]
//
// A thread owns columns (16 bytes at one place of the row) of all K rows of a batch entry:
// it reads the distinct rows that others take, then writes the rows that change, so no
// second buffer and no barrier is needed, a row that keeps its place is not written, and
// one that nobody else takes is not read.  What bounds it is memory: (distinct sources +
// rows that change) x the row's bytes.  32 x 4 rows of an 8-bit cache of 8 layers, 2.05 GB
// read and written, take 303 us: 6.8 TB/s, the measured copy rate; copies through a second
// buffer of the same rows would move half as much again.
//
// More than 8 distinct sources, or more than 32 beams, go through shared memory, a word at a
// time: rows of 512 tokens of 2 layers of 8 x 128 bf16 run at 82% of that rate with 8 x 32 of
// them (and with 16 x 16, where requests are of both kinds), at 56% with 4 x 64.  Tokens that
// lie apart are a block each, which finds out what moves again: 512 tokens of 64 rows in runs
// of 2 KB take 88 us, their bytes 25.
#include <algorithm>

#include "common.cuh"

namespace lp {
namespace {

constexpr int kMaxBeams = 256;
constexpr int kLaunchStates = 64;  // states of one launch (its parameters: 6 KB)
constexpr int kThreads = 256;
constexpr int kHeld = 8;           // sources whose columns fit in registers
constexpr int64_t kMostSeg = 32768, kLeastSeg = 8192;  // bytes of a row, a block
constexpr int64_t kEnoughBlocks = 152 * 16;

struct State {
  char* data;
  int64_t row_stride, run, token;   // bytes; token: 0: none, -1: outer[0] is the tokens' axis
  int64_t tokens;                   // of a run, where token is a size
  int64_t outer_stride[3];          // bytes
  int outer[3];
  int width;                        // bytes of an access: the alignment of base and strides
};

struct ReorderArgs {
  State st[kLaunchStates];
  unsigned first[kLaunchStates + 1];  // first block of each state
  int n;
  int64_t seg;                        // bytes of a row that a block moves
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
  uint8_t dest[kMaxBeams];      // the rows to write, source by source
  uint16_t first[kMaxBeams + 1];  // where a source's begin
  int sources;
};

struct Shared {                 // beside the slots that a launch asks for
  Plan plan;
  uint32_t taken[kMaxBeams / 32];
  uint8_t parent[kMaxBeams];    // itself: the row stays
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
    for (int i = 0; i < plan.sources; ++i) {
      const T v = *reinterpret_cast<const T*>(room + i * blockDim.x + threadIdx.x);
      for (int d = plan.first[i]; d < plan.first[i + 1]; ++d)
        *reinterpret_cast<T*>(p + plan.dest[d] * row_stride + at) = v;
    }
  }
}

// The same for S sources in registers, U columns at once.  source, to: the rows to read,
// and which take each.
template <int W, int S, int U>
__device__ __forceinline__ void move_held(char* p, int64_t row_stride, int64_t lo, int64_t hi,
                                          const int (&source)[kHeld], const uint32_t (&to)[kHeld]) {
  using T = typename Word<W>::T;
  const char* from[S];
#pragma unroll
  for (int i = 0; i < S; ++i) from[i] = p + source[i] * row_stride;
  const int64_t step = int64_t(blockDim.x) * W;
  for (int64_t at = lo + int64_t(threadIdx.x) * W; at < hi; at += U * step) {
    T v[U][S];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (at + u * step < hi)
          v[u][i] = *reinterpret_cast<const T*>(from[i] + at + u * step);
#pragma unroll
    for (int i = 0; i < S; ++i)
      for (uint32_t m = to[i]; m; m &= m - 1) {
        char* row = p + (__ffs(m) - 1) * row_stride + at;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (at + u * step < hi) *reinterpret_cast<T*>(row + u * step) = v[u][i];
      }
  }
}

template <int W>
__device__ __forceinline__ void move_few(int sources, char* p, int64_t row_stride, int64_t lo,
                                         int64_t hi, const int (&source)[kHeld],
                                         const uint32_t (&to)[kHeld]) {
  switch (sources) {
    case 1: move_held<W, 1, 4>(p, row_stride, lo, hi, source, to); break;
    case 2: move_held<W, 2, 4>(p, row_stride, lo, hi, source, to); break;
    case 3: move_held<W, 3, 2>(p, row_stride, lo, hi, source, to); break;
    case 4: move_held<W, 4, 2>(p, row_stride, lo, hi, source, to); break;
    case 5: move_held<W, 5, 1>(p, row_stride, lo, hi, source, to); break;
    case 6: move_held<W, 6, 1>(p, row_stride, lo, hi, source, to); break;
    case 7: move_held<W, 7, 1>(p, row_stride, lo, hi, source, to); break;
    default: move_held<W, 8, 1>(p, row_stride, lo, hi, source, to); break;
  }
}

__global__ void reorder_kernel(const __grid_constant__ ReorderArgs a) {
  extern __shared__ __align__(16) char raw[];
  uint4* room = reinterpret_cast<uint4*>(raw);
  __shared__ Shared sh;
  Plan& plan = sh.plan;
  uint32_t* taken = sh.taken;
  uint8_t* parent = sh.parent;

  int s = 0;  // the last state that begins at this block or before
  for (int half = kLaunchStates / 2; half; half >>= 1)
    if (s + half < a.n && a.first[s + half] <= blockIdx.x) s += half;
  const State& st = a.st[s];
  unsigned id = blockIdx.x - a.first[s];
  auto take = [&](unsigned of) {  // the next coordinate, of so many
    if (of == 1) return 0u;
    const unsigned q = id / of, r = id - q * of;
    id = q;
    return r;
  };
  const int64_t seg = take(unsigned((st.run + a.seg - 1) / a.seg));
  const int64_t b = take(unsigned(a.batch));
  const int32_t* parents = a.parents + b * a.beams;
  const int from = threadIdx.x % 32 < unsigned(a.beams) ? parents[threadIdx.x % 32] : -1;
  const int start = a.start ? a.start[b] : 0, stop = a.stop ? a.stop[b] : INT32_MAX;
  char* p = st.data + b * a.beams * st.row_stride;
  int64_t at0 = 0;  // place on the first outer axis
#pragma unroll
  for (int d = 2; d >= 0; --d) {
    at0 = take(unsigned(st.outer[d]));
    p += at0 * st.outer_stride[d];
  }

  // the bytes of this block: its segment within the batch entry's range
  int64_t lo = 0, hi = st.run;
  if (st.token > 0) {
    // cut to the run's tokens before they are bytes: an end far behind them, as where none is
    // given, times a token of 4 GB would pass 63 bits
    lo = min(int64_t(max(start, 0)), st.tokens) * st.token;
    hi = min(int64_t(max(stop, 0)), st.tokens) * st.token;
  } else if (st.token < 0) {
    if (at0 < start || at0 >= stop) return;
  }
  lo = max(lo, seg * a.seg);
  hi = min(hi, (seg + 1) * a.seg);
  if (lo >= hi) return;

  // A range of 16-byte words may begin and end inside one: those bytes one by one.
  int64_t mid_lo = lo, mid_hi = hi;
  if (st.width == 16) {
    mid_lo = min((lo + 15) & ~int64_t(15), hi);
    mid_hi = max(hi & ~int64_t(15), mid_lo);
  }

  // Up to 32 beams of few sources: each warp finds out for itself what moves.
  if (a.beams <= 32) {
    const int k = threadIdx.x & 31;
    const bool moves = from >= 0 && from < a.beams && from != k;
    uint32_t left = __reduce_or_sync(kFullWarp, moves ? 1u << from : 0u);
    const int sources = __popc(left);
    if (sources == 0) return;
    if (sources <= kHeld && st.width >= 4) {
      int source[kHeld];
      uint32_t to[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        source[i] = left ? __ffs(left) - 1 : 0;
        to[i] = __ballot_sync(kFullWarp, left && moves && from == source[i]);
        left &= left - 1;
      }
      if (st.width == 4) {
        move_few<4>(sources, p, st.row_stride, lo, hi, source, to);
      } else if (st.width == 8) {
        move_few<8>(sources, p, st.row_stride, lo, hi, source, to);
      } else {
        move_few<16>(sources, p, st.row_stride, mid_lo, mid_hi, source, to);
        if (lo < mid_lo) move_few<1>(sources, p, st.row_stride, lo, mid_lo, source, to);
        if (mid_hi < hi) move_few<1>(sources, p, st.row_stride, mid_hi, hi, source, to);
      }
      return;
    }
  }

  // which rows are read, which are written
  if (threadIdx.x < kMaxBeams / 32) taken[threadIdx.x] = 0;
  __syncthreads();
  for (int k = threadIdx.x; k < a.beams; k += blockDim.x) {
    const int from = parents[k];
    const bool moves = from >= 0 && from < a.beams && from != k;
    parent[k] = uint8_t(moves ? from : k);
    if (moves) atomicOr(&taken[from >> 5], 1u << (from & 31));
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int n_src = 0;
    for (int w = 0; w * 32 < a.beams; ++w) {
      const uint32_t below = (1u << threadIdx.x) - 1u;
      if (taken[w] >> threadIdx.x & 1u)
        plan.source[n_src + __popc(taken[w] & below)] = uint8_t(w * 32 + threadIdx.x);
      n_src += __popc(taken[w]);
    }
    if (threadIdx.x == 0) plan.sources = n_src;
    __syncwarp();
    // a lane lists the rows of its sources, behind those of the sources before
    int n_dst = 0;
    for (int i0 = 0; i0 < n_src; i0 += 32) {
      const int i = i0 + threadIdx.x;
      const int from = i < n_src ? plan.source[i] : -1;
      int mine = 0;
      for (int k = 0; k < a.beams; ++k) mine += parent[k] == from && k != from;
      int before = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kFullWarp, before, o);
        if (threadIdx.x >= o) before += up;
      }
      const int all = __shfl_sync(kFullWarp, before, 31);
      if (i < n_src) {
        int at = n_dst + before - mine;
        plan.first[i] = uint16_t(at);
        for (int k = 0; k < a.beams; ++k)
          if (parent[k] == from && k != from) plan.dest[at++] = uint8_t(k);
      }
      n_dst += all;
    }
    if (threadIdx.x == 0) plan.first[n_src] = uint16_t(n_dst);
  }
  __syncthreads();
  if (plan.sources == 0) return;

  switch (st.width) {
    case 16:
      move_columns<16>(p, st.row_stride, mid_lo, mid_hi, plan, room);
      move_columns<1>(p, st.row_stride, lo, mid_lo, plan, room);
      move_columns<1>(p, st.row_stride, mid_hi, hi, plan, room);
      break;
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

  auto blocks_of = [&](const lp_state& s, int64_t seg) -> int64_t {
    const int64_t segs = s.run_bytes / seg + (s.run_bytes % seg != 0);
    int64_t n = batch;
    for (int64_t f : {segs, s.outer[0], s.outer[1], s.outer[2]}) {
      if (f == 0) return 0;
      if (n > INT32_MAX / f) return -1;
      n *= f;
    }
    return n;
  };
  for (int64_t i = 0; i < n_states; ++i)
    if (blocks_of(states[i], kMostSeg) < 0) return LP_ERR_TOO_LARGE;
  // A block first finds out what moves, so its piece is large (with 64 KB no better: 135 us
  // to 132 for 16 x 5 rows laid out heads first), unless there would not be enough blocks
  // to keep all SMs busy: 4 rows of 128 tokens of 2 layers take 9.4 us in pieces of 32 KB,
  // 3.5 in 8 KB, 4.0 in 4 KB.
  int64_t seg = kMostSeg;
  for (; seg > kLeastSeg; seg /= 2) {
    int64_t blocks = 0;
    for (int64_t i = 0; i < n_states && blocks < kEnoughBlocks; ++i) {
      const int64_t n = blocks_of(states[i], seg);
      blocks = n < 0 ? kEnoughBlocks : blocks + n;
    }
    if (blocks >= kEnoughBlocks) break;
  }

  const int threads =
      int(std::max<int64_t>(32, std::min<int64_t>(kThreads, (98304 / 16 / beams) & ~31)));
  const size_t smem = size_t(threads) * 16 * size_t(beams);
  // A block's 48 KB without leave are for the kernel's own arrays too: with 12 beams the
  // slots alone are all of them (16 bytes: the alignment between the two)
  if (smem + sizeof(Shared) + 16 > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        reorder_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxBeams * 32 * 16);
    if (e != cudaSuccess) return status_of(e);
  }
  ReorderArgs a = {};
  a.batch = batch;
  a.seg = seg;
  a.beams = int(beams);
  a.parents = parents;
  a.start = start;
  a.stop = stop;
  for (int64_t i = 0; i < n_states;) {
    a.n = 0;
    for (; i < n_states && a.n < kLaunchStates; ++i) {
      const lp_state& s = states[i];
      const int64_t n = blocks_of(s, seg);
      if (n == 0) continue;
      if (a.n > 0 && int64_t(a.first[a.n]) + n > INT32_MAX) break;
      State& t = a.st[a.n];
      t.data = static_cast<char*>(s.data);
      t.row_stride = s.row_stride;
      t.run = s.run_bytes;
      t.token = s.token_bytes;
      t.tokens = s.token_bytes > 0 ? s.run_bytes / s.token_bytes : 0;
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
    const cudaError_t e = launch_kernel(reorder_kernel, a.first[a.n], threads, smem, stream, a);
    if (e != cudaSuccess) return status_of(e);
  }
  return LP_OK;
}
