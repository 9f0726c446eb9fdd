// attend_8w2.cu -- attention over a cache of 8 bits: queries and weights in two pieces, 16 rows.
#include "attend_mma.cuh"

namespace lp {

cudaError_t attend_8w2(const AttendArgs& a, int block, cudaStream_t stream) {
  return attend_mma<8, true, 2>(a, block, stream);
}

}  // namespace lp
