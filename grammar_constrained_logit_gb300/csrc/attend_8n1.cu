// attend_8n1.cu -- attention over a cache of 8 bits: queries and weights in one piece, 8 rows.
#include "attend_mma.cuh"

namespace lp {

cudaError_t attend_8n1(const AttendArgs& a, int block, cudaStream_t stream) {
  return attend_mma<8, false, 1>(a, block, stream);
}

}  // namespace lp
