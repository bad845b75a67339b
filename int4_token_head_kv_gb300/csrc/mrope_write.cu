// The write with a position rotation of several axes into the INT4 cache.
#include "rope_write.cuh"

namespace kvi4 {

cudaError_t launch_mrope_write(const RopeWriteParams& p, int head_size, DType dt, bool interleaved, cudaStream_t stream) {
    return launch_rope_write_mode<4, true>(p, head_size, dt, interleaved, stream);
}

}  // namespace kvi4
