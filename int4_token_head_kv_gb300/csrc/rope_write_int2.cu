// The write with the position rotation into the INT2 cache.
#include "rope_write.cuh"

namespace kvi4 {

cudaError_t launch_rope_write_int2(const RopeWriteParams& p, int head_size, DType dt, bool interleaved, cudaStream_t stream) {
    return launch_rope_write_mode<2>(p, head_size, dt, interleaved, stream);
}

}  // namespace kvi4
