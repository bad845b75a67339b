// The write with the position rotation into the INT8 cache.
#include "rope_write.cuh"

namespace kvi4 {

cudaError_t launch_rope_write_int8(const RopeWriteParams& p, int head_size, DType dt, bool interleaved, cudaStream_t stream) {
    return launch_rope_write_mode<8>(p, head_size, dt, interleaved, stream);
}

}  // namespace kvi4
