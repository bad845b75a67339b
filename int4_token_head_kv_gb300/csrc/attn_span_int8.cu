// Attention over key spans on the INT8 cache.
#include "attn_span.cuh"

namespace kvi4 {

cudaError_t launch_span_int8(const SpanParams& p, int head_size, cudaStream_t stream) {
    return head_size == 128 ? launch_span_head<128, 8>(p, stream) : launch_span_head<64, 8>(p, stream);
}

}  // namespace kvi4
