// Attention over key spans on the INT4 cache, and the entry that picks the cache mode.
#include "attn_span.cuh"

namespace kvi4 {

cudaError_t launch_span(const SpanParams& p, int bits, int head_size, cudaStream_t stream) {
    if (bits == 8) return launch_span_int8(p, head_size, stream);
    if (bits == 2) return launch_span_int2(p, head_size, stream);
    return head_size == 128 ? launch_span_head<128, 4>(p, stream) : launch_span_head<64, 4>(p, stream);
}

}  // namespace kvi4
