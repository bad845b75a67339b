// The shared-prefix kernel's instantiations, and the rule that splits the prefix.
#include "attn_prefix.cuh"

namespace kvi4 {

int prefix_splits(int64_t row_tiles, int num_kv_heads, int prefix_len) {
    // Time of a CTA is about its key tiles plus kFixed tiles' worth of start and end (rotation, partials);
    // the grid runs in waves of one CTA per SM.  The fewest splits with the smallest sum: more of them
    // only add partials to merge.
    constexpr int64_t kFixed = 6;
    const int64_t tiles = (prefix_len + kPfKeys - 1) / kPfKeys, base = row_tiles * num_kv_heads, sms = num_sms();
    int64_t best = 1, best_cost = INT64_MAX;
    for (int64_t s = 1; s <= tiles && s <= kMaxPrefixSplits; ++s) {
        const int64_t waves = (base * s + sms - 1) / sms;
        const int64_t cost = waves * ((tiles + s - 1) / s + kFixed);
        if (cost < best_cost) {
            best_cost = cost;
            best = s;
        }
    }
    return (int)best;
}

namespace {
template <int D, typename QT>
cudaError_t prefix_by_options(const AttnParams& p, cudaStream_t stream) {
    if (p.opts != 0) return launch_prefix_t<D, QT, true, true>(p, stream);
    return p.px_two ? launch_prefix_t<D, QT, false, true>(p, stream) : launch_prefix_t<D, QT, false, false>(p, stream);
}
}  // namespace

cudaError_t launch_prefix(const AttnParams& p, int head_size, DType q_dt, cudaStream_t stream) {
    if (head_size == 128)
        return q_dt == DType::BF16 ? prefix_by_options<128, __nv_bfloat16>(p, stream) : prefix_by_options<128, __half>(p, stream);
    return q_dt == DType::BF16 ? prefix_by_options<64, __nv_bfloat16>(p, stream) : prefix_by_options<64, __half>(p, stream);
}

}  // namespace kvi4
