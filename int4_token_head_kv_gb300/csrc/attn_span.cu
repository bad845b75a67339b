// Attention in which every query row sees the cached keys of a span of its own, over the INT4, INT8 and INT2
// caches: for the query at position pos of its sequence, over the keys begin <= j < end,
//   s_j = scale q . x_Kj,  s_j <- softcap tanh(s_j / softcap),  s_j <- s_j - slope |pos - j|,
//   out = sum_j softmax(s)_j x_Vj   (0 for an empty span).
//
// One warp per (query token, q head): lane l holds dimensions l D/32 .. of the (rotated) query and of the running
// output, the keys go by one at a time with a running maximum and sum.  Bound by its instructions: every key is
// decoded once for every query row.
#include "attn_common.cuh"

namespace kvi4 {
namespace {

constexpr int kSpanWarps = 4;

template <int D, int BITS>
__global__ void __launch_bounds__(kSpanWarps * 32) span_kernel(const __grid_constant__ SpanParams p, DType q_dt, DType out_dt) {
    constexpr int V = D / 32, RB = D * BITS / 8 + 4;
    __shared__ float rows[kSpanWarps][D];
    __shared__ float sgn[D];
    for (int i = threadIdx.x; i < D; i += blockDim.x) sgn[i] = BITS != 8 && p.signs[i] < 0.0f ? -1.0f : 1.0f;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tok = blockIdx.x;
    const int head = (int)blockIdx.y * kSpanWarps + warp;
    if (head >= p.Hq) return;
    int b = 0, hi = p.num_seqs;   // the last sequence with qsl[b] <= tok
    while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (__ldg(p.qsl + mid) <= tok) b = mid;
        else hi = mid;
    }
    const int q0 = __ldg(p.qsl + b), qlen = __ldg(p.qsl + b + 1) - q0;
    if (tok < q0 || tok >= (int64_t)q0 + min(qlen, p.max_query_len)) return;
    int L = __ldg(p.seq_lens + b);
    if (tok == q0 && head == 0 && lane == 0 && (L > p.len_cap || (qlen > L && L != 0) || qlen > p.max_query_len)) count_status(p.status, 2);
    L = max(0, min(L, p.len_cap));
    const int pos = __ldg(p.seq_lens + b) - qlen + (int)(tok - q0);
    const int begin = p.key_begin ? max(0, __ldg(p.key_begin + tok)) : 0;
    const int end = min(L, p.key_end ? __ldg(p.key_end + tok) : pos + 1);
    const int64_t at = (tok * p.Hq + head) * D;

    float x[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int64_t i = at + lane + 32 * k;
        x[k] = (q_dt == DType::BF16 ? load_elem<__nv_bfloat16>(p.q, i) : load_elem<__half>(p.q, i)) * sgn[lane + 32 * k];
    }
    if constexpr (BITS != 8) warp_fwht<D>(x);
    float* row = rows[warp];
#pragma unroll
    for (int k = 0; k < V; ++k) row[lane + 32 * k] = x[k];
    __syncwarp();
    float q[V], o[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        q[k] = row[lane * V + k];
        o[k] = 0.0f;
    }
    const float slope = p.alibi ? __ldg(p.alibi + head) : 0.0f;
    const float qs = p.c * p.softmax_scale;
    const int h = head / p.G;
    // this lane's dimensions of a row
    auto decode = [&](const uint8_t* r, float (&y)[V]) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(r + RB - 4);
        const float s = __uint_as_float(BITS == 4 ? w & 0xFFFFFFF0u : w);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int bit = (lane * V + k) * BITS, code = (r[bit >> 3] >> (bit & 7)) & ((1 << BITS) - 1);
            const float n = BITS == 4   ? (float)(code - (int)(w & 15u))
                            : BITS == 8 ? (float)(int8_t)code
                                        : (code < 2 ? -1.0f : 1.0f) * (code == 1 || code == 2 ? 0.45278f : 1.51042f);
            y[k] = n * s;
        }
    };
    float m = -INFINITY, l = 0.0f;
    for (int j = begin; j < end; ++j) {
        const int blk = __ldg(p.block_tables + (int64_t)b * p.max_blocks_per_seq + j / kBlockSize);
        if (blk < 0 || blk >= p.num_blocks) {
            if (tok == q0 && head == 0 && lane == 0 && j % kBlockSize == 0) count_status(p.status, 1);
            continue;
        }
        const uint8_t* r = p.cache + (((int64_t)blk * 2 * kBlockSize + j % kBlockSize) * p.H + h) * RB;
        float y[V], s = 0.0f;
        decode(r, y);
#pragma unroll
        for (int k = 0; k < V; ++k) s = fmaf(q[k], y[k], s);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= qs;
        if (p.softcap > 0.0f) s = p.softcap * tanhf(s / p.softcap);
        s -= slope * fabsf((float)(pos - j));
        decode(r + (int64_t)kBlockSize * p.H * RB, y);
        const float mn = fmaxf(m, s);   // a logit that is not a number shows through w
        const float f = m > -INFINITY ? __expf(m - mn) : 0.0f, w = s == -INFINITY ? 0.0f : __expf(s - mn);
        m = mn;
        l = fmaf(l, f, w);
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = fmaf(o[k], f, w * y[k]);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int k = 0; k < V; ++k) row[lane * V + k] = o[k] * inv;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < V; ++k) x[k] = row[lane + 32 * k];
    if constexpr (BITS != 8) warp_fwht<D>(x);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const float y = x[k] * p.c * sgn[lane + 32 * k];
        const int64_t i = at + lane + 32 * k;
        if (out_dt == DType::F16) store_elem<__half>(p.out, i, y);
        else if (out_dt == DType::BF16) store_elem<__nv_bfloat16>(p.out, i, y);
        else store_elem<float>(p.out, i, y);
    }
}

template <int BITS>
cudaError_t launch_span_mode(const SpanParams& p, int head_size, DType q_dt, DType out_dt, cudaStream_t s) {
    const dim3 grid((unsigned)p.num_q_tokens, (unsigned)((p.Hq + kSpanWarps - 1) / kSpanWarps));
    if (head_size == 128) span_kernel<128, BITS><<<grid, kSpanWarps * 32, 0, s>>>(p, q_dt, out_dt);
    else span_kernel<64, BITS><<<grid, kSpanWarps * 32, 0, s>>>(p, q_dt, out_dt);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_span(const SpanParams& p, int bits, int head_size, DType q_dt, DType out_dt, cudaStream_t s) {
    return bits == 8   ? launch_span_mode<8>(p, head_size, q_dt, out_dt, s)
           : bits == 2 ? launch_span_mode<2>(p, head_size, q_dt, out_dt, s)
                       : launch_span_mode<4>(p, head_size, q_dt, out_dt, s);
}

}  // namespace kvi4
