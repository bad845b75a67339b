// Cache write of the INT4 per-(token, head) KV cache: random Hadamard rotation, asymmetric 4-bit
// quantisation with the zero-point hidden in the scale's low mantissa bits, nibble packing and a
// paged store ("[Feature] Triton INT4 / INT2 per-token-head KV cache quantization", description;
// "PR #40835 report", get_kv_cache_shape).
//
// The encoders are in write_common.cuh; this file holds the kernel that feeds them K and V as they come.
#include "write_common.cuh"

namespace kvi4 {
namespace {

template <int D, typename T, int BITS>
__global__ void __launch_bounds__(kWriteThreads, WriteShape<BITS>::kMinBlocks)
    write_kernel(const __grid_constant__ WriteParams p) {
    using Gm = Geo<D>;
    using Sh = WriteShape<BITS>;
    constexpr bool INT8 = BITS == 8;
    constexpr int TPV = Sh::kTpv, TV = Sh::kTileVecs;
    constexpr int RB = INT8 ? D + 4 : (BITS == 2 ? D / 4 + 4 : Gm::RB);   // cache row bytes
    constexpr int NW = RB / 4 - 1;                                       // code words per row (then the scale)
    constexpr int OW = INT8 ? NW + 1 : NW / 2 + 1;   // words one thread stores (the last: the scale word)
    using Sm = WriteSmem<D, TV>;
    extern __shared__ __align__(128) uint8_t smem[];
    // Launched as a programmatic dependent: wait for the previous kernel of the stream (it may
    // produce K, V or the slots), then let the next kernel start its own set-up.
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int vl = lane / TPV, part = lane % TPV;   // this thread's vector of the tile and its part
    uint8_t* wbuf = smem + warp * Sm::kPerWarp;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sm::kBars) + warp * 2;   // this warp's [buffer]
    WriteSigns<D>& sgn = *reinterpret_cast<WriteSigns<D>*>(smem + Sm::kBars + kWriteWarps * 2 * 8);
    if (lane == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        fence_mbar_init();
    }
    for (int j = tid; j < (INT8 ? 0 : D / 2); j += kWriteThreads) {   // INT8 rows take no signs
        const float s0 = p.signs[2 * j], s1 = p.signs[2 * j + 1];
        // bf16 takes the even sign in the FMA (its mask flips only the odd element); fp16 in the XOR
        const uint32_t m = ((std::is_same<T, __nv_bfloat16>::value ? 0u : (__float_as_uint(s0) >> 31)) << 15) |
                           ((__float_as_uint(s1) >> 31) << 31);
        sgn.xmask[0][j] = m;
        sgn.xmask[1][j] = m ^ 0x80000000u;
        if ((j & 1) == 0) {   // the bf16 signs of elements 2j and 2j + 2
            const float s2 = p.signs[2 * j + 2];
            const int kk = j % (D / 4), half = j / (D / 4);
            sgn.esign[(kk & ~3) + ((kk >> 1) & 1) + 2 * half] =
                (s0 < 0.0f ? 0xBF80u : 0x3F80u) | ((s2 < 0.0f ? 0xBF80u : 0x3F80u) << 16);
        }
        if (blockIdx.x == 0 && ((fabsf(s0) != 1.0f) || (fabsf(s1) != 1.0f))) count_status(p.status, 4);
    }
    __syncthreads();

    const uint32_t H = (uint32_t)p.H;
    VecIndex vx;
    vx.H = H;
    vx.hmask = H - 1;
    vx.hshift = (H & (H - 1)) == 0 ? __ffs(H) - 1 : -1;
    const uint32_t nvec = (uint32_t)(p.num_tokens * H * 2);
    const uint32_t ntiles = (nvec + TV - 1) / TV;
    const uint32_t gwarp = blockIdx.x * kWriteWarps + warp, nwarps = gridDim.x * kWriteWarps;
    const uint32_t group_bytes = H * RB;
    const bool grouped = vx.hshift >= 0 && H <= (uint32_t)TV && (group_bytes % 16) == 0;
    const uint8_t* kin = static_cast<const uint8_t*>(p.k);
    const uint8_t* vin = static_cast<const uint8_t*>(p.v);

    // lane i < TV copies vector i of the tile (2D bytes) into row i of the buffer
    auto prefetch = [&](uint32_t tile, uint8_t* buf, uint64_t* bar) {
        const uint32_t v0 = tile * TV;
        const uint32_t live_vecs = min((uint32_t)TV, nvec - v0);
        if (lane == 0) mbar_arrive_expect_tx(bar, live_vecs * (uint32_t)(D * 2));
        __syncwarp();
        if ((uint32_t)lane < live_vecs) {
            uint32_t tok, h, pl;
            vx.split(v0 + lane, tok, h, pl);
            bulk_copy_g2s(buf + lane * Sm::kRowPad, (pl ? vin : kin) + (uint64_t)(tok * H + h) * (D * 2), D * 2, bar,
                          policy_evict_first());
        }
    };

    uint32_t tile = gwarp;
    int it = 0;
    bool waited_out = false;
    if (tile < ntiles) prefetch(tile, wbuf, &bars[0]);
    for (; tile < ntiles; tile += nwarps, ++it) {
        uint8_t* cur = wbuf + (it & 1) * Sm::kBuf;
        uint8_t* nxt = wbuf + ((it + 1) & 1) * Sm::kBuf;
        // the other buffer was last an output stage: its bulk stores must have read it
        if (grouped) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        if (tile + nwarps < ntiles) prefetch(tile + nwarps, nxt, &bars[(it + 1) & 1]);
        // this tile's rows: use (it >> 1) of buffer it & 1
        if (__any_sync(0xffffffffu, !mbar_wait(&bars[it & 1], (uint32_t)(it >> 1) & 1u))) {
            if (lane == 0) count_status(p.status, 3);
            waited_out = true;
            break;
        }
        const uint32_t v = tile * TV + vl;
        const bool live = v < nvec;
        uint32_t words[OW];
        if constexpr (INT8) {
            float u[D];
            if (live) load_vector_raw<D, T>(reinterpret_cast<const uint4*>(cur + vl * Sm::kRowPad), u);
            __syncwarp();   // the tile's inputs are in registers; its buffer becomes the output stage
            if (live) encode_vector_int8<D>(u, words);
        } else {
            // every lane runs the encoder (it exchanges values within the lane pair); a vector past
            // the end reads row 0, which every tile holds, and its words are discarded
            const uint32_t* in = reinterpret_cast<const uint32_t*>(cur + (live ? vl : 0) * Sm::kRowPad);
            if constexpr (BITS == 2) encode_half_int2<D, T>(in, sgn, part, p.c, words);
            else encode_half<D, T>(in, sgn, part, p.c, words);
            __syncwarp();   // the tile's inputs are consumed; its buffer becomes the output stage
        }
        // this thread's words of the row: all of them (INT8), or the first / second half of the code
        // words (INT4 / INT2 parts 0 / 1; part 1 also the scale word)
        const int w0 = INT8 ? 0 : part * (NW / 2);
        const int nw = INT8 ? OW : (part ? OW : OW - 1);
        uint32_t tok = 0, h = 0, pl = 0;
        if (live) vx.split(v, tok, h, pl);
        if (grouped) {
            uint32_t* orow = reinterpret_cast<uint32_t*>(cur + vl * RB) + w0;
            if (live) {
#pragma unroll
                for (int wi = 0; wi < OW; ++wi)
                    if (wi < nw) orow[wi] = words[wi];
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // staged rows -> bulk store
            __syncwarp();
            // the first thread of each row group stores the whole group
            if (live && h == 0 && part == 0) {
                const int64_t slot = __ldg(p.slots + tok);
                if (slot >= p.num_slots) {
                    if (pl == 0) count_status(p.status, 0);
                } else if (slot >= 0) {
                    const int64_t blk = slot / kBlockSize, off = slot % kBlockSize;
                    bulk_store_s2g(p.cache + ((blk * 2 + pl) * kBlockSize + off) * (int64_t)group_bytes,
                                   cur + vl * RB, group_bytes);
                }
            }
        } else if (live) {
            const int64_t slot = __ldg(p.slots + tok);
            if (slot >= p.num_slots) {
                if (pl == 0 && h == 0 && part == 0) count_status(p.status, 0);
            } else if (slot >= 0) {
                const int64_t blk = slot / kBlockSize, off = slot % kBlockSize;
                uint32_t* row =
                    reinterpret_cast<uint32_t*>(p.cache + (((blk * 2 + pl) * kBlockSize + off) * H + h) * RB) + w0;
#pragma unroll
                for (int wi = 0; wi < OW; ++wi)
                    if (wi < nw) row[wi] = words[wi];
            }
        }
    }
    if (waited_out && tile + nwarps < ntiles) {   // let the copy in flight land before the warp exits
        (void)mbar_wait(&bars[(it + 1) & 1], (uint32_t)((it + 1) >> 1) & 1u);
    }
    if (grouped) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    (void)kRoundMagicBits;
}

template <int D, typename T, int BITS>
cudaError_t launch_write_t(const WriteParams& p, cudaStream_t stream) {
    using Sh = WriteShape<BITS>;
    using Sm = WriteSmem<D, Sh::kTileVecs>;
    const int64_t ntiles = (p.num_tokens * p.H * 2 + Sh::kTileVecs - 1) / Sh::kTileVecs;
    int64_t blocks = (ntiles + kWriteWarps - 1) / kWriteWarps;
    const int64_t cap = (int64_t)num_sms() * Sh::kMinBlocks;
    if (blocks > cap) blocks = cap;
    if (blocks < 1) blocks = 1;
    cudaError_t err = opt_in_smem<write_kernel<D, T, BITS>>(Sm::kBytes);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kWriteThreads);
    cfg.dynamicSmemBytes = Sm::kBytes;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, write_kernel<D, T, BITS>, p);
}

}  // namespace

namespace {
template <int BITS>
cudaError_t launch_write_mode(const WriteParams& p, int head_size, DType dt, cudaStream_t stream) {
    if (head_size == 128) {
        return dt == DType::BF16 ? launch_write_t<128, __nv_bfloat16, BITS>(p, stream)
                                 : launch_write_t<128, __half, BITS>(p, stream);
    }
    return dt == DType::BF16 ? launch_write_t<64, __nv_bfloat16, BITS>(p, stream)
                             : launch_write_t<64, __half, BITS>(p, stream);
}
}  // namespace

cudaError_t launch_write(const WriteParams& p, int head_size, DType dt, cudaStream_t stream) {
    return launch_write_mode<4>(p, head_size, dt, stream);
}

cudaError_t launch_write_int8(const WriteParams& p, int head_size, DType dt, cudaStream_t stream) {
    return launch_write_mode<8>(p, head_size, dt, stream);
}

cudaError_t launch_write_int2(const WriteParams& p, int head_size, DType dt, cudaStream_t stream) {
    return launch_write_mode<2>(p, head_size, dt, stream);
}

}  // namespace kvi4
