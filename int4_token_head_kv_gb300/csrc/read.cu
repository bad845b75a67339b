// Read-back of cached rows: the keys and values that the rows at given slots stand for, the inverse of
// the cache writes (kv_int4.h: a reader reconstructs (code - zp) s', centroid(code) sigma or code s,
// and un-rotates the INT4 and INT2 rows by x = c D H_d y).
//
// Vectors are numbered (plane * num_tokens + token) * H + head, the order of the outputs.  A warp owns
// tiles of kTileVecs vectors and pipelines them on its own: the packed rows of the next tile arrive by
// bulk copies (one per token and plane, when the H rows of a token are a multiple of 16 bytes and a
// tile holds whole tokens; otherwise the lanes copy words) while this one is decoded; decoded rows are
// staged and leave as one bulk store per row.
//
// INT4 and INT2: a lane pair per vector, thread t with the outputs of the stride-1 butterflies of
// parity t, as the writes split it.  An INT4 row's butterflies run on the integers code - zp, whose sums
// stay within +-15 * 128: exact in fp16, two to a register, in any order of the strides; the one rounding
// before the output's is the product with fp32(c s').  INT2 centroids are not integers: fp32.
// What bounds it (65 536 tokens, 8 heads, d 128, bf16: 70 us, 4.9 TB/s, floor 51): 60 M warp-instructions at
// 60-70% issue, half of them logic on the codes and the two-byte exchange of the pair's outputs.  Selects in
// that exchange cost 8%; a warp's rows written by 16-byte stores instead of bulk copies cost 7%.
// INT8: a thread per vector, code * s.
#include "write_common.cuh"

namespace kvi4 {
namespace {

template <int BITS>
struct ReadShape {
    static constexpr int kTpv = BITS == 8 ? 1 : 2;
    static constexpr int kTileVecs = 32 / kTpv;
};

template <int D, int BITS, typename OT>
struct ReadSmem {
    static constexpr int TV = ReadShape<BITS>::kTileVecs;
    static constexpr int RB = D * BITS / 8 + 4;
    static constexpr int kOutRow = D * (int)sizeof(OT) + 16;   // padded: 16-byte accesses of 8 rows hit distinct banks
    static constexpr int kIn = (TV * RB + 15) / 16 * 16;       // packed rows of a tile, as the cache holds them
    static constexpr int kOut = TV * kOutRow;
    static constexpr int kPerWarp = 2 * kIn + kOut;
    static constexpr int kBars = kWriteWarps * kPerWarp;       // two mbarriers per warp
    static constexpr int kMask = kBars + kWriteWarps * 16;     // [D / 2] sign bits of an output pair (15: even, 31: odd)
    static constexpr int kBytes = kMask + D * 2;
    // Resident CTAs per SM, the grid's unit: what the shared memory leaves, up to 8 for INT4 (64 registers; 65 536
    // tokens of 8 heads, d 128: 70 us, 72 with 5, 77 with 4) and 5 for the others (INT2 spills below 96).
    static constexpr int kFit = 230000 / (kBytes + 1024);
    static constexpr int kBlocks = BITS == 4 ? (kFit < 8 ? kFit : 8) : (kFit < 5 ? kFit : 5);
};

__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// two neighbouring elements of an output row (element 2m in the low half for 16-bit types)
template <typename OT>
struct OutPair;
template <>
struct OutPair<__half> {
    static __device__ __forceinline__ void put(uint32_t* row, int m, float2 x, uint32_t mask) {
        __half2 h = __float22half2_rn(x);
        row[m] = *reinterpret_cast<uint32_t*>(&h) ^ mask;
    }
};
template <>
struct OutPair<__nv_bfloat16> {
    static __device__ __forceinline__ void put(uint32_t* row, int m, float2 x, uint32_t mask) {
        __nv_bfloat162 h = __float22bfloat162_rn(x);
        row[m] = *reinterpret_cast<uint32_t*>(&h) ^ mask;
    }
};
template <>
struct OutPair<float> {
    static __device__ __forceinline__ void put(uint32_t* row, int m, float2 x, uint32_t mask) {
        row[2 * m] = __float_as_uint(x.x) ^ ((mask << 16) & 0x80000000u);
        row[2 * m + 1] = __float_as_uint(x.y) ^ (mask & 0x80000000u);
    }
};

// One thread's half of the decoded row, elements part * D/2 .. + D/2 - 1, as 4-byte words of OT (a
// vector register array; the caller stores it).
template <typename OT>
__host__ __device__ constexpr int out_words(int n) { return n * (int)sizeof(OT) / 4; }

// INT4: w the row's D/8 code words, then the scale word.  Byte m of the row holds elements 2m (low nibble)
// and 2m + 1.  Thread t forms the outputs of parity t, then finishes the pairs m whose bit 4 is t: out[16 g + i]
// is pair 32 g + 16 t + i (the two threads' 16-byte stores then fall in different banks).
template <int D, typename OT>
__device__ __forceinline__ void decode_half(const uint32_t* w, const uint32_t* mask, int t, float c, bool live,
                                            uint32_t (&out)[out_words<OT>(D / 2)]) {
    constexpr int W = D / 8;   // code words
    const uint32_t sw = live ? w[W] : 0u;
    const uint32_t zp = sw & 15u;
    const float scale = __fmul_rn(__uint_as_float(sw & 0xFFFFFFF0u), c);   // dead rows: 0
    // stride 1: u_m = (e_2m - zp) + (e_2m+1 - zp) (t = 0) or e_2m - e_2m+1 (t = 1), from 1024 + e_2m and
    // 1024 + 16 e_2m+1: every sum and product below is an exact small integer
    const uint32_t sgn = t ? 0xBC00BC00u : 0x3C003C00u;                                     // +-1
    const uint32_t nsgn = sgn ^ 0x80008000u;
    const uint32_t sixteenth = t ? 0xAC00AC00u : 0x2C002C00u;                               // +-1/16
    const uint32_t bias = t ? 0xE380E380u : hsub2(0xE440E440u, hadd2(zp_lo_half(zp) * 0x10001u, hadd2(zp_lo_half(zp) * 0x10001u, 0xE800E800u)));   // -960 or -1088 - 2 zp
    uint32_t u[2 * W];   // u[2w + e]: pairs m = 4w + e (low half) and 4w + e + 2
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const uint32_t x = w[i], x8 = x >> 8;
        u[2 * i] = hfma2(lop3_and_or(x, 0x00F000F0u, 0x64006400u), sixteenth, hadd2(lop3_and_or(x, 0x000F000Fu, 0x64006400u), bias));
        u[2 * i + 1] = hfma2(lop3_and_or(x8, 0x00F000F0u, 0x64006400u), sixteenth, hadd2(lop3_and_or(x8, 0x000F000Fu, 0x64006400u), bias));
    }
    // bit 1 of m lies within a register
    const __half2 pm = __halves2half2(__ushort_as_half(0x3C00), __ushort_as_half(0xBC00));   // (1, -1)
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) {
        const __half2 v = *reinterpret_cast<const __half2*>(&u[i]);
        const __half2 r = __hfma2(__high2half2(v), pm, __low2half2(v));   // (a + b, a - b)
        u[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
    // bits 0, 2, 3 (and 5) between registers; bit 4 (register index bit 3) with the exchange below
#pragma unroll
    for (int st = 1; st < 2 * W; st <<= 1) {
        if (st == 8) continue;
#pragma unroll
        for (int i = 0; i < 2 * W; ++i) {
            if (i & st) continue;
            const uint32_t a = u[i], b = u[i + st];
            u[i] = hadd2(a, b);
            u[i + st] = hsub2(a, b);
        }
    }
    const float2 s2 = make_float2(scale, scale);
    const uint32_t sel_lo = t ? 0x1054u : 0x5410u, sel_hi = t ? 0x3276u : 0x7632u;   // (element 2m, element 2m + 1)
#pragma unroll
    for (int g = 0; g < W / 8; ++g) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {   // words 8 g + q and 8 g + q + 4
            const uint4 mk = *reinterpret_cast<const uint4*>(mask + 32 * g + 16 * t + 4 * q);
            uint32_t x[4];   // pairs 4 q .. 4 q + 3 of the group
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t a = u[16 * g + 2 * q + e], b = u[16 * g + 2 * q + 8 + e];
                const uint32_t mine = hfma2(b, sgn, a);
                const uint32_t other = __shfl_xor_sync(0xffffffffu, hfma2(b, nsgn, a), 1);
                x[e] = prmt(mine, other, sel_lo);
                x[e + 2] = prmt(mine, other, sel_hi);
            }
            const uint32_t m4[4] = {mk.x, mk.y, mk.z, mk.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                OutPair<OT>::put(out, 16 * g + 4 * q + e, mul_f32x2(half2_to_float2(x[e]), s2), m4[e]);
        }
    }
}

// INT2: w the row's D/16 code words (element 4j + k in bits 2k of byte j), then sigma.
template <int D, typename OT>
__device__ __forceinline__ void decode_half_int2(const uint32_t* w, const uint32_t* mask, int t, float c, bool live,
                                                 uint32_t (&out)[out_words<OT>(D / 2)]) {
    constexpr int Q = D / 4;
    const float sigma = live ? __uint_as_float(w[D / 16]) : 0.0f;
    auto centroid = [&](int e) -> float {
        const uint32_t code = (w[e / 16] >> (2 * (e % 16))) & 3u;
        const float a = (code == 1u || code == 2u) ? kLmA : kLmB;
        return code & 2u ? a : -a;
    };
    float2 P[Q];   // P[k] = elements 2k + t and 2(k + Q) + t of the stride-1 outputs
#pragma unroll
    for (int k = 0; k < Q; ++k) {
        const float a0 = centroid(2 * k), a1 = centroid(2 * k + 1);
        const float b0 = centroid(2 * (k + Q)), b1 = centroid(2 * (k + Q) + 1);
        P[k] = t ? make_float2(__fsub_rn(a0, a1), __fsub_rn(b0, b1)) : make_float2(__fadd_rn(a0, a1), __fadd_rn(b0, b1));
    }
    butterflies_half<D>(c, P);
#pragma unroll
    for (int k = 0; k < Q; ++k) {
        const float other = __shfl_xor_sync(0xffffffffu, t ? P[k].x : P[k].y, 1);
        const float mine = t ? P[k].y : P[k].x;
        const float2 x = make_float2((t ? other : mine) * sigma, (t ? mine : other) * sigma);
        OutPair<OT>::put(out, k, x, mask[k]);
    }
}

// INT8: elements D/2 * part .. of the row, no rotation
template <int D, typename OT>
__device__ __forceinline__ void decode_int8_words(const uint32_t* w, int first, float s, uint32_t (&out)[4]) {
    // 16 bytes of output: 8 elements of a 16-bit type, 4 of fp32
    constexpr int N = 16 / (int)sizeof(OT);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const uint32_t x = w[first / 4 + i];
        const float2 a = make_float2((float)(int8_t)(x & 0xFFu) * s, (float)(int8_t)((x >> 8) & 0xFFu) * s);
        const float2 b = make_float2((float)(int8_t)((x >> 16) & 0xFFu) * s, (float)(int8_t)(x >> 24) * s);
        OutPair<OT>::put(out, 2 * i, a, 0u);
        OutPair<OT>::put(out, 2 * i + 1, b, 0u);
    }
}

template <int D, int BITS, typename OT>
__global__ void __launch_bounds__(kWriteThreads, ReadSmem<D, BITS, OT>::kBlocks) read_kernel(const __grid_constant__ ReadParams p) {
    using Sh = ReadShape<BITS>;
    using Sm = ReadSmem<D, BITS, OT>;
    constexpr int TPV = Sh::kTpv, TV = Sh::kTileVecs, RB = Sm::RB, RW = RB / 4;
    extern __shared__ __align__(128) uint8_t smem[];
    // The cache and the slots may come from the previous kernel.  No dependent starts early.
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int vl = lane / TPV, part = lane % TPV;
    uint8_t* wbuf = smem + warp * Sm::kPerWarp;
    uint8_t* obuf = wbuf + 2 * Sm::kIn;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sm::kBars) + warp * 2;
    uint32_t* mask = reinterpret_cast<uint32_t*>(smem + Sm::kMask);
    if (lane == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        fence_mbar_init();
    }
    for (int j = tid; j < (BITS == 8 ? 0 : D / 2); j += kWriteThreads) {
        const float s0 = p.signs[2 * j], s1 = p.signs[2 * j + 1];
        mask[j] = ((__float_as_uint(s0) >> 31) << 15) | (__float_as_uint(s1) & 0x80000000u);
        if (blockIdx.x == 0 && ((fabsf(s0) != 1.0f) || (fabsf(s1) != 1.0f))) count_status(p.status, 4);
    }
    __syncthreads();

    const uint32_t H = (uint32_t)p.H;
    const int hshift = (H & (H - 1)) == 0 ? __ffs(H) - 1 : -1;
    const uint32_t nplane = (uint32_t)p.num_tokens * H, nvec = 2 * nplane;
    const uint32_t ntiles = (nvec + TV - 1) / TV;
    const uint32_t gwarp = blockIdx.x * kWriteWarps + warp, nwarps = gridDim.x * kWriteWarps;
    const bool grouped = hshift >= 0 && H <= (uint32_t)TV && (H * RB) % 16 == 0;
    auto split = [&](uint32_t v, uint32_t& tok, uint32_t& h, uint32_t& pl) {
        pl = v >= nplane ? 1u : 0u;
        const uint32_t u = v - (pl ? nplane : 0u);
        tok = hshift >= 0 ? u >> hshift : u / H;
        h = u - tok * H;
    };
    // byte offset of vector v's row in the cache, or -1 (a negative slot, or one outside the cache)
    auto row_at = [&](uint32_t v, bool count) -> int64_t {
        uint32_t tok, h, pl;
        split(v, tok, h, pl);
        const int64_t slot = __ldg(p.slots + tok);
        if (slot < 0 || slot >= p.num_slots) {
            if (count && slot >= 0 && pl == 0 && h == 0) count_status(p.status, 0);
            return -1;
        }
        const int64_t blk = slot / kBlockSize, off = slot % kBlockSize;
        return (((blk * 2 + pl) * kBlockSize + off) * (int64_t)H + h) * RB;
    };

    // Start the copy of a tile's packed rows; returns whether lane l < TV's vector has a row.  The buffer's
    // mbarrier completes once every row is there.
    auto prefetch = [&](uint32_t tile, uint8_t* buf, uint64_t* bar) -> bool {
        const uint32_t v0 = tile * TV;
        const bool mine = lane < TV && v0 + lane < nvec;
        const int64_t at = mine ? row_at(v0 + lane, true) : -1;
        if (grouped) {
            const bool lead = at >= 0 && (lane & (H - 1)) == 0;
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, lead)) * H * (uint32_t)RB;
            if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (lead) bulk_copy_g2s(buf + lane * RB, p.cache + at, H * (uint32_t)RB, bar, policy_evict_first());
        } else {
            uint32_t* dst = reinterpret_cast<uint32_t*>(buf);
            for (int i0 = 0; i0 < TV * RW; i0 += 32) {   // whole warps: the offsets come from other lanes
                const int i = i0 + lane, r = min(i / RW, TV - 1);
                const int64_t a = __shfl_sync(0xffffffffu, at, r);
                if (i < TV * RW && a >= 0) dst[i] = __ldg(reinterpret_cast<const uint32_t*>(p.cache + a) + (i - r * RW));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        }
        return at >= 0;
    };

    const uint32_t my_tiles = gwarp < ntiles ? (ntiles - gwarp - 1) / nwarps + 1 : 0u;
    uint32_t tile = gwarp;
    bool have_next = my_tiles > 0 ? prefetch(tile, wbuf, &bars[0]) : false;
    uint32_t it = 0;
    bool waited_out = false;
    for (; it < my_tiles; ++it, tile += nwarps) {
        const uint8_t* cur = wbuf + (it & 1) * Sm::kIn;
        const bool have = have_next;
        __syncwarp();   // the other buffer's rows have been read
        if (it + 1 < my_tiles) have_next = prefetch(tile + nwarps, wbuf + ((it + 1) & 1) * Sm::kIn, &bars[(it + 1) & 1]);
        if (__any_sync(0xffffffffu, !mbar_wait(&bars[it & 1], (it >> 1) & 1u))) {
            if (lane == 0) count_status(p.status, 3);
            waited_out = true;
            break;
        }
        const bool live = __shfl_sync(0xffffffffu, (int)have, vl) != 0;
        const uint32_t* row = reinterpret_cast<const uint32_t*>(cur + vl * RB);
        uint8_t* orow = obuf + vl * Sm::kOutRow;
        auto staging_free = [&] {   // the staged rows of the previous tile have left
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
        };
        if constexpr (BITS == 8) {
            const float s = live ? __uint_as_float(row[D / 4]) : 0.0f;
            staging_free();
#pragma unroll 8
            for (int e = 0; e < D; e += 16 / (int)sizeof(OT)) {
                uint32_t o[4];
                decode_int8_words<D, OT>(row, e, s, o);
                *reinterpret_cast<uint4*>(orow + e * sizeof(OT)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        } else {
            constexpr int OWD = out_words<OT>(D / 2);
            uint32_t o[OWD];
            if constexpr (BITS == 4) decode_half<D, OT>(row, mask, part, p.c, live, o);
            else decode_half_int2<D, OT>(row, mask + part * (D / 4), part, p.c, live, o);
            staging_free();
            // INT4: groups of 16 pairs, the thread's in every second group; INT2: its half of the row
            constexpr int kGroup = BITS == 4 ? out_words<OT>(32) : OWD;   // words
#pragma unroll
            for (int g = 0; g < OWD / kGroup; ++g) {
                uint4* dst = reinterpret_cast<uint4*>(orow + (2 * g + part) * (kGroup * 4));
#pragma unroll
                for (int i = 0; i < kGroup / 4; ++i) {
                    const uint32_t* q = o + g * kGroup + 4 * i;
                    dst[i] = make_uint4(q[0], q[1], q[2], q[3]);
                }
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // staged rows -> bulk store
        __syncwarp();
        const uint32_t v = tile * TV + lane;   // lane i < TV stores row i
        if (lane < TV && v < nvec) {
            const bool second = v >= nplane;
            uint8_t* dst = static_cast<uint8_t*>(second ? p.v_out : p.k_out) +
                           (uint64_t)(second ? v - nplane : v) * (D * sizeof(OT));
            bulk_store_s2g(dst, obuf + lane * Sm::kOutRow, D * sizeof(OT));
        }
    }
    if (waited_out && it + 1 < my_tiles) (void)mbar_wait(&bars[(it + 1) & 1], ((it + 1) >> 1) & 1u);
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <int D, int BITS, typename OT>
cudaError_t launch_read_t(const ReadParams& p, cudaStream_t stream) {
    using Sm = ReadSmem<D, BITS, OT>;
    constexpr int TV = ReadShape<BITS>::kTileVecs;
    const int64_t ntiles = (p.num_tokens * p.H * 2 + TV - 1) / TV;
    const int64_t blocks = (ntiles + kWriteWarps - 1) / kWriteWarps;
    cudaError_t err = opt_in_smem<read_kernel<D, BITS, OT>>(Sm::kBytes);
    if (err != cudaSuccess) return err;
    const int64_t cap = (int64_t)num_sms() * Sm::kBlocks;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < cap ? blocks : cap));
    cfg.blockDim = dim3(kWriteThreads);
    cfg.dynamicSmemBytes = Sm::kBytes;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, read_kernel<D, BITS, OT>, p);
}

template <int D, int BITS>
cudaError_t read_by_out(const ReadParams& p, DType out_dt, cudaStream_t s) {
    switch (out_dt) {
        case DType::F16: return launch_read_t<D, BITS, __half>(p, s);
        case DType::BF16: return launch_read_t<D, BITS, __nv_bfloat16>(p, s);
        default: return launch_read_t<D, BITS, float>(p, s);
    }
}

}  // namespace
}  // namespace kvi4

namespace kvi4 {

cudaError_t launch_read(const ReadParams& p, int bits, int head_size, DType out_dt, cudaStream_t s) {
    const bool wide = head_size == 128;
    if (bits == 8) return wide ? read_by_out<128, 8>(p, out_dt, s) : read_by_out<64, 8>(p, out_dt, s);
    if (bits == 2) return wide ? read_by_out<128, 2>(p, out_dt, s) : read_by_out<64, 2>(p, out_dt, s);
    return wide ? read_by_out<128, 4>(p, out_dt, s) : read_by_out<64, 4>(p, out_dt, s);
}

}  // namespace kvi4
