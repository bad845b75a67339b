// Attention of a decode batch over the cached prefix that its sequences share: every query row of the
// batch against the same keys, so the prefix is read and dequantised once per 128 query rows instead of
// once per sequence, and the products fill the tensor cores' tiles although each sequence has one query.
//
// The mathematics is the chunked prefill's (attn_prefill.cuh: rotated queries as fp16 high + low halves,
// S = Q' (K - zp)^T, logit = S s'_K k0 2^-e, weights 2^(logit - m + 127 - E) s'_V, O += P_w (V - zp), all
// accumulated in fp32), with these differences: a row is one (query token, q head) of any sequence and sees
// the prefix keys below its own limit (its sequence's length, when that ends inside the prefix; a padding
// row sees none), and a CTA writes its key range's partial (reference maximum m in log2 units, sum l,
// unnormalised O, still rotated), which the combine merges with the suffix's; the weights are raised (kPxRaise).
//
// Grid: (row tiles of 128 / G tokens) x kv heads x splits of the prefix's 128-key tiles, one CTA per SM.
// The splits fill the SMs when the batch alone does not (prefix_splits).
//
// Warp roles (640 threads): warps 0-7 own the rows (rotation, softmax, partials), warps 8-11 dequantise the K
// rows and warps 12-15 the V rows of a tile (one row per thread), warp 16 issues the MMAs, warps 17-18 stage
// packed rows four tiles ahead, warp 19 is idle (it completes the last warpgroup, which the register split
// needs).  The registers come from a setmaxnreg split: 136 for the rows, 72 for the dequantisation, 64 for the
// rest, together what 640 threads are launched with at 96.
//
// What bounds it (clock stamps in an instrumented copy, cycles per 128-key tile, d 128): about 3 000 a tile, of
// which the tensor pipe computes 1 600 (24 MMAs of 66; 32 with the weights in two halves).  A tile goes round the
// chain S (1 230 to issue) -> softmax (1 970, among the dequantisation's instructions) -> P.V (600) -> the S after
// next, which takes the same of the two S buffers, and each hand-over costs 300-700 until the MMAs issued have
// run and the other side is awake; tensor memory is full (two S, O, the queries' halves), so there is no third
// buffer.  Beside it K's and V's rows of a tile take 700 and 1 000.  Shared memory is what makes the MMAs run late:
// its data pipe is 83% busy (29% the MMAs' operands, 54% loads and stores: per tile 512 cycles of scales for the
// softmax, 512 of converted rows, 320 of packed ones).  What the steps gave on 128 sequences, 131 072
// shared tokens, 64 q / 8 kv heads (961 us at first): block ids looked up four tiles ahead and copies without a
// spilled table, descriptors in uniform registers: 812; one prescale per CTA, so that one FMA forms the
// exponent, and a fixed MMA order: 775; a walker grid for the tokens behind the prefix alone: 729; packed rows by
// TMA boxes instead of 16-byte copies: 696; polling in the chain's waits: 665; V rows read without bank conflicts:
// 661.  Since then blocks that hold keys are told from rows of zeros, the weights are raised and each row has its
// own V exponent: 679.  Tried and dropped: forming the weights before the maxima are known (no gain), 16 softmax
// warps with half of the keys each (923), output rows staged for bulk stores (no gain), S as two products of 64
// keys, so that one of them need not wait for P.V (713 against 683), weights handed over in two halves (674 against
// 665).
#pragma once

#include "attn_prefill.cuh"

namespace kvi4 {
namespace {

constexpr int kPxDequantWarp = kPfSoftmaxWarps;          // K group, then the V group
constexpr int kPxMmaWarp = kPxDequantWarp + 8;
constexpr int kPxLoadWarp = kPxMmaWarp + 1;              // one per plane (K, V)
constexpr int kPxThreads = (kPxMmaWarp + 4) * 32;
constexpr int kPxPolls = 128;                            // about 4 000 cycles, a tile and a bit
// Binades that a row's largest V scale may pass its reference exponent by, and the power of two the weights are
// raised by: w < 2^(kPfLazyMax + 0 + 1 + 6), half of fp16's range.  fp16's smallest step then stands for 2^-30 of
// the reference's weight.  (Without the raise it was 2^-24, and the weights of 2^16 keys some 25 binades below a
// dominant one, together 2^-9 of the sum, were lost from the output: a CTA's range can be the whole prefix, and it
// has one reference.)  A maximum that may trail less, 4 binades for a raise of 10, moves more often: 12% of the
// large calls with strong key channels.
constexpr uint32_t kPxLazyExp = 0;
constexpr int kPxRaise = 6;
constexpr int kPxLaunchRegs = 96, kPxRowRegs = 136, kPxDequantRegs = 72, kPxOtherRegs = 64;
static_assert(kPxRowRegs * 256 + kPxDequantRegs * 256 + kPxOtherRegs * 128 == kPxLaunchRegs * kPxThreads, "register split");

// Shared memory: the prefill's tiles and staging, then this kernel's own records and barriers.
template <int D>
struct PxLayout {
    using Pf = PfLayout<D>;
    static constexpr uint32_t kTile = Pf::kTile;
    static constexpr uint32_t kRaw = Pf::kRaw;
    static constexpr uint32_t kChunks = Pf::kChunks, kWindow = Pf::kWindow;
    static constexpr uint32_t kPlane = kPfKeys * kWindow * 4;                    // one plane of a staged tile
    static constexpr uint32_t kSk = kRaw + kPfRawStages * 2 * kPlane;            // [kring][128] f32 s'_K * k0
    static constexpr uint32_t kDeadF = kSk + kPfKRing * kPfKeys * 4;             // [kring][4] u32: positions with no key, one bit each
    static constexpr uint32_t kSv = kDeadF + kPfKRing * 4 * 4;                   // [pairs][128] f32 s'_V
    static constexpr uint32_t kEblk = kSv + kPfPairs * kPfKeys * 4;              // [pairs][4] per-warp max V exponent
    static constexpr uint32_t kQexp = kEblk + kPfPairs * 4 * 4;                  // u32: first usable row and its exponent
    static constexpr uint32_t kHeld = kQexp + 16;                                // [stages] u32: blocks of a staged tile that hold keys
    static constexpr uint32_t kRs = kHeld + kPfRawStages * 4;                    // [128] f32 2^-d of each row's own prescale
    static constexpr uint32_t kSignBits = kRs + 128 * 4;                         // [D / 32] u32
    static constexpr uint32_t kBars = (kSignBits + D / 8 + 7u) & ~7u;
    // k_full[kring], k_free[pairs], v_full[pairs], v_free[pairs], pv_done[2], s_full[2], p_full[2], q_ready,
    // flush, q_tma, rot_in, rot_done, q_max, raw_full[plane][stages], raw_free[plane][stages]
    static constexpr int kNumBars = kPfKRing + 3 * kPfPairs + 6 + 6 + 4 * kPfRawStages;
    static constexpr uint32_t kTmemSlot = kBars + kNumBars * 8;
    static constexpr uint32_t kFlags = kTmemSlot + 4;
    static constexpr uint32_t kBytes = kFlags + 4 + 1024;                        // + alignment slack
};

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// The CTA's query prescale exponent from its first usable row (row << 8 | biased exponent of its largest
// |v|; all ones: none): that row's to [2^7, 2^8), within the range a key's scale can take up.
__device__ __forceinline__ int rows_exponent(uint32_t first) {
    return first == 0xFFFFFFFFu ? 0 : max(-60, min(60, 7 + 127 - (int)(first & 0xFFu)));
}

// Key of V thread i (see the dequantisation): of a group of 16 keys 8a + 2b + c (rows 4b + 2a + c), the first
// eight threads take a = b / 2, the others the other half.
__host__ __device__ constexpr int v_key(int i) {
    const int b = (i >> 1) & 3, a = (b >> 1) ^ ((i >> 3) & 1);
    return (i & ~15) + 8 * a + 2 * b + (i & 1);
}
constexpr bool v_keys_spread() {
    for (int i = 0; i < 128; i += 8) {
        unsigned keys = 0, rows = 0;
        for (int j = i; j < i + 8; ++j) {
            keys |= 1u << (v_key(j) & 7);
            rows |= 1u << (slot_of_column(v_key(j)) & 7);
        }
        if (keys != 255u || rows != 255u) return false;
    }
    return true;
}
static_assert(v_keys_spread(), "eight neighbours, eight remainders");

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

template <int REGS>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS)); }
template <int REGS>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS)); }

// OPTS: the call has logit options; every tile then takes the masked path, which applies them.
// TWO: the weights too are carried as high + low halves (the low ones over S's last 64 columns), as the walker
// carries them with up to four query heads per kv head.  One fp16 weight per key errs by up to 2^-11, as much
// as the rounding of an fp16 output: results were 1.4-1.7 times as far off as that rounding alone.  With eight
// heads per kv head the walker has one half, and so has this kernel then for a bf16 output, whose error against
// 64 bits it raises by a hundredth (0.00167 to 0.00169 in the 2-norm).  The second half costs 11% (four heads per
// kv head) or 14% (eight) of a large call.
template <int D, typename QT, bool OPTS, bool TWO>
__global__ void __launch_bounds__(kPxThreads, 1) prefix_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap qmap,
                                                                  const __grid_constant__ CUtensorMap cmap) {
    using Gm = Geo<D>;
    using Ly = PxLayout<D>;
    using Tm = PfTmem<D>;
    constexpr int KSTEPS = D / 16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch_dependents();   // the combine waits for this grid before it reads anything

    const int G = p.G, Hq = p.Hq, H = p.H;
    const int BQ = kPfRows / G;
    const int h = (int)(blockIdx.x % (unsigned)H), qt0 = (int)(blockIdx.x / (unsigned)H) * BQ;
    const int split = blockIdx.y;
    const int tiles_all = (p.px_len + kPfKeys - 1) / kPfKeys;
    const int kt0 = (int)((int64_t)tiles_all * split / p.px_splits), kt1 = (int)((int64_t)tiles_all * (split + 1) / p.px_splits);
    const bool boxes = H % 4 == 0;   // rows of a multiple of 16 bytes: TMA loads packed rows (see the loaders)
    const int nkt = kt1 - kt0;   // at least one: the host takes no more splits than tiles

    float* sk = reinterpret_cast<float*>(smem + Ly::kSk);
    float* sv = reinterpret_cast<float*>(smem + Ly::kSv);
    uint32_t* eblkw = reinterpret_cast<uint32_t*>(smem + Ly::kEblk);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Ly::kBars);
    uint64_t* k_full = bars;                    // [kring] K tile and scales of tile j (128 arrivals)
    uint64_t* k_free = k_full + kPfKRing;       // [pairs] K tile j % 2 read by S of tile j (commit)
    uint64_t* v_full = k_free + kPfPairs;       // [pairs] V tile and scales of tile j (128 arrivals)
    uint64_t* v_free = v_full + kPfPairs;       // [pairs] V tile j % 2 read by P.V of tile j (commit)
    uint64_t* pv_done = v_free + kPfPairs;      // [2] P.V of tile j done (commit): S buffer j % 2 and O free
    uint64_t* s_full = pv_done + 2;             // [2] S of the tile in tensor memory (commit)
    uint64_t* p_full = s_full + 2;              // [2] P of the tile in tensor memory (256 arrivals)
    uint64_t* q_ready = p_full + 2;             // queries in tensor memory, staging free (256 arrivals)
    uint64_t* flush = q_ready + 1;              // the MMA thread's last commit (teardown)
    uint64_t* q_tma = flush + 1;                // the CTA's query rows in shared memory (bytes)
    uint64_t* rot_in = q_tma + 1;               // the rotation matrix in shared memory (256 arrivals)
    uint64_t* rot_done = rot_in + 1;            // the rotated queries in tensor memory (commit)
    uint64_t* q_max = rot_done + 1;             // the rows' exponent is known (256 arrivals)
    uint64_t* raw_full = q_max + 1;             // [plane][stages] packed rows of a key tile landed (one arrival and bytes, or and 32 lanes)
    uint64_t* raw_free = raw_full + 2 * kPfRawStages;   // [plane][stages] that plane converted (128 arrivals)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly::kTmemSlot);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Ly::kFlags);
    uint32_t* deadf = reinterpret_cast<uint32_t*>(smem + Ly::kDeadF);
    uint32_t* qexp = reinterpret_cast<uint32_t*>(smem + Ly::kQexp);
    uint32_t* held = reinterpret_cast<uint32_t*>(smem + Ly::kHeld);

    if (threadIdx.x == 0) {
        for (int b = 0; b < kPfKRing; ++b) mbar_init(&k_full[b], 128);
        for (int b = 0; b < kPfPairs; ++b) {
            mbar_init(&k_free[b], 1);
            mbar_init(&v_full[b], 128);
            mbar_init(&v_free[b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&pv_done[b], 1);
            mbar_init(&s_full[b], 1);
            mbar_init(&p_full[b], kPfSoftmaxThreads);
        }
        mbar_init(q_ready, kPfSoftmaxThreads);
        mbar_init(flush, 1);
        mbar_init(q_tma, 1);
        mbar_init(rot_in, kPfSoftmaxThreads);
        mbar_init(rot_done, 1);
        mbar_init(q_max, kPfSoftmaxThreads);
        *qexp = 0xFFFFFFFFu;
        for (int i = 0; i < 2 * kPfRawStages; ++i) {
            mbar_init(&raw_full[i], boxes ? 1 : 33);
            mbar_init(&raw_free[i], 128);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    // Metadata of this thread's two rows, loaded early and at once: (query start, end, length) as they are
    // when every sequence before a token has one query.
    struct RowMeta {
        int q0, q1, len;
    };
    auto row_meta = [&](int tok) -> RowMeta {
        const int b = min(tok, p.num_seqs - 1);
        return RowMeta{__ldg(p.qsl + b), __ldg(p.qsl + b + 1), __ldg(p.seq_lens + b)};
    };
    RowMeta meta_a = {}, meta_b = {};
    if (warp < kPfSoftmaxWarps) {
        const int r = 32 * (warp & 3) + 16 * (warp >> 2) + (lane >> 2);
        meta_a = row_meta(qt0 + r / G);
        meta_b = row_meta(qt0 + (r + 8) / G);
    }
    // cached tokens of a query token's sequence
    auto context = [&](int tok, const RowMeta& mt) -> int {
        if ((int64_t)tok >= p.num_q_tokens) return 0;
        int len = mt.len;
        if (tok >= p.num_seqs || mt.q0 != tok || mt.q1 != tok + 1) {   // some sequences have no query: search
            int lo = 0, hi = p.num_seqs;   // the last b with qsl[b] <= tok
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(p.qsl + mid) <= tok) lo = mid;
                else hi = mid;
            }
            if (__ldg(p.qsl + lo) != tok || __ldg(p.qsl + lo + 1) != tok + 1) return 0;
            len = __ldg(p.seq_lens + lo);
        }
        return max(0, min(len, p.len_cap));
    };
    uint32_t* signbits = reinterpret_cast<uint32_t*>(smem + Ly::kSignBits);
    if (threadIdx.x < D) {   // whole warps (D is a multiple of 32)
        const uint32_t m = __ballot_sync(0xffffffffu, p.signs[threadIdx.x] < 0.0f);
        if (lane == 0) signbits[warp] = m;
    }
    if (warp == kPxMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    uint8_t* tiles = smem;   // [K0][V0][K1][V1]
    auto ktile = [&](int b) { return tiles + (uint32_t)b * 2u * Ly::kTile; };
    auto vtile = [&](int b) { return tiles + (uint32_t)b * 2u * Ly::kTile + Ly::kTile; };
    // a wait that runs out counts once and winds the CTA down
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (*abort_flag) return false;
        if (mbar_wait(bar, parity)) return true;
        if (atomicExch(const_cast<int*>(abort_flag), 1) == 0) count_status(p.status, 3);
        return false;
    };
    // the same in the chain S -> weights -> P.V -> next S, where waking a suspended warp would add to every tile:
    // polled first
    auto soon = [&](uint64_t* bar, uint32_t parity) -> bool {
        for (int i = 0; i < kPxPolls; ++i)
            if (mbar_test_wait(bar, parity)) return true;
        return wait(bar, parity);
    };

    if (warp < kPfSoftmaxWarps) {
        more_registers<kPxRowRegs>();
        // ================================================================ rows: softmax + partials
        // Rows and tensor-memory layout as in the prefill: warp w owns the 16 rows 32 (w % 4) +
        // 16 (w / 4) ..; thread (g, t) holds rows ra = rbase + g and rb = ra + 8 and, of every group of
        // 8 columns, columns 2t and 2t + 1.
        const int rbase = 32 * (warp & 3) + 16 * (warp >> 2);
        const int t4 = lane & 3;
        const int ra = rbase + (lane >> 2), rb = ra + 8;
        const uint32_t trow = tmem + ((uint32_t)rbase << 16);
        // ---- the rotation matrix B[p][k] = sign_k (-1)^popcount(n(p) & k) in pair 1's V tile
        {
            constexpr int kRowChunks = D / 8, kThreadsPerRow = kPfSoftmaxThreads / D, kChunksPerThread = kRowChunks / kThreadsPerRow;
            uint8_t* qb = vtile(1);
            const uint32_t one = std::is_same<QT, __nv_bfloat16>::value ? 0x3F80u : 0x3C00u;
            const int prow = threadIdx.x / kThreadsPerRow;
            const int n = dim_of_column(slot_of_column(prow));
            uint32_t par8 = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) par8 |= ((uint32_t)__popc(n & j) & 1u) << j;
#pragma unroll
            for (int it = 0; it < kChunksPerThread; ++it) {
                const int k8 = (threadIdx.x % kThreadsPerRow) * kChunksPerThread + it;
                const uint32_t sb = (signbits[k8 / 4] >> (8 * (k8 % 4))) & 0xFFu;
                const uint32_t neg = par8 ^ sb ^ ((__popc(n & (8 * k8)) & 1) ? 0xFFu : 0u);
                uint32_t w[4];
                pm1_words(neg, one, w);
                *reinterpret_cast<uint4*>(qb + (uint32_t)(k8 / 8) * (uint32_t)(D * 128) + swz128((uint32_t)prow, (uint32_t)(k8 % 8))) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // generic writes -> tensor core reads
            mbar_arrive(rot_in);
        }
        // ---- each row's limit: keys [0, vis) of the prefix, from its token's sequence
        // A row that sees none (a padding row, or one past the batch) goes along as if it saw all, so that it
        // does not put its warp on the masked path, and its partial is empty at the end; a warp of such rows
        // leaves its weights unwritten.
        const int len_a = context(qt0 + ra / G, meta_a), len_b = context(qt0 + rb / G, meta_b);
        int vis_a = min(len_a, p.px_len), vis_b = min(len_b, p.px_len);
        const bool none_a = vis_a == 0, none_b = vis_b == 0;
        if (none_a) vis_a = p.px_len;
        if (none_b) vis_b = p.px_len;
        const bool idle = __all_sync(0xffffffffu, none_a && none_b);
        // ---- a power-of-two prescale of the rows, then fp16 high + low halves into tensor memory.  One exponent
        // serves the CTA, so that 2^-e sits in the keys' scales and not in a factor per row: it brings the first
        // usable row's max |v| (finite, not zero, of a row that sees keys) to [2^7, 2^8).  A row whose largest value
        // then lies in [2^-2, 2^15) keeps 22 bits of it (its elements err by 2^-25 at most, or 2^-23 relative); any
        // other (2^9 away, infinite) takes a further power of two of its own.  So a row's values reach another's
        // results in the last bits alone.
        float* rs = reinterpret_cast<float*>(smem + Ly::kRs);   // what a row's S is multiplied with
        bool own_a = false, own_b = false;
        bool ok = wait(rot_done, 0);
        if (__all_sync(0xffffffffu, ok)) {
            tc_fence_after();
            float v[D / 2];   // v[4i], v[4i + 1]: row a, columns 8i + 2t, + 1; v[4i + 2], v[4i + 3]: row b
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 64) tmem_ld_q8(trow + Tm::kS0 + c0, reinterpret_cast<uint32_t*>(v) + c0 / 2);
            tmem_ld_wait();
            // the rows' largest magnitudes by their bits (a NaN's are above infinity's)
            uint32_t mxa = 0u, mxb = 0u;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                mxa = max(mxa, max(__float_as_uint(v[4 * i]) & 0x7FFFFFFFu, __float_as_uint(v[4 * i + 1]) & 0x7FFFFFFFu));
                mxb = max(mxb, max(__float_as_uint(v[4 * i + 2]) & 0x7FFFFFFFu, __float_as_uint(v[4 * i + 3]) & 0x7FFFFFFFu));
            }
            mxa = max(mxa, __shfl_xor_sync(0xffffffffu, mxa, 1));
            mxb = max(mxb, __shfl_xor_sync(0xffffffffu, mxb, 1));
            mxa = max(mxa, __shfl_xor_sync(0xffffffffu, mxa, 2));
            mxb = max(mxb, __shfl_xor_sync(0xffffffffu, mxb, 2));
            const int xa = (int)(mxa >> 23), xb = (int)(mxb >> 23);   // biased exponents
            if (t4 == 0) {
                if (!none_a && xa > 0 && xa < 255) atomicMin(qexp, (uint32_t)ra << 8 | (uint32_t)xa);
                if (!none_b && xb > 0 && xb < 255) atomicMin(qexp, (uint32_t)rb << 8 | (uint32_t)xb);
            }
            __syncwarp();
            mbar_arrive(q_max);
            ok = __all_sync(0xffffffffu, wait(q_max, 0));
            const int e = rows_exponent(*reinterpret_cast<volatile uint32_t*>(qexp));
            auto own = [&](int x) -> int {   // a row's further exponent
                const int y = x - 127 + e;
                return x == 0 || (y >= -2 && y <= 14) ? 0 : max(-126 - e, min(127 - e, 7 - y));
            };
            const int da = own(xa), db = own(xb);
            own_a = da != 0;
            own_b = db != 0;
            if (t4 == 0) {
                rs[ra] = exp2f((float)-da);
                rs[rb] = exp2f((float)-db);
            }
            __syncwarp();
            const float sca = exp2i(e + da), scb = exp2i(e + db);
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
                uint32_t hw[4], lw[4];
#pragma unroll
                for (int i = 2 * q; i < 2 * q + 2; ++i) {
                    split_f16x2(v[4 * i] * sca, v[4 * i + 1] * sca, hw[i & 1], lw[i & 1]);
                    split_f16x2(v[4 * i + 2] * scb, v[4 * i + 3] * scb, hw[2 + (i & 1)], lw[2 + (i & 1)]);
                }
                tmem_st_q1(trow + Tm::kQh + 8 * q, hw);
                tmem_st_q1(trow + Tm::kQl + 8 * q, lw);
            }
            tmem_st_wait();
        } else {
            ok = false;
        }
        tc_fence_before();
        mbar_arrive(q_ready);
        // Keys below this one need no mask; rows with a prescale of their own (rare) go with the masked ones.
        const int plain_vis = own_a || own_b ? 0 : min(vis_a, vis_b);
        // ---- the key tiles
        // Reference maxima m (log2 units) as the exponents' offsets off = 127 + raise - E - m; E = 127 and off = 0
        // until a row has a key (any).
        float off_a = 0.0f, off_b = 0.0f;
        bool any_a = false, any_b = false;
        float l_a = 0.0f, l_b = 0.0f;           // this thread's part of the sums of 2^(127+raise-E) p
        // Reference biased exponents of the V scales that the rows see (0: none yet).  Each row has its own: a key
        // behind its sequence's end, infinite perhaps, must not move it.
        uint32_t E_a = 0, E_b = 0;
        if (idle) {   // a loop of its own: the test in the loop below cost 3% of the whole call
            for (int j = 0; j < nkt && ok; ++j) {
                ok = wait(&s_full[j & 1], (uint32_t)(j >> 1) & 1u);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) mbar_arrive(&p_full[j & 1]);
            }
        }
        for (int j = idle ? nkt : 0; j < nkt && ok; ++j) {
            const int b = j & 1;
            const uint32_t ph = (uint32_t)(j >> 1) & 1u;
            const int kb = j % kPfPairs, kr = j % kPfKRing;
            ok = soon(&s_full[b], ph) && wait(&k_full[kr], (uint32_t)(j / kPfKRing) & 1u) &&
                 wait(&v_full[kb], (uint32_t)(j / kPfPairs) & 1u);
            if (__any_sync(0xffffffffu, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t scol = trow + (b ? Tm::kS1 : Tm::kS0);
            uint32_t s[64];   // s[4i], s[4i + 1]: row a, columns 8i + 2t, + 1; s[4i + 2], s[4i + 3]: row b
            tmem_ld_q8(scol, s);
            tmem_ld_q8(scol + 64, s + 32);
            tmem_ld_wait();
            // Exponents e = S s'_K k0 2^-e - m + 127 + raise - E (one FMA) against the references as they
            // are, and their row maxima; a reference that moves is added to them afterwards, which is rare.
            const int key0 = (kt0 + j) * kPfKeys;
            const float4* skb = reinterpret_cast<const float4*>(sk + kr * kPfKeys) + t4;   // columns 16q + (2t, 2t + 1, 8 + 2t, 9 + 2t)
            const bool clean = (deadf[kr * 4] | deadf[kr * 4 + 1] | deadf[kr * 4 + 2] | deadf[kr * 4 + 3]) == 0u &&
                               key0 + kPfKeys <= plain_vis;
            float bma = -INFINITY, bmb = -INFINITY;
            const uint32_t* eb4 = eblkw + kb * 4;
            const float4* svb = reinterpret_cast<const float4*>(sv + kb * kPfKeys) + t4;
            uint32_t eb_a = max(max(eb4[0], eb4[1]), max(eb4[2], eb4[3])), eb_b = eb_a;
            if (!OPTS && __all_sync(0xffffffffu, clean)) {   // every key live and visible to both rows, rs 1
                const float2 moa2 = make_float2(off_a, off_a), mob2 = make_float2(off_b, off_b);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float4 k4 = skb[4 * (i / 2)];
                    const float2 k2 = (i & 1) ? make_float2(k4.z, k4.w) : make_float2(k4.x, k4.y);
                    const float2 ea = fma_f32x2(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), k2, moa2);
                    const float2 eb = fma_f32x2(make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), k2, mob2);
                    s[4 * i] = __float_as_uint(ea.x);
                    s[4 * i + 1] = __float_as_uint(ea.y);
                    s[4 * i + 2] = __float_as_uint(eb.x);
                    s[4 * i + 3] = __float_as_uint(eb.y);
                    bma = max3(bma, ea.x, ea.y);
                    bmb = max3(bmb, eb.x, eb.y);
                }
            } else {
                const float rs_a = rs[ra], rs_b = rs[rb];
                const bool alibi = OPTS && (p.opts & kOptAlibi);
                const float sl_a = alibi ? __ldg(p.alibi + h * G + ra % G) * kLog2e : 0.0f;
                const float sl_b = alibi ? __ldg(p.alibi + h * G + rb % G) * kLog2e : 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float4 k4 = skb[4 * (i / 2)];
                    const float2 k2 = (i & 1) ? make_float2(k4.z, k4.w) : make_float2(k4.x, k4.y);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float kk = e ? k2.y : k2.x;
                        const int key = key0 + 8 * i + 2 * t4 + e;
                        const bool live = ((deadf[kr * 4 + i / 4] >> (8 * (i % 4) + 2 * t4 + e)) & 1u) == 0u;
                        float ea, eb;
                        if constexpr (OPTS) {   // on the log2 logit
                            ea = live && key < vis_a ? __uint_as_float(s[4 * i + e]) * rs_a * kk : -INFINITY;
                            eb = live && key < vis_b ? __uint_as_float(s[4 * i + 2 + e]) * rs_b * kk : -INFINITY;
                            ea = apply_opts(ea, key, len_a - 1, sl_a, p, len_a - 1) + off_a;
                            eb = apply_opts(eb, key, len_b - 1, sl_b, p, len_b - 1) + off_b;
                        } else {
                            ea = live && key < vis_a ? fmaf(__uint_as_float(s[4 * i + e]) * rs_a, kk, off_a) : -INFINITY;
                            eb = live && key < vis_b ? fmaf(__uint_as_float(s[4 * i + 2 + e]) * rs_b, kk, off_b) : -INFINITY;
                        }
                        s[4 * i + e] = __float_as_uint(ea);
                        s[4 * i + 2 + e] = __float_as_uint(eb);
                        bma = fmaxf(bma, ea);
                        bmb = fmaxf(bmb, eb);
                    }
                }
                if (__any_sync(0xffffffffu, key0 + kPfKeys > min(vis_a, vis_b))) {   // the V scales of the visible keys alone
                    uint32_t ma = 0u, mb = 0u;
#pragma unroll 1
                    for (int q = 0; q < 8; ++q) {
                        const float4 v4 = svb[4 * q];
                        const float v[4] = {v4.x, v4.y, v4.z, v4.w};   // keys 16q + (2t, 2t + 1, 8 + 2t, 9 + 2t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = key0 + 16 * q + 8 * (e >> 1) + 2 * t4 + (e & 1);
                            const uint32_t bits = __float_as_uint(v[e]) + 1u;   // the largest finite value stands for infinity
                            if (key < vis_a) ma = max(ma, bits);
                            if (key < vis_b) mb = max(mb, bits);
                        }
                    }
#pragma unroll
                    for (int off = 1; off < 4; off <<= 1) {
                        ma = max(ma, __shfl_xor_sync(0xffffffffu, ma, off));
                        mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, off));
                    }
                    eb_a = ma >> 23;
                    eb_b = mb >> 23;
                }
            }
            bma = fmaxf(bma, __shfl_xor_sync(0xffffffffu, bma, 1));
            bmb = fmaxf(bmb, __shfl_xor_sync(0xffffffffu, bmb, 1));
            bma = fmaxf(bma, __shfl_xor_sync(0xffffffffu, bma, 2));
            bmb = fmaxf(bmb, __shfl_xor_sync(0xffffffffu, bmb, 2));
            // the four threads of a row take the same decisions; a row without a reference takes the first one
            const float eoff_a = (float)(127 + kPxRaise - (int)(E_a ? E_a : 127u)), eoff_b = (float)(127 + kPxRaise - (int)(E_b ? E_b : 127u));
            const bool newE_a = E_a == 0u ? eb_a > 0u : eb_a > E_a + kPxLazyExp;
            const bool newE_b = E_b == 0u ? eb_b > 0u : eb_b > E_b + kPxLazyExp;
            const bool up_a = any_a ? bma > eoff_a + kPfLazyMax : bma > -INFINITY;
            const bool up_b = any_b ? bmb > eoff_b + kPfLazyMax : bmb > -INFINITY;
            if (__any_sync(0xffffffffu, up_a || up_b || newE_a || newE_b)) {
                const float da = up_a ? eoff_a - bma : 0.0f, db = up_b ? eoff_b - bmb : 0.0f;   // old reference - new one
                const float fm_a = up_a ? (any_a ? fast_exp2(da) : 0.0f) : 1.0f, fm_b = up_b ? (any_b ? fast_exp2(db) : 0.0f) : 1.0f;
                any_a = any_a || up_a;
                any_b = any_b || up_b;
                // rebase from 2^(127 - E) to 2^(127 - eb); 0 when the jump underflows
                auto rebase = [](uint32_t& E, uint32_t eb, float& fe, float& de) {
                    const uint32_t Eeff = E ? E : 127u;
                    fe = eb > Eeff + 126u ? 0.0f : __uint_as_float((127u + Eeff - eb) << 23);
                    de = (float)((int)Eeff - (int)eb);
                    E = eb;
                };
                float fe_a = 1.0f, fe_b = 1.0f, de_a = 0.0f, de_b = 0.0f;
                if (newE_a) rebase(E_a, eb_a, fe_a, de_a);
                if (newE_b) rebase(E_b, eb_b, fe_b, de_b);
                const float f_a = fm_a * fe_a, f_b = fm_b * fe_b;
                l_a *= f_a;
                l_b *= f_b;
                off_a += da + de_a;
                off_b += db + de_b;
                const float2 da2 = make_float2(da + de_a, da + de_a), db2 = make_float2(db + de_b, db + de_b);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 ea = add_f32x2(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), da2);
                    const float2 eb2 = add_f32x2(make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), db2);
                    s[4 * i] = __float_as_uint(ea.x);
                    s[4 * i + 1] = __float_as_uint(ea.y);
                    s[4 * i + 2] = __float_as_uint(eb2.x);
                    s[4 * i + 3] = __float_as_uint(eb2.y);
                }
                if (j > 0 && __any_sync(0xffffffffu, f_a != 1.0f || f_b != 1.0f)) {
                    // O must hold P.V of the previous tile before it is rescaled
                    ok = wait(&pv_done[(j - 1) & 1], (uint32_t)((j - 1) >> 1) & 1u);
                    if (__any_sync(0xffffffffu, !ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const float2 fa2 = make_float2(f_a, f_a), fb2 = make_float2(f_b, f_b);
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 8) {
                        uint32_t o[4];
                        tmem_ld_q1(trow + Tm::kO + c0, o);
                        tmem_ld_wait();
                        const float2 oa = mul_f32x2(make_float2(__uint_as_float(o[0]), __uint_as_float(o[1])), fa2);
                        const float2 ob = mul_f32x2(make_float2(__uint_as_float(o[2]), __uint_as_float(o[3])), fb2);
                        o[0] = __float_as_uint(oa.x);
                        o[1] = __float_as_uint(oa.y);
                        o[2] = __float_as_uint(ob.x);
                        o[3] = __float_as_uint(ob.y);
                        tmem_st_q1(trow + Tm::kO + c0, o);
                    }
                    tmem_st_wait();
                }
            }
            // p' = 2^e, w = p' s'_V as fp16 pairs over the first 64 S columns: the pair of columns 8i + 2t, + 1
            // goes to column 8 (i / 2) + 2t + i % 2 (the V tile holds its rows in the matching order)
            float2 lsa = make_float2(0.0f, 0.0f), lsb = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                uint32_t pw[4], pl[4];
                const float4 v4 = svb[4 * q];
#pragma unroll
                for (int i = 2 * q; i < 2 * q + 2; ++i) {
                    const float2 v2 = (i & 1) ? make_float2(v4.z, v4.w) : make_float2(v4.x, v4.y);
                    const float2 pa = make_float2(fast_exp2(__uint_as_float(s[4 * i])), fast_exp2(__uint_as_float(s[4 * i + 1])));
                    const float2 pb = make_float2(fast_exp2(__uint_as_float(s[4 * i + 2])), fast_exp2(__uint_as_float(s[4 * i + 3])));
                    lsa = add_f32x2(lsa, pa);
                    lsb = add_f32x2(lsb, pb);
                    const float2 wa = mul_f32x2(pa, v2), wb = mul_f32x2(pb, v2);
                    const int e = i & 1;
                    if constexpr (TWO) {
                        split_f16x2(wa.x, wa.y, pw[e], pl[e]);
                        split_f16x2(wb.x, wb.y, pw[2 + e], pl[2 + e]);
                    } else {
                        pw[e] = pack_f16x2(wa.x, wa.y);
                        pw[2 + e] = pack_f16x2(wb.x, wb.y);
                    }
                }
                tmem_st_q1(scol + 8 * q, pw);
                if constexpr (TWO) tmem_st_q1(scol + 64 + 8 * q, pl);
            }
            l_a += lsa.x + lsa.y;
            l_b += lsb.x + lsb.y;
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&p_full[b]);
        }
        // ---- the partial: (m, l 2^(E - 127 - raise), O 2^(E - 127 - raise)), O's columns in the tile's dimension order
        if (ok && nkt > 0) ok = wait(&pv_done[(nkt - 1) & 1], (uint32_t)((nkt - 1) >> 1) & 1u);
        tc_fence_after();
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
        const bool good = __all_sync(0xffffffffu, ok) && nkt > 0;
        // a row that met only NaN (its query or the keys are not finite) shows it: no maximum tells
        any_a = (any_a || l_a != l_a) && !none_a;
        any_b = (any_b || l_b != l_b) && !none_b;
        E_a = E_a ? E_a : 127u;   // none: only rows of zeros
        E_b = E_b ? E_b : 127u;
        const float es_a = __uint_as_float(E_a << 23) * exp2i(-kPxRaise), es_b = __uint_as_float(E_b << 23) * exp2i(-kPxRaise);
        const float m_a = any_a ? (float)(127 + kPxRaise - (int)E_a) - off_a : kNegBig;
        const float m_b = any_b ? (float)(127 + kPxRaise - (int)E_b) - off_b : kNegBig;
        const int64_t rows = p.num_q_tokens * Hq;
        auto record = [&](int r) -> int64_t { return (int64_t)split * rows + (int64_t)(qt0 + r / G) * Hq + h * G + r % G; };
        auto in_batch = [&](int r) -> bool { return (int64_t)(qt0 + r / G) < p.num_q_tokens; };
        if (t4 == 0) {
            if (in_batch(ra)) reinterpret_cast<float2*>(p.px_ml)[record(ra)] = any_a && good ? make_float2(m_a, l_a * es_a) : make_float2(kNegBig, 0.0f);
            if (in_batch(rb)) reinterpret_cast<float2*>(p.px_ml)[record(rb)] = any_b && good ? make_float2(m_b, l_b * es_b) : make_float2(kNegBig, 0.0f);
        }
        const bool full_a = good && any_a, full_b = good && any_b, in_a = in_batch(ra), in_b = in_batch(rb);
        float* oa_row = p.px_o + (in_a ? record(ra) : 0) * D + 2 * t4;
        float* ob_row = p.px_o + (in_b ? record(rb) : 0) * D + 2 * t4;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[16];
            if (good) {
                tmem_ld_q4(trow + Tm::kO + c0, o);
                tmem_ld_wait();
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 oa = full_a ? make_float2(__uint_as_float(o[4 * i]) * es_a, __uint_as_float(o[4 * i + 1]) * es_a) : make_float2(0.0f, 0.0f);
                const float2 ob = full_b ? make_float2(__uint_as_float(o[4 * i + 2]) * es_b, __uint_as_float(o[4 * i + 3]) * es_b) : make_float2(0.0f, 0.0f);
                if (in_a) *reinterpret_cast<float2*>(oa_row + c0 + 8 * i) = oa;
                if (in_b) *reinterpret_cast<float2*>(ob_row + c0 + 8 * i) = ob;
            }
        }
    } else if (warp < kPxMmaWarp) {
        fewer_registers<kPxDequantRegs>();
        // ================================================================ dequantisation of key tiles
        const int pl = (warp - kPxDequantWarp) >> 2;      // 0: K rows, 1: V rows
        // This thread's key of every tile.  A V tile keeps its rows in the order the weights are laid out in, and V
        // threads take their keys in an order in which eight neighbours have keys, and rows, of eight different
        // remainders mod 8: the windows' reads and the swizzled rows' stores then hit no bank twice.
        const int i128 = (threadIdx.x - kPfSoftmaxThreads) & 127;
        const int k = pl ? v_key(i128) : i128;
        const uint32_t trow = (uint32_t)(pl ? slot_of_column(k) : k);
        constexpr int NW = D / 8 + 1;                     // words of a row: codes, then the scale word
        float k0 = p.c * p.softmax_scale * kLog2e;        // raw score -> log2 logit, with 2^-e once it is known
        // Word offset of this key's rows in their windows (the prefill's rule).  With 4 or 8 kv heads it is h % 4 for
        // the whole CTA, but a copy of the loop for each offset, without the 35 selects among a row's 270
        // instructions, made the large batch below 9% slower (762 us against 696).
        const int row_off = ((k % kBlockSize) * H + h) & 3;
        for (int j = 0; j < nkt; ++j) {
            const int kb = j % kPfPairs, st = j % kPfRawStages;
            bool ok = wait(&raw_full[pl * kPfRawStages + st], (uint32_t)(j / kPfRawStages) & 1u);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint4* win4 = reinterpret_cast<const uint4*>(smem + Ly::kRaw + (uint32_t)(st * 2 + pl) * Ly::kPlane) + k * Ly::kChunks;
            uint32_t kw[NW];
            {
                uint32_t wv[Ly::kWindow];
#pragma unroll
                for (int c = 0; c < (int)Ly::kChunks; ++c) {
                    const uint4 v = win4[c];
                    wv[4 * c] = v.x;
                    wv[4 * c + 1] = v.y;
                    wv[4 * c + 2] = v.z;
                    wv[4 * c + 3] = v.w;
                }
#pragma unroll
                for (int w = 0; w < NW + 1; ++w) wv[w] = (row_off & 2) ? wv[w + 2] : wv[w];
#pragma unroll
                for (int w = 0; w < NW; ++w) kw[w] = (row_off & 1) ? wv[w + 1] : wv[w];
            }
            const uint32_t blocks = pl == 0 ? held[st] : 0u;
            mbar_arrive(&raw_free[pl * kPfRawStages + st]);
            ok = j != 1 || wait(q_ready, 0);        // the query rows and the rotation matrix sat on pair 1
            if (ok && j >= kPfPairs) ok = wait(pl ? &v_free[kb] : &k_free[kb], (uint32_t)(j / kPfPairs - 1) & 1u);
            if (!__all_sync(0xffffffffu, ok)) break;
            uint8_t* t = pl ? vtile(kb) : ktile(kb);
            const uint32_t zp = kw[Gm::KW] & 15u;
            const uint32_t zl = zp_lo_half(zp) * 0x10001u, zh = zp_hi_half(zp) * 0x10001u;
#pragma unroll
            for (int w = 0; w < Gm::KW; ++w) {
                // code - zp of dimensions 8w + (0, 4), (1, 5), (2, 6), (3, 7): the tile order
                uint32_t o[4];
                unpack_word(kw[w], zl, zh, o);
                *reinterpret_cast<uint4*>(t + (uint32_t)(w / 8) * (kPfKeys * 128u) + swz128(trow, (uint32_t)(w % 8))) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
            if (pl == 0) {
                if (j == 0) {   // the rows' prescale
                    ok = wait(q_max, 0);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    k0 *= exp2i(-rows_exponent(*reinterpret_cast<volatile uint32_t*>(qexp)));
                }
                sk[(j % kPfKRing) * kPfKeys + slot_of_column(k)] = __uint_as_float(kw[Gm::KW] & 0xFFFFFFF0u) * k0;
                const uint32_t nokey = __ballot_sync(0xffffffffu, ((blocks >> (k / kBlockSize)) & 1u) == 0u);   // a row of zeros is a key, of logit 0
                if (lane == 0) deadf[(j % kPfKRing) * 4 + (warp & 3)] = nokey;
            } else {
                // finite, so that a weight of 0 stays one; an infinite scale shows in the exponent
                sv[kb * kPfKeys + (int)trow] = fminf(__uint_as_float(kw[Gm::KW] & 0xFFFFFFF0u), 3.4028234664e38f);
                const uint32_t wmax = __reduce_max_sync(0xffffffffu, kw[Gm::KW]);   // positive floats order like their bits
                if (lane == 0) eblkw[kb * 4 + (warp & 3)] = (wmax >> 23) & 0xFFu;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // generic writes -> tensor core reads
            mbar_arrive(pl ? &v_full[kb] : &k_full[j % kPfKRing]);
        }
    } else {
        fewer_registers<kPxOtherRegs>();
        if (warp == kPxLoadWarp || warp == kPxLoadWarp + 1) {
            // ============================================================ loads of packed rows
            // Each row's 16-byte-aligned window, keys past the prefix or in a block outside the cache zero-filled;
            // which blocks hold keys goes along with the K rows.  With 4 or 8 kv heads a token's rows are a multiple of 16 bytes and TMA
            // takes a block's windows at once; with 1 or 2 they are not, and the windows are 16-byte copies.
            // A pass moves kKeys whole windows (C lanes each; 30 of 32 lanes), so that a lane keeps its chunk
            // and the offsets are a few integer operations: a precomputed table of them spilled in this
            // warp's 64 registers and made a tile's copies 2 500 cycles.
            constexpr int C = Ly::kChunks, kKeys = 32 / C, kPasses = (kPfKeys + kKeys - 1) / kKeys;
            const int pl = warp - kPxLoadWarp;
            const int32_t* table = p.px_blocks;
            const int tok_stride = H * Gm::RB;
            const int64_t blk_stride = 2 * kBlockSize * (int64_t)tok_stride;
            const uint8_t* base = p.cache + (int64_t)pl * kBlockSize * tok_stride;
            const int ck = lane / C, cc = lane - ck * C;   // this lane's key of a pass and its chunk
            const bool mine = ck < kKeys;
            // Block ids of four tiles at a time, lane l's that of tile (group) + l / 8, block l % 8 of it
            // (-1: none, or not in the cache), loaded a group ahead: one tile ahead, the load's latency bounded every tile (the
            // K rows' wait was 2 100 of 3 600 cycles).
            const int nblocks = p.px_len / kBlockSize;
            auto inside = [&](int j) -> bool { return j + lane / 8 < nkt && (kt0 + j) * (kPfKeys / kBlockSize) + lane < nblocks; };
            auto lookup = [&](int j) -> int { return inside(j) ? __ldg(table + (kt0 + j) * (kPfKeys / kBlockSize) + lane) : -1; };
            int blk_next = lookup(0), blkv = -1;
            uint32_t blocks = 0;
            bool ok = true;
            int issued = 0;
            for (int j = 0; j < nkt && ok; ++j) {
                const int st = j % kPfRawStages;
                if ((j & 3) == 0) {
                    blkv = blk_next;
                    blk_next = lookup(j + 4);
                    if (blkv < 0 || (int64_t)blkv >= p.num_blocks) {
                        if (pl == 0 && h == 0 && qt0 == 0 && inside(j)) count_status(p.status, 1);
                        blkv = -1;
                    }
                    blocks = __ballot_sync(0xffffffffu, blkv >= 0);
                }
                if (j >= kPfRawStages) ok = wait(&raw_free[pl * kPfRawStages + st], (uint32_t)(j / kPfRawStages - 1) & 1u);
                if (!__all_sync(0xffffffffu, ok)) break;
                const uint32_t dst = smem_u32(smem + Ly::kRaw + (uint32_t)(st * 2 + pl) * Ly::kPlane);
                if (pl == 0 && lane == 0) held[st] = blocks >> (8 * (j & 3));   // this tile's: the low 8 bits; before the arrival below
                if (boxes) {
                    // one box [16 tokens][window bytes] per block; block -1 lies outside the tensor and reads as
                    // zeros, as do a last head's bytes past its token's rows
                    uint64_t* full = &raw_full[pl * kPfRawStages + st];
                    const int blk = __shfl_sync(0xffffffffu, blkv, (j & 3) * 8 + (lane & 7));
                    if (lane == 0) mbar_arrive_expect_tx(full, Ly::kPlane);
                    __syncwarp();
                    if (lane < kPfKeys / kBlockSize)
                        tma_load_4d(dst + (uint32_t)lane * (kBlockSize * Ly::kWindow * 4), &cmap, (h * Gm::RB) & ~15, 0, pl, blk, full);
                    issued = j + 1;
                    continue;
                }
#pragma unroll
                for (int t = 0; t < kPasses; ++t) {
                    const int key = t * kKeys + ck;
                    const int blk = __shfl_sync(0xffffffffu, blkv, (j & 3) * 8 + ((key / kBlockSize) & 7));
                    const bool live = blk >= 0;
                    const uint32_t row = (uint32_t)(h * Gm::RB + (key % kBlockSize) * tok_stride);
                    const uint8_t* src = base + (int64_t)(live ? blk : 0) * blk_stride + ((row & ~15u) + 16u * (uint32_t)cc);
                    if (mine && key < kPfKeys) cp_async16_zfill(dst + 16u * (uint32_t)(key * C + cc), src, live);
                }
                cp_async_arrive_noinc(&raw_full[pl * kPfRawStages + st]);
                if (lane == 0) mbar_arrive(&raw_full[pl * kPfRawStages + st]);
            }
            // no copy outlives the CTA
            cp_async_wait_all();
            for (int j = max(0, issued - kPfRawStages); j < issued; ++j)
                (void)mbar_wait(&raw_full[pl * kPfRawStages + j % kPfRawStages], (uint32_t)(j / kPfRawStages) & 1u);
        } else if (warp == kPxMmaWarp) {
            // ============================================================ the MMA issuer
            // S of tile t (its K tile dequantised, its S buffer read by P.V of tile t - 2), then P.V of tile t - 1
            // (its weights in tensor memory).  The whole warp runs the loop with uniform values and one elected
            // lane issues: descriptors are a base per tile pair plus a constant, in uniform registers (formed
            // by one lane alone, they cost 100 cycles per MMA against the 66 it takes).
            constexpr uint32_t idS = idesc_f16(kPfKeys, 0), idPV = idesc_f16(D, 1);
            const bool leader = elect_one();
            const uint64_t kd0 = smem_desc_sw128(smem_u32(ktile(0)), 16u, 1024u), kd1 = smem_desc_sw128(smem_u32(ktile(1)), 16u, 1024u);
            const uint64_t vd0 = smem_desc_sw128(smem_u32(vtile(0)), kPfKeys * 128u, 1024u);
            const uint64_t vd1 = smem_desc_sw128(smem_u32(vtile(1)), kPfKeys * 128u, 1024u);
            {
                if (leader) {
                    mbar_arrive_expect_tx(q_tma, Ly::kTile);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(ktile(1) + c * (kPfRows * 128), &qmap, 64 * c, h * G, qt0, q_tma);
                }
                __syncwarp();
                if (__all_sync(0xffffffffu, wait(q_tma, 0) && wait(rot_in, 0))) {
                    tc_fence_after();
                    constexpr uint32_t idR = std::is_same<QT, __nv_bfloat16>::value ? idesc_bf16(D, 0) : idesc_f16(D, 0);
                    const uint64_t rd = smem_desc_sw128(smem_u32(vtile(1)), 16u, 1024u);
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < KSTEPS; ++kk)
                            mma_ss(tmem + Tm::kS0, kd1 + (((kk / 4) * (kPfRows * 128) + (kk % 4) * 32) >> 4),
                                   rd + (((kk / 4) * (D * 128) + (kk % 4) * 32) >> 4), idR, kk > 0);
                        mma_commit(rot_done);
                    }
                    __syncwarp();
                }
            }
            auto issue_s = [&](int j) {
                const uint32_t sd = tmem + ((j & 1) ? Tm::kS1 : Tm::kS0);
                const uint64_t kd = (j & 1) ? kd1 : kd0;
                if (leader) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int kk = 0; kk < KSTEPS; ++kk)
                            mma_ts(sd, tmem + (half ? Tm::kQl : Tm::kQh) + 8u * kk,
                                   kd + (((kk / 4) * (kPfKeys * 128) + (kk % 4) * 32) >> 4), idS, half > 0 || kk > 0);
                    }
                    mma_commit(&s_full[j & 1]);
                    mma_commit(&k_free[j % kPfPairs]);
                }
                __syncwarp();
            };
            auto issue_pv = [&](int t) {
                const uint32_t pcol = tmem + ((t & 1) ? Tm::kS1 : Tm::kS0);
                const uint64_t vd = (t & 1) ? vd1 : vd0;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kPfKeys / 16; ++kk) {   // P of keys 16 kk .. 16 kk + 15 (in contraction order)
                        mma_ts(tmem + Tm::kO, pcol + 8u * kk, vd + ((kk * 16 * 128) >> 4), idPV, t > 0 || kk > 0);
                        if constexpr (TWO) mma_ts(tmem + Tm::kO, pcol + 64u + 8u * kk, vd + ((kk * 16 * 128) >> 4), idPV, true);
                    }
                    mma_commit(&pv_done[t & 1]);
                    mma_commit(&v_free[t % kPfPairs]);
                }
                __syncwarp();
            };
            static_assert(kPfPairs == 2, "one descriptor per pair");
            bool ok = __all_sync(0xffffffffu, nkt == 0 || wait(q_ready, 0));
            for (int t = 0; t <= nkt && ok; ++t) {
                if (t < nkt) {
                    ok = soon(&k_full[t % kPfKRing], (uint32_t)(t / kPfKRing) & 1u) &&
                         (t < 2 || soon(&pv_done[t & 1], (uint32_t)((t - 2) >> 1) & 1u));
                    if (!__all_sync(0xffffffffu, ok)) break;
                    tc_fence_after();
                    issue_s(t);
                }
                if (t > 0) {
                    ok = soon(&p_full[(t - 1) & 1], (uint32_t)((t - 1) >> 1) & 1u);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    tc_fence_after();
                    issue_pv(t - 1);
                }
            }
            // every MMA issued has completed before the CTA tears tensor memory down
            if (leader) mma_commit(flush);
            __syncwarp();
            (void)mbar_wait(flush, 0);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kPxMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
    // Complete only after the walker has: whoever waits for this kernel then also sees its partials.
    griddep_wait();
}

// The cache as bytes [block][plane][token][heads' rows], in boxes of one block's windows of one head (4 or 8 kv
// heads).  Block ids are int32, so a larger cache has no block past 2^31 that could be named.
template <int D>
cudaError_t cache_map(const AttnParams& p, CUtensorMap* map) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (enc == nullptr) return cudaErrorNotSupported;
    const cuuint64_t row = (cuuint64_t)p.H * Geo<D>::RB;
    const cuuint64_t blocks = (cuuint64_t)std::min<int64_t>(std::max<int64_t>(p.num_blocks, 1), (int64_t)1 << 31);
    const cuuint64_t dims[4] = {row, kBlockSize, 2, blocks};
    const cuuint64_t strides[3] = {row, row * kBlockSize, row * kBlockSize * 2};
    const cuuint32_t box[4] = {PxLayout<D>::kWindow * 4, kBlockSize, 1, 1};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(p.cache), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, typename QT, bool OPTS, bool TWO>
cudaError_t launch_prefix_t(const AttnParams& p, cudaStream_t stream) {
    const size_t smem = PxLayout<D>::kBytes;
    cudaError_t err = opt_in_smem<prefix_kernel<D, QT, OPTS, TWO>>(smem);
    if (err != cudaSuccess) return err;
    // the register split waits for registers the launch did not give out if this does not hold
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_acquire) == 0) {
        cudaFuncAttributes fa;
        err = cudaFuncGetAttributes(&fa, prefix_kernel<D, QT, OPTS, TWO>);
        if (err != cudaSuccess) return err;
        regs.store(fa.numRegs, std::memory_order_release);
    }
    if (regs.load(std::memory_order_acquire) != kPxLaunchRegs) return cudaErrorInvalidKernelImage;
    CUtensorMap qmap, cmap;
    err = query_map<D, QT>(p, &qmap);
    if (err != cudaSuccess) return err;
    if (p.H % 4 == 0) {
        err = cache_map<D>(p, &cmap);
        if (err != cudaSuccess) return err;
    } else {
        cmap = qmap;   // not used
    }
    const int64_t bq = kPfRows / p.G, tiles = (p.num_q_tokens + bq - 1) / bq;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.H), (unsigned)p.px_splits);
    cfg.blockDim = dim3(kPxThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefix_kernel<D, QT, OPTS, TWO>, p, qmap, cmap);
}

}  // namespace
}  // namespace kvi4
