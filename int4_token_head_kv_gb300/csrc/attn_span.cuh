// Attention in which every query row sees the cached keys of a span of its own, over the INT4, INT8 and INT2
// caches, for chunks of queries and single tokens.  For the query at position pos of its sequence, over its keys
// lo <= j < hi:
//   s_j = scale q . x_Kj,  s_j <- softcap tanh(s_j / softcap),  s_j <- s_j - slope |pos - j|,
//   out = sum_j softmax(s)_j x_Vj   (0 for an empty span).
//
// The products run on the fifth-generation tensor cores with the rows left in the domain they are stored in
// (rotated, but for INT8): S = Q' N_K^T with the stored numbers N exact in fp16 (INT4 code - zp, INT8 code, INT2
// centroid) and the rotated queries Q' as fp16 high + low halves, logit = S s_K k0 2^-e, one pass over the keys with
// one reference off per row, p = 2^(logit + off), weights w = p s_V in fp16 (two halves but for a bf16 output) with the
// largest of a row between 2^6 and 2^15.9, l += p, O += w N_V, everything accumulated in fp32, out = O / l un-rotated.
//
// A CTA takes 128 rows (128 / G query tokens of one sequence x the G query heads of a kv head) against the keys that
// some of them see, 128 at a time; tiles outside that range are not touched, so a document mask costs what its
// documents hold.  With few row tiles the range is split among CTAs and span_combine_kernel joins the partials.
// Tiles that every row of a warp sees whole take no mask; tiles that none of them sees take no arithmetic.
// With a distance bias the tiles go from the last key to the first: the largest logits come first, and the
// references, whose moves rescale O and stall the pipeline, settle at once (608 queries behind 8192 tokens, 32 q / 8 kv heads:
// 181 us forwards, 132 backwards).  Without one they go forwards: a causal row's last tile is cut off, and
// references taken from its few keys move again (107 us forwards, 121 backwards).
//
// What bounds it.  2048 queries behind 32768 INT4 tokens, 32 q / 8 kv heads, d 128, bf16: 1180 us, 961 TFLOP/s of the two
// products that a softmax needs.  The kernel does three, for the queries' halves: a tile takes 2240 cycles (the fullest
// SM's 1056 tiles, less the CTAs' starts and ends) and its 24 products 2130 if alone, 88.6 cycles each where the tensor
// pipe is busy for 62: their operands come through shared memory.  608 queries behind 8192, 93 us: tensor pipe 54%, issue
// slots 57%, shared-memory data pipe 48% besides the operands.  A tile goes through S, the softmax's registers, P.V and the S
// after next, with tensor memory full (two S, O and the queries), and each hand-over is a commit or an arrival, a poll and a
// fence through a busy shared memory.  A CTA's start (where it works, barriers, queries turned and split, first S) takes 7
// us and its end 3, which is half of the time of rows that see 1000 keys (one packed prompt of 16384 tokens: 568 us).
// Single tokens, 8 x 131072 INT2 keys, 64 q / 8 kv heads: 462 us, the same chain for 8 rows.
// Dropped after measuring: CTAs that stay for several row tiles, statically or by cluster launch control (that prompt: 821
// and 804 us against 667 then; the hardware balances as well, and queries turned in registers take longer than a
// product); a third V buffer (single tokens 513 against 505); two warps to a single token's softmax (560 against 504);
// K scales read ahead of S (+2%); one barrier polled after the other (1250 against 1222); the products formed in
// every tile, with the largest one looked at after the weights (1283 against 1200), in place of a bound before them.
#pragma once

#include "attn_prefix.cuh"

namespace kvi4 {
namespace {

// Warp roles (640 threads, the shared-prefix kernel's): warps 0-7 own the rows, 8-11 convert K rows, 12-15 V rows,
// 16 issues the MMAs, 17-18 load packed rows, 19 completes the last warpgroup for the register split.

// Shared memory: [K 0][V 0][K 1][V 1] fp16 tiles (as the prefill's), then staged packed rows, records, barriers.
template <int D, int BITS>
struct SpLayout {
    static constexpr uint32_t kRowBytes = D * BITS / 8 + 4;
    static constexpr uint32_t kRowWords = kRowBytes / 4;                          // codes, then the scale word
    static constexpr uint32_t kChunks = (kRowWords + 3 + 3) / 4;                  // 16-byte chunks of a row's aligned window
    static constexpr uint32_t kWindow = 4 * kChunks;
    static constexpr int kStages = kRowWords > 20 ? 2 : 4;                        // packed tiles staged ahead
    static constexpr uint32_t kTile = (D / 64) * kPfKeys * 128;
    // A block's rows of one head lie in boxes of 16 / m tokens, m the tokens whose rows make a multiple of 16 bytes: 1
    // with 4 or 8 kv heads, else 4 / H.  Boxes start on 128 bytes.  m > 1 is for INT8 rows alone, whose 16-byte copies
    // take longer than the rest of a tile (4864 queries on 4096 tokens, 2 kv heads, d 128: 222 us with them).
    static constexpr bool kGroups = BITS == 8;
    static constexpr uint32_t box_bytes(uint32_t m) { return (kBlockSize / m * kWindow * 4 + 127u) & ~127u; }
    static constexpr uint32_t kLoaded = kPfKeys * kWindow * 4;                    // bytes of one plane of a tile
    static constexpr uint32_t kPlane = kGroups ? kPfKeys / kBlockSize * 4 * box_bytes(4) : kLoaded;   // and their room
    static_assert(!kGroups || (2 * box_bytes(2) <= 4 * box_bytes(4) && box_bytes(1) <= 4 * box_bytes(4)), "room for every grouping");
    static constexpr uint32_t kRaw = 2 * kPfPairs * kTile;
    static constexpr uint32_t kSk = kRaw + kStages * 2 * kPlane;                  // [kring][128] f32 s_K k0 2^-e
    static constexpr uint32_t kDeadF = kSk + kPfKRing * kPfKeys * 4;              // [kring][4] u32: positions with no key
    static constexpr uint32_t kSv = kDeadF + kPfKRing * 4 * 4;                    // [kring][128] f32 s_V
    static constexpr uint32_t kEblk = kSv + kPfKRing * kPfKeys * 4;               // [kring][4] per-warp largest |s_V| (its bits)
    static constexpr uint32_t kWhere = kEblk + kPfKRing * 4 * 4;                               // i32: sequence, query tile, first key, end of the keys, first query's position
    static constexpr uint32_t kHeld = kWhere + 32;                                // [stages] u32: blocks of a staged tile that hold keys
    static constexpr uint32_t kScan = kHeld + kStages * 4;                        // [20] u32
    static constexpr uint32_t kRs = kScan + 20 * 4;                               // [128] f32 2^-d of each row's own prescale
    static constexpr uint32_t kFin = kRs + 128 * 4;                               // [128] f32 what a row's O is multiplied with
    static constexpr uint32_t kSignBits = kFin + 128 * 4;                         // [4] u32
    static constexpr uint32_t kCsign = (kSignBits + 16 + 15u) & ~15u;             // [D] f32 +-c of each dimension
    static constexpr uint32_t kBars = (kCsign + D * 4 + 7u) & ~7u;
    // k_full[kring], sv_full[kring], k_free[pairs], v_full[pairs], pv_done[pairs], s_full[2], p_full[2], q_ready,
    // flush, q_tma, rot_in, rot_done, epi, raw_full[plane][stages], raw_free[plane][stages]
    static constexpr int kNumBars = 2 * kPfKRing + 3 * kPfPairs + 4 + 6 + 4 * kStages;
    static constexpr uint32_t kTmemSlot = kBars + kNumBars * 8;
    static constexpr uint32_t kFlags = kTmemSlot + 4;
    static constexpr uint32_t kBytes = kFlags + 4 + 1024;                         // + alignment slack
    static_assert(kBytes <= 232448, "shared memory");
    static_assert(kSk % 16 == 0 && kSv % 16 == 0 && kEblk % 16 == 0 && kCsign % 16 == 0, "16-byte accesses");
    static_assert(kRaw % 1024 == 0 && kPlane % 128 == 0 && kTile % 1024 == 0 && kBars % 8 == 0, "boxes on 128 bytes, swizzled tiles on 1024");
};

// The INT2 centroids as the tiles hold them: of all pairs of fp16 numbers the one whose ratio is nearest b / a, 1.7939453 and
// 5.984375 (a byte table as kU2Lo, kU2Hi).  With a / 1.7939453 in the scales both are within 2.2e-7.
constexpr uint32_t kSpanU2Lo = 0xBF2DC5FCu, kSpanU2Hi = 0x45FC3F2Du;
constexpr float kU2Scale = 0.25239348f;

// The dimension a tile column holds.
template <int BITS>
__host__ __device__ constexpr int span_dim(int c) { return BITS == 8 ? c : dim_of_column(c); }

// 32 lanes x 16 columns: thread i gets row (lane) i of the address's lanes, 16 consecutive columns.
__device__ __forceinline__ void tmem_ld_row16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// The Walsh-Hadamard butterflies of a thread's own N values.
template <int N>
__device__ __forceinline__ void thread_fwht(float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float a = x[i], b = x[i + 1];
        x[i] = a + b;
        x[i + 1] = a - b;
    }
#pragma unroll
    for (int w = 2; w < N; w <<= 1) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            if (i & w) continue;
            const float2 a = make_float2(x[i], x[i + 1]), b = make_float2(x[i + w], x[i + w + 1]);
            const float2 u = add_f32x2(a, b), v = sub_f32x2(a, b);
            x[i] = u.x, x[i + 1] = u.y;
            x[i + w] = v.x, x[i + w + 1] = v.y;
        }
    }
}

// Eight values as a 16-byte word of a 16-bit type.
__device__ __forceinline__ uint4 pack8(DType dt, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (dt == DType::BF16) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&y);
        } else {
            w[e] = pack_f16x2(x[2 * e], x[2 * e + 1]);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Capped scores come as y, the logit over the cap (or over the nearest bound of SpanParams::cap_unit's range): C tanh(y) + off of
// two of them, C in log2 units, beyond the polynomial's range: C - 2 C / (e^(2y) + 1).  The error is a few 2^-24 of C,
// and of the result.
__device__ __forceinline__ float2 capped(float2 y, const SpanParams& p, float2 off) {
    const float2 z = mul_f32x2(y, make_float2(p.cap_exp, p.cap_exp));
    const float2 u = add_f32x2(make_float2(fast_exp2(z.x), fast_exp2(z.y)), make_float2(1.0f, 1.0f));
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(u.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(u.y));
    const float2 c2 = make_float2(p.cap_l2, p.cap_l2);
    return add_f32x2(fma_f32x2(mul_f32x2(r, make_float2(-2.0f, -2.0f)), c2, c2), off);
}
// The same for |y| <= 2 / 5, without the two special functions: y (C + C a1 y^2 + C a2 y^4 + C a3 y^6), a minimax fit of
// tanh(y) / y with the value 1 at 0 that is off by 1.2e-7 at most, two roundings.  A fourth term would take logits within
// half of the cap, and 1.3% longer (4 x 2048 queries behind 2048 keys, prefix masks, a cap of 50).
__device__ __forceinline__ float2 capped_small(float2 y, const SpanParams& p, float2 off) {
    const float2 t = mul_f32x2(y, y);
    float2 q = fma_f32x2(t, make_float2(p.cap_q[3], p.cap_q[3]), make_float2(p.cap_q[2], p.cap_q[2]));
    q = fma_f32x2(t, q, make_float2(p.cap_q[1], p.cap_q[1]));
    q = fma_f32x2(t, q, make_float2(p.cap_q[0], p.cap_q[0]));
    return fma_f32x2(y, q, off);
}

// The rows' power-of-two prescale: rotated queries of size 2^-4 .. 2^13 keep 22 bits in their fp16 halves; others take a
// further power of two of their own, and the masked path.
constexpr int kSpanExp = 2;

// The largest weights times scale, and weights, that a row may come to before its reference moves (log2), and the largest
// finite number, which stands for a V scale that is not finite.
constexpr float kSpanMaxW = 15.9f, kSpanMaxP = 90.0f, kSpanLargest = 3.4028234664e38f;

// INT8 queries are not rotated: their 8 or 11 bits are fp16 numbers, or lie on fp16's smallest step, as they are.  The low
// halves are 0, and the products with them are left out.
template <int BITS>
constexpr bool kSpanLow = BITS != 8;

// Where a query row's keys are: lo <= j < hi (none: an empty span, or no row).
struct Span {
    int lo, hi;
};

// OPTS: the call caps its scores or has a distance bias.  TWO: the weights as fp16 high + low halves.  FEW: no
// sequence has more than 64 rows (single tokens, drafts); a tile's rows are then the first eight of every sixteen, and the
// second eight hold the low halves of the first, of the queries and of the weights, so that half of the products do.
template <int D, int BITS, bool OPTS, bool TWO, bool FEW>
__global__ void __launch_bounds__(kPxThreads, 1) span_kernel(const __grid_constant__ SpanParams p, const __grid_constant__ CUtensorMap qmap,
                                                             const __grid_constant__ CUtensorMap cmap) {
    using Ly = SpLayout<D, BITS>;
    using Tm = PfTmem<D>;
    constexpr int KSTEPS = D / 16, RB = (int)Ly::kRowBytes, kStages = Ly::kStages;
    // Whether the softmax waits for the V scales alone and the MMA warp for the V tile.  608 queries on 8800 keys: INT8, whose
    // longer rows are converted in one go once their tile is free, 102 us with it and 107 without; with a cap 138.8 and
    // 139.7, with a bias 110 and 112.  Few rows: 8 x 131072 INT4 tokens 442 and 537.  INT4 and INT2 chunks without
    // options: 101 and 95, 108 and 104, as P.V waits for two barriers.
    constexpr bool EARLY = BITS == 8 || OPTS || FEW;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_wait();   // the previous kernel may produce any of the inputs
    if (p.splits > 1) griddep_launch_dependents();   // the combine, which waits for this grid before it reads anything

    if (threadIdx.x == kPxMmaWarp * 32) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&qmap)) : "memory");
    if (threadIdx.x == kPxLoadWarp * 32) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&cmap)) : "memory");
    const int G = p.G, Hq = p.Hq, H = p.H;
    const int BQ = (FEW ? kPfRows / 2 : kPfRows) / G;
    // the row (query token x head) of a tensor-memory lane; with FEW of the first eight of sixteen
    auto row_of = [](int r) -> int { return FEW ? (r >> 4) * 8 + (r & 7) : r; };
    const int h = (int)(blockIdx.x % (unsigned)H), split = (int)blockIdx.y;
    const int group = H >= 4 ? 1 : 4 / H;              // tokens whose rows are a multiple of 16 bytes
    const bool boxes = Ly::kGroups || group == 1;      // TMA loads packed rows (see the loaders)
    volatile int* where = reinterpret_cast<volatile int*>(smem + Ly::kWhere);

    // ---- the CTA's sequence and query tile, the last tiles (the longest causal rows) first
    auto tiles_of = [&](int b) -> int {
        const int ql = min(__ldg(p.qsl + b + 1) - __ldg(p.qsl + b), p.max_query_len);
        return ql > 0 ? (ql + BQ - 1) / BQ : 0;
    };
    int seq, qtile;
    if (p.tiled) {   // tile v of the batch's: its sequence by a scan over the sequences' tile counts
        const int v = (int)(blockIdx.x / (unsigned)H), per = (p.num_seqs + kPxThreads - 1) / kPxThreads;
        const int b0 = min(p.num_seqs, (int)threadIdx.x * per), b1 = min(p.num_seqs, b0 + per);
        int mine = 0;
        for (int b = b0; b < b1; ++b) mine += tiles_of(b);
        int x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        int* scan = reinterpret_cast<int*>(smem + Ly::kScan);
        if (lane == 31) scan[warp] = x;
        if (threadIdx.x == 0) where[0] = -1;
        __syncthreads();
        int before = x - mine;
        for (int w = 0; w < warp; ++w) before += scan[w];
        if (v >= before && v < before + mine) {
            int b = b0, left = v - before;
            for (int n = tiles_of(b); left >= n; n = tiles_of(b)) {
                left -= n;
                ++b;
            }
            where[0] = b;
            where[1] = tiles_of(b) - 1 - left;
        }
        __syncthreads();
        seq = where[0];
        qtile = where[1];
        if (seq < 0) return;   // past the batch's last tile
    } else {
        seq = (int)blockIdx.z;
        qtile = tiles_of(seq) - 1 - (int)(blockIdx.x / (unsigned)H);
        if (qtile < 0) return;
    }
    const int q0 = __ldg(p.qsl + seq);
    const int qlen = __ldg(p.qsl + seq + 1) - q0, qcount = min(qlen, p.max_query_len);
    const int qt0 = qtile * BQ;
    const int len = __ldg(p.seq_lens + seq), L = max(0, min(len, p.len_cap)), pos0 = len - qlen;
    const bool outside = q0 < 0 || (int64_t)q0 + qlen > p.num_q_tokens;
    if (qtile == 0 && h == 0 && split == 0 && threadIdx.x == 0 &&
        (outside || len > p.len_cap || (qlen > len && len != 0) || qlen > p.max_query_len))
        count_status(p.status, 2);
    if (outside) return;
    auto span_of = [&](int qt) -> Span {
        if (qt >= qcount) return Span{0, 0};
        const int r = q0 + qt;
        return Span{p.key_begin ? max(0, __ldg(p.key_begin + r)) : 0, min(L, p.key_end ? __ldg(p.key_end + r) : pos0 + qt + 1)};
    };

    float* sk = reinterpret_cast<float*>(smem + Ly::kSk);
    float* sv = reinterpret_cast<float*>(smem + Ly::kSv);
    uint32_t* eblkw = reinterpret_cast<uint32_t*>(smem + Ly::kEblk);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Ly::kBars);
    uint64_t* k_full = bars;                    // [kring] K tile and scales of tile j (4 warps)
    uint64_t* sv_full = k_full + kPfKRing;      // [kring] V scales of tile j (4 warps; EARLY)
    uint64_t* k_free = sv_full + kPfKRing;      // [pairs] K tile j % 2 read by S of tile j (commit)
    uint64_t* v_full = k_free + kPfPairs;       // [pairs] V tile j converted (4 warps)
    uint64_t* pv_done = v_full + kPfPairs;      // [pairs] P.V of tile j done (commit): V tile j % 2 and O free
    uint64_t* s_full = pv_done + kPfPairs;      // [2] S of the tile in tensor memory (commit)
    uint64_t* p_full = s_full + 2;              // [2] P of the tile in tensor memory (8 warps)
    uint64_t* q_ready = p_full + 2;             // queries in tensor memory, staging free (8 warps)
    uint64_t* flush = q_ready + 1;              // the MMA thread's last commit (teardown)
    uint64_t* q_tma = flush + 1;                // the CTA's query rows in shared memory (bytes)
    uint64_t* rot_in = q_tma + 1;               // the rotation matrix in shared memory (8 warps)
    uint64_t* rot_done = rot_in + 1;            // the rotated queries in tensor memory (commit)
    uint64_t* epi = rot_done + 1;                // the row warps meet (8 of them)
    uint64_t* raw_full = epi + 1;               // [plane][stages] packed rows of a key tile landed (one arrival and bytes, or and 32 lanes)
    uint64_t* raw_free = raw_full + 2 * kStages;   // [plane][stages] that plane converted (4 warps)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly::kTmemSlot);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Ly::kFlags);
    uint32_t* deadf = reinterpret_cast<uint32_t*>(smem + Ly::kDeadF);
    uint32_t* held = reinterpret_cast<uint32_t*>(smem + Ly::kHeld);
    float* fin = reinterpret_cast<float*>(smem + Ly::kFin);

    if (warp == 0) {   // the keys that some row sees
        int lo = 0x7FFFFFFF, hi = 0;
        for (int t = lane; t < BQ; t += 32) {
            const Span s = span_of(qt0 + t);
            if (s.hi > s.lo) {
                lo = min(lo, s.lo);
                hi = max(hi, s.hi);
            }
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
            where[2] = lo;
            where[3] = hi;
            where[4] = pos0 + qt0;
        }
    }
    if (threadIdx.x == 32) {
        for (int b = 0; b < 2 * kPfKRing; ++b) mbar_init(&k_full[b], 4);   // and sv_full
        for (int b = 0; b < kPfPairs; ++b) {
            mbar_init(&k_free[b], 1);
            mbar_init(&v_full[b], 4);
            mbar_init(&pv_done[b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&s_full[b], 1);
            mbar_init(&p_full[b], kPfSoftmaxWarps);
        }
        mbar_init(q_ready, kPfSoftmaxWarps);
        mbar_init(flush, 1);
        mbar_init(epi, kPfSoftmaxWarps);
        mbar_init(q_tma, 1);
        mbar_init(rot_in, kPfSoftmaxWarps);
        mbar_init(rot_done, 1);
        for (int i = 0; i < 2 * kStages; ++i) {
            mbar_init(&raw_full[i], boxes ? 1 : 33);
            mbar_init(&raw_free[i], 4);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    uint32_t* signbits = reinterpret_cast<uint32_t*>(smem + Ly::kSignBits);
    if (BITS != 8 && warp >= 4 && warp < 4 + D / 32) {
        const float s = p.signs[(warp - 4) * 32 + lane];
        reinterpret_cast<float*>(smem + Ly::kCsign)[(warp - 4) * 32 + lane] = s < 0.0f ? -p.c : p.c;
        const uint32_t m = __ballot_sync(0xffffffffu, s < 0.0f);
        if (lane == 0) signbits[warp - 4] = m;
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
    // this split's 128-key tiles, counted from the first key's block
    const int key_base = where[2] / kBlockSize * kBlockSize, key_end = where[3];
    const int tiles_all = key_end > where[2] ? (key_end - key_base + kPfKeys - 1) / kPfKeys : 0;
    const int kt0 = (int)((int64_t)tiles_all * split / p.splits), kt1 = (int)((int64_t)tiles_all * (split + 1) / p.splits);
    const int nkt = kt1 - kt0;
    auto tile_at = [&](int j) -> int { return OPTS && p.alibi != nullptr ? kt1 - 1 - j : kt0 + j; };   // the j-th tile taken
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
    // A warp's arrival, once all its lanes are there: 32 arrivals on one barrier keep the shared-memory pipe busy, which the
    // products' operands, the conversion and every wait of the chain below go through.
    auto arrive = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // the same in the chain S -> weights -> P.V -> next S, where waking a suspended warp would add to every tile:
    // polled first
    auto soon = [&](uint64_t* bar, uint32_t parity) -> bool {
        for (int i = 0; i < kPxPolls; ++i)
            if (mbar_test_wait(bar, parity)) return true;
        return wait(bar, parity);
    };
    // several at once: a poll takes 250 cycles or so behind the other users of shared memory
    auto soon2 = [&](uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb) -> bool {
        for (int i = 0; i < kPxPolls; ++i) {
            const bool x = mbar_test_wait(a, pa), y = mbar_test_wait(b, pb);
            if (x && y) return true;
        }
        return wait(a, pa) && wait(b, pb);
    };
    auto soon3 = [&](uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, uint64_t* c, uint32_t pc) -> bool {
        for (int i = 0; i < kPxPolls; ++i) {
            const bool x = mbar_test_wait(a, pa), y = mbar_test_wait(b, pb), z = mbar_test_wait(c, pc);
            if (x && y && z) return true;
        }
        return wait(a, pa) && wait(b, pb) && wait(c, pc);
    };

    if (nkt == 0) {
        // no keys: nothing below waits for any copy or product; the rows are written at the end
    } else if (warp < kPfSoftmaxWarps) {
        more_registers<kPxRowRegs>();
        // ================================================================ rows: softmax + output
        // Warp w owns the 16 rows 32 (w % 4) + 16 (w / 4) .. in the 16-lane tensor-memory layout: thread (g, t) holds
        // rows ra = rbase + g and rb = ra + 8 and, of every group of 8 columns, columns 2t and 2t + 1.
        const int rbase = 32 * (warp & 3) + 16 * (warp >> 2);
        const int t4 = lane & 3;
        const int ra = rbase + (lane >> 2), rb = ra + 8;
        const uint32_t trow = tmem + ((uint32_t)rbase << 16);
        // ---- the rotation matrix B[p][k] = sign_k (-1)^popcount(n(p) & k) (INT8: the identity) in pair 1's V tile
        {
            constexpr int kRowChunks = D / 8, kThreadsPerRow = kPfSoftmaxThreads / D, kChunksPerThread = kRowChunks / kThreadsPerRow;
            uint8_t* qb = vtile(1);
            const uint32_t one = p.q_bf16 ? 0x3F80u : 0x3C00u;
            const int prow = threadIdx.x / kThreadsPerRow;
            const int n = span_dim<BITS>(slot_of_column(prow));
            uint32_t par8 = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) par8 |= ((uint32_t)__popc(n & j) & 1u) << j;
#pragma unroll
            for (int it = 0; it < kChunksPerThread; ++it) {
                const int k8 = (threadIdx.x % kThreadsPerRow) * kChunksPerThread + it;
                uint32_t w[4];
                if constexpr (BITS == 8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = n / 2 == 4 * k8 + e ? one << (16 * (n & 1)) : 0u;
                } else {
                    const uint32_t sb = (signbits[k8 / 4] >> (8 * (k8 % 4))) & 0xFFu;
                    const uint32_t neg = par8 ^ sb ^ ((__popc(n & (8 * k8)) & 1) ? 0xFFu : 0u);
                    pm1_words(neg, one, w);
                }
                *reinterpret_cast<uint4*>(qb + (uint32_t)(k8 / 8) * (uint32_t)(D * 128) + swz128((uint32_t)prow, (uint32_t)(k8 % 8))) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // generic writes -> tensor core reads
            arrive(rot_in);
        }
        // ---- each row's keys.  A row that sees none goes along as if it saw all, so that it does not put its warp on
        // the masked path, and is zero at the end; a warp of such rows leaves its weights unwritten.
        const int wa = row_of(ra), wb = row_of(rb);
        Span sa = span_of(qt0 + wa / G), sb = FEW ? Span{0, 0} : span_of(qt0 + wb / G);
        const bool none_a = sa.hi <= sa.lo, none_b = sb.hi <= sb.lo;
        if (none_a) sa = Span{0, 0x7FFFFFFF};
        if (none_b) sb = Span{0, 0x7FFFFFFF};
        const bool idle = __all_sync(0xffffffffu, none_a && none_b);
        // the keys that all, and that any, of the warp's rows see
        const int all_lo = __reduce_max_sync(0xffffffffu, max(sa.lo, sb.lo)), all_hi = __reduce_min_sync(0xffffffffu, min(sa.hi, sb.hi));
        const int any_lo = __reduce_min_sync(0xffffffffu, min(none_a ? 0x7FFFFFFF : sa.lo, none_b ? 0x7FFFFFFF : sb.lo));
        const int any_hi = __reduce_max_sync(0xffffffffu, max(none_a ? 0 : sa.hi, none_b ? 0 : sb.hi));
        // ---- a power-of-two prescale of the rows, the same for all, so that 2^-e sits in the keys' scales, then fp16 high +
        // low halves into tensor memory.  A row whose largest value then lies outside [2^-2, 2^15) takes a further power
        // of two of its own.
        float* rs = reinterpret_cast<float*>(smem + Ly::kRs);   // what a row's S is multiplied with
        bool own_any = false;
        bool ok = soon(rot_done, 0);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && !idle) {
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
            auto own = [&](uint32_t m, bool none) -> int {   // a row's further exponent
                const int x = (int)(m >> 23), y = x - 127 + kSpanExp;
                return none || x == 0 || (y >= -2 && y <= 14) ? 0 : max(-126 - kSpanExp, min(127 - kSpanExp, 7 - y));
            };
            const int da = own(mxa, none_a), db = own(mxb, none_b);
            own_any = __any_sync(0xffffffffu, da != 0 || db != 0);
            if (t4 == 0) {
                rs[ra] = exp2f((float)-da);
                rs[rb] = exp2f((float)-db);
            }
            __syncwarp();
            const float sca = exp2i(kSpanExp + da), scb = exp2i(kSpanExp + db);
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
                uint32_t hw[4], lw[4];
#pragma unroll
                for (int i = 2 * q; i < 2 * q + 2; ++i) {
                    split_f16x2(v[4 * i] * sca, v[4 * i + 1] * sca, hw[i & 1], lw[i & 1]);
                    split_f16x2(v[4 * i + 2] * scb, v[4 * i + 3] * scb, hw[2 + (i & 1)], lw[2 + (i & 1)]);
                }
                if constexpr (FEW) {   // row b: the low halves of row a
                    hw[2] = lw[0];
                    hw[3] = lw[1];
                } else if constexpr (kSpanLow<BITS>) {
                    tmem_st_q1(trow + Tm::kQl + 8 * q, lw);
                }
                tmem_st_q1(trow + Tm::kQh + 8 * q, hw);
            }
            tmem_st_wait();
        }
        tc_fence_before();
        arrive(q_ready);
        // ---- the key tiles
        // A row's reference: what is added to its logits (log2 units), so that its largest weight times scale lies between 2^6
        // and 2^15.  The bound on its exponents that calls for another is the tile's, plus: 0, -inf for a row that has met
        // no key yet, inf for one that is none.
        float off_a = 0.0f, off_b = 0.0f;
        float set_a = none_a ? INFINITY : -INFINITY, set_b = none_b ? INFINITY : -INFINITY;
        float l_a = 0.0f, l_b = 0.0f;           // this thread's part of the sums of 2^(logit + off)
        const float pos_a = (float)(wa / G - 2 * t4), pos_b = (float)(wb / G - 2 * t4);   // the row's position - 2t from the tile's first one
        float sl_a = 0.0f, sl_b = 0.0f;
        if (OPTS && p.alibi) {
            sl_a = __ldg(p.alibi + h * G + wa % G) * kLog2e;
            sl_b = __ldg(p.alibi + h * G + wb % G) * kLog2e;
        }
        if (idle) {
            for (int j = 0; j < nkt && ok; ++j) {
                ok = wait(&s_full[j & 1], (uint32_t)(j >> 1) & 1u);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) arrive(&p_full[j & 1]);
            }
        }
        for (int j = idle ? nkt : 0; j < nkt && ok; ++j) {
            const int b = j & 1;
            const uint32_t ph = (uint32_t)(j >> 1) & 1u;
            const int kr = j % kPfKRing;
            const uint32_t rph = (uint32_t)(j / kPfKRing) & 1u;
            ok = EARLY ? soon3(&s_full[b], ph, &k_full[kr], rph, &sv_full[kr], rph)
                       : soon3(&s_full[b], ph, &k_full[kr], rph, &v_full[j % kPfPairs], (uint32_t)(j / kPfPairs) & 1u);
            if (__any_sync(0xffffffffu, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t scol = trow + (b ? Tm::kS1 : Tm::kS0);
            const int key0 = key_base + tile_at(j) * kPfKeys;
            if (key0 >= any_hi || key0 + kPfKeys <= any_lo) {   // none of the warp's rows sees any of it
                const uint32_t zero[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int q = 0; q < (TWO && !FEW ? 16 : 8); ++q) tmem_st_q1(scol + 8 * q, zero);
                tmem_st_wait();
                tc_fence_before();
                arrive(&p_full[b]);
                continue;
            }
            uint32_t s[64];   // s[4i], s[4i + 1]: row a, columns 8i + 2t, + 1; s[4i + 2], s[4i + 3]: row b
            tmem_ld_q8(scol, s);
            tmem_ld_q8(scol + 64, s + 32);
            tmem_ld_wait();
            if constexpr (FEW) {   // row b holds the low halves' share of row a
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s[4 * i] = __float_as_uint(__uint_as_float(s[4 * i]) + __uint_as_float(s[4 * i + 2]));
                    s[4 * i + 1] = __float_as_uint(__uint_as_float(s[4 * i + 1]) + __uint_as_float(s[4 * i + 3]));
                    s[4 * i + 2] = s[4 * i + 3] = 0u;
                }
            }
            // Exponents S s_K k0 2^-e + off (one FMA) with the references as they are, and the largest of the thread's; a
            // reference that moves is added to them afterwards, which is rare.
            float max_a = -INFINITY, max_b = -INFINITY;
            const float4* skb = reinterpret_cast<const float4*>(sk + kr * kPfKeys) + t4;   // columns 16q + (2t, 2t + 1, 8 + 2t, 9 + 2t)
            const uint32_t dead = deadf[kr * 4] | deadf[kr * 4 + 1] | deadf[kr * 4 + 2] | deadf[kr * 4 + 3];
            const bool clean = dead == 0u && !own_any && key0 >= all_lo && key0 + kPfKeys <= all_hi;   // warp-uniform
            const uint4 eb4 = *reinterpret_cast<const uint4*>(eblkw + kr * 4);
            const uint32_t largest = max(max(eb4.x, eb4.y), max(eb4.z, eb4.w));   // the tile's largest V scale
            const float4* svb = reinterpret_cast<const float4*>(sv + kr * kPfKeys) + t4;
            if (!OPTS && clean) {   // every key live and visible to both rows, rs 1
                const float2 moa2 = make_float2(off_a, off_a), mob2 = make_float2(off_b, off_b);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float4 k4 = skb[4 * (i / 2)];
                    const float2 k2 = (i & 1) ? make_float2(k4.z, k4.w) : make_float2(k4.x, k4.y);
                    const float2 ea = fma_f32x2(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), k2, moa2);
                    s[4 * i] = __float_as_uint(ea.x);
                    s[4 * i + 1] = __float_as_uint(ea.y);
                    max_a = max3(max_a, ea.x, ea.y);
                    if constexpr (!FEW) {
                        const float2 eb2 = fma_f32x2(make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), k2, mob2);
                        s[4 * i + 2] = __float_as_uint(eb2.x);
                        s[4 * i + 3] = __float_as_uint(eb2.y);
                        max_b = max3(max_b, eb2.x, eb2.y);
                    }
                }
            } else {
                // bit 2i + e of vis: the row sees the key of column 8i + 2t + e
                uint32_t vis_a = 0xFFFFFFFFu, vis_b = 0xFFFFFFFFu;
                if (!clean) {
                    auto below = [&](int key) -> uint32_t {   // the columns of keys before this one
                        const int y = max(0, min(kPfKeys, key - key0)), n = 2 * (y >> 3) + max(0, min(2, (y & 7) - 2 * t4));
                        return n < 32 ? (1u << n) - 1u : 0xFFFFFFFFu;
                    };
                    vis_a = below(sa.hi) & ~below(sa.lo);
                    vis_b = below(sb.hi) & ~below(sb.lo);
                    if (dead != 0u) {
                        uint32_t gone = 0u;
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t d = deadf[kr * 4 + w] >> (2 * t4);
                            gone |= ((d & 3u) | ((d >> 6) & 0xCu) | ((d >> 12) & 0x30u) | ((d >> 18) & 0xC0u)) << (8 * w);
                        }
                        vis_a &= ~gone;
                        vis_b &= ~gone;
                    }
                }
                const float rs_a = rs[ra], rs_b = rs[rb];
                const float2 rsa2 = make_float2(rs_a, rs_a), rsb2 = make_float2(rs_b, rs_b);
                const float2 moa2 = make_float2(off_a, off_a), mob2 = make_float2(off_b, off_b);
                auto at = [&](int i) -> float2 { return make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])); };
                auto set = [&](int i, float2 x) {
                    s[i] = __float_as_uint(x.x);
                    s[i + 1] = __float_as_uint(x.y);
                };
                if (own_any) {   // (rare) rows with a prescale of their own
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        set(4 * i, mul_f32x2(at(4 * i), rsa2));
                        set(4 * i + 2, mul_f32x2(at(4 * i + 2), rsb2));
                    }
                }
                const bool cap = OPTS && p.softcap > 0.0f;
                constexpr int kPairStep = FEW ? 4 : 2;   // (FEW: row b's are none)
                if (cap) {
                    float mag = 0.0f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float4 k4 = skb[4 * (i / 2)];
                        const float2 k2 = (i & 1) ? make_float2(k4.z, k4.w) : make_float2(k4.x, k4.y);
                        const float2 xa = mul_f32x2(at(4 * i), k2);
                        set(4 * i, xa);
                        mag = max3(mag, fabsf(xa.x), fabsf(xa.y));
                        if constexpr (!FEW) {
                            const float2 xb = mul_f32x2(at(4 * i + 2), k2);
                            set(4 * i + 2, xb);
                            mag = max3(mag, fabsf(xb.x), fabsf(xb.y));
                        }
                    }
                    if (__all_sync(0xffffffffu, mag <= p.cap_small)) {
#pragma unroll
                        for (int i = 0; i < 64; i += kPairStep) set(i, capped_small(at(i), p, (i & 2) ? mob2 : moa2));
                    } else {   // every logit takes the form of its own size, so that no hidden key and no other row reaches it
                        // (608 queries behind 8192 tokens: a cap of 4 185 us, of 50 139)
#pragma unroll
                        for (int i = 0; i < 64; i += kPairStep) {
                            const float2 y = at(i), off = (i & 2) ? mob2 : moa2;
                            const float2 lo = capped_small(y, p, off), hi = capped(y, p, off);
                            set(i, make_float2(fabsf(y.x) <= p.cap_small ? lo.x : hi.x, fabsf(y.y) <= p.cap_small ? lo.y : hi.y));
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float4 k4 = skb[4 * (i / 2)];
                        const float2 k2 = (i & 1) ? make_float2(k4.z, k4.w) : make_float2(k4.x, k4.y);
                        set(4 * i, fma_f32x2(at(4 * i), k2, moa2));
                        if constexpr (!FEW) set(4 * i + 2, fma_f32x2(at(4 * i + 2), k2, mob2));
                    }
                }
                if (OPTS && p.alibi) {
                    // distances, not positions, as fp32 numbers: near ones are exact however long the context.  (The first
                    // query's position from shared memory: registers are short here.)
                    const float first = (float)(where[4] - key0), da0 = first + pos_a, db0 = first + pos_b;
                    const float2 sla2 = make_float2(-sl_a, -sl_a), slb2 = make_float2(-sl_b, -sl_b);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float c = (float)(8 * i);
                        set(4 * i, fma_f32x2(make_float2(fabsf(da0 - c), fabsf(da0 - (c + 1.0f))), sla2, at(4 * i)));
                        if constexpr (!FEW) set(4 * i + 2, fma_f32x2(make_float2(fabsf(db0 - c), fabsf(db0 - (c + 1.0f))), slb2, at(4 * i + 2)));
                    }
                }
                if (!clean) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (!(vis_a & (1u << (2 * i)))) s[4 * i] = 0xFF800000u;
                        if (!(vis_a & (2u << (2 * i)))) s[4 * i + 1] = 0xFF800000u;
                        if (!(vis_b & (1u << (2 * i)))) s[4 * i + 2] = 0xFF800000u;
                        if (!(vis_b & (2u << (2 * i)))) s[4 * i + 3] = 0xFF800000u;
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    max_a = max3(max_a, __uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1]));
                    if constexpr (!FEW) max_b = max3(max_b, __uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3]));
                }
            }
            // Weights p = 2^e and w = p s_V; w stays below 2^15.99, which is within fp16's range, and p below 2^90.  A row
            // that meets its first key, or may pass a bound by the tile's largest scale, is looked at.  (A number's bits over
            // 2^23 are its logarithm + 127, at most 0.087 too low.)
            const float bound = fminf(fmaf((float)largest, -1.1920929e-7f, 127.0f + kSpanMaxW), kSpanMaxP);
            const bool broken = largest >= 0x7F800000u;
            if (__any_sync(0xffffffffu, max_a > bound + set_a || (!FEW && max_b > bound + set_b) || broken)) {
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    max_a = fmaxf(max_a, __shfl_xor_sync(0xffffffffu, max_a, o));
                    max_b = fmaxf(max_b, __shfl_xor_sync(0xffffffffu, max_b, o));
                }
                // The largest w itself, over that of the largest p (or of 1): the largest scale may belong to a key of next to no
                // weight, and a reference taken from it would leave the others' w below fp16's range.
                float top_a = 0.0f, top_b = 0.0f;
                const float2 ma2 = make_float2(-max_a, -max_a), mb2 = make_float2(-max_b, -max_b);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float4 v4 = svb[4 * (i / 2)];
                    const float vx = fabsf((i & 1) ? v4.z : v4.x), vy = fabsf((i & 1) ? v4.w : v4.y);
                    const float2 ea = add_f32x2(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), ma2);
                    top_a = max3(top_a, fast_exp2(ea.x) * vx, fast_exp2(ea.y) * vy);
                    if constexpr (!FEW) {
                        const float2 eb2 = add_f32x2(make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), mb2);
                        top_b = max3(top_b, fast_exp2(eb2.x) * vx, fast_exp2(eb2.y) * vy);
                    }
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    top_a = fmaxf(top_a, __shfl_xor_sync(0xffffffffu, top_a, o));
                    top_b = fmaxf(top_b, __shfl_xor_sync(0xffffffffu, top_b, o));
                }
                if (broken) {   // a visible value that is not finite shows in the sum, whatever its weight
#pragma unroll 1
                    for (int q = 0; q < 8; ++q) {
                        const float4 v4 = svb[4 * q];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = key0 + 16 * q + 8 * (e >> 1) + 2 * t4 + (e & 1);
                            const float v = e == 0 ? v4.x : e == 1 ? v4.y : e == 2 ? v4.z : v4.w;
                            if (fabsf(v) >= kSpanLargest) {
                                if (key >= sa.lo && key < sa.hi) l_a = __uint_as_float(0x7FC00000u);
                                if (key >= sb.lo && key < sb.hi) l_b = __uint_as_float(0x7FC00000u);
                            }
                        }
                    }
                }
                // What a row's reference moves by: the largest w goes to 2^6 .. 2^7, if that is p <= 2^80.  A reference that
                // holds stays, to the bit, whatever called: only what the row sees counts.
                auto move = [](float& set, float m, float top) -> float {
                    const float lg = fmaf((float)__float_as_uint(top), 1.1920929e-7f, -127.0f);
                    if (!(m > -INFINITY) || set > 0.0f || (set == 0.0f && !(m + lg > kSpanMaxW || m > kSpanMaxP))) return 0.0f;
                    set = 0.0f;
                    return (float)(top > 0.0f ? min(kPxRaise + 127 - (int)(__float_as_uint(top) >> 23), 80) : 0) - m;
                };
                const bool had_a = set_a == 0.0f, had_b = set_b == 0.0f;
                const float da = move(set_a, max_a, top_a), db = FEW ? 0.0f : move(set_b, max_b, top_b);
                off_a += da;
                off_b += db;
                const float f_a = had_a && da != 0.0f ? fast_exp2(da) : 1.0f;
                const float f_b = FEW ? f_a : had_b && db != 0.0f ? fast_exp2(db) : 1.0f;
                l_a *= f_a;
                l_b *= f_b;
                const float2 da2 = make_float2(da, da), db2 = make_float2(db, db);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 ea = add_f32x2(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), da2);
                    s[4 * i] = __float_as_uint(ea.x);
                    s[4 * i + 1] = __float_as_uint(ea.y);
                    if constexpr (!FEW) {
                        const float2 eb2 = add_f32x2(make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), db2);
                        s[4 * i + 2] = __float_as_uint(eb2.x);
                        s[4 * i + 3] = __float_as_uint(eb2.y);
                    }
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
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[16];
                        tmem_ld_q4(trow + Tm::kO + c0, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 oa = mul_f32x2(make_float2(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1])), fa2);
                            const float2 ob = mul_f32x2(make_float2(__uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3])), fb2);
                            const uint32_t w[4] = {__float_as_uint(oa.x), __float_as_uint(oa.y), __float_as_uint(ob.x), __float_as_uint(ob.y)};
                            tmem_st_q1(trow + Tm::kO + c0 + 8 * i, w);
                        }
                    }
                    tmem_st_wait();
                }
            }
            // w as fp16 pairs over the first 64 S columns: the pair of columns 8i + 2t, + 1 goes to column
            // 8 (i / 2) + 2t + i % 2 (the V tile holds its rows in the matching order)
            float2 lsa = make_float2(0.0f, 0.0f), lsb = make_float2(0.0f, 0.0f);
            if constexpr (FEW) {   // the low halves of the weights as row b
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    uint32_t pw[4];
                    const float4 v4 = svb[4 * q];
#pragma unroll
                    for (int i = 2 * q; i < 2 * q + 2; ++i) {
                        const float2 v2 = (i & 1) ? make_float2(v4.z, v4.w) : make_float2(v4.x, v4.y);
                        const float2 pa = make_float2(fast_exp2(__uint_as_float(s[4 * i])), fast_exp2(__uint_as_float(s[4 * i + 1])));
                        lsa = add_f32x2(lsa, pa);
                        const float2 wa = mul_f32x2(pa, v2);
                        split_f16x2(wa.x, wa.y, pw[i & 1], pw[2 + (i & 1)]);
                    }
                    tmem_st_q1(scol + 8 * q, pw);
                }
            } else {
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
            }
            l_a += lsa.x + lsa.y;
            l_b += lsb.x + lsb.y;
            tmem_st_wait();
            tc_fence_before();
            arrive(&p_full[b]);
        }
        // ---- the output, or the split's partial: (-off, l) with l normalised to 1 .. 2, and O / l
        if (ok) ok = wait(&pv_done[(nkt - 1) & 1], (uint32_t)((nkt - 1) >> 1) & 1u);
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
        // (a row that met NaN shows it in its sum)
        const bool any_a = l_a != 0.0f && !none_a, any_b = l_b != 0.0f && !none_b;
        if (t4 == 0) {
            fin[ra] = any_a ? 1.0f / l_a : 0.0f;
            fin[rb] = any_b ? 1.0f / l_b : 0.0f;
            if (p.splits > 1) {
                auto partial = [&](int r, bool any, float l, float off) {
                    const int qt = qt0 + r / G;
                    if (qt >= qcount) return;
                    const uint32_t bits = __float_as_uint(l);
                    float2 ml = make_float2((float)((int)(bits >> 23) - 127) - off, __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u));
                    if (!(l < INFINITY)) ml = make_float2(0.0f, l);
                    reinterpret_cast<float2*>(p.part_ml)[((int64_t)(q0 + qt) * Hq + h * G + r % G) * p.splits + split] =
                        any && ok ? ml : make_float2(kNegBig, 0.0f);
                };
                partial(wa, any_a, l_a, off_a);
                if constexpr (!FEW) partial(wb, any_b, l_b, off_b);
            }
        }
        __syncwarp();
        // Two threads per row from here on, the other layout: warp w takes the 32 rows 32 (w % 4) .. and column half w / 4.
        arrive(epi);
        ok = __all_sync(0xffffffffu, soon(epi, 0) && ok);
        tc_fence_after();
        constexpr int HD = D / 2;   // this thread's dimensions: half * HD ..
        const int row = 32 * (warp & 3) + lane, half = warp >> 2, nrows = min(BQ, qcount - qt0) * G;
        const bool whole = p.splits == 1;
        if (ok && nrows > row_of(32 * (warp & 3))) {
            const uint32_t trow32 = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + Tm::kO;
            const float f = fin[row];
            float x[HD];
#pragma unroll
            for (int c0 = 0; c0 < HD; c0 += 16) {
                // out = c D H x: the butterflies between the halves as they are read, the others in registers
                uint32_t a[16], b[16];
                tmem_ld_row16(trow32 + (BITS != 8 && whole ? 0 : half * HD) + c0, a);
                if (BITS != 8 && whole) tmem_ld_row16(trow32 + HD + c0, b);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    float y = __uint_as_float(a[c]);
                    if (BITS != 8 && whole) y = half ? y - __uint_as_float(b[c]) : y + __uint_as_float(b[c]);
                    if (FEW) y += __shfl_down_sync(0xffffffffu, y, 8);   // the low halves' share
                    x[c0 + span_dim<BITS>(c)] = f == 0.0f ? 0.0f : y * f;
                }
            }
            if (BITS != 8 && whole) {
                thread_fwht<HD>(x);
                const float4* cs = reinterpret_cast<const float4*>(smem + Ly::kCsign) + half * (HD / 4);
#pragma unroll
                for (int i = 0; i < HD / 4; ++i) {
                    const float4 c = cs[i];
                    x[4 * i] *= c.x;
                    x[4 * i + 1] *= c.y;
                    x[4 * i + 2] *= c.z;
                    x[4 * i + 3] *= c.w;
                }
            }
            // Through shared memory (the last P.V is done, so nothing reads the tiles), 64 bytes of each of the warp's rows
            // at a time, so that neighbouring lanes store neighbouring words.
            uint8_t* stage = tiles + warp * 2048;
            auto store_rows = [&](uint8_t* base, int64_t pitch, int bytes, int c, const uint4 (&w)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) *reinterpret_cast<uint4*>(stage + lane * 64 + 16 * (e ^ ((lane >> 1) & 3))) = w[e];
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int l = 8 * e + lane / 4, r = row_of(32 * (warp & 3) + l);
                    if (r < nrows && (!FEW || (l & 8) == 0)) {
                        const int64_t at = (int64_t)(q0 + qt0 + r / G) * Hq + h * G + r % G;
                        *reinterpret_cast<uint4*>(base + at * pitch + half * bytes + 64 * c + 16 * (lane & 3)) =
                            *reinterpret_cast<const uint4*>(stage + l * 64 + 16 * ((lane & 3) ^ ((l >> 1) & 3)));
                    }
                }
                __syncwarp();
            };
            if (!whole || p.out_dt == DType::F32) {
                uint8_t* base = whole ? static_cast<uint8_t*>(p.out) : reinterpret_cast<uint8_t*>(p.part_o) + (int64_t)split * (D * 4);
#pragma unroll
                for (int c = 0; c < HD / 16; ++c) {
                    uint4 w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = make_uint4(__float_as_uint(x[16 * c + 4 * e]), __float_as_uint(x[16 * c + 4 * e + 1]),
                                          __float_as_uint(x[16 * c + 4 * e + 2]), __float_as_uint(x[16 * c + 4 * e + 3]));
                    store_rows(base, (int64_t)p.splits * (D * 4), HD * 4, c, w);
                }
            } else {
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    uint4 w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = pack8(p.out_dt, x + 32 * c + 8 * e);
                    store_rows(static_cast<uint8_t*>(p.out), D * 2, HD * 2, c, w);
                }
            }
        }
    } else if (warp < kPxMmaWarp) {
        fewer_registers<kPxDequantRegs>();
        // ================================================================ conversion of key tiles
        const int pl = (warp - kPxDequantWarp) >> 2;      // 0: K rows, 1: V rows
        // This thread's key of every tile.  A V tile keeps its rows in the order the weights are laid out in, and V
        // threads take their keys in an order in which eight neighbours have keys, and rows, of eight different
        // remainders mod 8: the windows' reads and the swizzled rows' stores then hit no bank twice.
        const int i128 = (threadIdx.x - kPfSoftmaxThreads) & 127;
        const int k = pl ? v_key(i128) : i128;
        const uint32_t trow = (uint32_t)(pl ? slot_of_column(k) : k);
        constexpr int NW = (int)Ly::kRowWords;            // words of a row: codes, then the scale word
        // raw score -> log2 logit, or logit over the cap (finite, so that a row of zeros has a logit of 0)
        float k0 = p.c * p.softmax_scale * (OPTS ? p.cap_unit : kLog2e) * exp2i(-kSpanExp);
        if (OPTS) k0 = fmaxf(fminf(k0, 3.0e38f), -3.0e38f);
        const int row_off = ((k % kBlockSize) * H + h) & 3;   // the row's first word in its window (row bytes are 4 mod 16)
        const uint32_t row_at = boxes ? (uint32_t)(k / kBlockSize * group + k % group) * Ly::box_bytes((uint32_t)group) +
                                            (uint32_t)(k % kBlockSize / group) * Ly::kWindow * 4
                                      : (uint32_t)k * Ly::kWindow * 4;
        for (int j = 0; j < nkt; ++j) {
            const int kb = j % kPfPairs, st = j % kStages;
            bool ok = wait(&raw_full[pl * kStages + st], (uint32_t)(j / kStages) & 1u);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint4* win4 = reinterpret_cast<const uint4*>(smem + Ly::kRaw + (uint32_t)(st * 2 + pl) * Ly::kPlane + row_at);
            const uint32_t blocks = pl == 0 ? held[st] : 0u;
            uint8_t* t = pl ? vtile(kb) : ktile(kb);
            auto tile_free = [&]() -> bool {
                bool f = j != 1 || wait(q_ready, 0);        // the query rows and the rotation matrix sat on pair 1
                if (f && j >= kPfPairs) f = wait(pl ? &pv_done[kb] : &k_free[kb], (uint32_t)(j / kPfPairs - 1) & 1u);
                return __all_sync(0xffffffffu, f);
            };
            auto put = [&](int w, const uint32_t (&o)[4]) {   // dimensions 8w .. 8w + 7 in the tile's order
                *reinterpret_cast<uint4*>(t + (uint32_t)(w / 8) * (kPfKeys * 128u) + swz128(trow, (uint32_t)(w % 8))) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            };
            // EARLY: the V scales go ahead of the tile, which waits for P.V of tile j - 2; the weights wait for the scales alone.
            // Their place was last read for the weights of tile j - 4, and P.V of tile j - 3 is done.  The K scales' place
            // is free once S of tile j - 2 is done, as P.V of tile j - 4 came before it.
            auto publish = [&](uint32_t scale) {
                const float sc = BITS == 2 ? __uint_as_float(scale) * kU2Scale : __uint_as_float(scale);
                if (pl == 0) {
                    // (a key that is not finite: NaN, also where its products with a query have the same sign)
                    sk[(j % kPfKRing) * kPfKeys + slot_of_column(k)] = fabsf(sc) <= kSpanLargest ? sc * k0 : __uint_as_float(0x7FC00000u);
                    const uint32_t nokey = __ballot_sync(0xffffffffu, ((blocks >> (k / kBlockSize)) & 1u) == 0u);   // a row of zeros is a key, of logit 0
                    if (lane == 0) deadf[(j % kPfKRing) * 4 + (warp & 3)] = nokey;
                } else {
                    // finite, so that a weight of 0 stays one; a scale that is not finite shows in the largest one
                    sv[(j % kPfKRing) * kPfKeys + (int)trow] = fmaxf(fminf(sc, kSpanLargest), -kSpanLargest);
                    const uint32_t wmax = __reduce_max_sync(0xffffffffu, __float_as_uint(sc) & 0x7FFFFFFFu);   // magnitudes order like their bits
                    if (lane == 0) eblkw[(j % kPfKRing) * 4 + (warp & 3)] = wmax;
                    if (EARLY) arrive(&sv_full[j % kPfKRing]);
                }
            };
            uint32_t scale;   // the scale word, without a zero point
            if constexpr (NW > 20) {   // long rows: a chunk of 16 numbers at a time
                scale = reinterpret_cast<const uint32_t*>(win4)[NW - 1 + row_off];
                if (EARLY && pl == 1) publish(scale);
                ok = tile_free();
                if (!ok) break;
                uint4 c0 = win4[0];
#pragma unroll
                for (int c = 0; c < (NW - 1) / 4; ++c) {
                    const uint4 c1 = win4[c + 1];
                    const uint32_t u[6] = {(row_off & 2) ? c0.z : c0.x, (row_off & 2) ? c0.w : c0.y, (row_off & 2) ? c1.x : c0.z,
                                           (row_off & 2) ? c1.y : c0.w, (row_off & 2) ? c1.z : c1.x, 0u};
                    uint32_t w[4], o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = (row_off & 1) ? u[e + 1] : u[e];
                    unpack_i8(w[0], w[1], o);
                    put(2 * c, o);
                    unpack_i8(w[2], w[3], o);
                    put(2 * c + 1, o);
                    c0 = c1;
                }
                arrive(&raw_free[pl * kStages + st]);
            } else {
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
                arrive(&raw_free[pl * kStages + st]);
                scale = BITS == 4 ? kw[NW - 1] & 0xFFFFFFF0u : kw[NW - 1];
                if (EARLY && pl == 1) publish(scale);
                ok = tile_free();
                if (!ok) break;
                if constexpr (BITS == 4) {
                    const uint32_t zp = kw[NW - 1] & 15u, zl = zp_lo_half(zp) * 0x10001u, zh = zp_hi_half(zp) * 0x10001u;
#pragma unroll
                    for (int w = 0; w < NW - 1; ++w) {
                        uint32_t o[4];
                        unpack_word(kw[w], zl, zh, o);
                        put(w, o);
                    }
                } else if constexpr (BITS == 8) {
#pragma unroll
                    for (int w = 0; w < (NW - 1) / 2; ++w) {
                        uint32_t o[4];
                        unpack_i8(kw[2 * w], kw[2 * w + 1], o);
                        put(w, o);
                    }
                } else {
#pragma unroll
                    for (int w = 0; w < NW - 1; ++w) {
                        uint32_t oa[4], ob[4];
                        unpack_u2_x2<kSpanU2Lo, kSpanU2Hi>(kw[w], oa, ob);
                        put(2 * w, oa);
                        put(2 * w + 1, ob);
                    }
                }
            }
            if (!EARLY || pl == 0) publish(scale);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // generic writes -> tensor core reads
            arrive(pl ? &v_full[kb] : &k_full[j % kPfKRing]);
        }
    } else {
        fewer_registers<kPxOtherRegs>();
        if (warp == kPxLoadWarp || warp == kPxLoadWarp + 1) {
            // ============================================================ loads of packed rows
            // Each row's 16-byte-aligned window, keys in a block outside the cache or past the last key's block
            // zero-filled; which blocks hold keys goes along with the K rows.  With 4 or 8 kv heads a token's rows
            // are a multiple of 16 bytes and TMA takes a block's windows at once; with 1 or 2 the rows of 4 or 2 tokens
            // are, and INT8 rows take as many boxes.  INT4 and INT2 windows are then 16-byte copies, kKeys whole
            // windows (C lanes each) a pass.
            constexpr int C = Ly::kChunks, kKeys = 32 / C, kPasses = (kPfKeys + kKeys - 1) / kKeys;
            const int pl = warp - kPxLoadWarp;
            const int32_t* table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq + key_base / kBlockSize;
            const int tok_stride = H * RB;
            const int64_t blk_stride = 2 * kBlockSize * (int64_t)tok_stride;
            const uint8_t* base = p.cache + (int64_t)pl * kBlockSize * tok_stride;
            const int ck = lane / C, cc = lane - ck * C;   // this lane's key of a pass and its chunk
            const bool mine = ck < kKeys;
            // Block ids of four tiles at a time, lane l's that of the l / 8-th, block l % 8 of it (-1: none, or not in
            // the cache), loaded a group ahead.
            const int nblocks = (key_end + kBlockSize - 1) / kBlockSize - key_base / kBlockSize;
            auto block_of = [&](int j) -> int { return tile_at(j + lane / 8) * (kPfKeys / kBlockSize) + (lane & 7); };
            auto inside = [&](int j) -> bool { return j + lane / 8 < nkt && block_of(j) < nblocks; };
            auto lookup = [&](int j) -> int { return inside(j) ? __ldg(table + block_of(j)) : -1; };
            int blk_next = lookup(0), blkv = -1;
            uint32_t blocks = 0;
            bool ok = true;
            int issued = 0;
            for (int j = 0; j < nkt && ok; ++j) {
                const int st = j % kStages;
                if ((j & 3) == 0) {
                    blkv = blk_next;
                    blk_next = lookup(j + 4);
                    if (blkv < 0 || (int64_t)blkv >= p.num_blocks) {
                        if (pl == 0 && h == 0 && inside(j)) count_status(p.status, 1);
                        blkv = -1;
                    }
                    blocks = __ballot_sync(0xffffffffu, blkv >= 0);
                }
                if (j >= kStages) ok = wait(&raw_free[pl * kStages + st], (uint32_t)(j / kStages - 1) & 1u);
                if (!__all_sync(0xffffffffu, ok)) break;
                const uint32_t dst = smem_u32(smem + Ly::kRaw + (uint32_t)(st * 2 + pl) * Ly::kPlane);
                if (pl == 0 && lane == 0) held[st] = blocks >> (8 * (j & 3));   // this tile's: the low 8 bits; before the arrival below
                if (boxes) {
                    // boxes [16 / group tokens][window bytes]; block -1 lies outside the tensor and reads as zeros, as do
                    // a last head's bytes past its tokens' rows
                    uint64_t* full = &raw_full[pl * kStages + st];
                    const int blk = __shfl_sync(0xffffffffu, blkv, (j & 3) * 8 + (lane / group & 7));
                    if (lane == 0) mbar_arrive_expect_tx(full, Ly::kLoaded);
                    __syncwarp();
                    if (lane < kPfKeys / kBlockSize * group)
                        tma_load_4d(dst + (uint32_t)lane * Ly::box_bytes((uint32_t)group), &cmap, (lane % group * tok_stride + h * RB) & ~15, 0, pl,
                                    blk, full);
                    issued = j + 1;
                    continue;
                }
                if constexpr (!Ly::kGroups) {
#pragma unroll
                    for (int t = 0; t < kPasses; ++t) {
                        const int key = t * kKeys + ck;
                        const int blk = __shfl_sync(0xffffffffu, blkv, (j & 3) * 8 + ((key / kBlockSize) & 7));
                        const bool live = blk >= 0;
                        const uint32_t row = (uint32_t)(h * RB + (key % kBlockSize) * tok_stride);
                        const uint8_t* src = base + (int64_t)(live ? blk : 0) * blk_stride + ((row & ~15u) + 16u * (uint32_t)cc);
                        if (mine && key < kPfKeys) cp_async16_zfill(dst + 16u * (uint32_t)(key * C + cc), src, live);
                    }
                    cp_async_arrive_noinc(&raw_full[pl * kStages + st]);
                    if (lane == 0) mbar_arrive(&raw_full[pl * kStages + st]);
                }
            }
            // no copy outlives the CTA
            cp_async_wait_all();
            for (int j = max(0, issued - kStages); j < issued; ++j)
                (void)mbar_wait(&raw_full[pl * kStages + j % kStages], (uint32_t)(j / kStages) & 1u);
        } else if (warp == kPxMmaWarp) {
            // ============================================================ the MMA issuer
            // S of tile t (its K tile converted, its S buffer read by P.V of tile t - 2), then P.V of tile t - 1
            // (its weights in tensor memory).  The whole warp runs the loop with uniform values and one elected
            // lane issues, so that the descriptors sit in uniform registers.
            constexpr uint32_t idS = idesc_f16(kPfKeys, 0), idPV = idesc_f16(D, 1);
            const bool leader = elect_one();
            const uint64_t kd0 = smem_desc_sw128(smem_u32(ktile(0)), 16u, 1024u), kd1 = smem_desc_sw128(smem_u32(ktile(1)), 16u, 1024u);
            const uint64_t vd0 = smem_desc_sw128(smem_u32(vtile(0)), kPfKeys * 128u, 1024u);
            const uint64_t vd1 = smem_desc_sw128(smem_u32(vtile(1)), kPfKeys * 128u, 1024u);
            {
                if (leader) {
                    const int eights = (min(BQ, qcount - qt0) * G + 7) / 8;   // FEW: boxes of eight rows
                    mbar_arrive_expect_tx(q_tma, FEW ? (uint32_t)eights * (D / 64) * 1024u : Ly::kTile);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        if constexpr (FEW) {   // eight rows a box, in every second eight rows of the tile
                            for (int i = 0; i < eights; ++i)
                                tma_load_3d(ktile(1) + c * (kPfRows * 128) + i * 2048, &qmap, 64 * c, h * G, q0 + qt0 + i * (8 / G), q_tma);
                        } else {
                            tma_load_3d(ktile(1) + c * (kPfRows * 128), &qmap, 64 * c, h * G, q0 + qt0, q_tma);
                        }
                    }
                }
                __syncwarp();
                if (__all_sync(0xffffffffu, mbar_wait(q_tma, 0) && wait(rot_in, 0))) {
                    tc_fence_after();
                    const uint32_t idR = p.q_bf16 ? idesc_bf16(D, 0) : idesc_f16(D, 0);
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
                    for (int half = 0; half < (FEW || !kSpanLow<BITS> ? 1 : 2); ++half) {
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
                        if constexpr (TWO && !FEW) mma_ts(tmem + Tm::kO, pcol + 64u + 8u * kk, vd + ((kk * 16 * 128) >> 4), idPV, true);
                    }
                    mma_commit(&pv_done[t % kPfPairs]);
                }
                __syncwarp();
            };
            static_assert(kPfPairs == 2, "one descriptor per pair");
            bool ok = __all_sync(0xffffffffu, soon(q_ready, 0));
            for (int t = 0; t <= nkt && ok; ++t) {
                if (t < nkt) {
                    uint64_t* full = &k_full[t % kPfKRing];
                    const uint32_t ph = (uint32_t)(t / kPfKRing) & 1u;
                    ok = t < 2 ? soon(full, ph) : soon2(full, ph, &pv_done[t & 1], (uint32_t)((t - 2) >> 1) & 1u);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    tc_fence_after();
                    issue_s(t);
                }
                if (t > 0) {
                    const uint32_t ph = (uint32_t)((t - 1) >> 1) & 1u;
                    if constexpr (EARLY) ok = soon2(&p_full[(t - 1) & 1], ph, &v_full[(t - 1) & 1], ph);
                    else ok = soon(&p_full[(t - 1) & 1], ph);   // (which waited for the V tile)
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
    if (nkt == 0 && threadIdx.x < kPfRows) {   // rows that see nothing here
        const int row = threadIdx.x, qt = qt0 + row / G;
        if (qt < qcount) {
            const int64_t orow = (int64_t)(q0 + qt) * Hq + h * G + row % G;
            if (p.splits > 1) {
                reinterpret_cast<float2*>(p.part_ml)[orow * p.splits + split] = make_float2(kNegBig, 0.0f);
            } else {
                const int n = p.out_dt == DType::F32 ? D / 4 : D / 8;
                for (int i = 0; i < n; ++i) reinterpret_cast<uint4*>(p.out)[orow * n + i] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kPxMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
}

// Joins the splits of one row per warp: out = sum_s (l_s 2^(m_s - M)) o_s / sum_s l_s 2^(m_s - M), un-rotated.
constexpr int kSpanCombineWarps = 4;

template <int D, bool ROTATED>
__global__ void __launch_bounds__(kSpanCombineWarps * 32) span_combine_kernel(const __grid_constant__ SpanParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kSpanCombineWarps + warp, rows = p.num_q_tokens * p.Hq;
    const bool live = row < rows;
    const int tok = live ? (int)(row / p.Hq) : 0;
    float sgn[D / 32];
#pragma unroll
    for (int k = 0; k < D / 32; ++k) sgn[k] = ROTATED && p.signs[lane + 32 * k] < 0.0f ? -1.0f : 1.0f;
    int b = 0, hi = p.num_seqs;   // the last sequence with qsl[b] <= tok
    while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (__ldg(p.qsl + mid) <= tok) b = mid;
        else hi = mid;
    }
    const int q0 = __ldg(p.qsl + b), q1 = __ldg(p.qsl + b + 1);
    const bool mine = live && tok >= q0 && tok < q0 + min(q1 - q0, p.max_query_len) && q0 >= 0 && q1 <= p.num_q_tokens;
    griddep_wait();
    if (!mine) return;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + row * p.splits;
    // lane s holds split s (and s + 32)
    const float2 v0 = lane < p.splits ? ml[lane] : make_float2(kNegBig, 0.0f);
    const float2 v1 = lane + 32 < p.splits ? ml[lane + 32] : make_float2(kNegBig, 0.0f);
    const float M = warp_max(fmaxf(v0.x, v1.x));
    float w0 = v0.y == 0.0f ? 0.0f : v0.y * fast_exp2(v0.x - M), w1 = v1.y == 0.0f ? 0.0f : v1.y * fast_exp2(v1.x - M);
    float total = w0 + w1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    float x[D / 32];
#pragma unroll
    for (int k = 0; k < D / 32; ++k) x[k] = 0.0f;
    const float* po = p.part_o + row * p.splits * D + lane;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
        const float w = __shfl_sync(0xffffffffu, s < 32 ? w0 : w1, s & 31) * inv;
        if (w == 0.0f) continue;   // nothing seen: its output was not written
#pragma unroll
        for (int k = 0; k < D / 32; ++k) x[k] = fmaf(po[(int64_t)s * D + 32 * k], w, x[k]);
    }
    if constexpr (ROTATED) warp_fwht<D>(x);
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
        const float y = ROTATED ? x[k] * p.c * sgn[k] : x[k];
        const int64_t i = row * D + lane + 32 * k;
        if (p.out_dt == DType::BF16) store_elem<__nv_bfloat16>(p.out, i, y);
        else if (p.out_dt == DType::F16) store_elem<__half>(p.out, i, y);
        else store_elem<float>(p.out, i, y);
    }
}

// The queries as [token][q head][D], in boxes of [rows / G tokens][G heads][64 dims] with the 128-byte swizzle.
template <int D>
cudaError_t span_query_map(const SpanParams& p, int rows, CUtensorMap* map) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (enc == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)p.num_q_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)p.Hq * D * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)p.G, (cuuint32_t)(rows / p.G)};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    const CUresult r = enc(map, p.q_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                           const_cast<void*>(p.q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The cache as bytes [block][plane][16 / group tokens][rows of group tokens], in boxes of a block's windows of one head
// (of every group-th token).  Block ids are int32, so a larger cache has no block past 2^31 that could be named.
template <int D, int BITS>
cudaError_t span_cache_map(const SpanParams& p, CUtensorMap* map) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (enc == nullptr) return cudaErrorNotSupported;
    using Ly = SpLayout<D, BITS>;
    const cuuint64_t group = p.H >= 4 ? 1 : 4 / p.H, row = group * (cuuint64_t)p.H * Ly::kRowBytes, rows = kBlockSize / group;
    const cuuint64_t blocks = (cuuint64_t)std::min<int64_t>(std::max<int64_t>(p.num_blocks, 1), (int64_t)1 << 31);
    const cuuint64_t dims[4] = {row, rows, 2, blocks};
    const cuuint64_t strides[3] = {row, row * rows, row * rows * 2};
    const cuuint32_t box[4] = {Ly::kWindow * 4, (cuuint32_t)rows, 1, 1};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(p.cache), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int BITS, bool OPTS, bool TWO, bool FEW>
cudaError_t launch_span_t(const SpanParams& p, cudaStream_t stream) {
    const size_t smem = SpLayout<D, BITS>::kBytes;
    cudaError_t err = opt_in_smem<span_kernel<D, BITS, OPTS, TWO, FEW>>(smem);
    if (err != cudaSuccess) return err;
    // the register split waits for registers the launch did not give out if this does not hold
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_acquire) == 0) {
        cudaFuncAttributes fa;
        err = cudaFuncGetAttributes(&fa, span_kernel<D, BITS, OPTS, TWO, FEW>);
        if (err != cudaSuccess) return err;
        regs.store(fa.numRegs, std::memory_order_release);
    }
    if (regs.load(std::memory_order_acquire) != kPxLaunchRegs) return cudaErrorInvalidKernelImage;
    CUtensorMap qmap, cmap;
    err = span_query_map<D>(p, FEW ? 8 : kPfRows, &qmap);
    if (err != cudaSuccess) return err;
    if (p.H >= 4 || SpLayout<D, BITS>::kGroups) {
        err = span_cache_map<D, BITS>(p, &cmap);
        if (err != cudaSuccess) return err;
    } else {
        cmap = qmap;   // not used
    }
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.tiles * (unsigned)p.H, (unsigned)p.splits, p.tiled ? 1u : (unsigned)p.num_seqs);
    cfg.blockDim = dim3(kPxThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, span_kernel<D, BITS, OPTS, TWO, FEW>, p, qmap, cmap);
    if (err != cudaSuccess || p.splits == 1) return err;
    cfg.gridDim = dim3((unsigned)((p.num_q_tokens * p.Hq + kSpanCombineWarps - 1) / kSpanCombineWarps));
    cfg.blockDim = dim3(kSpanCombineWarps * 32);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, span_combine_kernel<D, BITS != 8>, p);
}

// Every (head size, options, weights) instantiation of one cache mode.
template <int D, int BITS>
cudaError_t launch_span_head(const SpanParams& p, cudaStream_t s) {
    const bool opts = p.softcap > 0.0f || p.alibi != nullptr;
    if (p.max_query_len <= kPfRows / 2 / p.G) return opts ? launch_span_t<D, BITS, true, true, true>(p, s) : launch_span_t<D, BITS, false, true, true>(p, s);
    if (p.out_dt == DType::BF16) return opts ? launch_span_t<D, BITS, true, false, false>(p, s) : launch_span_t<D, BITS, false, false, false>(p, s);
    return opts ? launch_span_t<D, BITS, true, true, false>(p, s) : launch_span_t<D, BITS, false, true, false>(p, s);
}

}  // namespace
}  // namespace kvi4
