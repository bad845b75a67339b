// Cache write with the position rotation applied on the way: queries and keys are rotated by their
// tokens' positions, the queries stored back in their type, keys and values encoded into the paged
// cache as the plain write does.
//
// For a token at position p with the table row cs = cos_sin[p] (rot/2 cosines, then rot/2 sines, fp32),
// the first rot dimensions of a head vector x (upcast exactly to fp32) are rotated in pairs (a, b) =
// (x_i, x_{i + rot/2}), or (x_{2i}, x_{2i+1}) when INTER:
//   a' = fl(fl(a c_i) - fl(b s_i)),   b' = fl(fl(b c_i) + fl(a s_i))
// and the others are left.  Rotated keys go to the encoder as fp32 (no rounding to 16 bits in between,
// so the cache holds more of them than a separate rotation would leave); rotated queries are rounded
// once, to their type.  Every step is an explicit round-to-nearest operation, so the cache bytes are
// bit-exact with this definition followed by the plain write's.
//
// The work of one launch is two kinds of warp items: cache tiles (kTileVecs vectors, as the plain
// write's, numbered plane by plane so that a tile is all keys or all values) and query items (one token,
// kRows heads).  A warp alternates them in proportion, because a cache tile is bound by its instructions
// and a query item by memory.
//
// A key tile is rotated by the whole warp before its vectors are encoded: a lane owns two words (pairs of
// elements) of every row, holds their cosines and sines, signed with the Hadamard rotation's signs, in
// registers for as long as the token lasts (its heads are neighbouring rows), and writes the rotated
// elements as fp32 where the encoding lane pair reads them as the operands of its first butterflies.
// (Rotated by the encoding threads themselves, each of a pair did the whole row: 64 table loads per thread
// and tile, and 180 us for 65 536 tokens of 8 kv heads instead of 88.7 without a rotation.)
//
// AXES: positions on several axes (time, height, width).  Pair i takes its cosine and sine from the table row of
// its own axis's position; the axis of every pair is two bits of a kernel parameter.  Everything else is the same.
// The positions of a tile's tokens are spread over the lanes a tile ahead, and a lane whose pairs share an axis loads 16
// bytes of the table at once: 65 536 tokens, three axes, 32 q / 8 kv heads, and the rows read back, 392 us (521 with
// each pair's position looked up where it is used).
#pragma once

#include "write_common.cuh"

namespace kvi4 {
namespace {

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float2 x);
template <>
__device__ __forceinline__ uint32_t pack_pair<__nv_bfloat16>(float2 x) {
    __nv_bfloat162 h = __float22bfloat162_rn(x);
    return *reinterpret_cast<uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack_pair<__half>(float2 x) {
    __half2 h = __float22half2_rn(x);
    return *reinterpret_cast<uint32_t*>(&h);
}

// A packed sum joined with the packed products that feed it becomes one FMA whatever their rounding
// modifiers say (measured: 2 of 18 944 rotated fp16 queries differed in the last bit), so the sums of
// products are scalar operations, which the compiler never contracts.
__device__ __forceinline__ float2 sum_of_products(float2 xc, float2 ys) {
    return make_float2(__fadd_rn(xc.x, ys.x), __fadd_rn(xc.y, ys.y));
}
__device__ __forceinline__ float2 diff_of_products(float2 xc, float2 ys) {
    return make_float2(__fsub_rn(xc.x, ys.x), __fsub_rn(xc.y, ys.y));
}

// (a c - b s, b c + a s) for two pairs at once, each product and sum rounded on its own
__device__ __forceinline__ void turn2(float2 a, float2 b, float2 c, float2 s, float2& ra, float2& rb) {
    ra = diff_of_products(mul_f32x2(a, c), mul_f32x2(b, s));
    rb = sum_of_products(mul_f32x2(b, c), mul_f32x2(a, s));
}

__device__ __forceinline__ float4 ldg4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }

// Rotated rows of a key tile, fp32, in shared memory: row r at r * kRopeRow<D> floats, in the order
// [4k .. 4k + 3] = elements 2k, 2k + D/2, 2k + 1, 2k + 1 + D/2 (k < D/4): one 16-byte access holds the two
// operand pairs of the encoder's stride-1 butterflies P[k].
template <int D>
constexpr int kRopeRow = D + 4;   // padded: 16-byte accesses of 8 rows hit distinct banks
constexpr int kRopeRows = 16;     // rows staged at a time

// What a lane keeps of a token's table row: x' = x c + partner s for its two words.
struct RopeTable {
    float2 c[2], s[2];
};

// The axis of pair i.
__device__ __forceinline__ int axis_of(const RopeWriteParams& p, int i) { return (int)((p.pair_axis[i >> 4] >> (2 * (i & 15))) & 3u); }

// Positions of eight tokens at once: lane 4t + a holds that of token tok0 + t on axis a (0 past the last token or axis).
__device__ __forceinline__ int64_t axis_positions(const RopeWriteParams& p, uint32_t tok0) {
    const uint32_t tok = tok0 + ((threadIdx.x & 31) >> 2), a = threadIdx.x & 3;
    return (int)a < p.axes && tok < (uint32_t)p.w.num_tokens ? __ldg(p.positions + (int64_t)a * p.w.num_tokens + tok) : 0;
}

// A position's table row (row 0 for one outside the table: its token is not stored).  The host refuses tables of more
// than 2^32 rows.
__device__ __forceinline__ uint32_t table_row(const RopeWriteParams& p, int64_t pos) {
    return pos >= 0 && pos < p.max_position ? (uint32_t)pos : 0u;
}

// One position that stands for a token's positions on all axes: in the table when all of them are, negative when
// all of them are, else behind the table.
__device__ __forceinline__ int64_t joint_position(const RopeWriteParams& p, uint32_t tok) {
    bool inside = true, negative = true;
    for (int a = 0; a < p.axes; ++a) {
        const int64_t pos = __ldg(p.positions + (int64_t)a * p.w.num_tokens + tok);
        inside = inside && pos >= 0 && pos < p.max_position;
        negative = negative && pos < 0;
    }
    return inside ? 0 : negative ? -1 : p.max_position;
}

// The lane's part of a token's table rows: rows holds them as axis_positions does, the token is its t-th.  All lanes
// call it.
template <int D, bool INTER>
__device__ __forceinline__ RopeTable load_axes(const RopeWriteParams& p, uint32_t rows, uint32_t t) {
    constexpr int Q = D / 4;
    const int k = (threadIdx.x & 31) % Q, rot = p.rot, hw = rot >> 2, half = rot >> 1;
    auto row = [&](int pair) -> const float* {
        return p.cos_sin + (int64_t)__shfl_sync(0xffffffffu, rows, 4 * t + axis_of(p, pair)) * rot;
    };
    RopeTable r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int m = k + i * Q;
        const bool turned = 2 * m < rot;
        r.c[i] = make_float2(1.0f, 1.0f);
        r.s[i] = make_float2(0.0f, 0.0f);
        if constexpr (INTER) {
            const float* cs = row(turned ? m : 0);
            if (turned) {
                r.c[i].x = __ldg(cs + m);
                r.s[i].x = __ldg(cs + half + m);
            }
        } else {
            const int j = turned ? 2 * (m < hw ? m : m - hw) : 0;   // pairs j and j + 1
            const float *ca = row(j), *cb = row(j + 1);
            if (turned) {
                if (ca == cb) {
                    r.c[i] = __ldg(reinterpret_cast<const float2*>(ca + j));
                    r.s[i] = __ldg(reinterpret_cast<const float2*>(ca + half + j));
                } else {
                    r.c[i] = make_float2(__ldg(ca + j), __ldg(cb + j + 1));
                    r.s[i] = make_float2(__ldg(ca + half + j), __ldg(cb + half + j + 1));
                }
            }
        }
    }
    return r;
}

// The lane's part of the table row of position pos (row 0 for one outside the table: its rows are not stored).
template <int D, bool INTER>
__device__ __forceinline__ RopeTable load_table(const RopeWriteParams& p, int64_t pos) {
    constexpr int Q = D / 4;
    const int k = (threadIdx.x & 31) % Q, rot = p.rot, hw = rot >> 2;
    const float* cs = p.cos_sin + (pos >= 0 && pos < p.max_position ? pos : 0) * rot;
    RopeTable t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int m = k + i * Q;
        t.c[i] = make_float2(1.0f, 1.0f);
        t.s[i] = make_float2(0.0f, 0.0f);
        if (2 * m < rot) {
            if constexpr (INTER) {   // the sines' signs follow in rope_rows
                t.c[i].x = __ldg(cs + m);
                t.s[i].x = __ldg(cs + (rot >> 1) + m);
            } else {
                const int j = m < hw ? m : m - hw;
                t.c[i] = __ldg(reinterpret_cast<const float2*>(cs + 2 * j));
                t.s[i] = __ldg(reinterpret_cast<const float2*>(cs + (rot >> 1) + 2 * j));
            }
        }
    }
    return t;
}

// Rotate rows r0 .. r0 + nrows - 1 of the tile (vectors v0 + r of the key plane, staged at in + r * ROWPAD)
// into stage rows 0 .. nrows - 1, nrows <= kRopeRows.  tab: the table row of the first row's token; pos: lane
// r * TPV holds the position of row r's token (with AXES: rows holds the table rows of the tokens from tok0 on, as
// axis_positions does).  fmask: per word m the signs to apply (bit 15: element 2m, bit
// 31: 2m + 1), or nullptr for none.  All lanes call it.
template <int D, typename T, bool INTER, bool AXES, int ROWPAD, int TPV>
__device__ __forceinline__ void rope_rows(const RopeWriteParams& p, const uint8_t* in, float* stage, uint32_t v0, int r0,
                                          int nrows, RopeTable tab, int64_t pos, uint32_t rows, uint32_t tok0, const uint32_t* fmask) {
    constexpr int Q = D / 4, kStep = 32 / Q;   // rows at once: a lane owns words k and k + Q of every kStep-th row
    const int lane = threadIdx.x & 31, k = lane % Q, sub = lane / Q;
    const uint32_t H = (uint32_t)p.w.H;
    const int rot = p.rot, hw = rot >> 2;       // words of a half of the rotated elements
    int pw[2];            // the partner word (split pairing)
    bool turned[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int m = k + i * Q;
        turned[i] = 2 * m < rot;
        pw[i] = INTER || !turned[i] ? m : (m < hw ? m + hw : m - hw);
    }
    const bool full = !INTER && rot == D;   // the lane's two words are each other's partners
    const uint32_t* src = reinterpret_cast<const uint32_t*>(in + r0 * ROWPAD);
    constexpr int kRowWords = ROWPAD / 4;
    int r = 0, r_end = (int)(H - (v0 + r0) % H);   // rows of the first token
    uint32_t tok = AXES ? (v0 + (uint32_t)r0) / H : 0u;
    while (r < nrows) {
        // a token's rows r .. r_end - 1, the next token's table row on its way
        if (r_end > nrows) r_end = nrows;
        RopeTable next = tab;
        if (r_end < nrows) {
            if constexpr (AXES) {
                if (++tok >= tok0 + 8) {   // (one or two kv heads)
                    tok0 = tok;
                    rows = table_row(p, axis_positions(p, tok));
                }
                next = load_axes<D, INTER>(p, rows, tok - tok0);
            } else next = load_table<D, INTER>(p, __shfl_sync(0xffffffffu, pos, (r0 + r_end) * TPV));
        }
        float2 c[2], s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = k + i * Q;
            c[i] = tab.c[i];
            s[i] = tab.s[i];
            if (turned[i]) {
                if constexpr (INTER) {
                    c[i].y = c[i].x;
                    s[i] = make_float2(-s[i].x, s[i].x);
                } else if (m < hw) {
                    s[i] = make_float2(-s[i].x, -s[i].y);
                }
            }
            if (fmask != nullptr) {   // products with the signed values round as the plain ones
                const uint32_t f = fmask[m], se = (f << 16) & 0x80000000u, so = f & 0x80000000u;
                c[i] = make_float2(__uint_as_float(__float_as_uint(c[i].x) ^ se), __uint_as_float(__float_as_uint(c[i].y) ^ so));
                s[i] = make_float2(__uint_as_float(__float_as_uint(s[i].x) ^ se), __uint_as_float(__float_as_uint(s[i].y) ^ so));
            }
        }
        if (full) {
#pragma unroll 4
            for (int q = r + sub; q < r_end; q += kStep) {
                const float2 x = upcast_pair<T>(src[q * kRowWords + k]), y = upcast_pair<T>(src[q * kRowWords + k + Q]);
                const float2 a = sum_of_products(mul_f32x2(x, c[0]), mul_f32x2(y, s[0]));
                const float2 b = sum_of_products(mul_f32x2(y, c[1]), mul_f32x2(x, s[1]));
                *reinterpret_cast<float4*>(stage + q * kRopeRow<D> + 4 * k) = make_float4(a.x, b.x, a.y, b.y);
            }
        } else {
#pragma unroll 2
            for (int q = r + sub; q < r_end; q += kStep) {
                float2 y[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 x = upcast_pair<T>(src[q * kRowWords + k + i * Q]);
                    float2 o;
                    if constexpr (INTER) o = make_float2(x.y, x.x);
                    else o = upcast_pair<T>(src[q * kRowWords + pw[i]]);
                    // c holds an unrotated word's signs; a product with its sine of 0 would make NaN of an infinity
                    const float2 xc = mul_f32x2(x, c[i]), z = sum_of_products(xc, mul_f32x2(o, s[i]));
                    y[i] = turned[i] ? z : xc;
                }
                *reinterpret_cast<float4*>(stage + q * kRopeRow<D> + 4 * k) = make_float4(y[0].x, y[1].x, y[0].y, y[1].y);
            }
        }
        tab = next;
        r = r_end;
        r_end += (int)H;
    }
}

// One thread's stride-1 outputs of a rotated key row (its signs are applied).
template <int D>
__device__ __forceinline__ void form_staged_half(const float* row, int t, float2 (&P)[D / 4]) {
    const float2 ts = t ? make_float2(-1.0f, -1.0f) : make_float2(1.0f, 1.0f);
#pragma unroll
    for (int k = 0; k < D / 4; ++k) {
        const float4 f = *reinterpret_cast<const float4*>(row + 4 * k);
        P[k] = fma_f32x2(make_float2(f.z, f.w), ts, make_float2(f.x, f.y));   // the product with +-1 is exact
    }
}

// The same for a value row as it comes.  fmask[m] (this thread's parity): bit 15 = sign of element 2m, bit
// 31 = sign of element 2m + 1 times (t ? -1 : +1).
template <int D, typename T>
__device__ __forceinline__ void form_plain_half(const uint32_t* row, const uint32_t* fmask, float2 (&P)[D / 4]) {
    constexpr int Q = D / 4;
#pragma unroll
    for (int k = 0; k < Q; k += 4) {
        const uint4 lo = *reinterpret_cast<const uint4*>(row + k), hi = *reinterpret_cast<const uint4*>(row + k + Q);
        const uint4 ml = *reinterpret_cast<const uint4*>(fmask + k), mh = *reinterpret_cast<const uint4*>(fmask + k + Q);
        const uint32_t wl[4] = {lo.x ^ ml.x, lo.y ^ ml.y, lo.z ^ ml.z, lo.w ^ ml.w};
        const uint32_t wh[4] = {hi.x ^ mh.x, hi.y ^ mh.y, hi.z ^ mh.z, hi.w ^ mh.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 a = upcast_pair<T>(wl[e]), b = upcast_pair<T>(wh[e]);
            P[k + e] = add_f32x2(make_float2(a.x, b.x), make_float2(a.y, b.y));
        }
    }
}

// Query items: kRows heads of one token, kPass rows (32 lanes, two 16-byte chunks each) at a time.
template <int D>
struct QueryItem {
    static constexpr int kSlots = D / 16;          // lanes per row
    static constexpr int kPassRows = 32 / kSlots;  // rows a warp holds at once
    static constexpr int kPasses = 2;
    static constexpr int kRows = kPassRows * kPasses;
};

template <int D, typename T, bool INTER, bool AXES>
__device__ __forceinline__ void rotate_queries(const RopeWriteParams& p, uint32_t item, uint32_t groups) {
    using Qi = QueryItem<D>;
    const int lane = threadIdx.x & 31, c = lane % Qi::kSlots, r = lane / Qi::kSlots;
    const uint32_t tok = item / groups, head0 = (item - tok * groups) * Qi::kRows;
    // (with AXES the lanes hold the token's positions, 0 past the last axis)
    const int64_t pos = AXES ? (lane < p.axes ? __ldg(p.positions + (int64_t)lane * p.w.num_tokens + tok) : 0) : __ldg(p.positions + tok);
    const bool out = pos < 0 || pos >= p.max_position;
    if (AXES ? __any_sync(0xffffffffu, out) : out) return;   // the cache tiles count it
    const int rot = p.rot;
    const bool turned = 16 * c < rot;
    // this lane's chunks of eight elements: a rotated lane holds the pairs 8c .. 8c + 7
    int ca, cb;
    if (INTER || !turned) {
        ca = 2 * c;
        cb = ca + 1;
    } else {
        ca = c;
        cb = c + (rot >> 4);
    }
    // the row's chunks are shared out among its lanes: rot / 16 rotated lanes own the first rot / 8
    // chunks, the others two neighbouring chunks behind them (2c, 2c + 1 in both cases)
    const T* src = static_cast<const T*>(p.q) + (int64_t)tok * p.q_stride;
    T* dst = static_cast<T*>(p.q_out) + (int64_t)tok * p.qo_stride;
    uint4 a[Qi::kPasses], b[Qi::kPasses];
#pragma unroll
    for (int i = 0; i < Qi::kPasses; ++i) {
        const int head = (int)head0 + i * Qi::kPassRows + r;
        if (head < p.Hq) {
            const uint4* row = reinterpret_cast<const uint4*>(src + (int64_t)head * D);
            a[i] = row[ca];
            b[i] = row[cb];
        }
    }
    float2 cv[4], sv[4];
    if constexpr (AXES) {
        // the axes of this lane's eight pairs: mostly the same, or at least those of the warp's lanes one each
        const uint32_t ax = (p.pair_axis[(c >> 1) & 3] >> (16 * (c & 1))) & (turned ? 0xFFFFu : 0u);
        if (__all_sync(0xffffffffu, ax == (ax & 3u) * 0x5555u)) {
            const float* cs = p.cos_sin + (int64_t)__shfl_sync(0xffffffffu, (uint32_t)pos, ax & 3u) * rot;
            if (turned) {
                const float4 c0 = ldg4(cs + 8 * c), c1 = ldg4(cs + 8 * c + 4);
                const float4 s0 = ldg4(cs + (rot >> 1) + 8 * c), s1 = ldg4(cs + (rot >> 1) + 8 * c + 4);
                cv[0] = make_float2(c0.x, c0.y), cv[1] = make_float2(c0.z, c0.w);
                cv[2] = make_float2(c1.x, c1.y), cv[3] = make_float2(c1.z, c1.w);
                sv[0] = make_float2(s0.x, s0.y), sv[1] = make_float2(s0.z, s0.w);
                sv[2] = make_float2(s1.x, s1.y), sv[3] = make_float2(s1.z, s1.w);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = 8 * c + 2 * e, half = rot >> 1;   // pairs j and j + 1
                const float* ra = p.cos_sin + (int64_t)__shfl_sync(0xffffffffu, (uint32_t)pos, (ax >> (4 * e)) & 3u) * rot;
                const float* rb = p.cos_sin + (int64_t)__shfl_sync(0xffffffffu, (uint32_t)pos, (ax >> (4 * e + 2)) & 3u) * rot;
                if (turned) {
                    cv[e] = make_float2(__ldg(ra + j), __ldg(rb + j + 1));
                    sv[e] = make_float2(__ldg(ra + half + j), __ldg(rb + half + j + 1));
                }
            }
        }
    } else if (turned) {
        const float* cs = p.cos_sin + pos * rot;
        const float4 c0 = ldg4(cs + 8 * c), c1 = ldg4(cs + 8 * c + 4);
        const float4 s0 = ldg4(cs + (rot >> 1) + 8 * c), s1 = ldg4(cs + (rot >> 1) + 8 * c + 4);
        cv[0] = make_float2(c0.x, c0.y), cv[1] = make_float2(c0.z, c0.w);
        cv[2] = make_float2(c1.x, c1.y), cv[3] = make_float2(c1.z, c1.w);
        sv[0] = make_float2(s0.x, s0.y), sv[1] = make_float2(s0.z, s0.w);
        sv[2] = make_float2(s1.x, s1.y), sv[3] = make_float2(s1.z, s1.w);
    }
#pragma unroll
    for (int i = 0; i < Qi::kPasses; ++i) {
        const int head = (int)head0 + i * Qi::kPassRows + r;
        if (head >= p.Hq) continue;
        if (turned) {
            uint32_t wa[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, wb[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
            if constexpr (INTER) {
                // pairs 8c + e sit in word e of the first chunk (e < 4) or word e - 4 of the second
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float ca_ = (e & 1) ? cv[e / 2].y : cv[e / 2].x, sa_ = (e & 1) ? sv[e / 2].y : sv[e / 2].x;
                    const float cb_ = (e & 1) ? cv[2 + e / 2].y : cv[2 + e / 2].x, sb_ = (e & 1) ? sv[2 + e / 2].y : sv[2 + e / 2].x;
                    const float2 x = upcast_pair<T>(wa[e]), y = upcast_pair<T>(wb[e]);
                    float2 ra, rb;   // pair e of both chunks at once
                    turn2(make_float2(x.x, y.x), make_float2(x.y, y.y), make_float2(ca_, cb_), make_float2(sa_, sb_), ra, rb);
                    wa[e] = pack_pair<T>(make_float2(ra.x, rb.x));
                    wb[e] = pack_pair<T>(make_float2(ra.y, rb.y));
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 ra, rb;
                    turn2(upcast_pair<T>(wa[e]), upcast_pair<T>(wb[e]), cv[e], sv[e], ra, rb);
                    wa[e] = pack_pair<T>(ra);
                    wb[e] = pack_pair<T>(rb);
                }
            }
            a[i] = make_uint4(wa[0], wa[1], wa[2], wa[3]);
            b[i] = make_uint4(wb[0], wb[1], wb[2], wb[3]);
        }
        uint4* row = reinterpret_cast<uint4*>(dst + (int64_t)head * D);
        row[ca] = a[i];
        row[cb] = b[i];
    }
}

// Resident CTAs per SM (register and shared-memory budget).
template <int BITS>
constexpr int kRopeBlocks = BITS == 8 ? 3 : 4;

// Shared memory of a warp: one tile of inputs, and the rotated rows, whose space holds the encoded rows once
// the tile is in registers.
template <int D, int BITS>
struct RopeSmem {
    static constexpr int TV = WriteShape<BITS>::kTileVecs;
    static constexpr int kRowPad = 2 * D + 16;
    static constexpr int kIn = TV * kRowPad;
    static constexpr int kStage = kRopeRows * kRopeRow<D> * 4;
    static_assert(TV * (D * BITS / 8 + 4) <= kStage, "encoded rows");
    static constexpr int kPerWarp = kIn + kStage;
    static constexpr int kBars = kWriteWarps * kPerWarp;   // one mbarrier per warp
    static constexpr int kBytes = kBars + kWriteWarps * 16 + (int)sizeof(WriteSigns<D>);
};

template <int D, typename T, int BITS, bool INTER, bool AXES>
__global__ void __launch_bounds__(kWriteThreads, kRopeBlocks<BITS>)
    rope_write_kernel(const __grid_constant__ RopeWriteParams p) {
    using Sh = WriteShape<BITS>;
    constexpr bool INT8 = BITS == 8;
    constexpr int TPV = Sh::kTpv, TV = Sh::kTileVecs;
    constexpr int RB = D * BITS / 8 + 4;             // cache row bytes
    constexpr int NW = RB / 4 - 1;                   // code words per row (then the scale)
    constexpr int OW = INT8 ? NW + 1 : NW / 2 + 1;   // words one thread stores (the last: the scale word)
    using Sm = RopeSmem<D, BITS>;
    extern __shared__ __align__(128) uint8_t smem[];
    // The previous kernel may produce any of the inputs.  Unlike the plain write, this kernel lets no
    // dependent start early.
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int vl = lane / TPV, part = lane % TPV;   // this thread's vector of the tile and its part
    uint8_t* in = smem + warp * Sm::kPerWarp;
    float* stage = reinterpret_cast<float*>(in + Sm::kIn);
    uint8_t* obuf = in + Sm::kIn;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + Sm::kBars) + warp * 2;   // this warp's inputs have landed
    WriteSigns<D>& sgn = *reinterpret_cast<WriteSigns<D>*>(smem + Sm::kBars + kWriteWarps * 16);
    if (lane == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
    }
    for (int j = tid; j < (INT8 ? 0 : D / 2); j += kWriteThreads) {   // INT8 rows take no signs
        const float s0 = p.w.signs[2 * j], s1 = p.w.signs[2 * j + 1];
        const uint32_t m = ((__float_as_uint(s0) >> 31) << 15) | ((__float_as_uint(s1) >> 31) << 31);
        sgn.xmask[0][j] = m;
        sgn.xmask[1][j] = m ^ 0x80000000u;
        if (blockIdx.x == 0 && ((fabsf(s0) != 1.0f) || (fabsf(s1) != 1.0f))) count_status(p.w.status, 4);
    }
    __syncthreads();

    const uint32_t H = (uint32_t)p.w.H;
    const int hshift = (H & (H - 1)) == 0 ? __ffs(H) - 1 : -1;   // -1: not a power of two
    const uint32_t nplane = (uint32_t)p.w.num_tokens * H, nvec = 2 * nplane;
    // vectors are numbered (plane * num_tokens + token) * H + head
    auto split = [&](uint32_t v, uint32_t& tok, uint32_t& h, uint32_t& pl) {
        pl = v >= nplane ? 1u : 0u;
        const uint32_t u = v - (pl ? nplane : 0u);
        tok = hshift >= 0 ? u >> hshift : u / H;
        h = u - tok * H;
    };
    const uint32_t ntiles = (nvec + TV - 1) / TV;
    const uint32_t gwarp = blockIdx.x * kWriteWarps + warp, nwarps = gridDim.x * kWriteWarps;
    const uint32_t group_bytes = H * RB;
    const bool grouped = hshift >= 0 && H <= (uint32_t)TV && (group_bytes % 16) == 0;
    const uint8_t* kin = static_cast<const uint8_t*>(p.w.k);
    const uint8_t* vin = static_cast<const uint8_t*>(p.w.v);
    const int64_t kst = p.k_stride * 2, vst = p.v_stride * 2;   // bytes per token

    // this warp's query items: the warps behind the last tile's start first
    const uint32_t groups = ((uint32_t)p.Hq + QueryItem<D>::kRows - 1) / QueryItem<D>::kRows;
    const uint32_t nitems = (uint32_t)p.w.num_tokens * groups;
    uint32_t item = (gwarp + nwarps - ntiles % nwarps) % nwarps;
    const uint32_t my_tiles = gwarp < ntiles ? (ntiles - gwarp - 1) / nwarps + 1 : 0u;
    const uint32_t my_items = item < nitems ? (nitems - item - 1) / nwarps + 1 : 0u;
    uint32_t items_done = 0;

    // lane i < TV copies vector i of the tile (2D bytes) into row i of the buffer
    auto prefetch = [&](uint32_t tile) {
        const uint32_t v0 = tile * TV;
        const uint32_t live_vecs = min((uint32_t)TV, nvec - v0);
        if (lane == 0) mbar_arrive_expect_tx(bar, live_vecs * (uint32_t)(D * 2));
        __syncwarp();
        if ((uint32_t)lane < live_vecs) {
            uint32_t tok, h, pl;
            split(v0 + lane, tok, h, pl);
            const uint8_t* src = (pl ? vin + (int64_t)tok * vst : kin + (int64_t)tok * kst) + (int64_t)h * (D * 2);
            bulk_copy_g2s(in + lane * Sm::kRowPad, src, D * 2, bar, policy_evict_first());
        }
    };

    uint32_t tile = gwarp;
    uint32_t it = 0;
    bool waited_out = false;
    // position and slot of this lane's vector of a tile (past the end: the tile's first vector), loaded one
    // tile ahead with its rows
    auto indices = [&](uint32_t tile, int64_t& pos, int64_t& slot) {
        const uint32_t v = tile * TV + vl;
        uint32_t tok, h, pl;
        split(v < nvec ? v : tile * TV, tok, h, pl);
        if constexpr (AXES) {
            uint32_t tok0;
            split(tile * TV, tok0, h, pl);
            pos = axis_positions(p, tok0);   // of the tile's first eight tokens (of the plane it begins in)
        } else pos = __ldg(p.positions + tok);
        slot = __ldg(p.w.slots + tok);
    };
    // The lane's table entries of vector v of the key plane; pos: lane src holds its token's position (with AXES: rows and
    // tok0 as rope_rows takes them).
    auto table_of = [&](uint32_t v, int64_t pos, int src, uint32_t rows, uint32_t tok0) -> RopeTable {
        if constexpr (AXES) {
            const uint32_t tok = v / H;
            if (tok >= tok0 + 8) return load_axes<D, INTER>(p, table_row(p, axis_positions(p, tok)), 0);
            return load_axes<D, INTER>(p, rows, tok - tok0);
        } else return load_table<D, INTER>(p, __shfl_sync(0xffffffffu, pos, src));
    };
    int64_t pos_next = 0, slot_next = 0;
    if (my_tiles > 0) {
        prefetch(tile);
        indices(tile, pos_next, slot_next);
    }
    for (; it < my_tiles; tile += nwarps, ++it) {
        int64_t pos = pos_next;
        const int64_t slot = slot_next;
        const uint32_t v0 = tile * TV, v = v0 + vl;
        const bool live = v < nvec;
        uint32_t rows = 0, tok0 = 0;
        if constexpr (AXES) {   // the table rows of the tile's first tokens, and what stands for this vector's positions
            uint32_t tok, h, pl;
            split(v0, tok0, h, pl);
            split(live ? v : v0, tok, h, pl);
            const bool none = (lane & 3) >= p.axes;
            const uint32_t in = __ballot_sync(0xffffffffu, none || (pos >= 0 && pos < p.max_position));
            const uint32_t neg = __ballot_sync(0xffffffffu, none || pos < 0);
            rows = table_row(p, pos);
            const uint32_t t = tok - tok0;
            pos = t < 8u ? (((in >> (4 * t)) & 15u) == 15u ? 0 : ((neg >> (4 * t)) & 15u) == 15u ? -1 : p.max_position) : joint_position(p, tok);
        }
        const int keys = v0 < nplane ? (int)min((uint32_t)TV, nplane - v0) : 0;   // key rows of the tile, its first ones
        RopeTable tab = {};
        if (keys > 0) tab = table_of(v0, pos, 0, rows, tok0);
        // this tile's share of the query items
        const uint32_t until = (uint32_t)((uint64_t)my_items * (it + 1) / my_tiles);
        for (; items_done < until; ++items_done, item += nwarps) rotate_queries<D, T, INTER, AXES>(p, item, groups);
        __syncwarp();
        if (__any_sync(0xffffffffu, !mbar_wait(bar, it & 1u))) {
            if (lane == 0) count_status(p.w.status, 3);
            waited_out = true;
            break;
        }
        // the previous tile's bulk stores have read the staged rows
        if (grouped) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        uint32_t tok = 0, h = 0, pl = 0;
        split(live ? v : v0, tok, h, pl);   // past the end: the tile's first vector, its words discarded
        // a token outside the table is skipped whole; a padding token (no slot, no position) is not counted
        const bool placed = pos >= 0 && pos < p.max_position;
        if (!placed && live && pl == 0 && h == 0 && part == 0 && (pos >= 0 || slot >= 0)) count_status(p.w.status, 5);
        const int row = live ? vl : 0;
        uint32_t words[OW];
        if constexpr (INT8) {
            float u[D];
            for (int r0 = 0; r0 < keys; r0 += kRopeRows) {
                if (r0 > 0) tab = table_of(v0 + (uint32_t)r0, pos, r0 * TPV, rows, tok0);
                rope_rows<D, T, INTER, AXES, Sm::kRowPad, TPV>(p, in, stage, v0, r0, min(kRopeRows, keys - r0), tab, pos, rows, tok0, nullptr);
                __syncwarp();
                if (row >= r0 && row < min(r0 + kRopeRows, keys)) {
#pragma unroll
                    for (int k = 0; k < D / 4; ++k) {
                        const float4 f = *reinterpret_cast<const float4*>(stage + (row - r0) * kRopeRow<D> + 4 * k);
                        u[2 * k] = f.x;
                        u[2 * k + D / 2] = f.y;
                        u[2 * k + 1] = f.z;
                        u[2 * k + 1 + D / 2] = f.w;
                    }
                }
                __syncwarp();
            }
            if (row >= keys) load_vector_raw<D, T>(reinterpret_cast<const uint4*>(in + row * Sm::kRowPad), u);
            __syncwarp();   // the tile is in registers
            if (it + 1 < my_tiles) {
                prefetch(tile + nwarps);
                indices(tile + nwarps, pos_next, slot_next);
            }
            if (live) encode_vector_int8<D>(u, words);
        } else {
            // every lane runs the encoder (it exchanges values within the lane pair)
            float2 P[D / 4];
            if (keys > 0) {
                rope_rows<D, T, INTER, AXES, Sm::kRowPad, TPV>(p, in, stage, v0, 0, keys, tab, pos, rows, tok0, sgn.xmask[0]);
                __syncwarp();
            }
            if (row < keys) form_staged_half<D>(stage + row * kRopeRow<D>, part, P);
            else form_plain_half<D, T>(reinterpret_cast<const uint32_t*>(in + row * Sm::kRowPad), sgn.xmask[part], P);
            __syncwarp();   // the tile is in registers
            if (it + 1 < my_tiles) {
                prefetch(tile + nwarps);
                indices(tile + nwarps, pos_next, slot_next);
            }
            butterflies_half<D>(p.w.c, P);
            if constexpr (BITS == 2) quantise_half_int2<D>(P, part, words);
            else quantise_half<D>(P, part, words);
        }
        // this thread's words of the row: all of them (INT8), or the first / second half of the code
        // words (INT4 / INT2 parts 0 / 1; part 1 also the scale word)
        const int w0 = INT8 ? 0 : part * (NW / 2);
        const int nw = INT8 ? OW : (part ? OW : OW - 1);
        const bool in_range = slot < p.w.num_slots;
        if (!in_range && placed && live && pl == 0 && h == 0 && part == 0) count_status(p.w.status, 0);
        const bool store = live && placed && slot >= 0 && in_range;
        const int64_t blk = slot / kBlockSize, off = slot % kBlockSize;
        if (grouped) {
            uint32_t* orow = reinterpret_cast<uint32_t*>(obuf + vl * RB) + w0;
            if (live) {
#pragma unroll
                for (int wi = 0; wi < OW; ++wi)
                    if (wi < nw) orow[wi] = words[wi];
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // staged rows -> bulk store
            __syncwarp();
            // the first thread of each row group stores the whole group
            if (store && h == 0 && part == 0)
                bulk_store_s2g(p.w.cache + ((blk * 2 + pl) * kBlockSize + off) * (int64_t)group_bytes, obuf + vl * RB, group_bytes);
        } else if (store) {
            uint32_t* orow = reinterpret_cast<uint32_t*>(p.w.cache + (((blk * 2 + pl) * kBlockSize + off) * (int64_t)H + h) * RB) + w0;
#pragma unroll
            for (int wi = 0; wi < OW; ++wi)
                if (wi < nw) orow[wi] = words[wi];
        }
    }
    if (waited_out) (void)mbar_wait(bar, it & 1u);   // let the copy in flight land before the warp exits
    for (; items_done < my_items; ++items_done, item += nwarps) rotate_queries<D, T, INTER, AXES>(p, item, groups);
    if (grouped) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <int D, typename T, int BITS, bool INTER, bool AXES>
cudaError_t launch_rope_write_t(const RopeWriteParams& p, cudaStream_t stream) {
    using Sh = WriteShape<BITS>;
    using Sm = RopeSmem<D, BITS>;
    const int64_t ntiles = (p.w.num_tokens * p.w.H * 2 + Sh::kTileVecs - 1) / Sh::kTileVecs;
    const int64_t groups = (p.Hq + QueryItem<D>::kRows - 1) / QueryItem<D>::kRows;
    const int64_t blocks = (ntiles + p.w.num_tokens * groups + kWriteWarps - 1) / kWriteWarps;
    const int64_t cap = (int64_t)num_sms() * kRopeBlocks<BITS>;
    cudaError_t err = opt_in_smem<rope_write_kernel<D, T, BITS, INTER, AXES>>(Sm::kBytes);
    if (err != cudaSuccess) return err;
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
    return cudaLaunchKernelEx(&cfg, rope_write_kernel<D, T, BITS, INTER, AXES>, p);
}

// Every (head size, type, pairing) instantiation of one cache mode.
template <int BITS, bool AXES = false>
cudaError_t launch_rope_write_mode(const RopeWriteParams& p, int head_size, DType dt, bool inter, cudaStream_t s) {
    if (head_size == 128) {
        if (dt == DType::BF16)
            return inter ? launch_rope_write_t<128, __nv_bfloat16, BITS, true, AXES>(p, s)
                         : launch_rope_write_t<128, __nv_bfloat16, BITS, false, AXES>(p, s);
        return inter ? launch_rope_write_t<128, __half, BITS, true, AXES>(p, s)
                     : launch_rope_write_t<128, __half, BITS, false, AXES>(p, s);
    }
    if (dt == DType::BF16)
        return inter ? launch_rope_write_t<64, __nv_bfloat16, BITS, true, AXES>(p, s)
                     : launch_rope_write_t<64, __nv_bfloat16, BITS, false, AXES>(p, s);
    return inter ? launch_rope_write_t<64, __half, BITS, true, AXES>(p, s)
                 : launch_rope_write_t<64, __half, BITS, false, AXES>(p, s);
}

}  // namespace
}  // namespace kvi4
