// pa_fp4.cuh -- 4-bit (E2M1) KV cache: conversions and the per-warp attention
// arithmetic over its tiles.
//
// A tile holds the 16 rows of one (block, KV head): the codes of the rows, D/2
// bytes each (element 2i in the low half of byte i), then the rows' scales, D/16
// bytes each: one E4M3 number for every 16 neighbouring elements.  With the head's
// float scale_j an element stands for E2M1(code) * E4M3(scale) * scale_j.  A tile is
// 9 D contiguous bytes, so one bulk copy fetches it.
//
// The first product is exact in f16 (an E2M1 value has two significant bits, an
// E4M3 one four; 2^-10 <= product <= 2688), so the tiles are dequantised to f16 in
// registers and both contractions run on the f16 tensor cores with fp32
// accumulation; scale_j folds into the score scale (keys) and the normalisation
// (values).  q is rounded to f16 once, P as it is used.
#pragma once

#include "pa_common.cuh"
#include "pa_decode.cuh"
#include "pa_fp8.cuh"
#include "pa_mma.cuh"

namespace pa {

struct e2m1 {                              // the cache's storage type, as a tag
    unsigned char byte;
};

// Bytes of one tile: 16 rows of D elements of KV.
template <typename KV, int D>
__host__ __device__ constexpr int tile_bytes() {
    return std::is_same<KV, e2m1>::value ? 9 * D : 16 * D * (int)sizeof(KV);
}

// A condition whose code the loop should not step over.
__device__ __forceinline__ bool rarely(bool c) { return __builtin_expect(c, 0); }

// The eight E2M1 codes of w as f16 pairs, byte i in r[i] (low half: low code).
__device__ __forceinline__ void f16x2_from_e2m1x8(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}

// Two binary32 values to E2M1 codes (nearest, ties to even, saturating at 6): lo in
// bits 0-3, hi in bits 4-7.
__device__ __forceinline__ uint32_t e2m1x2_from_f32(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 a;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.u32.u8 %0, a;\n\t}"
        : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// a times the low or the high half of s.
__device__ __forceinline__ uint32_t mul_by_half(uint32_t a, uint32_t s, bool hi) {
    const __half2 x = *reinterpret_cast<const __half2 *>(&a), y = *reinterpret_cast<const __half2 *>(&s);
    const __half2 r = __hmul2(x, hi ? __high2half2(y) : __low2half2(y));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// d = a . b on the f16 tensor cores.
__device__ __forceinline__ void mma_f16_first(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// A transposed 8 x 8 matrix of 16-bit elements: lane (g, t) gives row g, columns 2t
// and 2t + 1, and gets rows 2t and 2t + 1 of column g.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// Token of row r (0..7) of a score tile.  Every group of rows that one load
// instruction serves falls on distinct banks (or on two, for 8-byte loads of 64-byte
// rows): 0 and 1, 2 and 3, .. differ in parity; 0-3, 4-7, the even and the odd rows
// are all four residues of 4.
__device__ __forceinline__ int fp4_token(int r) { return r ^ ((r >> 2) & 1); }

// Attention of one warp over E2M1 tiles, for NT tiles of eight query rows that share
// a KV head: the G heads of one token (NT = 1), or 16 (token, head) pairs of a
// multi-token query (NT = 2) with a causal limit each.
//
// Both contractions have the tokens or head_dim on the 16-row side and the query
// rows on the 8-column side, so no half of a matrix instruction is padding:
//   S^T[token][row] = K Q^T    A: K as lane (g, t) holds it, rows fp4_token(g) and
//       8 more, D/4 neighbouring elements from (D/4) t (two groups at D = 128); the
//       order of elements in the product is free, q follows it
//   O^T[d][row] += V^T P^T     B: P^T, the transposed scores (two movmatrix a
//       tile); A: V^T, lane (g, t): elements (D/8) g .. of the tokens of rows 2t,
//       2t + 1, 8 + 2t and 9 + 2t
// Lane (g, t) holds rows 2t and 2t + 1 of each tile throughout (scores, statistics
// and outputs), so nothing is exchanged when a row is rescaled.
//
// A row's reference level moves only when a score exceeds it by more than
// F8_TOP_LOG2, as in WarpAttnF8x16; (m, l, acc) are to that level.
//
// Bound by instructions: a block of 16 keys takes about 330 (the conversions of its
// codes, at half rate, lead), issued on 0.55-0.58 of the cycles, where its 2.3 KB would
// come in two thirds of the time (serving mix of 256 sequences, 32 / 8 heads of 128: 48 us,
// the copies alone 41; 256 sequences of four rows: 71 and 49; eight of up to 131071
// keys, partitioned: 149 us = 4.3 TB/s, the copies alone 146, with partitions of 2048
// keys 109).  Two blocks at a time keep the chains of one beside the other's (54 us
// against 61).
template <typename T, int D, int NT, int R>
struct WarpAttnF4 {
    static_assert(sizeof(T) == 2, "q and out are 16-bit");
    static_assert(D == 64 || D == 128, "head_dim");
    static_assert(NT == 1 || R == 8, "rows of a tile: 8, or the G heads of one token");
    static constexpr int KS = D / 16;      // k-steps of the score product
    static constexpr int MT = D / 16;      // 16-row tiles of the value product
    static constexpr int DL = D / 8;       // elements of a lane in it
    static constexpr int ROWB = D / 2, OFF_SC = 16 * ROWB, SCB = D / 16;

    int lane, g, t;
    uint32_t qb[NT][KS][2];                // f16 B fragments
    // acc[n][mt]: elements DL g + 2mt (0, 1) and + 1 (2, 3) of rows 2t and 2t + 1
    float acc[NT][MT][4];
    // a row's level as what is added to its scores (minus it; 0 before the first one)
    // and the score that moves it (-inf before); this lane's part of its sum
    float down[NT][2], limit[NT][2], l_run[NT][2];
    int lim[NT][2];                        // last visible position, -1: no such row (multi-token queries)

    __device__ __forceinline__ void init(int lane_) {
        lane = lane_;
        g = lane >> 2;
        t = lane & 3;
        reset();
    }

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            down[n][0] = down[n][1] = 0.f;
            limit[n][0] = limit[n][1] = -INFINITY;
            l_run[n][0] = l_run[n][1] = 0.f;
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[n][j][e] = 0.f;
        }
    }

    // query row g of tile n (nullptr: no such row)
    __device__ __forceinline__ void load_row(int n, const T *q) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 x = q ? __ldg(reinterpret_cast<const uint4 *>(q + (D / 4) * t + 8 * i))
                              : make_uint4(0, 0, 0, 0);
            qb[n][2 * i][0] = WarpAttnF8<T, D, 1>::to_f16x2(x.x);
            qb[n][2 * i][1] = WarpAttnF8<T, D, 1>::to_f16x2(x.y);
            qb[n][2 * i + 1][0] = WarpAttnF8<T, D, 1>::to_f16x2(x.z);
            qb[n][2 * i + 1][1] = WarpAttnF8<T, D, 1>::to_f16x2(x.w);
        }
    }

    // Scores of a block's 16 tokens: v[n][0], [1]: token fp4_token(g) of rows 2t,
    // 2t + 1; [2], [3]: 8 tokens on.
    template <int CHAINS>
    __device__ __forceinline__ void scores(uint32_t kt, float2 (&v)[NT][2]) const {
        const int r0 = fp4_token(g);
        constexpr int W = D / 32;          // 32-bit words of codes of a row
        uint32_t w0[W], w1[W], s0, s1;
        if constexpr (D == 128) {
            const uint4 a = lds128(kt + r0 * ROWB + 16 * t), b = lds128(kt + (r0 + 8) * ROWB + 16 * t);
            w0[0] = a.x; w0[1] = a.y; w0[2] = a.z; w0[3] = a.w;
            w1[0] = b.x; w1[1] = b.y; w1[2] = b.z; w1[3] = b.w;
            s0 = f16x2_from_e4m3x2(lds16(kt + OFF_SC + r0 * SCB + 2 * t));
            s1 = f16x2_from_e4m3x2(lds16(kt + OFF_SC + (r0 + 8) * SCB + 2 * t));
        } else {
            const uint2 a = lds64(kt + r0 * ROWB + 8 * t), b = lds64(kt + (r0 + 8) * ROWB + 8 * t);
            w0[0] = a.x; w0[1] = a.y;
            w1[0] = b.x; w1[1] = b.y;
            s0 = f16x2_from_e4m3x2(lds8(kt + OFF_SC + r0 * SCB + t));
            s1 = f16x2_from_e4m3x2(lds8(kt + OFF_SC + (r0 + 8) * SCB + t));
        }
        float c[NT][CHAINS][4];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            // the low group's scale for the first half of the run, then the high one's
            const bool hi = D == 128 && i >= W / 2;
            uint32_t a[4], b[4];
            f16x2_from_e2m1x8(w0[i], a);
            f16x2_from_e2m1x8(w1[i], b);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = mul_by_half(a[e], s0, hi);
                b[e] = mul_by_half(b[e], s1, hi);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (i == 0) mma_f16_first(c[n][0], a[0], b[0], a[1], b[1], qb[n][0][0], qb[n][0][1]);
                else mma_f16(c[n][0], a[0], b[0], a[1], b[1], qb[n][2 * i][0], qb[n][2 * i][1]);
                if (i == 0 && CHAINS > 1)
                    mma_f16_first(c[n][CHAINS - 1], a[2], b[2], a[3], b[3], qb[n][1][0], qb[n][1][1]);
                else
                    mma_f16(c[n][CHAINS - 1], a[2], b[2], a[3], b[3], qb[n][2 * i + 1][0], qb[n][2 * i + 1][1]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                v[n][e] = make_float2(c[n][0][2 * e], c[n][0][2 * e + 1]);
                if (CHAINS > 1)
                    v[n][e] = add2(v[n][e], make_float2(c[n][CHAINS - 1][2 * e], c[n][CHAINS - 1][2 * e + 1]));
            }
    }

    // NB neighbouring blocks of a sequence with tiles kt, vt.  rows: tokens of each
    // that count (0..16, the first ones); pos0: the first one's position
    // (multi-token queries).  scale_log2 carries K's head scale.
    template <bool CAUSAL, int NB>
    __device__ __forceinline__ void step(const uint32_t (&kt)[NB], const uint32_t (&vt)[NB],
                                         const int (&rows)[NB], int pos0, float scale_log2) {
        float2 sc[NB][NT][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) scores<(NB * NT > 1 ? 1 : 2)>(kt[b], sc[b]);
        const float2 sl = make_float2(scale_log2, scale_log2);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) sc[b][n][e] = mul2(sc[b][n][e], sl);
        const int tok = fp4_token(g);
        bool part = false;                 // some block is not whole
#pragma unroll
        for (int b = 0; b < NB; ++b) part = part || rows[b] < 16;
        if constexpr (CAUSAL) {
            bool cut = part;
#pragma unroll
            for (int n = 0; n < NT; ++n) cut = cut || pos0 + 16 * NB - 1 > min(lim[n][0], lim[n][1]);
            if (rarely(__any_sync(0xffffffffu, cut))) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int i = tok + 8 * e, at = i < rows[b] ? pos0 + 16 * b + i : INT32_MAX;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            sc[b][n][e].x = at <= lim[n][0] ? sc[b][n][e].x : -INFINITY;
                            sc[b][n][e].y = at <= lim[n][1] ? sc[b][n][e].y : -INFINITY;
                        }
                    }
            }
        } else if (rarely(part)) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (tok + 8 * e >= rows[b]) sc[b][n][e] = make_float2(-INFINITY, -INFINITY);
        }
        bool above = false;
        float mx[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mx[n][0] = fmaxf(sc[0][n][0].x, sc[0][n][1].x);
            mx[n][1] = fmaxf(sc[0][n][0].y, sc[0][n][1].y);
            if constexpr (NB > 1) {
                mx[n][0] = max3f(mx[n][0], sc[NB - 1][n][0].x, sc[NB - 1][n][1].x);
                mx[n][1] = max3f(mx[n][1], sc[NB - 1][n][0].y, sc[NB - 1][n][1].y);
            }
            above = above || mx[n][0] > limit[n][0] || mx[n][1] > limit[n][1];
        }
        if (rarely(__any_sync(0xffffffffu, above))) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float m = mx[n][h];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    if (!(m > limit[n][h])) continue;
                    const float to = F8_BELOW_LOG2 - m;
                    const float alpha = limit[n][h] == -INFINITY ? 0.f : ex2(to - down[n][h]);
                    down[n][h] = to;
                    limit[n][h] = m + (F8_TOP_LOG2 - F8_BELOW_LOG2);
                    l_run[n][h] *= alpha;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        acc[n][mt][h] *= alpha;
                        acc[n][mt][2 + h] *= alpha;
                    }
                }
        }
        uint32_t pb[NB][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float2 nm = make_float2(down[n][0], down[n][1]);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 x = add2(sc[b][n][e], nm);
                    const uint32_t w = Mma<__half>::pack(ex2(x.x), ex2(x.y));
                    add_halves(l_run[n][0], l_run[n][1], w);       // the weights as they are used
                    pb[b][n][e] = transpose8(w);
                }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) values(vt[b], rows[b], pb[b]);
    }

    __device__ __forceinline__ void values(uint32_t vt, int rows, const uint32_t (&pb)[NT][2]) {
        const int tok[4] = {fp4_token(2 * t), fp4_token(2 * t + 1), 8 + fp4_token(2 * t), 8 + fp4_token(2 * t + 1)};
        constexpr int W = D / 64;          // 32-bit words of codes of a token
        uint32_t w[4][W], s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (D == 128) {
                const uint2 v = lds64(vt + tok[i] * ROWB + 8 * g);
                w[i][0] = v.x; w[i][1] = v.y;
                s[i] = lds8(vt + OFF_SC + tok[i] * SCB + g);
            } else {
                w[i][0] = lds32(vt + tok[i] * ROWB + 4 * g);
                s[i] = lds8(vt + OFF_SC + tok[i] * SCB + (g >> 1));
            }
        }
        // rows that do not count hold anything; their weight is 0, so what must not
        // stay is a scale that is NaN
        if (rarely(rows < 16)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = tok[i] < rows ? s[i] : 0u;
        }
        const uint32_t x01 = f16x2_from_e4m3x2(s[0] | (s[1] << 8)), x23 = f16x2_from_e4m3x2(s[2] | (s[3] << 8));
        constexpr uint32_t LO = 0x0f0f0f0fu;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            // byte e: the codes of two tokens, element 2 (4i + e) (even) and the one after
            uint32_t ea[4], oa[4], eb[4], ob[4];
            f16x2_from_e2m1x8((w[0][i] & LO) | ((w[1][i] << 4) & ~LO), ea);
            f16x2_from_e2m1x8(((w[0][i] >> 4) & LO) | (w[1][i] & ~LO), oa);
            f16x2_from_e2m1x8((w[2][i] & LO) | ((w[3][i] << 4) & ~LO), eb);
            f16x2_from_e2m1x8(((w[2][i] >> 4) & LO) | (w[3][i] & ~LO), ob);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t a0 = mul_f16x2(ea[e], x01), a1 = mul_f16x2(oa[e], x01);
                const uint32_t a2 = mul_f16x2(eb[e], x23), a3 = mul_f16x2(ob[e], x23);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(acc[n][4 * i + e], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            }
        }
    }

    // Sum the lanes of each row.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h)
            {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l_run[n][h] += __shfl_xor_sync(0xffffffffu, l_run[n][h], o);
            }
    }

    // The level of a row, -inf where it has none: nothing seen yet, if the sum is 0
    // (with a sum, of NaN, one that a merge does not take for an empty partial).
    __device__ __forceinline__ float level(int n, int h) const {
        return limit[n][h] == -INFINITY && l_run[n][h] == 0.f ? -INFINITY : -down[n][h];
    }

    // A partial, of 8 NT (NT = 1: R) rows of D floats: the accumulators as the lanes
    // hold them, (m, l) of the rows behind them; every warp's lie alike, so a merge
    // adds up what the same lane has stored.
    static constexpr int ROWS = NT > 1 ? 8 * NT : R;
    static constexpr int LANES = R > 1 ? 4 * R : 8;        // that hold rows
    static constexpr int HS = R > 1 ? 2 : 1;               // rows of a lane in a tile
    __device__ __forceinline__ bool holds() const { return 2 * t < R; }
    __device__ __forceinline__ int slot(int n, int mt) const {     // in floats
        return ((n * MT + mt) * LANES + (R > 1 ? g * (R / 2) + t : g)) * (R > 1 ? 4 : 2);
    }
    __device__ __forceinline__ void store_partial(float *P) const {
        if (!holds()) return;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if constexpr (R > 1)
                    *reinterpret_cast<float4 *>(P + slot(n, mt)) =
                        make_float4(acc[n][mt][0], acc[n][mt][1], acc[n][mt][2], acc[n][mt][3]);
                else
                    *reinterpret_cast<float2 *>(P + slot(n, mt)) = make_float2(acc[n][mt][0], acc[n][mt][2]);
            }
#pragma unroll
            for (int h = 0; h < (R > 1 ? 2 : 1); ++h) {
                if (g == 0) {
                    P[ROWS * D + 8 * n + 2 * t + h] = level(n, h);
                    P[ROWS * D + ROWS + 8 * n + 2 * t + h] = l_run[n][h];
                }
            }
        }
    }

    // The state becomes the merge of partials: merge_begin, merge_levels of all of
    // them, merge_add of all of them, merge_end.  Lane i of `which` gives where a partial
    // lies in shared memory (FAR: the cluster's); they are taken in the lanes' order, the
    // loads of two (of four, for the levels) in flight.
    template <bool FAR> __device__ __forceinline__ static float get(uint32_t at) {
        if constexpr (FAR) return ld_dsmem_f32(at);
        else return __uint_as_float(lds32(at));
    }
    template <bool FAR> __device__ __forceinline__ static float4 get4(uint32_t at) {
        if constexpr (FAR) return ld_dsmem_f32x4(at);
        const uint4 v = lds128(at);
        return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
    }
    float top[NT][2];
    __device__ __forceinline__ void merge_begin() {
        reset();
#pragma unroll
        for (int n = 0; n < NT; ++n) top[n][0] = top[n][1] = -INFINITY;
    }
    template <bool FAR>
    __device__ __forceinline__ void merge_levels(uint32_t at, unsigned which) {
        while (which) {
            uint32_t P[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {          // the last ones again where there are no more
                const int l = __ffs(which) - 1;
                P[i] = l >= 0 ? __shfl_sync(0xffffffffu, at, l & 31) : P[i ? i - 1 : 0];
                which &= which - 1;
            }
            if (holds()) {
                float m[4][NT][2];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int h = 0; h < HS; ++h) m[i][n][h] = get<FAR>(P[i] + (ROWS * D + 8 * n + 2 * t + h) * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int h = 0; h < HS; ++h) top[n][h] = fmaxf(top[n][h], m[i][n][h]);
            }
        }
    }
    template <bool FAR>
    __device__ __forceinline__ void merge_add(uint32_t at, unsigned which) {
        while (which) {
            const int l0 = __ffs(which) - 1;
            which &= which - 1;
            const int l1 = __ffs(which) - 1;       // -1: a single one
            which &= which - 1;
            uint32_t P[2];
            P[0] = __shfl_sync(0xffffffffu, at, l0);
            P[1] = __shfl_sync(0xffffffffu, at, l1 & 31);
            if (!holds()) continue;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float m[2][2], l[2][2];
                float4 a[2][MT];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (i == 1 && l1 < 0) break;
#pragma unroll
                    for (int h = 0; h < HS; ++h) {
                        m[i][h] = get<FAR>(P[i] + (ROWS * D + 8 * n + 2 * t + h) * 4);
                        l[i][h] = get<FAR>(P[i] + (ROWS * D + ROWS + 8 * n + 2 * t + h) * 4);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        if constexpr (R > 1) {
                            a[i][mt] = get4<FAR>(P[i] + slot(n, mt) * 4);
                        } else {
                            a[i][mt].x = get<FAR>(P[i] + slot(n, mt) * 4);
                            a[i][mt].z = get<FAR>(P[i] + slot(n, mt) * 4 + 4);
                            a[i][mt].y = a[i][mt].w = 0.f;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (i == 1 && l1 < 0) break;
                    float f[2] = {0.f, 0.f};
#pragma unroll
                    for (int h = 0; h < HS; ++h) {
                        f[h] = m[i][h] == -INFINITY ? 0.f : ex2(m[i][h] - top[n][h]);
                        l_run[n][h] = fmaf(f[h], l[i][h], l_run[n][h]);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        acc[n][mt][0] = fmaf(f[0], a[i][mt].x, acc[n][mt][0]);
                        acc[n][mt][1] = fmaf(f[1], a[i][mt].y, acc[n][mt][1]);
                        acc[n][mt][2] = fmaf(f[0], a[i][mt].z, acc[n][mt][2]);
                        acc[n][mt][3] = fmaf(f[1], a[i][mt].w, acc[n][mt][3]);
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void merge_end() {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < HS; ++h)
                if (top[n][h] != -INFINITY) {
                    down[n][h] = -top[n][h];
                    limit[n][h] = top[n][h];
                }
    }

    // After finish(): f(row, d, v, m, l) with the normalised outputs v[0 .. D/8) at d ..
    // of the rows that exist.
    template <typename Fn>
    __device__ __forceinline__ void for_each_row(Fn &&f) const {
        if (!holds()) return;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < (R > 1 ? 2 : 1); ++h) {
                if (NT > 1 && lim[n][h] < 0) continue;
                const float l = l_run[n][h], inv = l > 0.f ? 1.f / l : 0.f;
                float v[DL];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    v[2 * mt] = acc[n][mt][h] * inv;
                    v[2 * mt + 1] = acc[n][mt][2 + h] * inv;
                }
                f(8 * n + 2 * t + h, DL * g, v, level(n, h), l);
            }
    }
};

}  // namespace pa
