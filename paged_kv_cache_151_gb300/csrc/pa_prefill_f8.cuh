// pa_prefill_f8.cuh -- multi-token queries with many rows per sequence (a chunk
// of a prompt) over E4M3 caches, on the fifth-generation tensor cores.
//
// "vLLM: Architecture, PagedAttention & Internals", *Prefill, decode, and
// chunked prefill*.  Row r of sequence s's run (token i = r / G, head r % G of
// the KV head's group) attends over positions 0 .. L - n + i.  As in the
// decode path every code is exactly an f16 value, so q is rounded to f16, the
// codes are converted on the way into shared memory and both products run as
// kind::f16 with fp32 accumulation; K's scale folds into the score scale and
// V's into the final normalisation.
//
// A work item is 256 rows of one (sequence, KV head), as two tiles of 128 rows
// (the M side of an MMA), so that every key is loaded and converted once for
// 256 rows; one block per SM works through its items, 64 keys a step:
//   S = Q K^T   M = 128, N = 64, K = head_dim: the first 64 elements of Q from
//               TMEM (written there once per item by the threads that own its
//               rows), the rest and K from shared memory.  With all of Q in
//               shared memory the product would read 192 bytes a clock, more
//               than the 128 that there are.
//   softmax     one thread per row (four warps a tile): 64 scores from TMEM --
//               after which the next step's S may overwrite them -- causal
//               mask, online softmax in fp32 with lazy rescaling, P as f16
//               pairs to TMEM once P V of the step before is done
//   O += P V    M = 128, N = head_dim, K = 64: P from TMEM, V from shared memory
//               MN-major; O stays in TMEM over the item
// TMEM columns: S of tile 0 and 1 (64 each), P (32 each), O (head_dim each),
// Q (32 each): 512 at head_dim 128.  S of the next step is in place when a
// softmax warp comes back for it, so neither the tensor pipe nor the softmax
// warps wait for a whole chain of S, softmax and P V.  (P over the scores' own
// columns, with all of Q in TMEM, ties the three into one chain: a step of
// both tiles took 3160 clocks, the two tiles in step with each other.)
//
// A cluster of C blocks (1, 2 or 4) shares an item by its keys where the items
// alone would leave SMs idle: each block takes n / C consecutive steps, and at
// the end block r owns head_dim / C columns of O: every softmax thread writes
// the other blocks' columns of its row, and its (m, l), into their shared memory,
// and merges its own columns in the order of the ranks (so the result is a
// function of the sizes and of C only).
//
// Roles of the 16 warps: 0-3 and 4-7 softmax of tile 0 and 1; 8, 9 convert K and
// 10, 11 V (32 rows of a step each: 16-byte loads of codes two steps ahead in
// registers, f16 to the 128-byte swizzled stages of K and V); lane 0 of warps 12
// and 13 issues S of tile 0 and 1, of warps 14 and 15 P V (an issue blocks while
// the pipe is busy, so one warp for both would hold the next S back behind a
// P V, or the reverse).  Completion comes back through tcgen05.commit on
// mbarriers; one lane of a warp polls.  Every wait is bounded; on a timeout the
// block stops and the error word says so.
//
// Measured: 2048 rows of 32 query heads (8 KV heads of 128) over 14 to 16 thousand
// keys 510 us a call over three sets of inputs in turn: 1.00 PFLOP/s, 0.53 of the
// measured bf16 peak (467 us over one set, whose codes stay in L2); 256 items are
// 1.68 waves of the 152 SMs, so the SMs that work run at 0.63.  Three
// runs of 200 to 500 tokens (16 heads over 2, head_dim 64) over up to 6000 keys:
// 54.6 us.  Over E2M1 caches 3008 rows (f16) of 32 heads over up to 16000 keys take
// 357 us, 0.99 PFLOP/s: half the bytes, the same steps.  A step of one tile alone takes 0.82 us and not for its arithmetic
// (without the exponentials, the maximum or the sum 0.80 us and more): what is
// left is the chain S, wait, load, softmax, wait, store, P V and the converters'
// loads, which were not timed apart.  Short lists of items are bound by the step.
// Summing the weights as rounded instead of in fp32 is 2 % of both, the masks of
// bad blocks 1.5 %.
#pragma once

#include <atomic>

#include "pa_common.cuh"
#include "pa_decode.cuh"
#include "pa_fp4.cuh"
#include "pa_fp8.cuh"
#include "pa_internal.h"
#include "pa_mma.cuh"
#include "pa_prefill.cuh"
#include "pa_tc5.cuh"

namespace pa {

constexpr int PF8_ROWS = PREFILL_F8_ROWS;      // rows of one item: two tiles of 128
constexpr int PF8_KEYS = 64;                   // keys of a step: four cache blocks
// stages of K, and of V: what the exchange buffers of a cluster leave room for
__host__ __device__ constexpr int pf8_stages(int C) { return C == 1 ? 4 : C == 2 ? 3 : 2; }
constexpr int PF8_THREADS = 16 * 32;
#ifndef PF4_AHEAD
#define PF4_AHEAD 6
#endif
constexpr int PF8_K_WARP = 8;                  // and 9; V: 10, 11
constexpr int PF8_MMA_WARP = 12;               // and 13: S; 14, 15: P V

template <int D, int C>
struct PrefillF8Layout {
    static constexpr int STAGES = pf8_stages(C);
    static constexpr int NH = D / 64;                                // 128-byte groups of an f16 row
    static constexpr uint32_t KV_BYTES = PF8_KEYS * D * 2;           // [NH][64 keys][128 B]
    static constexpr uint32_t Q_BYTES = (NH - 1) * 128 * 128;        // a tile's [NH - 1][128 rows][128 B]
    // from the other blocks of the cluster, a tile: columns of O [C][D / C / 4][128
    // rows] float4 (the own rank's slot is not there), and (m, l) [C][128]
    static constexpr uint32_t XO_BYTES = (C - 1) * (D / C) * 128 * 4;
    static constexpr uint32_t XS_BYTES = C > 1 ? C * 128 * 8 : 0;
    static constexpr size_t OFF_K = 0;
    static constexpr size_t OFF_V = (size_t)STAGES * KV_BYTES;
    static constexpr size_t OFF_Q = 2 * (size_t)STAGES * KV_BYTES;
    static constexpr size_t OFF_XO = OFF_Q + 2 * (size_t)Q_BYTES;
    static constexpr size_t OFF_XS = OFF_XO + 2 * (size_t)XO_BYTES;
    static constexpr size_t OFF_BARS = OFF_XS + 2 * (size_t)XS_BYTES;
    static constexpr int NBARS = 4 * STAGES + 14 + 1;
    static constexpr size_t OFF_TMEM = OFF_BARS + (size_t)NBARS * 8;
    static constexpr size_t BYTES = OFF_TMEM + 16 + 1024;            // + alignment of the base
    // first TMEM columns of tile 0's S, P, O and Q; tile 1's come 64, 32, D and
    // 32 later
    static constexpr uint32_t TMEM_S = 0, TMEM_P = 128, TMEM_O = 192, TMEM_Q = 192 + 2 * D;
    static_assert(TMEM_Q + 64 <= 512 && KV_BYTES % 1024 == 0, "TMEM columns; swizzle atoms");
};

// A remote or local shared-memory float4 / float2, and an arrival at another
// block's barrier that publishes what this warp wrote there.
__device__ __forceinline__ void st_dsmem_f32x4(uint32_t addr, float a, float b, float c, float d) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" :: "r"(addr), "f"(a), "f"(b),
                 "f"(c), "f"(d) : "memory");
}
__device__ __forceinline__ void st_dsmem_f32x2(uint32_t addr, float a, float b) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" :: "r"(addr), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ float2 lds_f32x2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 lds_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
// the address `addr` of this block's shared memory in block `rank` of the cluster
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t out;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(addr), "r"(rank));
    return out;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(addr) : "memory");
}

template <typename T, typename KV, int D, int G, int C>
__global__ void __launch_bounds__(PF8_THREADS, 1)
prefill_f8_kernel(const __grid_constant__ DecodeParams p, int groups) {
    static_assert(sizeof(T) == 2 && (D == 64 || D == 128), "16-bit q and out, head_dim 64 or 128");
    static_assert(128 % G == 0, "a tile holds whole tokens");
    static_assert(C == 1 || C == 2 || C == 4, "blocks that share an item");
    constexpr bool F4 = std::is_same<KV, e2m1>::value;
    static_assert(F4 || std::is_same<KV, e4m3>::value, "cache type");
    using Lay = PrefillF8Layout<D, C>;
    constexpr uint32_t KVB = Lay::KV_BYTES;
    constexpr int NS = Lay::STAGES;
    constexpr uint32_t ID_S = tc5_idesc<__half>(128, PF8_KEYS, 0);   // Q K^T: K K-major
    constexpr uint32_t ID_O = tc5_idesc<__half>(128, D, 1);          // P V: V MN-major

    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::OFF_BARS);
    uint64_t *kfull = bars;                // [NS] K of a step converted (two warps)
    uint64_t *vfull = bars + NS;           // [NS] V of a step converted
    uint64_t *kfree = bars + 2 * NS;       // [NS] both tiles' S of a step done
    uint64_t *vfree = bars + 3 * NS;       // [NS] both tiles' P V of a step done
    uint64_t *q_full = bars + 4 * NS;      // [2] a tile's Q in TMEM (four warps)
    uint64_t *s_full = q_full + 2;         // [2] a tile's S of a step in TMEM
    uint64_t *p_full = q_full + 4;         // [2] a tile's P of a step in TMEM (four warps)
    uint64_t *pv_done = q_full + 6;        // [2] a tile's P V of a step done: P free, O whole
    uint64_t *s_free = q_full + 8;         // [2] a tile's S of a step read (four warps)
    uint64_t *x_full = q_full + 10;        // [2] a tile's rows from the other blocks are here
    uint64_t *x_free = q_full + 12;        // [2] the other blocks have read this one's rows
    uint64_t *mma_idle = q_full + 14;      // the block's MMAs are all done
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Lay::OFF_TMEM);
    __shared__ PrefillSched sched;
    __shared__ int bad_seq[8];             // softmax warps: sequence of an item with bad blocks

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hkv = p.num_kv_heads, H = p.num_heads;

    // the kernel launched next (the rows of the short runs) may set up; it waits
    // for this grid before it touches the caches or out
    launch_dependents();
    if (tid == 0) {
        // test hook: with one arrival more than there are, a block's first K never
        // counts as converted, and the waits for it and for what it holds up run out
        for (int i = 0; i < 4 * NS; ++i) mbar_init(&bars[i], i == 0 && p.test_stall ? 3 : 2);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&q_full[t], 4);
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 4);
            mbar_init(&pv_done[t], 1);
            mbar_init(&s_free[t], 4);
            mbar_init(&x_full[t], C > 1 ? 4 * (C - 1) : 1);
            mbar_init(&x_free[t], C > 1 ? 4 * (C - 1) : 1);
        }
        mbar_init(mma_idle, 4);
        fence_mbar_init();
    }
    if (warp == 0) tc5_alloc(tmem_slot, 512);
    tc5_fence_before_sync();
    __syncthreads();
    tc5_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    if constexpr (C > 1) cluster_sync();   // the peers' barriers are there

    const int total = prefill_schedule<G, PF8_ROWS>(p, groups, sched);
    grid_dependency_wait();                // q, the caches and out from here on

    const int R = (int)gridDim.x / C, me = (int)blockIdx.x / C;    // clusters
    const int rank = C > 1 ? (int)cluster_ctarank() : 0;
    // The geometry of an item, and this block's steps of it; every role computes
    // it alike.
    struct Item {
        int s, j, row0, q0, nq, L, nrows, step0, nsteps;
    };
    auto item_at = [&](int k, Item &it) -> bool {  // all lanes of a warp
        const long long x = (long long)k * R + ((k & 1) ? (R - 1 - me) : me);   // snake
        if (x >= total) return false;
        int grp;
        prefill_item<G, PF8_ROWS>(p, groups, sched, (int)x, it.s, it.j, grp);
        it.q0 = p.query_start[it.s];
        it.nq = p.query_start[it.s + 1] - it.q0;
        it.L = p.seq_lens[it.s];
        it.row0 = grp * PF8_ROWS;
        it.nrows = min(PF8_ROWS, it.nq * G - it.row0);           // >= 1
        const int n_keys = it.L - it.nq + (it.row0 + it.nrows - 1) / G + 1;   // keys any row sees
        const int n = (n_keys + PF8_KEYS - 1) / PF8_KEYS;
        it.step0 = n * rank / C;
        it.nsteps = n * (rank + 1) / C - it.step0;
        return true;
    };

    if (warp >= PF8_K_WARP && warp < PF8_MMA_WARP) {
        // ---- convert K (warps 8, 9) or V (10, 11): rows 32 * half .. + 31 of each
        // step.  A lane holds 16 codes of a row: the pieces 0-3 of two
        // neighbouring rows lie in eight neighbouring lanes, whose f16 chunks 2 jl
        // (and 2 jl + 1) then fall on all banks under the swizzle.
        const bool kside = warp < PF8_K_WARP + 2;
        const int half = warp & 1;
        constexpr int RPI = 512 / D, NI = 32 / RPI;       // rows of an instruction; instructions
        const int jl = (lane & 3) | (D == 128 ? (lane >> 1) & 4 : 0);
        const int r0 = D == 128 ? ((lane >> 2) & 1) | ((lane >> 3) & 2) : lane >> 2;
        constexpr int ROWB = F4 ? D / 2 : D;              // bytes of a row's codes
        constexpr int TILE = tile_bytes<KV, D>();
        const unsigned char *cache = static_cast<const unsigned char *>(kside ? p.k_cache : p.v_cache) +
                                     r0 * ROWB + (ROWB / (D / 16)) * jl;
        const unsigned char *scales = static_cast<const unsigned char *>(kside ? p.k_cache : p.v_cache) +
                                      8 * D + r0 * (D / 16) + jl;    // E2M1: of this lane's 16 codes
        // f16 chunk cc of row r lies at cc ^ (r & 7) of its 128-byte group; with
        // four rows an instruction, every second one flips bit 2 of that
        unsigned char *const stage0 = smem + (kside ? Lay::OFF_K : Lay::OFF_V) +
                                      (jl >> 2) * (PF8_KEYS * 128) + (32 * half + r0) * 128;
        const int lo0 = ((2 * (jl & 3)) ^ r0) << 4, hi0 = ((2 * (jl & 3) + 1) ^ r0) << 4;
        uint64_t *const full = kside ? kfull : vfull;
        uint64_t *const empty = kside ? kfree : vfree;

        // the load cursor: step c of item k, and the physical blocks of this
        // warp's two cache blocks of it
        Item it;
        int k = -1, c = 0, pb[2] = {-1, -1};
        const int32_t *tab = nullptr;
        long long joff = 0;
        const long long bstride = (long long)Hkv * TILE;
        bool more = false;
        auto item_next = [&]() {                   // the next item with steps of this block's
            do more = item_at(++k, it); while (more && it.nsteps == 0);
            if (!more) return;
            c = 0;
            tab = p.block_tables + (long long)it.s * p.max_blocks + 4 * it.step0 + 2 * half;
            joff = (long long)it.j * TILE;
        };
        auto blocks_of = [&]() {
            if (!more) return;
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (64 * (it.step0 + c) + 32 * half + 16 * b < it.L) pb[b] = tab[4 * c + b];
        };
        // E2M1: the tiles PF4_AHEAD steps on are brought into L2.  The items of a head
        // walk the same keys in step, so all of them would wait for what the first
        // one meets (3008 rows over up to 16 k keys from HBM: 389 us without, 359 with).
        constexpr int LINES = (TILE + 127) / 128;
        int ahead = -1;                            // a block of the step, in lanes of its lines
        auto look_ahead = [&]() {
            ahead = -1;
            if constexpr (F4) {
                const int a = c + PF4_AHEAD, b = lane / LINES;
                if (more && a < it.nsteps && b < 2 && 64 * (it.step0 + a) + 32 * half + 16 * b < it.L)
                    ahead = tab[4 * a + b];
            }
        };
        auto bring = [&]() {
            if (F4 && ahead >= 0 && (long long)ahead < p.num_blocks) {
                const unsigned char *t = static_cast<const unsigned char *>(kside ? p.k_cache : p.v_cache) +
                                         ahead * bstride + joff;
                asm volatile("prefetch.global.L2 [%0];" :: "l"(t + min(lane % LINES * 128, TILE - 1)));
            }
        };
        item_next();
        blocks_of();
        look_ahead();
        // 16 codes of a row: E4M3 four words, E2M1 two and their scale
        using Codes = std::conditional_t<F4, uint3, uint4>;
        auto load = [&](Codes (&buf)[NI]) -> bool {        // the cursor's step; moves on
            if (!more) return false;
            bring();
            const int key0 = 64 * (it.step0 + c) + 32 * half;
            const bool whole = key0 + 32 <= it.L;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                // rows past the sequence and bad blocks: zeros
                int rows = whole ? 16 : min(16, it.L - key0 - 16 * b);
                if (rows > 0 && (pb[b] < 0 || (long long)pb[b] >= p.num_blocks)) {
                    if (kside && lane == 0) set_error(p.err, ERR_BLOCK_ID);
                    rows = 0;
                }
                const long long off = (rows > 0 ? pb[b] : 0) * bstride + joff;
#pragma unroll
                for (int i = 0; i < NI / 2; ++i) {
                    Codes &x = buf[b * (NI / 2) + i];
                    x = {};
                    if (i * RPI + r0 < rows) {
                        if constexpr (F4) {
                            const uint2 w = *reinterpret_cast<const uint2 *>(cache + off + i * RPI * ROWB);
                            x = make_uint3(w.x, w.y, scales[off + i * RPI * (D / 16)]);
                        } else {
                            x = *reinterpret_cast<const uint4 *>(cache + off + i * RPI * ROWB);
                        }
                    }
                }
            }
            if (++c == it.nsteps) item_next();
            blocks_of();
            look_ahead();
            return true;
        };
        auto store = [&](unsigned char *st, const Codes (&buf)[NI]) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const Codes w = buf[i];
                const int flip = RPI == 4 && (i & 1) ? 64 : 0;
                unsigned char *row = st + i * RPI * 128;
                uint4 lo, hi;
                if constexpr (F4) {
                    const uint32_t x = f16x2_from_e4m3x2(w.z | (w.z << 8));
                    uint32_t a[4], b[4];
                    f16x2_from_e2m1x8(w.x, a);
                    f16x2_from_e2m1x8(w.y, b);
                    lo = make_uint4(mul_f16x2(a[0], x), mul_f16x2(a[1], x), mul_f16x2(a[2], x), mul_f16x2(a[3], x));
                    hi = make_uint4(mul_f16x2(b[0], x), mul_f16x2(b[1], x), mul_f16x2(b[2], x), mul_f16x2(b[3], x));
                } else {
                    lo = make_uint4(f16x2_from_e4m3x2(w.x), f16x2_from_e4m3x2(w.x >> 16),
                                    f16x2_from_e4m3x2(w.y), f16x2_from_e4m3x2(w.y >> 16));
                    hi = make_uint4(f16x2_from_e4m3x2(w.z), f16x2_from_e4m3x2(w.z >> 16),
                                    f16x2_from_e4m3x2(w.w), f16x2_from_e4m3x2(w.w >> 16));
                }
                *reinterpret_cast<uint4 *>(row + (lo0 ^ flip)) = lo;
                *reinterpret_cast<uint4 *>(row + (hi0 ^ flip)) = hi;
            }
        };
        unsigned g = 0;
        auto put = [&](const Codes (&buf)[NI]) -> bool {
            const int st = (int)(g % NS);
            bool w = true;
            if (lane == 0 && g >= NS) w = mbar_wait_bounded(&empty[st], (g / NS - 1) & 1, p.err);
            if (!__shfl_sync(0xffffffffu, w, 0)) return false;
            store(stage0 + (size_t)st * KVB, buf);
            fence_proxy_async_smem();              // the rows before the MMAs
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
            ++g;
            return true;
        };
        Codes b0[NI], b1[NI];
        bool h0 = load(b0), h1 = load(b1);
        while (h0) {
            if (!put(b0)) break;
            h0 = load(b0);
            if (!h1) break;
            if (!put(b1)) break;
            h1 = load(b1);
        }
    } else if (warp >= PF8_MMA_WARP) {
        // ---- the MMAs of tile t: S (warps 12, 13) or P V (14, 15)
        const int t = warp & 1;
        const bool sside = warp < PF8_MMA_WARP + 2;
        bool ok = true;
        unsigned g = 0, gt = 0;                    // steps so far; of this tile
        unsigned kt = 0;                           // items with this tile and steps
        Item it;
        const uint64_t dk = tc5_desc_sw128(smem_u32(smem + Lay::OFF_K), 16, 1024);
        const uint64_t dv = tc5_desc_sw128(smem_u32(smem + Lay::OFF_V), PF8_KEYS * 128, 1024);
        const uint64_t dq = tc5_desc_sw128(smem_u32(smem + Lay::OFF_Q + t * Lay::Q_BYTES), 16, 1024);
        const uint32_t tS = tmem + Lay::TMEM_S + 64 * t, tP = tmem + Lay::TMEM_P + 32 * t;
        const uint32_t tO = tmem + Lay::TMEM_O + D * t, tQ = tmem + Lay::TMEM_Q + 32 * t;
        auto wait = [&](uint64_t *bar, unsigned phase) -> bool {
            return mbar_wait_bounded(bar, phase & 1, p.err);
        };
        for (int k = 0; ok && item_at(k, it); ++k) {
            const int n = it.nsteps;
            if (lane == 0 && it.nrows <= 128 * t) {
                // an idle tile gives the stages back
                uint64_t *const full = sside ? kfull : vfull, *const empty = sside ? kfree : vfree;
                for (int c = 0; ok && c < n; ++c, ++g) {
                    ok = wait(&full[g % NS], g / NS);
                    if (ok) mbar_arrive(&empty[g % NS]);
                }
            } else if (lane == 0 && sside && n > 0) {
                ok = wait(&q_full[t], kt++);
                for (int c = 0; ok && c < n; ++c, ++g, ++gt) {
                    const unsigned st = g % NS;
                    // K has landed, and S of the step before has been read (by the
                    // item before, if this is an item's first)
                    ok = wait(&kfull[st], g / NS) && (gt == 0 || wait(&s_free[t], gt - 1));
                    if (!ok) break;
                    tc5_fence_after_sync();
                    const uint64_t kb = dk + (uint64_t)(st * KVB >> 4);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)             // 16 elements = 32 bytes
                        tc5_mma_ta(tS, tQ + 8 * ks, kb + (uint32_t)(ks * 32 >> 4), ID_S, ks > 0);
#pragma unroll
                    for (int ks = 4; ks < D / 16; ++ks)
                        tc5_mma(tS, dq + (uint32_t)(((ks >> 2) - 1) * (128 * 128) + (ks & 3) * 32 >> 4),
                                kb + (uint32_t)(((ks >> 2) * (PF8_KEYS * 128) + (ks & 3) * 32) >> 4), ID_S, 1);
                    tc5_commit(&s_full[t]);
                    tc5_commit(&kfree[st]);
                }
            } else if (lane == 0) {
                for (int c = 0; ok && c < n; ++c, ++g, ++gt) {
                    const unsigned st = g % NS;
                    ok = wait(&vfull[st], g / NS) && wait(&p_full[t], gt);
                    if (!ok) break;
                    tc5_fence_after_sync();
                    const uint64_t vb = dv + (uint64_t)(st * KVB >> 4);
#pragma unroll
                    for (int ks = 0; ks < PF8_KEYS / 16; ++ks) // 16 keys = 2048 bytes
                        tc5_mma_ta(tO, tP + 8 * ks, vb + (uint32_t)(ks * 2048 >> 4), ID_O, c > 0 || ks > 0);
                    tc5_commit(&pv_done[t]);
                    tc5_commit(&vfree[st]);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        // MMAs may still be running (after a timeout): wait for them
        if (lane == 0) {
            tc5_commit(mma_idle);
            mbar_wait_bounded(mma_idle, 0, p.err);
        }
    } else if (warp < PF8_K_WARP) {
        // ---- softmax: thread r of tile t owns row 128 t + r of every item
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;   // this warp's TMEM lanes
        const uint32_t tS = tmem + Lay::TMEM_S + 64 * t + lane_base, tP = tmem + Lay::TMEM_P + 32 * t + lane_base;
        const uint32_t tO = tmem + Lay::TMEM_O + D * t + lane_base, tQ = tmem + Lay::TMEM_Q + 32 * t + lane_base;
        unsigned char *const qrow = smem + Lay::OFF_Q + t * Lay::Q_BYTES + r * 128;
        unsigned g = 0;                            // steps of this tile
        unsigned kt = 0;                           // items of it
        bool ok = true;
        auto wait = [&](uint64_t *bar, unsigned phase) -> bool {       // the whole warp
            bool w = true;
            if (lane == 0) w = mbar_wait_bounded(bar, phase & 1, p.err);
            w = __shfl_sync(0xffffffffu, w, 0);
            tc5_fence_after_sync();
            return w;
        };
        auto wait_cluster = [&](uint64_t *bar, unsigned phase) -> bool {
            const bool w = wait(bar, phase);
            fence_acq_rel_cluster();               // what the other blocks wrote before it
            return w;
        };
        Item it;
        for (int k = 0; ok && item_at(k, it); ++k) {
            if (it.nrows <= 128 * t) continue;     // no rows of this tile
            const int rr = it.row0 + 128 * t + r;
            const int tok = rr / G, head = rr % G;
            const bool row_ok = 128 * t + r < it.nrows;
            // last visible position; rows past the run see what its last row sees
            const int lim = it.L - it.nq + min(tok, it.nq - 1);
            int cmask = (__reduce_min_sync(0xffffffffu, lim) + 1) / PF8_KEYS;   // steps before: no mask
            // the score scale; a negative one moves its sign to q, and one of 0 is
            // a tiny one, so that masked scores stay -inf; a NaN stays one
            float sl2 = p.scale_log2 * __ldg(p.k_scale + it.j);
            const uint32_t sign = sl2 < 0.f ? 0x80008000u : 0u;
            sl2 = fabsf(sl2) < 1e-30f ? 1e-30f : fabsf(sl2);

            // -- Q of this row as f16: the first 64 elements to TMEM as pairs, the
            // rest to shared memory (128-byte swizzle); the item before is done
            // with both.  Only for an item with steps here: S of its first step then
            // shows that q_full was seen before the next item completes it again.
            if (C == 1 || it.nsteps > 0) {
                const T *q = static_cast<const T *>(p.q) + (long long)(it.q0 + tok) * p.q_seq_stride +
                             (long long)(it.j * G + head) * D;
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    uint32_t w[32];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 x = row_ok ? reinterpret_cast<const uint4 *>(q + 64 * h)[i]
                                               : make_uint4(0, 0, 0, 0);
                        w[4 * i] = WarpAttnF8<T, D, 1>::to_f16x2(x.x) ^ sign;
                        w[4 * i + 1] = WarpAttnF8<T, D, 1>::to_f16x2(x.y) ^ sign;
                        w[4 * i + 2] = WarpAttnF8<T, D, 1>::to_f16x2(x.z) ^ sign;
                        w[4 * i + 3] = WarpAttnF8<T, D, 1>::to_f16x2(x.w) ^ sign;
                    }
                    if (h == 0) {
                        tc5_st32u(tQ, w);          // waits for the store
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4 *>(qrow + (h - 1) * (128 * 128) + ((i ^ (r & 7)) << 4)) =
                                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    }
                }
                if (D > 64) fence_proxy_async_smem();
                tc5_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[t]);
            }

            // If this block's steps name a block outside the pool, its keys (zeros in
            // the stages) are masked, as if no row saw them: every step goes through
            // the masks below then (cmask < 0).
            {
                const int32_t *tab = p.block_tables + (long long)it.s * p.max_blocks;
                const int end = min(4 * (it.step0 + it.nsteps), (it.L + 15) >> 4);
                bool bad = false;
#pragma unroll 8
                for (int i = 4 * it.step0 + lane; i < end; i += 32)
                    bad |= (unsigned long long)(long long)tab[i] >= (unsigned long long)p.num_blocks;
                if (__any_sync(0xffffffffu, bad)) {
                    cmask = -1;
                    if (lane == 0) bad_seq[warp] = it.s;   // no register over the steps
                    __syncwarp();
                }
            }

            float m_run = -INFINITY, l_run = 0.f;
            for (int c = 0; c < it.nsteps; ++c, ++g) {
                const int step = it.step0 + c;
                if (!wait(&s_full[t], g)) { ok = false; break; }
                float sv[PF8_KEYS];
                tc5_ld64u(tS, *reinterpret_cast<uint32_t(*)[PF8_KEYS]>(&sv[0]));
                tc5_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_free[t]);
                if (step >= cmask) {
                    const int nvis = lim - step * PF8_KEYS + 1;     // positions of this step the row sees
                    uint64_t vis = nvis >= 64 ? ~0ull : nvis > 0 ? (1ull << nvis) - 1 : 0ull;
                    if (cmask < 0) {
                        const int s = *(volatile int *)&bad_seq[warp];
                        const int32_t *tab = p.block_tables + (long long)s * p.max_blocks + 4 * step;
                        const int left = p.seq_lens[s] - step * PF8_KEYS;
                        for (int b = 0; b < 4; ++b)
                            if (16 * b < left &&
                                (unsigned long long)(long long)tab[b] >= (unsigned long long)p.num_blocks)
                                vis &= ~(0xffffull << (16 * b));
                    }
                    const uint32_t vl = (uint32_t)vis, vh = (uint32_t)(vis >> 32);
#pragma unroll
                    for (int e = 0; e < PF8_KEYS; ++e)
                        sv[e] = ((e < 32 ? vl : vh) >> (e & 31)) & 1 ? sv[e] : -INFINITY;
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < PF8_KEYS; e += 8) {
                    m4[0] = max3f(m4[0], sv[e], sv[e + 1]);
                    m4[1] = max3f(m4[1], sv[e + 2], sv[e + 3]);
                    m4[2] = max3f(m4[2], sv[e + 4], sv[e + 5]);
                    m4[3] = max3f(m4[3], sv[e + 6], sv[e + 7]);
                }
                const float mxs = max3f(m4[0], m4[1], fmaxf(m4[2], m4[3])) * sl2;
                // lazy rescaling: see F8_BELOW_LOG2
                const float m_new = mxs > m_run + F8_TOP_LOG2 ? mxs - F8_BELOW_LOG2 : m_run;
                const float ms = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = m_new == m_run ? 1.f : ex2(m_run - ms);
                uint32_t pw[PF8_KEYS / 2];
                float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                 make_float2(0.f, 0.f)};
                const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(-ms, -ms);
#pragma unroll
                for (int e = 0; e < PF8_KEYS / 2; ++e) {
                    const float2 x = fma2(make_float2(sv[2 * e], sv[2 * e + 1]), sc2, nm2);
                    pw[e] = Mma<__half>::pack(ex2(x.x), ex2(x.y));
                    // the weights as P V uses them: their rounding cancels in O / l
                    add_halves(acc[e & 3].x, acc[e & 3].y, pw[e]);
                }
                const float2 a2 = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
                l_run = l_run * alpha + (a2.x + a2.y);
                m_run = m_new;
                // P V of the step before is done: its P may be overwritten, and this
                // row of O taken to the new level (O holds nothing before the
                // item's first)
                if (g > 0 && !wait(&pv_done[t], g - 1)) { ok = false; break; }
                tc5_st32u(tP, pw);
                if (c > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        float o[32];
                        tc5_ld32(tO + c0, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= alpha;
                        tc5_st32(tO + c0, o);
                    }
                }
                tc5_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[t]);
            }
            if (!ok) break;

            // -- O / l, in V's scale, into out (this thread's row)
            if (g > 0 && !wait(&pv_done[t], g - 1)) { ok = false; break; }
            T *o = static_cast<T *>(p.out) + ((long long)(it.q0 + tok) * H + it.j * G + head) * D;
            const float vsc = __ldg(p.v_scale + it.j);
            auto write = [&](int c0, const float *v, float f) {    // 8 columns
                uint4 w;
                w.x = Mma<T>::pack(v[0] * f, v[1] * f);
                w.y = Mma<T>::pack(v[2] * f, v[3] * f);
                w.z = Mma<T>::pack(v[4] * f, v[5] * f);
                w.w = Mma<T>::pack(v[6] * f, v[7] * f);
                *reinterpret_cast<uint4 *>(o + c0) = w;
            };
            if constexpr (C == 1) {
                const float inv = l_run > 0.f ? vsc / l_run : 0.f;
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 32) {
                    float v[32];
                    tc5_ld32(tO + c0, v);
                    if (row_ok) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) write(c0 + e, v + e, inv);
                    }
                }
            } else {
                constexpr int DC = D / C;                          // columns of a block
                constexpr int CH = DC < 32 ? DC : 32;              // of them at a time
                const uint32_t xo = smem_u32(smem + Lay::OFF_XO + t * Lay::XO_BYTES) + 16 * r;
                const uint32_t xs = smem_u32(smem + Lay::OFF_XS + t * Lay::XS_BYTES) + 8 * r;
                // the other blocks have read the item before
                if (kt > 0 && !wait_cluster(&x_free[t], kt - 1)) { ok = false; break; }
#pragma unroll 1
                for (int i = 1; i < C; ++i) {
                    const int to = (rank + i) % C;                 // its columns of this row
                    const uint32_t xoff = map_rank(xo, to) + (rank < to ? rank : rank - 1) * (DC * 512);
                    if (it.nsteps > 0) {
#pragma unroll
                        for (int c0 = 0; c0 < DC; c0 += CH) {
                            float v[32];
                            tc5_ld32(tO + to * DC + c0, v);
#pragma unroll
                            for (int e = 0; e < CH; e += 4)
                                st_dsmem_f32x4(xoff + (c0 + e) * 512, v[e], v[e + 1], v[e + 2], v[e + 3]);
                        }
                    }
                    st_dsmem_f32x2(map_rank(xs, to) + rank * 1024, m_run, l_run);
                    fence_acq_rel_cluster();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&x_full[t]), to));
                }
                st_dsmem_f32x2(xs + rank * 1024, m_run, l_run);
                if (!wait_cluster(&x_full[t], kt)) { ok = false; break; }
                // the common level, each block's weight, and the sum; a block that saw
                // nothing of the row has l = 0, one that saw a NaN has l = NaN (at any
                // level) and makes the row NaN
                float w[C], M = -INFINITY, sum = 0.f;
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const float2 ml = lds_f32x2(xs + i * 1024);
                    w[i] = ml.y == 0.f ? -INFINITY : ml.x == -INFINITY ? 0.f : ml.x;
                    M = fmaxf(M, w[i]);
                }
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    w[i] = w[i] == -INFINITY ? 0.f : ex2(w[i] - M);
                    sum = fmaf(w[i], lds_f32x2(xs + i * 1024).y, sum);
                }
                const float inv = sum > 0.f ? vsc / sum : 0.f;
#pragma unroll
                for (int c0 = 0; c0 < DC; c0 += CH) {
                    float v[32], x[32];
                    tc5_ld32(tO + rank * DC + c0, v);
#pragma unroll
                    for (int e = 0; e < CH; ++e) x[e] = 0.f;
#pragma unroll
                    for (int i = 0; i < C; ++i) {
                        // nothing of the row there (or no step at all): no O to read
                        if (lds_f32x2(xs + i * 1024).y == 0.f) continue;
                        if (i == rank) {
#pragma unroll
                            for (int e = 0; e < CH; ++e) x[e] = fmaf(w[i], v[e], x[e]);
                        } else {
                            const uint32_t from = xo + (i < rank ? i : i - 1) * (DC * 512) + c0 * 512;
#pragma unroll
                            for (int e = 0; e < CH; e += 4) {
                                const float4 y = lds_f32x4(from + e * 512);
                                x[e] = fmaf(w[i], y.x, x[e]);
                                x[e + 1] = fmaf(w[i], y.y, x[e + 1]);
                                x[e + 2] = fmaf(w[i], y.z, x[e + 2]);
                                x[e + 3] = fmaf(w[i], y.w, x[e + 3]);
                            }
                        }
                    }
                    if (row_ok) {
#pragma unroll
                        for (int e = 0; e < CH; e += 8) write(rank * DC + c0 + e, x + e, inv);
                    }
                }
                // the others may write the next item's rows
                __syncwarp();
                if (lane < C && lane != rank) mbar_arrive_cluster(map_rank(smem_u32(&x_free[t]), lane));
                ++kt;
            }
            // O and S read before the next item's MMAs overwrite them (they wait for
            // this warp's next arrivals)
            tc5_fence_before_sync();
        }
    }

    tc5_fence_before_sync();
    __syncthreads();
    if (warp == 0) tc5_dealloc(tmem, 512);
    if constexpr (C > 1) cluster_sync();   // no block leaves while a peer may write to it
}

// Clusters of C blocks that the device holds at once (blocks for C = 1), with the
// kernel's attributes set; looked up once per device.
template <typename T, typename KV, int D, int G, int C>
cudaError_t prefill_f8_fit(int *clusters) {
    constexpr size_t smem = PrefillF8Layout<D, C>::BYTES;
    static_assert(smem + sizeof(PrefillSched) + 1024 <= 227 * 1024, "shared memory");
    auto kern = prefill_f8_kernel<T, KV, D, G, C>;
    static std::atomic<int> fitted[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int nc = dev >= 0 && dev < 64 ? fitted[dev].load(std::memory_order_acquire) : 0;
    if (nc <= 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        nc = sm_count_of_current_device();
        if (C > 1) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(C * 64, 1, 1);
            cfg.blockDim = dim3(PF8_THREADS, 1, 1);
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = C;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&nc, kern, &cfg);
            if (e != cudaSuccess) return e;
        }
        if (nc < 1) nc = 1;
        if (dev >= 0 && dev < 64) fitted[dev].store(nc, std::memory_order_release);
    }
    *clusters = nc;
    return cudaSuccess;
}

template <typename T, typename KV, int D, int G, int C>
cudaError_t launch_prefill_f8(const DecodeParams &p, int groups, long long items, int clusters,
                              cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((items < clusters ? items : clusters) * C), 1, 1);
    cfg.blockDim = dim3(PF8_THREADS, 1, 1);
    cfg.dynamicSmemBytes = PrefillF8Layout<D, C>::BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, prefill_f8_kernel<T, KV, D, G, C>, p, groups);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

// Blocks that share an item.  `items` bounds the items from above (their keys
// are known on the device only).  A wave of items takes as long as its longest,
// so what counts is how full the last wave is: with few items the split that
// fills the SMs wins.  Sharing costs an exchange per item and stages, so the
// larger split has to be better by an eighth.
template <typename T, typename KV, int D, int G>
cudaError_t run_prefill_f8(const DecodeParams &p, int groups, long long items, cudaStream_t st) {
    int fit[3];
    cudaError_t e = prefill_f8_fit<T, KV, D, G, 1>(&fit[0]);
    if (e == cudaSuccess) e = prefill_f8_fit<T, KV, D, G, 2>(&fit[1]);
    if (e == cudaSuccess) e = prefill_f8_fit<T, KV, D, G, 4>(&fit[2]);
    if (e != cudaSuccess) return e;
    int best = 0;
    double best_t = 0.;
    for (int i = 0; i < 3; ++i) {
        const double t = (double)((items + fit[i] - 1) / fit[i]) / (1 << i);     // waves, in whole items
        if (i == 0 || t * 1.125 < best_t) {
            best = i;
            best_t = t;
        }
    }
    if (best == 0) return launch_prefill_f8<T, KV, D, G, 1>(p, groups, items, fit[0], st);
    if (best == 1) return launch_prefill_f8<T, KV, D, G, 2>(p, groups, items, fit[1], st);
    return launch_prefill_f8<T, KV, D, G, 4>(p, groups, items, fit[2], st);
}

template <typename T, typename KV = e4m3>
cudaError_t dispatch_prefill_f8(const DecodeParams &p, int D, int G, int groups, cudaStream_t st) {
    // at most `groups` items a run, and one more than the full items of all rows
    // for each run (a run has at least mq_split_rows rows)
    const long long rows_all = (long long)p.num_q_rows * G;
    long long runs = rows_all / p.mq_split_rows;
    if (runs > p.num_seqs) runs = p.num_seqs;
    long long items = rows_all / PF8_ROWS + runs;
    if (items > groups * (long long)p.num_seqs) items = groups * (long long)p.num_seqs;
    items *= p.num_kv_heads;
    if (items <= 0) return cudaSuccess;
#define PA_CASE(DD, GG) \
    if (D == DD && G == GG) return run_prefill_f8<T, KV, DD, GG>(p, groups, items, st);
    PA_CASE(64, 1) PA_CASE(64, 2) PA_CASE(64, 4) PA_CASE(64, 8)
    PA_CASE(128, 1) PA_CASE(128, 2) PA_CASE(128, 4) PA_CASE(128, 8)
#undef PA_CASE
    return cudaErrorNotSupported;
}

}  // namespace pa
