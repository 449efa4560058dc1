// pa_logits.cuh -- logits made ready for sampling or for the verification of drafts:
// penalties for repeated tokens, biases, masks of allowed tokens, temperature and
// softmax, in one pass over the vocabulary.
//
// For token v of row i of a sequence, x its logit, c the times v occurs in the output
// so far (the history behind the prompt, and the drafts before the row), seen whether
// it occurs there or in the prompt:
//   x = x > 0 ? x / theta : x theta        if seen
//   x = x - alpha c - beta [c > 0]
//   x = x + the biases of v
//   x = -inf                               if the row's mask does not allow v
//   x = x / tau                            (tau > 0)
// and the row of x, or softmax(x); with tau not above 0 the one-hot row of the first
// largest x instead.
//
// Bound by HBM: a row is read once and written once.  A cluster of C blocks takes a
// row, each block a run of the vocabulary that its threads hold in registers (up to
// LG_EPT elements each) from the load to the store, so that the maximum and the sum
// cost no second read; the blocks' (maximum, sum) meet through distributed shared
// memory.  The history is turned into counts per token of the run in shared memory
// while the logits are on their way.  What such a kernel spends its time on is
// instructions (with an element a lane and a bounds check, a vote and a mask bit each
// it took 68 an element, and 143 us for 237 rows of 131071): a thread holds four neighbours,
// a quad, read, counted, masked and written by one access each.  Quads lie on
// 16-byte borders of the output (rows of an odd vocabulary start anywhere); where
// the input's borders fall elsewhere it is read an element at a time.  Runs that do
// not fit into registers are read twice, the second time mostly from L2.
#pragma once
#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_mma.cuh"

#include <atomic>
#include <type_traits>

namespace pa {

namespace {

constexpr int LG_EPT = 36;                 // elements of a thread, at most
constexpr int LG_CLUSTER = 8;

// A token's word: whether it is in the prompt, whether it has biases, times in the output.
constexpr uint32_t LG_PROMPT = 0x80000000u, LG_BIAS = 0x40000000u, LG_COUNT = 0x3fffffffu;

// The factor that takes a sum to the level m (log2 units) over to base; a NaN sum
// without a level stays one.
__device__ __forceinline__ float carry(float m, float l, float base) {
    return m == -INFINITY ? (l != l ? 1.f : 0.f) : ex2(m - base);
}

__device__ __forceinline__ bool before(float m, int at, float m2, int at2) {   // (m, at) goes first
    return m > m2 || (m == m2 && at < at2);
}

// Four neighbouring elements as loaded.
template <typename T> struct Quad {
    using Raw = std::conditional_t<sizeof(T) == 4, uint4, uint2>;
    Raw w;
    // from an address that is a multiple of their size
    __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const Raw *>(p); }
    // one at a time, -inf where there is none
    template <typename In>
    __device__ __forceinline__ void load_some(const T *p, In &&in) {
        constexpr uint32_t NONE = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
        uint32_t c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            c[e] = NONE;
            if (in(e)) {
                if constexpr (sizeof(T) == 4) c[e] = reinterpret_cast<const uint32_t *>(p)[e];
                else c[e] = reinterpret_cast<const unsigned short *>(p)[e];
            }
        }
        if constexpr (sizeof(T) == 4) w = make_uint4(c[0], c[1], c[2], c[3]);
        else w = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
    __device__ __forceinline__ void widen(float *x) const {
        if constexpr (sizeof(T) == 4) {
            Elem<float>::to_f32(w, x);
        } else {
            Elem<T>::pair(w.x, x[0], x[1]);
            Elem<T>::pair(w.y, x[2], x[3]);
        }
    }
};
template <typename T>
__device__ __forceinline__ void store_quad(T *p, const float *x) {
    if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else
        *reinterpret_cast<uint2 *>(p) = make_uint2(Mma<T>::pack(x[0], x[1]), Mma<T>::pack(x[2], x[3]));
}

// sequence of row r: the last s with query_start[s] <= r; -1 if no sequence has it
__device__ __forceinline__ int sequence_of(const int32_t *qs, int B, int r, int lane) {
    int lo = 0, n = B;                     // in [lo, lo + n)
    while (n > 256) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const unsigned ok = __ballot_sync(0xffffffffu, lane * step < n && qs[at] <= r);
        // the probes hold for a first part of the lanes when the starts do not decrease
        const int k = ok ? 31 - __clz(ok) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    int mine = 0;                          // starts at or before r, of up to 256 at once
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e * 32 + lane < n) mine += qs[lo + e * 32 + lane] <= r;
    lo += max((int)__reduce_add_sync(0xffffffffu, mine) - 1, 0);
    return qs[lo] <= r && r < qs[lo + 1] ? lo : -1;
}

// What a row's sequence gives: its words as they are in memory, then checked.
struct Words {
    float theta, alpha, beta, tau;
    int first, len, asked, b0, b1;         // the history's length, of it the prompt's; the biases
    bool penalise, count;
    float inv_theta, inv_tau;
    __device__ __forceinline__ void read(const LogitsParams &p, int s) {
        theta = p.repetition ? p.repetition[s] : 1.f;
        alpha = p.frequency ? p.frequency[s] : 0.f;
        beta = p.presence ? p.presence[s] : 0.f;
        tau = p.temperature ? p.temperature[s] : 1.f;
        first = p.query_start[s];
        len = asked = b0 = b1 = 0;
        if (p.history) {
            len = p.history_lens[s];
            asked = p.prompt_lens ? p.prompt_lens[s] : 0;
        }
        if (p.bias_start) {
            b0 = p.bias_start[s];
            b1 = p.bias_start[s + 1];
        }
    }
    // The same by a warp, a word a lane: on their way to shared memory, and from there.
    static constexpr int RAW = 9;
    static __device__ __forceinline__ void fetch(const LogitsParams &p, int s, uint32_t *raw) {
        const int lane = threadIdx.x & 31;
        const void *at = nullptr;
        if (s >= 0) {                                      // else what changes nothing
            if (lane == 0 && p.repetition) at = p.repetition + s;
            if (lane == 1 && p.frequency) at = p.frequency + s;
            if (lane == 2 && p.presence) at = p.presence + s;
            if (lane == 3 && p.temperature) at = p.temperature + s;
            if (lane == 4) at = p.query_start + s;
            if (lane == 5 && p.history) at = p.history_lens + s;
            if (lane == 6 && p.history && p.prompt_lens) at = p.prompt_lens + s;
            if (lane == 7 && p.bias_start) at = p.bias_start + s;
            if (lane == 8 && p.bias_start) at = p.bias_start + s + 1;
        }
        if (at)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(smem_u32(&raw[lane])), "l"(at) : "memory");
        else if (lane < RAW)
            raw[lane] = lane == 0 || lane == 3 ? __float_as_uint(1.f) : 0u;
    }
    __device__ __forceinline__ void gather(const uint32_t *raw) {
        theta = __uint_as_float(raw[0]);
        alpha = __uint_as_float(raw[1]);
        beta = __uint_as_float(raw[2]);
        tau = __uint_as_float(raw[3]);
        first = (int)raw[4];
        len = (int)raw[5];
        asked = (int)raw[6];
        b0 = (int)raw[7];
        b1 = (int)raw[8];
    }
    __device__ __forceinline__ void check(const LogitsParams &p, bool flag) {
        if (len < 0 || len > p.history_stride || asked < 0 || asked > len) {
            if (flag) set_error(p.err, ERR_SEQ_LEN);
            len = max(0, (int)min((int64_t)len, p.history_stride));
            asked = min(max(asked, 0), len);
        }
        if (b0 < 0 || b1 < b0 || b1 > p.num_bias) {
            if (flag) set_error(p.err, ERR_SEQ_LEN);
            b0 = b1 = 0;
        }
        penalise = theta != 1.f || alpha != 0.f || beta != 0.f;
        count = penalise || b1 > b0;
        inv_theta = 1.f / theta;
        inv_tau = tau > 0.f ? 1.f / tau : 1.f;
        if (!penalise) len = 0;
    }
    // a quad by its tokens' words
    __device__ __forceinline__ void penalties(const uint32_t *c, float *x) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t n = c[e] & LG_COUNT;
            const float z = (x[e] > 0.f ? x[e] * inv_theta : x[e] * theta) - alpha * (float)n - (n ? beta : 0.f);
            x[e] = c[e] & ~LG_BIAS ? z : x[e];
        }
    }
};

// The part of row r that block `rank` of C has.  Quads, four elements, lie on borders
// of the output's; the first may begin before the row.
template <typename T, typename O> struct Part {
    const T *in;
    O *out;
    const uint32_t *mask;
    int v0, v1;
    bool wide;                             // the input's quads lie on its borders too
    __device__ __forceinline__ Part(const LogitsParams &p, int r, int rank, int C) {
        in = static_cast<const T *>(p.logits) + (int64_t)r * p.logits_stride;
        out = static_cast<O *>(p.out) + (int64_t)r * p.out_stride;
        mask = p.allowed ? p.allowed + (int64_t)r * p.allowed_stride : nullptr;
        const int lead = (int)((reinterpret_cast<uintptr_t>(out) / sizeof(O)) & 3);
        wide = (int)((reinterpret_cast<uintptr_t>(in) / sizeof(T)) & 3) == lead;
        const int run = ((p.vocab + lead + 3) / 4 + C - 1) / C * 4;
        v0 = rank * run - lead;
        v1 = min(p.vocab, v0 + run);
    }
};

// the words of the mask of elements t0 .. t1, on their way to shared memory
template <int NT>
__device__ __forceinline__ void fetch_mask(uint32_t *bits, const uint32_t *mask, int t0, int t1) {
    const int w0 = max(t0, 0) >> 5, n = ((t1 - 1) >> 5) - w0 + 1;
    for (int i = threadIdx.x; i < n; i += NT)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(smem_u32(&bits[i])), "l"(mask + w0 + i)
                     : "memory");
}
// they are here once the block has met behind this
__device__ __forceinline__ void mask_here() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// -inf for what the mask forbids in the quad at v
__device__ __forceinline__ void forbid(const uint32_t *bits, int w0, int v, float *x) {
    const int at = max(v, 0);
    const uint32_t w = bits[(at >> 5) - w0], w2 = bits[(at >> 5) - w0 + 1];
    const uint32_t ok = __funnelshift_r(w, w2, at & 31) << (at - v);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (ok >> e) & 1 ? x[e] : -INFINITY;
}

// What a thread counts first, loaded ahead: some of the history's tokens, a draft and
// an entry of the biases.
// AHEAD: history loads of a thread in flight.
template <int AHEAD> struct Tokens {
    int32_t h[AHEAD], draft, entry;
    float value;                           // of the entry; for the warp that adds the biases up
    template <int NT>
    __device__ __forceinline__ void read(const LogitsParams &p, const Words &q, const int32_t *hist, int r) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) h[e] = tid + e * NT < q.len ? hist[tid + e * NT] : -1;
        draft = p.tokens && q.penalise && q.first + 1 + tid <= r ? p.tokens[q.first + 1 + tid] : -1;
        entry = q.b0 + tid < q.b1 ? p.bias_tokens[q.b0 + tid] : -1;
        value = tid < 32 && q.b0 + tid < q.b1 ? p.bias_values[q.b0 + tid] : 0.f;
    }
};

// The words of the tokens of elements t0 .. t1 of a row: its history, the drafts
// before it, its biases.  Returns whether a token lies outside the vocabulary.
template <int NT, int AHEAD>
__device__ __forceinline__ bool count_tokens(const LogitsParams &p, const Words &q, const int32_t *hist, int r,
                                             int t0, int t1, uint32_t *counts, Tokens<AHEAD> &k) {
    const int tid = threadIdx.x, lo = max(t0, 0);
    bool bad = false;
    auto add = [&](int32_t v, bool prompt) {
        bad = bad || (uint32_t)v >= (uint32_t)p.vocab;
        if (v >= lo && v < t1) {
            if (prompt) atomicOr(&counts[v - t0], LG_PROMPT);
            else atomicAdd(&counts[v - t0], 1u);
        }
    };
    for (int i = tid; i < q.len; i += AHEAD * NT) {
        int32_t next[AHEAD];
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
            const int at = i + (AHEAD + e) * NT;
            next[e] = at < q.len ? hist[at] : -1;
        }
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
            if (i + e * NT < q.len) add(k.h[e], i + e * NT < q.asked);
            k.h[e] = next[e];
        }
    }
    if (p.tokens && q.penalise)            // the drafts before this row
        for (int i = q.first + 1 + tid; i <= r; i += NT) add(i < q.first + 1 + NT ? k.draft : p.tokens[i], false);
    for (int i = q.b0 + tid; i < q.b1; i += NT) {
        const int32_t v = i < q.b0 + NT ? k.entry : p.bias_tokens[i];
        bad = bad || (uint32_t)v >= (uint32_t)p.vocab;
        if (v >= lo && v < t1) atomicOr(&counts[v - t0], LG_BIAS);
    }
    return bad;
}

// The first warp adds the biases up in the order of the list, 32 at a time (the first
// ones loaded ahead): of the entries that name one token the first takes them all.
__device__ __forceinline__ void add_biases(const LogitsParams &p, const Words &q, int t0, int t1, uint32_t *counts,
                                           int32_t entry, float value) {
    const int lane = threadIdx.x & 31;
    for (int i = q.b0; i < q.b1; i += 32) {
        const bool in_list = i + lane < q.b1, first = i == q.b0;
        const int32_t v = !in_list ? -1 - lane : first ? entry : p.bias_tokens[i + lane];
        const float y = !in_list ? 0.f : first ? value : p.bias_values[i + lane];
        const unsigned same = __match_any_sync(0xffffffffu, v);
        float sum = y;
        const bool leads = lane == __ffs(same) - 1;
        if (__any_sync(0xffffffffu, __popc(same) > 1)) {
            sum = 0.f;
            for (int e = 0; e < 32; ++e) {
                const float z = __shfl_sync(0xffffffffu, y, e);
                if ((same >> e) & 1) sum += z;
            }
        }
        if (leads && v >= max(t0, 0) && v < t1) {
            float *to = reinterpret_cast<float *>(counts) + (v - t0);
            *to += sum;
        }
        __syncwarp();
    }
}
__device__ __forceinline__ void take_biases(const uint32_t *sums, float *x) {
    const float4 y = *reinterpret_cast<const float4 *>(sums);
    const float add[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)            // what is not allowed stays so
        x[e] = x[e] == -INFINITY ? -INFINITY : x[e] + add[e];
}

// The largest and the sum of a run: level m in log2 units and the sum l to it, or for
// a row that takes the first largest that element and its place.
struct Stat {
    float m = -INFINITY, l = 0.f, top = -INFINITY;
    int top_at = INT32_MAX;
    // over `lanes` neighbouring lanes
    __device__ __forceinline__ void join(int lanes, bool greedy) {
        if (greedy) {
            for (int o = lanes / 2; o > 0; o >>= 1) {
                const float t2 = __shfl_xor_sync(0xffffffffu, top, o);
                const int at2 = __shfl_xor_sync(0xffffffffu, top_at, o);
                if (before(t2, at2, top, top_at)) {
                    top = t2;
                    top_at = at2;
                }
            }
        } else {
            float up = m;
            for (int o = lanes / 2; o > 0; o >>= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, o));
            l *= carry(m, l, up == -INFINITY ? 0.f : up);
            for (int o = lanes / 2; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            m = up;
        }
    }
    // EPT elements more; KEEP: x becomes 2^(x log2 e - m)
    template <int EPT, bool KEEP>
    __device__ __forceinline__ void add(float *x) {
        float big = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPT; i += 2) big = max3f(big, x[i], x[i + 1]);
        const float up = fmaxf(m, big * LOG2E), base = up == -INFINITY ? 0.f : up;
        float sum[4] = {l * carry(m, l, base), 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const float e = ex2(fmaf(x[i], LOG2E, -base));
            if constexpr (KEEP) x[i] = e;
            sum[i & 3] += e;
        }
        m = up;
        l = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
    // sent to place `rank` of every block of the cluster, by a whole warp
    __device__ __forceinline__ void send(float4 *to, int rank, int C) const {
        const int lane = threadIdx.x & 31;
        if (lane < C)
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::
                         "r"(map_to_rank(&to[rank], (uint32_t)lane)), "f"(m), "f"(l), "f"(top),
                         "f"(__int_as_float(top_at)) : "memory");
        __syncwarp();                      // the cluster's barrier is one of whole warps
    }
};
// over the cluster's blocks: the place of the first largest
__device__ __forceinline__ int first_largest(const float4 *blocks, int C) {
    float best = -INFINITY;
    int at = INT32_MAX;
    for (int i = 0; i < C; ++i)
        if (before(blocks[i].z, __float_as_int(blocks[i].w), best, at)) {
            best = blocks[i].z;
            at = __float_as_int(blocks[i].w);
        }
    return at;
}
// and the level with the reciprocal of the sum to it (nothing allowed: 0)
__device__ __forceinline__ void level_and_scale(const float4 *blocks, int C, float &base, float &inv) {
    float up = -INFINITY, sum = 0.f;
    for (int i = 0; i < C; ++i) up = fmaxf(up, blocks[i].x);
    base = up == -INFINITY ? 0.f : up;
    for (int i = 0; i < C; ++i) sum += blocks[i].y * carry(blocks[i].x, blocks[i].y, base);
    inv = sum == 0.f ? 0.f : 1.f / sum;
}

template <typename O, int NT, int EPT>
__device__ __forceinline__ void store_tile(O *out, int t0, int t1, const float *x) {
#pragma unroll
    for (int i = 0; i < EPT / 4; ++i) {
        const int v = t0 + 4 * (i * NT + (int)threadIdx.x);
        if (v >= 0 && v + 4 <= t1) {
            store_quad<O>(out + v, x + 4 * i);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (v + e >= 0 && v + e < t1) Elem<O>::store1(out + v + e, x[4 * i + e]);
        }
    }
}

template <typename T, typename O, int NT, int EPT, bool RESIDENT>
__global__ void __launch_bounds__(NT, 1024 / NT) process_logits_kernel(const __grid_constant__ LogitsParams p) {
    constexpr int TILE = NT * EPT, WARPS = NT / 32, Q = EPT / 4;
    extern __shared__ __align__(16) uint32_t counts[];      // [tile], as the threads hold it
    __shared__ uint32_t bits[TILE / 32 + 2];                // words of the mask that the tile meets
    __shared__ float sh_m[WARPS], sh_l[WARPS], sh_top[WARPS];
    __shared__ int sh_at[WARPS];
    __shared__ float4 sh_blocks[LG_CLUSTER];                // (m, l, top, at) of the cluster's blocks
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
    const int r = (int)(blockIdx.x / C);
    const Part<T, O> part(p, r, rank, C);
    const int v0 = part.v0, v1 = part.v1;

    // The tile at t0: quad i NT + tid of it (-inf outside the row).
    constexpr bool NARROW = sizeof(T) == 2;     // widened only when the rest is here
    Quad<T> raw[NARROW ? Q : 1];
    float x[EPT];
    auto quad_at = [&](int t0, int i) -> int { return t0 + 4 * (i * NT + tid); };
    auto load = [&](int t0, int t1) {
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const int v = quad_at(t0, i);
            Quad<T> &q = raw[NARROW ? i : 0];
            if (part.wide && v >= 0 && v + 4 <= t1) q.load(part.in + v);
            else q.load_some(part.in + v, [&](int e) { return v + e >= 0 && v + e < t1; });
            if constexpr (!NARROW) q.widen(x + 4 * i);
        }
        if (part.mask) fetch_mask<NT>(bits, part.mask, t0, t1);
    };
    const int s = sequence_of(p.query_start, p.num_seqs, r, lane);
    if (s < 0) return;                                      // the whole cluster: no such row
    if (C > 1) cluster_arrive();                            // this block runs (see cluster_wait below)
    Words q;
    q.read(p, s);
    // The logits behind these few words (in front of them they hold them up, as the memory
    // answers in order: 3 us of a block's 14), and on their way while the history is
    // counted.
    load(v0, min(v1, v0 + TILE));
    q.check(p, rank == 0 && tid == 0);

    // counts of the tile's tokens: prompt and bias flags, times in the output
    const int32_t *hist = p.history ? p.history + (int64_t)s * p.history_stride : nullptr;
    Tokens<4> k;
    auto build = [&](int t0, int t1) {
        k.read<NT>(p, q, hist, r);
#pragma unroll
        for (int i = 0; i < Q; ++i)
            if (4 * (i * NT + tid) < t1 - t0)
                reinterpret_cast<uint4 *>(counts)[i * NT + tid] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        if (count_tokens<NT>(p, q, hist, r, t0, t1, counts, k) && rank == 0) set_error(p.err, ERR_TOKEN);
        mask_here();
        __syncthreads();
    };
    auto process = [&](int t0, int t1) {
        if (!q.count && part.mask) {
            mask_here();
            __syncthreads();
        }
        uint32_t biased = 0;               // bit i: quad i has biases
        const int w0 = max(t0, 0) >> 5;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            if constexpr (NARROW) raw[i].widen(x + 4 * i);
            const int v = quad_at(t0, i);
            if (v >= t1) continue;
            if (q.count) {
                uint4 &c4 = reinterpret_cast<uint4 *>(counts)[i * NT + tid];
                const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w}, any = c[0] | c[1] | c[2] | c[3];
                if (any) {
                    q.penalties(c, x + 4 * i);
                    if (any & LG_BIAS) {
                        biased |= 1u << i;
                        c4 = make_uint4(0, 0, 0, 0);        // the sums of the biases from here on
                    }
                }
            }
            if (part.mask) forbid(bits, w0, v, x + 4 * i);
        }
        if (q.b1 > q.b0) {
            __syncthreads();
            if (warp == 0) add_biases(p, q, t0, t1, counts, k.entry, k.value);
            __syncthreads();
            if (biased) {
#pragma unroll
                for (int i = 0; i < Q; ++i)
                    if ((biased >> i) & 1) take_biases(counts + 4 * (i * NT + tid), x + 4 * i);
            }
        }
        if (q.inv_tau != 1.f) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) x[i] *= q.inv_tau;
        }
    };
    auto store = [&](int t0, int t1) { store_tile<O, NT, EPT>(part.out, t0, t1, x); };

    if (!p.probs) {
        for (int t0 = v0; t0 < v1; t0 += TILE) {
            const int t1 = min(v1, t0 + TILE);
            if (t0 > v0) load(t0, t1);
            if (q.count) build(t0, t1);
            process(t0, t1);
            store(t0, t1);
            if (t0 + TILE < v1) __syncthreads();            // before the next counts and words
        }
        if (C > 1) cluster_wait();
        return;
    }

    Stat st;
    const bool greedy = !(q.tau > 0.f);
    for (int t0 = v0; t0 < v1; t0 += TILE) {
        const int t1 = min(v1, t0 + TILE);
        if (t0 > v0) load(t0, t1);
        if (q.count) build(t0, t1);
        process(t0, t1);
        if (greedy) {
#pragma unroll
            for (int i = 0; i < EPT; ++i)
                if (x[i] > st.top) {
                    st.top = x[i];
                    st.top_at = quad_at(t0, i >> 2) + (i & 3);
                }
        } else {
            st.template add<EPT, RESIDENT>(x);
        }
        if (!RESIDENT) __syncthreads();
    }
    const float mine = st.m;               // the level that x is to (resident)
    // over the warp, the block's warps, the cluster's blocks
    st.join(32, greedy);
    if (lane == 0) {
        sh_m[warp] = st.m;
        sh_l[warp] = st.l;
        sh_top[warp] = st.top;
        sh_at[warp] = st.top_at;
    }
    __syncthreads();
    // a peer's shared memory may be written once that block is known to run
    if (C > 1) cluster_wait();
    if (warp == 0) {
        const int w = lane & (WARPS - 1);
        st.m = sh_m[w];
        st.l = sh_l[w];
        st.top = sh_top[w];
        st.top_at = sh_at[w];
        st.join(WARPS, greedy);
        st.send(sh_blocks, rank, C);
    }
    cluster_sync();

    // ---- the row
    if (greedy) {
        const int at = first_largest(sh_blocks, C);
        for (int t0 = v0; t0 < v1; t0 += TILE) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) x[i] = quad_at(t0, i >> 2) + (i & 3) == at ? 1.f : 0.f;
            store(t0, min(v1, t0 + TILE));
        }
        return;
    }
    float base, inv;
    level_and_scale(sh_blocks, C, base, inv);
    if constexpr (RESIDENT) {
        const float f = (mine == -INFINITY ? 0.f : ex2(mine - base)) * inv;
#pragma unroll
        for (int i = 0; i < EPT; ++i) x[i] *= f;
        store(v0, v1);
    } else {
        for (int t0 = v0; t0 < v1; t0 += TILE) {
            const int t1 = min(v1, t0 + TILE);
            load(t0, t1);
            if (q.count) build(t0, t1);
            process(t0, t1);
#pragma unroll
            for (int i = 0; i < EPT; ++i) x[i] = ex2(fmaf(x[i], LOG2E, -base)) * inv;
            store(t0, t1);
            __syncthreads();
        }
    }
}

// Many rows: a cluster (without probabilities: C blocks that need not meet) takes one
// row after the other.  While a row is in its registers, the next one's logits come
// into shared memory by a bulk copy and its mask and its sequence's words by small ones,
// and its tokens are counted while the blocks exchange the first one's sums; counts are
// cleared as they are read.  237 rows of 131071 (bf16 to f32, a history of 4000, biases,
// masks, probabilities) take 82 us where a row a cluster at a time took 94, 256 rows of
// 50021 (f32, no probabilities) 33 us instead of 38.  What is left of a row's 26 thousand
// clocks (two blocks of 512 an SM): 5 the penalties and masks, 5 the counting, 3 each the
// joining of the warps' sums and the stores.  Registers are the limit: with 250 bytes
// of spills the same loop took 95 us, so what the next row needs stays in shared memory,
// and two loads of the history are in flight (80.4 us), not four (82.5) or eight (90).
template <typename T, typename O, int NT, int EPT, bool PROBS>
__global__ void __launch_bounds__(NT, 1024 / NT) process_rows_kernel(const __grid_constant__ LogitsParams p, int C) {
    constexpr int TILE = NT * EPT, WARPS = NT / 32, Q = EPT / 4, ES = (int)sizeof(T);
    extern __shared__ __align__(16) uint32_t counts[];      // [p.run], and behind them the next row's run
    __shared__ uint32_t bits[TILE / 32 + 2];
    __shared__ float sh_m[WARPS], sh_l[WARPS], sh_top[WARPS];
    __shared__ int sh_at[WARPS];
    __shared__ float4 sh_blocks[2][LG_CLUSTER];             // of this row and the last one that a sequence has
    constexpr int KNOWN = 32;
    __shared__ int sequences[KNOWN];                        // of rows r_known + i step
    __shared__ Words words[2];                              // of this row's sequence and the next one's
    __shared__ uint32_t raw_words[Words::RAW];              // and as they come
    __shared__ int sh_dead;                                 // 1 + the phase of a copy that did not come
    __shared__ int32_t entries[32];                         // the row's first biases
    __shared__ float values[32];
    __shared__ __align__(8) uint64_t bar;
    const bool counting = p.repetition || p.frequency || p.presence || p.bias_start;
    unsigned char *stage = reinterpret_cast<unsigned char *>(counts) + (counting ? (size_t)p.run * 4 : 0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)(blockIdx.x % C), step = (int)(gridDim.x / C);
    int r_known = 0;

    if (tid == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
        sh_dead = 0;
    }
    if (counting)
        for (int i = tid; i < p.run / 4; i += NT) reinterpret_cast<uint4 *>(counts)[i] = make_uint4(0, 0, 0, 0);
    auto sequence = [&](int r) { return r < p.num_rows ? sequences[(r - r_known) / step] : -1; };
    // The sequences of the next KNOWN rows from r on, a warp each: looked up row by row
    // the search's loads took 4 of 28 thousand clocks.
    auto know = [&](int r) {
        r_known = r;
        for (int i = warp; i < KNOWN && r + i * step < p.num_rows; i += WARPS) {
            const int s = sequence_of(p.query_start, p.num_seqs, r + i * step, lane);
            if (lane == 0) sequences[i] = s;
        }
    };
    know((int)(blockIdx.x / C));
    __syncthreads();
    if (PROBS && C > 1) cluster_arrive();                   // this block runs (see cluster_wait below)

    // One bulk copy of the 16-byte pieces that the run lies in; at the tensor's own ends,
    // of those that lie in it, and the up to 7 elements beside them one by one.  The
    // run's first byte is at its address modulo 16.
    struct Pieces {
        uintptr_t a, e, from, to;          // the run, the copy
    };
    auto pieces_of = [&](const Part<T, O> &w, int r) -> Pieces {
        Pieces c;
        c.a = reinterpret_cast<uintptr_t>(w.in + max(w.v0, 0));
        c.e = reinterpret_cast<uintptr_t>(w.in + w.v1);
        c.from = (r > 0 || w.v0 > 0 ? c.a : c.a + 15) & ~uintptr_t(15);
        c.to = (r < p.num_rows - 1 || w.v1 < p.vocab ? c.e + 15 : c.e) & ~uintptr_t(15);
        return c;
    };
    auto edge_of = [&](const Part<T, O> &w, const Pieces &c) -> int {      // this thread's element, -1: none
        if (tid >= 16 || c.e <= c.a) return -1;
        if (tid < 8) return c.from > c.a && tid < (int)((min(c.from, c.e) - c.a) / ES) ? max(w.v0, 0) + tid : -1;
        return c.to >= c.from && c.to < c.e && tid - 8 < (int)((c.e - c.to) / ES) ? w.v1 - 1 - (tid - 8) : -1;
    };
    auto staged = [&](const Part<T, O> &w, int v) -> T * {  // element v of the run
        return reinterpret_cast<T *>(stage + (reinterpret_cast<uintptr_t>(w.in + max(w.v0, 0)) & 15)) + (v - max(w.v0, 0));
    };
    auto fetch = [&](const Part<T, O> &w, int r) {
        if (tid == 0) {
            const Pieces c = pieces_of(w, r);
            if (c.e > c.a && c.to > c.from) {
                mbar_arrive_expect_tx(&bar, (uint32_t)(c.to - c.from));
                bulk_g2s(stage + (c.from - (c.a & ~uintptr_t(15))), reinterpret_cast<const void *>(c.from),
                         (uint32_t)(c.to - c.from), &bar, policy_evict_first());
            } else {
                mbar_arrive(&bar);
            }
        }
        if (w.mask && w.v1 > max(w.v0, 0)) fetch_mask<NT>(bits, w.mask, w.v0, w.v1);
    };
    auto history_of = [&](int s) { return p.history ? p.history + (int64_t)s * p.history_stride : nullptr; };
    auto count_row = [&](const Words &q, const Part<T, O> &w, int r, int s, Tokens<2> &k) {
        if (counting && q.count && count_tokens<NT>(p, q, history_of(s), r, w.v0, w.v1, counts, k) && rank == 0)
            set_error(p.err, ERR_TOKEN);
        if (tid < 32) {
            entries[tid] = k.entry;
            values[tid] = k.value;
        }
    };
    // the last warp brings a sequence's words
    auto ask_words = [&](int r, int s) {
        if (warp == WARPS - 1 && r < p.num_rows) Words::fetch(p, s, raw_words);
    };
    auto put_words = [&](int i) {
        if (warp != WARPS - 1) return;
        Words q;
        q.gather(raw_words);
        q.check(p, rank == 0 && lane == 0);
        if (lane == 0) words[i] = q;
    };
    auto put_edge = [&](const Part<T, O> &w, int r) {
        const int at = edge_of(w, pieces_of(w, r));
        if (at < 0) return;
        *staged(w, at) = w.in[at];
        fence_proxy_async_smem();          // the stage is a copy's again
    };

    int r = (int)(blockIdx.x / C);
    uint32_t phase = 0, now = 0;           // of the copies; the row's place in what is double
    {
        const Part<T, O> w(p, r, rank, C);
        const int s = sequence(r);
        ask_words(r, s);
        if (s >= 0) {
            fetch(w, r);
            put_edge(w, r);
        }
        mask_here();
        __syncthreads();
        put_words(0);
        __syncthreads();
        ask_words(r + step, sequence(r + step));
        if (s >= 0) {
            Tokens<2> k;
            k.read<NT>(p, words[0], history_of(s), r);
            count_row(words[0], w, r, s, k);
        }
        mask_here();
    }
    __syncthreads();
    if (PROBS && C > 1) cluster_wait();                     // every block of the cluster runs

    for (; r < p.num_rows; r += step, now ^= 1) {
        const Part<T, O> w(p, r, rank, C);
        const bool here = sequence(r) >= 0;                 // as in all blocks of the cluster
        const Words q = words[now];
        const bool count = counting && q.count;             // (no memory for counts otherwise)
        put_words(now ^ 1);                // (of no use behind the last row)
        float x[EPT];
        uint32_t biased = 0;               // bit i: quad i has biases
        if (here) {
            if (!sh_dead && !mbar_wait_bounded(&bar, phase, p.err)) sh_dead = 1 + phase;
            phase ^= 1;
        }
        const int w0 = max(w.v0, 0) >> 5;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const int v = w.v0 + 4 * (i * NT + tid);
            Quad<T> raw;
            if (w.wide && v >= 0 && v + 4 <= w.v1) raw.load(staged(w, v));
            else raw.load_some(staged(w, v), [&](int e) { return v + e >= 0 && v + e < w.v1; });
            raw.widen(x + 4 * i);
            if (v >= w.v1) continue;
            if (count) {
                uint4 &c4 = reinterpret_cast<uint4 *>(counts)[i * NT + tid];
                const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w}, any = c[0] | c[1] | c[2] | c[3];
                if (any) {
                    q.penalties(c, x + 4 * i);
                    if (any & LG_BIAS) biased |= 1u << i;   // the sums of the biases from here on
                    c4 = make_uint4(0, 0, 0, 0);
                }
            }
            if (w.mask) forbid(bits, w0, v, x + 4 * i);
        }
        if (counting && q.b1 > q.b0) {
            __syncthreads();
            if (warp == 0) add_biases(p, q, w.v0, w.v1, counts, entries[lane], values[lane]);
            __syncthreads();
            if (biased) {
#pragma unroll
                for (int i = 0; i < Q; ++i)
                    if ((biased >> i) & 1) {
                        take_biases(counts + 4 * (i * NT + tid), x + 4 * i);
                        reinterpret_cast<uint4 *>(counts)[i * NT + tid] = make_uint4(0, 0, 0, 0);
                    }
            }
        }
        __syncthreads();                   // the stage, the counts and the words are free
        const int r2 = r + step, s2 = sequence(r2);
        if (s2 >= 0 && !sh_dead) fetch(Part<T, O>(p, r2, rank, C), r2);
        ask_words(r2 + step, sequence(r2 + step));
        if (q.inv_tau != 1.f) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) x[i] *= q.inv_tau;
        }
        const bool greedy = !(q.tau > 0.f);
        float mine = 0.f;                  // the level that x is to
        float4 *blocks = sh_blocks[phase];                  // (turns with the cluster's barriers)
        if (PROBS && here) {
            Stat st;
            if (greedy) {
#pragma unroll
                for (int i = 0; i < EPT; ++i)
                    if (x[i] > st.top) {
                        st.top = x[i];
                        st.top_at = w.v0 + 4 * ((i >> 2) * NT + tid) + (i & 3);
                    }
            } else {
                st.template add<EPT, true>(x);
            }
            mine = st.m;
            st.join(32, greedy);
            if (lane == 0) {
                sh_m[warp] = st.m;
                sh_l[warp] = st.l;
                sh_top[warp] = st.top;
                sh_at[warp] = st.top_at;
            }
            __syncthreads();
            if (warp == 0) {
                const int i = lane & (WARPS - 1);
                st.m = sh_m[i];
                st.l = sh_l[i];
                st.top = sh_top[i];
                st.top_at = sh_at[i];
                st.join(WARPS, greedy);
                st.send(blocks, rank, C);
            }
            cluster_arrive();
        }
        if (s2 >= 0) {
            const Part<T, O> w2(p, r2, rank, C);
            Tokens<2> k;
            k.read<NT>(p, words[now ^ 1], history_of(s2), r2);
            put_edge(w2, r2);
            count_row(words[now ^ 1], w2, r2, s2, k);
        }
        mask_here();
        if (PROBS && here) {
            __syncwarp();                  // the barrier is one of whole warps
            cluster_wait();
            if (greedy) {
                const int at = first_largest(blocks, C);
#pragma unroll
                for (int i = 0; i < EPT; ++i)
                    x[i] = w.v0 + 4 * ((i >> 2) * NT + tid) + (i & 3) == at ? 1.f : 0.f;
            } else {
                float base, inv;
                level_and_scale(blocks, C, base, inv);
                const float f = (mine == -INFINITY ? 0.f : ex2(mine - base)) * inv;
#pragma unroll
                for (int i = 0; i < EPT; ++i) x[i] *= f;
            }
        }
        if (here) store_tile<O, NT, EPT>(w.out, w.v0, w.v1, x);
        if (r2 - r_known >= KNOWN / 2 * step) {
            __syncthreads();               // every warp has looked its rows up
            know(r2);
        }
        __syncthreads();                   // counts, words and edges of the next row are here
    }
    // after a timeout: wait (bounded) for the copy still in flight
    if (sh_dead) mbar_wait_bounded(&bar, sh_dead - 1, p.err);
}

// How many clusters of C blocks the device holds at a time: asked of the runtime once
// for a shape (answers are kept for the last one).
template <typename Kernel>
int resident_clusters(Kernel kern, cudaLaunchConfig_t cfg, int C, std::atomic<uint64_t> &last) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const uint64_t key = ((uint64_t)cfg.dynamicSmemBytes << 24) | ((uint64_t)C << 20) | ((uint64_t)(dev & 15) << 16);
    const uint64_t was = last.load(std::memory_order_relaxed);
    if (was && (was & ~uint64_t(0xffff)) == key) return (int)(was & 0xffff);
    int n = 0;
    if (C > 1) {
        cfg.gridDim.x = (unsigned)C;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) n = 0;
    } else if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, (int)cfg.blockDim.x,
                                                             cfg.dynamicSmemBytes) != cudaSuccess) {
        n = 0;
    } else {
        n *= sm_count_of_current_device();
    }
    if (n > 0 && n <= 0xffff) last.store(key | (uint64_t)n, std::memory_order_relaxed);
    return n;
}

// Rows one after the other by the blocks that are resident: where there are more rows
// than that, and shared memory holds a run and its counts for as many blocks as the
// registers.  -1: not such a case.
template <typename T, typename O, int NT, int EPT, bool PROBS>
int launch_rows(const LogitsParams &p, int C, int run, cudaStream_t st, cudaError_t &e) {
    auto kern = process_rows_kernel<T, O, NT, EPT, PROBS>;
    const bool count = p.repetition || p.frequency || p.presence || p.bias_start;
    LogitsParams q = p;
    q.run = run;
    const size_t smem = (count ? (size_t)run * 4 : 0) + (size_t)run * sizeof(T) + 32;
    const size_t fixed = (NT * EPT / 32 + 2) * 4 + NT / 32 * 16 + 2 * LG_CLUSTER * 16 + 32 * 12 + 2 * 64 + 128;
    if ((smem + fixed + 1024) * (1024 / NT) > 228 * 1024) return -1;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(NT, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PROBS ? 1 : 0;
    static std::atomic<uint64_t> last{0};
    const int n = PROBS ? resident_clusters(kern, cfg, C, last) : resident_clusters(kern, cfg, 1, last) / C;
    if (n <= 0 || p.num_rows <= n) return -1;
    cfg.gridDim = dim3((unsigned)(n * C), 1, 1);
    e = cudaLaunchKernelEx(&cfg, kern, q, C);
    return 0;
}

template <typename T, typename O, int NT, int EPT, bool RESIDENT>
cudaError_t launch_ept(const LogitsParams &p, int C, int tile, cudaStream_t st) {
    if constexpr (RESIDENT && EPT == LG_EPT) {
        cudaError_t e = cudaSuccess;
        if ((p.probs ? launch_rows<T, O, NT, EPT, true>(p, C, tile, st, e)
                     : launch_rows<T, O, NT, EPT, false>(p, C, tile, st, e)) == 0)
            return e;
    }
    auto kern = process_logits_kernel<T, O, NT, EPT, RESIDENT>;
    const bool count = p.repetition || p.frequency || p.presence || p.bias_start;
    const size_t smem = count ? (size_t)tile * 4 : 0;
    if (smem > 46 * 1024) {                        // beside the static part
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, NT * EPT * 4);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)p.num_rows * C), 1, 1);
    cfg.blockDim = dim3(NT, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T, typename O>
cudaError_t launch_logits(const LogitsParams &p, cudaStream_t st) {
    const int sms = sm_count_of_current_device();
    // as few blocks a row as hold it, more where the rows alone do not fill the SMs
    int C = 1;
    while (C < LG_CLUSTER && (p.vocab > C * (256 * LG_EPT - 8) ||
                              (int64_t)p.num_rows * C * 2 <= 2 * (sms > 0 ? sms : 152))) C *= 2;
    if ((int64_t)p.num_rows * C > (int64_t)INT32_MAX) return cudaErrorNotSupported;
    const int run = (int)((((int64_t)p.vocab + 6) / 4 + C - 1) / C * 4);     // wherever the rows start
    if (run <= 256 * 8) return launch_ept<T, O, 256, 8, true>(p, C, run, st);
    if (run <= 256 * 16) return launch_ept<T, O, 256, 16, true>(p, C, run, st);
    if (run <= 256 * LG_EPT) return launch_ept<T, O, 256, LG_EPT, true>(p, C, run, st);
    if (run <= 512 * LG_EPT) return launch_ept<T, O, 512, LG_EPT, true>(p, C, run, st);
    return launch_ept<T, O, 512, 32, false>(p, C, 512 * 32, st);
}

}  // namespace

}  // namespace pa
