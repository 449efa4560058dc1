// pa_logits.cu -- logits made ready for sampling or for the verification of drafts:
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
#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_mma.cuh"

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
    const int V = p.vocab;
    const T *in = static_cast<const T *>(p.logits) + (int64_t)r * p.logits_stride;
    O *out = static_cast<O *>(p.out) + (int64_t)r * p.out_stride;
    // quads: four elements on borders of the output's; the first may begin before the row
    const int lead = (int)((reinterpret_cast<uintptr_t>(out) / sizeof(O)) & 3);
    const bool wide = (int)((reinterpret_cast<uintptr_t>(in) / sizeof(T)) & 3) == lead;
    const int run = ((V + lead + 3) / 4 + C - 1) / C * 4;   // a block's part, in elements
    const int v0 = rank * run - lead, v1 = min(V, v0 + run);
    const uint32_t *mask = p.allowed ? p.allowed + (int64_t)r * p.allowed_stride : nullptr;

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
            if (wide && v >= 0 && v + 4 <= t1) q.load(in + v);
            else q.load_some(in + v, [&](int e) { return v + e >= 0 && v + e < t1; });
            if constexpr (!NARROW) q.widen(x + 4 * i);
        }
        if (mask) {
            const int w0 = max(t0, 0) >> 5, n = ((t1 - 1) >> 5) - w0 + 1;
            for (int i = tid; i < n; i += NT)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(smem_u32(&bits[i])), "l"(mask + w0 + i)
                             : "memory");
        }
    };
    // the tile's words of the mask are here once the block has met behind this
    auto words_here = [&]() { asm volatile("cp.async.wait_all;" ::: "memory"); };
    const int s = sequence_of(p.query_start, p.num_seqs, r, lane);
    if (s < 0) return;                                      // the whole cluster: no such row
    if (C > 1) cluster_arrive();                            // this block runs (see cluster_wait below)
    const float theta = p.repetition ? p.repetition[s] : 1.f;
    const float alpha = p.frequency ? p.frequency[s] : 0.f;
    const float beta = p.presence ? p.presence[s] : 0.f;
    const float tau = p.temperature ? p.temperature[s] : 1.f;
    const int first = p.query_start[s];
    int len = 0, asked = 0, b0 = 0, b1 = 0;                 // of the history; of these the prompt's; biases
    if (p.history) {
        len = p.history_lens[s];
        asked = p.prompt_lens ? p.prompt_lens[s] : 0;
    }
    if (p.bias_start) {
        b0 = p.bias_start[s];
        b1 = p.bias_start[s + 1];
    }
    // The logits behind these few words (in front of them they hold them up, as the memory
    // answers in order: 3 us of a block's 14), and on their way while the history is
    // counted.
    load(v0, min(v1, v0 + TILE));
    if (len < 0 || len > p.history_stride || asked < 0 || asked > len) {
        if (rank == 0 && tid == 0) set_error(p.err, ERR_SEQ_LEN);
        len = max(0, (int)min((int64_t)len, p.history_stride));
        asked = min(max(asked, 0), len);
    }
    if (b0 < 0 || b1 < b0 || b1 > p.num_bias) {
        if (rank == 0 && tid == 0) set_error(p.err, ERR_SEQ_LEN);
        b0 = b1 = 0;
    }
    const bool penalise = theta != 1.f || alpha != 0.f || beta != 0.f;
    const bool count = penalise || b1 > b0;
    const float inv_theta = 1.f / theta, inv_tau = tau > 0.f ? 1.f / tau : 1.f;

    // counts of the tile's tokens: prompt and bias flags, times in the output
    const int32_t *hist = p.history ? p.history + (int64_t)s * p.history_stride : nullptr;
    if (!penalise) len = 0;
    constexpr int AHEAD = 4;               // history loads of a thread in flight
    auto build = [&](int t0, int t1) {
        int32_t h[AHEAD];
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) h[e] = tid + e * NT < len ? hist[tid + e * NT] : -1;
#pragma unroll
        for (int i = 0; i < Q; ++i)
            if (4 * (i * NT + tid) < t1 - t0)
                reinterpret_cast<uint4 *>(counts)[i * NT + tid] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        const int lo = max(t0, 0);
        bool bad = false;
        auto add = [&](int32_t v, bool prompt) {
            bad = bad || (uint32_t)v >= (uint32_t)V;
            if (v >= lo && v < t1) {
                if (prompt) atomicOr(&counts[v - t0], LG_PROMPT);
                else atomicAdd(&counts[v - t0], 1u);
            }
        };
        for (int i = tid; i < len; i += AHEAD * NT) {
            int32_t next[AHEAD];
#pragma unroll
            for (int e = 0; e < AHEAD; ++e) {
                const int at = i + (AHEAD + e) * NT;
                next[e] = at < len ? hist[at] : -1;
            }
#pragma unroll
            for (int e = 0; e < AHEAD; ++e) {
                if (i + e * NT < len) add(h[e], i + e * NT < asked);
                h[e] = next[e];
            }
        }
        if (p.tokens && penalise)          // the drafts before this row
            for (int i = first + 1 + tid; i <= r; i += NT) add(p.tokens[i], false);
        for (int i = b0 + tid; i < b1; i += NT) {
            const int32_t v = p.bias_tokens[i];
            bad = bad || (uint32_t)v >= (uint32_t)V;
            if (v >= lo && v < t1) atomicOr(&counts[v - t0], LG_BIAS);
        }
        if (bad && rank == 0) set_error(p.err, ERR_TOKEN);
        words_here();
        __syncthreads();
    };
    auto process = [&](int t0, int t1) {
        if (!count && mask) {
            words_here();
            __syncthreads();
        }
        uint32_t biased = 0;               // bit i: quad i has biases
        const int w0 = max(t0, 0) >> 5;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            if constexpr (NARROW) raw[i].widen(x + 4 * i);
            const int v = quad_at(t0, i);
            if (v >= t1) continue;
            if (count) {
                uint4 &c4 = reinterpret_cast<uint4 *>(counts)[i * NT + tid];
                uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
                if (c[0] | c[1] | c[2] | c[3]) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float &y = x[4 * i + e];
                        const uint32_t n = c[e] & LG_COUNT;
                        const float z = (y > 0.f ? y * inv_theta : y * theta) - alpha * (float)n - (n ? beta : 0.f);
                        y = c[e] & ~LG_BIAS ? z : y;
                    }
                    if ((c[0] | c[1] | c[2] | c[3]) & LG_BIAS) {
                        biased |= 1u << i;
                        c4 = make_uint4(0, 0, 0, 0);        // the sums of the biases from here on
                    }
                }
            }
            if (mask) {
                const int at = max(v, 0);
                const uint32_t w = bits[(at >> 5) - w0], w2 = bits[(at >> 5) - w0 + 1];
                const uint32_t ok = __funnelshift_r(w, w2, at & 31) << (at - v);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * i + e] = (ok >> e) & 1 ? x[4 * i + e] : -INFINITY;
            }
        }
        if (b1 > b0) {
            // one warp adds the biases up in the order of the list, 32 at a time: of
            // the entries that name one token the first takes them all.
            __syncthreads();
            if (warp == 0) {
                for (int i = b0; i < b1; i += 32) {
                    const bool in_list = i + lane < b1;
                    const int32_t v = in_list ? p.bias_tokens[i + lane] : -1 - lane;
                    const float y = in_list ? p.bias_values[i + lane] : 0.f;
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
            __syncthreads();
            if (biased) {
#pragma unroll
                for (int i = 0; i < Q; ++i)
                    if ((biased >> i) & 1) {
                        const float4 y = reinterpret_cast<const float4 *>(counts)[i * NT + tid];
                        const float add[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)        // what is not allowed stays so
                            x[4 * i + e] = x[4 * i + e] == -INFINITY ? -INFINITY : x[4 * i + e] + add[e];
                    }
            }
        }
        if (inv_tau != 1.f) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) x[i] *= inv_tau;
        }
    };
    auto store = [&](int t0, int t1) {
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const int v = quad_at(t0, i);
            if (v >= 0 && v + 4 <= t1) {
                store_quad<O>(out + v, x + 4 * i);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (v + e >= 0 && v + e < t1) Elem<O>::store1(out + v + e, x[4 * i + e]);
            }
        }
    };

    if (!p.probs) {
        for (int t0 = v0; t0 < v1; t0 += TILE) {
            const int t1 = min(v1, t0 + TILE);
            if (t0 > v0) load(t0, t1);
            if (count) build(t0, t1);
            process(t0, t1);
            store(t0, t1);
            if (t0 + TILE < v1) __syncthreads();            // before the next counts and words
        }
        if (C > 1) cluster_wait();
        return;
    }

    // ---- the run's largest element and sum: levels m in log2 units, and for a row
    // that takes the first largest that element and its place
    float m = -INFINITY, l = 0.f, top = -INFINITY;
    int top_at = INT32_MAX;
    const bool greedy = !(tau > 0.f);
    for (int t0 = v0; t0 < v1; t0 += TILE) {
        const int t1 = min(v1, t0 + TILE);
        if (t0 > v0) load(t0, t1);
        if (count) build(t0, t1);
        process(t0, t1);
        if (greedy) {
#pragma unroll
            for (int i = 0; i < EPT; ++i)
                if (x[i] > top) {
                    top = x[i];
                    top_at = quad_at(t0, i >> 2) + (i & 3);
                }
        } else {
            float big = -INFINITY;
#pragma unroll
            for (int i = 0; i < EPT; i += 2) big = max3f(big, x[i], x[i + 1]);
            const float up = fmaxf(m, big * LOG2E), base = up == -INFINITY ? 0.f : up;
            float sum[4] = {l * carry(m, l, base), 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const float e = ex2(fmaf(x[i], LOG2E, -base));
                if constexpr (RESIDENT) x[i] = e;
                sum[i & 3] += e;
            }
            m = up;
            l = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        if (!RESIDENT) __syncthreads();
    }
    const float mine = m;                  // the level that x is to (resident)
    // over the warp, the block's warps, the cluster's blocks
    auto join = [&](int lanes) {
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
    };
    join(32);
    if (lane == 0) {
        sh_m[warp] = m;
        sh_l[warp] = l;
        sh_top[warp] = top;
        sh_at[warp] = top_at;
    }
    __syncthreads();
    // a peer's shared memory may be written once that block is known to run
    if (C > 1) cluster_wait();
    if (warp == 0) {
        const int w = lane & (WARPS - 1);
        m = sh_m[w];
        l = sh_l[w];
        top = sh_top[w];
        top_at = sh_at[w];
        join(WARPS);
        if (lane < C)
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::
                         "r"(map_to_rank(&sh_blocks[rank], (uint32_t)lane)), "f"(m), "f"(l), "f"(top),
                         "f"(__int_as_float(top_at)) : "memory");
        __syncwarp();                                       // the barrier below is one of whole warps
    }
    cluster_sync();

    // ---- the row
    if (greedy) {
        float best = -INFINITY;
        int at = INT32_MAX;
        for (int i = 0; i < C; ++i)
            if (before(sh_blocks[i].z, __float_as_int(sh_blocks[i].w), best, at)) {
                best = sh_blocks[i].z;
                at = __float_as_int(sh_blocks[i].w);
            }
        for (int t0 = v0; t0 < v1; t0 += TILE) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) x[i] = quad_at(t0, i >> 2) + (i & 3) == at ? 1.f : 0.f;
            store(t0, min(v1, t0 + TILE));
        }
        return;
    }
    float up = -INFINITY, sum = 0.f;
    for (int i = 0; i < C; ++i) up = fmaxf(up, sh_blocks[i].x);
    const float base = up == -INFINITY ? 0.f : up;
    for (int i = 0; i < C; ++i) sum += sh_blocks[i].y * carry(sh_blocks[i].x, sh_blocks[i].y, base);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;         // nothing allowed: zeros
    if constexpr (RESIDENT) {
        const float f = (mine == -INFINITY ? 0.f : ex2(mine - base)) * inv;
#pragma unroll
        for (int i = 0; i < EPT; ++i) x[i] *= f;
        store(v0, v1);
    } else {
        for (int t0 = v0; t0 < v1; t0 += TILE) {
            const int t1 = min(v1, t0 + TILE);
            load(t0, t1);
            if (count) build(t0, t1);
            process(t0, t1);
#pragma unroll
            for (int i = 0; i < EPT; ++i) x[i] = ex2(fmaf(x[i], LOG2E, -base)) * inv;
            store(t0, t1);
            __syncthreads();
        }
    }
}

template <typename T, typename O, int NT, int EPT, bool RESIDENT>
cudaError_t launch_ept(const LogitsParams &p, int C, int tile, cudaStream_t st) {
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

cudaError_t process_logits(const LogitsParams &p, int dtype, int out_dtype, cudaStream_t st) {
    switch (dtype) {
        case 0: return launch_logits<float, float>(p, st);
        case 1:
            return out_dtype == 0 ? launch_logits<__nv_bfloat16, float>(p, st)
                                  : launch_logits<__nv_bfloat16, __nv_bfloat16>(p, st);
        default:
            return out_dtype == 0 ? launch_logits<__half, float>(p, st) : launch_logits<__half, __half>(p, st);
    }
}

}  // namespace pa
