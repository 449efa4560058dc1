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
// while the logits are on their way.  Neighbouring lanes hold neighbouring
// elements: rows may start anywhere (vocabularies are odd), and a warp's 32 elements
// share one word of the mask.  Runs that do not fit into registers are read twice,
// the second time mostly from L2.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int LG_THREADS = 512;
constexpr int LG_WARPS = LG_THREADS / 32;
constexpr int LG_EPT = 32;                 // elements of a thread, at most
constexpr int LG_TILE = LG_THREADS * LG_EPT;
constexpr int LG_CLUSTER = 8;

constexpr uint32_t LG_PROMPT = 0x80000000u, LG_BIAS = 0x40000000u, LG_COUNT = 0x3fffffffu;

// The largest element, the first place of it, and the sum of exp2 to it.
struct Top {
    float m, l;
    int at;
};

// The factor that takes a sum to m over to base; a NaN sum without a largest element
// stays one.
__device__ __forceinline__ float carry(float m, float l, float base) {
    return m == -INFINITY ? (l != l ? 1.f : 0.f) : ex2((m - base) * LOG2E);
}

__device__ __forceinline__ bool before(float m, int at, float m2, int at2) {   // (m, at) goes first
    return m > m2 || (m == m2 && at < at2);
}

// sequence of row r: the last s with query_start[s] <= r; -1 if no sequence has it
__device__ __forceinline__ int sequence_of(const int32_t *qs, int B, int r, int lane) {
    int lo = 0, n = B;                     // in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const unsigned ok = __ballot_sync(0xffffffffu, lane * step < n && qs[at] <= r);
        // the probes hold for a first part of the lanes when the starts do not decrease
        const int k = ok ? 31 - __clz(ok) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return qs[lo] <= r && r < qs[lo + 1] ? lo : -1;
}

template <typename T, typename O, int EPT, bool RESIDENT>
__global__ void __launch_bounds__(LG_THREADS, 2) process_logits_kernel(const __grid_constant__ LogitsParams p) {
    extern __shared__ uint32_t counts[];                    // [tile]
    __shared__ float sh_m[LG_WARPS], sh_l[LG_WARPS];
    __shared__ int sh_at[LG_WARPS];
    __shared__ float4 sh_blocks[LG_CLUSTER];                // (m, l, at) of the cluster's blocks
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
    const int r = (int)(blockIdx.x / C);
    const int s = sequence_of(p.query_start, p.num_seqs, r, lane);
    if (s < 0) return;                                      // the whole cluster: no such row
    if (C > 1) cluster_arrive();                            // this block runs (see cluster_wait below)

    const int V = p.vocab;
    const int run = (V + 32 * C - 1) / (32 * C) * 32;       // a block's part of the vocabulary
    const int v0 = min(V, rank * run), v1 = min(V, v0 + run);
    const T *in = static_cast<const T *>(p.logits) + (int64_t)r * p.logits_stride;
    O *out = static_cast<O *>(p.out) + (int64_t)r * p.out_stride;

    const float theta = p.repetition ? p.repetition[s] : 1.f;
    const float alpha = p.frequency ? p.frequency[s] : 0.f;
    const float beta = p.presence ? p.presence[s] : 0.f;
    const float tau = p.temperature ? p.temperature[s] : 1.f;
    const bool penalise = theta != 1.f || alpha != 0.f || beta != 0.f;
    const float inv_theta = 1.f / theta, inv_tau = tau > 0.f ? 1.f / tau : 1.f;
    int b0 = 0, b1 = 0;
    if (p.bias_start) {
        b0 = p.bias_start[s];
        b1 = p.bias_start[s + 1];
        if (b0 < 0 || b1 < b0 || b1 > p.num_bias) {
            if (rank == 0 && tid == 0) set_error(p.err, ERR_SEQ_LEN);
            b0 = b1 = 0;
        }
    }
    const bool count = penalise || b1 > b0;
    const uint32_t *mask = p.allowed ? p.allowed + (int64_t)r * p.allowed_stride : nullptr;

    // counts of tokens [t0, t1): prompt and bias flags, times in the output
    auto build = [&](int t0, int t1) {
        for (int i = tid; i < t1 - t0; i += LG_THREADS) counts[i] = 0;
        __syncthreads();
        bool bad = false;
        auto add = [&](int32_t v, bool prompt) {
            if (v < 0 || v >= V) {
                bad = true;
            } else if (v >= t0 && v < t1) {
                if (prompt) atomicOr(&counts[v - t0], LG_PROMPT);
                else atomicAdd(&counts[v - t0], 1u);
            }
        };
        if (penalise) {
            if (p.history) {
                int len = p.history_lens[s], pl = p.prompt_lens ? p.prompt_lens[s] : 0;
                if (len < 0 || len > p.history_stride || pl < 0 || pl > len) {
                    if (rank == 0 && tid == 0) set_error(p.err, ERR_SEQ_LEN);
                    len = max(0, (int)min((int64_t)len, p.history_stride));
                    pl = min(max(pl, 0), len);
                }
                const int32_t *h = p.history + (int64_t)s * p.history_stride;
#pragma unroll 4
                for (int i = tid; i < len; i += LG_THREADS) add(h[i], i < pl);
            }
            if (p.tokens)                  // the drafts before this row
                for (int i = p.query_start[s] + 1 + tid; i <= r; i += LG_THREADS) add(p.tokens[i], false);
        }
        for (int i = b0 + tid; i < b1; i += LG_THREADS) {
            const int32_t v = p.bias_tokens[i];
            if (v < 0 || v >= V) bad = true;
            else if (v >= t0 && v < t1) atomicOr(&counts[v - t0], LG_BIAS);
        }
        if (bad && rank == 0) set_error(p.err, ERR_TOKEN);
        __syncthreads();
    };
    // the biases of token v, added in the order of the list; the warp together
    auto bias_of = [&](int v) -> float {
        float sum = 0.f;
        for (int i = b0; i < b1; i += 32) {
            const int e = i + lane;
            const bool mine = e < b1 && p.bias_tokens[e] == v;
            const float x = mine ? p.bias_values[e] : 0.f;
            unsigned hit = __ballot_sync(0xffffffffu, mine);
            while (hit) {
                sum += __shfl_sync(0xffffffffu, x, __ffs(hit) - 1);
                hit &= hit - 1;
            }
        }
        return sum;
    };
    // EPT elements of the tile at t0 from tid on, as processed (-inf past its end)
    auto load = [&](float (&x)[EPT], int t0, int t1) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const int v = t0 + i * LG_THREADS + tid;
            x[i] = v < t1 ? Elem<T>::load1(in + v) : -INFINITY;
        }
    };
    auto process = [&](float (&x)[EPT], int t0, int t1) {
        if (count) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const int k = i * LG_THREADS + tid;
                const uint32_t c = t0 + k < t1 ? counts[k] : 0u;
                if (__any_sync(0xffffffffu, c != 0)) {
                    if (c & ~LG_BIAS) {
                        const uint32_t n = c & LG_COUNT;
                        x[i] = x[i] > 0.f ? x[i] * inv_theta : x[i] * theta;
                        x[i] = x[i] - alpha * (float)n - (n ? beta : 0.f);
                    }
                    unsigned hit = __ballot_sync(0xffffffffu, (c & LG_BIAS) != 0);
                    while (hit) {
                        const int l = __ffs(hit) - 1;
                        const float b = bias_of(t0 + i * LG_THREADS + (warp * 32) + l);
                        if (lane == l) x[i] += b;
                        hit &= hit - 1;
                    }
                }
            }
        }
        if (mask) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const int v = t0 + i * LG_THREADS + tid;
                if (v < t1 && !((mask[v >> 5] >> (v & 31)) & 1)) x[i] = -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < EPT; ++i) x[i] *= inv_tau;
    };

    float x[EPT];
    if (!p.probs) {
        for (int t0 = v0; t0 < v1; t0 += LG_TILE) {
            const int t1 = min(v1, t0 + LG_TILE);
            load(x, t0, t1);
            if (count) build(t0, t1);
            process(x, t0, t1);
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const int v = t0 + i * LG_THREADS + tid;
                if (v < t1) Elem<O>::store1(out + v, x[i]);
            }
            if (count && t0 + LG_TILE < v1) __syncthreads();     // before the next counts
        }
        if (C > 1) cluster_wait();
        return;
    }

    // ---- the run's largest element and sum
    Top top{-INFINITY, 0.f, INT32_MAX};
    for (int t0 = v0; t0 < v1; t0 += LG_TILE) {
        const int t1 = min(v1, t0 + LG_TILE);
        load(x, t0, t1);
        if (count) build(t0, t1);
        process(x, t0, t1);
        float m = -INFINITY;
        int at = INT32_MAX;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const int v = t0 + i * LG_THREADS + tid;
            if (x[i] > m) {
                m = x[i];
                at = v;
            }
        }
        const float up = fmaxf(m, top.m), base = up == -INFINITY ? 0.f : up;
        float l = top.l * carry(top.m, top.l, base);
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const float e = ex2((x[i] - base) * LOG2E);
            if constexpr (RESIDENT) x[i] = e;
            l += e;
        }
        if (before(m, at, top.m, top.at)) top.at = at;
        top.m = up;
        top.l = l;
        if (!RESIDENT && count) __syncthreads();
    }
    const float mine = top.m;              // what x holds is relative to (resident)
    auto join = [](Top &a, const Top &b) {
        const float up = fmaxf(a.m, b.m), base = up == -INFINITY ? 0.f : up;
        a.l = a.l * carry(a.m, a.l, base) + b.l * carry(b.m, b.l, base);
        if (before(b.m, b.at, a.m, a.at)) a.at = b.at;
        a.m = up;
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        join(top, Top{__shfl_xor_sync(0xffffffffu, top.m, o), __shfl_xor_sync(0xffffffffu, top.l, o),
                      __shfl_xor_sync(0xffffffffu, top.at, o)});
    if (lane == 0) {
        sh_m[warp] = top.m;
        sh_l[warp] = top.l;
        sh_at[warp] = top.at;
    }
    __syncthreads();
    // a peer's shared memory may be written once that block is known to run
    if (C > 1) cluster_wait();
    if (warp == 0) {
        Top b{-INFINITY, 0.f, INT32_MAX};
        if (lane < LG_WARPS) b = Top{sh_m[lane], sh_l[lane], sh_at[lane]};
#pragma unroll
        for (int o = LG_WARPS / 2; o > 0; o >>= 1)
            join(b, Top{__shfl_xor_sync(0xffffffffu, b.m, o), __shfl_xor_sync(0xffffffffu, b.l, o),
                        __shfl_xor_sync(0xffffffffu, b.at, o)});
        if (lane < C)
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::
                         "r"(map_to_rank(&sh_blocks[rank], (uint32_t)lane)), "f"(b.m), "f"(b.l),
                         "f"(__int_as_float(b.at)), "f"(0.f) : "memory");
        __syncwarp();                                       // the barrier below is one of whole warps
    }
    cluster_sync();
    Top all{-INFINITY, 0.f, INT32_MAX};
    for (int i = 0; i < C; ++i) {
        const float4 b = sh_blocks[i];
        join(all, Top{b.x, b.y, __float_as_int(b.z)});
    }

    // ---- the row
    if (!(tau > 0.f)) {
        for (int v = v0 + tid; v < v1; v += LG_THREADS) Elem<O>::store1(out + v, v == all.at ? 1.f : 0.f);
        return;
    }
    const float inv = all.l == 0.f ? 0.f : 1.f / all.l;     // nothing allowed: zeros
    const float base = all.m == -INFINITY ? 0.f : all.m;
    if constexpr (RESIDENT) {
        const float f = (mine == -INFINITY ? 0.f : ex2((mine - base) * LOG2E)) * inv;   // x is to this thread's maximum
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const int v = v0 + i * LG_THREADS + tid;
            if (v < v1) Elem<O>::store1(out + v, x[i] * f);
        }
    } else {
        for (int t0 = v0; t0 < v1; t0 += LG_TILE) {
            const int t1 = min(v1, t0 + LG_TILE);
            load(x, t0, t1);
            if (count) build(t0, t1);
            process(x, t0, t1);
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const int v = t0 + i * LG_THREADS + tid;
                if (v < t1) Elem<O>::store1(out + v, ex2((x[i] - base) * LOG2E) * inv);
            }
            if (count) __syncthreads();
        }
    }
}

template <typename T, typename O, int EPT, bool RESIDENT>
cudaError_t launch_ept(const LogitsParams &p, int C, int tile, cudaStream_t st) {
    auto kern = process_logits_kernel<T, O, EPT, RESIDENT>;
    const bool count = p.repetition || p.frequency || p.presence || p.bias_start;
    const size_t smem = count ? (size_t)tile * 4 : 0;
    if (smem > 46 * 1024) {                        // beside the static part
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, LG_TILE * 4);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)p.num_rows * C), 1, 1);
    cfg.blockDim = dim3(LG_THREADS, 1, 1);
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
    while (C < LG_CLUSTER && (p.vocab > C * LG_TILE || (int64_t)p.num_rows * C * 2 <= 2 * (sms > 0 ? sms : 152))) C *= 2;
    if ((int64_t)p.num_rows * C > (int64_t)INT32_MAX) return cudaErrorNotSupported;
    const int run = (int)(((int64_t)p.vocab + 32 * C - 1) / (32 * C) * 32);
    if (run <= 8 * LG_THREADS) return launch_ept<T, O, 8, true>(p, C, run, st);
    if (run <= 16 * LG_THREADS) return launch_ept<T, O, 16, true>(p, C, run, st);
    if (run <= LG_TILE) return launch_ept<T, O, 32, true>(p, C, run, st);
    return launch_ept<T, O, 32, false>(p, C, LG_TILE, st);
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
