// pa_verify.cu -- verification of drafted tokens: the accept test of every
// draft of a sequence and the token drawn after the accepted ones.
//
// With target row p_i and draft row q_i behind draft x_i and a uniform u_i,
// drafts are accepted in order while u_i q_i(x_i) < p_i(x_i).  At the first
// rejection the next token comes from w = max(p_i - q_i, 0), and when all are
// accepted from w = p of the row behind the last one: the first v whose
// cumulative weight C_v exceeds u W (W the row's sum).  The vocabulary's
// cumulative sums decide a whole number, and a row has 10^4 to 10^5 borders that
// u W can fall next to, so sums carry about 48 bits or more: a lane adds its
// elements in pairs of floats (the rounding error of every addition is kept
// and added up beside it), and everything above a lane is binary64.
//
// Bound by HBM for batches (one or two rows of the vocabulary per sequence),
// by latency for one sequence.  A cluster of C blocks takes one sequence: the
// row is cut into C * 16 runs, one per warp, each summed in one pass; the
// block sums meet through distributed shared memory, and only the run that
// holds the border is read again, by the whole block that owns it.  One launch,
// no workspace, no atomics on global memory, a fixed order of additions.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int VF_THREADS = 512;
constexpr int VF_WARPS = VF_THREADS / 32;

// Negative entries and NaN count as 0; the comparison also drops +inf.
__device__ __forceinline__ float weight_of(float p, float q) {
    const float w = fmaxf(p - fmaxf(q, 0.f), 0.f);
    return w < INFINITY ? w : 0.f;
}

template <typename T>
struct Row {
    const T *p, *q;      // q: nullptr without draft probabilities or rejection
    int64_t hole;        // token whose weight is 0 (rejected, no probabilities), or -1
    __device__ __forceinline__ float at(int64_t v) const {
        const float w = weight_of(Elem<T>::load1(p + v), q ? Elem<T>::load1(q + v) : 0.f);
        return v == hole ? 0.f : w;
    }
};

// hi + lo += x with the rounding error of hi + x kept in lo
__device__ __forceinline__ void add_pair(float &hi, float &lo, float x) {
    const float s = hi + x, z = s - hi;
    lo += (hi - (s - z)) + (x - z);
    hi = s;
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ double ld_dsmem_f64(uint32_t addr) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}

template <typename T>
__global__ void __launch_bounds__(VF_THREADS) verify_drafts_kernel(const __grid_constant__ VerifyParams p) {
    __shared__ int sh_acc;                          // accepted drafts
    __shared__ int sh_reject;                       // a draft was rejected
    __shared__ double sh_warp[VF_WARPS];            // sums of the warps' runs
    __shared__ double sh_block;                     // and of the block's
    __shared__ double sh_scan[VF_WARPS];
    __shared__ unsigned sh_first, sh_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
    const int s = (int)(blockIdx.x / C);
    const int64_t V = p.vocab;
    int32_t *out = p.out_tokens + (int64_t)s * p.max_query_len;

    const int q0 = p.query_start[s], q1 = p.query_start[s + 1], n = q1 - q0;
    if (q0 < 0 || n <= 0 || q1 > p.num_rows || n > p.max_query_len) {
        // the whole cluster leaves here, so no peer waits for this block
        if (rank == 0) {
            if (n != 0 && tid == 0) set_error(p.err, ERR_SEQ_LEN);
            for (int j = tid; j < p.max_query_len; j += VF_THREADS) out[j] = -1;
            if (tid == 0) p.num_accepted[s] = 0;
        }
        return;
    }
    const T *target = static_cast<const T *>(p.target);
    const T *draft = static_cast<const T *>(p.draft);

    // ---- the accept test, 32 drafts at a time, in every block of the cluster
    if (warp == 0) {
        int acc = 0;
        bool reject = false;
        for (int i0 = 1; i0 < n && !reject; i0 += 32) {
            const int i = i0 + lane;
            bool ok = true, outside = false;        // lanes past the last draft
            if (i < n) {
                const int64_t r = (int64_t)q0 + i;
                const int32_t x = p.tokens[r];
                ok = false;
                if (x >= 0 && x < V) {
                    const float pt = weight_of(Elem<T>::load1(target + (r - 1) * p.target_stride + x), 0.f);
                    const float qt = draft ? fmaxf(Elem<T>::load1(draft + r * p.draft_stride + x), 0.f) : 1.f;
                    // the product of two floats is exact in binary64
                    ok = (double)p.accept_u[r] * (double)qt < (double)pt;
                } else {
                    outside = true;
                }
            }
            const unsigned bad = ~__ballot_sync(0xffffffffu, ok);
            if (bad) {
                reject = true;
                acc = i0 - 1 + __ffs(bad) - 1;
                if (outside && lane == __ffs(bad) - 1 && rank == 0) set_error(p.err, ERR_TOKEN);
            } else {
                acc = min(n - 1, i0 + 31);
            }
        }
        if (lane == 0) {
            sh_acc = acc;
            sh_reject = reject;
        }
    }
    __syncthreads();
    const int a = sh_acc;
    const bool reject = sh_reject != 0;
    Row<T> row;
    row.p = target + ((int64_t)q0 + a) * p.target_stride;
    row.q = nullptr;
    row.hole = -1;
    if (reject) {
        if (draft) row.q = draft + ((int64_t)q0 + a + 1) * p.draft_stride;
        else row.hole = p.tokens[q0 + a + 1];
    }
    const int64_t chunk = ((V + (int64_t)C * VF_WARPS - 1) / ((int64_t)C * VF_WARPS) + 31) / 32 * 32;
    auto run_lo = [&](int w) -> int64_t {           // first element of warp w's run in this block
        const int64_t x = ((int64_t)rank * VF_WARPS + w) * chunk;
        return x < V ? x : V;
    };

    double W = 0., before = 0., mine = 0.;
    for (int pass = 0; pass < 2; ++pass) {
        // ---- sums of the runs
        const int64_t lo = run_lo(warp), hi = run_lo(warp + 1);
        float sh = 0.f, sl = 0.f;
        constexpr int U = 8;
        for (int64_t v0 = lo + lane; v0 < hi; v0 += 32 * U) {
            float x[U];
#pragma unroll
            for (int e = 0; e < U; ++e) x[e] = v0 + 32 * e < hi ? row.at(v0 + 32 * e) : 0.f;
#pragma unroll
            for (int e = 0; e < U; ++e) add_pair(sh, sl, x[e]);
        }
        const double sum = warp_sum((double)sh + (double)sl);
        if (lane == 0) sh_warp[warp] = sum;
        __syncthreads();
        if (tid == 0) {
            double b = 0.;
            for (int w = 0; w < VF_WARPS; ++w) b += sh_warp[w];
            sh_block = b;
        }
        cluster_sync();
        W = before = mine = 0.;
        for (int c = 0; c < C; ++c) {
            const double b = ld_dsmem_f64(map_to_rank(&sh_block, (uint32_t)c));
            if (c == rank) {
                before = W;
                mine = b;
            }
            W += b;
        }
        cluster_sync();                             // peers have read sh_block
        // nothing left of max(p - q, 0): the target's own row; every block
        // sees the same W
        if (W > 0. || (!row.q && row.hole < 0)) break;
        row.q = nullptr;
        row.hole = -1;
    }

    // ---- the border u W, in the block whose sums reach past it (the last
    // block with any weight if rounding leaves none)
    const float us = p.sample_u[s];
    const double u = us > 0.f ? (us < 1.f ? (double)us : 1.) : 0.;
    const double x = u * W;
    const bool drawn = W > 0. && W < INFINITY;
    if (rank == 0) {
        for (int j = tid; j < p.max_query_len; j += VF_THREADS) {
            if (j < a) out[j] = p.tokens[q0 + 1 + j];
            else if (j > a || !drawn) out[j] = -1;
        }
        if (tid == 0) p.num_accepted[s] = a;
    }
    if (!drawn) return;
    const bool here = mine > 0. && x >= before && (x < before + mine || before + mine >= W);
    if (!here) return;
    // the run of this block
    double base = before;
    int own = -1, lastw = 0;
    double ob = base;
    for (int w = 0; w < VF_WARPS; ++w) {
        const double b = sh_warp[w];
        if (b > 0.) {
            lastw = w;
            ob = base;
            if (x < base + b) {
                own = w;
                break;
            }
        }
        base += b;
    }
    if (own < 0) own = lastw;
    base = ob;
    // its elements, dealt to the threads in order; a scan finds the thread
    const int64_t lo = run_lo(own), len = run_lo(own + 1) - lo;
    const int64_t per = (len + VF_THREADS - 1) / VF_THREADS;
    const int64_t e0 = lo + min(len, per * tid), e1 = lo + min(len, per * (tid + 1));
    double sum = 0.;
    for (int64_t v = e0; v < e1; ++v) sum += (double)row.at(v);
    double inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) sh_scan[warp] = inc;
    if (tid == 0) {
        sh_first = 0xffffffffu;
        sh_last = 0;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) base += sh_scan[w];
    if (sum > 0.) {
        if (x < base + inc) atomicMin(&sh_first, (unsigned)tid);
        atomicMax(&sh_last, (unsigned)tid);
    }
    __syncthreads();
    const unsigned chosen = sh_first != 0xffffffffu ? sh_first : sh_last;
    if ((unsigned)tid != chosen) return;
    double run = base + (inc - sum);
    int64_t token = -1;
    for (int64_t v = e0; v < e1; ++v) {
        const float w = row.at(v);
        if (w > 0.f) {
            token = v;
            run += (double)w;
            if (x < run) break;
        }
    }
    out[a] = (int32_t)token;
}

template <typename T>
cudaError_t launch_verify(const VerifyParams &p, cudaStream_t st) {
    const int sms = sm_count_of_current_device();
    const int64_t slots = (int64_t)(sms > 0 ? sms : 152) * 2;
    int C = 1;
    while (C < 8 && (int64_t)p.num_seqs * C * 2 <= slots) C *= 2;
    if ((int64_t)p.num_seqs * C > (int64_t)INT32_MAX) return cudaErrorNotSupported;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.num_seqs * C), 1, 1);
    cfg.blockDim = dim3(VF_THREADS, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<T>, p);
}

}  // namespace

cudaError_t verify_drafts(const VerifyParams &p, int dtype, cudaStream_t st) {
    switch (dtype) {
        case 0: return launch_verify<float>(p, st);
        case 1: return launch_verify<__nv_bfloat16>(p, st);
        default: return launch_verify<__half>(p, st);
    }
}

}  // namespace pa
