// pa_verify.cu -- verification of drafted tokens: the accept test of every
// draft of a sequence and the token drawn after the accepted ones.
//
// With target row p_i and draft row q_i behind draft x_i and a uniform u_i,
// drafts are accepted in order while u_i q_i(x_i) < p_i(x_i).  At the first
// rejection the next token comes from w = max(p_i - q_i, 0), and when all are
// accepted from w = p of the row behind the last one: the first v whose
// cumulative weight C_v exceeds u W (W the row's sum).  The vocabulary's
// cumulative sums decide a whole number, and a row has 10^4 to 10^5 borders that
// u W can fall next to, so every sum is a pair of floats (the rounding error of
// every addition is kept and added up beside it: about 46 bits), as Knuth's
// two-sum gives it without a comparison.  Binary64 would be simpler and
// costs more than the row's traffic: a batch of 64 over 131071 tokens spent
// 5 of its 19 us in the 16 binary64 steps that one warp took.
//
// Bound by HBM for batches (one or two rows of the vocabulary per sequence),
// by latency for one sequence.  A cluster of C blocks takes one sequence: the
// row is cut into C * 16 runs, one per warp, each summed in one pass; the
// block sums meet through distributed shared memory (after a first cluster
// barrier, whose wait the sums hide: no peer is written to before it is known to
// run), and only the run that holds the border is read again, by the whole block
// that owns it.  One launch, no workspace, no atomics on global memory, a fixed
// order of additions.
//
// Measured, calls of a captured graph: one sequence over 32000 tokens 5.7 us (rows,
// tokens and uniforms 1 us, the sums 1.5, the cluster's exchange 1.2, the border
// and its run 2); 64 sequences over 131071 tokens in fp32 (53 MB) 17.2 us, 8 to 10
// of them streaming; 256 over 50021 in bf16 without draft probabilities (26 MB)
// 14.6 us, read two bytes a lane (rows of an odd stride start anywhere), eight
// loads in flight: some twelve round trips to memory in a row.
#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int VF_THREADS = 512;
constexpr int VF_WARPS = VF_THREADS / 32;
constexpr int VF_MAX_CLUSTER = 8;

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

// A sum as hi + lo: the rounding error of every addition to hi goes to lo.
struct Pair {
    float hi, lo;
    __device__ __forceinline__ void add(float x) {
        const float s = hi + x, z = s - hi;
        lo += (hi - (s - z)) + (x - z);
        hi = s;
    }
    __device__ __forceinline__ void add(const Pair &o) {
        add(o.hi);
        lo += o.lo;
    }
    // *this > o, by the difference (its first part is exact where it matters)
    __device__ __forceinline__ bool above(const Pair &o) const { return (hi - o.hi) + (lo - o.lo) > 0.f; }
};

__device__ __forceinline__ Pair shfl(const Pair &a, int src) {
    return Pair{__shfl_sync(0xffffffffu, a.hi, src), __shfl_sync(0xffffffffu, a.lo, src)};
}
__device__ __forceinline__ Pair shfl_xor(const Pair &a, int o) {
    return Pair{__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
}
// Inclusive sums over the first W lanes; *before: the lanes below this one.
template <int W>
__device__ __forceinline__ Pair scan(const Pair &a, int lane, Pair *before) {
    Pair inc = a;
#pragma unroll
    for (int o = 1; o < W; o <<= 1) {
        const Pair y{__shfl_up_sync(0xffffffffu, inc.hi, o), __shfl_up_sync(0xffffffffu, inc.lo, o)};
        if (lane >= o) inc.add(y);
    }
    *before = Pair{__shfl_up_sync(0xffffffffu, inc.hi, 1), __shfl_up_sync(0xffffffffu, inc.lo, 1)};
    if (lane == 0) *before = Pair{0.f, 0.f};
    return inc;
}

// u q < p for u, p, q >= 0, exactly: the product's rounding error is one fma
// away where it does not underflow.  It is a multiple of the factors' last bits,
// 2^-73 each above 2^-50, and those of 2^-149 are binary32 numbers.
__device__ __forceinline__ bool product_below(float u, float q, float p) {
    if (u > 0x1p-50f && q > 0x1p-50f) {
        const float h = u * q, e = fmaf(u, q, -h);
        return h < p || (h == p && e < 0.f);
    }
    return (double)u * (double)q < (double)p;
}

// Two Pairs in the packed arithmetic: x - y as fma(y, -1, x), rounded once.
struct Pair2 {
    float2 hi, lo;
    __device__ __forceinline__ static float2 sub(float2 x, float2 y) {
        return fma2(y, make_float2(-1.f, -1.f), x);
    }
    __device__ __forceinline__ void add(float2 x) {
        const float2 s = add2(hi, x), z = sub(s, hi);
        lo = add2(lo, add2(sub(hi, sub(s, z)), sub(x, z)));
        hi = s;
    }
    __device__ __forceinline__ Pair sum() const {
        Pair r{hi.x, lo.x};
        r.add(Pair{hi.y, lo.y});
        return r;
    }
};

// This lane's part of the weights of n elements: lane + 32 i, 2 U of them in
// flight.  Element `hole` (one row only) is left out.  Infinite entries are not
// dropped here: they make the sum infinite or NaN, which the caller looks for.
template <typename T, bool TWO, int U>
__device__ __forceinline__ Pair sum_run(const T *p, const T *q, int n, int hole, int lane) {
    Pair2 acc{make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    constexpr int STEP = 64 * U;
    p += lane;
    q += lane;
    n -= lane;
    hole -= lane;
    auto step = [&](int at, auto &&in) {
        T x[2 * U];
        [[maybe_unused]] T y[2 * U];
#pragma unroll
        for (int e = 0; e < 2 * U; ++e) {
            x[e] = in(at + 32 * e) ? p[at + 32 * e] : T(0.f);
            if constexpr (TWO) y[e] = in(at + 32 * e) ? q[at + 32 * e] : T(0.f);
        }
#pragma unroll
        for (int e = 0; e < 2 * U; e += 2) {
            float2 w = make_float2((float)x[e], (float)x[e + 1]);
            if constexpr (TWO)
                w = Pair2::sub(w, make_float2(fmaxf((float)y[e], 0.f), fmaxf((float)y[e + 1], 0.f)));
            w = make_float2(fmaxf(w.x, 0.f), fmaxf(w.y, 0.f));
            if constexpr (!TWO) {
                w.x = at + 32 * e == hole ? 0.f : w.x;
                w.y = at + 32 * e + 32 == hole ? 0.f : w.y;
            }
            acc.add(w);
        }
    };
    int at = 0;
    for (; at + STEP - 32 < n; at += STEP) step(at, [](int) { return true; });
    if (at < n) step(at, [&](int i) { return i < n; });
    return acc.sum();
}

// The same with every check, one element at a time: a run with an infinite
// entry.
template <typename T>
__device__ __forceinline__ Pair sum_run_checked(const Row<T> &row, int64_t lo, int64_t hi, int lane) {
    Pair acc{0.f, 0.f};
    for (int64_t v = lo + lane; v < hi; v += 32) acc.add(row.at(v));
    return acc;
}

__device__ __forceinline__ void st_dsmem(uint32_t addr, const Pair &v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" :: "r"(addr), "f"(v.hi), "f"(v.lo) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(VF_THREADS, 2) verify_drafts_kernel(const __grid_constant__ VerifyParams p) {
    __shared__ int sh_acc, sh_reject;               // accepted drafts; whether one was rejected
    __shared__ Pair sh_warp[VF_WARPS];              // sums of the warps' runs
    __shared__ Pair sh_blocks[2][VF_MAX_CLUSTER];   // of the cluster's blocks, a pass each
    __shared__ int sh_own;                          // run that holds the border, -1: another block's,
                                                    // -2: nothing to draw from
    __shared__ Pair sh_goal;                        // the border from the run's start
    __shared__ Pair sh_scan[VF_WARPS];
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
    if (C > 1) cluster_arrive();                    // this block runs (see cluster_wait below)
    const float us = p.sample_u[s];
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
                const float u = p.accept_u[r];
                ok = false;
                if (x >= 0 && x < V) {
                    const float pt = weight_of(Elem<T>::load1(target + (r - 1) * p.target_stride + x), 0.f);
                    const float qt = draft ? fmaxf(Elem<T>::load1(draft + r * p.draft_stride + x), 0.f) : 1.f;
                    ok = product_below(u, qt, pt);
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
            sh_first = 0xffffffffu;
            sh_last = 0;
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
    if (rank == 0) {
        for (int j = tid; j < p.max_query_len; j += VF_THREADS)
            if (j != a) out[j] = j < a ? p.tokens[q0 + 1 + j] : -1;
        if (tid == 0) p.num_accepted[s] = a;
    }

    int own = -2;
    for (int pass = 0; pass < 2; ++pass) {
        // ---- sums of the runs, and of the blocks
        const int64_t lo = run_lo(warp), hi = run_lo(warp + 1);
        const int len = (int)(hi - lo);
        const int hole = row.hole >= lo && row.hole < hi ? (int)(row.hole - lo) : -1;
        Pair sum = row.q ? sum_run<T, true, 4>(row.p + lo, row.q + lo, len, -1, lane)
                         : sum_run<T, false, 4>(row.p + lo, row.p + lo, len, hole, lane);
        if (__any_sync(0xffffffffu, !(sum.hi < INFINITY && sum.lo < INFINITY)))
            sum = sum_run_checked(row, lo, hi, lane);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum.add(shfl_xor(sum, o));
        if (lane == 0) sh_warp[warp] = sum;
        __syncthreads();
        // a peer's shared memory may be written once that block is known to run
        if (pass == 0 && C > 1) cluster_wait();
        Pair mine{0.f, 0.f}, upto, below;           // lane w of warp 0: run w's sum, up to it, below it
        if (warp == 0) {
            if (lane < VF_WARPS) mine = sh_warp[lane];
            upto = scan<VF_WARPS>(mine, lane, &below);
            const Pair block = shfl(upto, VF_WARPS - 1);
            if (lane < C) st_dsmem(map_to_rank(&sh_blocks[pass][rank], (uint32_t)lane), block);
            __syncwarp();                           // the barrier below is one of whole warps
        }
        cluster_sync();
        // ---- the border u W: the first block whose sums reach past it (or the
        // last with any weight), and the run
        if (warp == 0) {
            const Pair b = lane < C ? sh_blocks[pass][lane] : Pair{0.f, 0.f};
            Pair before;
            const Pair sums = scan<VF_MAX_CLUSTER>(b, lane, &before);      // blocks 0 .. lane
            const Pair W = shfl(sums, VF_MAX_CLUSTER - 1);
            const float u = us > 0.f ? fminf(us, 1.f) : 0.f;
            // u = 1 takes the last weight, however far below the sums' last bit it
            // is: no sum is past the border then, at any level
            const bool last = u == 1.f;
            Pair x;                                 // u W
            x.hi = u * W.hi;
            x.lo = fmaf(u, W.hi, -x.hi) + u * W.lo;
            const unsigned past = __ballot_sync(0xffffffffu, lane < C && b.hi > 0.f && !last && sums.above(x));
            const unsigned any = __ballot_sync(0xffffffffu, lane < C && b.hi > 0.f);
            int o = -2;
            if (any && W.hi < INFINITY && W.lo < INFINITY) {
                const int blk = past ? __ffs(past) - 1 : 31 - __clz(any);
                o = -1;
                if (blk == rank) {
                    const Pair base = shfl(before, blk);
                    x.add(Pair{-base.hi, -base.lo});               // from the block's start
                    const unsigned rp = __ballot_sync(0xffffffffu, mine.hi > 0.f && !last && upto.above(x));
                    const unsigned ra = __ballot_sync(0xffffffffu, mine.hi > 0.f);
                    o = rp ? __ffs(rp) - 1 : 31 - __clz(ra);
                    const Pair run = shfl(below, o);
                    x.add(Pair{-run.hi, -run.lo});                 // from the run's start
                    if (lane == 0) sh_goal = last ? Pair{INFINITY, 0.f} : x;
                }
            }
            if (lane == 0) sh_own = o;
        }
        __syncthreads();
        own = sh_own;
        // nothing left of max(p - q, 0): the target's own row; every block
        // sees the same sums
        if (own != -2 || (!row.q && row.hole < 0)) break;
        row.q = nullptr;
        row.hole = -1;
    }
    if (own == -2 && rank == 0 && tid == 0) out[a] = -1;
    if (own < 0) return;

    // ---- the run's elements, dealt to the threads in order; a scan finds the
    // thread, and it the element
    const Pair goal = sh_goal;
    const int64_t lo = run_lo(own), len = run_lo(own + 1) - lo;
    const int64_t per = (len + VF_THREADS - 1) / VF_THREADS;
    const int64_t e0 = lo + min(len, per * tid), e1 = lo + min(len, per * (tid + 1));
    Pair sum{0.f, 0.f};
    for (int64_t v = e0; v < e1; ++v) sum.add(row.at(v));
    Pair before;                                    // the warp's lanes below this one
    const Pair inc = scan<32>(sum, lane, &before);
    if (lane == 31) sh_scan[warp] = inc;
    __syncthreads();
    Pair base{0.f, 0.f};
    for (int w = 0; w < warp; ++w) base.add(sh_scan[w]);
    Pair end = base;
    end.add(inc);
    if (sum.hi > 0.f) {
        if (end.above(goal)) atomicMin(&sh_first, (unsigned)tid);
        atomicMax(&sh_last, (unsigned)tid);
    }
    __syncthreads();
    const unsigned chosen = sh_first != 0xffffffffu ? sh_first : sh_last;
    if ((unsigned)tid != chosen) return;
    Pair run = base;                                // up to this thread's elements
    run.add(before);
    int64_t token = -1;
    for (int64_t v = e0; v < e1; ++v) {
        const float w = row.at(v);
        if (w > 0.f) {
            token = v;
            run.add(w);
            if (run.above(goal)) break;
        }
    }
    out[a] = (int32_t)token;
}

template <typename T>
cudaError_t launch_verify(const VerifyParams &p, cudaStream_t st) {
    const int sms = sm_count_of_current_device();
    // two blocks per SM fit; more would queue behind each other's chains of loads
    // (64 sequences of 131071 tokens: 18.5 us a call at 4 blocks each, 22.5 at 8)
    const int64_t slots = (int64_t)(sms > 0 ? sms : 152) * 2;
    int C = 1;
    while (C < VF_MAX_CLUSTER && (int64_t)p.num_seqs * C * 2 <= slots) C *= 2;
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
