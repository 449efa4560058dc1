// pa_rope.cu -- the cache write with what comes right before it in the
// attention layer: per-head norms of the new queries and keys and the
// rotation by their positions, in one pass over q, k and v.
//
// For a head x of D elements (q or k) of a token at position p:
//   y = x / sqrt(mean(x^2) + eps) * w           (only with a weight row w)
//   (a, b) -> (a cos - b sin, b cos + a sin)    for the R/2 pairs of the first
//       R elements: (i, i + R/2), or (2i, 2i + 1) when interleaved; cos and
//       sin of pair i at columns i and R/2 + i of row p of the table;
// q goes to q_out, k to its cache slot, v to its slot as it is.  Everything
// between the load and the one rounding of the stored value is fp32: the sum
// of squares of at most 256 elements loses less than the 2^-9 (bf16) of the
// result's own rounding.  E4M3 caches store E4M3(x / scale) as the plain cache
// write does (quotient rounded to binary32, then to E4M3).
//
// Bound by HBM: each element is read once and written once (about 9 flop per
// element).  A lane holds two 8-element chunks whose elements are each
// other's partners in the rotation (chunk l of the first half and chunk l of
// the second, or two neighbouring chunks when interleaved), so the rotation
// needs no exchange between lanes and every access is 16 bytes; the D/16
// lanes of a head add up its squares with shuffles.  The same lane keeps the
// same pairs for every head of a token, so a warp folds weights, cos and sin
// into four factors a pair once and runs over several heads with them, the
// next heads' loads in flight.
//
// Measured: 32768 tokens (32 + 8 + 8 heads of 128, norms, E4M3 cache; 755 MB) 150 us =
// 5.0 TB/s, 0.75 of the measured copy rate; 1024 tokens 10.3 us and one token
// 4.1 us on the device, where a warp's chain of slot and position, table and data
// loads counts.  The launch cuts a call for 32 warps an SM and 20 fit: 1024
// tokens are 4096 warps of three iterations, 1.35 waves of 3040, and 4099 tokens
// of 16 + 4 + 4 heads of 64 are 8198 of two, 2.70 waves (10.3 us as well), so the
// chain is paid more than once.
#include <type_traits>

#include "pa_common.cuh"
#include "pa_fp8.cuh"
#include "pa_internal.h"
#include "pa_mma.cuh"

namespace pa {

namespace {

template <typename T> struct Raw8 {                 // eight elements as loaded
    uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T *src) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4 *>(src)[i];
    return r;
}

template <typename T>
__device__ __forceinline__ void store_raw8(T *dst, const Raw8<T> &r) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(dst)[i] = r.w[i];
}

template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T> &r, float *x) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) Elem<T>::to_f32(r.w[i], x + i * (16 / (int)sizeof(T)));
}

template <typename T>
__device__ __forceinline__ Raw8<T> narrow8(const float *x) {
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
        r.w[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                            __float_as_uint(x[3]));
        r.w[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]),
                            __float_as_uint(x[7]));
    } else {
        r.w[0] = make_uint4(Mma<T>::pack(x[0], x[1]), Mma<T>::pack(x[2], x[3]),
                            Mma<T>::pack(x[4], x[5]), Mma<T>::pack(x[6], x[7]));
    }
    return r;
}

// The codes of x[0..7] / scale as the plain cache write stores them.  x times
// the reciprocal r is within 2^-22.4 of the quotient, so where it gives the
// same code from 2^-21 below and above, that is the quotient's code (rounding
// is monotonic); the rest -- about one element in 2^17 -- is divided.
// r == 0: always divide.
__device__ __forceinline__ uint2 e4m3_of8(const float *x, float scale, float r) {
    uint32_t lo[2], hi[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float2 a = mul2(make_float2(x[4 * h], x[4 * h + 1]), make_float2(r, r));
        const float2 b = mul2(make_float2(x[4 * h + 2], x[4 * h + 3]), make_float2(r, r));
        constexpr float DN = 1.f - 0x1p-21f, UP = 1.f + 0x1p-21f;
        const float2 al = mul2(a, make_float2(DN, DN)), ah = mul2(a, make_float2(UP, UP));
        const float2 bl = mul2(b, make_float2(DN, DN)), bh = mul2(b, make_float2(UP, UP));
        lo[h] = e4m3x2_from_f32(al.x, al.y) | (e4m3x2_from_f32(bl.x, bl.y) << 16);
        hi[h] = e4m3x2_from_f32(ah.x, ah.y) | (e4m3x2_from_f32(bh.x, bh.y) << 16);
    }
    if (lo[0] != hi[0] || lo[1] != hi[1] || r == 0.f) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            lo[h] = e4m3x2_from_f32(__fdiv_rn(x[4 * h], scale), __fdiv_rn(x[4 * h + 1], scale)) |
                    (e4m3x2_from_f32(__fdiv_rn(x[4 * h + 2], scale), __fdiv_rn(x[4 * h + 3], scale)) << 16);
    }
    return make_uint2(lo[0], lo[1]);
}

// A lane's two chunks of a head, and the factors of their pairs: with weights w
// (1 without a norm) a' = f (a A1 - b A2), b' = f (b B1 + a B2), A1 = w_a cos,
// A2 = w_b sin, B1 = w_b cos, B2 = w_a sin; a lane past the rotation only has
// w_a = A1 and w_b = B1 (a product with 0 would spread infinities).  In the
// interleaved layout the pairs are neighbours and factor e belongs to element
// e: the partner of x[2i] is x[2i + 1].
struct Factors {
    float A1[8], A2[8], B1[8], B2[8];
};

template <typename T>
__device__ __forceinline__ void load_factors(Factors &f, const void *weight, const float *tr,
                                             int half, bool rot, bool live, bool interleaved, int ea,
                                             int eb) {
    float wa[8], wb[8], cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) wa[e] = wb[e] = 1.f;
    if (weight && live) {
        const T *w = reinterpret_cast<const T *>(weight);
        widen8<T>(load_raw8<T>(w + ea), wa);
        widen8<T>(load_raw8<T>(w + eb), wb);
    }
    if (!rot) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f.A1[e] = wa[e];
            f.B1[e] = wb[e];
            f.A2[e] = f.B2[e] = 0.f;
        }
        return;
    }
    Elem<float>::to_f32(__ldg(reinterpret_cast<const uint4 *>(tr)), cs);
    Elem<float>::to_f32(__ldg(reinterpret_cast<const uint4 *>(tr) + 1), cs + 4);
    Elem<float>::to_f32(__ldg(reinterpret_cast<const uint4 *>(tr + half)), sn);
    Elem<float>::to_f32(__ldg(reinterpret_cast<const uint4 *>(tr + half) + 1), sn + 4);
    if (interleaved) {
        // pair i of this lane: elements 2i, 2i + 1 of (a, b) taken as one run of 16
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = e >> 1;
            f.A1[e] = wa[e] * cs[i];
            f.A2[e] = wa[e ^ 1] * sn[i];
            f.B1[e] = wb[e] * cs[4 + i];
            f.B2[e] = wb[e ^ 1] * sn[4 + i];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f.A1[e] = wa[e] * cs[e];
            f.A2[e] = wb[e] * sn[e];
            f.B1[e] = wb[e] * cs[e];
            f.B2[e] = wa[e] * sn[e];
        }
    }
}

// Five blocks of four warps per SM, two iterations in flight (32768 tokens of
// 32 + 8 + 8 heads of 128 into E4M3): 148 us; one iteration 170, four blocks 157, six
// (which spill) 213.
constexpr int ROPE_THREADS = 128, ROPE_BLOCKS = 5, ROPE_AHEAD = 2;

// One warp per (token, part of its heads); L lanes per head, HW = 32 / L heads
// an iteration, of one kind: ceil(H / HW) iterations of q, then of k, then of v.
// Loads run AHEAD iterations ahead, across the kinds.  q may be q_out: a head is
// read and written by the same lanes, reads first.
template <typename T, bool F8, bool INTER, int L>
__global__ void __launch_bounds__(ROPE_THREADS, ROPE_BLOCKS) rope_and_cache_kernel(const __grid_constant__ RopeParams p) {
    // Without queries this is a cache write like the others: a decode launched
    // next may set up meanwhile.  With queries it may not: the decodes read q
    // through the non-coherent path, which must not see it being written.
    if (p.num_heads == 0) launch_dependents();
    constexpr int HW = 32 / L;
    constexpr int AHEAD = ROPE_AHEAD;
    const int lane = threadIdx.x & 31, l = lane % L, sub = lane / L;
    const unsigned item = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const unsigned t = item / (unsigned)p.parts, part = item - t * (unsigned)p.parts;
    if (t >= (unsigned)p.num_tokens) return;
    const int D = p.head_dim, R = p.rot_dim, H = p.num_heads, Hkv = p.num_kv_heads;
    const int nq = (H + HW - 1) / HW, nk = (Hkv + HW - 1) / HW;
    const int it0 = (int)part * p.part_iters;
    int it1 = min(nq + 2 * nk, it0 + p.part_iters);
    const bool lane_ok = l < D / 16;

    const int64_t slot = p.slot_mapping[t];
    const int64_t pos = R > 0 ? p.positions[t] : 0;

    // this lane's two chunks (of v: any two do)
    const int RL = R / 16;                          // lanes that rotate
    const bool rot = l < RL;
    int ea, eb;
    if (INTER) {
        ea = 16 * l;
        eb = ea + 8;
    } else if (rot) {
        ea = 8 * l;
        eb = ea + R / 2;
    } else {
        ea = R + 8 * (l - RL);
        eb = ea + (D - R) / 2;
    }
    const T *q = reinterpret_cast<const T *>(p.q) + (int64_t)t * p.q_stride;
    const T *k = reinterpret_cast<const T *>(p.k) + (int64_t)t * p.k_stride;
    const T *v = reinterpret_cast<const T *>(p.v) + (int64_t)t * p.v_stride;
    Raw8<T> na[AHEAD] = {}, nb[AHEAD] = {};
    auto fetch = [&](int it, Raw8<T> &xa, Raw8<T> &xb) {
        const bool is_q = it < nq, is_k = !is_q && it < nq + nk;
        const int h = (it - (is_q ? 0 : is_k ? nq : nq + nk)) * HW + sub;
        const T *src = (is_q ? q : is_k ? k : v) + h * D;
        if (lane_ok && it < it1 && h < (is_q ? H : Hkv)) {
            xa = load_raw8<T>(src + ea);
            xb = load_raw8<T>(src + eb);
        }
    };
    // k and v of a padding token are not looked at, so its loads wait for the slot
    if (slot < 0 || slot >= p.num_slots) it1 = min(it1, nq);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(it0 + i, na[i], nb[i]);

    if (slot >= p.num_slots && part == 0 && lane == 0) set_error(p.err, ERR_SLOT);
    if (R > 0 && (pos < 0 || pos >= p.num_positions)) {
        // a padding token may have any position; nothing of the token is written
        if (slot >= 0 && part == 0 && lane == 0) set_error(p.err, ERR_POSITION);
        return;
    }
    const float *tr = p.rope_table + pos * R + 8 * l;
    const float inv_d = 1.f / (float)D;
    T *qo = reinterpret_cast<T *>(p.q_out) + (int64_t)t * p.q_out_stride;
    const int64_t row0 = ((slot >> 4) * Hkv * 16 + (slot & 15)) * D;   // KV head 0's row (block_size 16)
    Factors f;

    auto body = [&](int it, Raw8<T> &xa, Raw8<T> &xb) {
        const bool is_q = it < nq, is_v = it >= nq + nk;
        const int h = (it - (is_q ? 0 : is_v ? nq + nk : nq)) * HW + sub;
        const bool live = lane_ok && h < (is_q ? H : Hkv);
        const int64_t at = row0 + (int64_t)h * 16 * D;
        if (is_v && !F8) {                          // bit for bit
            const Raw8<T> ya = xa, yb = xb;
            fetch(it + AHEAD, xa, xb);
            if (live) {
                store_raw8<T>(static_cast<T *>(p.v_cache) + at + ea, ya);
                store_raw8<T>(static_cast<T *>(p.v_cache) + at + eb, yb);
            }
            return;
        }
        const void *weight = is_q ? p.q_weight : p.k_weight;
        if (!is_v && (it == it0 || it == nq))
            load_factors<T>(f, weight, tr, R / 2, rot, lane_ok, INTER, ea, eb);
        float a[8], b[8];
        widen8<T>(xa, a);
        widen8<T>(xb, b);
        fetch(it + AHEAD, xa, xb);
        float ra[8], rb[8];
        if (is_v) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ra[e] = a[e];
                rb[e] = b[e];
            }
        } else {
            float g = 1.f;
            if (weight) {                           // the sum needs every lane of the warp
                float2 ss = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 x = make_float2(a[e], a[e + 1]), y = make_float2(b[e], b[e + 1]);
                    ss = fma2(x, x, fma2(y, y, ss));
                }
                float sum = live ? ss.x + ss.y : 0.f;
#pragma unroll
                for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                g = rsqrtf(sum * inv_d + p.eps);
            }
            if (!rot) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ra[e] = a[e] * f.A1[e] * g;
                    rb[e] = b[e] * f.B1[e] * g;
                }
            } else if (INTER) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    ra[e] = (a[e] * f.A1[e] - a[e + 1] * f.A2[e]) * g;
                    ra[e + 1] = (a[e + 1] * f.A1[e + 1] + a[e] * f.A2[e + 1]) * g;
                    rb[e] = (b[e] * f.B1[e] - b[e + 1] * f.B2[e]) * g;
                    rb[e + 1] = (b[e + 1] * f.B1[e + 1] + b[e] * f.B2[e + 1]) * g;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ra[e] = (a[e] * f.A1[e] - b[e] * f.A2[e]) * g;
                    rb[e] = (b[e] * f.B1[e] + a[e] * f.B2[e]) * g;
                }
            }
        }
        if (!live) return;
        if (F8 && !is_q) {
            const float sc = __ldg((is_v ? p.v_scale : p.k_scale) + h);
            const float r = sc > 0x1p-100f && sc < 0x1p100f ? 1.f / sc : 0.f;
            unsigned char *dst = static_cast<unsigned char *>(is_v ? p.v_cache : p.k_cache) + at;
            *reinterpret_cast<uint2 *>(dst + ea) = e4m3_of8(ra, sc, r);
            *reinterpret_cast<uint2 *>(dst + eb) = e4m3_of8(rb, sc, r);
        } else {
            T *dst = is_q ? qo + h * D : static_cast<T *>(p.k_cache) + at;
            store_raw8<T>(dst + ea, narrow8<T>(ra));
            store_raw8<T>(dst + eb, narrow8<T>(rb));
        }
    };
    for (int it = it0; it < it1; it += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (it + i < it1) body(it + i, na[i], nb[i]);
    }
}

template <typename T, bool F8, bool INTER, int L>
cudaError_t launch_rope(RopeParams p, cudaStream_t st) {
    constexpr int HW = 32 / L;
    const int iters = (p.num_heads + HW - 1) / HW + 2 * ((p.num_kv_heads + HW - 1) / HW);
    const int sms = sm_count_of_current_device();
    const int64_t want = (int64_t)(sms > 0 ? sms : 152) * 32;
    int64_t parts = (want + p.num_tokens - 1) / p.num_tokens;
    if (parts > iters) parts = iters;
    p.part_iters = (int)((iters + parts - 1) / parts);
    p.parts = (iters + p.part_iters - 1) / p.part_iters;
    const int64_t items = p.num_tokens * p.parts;
    if (items > (int64_t)INT32_MAX) return cudaErrorNotSupported;
    const int64_t blocks = (items * 32 + ROPE_THREADS - 1) / ROPE_THREADS;
    prefer_shared_carveout<rope_and_cache_kernel<T, F8, INTER, L>>();
    rope_and_cache_kernel<T, F8, INTER, L><<<(unsigned)blocks, ROPE_THREADS, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T, bool F8, bool INTER>
cudaError_t dispatch_lanes(const RopeParams &p, cudaStream_t st) {
    if (p.head_dim <= 64) return launch_rope<T, F8, INTER, 4>(p, st);
    if (p.head_dim <= 128) return launch_rope<T, F8, INTER, 8>(p, st);
    return launch_rope<T, F8, INTER, 16>(p, st);
}

template <typename T>
cudaError_t dispatch_cache(const RopeParams &p, cudaStream_t st) {
    if (p.interleaved)
        return p.k_scale ? dispatch_lanes<T, true, true>(p, st) : dispatch_lanes<T, false, true>(p, st);
    return p.k_scale ? dispatch_lanes<T, true, false>(p, st) : dispatch_lanes<T, false, false>(p, st);
}

}  // namespace

cudaError_t rope_and_cache(const RopeParams &p, int dtype, cudaStream_t st) {
    switch (dtype) {
        case 0: return dispatch_cache<float>(p, st);
        case 1: return dispatch_cache<__nv_bfloat16>(p, st);
        default: return dispatch_cache<__half>(p, st);
    }
}

}  // namespace pa
