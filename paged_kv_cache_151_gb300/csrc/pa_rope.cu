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

// One warp per (token, part of its heads); L lanes per head, 32 / L heads at
// a time.  The heads of a token are numbered q, then k, then v.  q may be
// q_out: a head is read and written by the same lanes, reads first.
template <typename T, bool F8, int L>
__global__ void __launch_bounds__(256) rope_and_cache_kernel(const __grid_constant__ RopeParams p) {
    launch_dependents();      // a decode launched next may set up meanwhile
    constexpr int HW = 32 / L;                      // heads of one iteration
    const int lane = threadIdx.x & 31, l = lane % L, sub = lane / L;
    const unsigned item = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const unsigned t = item / (unsigned)p.parts, part = item - t * (unsigned)p.parts;
    if (t >= (unsigned)p.num_tokens) return;
    const int D = p.head_dim, R = p.rot_dim, H = p.num_heads, Hkv = p.num_kv_heads;
    const int h0 = (int)part * p.part_heads, h1 = min(H + 2 * Hkv, h0 + p.part_heads);
    const bool lane_ok = l < D / 16;

    const int64_t slot = p.slot_mapping[t];
    const int64_t pos = R > 0 ? p.positions[t] : 0;
    const bool write = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots && part == 0 && lane == 0) set_error(p.err, ERR_SLOT);
    if (R > 0 && (pos < 0 || pos >= p.num_positions)) {
        // a padding token may have any position; nothing of the token is written
        if (slot >= 0 && part == 0 && lane == 0) set_error(p.err, ERR_POSITION);
        return;
    }

    // this lane's two chunks
    const int RL = R / 16;                          // lanes that rotate
    const bool rot = l < RL;
    int ea, eb;
    if (p.interleaved) {
        ea = 16 * l;
        eb = ea + 8;
    } else if (rot) {
        ea = 8 * l;
        eb = ea + R / 2;
    } else {
        ea = R + 8 * (l - RL);
        eb = ea + (D - R) / 2;
    }
    const float *tr = p.rope_table + pos * R + 8 * l;
    const float inv_d = 1.f / (float)D;

    // heads [lo, hi) of q (or of k): from src on, the result to put(head, a, b)
    auto turn = [&](const T *src, int lo, int hi, const void *weight, auto &&put) {
        if (lo >= hi) return;
        Raw8<T> na = {}, nb = {};
        auto fetch = [&](int h) {
            if (lane_ok && h < hi) {
                na = load_raw8<T>(src + (int64_t)h * D + ea);
                nb = load_raw8<T>(src + (int64_t)h * D + eb);
            }
        };
        fetch(lo + sub);
        Factors f;
        load_factors<T>(f, weight, tr, R / 2, rot, lane_ok, p.interleaved, ea, eb);
        for (int hb = lo; hb < hi; hb += HW) {
            const int h = hb + sub;
            float a[8], b[8];
            widen8<T>(na, a);
            widen8<T>(nb, b);
            fetch(h + HW);
            float g = 1.f;
            if (weight) {                           // the sum needs every lane of the warp
                float2 ss = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 x = make_float2(a[e], a[e + 1]), y = make_float2(b[e], b[e + 1]);
                    ss = fma2(x, x, fma2(y, y, ss));
                }
                float sum = lane_ok ? ss.x + ss.y : 0.f;
#pragma unroll
                for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                g = rsqrtf(sum * inv_d + p.eps);
            }
            float ra[8], rb[8];
            if (!rot) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ra[e] = a[e] * f.A1[e] * g;
                    rb[e] = b[e] * f.B1[e] * g;
                }
            } else if (p.interleaved) {
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
            if (lane_ok && h < hi) put(h, ra, rb);
        }
    };

    T *qo = reinterpret_cast<T *>(p.q_out) + (int64_t)t * p.q_out_stride;
    turn(reinterpret_cast<const T *>(p.q) + (int64_t)t * p.q_stride, h0, min(h1, H), p.q_weight,
         [&](int h, const float *a, const float *b) {
             store_raw8<T>(qo + (int64_t)h * D + ea, narrow8<T>(a));
             store_raw8<T>(qo + (int64_t)h * D + eb, narrow8<T>(b));
         });
    if (!write) return;

    // a row of KV head j of this token (block_size 16); chunk ea of it
    auto cache_at = [&](int j) { return (((slot >> 4) * Hkv + j) * 16 + (slot & 15)) * D; };
    auto recip = [&](float sc) { return sc > 0x1p-100f && sc < 0x1p100f ? 1.f / sc : 0.f; };
    turn(reinterpret_cast<const T *>(p.k) + (int64_t)t * p.k_stride, max(h0 - H, 0),
         min(h1 - H, Hkv), p.k_weight, [&](int j, const float *a, const float *b) {
             if constexpr (F8) {
                 const float sc = __ldg(p.k_scale + j), r = recip(sc);
                 unsigned char *dst = static_cast<unsigned char *>(p.k_cache) + cache_at(j);
                 *reinterpret_cast<uint2 *>(dst + ea) = e4m3_of8(a, sc, r);
                 *reinterpret_cast<uint2 *>(dst + eb) = e4m3_of8(b, sc, r);
             } else {
                 T *dst = static_cast<T *>(p.k_cache) + cache_at(j);
                 store_raw8<T>(dst + ea, narrow8<T>(a));
                 store_raw8<T>(dst + eb, narrow8<T>(b));
             }
         });
    // v: as it is (16-byte chunks l and D/16 + l of the head's 8-element ones)
    const T *v = reinterpret_cast<const T *>(p.v) + (int64_t)t * p.v_stride;
    const int va = 8 * l, vb = D / 2 + 8 * l;
    for (int j = max(h0 - H - Hkv, 0) + sub; j < h1 - H - Hkv; j += HW) {
        if (!lane_ok) continue;
        const Raw8<T> ra = load_raw8<T>(v + (int64_t)j * D + va);
        const Raw8<T> rb = load_raw8<T>(v + (int64_t)j * D + vb);
        if constexpr (F8) {
            const float sc = __ldg(p.v_scale + j), r = recip(sc);
            unsigned char *dst = static_cast<unsigned char *>(p.v_cache) + cache_at(j);
            float a[8], b[8];
            widen8<T>(ra, a);
            widen8<T>(rb, b);
            *reinterpret_cast<uint2 *>(dst + va) = e4m3_of8(a, sc, r);
            *reinterpret_cast<uint2 *>(dst + vb) = e4m3_of8(b, sc, r);
        } else {
            T *dst = static_cast<T *>(p.v_cache) + cache_at(j);
            store_raw8<T>(dst + va, ra);
            store_raw8<T>(dst + vb, rb);
        }
    }
}

template <typename T, bool F8, int L>
cudaError_t launch_rope(RopeParams p, cudaStream_t st) {
    constexpr int HW = 32 / L;
    const int rows = p.num_heads + 2 * p.num_kv_heads;
    const int most = (rows + HW - 1) / HW;          // parts of one iteration each
    const int sms = sm_count_of_current_device();
    const int64_t want = (int64_t)(sms > 0 ? sms : 152) * 32;
    int64_t parts = (want + p.num_tokens - 1) / p.num_tokens;
    if (parts > most) parts = most;
    const int iters = (int)((most + parts - 1) / parts);
    p.part_heads = iters * HW;
    p.parts = (rows + p.part_heads - 1) / p.part_heads;
    const int64_t items = p.num_tokens * p.parts;
    if (items > (int64_t)INT32_MAX) return cudaErrorNotSupported;
    const int threads = 256;
    const int64_t blocks = (items * 32 + threads - 1) / threads;
    prefer_shared_carveout<rope_and_cache_kernel<T, F8, L>>();
    rope_and_cache_kernel<T, F8, L><<<(unsigned)blocks, threads, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T, bool F8>
cudaError_t dispatch_lanes(const RopeParams &p, cudaStream_t st) {
    if (p.head_dim <= 64) return launch_rope<T, F8, 4>(p, st);
    if (p.head_dim <= 128) return launch_rope<T, F8, 8>(p, st);
    return launch_rope<T, F8, 16>(p, st);
}

template <typename T>
cudaError_t dispatch_cache(const RopeParams &p, cudaStream_t st) {
    return p.k_scale ? dispatch_lanes<T, true>(p, st) : dispatch_lanes<T, false>(p, st);
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
