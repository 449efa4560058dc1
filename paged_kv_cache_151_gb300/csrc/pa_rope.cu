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
// same pairs for every head of a token, so a warp loads its cos and sin once
// and runs over several heads with them.
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

__device__ __forceinline__ uint2 e4m3_of8(const float *x, float scale) {
    uint2 r;
    r.x = e4m3x2_from_f32(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale)) |
          (e4m3x2_from_f32(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale)) << 16);
    r.y = e4m3x2_from_f32(__fdiv_rn(x[4], scale), __fdiv_rn(x[5], scale)) |
          (e4m3x2_from_f32(__fdiv_rn(x[6], scale), __fdiv_rn(x[7], scale)) << 16);
    return r;
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
    const int rows = H + 2 * Hkv;
    const int h0 = (int)part * p.part_heads, h1 = min(rows, h0 + p.part_heads);
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

    // this lane's two chunks, and the cos and sin of their pairs
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
    float cs[8], sn[8];
    if (rot) {
        const float *tr = p.rope_table + pos * R + 8 * l;
        Elem<float>::to_f32(__ldg(reinterpret_cast<const uint4 *>(tr)), cs);
        Elem<float>::to_f32(__ldg(reinterpret_cast<const uint4 *>(tr) + 1), cs + 4);
        tr += R / 2;
        Elem<float>::to_f32(__ldg(reinterpret_cast<const uint4 *>(tr)), sn);
        Elem<float>::to_f32(__ldg(reinterpret_cast<const uint4 *>(tr) + 1), sn + 4);
    }
    const T *q = reinterpret_cast<const T *>(p.q) + (int64_t)t * p.q_stride;
    const T *k = reinterpret_cast<const T *>(p.k) + (int64_t)t * p.k_stride;
    const T *v = reinterpret_cast<const T *>(p.v) + (int64_t)t * p.v_stride;
    T *qo = reinterpret_cast<T *>(p.q_out) + (int64_t)t * p.q_out_stride;
    const int64_t crow = ((slot >> 4) * Hkv * 16 + (slot & 15)) * D;   // row of KV head 0 (block_size 16)

    for (int hb = h0; hb < h1; hb += HW) {
        const int h = hb + sub;
        const bool is_q = h < H, is_k = !is_q && h < H + Hkv;
        const int j = is_q ? h : (is_k ? h - H : h - H - Hkv);
        const bool live = lane_ok && h < h1 && (is_q || write);
        const T *src = (is_q ? q : is_k ? k : v) + (int64_t)j * D;
        Raw8<T> ra = {}, rb = {};
        if (live) {
            ra = load_raw8<T>(src + ea);
            rb = load_raw8<T>(src + eb);
        }
        float a[8], b[8];
        widen8<T>(ra, a);
        widen8<T>(rb, b);
        const T *w = reinterpret_cast<const T *>(is_q ? p.q_weight : is_k ? p.k_weight : nullptr);
        if (p.q_weight || p.k_weight) {             // the sum needs every lane of the warp
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
            for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (w && live) {
                const float f = 1.f / sqrtf(ss / (float)D + p.eps);
                float wa[8], wb[8];
                widen8<T>(load_raw8<T>(w + ea), wa);
                widen8<T>(load_raw8<T>(w + eb), wb);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    a[e] *= f * wa[e];
                    b[e] *= f * wb[e];
                }
            }
        }
        if (rot && (is_q || is_k)) {
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], u = b[2 * i + 1];
                    a[2 * i] = x * cs[i] - y * sn[i];
                    a[2 * i + 1] = y * cs[i] + x * sn[i];
                    b[2 * i] = z * cs[4 + i] - u * sn[4 + i];
                    b[2 * i + 1] = u * cs[4 + i] + z * sn[4 + i];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = a[e], y = b[e];
                    a[e] = x * cs[e] - y * sn[e];
                    b[e] = y * cs[e] + x * sn[e];
                }
            }
        }
        if (!live) continue;
        if (is_q) {
            T *dst = qo + (int64_t)j * D;
            store_raw8<T>(dst + ea, narrow8<T>(a));
            store_raw8<T>(dst + eb, narrow8<T>(b));
        } else {
            const int64_t at = crow + (int64_t)j * 16 * D;
            void *cache = is_k ? p.k_cache : p.v_cache;
            if constexpr (F8) {
                const float sc = __ldg((is_k ? p.k_scale : p.v_scale) + j);
                unsigned char *dst = static_cast<unsigned char *>(cache) + at;
                *reinterpret_cast<uint2 *>(dst + ea) = e4m3_of8(a, sc);
                *reinterpret_cast<uint2 *>(dst + eb) = e4m3_of8(b, sc);
            } else {
                T *dst = static_cast<T *>(cache) + at;
                store_raw8<T>(dst + ea, is_k ? narrow8<T>(a) : ra);   // v bit for bit
                store_raw8<T>(dst + eb, is_k ? narrow8<T>(b) : rb);
            }
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
