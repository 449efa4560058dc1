// pa_fp4.cu -- the cache write into E2M1 caches, and the rows read back.
//
// For the 16 neighbouring elements x of a group of a new row, KV head j:
//   y = x / scale_j                      (binary32, IEEE division)
//   S = E4M3(max |y| / 6)                (nearest even, saturating at 448; NaN if any y is)
//   code = E2M1(y / S)                   (nearest even, saturating at 6; S = 0: the codes are 0)
// and an element read back is value(code) * value(S) * scale_j: the first product is
// exact, the second rounded to binary32 and then to the output's type.
#include "pa_common.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

// Sixteen elements as fp32.  With WIDE, 32 bytes an access (every row starts on 32
// bytes): two of 16 touch each sector twice (32001 x 16 rows of 128 in bf16: 58 us a
// write against 44, reading them back 37 against 30; the write is at 3.8 TB/s, bound by
// its instructions: a group's largest, its quotients and their codes).
__device__ __forceinline__ void load_b256(const void *p, uint32_t (&w)[8]) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}
__device__ __forceinline__ void store_b256(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
                 :: "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
                 : "memory");
}
template <typename T, bool WIDE>
__device__ __forceinline__ void load16(const T *src, float (&x)[16]) {
    constexpr int E = Elem<T>::E;
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < 16 / (2 * E); ++i) {
            uint32_t w[8];
            load_b256(src + i * 2 * E, w);
            Elem<T>::to_f32(make_uint4(w[0], w[1], w[2], w[3]), x + i * 2 * E);
            Elem<T>::to_f32(make_uint4(w[4], w[5], w[6], w[7]), x + i * 2 * E + E);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16 / E; ++i) Elem<T>::to_f32(__ldg(reinterpret_cast<const uint4 *>(src) + i), x + i * E);
    }
}

template <typename T, bool WIDE>
__device__ __forceinline__ void store16(T *dst, const float (&x)[16]) {
    constexpr int N = 16 * (int)sizeof(T) / 4;     // words
    uint32_t w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x[i]);
        else w[i] = Mma<T>::pack(x[2 * i], x[2 * i + 1]);
    }
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < N; i += 8)
            store_b256(reinterpret_cast<uint32_t *>(dst) + i, *reinterpret_cast<const uint32_t(*)[8]>(&w[i]));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            reinterpret_cast<uint4 *>(dst)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
}

// Codes (element 2i in the low half of byte i) and scale of a group, as defined.
template <typename T>
__device__ __noinline__ uint2 quantise16_divided(const T *src, float scale, uint32_t &sc) {
    float x[16], y[16], top = 0.f;
    load16<T, false>(src, x);
    bool nan = false;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        y[e] = __fdiv_rn(x[e], scale);
        top = fmaxf(top, fabsf(y[e]));
        nan = nan || y[e] != y[e];
    }
    sc = nan ? 0x7fu : e4m3x2_from_f32(__fdiv_rn(top, 6.f), 0.f) & 0xffu;
    float S, unused;
    Mma<__half>::unpack(f16x2_from_e4m3x2(sc), S, unused);
    uint32_t w[2] = {0, 0};
    if (S > 0.f) {                                 // NaN: codes of 0 beside it
#pragma unroll
        for (int e = 0; e < 16; e += 2)
            w[e / 8] |= e2m1x2_from_f32(__fdiv_rn(y[e], S), __fdiv_rn(y[e + 1], S)) << (4 * (e & 7));
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The same without its 33 divisions, a third of the write's time.  y times a
// reciprocal is within 2^-22.4 of the quotient, and twice so within 2^-21.2; where
// 2^-20 below and above give the same scale and the same codes those are the
// quotients' (rounding is monotonic), and the rest -- a group in 2^13 or so -- is
// divided.  r: 1 / scale, 0: always divide.
template <typename T>
__device__ __forceinline__ uint2 quantise16(const T *src, const float (&x)[16], float scale, float r, uint32_t &sc) {
    constexpr float DN = 1.f - 0x1p-20f, UP = 1.f + 0x1p-20f;
    float2 y[8];
    float top = 0.f;                               // NaN if one of them is
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        y[e] = mul2(make_float2(x[2 * e], x[2 * e + 1]), make_float2(r, r));
        top = max_nan(top, fabsf(y[e].x), fabsf(y[e].y));
    }
    const float t = top * (1.f / 6.f);
    const uint32_t both = e4m3x2_from_f32(t * DN, t * UP);
    sc = both & 0xffu;
    float S, unused;
    Mma<__half>::unpack(f16x2_from_e4m3x2(sc), S, unused);
    const float rs = S > 0.f ? __frcp_rn(S) : 0.f;
    uint32_t lo[2] = {0, 0}, hi[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 z = mul2(y[e], make_float2(rs, rs));
        const float2 zl = mul2(z, make_float2(DN, DN)), zh = mul2(z, make_float2(UP, UP));
        lo[e / 4] |= e2m1x2_from_f32(zl.x, zl.y) << (8 * (e & 3));
        hi[e / 4] |= e2m1x2_from_f32(zh.x, zh.y) << (8 * (e & 3));
    }
    // (a scale of 0: codes of +0)
    if (sc != both >> 8 || lo[0] != hi[0] || lo[1] != hi[1] || !(top < INFINITY) || r == 0.f)
        return quantise16_divided(src, scale, sc);
    return S > 0.f ? make_uint2(lo[0], lo[1]) : make_uint2(0, 0);
}

// Where a thread's group of 16 elements of a (token, KV head) row is, in K and V.
struct Place {
    unsigned t;                                    // token
    int j, grp;                                    // KV head, group of its row
    int64_t tile;                                  // its tile's first byte
    int row;                                       // row of the tile, -1: no slot
};
__device__ __forceinline__ Place place_of(const Fp4RowsParams &p, unsigned item) {
    const unsigned per_row = (unsigned)p.head_dim / 16, per_tok = per_row * (unsigned)p.num_kv_heads;
    Place at;
    at.t = item / per_tok;
    const unsigned rem = item - at.t * per_tok;
    at.j = (int)(rem / per_row);
    at.grp = (int)(rem - (unsigned)at.j * per_row);
    const int64_t slot = p.slot_mapping[at.t];
    at.row = -1;
    at.tile = 0;
    if (slot >= p.num_slots) {
        if (rem == 0) set_error(p.err, ERR_SLOT);
    } else if (slot >= 0) {                        // negative: a padding token
        at.row = (int)(slot & 15);
        at.tile = ((slot >> 4) * p.num_kv_heads + at.j) * (9 * (int64_t)p.head_dim);
    }
    return at;
}

// One thread per group of a (token, KV head) row, of K and V.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) reshape_and_cache_fp4_kernel(const __grid_constant__ Fp4RowsParams p) {
    launch_dependents();      // a decode launched next may set up meanwhile
    const unsigned item = blockIdx.x * blockDim.x + threadIdx.x;
    if (item >= p.num_items) return;
    const Place at = place_of(p, item);
    if (at.row < 0) return;
    const int64_t src = (int64_t)at.j * p.head_dim + at.grp * 16;
    const int codes = at.row * (p.head_dim / 2) + at.grp * 8;
    const int scale = 8 * p.head_dim + at.row * (p.head_dim / 16) + at.grp;
    float x[2][16];
    const T *from[2] = {static_cast<const T *>(p.k) + at.t * p.k_stride + src,
                        static_cast<const T *>(p.v) + at.t * p.v_stride + src};
    load16<T, WIDE>(from[0], x[0]);
    load16<T, WIDE>(from[1], x[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float s = __ldg((i ? p.v_scale : p.k_scale) + at.j);
        const float r = s > 0x1p-100f && s < 0x1p100f ? __frcp_rn(s) : 0.f;
        uint32_t sc;
        const uint2 w = quantise16<T>(from[i], x[i], s, r, sc);
        unsigned char *tile = static_cast<unsigned char *>(i ? p.v_cache : p.k_cache) + at.tile;
        *reinterpret_cast<uint2 *>(tile + codes) = w;
        tile[scale] = (unsigned char)sc;
    }
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) gather_cache_fp4_kernel(const __grid_constant__ Fp4RowsParams p) {
    const unsigned item = blockIdx.x * blockDim.x + threadIdx.x;
    if (item >= p.num_items) return;
    const Place at = place_of(p, item);
    if (at.row < 0) return;                        // padding token: its row stays
    const int64_t dst = (int64_t)at.j * p.head_dim + at.grp * 16;
    const int codes = at.row * (p.head_dim / 2) + at.grp * 8;
    const int scale = 8 * p.head_dim + at.row * (p.head_dim / 16) + at.grp;
    uint2 w[2];
    uint32_t sc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const unsigned char *tile = static_cast<const unsigned char *>(i ? p.v_cache : p.k_cache) + at.tile;
        w[i] = *reinterpret_cast<const uint2 *>(tile + codes);
        sc[i] = tile[scale];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t s2 = f16x2_from_e4m3x2(sc[i] | (sc[i] << 8));
        const float s = __ldg((i ? p.v_scale : p.k_scale) + at.j);
        uint32_t h[2][4];
        f16x2_from_e2m1x8(w[i].x, h[0]);
        f16x2_from_e2m1x8(w[i].y, h[1]);
        float x[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            Mma<__half>::unpack(mul_f16x2(h[e / 4][e & 3], s2), x[2 * e], x[2 * e + 1]);
            x[2 * e] *= s;
            x[2 * e + 1] *= s;
        }
        T *to = static_cast<T *>(i ? p.v_out : p.k_out) + at.t * (i ? p.v_stride : p.k_stride) + dst;
        store16<T, WIDE>(to, x);
    }
}

template <typename T, bool GATHER>
cudaError_t launch_rows(Fp4RowsParams p, cudaStream_t st) {
    // items are numbered in 32 bits: more tokens than that go in several launches
    const int64_t per_tok = (int64_t)p.num_kv_heads * (p.head_dim / 16);
    const int64_t step = (int64_t)(1u << 31) / per_tok;            // at least 2^9 tokens
    const Fp4RowsParams all = p;
    const uintptr_t starts = GATHER ? (uintptr_t)p.k_out | (uintptr_t)p.v_out : (uintptr_t)p.k | (uintptr_t)p.v;
    const bool wide = ((starts | (uintptr_t)(p.k_stride * sizeof(T)) | (uintptr_t)(p.v_stride * sizeof(T))) & 31) == 0;
    for (int64_t t = 0; t < all.num_tokens; t += step) {
        const int64_t n = all.num_tokens - t < step ? all.num_tokens - t : step;
        p = all;
        p.slot_mapping += t;
        const int64_t ko = t * p.k_stride * (int64_t)sizeof(T), vo = t * p.v_stride * (int64_t)sizeof(T);
        if (GATHER) {
            p.k_out = static_cast<char *>(p.k_out) + ko;
            p.v_out = static_cast<char *>(p.v_out) + vo;
        } else {
            p.k = static_cast<const char *>(p.k) + ko;
            p.v = static_cast<const char *>(p.v) + vo;
        }
        p.num_items = (unsigned)(n * per_tok);
        const unsigned blocks = (p.num_items + 255) / 256;
        if constexpr (GATHER) {
            if (wide) gather_cache_fp4_kernel<T, true><<<blocks, 256, 0, st>>>(p);
            else gather_cache_fp4_kernel<T, false><<<blocks, 256, 0, st>>>(p);
        } else if (wide) {
            prefer_shared_carveout<reshape_and_cache_fp4_kernel<T, true>>();
            reshape_and_cache_fp4_kernel<T, true><<<blocks, 256, 0, st>>>(p);
        } else {
            prefer_shared_carveout<reshape_and_cache_fp4_kernel<T, false>>();
            reshape_and_cache_fp4_kernel<T, false><<<blocks, 256, 0, st>>>(p);
        }
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <bool GATHER>
cudaError_t dispatch_rows(const Fp4RowsParams &p, int dtype, cudaStream_t st) {
    switch (dtype) {
        case 0: return launch_rows<float, GATHER>(p, st);
        case 1: return launch_rows<__nv_bfloat16, GATHER>(p, st);
        default: return launch_rows<__half, GATHER>(p, st);
    }
}

}  // namespace

cudaError_t reshape_and_cache_fp4(const Fp4RowsParams &p, int dtype, cudaStream_t st) {
    return dispatch_rows<false>(p, dtype, st);
}
cudaError_t gather_cache_fp4(const Fp4RowsParams &p, int dtype, cudaStream_t st) {
    return dispatch_rows<true>(p, dtype, st);
}

}  // namespace pa
