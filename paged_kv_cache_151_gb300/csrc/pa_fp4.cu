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

// Sixteen elements as fp32.
template <typename T>
__device__ __forceinline__ void load16(const T *src, float (&x)[16]) {
    constexpr int E = Elem<T>::E;
#pragma unroll
    for (int i = 0; i < 16 / E; ++i) Elem<T>::to_f32(reinterpret_cast<const uint4 *>(src)[i], x + i * E);
}

template <typename T>
__device__ __forceinline__ void store16(T *dst, const float (&x)[16]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4 *>(dst)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            reinterpret_cast<uint4 *>(dst)[i] =
                make_uint4(Mma<T>::pack(x[8 * i], x[8 * i + 1]), Mma<T>::pack(x[8 * i + 2], x[8 * i + 3]),
                           Mma<T>::pack(x[8 * i + 4], x[8 * i + 5]), Mma<T>::pack(x[8 * i + 6], x[8 * i + 7]));
    }
}

// Codes (element 2i in the low half of byte i) and scale of a group.
__device__ __forceinline__ uint2 quantise16(float (&x)[16], float scale, uint32_t &sc) {
    float top = 0.f;
    bool nan = false;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        x[e] = __fdiv_rn(x[e], scale);
        top = fmaxf(top, fabsf(x[e]));
        nan = nan || x[e] != x[e];
    }
    sc = nan ? 0x7fu : e4m3x2_from_f32(__fdiv_rn(top, 6.f), 0.f) & 0xffu;
    float S, unused;
    Mma<__half>::unpack(f16x2_from_e4m3x2(sc), S, unused);
    uint32_t w[2] = {0, 0};
    if (S > 0.f) {                                 // NaN: codes of 0 beside it
#pragma unroll
        for (int e = 0; e < 16; e += 2)
            w[e / 8] |= e2m1x2_from_f32(__fdiv_rn(x[e], S), __fdiv_rn(x[e + 1], S)) << (4 * (e & 7));
    }
    return make_uint2(w[0], w[1]);
}

// One thread per group of 16 elements of a (token, KV head) row, of K or V.
template <typename T>
__global__ void __launch_bounds__(256) reshape_and_cache_fp4_kernel(const __grid_constant__ Fp4RowsParams p) {
    launch_dependents();      // a decode launched next may set up meanwhile
    const int per_row = p.head_dim / 16;
    const int64_t per_tok = 2 * (int64_t)p.num_kv_heads * per_row;
    const int64_t total = p.num_tokens * per_tok;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = i / per_tok;
        int rem = (int)(i - t * per_tok);
        const bool is_v = rem >= p.num_kv_heads * per_row;
        if (is_v) rem -= p.num_kv_heads * per_row;
        const int j = rem / per_row, grp = rem - j * per_row;
        const int64_t slot = p.slot_mapping[t];
        if (slot < 0) continue;                        // padding token
        if (slot >= p.num_slots) {
            if (rem == 0 && !is_v) set_error(p.err, ERR_SLOT);
            continue;
        }
        const T *src = static_cast<const T *>(is_v ? p.v : p.k) + t * (is_v ? p.v_stride : p.k_stride) +
                       (int64_t)j * p.head_dim + grp * 16;
        float x[16];
        load16<T>(src, x);
        uint32_t sc;
        const uint2 w = quantise16(x, __ldg((is_v ? p.v_scale : p.k_scale) + j), sc);
        unsigned char *tile = static_cast<unsigned char *>(is_v ? p.v_cache : p.k_cache) +
                              ((slot >> 4) * p.num_kv_heads + j) * (9 * (int64_t)p.head_dim);
        const int row = (int)(slot & 15);
        *reinterpret_cast<uint2 *>(tile + row * (p.head_dim / 2) + grp * 8) = w;
        tile[8 * p.head_dim + row * per_row + grp] = (unsigned char)sc;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) gather_cache_fp4_kernel(const __grid_constant__ Fp4RowsParams p) {
    const int per_row = p.head_dim / 16;
    const int64_t per_tok = 2 * (int64_t)p.num_kv_heads * per_row;
    const int64_t total = p.num_tokens * per_tok;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = i / per_tok;
        int rem = (int)(i - t * per_tok);
        const bool is_v = rem >= p.num_kv_heads * per_row;
        if (is_v) rem -= p.num_kv_heads * per_row;
        const int j = rem / per_row, grp = rem - j * per_row;
        const int64_t slot = p.slot_mapping[t];
        if (slot < 0) continue;                        // padding token: its row stays
        if (slot >= p.num_slots) {
            if (rem == 0 && !is_v) set_error(p.err, ERR_SLOT);
            continue;
        }
        const unsigned char *tile = static_cast<const unsigned char *>(is_v ? p.v_cache : p.k_cache) +
                                    ((slot >> 4) * p.num_kv_heads + j) * (9 * (int64_t)p.head_dim);
        const int row = (int)(slot & 15);
        const uint2 w = *reinterpret_cast<const uint2 *>(tile + row * (p.head_dim / 2) + grp * 8);
        const uint32_t sc = tile[8 * p.head_dim + row * per_row + grp];
        const uint32_t s2 = f16x2_from_e4m3x2(sc | (sc << 8));
        const float scale = __ldg((is_v ? p.v_scale : p.k_scale) + j);
        uint32_t h[8];
        f16x2_from_e2m1x8(w.x, *reinterpret_cast<uint32_t(*)[4]>(&h[0]));
        f16x2_from_e2m1x8(w.y, *reinterpret_cast<uint32_t(*)[4]>(&h[4]));
        float x[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            Mma<__half>::unpack(mul_f16x2(h[e], s2), x[2 * e], x[2 * e + 1]);
            x[2 * e] *= scale;
            x[2 * e + 1] *= scale;
        }
        T *dst = static_cast<T *>(is_v ? p.v_out : p.k_out) + t * (is_v ? p.v_stride : p.k_stride) +
                 (int64_t)j * p.head_dim + grp * 16;
        store16<T>(dst, x);
    }
}

template <typename T, bool GATHER>
cudaError_t launch_rows(const Fp4RowsParams &p, cudaStream_t st) {
    const int64_t total = p.num_tokens * 2 * p.num_kv_heads * (p.head_dim / 16);
    const int sms = sm_count_of_current_device();
    int64_t blocks = (total + 255) / 256;
    const int64_t cap = (int64_t)(sms > 0 ? sms : 152) * 16;
    if (blocks > cap) blocks = cap;
    if constexpr (GATHER) {
        gather_cache_fp4_kernel<T><<<(unsigned)blocks, 256, 0, st>>>(p);
    } else {
        prefer_shared_carveout<reshape_and_cache_fp4_kernel<T>>();
        reshape_and_cache_fp4_kernel<T><<<(unsigned)blocks, 256, 0, st>>>(p);
    }
    return cudaGetLastError();
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
