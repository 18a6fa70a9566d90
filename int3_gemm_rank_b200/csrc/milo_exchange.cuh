// milo_exchange.cuh -- pieces shared by the kernels that move token rows into
// expert order and back and their gradients (exchange.cu, exchange_rows.cuh).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "milo_device.cuh"

namespace milo {

struct ExchangeParams {
    const void* src;            // token rows [T, H] (dispatch, combine_backward: dy) or expert rows [T*k, H]
    const void* other;          // combine: residual [T, H] (output type) or NULL; gradients: the second row operand
    const int32_t* inv_perm;    // [T*k] expert row of each flat slot, -1: dropped
    const float* w;             // [T*k] or NULL (1)
    void* out;
    float* dw;                  // gradients: [T*k] or NULL
    int32_t* dev_status;
    int T, k, H;
    uint32_t nv;                // ceil(H / 8): vectors of a row
    uint32_t div_m, div_s;      // i / nv for i < 2^31 (see fast_div)
    int wide;                   // T * nv does not fit 31 bits: 64-bit indices
};

// i / d for 0 <= i < 2^31 (Granlund and Montgomery 1994, division by invariant
// integers): s = ceil(log2 d), m = floor(2^32 (2^s - d) / d) + 1,
// q = (mulhi(m, i) + i) >> s; the sum stays below 2^32 because both terms are
// below 2^31.
__device__ __forceinline__ uint32_t fast_div(uint32_t i, uint32_t m, uint32_t s) { return (__umulhi(m, i) + i) >> s; }

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Round once to the output type; FP16_RANGE when a finite value does not fit fp16.
template <typename T>
__device__ __forceinline__ T from_f32(float v, int32_t& st);
template <>
__device__ __forceinline__ float from_f32<float>(float v, int32_t&) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v, int32_t& st) {
    const __half h = __float2half_rn(v);
    if (__hisinf(h) && !isinf(v)) st |= MILO_DEV_FP16_RANGE;
    return h;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v, int32_t&) { return __float2bfloat16_rn(v); }

// Two fp32 values rounded to 16 bits each, as one word.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// FP16_RANGE for eight values and their packed halves: one whose exponent field is
// all ones (adding one there carries into the sign's place) is looked at again,
// since an infinity may have been one before.
__device__ __forceinline__ void half_overflow(const float (&v)[8], const uint32_t (&w)[4], int32_t& st) {
    uint32_t e = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) e |= (w[q] & 0x7C007C00u) + 0x04000400u;
    if (e & 0x80008000u) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (fabsf(v[q]) >= 65520.0f && !isinf(v[q])) st |= MILO_DEV_FP16_RANGE;
    }
}

// Eight values rounded to T.
template <typename T>
__device__ __forceinline__ void to_elems(const float (&v)[8], T (&e)[8], int32_t& st) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int q = 0; q < 8; ++q) e[q] = v[q];
    } else {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = pack2<T>(v[2 * q], v[2 * q + 1]);
        if constexpr (std::is_same<T, __half>::value) half_overflow(v, w, st);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint16_t h = static_cast<uint16_t>(q & 1 ? w[q / 2] >> 16 : w[q / 2] & 0xFFFFu);
            e[q] = *reinterpret_cast<const T*>(&h);
        }
    }
}

// Eight values to a 16-byte aligned address.
template <typename T>
__device__ __forceinline__ void store8(void* dst, const float (&v)[8], int32_t& st) {
    if constexpr (sizeof(T) == 4) {
        float4* d = static_cast<float4*>(dst);
        d[0] = make_float4(v[0], v[1], v[2], v[3]);
        d[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = pack2<T>(v[2 * q], v[2 * q + 1]);
        if constexpr (std::is_same<T, __half>::value) half_overflow(v, w, st);
        *static_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Eight values from a 16-byte aligned address.
template <typename T>
__device__ __forceinline__ void load8(const void* src, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4* p = static_cast<const float4*>(src);
        const float4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = *static_cast<const uint4*>(src);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (std::is_same<T, __half>::value) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[q]));
                v[2 * q] = f.x;
                v[2 * q + 1] = f.y;
            } else {
                v[2 * q] = __uint_as_float(w[q] << 16);
                v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
            }
        }
    }
}

// The expert row of a flat slot, or -1: a dropped slot, or (flagged, in every
// build) an entry outside the T*k rows.
__device__ __forceinline__ int slot_row(int r, int rows, int32_t& st) {
    if (r >= 0 && r < rows) return r;
    if (r != -1) st |= MILO_DEV_BOUNDS;
    return -1;
}

struct ExchangeTypes {
    milo_dtype in, out;
    bool aligned;               // rows of whole 16-byte pieces at 16-byte addresses
};

cudaError_t launch_dispatch(const ExchangeParams& p, const ExchangeTypes& t, cudaStream_t s);
cudaError_t launch_dispatch_rows(const ExchangeParams& p, const ExchangeTypes& t, cudaStream_t s);
cudaError_t launch_combine_rows(const ExchangeParams& p, const ExchangeTypes& t, cudaStream_t s);
cudaError_t launch_combine_grad(const ExchangeParams& p, const ExchangeTypes& t, cudaStream_t s);
cudaError_t launch_dispatch_grad(const ExchangeParams& p, const ExchangeTypes& t, cudaStream_t s);

}  // namespace milo
