// milo_exchange.cuh -- pieces shared by the kernels that move token rows into
// expert order and back (exchange.cu) and their gradients (exchange_grad.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
    uint32_t nv;                // H / V: vectors of a row
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

// V consecutive elements, moved in 16-byte pieces (V = 8; the address is
// 16-byte aligned) or one element at a time (V = 1).
template <typename T, int V>
struct alignas(V == 1 ? sizeof(T) : 16) RowVec {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ RowVec<T, V> load_vec(const void* base, size_t row, size_t H, uint32_t c) {
    RowVec<T, V> r;
    const T* p = static_cast<const T*>(base) + row * H + static_cast<size_t>(c) * V;
    if constexpr (V == 1) {
        r.v[0] = *p;
    } else {
#pragma unroll
        for (int q = 0; q < static_cast<int>(V * sizeof(T) / 16); ++q)
            reinterpret_cast<uint4*>(r.v)[q] = reinterpret_cast<const uint4*>(p)[q];
    }
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(void* base, size_t row, size_t H, uint32_t c, const RowVec<T, V>& r) {
    T* p = static_cast<T*>(base) + row * H + static_cast<size_t>(c) * V;
    if constexpr (V == 1) {
        *p = r.v[0];
    } else {
#pragma unroll
        for (int q = 0; q < static_cast<int>(V * sizeof(T) / 16); ++q)
            reinterpret_cast<uint4*>(p)[q] = reinterpret_cast<const uint4*>(r.v)[q];
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
    int vec;                    // 8 or 1
};

cudaError_t launch_exchange(const ExchangeParams& p, const ExchangeTypes& t, bool combine, cudaStream_t s);
cudaError_t launch_exchange_grad(const ExchangeParams& p, const ExchangeTypes& t, bool combine, cudaStream_t s);

}  // namespace milo
