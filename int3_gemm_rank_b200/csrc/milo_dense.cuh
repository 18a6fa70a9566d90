// milo_dense.cuh -- the dense 16-bit product's parameter block, activations
// and their derivatives (dense.cu, dense_tc.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "milo_device.cuh"

namespace milo {

// D[p, q] = sum_c A(p, c) B(q, c), then the epilogue of y[p, q].
// K-major operand: element (r, c) at base[r * ld + c]; MN-major: base[c * ld + r].
struct DenseGemm {
    const void *a, *b;
    long long lda, ldb;
    int a_mn, b_mn;
    int P, Q, C;
    int bf16;                   // type of a, b, bias and z: bf16 or fp16
    const void* bias;           // [Q] or NULL
    const void* residual;       // [P, Q] in y_dt or NULL
    int act;
    void* y;                    // [P, Q]
    int y_dt;
    void* z;                    // [P, Q] or NULL
    int32_t* dev_status;
};

__device__ __forceinline__ float dense_act(int act, float z) {
    switch (act) {
        case MILO_ACT_RELU: return z <= 0.0f ? 0.0f : z;     // NaN stays
        case MILO_ACT_SILU: return z / (1.0f + expf(-z));
        case MILO_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
        case MILO_ACT_GELU_TANH: {
            // (1 + tanh u) / 2 = 1 / (1 + exp(-2u)), without the cancellation near -1
            const float u = 0.79788456080286536f * (z + 0.044715f * z * z * z);
            return z / (1.0f + expf(-2.0f * u));
        }
        default: return z;
    }
}

__device__ __forceinline__ float dense_dact(int act, float z) {
    switch (act) {
        case MILO_ACT_RELU: return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
        case MILO_ACT_SILU: {
            const float g = 1.0f / (1.0f + expf(-z));
            return g * (1.0f + z * (1.0f - g));
        }
        case MILO_ACT_GELU:
            return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) +
                   z * expf(-0.5f * z * z) * 0.39894228040143268f;
        case MILO_ACT_GELU_TANH: {
            // past |z| = 16 the slope is 0 or 1 to the last bit, and z^2 may overflow
            if (fabsf(z) > 16.0f) return z > 0.0f ? 1.0f : 0.0f;
            const float u = 0.79788456080286536f * (z + 0.044715f * z * z * z);
            const float g = 1.0f / (1.0f + expf(-2.0f * u));
            return g + z * g * (1.0f - g) * 1.59576912160573071f * (1.0f + 0.134145f * z * z);
        }
        default: return 1.0f;
    }
}

__device__ __forceinline__ float load16(const void* p, size_t i, int bf16) {
    return act_f32(static_cast<const uint16_t*>(p)[i], bf16);
}

__device__ __forceinline__ float load_any(const void* p, size_t i, int dt) {
    return dt == MILO_F32 ? static_cast<const float*>(p)[i] : load16(p, i, dt == MILO_BF16);
}

// fp16 (FP16_RANGE when a finite value does not fit) or bf16 bits of v.
__device__ __forceinline__ uint16_t round16(float v, int bf16, int32_t& st) {
    if (bf16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    const __half h = __float2half_rn(v);
    if (__hisinf(h) && !isinf(v)) st |= MILO_DEV_FP16_RANGE;
    return __half_as_ushort(h);
}

__device__ __forceinline__ void store_any(void* p, size_t i, int dt, float v, int32_t& st) {
    if (dt == MILO_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = round16(v, dt == MILO_BF16, st);
}

milo_status launch_dense_gemm(const DenseGemm& g, const char* what, cudaStream_t s);

}  // namespace milo
