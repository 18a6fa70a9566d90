// milo_dense.cuh -- the dense 16-bit product's parameter block, activations
// and their derivatives (dense.cu, dense_tc.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

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

// The activations in fp32, act by act so that a loop over a register tile has
// no branch in it.  1 / (1 + exp(-v)) by the fast exponential and reciprocal
// (2^-22.5 and 2^-23) is within 2^-21 + 2^-23 |v| of its value, relative to it (|v|
// from the exponential's argument), and so is silu; gelu_tanh, whose argument
// has three roundings of its own, within 2^-21 + 2^-21 |v|.  That is far below the
// half step of a 16-bit result; an fp32 result is a few steps off, tens of steps
// where |v| is in the tens and the result below 1e-12.  Past v = -87.3 the reciprocal
// is flushed: a result below 2^-119 may be 0.  (__expf in place of the bare ex2:
// 8192 x 14336 x 4096 with gelu_tanh 619 us against 612.)
__device__ __forceinline__ float exp_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.44269504088896f));
    return r;
}
__device__ __forceinline__ float sigmoid_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + exp_fast(-v)));
    return r;
}

// The normal distribution's lower tail, Phi(-a) = exp(-a^2 / 2) r(a) for a >= 0:
// e = exp(-a^2 / 2) and r.  r falls slowly (like 0.4 / a), and is t P(t) with t = 1 /
// (1 + a / 4): a polynomial in the reciprocal of a linear function times the
// exponential, the form of Hastings' approximations (1955), its coefficients a
// fit of our own to erfc in 64 bits (degree 8, within 2^-24 of r relative to it
// for a <= 13.3, where exp(-a^2 / 2) leaves fp32's normal range).  With the
// roundings Phi(-a) is within (a^2 + 9) 2^-23 of its value, relative to it (a^2
// from the exponential's argument; the reciprocal counts up to 3.2 times); 1 + erf
// cancels below zero (4% off at -5, nothing left from -5.6 on).  erfcf is as exact
// but dearer: 8192 x 14336 x 4096 with gelu 680 us against 633 with erff and with
// this, the slope's pass (8192 x 8192, sums alone) 136, 91 and 69.  a is cut at 16,
// where e is 0, so that an infinity does not meet it.
__device__ __forceinline__ void normal_tail(float z, float& a, float& e, float& r) {
    a = fminf(fabsf(z), 16.0f);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a * a * -0.72134752044448f));
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.25f, a, 1.0f)));
    float p = 0.0265311133f;
    p = fmaf(p, t, -0.156805381f);
    p = fmaf(p, t, 0.304548144f);
    p = fmaf(p, t, -0.215653077f);
    p = fmaf(p, t, 0.208767325f);
    p = fmaf(p, t, 0.0298440605f);
    p = fmaf(p, t, 0.104566082f);
    p = fmaf(p, t, 0.0983968228f);
    p = fmaf(p, t, 0.0998048931f);
    r = t * p;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == MILO_ACT_RELU) {
        return z <= 0.0f ? 0.0f : z;                             // NaN stays
    } else if constexpr (ACT == MILO_ACT_SILU) {
        return z * sigmoid_fast(z);
    } else if constexpr (ACT == MILO_ACT_GELU) {
        // max(z, 0) - |z| Phi(-|z|); NaN stays
        float a, e, r;
        normal_tail(z, a, e, r);
        return fmaf(-a, e * r, z <= 0.0f ? 0.0f : z);
    } else if constexpr (ACT == MILO_ACT_GELU_TANH) {
        // (1 + tanh u) / 2 = 1 / (1 + exp(-2u)), without the cancellation near -1
        return z * sigmoid_fast(z * fmaf(0.07135481627260f, z * z, 1.59576912160573f));
    } else {
        return z;
    }
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == MILO_ACT_RELU) {
        return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
    } else if constexpr (ACT == MILO_ACT_SILU) {
        const float g = sigmoid_fast(z);
        return g * fmaf(z, 1.0f - g, 1.0f);
    } else if constexpr (ACT == MILO_ACT_GELU) {
        // Phi(z) + z phi(z), below zero e (r - |z| / sqrt(2 pi)); NaN stays
        float a, e, r;
        normal_tail(z, a, e, r);
        const float low = e * fmaf(-0.39894228040143f, a, r);
        return z > 0.0f ? 1.0f - low : z <= 0.0f ? low : z;
    } else if constexpr (ACT == MILO_ACT_GELU_TANH) {
        // past |z| = 16 the slope is 0 or 1 to the last bit, and z^2 may overflow
        const float c = fminf(fmaxf(z, -16.0f), 16.0f);
        const float g = sigmoid_fast(c * fmaf(0.07135481627260f, c * c, 1.59576912160573f));
        return z == z ? fmaf(c * g * (1.0f - g), fmaf(0.21406444881780f, c * c, 1.59576912160573f), g) : z;
    } else {
        return 1.0f;
    }
}

// f(std::integral_constant<int, act>) for a run-time act.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case MILO_ACT_RELU: f(std::integral_constant<int, MILO_ACT_RELU>{}); break;
        case MILO_ACT_SILU: f(std::integral_constant<int, MILO_ACT_SILU>{}); break;
        case MILO_ACT_GELU: f(std::integral_constant<int, MILO_ACT_GELU>{}); break;
        case MILO_ACT_GELU_TANH: f(std::integral_constant<int, MILO_ACT_GELU_TANH>{}); break;
        default: f(std::integral_constant<int, MILO_ACT_NONE>{}); break;
    }
}

// f(std::integral_constant<int, dt>) for a run-time dtype: the loops inside have
// no branch on it.
template <typename F>
__device__ __forceinline__ void with_dtype(int dt, F&& f) {
    if (dt == MILO_BF16) f(std::integral_constant<int, MILO_BF16>{});
    else if (dt == MILO_F16) f(std::integral_constant<int, MILO_F16>{});
    else f(std::integral_constant<int, MILO_F32>{});
}

// Two fp32 values rounded to fp16 or bf16, as one word.
template <int DT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (DT == MILO_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// FP16_RANGE for N values and their packed halves: one whose exponent field is
// all ones (adding one there carries into the sign's place) is looked at again,
// since an infinity may have been one before.
template <int N>
__device__ __forceinline__ void half_range(const float (&v)[N], const uint32_t* w, int32_t& st) {
    uint32_t e = 0;
#pragma unroll
    for (int q = 0; q < N / 2; ++q) e |= (w[q] & 0x7C007C00u) + 0x04000400u;
    if (e & 0x80008000u) {
#pragma unroll
        for (int q = 0; q < N; ++q)
            if (fabsf(v[q]) >= 65520.0f && !isinf(v[q])) st |= MILO_DEV_FP16_RANGE;
    }
}

template <int DT>
__device__ __forceinline__ float unpack16(uint32_t w, int hi) {
    if constexpr (DT == MILO_BF16) return __uint_as_float(hi ? w & 0xFFFF0000u : w << 16);
    else return __half2float(__ushort_as_half(static_cast<uint16_t>(hi ? w >> 16 : w & 0xFFFFu)));
}

// One element of a tensor of type DT.
template <int DT>
__device__ __forceinline__ float elem_load(const void* p, size_t i) {
    if constexpr (DT == MILO_F32) return static_cast<const float*>(p)[i];
    else return unpack16<DT>(static_cast<const uint16_t*>(p)[i], 0);
}
template <int DT>
__device__ __forceinline__ void elem_store(void* p, size_t i, float v, int32_t& st) {
    if constexpr (DT == MILO_F32) {
        static_cast<float*>(p)[i] = v;
    } else if constexpr (DT == MILO_BF16) {
        static_cast<uint16_t*>(p)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    } else {
        static_cast<uint16_t*>(p)[i] = __half_as_ushort(__float2half_rn(v));
        if (fabsf(v) >= 65520.0f && !isinf(v)) st |= MILO_DEV_FP16_RANGE;
    }
}

template <int N>
__device__ __forceinline__ void act_tile(int act, float (&v)[N]) {
    with_act(act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = act_value<decltype(a)::value>(v[i]);
    });
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

// Tokens up to which the forward product goes to the kernel for few rows.
constexpr int kDenseFewRows = 16;

milo_status launch_dense_gemm(const DenseGemm& g, const char* what, cudaStream_t s);       // dense_tc.cu
// Two products without an epilogue, of the same types, in one launch; one whose y
// is NULL is left out, and the other's bits do not depend on that.
milo_status launch_dense_pair(const DenseGemm& g0, const DenseGemm& g1, const char* what, cudaStream_t s);
milo_status launch_dense_few(const DenseGemm& g, const char* what, cudaStream_t s);        // dense_few.cu

}  // namespace milo
