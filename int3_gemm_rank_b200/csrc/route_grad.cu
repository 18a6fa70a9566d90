// route_grad.cu -- gradient of the router's top-k softmax weights
// (milo_route_backward).
#include <cuda_runtime.h>

#include <string>

#include "milo_exchange.cuh"
#include "milo_host.h"

namespace milo {

constexpr int kRgThreads = 128;

struct RouteGradArgs {
    const uint16_t* logits;
    const int32_t* ids;
    const float *w, *dw;
    int T, E, k, renorm, vec;   // vec: rows of whole 16-byte pieces at 16-byte addresses
    void* dl;
    int32_t* dev_status;
};

// Gradient of the top-k softmax weights:
//     s = sum_j w_j dw_j
//     renormalised:  dl[e_j] = w_j (dw_j - s),  0 elsewhere
//     full softmax:  dl[e] = [e = e_j] w_j dw_j - p_e s,  p = softmax(l)
// (the Jacobian of a softmax q is q_i ([i = l] - q_l); the renormalised one
// runs over the picked experts only).  L lanes share a token, eight experts
// each, so a warp takes 32 / L tokens and every reduction has log2 L steps:
// the instructions, not the bytes, bound a warp that gives a whole token to
// its 32 lanes (65536 x 64, k 6: 18.7 us that way).  The k <= KM picks are few
// and read by all L lanes (one L1 line) before anything else, each lane adding
// those that are its own.
template <typename TO, int L, int KM, bool VEC>
__global__ void __launch_bounds__(kRgThreads) route_grad_kernel(const RouteGradArgs p) {
    grid_dep_launch();
    grid_dep_wait();
    const long long i = static_cast<long long>(blockIdx.x) * kRgThreads + threadIdx.x;
    const bool in = i / L < p.T;                          // the last warp may be part empty
    const long long t = in ? i / L : p.T - 1;
    const int E = p.E, k = p.k;
    // the lane's experts: eight in a row, or every L-th where rows do not start on
    // 16-byte boundaries
    constexpr int step = VEC ? 1 : L;
    const int e0 = static_cast<int>(i % L) * (VEC ? 8 : 1);
    int32_t st = 0;
    float v[8], wj[KM], dj[KM];
    int id[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) {
        id[j] = -1;
        wj[j] = dj[j] = 0.0f;
        if (j < k) {
            id[j] = p.ids[t * k + j];
            wj[j] = p.w[t * k + j];
            dj[j] = p.dw[t * k + j];
        }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = 0.0f;
    if (!p.renorm) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = -INFINITY;
        const uint16_t* l = p.logits + t * E + e0;
        if constexpr (VEC) {
            if (e0 < E) load8<__half>(l, v);
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (e0 + q * step < E) v[q] = __half2float(__ushort_as_half(l[q * step]));
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < KM; ++j)
        if (j < k) {
            if (id[j] < 0 || id[j] >= E) st |= MILO_DEV_BAD_EXPERT_ID;
            else s = fmaf(wj[j], dj[j], s);
        }
    if (!p.renorm) {
        float m = -INFINITY, den = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (!isfinite(v[q]) && e0 + q * step < E) st |= MILO_DEV_NONFINITE;
            m = fmaxf(m, v[q]);                           // NaN counts as -inf, as in milo_route
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            v[q] = v[q] == v[q] ? expf(v[q] - m) : 0.0f;
            den += v[q];
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) den += __shfl_xor_sync(0xFFFFFFFFu, den, o);
        const float c = -s / den;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] *= c;
    }
#pragma unroll
    for (int j = 0; j < KM; ++j)
        if (j < k) {
            const float g = p.renorm ? wj[j] * (dj[j] - s) : wj[j] * dj[j];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (id[j] == e0 + q * step) v[q] += g;
        }
    if (!in) return;
    TO* d = static_cast<TO*>(p.dl) + t * E + e0;
    if constexpr (VEC) {
        if (e0 < E) store8<TO>(d, v, st);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (e0 + q * step < E) d[q * step] = from_f32<TO>(v[q], st);
    }
    flag(p.dev_status, st);
}

template <typename TO, int L>
static cudaError_t run_route_grad_l(const RouteGradArgs& a, cudaStream_t s) {
    const long long blocks = (static_cast<long long>(a.T) * L + kRgThreads - 1) / kRgThreads;
    auto k = a.vec ? (a.k <= 8 ? route_grad_kernel<TO, L, 8, true> : route_grad_kernel<TO, L, 16, true>)
                   : (a.k <= 8 ? route_grad_kernel<TO, L, 8, false> : route_grad_kernel<TO, L, 16, false>);
    return launch_pdl(k, dim3(static_cast<unsigned>(blocks)), dim3(kRgThreads), 0, s, a);
}

// Lanes of a token: eight experts each.
template <typename TO>
static cudaError_t run_route_grad(const RouteGradArgs& a, cudaStream_t s) {
    if (a.E <= 8) return run_route_grad_l<TO, 1>(a, s);
    if (a.E <= 16) return run_route_grad_l<TO, 2>(a, s);
    if (a.E <= 32) return run_route_grad_l<TO, 4>(a, s);
    if (a.E <= 64) return run_route_grad_l<TO, 8>(a, s);
    if (a.E <= 128) return run_route_grad_l<TO, 16>(a, s);
    return run_route_grad_l<TO, 32>(a, s);
}

}  // namespace milo

using namespace milo;

extern "C" milo_status milo_route_backward(const uint16_t* logits, const int32_t* topk_ids, const float* topk_w,
                                           const float* dw, int32_t T, int32_t E, int32_t k, uint32_t flags,
                                           void* dlogits, milo_dtype dl_dt, int32_t* dev_status, void* stream) {
    clear_error();
    if (T < 0) return fail(MILO_ERR_INVALID_ARG, "milo_route_backward: T must be >= 0");
    if (E < 1 || E > MILO_MAX_EXPERTS)
        return fail(MILO_ERR_UNSUPPORTED_SHAPE, "milo_route_backward: E must be in [1, 256]");
    if (k < 1 || k > E || k > MILO_MAX_TOPK)
        return fail(MILO_ERR_UNSUPPORTED_SHAPE, "milo_route_backward: k must be in [1, min(E, 16)]");
    if (flags & ~MILO_ROUTE_RENORM) return fail(MILO_ERR_INVALID_ARG, "milo_route_backward: unknown flag");
    if (dl_dt != MILO_F16 && dl_dt != MILO_BF16 && dl_dt != MILO_F32)
        return fail(MILO_ERR_INVALID_ARG, "milo_route_backward: bad dtype");
    if (static_cast<long long>(T) * k > MILO_MAX_ROWS)
        return fail(MILO_ERR_UNSUPPORTED_SHAPE, "milo_route_backward: T*k above MILO_MAX_ROWS");
    if (T == 0) return MILO_OK;
    const bool renorm = flags & MILO_ROUTE_RENORM;
    if (!topk_ids || !topk_w || !dw || !dlogits || (!renorm && !logits))
        return fail(MILO_ERR_INVALID_ARG, "milo_route_backward: NULL pointer");
    if (!aligned(dlogits, dl_dt == MILO_F32 ? 4 : 2))
        return fail(MILO_ERR_INVALID_ARG, "milo_route_backward: dlogits must be aligned to its elements");
    const int vec = E % 8 == 0 && aligned(logits, 16) && aligned(dlogits, 16);
    const RouteGradArgs a = {logits, topk_ids, topk_w, dw, T, E, k, renorm ? 1 : 0, vec, dlogits, dev_status};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dl_dt == MILO_F32   ? run_route_grad<float>(a, st)
                          : dl_dt == MILO_F16 ? run_route_grad<__half>(a, st)
                                              : run_route_grad<__nv_bfloat16>(a, st);
    return check_cuda(e, "milo_route_backward");
}
