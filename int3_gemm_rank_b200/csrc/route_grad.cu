// route_grad.cu -- gradient of the router's top-k softmax weights
// (milo_route_backward).
#include <cuda_runtime.h>

#include <string>

#include "milo_exchange.cuh"
#include "milo_host.h"

namespace milo {

constexpr int kRgThreads = 128;

// Gradient of the top-k softmax weights, one warp per token:
//     s = sum_j w_j dw_j
//     renormalised:  dl[e_j] = w_j (dw_j - s),  0 elsewhere
//     full softmax:  dl[e] = [e = e_j] w_j dw_j - p_e s,  p = softmax(l)
// (the Jacobian of a softmax q is q_i ([i = l] - q_l); the renormalised one
// runs over the picked experts only).  Lane j holds pick j; lanes then own
// experts 32 i + lane, i < S.  A warp takes UT tokens side by side: their
// chains of dependent reductions overlap, and so do their loads.
template <typename TO, int S, int UT>
__global__ void __launch_bounds__(kRgThreads)
route_grad_kernel(const uint16_t* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ w,
                  const float* __restrict__ dw, int T, int E, int k, int renorm, TO* __restrict__ dl,
                  int32_t* __restrict__ dev_status) {
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const long long t0 = (static_cast<long long>(blockIdx.x) * (kRgThreads / 32) + (threadIdx.x >> 5)) * UT;
    if (t0 >= T) return;
    int32_t st = 0;
    int id[UT];
    float wj[UT], g[UT], s[UT], v[UT][S];
#pragma unroll
    for (int u = 0; u < UT; ++u) {
        id[u] = -1;
        wj[u] = g[u] = 0.0f;
        if (lane < k && t0 + u < T) {
            id[u] = ids[(t0 + u) * k + lane];
            wj[u] = w[(t0 + u) * k + lane];
            g[u] = dw[(t0 + u) * k + lane];
        }
#pragma unroll
        for (int i = 0; i < S; ++i) {
            v[u][i] = -INFINITY;
            if (!renorm && 32 * i + lane < E && t0 + u < T) {
                const float x = __half2float(__ushort_as_half(logits[(t0 + u) * E + 32 * i + lane]));
                if (!isfinite(x)) st |= MILO_DEV_NONFINITE;
                if (x == x) v[u][i] = x;          // NaN counts as -inf, as in milo_route
            }
        }
    }
#pragma unroll
    for (int u = 0; u < UT; ++u) {
        if (id[u] < 0 || id[u] >= E) {
            if (lane < k && t0 + u < T) st |= MILO_DEV_BAD_EXPERT_ID;
            id[u] = -1;
            wj[u] = g[u] = 0.0f;
        }
        g[u] *= wj[u];
        s[u] = g[u];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < UT; ++u) s[u] += __shfl_xor_sync(0xFFFFFFFFu, s[u], o);
    if (renorm) {
#pragma unroll
        for (int u = 0; u < UT; ++u) {
            g[u] -= wj[u] * s[u];
#pragma unroll
            for (int i = 0; i < S; ++i) v[u][i] = 0.0f;
        }
    } else {
        float m[UT], den[UT];
#pragma unroll
        for (int u = 0; u < UT; ++u) {
            m[u] = v[u][0];
#pragma unroll
            for (int i = 1; i < S; ++i) m[u] = fmaxf(m[u], v[u][i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < UT; ++u) m[u] = fmaxf(m[u], __shfl_xor_sync(0xFFFFFFFFu, m[u], o));
#pragma unroll
        for (int u = 0; u < UT; ++u) {
            den[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                v[u][i] = 32 * i + lane < E ? expf(v[u][i] - m[u]) : 0.0f;
                den[u] += v[u][i];
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < UT; ++u) den[u] += __shfl_xor_sync(0xFFFFFFFFu, den[u], o);
#pragma unroll
        for (int u = 0; u < UT; ++u) {
            const float c = -s[u] / den[u];
#pragma unroll
            for (int i = 0; i < S; ++i) v[u][i] *= c;
        }
    }
    for (int j = 0; j < k; ++j) {
#pragma unroll
        for (int u = 0; u < UT; ++u) {
            const int e = __shfl_sync(0xFFFFFFFFu, id[u], j);
            const float ge = __shfl_sync(0xFFFFFFFFu, g[u], j);
#pragma unroll
            for (int i = 0; i < S; ++i)
                if (32 * i + lane == e) v[u][i] += ge;
        }
    }
#pragma unroll
    for (int u = 0; u < UT; ++u)
#pragma unroll
        for (int i = 0; i < S; ++i)
            if (32 * i + lane < E && t0 + u < T) dl[(t0 + u) * E + 32 * i + lane] = from_f32<TO>(v[u][i], st);
    flag(dev_status, st);
}

struct RouteGradArgs {
    const uint16_t* logits;
    const int32_t* ids;
    const float *w, *dw;
    int T, E, k, renorm;
    void* dl;
    int32_t* dev_status;
};

template <typename TO, int S, int UT>
static cudaError_t run_route_grad_s(const RouteGradArgs& a, cudaStream_t s) {
    constexpr int kTok = kRgThreads / 32 * UT;
    return launch_pdl(route_grad_kernel<TO, S, UT>, dim3((a.T + kTok - 1) / kTok), dim3(kRgThreads), 0, s, a.logits,
                      a.ids, a.w, a.dw, a.T, a.E, a.k, a.renorm, static_cast<TO*>(a.dl), a.dev_status);
}

// One token per warp while the tokens do not fill the GPU's warps, four after
// (two where a lane holds eight experts).
template <typename TO>
static cudaError_t run_route_grad(const RouteGradArgs& a, cudaStream_t s) {
    const bool few = a.T < 148 * 32;
    if (a.E <= 32) return few ? run_route_grad_s<TO, 1, 1>(a, s) : run_route_grad_s<TO, 1, 4>(a, s);
    if (a.E <= 64) return few ? run_route_grad_s<TO, 2, 1>(a, s) : run_route_grad_s<TO, 2, 4>(a, s);
    if (a.E <= 128) return few ? run_route_grad_s<TO, 4, 1>(a, s) : run_route_grad_s<TO, 4, 4>(a, s);
    return few ? run_route_grad_s<TO, 8, 1>(a, s) : run_route_grad_s<TO, 8, 2>(a, s);
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
    const RouteGradArgs a = {logits, topk_ids, topk_w, dw, T, E, k, renorm ? 1 : 0, dlogits, dev_status};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dl_dt == MILO_F32   ? run_route_grad<float>(a, st)
                          : dl_dt == MILO_F16 ? run_route_grad<__half>(a, st)
                                              : run_route_grad<__nv_bfloat16>(a, st);
    return check_cuda(e, "milo_route_backward");
}
