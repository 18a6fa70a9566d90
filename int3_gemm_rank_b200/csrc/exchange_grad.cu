// exchange_grad.cu -- gradients of milo_dispatch and milo_combine with router
// weights, and of the router's softmax weights (milo_route_backward).
//
// With f = t*k + j, p = inv_perm[f]:
//     combine_backward:   dys[p] = w[f] dy[t],           dw[f] = <dy[t], ys[p]>
//     dispatch_backward:  dx[t] = sum_j w[f] dxs[p],     dw[f] = <dxs[p], x[t]>
// One pass over the rows gives both results: a group of threads owns a token,
// keeps its k partial dot products in fp32 registers over the row and adds
// them by a fixed tree, so the result does not depend on timing.
#include <cuda_runtime.h>

#include <string>

#include "milo_exchange.cuh"
#include "milo_host.h"

namespace milo {

constexpr int kGThreads = 256;

// One block per token.  COMBINE: src = dy [T, H], other = ys, out = dys;
// else src = dxs, other = x, out = dx.  KM: slots a token may have (8 or 16).
template <typename TI, typename TO, int V, int KM, bool COMBINE>
__global__ void __launch_bounds__(kGThreads) exchange_grad_kernel(const ExchangeParams p) {
    __shared__ float part[kGThreads / 32][KM];
    grid_dep_launch();
    grid_dep_wait();
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rows = p.T * p.k;
    int32_t st = 0;
    int r[KM];
    float w[KM], dot[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) {
        r[j] = -1;
        w[j] = 0.0f;
        dot[j] = 0.0f;
        if (j < p.k) {
            r[j] = slot_row(p.inv_perm[t * p.k + j], rows, st);
            w[j] = p.w[t * p.k + j];
        }
    }
    for (uint32_t c = threadIdx.x; c < p.nv; c += kGThreads) {
        const RowVec<TI, V> tok = load_vec<TI, V>(COMBINE ? p.src : p.other, t, p.H, c);
        float acc[V];
#pragma unroll
        for (int q = 0; q < V; ++q) acc[q] = 0.0f;
#pragma unroll
        for (int j0 = 0; j0 < KM; j0 += 8) {
            RowVec<TI, V> v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (r[j0 + j] >= 0) v[j] = load_vec<TI, V>(COMBINE ? p.other : p.src, r[j0 + j], p.H, c);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (r[j0 + j] >= 0) {
                    RowVec<TO, V> o;
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        const float a = to_f32(tok.v[q]), b = to_f32(v[j].v[q]);
                        dot[j0 + j] = fmaf(a, b, dot[j0 + j]);
                        if constexpr (COMBINE) o.v[q] = from_f32<TO>(w[j0 + j] * a, st);
                        else acc[q] = fmaf(w[j0 + j], b, acc[q]);
                    }
                    if constexpr (COMBINE) store_vec<TO, V>(p.out, r[j0 + j], p.H, c, o);
                }
        }
        if constexpr (!COMBINE) {
            RowVec<TO, V> o;
#pragma unroll
            for (int q = 0; q < V; ++q) o.v[q] = from_f32<TO>(acc[q], st);
            store_vec<TO, V>(p.out, t, p.H, c, o);
        }
    }
#pragma unroll
    for (int j = 0; j < KM; ++j)
        if (j < p.k) {
            float d = dot[j];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
            if (lane == 0) part[warp][j] = d;
        }
    __syncthreads();
    if (threadIdx.x < p.k) {
        float d = 0.0f;
#pragma unroll
        for (int q = 0; q < kGThreads / 32; ++q) d += part[q][threadIdx.x];
        p.dw[t * p.k + threadIdx.x] = d;      // 0 for a dropped slot
    }
    flag(p.dev_status, st);
}

template <typename TI, typename TO, int V, bool COMBINE>
static cudaError_t run_grad(const ExchangeParams& p, cudaStream_t s) {
    return launch_pdl(p.k <= 8 ? exchange_grad_kernel<TI, TO, V, 8, COMBINE> : exchange_grad_kernel<TI, TO, V, 16, COMBINE>,
                      dim3(static_cast<unsigned>(p.T)), dim3(kGThreads), 0, s, p);
}

template <typename TI, typename TO>
static cudaError_t run_grad_v(const ExchangeParams& p, int vec, bool combine, cudaStream_t s) {
    if (vec == 8) return combine ? run_grad<TI, TO, 8, true>(p, s) : run_grad<TI, TO, 8, false>(p, s);
    return combine ? run_grad<TI, TO, 1, true>(p, s) : run_grad<TI, TO, 1, false>(p, s);
}

template <typename TI>
static cudaError_t run_grad_o(const ExchangeParams& p, const ExchangeTypes& t, bool combine, cudaStream_t s) {
    if (t.out == MILO_F32) return run_grad_v<TI, float>(p, t.vec, combine, s);
    if (t.out == MILO_F16) return run_grad_v<TI, __half>(p, t.vec, combine, s);
    return run_grad_v<TI, __nv_bfloat16>(p, t.vec, combine, s);
}

cudaError_t launch_exchange_grad(const ExchangeParams& p, const ExchangeTypes& t, bool combine, cudaStream_t s) {
    if (t.in == MILO_F32) return run_grad_o<float>(p, t, combine, s);
    if (t.in == MILO_F16) return run_grad_o<__half>(p, t, combine, s);
    return run_grad_o<__nv_bfloat16>(p, t, combine, s);
}

// ---------------------------------------------------------------------------
// router weights
// ---------------------------------------------------------------------------

constexpr int kRgThreads = 256;

// Gradient of the top-k softmax weights, one warp per token:
//     s = sum_j w_j dw_j
//     renormalised:  dl[e_j] = w_j (dw_j - s),  0 elsewhere
//     full softmax:  dl[e] = [e = e_j] w_j dw_j - p_e s,  p = softmax(l)
// (the Jacobian of a softmax q is q_i ([i = l] - q_l); the renormalised one
// runs over the picked experts only).  Lane j holds pick j; lanes then own
// experts 32 i + lane.
template <typename TO>
__global__ void __launch_bounds__(kRgThreads)
route_grad_kernel(const uint16_t* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ w,
                  const float* __restrict__ dw, int T, int E, int k, int renorm, TO* __restrict__ dl,
                  int32_t* __restrict__ dev_status) {
    constexpr int kSlots = (MILO_MAX_EXPERTS + 31) / 32;
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const long long t = static_cast<long long>(blockIdx.x) * (kRgThreads / 32) + (threadIdx.x >> 5);
    if (t >= T) return;
    int32_t st = 0;
    int id = -1;
    float wj = 0.0f, g = 0.0f;
    if (lane < k) {
        id = ids[t * k + lane];
        if (id < 0 || id >= E) {
            st |= MILO_DEV_BAD_EXPERT_ID;
            id = -1;
        } else {
            wj = w[t * k + lane];
            g = wj * dw[t * k + lane];
        }
    }
    float s = g;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    float v[kSlots];
    if (renorm) {
        g -= wj * s;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) v[i] = 0.0f;
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            const int e = 32 * i + lane;
            v[i] = -INFINITY;
            if (e < E) {
                const float x = __half2float(__ushort_as_half(logits[t * E + e]));
                if (!isfinite(x)) st |= MILO_DEV_NONFINITE;
                if (x == x) v[i] = x;              // NaN counts as -inf, as in milo_route
            }
            m = fmaxf(m, v[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        float den = 0.0f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            v[i] = 32 * i + lane < E ? expf(v[i] - m) : 0.0f;
            den += v[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xFFFFFFFFu, den, o);
        const float c = -s / den;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) v[i] *= c;
    }
    for (int j = 0; j < k; ++j) {
        const int e = __shfl_sync(0xFFFFFFFFu, id, j);
        const float ge = __shfl_sync(0xFFFFFFFFu, g, j);
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
            if (32 * i + lane == e) v[i] += ge;
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
        if (32 * i + lane < E) dl[t * E + 32 * i + lane] = from_f32<TO>(v[i], st);
    flag(dev_status, st);
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
    const dim3 grid((T + kRgThreads / 32 - 1) / (kRgThreads / 32)), block(kRgThreads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dl_dt == MILO_F32)
        e = launch_pdl(route_grad_kernel<float>, grid, block, 0, st, logits, topk_ids, topk_w, dw, T, E, k,
                       renorm ? 1 : 0, static_cast<float*>(dlogits), dev_status);
    else if (dl_dt == MILO_F16)
        e = launch_pdl(route_grad_kernel<__half>, grid, block, 0, st, logits, topk_ids, topk_w, dw, T, E, k,
                       renorm ? 1 : 0, static_cast<__half*>(dlogits), dev_status);
    else
        e = launch_pdl(route_grad_kernel<__nv_bfloat16>, grid, block, 0, st, logits, topk_ids, topk_w, dw, T, E, k,
                       renorm ? 1 : 0, static_cast<__nv_bfloat16*>(dlogits), dev_status);
    return check_cuda(e, "milo_route_backward");
}
