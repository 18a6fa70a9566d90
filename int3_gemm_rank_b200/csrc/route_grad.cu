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
// and every L-th pick each, so a warp takes 32 / L tokens and every reduction
// has log2 L steps; the picks meet their experts in shared memory.  What
// bounds it is each warp's one chain of loads, shuffles and shared memory: 65536 x
// 64, k 6, took 18.7 us with a warp per token, 11 us with the picks compared in
// registers, and takes 9.5 us (0.48 of the measured copy rate) so, with 46% of the
// issue slots taken and warps waiting for global (9.5 of 24 cycles an issue) and
// shared memory (9.4).
template <typename TO, int L, int KM, bool VEC>
__global__ void __launch_bounds__(kRgThreads) route_grad_kernel(const RouteGradArgs p) {
    constexpr int kTok = kRgThreads / L, kRow = 8 * L + 4;
    constexpr int kPicks = (KM + L - 1) / L;              // of a lane
    __shared__ __align__(16) float rows[kTok][kRow];
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, sub = threadIdx.x % L;
    const long long i = static_cast<long long>(blockIdx.x) * kTok + threadIdx.x / L;
    const bool in = i < p.T;                              // the last block may be part empty
    const long long t = in ? i : p.T - 1;
    const int E = p.E, k = p.k;
    // the lane's experts: eight in a row, or every L-th where rows do not start on
    // 16-byte boundaries
    constexpr int step = VEC ? 1 : L;
    const int e0 = sub * (VEC ? 8 : 1);
    int32_t st = 0;
    float v[8], g[kPicks], wj[kPicks];
    int id[kPicks];
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < kPicks; ++r) {
        const int j = sub + r * L;
        id[r] = -1;
        g[r] = wj[r] = 0.0f;
        if (j < k) {
            id[r] = p.ids[t * k + j];
            wj[r] = p.w[t * k + j];
            g[r] = p.dw[t * k + j];
            if (id[r] < 0 || id[r] >= E) {
                st |= MILO_DEV_BAD_EXPERT_ID;
                id[r] = -1;
                g[r] = wj[r] = 0.0f;
            }
        }
    }
    if (!p.renorm) {
        const uint16_t* l = p.logits + t * E + e0;
        if constexpr (VEC) {
            if (e0 < E) {
                load8<__half>(l, v);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = -INFINITY;
            }
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = e0 + q * step < E ? __half2float(__ushort_as_half(l[q * step])) : -INFINITY;
        }
    }
#pragma unroll
    for (int r = 0; r < kPicks; ++r) {
        g[r] *= wj[r];
        s += g[r];
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (p.renorm) {
#pragma unroll
        for (int r = 0; r < kPicks; ++r) g[r] -= wj[r] * s;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = 0.0f;
    } else {
        bool ok = true;
        float m = -INFINITY, den = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            ok = ok && (fabsf(v[q]) <= 65504.0f || e0 + q * step >= E);
            m = fmaxf(m, v[q]);                           // a NaN counts as -inf, as in milo_route
        }
        if (!ok) {
            st |= MILO_DEV_NONFINITE;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (v[q] != v[q]) v[q] = -INFINITY;
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            v[q] = __expf(v[q] - m);
            den += v[q];
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) den += __shfl_xor_sync(0xFFFFFFFFu, den, o);
        const float c = -s / den;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] *= c;
    }
    float* row = rows[threadIdx.x / L];
    if constexpr (VEC) {
        reinterpret_cast<float4*>(row + e0)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(row + e0)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) row[e0 + q * step] = v[q];
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kPicks; ++r) {
        // picks of a token are distinct (milo_route's); two alike would be added one
        // after the other, lowest first
        const unsigned same = __match_any_sync(0xFFFFFFFFu, id[r] >= 0 ? (lane / L) << 16 | id[r] : -1 - lane);
        unsigned left = same;
        bool mine = __ffs(left) - 1 == lane;
        while (true) {
            if (mine && id[r] >= 0) row[id[r]] += g[r];
            __syncwarp();
            left &= left - 1;
            if (!__any_sync(0xFFFFFFFFu, left != 0)) break;
            mine = left != 0 && __ffs(left) - 1 == lane;
        }
    }
    if constexpr (VEC) {
        const float4 a = reinterpret_cast<const float4*>(row + e0)[0], b = reinterpret_cast<const float4*>(row + e0)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = row[e0 + q * step];
    }
    if (in) {
        TO* d = static_cast<TO*>(p.dl) + t * E + e0;
        if constexpr (VEC) {
            if (e0 < E) store8<TO>(d, v, st);
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (e0 + q * step < E) d[q * step] = from_f32<TO>(v[q], st);
        }
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
    if ((!renorm && !aligned(logits, 2)) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(dw, 4) || !aligned(dev_status, 4))
        return fail(MILO_ERR_INVALID_ARG,
                    "milo_route_backward: logits, topk_ids, topk_w, dw and dev_status must be aligned to their elements");
    const int vec = E % 8 == 0 && aligned(logits, 16) && aligned(dlogits, 16);
    const RouteGradArgs a = {logits, topk_ids, topk_w, dw, T, E, k, renorm ? 1 : 0, vec, dlogits, dev_status};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dl_dt == MILO_F32   ? run_route_grad<float>(a, st)
                          : dl_dt == MILO_F16 ? run_route_grad<__half>(a, st)
                                              : run_route_grad<__nv_bfloat16>(a, st);
    return check_cuda(e, "milo_route_backward");
}
