// exchange.cu -- token rows into expert order and back (milo_dispatch,
// milo_combine, and their gradients' host side).
//
// "MiLo: Efficient Quantized MoE Inference with Mixture of Low-Rank
// Compensators", "Background": an MoE layer sends each token to a subset of
// its experts and mixes their outputs with the router's weights.  With f =
// t*k + j the flat slot of token t's j-th pick and p = inv_perm[f] its row in
// expert order:
//     dispatch:  xs[p] = w[f] x[t]               (w optional)
//     combine:   y[t]  = r[t] + sum_j w[f] ys[p]  (w, r optional)
// Both walk the tokens, not the expert rows: dispatch then reads each token
// row once for its k copies, and combine writes each output row once, its
// sum in slot order in fp32.
//
// Bound by memory: dispatch moves T H + T k H elements, combine T k H + T H
// (and T H of residual).
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "milo_exchange.cuh"
#include "milo_host.h"

namespace milo {

constexpr int kXThreads = 256;

// One thread per (token, vector of V columns).
template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(kXThreads) dispatch_kernel(const ExchangeParams p) {
    grid_dep_launch();
    grid_dep_wait();
    const long long i = static_cast<long long>(blockIdx.x) * kXThreads + threadIdx.x;
    if (i >= static_cast<long long>(p.T) * p.nv) return;
    const int t = p.wide ? static_cast<int>(i / p.nv) : static_cast<int>(fast_div(static_cast<uint32_t>(i), p.div_m, p.div_s));
    const uint32_t c = static_cast<uint32_t>(i - static_cast<long long>(t) * p.nv);
    const int rows = p.T * p.k;
    int32_t st = 0;
    const RowVec<TI, V> x = load_vec<TI, V>(p.src, t, p.H, c);
    for (int j = 0; j < p.k; ++j) {
        const int f = t * p.k + j;
        const int r = slot_row(p.inv_perm[f], rows, st);
        if (r < 0) continue;
        RowVec<TO, V> o;
        const float w = p.w ? p.w[f] : 1.0f;
#pragma unroll
        for (int q = 0; q < V; ++q) o.v[q] = from_f32<TO>(w * to_f32(x.v[q]), st);
        store_vec<TO, V>(p.out, r, p.H, c, o);
    }
    flag(p.dev_status, st);
}

// One thread per (token, vector of V columns): eight slots' rows in flight,
// added in slot order.
template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(kXThreads) combine_rows_kernel(const ExchangeParams p) {
    grid_dep_launch();
    grid_dep_wait();
    const long long i = static_cast<long long>(blockIdx.x) * kXThreads + threadIdx.x;
    if (i >= static_cast<long long>(p.T) * p.nv) return;
    const int t = p.wide ? static_cast<int>(i / p.nv) : static_cast<int>(fast_div(static_cast<uint32_t>(i), p.div_m, p.div_s));
    const uint32_t c = static_cast<uint32_t>(i - static_cast<long long>(t) * p.nv);
    const int rows = p.T * p.k;
    int32_t st = 0;
    float acc[V];
#pragma unroll
    for (int q = 0; q < V; ++q) acc[q] = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        int r[8];
        float w[8];
        RowVec<TI, V> v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[j] = -1;
            if (j0 + j < p.k) {
                const int f = t * p.k + j0 + j;
                r[j] = slot_row(p.inv_perm[f], rows, st);
                w[j] = p.w ? p.w[f] : 1.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (r[j] >= 0) v[j] = load_vec<TI, V>(p.src, r[j], p.H, c);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (r[j] >= 0) {
#pragma unroll
                for (int q = 0; q < V; ++q) acc[q] = fmaf(w[j], to_f32(v[j].v[q]), acc[q]);
            }
    }
    if (p.other) {
        const RowVec<TO, V> res = load_vec<TO, V>(p.other, t, p.H, c);
#pragma unroll
        for (int q = 0; q < V; ++q) acc[q] += to_f32(res.v[q]);
    }
    RowVec<TO, V> o;
#pragma unroll
    for (int q = 0; q < V; ++q) o.v[q] = from_f32<TO>(acc[q], st);
    store_vec<TO, V>(p.out, t, p.H, c, o);
    flag(p.dev_status, st);
}

template <typename TI, typename TO, int V>
static cudaError_t run_exchange(const ExchangeParams& p, bool combine, cudaStream_t s) {
    const long long blocks = (static_cast<long long>(p.T) * p.nv + kXThreads - 1) / kXThreads;
    return launch_pdl(combine ? combine_rows_kernel<TI, TO, V> : dispatch_kernel<TI, TO, V>,
                      dim3(static_cast<unsigned>(blocks)), dim3(kXThreads), 0, s, p);
}

template <typename TI, typename TO>
static cudaError_t run_exchange_v(const ExchangeParams& p, int vec, bool combine, cudaStream_t s) {
    return vec == 8 ? run_exchange<TI, TO, 8>(p, combine, s) : run_exchange<TI, TO, 1>(p, combine, s);
}

template <typename TI>
static cudaError_t run_exchange_o(const ExchangeParams& p, const ExchangeTypes& t, bool combine, cudaStream_t s) {
    if (t.out == MILO_F32) return run_exchange_v<TI, float>(p, t.vec, combine, s);
    if (t.out == MILO_F16) return run_exchange_v<TI, __half>(p, t.vec, combine, s);
    return run_exchange_v<TI, __nv_bfloat16>(p, t.vec, combine, s);
}

cudaError_t launch_exchange(const ExchangeParams& p, const ExchangeTypes& t, bool combine, cudaStream_t s) {
    if (t.in == MILO_F32) return run_exchange_o<float>(p, t, combine, s);
    if (t.in == MILO_F16) return run_exchange_o<__half>(p, t, combine, s);
    return run_exchange_o<__nv_bfloat16>(p, t, combine, s);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

static size_t dtype_size(milo_dtype d) { return d == MILO_F32 ? 4 : 2; }
static bool dtype_ok(milo_dtype d) { return d == MILO_F16 || d == MILO_BF16 || d == MILO_F32; }

// Sizes and types of the four calls.
static milo_status check_exchange(const char* what, milo_dtype in, milo_dtype out, int T, int k, int H) {
    const std::string f = what;
    if (!dtype_ok(in) || !dtype_ok(out)) return fail(MILO_ERR_INVALID_ARG, f + ": bad dtype");
    if (T < 0 || H < 1) return fail(MILO_ERR_INVALID_ARG, f + ": T must be >= 0 and H >= 1");
    if (k < 1 || k > MILO_MAX_TOPK) return fail(MILO_ERR_UNSUPPORTED_SHAPE, f + ": k must be in [1, 16]");
    if (H > kMaxProjK) return fail(MILO_ERR_UNSUPPORTED_SHAPE, f + ": H above 2^24");
    if (static_cast<long long>(T) * k > MILO_MAX_ROWS)
        return fail(MILO_ERR_UNSUPPORTED_SHAPE, f + ": T*k above MILO_MAX_ROWS");
    // one block per 256 elements of the token rows at the least
    if (static_cast<long long>(T) * H > (1LL << 38))
        return fail(MILO_ERR_UNSUPPORTED_SHAPE, f + ": T*H above 2^38");
    return MILO_OK;
}

// The 16-byte path needs rows of whole 16-byte pieces at 16-byte addresses;
// every other width or address goes element by element.
static int exchange_vec(int H, std::initializer_list<const void*> ptrs) {
    if (H % 8) return 1;
    for (const void* q : ptrs)
        if (q && !aligned(q, 16)) return 1;
    return 8;
}

static void exchange_index(ExchangeParams& p, int vec) {
    p.nv = static_cast<uint32_t>(p.H / vec);
    uint32_t s = 0;
    while ((1ULL << s) < p.nv) ++s;
    p.div_s = s;
    p.div_m = static_cast<uint32_t>(((1ULL << 32) * ((1ULL << s) - p.nv)) / p.nv + 1);
    p.wide = static_cast<long long>(p.T) * p.nv >= (1LL << 31);
}

static milo_status check_rows(const char* what, std::initializer_list<std::pair<const void*, milo_dtype>> rows) {
    for (const auto& r : rows)
        if (r.first && !aligned(r.first, dtype_size(r.second)))
            return fail(MILO_ERR_INVALID_ARG, std::string(what) + ": rows must be aligned to their elements");
    return MILO_OK;
}

}  // namespace milo

using namespace milo;

extern "C" milo_status milo_dispatch(const void* x, milo_dtype x_dt, int32_t T, int32_t k, int32_t H,
                                     const int32_t* inv_perm, const float* w, void* xs, milo_dtype xs_dt,
                                     int32_t* dev_status, void* stream) {
    clear_error();
    milo_status s = check_exchange("milo_dispatch", x_dt, xs_dt, T, k, H);
    if (s != MILO_OK) return s;
    if (T == 0) return MILO_OK;
    if (!x || !xs || !inv_perm) return fail(MILO_ERR_INVALID_ARG, "milo_dispatch: NULL pointer");
    if ((s = check_rows("milo_dispatch", {{x, x_dt}, {xs, xs_dt}})) != MILO_OK) return s;
    const ExchangeTypes ty{x_dt, xs_dt, exchange_vec(H, {x, xs})};
    ExchangeParams p = {x, nullptr, inv_perm, w, xs, nullptr, dev_status, T, k, H, 0, 0, 0, 0};
    exchange_index(p, ty.vec);
    return check_cuda(launch_exchange(p, ty, false, static_cast<cudaStream_t>(stream)), "milo_dispatch");
}

extern "C" milo_status milo_combine(const void* ys, milo_dtype ys_dt, int32_t T, int32_t k, int32_t H,
                                    const int32_t* inv_perm, const float* w, const void* residual, void* y,
                                    milo_dtype y_dt, int32_t* dev_status, void* stream) {
    clear_error();
    milo_status s = check_exchange("milo_combine", ys_dt, y_dt, T, k, H);
    if (s != MILO_OK) return s;
    if (T == 0) return MILO_OK;
    if (!ys || !y || !inv_perm) return fail(MILO_ERR_INVALID_ARG, "milo_combine: NULL pointer");
    if ((s = check_rows("milo_combine", {{ys, ys_dt}, {y, y_dt}, {residual, y_dt}})) != MILO_OK) return s;
    const ExchangeTypes ty{ys_dt, y_dt, exchange_vec(H, {ys, y, residual})};
    ExchangeParams p = {ys, residual, inv_perm, w, y, nullptr, dev_status, T, k, H, 0, 0, 0, 0};
    exchange_index(p, ty.vec);
    return check_cuda(launch_exchange(p, ty, true, static_cast<cudaStream_t>(stream)), "milo_combine");
}

extern "C" milo_status milo_dispatch_backward(const void* dxs, milo_dtype dxs_dt, int32_t T, int32_t k, int32_t H,
                                              const int32_t* inv_perm, const float* w, const void* x, void* dx,
                                              milo_dtype dx_dt, float* dw, int32_t* dev_status, void* stream) {
    clear_error();
    milo_status s = check_exchange("milo_dispatch_backward", dxs_dt, dx_dt, T, k, H);
    if (s != MILO_OK) return s;
    if (dw && (!w || !x))
        return fail(MILO_ERR_INVALID_ARG, "milo_dispatch_backward: dw needs the call's w and x");
    if (T == 0) return MILO_OK;
    if (!dxs || !dx || !inv_perm) return fail(MILO_ERR_INVALID_ARG, "milo_dispatch_backward: NULL pointer");
    if ((s = check_rows("milo_dispatch_backward", {{dxs, dxs_dt}, {dx, dx_dt}, {dw ? x : nullptr, dxs_dt}})) != MILO_OK)
        return s;
    const ExchangeTypes ty{dxs_dt, dx_dt, exchange_vec(H, {dxs, dx, dw ? x : nullptr})};
    ExchangeParams p = {dxs, nullptr, inv_perm, w, dx, dw, dev_status, T, k, H, 0, 0, 0, 0};
    exchange_index(p, ty.vec);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // without a weight gradient this is the combine of the gradients' rows
    if (!dw) return check_cuda(launch_exchange(p, ty, true, st), "milo_dispatch_backward");
    p.other = x;
    return check_cuda(launch_exchange_grad(p, ty, false, st), "milo_dispatch_backward");
}

extern "C" milo_status milo_combine_backward(const void* dy, milo_dtype dy_dt, int32_t T, int32_t k, int32_t H,
                                             const int32_t* inv_perm, const float* w, const void* ys, void* dys,
                                             milo_dtype dys_dt, float* dw, int32_t* dev_status, void* stream) {
    clear_error();
    milo_status s = check_exchange("milo_combine_backward", dy_dt, dys_dt, T, k, H);
    if (s != MILO_OK) return s;
    if (dw && (!w || !ys))
        return fail(MILO_ERR_INVALID_ARG, "milo_combine_backward: dw needs the call's w and ys");
    if (T == 0) return MILO_OK;
    if (!dy || !dys || !inv_perm) return fail(MILO_ERR_INVALID_ARG, "milo_combine_backward: NULL pointer");
    if ((s = check_rows("milo_combine_backward", {{dy, dy_dt}, {dys, dys_dt}, {dw ? ys : nullptr, dy_dt}})) != MILO_OK)
        return s;
    const ExchangeTypes ty{dy_dt, dys_dt, exchange_vec(H, {dy, dys, dw ? ys : nullptr})};
    ExchangeParams p = {dy, nullptr, inv_perm, w, dys, dw, dev_status, T, k, H, 0, 0, 0, 0};
    exchange_index(p, ty.vec);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // without a weight gradient this is the dispatch of the output's gradient
    if (!dw) return check_cuda(launch_exchange(p, ty, false, st), "milo_combine_backward");
    p.other = ys;
    return check_cuda(launch_exchange_grad(p, ty, true, st), "milo_combine_backward");
}
