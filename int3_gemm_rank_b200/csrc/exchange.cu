// exchange.cu -- token rows into expert order (milo_dispatch), and the host side
// of the way back and of the gradients (exchange_rows.cuh).
//
// "MiLo: Efficient Quantized MoE Inference with Mixture of Low-Rank
// Compensators", "Background": an MoE layer sends each token to a subset of
// its experts and mixes their outputs with the router's weights.  With f =
// t*k + j the flat slot of token t's j-th pick and p = inv_perm[f] its row in
// expert order: xs[p] = w[f] x[t] (w optional).  The kernel walks the tokens,
// not the expert rows, so it reads each token row once for its k copies.
// Bound by memory: T H elements read, T k H written.  Measured (B200, bf16):
// 8192 x 2048, k 6, 39.4 us = 0.91 of the measured copy rate; 8192 x 4096, k 2,
// 37.9 us = 0.81 (four groups of columns a thread 39.5, the rows through
// shared memory 37.9 and, k 6, 46).
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "milo_exchange.cuh"
#include "milo_host.h"

namespace milo {

constexpr int kXThreads = 256;

// Rows of whole 16-byte pieces: a thread takes U groups of eight columns, all
// loaded before the first store.  (Other rows: exchange_rows.cuh.)
template <typename TI, typename TO, int U>
__global__ void __launch_bounds__(kXThreads) dispatch_kernel(const ExchangeParams p) {
    grid_dep_launch();
    grid_dep_wait();
    const long long i0 = static_cast<long long>(blockIdx.x) * (kXThreads * U) + threadIdx.x;
    const int rows = p.T * p.k;
    int32_t st = 0;
    int t[U], c[U];
    float x[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long i = i0 + u * kXThreads;
        t[u] = -1;
        if (i < static_cast<long long>(p.T) * p.nv) {
            t[u] = p.wide ? static_cast<int>(i / p.nv)
                          : static_cast<int>(fast_div(static_cast<uint32_t>(i), p.div_m, p.div_s));
            c[u] = static_cast<int>(i - static_cast<long long>(t[u]) * p.nv) * 8;
            load8<TI>(static_cast<const TI*>(p.src) + static_cast<long long>(t[u]) * p.H + c[u], x[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (t[u] < 0) continue;
        for (int j = 0; j < p.k; ++j) {
            const int f = t[u] * p.k + j;
            const int r = slot_row(p.inv_perm[f], rows, st);
            if (r < 0) continue;
            const float w = p.w ? p.w[f] : 1.0f;
            float o[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = w * x[u][q];
            store8<TO>(static_cast<TO*>(p.out) + static_cast<long long>(r) * p.H + c[u], o, st);
        }
    }
    flag(p.dev_status, st);
}

template <typename TI, typename TO>
static cudaError_t run_dispatch(const ExchangeParams& p, cudaStream_t s) {
    constexpr int U = 2;
    const long long blocks = (static_cast<long long>(p.T) * p.nv + kXThreads * U - 1) / (kXThreads * U);
    return launch_pdl(dispatch_kernel<TI, TO, U>, dim3(static_cast<unsigned>(blocks)), dim3(kXThreads), 0, s, p);
}

cudaError_t launch_dispatch(const ExchangeParams& p, const ExchangeTypes& t, cudaStream_t s) {
    if (!t.aligned) return launch_dispatch_rows(p, t, s);
    auto by_out = [&](auto in) {
        using TI = decltype(in);
        if (t.out == MILO_F32) return run_dispatch<TI, float>(p, s);
        if (t.out == MILO_F16) return run_dispatch<TI, __half>(p, s);
        return run_dispatch<TI, __nv_bfloat16>(p, s);
    };
    if (t.in == MILO_F32) return by_out(float{});
    if (t.in == MILO_F16) return by_out(__half{});
    return by_out(__nv_bfloat16{});
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
    // the kernels' blocks, 256 vectors of eight columns each at the least, stay a 31-bit count
    if (static_cast<long long>(T) * H > (1LL << 38))
        return fail(MILO_ERR_UNSUPPORTED_SHAPE, f + ": T*H above 2^38");
    return MILO_OK;
}

static bool exchange_aligned(int H, std::initializer_list<const void*> ptrs) {
    if (H % 8) return false;
    for (const void* q : ptrs)
        if (q && !aligned(q, 16)) return false;
    return true;
}

static void exchange_index(ExchangeParams& p) {
    p.nv = static_cast<uint32_t>((p.H + 7) / 8);
    uint32_t s = 0;
    while ((1ULL << s) < p.nv) ++s;
    p.div_s = s;
    p.div_m = static_cast<uint32_t>(((1ULL << 32) * ((1ULL << s) - p.nv)) / p.nv + 1);
    p.wide = static_cast<long long>(p.T) * p.nv >= (1LL << 31);
}

// Addresses: rows at their elements, indices, weights and status at 32-bit words.
static milo_status check_addresses(const char* what, std::initializer_list<std::pair<const void*, milo_dtype>> rows,
                                   std::initializer_list<const void*> words) {
    for (const auto& r : rows)
        if (r.first && !aligned(r.first, dtype_size(r.second)))
            return fail(MILO_ERR_INVALID_ARG, std::string(what) + ": rows must be aligned to their elements");
    for (const void* q : words)
        if (!aligned(q, 4))
            return fail(MILO_ERR_INVALID_ARG,
                        std::string(what) + ": inv_perm, w, dw and dev_status must be aligned to 4 bytes");
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
    if ((s = check_addresses("milo_dispatch", {{x, x_dt}, {xs, xs_dt}}, {inv_perm, w, dev_status})) != MILO_OK) return s;
    const ExchangeTypes ty{x_dt, xs_dt, exchange_aligned(H, {x, xs})};
    ExchangeParams p = {x, nullptr, inv_perm, w, xs, nullptr, dev_status, T, k, H, 0, 0, 0, 0};
    exchange_index(p);
    return check_cuda(launch_dispatch(p, ty, static_cast<cudaStream_t>(stream)), "milo_dispatch");
}

extern "C" milo_status milo_combine(const void* ys, milo_dtype ys_dt, int32_t T, int32_t k, int32_t H,
                                    const int32_t* inv_perm, const float* w, const void* residual, void* y,
                                    milo_dtype y_dt, int32_t* dev_status, void* stream) {
    clear_error();
    milo_status s = check_exchange("milo_combine", ys_dt, y_dt, T, k, H);
    if (s != MILO_OK) return s;
    if (T == 0) return MILO_OK;
    if (!ys || !y || !inv_perm) return fail(MILO_ERR_INVALID_ARG, "milo_combine: NULL pointer");
    if ((s = check_addresses("milo_combine", {{ys, ys_dt}, {y, y_dt}, {residual, y_dt}}, {inv_perm, w, dev_status})) != MILO_OK)
        return s;
    const ExchangeTypes ty{ys_dt, y_dt, exchange_aligned(H, {ys, y, residual})};
    ExchangeParams p = {ys, residual, inv_perm, w, y, nullptr, dev_status, T, k, H, 0, 0, 0, 0};
    exchange_index(p);
    return check_cuda(launch_combine_rows(p, ty, static_cast<cudaStream_t>(stream)), "milo_combine");
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
    if ((s = check_addresses("milo_dispatch_backward", {{dxs, dxs_dt}, {dx, dx_dt}, {dw ? x : nullptr, dxs_dt}},
                             {inv_perm, w, dw, dev_status})) != MILO_OK)
        return s;
    const ExchangeTypes ty{dxs_dt, dx_dt, exchange_aligned(H, {dxs, dx, dw ? x : nullptr})};
    ExchangeParams p = {dxs, nullptr, inv_perm, w, dx, dw, dev_status, T, k, H, 0, 0, 0, 0};
    exchange_index(p);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // without a weight gradient this is the combine of the gradients' rows
    if (!dw) return check_cuda(launch_combine_rows(p, ty, st), "milo_dispatch_backward");
    p.other = x;
    return check_cuda(launch_dispatch_grad(p, ty, st), "milo_dispatch_backward");
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
    if ((s = check_addresses("milo_combine_backward", {{dy, dy_dt}, {dys, dys_dt}, {dw ? ys : nullptr, dy_dt}},
                             {inv_perm, w, dw, dev_status})) != MILO_OK)
        return s;
    const ExchangeTypes ty{dy_dt, dys_dt, exchange_aligned(H, {dy, dys, dw ? ys : nullptr})};
    ExchangeParams p = {dy, nullptr, inv_perm, w, dys, dw, dev_status, T, k, H, 0, 0, 0, 0};
    exchange_index(p);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // without a weight gradient this is the dispatch of the output's gradient
    if (!dw) return check_cuda(launch_dispatch(p, ty, st), "milo_combine_backward");
    p.other = ys;
    return check_cuda(launch_combine_grad(p, ty, st), "milo_combine_backward");
}
