// dense_few.cu -- the dense 16-bit projection for a handful of tokens (decode):
// y = act(x W^T + b) + r with x [M <= 16, K], W [N, K] (see dense.cu).
//
// Bound by the weight's bytes: every element of W is used once per token, so
// the kernel is a stream of W through the registers into mma.sync (m16n8k16,
// fp32), with no shared memory on the way.  A block owns 16 rows of W, its
// warps share K in steps of 32; a lane's A fragments of two k16 steps are 16
// contiguous bytes of two rows (the k order inside a step is free as long as x
// uses the same), so W and x come by 16-byte loads, S steps of them in flight
// per lane: each step's registers are loaded anew as soon as its product is
// issued.  The warps' partial sums meet in shared memory
// in warp order.  (The tcgen05 tile of 16 columns, fed by TMA and split over a
// cluster, took 26 us for 1 x 4096 x 4096 bf16.)
#include <cuda_runtime.h>

#include "milo_dense.cuh"
#include "milo_host.h"

namespace milo {

constexpr int kFewRows = 16;                // rows of W per block

struct DenseFew {
    const uint16_t *x, *W;
    int M, N, K, bf16;
    const void *bias, *residual;
    void *y, *z;
    int act, y_dt;
    int32_t* dev_status;
};

__device__ __forceinline__ void mma16816_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT tiles of 8 tokens; WARPS warps share K.
template <bool BF16, int NT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) dense_few_kernel(const DenseFew p) {
    constexpr int S = NT == 1 ? 8 : 4;          // k32 steps in flight
    __shared__ float part[WARPS][NT * 8][kFewRows + 1];
    grid_dep_launch();
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int n0 = blockIdx.x * kFewRows;
    const bool r0 = n0 + g < p.N, r1 = n0 + g + 8 < p.N;
    const uint16_t* w0 = p.W + static_cast<size_t>(r0 ? n0 + g : 0) * p.K + 8 * c;
    const uint16_t* w1 = p.W + static_cast<size_t>(r1 ? n0 + g + 8 : 0) * p.K + 8 * c;
    const uint16_t* xr[NT];
    bool xin[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        xin[t] = 8 * t + g < p.M;
        xr[t] = p.x + static_cast<size_t>(xin[t] ? 8 * t + g : 0) * p.K + 8 * c;
    }
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 a[S], b[S], xv[S][NT];
    auto load = [&](int s, int k) {
        const bool in = k + 8 * c < p.K;                  // K is a multiple of 8
        a[s] = in && r0 ? __ldcs(reinterpret_cast<const uint4*>(w0 + k)) : zero;
        b[s] = in && r1 ? __ldcs(reinterpret_cast<const uint4*>(w1 + k)) : zero;
#pragma unroll
        for (int t = 0; t < NT; ++t) xv[s][t] = in && xin[t] ? *reinterpret_cast<const uint4*>(xr[t] + k) : zero;
    };
    constexpr int kStep = 32 * WARPS;
#pragma unroll
    for (int s = 0; s < S; ++s) load(s, 32 * warp + s * kStep);
    for (int k0 = 32 * warp; k0 < p.K; k0 += S * kStep)
#pragma unroll
        for (int s = 0; s < S; ++s) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if constexpr (BF16) {
                    mma16816_bf16(acc[t], a[s].x, b[s].x, a[s].y, b[s].y, xv[s][t].x, xv[s][t].y);
                    mma16816_bf16(acc[t], a[s].z, b[s].z, a[s].w, b[s].w, xv[s][t].z, xv[s][t].w);
                } else {
                    mma16816(acc[t], a[s].x, b[s].x, a[s].y, b[s].y, xv[s][t].x, xv[s][t].y);
                    mma16816(acc[t], a[s].z, b[s].z, a[s].w, b[s].w, xv[s][t].z, xv[s][t].w);
                }
            }
            load(s, k0 + (S + s) * kStep);
        }
    // acc[t][i]: W row g + 8 (i >> 1), token 8 t + 2 c + (i & 1)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[warp][8 * t + 2 * c + (i & 1)][g + 8 * (i >> 1)] = acc[t][i];
    __syncthreads();
    int32_t st = 0;
    for (int i = threadIdx.x; i < NT * 8 * kFewRows; i += 32 * WARPS) {
        const int m = i / kFewRows, r = i % kFewRows;
        if (m >= p.M || n0 + r >= p.N) continue;
        float v[1] = {0.0f};
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v[0] += part[w][m][r];
        const size_t o = static_cast<size_t>(m) * p.N + n0 + r;
        if (p.bias) v[0] += load16(p.bias, n0 + r, p.bf16);
        if (p.z) static_cast<uint16_t*>(p.z)[o] = round16(v[0], p.bf16, st);
        act_tile(p.act, v);
        if (p.residual) v[0] += load_any(p.residual, o, p.y_dt);
        store_any(p.y, o, p.y_dt, v[0], st);
    }
    flag(p.dev_status, st);
}

template <bool BF16, int NT>
static cudaError_t run_few(const DenseFew& p, cudaStream_t s) {
    const int blocks = (p.N + kFewRows - 1) / kFewRows;
    // blocks that do not fill the SMs take K with twice the warps
    if (blocks < 148) return launch_pdl(dense_few_kernel<BF16, NT, 16>, dim3(blocks), dim3(512), 0, s, p);
    return launch_pdl(dense_few_kernel<BF16, NT, 8>, dim3(blocks), dim3(256), 0, s, p);
}

milo_status launch_dense_few(const DenseGemm& g, const char* what, cudaStream_t s) {
    const DenseFew p = {static_cast<const uint16_t*>(g.a), static_cast<const uint16_t*>(g.b), g.P, g.Q, g.C, g.bf16,
                        g.bias, g.residual, g.y, g.z, g.act, g.y_dt, g.dev_status};
    cudaError_t e;
    if (g.bf16) e = g.P <= 8 ? run_few<true, 1>(p, s) : run_few<true, 2>(p, s);
    else e = g.P <= 8 ? run_few<false, 1>(p, s) : run_few<false, 2>(p, s);
    return check_cuda(e, what);
}

}  // namespace milo
