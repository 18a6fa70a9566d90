// dense_few.cu -- the dense 16-bit projection for a handful of tokens (decode):
// y = act(x W^T + b) + r with x [M <= 16, K], W [N, K] (see dense.cu).
//
// Bound by the weight's bytes: every element of W is used once per token, so
// the kernel is a stream of W through the registers into mma.sync (m16n8k16,
// fp32), with no shared memory on the way.  A block owns 16 or 32 rows of W,
// its warps share K in steps of 32; a lane's A fragments of two k16 steps are
// 16 contiguous bytes of two rows (the k order inside a step is free as long
// as x uses the same), so W and x come by 16-byte loads, S steps of them in
// flight per lane: each step's registers are loaded anew as soon as its
// product is issued.  9 to 16 tokens need twice the x per row of W, so their
// blocks take 32 rows.  The warps' partial sums meet in shared memory in warp
// order; where the blocks are few, those of a cluster share K and meet in
// rank order.  Measured (B200, bf16): 1 x 4096 x 4096 7.6 us = 0.68 of the
// measured copy rate, launch included (the tcgen05 tile of 16 columns, split
// over a cluster, 26 us), 1 x 14336 x 4096 21.3 us = 0.84, 16 x 4096 x 4096
// 9.8 us.
#include <cuda_runtime.h>

#include "milo_dense.cuh"
#include "milo_host.h"

namespace milo {


struct DenseFew {
    const uint16_t *x, *W;
    int M, N, K, bf16, cluster;  // cluster: blocks that share K
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

__device__ __forceinline__ void few_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// *p in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ float ld_peer(const float* p, int rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// MT tiles of 16 rows of W, NT tiles of 8 tokens; WARPS warps of `cluster` blocks share K.
template <bool BF16, int MT, int NT, int WARPS, bool CLUSTER>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS) dense_few_kernel(const DenseFew p) {
    // k32 steps of W in flight, as many as 128 registers hold, and of x, which comes
    // from L1 or L2 sooner (SX divides S)
    constexpr int S = NT == 1 ? (CLUSTER ? 6 : 8) : (CLUSTER ? 2 : 4), SX = NT == 1 ? S / 2 : 2;
    constexpr int kRows = 16 * MT;
    __shared__ float part[WARPS][NT * 8][kRows + 1];
    __shared__ float sum[CLUSTER ? NT * 8 : 1][kRows];
    grid_dep_launch();
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int cluster = CLUSTER ? p.cluster : 1;
    const int rank = CLUSTER ? static_cast<int>(blockIdx.x) % cluster : 0;
    const int n0 = (CLUSTER ? static_cast<int>(blockIdx.x) / cluster : static_cast<int>(blockIdx.x)) * kRows;
    const uint16_t *wr[2 * MT], *xr[NT];        // row 8 i + g of the block's, token 8 t + g
    bool win[2 * MT], xin[NT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
        win[i] = n0 + 8 * i + g < p.N;
        wr[i] = p.W + static_cast<size_t>(win[i] ? n0 + 8 * i + g : 0) * p.K + 8 * c;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        xin[t] = 8 * t + g < p.M;
        xr[t] = p.x + static_cast<size_t>(xin[t] ? 8 * t + g : 0) * p.K + 8 * c;
    }
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][t][i] = 0.0f;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 w[S][2 * MT], xv[SX][NT];
    auto load_w = [&](int s, int k) {
        const bool in = k + 8 * c < p.K;                  // K is a multiple of 8
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) w[s][i] = in && win[i] ? __ldcs(reinterpret_cast<const uint4*>(wr[i] + k)) : zero;
    };
    auto load_x = [&](int s, int k) {
        const bool in = k + 8 * c < p.K;
#pragma unroll
        for (int t = 0; t < NT; ++t) xv[s][t] = in && xin[t] ? *reinterpret_cast<const uint4*>(xr[t] + k) : zero;
    };
    const int kstep = 32 * WARPS * cluster, kfirst = 32 * (rank * WARPS + warp);
#pragma unroll
    for (int s = 0; s < S; ++s) {
        load_w(s, kfirst + s * kstep);
        if (s < SX) load_x(s, kfirst + s * kstep);
    }
    for (int k0 = kfirst; k0 < p.K; k0 += S * kstep)
#pragma unroll
        for (int s = 0; s < S; ++s) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint4 a = w[s][2 * m], b = w[s][2 * m + 1], x = xv[s % SX][t];
                    if constexpr (BF16) {
                        mma16816_bf16(acc[m][t], a.x, b.x, a.y, b.y, x.x, x.y);
                        mma16816_bf16(acc[m][t], a.z, b.z, a.w, b.w, x.z, x.w);
                    } else {
                        mma16816(acc[m][t], a.x, b.x, a.y, b.y, x.x, x.y);
                        mma16816(acc[m][t], a.z, b.z, a.w, b.w, x.z, x.w);
                    }
                }
            load_w(s, k0 + (S + s) * kstep);
            load_x(s % SX, k0 + (SX + s) * kstep);
        }
    // acc[m][t][i]: W row 16 m + g + 8 (i >> 1), token 8 t + 2 c + (i & 1)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[warp][8 * t + 2 * c + (i & 1)][16 * m + g + 8 * (i >> 1)] = acc[m][t][i];
    __syncthreads();
    auto block_sum = [&](int m, int r) {
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < WARPS; ++q) v += part[q][m][r];
        return v;
    };
    if constexpr (CLUSTER) {
        for (int i = threadIdx.x; i < NT * 8 * kRows; i += 32 * WARPS) sum[i / kRows][i % kRows] = block_sum(i / kRows, i % kRows);
        few_cluster_sync();
    }
    int32_t st = 0;
    for (int i = threadIdx.x * cluster + rank; i < NT * 8 * kRows; i += 32 * WARPS * cluster) {
        const int m = i / kRows, r = i % kRows;
        if (m >= p.M || n0 + r >= p.N) continue;
        float v[1] = {0.0f};
        if constexpr (CLUSTER) {
            for (int q = 0; q < cluster; ++q) v[0] += ld_peer(&sum[m][r], q);
        } else {
            v[0] = block_sum(m, r);
        }
        const size_t o = static_cast<size_t>(m) * p.N + n0 + r;
        if (p.bias) v[0] += load16(p.bias, n0 + r, p.bf16);
        if (p.z) static_cast<uint16_t*>(p.z)[o] = round16(v[0], p.bf16, st);
        act_tile(p.act, v);
        if (p.residual) v[0] += load_any(p.residual, o, p.y_dt);
        store_any(p.y, o, p.y_dt, v[0], st);
    }
    flag(p.dev_status, st);
    if constexpr (CLUSTER) few_cluster_sync();       // no block leaves while another reads its sums
}

template <bool BF16, int MT, int NT, int WARPS>
static cudaError_t launch_few(const DenseFew& p, int blocks, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * p.cluster));
    cfg.blockDim = dim3(32 * WARPS);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    if constexpr (WARPS == 16)
        if (p.cluster > 1) return cudaLaunchKernelEx(&cfg, dense_few_kernel<BF16, MT, NT, WARPS, true>, p);
    return cudaLaunchKernelEx(&cfg, dense_few_kernel<BF16, MT, NT, WARPS, false>, p);
}

// Blocks that do not fill the SMs take K with twice the warps, and far fewer of
// them in clusters, as long as a warp keeps at least two steps.
template <bool BF16, int MT, int NT>
static cudaError_t run_few(DenseFew p, cudaStream_t s) {
    const int blocks = (p.N + 16 * MT - 1) / (16 * MT);
    p.cluster = 1;
    if (blocks >= 148) return launch_few<BF16, MT, NT, 8>(p, blocks, s);
    while (p.cluster < 8 && blocks * p.cluster * 2 <= 148 && p.K >= 2 * 32 * 16 * p.cluster * 2) p.cluster *= 2;
    return launch_few<BF16, MT, NT, 16>(p, blocks, s);
}

milo_status launch_dense_few(const DenseGemm& g, const char* what, cudaStream_t s) {
    const DenseFew p = {static_cast<const uint16_t*>(g.a), static_cast<const uint16_t*>(g.b), g.P, g.Q, g.C, g.bf16,
                        1, g.bias, g.residual, g.y, g.z, g.act, g.y_dt, g.dev_status};
    cudaError_t e;
    if (g.bf16) e = g.P <= 8 ? run_few<true, 1, 1>(p, s) : run_few<true, 2, 2>(p, s);
    else e = g.P <= 8 ? run_few<false, 1, 1>(p, s) : run_few<false, 2, 2>(p, s);
    return check_cuda(e, what);
}

}  // namespace milo
