// dense_tc.cu -- the dense 16-bit product D[p, q] = sum_c A(p, c) B(q, c) on the
// 5th-generation tensor cores (tcgen05, TMEM), with bias, activation and
// residual in its epilogue (see dense.cu for the three products it serves).
//
// Design (B200):
//   - A work item is a 128 x BN tile of D.  One warp brings 64-deep slices of A
//     and B by 2-D TMA (128-byte swizzle) into a ring of stages, one warp
//     issues tcgen05.mma (M = 128, N = BN, K = 16, fp32 accumulator in TMEM),
//     eight warps turn the finished accumulator into output.
//   - Either operand may lie along c (K-major: a box of 64 c by 128 rows) or
//     along its rows (MN-major: boxes of 64 rows by 64 c); only the boxes'
//     coordinates and the matrix descriptors differ, so W and x are read as
//     they are stored by the forward product and by both gradients.
//   - Many tiles: a persistent grid, two accumulators in TMEM, so that the
//     epilogue of one tile runs under the products of the next.
//   - Few tiles: c is split over the CTAs of a cluster.  The tile's blocks of
//     32 rows by 32 (SWAP: 16) columns are dealt out to the CTAs; each sends its
//     partial blocks to their owners' shared memory, and after a cluster
//     barrier the owners add them in rank order (no workspace, no atomics, the
//     same bits every time).
//   - Few tokens: the operands change places (SWAP), the weight's rows fill
//     the 128 rows of the tile and the tokens its BN columns, so one token
//     costs a tile of 16 columns, not of 128 rows.
//   - Ragged edges need no care in the loads (TMA fills zeros) and are cut in
//     the epilogue's stores.
//   - Every wait is bounded: on a timeout the kernel flags MILO_DEV_TIMEOUT,
//     waits for its copies and products and frees TMEM before it leaves.
#include <cuda.h>
#include <cuda_runtime.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "milo_dense.cuh"
#include "milo_host.h"
#include "milo_tc.cuh"

namespace milo {

constexpr int kDtRows = 128;                 // rows of A in a tile (MMA M)
constexpr int kDtK = 64;                     // c per stage: one 128-byte swizzled row
constexpr int kDtAtom = kDtRows * kDtK * 2;  // bytes of an A stage
constexpr int kDtBox = 64 * kDtK * 2;        // bytes of an MN-major box (64 rows x 64 c)
constexpr int kDtEpiWarps = 8;               // two per TMEM lane quarter, every other block of columns each
constexpr int kDtThreads = 32 * (2 + kDtEpiWarps);   // producer, MMA, epilogue
constexpr int kDtMaxStages = 12;
constexpr int kDtMaxSplit = 8;               // portable cluster size
constexpr int kDtChunk = 32;                 // accumulator columns handled at a time
constexpr int kDtBias = 128;                 // fp32 bias columns, per epilogue warp (its half of 256)

// Output staging of an epilogue warp: 32 rows of 32 elements, 16 bytes apart
// from a multiple of 128 so that 16-byte pieces of a column fall on different
// banks.
constexpr int dense_pitch(int esize) { return 32 * esize + 16; }

struct DenseTc {
    CUtensorMap a_map, b_map;
    int P, Q, C;
    int a_mn, b_mn, bf16;
    int bn, stages, split, kblocks;          // columns of a tile; c slices of 64
    int tiles_p, tiles_q, tiles;
    uint32_t idesc, tmem_cols;
    int bufs;                                // accumulators in TMEM (2: persistent)
    int stage_bytes, staging, off_staging, off_bias, off_bar;
    int vec;                                 // 16-byte output rows
    // epilogue (y, residual and z are [M, N]; SWAP: p is the feature)
    const void *bias, *residual;
    void *y, *z;
    int act, y_dt;
    int32_t* dev_status;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Four floats to the same shared-memory address of CTA `rank` of the cluster.
__device__ __forceinline__ void st_peer4(uint32_t saddr, uint32_t rank, float4 v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// Matrix descriptor of an MN-major operand in the 128-byte swizzled layout:
// rows of 64 elements along MN, 8-c groups 1024 bytes apart, blocks of 64
// elements along MN one box apart.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(kDtBox >> 4) << 16;           // leading byte offset: next 64 rows
    d |= static_cast<uint64_t>(1024 >> 4) << 32;             // stride byte offset: next 8 c
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// Item order: bands of kDtBand row tiles, columns inside a band, the band's
// row tiles fastest, so that the CTAs at work share operand tiles in L2.
constexpr int kDtBand = 16;
__device__ __forceinline__ void dense_tile(const DenseTc& p, int item, int& tp, int& tq) {
    const int per = kDtBand * p.tiles_q;
    const int band = item / per, in = item - band * per;
    const int h = min(kDtBand, p.tiles_p - band * kDtBand);
    tq = in / h;
    tp = band * kDtBand + in - tq * h;
}

// ---------------------------------------------------------------------------
// epilogue of 32 rows (lane = row p) by 32 columns q0.. of D, normal form:
// y[p, q].  v holds the lane's row.  st32 is the warp's staging buffer.
// ---------------------------------------------------------------------------

// The warp's 32 x 32 block between staging rows and global rows p0.., columns
// q0..; 16-byte pieces when p.vec.
template <int DT, bool LOAD>
__device__ __forceinline__ void dense_block(const DenseTc& p, void* g, uint8_t* stg, int p0, int q0, int lane) {
    constexpr int E = DT == MILO_F32 ? 4 : 2, kPitch = dense_pitch(E);
    constexpr int kPieces = 32 * E / 16;              // 16-byte pieces of a row
    constexpr int kRows = 32 / kPieces;               // rows of one pass
    if (p.vec) {
        const int piece = lane % kPieces, r0 = lane / kPieces;
        const bool in = q0 + piece * (16 / E) < p.Q;  // Q is a multiple of a piece here
        uint8_t* gp = static_cast<uint8_t*>(g) + (static_cast<size_t>(p0 + r0) * p.Q + q0) * E + piece * 16;
        uint4 t[32 / kRows];
#pragma unroll
        for (int i = 0; i < 32 / kRows; ++i) {
            if constexpr (LOAD) {
                if (in && p0 + r0 + i * kRows < p.P) t[i] = *reinterpret_cast<const uint4*>(gp + static_cast<size_t>(i) * kRows * p.Q * E);
            } else {
                t[i] = *reinterpret_cast<const uint4*>(stg + (r0 + i * kRows) * kPitch + piece * 16);
            }
        }
#pragma unroll
        for (int i = 0; i < 32 / kRows; ++i) {
            if constexpr (LOAD) {
                *reinterpret_cast<uint4*>(stg + (r0 + i * kRows) * kPitch + piece * 16) = t[i];
            } else {
                if (in && p0 + r0 + i * kRows < p.P) *reinterpret_cast<uint4*>(gp + static_cast<size_t>(i) * kRows * p.Q * E) = t[i];
            }
        }
    } else {
        using T = typename std::conditional<E == 4, uint32_t, uint16_t>::type;
        if (q0 + lane < p.Q) {
            T* gp = static_cast<T*>(g) + static_cast<size_t>(p0) * p.Q + q0 + lane;
            T* sp = reinterpret_cast<T*>(stg) + lane;
            const int n = min(32, p.P - p0);
#pragma unroll 8
            for (int r = 0; r < n; ++r) {
                if constexpr (LOAD) sp[r * (kPitch / E)] = gp[static_cast<size_t>(r) * p.Q];
                else gp[static_cast<size_t>(r) * p.Q] = sp[r * (kPitch / E)];
            }
        }
    }
}

// The lane's 32 values to its staging row, and the block to global memory.
template <int DT>
__device__ __forceinline__ void dense_put(const DenseTc& p, void* g, const float (&v)[32], uint8_t* stg, int p0, int q0,
                                          int lane, int32_t& st) {
    uint8_t* row = stg + lane * dense_pitch(DT == MILO_F32 ? 4 : 2);
    if constexpr (DT == MILO_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            reinterpret_cast<float4*>(row)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack16<DT>(v[2 * i], v[2 * i + 1]);
        if constexpr (DT == MILO_F16) half_range(v, w, st);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<uint4*>(row)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    __syncwarp();
    dense_block<DT, false>(p, g, stg, p0, q0, lane);
    __syncwarp();
}

// v += the block of the residual.
template <int DT>
__device__ __forceinline__ void dense_add(const DenseTc& p, float (&v)[32], uint8_t* stg, int p0, int q0, int lane) {
    dense_block<DT, true>(p, const_cast<void*>(p.residual), stg, p0, q0, lane);
    __syncwarp();
    const uint8_t* row = stg + lane * dense_pitch(DT == MILO_F32 ? 4 : 2);
    if constexpr (DT == MILO_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 t = reinterpret_cast<const float4*>(row)[i];
            v[4 * i] += t.x;
            v[4 * i + 1] += t.y;
            v[4 * i + 2] += t.z;
            v[4 * i + 3] += t.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 t = reinterpret_cast<const uint4*>(row)[i];
            const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
            for (int q = 0; q < 8; ++q) v[8 * i + q] += unpack16<DT>(w[q / 2], q & 1);
        }
    }
    __syncwarp();
}

__device__ __forceinline__ void dense_store_chunk(const DenseTc& p, float (&v)[32], uint8_t* stg, const float* bias,
                                                  int p0, int q0, int lane, int32_t& st) {
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 t = reinterpret_cast<const float4*>(bias)[i];
            v[4 * i] += t.x;
            v[4 * i + 1] += t.y;
            v[4 * i + 2] += t.z;
            v[4 * i + 3] += t.w;
        }
    }
    if (p.z) {
        if (p.bf16) dense_put<MILO_BF16>(p, p.z, v, stg, p0, q0, lane, st);
        else dense_put<MILO_F16>(p, p.z, v, stg, p0, q0, lane, st);
    }
    act_tile(p.act, v);
    with_dtype(p.y_dt, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (p.residual) dense_add<DT>(p, v, stg, p0, q0, lane);
        dense_put<DT>(p, p.y, v, stg, p0, q0, lane, st);
    });
}

// Swapped form: the lane's row is feature p0 + lane, its N values tokens q0..:
// y[q, p], consecutive lanes at consecutive addresses.
template <int N>
__device__ __forceinline__ void dense_store_swapped(const DenseTc& p, float (&v)[N], int p0, int q0, int lane,
                                                    int32_t& st) {
    const int f = p0 + lane;
    if (f >= p.P) return;
    if (p.bias) {
        const float b = load16(p.bias, f, p.bf16);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += b;
    }
    const int n = min(N, p.Q - q0);
    const size_t o = static_cast<size_t>(q0) * p.P + f;
    if (p.z)
        with_dtype(p.bf16 ? MILO_BF16 : MILO_F16, [&](auto dt) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < n) elem_store<decltype(dt)::value>(p.z, o + static_cast<size_t>(i) * p.P, v[i], st);
        });
    act_tile(p.act, v);
    with_dtype(p.y_dt, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (p.residual) {
            float r[N];
#pragma unroll
            for (int i = 0; i < N; ++i) r[i] = i < n ? elem_load<DT>(p.residual, o + static_cast<size_t>(i) * p.P) : 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += r[i];
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) elem_store<DT>(p.y, o + static_cast<size_t>(i) * p.P, v[i], st);
    });
}

template <bool SWAP>
__global__ void __launch_bounds__(kDtThreads) dense_tc_kernel(const __grid_constant__ DenseTc p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.off_bar);
    uint64_t* empty = full + kDtMaxStages;
    uint64_t* afull = empty + kDtMaxStages;      // accumulator finished
    uint64_t* aempty = afull + 2;                // accumulator read
    uint64_t* done_bar = aempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = p.split > 1 ? cluster_rank() : 0u;
    constexpr int W = SWAP ? 16 : kDtChunk;      // columns of a block of the split epilogue

    grid_dep_launch();
    if (warp == 0) {
        if (elect_one()) {
            prefetch_map(&p.a_map);
            prefetch_map(&p.b_map);
            for (int s = 0; s < p.stages; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(&afull[b], 1);
                mbar_init(&aempty[b], kDtEpiWarps);
            }
            mbar_init(done_bar, 1);
            fence_barrier_init();
        }
        __syncwarp();
    }
    // TMEM only once the kernels before have left: a CTA that held columns while
    // it waits for them could keep one of their CTAs from its own.  The producer
    // does not wait for it.
    grid_dep_wait();
    uint32_t tbase = 0;
    if (warp == 0) {
        asm volatile("bar.arrive 1, %0;" ::"n"(kDtThreads) : "memory");
    } else {
        if (warp == 1) tmem_alloc(tmem_slot, p.tmem_cols);
        tc_fence_before();
        named_sync(1, kDtThreads);
        tc_fence_after();
        tbase = *tmem_slot;
    }

    // this CTA's share of c (all of it without a split)
    const int kb0 = static_cast<int>(static_cast<long long>(p.kblocks) * rank / p.split);
    const int kb1 = static_cast<int>(static_cast<long long>(p.kblocks) * (rank + 1) / p.split);
    const int first = static_cast<int>(blockIdx.x) / p.split, step = static_cast<int>(gridDim.x) / p.split;
    int32_t st_bits = 0;
    // epilogue warps: lane quarter, which half of the column blocks, own buffers
    const int quarter = warp & 3, half = (warp - 2) >> 2, ew = warp - 2;
    const uint32_t lane_base = tbase + (static_cast<uint32_t>(32 * quarter) << 16);
    uint8_t* stg = smem + p.off_staging + ew * p.staging;
    float* sbias = reinterpret_cast<float*>(smem + p.off_bias) + ew * kDtBias;

    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        int stage = 0;
        uint32_t phase = 0, filled = 0, fph = 0;
        bool fail = false;
        const uint32_t tx = kDtAtom + p.bn * 128;
        for (int it = first; it < p.tiles && !fail; it += step) {
            int tp, tq;
            dense_tile(p, it, tp, tq);
            const int p0 = tp * kDtRows, q0 = tq * p.bn;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!warp_wait(&empty[stage], phase ^ 1)) {
                    fail = true;
                    break;
                }
                uint8_t* sa = smem + stage * p.stage_bytes;
                uint8_t* sb = sa + kDtAtom;
                uint64_t* fb = &full[stage];
                filled |= 1u << stage;
                fph = (fph & ~(1u << stage)) | (phase << stage);
                if (elect_one()) {
                    mbar_arrive_expect_tx(fb, tx);
                    if (p.a_mn) {
                        tma_load_2d(sa, &p.a_map, fb, p0, kb * kDtK);
                        tma_load_2d(sa + kDtBox, &p.a_map, fb, p0 + 64, kb * kDtK);
                    } else {
                        tma_load_2d(sa, &p.a_map, fb, kb * kDtK, p0);
                    }
                    if (p.b_mn) {
                        for (int j = 0; j < p.bn / 64; ++j)
                            tma_load_2d(sb + j * kDtBox, &p.b_map, fb, q0 + 64 * j, kb * kDtK);
                    } else {
                        tma_load_2d(sb, &p.b_map, fb, kb * kDtK, q0);
                    }
                }
                __syncwarp();
                if (++stage == p.stages) { stage = 0; phase ^= 1; }
            }
        }
        // no copy may still be landing in shared memory when the CTA leaves
        for (int s = 0; s < p.stages; ++s)
            if (((filled >> s) & 1u) && !warp_wait(&full[s], (fph >> s) & 1u)) fail = true;
        if (fail) st_bits |= MILO_DEV_TIMEOUT;
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        int stage = 0, buf = 0;
        uint32_t phase = 0, bph = 0;
        bool fail = false;
        const uint64_t astep = p.a_mn ? 128u : 2u, bstep = p.b_mn ? 128u : 2u;   // 16 c further, in 16-byte units
        for (int it = first; it < p.tiles && !fail; it += step) {
            if (!warp_wait(&aempty[buf], bph ^ 1)) {
                fail = true;
                break;
            }
            tc_fence_after();
            const uint32_t d = tbase + static_cast<uint32_t>(buf * p.bn);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!warp_wait(&full[stage], phase)) {
                    fail = true;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = smem_u32(smem + stage * p.stage_bytes), sb = sa + kDtAtom;
                const uint64_t da = p.a_mn ? sw128_mnmajor_desc(sa) : sw128_kmajor_desc(sa);
                const uint64_t db = p.b_mn ? sw128_mnmajor_desc(sb) : sw128_kmajor_desc(sb);
#pragma unroll
                for (int q = 0; q < kDtK / 16; ++q)
                    tc_mma_ss(d, da + q * astep, db + q * bstep, p.idesc, kb > kb0 || q > 0 ? 1u : 0u);
                tc_commit(&empty[stage]);
                if (++stage == p.stages) { stage = 0; phase ^= 1; }
            }
            tc_commit(&afull[buf]);
            if (++buf == p.bufs) { buf = 0; bph ^= 1; }
        }
        if (fail) st_bits |= MILO_DEV_TIMEOUT;
        // every issued MMA has completed before TMEM is released
        tc_commit(done_bar);
        if (!warp_wait(done_bar, 0)) st_bits |= MILO_DEV_TIMEOUT;
    } else if (p.split == 1) {
        // ---------------------------------------------------------------- epilogue, whole tiles
        int buf = 0;
        uint32_t bph = 0;
        for (int it = first; it < p.tiles; it += step) {
            int tp, tq;
            dense_tile(p, it, tp, tq);
            const int p0 = tp * kDtRows + 32 * quarter, q0 = tq * p.bn;
            if constexpr (!SWAP) {
                if (p.bias) {
                    // the columns of this warp's blocks, block after block
                    for (int i = lane; i < p.bn / 2; i += 32) {
                        const int q = q0 + (i / 32 * 2 + half) * 32 + lane;
                        sbias[i] = q < p.Q ? load16(p.bias, q, p.bf16) : 0.0f;
                    }
                    __syncwarp();
                }
            }
            if (!warp_wait(&afull[buf], bph)) {
                st_bits |= MILO_DEV_TIMEOUT;
                break;
            }
            tc_fence_after();
            const uint32_t acc = lane_base + static_cast<uint32_t>(buf * p.bn);
            for (int c = W * half; c < p.bn; c += 2 * W) {
                uint32_t d[W];
                tc_ld(acc + c, d);
                tc_wait_ld();
                float v[W];
#pragma unroll
                for (int i = 0; i < W; ++i) v[i] = __uint_as_float(d[i]);
                if (p0 >= p.P || q0 + c >= p.Q) continue;
                if constexpr (SWAP) dense_store_swapped(p, v, p0, q0 + c, lane, st_bits);
                else dense_store_chunk(p, v, stg, sbias + c / 2 - W / 2 * half, p0, q0 + c, lane, st_bits);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&aempty[buf]);
            if (++buf == p.bufs) { buf = 0; bph ^= 1; }
        }
    } else {
        // ---------------------------------------------------------------- epilogue, split over the cluster:
        // this CTA's partial blocks to their owners: block u (rows 32 (u % 4)..,
        // columns W (u / 4)..) to CTA u % split, there at [u / split][rank], four
        // columns of a lane's row together
        if (!warp_wait(&afull[0], 0)) st_bits |= MILO_DEV_TIMEOUT;
        tc_fence_after();
        __syncwarp();
        cluster_arrive();        // this CTA is done with its ring ...
        cluster_wait();          // ... and so are the others: the blocks go there
        for (int c = half; c < p.bn / W; c += 2) {
            const int u = 4 * c + quarter;
            const uint32_t dst = smem_u32(smem) + (u / p.split * p.split + rank) * (W * 128) + lane * 16;
            uint32_t d[W];
            tc_ld(lane_base + W * c, d);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < W / 4; ++i)
                st_peer4(dst + i * 512, u % p.split,
                         make_float4(__uint_as_float(d[4 * i]), __uint_as_float(d[4 * i + 1]), __uint_as_float(d[4 * i + 2]),
                                     __uint_as_float(d[4 * i + 3])));
        }
        tc_fence_before();
    }

    if (p.split > 1) {
        __syncwarp();
        if (warp < 2) {
            cluster_arrive();
            cluster_wait();
        }
        cluster_arrive();
        cluster_wait();
        if (warp >= 2) {
            int tp, tq;
            dense_tile(p, first, tp, tq);
            for (int i = ew; i * p.split + static_cast<int>(rank) < 4 * (p.bn / W); i += kDtEpiWarps) {
                const int u = i * p.split + static_cast<int>(rank);
                const int p0 = tp * kDtRows + 32 * (u & 3), q0 = tq * p.bn + W * (u >> 2);
                if (p0 >= p.P || q0 >= p.Q) continue;
                const float4* src = reinterpret_cast<const float4*>(smem + i * p.split * (W * 128)) + lane;
                float v[W];
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] = 0.0f;
                for (int s = 0; s < p.split; ++s)
#pragma unroll
                    for (int j = 0; j < W / 4; ++j) {
                        const float4 t = src[(s * (W / 4) + j) * 32];
                        v[4 * j] += t.x;
                        v[4 * j + 1] += t.y;
                        v[4 * j + 2] += t.z;
                        v[4 * j + 3] += t.w;
                    }
                if constexpr (SWAP) {
                    dense_store_swapped(p, v, p0, q0, lane, st_bits);
                } else {
                    if (p.bias) {
                        sbias[lane] = q0 + lane < p.Q ? load16(p.bias, q0 + lane, p.bf16) : 0.0f;
                        __syncwarp();
                    }
                    dense_store_chunk(p, v, stg, sbias, p0, q0, lane, st_bits);
                }
            }
        }
    }
    flag(p.dev_status, st_bits);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, p.tmem_cols);
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

constexpr int kDtSmemMax = 227 * 1024 - 1024;     // less the slack that aligns the base

static int dense_sms() {
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

// Instruction descriptor: D f32, A and B both fp16 or both bf16, each K- or
// MN-major, M = 128, N = bn.
static uint32_t dense_idesc(int bf16, int a_mn, int b_mn, int bn) {
    const uint32_t t = bf16 ? 1u : 0u;
    return (1u << 4) | (t << 7) | (t << 10) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(bn >> 3) << 17) | (static_cast<uint32_t>(kDtRows >> 4) << 24);
}

template <bool SWAP>
static cudaError_t launch_dense_tc(const DenseTc& p, int grid, int smem, cudaStream_t s) {
    static std::atomic<bool> configured[64];     // set once per device (a repeat is harmless)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(dense_tc_kernel<SWAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDtSmemMax + 1024);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kDtThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, dense_tc_kernel<SWAP>, p);
}

// Columns of a tile and split of c, by an estimate in SM cycles of a CTA's
// work: a slice of c takes bn * 2 cycles of the tensor core or its bytes at 90
// bytes a cycle (what one SM was seen to draw from L2), whichever is longer; a
// wave of tiles takes its slices and, when nothing follows to hide it, an
// epilogue; all of it at least the operands' bytes at the measured copy rate
// (3.4 bytes a cycle and SM each way, at 148 SMs and 1.9 GHz: 23 in all).
static void dense_plan(DenseTc& p, bool swap, int sms) {
    double best = -1.0;
    const double dram = (static_cast<double>(p.P) + p.Q) * p.C * 2.0 / (23.0 * 148.0);
    const int bn_swap = static_cast<int>(round_up(p.Q, 16));
    for (int bn = swap ? bn_swap : 64; bn <= (swap ? bn_swap : 256); bn *= 2) {
        if (!swap && bn > 64 && bn / 2 >= p.Q) break;            // the tile would be mostly empty
        const double tiles = std::ceil(p.P / 128.0) * std::ceil(p.Q / static_cast<double>(bn));
        const double slice = std::max(2.0 * bn, (kDtAtom + bn * 128) / 90.0);
        for (int split = 1; split <= kDtMaxSplit && (split == 1 || p.kblocks >= 2 * split); split *= 2) {
            const double waves = std::ceil(tiles * split / sms);
            if (split > 1 && waves > 1.0) break;                 // clusters only where one wave holds them
            const double epilogue = 8.0 * bn * (split > 1 ? 1.0 / split : 1.0);
            const double cost = std::max(dram, waves * std::ceil(p.kblocks / static_cast<double>(split)) * slice) + epilogue +
                                (split > 1 ? 1500.0 + 100.0 * split : 0.0);
            if (best < 0.0 || cost < best) {
                best = cost;
                p.bn = bn;
                p.split = split;
            }
        }
    }
    p.tiles_p = (p.P + kDtRows - 1) / kDtRows;
    p.tiles_q = (p.Q + p.bn - 1) / p.bn;
}

milo_status launch_dense_gemm(const DenseGemm& g, const char* what, cudaStream_t s) {
    if (g.P <= kDenseFewRows && !g.a_mn && !g.b_mn) return launch_dense_few(g, what, s);
    DenseTc p;
    memset(&p, 0, sizeof(p));
    // few rows of A (tokens): they become the columns
    const bool swap = g.P <= 128 && !g.a_mn;
    p.P = swap ? g.Q : g.P;
    p.Q = swap ? g.P : g.Q;
    p.C = g.C;
    p.a_mn = swap ? g.b_mn : g.a_mn;
    p.b_mn = swap ? g.a_mn : g.b_mn;
    const void* a = swap ? g.b : g.a;
    const void* b = swap ? g.a : g.b;
    const long long lda = swap ? g.ldb : g.lda, ldb = swap ? g.lda : g.ldb;
    p.bf16 = g.bf16;
    p.kblocks = (p.C + kDtK - 1) / kDtK;
    const int sms = dense_sms();
    dense_plan(p, swap, sms);
    const long long tiles = static_cast<long long>(p.tiles_p) * p.tiles_q;
    if (tiles > 0x3FFFFFFF) return fail(MILO_ERR_UNSUPPORTED_SHAPE, std::string(what) + ": too many tiles");
    p.tiles = static_cast<int>(tiles);
    p.bufs = p.split == 1 && p.tiles > sms ? 2 : 1;
    p.stage_bytes = kDtAtom + p.bn * 128;
    // shared memory: the ring (then a split's partial blocks), the row form's
    // staging and bias, barriers
    p.staging = swap ? 0 : 32 * dense_pitch(g.y_dt == MILO_F32 ? 4 : 2);
    const int staging = kDtEpiWarps * p.staging, bias = swap ? 0 : kDtEpiWarps * kDtBias * 4;
    const int w = swap ? 16 : kDtChunk;
    const int part = p.split > 1 ? static_cast<int>(round_up(4 * (p.bn / w), p.split)) * w * 128 : 0;
    const int kper = (p.kblocks + p.split - 1) / p.split;
    p.stages = std::min({kDtMaxStages, (kDtSmemMax - staging - bias - 512) / p.stage_bytes,
                         std::max(2, p.bufs == 2 ? kDtMaxStages : kper)});
    p.off_staging = std::max(p.stages * p.stage_bytes, part);
    p.off_bias = p.off_staging + staging;
    p.off_bar = p.off_bias + bias;
    const int smem = p.off_bar + 512 + 1024;
    p.tmem_cols = 32;
    while (p.tmem_cols < static_cast<uint32_t>(p.bufs * p.bn)) p.tmem_cols *= 2;
    p.idesc = dense_idesc(p.bf16, p.a_mn, p.b_mn, p.bn);
    p.bias = g.bias;
    p.residual = g.residual;
    p.y = g.y;
    p.z = g.z;
    p.act = g.act;
    p.y_dt = g.y_dt;
    p.dev_status = g.dev_status;
    p.vec = g.Q % 8 == 0 && aligned(g.y, 16) && aligned(g.residual, 16) && aligned(g.z, 16);

    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_UINT16;
    milo_status st;
    // K-major [rows, c]: box 64 c by the tile's rows; MN-major [c, rows]: box 64 rows by 64 c
    st = p.a_mn ? make_map(&p.a_map, a, dt, p.P, p.C, lda * 2, 64, kDtK, what, CU_TENSOR_MAP_SWIZZLE_128B)
                : make_map(&p.a_map, a, dt, p.C, p.P, lda * 2, kDtK, kDtRows, what, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != MILO_OK) return st;
    st = p.b_mn ? make_map(&p.b_map, b, dt, p.Q, p.C, ldb * 2, 64, kDtK, what, CU_TENSOR_MAP_SWIZZLE_128B)
                : make_map(&p.b_map, b, dt, p.C, p.Q, ldb * 2, kDtK, p.bn, what, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != MILO_OK) return st;
    const int grid = p.split > 1 ? p.tiles * p.split : std::min(p.tiles, sms);
    return check_cuda(swap ? launch_dense_tc<true>(p, grid, smem, s) : launch_dense_tc<false>(p, grid, smem, s), what);
}

}  // namespace milo
