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
//   - Large products: pairs of CTAs (cta_group::2) share tiles of 256 x 256; each
//     brings 128 rows of A and of B, 32 KB a slice instead of 48, since what
//     an SM can draw from L2 (about 66 bytes a cycle) bounds the single form.
//   - Two products may share a launch (a layer's dx and dW): their tiles follow
//     one another on the same grid (dense_item), so neither's last wave leaves
//     SMs idle.
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
//   - Outputs of whole 16-byte pieces leave by TMA, and a residual's blocks come
//     by it, up to three ahead of the accumulators (2780 x 8424 x 72 with both: 47
//     us, 99 with loads that a warp waits for).  Other widths go through a staging
//     buffer by words or elements, eight loads under way (2780 x 8420 x 72: 70 us,
//     2780 x 8419 x 72: 96; one load at a time 268).  The two forms are kernels of
//     their own: in one, the second's registers slowed the first by 3 to 15%.
//   - Every wait is bounded: on a timeout the kernel flags MILO_DEV_TIMEOUT,
//     waits for its copies and products and frees TMEM before it leaves.
//
// Measured (B200, device time): 8192 x 14336 x 4096 bf16 with bias and gelu_tanh
// 612 to 633 us from GPU to GPU = 1520 to 1570 TFLOP/s, 0.93 to 0.96 of the cuBLAS
// burst rate (single CTAs 690 us: the operands' way from L2); dx and dW of 8192 x
// 4096 x 4096 370 to 388 us together (385 with their tiles dealt round without
// regard to length, where 370 was).  Small products are bound by latency, not by
// the tensor cores or memory (5% of the pipe, 10 to 13% of DRAM): 64 x 2816 x 2048
// fp16 8.6 us and 4999 x 64 x 2048 9.4 to 10.0 us, of which the first loads take about
// 1.6 us, the cluster's exchange 1.5 and the launch 2; the rest, barriers and output,
// has not been told apart.
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
constexpr int kDtMaxStages = 12;             // below 31 (a lane each at the end)
constexpr int kDtMaxSplit = 8;               // portable cluster size
constexpr int kDtChunk = 32;                 // accumulator columns handled at a time
constexpr int kDtOutBufs = 4;                // output buffers of an epilogue warp, at most
constexpr int kDtBias = 128;                 // fp32 bias columns, per epilogue warp (its half of 256)

// Output staging of an epilogue warp (narrow form): 32 rows of 32 elements, 16
// bytes apart from a multiple of 128 so that 16-byte pieces of a column fall on
// different banks.
constexpr int dense_pitch(int esize) { return 32 * esize + 16; }

// One product of a launch.
struct DenseProb {
    CUtensorMap a_map, b_map;
    CUtensorMap y_map;                       // wide form only
    int P, Q, C;
    int a_mn, b_mn;
    int kblocks;                             // slices of 64 c
    int tiles_p, tiles_q, tiles;
    uint32_t idesc;
    void* y;                                 // [P, Q] (SWAP: [Q, P])
};

struct DenseTc {
    CUtensorMap z_map, r_map;                // wide form only
    DenseProb prob[2];                       // one product, or two that share the grid (a layer's dx and dW)
    int tiles;                               // of both
    int rounds, extra, fill;                 // the schedule (dense_item)
    int bf16, bn, stages, split;             // columns of a tile; CTAs that share a tile's c
    int two;                                 // pairs of CTAs on tiles of 256 rows
    uint32_t tmem_cols;
    int bufs;                                // accumulators in TMEM (2: persistent)
    int stage_bytes, staging, off_staging, off_bias, off_bar;
    int out_bufs, out_bytes;                 // wide form: output buffers of an epilogue warp, bytes of one
    // epilogue (residual and z as y; SWAP: p is the feature)
    const void *bias, *residual;
    void* z;
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

// Pairs of CTAs (cta_group::2): the same shared-memory address in CTA `rank` of
// the cluster, and the forms of the TMEM, copy, MMA and commit instructions that
// work for both.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void mbar_arrive_peer(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_alloc2(uint32_t* dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// To this CTA's shared memory, completing on a barrier of either CTA (no multicast).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4}], [%2];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void tc_mma_ss2(uint32_t d_addr, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_addr), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// One arrival on this barrier in both CTAs.
__device__ __forceinline__ void tc_commit2(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
        ::"r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3)) : "memory");
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
struct DenseItem {
    int i;                                   // product
    int tp, tq;
};
// Item n of CTA (or pair, or cluster) `slot` of S, or -1 behind its last one; item
// 0 is tile `slot`.
// The first product's tiles, which take the longest, go round: `rounds` to
// each slot and one more to the first `extra`.  The other slots then take
// `fill` of the second's, about as long as that one, and the rest goes round
// again.
__device__ __forceinline__ int dense_item(const DenseTc& p, int slot, int S, int n) {
    const int own = p.rounds + (slot < p.extra ? 1 : 0);
    if (n < own) return n * S + slot;
    const int m = n - own, others = S - p.extra;
    int i = p.prob[0].tiles;
    if (slot < p.extra) i += p.fill * others + m * S + slot;
    else if (m < p.fill) i += m * others + slot - p.extra;
    else i += p.fill * others + (m - p.fill) * S + slot;
    return i < p.tiles ? i : -1;
}
__device__ __forceinline__ DenseItem dense_tile(const DenseTc& p, int item) {
    DenseItem r;
    r.i = item >= p.prob[0].tiles;
    if (r.i) item -= p.prob[0].tiles;
    const DenseProb& d = p.prob[r.i];
    const int per = kDtBand * d.tiles_q;
    const int band = item / per, in = item - band * per;
    const int h = min(kDtBand, d.tiles_p - band * kDtBand);
    r.tq = in / h;
    r.tp = band * kDtBand + in - r.tq * h;
    return r;
}

// ---------------------------------------------------------------------------
// epilogue of 32 rows (lane = row p) by 32 columns q0.. of D, row form: y[p, q].
// v holds the lane's row.  Wide form: rows of whole 16-byte pieces at 16-byte
// addresses, blocks come and go by TMA, which cuts what lies outside.  Narrow
// form: every other width and address.
// ---------------------------------------------------------------------------

// 16-byte piece i of the lane's row in a buffer of the maps' swizzled layout
// (64-byte rows: piece i at i ^ ((row / 2) % 4); 128-byte rows: i ^ (row % 8), so
// that eight lanes' pieces fall on different banks).
template <int DT>
__device__ __forceinline__ uint4* out_piece(uint8_t* buf, int lane, int i) {
    if constexpr (DT == MILO_F32) return reinterpret_cast<uint4*>(buf + lane * 128 + ((i ^ (lane & 7)) << 4));
    else return reinterpret_cast<uint4*>(buf + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4));
}

template <int DT>
__device__ __forceinline__ void wide_put(const CUtensorMap* map, const float (&v)[32], uint8_t* buf, int p0, int q0, int lane,
                                         int32_t& st) {
    if constexpr (DT == MILO_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(out_piece<DT>(buf, lane, i)) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack16<DT>(v[2 * i], v[2 * i + 1]);
        if constexpr (DT == MILO_F16) half_range(v, w, st);
#pragma unroll
        for (int i = 0; i < 4; ++i) *out_piece<DT>(buf, lane, i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0)
        asm volatile(
            "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];\n\t"
            "cp.async.bulk.commit_group;"
            ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(buf)), "r"(q0), "r"(p0) : "memory");
}

// All but the `newest` last stores of this thread have left shared memory.
__device__ __forceinline__ void stores_read(int newest) {
    if (newest >= 3) asm volatile("cp.async.bulk.wait_group.read 3;" ::: "memory");
    else if (newest == 2) asm volatile("cp.async.bulk.wait_group.read 2;" ::: "memory");
    else if (newest == 1) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    else asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

__device__ __forceinline__ void add_bias(float (&v)[32], const float* bias) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 t = reinterpret_cast<const float4*>(bias)[i];
        v[4 * i] += t.x;
        v[4 * i + 1] += t.y;
        v[4 * i + 2] += t.z;
        v[4 * i + 3] += t.w;
    }
}

// One 32 x 32 block.  `buf` holds the residual's block if there is one; the
// stores up to the `left` newest have to be out of `zbuf`, and without a residual
// out of `buf`, before they are written.
__device__ __forceinline__ void wide_chunk(const DenseTc& p, const DenseProb& d, float (&v)[32], uint8_t* buf, uint8_t* zbuf,
                                           int left, const float* bias, int p0, int q0, int lane, int32_t& flags) {
    int32_t st = 0;                          // counts where the lane's row exists: behind the last one it is act(bias)
    if (p.bias) add_bias(v, bias);
    if (p.z) {
        if (lane == 0) stores_read(left);
        __syncwarp();
        if (p.bf16) wide_put<MILO_BF16>(&p.z_map, v, zbuf, p0, q0, lane, st);
        else wide_put<MILO_F16>(&p.z_map, v, zbuf, p0, q0, lane, st);
    }
    act_tile(p.act, v);
    with_dtype(p.y_dt, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < (DT == MILO_F32 ? 8 : 4); ++i) {
                const uint4 t = *out_piece<DT>(buf, lane, i);
                const uint32_t w[4] = {t.x, t.y, t.z, t.w};
                if constexpr (DT == MILO_F32) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[4 * i + q] += __uint_as_float(w[q]);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[8 * i + q] += unpack16<DT>(w[q / 2], q & 1);
                }
            }
        } else {
            if (lane == 0) stores_read(left);
            __syncwarp();
        }
        wide_put<DT>(&d.y_map, v, buf, p0, q0, lane, st);
    });
    if (p0 + lane < d.P) flags |= st;
}

// Narrow form: the warp's block between staging rows (dense_pitch) and global
// rows p0.., columns q0.., in pieces of T, R rows a pass.  All of a batch's
// loads come before its stores: one at a time they would wait for each other
// (the compiler cannot tell the two buffers apart).
template <typename T, int E, bool LOAD>
__device__ __forceinline__ void narrow_block_by(const DenseProb& d, void* g, uint8_t* stg, int p0, int q0, int lane) {
    constexpr int kPitch = dense_pitch(E), kEl = static_cast<int>(sizeof(T)) / E;
    constexpr int kLanes = 32 / kEl, R = 32 / kLanes, kBatch = 8;
    const int col = lane % kLanes * kEl, r0 = lane / kLanes;
    const int rows = q0 + col < d.Q ? d.P - p0 - r0 : 0;  // (Q is a multiple of kEl)
    const size_t pitch = static_cast<size_t>(d.Q) * E;
    uint8_t* gp = static_cast<uint8_t*>(g) + static_cast<size_t>(p0 + r0) * pitch + static_cast<size_t>(q0 + col) * E;
    uint8_t* sp = stg + r0 * kPitch + col * E;
#pragma unroll 1
    for (int r = 0; r < 32; r += kBatch * R, gp += kBatch * R * pitch, sp += kBatch * R * kPitch) {
        T t[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if constexpr (LOAD) t[i] = r + i * R < rows ? *reinterpret_cast<const T*>(gp + i * R * pitch) : T(0);
            else t[i] = *reinterpret_cast<const T*>(sp + i * R * kPitch);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if constexpr (LOAD) *reinterpret_cast<T*>(sp + i * R * kPitch) = t[i];
            else if (r + i * R < rows) *reinterpret_cast<T*>(gp + i * R * pitch) = t[i];
        }
    }
}

template <int DT, bool LOAD>
__device__ __forceinline__ void narrow_block(const DenseProb& d, const void* g, uint8_t* stg, int p0, int q0, int lane) {
    if constexpr (DT == MILO_F32) {
        narrow_block_by<uint32_t, 4, LOAD>(d, const_cast<void*>(g), stg, p0, q0, lane);
    } else {
        // words where every row starts on one, else elements
        if (((reinterpret_cast<uintptr_t>(g) & 3) | (d.Q & 1)) == 0)
            narrow_block_by<uint32_t, 2, LOAD>(d, const_cast<void*>(g), stg, p0, q0, lane);
        else
            narrow_block_by<uint16_t, 2, LOAD>(d, const_cast<void*>(g), stg, p0, q0, lane);
    }
}

template <int DT>
__device__ __forceinline__ void narrow_put(const DenseProb& d, void* g, const float (&v)[32], uint8_t* stg, int p0, int q0,
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
    narrow_block<DT, false>(d, g, stg, p0, q0, lane);
    __syncwarp();
}

__device__ __forceinline__ void narrow_chunk(const DenseTc& p, const DenseProb& d, float (&v)[32], uint8_t* stg,
                                             const float* bias, int p0, int q0, int lane, int32_t& flags) {
    int32_t st = 0;                          // as in wide_chunk
    if (p.bias) add_bias(v, bias);
    if (p.z) {
        if (p.bf16) narrow_put<MILO_BF16>(d, p.z, v, stg, p0, q0, lane, st);
        else narrow_put<MILO_F16>(d, p.z, v, stg, p0, q0, lane, st);
    }
    act_tile(p.act, v);
    with_dtype(p.y_dt, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (p.residual) {
            narrow_block<DT, true>(d, p.residual, stg, p0, q0, lane);
            __syncwarp();
            const uint8_t* row = stg + lane * dense_pitch(DT == MILO_F32 ? 4 : 2);
#pragma unroll
            for (int i = 0; i < (DT == MILO_F32 ? 8 : 4); ++i) {
                const uint4 t = reinterpret_cast<const uint4*>(row)[i];
                const uint32_t w[4] = {t.x, t.y, t.z, t.w};
                if constexpr (DT == MILO_F32) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[4 * i + q] += __uint_as_float(w[q]);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[8 * i + q] += unpack16<DT>(w[q / 2], q & 1);
                }
            }
            __syncwarp();
        }
        narrow_put<DT>(d, d.y, v, stg, p0, q0, lane, st);
    });
    if (p0 + lane < d.P) flags |= st;
}

// Swapped form: the lane's row is feature p0 + lane, its N values tokens q0..:
// y[q, p], consecutive lanes at consecutive addresses.
template <int N>
__device__ __forceinline__ void dense_store_swapped(const DenseTc& p, const DenseProb& d, float (&v)[N], int p0, int q0, int lane,
                                                    int32_t& st) {
    const int f = p0 + lane;
    if (f >= d.P) return;
    if (p.bias) {
        const float b = load16(p.bias, f, p.bf16);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += b;
    }
    const int n = min(N, d.Q - q0);
    const size_t o = static_cast<size_t>(q0) * d.P + f;
    if (p.z)
        with_dtype(p.bf16 ? MILO_BF16 : MILO_F16, [&](auto dt) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < n) elem_store<decltype(dt)::value>(p.z, o + static_cast<size_t>(i) * d.P, v[i], st);
        });
    act_tile(p.act, v);
    with_dtype(p.y_dt, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (p.residual) {
            float r[N];
#pragma unroll
            for (int i = 0; i < N; ++i) r[i] = i < n ? elem_load<DT>(p.residual, o + static_cast<size_t>(i) * d.P) : 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += r[i];
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) elem_store<DT>(d.y, o + static_cast<size_t>(i) * d.P, v[i], st);
    });
}

// (SWAP: left alone the compiler takes 48 registers and spills; 128 x 4096 x 4096
// 14.2 us, so 13.0)
template <bool SWAP, bool TWO, bool WIDE>
__global__ void __launch_bounds__(kDtThreads, SWAP ? 2 : 0) dense_tc_kernel(const __grid_constant__ DenseTc p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.off_bar);
    uint64_t* empty = full + kDtMaxStages;
    uint64_t* afull = empty + kDtMaxStages;      // accumulator finished
    uint64_t* aempty = afull + 2;                // accumulator read
    uint64_t* done_bar = aempty + 2;
    uint64_t* rbar = done_bar + 1;               // residual blocks, per epilogue warp and buffer
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rbar + kDtEpiWarps * kDtOutBufs);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t cta = TWO || p.split > 1 ? cluster_rank() : 0u;
    const uint32_t rank = TWO ? 0u : cta;        // of a split of c
    constexpr int W = SWAP ? 16 : kDtChunk;      // columns of a block of the epilogue
    constexpr int kTileRows2 = TWO ? 2 * kDtRows : kDtRows;
    const int group = TWO ? 2 : p.split;         // CTAs of a tile

    grid_dep_launch();
    if (warp == 0) {
        if (elect_one()) {
            for (int i = 0; i < (p.tiles > p.prob[0].tiles ? 2 : 1); ++i) {
                prefetch_map(&p.prob[i].a_map);
                prefetch_map(&p.prob[i].b_map);
            }
            for (int s = 0; s < p.stages; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(&afull[b], 1);
                mbar_init(&aempty[b], TWO ? 2 * kDtEpiWarps : kDtEpiWarps);
            }
            mbar_init(done_bar, 1);
            if (WIDE && p.residual)
                for (int i = 0; i < kDtEpiWarps * kDtOutBufs; ++i) mbar_init(&rbar[i], 1);
            fence_barrier_init();
        }
        __syncwarp();
    }
    // TMEM only once the kernels before have left: a CTA that held columns while
    // it waits for them could keep one of their CTAs from its own.  The producer
    // does not wait for it.
    grid_dep_wait();
    uint32_t tbase = 0;
    if constexpr (TWO) {
        // both CTAs' barriers and columns exist before either's copies and products
        if (warp == 1) tmem_alloc2(tmem_slot, p.tmem_cols);
        tc_fence_before();
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        tc_fence_after();
        tbase = *tmem_slot;
    } else if (warp == 0) {
        asm volatile("bar.arrive 1, %0;" ::"n"(kDtThreads) : "memory");
    } else {
        if (warp == 1) tmem_alloc(tmem_slot, p.tmem_cols);
        tc_fence_before();
        named_sync(1, kDtThreads);
        tc_fence_after();
        tbase = *tmem_slot;
    }

    // this CTA's share of a product's c (all of it without a split)
    const auto slice = [&](const DenseProb& d, uint32_t r) {
        return static_cast<int>(static_cast<long long>(d.kblocks) * r / p.split);
    };
    const int first = static_cast<int>(blockIdx.x) / group, slots = static_cast<int>(gridDim.x) / group;
    int32_t st_bits = 0;
    // epilogue warps: lane quarter, which half of the column blocks, own buffers
    const int quarter = warp & 3, half = (warp - 2) >> 2, ew = warp - 2;
    const uint32_t lane_base = tbase + (static_cast<uint32_t>(32 * quarter) << 16);
    uint8_t* stg = smem + p.off_staging + ew * p.staging;
    // z's buffer, wide form: the one behind the others when those hold residuals
    uint8_t* zbuf = stg + p.out_bufs * p.out_bytes;
    auto load_residual = [&](int buf, int p0, int q0) {       // one lane
        uint64_t* bar = &rbar[ew * kDtOutBufs + buf];
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(p.out_bytes));
        tma_load_2d(stg + buf * p.out_bytes, &p.r_map, bar, q0, p0);
    };
    float* sbias = reinterpret_cast<float*>(smem + p.off_bias) + ew * kDtBias;
    uint32_t filled = 0, fph = 0;                // producer: stages filled, their last phases

    if (warp == 0) {
        // ---------------------------------------------------------------- producer
        int stage = 0;
        uint32_t phase = 0;
        bool fail = false;
        const uint32_t tx = (TWO ? 2 : 1) * p.stage_bytes;
        const int bq = TWO ? p.bn / 2 : p.bn;        // B rows this CTA brings
        for (int n = 0, it = first; it >= 0 && !fail; it = dense_item(p, first, slots, ++n)) {
            const DenseItem t = dense_tile(p, it);
            const DenseProb& d = p.prob[t.i];
            const int p0 = t.tp * kTileRows2 + (TWO ? kDtRows * cta : 0), q0 = t.tq * p.bn + (TWO ? bq * cta : 0);
            const int kb1 = slice(d, rank + 1);
            for (int kb = slice(d, rank); kb < kb1; ++kb) {
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
                    // a pair's copies complete on the first CTA's barrier
                    const uint32_t pb = TWO ? peer_addr(fb, 0) : 0u;
                    auto load = [&](void* dst, const CUtensorMap* map, int x, int y) {
                        if constexpr (TWO) tma_load_2d_pair(dst, map, pb, x, y);
                        else tma_load_2d(dst, map, fb, x, y);
                    };
                    if (!TWO || cta == 0) mbar_arrive_expect_tx(fb, tx);
                    if (d.a_mn) {
                        load(sa, &d.a_map, p0, kb * kDtK);
                        load(sa + kDtBox, &d.a_map, p0 + 64, kb * kDtK);
                    } else {
                        load(sa, &d.a_map, kb * kDtK, p0);
                    }
                    if (d.b_mn) {
                        for (int j = 0; j < bq / 64; ++j) load(sb + j * kDtBox, &d.b_map, q0 + 64 * j, kb * kDtK);
                    } else {
                        load(sb, &d.b_map, kb * kDtK, q0);
                    }
                }
                __syncwarp();
                if (++stage == p.stages) { stage = 0; phase ^= 1; }
            }
        }
        // no copy may still be landing in shared memory when the CTA leaves
        // (a pair's first CTA sees both CTAs' copies)
        for (int s = 0; s < p.stages && (!TWO || cta == 0); ++s)
            if (((filled >> s) & 1u) && !warp_wait(&full[s], (fph >> s) & 1u)) fail = true;
        if (fail) st_bits |= MILO_DEV_TIMEOUT;
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        int stage = 0, buf = 0;
        uint32_t phase = 0, bph = 0;
        bool fail = false;
        for (int n = 0, it = first; it >= 0 && !fail && (!TWO || cta == 0); it = dense_item(p, first, slots, ++n)) {
            if (!warp_wait(&aempty[buf], bph ^ 1)) {
                fail = true;
                break;
            }
            tc_fence_after();
            const DenseProb& d = p.prob[dense_tile(p, it).i];
            const int a_mn = d.a_mn, b_mn = d.b_mn, kb0 = slice(d, rank), kb1 = slice(d, rank + 1);
            const uint64_t astep = a_mn ? 128u : 2u, bstep = b_mn ? 128u : 2u;   // 16 c further, in 16-byte units
            const uint32_t idesc = d.idesc;
            const uint32_t acc = tbase + static_cast<uint32_t>(buf * p.bn);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!warp_wait(&full[stage], phase)) {
                    fail = true;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = smem_u32(smem + stage * p.stage_bytes), sb = sa + kDtAtom;
                const uint64_t da = a_mn ? sw128_mnmajor_desc(sa) : sw128_kmajor_desc(sa);
                const uint64_t db = b_mn ? sw128_mnmajor_desc(sb) : sw128_kmajor_desc(sb);
#pragma unroll
                for (int q = 0; q < kDtK / 16; ++q) {
                    if constexpr (TWO) tc_mma_ss2(acc, da + q * astep, db + q * bstep, idesc, kb > kb0 || q > 0 ? 1u : 0u);
                    else tc_mma_ss(acc, da + q * astep, db + q * bstep, idesc, kb > kb0 || q > 0 ? 1u : 0u);
                }
                if constexpr (TWO) tc_commit2(&empty[stage]);
                else tc_commit(&empty[stage]);
                if (++stage == p.stages) { stage = 0; phase ^= 1; }
            }
            if constexpr (TWO) tc_commit2(&afull[buf]);
            else tc_commit(&afull[buf]);
            if (++buf == p.bufs) { buf = 0; bph ^= 1; }
        }
        if (fail) st_bits |= MILO_DEV_TIMEOUT;
        // every issued MMA has completed before TMEM is released
        if constexpr (TWO) {
            if (cta == 0) {
                tc_commit2(done_bar);
                if (!warp_wait(done_bar, 0)) st_bits |= MILO_DEV_TIMEOUT;
            }
        } else {
            tc_commit(done_bar);
            if (!warp_wait(done_bar, 0)) st_bits |= MILO_DEV_TIMEOUT;
        }
    } else if (TWO || p.split == 1) {
        // ---------------------------------------------------------------- epilogue, whole tiles
        int buf = 0;
        uint32_t bph = 0;
        bool dead = false;
        // Wide form: the output buffers in turn; with a residual, its block comes
        // to the buffer of y's, under way out_bufs - 1 blocks ahead.
        int at = 0, flying = 0, ahead_n = 0, ahead_it = first, ahead_c = -2 * W + W * half;
        uint32_t rph = 0;
        const bool res = WIDE && p.residual;
        auto ahead = [&](int b) {                             // the next block's residual to buffer b
            while (!dead) {
                ahead_c += 2 * W;
                if (ahead_c >= p.bn) {
                    ahead_c = W * half;
                    if (ahead_it >= 0) ahead_it = dense_item(p, first, slots, ++ahead_n);
                }
                if (ahead_it < 0) return;
                const DenseItem t = dense_tile(p, ahead_it);
                const DenseProb& d = p.prob[t.i];
                const int p0 = t.tp * kTileRows2 + (TWO ? kDtRows * cta : 0) + 32 * quarter, q0 = t.tq * p.bn + ahead_c;
                if (p0 >= d.P || q0 >= d.Q || ahead_c >= p.bn) continue;
                if (lane == 0) load_residual(b, p0, q0);
                ++flying;
                return;
            }
        };
        if (res)
            for (int b = 0; b < p.out_bufs - 1; ++b) ahead(b);
        for (int n = 0, it = first; it >= 0; it = dense_item(p, first, slots, ++n)) {
            const DenseItem t = dense_tile(p, it);
            const DenseProb& d = p.prob[t.i];
            const int p0 = t.tp * kTileRows2 + (TWO ? kDtRows * cta : 0) + 32 * quarter, q0 = t.tq * p.bn;
            if constexpr (!SWAP) {
                if (p.bias) {
                    // the columns of this warp's blocks, block after block
                    for (int i = lane; i < p.bn / 2; i += 32) {
                        const int q = q0 + (i / 32 * 2 + half) * 32 + lane;
                        sbias[i] = q < d.Q ? load16(p.bias, q, p.bf16) : 0.0f;
                    }
                    __syncwarp();
                }
            }
            // after a timeout nothing is waited for again (the outputs are invalid)
            if (!dead && !warp_wait(&afull[buf], bph)) dead = true;
            tc_fence_after();
            const uint32_t acc = lane_base + static_cast<uint32_t>(buf * p.bn);
            for (int c = W * half; c < p.bn; c += 2 * W) {
                uint32_t r[W];
                tc_ld(acc + c, r);
                tc_wait_ld();
                float v[W];
#pragma unroll
                for (int i = 0; i < W; ++i) v[i] = __uint_as_float(r[i]);
                if (p0 >= d.P || q0 + c >= d.Q) continue;
                const float* cb = sbias + c / 2 - W / 2 * half;
                if constexpr (SWAP) {
                    dense_store_swapped(p, d, v, p0, q0 + c, lane, st_bits);
                } else if constexpr (WIDE) {
                    if (res) {
                        if (flying > 0) {
                            --flying;
                            if (!warp_wait(&rbar[ew * kDtOutBufs + at], rph)) dead = true;
                        }
                        wide_chunk(p, d, v, stg + at * p.out_bytes, zbuf, 1, cb, p0, q0 + c, lane, st_bits);
                        // the buffer of the block before takes the next residual
                        if (lane == 0) stores_read(1);
                        __syncwarp();
                        ahead(at == 0 ? p.out_bufs - 1 : at - 1);
                        if (++at == p.out_bufs) { at = 0; rph ^= 1; }
                    } else {
                        uint8_t* zb = stg + at * p.out_bytes;
                        if (p.z && ++at == p.out_bufs) at = 0;
                        uint8_t* yb = stg + at * p.out_bytes;
                        if (++at == p.out_bufs) at = 0;
                        wide_chunk(p, d, v, yb, zb, p.out_bufs - 1, cb, p0, q0 + c, lane, st_bits);
                    }
                } else {
                    narrow_chunk(p, d, v, stg, cb, p0, q0 + c, lane, st_bits);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (TWO) mbar_arrive_peer(peer_addr(&aempty[buf], 0));
                else mbar_arrive(&aempty[buf]);
            }
            if (++buf == p.bufs) { buf = 0; bph ^= 1; }
        }
        if (dead) st_bits |= MILO_DEV_TIMEOUT;
    } else {
        // ---------------------------------------------------------------- epilogue, split over the cluster:
        // this CTA's partial blocks to their owners: block u (rows 32 (u % 4)..,
        // columns W (u / 4)..) to CTA u % split, there at [u / split][rank], four
        // columns of a lane's row together
        const DenseProb& d = p.prob[dense_tile(p, first).i];
        const bool none = slice(d, rank) == slice(d, rank + 1);      // a short c leaves some CTAs nothing
        if (WIDE && p.residual && lane == 0) {
            // the residual of the first block this warp will finish
            const DenseItem t = dense_tile(p, first);
            const int u = ew * p.split + static_cast<int>(rank);
            const int p0 = t.tp * kDtRows + 32 * (u & 3), q0 = t.tq * p.bn + W * (u >> 2);
            if (u < 4 * (p.bn / W) && p0 < d.P && q0 < d.Q) load_residual(0, p0, q0);
        }
        if (!warp_wait(&afull[0], 0)) st_bits |= MILO_DEV_TIMEOUT;
        tc_fence_after();
        __syncwarp();
        cluster_arrive();        // this CTA is done with its ring ...
        cluster_wait();          // ... and so are the others: the blocks go there
        for (int c = half; c < p.bn / W; c += 2) {
            const int u = 4 * c + quarter;
            const uint32_t dst = smem_u32(smem) + (u / p.split * p.split + rank) * (W * 128) + lane * 16;
            uint32_t r[W];
            tc_ld(lane_base + W * c, r);
            tc_wait_ld();
            if (none) {
#pragma unroll
                for (int i = 0; i < W; ++i) r[i] = 0u;
            }
#pragma unroll
            for (int i = 0; i < W / 4; ++i)
                st_peer4(dst + i * 512, u % p.split,
                         make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]), __uint_as_float(r[4 * i + 2]),
                                     __uint_as_float(r[4 * i + 3])));
        }
        tc_fence_before();
    }

    if constexpr (TWO) {
        // neither CTA leaves while the other's copies, products or remote arrivals reach
        // it (the commits' arrivals, which no barrier of the cluster orders: below)
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    } else if (p.split > 1) {
        __syncwarp();
        if (warp < 2) {
            cluster_arrive();
            cluster_wait();
        }
        cluster_arrive();
        cluster_wait();
        if (warp >= 2) {
            const DenseItem t = dense_tile(p, first);
            const DenseProb& d = p.prob[t.i];
            uint32_t uph = 0;
            for (int i = ew; i * p.split + static_cast<int>(rank) < 4 * (p.bn / W); i += kDtEpiWarps) {
                const int u = i * p.split + static_cast<int>(rank);
                const int p0 = t.tp * kDtRows + 32 * (u & 3), q0 = t.tq * p.bn + W * (u >> 2);
                if (p0 >= d.P || q0 >= d.Q) continue;
                const float4* src = reinterpret_cast<const float4*>(smem + i * p.split * (W * 128)) + lane;
                float v[W];
#pragma unroll
                for (int j = 0; j < W; ++j) v[j] = 0.0f;
                for (int s = 0; s < p.split; ++s)
#pragma unroll
                    for (int j = 0; j < W / 4; ++j) {
                        const float4 f = src[(s * (W / 4) + j) * 32];
                        v[4 * j] += f.x;
                        v[4 * j + 1] += f.y;
                        v[4 * j + 2] += f.z;
                        v[4 * j + 3] += f.w;
                    }
                if constexpr (SWAP) {
                    dense_store_swapped(p, d, v, p0, q0, lane, st_bits);
                } else {
                    if (p.bias) {
                        sbias[lane] = q0 + lane < d.Q ? load16(p.bias, q0 + lane, p.bf16) : 0.0f;
                        __syncwarp();
                    }
                    if constexpr (WIDE) {
                        if (p.residual) {
                            // (the first block's is under way, the others' come now)
                            if (i != ew && lane == 0) {
                                stores_read(0);
                                load_residual(0, p0, q0);
                            }
                            __syncwarp();
                            if (!warp_wait(&rbar[ew * kDtOutBufs], uph)) st_bits |= MILO_DEV_TIMEOUT;
                            uph ^= 1;
                            wide_chunk(p, d, v, stg, zbuf, 1, sbias, p0, q0, lane, st_bits);
                        } else {
                            if (lane == 0) stores_read(0);
                            __syncwarp();
                            wide_chunk(p, d, v, zbuf - p.out_bytes, stg, p.out_bufs - 1, sbias, p0, q0, lane, st_bits);
                        }
                    } else {
                        narrow_chunk(p, d, v, stg, sbias, p0, q0, lane, st_bits);
                    }
                }
            }
        }
    }
    // Nor does a CTA leave while a commit's arrival is on its way to its barriers (a
    // pair's commits arrive in both CTAs): those on the stages filled last and the
    // second CTA's done_bar are waited for here, a lane each, beside the epilogue's
    // last blocks (32 x 4096 x 4096 11.4 us; stage by stage 12.0, in the producer's branch
    // above, ahead of a split's barriers, 12.7); afull's were in the epilogue,
    // done_bar's in the MMA warp.
    if (warp == 0) {
        bool ok = true;
        if (lane < p.stages && ((filled >> lane) & 1u)) ok = mbar_wait(&empty[lane], (fph >> lane) & 1u);
        if (TWO && cta == 1 && lane == 31) ok = mbar_wait(done_bar, 0);
        if (!__all_sync(0xFFFFFFFFu, ok)) st_bits |= MILO_DEV_TIMEOUT;
    }
    // the stores have left shared memory and reached the outputs
    if (WIDE && warp >= 2 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    flag(p.dev_status, st_bits);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (TWO) tmem_dealloc2(tbase, p.tmem_cols);
        else tmem_dealloc(tbase, p.tmem_cols);
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
// MN-major, M = rows, N = bn.
static uint32_t dense_idesc(int bf16, int a_mn, int b_mn, int rows, int bn) {
    const uint32_t t = bf16 ? 1u : 0u;
    return (1u << 4) | (t << 7) | (t << 10) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(bn >> 3) << 17) | (static_cast<uint32_t>(rows >> 4) << 24);
}

template <bool SWAP, bool TWO, bool WIDE>
static cudaError_t dense_configure() {
    static std::atomic<bool> configured[64];     // set once per device (a repeat is harmless)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(dense_tc_kernel<SWAP, TWO, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDtSmemMax + 1024);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
    }
    return cudaSuccess;
}

template <bool SWAP, bool TWO, bool WIDE>
static cudaError_t launch_dense_tc(const DenseTc& p, int grid, int smem, cudaStream_t s) {
    const cudaError_t e = dense_configure<SWAP, TWO, WIDE>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kDtThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(TWO ? 2 : p.split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = TWO || p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, dense_tc_kernel<SWAP, TWO, WIDE>, p);
}

// Clusters of `split` CTAs (with a whole SM's shared memory each) that run at
// once on the current device; asked once per device and size.
static int max_clusters(int split) {
    static std::atomic<int> known[64][kDtMaxSplit + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[dev][split].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (dense_configure<false, false, true>() != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(split));
    cfg.blockDim = dim3(kDtThreads);
    cfg.dynamicSmemBytes = kDtSmemMax + 1024;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, dense_tc_kernel<false, false, true>, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        return 0;
    }
    known[dev][split].store(n, std::memory_order_relaxed);
    return n;
}

struct DensePlan {
    int bn, split, two;
};

// Columns of a tile and split of c, by an estimate in SM cycles of a CTA's
// work: a slice of c takes bn * 2 cycles of the tensor core or its bytes at 66
// bytes a cycle (what one SM was seen to draw from L2: 0.385 us for the 48 KB
// of a 256-column slice), whichever is longer; a tile takes its slices or, where
// these are few and another tile follows, its epilogue (600 and 20 a column: 3
// us for 256); and the last tile an epilogue.  All of it at least the operands'
// bytes at the measured copy rate (23 bytes a cycle and SM).
static double tile_cycles(double slices, double slice, int bn, double waves) {
    return waves > 1.0 ? std::max(slices * slice, 600.0 + 20.0 * bn) : slices * slice;
}
static double slice_cycles(int bn, int two) { return two ? 512.0 : std::max(2.0 * bn, (kDtAtom + bn * 128) / 66.0); }

// Tiles of the second product for a slot without an extra one of the first's.
static double fill_tiles(double c0, double c1) { return std::max(1.0, std::floor(c0 / c1)); }

// The longest slot of dense_item's schedule: t0 tiles of c0 cycles, t1 of c1.
static double schedule_cycles(double t0, double c0, double t1, double c1, double slots) {
    const double rounds = std::floor(t0 / slots), extra = t0 - rounds * slots, others = slots - extra;
    const double filled = std::min(t1, fill_tiles(c0, c1) * others);
    return rounds * c0 + std::max(extra > 0.0 ? c0 : 0.0, std::ceil(filled / others) * c1) +
           std::ceil((t1 - filled) / slots) * c1;
}

static double dense_plan(const DenseGemm* gs, int n, bool swap, int sms, DensePlan* plan) {
    double best = -1.0, dram = 0.0;
    int qmax = 0, kmax = 0;
    double P[2], Q[2], kblocks[2];
    for (int i = 0; i < n; ++i) {
        P[i] = swap ? gs[i].Q : gs[i].P;
        Q[i] = swap ? gs[i].P : gs[i].Q;
        kblocks[i] = (gs[i].C + kDtK - 1) / kDtK;
        dram += (P[i] + Q[i]) * gs[i].C * 2.0 / (23.0 * 148.0);
        qmax = std::max(qmax, static_cast<int>(Q[i]));
        kmax = std::max(kmax, static_cast<int>(kblocks[i]));
    }
    const int bn_swap = static_cast<int>(round_up(qmax, 16));
    for (int bn = swap ? bn_swap : 64; bn <= (swap ? bn_swap : 256); bn += 64) {
        if (!swap && bn > 64 && bn - 64 >= qmax) break;          // the tile would be part empty
        const double slice = slice_cycles(bn, 0);
        for (int split = 1; split <= kDtMaxSplit && (split == 1 || kmax >= 2 * split); ++split) {
            const auto count = [&](int i) { return std::ceil(P[i] / 128.0) * std::ceil(Q[i] / static_cast<double>(bn)); };
            const double tiles = count(0) + (n > 1 ? count(1) : 0.0);
            // clusters only where one wave holds them all
            if (split > 1 && tiles > max_clusters(split)) break;
            const double waves = split > 1 ? 1.0 : std::ceil(tiles / sms);
            const auto cycles = [&](int i) { return tile_cycles(std::ceil(kblocks[i] / split), slice, bn, waves); };
            const double work = split > 1 ? cycles(0)
                                          : schedule_cycles(count(0), cycles(0), n > 1 ? count(1) : 0.0, cycles(n - 1), sms);
            const double epilogue = 8.0 * bn * (split > 1 ? 1.0 / split : 1.0);
            const double cost = std::max(dram, work + 0.5 * waves * slice) + epilogue +
                                (split > 1 ? 1500.0 + 100.0 * split : 0.0);
            if (best < 0.0 || cost < best) {
                best = cost;
                *plan = DensePlan{bn, split, 0};
            }
        }
    }
    if (!swap && qmax > 128) {
        // pairs of CTAs: 256 x 256 tiles, each CTA bringing half of either operand
        // (32 KB a slice against the tensor cores' 512 cycles)
        const int pairs = max_clusters(2);
        const auto count = [&](int i) { return std::ceil(P[i] / 256.0) * std::ceil(Q[i] / 256.0); };
        if (pairs > 0) {
            const double waves = std::ceil((count(0) + (n > 1 ? count(1) : 0.0)) / pairs);
            const auto cycles = [&](int i) { return tile_cycles(kblocks[i], slice_cycles(256, 1), 256, waves); };
            const double work = schedule_cycles(count(0), cycles(0), n > 1 ? count(1) : 0.0, cycles(n - 1), pairs);
            const double cost = std::max(dram, work + 0.5 * waves * 512.0) + 8.0 * 256 + 500.0;
            if (cost < best) {
                best = cost;
                *plan = DensePlan{256, 1, 1};
            }
        }
    }
    return best;
}

// n products (two share a grid and an epilogue without bias, residual, z and
// act).  One without an output only takes part in the plan, so that the other's
// sums do not depend on it.
static milo_status launch_dense(const DenseGemm* gs, int n, bool swap, const char* what, cudaStream_t s) {
    DenseTc p;
    memset(&p, 0, sizeof(p));
    const void *a[2] = {}, *b[2] = {};
    bool wide = !swap;
    long long lda[2] = {}, ldb[2] = {};
    for (int i = 0; i < n; ++i) {
        const DenseGemm& g = gs[i];
        DenseProb& d = p.prob[i];
        d.P = swap ? g.Q : g.P;
        d.Q = swap ? g.P : g.Q;
        d.C = g.C;
        d.a_mn = swap ? g.b_mn : g.a_mn;
        d.b_mn = swap ? g.a_mn : g.b_mn;
        a[i] = swap ? g.b : g.a;
        b[i] = swap ? g.a : g.b;
        lda[i] = swap ? g.ldb : g.lda;
        ldb[i] = swap ? g.lda : g.ldb;
        d.kblocks = (d.C + kDtK - 1) / kDtK;
        d.y = g.y;
    }
    const DenseGemm& g = gs[0];
    const int sms = dense_sms();
    DensePlan plan{};
    dense_plan(gs, n, swap, sms, &plan);
    p.bn = plan.bn;
    p.split = plan.split;
    p.two = plan.two;
    const int tile_rows = p.two ? 2 * kDtRows : kDtRows;
    const int slots = p.two ? max_clusters(2) : sms;         // tiles at work at once
    int live = 0;
    for (int i = 0; i < n; ++i)
        if (p.prob[i].y) {
            p.prob[live] = p.prob[i];
            a[live] = a[i];
            b[live] = b[i];
            lda[live] = lda[i];
            ldb[live] = ldb[i];
            ++live;
        }
    if (live < n) memset(&p.prob[live], 0, sizeof(DenseProb));
    n = live;
    p.bf16 = g.bf16;
    long long tiles = 0;
    int kper = 0;
    for (int i = 0; i < n; ++i) {
        DenseProb& d = p.prob[i];
        d.tiles_p = (d.P + tile_rows - 1) / tile_rows;
        d.tiles_q = (d.Q + p.bn - 1) / p.bn;
        const long long t = static_cast<long long>(d.tiles_p) * d.tiles_q;
        if ((tiles += t) > 0x3FFFFFFF) return fail(MILO_ERR_UNSUPPORTED_SHAPE, std::string(what) + ": too many tiles");
        d.tiles = static_cast<int>(t);
        d.idesc = dense_idesc(p.bf16, d.a_mn, d.b_mn, p.two ? 2 * kDtRows : kDtRows, p.bn);
        kper = std::max(kper, (d.kblocks + p.split - 1) / p.split);
    }
    p.tiles = static_cast<int>(tiles);
    p.bufs = p.split == 1 && p.tiles > slots ? 2 : 1;
    const int b_rows = p.two ? p.bn / 2 : p.bn;              // of B per CTA
    p.stage_bytes = kDtAtom + b_rows * 128;
    // shared memory: the ring (then a split's partial blocks), the row form's
    // output buffers and bias, barriers
    const int es = g.y_dt == MILO_F32 ? 4 : 2, bias = swap ? 0 : kDtEpiWarps * kDtBias * 4;
    const int want = std::max(2, p.bufs == 2 ? kDtMaxStages : kper);
    for (int i = 0; i < n; ++i)
        wide = wide && p.prob[i].Q % 8 == 0 && aligned(p.prob[i].y, 16) && aligned(g.residual, 16) && aligned(g.z, 16);
    const auto ring = [&](int staging) {
        return std::min({kDtMaxStages, (kDtSmemMax - kDtEpiWarps * staging - bias - 1024) / p.stage_bytes, want});
    };
    p.out_bytes = 32 * 32 * es;
    p.out_bufs = 1;
    p.staging = swap ? 0 : 32 * dense_pitch(es);
    if (wide) {
        // Without a residual two buffers a warp let a store drain under the next
        // block; with one they cover its latency (a split loads one block ahead
        // and needs one).  As many as leave the ring four stages, or with a
        // residual three, if it can have those at all.
        const int z = g.residual && g.z ? 32 * 32 * 2 : 0;       // z's own, behind the others
        const int least = g.residual && p.split == 1 ? 2 : 1, most = !g.residual ? 2 : p.split == 1 ? kDtOutBufs : 1;
        const int enough = std::min(ring(least * p.out_bytes + z), g.residual ? 3 : 4);
        p.out_bufs = most;
        while (p.out_bufs > least && ring(p.out_bufs * p.out_bytes + z) < enough) --p.out_bufs;
        p.staging = p.out_bufs * p.out_bytes + z;
    }
    p.stages = ring(p.staging);
    const int staging = kDtEpiWarps * p.staging;
    const int w = swap ? 16 : kDtChunk;
    const int part = p.split > 1 ? static_cast<int>(round_up(4 * (p.bn / w), p.split)) * w * 128 : 0;
    p.off_staging = std::max(p.stages * p.stage_bytes, part);
    p.off_bias = p.off_staging + staging;
    p.off_bar = p.off_bias + bias;
    p.tmem_cols = 32;
    while (p.tmem_cols < static_cast<uint32_t>(p.bufs * p.bn)) p.tmem_cols *= 2;
    // A CTA takes at least its columns' share of the SM's shared memory, so CTAs
    // that run side by side never ask for more than the SM's 512 columns: an
    // allocation that waited while its cluster's other CTAs hold theirs could
    // wait for ever on a cluster of another stream in the same position.
    const int smem = std::max({p.off_bar + 512 + 1024, kTmemLeastShared,
                               static_cast<int>(p.tmem_cols) * ((kDtSmemMax + 1024) / 512)});
    p.bias = g.bias;
    p.residual = g.residual;
    p.z = g.z;
    p.act = g.act;
    p.y_dt = g.y_dt;
    p.dev_status = g.dev_status;

    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_UINT16;
    const CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B;
    for (int i = 0; i < n; ++i) {
        // K-major [rows, c]: box 64 c by the tile's rows; MN-major [c, rows]: box 64 rows by 64 c
        DenseProb& d = p.prob[i];
        milo_status st = d.a_mn ? make_map(&d.a_map, a[i], dt, d.P, d.C, lda[i] * 2, 64, kDtK, what, swz)
                                : make_map(&d.a_map, a[i], dt, d.C, d.P, lda[i] * 2, kDtK, kDtRows, what, swz);
        if (st != MILO_OK) return st;
        st = d.b_mn ? make_map(&d.b_map, b[i], dt, d.Q, d.C, ldb[i] * 2, 64, kDtK, what, swz)
                    : make_map(&d.b_map, b[i], dt, d.C, d.Q, ldb[i] * 2, kDtK, b_rows, what, swz);
        if (st != MILO_OK) return st;
        if (!wide) continue;
        // output blocks of 32 x 32
        const CUtensorMapDataType ydt = es == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : dt;
        const CUtensorMapSwizzle yswz = es == 4 ? swz : CU_TENSOR_MAP_SWIZZLE_64B;
        st = make_map(&d.y_map, d.y, ydt, d.Q, d.P, static_cast<uint64_t>(d.Q) * es, 32, 32, what, yswz);
        if (st == MILO_OK && p.z)
            st = make_map(&p.z_map, p.z, dt, d.Q, d.P, static_cast<uint64_t>(d.Q) * 2, 32, 32, what, CU_TENSOR_MAP_SWIZZLE_64B);
        if (st == MILO_OK && p.residual)
            st = make_map(&p.r_map, p.residual, ydt, d.Q, d.P, static_cast<uint64_t>(d.Q) * es, 32, 32, what, yswz);
        if (st != MILO_OK) return st;
    }
    const int used = p.split > 1 ? p.tiles : std::min(p.tiles, slots);       // CTAs, pairs or clusters at work
    const int grid = used * (p.two ? 2 : p.split);
    const double slice = slice_cycles(p.bn, p.two);
    const auto cycles = [&](int i) { return tile_cycles(p.prob[i].kblocks, slice, p.bn, p.bufs); };
    p.rounds = p.prob[0].tiles / used;
    p.extra = p.prob[0].tiles % used;
    p.fill = n > 1 ? static_cast<int>(fill_tiles(cycles(0), cycles(1))) : 0;
    cudaError_t e;
    if (swap) e = launch_dense_tc<true, false, false>(p, grid, smem, s);
    else if (p.two) e = wide ? launch_dense_tc<false, true, true>(p, grid, smem, s) : launch_dense_tc<false, true, false>(p, grid, smem, s);
    else e = wide ? launch_dense_tc<false, false, true>(p, grid, smem, s) : launch_dense_tc<false, false, false>(p, grid, smem, s);
    return check_cuda(e, what);
}

// Few rows of A (tokens): they become the columns.
static bool few_rows(const DenseGemm& g) { return g.P <= 128 && !g.a_mn; }

milo_status launch_dense_gemm(const DenseGemm& g, const char* what, cudaStream_t s) {
    if (g.P <= kDenseFewRows && !g.a_mn && !g.b_mn) return launch_dense_few(g, what, s);
    return launch_dense(&g, 1, few_rows(g), what, s);
}

milo_status launch_dense_pair(const DenseGemm& g0, const DenseGemm& g1, const char* what, cudaStream_t s) {
    // the longer sums first: the shorter ones fill the last wave
    const DenseGemm gs[2] = {g0.C >= g1.C ? g0 : g1, g0.C >= g1.C ? g1 : g0};
    if (!g0.y && !g1.y) return MILO_OK;
    // one launch unless the two want different forms, tiles or splits by more
    // than a second launch costs (about 4000 cycles).  By the shapes alone: a
    // gradient without the other has the same bits.
    DensePlan plan;
    const int sms = dense_sms();
    const bool few0 = few_rows(g0), few1 = few_rows(g1);
    const double apart = dense_plan(&g0, 1, few0, sms, &plan) + dense_plan(&g1, 1, few1, sms, &plan) + 4000.0;
    if (dense_plan(gs, 2, false, sms, &plan) <= apart) return launch_dense(gs, 2, false, what, s);
    milo_status r = g0.y ? launch_dense(&g0, 1, few0, what, s) : MILO_OK;
    if (r == MILO_OK && g1.y) r = launch_dense(&g1, 1, few1, what, s);
    return r;
}

}  // namespace milo
