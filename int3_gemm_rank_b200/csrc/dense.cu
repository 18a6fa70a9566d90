// dense.cu -- the dense 16-bit projection and its gradients
// (milo_dense_linear, milo_dense_linear_backward): host side, and the pass
// that turns dy into dz.
//
//     z = x W^T + b,  y = act(z) + r
//     dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum_m dz
// All three products are D[p, q] = sum_c A(p, c) B(q, c) with each operand
// stored along c (K-major) or along its rows (MN-major):
//     forward  A = x  [M, K] K-major,   B = W [N, K] K-major
//     dx       A = dz [M, N] K-major,   B = W [N, K] MN-major (c = n)
//     dW       A = dz [M, N] MN-major,  B = x [M, K] MN-major (c = m)
// so nothing is ever transposed in memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "milo_dense.cuh"
#include "milo_host.h"

namespace milo {

// ---------------------------------------------------------------------------
// dz = dy act'(z), and its column sums
//
// dz is computed in fp32 and rounded once, to the product's type, before it is
// multiplied: the tensor cores take 16-bit operands, and dz held in two 16-bit
// parts would double both products (8192 x 4096 x 4096: 375 us more).  It puts
// dx and dW 1.4 times as far from the exact gradient as the rounding of their own
// output (there, bf16, silu: 0.0023 against 0.0017 in norm), whatever dy's type.
// db sums dz unrounded; without an activation and with dy in the product's type
// nothing is rounded.
// ---------------------------------------------------------------------------
constexpr int kDzCols = 256;        // columns of a block
constexpr int kDzThreads = 256;     // 32 column lanes by 8 row lanes

struct DzParams {
    const void* dy;             // [M, N] in dy_dt
    const void* z;              // [M, N] or NULL
    void* dz;                   // [M, ldz] in the product's type, columns N..ldz-1 zero; NULL: not written
    float* part;                // [row blocks][N] column sums, or NULL
    void* db;                   // with one row block: the sums themselves, in the product's type
    int32_t* dev_status;
    int M, N, ldz, dy_dt, bf16, act;
    int rows, col_blocks;       // rows of a block; blocks of columns
};

// A lane's eight columns of a row of 256 that starts at column n0: VEC (dy and z
// in whole 16-byte pieces) n0 + 8 lane.., else n0 + lane, + 32, ...
template <int DT, bool VEC>
__device__ __forceinline__ void dz_load(const void* p, size_t row, int N, int n0, int lane, float (&v)[8]) {
    const size_t i = row * N + n0;
    if constexpr (VEC) {
        if (n0 + 8 * lane < N) {
            if constexpr (DT == MILO_F32) {
                const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + 8 * lane);
                const float4 a = q[0], b = q[1];
                v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
                v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
            } else {
                const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i + 8 * lane);
                const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = unpack16<DT>(w[q / 2], q & 1);
            }
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = 0.0f;
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = n0 + lane + 32 * q < N ? elem_load<DT>(p, i + lane + 32 * q) : 0.0f;
    }
}

// One block: p.rows rows of 256 columns; a row lane takes every eighth row.  The
// column sums of a thread's rows are its own, and the eight row lanes meet in
// shared memory in lane order.  Bound by memory (dy and z read, dz written
// once); many small blocks carry it: with two or four rows of a thread in
// flight the registers cost more warps than the loads gain (8192 x 4096 bf16,
// silu, sums alone: 28 us with one, 37 with two, 57 with four).
// Blocks an SM should hold at the least, 0: as the compiler likes.  Sums alone,
// 8192 x 8192, 16-bit dy: silu 49 us with seven, 56 without; gelu 76 with one
// (so, as many registers as its loads like), 72 with seven and 69 without; no
// activation 26 with one and 29 without; at width 8191 silu 75 with one and 69
// without.
template <int DYT, bool VEC, int ACT>
constexpr int dz_blocks() {
    if (ACT == MILO_ACT_NONE || (ACT == MILO_ACT_RELU && !VEC)) return 1;
    return ACT == MILO_ACT_SILU && VEC && DYT != MILO_F32 ? 7 : 0;
}
template <int DYT, int ZT, bool VEC, int ACT>
__global__ void __launch_bounds__(kDzThreads, dz_blocks<DYT, VEC, ACT>()) dense_dz_kernel(const DzParams p) {
    __shared__ float red[8][kDzCols];
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int rb = static_cast<int>(blockIdx.x) / p.col_blocks, cb = static_cast<int>(blockIdx.x) % p.col_blocks;
    const int n0 = cb * kDzCols;
    const int m0 = rb * p.rows, m1 = min(p.M, m0 + p.rows);
    int32_t st = 0;
    float sum[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[q] = 0.0f;
    for (int m = m0 + rl; m < m1; m += 8) {
        float v[8];
        dz_load<DYT, VEC>(p.dy, m, p.N, n0, lane, v);
        if constexpr (ACT != MILO_ACT_NONE) {
            float z[8];
            dz_load<ZT, VEC>(p.z, m, p.N, n0, lane, z);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = __fmul_rn(v[q], act_slope<ACT>(z[q]));    // no FMA into the sum: db alone has the same bits
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] += v[q];
        if (p.dz) {
            uint16_t* d = static_cast<uint16_t*>(p.dz) + static_cast<size_t>(m) * p.ldz + n0;
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = pack16<ZT>(v[2 * q], v[2 * q + 1]);
            if constexpr (ZT == MILO_F16) half_range(v, w, st);
            if constexpr (VEC) {
                if (n0 + 8 * lane < p.ldz) *reinterpret_cast<uint4*>(d + 8 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (n0 + lane + 32 * q < p.ldz)
                        d[lane + 32 * q] = static_cast<uint16_t>(q & 1 ? w[q / 2] >> 16 : w[q / 2] & 0xFFFFu);
            }
        }
    }
    if (p.part) {
#pragma unroll
        for (int q = 0; q < 8; ++q) red[rl][VEC ? 8 * lane + q : lane + 32 * q] = sum[q];
        __syncthreads();
        const int n = n0 + threadIdx.x;
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s += red[q][threadIdx.x];
        if (n < p.N) {
            if (p.db) elem_store<ZT>(p.db, n, s, st);
            else p.part[static_cast<size_t>(rb) * p.N + n] = s;
        }
    }
    flag(p.dev_status, st);
}

template <int DYT, int ZT, bool VEC>
static cudaError_t run_dz_act(const DzParams& p, int grid, cudaStream_t s) {
    void (*k)(DzParams) = dense_dz_kernel<DYT, ZT, VEC, MILO_ACT_NONE>;
    if (p.act == MILO_ACT_RELU) k = dense_dz_kernel<DYT, ZT, VEC, MILO_ACT_RELU>;
    else if (p.act == MILO_ACT_SILU) k = dense_dz_kernel<DYT, ZT, VEC, MILO_ACT_SILU>;
    else if (p.act == MILO_ACT_GELU) k = dense_dz_kernel<DYT, ZT, VEC, MILO_ACT_GELU>;
    else if (p.act == MILO_ACT_GELU_TANH) k = dense_dz_kernel<DYT, ZT, VEC, MILO_ACT_GELU_TANH>;
    return launch_pdl(k, dim3(static_cast<unsigned>(grid)), dim3(kDzThreads), 0, s, p);
}

template <int DYT, int ZT>
static cudaError_t run_dz_vec(const DzParams& p, bool vec, int grid, cudaStream_t s) {
    return vec ? run_dz_act<DYT, ZT, true>(p, grid, s) : run_dz_act<DYT, ZT, false>(p, grid, s);
}

template <int ZT>
static cudaError_t run_dz(const DzParams& p, bool vec, int grid, cudaStream_t s) {
    if (p.dy_dt == MILO_F32) return run_dz_vec<MILO_F32, ZT>(p, vec, grid, s);
    if (p.dy_dt == MILO_F16) return run_dz_vec<MILO_F16, ZT>(p, vec, grid, s);
    return run_dz_vec<MILO_BF16, ZT>(p, vec, grid, s);
}

// db[n] = the row blocks' sums: LANES lanes of a column take every LANES'th block
// in order, and meet in lane order.  Bound by the latency of its loads: 32 lanes
// where there are many blocks (979 blocks of 78 columns, db in all 7.0 us, with
// eight lanes 10.0; 96 blocks of 1411 columns 8.7 and 7.8).
template <int LANES>
__global__ void __launch_bounds__(32 * LANES) dense_db_kernel(const float* __restrict__ part, int blocks, int N, int bf16,
                                                                 uint16_t* __restrict__ db, int32_t* dev_status) {
    __shared__ float red[LANES][32];
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int n = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (n < N)
#pragma unroll 8
        for (int b = rl; b < blocks; b += LANES) s += part[static_cast<size_t>(b) * N + n];
    red[rl][lane] = s;
    __syncthreads();
    if (rl > 0 || n >= N) return;
    int32_t st = 0;
#pragma unroll
    for (int q = 1; q < LANES; ++q) s += red[q][lane];
    db[n] = round16(s, bf16, st);
    flag(dev_status, st);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

constexpr long long kDenseMaxElems = 1LL << 38;

static milo_status check_dense(const char* what, milo_dtype dt, int M, int N, int K, int act) {
    const std::string f = what;
    if (dt != MILO_F16 && dt != MILO_BF16) return fail(MILO_ERR_INVALID_ARG, f + ": x and W must be fp16 or bf16");
    if (M < 0 || N < 1 || K < 1) return fail(MILO_ERR_INVALID_ARG, f + ": M must be >= 0, N and K >= 1");
    if (act < MILO_ACT_NONE || act > MILO_ACT_GELU_TANH) return fail(MILO_ERR_INVALID_ARG, f + ": unknown activation");
    if (K % 8) return fail(MILO_ERR_UNSUPPORTED_SHAPE, f + ": K must be a multiple of 8");
    if (M > kMaxProjK || N > kMaxProjK || K > kMaxProjK)
        return fail(MILO_ERR_UNSUPPORTED_SHAPE, f + ": M, N and K must be at most 2^24");
    if (static_cast<long long>(M) * N > kDenseMaxElems || static_cast<long long>(M) * K > kDenseMaxElems ||
        static_cast<long long>(N) * K > kDenseMaxElems)
        return fail(MILO_ERR_UNSUPPORTED_SHAPE, f + ": M*N, M*K and N*K must be at most 2^38");
    return MILO_OK;
}

static bool out_ok(milo_dtype d) { return d == MILO_F16 || d == MILO_BF16 || d == MILO_F32; }
static uintptr_t elem(milo_dtype d) { return d == MILO_F32 ? 4 : 2; }

// Scratch of the backward pass: dz [M, ldz] in the product's type (rows padded
// to 128 bytes, what one row of a TMA box brings) and the column sums of each
// row block.
struct DenseWs {
    size_t dz, part, total;
    int ldz, rows, blocks;
};

static DenseWs dense_ws(int M, int N) {
    DenseWs w;
    w.ldz = static_cast<int>(round_up(N, 64));
    // rows of a block: 64, fewer while the blocks do not fill the SMs four deep --
    // but up to 64 rows in one, whose column sums then need no second kernel (128
    // rows: 8192 x 8192 bf16 without an activation, sums alone, 26 us against 27,
    // but 8192 x 4096 with gelu 43 against 38 and with silu 32 against 28)
    w.rows = 64;
    const long long col_blocks = (N + kDzCols - 1) / kDzCols;
    while (M > 64 && w.rows > 8 && (M + w.rows - 1) / w.rows * col_blocks < 4 * 148) w.rows /= 2;
    w.blocks = (M + w.rows - 1) / w.rows;
    w.dz = 0;
    w.part = round_up(static_cast<size_t>(M) * w.ldz * 2, 256);
    w.total = w.part + round_up(static_cast<size_t>(w.blocks) * N * 4, 256);
    return w;
}

}  // namespace milo

using namespace milo;

extern "C" milo_status milo_dense_linear(const void* x, const void* W, milo_dtype dt, int32_t M, int32_t N,
                                         int32_t K, const void* bias, const void* residual, int32_t act, void* y,
                                         milo_dtype y_dt, void* z, int32_t* dev_status, void* stream) {
    clear_error();
    milo_status s = check_dense("milo_dense_linear", dt, M, N, K, act);
    if (s != MILO_OK) return s;
    if (!out_ok(y_dt)) return fail(MILO_ERR_INVALID_ARG, "milo_dense_linear: bad y dtype");
    if (M == 0) return MILO_OK;
    if (!x || !W || !y) return fail(MILO_ERR_INVALID_ARG, "milo_dense_linear: NULL pointer");
    if (!aligned(x, 16) || !aligned(W, 16))
        return fail(MILO_ERR_INVALID_ARG, "milo_dense_linear: x and W must be 16-byte aligned");
    if (!aligned(y, elem(y_dt)) || !aligned(residual, elem(y_dt)) || !aligned(bias, 2) || !aligned(z, 2) ||
        !aligned(dev_status, 4))
        return fail(MILO_ERR_INVALID_ARG,
                    "milo_dense_linear: bias, residual, y, z and dev_status must be aligned to their elements");
    const DenseGemm g = {x, W, K, K, 0, 0, M, N, K, dt == MILO_BF16, bias, residual, act, y, y_dt, z, dev_status};
    return launch_dense_gemm(g, "milo_dense_linear", static_cast<cudaStream_t>(stream));
}

extern "C" milo_status milo_dense_linear_backward_workspace_bytes(int32_t M, int32_t N, int32_t K, size_t* bytes) {
    clear_error();
    if (!bytes) return fail(MILO_ERR_INVALID_ARG, "milo_dense_linear_backward_workspace_bytes: NULL argument");
    const milo_status s = check_dense("milo_dense_linear_backward_workspace_bytes", MILO_BF16, M, N, K, MILO_ACT_NONE);
    if (s != MILO_OK) return s;
    *bytes = dense_ws(M, N).total;
    return MILO_OK;
}

extern "C" milo_status milo_dense_linear_backward(const void* dy, milo_dtype dy_dt, const void* x, const void* W,
                                                  milo_dtype dt, int32_t M, int32_t N, int32_t K, int32_t act,
                                                  const void* z, void* dx, void* dW, void* db, void* ws,
                                                  size_t ws_bytes, int32_t* dev_status, void* stream) {
    clear_error();
    milo_status s = check_dense("milo_dense_linear_backward", dt, M, N, K, act);
    if (s != MILO_OK) return s;
    if (!out_ok(dy_dt)) return fail(MILO_ERR_INVALID_ARG, "milo_dense_linear_backward: bad dy dtype");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!dx && !dW && !db) return MILO_OK;
    if (M == 0) {
        // an empty batch: the parameters' gradients are zero
        if (dW && (s = check_cuda(cudaMemsetAsync(dW, 0, static_cast<size_t>(N) * K * 2, st), "dW")) != MILO_OK) return s;
        if (db && (s = check_cuda(cudaMemsetAsync(db, 0, static_cast<size_t>(N) * 2, st), "db")) != MILO_OK) return s;
        return MILO_OK;
    }
    if (!dy || (dW && !x) || (dx && !W) || (act != MILO_ACT_NONE && !z) || !ws)
        return fail(MILO_ERR_INVALID_ARG, "milo_dense_linear_backward: NULL pointer");
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(dx, 16) || !aligned(dW, 16))
        return fail(MILO_ERR_INVALID_ARG, "milo_dense_linear_backward: x, W, dx and dW must be 16-byte aligned");
    if (!aligned(dy, elem(dy_dt)) || !aligned(z, 2) || !aligned(db, 2) || !aligned(dev_status, 4))
        return fail(MILO_ERR_INVALID_ARG,
                    "milo_dense_linear_backward: dy, z, db and dev_status must be aligned to their elements");
    if (!aligned(ws, 256)) return fail(MILO_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    const DenseWs w = dense_ws(M, N);
    if (ws_bytes < w.total) return fail(MILO_ERR_WORKSPACE, "milo_dense_linear_backward: workspace too small");
    char* base = static_cast<char*>(ws);

    // dy itself serves as dz when nothing has to be applied, converted or padded
    const bool direct = act == MILO_ACT_NONE && dy_dt == dt && N % 8 == 0 && aligned(dy, 16);
    const bool want_dz = !direct && (dx || dW);
    if (want_dz || db) {
        const DzParams p = {dy, act == MILO_ACT_NONE ? nullptr : z, want_dz ? base + w.dz : nullptr,
                            db ? reinterpret_cast<float*>(base + w.part) : nullptr, w.blocks == 1 ? db : nullptr,
                            dev_status, M, N, w.ldz,
                            static_cast<int>(dy_dt), dt == MILO_BF16, act, w.rows, (w.ldz + kDzCols - 1) / kDzCols};
        const bool vec = N % 8 == 0 && aligned(dy, 16) && (act == MILO_ACT_NONE || aligned(z, 16));
        const int grid = w.blocks * p.col_blocks;
        s = check_cuda(dt == MILO_BF16 ? run_dz<MILO_BF16>(p, vec, grid, st) : run_dz<MILO_F16>(p, vec, grid, st), "dz");
        if (s != MILO_OK) return s;
    }
    if (db && w.blocks > 1) {
        const bool many = w.blocks >= 256;
        s = check_cuda(launch_pdl(many ? dense_db_kernel<32> : dense_db_kernel<8>, dim3((N + 31) / 32), dim3(many ? 1024 : 256), 0, st,
                                  reinterpret_cast<const float*>(base + w.part), w.blocks, N, dt == MILO_BF16 ? 1 : 0,
                                  static_cast<uint16_t*>(db), dev_status),
                       "db");
        if (s != MILO_OK) return s;
    }
    const void* dz = direct ? dy : base + w.dz;
    const long long ldz = direct ? N : w.ldz;
    const DenseGemm gx = {dz, W, ldz, K, 0, 1, M, K, N, dt == MILO_BF16, nullptr, nullptr, MILO_ACT_NONE, dx, dt,
                          nullptr, dev_status};
    const DenseGemm gw = {dz, x, ldz, K, 1, 1, N, K, M, dt == MILO_BF16, nullptr, nullptr, MILO_ACT_NONE, dW, dt,
                          nullptr, dev_status};
    return launch_dense_pair(gx, gw, "dx and dW", st);
}
