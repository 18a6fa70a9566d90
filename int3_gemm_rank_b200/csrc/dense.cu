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
// ---------------------------------------------------------------------------
constexpr int kDzRows = 64;         // rows of a block
constexpr int kDzThreads = 256;

struct DzParams {
    const void* dy;             // [M, N] in dy_dt
    const void* z;              // [M, N] or NULL
    void* dz;                   // [M, ldz] in the product's type, columns N..ldz-1 zero; NULL: not written
    float* part;                // [row blocks][N] column sums, or NULL
    int32_t* dev_status;
    int M, N, ldz, dy_dt, bf16, act;
};

// One block: kDzRows rows of 256 columns, a thread per column, so the column
// sum is the thread's own (fp32, row order).
__global__ void __launch_bounds__(kDzThreads) dense_dz_kernel(const DzParams p) {
    grid_dep_launch();
    grid_dep_wait();
    const int n = blockIdx.y * kDzThreads + threadIdx.x;
    const int m0 = blockIdx.x * kDzRows;
    if (n >= (p.dz ? p.ldz : p.N)) return;
    int32_t st = 0;
    float sum = 0.0f;
    for (int m = m0; m < min(p.M, m0 + kDzRows); ++m) {
        float v = 0.0f;
        if (n < p.N) {
            const size_t i = static_cast<size_t>(m) * p.N + n;
            v = load_any(p.dy, i, p.dy_dt);
            if (p.z) v *= dense_dact(p.act, load16(p.z, i, p.bf16));
        }
        sum += v;
        if (p.dz) static_cast<uint16_t*>(p.dz)[static_cast<size_t>(m) * p.ldz + n] = round16(v, p.bf16, st);
    }
    if (p.part && n < p.N) p.part[static_cast<size_t>(blockIdx.x) * p.N + n] = sum;
    flag(p.dev_status, st);
}

// db[n] = the row blocks' sums, in order.
__global__ void __launch_bounds__(256) dense_db_kernel(const float* __restrict__ part, int blocks, int N, int bf16,
                                                       uint16_t* __restrict__ db, int32_t* dev_status) {
    grid_dep_launch();
    grid_dep_wait();
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    int32_t st = 0;
    float s = 0.0f;
    for (int b = 0; b < blocks; ++b) s += part[static_cast<size_t>(b) * N + n];
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
// to 16 bytes, as the products' tiles are copied) and the column sums of each
// row block.
struct DenseWs {
    size_t dz, part, total;
    int ldz, blocks;
};

static DenseWs dense_ws(int M, int N) {
    DenseWs w;
    w.ldz = static_cast<int>(round_up(N, 8));
    w.blocks = (M + kDzRows - 1) / kDzRows;
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
    if (!aligned(y, elem(y_dt)) || !aligned(residual, elem(y_dt)) || !aligned(bias, 2) || !aligned(z, 2))
        return fail(MILO_ERR_INVALID_ARG, "milo_dense_linear: bias, residual, y and z must be aligned to their elements");
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
    if (!aligned(dy, elem(dy_dt)) || !aligned(z, 2) || !aligned(db, 2))
        return fail(MILO_ERR_INVALID_ARG, "milo_dense_linear_backward: dy, z and db must be aligned to their elements");
    if (!aligned(ws, 256)) return fail(MILO_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    const DenseWs w = dense_ws(M, N);
    if (ws_bytes < w.total) return fail(MILO_ERR_WORKSPACE, "milo_dense_linear_backward: workspace too small");
    char* base = static_cast<char*>(ws);

    // dy itself serves as dz when nothing has to be applied, converted or padded
    const bool direct = act == MILO_ACT_NONE && dy_dt == dt && N % 8 == 0 && aligned(dy, 16);
    const bool want_dz = !direct && (dx || dW);
    if (want_dz || db) {
        DzParams p = {dy, act == MILO_ACT_NONE ? nullptr : z, want_dz ? base + w.dz : nullptr,
                      db ? reinterpret_cast<float*>(base + w.part) : nullptr, dev_status, M, N, w.ldz,
                      static_cast<int>(dy_dt), dt == MILO_BF16, act};
        const dim3 grid(static_cast<unsigned>(w.blocks), static_cast<unsigned>((w.ldz + kDzThreads - 1) / kDzThreads));
        if (grid.y > 65535) return fail(MILO_ERR_UNSUPPORTED_SHAPE, "milo_dense_linear_backward: N too large");
        if ((s = check_cuda(launch_pdl(dense_dz_kernel, grid, dim3(kDzThreads), 0, st, p), "dz")) != MILO_OK) return s;
    }
    if (db) {
        s = check_cuda(launch_pdl(dense_db_kernel, dim3((N + 255) / 256), dim3(256), 0, st,
                                  reinterpret_cast<const float*>(base + w.part), w.blocks, N, dt == MILO_BF16 ? 1 : 0,
                                  static_cast<uint16_t*>(db), dev_status),
                       "db");
        if (s != MILO_OK) return s;
    }
    const void* dz = direct ? dy : base + w.dz;
    const long long ldz = direct ? N : w.ldz;
    if (dx) {
        const DenseGemm g = {dz, W, ldz, K, 0, 1, M, K, N, dt == MILO_BF16, nullptr, nullptr, MILO_ACT_NONE, dx, dt,
                             nullptr, dev_status};
        if ((s = launch_dense_gemm(g, "dx", st)) != MILO_OK) return s;
    }
    if (dW) {
        const DenseGemm g = {dz, x, ldz, K, 1, 1, N, K, M, dt == MILO_BF16, nullptr, nullptr, MILO_ACT_NONE, dW, dt,
                             nullptr, dev_status};
        if ((s = launch_dense_gemm(g, "dW", st)) != MILO_OK) return s;
    }
    return MILO_OK;
}
