// exchange_rows.cuh -- the kernel behind milo_combine, the gradients of both moves
// and the dispatch of rows that do not start on 16-byte boundaries: a token's
// k expert rows (and its own row) streamed through shared memory
// (instantiated in exchange_*.cu).
//
// With f = t*k + j, p = inv_perm[f]:
//     dispatch           xs[p] = w[f] x[t]
//     combine            y[t]  = r[t] + sum_j w[f] ys[p]
//     combine_backward   dys[p] = w[f] dy[t],       dw[f] = <dy[t], ys[p]>
//     dispatch_backward  dx[t] = sum_j w[f] dxs[p], dw[f] = <dxs[p], x[t]>
//
// Bound by memory, and the rows lie scattered, so what counts is bytes in
// flight.  Every warp works alone: lane j fetches slot j's index and brings
// that row's piece to the warp's own ring in shared memory with one bulk copy
// (lane k the token's), two items ahead of the one being added up, so that a
// block keeps its whole ring (about 200 KB) in flight whatever the registers
// hold, and no warp waits for another.  Dropped slots get no place in the
// ring, so the sums run over the live ones without a test.  Sums and dot
// products run in fp32 in a fixed order.
//
// A row that starts off a 16-byte boundary comes in the aligned pieces that
// cover it; its columns are then read one element per lane (lane, lane + 32,
// ...), which no misalignment slows down, and written the same way.
//
// Measured (B200, device time, of the measured copy rate): combine 8192 x 2048,
// k 6, bf16 with a residual 42.3 us (0.97; 54 with 8 warps a block, 48 with
// 16), at width 2047 48.5 us (0.85); dispatch's gradient 8192 x 4096, k 2, bf16 32.3
// us (0.95), with router weights 43.1 us (0.95); combine's gradient 5003 x 2048, k
// 6, fp16 47 us (0.82), and at width 2051 56 us (0.70), where the one-element
// reads and stores bound it; dispatch 8192 x 2047, k 6, bf16 53 us (0.68).  Threads that load
// the rows into registers reached 0.62 of the rate at best.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "milo_exchange.cuh"
#include "milo_host.h"
#include "milo_tc.cuh"

namespace milo {

enum { kXDispatch, kXCombine, kXCombineGrad, kXDispatchGrad };

constexpr int kXrWarps = 12;
constexpr int kXrTeams[] = {1, 2, 4};        // warps that may share a token's pieces (gradients)
constexpr int kXrThreads = 32 * kXrWarps;
constexpr int kXrStages = 2;
constexpr int kXrSlack = 32;                 // bytes a row that starts off a 16-byte boundary may add
constexpr int kXrSmem = 216 * 1024;

struct XRowsParams {
    ExchangeParams x;
    int cols, nch;              // columns of a piece (a multiple of 64; the last may be up to 64 longer), pieces of a row
    int pitch, nrows;           // bytes between a stage's rows; rows of a stage
    int team;                   // gradients: warps per token
};

struct alignas(16) XMeta {      // a live slot of a stage
    int32_t row, m;             // expert row; elements before its first column in shared memory
    float w;
    int32_t slot;
};

// Brings `len` bytes at global address `a` to shared memory so that the byte
// at address g lands at dst + (g - floor16(a)).  [tb, te) is the tensor: a
// 16-byte piece that would leave it is copied by element instead.  Returns the
// bytes of the bulk copy [lo, lo + bytes).
template <typename T, bool AL>
__device__ __forceinline__ uint32_t row_window(uintptr_t a, uint32_t len, uintptr_t tb, uintptr_t te, uint8_t* dst,
                                               uintptr_t& lo) {
    if constexpr (AL) {
        lo = a;
        return len;
    } else {
        const uintptr_t base = a & ~static_cast<uintptr_t>(15);
        uintptr_t hi = (a + len + 15) & ~static_cast<uintptr_t>(15);
        lo = base;
        if (lo < tb) lo += 16;
        if (hi > te) hi -= 16;
        if (hi < lo) hi = lo;
        auto copy = [&](uintptr_t g0, uintptr_t g1) {
            for (uintptr_t g = g0; g < g1; g += sizeof(T))
                *reinterpret_cast<T*>(dst + (g - base)) = *reinterpret_cast<const T*>(g);
        };
        copy(a, a + len < lo ? a + len : lo);
        copy(a > hi ? a : hi, a + len);
        // a later bulk copy to this place of the ring must not be overtaken by these
        // stores (two pieces of a tensor at most have any)
        if (lo > base || hi < a + len) fence_proxy_async_smem();
        return static_cast<uint32_t>(hi - lo);
    }
}

// The lane's eight columns of a block of 256 that starts at column v0 of a row
// in shared memory (m elements in, see row_window); 0 from column nc on (FULL:
// the block ends before).  AL: columns v0 + 8 lane.., else v0 + lane, + 32, ...
template <typename T, bool AL, bool FULL>
__device__ __forceinline__ void read_cols(const uint8_t* row, int m, int v0, int lane, int nc, float (&v)[8]) {
    if constexpr (AL) {
        if (FULL || v0 + 8 * lane < nc) load8<T>(row + (v0 + 8 * lane) * sizeof(T), v);
    } else {
        const T* p = reinterpret_cast<const T*>(row) + m + v0 + lane;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = FULL || v0 + lane + 32 * q < nc ? to_f32(p[32 * q]) : 0.0f;
    }
}

// The same columns of a row in global memory (`row` points to column 0 of the piece).
template <typename T, bool AL, bool FULL>
__device__ __forceinline__ void write_cols(T* row, int v0, int lane, int nc, const float (&v)[8], int32_t& st) {
    if constexpr (AL) {
        if (FULL || v0 + 8 * lane < nc) store8<T>(row + v0 + 8 * lane, v, st);
    } else {
        T e[8];
        to_elems<T>(v, e, st);
        T* d = row + v0 + lane;
        if (FULL || v0 + 256 <= nc) {
#pragma unroll
            for (int q = 0; q < 8; ++q) d[32 * q] = e[q];
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (v0 + lane + 32 * q < nc) d[32 * q] = e[q];
        }
    }
}

template <typename TI, typename TO, bool AL, int KM, int MODE>
__global__ void __launch_bounds__(kXrThreads, 1) exchange_rows_kernel(const XRowsParams P) {
    using TT = typename std::conditional<MODE == kXCombine, TO, TI>::type;   // the token row's type
    constexpr bool kLoadRows = MODE != kXDispatch, kDot = MODE == kXCombineGrad || MODE == kXDispatchGrad;
    constexpr bool kToRows = MODE == kXDispatch || MODE == kXCombineGrad;    // writes expert rows
    constexpr int KB = KM < 4 ? KM : 4;                                       // slots read side by side
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kXrWarps][kXrStages];
    __shared__ XMeta meta[kXrWarps][kXrStages][KM + 1];                      // live slots, then the token's row
    __shared__ int live[kXrWarps][kXrStages];
    // gradients with several warps per token: their partial dot products, two
    // tokens deep (filled: all but the leader have written; taken: read)
    __shared__ float part[kDot ? kXrWarps : 1][2][KM];
    __shared__ uint64_t filled[kXrWarps][2], taken[kXrWarps][2];
    const ExchangeParams& p = P.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_launch();
    if (lane < kXrStages) mbar_init(&full[warp][lane], 1);
    if (kDot && lane < 2) {
        mbar_init(&filled[warp][lane], max(1, P.team - 1));
        mbar_init(&taken[warp][lane], 1);
    }
    fence_barrier_init();
    if (kDot && P.team > 1) __syncthreads();      // the barriers of the team's first warp
    __syncwarp();
    grid_dep_wait();

    const int rows = p.T * p.k;
    const bool tok_is_src = MODE == kXDispatch || MODE == kXCombineGrad;
    const TI* exp_rows = static_cast<const TI*>(tok_is_src ? p.other : p.src);
    const TT* tok_rows = static_cast<const TT*>(tok_is_src ? p.src : p.other);
    const bool has_tok = MODE != kXCombine || p.other;
    const int tok_at = kLoadRows ? p.k : 0;                                  // the token's row of a stage
    uint8_t* ring = smem + static_cast<size_t>(warp) * kXrStages * P.nrows * P.pitch;
    // The pieces of all tokens are spread over the warps, over the blocks first.
    // A gradient's token belongs to a team of warps of one block, whose
    // registers hold its dot products: member g takes pieces g, g + team, ...
    const int team = kDot ? P.team : 1, g = kDot ? warp % team : 0, lead = warp - g;
    const int gw = warp / team * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    const int nw = kXrWarps / team * static_cast<int>(gridDim.x);
    struct Cursor {
        int t, ch;
    };
    const int dt = kDot ? 0 : nw / P.nch, dch = kDot ? team : nw - nw / P.nch * P.nch;
    auto advance = [&](Cursor& c) {
        c.ch += dch;
        c.t += dt;
        if (c.ch >= P.nch) {
            c.ch = kDot ? g : c.ch - P.nch;
            c.t += kDot ? nw : 1;
        }
    };
    int32_t st = 0;
    int nidx = -1;
    float nwt = 1.0f;
    // lane j's index and weight of an item, ahead of its copies
    auto fetch = [&](const Cursor& c) {
        nidx = -1;
        if (c.t < p.T && lane < p.k) {
            nidx = p.inv_perm[c.t * p.k + lane];
            nwt = p.w ? p.w[c.t * p.k + lane] : 1.0f;
        }
    };
    Cursor head{kDot ? gw : gw / P.nch, kDot ? g : gw - gw / P.nch * P.nch};
    Cursor tail = head;
    auto issue = [&](int s) {
        const int c0 = head.ch * P.cols, nc = head.ch == P.nch - 1 ? p.H - c0 : P.cols;
        const int r = lane < p.k ? slot_row(nidx, rows, st) : -1;
        const unsigned mask = __ballot_sync(0xFFFFFFFFu, r >= 0);
        const int pos = __popc(mask & ((1u << lane) - 1u));
        const bool tok = lane == p.k && has_tok;
        uint8_t* dst = ring + (s * P.nrows + (tok ? tok_at : pos)) * P.pitch;
        uintptr_t lo = 0, a = 0;
        uint32_t bytes = 0;
        if (tok) {
            const uintptr_t tb = reinterpret_cast<uintptr_t>(tok_rows);
            a = reinterpret_cast<uintptr_t>(tok_rows + static_cast<long long>(head.t) * p.H + c0);
            bytes = row_window<TT, AL>(a, nc * sizeof(TT), tb, tb + static_cast<size_t>(p.T) * p.H * sizeof(TT), dst, lo);
            meta[warp][s][KM].m = static_cast<int32_t>((a & 15) / sizeof(TT));
        } else if (r >= 0) {
            if constexpr (kLoadRows) {
                const uintptr_t tb = reinterpret_cast<uintptr_t>(exp_rows);
                a = reinterpret_cast<uintptr_t>(exp_rows + static_cast<long long>(r) * p.H + c0);
                bytes = row_window<TI, AL>(a, nc * sizeof(TI), tb, tb + static_cast<size_t>(rows) * p.H * sizeof(TI), dst, lo);
            }
            meta[warp][s][pos] = XMeta{r, static_cast<int32_t>((a & 15) / sizeof(TI)), nwt, lane};
        }
        const uint32_t tx = __reduce_add_sync(0xFFFFFFFFu, bytes);
        if (lane == 0) {
            live[warp][s] = __popc(mask);
            mbar_arrive_expect_tx(&full[warp][s], tx);
        }
        __syncwarp();
        if (bytes)
            bulk_load(dst + (AL ? 0 : lo - (a & ~static_cast<uintptr_t>(15))), reinterpret_cast<const void*>(lo), bytes,
                      &full[warp][s]);
        advance(head);
        fetch(head);
    };

    float dot[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) dot[j] = 0.0f;
    fetch(head);
    for (int s = 0; s < kXrStages; ++s)
        if (head.t < p.T) issue(s);
    int s = 0, nth = 0, under_way = kXrStages;
    uint32_t phase = 0;
    bool drain = false;
    while (tail.t < p.T) {
        if (!warp_wait(&full[warp][s], phase)) {
            st |= MILO_DEV_TIMEOUT;
            drain = true;
        }
        if (drain) {
            // the copies under way land before the block leaves
            if (head.t < p.T) head.t = p.T;
            advance(tail);
            if (tail.t >= p.T || --under_way <= 0) break;
            if (++s == kXrStages) { s = 0; phase ^= 1; }
            continue;
        }
        const int t = tail.t, c0 = tail.ch * P.cols, nc = tail.ch == P.nch - 1 ? p.H - c0 : P.cols;
        const uint8_t* stage = ring + s * P.nrows * P.pitch;
        const XMeta* mt = meta[warp][s];
        const int cnt = live[warp][s];
        auto block = [&](auto full, int v0) {
            constexpr bool FULL = decltype(full)::value;
            float a[8], acc[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) a[q] = acc[q] = 0.0f;
            if (has_tok) read_cols<TT, AL, FULL>(stage + tok_at * P.pitch, mt[KM].m, v0, lane, nc, a);
            // slots j..j + N - 1 of the live ones
            auto slots = [&](auto count, int j, float* d) {
                constexpr int N = decltype(count)::value;
                XMeta x[N];
                float b[N][8];
#pragma unroll
                for (int u = 0; u < N; ++u) {
                    x[u] = mt[j + u];
#pragma unroll
                    for (int q = 0; q < 8; ++q) b[u][q] = 0.0f;
                    if constexpr (kLoadRows) read_cols<TI, AL, FULL>(stage + (j + u) * P.pitch, x[u].m, v0, lane, nc, b[u]);
                }
#pragma unroll
                for (int u = 0; u < N; ++u) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        if constexpr (kDot) d[u] = fmaf(a[q], b[u][q], d[u]);
                        if constexpr (kToRows) b[u][q] = x[u].w * a[q];
                        else acc[q] = fmaf(x[u].w, b[u][q], acc[q]);
                    }
                    if constexpr (kToRows)
                        write_cols<TO, AL, FULL>(static_cast<TO*>(p.out) + static_cast<long long>(x[u].row) * p.H + c0, v0, lane, nc,
                                           b[u], st);
                }
            };
            if constexpr (FULL || !kDot) {
#pragma unroll
                for (int g4 = 0; g4 < KM; g4 += KB) {
                    if (g4 + KB <= cnt) {
                        slots(std::integral_constant<int, KB>{}, g4, dot + g4);
                    } else {
#pragma unroll
                        for (int u = 0; u < KB - 1; ++u)
                            if (g4 + u < cnt) slots(std::integral_constant<int, 1>{}, g4 + u, dot + g4 + u);
                    }
                }
            } else {
                // a row's rest: one body for all slots
#pragma unroll 1
                for (int j = 0; j < cnt; ++j) {
                    float d1[1] = {0.0f};
                    slots(std::integral_constant<int, 1>{}, j, d1);
#pragma unroll
                    for (int u = 0; u < KM; ++u) dot[u] += u == j ? d1[0] : 0.0f;
                }
            }
            if constexpr (!kToRows) {
                if constexpr (MODE == kXCombine) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) acc[q] += a[q];
                }
                write_cols<TO, AL, FULL>(static_cast<TO*>(p.out) + static_cast<long long>(t) * p.H + c0, v0, lane, nc, acc, st);
            }
        };
        // whole blocks without a test per column, where that is worth a second copy
        // of the code (combine's gradient at width 2051 55 us against 59; but
        // misaligned dispatch 53 us with one copy and 65 with two, combine's
        // gradient at aligned rows 47 and 51)
        int v0 = 0;
        if constexpr (MODE != kXDispatch && !(AL && MODE == kXCombineGrad))
            for (; v0 + 256 <= nc; v0 += 256) block(std::true_type{}, v0);
        for (; v0 < nc; v0 += 256) block(std::false_type{}, v0);
        if constexpr (kDot) {
            if (tail.ch + team >= P.nch) {
                // this warp's last piece of the token: the sums over its lanes, to
                // lane j for live slot j
                float mine = 0.0f;
#pragma unroll
                for (int j = 0; j < KM; ++j) {
                    if (j < cnt) {
                        float d = dot[j];
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
                        if (lane == j) mine = d;
                    }
                    dot[j] = 0.0f;
                }
                bool ok = true;
                if (g > 0) {
                    // a member: its sums to the leader, once the token two before has been read
                    ok = warp_wait(&taken[lead][nth & 1], ((nth >> 1) & 1) ^ 1);
                    if (ok) {
                        if (lane < KM) part[warp][nth & 1][lane] = mine;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&filled[lead][nth & 1]);
                    }
                } else {
                    if (team > 1) {
                        ok = warp_wait(&filled[lead][nth & 1], (nth >> 1) & 1);
                        for (int q = 1; q < team; ++q)
                            if (lane < KM) mine += part[lead + q][nth & 1][lane];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&taken[lead][nth & 1]);
                    }
                    if (lane < p.k) p.dw[t * p.k + lane] = 0.0f;        // a dropped slot keeps this
                    __syncwarp();
                    if (lane < cnt) p.dw[t * p.k + mt[lane].slot] = mine;
                }
                if (!ok) {
                    st |= MILO_DEV_TIMEOUT;
                    drain = true;
                }
                ++nth;
            }
        }
        __syncwarp();
        advance(tail);
        if (head.t < p.T) issue(s);
        if (++s == kXrStages) { s = 0; phase ^= 1; }
    }
    flag(p.dev_status, st);
}

template <typename TI, typename TO, bool AL, int KM, int MODE>
inline cudaError_t launch_rows(const XRowsParams& P, size_t smem, cudaStream_t s) {
    static std::atomic<bool> configured[64];     // set once per device (a repeat is harmless)
    auto kernel = exchange_rows_kernel<TI, TO, AL, KM, MODE>;
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kXrSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
    }
    const bool dot = MODE == kXCombineGrad || MODE == kXDispatchGrad;
    const long long items = static_cast<long long>(P.x.T) * (dot ? 1 : P.nch);
    const long long grid = std::min<long long>(sms, items);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kXrThreads), smem, s, P);
}

template <typename TI, typename TO, int MODE>
inline cudaError_t run_rows(const ExchangeParams& p, bool al, cudaStream_t s) {
    constexpr int es = MODE == kXCombine && sizeof(TO) > sizeof(TI) ? sizeof(TO) : sizeof(TI);   // widest staged type
    XRowsParams P;
    P.x = p;
    P.nrows = MODE == kXDispatch ? 1 : p.k + (MODE != kXCombine || p.other ? 1 : 0);
    const int slack = al ? 0 : kXrSlack;
    const int max_cols = ((kXrSmem / (kXrWarps * kXrStages * P.nrows) - slack) / es) / 64 * 64;
    // Piece length (b blocks of 256 columns, as the ring allows) and team: the
    // work is dealt out in whole items, so what counts is how evenly they fill
    // the warps' rounds, against a fixed cost per item (0.15 us of a warp) and,
    // with teams, per token; a block of 256 columns costs 0.14 us per row moved
    // (12 warps sharing an SM's part of the bandwidth).
    const bool dot = MODE == kXCombineGrad || MODE == kXDispatchGrad;
    const double rows_moved = (MODE == kXDispatch ? 1 : p.k + 1) + (MODE == kXCombineGrad || MODE == kXDispatch ? p.k : 1);
    const long long nw = 148LL * kXrWarps;
    double best = -1.0;
    // a rest of up to 64 columns goes with the last piece where the ring has room
    const int rest = max_cols >= 320 ? 64 : 0;
    for (int b = std::max(1, (max_cols - rest) / 256); b >= 1; --b) {
        const int cols = std::min(max_cols - rest, 256 * b);
        const int nch = std::max(1, (p.H - rest + cols - 1) / cols);
        for (int team : kXrTeams) {
            if (team > 1 && (!dot || team > nch)) break;
            const long long warps = nw / team;
            const long long items = dot ? (p.T + warps - 1) / warps * ((nch + team - 1) / team)
                                        : (static_cast<long long>(p.T) * nch + nw - 1) / nw;
            double cost = items * (0.15 + 0.14 * rows_moved * std::min(static_cast<double>(b), p.H / 256.0));
            if (team > 1) cost += 0.2 * ((p.T + warps - 1) / warps);
            if (best < 0.0 || cost < best * 0.999) {
                best = cost;
                P.cols = cols;
                P.nch = nch;
                P.team = team;
            }
        }
    }
    P.pitch = std::min(P.cols + rest, (p.H + 63) / 64 * 64) * es + slack;
    const size_t smem = static_cast<size_t>(kXrWarps) * kXrStages * P.nrows * P.pitch;
    if (MODE != kXDispatch && al) {
        if (p.k <= 2) return launch_rows<TI, TO, MODE != kXDispatch, 2, MODE>(P, smem, s);
        if (p.k <= 8) return launch_rows<TI, TO, MODE != kXDispatch, 8, MODE>(P, smem, s);
        return launch_rows<TI, TO, MODE != kXDispatch, 16, MODE>(P, smem, s);
    }
    if (p.k <= 2) return launch_rows<TI, TO, false, 2, MODE>(P, smem, s);
    if (p.k <= 8) return launch_rows<TI, TO, false, 8, MODE>(P, smem, s);
    return launch_rows<TI, TO, false, 16, MODE>(P, smem, s);
}

template <int MODE>
inline cudaError_t run_rows_types(const ExchangeParams& p, const ExchangeTypes& t, cudaStream_t s) {
    auto by_out = [&](auto in) {
        using TI = decltype(in);
        if (t.out == MILO_F32) return run_rows<TI, float, MODE>(p, t.aligned, s);
        if (t.out == MILO_F16) return run_rows<TI, __half, MODE>(p, t.aligned, s);
        return run_rows<TI, __nv_bfloat16, MODE>(p, t.aligned, s);
    };
    if (t.in == MILO_F32) return by_out(float{});
    if (t.in == MILO_F16) return by_out(__half{});
    return by_out(__nv_bfloat16{});
}

}  // namespace milo
