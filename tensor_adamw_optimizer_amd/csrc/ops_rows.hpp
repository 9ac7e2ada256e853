// ops_rows.hpp -- the product of a few rows with a large matrix, under the
// feed-forward block and the loss where only a few tokens are answered or scored.
//
//     C(m, n) = sum_k A(m, k) B(n, k),   m < 16 MF <= 64
//
// B's bytes are the time, so every wave reads fragments of B straight from memory
// to registers, 16 rows by 64 bytes a load, with the next chunk's loads under way
// while a chunk is multiplied; A comes from the caches.  A workgroup takes 16 NF
// columns; its eight waves take chunks of k in turn and add up their sums through
// LDS, so that a product with few columns still has enough loads under way.  What
// happens to the result is the same as under ops_gemm.hpp.
//
// Measured on an MI355X, bf16: one row, 28672 x 4096 42 us (5.6 TB/s), 4096 x 14336
// 22 us (5.3 TB/s); 16 rows, 32000 x 2048 26 us (5.0 TB/s, with the matrix's 131 MB
// in the 256 MB Infinity Cache from the call before; eight such matrices in turn take
// 3 us more a call).  With branches around the loads the compiler waits for all of
// them at once: 51, 30 and 31 us.
//
// Rows need no padding: a 16-byte load is made at any element's alignment, and
// the end of a row that is no whole step is read value by value.
#pragma once

#include "ops_gemm.hpp"

namespace apexw {
namespace {

constexpr int kRowsMax = 64;

struct RowsArgs {
    const char *a;
    const char *b0, *b1;     // b1: the other matrix of a pair (kEpiGate)
    int64_t lda, ldb;        // bytes
    int32_t M, N, K;         // N: columns of one matrix of a pair
    EpiArgs e;
    const int64_t *target;   // kEpiLse: each row's class as the caller gave it
    int64_t ignore, vocab;
};

// A row's class; -1: carries no loss, -2: outside the vocabulary.
__device__ __forceinline__ int class_of(int64_t target, int64_t ignore, int64_t vocab) {
    return target == ignore ? -1 : target >= 0 && target < vocab ? (int)target : -2;
}

template <class T>
__device__ __forceinline__ Frag piece_at(const char *p) {
    Frag f;
    __builtin_memcpy(&f.v, p, 16);
    return f;
}
// The first n values of a piece, zeros behind them.
template <class T>
__device__ __forceinline__ Frag piece_of(const char *p, int n) {
    constexpr int V = 16 / sizeof(T);
    union { T t[V]; i32x4 v; } u;
#pragma unroll
    for (int j = 0; j < V; ++j) u.t[j] = j < n ? reinterpret_cast<const T *>(p)[j] : (T)0.0f;
    return Frag{u.v};
}

template <class T, int MF, int NF, int U, int W, int EPI>
__global__ __launch_bounds__(W * 64) void rows_product_kernel(const RowsArgs g) {
    constexpr int V = 16 / sizeof(T), STEP = 4 * V;           // values of k: a piece, a step
    constexpr bool PAIR = EPI == kEpiGate;
    constexpr int CHUNK = 64 * U;                              // bytes of k
    static_assert(!PAIR || NF % 2 == 0, "gate and up take turns");
    __shared__ __attribute__((aligned(16))) f32x4 lds[W][MF * NF][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = lane & 15, kg = lane >> 4;
    const int n0 = blockIdx.x * NF * (PAIR ? 8 : 16);          // first column

    // rows past the end repeat the last one: their results are not used
    const char *pa[MF], *pb[NF];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
        const int m = i * 16 + t;
        pa[i] = g.a + (int64_t)(m < g.M ? m : g.M - 1) * g.lda + kg * 16;
    }
#pragma unroll
    for (int j = 0; j < NF; ++j) {
        const int n = n0 + (PAIR ? j / 2 : j) * 16 + t;
        pb[j] = (PAIR && j % 2 ? g.b1 : g.b0) + (int64_t)(n < g.N ? n : g.N - 1) * g.ldb + kg * 16;
    }

    f32x4 acc[MF][NF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    // Whole chunks first, without a branch around a load in the loop: where paths
    // with and without one meet, the compiler waits for all of them.
    const int steps = g.K / STEP, whole = steps / U;
    const int mine = (whole - wave + W - 1) / W;
    Frag fa[2][U][MF], fb[2][U][NF];
    auto load = [&](int i, auto buf) {
        constexpr int B = decltype(buf)::value;
        const int64_t at = (int64_t)(wave + i * W) * CHUNK;
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < NF; ++j) fb[B][u][j] = piece_at<T>(pb[j] + at + u * 64);
#pragma unroll
            for (int i = 0; i < MF; ++i) fa[B][u][i] = piece_at<T>(pa[i] + at + u * 64);
        }
        __builtin_amdgcn_sched_barrier(0);     // (not to be put off until they are used)
    };
    auto multiply = [&](auto buf) {
        constexpr int B = decltype(buf)::value;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int j = 0; j < NF; ++j)
                    mma(fb[B][u][j], fa[B][u][i], acc[i][j], (T *)nullptr);
    };
    if (mine > 0) {
        load(0, Int<0>());
        int i = 0;
        for (; i + 2 < mine; i += 2) {
            load(i + 1, Int<1>());
            multiply(Int<0>());
            load(i + 2, Int<0>());
            multiply(Int<1>());
        }
        if (i + 1 < mine) {
            load(i + 1, Int<1>());
            multiply(Int<0>());
            multiply(Int<1>());
        } else {
            multiply(Int<0>());
        }
    }
    // the steps of the last chunk, which is not a whole one, by the waves in turn
    for (int step = whole * U; step < steps; ++step) {
        if (step % W != wave) continue;
        Frag a[MF], b[NF];
#pragma unroll
        for (int j = 0; j < NF; ++j) b[j] = piece_at<T>(pb[j] + (int64_t)step * 64);
#pragma unroll
        for (int i = 0; i < MF; ++i) a[i] = piece_at<T>(pa[i] + (int64_t)step * 64);
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j) mma(b[j], a[i], acc[i][j], (T *)nullptr);
    }
    if (g.K % STEP != 0 && wave == W - 1) {
        const int left = g.K % STEP - kg * V;                  // values of this lane's piece
        const int64_t at = (int64_t)steps * 64;
        Frag a[MF], b[NF];
#pragma unroll
        for (int j = 0; j < NF; ++j) b[j] = piece_of<T>(pb[j] + at, left);
#pragma unroll
        for (int i = 0; i < MF; ++i) a[i] = piece_of<T>(pa[i] + at, left);
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j) mma(b[j], a[i], acc[i][j], (T *)nullptr);
    }

#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) lds[wave][i * NF + j][lane] = acc[i][j];
    __syncthreads();
    auto total = [&](int f) {
        f32x4 s = lds[0][f][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) s += lds[w][f][lane];
        return s;
    };
    if constexpr (EPI == kEpiLse) {
        // the block's logits, rows of 16 NF, then a lane a row
        constexpr int WC = 16 * NF, C = WC / 4, OWN = (MF * NF + W - 1) / W;
        f32x4 z[OWN];
#pragma unroll
        for (int o = 0; o < OWN; ++o)
            if (o * W + wave < MF * NF) z[o] = total(o * W + wave);
        __syncthreads();
        char *rows = reinterpret_cast<char *>(lds);
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            const int f = o * W + wave, r = f / NF * 16 + t, at = f % NF * 4 + kg;
            if (f < MF * NF)
                *reinterpret_cast<f32x4 *>(rows + r * (WC * 4) + ((at ^ r % C) * 16)) = z[o];
        }
        __syncthreads();
        const int m = threadIdx.x;
        if (m < MF * 16 && m < g.M)
            reduce_row<WC>(rows, g.e, m, m, n0, g.N, class_of(g.target[m], g.ignore, g.vocab));
    } else {
        for (int f = wave; f < MF * NF / (PAIR ? 2 : 1); f += W) {
            const int i = f / (PAIR ? NF / 2 : NF), j = f % (PAIR ? NF / 2 : NF);
            const int m = i * 16 + t, n = n0 + j * 16 + kg * 4;
            f32x4 v = total(PAIR ? i * NF + 2 * j : f);
            f32x4 up = PAIR ? total(i * NF + 2 * j + 1) : v;
            if (PAIR && n + 4 > g.N) {                         // padding is zeros
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (n + q >= g.N) v[q] = up[q] = 0.0f;
            }
            if (m < g.M && n < g.e.n_store)
                finish<T, EPI, true>(v, up, Beside<EPI>(), g.e, m, n, g.N, 0);
        }
    }
}

// Groups of 16 columns of a workgroup, and its waves.  Measured, 32000 columns of
// 2048, 16 rows, bf16: two groups and eight waves 26 us (5.0 TB/s), four waves 29,
// one group and eight waves 37.  Four waves are enough from 1024 workgroups on.
struct RowsTiling {
    int nf, waves;
};
inline RowsTiling rows_tiling(int64_t n, int least) {
    const int64_t frags = div_up(n, 16);
    RowsTiling t{least, 8};
    if (frags / 2 >= 256) t.nf = 2;
    if (frags / t.nf >= 1024) t.waves = 4;
    return t;
}

template <class T, int EPI, int MF, int W>
int launch_rows(const RowsArgs &g, int nf, hipStream_t stream) {
    const int blocks = (int)div_up(g.N, nf * (EPI == kEpiGate ? 8 : 16));
    constexpr int U = MF == 1 ? 4 : 2;                         // (what the registers hold)
    if (nf == 2)
        rows_product_kernel<T, MF, 2, U, W, EPI><<<blocks, W * 64, 0, stream>>>(g);
    else if constexpr (EPI != kEpiGate)
        rows_product_kernel<T, MF, 1, U, W, EPI><<<blocks, W * 64, 0, stream>>>(g);
    APEXW_TRY_HIP(hipGetLastError());
    return APEXW_OK;
}

template <class T, int EPI>
int run_rows(const RowsArgs &g, const RowsTiling &t, hipStream_t stream) {
    if (g.M < 1) return APEXW_OK;
    const bool few = t.waves == 4;
    if (g.M <= 16)
        return few ? launch_rows<T, EPI, 1, 4>(g, t.nf, stream) : launch_rows<T, EPI, 1, 8>(g, t.nf, stream);
    if (g.M <= 32)
        return few ? launch_rows<T, EPI, 2, 4>(g, t.nf, stream) : launch_rows<T, EPI, 2, 8>(g, t.nf, stream);
    return few ? launch_rows<T, EPI, 4, 4>(g, t.nf, stream) : launch_rows<T, EPI, 4, 8>(g, t.nf, stream);
}

}  // namespace
}  // namespace apexw
