// ops_gemm.hpp -- the tiled matrix product under the gated feed-forward block
// and the linear cross entropy.
//
//     C(m, n) = sum_k A(m, k) B(n, k)
//
// Each operand lies in memory either k-contiguous (row major over k, "KC") or
// k-strided ("KS": k is the row, m or n runs along it), so that x W^T, dy W
// and dy^T x are read as they are, without a transposed copy.
//
// One workgroup computes a BM x BN tile in fp32 accumulators.  Both operands
// pass through LDS in slices of 128 or 256 bytes of k, a ring of two or four of
// them, brought in by direct loads (16 bytes a lane, no registers) through buffer
// descriptors whose bounds make every element past the matrix read as zero, so
// ragged sizes need no other care.  The matrix instructions are 16x16x32 (bf16)
// and 16x16x4 (fp32), fp32 accumulation in both.  What happens to the tile
// afterwards is the epilogue, a template argument.
//
// Measured on an MI355X, bf16, 8192 x 8192 x 8192: 770 us (1430 TFLOP/s), 755 to
// 790 with an operand or both k-strided; the same loop without its loads runs at
// 1650.  No LDS bank conflicts; the matrix pipe is busy 63-75% of the cycles, at
// a clock that the power of this work holds at 1.4 to 1.9 GHz (of 2.4).  Eight
// waves of 128 x 64 against four of 128 x 128: 790 and 860 us; instructions of
// 32x32x16 instead: 890 (two-way bank conflicts on the same tiles).
#pragma once

#include <hip/hip_bf16.h>

#include <utility>

#include "ops_common.hpp"

namespace apexw {
namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(2))) int i32x2;
typedef __attribute__((ext_vector_type(4))) short i16x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
typedef __attribute__((ext_vector_type(4))) float f32x4;

#define APEXW_LDS __attribute__((address_space(3)))

// f(Int<0>()), ..., f(Int<N - 1>()): a loop whose index is a constant.
template <int I> struct Int { static constexpr int value = I; };
template <class F, int... I>
__device__ __forceinline__ void unroll_of(F &&f, std::integer_sequence<int, I...>) {
    (f(Int<I>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void unroll(F &&f) {
    unroll_of(f, std::make_integer_sequence<int, N>());
}

// One matrix operand: `rows` along m (or n), `ldb` bytes from one row (KC) or
// one k (KS) to the next.  p1 is the second matrix of a pair: interleaved with
// p0 in groups of 16 rows (gate and up projections), or the second half of a
// sum over k (dx = dg Wg + du Wu).
struct MatArg {
    const char *p0;
    const char *p1;
    int64_t ldb;
};

enum { kEpiStore, kEpiSlab, kEpiGate, kEpiGateBwd, kEpiLse, kEpiProb };

struct EpiArgs {
    void *out0;            // C; h; dg; p
    void *out1;            // du
    float *f0;             // slab; kept gate pre-activations; LSE partials (pairs)
    float *f1;             // kept up pre-activations; target logits
    const float *row;      // per-row lse (kEpiProb)
    const float *row_scale;// per-row factor (kEpiProb)
    const float *scale;    // one device factor for the whole product, or NULL
    const int32_t *target; // per-row class, -1 for none
    int64_t ld;            // leading dimension of out0/out1 (elements); slab: of f0
    int64_t slab;          // elements of one split's slab
    int32_t n_store;       // columns to write (>= N where padding is zeroed)
    int32_t col0;          // global class of column 0
    int32_t act;
    int32_t accumulate;
    int32_t keep;
};

// Further products of the same launch, of the same k: operands, place and shape.
struct MoreArgs {
    MatArg a, b;
    void *out;
    int64_t ld;
    int32_t M, N;
};

struct GemmArgs {
    MatArg a, b;
    int32_t M, N, K;
    int32_t products;      // blockIdx.z counts them
    MoreArgs more[2];
    int32_t nk;            // slices of one matrix pair
    int32_t nkt;           // slices of the whole sum (2 nk where K is a pair)
    int32_t per_split;     // slices per split of k
    const int32_t *m_dev;  // if not NULL: the number of rows m in fact
    const int32_t *k_dev;  // if not NULL: the length of k in fact
    EpiArgs e;
};


// A fragment: 16 rows of an operand by four groups of lanes with 16 bytes of k
// each: lane l holds row l % 16 and group l / 16.  The result of 16 columns (the
// first operand) by 16 rows: lane l holds row l % 16 and columns 4 (l / 16) .. + 3.
struct Frag { i32x4 v; };

__device__ __forceinline__ void mma(const Frag &n, const Frag &m, f32x4 &c, __bf16 *) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, n.v),
                                                __builtin_bit_cast(bf16x8, m.v), c, 0, 0, 0);
}
__device__ __forceinline__ void mma_part(const Frag &n, const Frag &m, f32x4 &c, int part) {
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(f32x4, n.v)[part],
                                             __builtin_bit_cast(f32x4, m.v)[part], c, 0, 0, 0);
}
__device__ __forceinline__ void mma(const Frag &n, const Frag &m, f32x4 &c, float *) {
#pragma unroll
    for (int j = 0; j < 4; ++j) mma_part(n, m, c, j);
}

// The same with the accumulator held in place: with this many accumulators the
// register allocator has no room to rename one, and moves them about instead.
// No other instruction may touch the accumulators right before or after (see
// settle), and a kernel that uses this form has many of them in turn.
__device__ __forceinline__ void mma_in_place(const Frag &n, const Frag &m, f32x4 &c) {
    asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(n.v), "v"(m.v));
}

// Stands between mma_in_place and other uses of the accumulators, either way: all
// that writes them comes before the wait, all that reads them after it.
template <int M, int N>
__device__ __forceinline__ void settle(f32x4 (&acc)[M][N]) {
    auto hold = [&] {
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) asm volatile("" : "+a"(acc[i][j]));
    };
    hold();
    asm volatile("s_nop 15" ::);
    hold();
}

// ---- the operand's way through LDS
//
// KC tile: ROWS rows of P 16-byte pieces (8 or 16); piece c of row r lies at
// position c ^ (r % P), so the 16 lanes that read 16 rows at one c spread over
// all banks.  KS tile: one row per k, ROWS values long; the piece that holds 16
// consecutive rows (a granule, 32 or 64 bytes) is displaced by a function of k,
// so the k's that one read takes spread over the banks.
template <class T, bool KS, int ROWS, int P, int NT>
struct Tile {
    static constexpr int EB = sizeof(T), BK = P * 16 / EB;
    static constexpr int BYTES = ROWS * P * 16;
    static constexpr int LOADS = BYTES / 16 / NT;      // direct loads per thread and slice
    static constexpr int CPR = ROWS * EB / 16;         // KS: 16-byte pieces per k
    static_assert(BYTES / 16 % NT == 0, "a slice is a whole number of loads");
    static_assert(!KS || ROWS == 64 || ROWS % 128 == 0, "as many granules as displacements");

    static __device__ __forceinline__ int shift(int k) {
        if (EB == 4) return (k >> 2) & 3;
        return ROWS == 64 ? (k ^ k >> 3) & 3 : (k & 3) | ((k >> 3) & 1) << 2;
    }

    // Byte offset, from the tile's origin in memory, of the piece that load i
    // of this thread brings in.  pair: rows alternate between two matrices in
    // groups of so many.
    static __device__ __forceinline__ uint32_t offset(int i, int tid, int64_t ldb, int pair) {
        const int q = i * NT + tid;
        if constexpr (KS) {
            const int k = q / CPR, pos = q % CPR;
            constexpr int G = EB == 2 ? 2 : 4;         // pieces per granule
            const int c = ((pos / G) ^ shift(k)) * G + pos % G;
            return (uint32_t)(k * ldb + c * 16);
        } else {
            int r = q / P;
            const int c = q % P ^ r % P;
            if (pair) r = r / (2 * pair) * pair + r % pair;
            return (uint32_t)(r * ldb + c * 16);
        }
    }
};

// The fragment of rows row .. row + 15 and k step `s`.
template <class T, bool KS, int ROWS, int P>
__device__ __forceinline__ Frag load_frag(const char *tile, int row, int s, int lane) {
    Frag f;
    const int t = lane & 15, kg = lane >> 4;
    if constexpr (!KS) {
        f.v = *reinterpret_cast<const i32x4 *>(tile + (row + t) * (P * 16) +
                                               (((s * 4 + kg) ^ t % P) * 16));
    } else if constexpr (sizeof(T) == 2) {
        // the transposing read: 16 lanes take a 4 x 16 block, four values of k each
        const int k = s * 32 + kg * 8 + (t >> 2);
        const int g = (row >> 4) ^ (ROWS == 64 ? (t >> 2) ^ kg : (t >> 2) | (kg & 1) << 2);
        const char *p = tile + k * (ROWS * 2) + g * 32 + (t & 3) * 8;
        union { i16x4 h[2]; i32x4 v; } u;
        u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((APEXW_LDS i16x4 *)p);
        u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((APEXW_LDS i16x4 *)(p + 4 * ROWS * 2));
        f.v = u.v;
    } else {
        const int g = (row >> 4) ^ kg;
        const char *p = tile + (s * 16 + kg * 4) * (ROWS * 4) + g * 64 + t * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) f.v[j] = *reinterpret_cast<const int *>(p + j * (ROWS * 4));
    }
    return f;
}

// Direct load of 16 bytes per lane to LDS at lds + AT + 16 * lane.  It has no
// output register and is waited for by count, by hand: the compiler does not
// track it.  No memory clobber: reads of LDS may move over it, since between two
// barriers nobody reads the buffer that it fills; `arrive` is what orders them.
template <int AT>
__device__ __forceinline__ void lds_load(uint32_t lds, uint32_t off, i32x4 rsrc) {
    asm volatile("s_add_i32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(off), "s"(rsrc), "n"(AT) : "m0", "scc");
}

// All but the last N direct loads have landed and all reads of LDS are done,
// for every wave of the workgroup.
template <int N>
__device__ __forceinline__ void arrive() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Bytes of n values of EB bytes in whole 16-byte pieces.
template <int EB>
__device__ __forceinline__ int64_t pieces(int n) { return (int64_t)(n + 16 / EB - 1) / (16 / EB) * 16; }

// The same in every lane: kept in scalar registers.
__device__ __forceinline__ const char *uniform(const char *p) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint64_t)p);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)((uint64_t)p >> 32));
    return reinterpret_cast<const char *>((uint64_t)hi << 32 | lo);
}

constexpr uint32_t kOutside = 0x80000000u;   // an offset past every descriptor

// An operand's way through memory, a slice of k after the other: the buffer
// descriptor of the tile's part of the slice, whose bound moves along with its
// base, and each load's offset from the base.  This runs in every slice on the
// scalar unit, in line with everything else: it is kept to a few instructions.
template <class T, bool KS, int ROWS, int P, int NT>
struct Slice {
    using TL = Tile<T, KS, ROWS, P, NT>;
    uint64_t base, left, step;     // address; bytes from there to the bound; bytes a slice
    uint32_t off[TL::LOADS];

    // rows_left >= 1, k < K
    __device__ __forceinline__ void start(const char *p, int64_t ldb, int64_t row0, int rows_left,
                                          int k, int K, int tid, int pair) {
        if constexpr (KS) {
            // (a bound inside a dword would drop the dword: rows count in whole
            // 16-byte pieces, which the leading dimension has room for)
            step = TL::BK * ldb;
            base = (uint64_t)p + k * ldb + row0 * TL::EB;
            left = (int64_t)(K - k - 1) * ldb + pieces<TL::EB>(rows_left);
        } else {
            step = TL::BK * TL::EB;
            base = (uint64_t)p + row0 * ldb + (int64_t)k * TL::EB;
            left = (int64_t)(rows_left - 1) * ldb + pieces<TL::EB>(K - k);
        }
#pragma unroll
        for (int i = 0; i < TL::LOADS; ++i) off[i] = TL::offset(i, tid, ldb, pair);
    }
    __device__ __forceinline__ void next() {
        base += step;
        left -= step;
    }
    // In the last slice of a k-contiguous operand, `in` values long: pieces past
    // the end of a row would read the next row.
    __device__ __forceinline__ void ragged(int in, int tid) {
        if constexpr (!KS) {
            const uint32_t out = (tid % P ^ tid / P % P) * (16 / TL::EB) >= in ? kOutside : 0;
#pragma unroll
            for (int i = 0; i < TL::LOADS; ++i) off[i] |= out;
        }
    }
    // (the last bytes are all that a bound is for: nothing beyond is asked for
    // before there)
    __device__ __forceinline__ i32x4 rsrc(bool alive) const {
        const uint32_t lo = (uint32_t)left, hi = (uint32_t)(left >> 32);
        const uint32_t n = hi != 0 || lo > 0x7fffffffu ? 0x7fffffffu : lo;
        return i32x4{__builtin_amdgcn_readfirstlane((int)base),
                     __builtin_amdgcn_readfirstlane((int)(base >> 32)),
                     __builtin_amdgcn_readfirstlane(alive ? (int)n : 0), 0x00020000};
    }
};

// ---- epilogues

__device__ __forceinline__ float fast_exp(float x) {
    return __builtin_amdgcn_exp2f(x * 1.4426950408889634f);
}

// The activation and its derivative, in fp32.
__device__ __forceinline__ float act_fwd(float g, int act) {
    if (act == APEXW_ACT_SILU) return g / (1.0f + __expf(-g));
    const float z = 0.7978845608028654f * (g + 0.044715f * g * g * g);
    // 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z))
    return g / (1.0f + __expf(-2.0f * z));
}
__device__ __forceinline__ void act_both(float g, int act, float &f, float &d) {
    if (act == APEXW_ACT_SILU) {
        const float s = 1.0f / (1.0f + __expf(-g));
        f = g * s;
        d = s * (1.0f + g * (1.0f - s));
    } else {
        const float c = 0.7978845608028654f;
        const float z = c * (g + 0.044715f * g * g * g);
        const float s = 1.0f / (1.0f + __expf(-2.0f * z));
        f = g * s;
        d = s + 2.0f * g * s * (1.0f - s) * c * (1.0f + 3.0f * 0.044715f * g * g);
    }
}

template <class T> struct Vec4;
template <> struct Vec4<float> { typedef f32x4 type; };
template <> struct Vec4<__bf16> { typedef bf16x4 type; };

// Four consecutive values, as one aligned vector.
template <class T>
__device__ __forceinline__ void store4(T *p, f32x4 v) {
    typename Vec4<T>::type b;
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = (T)v[j];
    *reinterpret_cast<typename Vec4<T>::type *>(p) = b;
}

// A lane's four consecutive values of row m at columns n .. n+3.  SAFE false:
// the caller knows that all four are inside and aligned.
template <class T, bool SAFE = true>
__device__ __forceinline__ void put4(T *base, int64_t ld, int m, int n, int n_store, f32x4 v) {
    T *p = base + (int64_t)m * ld + n;
    if constexpr (SAFE) {
        if (n >= n_store) return;
        if (n + 4 > n_store || ((uintptr_t)p & (4 * sizeof(T) - 1)) != 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < n_store) p[j] = (T)v[j];
            return;
        }
    }
    store4(p, v);
}

// What an epilogue reads for four values at row m and columns n .. n+3, and what
// it does with them: v of the product (kEpiGate: v and up, of the two projections'
// column n).  Reading stands apart, so that a few rows' reads are under way at
// once.  SAFE false: row and columns are known to be inside and aligned.
template <int EPI>
struct Beside {
    f32x4 a, b;
    float lse, s;
    int t;

    __device__ __forceinline__ void read(const EpiArgs &e, int m, int n, int split) {
        if constexpr (EPI == kEpiSlab) {
            if (e.accumulate)
                a = *reinterpret_cast<const f32x4 *>(e.f0 + split * e.slab + (int64_t)m * e.ld + n);
        } else if constexpr (EPI == kEpiGateBwd) {
            a = *reinterpret_cast<const f32x4 *>(e.f0 + (int64_t)m * e.ld + n);
            b = *reinterpret_cast<const f32x4 *>(e.f1 + (int64_t)m * e.ld + n);
        } else if constexpr (EPI == kEpiProb) {
            lse = e.row[m];
            s = e.row_scale[m];
            t = e.target[m] - e.col0;                  // below 0: none of these
        }
    }
};

template <class T, int EPI, bool SAFE>
__device__ __forceinline__ void finish(f32x4 v, f32x4 up, const Beside<EPI> &x, const EpiArgs &e,
                                       int m, int n, int N, int split) {
    if constexpr (EPI == kEpiStore) {
        put4<T, SAFE>((T *)e.out0, e.ld, m, n, e.n_store, v);
    } else if constexpr (EPI == kEpiSlab) {
        if (e.accumulate) v += x.a;
        *reinterpret_cast<f32x4 *>(e.f0 + split * e.slab + (int64_t)m * e.ld + n) = v;
    } else if constexpr (EPI == kEpiGate) {
        f32x4 h;
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = act_fwd(v[q], e.act) * up[q];
        put4<T, SAFE>((T *)e.out0, e.ld, m, n, e.n_store, h);
        if (e.keep) {
            *reinterpret_cast<f32x4 *>(e.f0 + (int64_t)m * e.ld + n) = v;
            *reinterpret_cast<f32x4 *>(e.f1 + (int64_t)m * e.ld + n) = up;
        }
    } else if constexpr (EPI == kEpiGateBwd) {
        f32x4 dg, du;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float f, d;
            act_both(x.a[q], e.act, f, d);
            dg[q] = v[q] * x.b[q] * d;
            du[q] = v[q] * f;
        }
        put4<T, SAFE>((T *)e.out0, e.ld, m, n, e.n_store, dg);
        put4<T, SAFE>((T *)e.out1, e.ld, m, n, e.n_store, du);
    } else {
        static_assert(EPI == kEpiProb, "an epilogue");
        f32x4 p;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            p[q] = fast_exp(v[q] - x.lse) - (n + q == x.t ? 1.0f : 0.0f);
            p[q] = !SAFE || n + q < N ? p[q] * x.s : 0.0f;
        }
        put4<T, SAFE>((T *)e.out0, e.ld, m, n, e.n_store, p);
    }
}

// kEpiLse: a lane takes a row of the wave's part, whole: its largest logit and the
// sum of exp(z - largest) over the part's columns go to f0, which has ld such pairs
// for each group of that many columns.
template <int WC>
__device__ __forceinline__ void reduce_row(const char *lds, const EpiArgs &e, int r, int m, int n0,
                                           int N, int target) {
    constexpr int C = WC / 4;
    const char *p = lds + r * (WC * 4);
    const int t = target - n0;
    if (t >= 0 && t < WC && n0 + t < N)
        e.f1[m] = reinterpret_cast<const float *>(p + ((t / 4 ^ r % C) * 16))[t % 4];
    f32x4 v[C];
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        v[c] = *reinterpret_cast<const f32x4 *>(p + ((c ^ r % C) * 16));
        if (n0 + WC > N) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (n0 + c * 4 + q >= N) v[c][q] = -INFINITY;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) top = fmaxf(top, v[c][q]);
    }
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) sum += fast_exp(v[c][q] - ref);
    reinterpret_cast<float2 *>(e.f0)[(int64_t)(n0 / WC) * e.ld + m] = make_float2(top, sum);
}

// A wave's part of the tile, 16 FM x 16 FN: acc[i][j] holds row 16 i + lane % 16
// and columns 16 j + 4 (lane / 16) .. + 3.  It passes through the wave's own piece
// of LDS, so that whole rows are stored, by a loop over a few rows at a time.
template <class T, int EPI, int ROOM, int FM, int FN>
__device__ __forceinline__ void epilogue(f32x4 (&acc)[FM][FN], char *lds, const EpiArgs &e, int m0,
                                         int n0, int M, int N, int split, int lane) {
    constexpr bool GATE = EPI == kEpiGate;
    constexpr int WC = FN * 16, C = WC / 4;            // columns; runs of four in a row
    constexpr int FIT = ROOM / (WC * 64), PASS = FIT < FM ? FIT : FM;
    static_assert(FM % PASS == 0, "whole passes");
    constexpr int L = GATE ? C / 2 : C, AT_ONCE = 64 / L;        // lanes a row; rows at once
    constexpr int ITER = PASS * 16 / AT_ONCE, U = ITER < 4 ? ITER : 4;
    static_assert(ITER % U == 0, "whole batches");
    const int c = lane % L, r0 = lane / L;
    const int c0 = GATE ? c / 4 * 8 + c % 4 : c;       // (groups of 16 columns alternate)
    const int nw = GATE ? n0 / 2 : n0, n = nw + c * 4, n1 = nw + (GATE ? WC / 2 : WC);
    const float factor = EPI == kEpiStore && e.scale != nullptr ? *e.scale : 1.0f;
    // columns that the lane may touch: those to be stored, or of the product
    const int n_end = e.n_store;
    const bool inside = m0 + FM * 16 <= M && n1 <= n_end && (EPI != kEpiProb || n1 <= N) &&
                        (((uintptr_t)e.out0 | (uintptr_t)e.out1 | (uintptr_t)(e.ld * sizeof(T))) &
                         (4 * sizeof(T) - 1)) == 0;
    unroll<FM / PASS>([&](auto pc) {
        constexpr int P0 = decltype(pc)::value * PASS;
#pragma unroll
        for (int i = 0; i < PASS; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int r = i * 16 + (lane & 15), at = j * 4 + (lane >> 4);
                *reinterpret_cast<f32x4 *>(lds + r * (WC * 4) + ((at ^ r % C) * 16)) = acc[P0 + i][j];
            }
        auto rows = [&](auto safe) {
            constexpr bool SAFE = decltype(safe)::value != 0;
#pragma unroll 1
            for (int r = r0; r < PASS * 16; r += AT_ONCE * U) {
                f32x4 v[U], up[U];
                Beside<EPI> x[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int ru = r + u * AT_ONCE, m = m0 + P0 * 16 + ru;
                    if (!SAFE || (m < M && n < n_end)) x[u].read(e, m, n, split);
                    const char *p = lds + ru * (WC * 4);
                    v[u] = *reinterpret_cast<const f32x4 *>(p + ((c0 ^ ru % C) * 16));
                    if constexpr (EPI == kEpiStore) v[u] *= factor;
                    if constexpr (GATE)
                        up[u] = *reinterpret_cast<const f32x4 *>(p + (((c0 + 4) ^ ru % C) * 16));
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int m = m0 + P0 * 16 + r + u * AT_ONCE;
                    if (!SAFE || (m < M && n < n_end))
                        finish<T, EPI, SAFE>(v[u], up[u], x[u], e, m, n, N, split);
                }
            }
        };
        if constexpr (EPI == kEpiLse) {
            static_assert(PASS * 16 <= 64, "a lane a row");
            const int m = m0 + P0 * 16 + lane;
            if (lane < PASS * 16 && m < M) reduce_row<WC>(lds, e, lane, m, n0, N, e.target[m] - e.col0);
        } else if (inside) {
            rows(Int<0>());
        } else {
            rows(Int<1>());
        }
    });
}

// Which tile a workgroup computes.  Workgroups go to the eight dies in turn,
// each with an L2 of its own: die d takes a run of consecutive places, and
// places walk down 8 tile rows before the next tile column, so the workgroups of
// one die share a few rows of A and columns of B.
__device__ __forceinline__ bool tile_of(int id, int tiles_m, int tiles_n, int &tm, int &tn) {
    const int total = tiles_m * tiles_n;
    if (id >= total) return false;       // rows counted on the device: fewer than the grid is for
    const int per = total / 8, rest = total % 8, die = id % 8, idx = id / 8;
    const int place = die * per + (die < rest ? die : rest) + idx;
    constexpr int G = 8;
    const int band = place / (G * tiles_n), first = band * G;
    const int height = tiles_m - first < G ? tiles_m - first : G;
    const int in = place - band * G * tiles_n;
    tm = first + in % height;
    tn = in / height;
    return true;
}

enum { kPairNone, kPairRows, kPairK };

// The loop over k.  A ring of NS slices in LDS is filled by direct loads, a slice
// NS ahead of the one whose place it takes.  A slice is two steps of 32 (bf16) or 16 (fp32) k; the fragments
// of one step are read from LDS between the matrix instructions of the step
// before it, so that the matrix pipe waits for neither.  The one barrier of a
// slice stands before its last step: by then its reads are done (its place in
// the ring is free for new loads) and the next slice has landed.
template <class T, bool AKS, bool BKS, int BM, int BN, int WM, int WN, int P, int Q, int NS,
          int PAIR, int EPI>
__global__ __launch_bounds__(WM *WN * 64, 1) void gemm_kernel(const GemmArgs g) {
    constexpr int NT = WM * WN * 64;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16, CW = 16;
    constexpr int STEPS = P / (4 * Q);                 // Q times four pieces of k a step
    static_assert(STEPS % 2 == 0, "the steps' fragments take turns");
    using TA = Tile<T, AKS, BM, P, NT>;
    using TB = Tile<T, BKS, BN, P, NT>;
    constexpr int BK = TA::BK, STAGE = TA::BYTES + TB::BYTES, LOADS = TA::LOADS + TB::LOADS;
    __shared__ __attribute__((aligned(1024))) char lds[NS * STAGE];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    // (which product: by comparison, so that all of it stays in scalar registers)
    MatArg oa = g.a, ob = g.b;
    EpiArgs e = g.e;
    int gm = g.M, gn = g.N;
    if constexpr (EPI == kEpiStore) {
#pragma unroll
        for (int z = 1; z < 3; ++z)
            if (blockIdx.z == z) {
                const MoreArgs &p = g.more[z - 1];
                oa = p.a;
                ob = p.b;
                gm = p.M;
                gn = p.N;
                e.out0 = p.out;
                e.ld = p.ld;
                e.n_store = p.N;
            }
    }
    const int M = g.m_dev == nullptr ? gm : __builtin_amdgcn_readfirstlane(*g.m_dev);
    const int K = g.k_dev == nullptr ? g.K : __builtin_amdgcn_readfirstlane(*g.k_dev);
    int tm, tn;
    if (!tile_of(blockIdx.x, (M + BM - 1) / BM, (gn + BN - 1) / BN, tm, tn)) return;
    const int m0 = tm * BM, n0 = tn * BN;

    const int split = blockIdx.y;
    int nkt = g.nkt;
    if (g.k_dev != nullptr) nkt = (K + BK - 1) / BK;
    const int kt0 = split * g.per_split;
    const int kt1 = kt0 + g.per_split < nkt ? kt0 + g.per_split : nkt;

    // (a wave's rows of a load are of one matrix, the same one for every load)
    static_assert(PAIR != kPairRows || (64 / P <= CW && NT / P % (2 * CW) == 0), "one matrix a wave");
    const bool second = PAIR == kPairRows && wave * (64 / P) / CW % 2;
    const int b_row0 = PAIR == kPairRows ? n0 / 2 : n0;
    const int b_rows = (PAIR == kPairRows ? gn / 2 : gn) - b_row0;

    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(size_t)(APEXW_LDS char *)lds) +
                          wave * 1024;

    // Slices past the last one are read too, as zeros: the waits count loads.
    Slice<T, AKS, BM, P, NT> sa;
    Slice<T, BKS, BN, P, NT> sb;
    // the last slice of each matrix, where it is not a whole one
    const int in = K % BK, ragged_at = in == 0 ? -1 : (K - 1) / BK;
    const char *const a0 = uniform(oa.p0), *const a1 = PAIR == kPairK ? uniform(oa.p1) : nullptr;
    const char *const b0 = uniform(ob.p0), *const b1 = PAIR != kPairNone ? uniform(ob.p1) : nullptr;
    auto start = [&](int kt) {
        const bool late = PAIR == kPairK && kt >= g.nk;
        const int k = (late ? kt - g.nk : kt) * BK;
        sa.start(PAIR == kPairK && late ? a1 : a0, oa.ldb, m0, M - m0, k, K, tid, 0);
        sb.start(PAIR != kPairNone && (late || second) ? b1 : b0, ob.ldb, b_row0, b_rows, k, K, tid,
                 PAIR == kPairRows ? CW : 0);
        if (k / BK == ragged_at) {
            sa.ragged(in, tid);
            sb.ragged(in, tid);
        }
    };
    i32x4 ra, rb;
    // on to slice kt and its descriptors, in four parts
    auto next = [&](int part, int kt) {
        if (part == 0) sa.next();
        if (part == 1) sb.next();
        if (part == 2) {
            if (PAIR == kPairK && kt == g.nk) {
                start(kt);
            } else if (kt == ragged_at || (PAIR == kPairK && in != 0 && kt == g.nk + ragged_at)) {
                sa.ragged(in, tid);
                sb.ragged(in, tid);
            }
            ra = sa.rsrc(kt < kt1);
        }
        if (part == 3) rb = sb.rsrc(kt < kt1);
    };
    auto load = [&](uint32_t at, auto l) {
        constexpr int i = decltype(l)::value;
        if constexpr (i < TA::LOADS) lds_load<i * NT * 16>(at, sa.off[i], ra);
        else lds_load<TA::BYTES + (i - TA::LOADS) * NT * 16>(at, sb.off[i - TA::LOADS], rb);
    };

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    constexpr bool IN_PLACE = sizeof(T) == 2 && FM * FN >= 32;
    auto settled = [&] {
        if constexpr (IN_PLACE) settle(acc);
    };

    Frag fa[2][Q][FM], fb[2][Q][FN];
    const char *la = lds, *lb;
    auto fetch = [&](int s, int f) {
        const int q = f / (FN + FM);
        f %= FN + FM;
        if (f < FN) fb[s & 1][q][f] = load_frag<T, BKS, BN, P>(lb, (wn * FN + f) * 16, s * Q + q, lane);
        else fa[s & 1][q][f - FN] = load_frag<T, AKS, BM, P>(la, (wm * FM + f - FN) * 16, s * Q + q, lane);
    };
    // (fp32: a fragment is four instructions' worth; those of one accumulator stand
    // apart, since each waits for the one before)
    constexpr int SUB = sizeof(T) == 4 ? 4 : 1;
    // one step's matrix instructions, with the other step's fragments read, in a
    // slice's first step the way to slice kt prepared and in its last step that
    // slice's loads issued in between, evenly
    auto step = [&](auto st, uint32_t at, int kt) {
        constexpr int s = decltype(st)::value, G = Q * SUB * FM * FN, F = Q * (FM + FN);
        constexpr bool loading = s == STEPS - 1;
        constexpr int E = G < 8 ? 1 : G / 8;
        static_assert(G >= 4, "room for the four parts of next");
        unroll<G>([&](auto xc) {
            constexpr int x = decltype(xc)::value, q = x / (SUB * FM * FN), sub = x / (FM * FN) % SUB,
                          i = x / FN % FM, j = x % FN;
            if constexpr (IN_PLACE) mma_in_place(fb[s & 1][q][j], fa[s & 1][q][i], acc[i][j]);
            else if constexpr (SUB == 4) mma_part(fb[s & 1][q][j], fa[s & 1][q][i], acc[i][j], sub);
            else mma(fb[s & 1][q][j], fa[s & 1][q][i], acc[i][j], (T *)nullptr);
            if constexpr (s == 0 && x % E == 0 && x / E < 4) next(x / E, kt);
            constexpr int f0 = x * F / G, f1 = (x + 1) * F / G;
#pragma unroll
            for (int f = f0; f < f1; ++f) fetch((s + 1) % STEPS, f);
            constexpr int l0 = loading ? x * LOADS / G : 0, l1 = loading ? (x + 1) * LOADS / G : 0;
            unroll<l1 - l0>([&](auto l) { load(at, Int<l0 + decltype(l)::value>()); });
            if constexpr (f1 > f0 || l1 > l0) __builtin_amdgcn_sched_barrier(0);
        });
    };

    start(kt0);
    unroll<NS>([&](auto i) {
        constexpr int n = decltype(i)::value;
        if (n == 0) {
            ra = sa.rsrc(kt0 < kt1);
            rb = sb.rsrc(kt0 < kt1);
        } else {
            for (int part = 0; part < 4; ++part) next(part, kt0 + n);
        }
        unroll<LOADS>([&](auto l) { load(lds0 + n * STAGE, l); });
    });
    arrive<(NS - 1) * LOADS>();
    lb = la + TA::BYTES;
#pragma unroll
    for (int f = 0; f < Q * (FM + FN); ++f) fetch(0, f);

    settled();
    int stage = 0;
    for (int kt = kt0; kt < kt1; ++kt) {
        unroll<STEPS - 1>([&](auto s) { step(s, 0, kt + NS); });
        arrive<(NS - 2) * LOADS>();
        const uint32_t at = lds0 + stage * STAGE;
        stage = stage + 1 == NS ? 0 : stage + 1;
        la = lds + stage * STAGE;
        lb = la + TA::BYTES;
        step(Int<STEPS - 1>(), at, 0);
    }
    arrive<0>();                         // LDS is the epilogue's from here on
    settled();
    constexpr int ROOM = NS * STAGE / (WM * WN);
    epilogue<T, EPI, ROOM>(acc, lds + wave * ROOM, e, m0 + wm * FM * 16, n0 + wn * FN * 16, M,
                           gn, split, lane);
}

// ---- host side

// The tile shapes.  Measured on an MI355X, bf16, us: 8192 x 8192 x 8192 770 with
// kBig, 990 with kMid; 2048 x 4096 x 4096 63 with kMid, 77 with kBig; 512 x 5632
// x 1024 11.7 with kSmall, 13.1 with kMid, 28 with kBig; 512 x 1024 x 2816, split
// in four, 8.9 with kTiny, 10.9 with kSmall.
//   kBig    256 x 256, 8 waves, one workgroup a compute unit; fp32: 128 x 128, 4 waves
//   kMid    128 x 128, 4 waves, two workgroups; fp32: 64 x 128
//   kSmall  128 x 128, 8 waves, a ring of four slices, one workgroup (bf16)
//   kTiny   64 x 64, 4 waves; bf16: a ring of four slices of twice the length
enum Kind { kBig, kMid, kSmall, kTiny };

struct Tiling {
    Kind kind;
    int bm, bn, wave_cols, splits;   // wave_cols: columns of a wave's part of the tile
};

// The shape, and the splits of the sum over k where a product may be split, that
// cost least by a model of the measurements: each round of 256 workgroups, one a
// compute unit, takes some time itself and some for each 128 bytes of k (two
// workgroups of kMid share a unit and overlap); a split product is added up by a
// second launch.
template <class T>
Tiling least_cost(int64_t m, int64_t n, int64_t k, bool pair_k, bool may_split, int products) {
    constexpr bool BF = sizeof(T) == 2;
    const Tiling shapes[4] = {BF ? Tiling{kBig, 256, 256, 64, 1} : Tiling{kBig, 128, 128, 64, 1},
                              BF ? Tiling{kMid, 128, 128, 64, 1} : Tiling{kMid, 64, 128, 64, 1},
                              Tiling{kTiny, 64, 64, 32, 1}, Tiling{kSmall, 128, 128, 32, 1}};
    const int64_t slices = div_up(k * (int64_t)sizeof(T), 128) * (pair_k ? 2 : 1);
    Tiling best = shapes[0];
    double best_cost = 1e300;
    for (const Tiling &t : shapes) {
        if (!BF && t.kind == kSmall) break;
        const int64_t tiles = div_up(m, t.bm) * div_up(n, t.bn) * products;
        for (int splits = 1; splits <= (may_split ? 64 : 1); splits = splits < 4 ? splits + 1 : splits * 5 / 4) {
            if (splits > 1 && (splits * 4 > slices || splits * tiles > 2048)) break;
            const double s = (double)div_up(slices, splits);
            const int64_t all = tiles * splits, rounds = div_up(all, 256);
            double cost;
            if (!BF)           // the matrix instructions' rate; one workgroup alone waits
                cost = 3 + s * t.bm * t.bn / 4096 * (rounds * 0.45 < 0.62 ? 0.62 : rounds * 0.45);
            else if (t.kind == kBig)
                cost = rounds * (5.5 + 1.45 * s);
            else if (t.kind == kMid)
                cost = all / 512 * (4 + 0.95 * s) + (all % 512 == 0 ? 0 : all % 512 <= 256 ? 3 + 0.5 * s : 4 + 0.95 * s);
            else if (t.kind == kSmall)
                cost = rounds * (3.5 + (rounds > 1 ? 0.6 : 0.42) * s);
            else
                cost = rounds * (1.3 + 0.24 * s);
            if (splits > 1) cost += 4 + (splits + 1.0) * m * n * 4 / 3e6;
            if (cost < best_cost) {
                best_cost = cost;
                best = t;
                best.splits = splits;
            }
        }
    }
    return best;
}

// (The same products come again with every step: the model is not worked out
// anew for the last few of them.)
template <class T>
Tiling pick_tiling(int64_t m, int64_t n, int64_t k, bool pair_k, bool may_split, int products = 1) {
    struct Known {
        int64_t m, n, k;
        int how;
        Tiling t;
    };
    static thread_local Known known[32] = {};
    const int how = 1 + pair_k + 2 * may_split + 4 * products;       // (0: an empty place)
    Known &e = known[(uint64_t)(m * 31 + n * 7 + k * 3 + how) % 32];
    if (e.how != how || e.m != m || e.n != n || e.k != k)
        e = Known{m, n, k, how, least_cost<T>(m, n, k, pair_k, may_split, products)};
    return e.t;
}

template <class T, bool AKS, bool BKS, int BM, int BN, int WM, int WN, int P, int Q, int NS,
          int PAIR, int EPI>
int launch_gemm(GemmArgs g, int splits, hipStream_t stream) {
    int64_t tiles = div_up(g.M, BM) * div_up(g.N, BN);
    for (int i = 0; i + 1 < g.products; ++i) {
        const int64_t n = div_up(g.more[i].M, BM) * div_up(g.more[i].N, BN);
        if (n > tiles) tiles = n;
    }
    g.nk = (int)div_up(g.K, P * 16 / (int64_t)sizeof(T));
    g.nkt = PAIR == kPairK ? 2 * g.nk : g.nk;
    g.per_split = (int)div_up(g.nkt, splits);
    if (tiles <= 0) return APEXW_OK;
    gemm_kernel<T, AKS, BKS, BM, BN, WM, WN, P, Q, NS, PAIR, EPI>
        <<<dim3(tiles, splits, g.products < 1 ? 1 : g.products), WM * WN * 64, 0, stream>>>(g);
    APEXW_TRY_HIP(hipGetLastError());
    return APEXW_OK;
}

template <class T, bool AKS, bool BKS, int PAIR, int EPI>
int run_gemm(const GemmArgs &g, const Tiling &t, hipStream_t stream) {
    if constexpr (sizeof(T) == 2) {
        switch (t.kind) {
            case kBig:
                return launch_gemm<T, AKS, BKS, 256, 256, 2, 4, 8, 1, 2, PAIR, EPI>(g, t.splits, stream);
            case kMid:
                return launch_gemm<T, AKS, BKS, 128, 128, 2, 2, 8, 1, 2, PAIR, EPI>(g, t.splits, stream);
            case kSmall:
                return launch_gemm<T, AKS, BKS, 128, 128, 2, 4, 8, 1, 4, PAIR, EPI>(g, t.splits, stream);
            default:
                // (a pair's rows alternate within a load of the longer slices)
                return launch_gemm<T, AKS, BKS, 64, 64, 2, 2, PAIR == kPairRows ? 8 : 16,
                                   PAIR == kPairRows ? 1 : 2, 4, PAIR, EPI>(g, t.splits, stream);
        }
    } else {
        switch (t.kind) {
            case kBig:
                return launch_gemm<T, AKS, BKS, 128, 128, 2, 2, 8, 1, 2, PAIR, EPI>(g, t.splits, stream);
            case kMid:
                return launch_gemm<T, AKS, BKS, 64, 128, 2, 2, 8, 1, 2, PAIR, EPI>(g, t.splits, stream);
            default:
                return launch_gemm<T, AKS, BKS, 64, 64, 2, 2, 8, 1, 2, PAIR, EPI>(g, t.splits, stream);
        }
    }
}

// ---- products split over k, and operands whose rows are not 16-byte pieces

// Copies a row of `cols` values, from any element's alignment, to a row of `ld` (a
// multiple of 8) with zeros past the end, by 256 threads.
template <class T>
__device__ __forceinline__ void pad_row(const T *src, T *dst, int64_t ld, int32_t cols) {
    constexpr int V = 16 / sizeof(T);
    for (int c = threadIdx.x * V; c < ld; c += 256 * V) {
        if (c + V <= cols) {
            i32x4 v;
            __builtin_memcpy(&v, src + c, 16);
            *reinterpret_cast<i32x4 *>(dst + c) = v;
        } else {
            for (int j = 0; j < V; ++j) dst[c + j] = c + j < cols ? src[c + j] : (T)0.0f;
        }
    }
}

// The way of an operand whose rows are not whole 16-byte pieces.
template <class T>
__global__ __launch_bounds__(256) void pad_rows_kernel(const T *src, int64_t src_ld, T *dst,
                                                       int64_t ld, int32_t rows, int32_t cols) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        pad_row(src + r * src_ld, dst + r * ld, ld, cols);
}

// The sum of the splits' slabs, in order, through an epilogue.  kEpiGate: the
// slabs' columns alternate between the two projections in groups of 16.
template <class T, int EPI>
__global__ __launch_bounds__(256) void sum_slabs_kernel(const float *slab, int64_t slab_elems,
                                                        int splits, int64_t ld, const EpiArgs e,
                                                        int32_t rows, int32_t cols) {
    constexpr bool GATE = EPI == kEpiGate;
    const float factor = EPI == kEpiStore && e.scale != nullptr ? *e.scale : 1.0f;
    const int64_t groups = (e.n_store + 3) / 4, total = rows * groups;
    for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int m = (int)(i / groups), n = (int)(i % groups) * 4;
        Beside<EPI> x;
        x.read(e, m, n, 0);
        const float *p = slab + m * ld + (GATE ? n / 16 * 32 + n % 16 : n);
        f32x4 v = {0, 0, 0, 0}, up = {0, 0, 0, 0};
        for (int k = 0; k < splits; ++k) {
            v += *reinterpret_cast<const f32x4 *>(p + k * slab_elems);
            if (GATE) up += *reinterpret_cast<const f32x4 *>(p + k * slab_elems + 16);
        }
        if (EPI == kEpiStore) v *= factor;
        finish<T, EPI, true>(v, up, x, e, m, n, cols, 0);
    }
}

inline int64_t pad8(int64_t n) { return (n + 7) / 8 * 8; }

// Elements of the slabs of a product that may be split.
template <class T>
int64_t slab_elems(int64_t m, int64_t n, int64_t k, bool pair_k = false) {
    const int splits = pick_tiling<T>(m, n, k, pair_k, true).splits;
    return splits == 1 ? 0 : splits * m * ((n + 31) / 32 * 32);
}

template <class T>
MatArg mat(const T *p, int64_t ld, const T *p1 = nullptr) {
    return MatArg{(const char *)p, (const char *)p1, ld * (int64_t)sizeof(T)};
}

// A product with epilogue EPI, split over k where that helps (slab: slab_elems).
template <class T, bool AKS, bool BKS, int PAIR, int EPI>
int run_split(const GemmArgs &a, float *slab, hipStream_t stream) {
    if (a.M < 1 || a.N < 1) return APEXW_OK;           // (a grid of no blocks is refused)
    const Tiling t = pick_tiling<T>(a.M, a.N, a.K, PAIR == kPairK, true);
    if (t.splits == 1) return run_gemm<T, AKS, BKS, PAIR, EPI>(a, t, stream);
    const int64_t ld = (a.N + 31) / 32 * 32, groups = (a.e.n_store + 3) / 4;
    GemmArgs p = a;
    p.e = EpiArgs{};
    p.e.f0 = slab;
    p.e.ld = ld;
    p.e.slab = a.M * ld;
    p.e.n_store = (int)ld;
    APEXW_TRY((run_gemm<T, AKS, BKS, PAIR, kEpiSlab>(p, t, stream)));
    const int64_t blocks = div_up(a.M * groups, 256);
    sum_slabs_kernel<T, EPI><<<(int)(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(
        slab, a.M * ld, t.splits, ld, a.e, a.M, a.N);
    APEXW_TRY_HIP(hipGetLastError());
    return APEXW_OK;
}

// out[M, N] = A B^T in T.
template <class T, bool AKS, bool BKS, int PAIR>
int run_product(GemmArgs a, T *out, int64_t out_ld, float *slab, hipStream_t stream) {
    a.e.out0 = out;
    a.e.ld = out_ld;
    a.e.n_store = a.N;
    return run_split<T, AKS, BKS, PAIR, kEpiStore>(a, slab, stream);
}

// Copies an operand to padded rows where dst is not NULL, and has it read there.
template <class T>
int pad_operand(const T *&src, int64_t &ld, T *dst, int64_t dst_ld, int64_t rows, int64_t cols,
                hipStream_t stream) {
    if (dst == nullptr || rows == 0) return APEXW_OK;
    pad_rows_kernel<T><<<(int)(rows < 8192 ? rows : 8192), 256, 0, stream>>>(
        src, ld, dst, dst_ld, (int)rows, (int)cols);
    APEXW_TRY_HIP(hipGetLastError());
    src = dst;
    ld = dst_ld;
    return APEXW_OK;
}

}  // namespace
}  // namespace apexw
