// ops_qk_norm_rope.hip -- the norm of each head of queries and keys with the
// position rotation, forward and backward, one pass over the data each.
//
//     n = x / sqrt(mean x^2 + eps)      y = R(pos) (n w)
//     dn = R(pos)^T dy    dw = sum dn n    dx = (dn w - n mean(dn w n)) / sqrt(..)
//
// R turns pair i of a head's first rotary_dim values by pos theta^(-2 i /
// rotary_dim).  A group of G lanes holds one head in registers, eight values a
// lane, so that both values of a pair are in one lane: two runs of four, the
// pair's first values and its second ones (or eight adjacent values where pairs
// lie side by side).  A workgroup takes all heads of a token, queries and keys
// together; the angles of a token are formed once, for all of its heads.
//
// Angles: turns = pos theta^(..) / 2 pi in fp64, of which the whole ones are
// dropped before sin and cos in fp32, so that positions of a million lose
// nothing.  Norms and rotations are fp32, one rounding at the end.  The weights'
// gradients are summed in registers over a workgroup's tokens and heads, then
// over workgroups in a fixed order by a second launch: no atomics.
//
// Bound by memory: 16384 tokens, 32 + 8 heads of 128, bf16, forward 69 us (4.9
// TB/s) and backward 103 us (4.9 TB/s) on an MI355X, fp32 131 (5.1) and 203 (5.0);
// 32 tokens 3.6 us.  With the angles formed by every lane for itself the two took
// 91 and 146 us, without the next row's values under way the backward pass 122; of
// 3 to 6 waves a unit's fourth, 4 measured best in bf16 (6 spill: 288 us for both).
// In fp32 four waves leave the backward pass's vector modes two or four registers
// short, which pass through 12 or 20 bytes of scratch memory a lane.
#include "ops_common.hpp"
#include "ops_rounds.hpp"

// Multiply-adds are written out: what the values are reached by (Mode) does not
// change a bit.
#pragma clang fp contract(off)

namespace apexw {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;

struct Heads {
    const void *p;
    int64_t token, head;   // strides in elements
};

struct QkArgs {
    Heads q, k, dq, dk;
    const void *q_weight, *k_weight;
    const int64_t *positions;
    void *q_out, *k_out;   // forward: y; backward: the gradients of q and k
    float *part;           // backward: a row of 2 * head_dim sums per workgroup
    int32_t tokens, q_heads, k_heads, head_dim, rotary_dim, interleaved;
    double log2_theta;
    float eps;
};

constexpr int kThreads = 256, kTokens = 4;

// How a head's values are reached: one by one; or as two aligned vectors of four a
// lane, the pairs' first values and their second ones (kSplit) or pairs side by
// side (kPairs), the lane's pairs all turned or none of them.
enum Mode { kSingle, kSplit, kPairs };

// The eight places of lane g of a head's G lanes: `at(j)` is the element of
// value j, head_dim or more where there is none.
struct Places {
    int s0, r2;              // the lane's first pair; pairs that turn
    int a, b;                // first element of each run of four
    int hd, half;            // half: pairs of the values past rotary_dim
    bool split;              // pairs in two runs (not side by side)

    __device__ Places(const QkArgs &q, int g) {
        hd = q.head_dim;
        split = !q.interleaved;
        s0 = 4 * g;
        r2 = q.rotary_dim / 2;
        half = (hd - q.rotary_dim + 1) / 2;
        a = at(0);
        b = at(4);
    }
    __device__ int at(int j) const {
        if (!split) return 2 * s0 + j;
        const int s = s0 + (j & 3), second = j >> 2;
        if (s < r2) return second ? s + r2 : s;
        const int u = s - r2;
        if (u >= half) return hd;
        return second ? (half + u < hd - 2 * r2 ? 2 * r2 + half + u : hd) : 2 * r2 + u;
    }
};

template <class T> struct Vec4;
template <> struct Vec4<float> { typedef f32x4 type; };
template <> struct Vec4<__bf16> { typedef bf16x4 type; };

// Eight values of a head, as they lie in memory: the next row's are on their way
// while a row is worked on.
template <class T, Mode MODE>
struct Raw {
    T v[8];
    __device__ __forceinline__ Raw(const T *p, const Places &pl) {
        if constexpr (MODE != kSingle) {
            typedef typename Vec4<T>::type V;
            V x, y;
            if (pl.a < pl.hd) {
                x = *reinterpret_cast<const V *>(p + pl.a);
                y = *reinterpret_cast<const V *>(p + pl.b);
            } else {
                x = y = (V)(T)0.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = x[j];
                v[4 + j] = y[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = pl.at(j);
                v[j] = e < pl.hd ? p[e] : (T)0.0f;
            }
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = (float)v[j];
    }
};

template <class T, Mode MODE>
__device__ __forceinline__ void store8(T *p, const Places &pl, const float (&v)[8]) {
    if constexpr (MODE != kSingle) {
        typedef typename Vec4<T>::type V;
        if (pl.a >= pl.hd) return;
        V x, y;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = (T)v[j];
            y[j] = (T)v[4 + j];
        }
        *reinterpret_cast<V *>(p + pl.a) = x;
        *reinterpret_cast<V *>(p + pl.b) = y;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = pl.at(j);
            if (e < pl.hd) p[e] = (T)v[j];
        }
    }
}

// Turns the lane's four pairs by their angles (SIGN -1: back).  Pairs past
// rotary_dim are left alone: an infinity there stays in its place.
template <Mode MODE, int SIGN>
__device__ __forceinline__ void turn(float (&v)[8], const float (&c)[4], const float (&s)[4],
                                     const Places &pl) {
    const bool split = MODE == kSplit || (MODE == kSingle && pl.split);
    if (pl.s0 >= pl.r2) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float &a = split ? v[i] : v[2 * i], &b = split ? v[4 + i] : v[2 * i + 1];
        if (MODE == kSingle && pl.s0 + i >= pl.r2) continue;
        const float x = fmaf(a, c[i], -SIGN * (b * s[i])), y = fmaf(b, c[i], SIGN * (a * s[i]));
        a = x;
        b = y;
    }
}

template <int CTRL>
__device__ __forceinline__ float across(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL,
                                                                 0xf, 0xf, true));
}
// The sum over a row's G lanes, in all of them.
template <int G>
__device__ __forceinline__ float row_sum(float x) {
    x += across<0xb1>(x);                    // the neighbour, quad_perm 1 0 3 2
    x += across<0x4e>(x);                    // quad_perm 2 3 0 1
    x += across<0x141>(x);                   // the other four of eight, row_half_mirror
    if (G >= 16) x += across<0x140>(x);      // the other eight of sixteen, row_mirror
    if (G >= 32) x += __shfl_xor(x, 16);
    if (G >= 64) x += __shfl_xor(x, 32);
    return x;
}

// The angles of TPI tokens' pairs, formed once by the workgroup's threads: sin and
// cos of a position cost more than all of a head's other work in one lane.  Two
// sets take turns, so that one barrier a round is enough.
constexpr int kMaxPairs = 256;

template <int TPI>
struct Angles {
    double turns[kMaxPairs];         // of one position's step, for each pair
    float cs[2][2][TPI][kMaxPairs];  // cos, sin

    __device__ __forceinline__ void start(const QkArgs &q) {
        const int r2 = q.rotary_dim / 2;
        for (int i = threadIdx.x; i < r2; i += kThreads)
            // 1 / 2 pi
            turns[i] = exp2(-(double)i / r2 * q.log2_theta) * 0.15915494309189535;
        __syncthreads();
    }
    __device__ __forceinline__ void round(const QkArgs &q, int set, int first) {
        const int r2 = q.rotary_dim / 2;
        for (int i = threadIdx.x; i < TPI * r2; i += kThreads) {
            const int t = i / r2, pair = i - t * r2;
            if (first + t >= q.tokens) break;
            const double a = (double)q.positions[first + t] * turns[pair];
            sincospif((float)(2.0 * (a - rint(a))), &cs[set][1][t][pair], &cs[set][0][t][pair]);
        }
        __syncthreads();
    }
    // a lane's four pairs (read where the lane has such pairs at all)
    __device__ __forceinline__ void get(int set, int t, const Places &pl, float (&c)[4], float (&s)[4]) const {
        if (pl.s0 >= pl.r2) return;
        *reinterpret_cast<f32x4 *>(c) = *reinterpret_cast<const f32x4 *>(&cs[set][0][t][pl.s0]);
        *reinterpret_cast<f32x4 *>(s) = *reinterpret_cast<const f32x4 *>(&cs[set][1][t][pl.s0]);
    }
};

// One of queries and keys: its rows (token, head) of a round's TPI tokens, and
// which of them this thread's group of lanes takes.
struct Rows {
    int heads, first, step;
    // parts: workgroups that share the rows; part: this one, none of its rows
    // where it is not among them
    __device__ __forceinline__ Rows(int heads, int at, int rows, int part, int parts, int tokens)
        : heads(heads), first(part >= 0 && part < parts ? part * rows + at : tokens * heads),
          step(parts * rows) {}
};
// (passes over one token's queries by R rows at a time)
__device__ __forceinline__ int passes(int heads, int rows) { return (heads + rows - 1) / rows; }

template <class T, int G, Mode MODE, int TPI>
__global__ __launch_bounds__(kThreads, 4) void forward_kernel(const QkArgs a) {
    constexpr int R = kThreads / G;
    __shared__ __attribute__((aligned(16))) Angles<TPI> angles;
    angles.start(a);
    const Places pl(a, threadIdx.x % G);
    const float inv = 1.0f / a.head_dim;
    const int at = threadIdx.x / G, pq = gridDim.y == 1 ? 1 : passes(a.q_heads, R);
    int set = 0;
    for (int t0 = blockIdx.x * TPI; t0 < a.tokens;
         t0 = next_round(t0, gridDim.x * TPI, a.tokens), set ^= 1) {
        angles.round(a, set, t0);
        const int left = a.tokens - t0 < TPI ? a.tokens - t0 : TPI;
        auto rows = [&](const Heads &in, const void *weight, void *out, Rows r) {
            const int end = left * r.heads;
            if (r.first >= end) return;
            float w[8];
            Raw<T, MODE>((const T *)weight, pl).get(w);
            int tt = r.first / r.heads, h = r.first - tt * r.heads;
            auto load = [&] { return Raw<T, MODE>((const T *)in.p + (t0 + tt) * in.token + h * in.head, pl); };
            Raw<T, MODE> ahead = load();
            for (int i = r.first; i < end; i += r.step) {
                const int hh = h, at_t = tt;
                float v[8], c[4], s[4];
                ahead.get(v);
                if (i + r.step < end) {
                    tt = (i + r.step) / r.heads;
                    h = i + r.step - tt * r.heads;
                    ahead = load();
                }
                angles.get(set, at_t, pl, c, s);
                float ss = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
                const float rstd = rsqrtf(fmaf(row_sum<G>(ss), inv, a.eps));
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * w[j];
                turn<MODE, 1>(v, c, s, pl);
                store8<T, MODE>((T *)out + ((int64_t)(t0 + at_t) * r.heads + hh) * a.head_dim, pl, v);
            }
        };
        rows(a.q, a.q_weight, a.q_out, Rows(a.q_heads, at, R, blockIdx.y, pq, TPI));
        rows(a.k, a.k_weight, a.k_out,
             Rows(a.k_heads, at, R, gridDim.y == 1 ? 0 : blockIdx.y - pq, gridDim.y == 1 ? 1 : gridDim.y - pq, TPI));
    }
}

// (value by value the places take registers too: two waves, or they would spill)
template <class T, int G, Mode MODE, int TPI>
__global__ __launch_bounds__(kThreads, MODE == kSingle ? 2 : 4) void backward_kernel(const QkArgs a) {
    constexpr int R = kThreads / G, WAVES = kThreads / 64;
    __shared__ __attribute__((aligned(16))) Angles<TPI> angles;
    __shared__ float lds[WAVES][2][G * 8];
    angles.start(a);
    const Places pl(a, threadIdx.x % G);
    const float inv = 1.0f / a.head_dim;
    const int at = threadIdx.x / G, pq = gridDim.y == 1 ? 1 : passes(a.q_heads, R);
    float sum_q[8], sum_k[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum_q[j] = sum_k[j] = 0.0f;
    int set = 0;
    for (int t0 = blockIdx.x * TPI; t0 < a.tokens;
         t0 = next_round(t0, gridDim.x * TPI, a.tokens), set ^= 1) {
        angles.round(a, set, t0);
        const int left = a.tokens - t0 < TPI ? a.tokens - t0 : TPI;
        auto rows = [&](const Heads &in, const Heads &gr, const void *weight, void *out,
                        float (&sum)[8], Rows r) {
            const int end = left * r.heads;
            if (r.first >= end) return;
            float w[8];
            Raw<T, MODE>((const T *)weight, pl).get(w);
            int tt = r.first / r.heads, h = r.first - tt * r.heads;
            auto load = [&](const Heads &of) {
                return Raw<T, MODE>((const T *)of.p + (t0 + tt) * of.token + h * of.head, pl);
            };
            Raw<T, MODE> ahead = load(in), d_ahead = load(gr);
            for (int i = r.first; i < end; i += r.step) {
                const int hh = h, at_t = tt;
                float v[8], d[8], c[4], s[4];
                ahead.get(v);
                d_ahead.get(d);
                if (i + r.step < end) {
                    tt = (i + r.step) / r.heads;
                    h = i + r.step - tt * r.heads;
                    ahead = load(in);
                    d_ahead = load(gr);
                }
                angles.get(set, at_t, pl, c, s);
                turn<MODE, -1>(d, c, s, pl);
                float ss = 0.0f, dot = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    ss = fmaf(v[j], v[j], ss);
                    dot = fmaf(v[j], d[j] * w[j], dot);
                }
                const float rstd = rsqrtf(fmaf(row_sum<G>(ss), inv, a.eps));
                const float mean = row_sum<G>(dot) * inv * rstd;      // mean(dn w n)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float n = v[j] * rstd;
                    sum[j] = fmaf(d[j], n, sum[j]);
                    v[j] = rstd * fmaf(-n, mean, d[j] * w[j]);
                }
                if (out != nullptr)
                    store8<T, MODE>((T *)out + ((int64_t)(t0 + at_t) * r.heads + hh) * a.head_dim, pl, v);
            }
        };
        rows(a.q, a.dq, a.q_weight, a.q_out, sum_q, Rows(a.q_heads, at, R, blockIdx.y, pq, TPI));
        rows(a.k, a.dk, a.k_weight, a.k_out, sum_k,
             Rows(a.k_heads, at, R, gridDim.y == 1 ? 0 : blockIdx.y - pq, gridDim.y == 1 ? 1 : gridDim.y - pq, TPI));
    }
    // the wave's heads, then the workgroup's waves
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int d = G; d < 64; d *= 2) {
            sum_q[j] += __shfl_xor(sum_q[j], d);
            sum_k[j] += __shfl_xor(sum_k[j], d);
        }
    const int g = threadIdx.x % G;
    if (threadIdx.x % 64 < G) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            lds[threadIdx.x / 64][0][g * 8 + j] = sum_q[j];
            lds[threadIdx.x / 64][1][g * 8 + j] = sum_k[j];
        }
    }
    __syncthreads();
    if (threadIdx.x >= 2 * G) return;
    const int which = threadIdx.x / G;               // (2 G <= 128: G lanes for each weight)
    float *part = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * a.head_dim +
                  which * a.head_dim;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float x = 0.0f;
        for (int w = 0; w < WAVES; ++w) x += lds[w][which][g * 8 + j];
        const int e = pl.at(j);
        if (e < a.head_dim) part[e] = x;
    }
}

// The workgroups' sums added up: 16 columns a workgroup, 64 strands of rows, each
// with eight loads under way.
template <class T>
__global__ __launch_bounds__(1024) void weights_kernel(const float *part, int32_t rows,
                                                       int32_t head_dim, T *dqw, T *dkw) {
    __shared__ float lds[64][17];
    const int c = threadIdx.x & 15, k = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
    float x = 0.0f;
    if (col < 2 * head_dim) {
        const float *p = part + col;
#pragma unroll 8
        for (int r = k; r < rows; r += 64) x += p[(int64_t)r * 2 * head_dim];
    }
    lds[k][c] = x;
    for (int half = 32; half > 0; half /= 2) {
        __syncthreads();
        if (k < half) lds[k][c] += lds[k + half][c];
    }
    if (k != 0 || col >= 2 * head_dim) return;
    T *out = col < head_dim ? dqw : dkw;
    if (out != nullptr) out[col < head_dim ? col : col - head_dim] = (T)lds[0][c];
}

struct Shape {
    apexw_qk_norm_rope_shape p;
    bool many;
    int gx, gy, rows;     // grid; heads a workgroup takes at once
};

int lanes(int head_dim) { return head_dim <= 64 ? 8 : head_dim <= 128 ? 16 : head_dim <= 256 ? 32 : 64; }

int check_shape(const apexw_qk_norm_rope_shape *p, bool backward, Shape &s) {
    if (p == nullptr) return fail(APEXW_EINVAL, "shape is NULL");
    if (p->dtype != APEXW_F32 && p->dtype != APEXW_BF16)
        return fail(APEXW_EDTYPE, "unknown element type %d", p->dtype);
    if (p->tokens < 0 || p->tokens >= (int64_t)1 << 31 || p->q_heads < 1 || p->q_heads > 4096 ||
        p->k_heads < 1 || p->k_heads > 4096 || p->head_dim < 1 || p->head_dim > 512)
        return fail(APEXW_EINVAL, "tokens %lld, heads %d and %d or head_dim %d out of range",
                    (long long)p->tokens, p->q_heads, p->k_heads, p->head_dim);
    if (p->rotary_dim < 0 || p->rotary_dim > p->head_dim || p->rotary_dim % 2 != 0)
        return fail(APEXW_EINVAL, "rotary_dim %d: even, at most head_dim %d", p->rotary_dim,
                    p->head_dim);
    if (!(p->theta > 0) || p->theta > 1e300) return fail(APEXW_EINVAL, "theta %g out of range", p->theta);
    if (!(p->eps >= 0)) return fail(APEXW_EINVAL, "eps %g is negative", p->eps);
    s.p = *p;
    // strides: 0 stands for contiguous
    const int64_t hd = p->head_dim;
    int64_t *const st[4] = {s.p.q_stride, s.p.k_stride, s.p.dq_stride, s.p.dk_stride};
    for (int i = 0; i < 4; ++i) {
        if (st[i][0] < 0 || st[i][1] < 0) return fail(APEXW_EINVAL, "a stride is negative");
        if (st[i][1] == 0) st[i][1] = hd;
        if (st[i][0] == 0) st[i][0] = hd * (i % 2 == 0 ? p->q_heads : p->k_heads);
    }
    s.rows = kThreads / lanes(p->head_dim);
    // Few tokens: a token a round, and a workgroup for each pass over its heads.
    // Many: rounds of four tokens with all of their heads, workgroups walking
    // over them.  Measured, us, few against many, 32 + 8 heads of 128, bf16: forward
    // 256 tokens 4.2 and 8.0, 768 7.1 and 8.7, 1024 8.5 and 9.1, 1536 11.1 and 9.8;
    // backward, whose workgroups leave a row of sums each, 256 tokens 10.6 and 13.1,
    // 512 14.8 and 13.8, 1024 23.5 and 15.1.  12 + 3 heads of 96 and fp32 meet at the
    // same numbers of tokens.
    const int passes = (int)(div_up(p->q_heads, s.rows) + div_up(p->k_heads, s.rows));
    s.many = p->tokens >= (backward ? 512 : 1024);
    s.gx = !s.many ? (int)p->tokens : (int)(div_up(p->tokens, kTokens) < 1024 ? div_up(p->tokens, kTokens) : 1024);
    s.gy = s.many ? 1 : passes;
    return APEXW_OK;
}

// The vector modes where all of a lane's values are two aligned vectors of four,
// in pairs that are all turned or none of them.
Mode mode_of(const Shape &s, const void *const *ptrs, int n, bool backward) {
    const auto &p = s.p;
    const int bytes = p.dtype == APEXW_BF16 ? 8 : 16;
    if (p.rotary_dim % 8 != 0 || p.head_dim % 8 != 0) return kSingle;
    for (int i = 0; i < 2; ++i)
        if (p.q_stride[i] % 4 != 0 || p.k_stride[i] % 4 != 0 ||
            (backward && (p.dq_stride[i] % 4 != 0 || p.dk_stride[i] % 4 != 0)))
            return kSingle;
    for (int i = 0; i < n; ++i)
        if ((uintptr_t)ptrs[i] % bytes != 0) return kSingle;
    return p.interleaved ? kPairs : kSplit;
}

QkArgs arguments(const Shape &s, const void *q, const void *k, const void *qw, const void *kw,
                 const int64_t *positions, void *q_out, void *k_out) {
    const auto &p = s.p;
    QkArgs a{};
    a.q = {q, p.q_stride[0], p.q_stride[1]};
    a.k = {k, p.k_stride[0], p.k_stride[1]};
    a.q_weight = qw;
    a.k_weight = kw;
    a.positions = positions;
    a.q_out = q_out;
    a.k_out = k_out;
    a.tokens = (int32_t)p.tokens;
    a.q_heads = p.q_heads;
    a.k_heads = p.k_heads;
    a.head_dim = p.head_dim;
    a.rotary_dim = p.rotary_dim;
    a.interleaved = p.interleaved != 0;
    a.log2_theta = __builtin_log2(p.theta);
    a.eps = p.eps;
    return a;
}

template <class T, int G, Mode MODE>
int launch(const Shape &s, const QkArgs &a, bool backward, hipStream_t stream) {
    const dim3 grid(s.gx, s.gy);
    if (backward) {
        if (s.many) backward_kernel<T, G, MODE, kTokens><<<grid, kThreads, 0, stream>>>(a);
        else backward_kernel<T, G, MODE, 1><<<grid, kThreads, 0, stream>>>(a);
    } else {
        if (s.many) forward_kernel<T, G, MODE, kTokens><<<grid, kThreads, 0, stream>>>(a);
        else forward_kernel<T, G, MODE, 1><<<grid, kThreads, 0, stream>>>(a);
    }
    APEXW_TRY_HIP(hipGetLastError());
    return APEXW_OK;
}

template <class T, int G>
int launch(const Shape &s, const QkArgs &a, bool backward, Mode mode, hipStream_t stream) {
    switch (mode) {
        case kSplit: return launch<T, G, kSplit>(s, a, backward, stream);
        case kPairs: return launch<T, G, kPairs>(s, a, backward, stream);
        default: return launch<T, G, kSingle>(s, a, backward, stream);
    }
}

template <class T>
int launch(const Shape &s, const QkArgs &a, bool backward, Mode mode, hipStream_t stream) {
    switch (lanes(s.p.head_dim)) {
        case 8: return launch<T, 8>(s, a, backward, mode, stream);
        case 16: return launch<T, 16>(s, a, backward, mode, stream);
        case 32: return launch<T, 32>(s, a, backward, mode, stream);
        default: return launch<T, 64>(s, a, backward, mode, stream);
    }
}

int64_t work_bytes(const Shape &s) {
    return ws_round((int64_t)s.gx * s.gy * 2 * s.p.head_dim * (int64_t)sizeof(float));
}

// Element accesses are as wide as an element at least.
int check_element(const void *p, const Shape &s, const char *name, bool optional = false) {
    if (p == nullptr) return optional ? APEXW_OK : fail(APEXW_EINVAL, "%s is NULL", name);
    const int eb = s.p.dtype == APEXW_BF16 ? 2 : 4;
    if ((uintptr_t)p % eb != 0)
        return fail(APEXW_EINVAL, "%s is not aligned to its %d-byte elements", name, eb);
    return APEXW_OK;
}

}  // namespace
}  // namespace apexw

using namespace apexw;

extern "C" int apexw_qk_norm_rope_forward(const apexw_qk_norm_rope_shape *shape, const void *q,
                                          const void *k, const void *q_weight,
                                          const void *k_weight, const int64_t *positions,
                                          void *q_out, void *k_out, void *stream) {
    Shape s;
    APEXW_TRY(check_shape(shape, false, s));
    if (s.p.tokens == 0) return APEXW_OK;
    const void *const ptrs[6] = {q, k, q_weight, k_weight, q_out, k_out};
    const char *const names[6] = {"q", "k", "q_weight", "k_weight", "q_out", "k_out"};
    for (int i = 0; i < 6; ++i) APEXW_TRY(check_element(ptrs[i], s, names[i]));
    if (positions == nullptr) return fail(APEXW_EINVAL, "positions is NULL");
    const QkArgs a = arguments(s, q, k, q_weight, k_weight, positions, q_out, k_out);
    const Mode mode = mode_of(s, ptrs, 6, false);
    return s.p.dtype == APEXW_BF16 ? launch<__bf16>(s, a, false, mode, (hipStream_t)stream)
                                   : launch<float>(s, a, false, mode, (hipStream_t)stream);
}

extern "C" int apexw_qk_norm_rope_workspace_bytes(const apexw_qk_norm_rope_shape *shape,
                                                  size_t *out_bytes) {
    Shape s;
    APEXW_TRY(check_shape(shape, true, s));
    if (out_bytes == nullptr) return fail(APEXW_EINVAL, "out_bytes is NULL");
    *out_bytes = (size_t)work_bytes(s);
    return APEXW_OK;
}

extern "C" int apexw_qk_norm_rope_backward(const apexw_qk_norm_rope_shape *shape, const void *dq,
                                           const void *dk, const void *q, const void *k,
                                           const void *q_weight, const void *k_weight,
                                           const int64_t *positions, void *q_grad, void *k_grad,
                                           void *dq_weight, void *dk_weight, void *workspace,
                                           size_t workspace_len, void *stream) {
    Shape s;
    APEXW_TRY(check_shape(shape, true, s));
    const void *const ptrs[10] = {dq, dk, q, k, q_weight, k_weight, q_grad, k_grad, dq_weight, dk_weight};
    const char *const names[10] = {"dq", "dk", "q", "k", "q_weight", "k_weight", "q_grad", "k_grad",
                                   "dq_weight", "dk_weight"};
    for (int i = 0; i < 10; ++i)
        APEXW_TRY(check_element(ptrs[i], s, names[i], i >= 6 || s.p.tokens == 0));
    if (positions == nullptr && s.p.tokens > 0) return fail(APEXW_EINVAL, "positions is NULL");
    APEXW_TRY(check_room(workspace, workspace_len, work_bytes(s), "workspace"));
    QkArgs a = arguments(s, q, k, q_weight, k_weight, positions, q_grad, k_grad);
    a.dq = {dq, s.p.dq_stride[0], s.p.dq_stride[1]};
    a.dk = {dk, s.p.dk_stride[0], s.p.dk_stride[1]};
    a.part = (float *)workspace;
    const hipStream_t st = (hipStream_t)stream;
    const bool bf = s.p.dtype == APEXW_BF16;
    const Mode mode = mode_of(s, ptrs, 8, true);
    if (s.p.tokens > 0)
        APEXW_TRY(bf ? launch<__bf16>(s, a, true, mode, st) : launch<float>(s, a, true, mode, st));
    if (dq_weight == nullptr && dk_weight == nullptr) return APEXW_OK;
    const int grid = (int)div_up(2 * s.p.head_dim, 16);
    if (bf)
        weights_kernel<<<grid, 1024, 0, st>>>(a.part, s.gx * s.gy, s.p.head_dim,
                                              (__bf16 *)dq_weight, (__bf16 *)dk_weight);
    else
        weights_kernel<<<grid, 1024, 0, st>>>(a.part, s.gx * s.gy, s.p.head_dim,
                                              (float *)dq_weight, (float *)dk_weight);
    APEXW_TRY_HIP(hipGetLastError());
    return APEXW_OK;
}
