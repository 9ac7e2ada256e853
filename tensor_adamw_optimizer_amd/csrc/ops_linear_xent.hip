// ops_linear_xent.hip -- softmax cross entropy of a linear layer's outputs over
// a vocabulary, forward and backward, without the logits ever in memory.
//
//     z = x W^T    lse = log sum_n exp z_n    loss = lse - z_target
//     p = (exp(z - lse) - onehot(target)) s   dx = p W   dW = p^T x
//
// s is the gradient of the token's loss.  Tokens that carry no loss are left
// out before the products: their rows are skipped when x is gathered, and the
// products take the number of rows that are left from the device.
//
// Forward: one product whose epilogue reduces each 32 or 64 columns of a row to
// their largest logit and the sum of exp(z - largest); a second kernel joins
// these pairs.  More than 2^30 logits are formed in pieces of the vocabulary, the
// pairs of a piece joined to those before it.  Backward, in pieces of the vocabulary: p of a piece from a
// second product over x and W, then the piece's rows of dW, and the piece's
// share of dx added to an fp32 array.  Forming z twice costs a quarter of the
// pass (8 instead of 6 T D V); the logits would take 4 T V bytes.
//
// Roundings in bf16: p once, where it becomes an operand of the matrix
// instructions, and each output once.  A factor that all tokens share (of a mean
// or a sum) is applied to the fp32 products, not to p: s (p - 1) of the many
// targets with a small p would all round by the same share of s.  z, lse, the softmax sums and dx's sum
// over the pieces are fp32, the mean's sum is fp64.
//
// Measured on an MI355X, bf16: 8192 tokens, 4096 x 131072, forward and backward
// 26.2 ms (1340 TFLOP/s of the 8 T D V, the products' rate); 4096 tokens, a quarter
// of them without a loss, 2048 x 49999, 2.3 ms; 16 tokens scored, 2048 x 32000, 33
// us (26 us of it the weight's 131 MB).
#include "ops_rows.hpp"

namespace apexw {
namespace {

// Rows that count, in order: their number, each one's token and class, each
// token's row (-1 for none) and, where a backward pass asks, each row's factor
// s.  One workgroup walks the tokens, 4096 at a time.  A class outside the
// vocabulary is marked -2: its row's loss and factor are NaN.
enum { kMean, kSum, kNone };

__global__ __launch_bounds__(1024) void rows_kernel(const int64_t *target, int64_t ignore,
                                                    int64_t vocab, int32_t tokens, int32_t *count,
                                                    int32_t *token_of, int32_t *class_of,
                                                    int32_t *row_of) {
    __shared__ int sums[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int base = 0;
    for (int t0 = 0; t0 < tokens; t0 += 4096) {
        const int first = t0 + tid * 4;
        int64_t c[4];
        int n = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c[j] = first + j < tokens ? target[first + j] : ignore;
            n += c[j] != ignore;
        }
        int before = n;                                // inclusive sum over the wave
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int v = __shfl_up(before, d);
            if (lane >= d) before += v;
        }
        if (lane == 63) sums[wave] = before;
        __syncthreads();
        int at = base + before - n;
        for (int w = 0; w < 16; ++w) {
            if (w < wave) at += sums[w];
            base += sums[w];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (first + j >= tokens) break;
            const bool on = c[j] != ignore;
            row_of[first + j] = on ? at : -1;
            if (on) {
                token_of[at] = first + j;
                class_of[at] = c[j] >= 0 && c[j] < vocab ? (int32_t)c[j] : -2;
                ++at;
            }
        }
        __syncthreads();
    }
    if (tid == 0) *count = base;
}

// Row r of dst is x's row token_of[r].
template <class T>
__global__ __launch_bounds__(256) void gather_kernel(const T *x, int64_t x_ld, T *dst, int64_t ld,
                                                     int32_t cols, const int32_t *count,
                                                     const int32_t *token_of) {
    const int rows = *count;
    for (int r = blockIdx.x; r < rows; r += gridDim.x)
        pad_row(x + (int64_t)token_of[r] * x_ld, dst + r * ld, ld, cols);
}

// What a backward pass asks of the rows beside.
struct Factors {
    const float *lse, *dloss;
    int32_t reduction;
    float *row_lse, *factor, *common;
};
__device__ __forceinline__ void put_factors(const Factors &f, int r, int t, int cls) {
    f.row_lse[r] = f.lse[t];
    f.factor[r] = cls < 0 ? NAN : f.reduction == kNone ? f.dloss[t] : 1.0f;
}
// (0 where no token carries a loss: their zeros stay so if dloss is not finite)
__device__ __forceinline__ void put_common(const Factors &f, int n) {
    *f.common = n == 0 ? 0.0f
                : f.reduction == kNone ? 1.0f
                : f.reduction == kMean ? *f.dloss / (float)n : *f.dloss;
}

// rows_kernel, gather_kernel and factors_kernel in one launch, for at most kAtOnce
// tokens: a workgroup a token, which counts the rows before it for itself.
constexpr int kAtOnce = 2048;
template <class T>
__global__ __launch_bounds__(256) void rows_at_once_kernel(
    const int64_t *target, int64_t ignore, int64_t vocab, int32_t tokens, int32_t *count,
    int32_t *token_of, int32_t *class_of, int32_t *row_of, const T *x, int64_t x_ld, T *dst,
    int64_t ld, int32_t cols, const Factors f) {
    __shared__ int sums[4][2];
    const int t = blockIdx.x;
    int before = 0, all = 0;
    for (int s = threadIdx.x; s < tokens; s += 256) {
        const int on = target[s] != ignore;
        all += on;
        before += s < t ? on : 0;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        all += __shfl_xor(all, d);
        before += __shfl_xor(before, d);
    }
    if (threadIdx.x % 64 == 0) {
        sums[threadIdx.x / 64][0] = before;
        sums[threadIdx.x / 64][1] = all;
    }
    __syncthreads();
    before = sums[0][0] + sums[1][0] + sums[2][0] + sums[3][0];
    all = sums[0][1] + sums[1][1] + sums[2][1] + sums[3][1];
    const int cls = apexw::class_of(target[t], ignore, vocab);
    if (threadIdx.x == 0) {
        row_of[t] = cls == -1 ? -1 : before;
        if (cls != -1) {
            token_of[before] = t;
            class_of[before] = cls;
            if (f.lse != nullptr) put_factors(f, before, t, cls);
        }
        if (t == 0) {
            *count = all;
            if (f.lse != nullptr) put_common(f, all);
        }
    }
    if (cls != -1)
        pad_row(x + (int64_t)t * x_ld, dst + before * ld, ld, cols);
}

// The joined pair of two parts of a row.
__device__ __forceinline__ void join(float &top, float &sum, float2 p) {
    const float m = fmaxf(top, p.x), ref = m == -INFINITY ? 0.0f : m;
    sum = sum * fast_exp(top - ref) + p.y * fast_exp(p.x - ref);
    top = m;
}

// A row's pair and its target's logit from slabs of a product split over k (small
// vocabularies, whose tiles alone would not fill the chip): a workgroup a row.
__global__ __launch_bounds__(256) void reduce_slabs_kernel(const float *slab, int64_t slab_elems,
                                                           int splits, int64_t ld, int32_t col0,
                                                           int32_t cols, const int32_t *count,
                                                           const int32_t *class_of, float2 *part,
                                                           float *z_target) {
    __shared__ float2 lds[256];
    const int r = blockIdx.x;
    if (r >= *count) return;
    const int t = class_of[r] - col0;
    float top = -INFINITY, sum = 0.0f;
    for (int n = threadIdx.x * 4; n < cols; n += 1024) {
        f32x4 v = {0, 0, 0, 0};
        for (int k = 0; k < splits; ++k)
            v += *reinterpret_cast<const f32x4 *>(slab + k * slab_elems + r * ld + n);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (n + q >= cols) continue;
            if (n + q == t) z_target[r] = v[q];
            join(top, sum, make_float2(v[q], 1.0f));
        }
    }
    lds[threadIdx.x] = make_float2(top, sum);
    for (int half = 128; half > 0; half /= 2) {
        __syncthreads();
        if ((int)threadIdx.x < half) {
            join(top, sum, lds[threadIdx.x + half]);
            lds[threadIdx.x] = make_float2(top, sum);
        }
    }
    if (threadIdx.x == 0) part[r] = make_float2(top, sum);
}

// Joins each row's pairs, in pieces of the vocabulary to that of the pieces before:
// 16 rows a workgroup, 16 threads a row.  The last piece has the row's results.
__global__ __launch_bounds__(256) void join_kernel(const float2 *part, int64_t ld, int32_t groups,
                                                   float2 *before, bool first, bool last,
                                                   const int32_t *count, const int32_t *token_of,
                                                   const int32_t *class_of, const float *z_target,
                                                   float *token_loss, float *lse) {
    __shared__ float2 lds[256];
    const int rows = *count, r = blockIdx.x * 16 + (threadIdx.x & 15), k = threadIdx.x >> 4;
    if ((int)blockIdx.x * 16 >= rows) return;
    float top = -INFINITY, sum = 0.0f;
    if (r < rows) {
        for (int g = k; g < groups; g += 16) {
            join(top, sum, part[g * ld + r]);
        }
    }
    lds[threadIdx.x] = make_float2(top, sum);
    __syncthreads();
    if (k != 0 || r >= rows) return;
    for (int j = 1; j < 16; ++j) join(top, sum, lds[threadIdx.x + 16 * j]);
    if (!first) join(top, sum, before[r]);
    if (!last) {
        before[r] = make_float2(top, sum);
        return;
    }
    const float l = top + logf(sum);
    const int t = token_of[r];
    lse[t] = l;
    token_loss[t] = class_of[r] < 0 ? NAN : l - z_target[r];
}

// The mean or sum of at most 64 tokens' losses, by one wave.
__device__ __forceinline__ void few_loss(float mine, bool on, int reduction, float *loss) {
    double sum = on ? mine : 0.0, n = on ? 1.0 : 0.0;
#pragma unroll
    for (int d = 32; d > 0; d /= 2) {
        sum += __shfl_xor(sum, d);
        n += __shfl_xor(n, d);
    }
    if ((threadIdx.x & 63) == 0 && reduction != kNone)
        *loss = (float)(reduction == kMean ? sum / (n > 0 ? n : 1.0) : sum);
}

// Joins the pairs of a few tokens: one workgroup does all of them, and the loss,
// where they are soon read; else a workgroup takes a token.
__global__ __launch_bounds__(1024) void few_join_kernel(const float2 *part, int32_t tokens,
                                                        int32_t groups, const int64_t *target,
                                                        int64_t ignore, int64_t vocab,
                                                        const float *z_target, float *token_loss,
                                                        float *lse, int32_t reduction, float *loss) {
    __shared__ float2 lds[1024];
    __shared__ float done[kRowsMax];
    int width = 1;                                    // a power of two of rows at once
    if (gridDim.x == 1)
        while (width < tokens) width *= 2;
    const int strands = 1024 / width, k = threadIdx.x / width;
    const int r = gridDim.x == 1 ? threadIdx.x % width : blockIdx.x;
    float top = -INFINITY, sum = 0.0f;
    if (r < tokens) {
        int g = k;
        for (; g + 3 * strands < groups; g += 4 * strands) {
            float2 p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = part[(int64_t)(g + j * strands) * tokens + r];
#pragma unroll
            for (int j = 0; j < 4; ++j) join(top, sum, p[j]);
        }
        for (; g < groups; g += strands) join(top, sum, part[(int64_t)g * tokens + r]);
    }
    lds[threadIdx.x] = make_float2(top, sum);
    for (int half = strands / 2; half > 0; half /= 2) {
        __syncthreads();
        if (k < half) {
            join(top, sum, lds[threadIdx.x + half * width]);
            lds[threadIdx.x] = make_float2(top, sum);
        }
    }
    if (k == 0 && r < tokens) {
        const float l = top + logf(sum);
        const int c = class_of(target[r], ignore, vocab);
        const float mine = c == -1 ? 0.0f : c < 0 ? NAN : l - z_target[r];
        lse[r] = c == -1 ? 0.0f : l;
        token_loss[r] = mine;
        if (gridDim.x == 1) done[r] = mine;
    }
    if (gridDim.x != 1) return;
    __syncthreads();
    if (threadIdx.x < 64) {
        const bool on = (int)threadIdx.x < tokens && target[threadIdx.x] != ignore;
        few_loss(on ? done[threadIdx.x] : 0.0f, on, reduction, loss);
    }
}

__global__ __launch_bounds__(64) void few_reduce_kernel(const int64_t *target, int64_t ignore,
                                                        int32_t tokens, int32_t reduction,
                                                        const float *token_loss, float *loss) {
    const bool on = (int)threadIdx.x < tokens && target[threadIdx.x] != ignore;
    few_loss(on ? token_loss[threadIdx.x] : 0.0f, on, reduction, loss);
}

// Zeros for the tokens that carry no loss, and the loss of all of them.
__global__ __launch_bounds__(1024) void reduce_kernel(const int32_t *row_of, const int32_t *count,
                                                      int32_t tokens, int32_t reduction,
                                                      float *token_loss, float *lse, float *loss) {
    __shared__ double sums[16];
    double sum = 0;
    for (int t = threadIdx.x; t < tokens; t += 1024) {
        if (row_of[t] < 0) {
            token_loss[t] = 0.0f;
            lse[t] = 0.0f;
        } else {
            sum += token_loss[t];
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d /= 2) sum += __shfl_xor(sum, d);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x != 0 || reduction == kNone) return;
    for (int w = 1; w < 16; ++w) sum += sums[w];
    const int n = *count;
    *loss = (float)(reduction == kMean ? sum / (n > 0 ? n : 1) : sum);
}

// Each row's lse and factor, in the rows' order, and the factor of them all.
__global__ __launch_bounds__(256) void factors_kernel(const int32_t *count, const int32_t *token_of,
                                                      const int32_t *class_of, const Factors f) {
    const int r = blockIdx.x * 256 + threadIdx.x, n = *count;
    if (r == 0) put_common(f, n);
    if (r < n) put_factors(f, r, token_of[r], class_of[r]);
}

// dx's rows back in their places: the sum of the splits' slabs times the common
// factor, rounded once, and zeros for tokens that carry no loss.
template <class T>
__global__ __launch_bounds__(256) void scatter_kernel(const float *slab, int64_t slab_elems,
                                                      int splits, int64_t ld, const int32_t *row_of,
                                                      T *out, int32_t tokens, int32_t cols,
                                                      const float *common) {
    const float factor = *common;
    for (int t = blockIdx.x; t < tokens; t += gridDim.x) {
        const int r = row_of[t];
        for (int n = threadIdx.x * 4; n < cols; n += 1024) {
            f32x4 s = {0, 0, 0, 0};
            if (r >= 0) {
                for (int k = 0; k < splits; ++k)
                    s += *reinterpret_cast<const f32x4 *>(slab + k * slab_elems + r * ld + n);
                s *= factor;                           // (0 times a factor that is not finite: NaN)
            }
            put4(out, (int64_t)cols, t, n, cols, s);
        }
    }
}

struct Shape {
    int64_t T, D, V, x_ld, ignore, Dp;
    int32_t reduction;
};

template <class T>
struct Xent {
    Shape s;
    hipStream_t stream;
    const T *x, *w;
    const int64_t *target;
    // workspace
    int32_t *count, *token_of, *class_of, *row_of;
    T *xc, *wp, *p;
    float *part, *before, *z_target, *row_lse, *factor, *common, *slab, *dw_slab;

    bool pad_d() const { return s.D % (16 / sizeof(T)) != 0; }

    // Classes in a piece of the backward pass: whole tiles, and p within 256 MiB, up
    // to 2^16 tokens in bf16 and 2^15 in fp32.  Of more tokens p has 2048 classes all
    // the same, 4 GiB of 2^20 in bf16: each piece reads and writes dx's fp32 sums, 8
    // bytes a token and width, half the time of such a piece's product; of narrower
    // pieces, four times it at 256 classes.
    int64_t piece() const {
        const int64_t c = ((int64_t)1 << 28) / ((s.T > 0 ? s.T : 1) * (int64_t)sizeof(T)) / 2048 * 2048;
        return c < 2048 ? (s.V < 2048 ? s.V : 2048) : c < s.V ? c : s.V;
    }

    void place_rows(Bump &b) {
        count = b.take<int32_t>(1);
        token_of = b.take<int32_t>(s.T);
        class_of = b.take<int32_t>(s.T);
        row_of = b.take<int32_t>(s.T);
        xc = b.take<T>(s.T * s.Dp);
        wp = pad_d() ? b.take<T>(s.V * s.Dp) : nullptr;
    }
    int64_t w_ld;
    int rows(const Factors &f) {
        if (s.T > 0 && s.T <= kAtOnce) {
            rows_at_once_kernel<T><<<(int)s.T, 256, 0, stream>>>(
                target, s.ignore, s.V, (int)s.T, count, token_of, class_of, row_of, x, s.x_ld, xc,
                s.Dp, (int)s.D, f);
            APEXW_TRY_HIP(hipGetLastError());
        } else {
            rows_kernel<<<1, 1024, 0, stream>>>(target, s.ignore, s.V, (int)s.T, count, token_of,
                                                class_of, row_of);
            APEXW_TRY_HIP(hipGetLastError());
            if (s.T > 0) {
                gather_kernel<T><<<(int)(s.T < 8192 ? s.T : 8192), 256, 0, stream>>>(
                    x, s.x_ld, xc, s.Dp, (int)s.D, count, token_of);
                APEXW_TRY_HIP(hipGetLastError());
                if (f.lse != nullptr) {
                    factors_kernel<<<(int)div_up(s.T, 256), 256, 0, stream>>>(count, token_of,
                                                                              class_of, f);
                    APEXW_TRY_HIP(hipGetLastError());
                }
            }
        }
        w_ld = s.D;
        return pad_operand(w, w_ld, wp, s.Dp, s.V, s.D, stream);
    }

    GemmArgs logits(int64_t c0, int64_t classes) const {
        GemmArgs a{};
        a.a = mat(xc, s.Dp);
        a.b = mat(w + c0 * w_ld, w_ld);
        a.M = (int)s.T;
        a.N = (int)classes;
        a.K = (int)s.D;
        a.m_dev = count;
        a.e.target = class_of;
        return a;
    }

    // Classes in a piece of the forward pass: whole tiles, and at most 2^30 logits, so
    // that their pairs stay within some 256 MiB and a launch's threads far below 2^32.
    int64_t forward_piece() const {
        const int64_t most = ((int64_t)1 << 30) / (s.T > 0 ? s.T : 1) / 256 * 256;
        if (s.V <= most) return s.V;
        return div_up(div_up(s.V, div_up(s.V, most)), 256) * 256;
    }
    int64_t forward_last() const { return s.V - (s.V - 1) / forward_piece() * forward_piece(); }

    Tiling tiling(int64_t classes) const { return pick_tiling<T>(s.T, classes, s.D, false, true); }
    // Groups of columns that are reduced to a pair, those of the last tile's
    // columns past the piece too.
    int64_t groups(int64_t classes) const {
        const Tiling t = tiling(classes);
        return t.splits > 1 ? 1 : div_up(classes, t.bn) * (t.bn / t.wave_cols);
    }

    // A few tokens: all of them go through the product of ops_rows.hpp, which reads
    // the weight where it lies.  More than 32 with a large weight: the tiles fetch that
    // faster, unless it would have to be copied to padded rows first.  Measured, us,
    // rows against tiles: 24 tokens, bf16, 2048 x 32000 37 and 49, 4096 x 131072 249
    // and 233, fp32 506 and 569; 48 tokens, bf16, 1024 x 32000 (63 MiB) 34 and 40,
    // 2048 x 32000 53 and 49, 4096 x 131072 346 and 235, 1030 x 32000 (padded) 32
    // and 74; 64 tokens, fp32, 512 x 32000 43 and 50, 4096 x 32000 225 and 173.
    bool few() const {
        return s.T <= 32 || (s.T <= kRowsMax && (s.V * s.D * (int64_t)sizeof(T) <= (int64_t)64 << 20 ||
                                                 pad_d()));
    }
    RowsTiling few_tiling() const { return rows_tiling(s.V, 1); }
    int64_t few_groups() const { return div_up(s.V, few_tiling().nf * 16); }
    bool at_once() const { return few_groups() * s.T <= 32768; }

    int64_t place_forward(Bump &b) {
        if (few()) {
            part = b.take<float>(few_groups() * s.T * 2);
            z_target = b.take<float>(s.T);
            return b.used;
        }
        place_rows(b);
        const int64_t c = forward_piece(), last = forward_last();
        part = b.take<float>((groups(c) > groups(last) ? groups(c) : groups(last)) * s.T * 2);
        before = b.take<float>(c < s.V ? s.T * 2 : 0);
        z_target = b.take<float>(s.T);
        const int64_t n0 = slab_elems<T>(s.T, c, s.D), n1 = slab_elems<T>(s.T, last, s.D);
        slab = b.take<float>(n0 > n1 ? n0 : n1);
        return b.used;
    }

    int few_forward(float *loss, float *token_loss, float *lse) {
        RowsArgs r{};
        r.a = (const char *)x;
        r.b0 = (const char *)w;
        r.lda = s.x_ld * (int64_t)sizeof(T);
        r.ldb = s.D * (int64_t)sizeof(T);
        r.M = (int)s.T;
        r.N = (int)s.V;
        r.K = (int)s.D;
        r.e.f0 = part;
        r.e.f1 = z_target;
        r.e.ld = s.T;
        r.target = target;
        r.ignore = s.ignore;
        r.vocab = s.V;
        if (s.T > 0) APEXW_TRY((run_rows<T, kEpiLse>(r, few_tiling(), stream)));
        few_join_kernel<<<at_once() ? 1 : (int)s.T, 1024, 0, stream>>>(
            (const float2 *)part, (int)s.T, (int)few_groups(), target, s.ignore, s.V, z_target,
            token_loss, lse, s.reduction, loss);
        APEXW_TRY_HIP(hipGetLastError());
        if (at_once() || s.reduction == kNone) return APEXW_OK;
        few_reduce_kernel<<<1, 64, 0, stream>>>(target, s.ignore, (int)s.T, s.reduction, token_loss, loss);
        APEXW_TRY_HIP(hipGetLastError());
        return APEXW_OK;
    }

    int forward(float *loss, float *token_loss, float *lse) {
        if (few()) return few_forward(loss, token_loss, lse);
        APEXW_TRY(rows(Factors{}));
        const int64_t c = forward_piece();
        for (int64_t c0 = 0; c0 < s.V; c0 += c) {
            const int64_t n = s.V - c0 < c ? s.V - c0 : c;
            GemmArgs a = logits(c0, n);
            const Tiling t = tiling(n);
            if (t.splits == 1) {
                a.e.f0 = part;
                a.e.f1 = z_target;
                a.e.ld = s.T;
                a.e.col0 = (int)c0;
                APEXW_TRY((run_gemm<T, false, false, kPairNone, kEpiLse>(a, t, stream)));
            } else {
                const int64_t ld = (n + 31) / 32 * 32;
                a.e.f0 = slab;
                a.e.ld = ld;
                a.e.slab = s.T * ld;
                a.e.n_store = (int)ld;
                APEXW_TRY((run_gemm<T, false, false, kPairNone, kEpiSlab>(a, t, stream)));
                reduce_slabs_kernel<<<(int)s.T, 256, 0, stream>>>(slab, s.T * ld, t.splits, ld,
                                                                  (int)c0, (int)n, count, class_of,
                                                                  (float2 *)part, z_target);
                APEXW_TRY_HIP(hipGetLastError());
            }
            join_kernel<<<(int)div_up(s.T, 16), 256, 0, stream>>>(
                (const float2 *)part, s.T, (int)groups(n), (float2 *)before, c0 == 0, c0 + n == s.V,
                count, token_of, class_of, z_target, token_loss, lse);
            APEXW_TRY_HIP(hipGetLastError());
        }
        reduce_kernel<<<1, 1024, 0, stream>>>(row_of, count, (int)s.T, s.reduction, token_loss, lse,
                                              loss);
        APEXW_TRY_HIP(hipGetLastError());
        return APEXW_OK;
    }

    Tiling dx_tiling() const { return pick_tiling<T>(s.T, s.D, piece(), false, true); }

    int64_t place_backward(Bump &b) {
        place_rows(b);
        const int64_t c = piece();
        row_lse = b.take<float>(s.T);
        factor = b.take<float>(s.T);
        common = b.take<float>(1);
        p = b.take<T>(s.T * pad8(c));
        slab = b.take<float>(dx_tiling().splits * s.T * pad8(s.D));
        const int64_t last = s.V % c == 0 ? c : s.V % c;
        const int64_t n0 = slab_elems<T>(c, s.D, s.T),
                      n1 = slab_elems<T>(last, s.D, s.T);
        const int64_t n2 = slab_elems<T>(s.T, c, s.D), n3 = slab_elems<T>(s.T, last, s.D);
        const int64_t dw = n0 > n1 ? n0 : n1, p_z = n2 > n3 ? n2 : n3;
        dw_slab = b.take<float>(dw > p_z ? dw : p_z);
        return b.used;
    }

    int backward(const float *dloss, const float *lse, T *dx, T *dw) {
        APEXW_TRY(rows(Factors{lse, dloss, s.reduction, row_lse, factor, common}));
        const int64_t c = piece(), ld = pad8(c), dx_ld = pad8(s.D);
        const Tiling dx_tiles = dx_tiling();
        for (int64_t c0 = 0; c0 < s.V; c0 += c) {
            const int64_t n = s.V - c0 < c ? s.V - c0 : c;
            if (s.T > 0) {
                GemmArgs a = logits(c0, n);
                a.e.out0 = p;
                a.e.ld = ld;
                a.e.n_store = (int)pad8(n);
                a.e.row = row_lse;
                a.e.row_scale = factor;
                a.e.col0 = (int)c0;
                APEXW_TRY((run_split<T, false, false, kPairNone, kEpiProb>(a, dw_slab, stream)));
            }
            if (dw != nullptr) {
                GemmArgs a{};
                a.a = mat(p, ld);
                a.b = mat(xc, s.Dp);
                a.M = (int)n;
                a.N = (int)s.D;
                a.K = (int)s.T;
                a.k_dev = count;
                a.e.scale = s.T > 0 ? common : nullptr;
                APEXW_TRY((run_product<T, true, true, kPairNone>(a, dw + c0 * s.D, s.D, dw_slab,
                                                                 stream)));
            }
            if (dx != nullptr && s.T > 0) {
                GemmArgs a{};
                a.a = mat(p, ld);
                a.b = mat(w + c0 * w_ld, w_ld);
                a.M = (int)s.T;
                a.N = (int)s.D;
                a.K = (int)n;
                a.m_dev = count;
                a.e.f0 = slab;
                a.e.ld = dx_ld;
                a.e.slab = s.T * dx_ld;
                a.e.n_store = (int)dx_ld;
                a.e.accumulate = c0 > 0;
                APEXW_TRY((run_gemm<T, false, true, kPairNone, kEpiSlab>(a, dx_tiles, stream)));
            }
        }
        if (dx != nullptr && s.T > 0) {
            scatter_kernel<T><<<(int)(s.T < 8192 ? s.T : 8192), 256, 0, stream>>>(
                slab, s.T * dx_ld, dx_tiles.splits, dx_ld, row_of, dx, (int)s.T, (int)s.D, common);
            APEXW_TRY_HIP(hipGetLastError());
        }
        return APEXW_OK;
    }
};

int check_shape(const apexw_linear_xent_shape *p, Shape &s) {
    if (p == nullptr) return fail(APEXW_EINVAL, "shape is NULL");
    if (p->dtype != APEXW_F32 && p->dtype != APEXW_BF16)
        return fail(APEXW_EDTYPE, "unknown element type %d", p->dtype);
    if (p->reduction != APEXW_LOSS_MEAN && p->reduction != APEXW_LOSS_SUM &&
        p->reduction != APEXW_LOSS_NONE)
        return fail(APEXW_EINVAL, "unknown reduction %d", p->reduction);
    if (p->tokens < 0 || p->tokens > kMaxDim || p->d_model < 1 || p->d_model > kMaxDim ||
        p->vocab < 1 || p->vocab > kMaxDim)
        return fail(APEXW_EINVAL, "tokens %lld, d_model %lld or vocab %lld out of range",
                    (long long)p->tokens, (long long)p->d_model, (long long)p->vocab);
    s.T = p->tokens;
    s.D = p->d_model;
    s.V = p->vocab;
    s.x_ld = p->x_stride == 0 ? s.D : p->x_stride;
    if (s.x_ld < s.D || s.x_ld > kMaxDim)
        return fail(APEXW_EINVAL, "row stride %lld: at least d_model, at most %lld",
                    (long long)p->x_stride, (long long)kMaxDim);
    s.ignore = p->ignore_index;
    s.Dp = pad8(s.D);
    s.reduction = p->reduction == APEXW_LOSS_MEAN ? kMean
                  : p->reduction == APEXW_LOSS_SUM ? kSum : kNone;
    return APEXW_OK;
}

template <class T>
int64_t work_bytes(const Shape &s, bool backward) {
    Xent<T> f{s};
    Bump b{nullptr};
    return backward ? f.place_backward(b) : f.place_forward(b);
}

template <class T>
int forward(const Shape &s, const void *x, const void *w, const int64_t *target, float *loss,
            float *token_loss, float *lse, void *ws, hipStream_t stream) {
    Xent<T> f{s, stream, (const T *)x, (const T *)w, target};
    Bump b{(char *)ws};
    f.place_forward(b);
    return f.forward(loss, token_loss, lse);
}

template <class T>
int backward(const Shape &s, const float *dloss, const void *x, const void *w,
             const int64_t *target, const float *lse, void *dx, void *dw, void *ws,
             hipStream_t stream) {
    Xent<T> f{s, stream, (const T *)x, (const T *)w, target};
    Bump b{(char *)ws};
    f.place_backward(b);
    return f.backward(dloss, lse, (T *)dx, (T *)dw);
}

}  // namespace
}  // namespace apexw

using namespace apexw;

extern "C" int apexw_linear_xent_workspace_bytes(const apexw_linear_xent_shape *shape,
                                                 int32_t backward, size_t *out_bytes) {
    Shape s;
    APEXW_TRY(check_shape(shape, s));
    if (out_bytes == nullptr) return fail(APEXW_EINVAL, "out_bytes is NULL");
    *out_bytes = (size_t)(shape->dtype == APEXW_BF16 ? work_bytes<__bf16>(s, backward)
                                                     : work_bytes<float>(s, backward));
    return APEXW_OK;
}

extern "C" int apexw_linear_xent_forward(const apexw_linear_xent_shape *shape, const void *x,
                                         const void *weight, const int64_t *target, float *loss,
                                         float *token_loss, float *lse, void *workspace,
                                         size_t workspace_len, void *stream) {
    Shape s;
    APEXW_TRY(check_shape(shape, s));
    if (s.T > 0) {
        APEXW_TRY(check_ptr(x, "x"));
        APEXW_TRY(check_ptr(weight, "weight"));
        if (target == nullptr) return fail(APEXW_EINVAL, "target is NULL");
        if (token_loss == nullptr) return fail(APEXW_EINVAL, "token_loss is NULL");
        if (lse == nullptr) return fail(APEXW_EINVAL, "lse is NULL");
    }
    if (loss == nullptr && s.reduction != kNone) return fail(APEXW_EINVAL, "loss is NULL");
    const bool bf = shape->dtype == APEXW_BF16;
    APEXW_TRY(check_room(workspace, workspace_len,
                         bf ? work_bytes<__bf16>(s, false) : work_bytes<float>(s, false),
                         "workspace"));
    return bf ? forward<__bf16>(s, x, weight, target, loss, token_loss, lse, workspace,
                                (hipStream_t)stream)
              : forward<float>(s, x, weight, target, loss, token_loss, lse, workspace,
                               (hipStream_t)stream);
}

extern "C" int apexw_linear_xent_backward(const apexw_linear_xent_shape *shape, const float *dloss,
                                          const void *x, const void *weight, const int64_t *target,
                                          const float *lse, void *dx, void *dweight,
                                          void *workspace, size_t workspace_len, void *stream) {
    Shape s;
    APEXW_TRY(check_shape(shape, s));
    if (s.T > 0) {
        APEXW_TRY(check_ptr(x, "x"));
        if (target == nullptr) return fail(APEXW_EINVAL, "target is NULL");
        if (dloss == nullptr) return fail(APEXW_EINVAL, "dloss is NULL");
        if (lse == nullptr) return fail(APEXW_EINVAL, "lse is NULL");
    }
    APEXW_TRY(check_ptr(weight, "weight"));
    if (dx != nullptr) APEXW_TRY(check_ptr(dx, "dx"));
    if (dweight != nullptr) APEXW_TRY(check_ptr(dweight, "dweight"));
    const bool bf = shape->dtype == APEXW_BF16;
    APEXW_TRY(check_room(workspace, workspace_len,
                         bf ? work_bytes<__bf16>(s, true) : work_bytes<float>(s, true),
                         "workspace"));
    return bf ? backward<__bf16>(s, dloss, x, weight, target, lse, dx, dweight, workspace,
                                 (hipStream_t)stream)
              : backward<float>(s, dloss, x, weight, target, lse, dx, dweight, workspace,
                                (hipStream_t)stream);
}
