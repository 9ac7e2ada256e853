// ops_gated_ffn.hip -- the gated feed-forward block, forward and backward.
//
//     g = x Wg^T   u = x Wu^T   h = act(g) u   y = h Wd^T
//     dh = dy Wd   dg = dh u act'(g)   du = dh act(g)
//     dx = dg Wg + du Wu   dWg = dg^T x   dWu = du^T x   dWd = dy^T h
//
// Every product runs in gemm_kernel (ops_gemm.hpp) on the operands as they
// lie in memory.  The activation and the product of the two projections are
// the epilogue of one launch that computes both (their weights' rows alternate
// in groups of 16 in the tile, so a lane holds g and u of the same element);
// the backward's dg and du are the epilogue of dh = dy Wd.
//
// Roundings in bf16: h, dg and du are rounded once where they become an
// operand of a matrix instruction; g and u are kept for the backward pass in
// fp32, since act'(g) and the product would each take a further rounding from
// bf16 copies.  All sums are fp32.
//
// Measured on an MI355X, bf16: 8192 tokens, 4096 x 14336, forward and backward
// 6.7 ms (1285 TFLOP/s; the products' rate, 1.3 to 1.4 PFLOP/s, and 0.4 ms for the
// kept fp32 values' 2.3 GB); 512 tokens, 1024 x 2816, 75 us in six launches, bound
// by each launch's fill and drain; one token, 4096 x 14336, forward 65 us (5.4
// TB/s of weights).
#include <initializer_list>

#include "ops_rows.hpp"

namespace apexw {
namespace {

struct Shape {
    int64_t T, D, F, x_ld, dy_ld, Dp, Fp;
    int32_t act;
};

template <class T>
struct Ffn {
    Shape s;
    hipStream_t stream;
    const T *x, *wg, *wu, *wd, *dy;
    // workspace
    T *xp, *dyp, *wgp, *wup, *wdp, *h, *dg, *du;
    float *g, *u, *slab;

    // A few tokens: the products of ops_rows.hpp, which need no padded operands.
    // More than 16 with large weights: the tiles fetch those faster (23 tokens, bf16,
    // 2048 x 5504: 22 us against 30; 3584 x 1216: 26 against 18), unless they would
    // have to be copied to padded rows first (24 tokens, 3114 x 5312: 87 against 44).
    bool few() const {
        return s.T <= 16 || (s.T <= kRowsMax && (s.D * s.F * (int64_t)sizeof(T) <= (int64_t)16 << 20 ||
                                                 pad_d() || pad_f()));
    }

    bool pad_d() const { return s.D % (16 / sizeof(T)) != 0; }
    bool pad_f() const { return s.F % (16 / sizeof(T)) != 0; }
    static bool pad_ld(int64_t ld) { return ld % (16 / sizeof(T)) != 0; }

    void place_pads(Bump &b, bool backward) {
        xp = pad_d() || pad_ld(s.x_ld) ? b.take<T>(s.T * s.Dp) : nullptr;
        wgp = pad_d() ? b.take<T>(s.F * s.Dp) : nullptr;
        wup = pad_d() ? b.take<T>(s.F * s.Dp) : nullptr;
        wdp = pad_f() ? b.take<T>(s.D * s.Fp) : nullptr;
        dyp = backward && (pad_d() || pad_ld(s.dy_ld)) ? b.take<T>(s.T * s.Dp) : nullptr;
    }

    int64_t x_ld, dy_ld, wg_ld, wu_ld, wd_ld;
    int pad_all(bool backward) {
        x_ld = s.x_ld;
        dy_ld = s.dy_ld;
        wg_ld = wu_ld = s.D;
        wd_ld = s.F;
        APEXW_TRY(pad_operand(x, x_ld, xp, s.Dp, s.T, s.D, stream));
        APEXW_TRY(pad_operand(wg, wg_ld, wgp, s.Dp, s.F, s.D, stream));
        APEXW_TRY(pad_operand(wu, wu_ld, wup, s.Dp, s.F, s.D, stream));
        APEXW_TRY(pad_operand(wd, wd_ld, wdp, s.Fp, s.D, s.F, stream));
        if (backward) APEXW_TRY(pad_operand(dy, dy_ld, dyp, s.Dp, s.T, s.D, stream));
        return APEXW_OK;
    }

    // h, and g and u where they are kept
    int gate(bool keep) {
        if (few()) {
            RowsArgs r{};
            r.a = (const char *)x;
            r.b0 = (const char *)wg;
            r.b1 = (const char *)wu;
            r.lda = x_ld * (int64_t)sizeof(T);
            r.ldb = wg_ld * (int64_t)sizeof(T);
            r.M = (int)s.T;
            r.N = (int)s.F;
            r.K = (int)s.D;
            r.e.out0 = h;
            r.e.f0 = g;
            r.e.f1 = u;
            r.e.ld = s.Fp;
            r.e.n_store = (int)s.Fp;
            r.e.act = s.act;
            r.e.keep = keep;
            return run_rows<T, kEpiGate>(r, rows_tiling(2 * s.F, 2), stream);
        }
        GemmArgs a{};
        a.a = mat(x, x_ld);
        a.b = mat(wg, wg_ld, wu);
        a.M = (int)s.T;
        a.N = (int)(2 * s.F);
        a.K = (int)s.D;
        a.e.out0 = h;
        a.e.f0 = g;
        a.e.f1 = u;
        a.e.ld = s.Fp;
        a.e.n_store = (int)s.Fp;
        a.e.act = s.act;
        a.e.keep = keep;
        return run_split<T, false, false, kPairRows, kEpiGate>(a, slab, stream);
    }

    // out[M, N] = A B^T in T
    template <bool AKS, bool BKS, int PAIR>
    int product(MatArg ma, MatArg mb, int64_t M, int64_t N, int64_t K, T *out) {
        GemmArgs a{};
        a.a = ma;
        a.b = mb;
        a.M = (int)M;
        a.N = (int)N;
        a.K = (int)K;
        return run_product<T, AKS, BKS, PAIR>(a, out, N, slab, stream);
    }

    int64_t gate_slab() const {
        return few() ? 0 : slab_elems<T>(s.T, 2 * s.F, s.D);
    }
    static int64_t most(std::initializer_list<int64_t> n) {
        int64_t m = 0;
        for (int64_t x : n) m = x > m ? x : m;
        return m;
    }

    int64_t place_kept(Bump &b) {
        g = b.take<float>(s.T * s.Fp);
        u = b.take<float>(s.T * s.Fp);
        h = b.take<T>(s.T * s.Fp);
        return b.used;
    }

    int64_t place_forward(Bump &b, bool keep) {
        if (!keep) h = b.take<T>(s.T * s.Fp);
        if (few()) return b.used;
        place_pads(b, false);
        slab = b.take<float>(most({gate_slab(), slab_elems<T>(s.T, s.D, s.F)}));
        return b.used;
    }

    int forward(T *y, bool keep) {
        if (few()) {
            x_ld = s.x_ld;
            wg_ld = s.D;
            APEXW_TRY(gate(keep));
            RowsArgs r{};
            r.a = (const char *)h;
            r.b0 = (const char *)wd;
            r.lda = s.Fp * (int64_t)sizeof(T);
            r.ldb = s.F * (int64_t)sizeof(T);
            r.M = (int)s.T;
            r.N = (int)s.D;
            r.K = (int)s.F;
            r.e.out0 = y;
            r.e.ld = s.D;
            r.e.n_store = (int)s.D;
            return run_rows<T, kEpiStore>(r, rows_tiling(s.D, 1), stream);
        }
        APEXW_TRY(pad_all(false));
        APEXW_TRY(gate(keep));
        return product<false, false, kPairNone>(mat(h, s.Fp), mat(wd, wd_ld), s.T, s.D, s.F, y);
    }

    // The weights' gradients are one launch of as many products, those asked for,
    // of one k and (but for the order of their two sizes) one shape, if the sum
    // over tokens need not be split to fill the chip.
    Tiling together(int products) const {
        return pick_tiling<T>(s.F, s.D, s.T, false, true, products);
    }

    int64_t place_backward(Bump &b, bool kept) {
        place_pads(b, true);
        if (!kept) place_kept(b);
        dg = b.take<T>(s.T * s.Fp);
        du = b.take<T>(s.T * s.Fp);
        slab = b.take<float>(most({kept ? 0 : gate_slab(), slab_elems<T>(s.T, s.F, s.D),
                                   slab_elems<T>(s.T, s.D, s.F, true), slab_elems<T>(s.F, s.D, s.T),
                                   slab_elems<T>(s.D, s.F, s.T)}));
        return b.used;
    }

    int weights(T *dwg, T *dwu, T *dwd) {
        const struct { T *out; MatArg a, b; int64_t M, N; } all[3] = {
            {dwg, mat(dg, s.Fp), mat(x, x_ld), s.F, s.D},
            {dwu, mat(du, s.Fp), mat(x, x_ld), s.F, s.D},
            {dwd, mat(dy, dy_ld), mat(h, s.Fp), s.D, s.F}};
        GemmArgs a{};
        for (const auto &p : all) {
            if (p.out == nullptr) continue;
            if (a.products++ == 0) {
                a.a = p.a;
                a.b = p.b;
                a.M = (int)p.M;
                a.N = (int)p.N;
                a.e.out0 = p.out;
                a.e.ld = p.N;
                a.e.n_store = (int)p.N;
            } else {
                a.more[a.products - 2] = MoreArgs{p.a, p.b, p.out, p.N, (int)p.M, (int)p.N};
            }
        }
        if (a.products == 0) return APEXW_OK;
        a.K = (int)s.T;
        const Tiling t = together(a.products);
        if (t.splits == 1)
            return run_gemm<T, true, true, kPairNone, kEpiStore>(a, t, stream);
        for (const auto &p : all)
            if (p.out != nullptr)
                APEXW_TRY((product<true, true, kPairNone>(p.a, p.b, p.M, p.N, s.T, p.out)));
        return APEXW_OK;
    }

    int backward(bool kept, T *dx, T *dwg, T *dwu, T *dwd) {
        APEXW_TRY(pad_all(true));
        if (!kept) APEXW_TRY(gate(true));
        if (dx != nullptr || dwg != nullptr || dwu != nullptr) {
            GemmArgs a{};
            a.a = mat(dy, dy_ld);
            a.b = mat(wd, wd_ld);
            a.M = (int)s.T;
            a.N = (int)s.F;
            a.K = (int)s.D;
            a.e.out0 = dg;
            a.e.out1 = du;
            a.e.f0 = g;
            a.e.f1 = u;
            a.e.ld = s.Fp;
            a.e.n_store = (int)s.Fp;
            a.e.act = s.act;
            APEXW_TRY((run_split<T, false, true, kPairNone, kEpiGateBwd>(a, slab, stream)));
        }
        APEXW_TRY(weights(dwg, dwu, dwd));
        if (dx != nullptr)
            APEXW_TRY((product<false, true, kPairK>(mat(dg, s.Fp, du), mat(wg, wg_ld, wu), s.T, s.D,
                                                    s.F, dx)));
        return APEXW_OK;
    }
};

int check_shape(const apexw_gated_ffn_shape *p, Shape &s) {
    if (p == nullptr) return fail(APEXW_EINVAL, "shape is NULL");
    if (p->dtype != APEXW_F32 && p->dtype != APEXW_BF16)
        return fail(APEXW_EDTYPE, "unknown element type %d", p->dtype);
    if (p->activation != APEXW_ACT_SILU && p->activation != APEXW_ACT_GELU_TANH)
        return fail(APEXW_EINVAL, "unknown activation %d", p->activation);
    if (p->tokens < 0 || p->tokens > kMaxDim || p->d_model < 1 || p->d_model > kMaxDim ||
        p->d_ff < 1 || p->d_ff > kMaxDim / 2)
        return fail(APEXW_EINVAL, "tokens %lld, d_model %lld or d_ff %lld out of range",
                    (long long)p->tokens, (long long)p->d_model, (long long)p->d_ff);
    s.T = p->tokens;
    s.D = p->d_model;
    s.F = p->d_ff;
    s.x_ld = p->x_stride == 0 ? s.D : p->x_stride;
    s.dy_ld = p->dy_stride == 0 ? s.D : p->dy_stride;
    if (s.x_ld < s.D || s.x_ld > kMaxDim || s.dy_ld < s.D || s.dy_ld > kMaxDim)
        return fail(APEXW_EINVAL, "row strides %lld, %lld: at least d_model, at most %lld",
                    (long long)p->x_stride, (long long)p->dy_stride, (long long)kMaxDim);
    s.Dp = pad8(s.D);
    s.Fp = pad8(s.F);
    s.act = p->activation;
    return APEXW_OK;
}

template <class T>
int64_t kept_bytes(const Shape &s) {
    Ffn<T> f{s};
    Bump b{nullptr};
    return f.place_kept(b);
}

template <class T>
int64_t work_bytes(const Shape &s, bool backward, bool kept) {
    Ffn<T> f{s};
    Bump b{nullptr};
    return backward ? f.place_backward(b, kept) : f.place_forward(b, kept);
}

template <class T>
int forward(const Shape &s, const void *x, const void *wg, const void *wu, const void *wd, void *y,
            void *kept, void *ws, hipStream_t stream) {
    Ffn<T> f{s, stream, (const T *)x, (const T *)wg, (const T *)wu, (const T *)wd, nullptr};
    if (kept != nullptr) {
        Bump k{(char *)kept};
        f.place_kept(k);
    }
    Bump b{(char *)ws};
    f.place_forward(b, kept != nullptr);
    return f.forward((T *)y, kept != nullptr);
}

template <class T>
int backward(const Shape &s, const void *dy, const void *x, const void *wg, const void *wu,
             const void *wd, const void *kept, void *dx, void *dwg, void *dwu, void *dwd, void *ws,
             hipStream_t stream) {
    Ffn<T> f{s, stream, (const T *)x, (const T *)wg, (const T *)wu, (const T *)wd, (const T *)dy};
    if (kept != nullptr) {
        Bump k{(char *)kept};
        f.place_kept(k);
    }
    Bump b{(char *)ws};
    f.place_backward(b, kept != nullptr);
    return f.backward(kept != nullptr, (T *)dx, (T *)dwg, (T *)dwu, (T *)dwd);
}

}  // namespace
}  // namespace apexw

using namespace apexw;

extern "C" int apexw_gated_ffn_kept_bytes(const apexw_gated_ffn_shape *shape, size_t *out_bytes) {
    Shape s;
    APEXW_TRY(check_shape(shape, s));
    if (out_bytes == nullptr) return fail(APEXW_EINVAL, "out_bytes is NULL");
    *out_bytes = (size_t)(shape->dtype == APEXW_BF16 ? kept_bytes<__bf16>(s) : kept_bytes<float>(s));
    return APEXW_OK;
}

extern "C" int apexw_gated_ffn_workspace_bytes(const apexw_gated_ffn_shape *shape, int32_t backward,
                                               int32_t kept, size_t *out_bytes) {
    Shape s;
    APEXW_TRY(check_shape(shape, s));
    if (out_bytes == nullptr) return fail(APEXW_EINVAL, "out_bytes is NULL");
    *out_bytes = (size_t)(shape->dtype == APEXW_BF16 ? work_bytes<__bf16>(s, backward, kept)
                                                     : work_bytes<float>(s, backward, kept));
    return APEXW_OK;
}

extern "C" int apexw_gated_ffn_forward(const apexw_gated_ffn_shape *shape, const void *x,
                                       const void *w_gate, const void *w_up, const void *w_down,
                                       void *y, void *kept, size_t kept_len, void *workspace,
                                       size_t workspace_len, void *stream) {
    Shape s;
    APEXW_TRY(check_shape(shape, s));
    if (s.T == 0) return APEXW_OK;
    APEXW_TRY(check_ptr(x, "x"));
    APEXW_TRY(check_ptr(w_gate, "w_gate"));
    APEXW_TRY(check_ptr(w_up, "w_up"));
    APEXW_TRY(check_ptr(w_down, "w_down"));
    APEXW_TRY(check_ptr(y, "y"));
    const bool bf = shape->dtype == APEXW_BF16;
    if (kept != nullptr)
        APEXW_TRY(check_room(kept, kept_len, bf ? kept_bytes<__bf16>(s) : kept_bytes<float>(s), "kept"));
    APEXW_TRY(check_room(workspace, workspace_len,
                         bf ? work_bytes<__bf16>(s, false, kept != nullptr)
                            : work_bytes<float>(s, false, kept != nullptr),
                         "workspace"));
    return bf ? forward<__bf16>(s, x, w_gate, w_up, w_down, y, kept, workspace, (hipStream_t)stream)
              : forward<float>(s, x, w_gate, w_up, w_down, y, kept, workspace, (hipStream_t)stream);
}

extern "C" int apexw_gated_ffn_backward(const apexw_gated_ffn_shape *shape, const void *dy,
                                        const void *x, const void *w_gate, const void *w_up,
                                        const void *w_down, const void *kept, size_t kept_len,
                                        void *dx, void *dw_gate, void *dw_up, void *dw_down,
                                        void *workspace, size_t workspace_len, void *stream) {
    Shape s;
    APEXW_TRY(check_shape(shape, s));
    if (s.T > 0) {
        APEXW_TRY(check_ptr(dy, "dy"));
        APEXW_TRY(check_ptr(x, "x"));
    }
    APEXW_TRY(check_ptr(w_gate, "w_gate"));
    APEXW_TRY(check_ptr(w_up, "w_up"));
    APEXW_TRY(check_ptr(w_down, "w_down"));
    void *const outs[4] = {dx, dw_gate, dw_up, dw_down};
    for (void *o : outs)
        if (o != nullptr && !aligned16(o))
            return fail(APEXW_EINVAL, "a gradient is not 16-byte aligned");
    const bool bf = shape->dtype == APEXW_BF16;
    if (kept != nullptr)
        APEXW_TRY(check_room(kept, kept_len, bf ? kept_bytes<__bf16>(s) : kept_bytes<float>(s), "kept"));
    APEXW_TRY(check_room(workspace, workspace_len,
                         bf ? work_bytes<__bf16>(s, true, kept != nullptr)
                            : work_bytes<float>(s, true, kept != nullptr),
                         "workspace"));
    return bf ? backward<__bf16>(s, dy, x, w_gate, w_up, w_down, kept, dx, dw_gate, dw_up, dw_down,
                                 workspace, (hipStream_t)stream)
              : backward<float>(s, dy, x, w_gate, w_up, w_down, kept, dx, dw_gate, dw_up, dw_down,
                                workspace, (hipStream_t)stream);
}
