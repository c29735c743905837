// Gated feed-forward block (a shared expert) and its gradients.
//
//   forward   h = act(x Wg^T + bg) * (x Wu^T + bu)   one product over the rows
//             [Wg; Wu], whose tiles pair the G and U columns of the same h
//             columns in one wave, so that act, the product and the save of
//             [G, U] run on the accumulators;  y = h W2^T + b2 + residual
//   backward  dh = dy W2 with [dG, dU] and h formed on its accumulators (dh is
//             never written);  dx, dW13, dW2 products;  bias column sums, db13's
//             over [dG, dU] as rounded for the products: fp32 values of them would
//             have to be written and read again, 8 T f bytes more, for a sum whose
//             terms' roundings (2^-9 of each on average) mostly cancel
#include "dense_gemm.hpp"

namespace moe {
namespace {

constexpr int64_t MAX_DIM = 1 << 20, MAX_LD = 1 << 22, MAX_T = 1 << 30;

int check_sizes(int64_t T, int64_t d, int64_t f) {
    MOE_REQUIRE(T >= 0 && T <= MAX_T, MOE_ERR_SHAPE, "T=%lld outside [0, 2^30]", (long long)T);
    MOE_REQUIRE(d >= 8 && d <= MAX_DIM && d % 8 == 0, MOE_ERR_SHAPE, "d=%lld: a multiple of 8 up to 2^20", (long long)d);
    MOE_REQUIRE(f >= 8 && 2 * f <= MAX_DIM && f % 8 == 0, MOE_ERR_SHAPE, "f=%lld: a multiple of 8 up to 2^19",
                (long long)f);
    return MOE_OK;
}
int check_kind(int32_t act, int32_t save, int64_t f) {
    MOE_REQUIRE(act >= MOE_ACT_NONE && act <= MOE_ACT_SIGMOID, MOE_ERR_UNSUPPORTED, "unknown activation %d", act);
    MOE_REQUIRE(save >= MOE_SAVE_NONE && save <= MOE_SAVE_INT8, MOE_ERR_UNSUPPORTED, "unknown save mode %d", save);
    MOE_REQUIRE(save != MOE_SAVE_INT8 || f % 128 == 0, MOE_ERR_SHAPE, "MOE_SAVE_INT8: f=%lld is no multiple of 128",
                (long long)f);
    return MOE_OK;
}

// one launch for the gradients behind [dG, dU] that are wanted
bool grouped(int64_t T, int64_t d, int64_t f, bool dx, bool dW13, bool dW2, bool dbias) {
    DenseArgs gx = {}, g13 = {}, g2 = {};
    gx.M = g13.K = g2.K = (int)T;
    gx.N = g13.N = g2.M = (int)d;
    gx.K = g13.M = (int)(2 * f);
    g2.N = (int)f;
    return dense_group_pays(dx ? &gx : nullptr, dW13 ? &g13 : nullptr, dW2 ? &g2 : nullptr, dbias ? T : 0);
}

struct BackwardWs {
    size_t dgu, h, part, gemm, total;
};
BackwardWs backward_ws(int64_t T, int64_t d, int64_t f) {
    BackwardWs w;
    w.dgu = 0;
    w.h = (size_t)round_up(T * 2 * f * 2, 256);
    w.part = w.h + (size_t)round_up(T * f * 2, 256);
    w.gemm = w.part + (size_t)round_up((int64_t)(colsum_ws(T, 2 * f) + colsum_ws(T, d)), 256);
    size_t g = 0;
    for (const size_t s : {dense_ws(T, f, d, OP_KC, OP_KS, EPI_DGATE), dense_ws(T, d, 2 * f, OP_KC, OP_KS, EPI_LINEAR),
                           dense_ws(2 * f, d, T, OP_KS, OP_KS, EPI_LINEAR), dense_ws(d, f, T, OP_KS, OP_KS, EPI_LINEAR)})
        if (s > g) g = s;
    w.total = w.gemm + g;
    return w;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_gated_ffn_workspace(int64_t T, int64_t d, int64_t f, size_t* bytes) {
    clear_error();
    MOE_REQUIRE(bytes, MOE_ERR_NULL, "bytes is NULL");
    if (const int rc = check_sizes(T, d, f)) return rc;
    *bytes = 0;
    for (const size_t s : {dense_ws(T, 2 * f, d, OP_KC, OP_KC, EPI_GATE), dense_ws(T, 2 * f, d, OP_KC, OP_KC, EPI_GATE8),
                           dense_ws(T, d, f, OP_KC, OP_KC, EPI_LINEAR)})
        if (s > *bytes) *bytes = s;
    return MOE_OK;
}

extern "C" int moe_gated_ffn(const uint16_t* x, int64_t ldx, const uint16_t* W13, const uint16_t* b13,
                             const uint16_t* W2, const uint16_t* b2, const uint16_t* residual, int64_t T, int64_t d,
                             int64_t f, int32_t act, uint16_t* h, uint16_t* y, int32_t save, void* gu, float* gu_s,
                             void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    if (const int rc = check_sizes(T, d, f)) return rc;
    if (const int rc = check_kind(act, save, f)) return rc;
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(x && W13 && h, MOE_ERR_NULL, "x, W13 or h is NULL");
    MOE_REQUIRE(!y || W2, MOE_ERR_NULL, "y without W2");
    MOE_REQUIRE(save == MOE_SAVE_NONE || gu, MOE_ERR_NULL, "gu is NULL with a save mode");
    MOE_REQUIRE(save != MOE_SAVE_INT8 || gu_s, MOE_ERR_NULL, "gu_s is NULL with MOE_SAVE_INT8");
    MOE_REQUIRE(ldx >= d && ldx <= MAX_LD && ldx % 8 == 0, MOE_ERR_SHAPE, "ldx=%lld: a multiple of 8 in [d, 2^22]",
                (long long)ldx);
    MOE_REQUIRE(aligned16(x) && aligned16(W13) && aligned16(b13) && aligned16(W2) && aligned16(b2) &&
                    aligned16(residual) && aligned16(h) && aligned16(y) && aligned16(gu),
                MOE_ERR_SHAPE, "pointers must be 16-byte aligned");
    DenseArgs g = {};
    g.a = x;
    g.lda = ldx;
    g.b = W13;
    g.ldb = d;
    g.M = (int)T;
    g.N = (int)(2 * f);
    g.K = (int)d;
    g.f = (int)f;
    g.bias = b13;
    g.act = act;
    g.h = h;
    g.save = save;
    g.gu = gu;
    g.gu_s = gu_s;
    if (const int rc = dense_launch(g, OP_KC, OP_KC, EPI_GATE, ws, ws_bytes, stream)) return rc;
    if (!y) return MOE_OK;
    g = {};
    g.a = h;
    g.lda = f;
    g.b = W2;
    g.ldb = f;
    g.M = (int)T;
    g.N = (int)d;
    g.K = (int)f;
    g.bias = b2;
    g.res = residual;
    g.ldr = d;
    g.out = y;
    g.ldo = d;
    g.vec = 1;
    return dense_launch(g, OP_KC, OP_KC, EPI_LINEAR, ws, ws_bytes, stream);
}

extern "C" int moe_gated_ffn_backward_workspace(int64_t T, int64_t d, int64_t f, size_t* bytes) {
    clear_error();
    MOE_REQUIRE(bytes, MOE_ERR_NULL, "bytes is NULL");
    if (const int rc = check_sizes(T, d, f)) return rc;
    *bytes = backward_ws(T, d, f).total;
    return MOE_OK;
}

extern "C" int moe_gated_ffn_backward_grouped(int64_t T, int64_t d, int64_t f, int32_t dx, int32_t dW13, int32_t dW2,
                                              int32_t dbias, int32_t* yes) {
    clear_error();
    MOE_REQUIRE(yes, MOE_ERR_NULL, "yes is NULL");
    if (const int rc = check_sizes(T, d, f)) return rc;
    *yes = T > 0 && grouped(T, d, f, dx, dW13, dW2, dbias);
    return MOE_OK;
}

extern "C" int moe_gated_ffn_backward(const uint16_t* dy, const uint16_t* x, int64_t ldx, const uint16_t* W13,
                                      const uint16_t* W2, int32_t save, const void* gu, const float* gu_s,
                                      const uint16_t* dx_add, int64_t T, int64_t d, int64_t f, int32_t act,
                                      uint16_t* dx, uint16_t* dW13, uint16_t* dW2, uint16_t* db13, uint16_t* db2,
                                      void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    if (const int rc = check_sizes(T, d, f)) return rc;
    if (const int rc = check_kind(act, save, f)) return rc;
    MOE_REQUIRE(save != MOE_SAVE_NONE, MOE_ERR_UNSUPPORTED, "the backward needs the saved [G, U]");
    MOE_REQUIRE(aligned16(dx) && aligned16(dW13) && aligned16(dW2) && aligned16(dx_add), MOE_ERR_SHAPE,
                "dx, dW13, dW2 and dx_add: 16-byte aligned");
    if (T == 0) {
        int rc = MOE_OK;
        if (dW13) rc = zero16_launch(dW13, 2 * f * d, stream);
        if (rc == MOE_OK && dW2) rc = zero16_launch(dW2, d * f, stream);
        if (rc == MOE_OK && db13) rc = zero16_launch(db13, 2 * f, stream);
        if (rc == MOE_OK && db2) rc = zero16_launch(db2, d, stream);
        return rc;
    }
    const bool need_dgu = dx || dW13 || db13;
    MOE_REQUIRE(dy && gu && W2, MOE_ERR_NULL, "dy, W2 or gu is NULL");
    MOE_REQUIRE((!dW13 || x) && (!dx || W13), MOE_ERR_NULL, "x or W13 is NULL");
    MOE_REQUIRE(save != MOE_SAVE_INT8 || gu_s, MOE_ERR_NULL, "gu_s is NULL with MOE_SAVE_INT8");
    MOE_REQUIRE(!dW13 || (ldx >= d && ldx <= MAX_LD && ldx % 8 == 0), MOE_ERR_SHAPE,
                "ldx=%lld: a multiple of 8 in [d, 2^22]", (long long)ldx);
    MOE_REQUIRE(aligned16(dy) && aligned16(x) && aligned16(W13) && aligned16(W2) && aligned16(gu), MOE_ERR_SHAPE,
                "pointers must be 16-byte aligned");
    const BackwardWs w = backward_ws(T, d, f);
    MOE_REQUIRE(ws && aligned16(ws), MOE_ERR_NULL, "ws is NULL or not 16-byte aligned");
    MOE_REQUIRE(ws_bytes >= w.total, MOE_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, w.total);
    uint8_t* wp = (uint8_t*)ws;
    uint16_t* dgu = (uint16_t*)(wp + w.dgu);
    uint16_t* h = (uint16_t*)(wp + w.h);
    float* part = (float*)(wp + w.part);
    void* gw = wp + w.gemm;
    const size_t gwb = ws_bytes - w.gemm;

    if (need_dgu || dW2) {
        DenseArgs g = {};
        g.a = dy;  // [T, d] x [d, f]
        g.lda = d;
        g.b = W2;
        g.ldb = f;
        g.M = (int)T;
        g.N = (int)f;
        g.K = (int)d;
        g.b_cols = (int)f;
        g.f = (int)f;
        g.act = act;
        g.save = save;
        g.gu = const_cast<void*>(gu);
        g.gu_s = const_cast<float*>(gu_s);
        g.dgu = dgu;
        g.h = dW2 ? h : nullptr;
        if (const int rc = dense_launch(g, OP_KC, OP_KS, EPI_DGATE, gw, gwb, stream)) return rc;
    }
    // dx [T, 2f] x [2f, d]
    DenseArgs gx = {}, g13 = {}, g2 = {};
    gx.vec = g13.vec = g2.vec = 1;
    gx.a = dgu;
    gx.lda = 2 * f;
    gx.b = W13;
    gx.ldb = d;
    gx.M = (int)T;
    gx.N = gx.b_cols = (int)d;
    gx.K = (int)(2 * f);
    gx.res = dx_add;
    gx.ldr = d;
    gx.out = dx;
    gx.ldo = d;
    // dW13 [T, 2f]^T x [T, d]
    g13.a = dgu;
    g13.lda = 2 * f;
    g13.b = x;
    g13.ldb = ldx;
    g13.M = g13.a_cols = (int)(2 * f);
    g13.N = g13.b_cols = (int)d;
    g13.K = (int)T;
    g13.out = dW13;
    g13.ldo = d;
    // dW2 [T, d]^T x [T, f]
    g2.a = dy;
    g2.lda = d;
    g2.b = h;
    g2.ldb = f;
    g2.M = g2.a_cols = (int)d;
    g2.N = g2.b_cols = (int)f;
    g2.K = (int)T;
    g2.out = dW2;
    g2.ldo = f;
    const DenseArgs *px = dx ? &gx : nullptr, *p13 = dW13 ? &g13 : nullptr, *p2 = dW2 ? &g2 : nullptr;
    if (grouped(T, d, f, dx, dW13, dW2, db13 || db2)) {
        ColSum sums[2];
        int n = 0;
        if (db13) sums[n++] = ColSum{dgu, 0, 2 * f, T, 2 * f, db13, 0};
        if (db2) sums[n++] = ColSum{dy, 0, d, T, d, db2, 0};
        return dense_group_launch(px, p13, p2, sums, n, stream);
    }
    if (dx)
        if (const int rc = dense_launch(gx, OP_KC, OP_KS, EPI_LINEAR, gw, gwb, stream)) return rc;
    if (dW13)
        if (const int rc = dense_launch(g13, OP_KS, OP_KS, EPI_LINEAR, gw, gwb, stream)) return rc;
    if (dW2)
        if (const int rc = dense_launch(g2, OP_KS, OP_KS, EPI_LINEAR, gw, gwb, stream)) return rc;
    return colsum_launch(dgu, 2 * f, db13, dy, d, db2, T, part, stream);
}
