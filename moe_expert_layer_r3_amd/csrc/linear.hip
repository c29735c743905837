// Matrix product with bias, activation and residual in its epilogue, and its
// gradients: the router's projection and a shared expert's second projection.
#include "dense_gemm.hpp"

namespace moe {
namespace {

constexpr int64_t MAX_DIM = 1 << 20, MAX_LD = 1 << 22, MAX_T = 1 << 30;

// dz is made where dy cannot be the products' operand itself
bool needs_dz(int32_t dy_type, int64_t N, int32_t act) {
    return act != MOE_ACT_NONE || dy_type == MOE_SRC_F32 || N % 8 != 0;
}

int check_sizes(int64_t T, int64_t N, int64_t K) {
    MOE_REQUIRE(T >= 0 && T <= MAX_T, MOE_ERR_SHAPE, "T=%lld outside [0, 2^30]", (long long)T);
    MOE_REQUIRE(N >= 1 && N <= MAX_DIM, MOE_ERR_SHAPE, "N=%lld outside [1, 2^20]", (long long)N);
    MOE_REQUIRE(K >= 8 && K <= MAX_DIM && K % 8 == 0, MOE_ERR_SHAPE, "K=%lld: a multiple of 8 up to 2^20", (long long)K);
    return MOE_OK;
}
bool operand_ok(const void* p, int64_t ld, int64_t cols) {
    return aligned16(p) && ld >= cols && ld <= MAX_LD && ld % 8 == 0;
}

// one launch for the gradients that are wanted
bool grouped(int64_t T, int64_t N, int64_t K, bool own, bool dx, bool dW, bool dbias) {
    DenseArgs gx = {}, gw = {};
    gx.M = gw.K = (int)T;
    gx.N = gw.N = (int)K;
    gx.K = gw.M = (int)N;
    return dense_group_pays(dx ? &gx : nullptr, dW ? &gw : nullptr, nullptr, !dbias ? 0 : own ? colsum_parts(T) : T);
}

struct BackwardWs {
    size_t dz, part, gemm, total;
};
BackwardWs backward_ws(int64_t T, int64_t N, int64_t K) {
    BackwardWs w;
    const int64_t ldz = round_up(N, 8);
    w.dz = 0;
    w.part = (size_t)round_up(T * ldz * 2, 256);
    w.gemm = w.part + (size_t)round_up((int64_t)colsum_ws(T, ldz), 256);
    size_t g = dense_ws(T, K, N, OP_KC, OP_KS, EPI_LINEAR);
    const size_t g2 = dense_ws(N, K, T, OP_KS, OP_KS, EPI_LINEAR);
    if (g2 > g) g = g2;
    w.total = w.gemm + g;
    return w;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_linear_workspace(int64_t T, int64_t N, int64_t K, size_t* bytes) {
    clear_error();
    MOE_REQUIRE(bytes, MOE_ERR_NULL, "bytes is NULL");
    if (const int rc = check_sizes(T, N, K)) return rc;
    *bytes = dense_ws(T, N, K, OP_KC, OP_KC, EPI_LINEAR);
    return MOE_OK;
}

extern "C" int moe_linear(const uint16_t* x, int64_t ldx, const uint16_t* W, int64_t ldw, const uint16_t* bias,
                          const uint16_t* residual, int64_t ldr, int64_t T, int64_t N, int64_t K, int32_t act,
                          void* out, int32_t out_type, int64_t ldo, uint16_t* pre, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
    clear_error();
    if (const int rc = check_sizes(T, N, K)) return rc;
    MOE_REQUIRE(act >= MOE_ACT_NONE && act <= MOE_ACT_SIGMOID, MOE_ERR_UNSUPPORTED, "unknown activation %d", act);
    MOE_REQUIRE(out_type == MOE_SRC_BF16 || out_type == MOE_SRC_F32, MOE_ERR_UNSUPPORTED, "unknown output type %d",
                out_type);
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(x && W && out, MOE_ERR_NULL, "x, W or out is NULL");
    MOE_REQUIRE(operand_ok(x, ldx, K), MOE_ERR_SHAPE, "x: 16-byte aligned, ldx=%lld a multiple of 8 in [K, 2^22]",
                (long long)ldx);
    MOE_REQUIRE(operand_ok(W, ldw, K), MOE_ERR_SHAPE, "W: 16-byte aligned, ldw=%lld a multiple of 8 in [K, 2^22]",
                (long long)ldw);
    MOE_REQUIRE(ldo >= N && ldo <= MAX_LD, MOE_ERR_SHAPE, "ldo=%lld outside [N, 2^22]", (long long)ldo);
    MOE_REQUIRE(!residual || (ldr >= N && ldr <= MAX_LD), MOE_ERR_SHAPE, "ldr=%lld outside [N, 2^22]", (long long)ldr);
    DenseArgs g = {};
    g.a = x;
    g.lda = ldx;
    g.b = W;
    g.ldb = ldw;
    g.M = (int)T;
    g.N = (int)N;
    g.K = (int)K;
    g.bias = bias;
    g.res = residual;
    g.ldr = ldr;
    g.out = out;
    g.ldo = ldo;
    g.pre = pre;
    g.act = act;
    g.out_f32 = out_type == MOE_SRC_F32;
    g.vec = N % 4 == 0 && ldo % 4 == 0 && aligned16(out) && aligned16(bias) && aligned16(pre) &&
            (!residual || (ldr % 4 == 0 && aligned16(residual)));
    return dense_launch(g, OP_KC, OP_KC, EPI_LINEAR, ws, ws_bytes, stream);
}

extern "C" int moe_linear_backward_workspace(int64_t T, int64_t N, int64_t K, size_t* bytes) {
    clear_error();
    MOE_REQUIRE(bytes, MOE_ERR_NULL, "bytes is NULL");
    if (const int rc = check_sizes(T, N, K)) return rc;
    *bytes = backward_ws(T, N, K).total;
    return MOE_OK;
}

extern "C" int moe_linear_backward_grouped(int64_t T, int64_t N, int64_t K, int32_t dy_type, int32_t act, int32_t dx,
                                           int32_t dW, int32_t dbias, int32_t* yes) {
    clear_error();
    MOE_REQUIRE(yes, MOE_ERR_NULL, "yes is NULL");
    if (const int rc = check_sizes(T, N, K)) return rc;
    *yes = T > 0 && grouped(T, N, K, needs_dz(dy_type, N, act), dx, dW, dbias);
    return MOE_OK;
}

extern "C" int moe_linear_backward(const void* dy, int32_t dy_type, const uint16_t* pre, const uint16_t* x, int64_t ldx,
                                   const uint16_t* W, int64_t ldw, const uint16_t* dx_add, int64_t T, int64_t N,
                                   int64_t K, int32_t act, uint16_t* dx, uint16_t* dW, uint16_t* dbias, void* ws,
                                   size_t ws_bytes, hipStream_t stream) {
    clear_error();
    if (const int rc = check_sizes(T, N, K)) return rc;
    MOE_REQUIRE(act >= MOE_ACT_NONE && act <= MOE_ACT_SIGMOID, MOE_ERR_UNSUPPORTED, "unknown activation %d", act);
    MOE_REQUIRE(dy_type == MOE_SRC_BF16 || dy_type == MOE_SRC_F32, MOE_ERR_UNSUPPORTED, "unknown gradient type %d",
                dy_type);
    MOE_REQUIRE(aligned16(dx) && aligned16(dW) && aligned16(dx_add), MOE_ERR_SHAPE,
                "dx, dW and dx_add: 16-byte aligned");
    if (T == 0) {
        int rc = MOE_OK;
        if (dW) rc = zero16_launch(dW, N * K, stream);
        if (rc == MOE_OK && dbias) rc = zero16_launch(dbias, N, stream);
        return rc;
    }
    MOE_REQUIRE(dy && (!dW || x) && (!dx || W), MOE_ERR_NULL, "dy, x or W is NULL");
    MOE_REQUIRE(act == MOE_ACT_NONE || pre, MOE_ERR_NULL, "pre is NULL with an activation");
    MOE_REQUIRE(aligned16(dy) && aligned16(pre), MOE_ERR_SHAPE, "dy and pre: 16-byte aligned");
    MOE_REQUIRE(!dW || operand_ok(x, ldx, K), MOE_ERR_SHAPE, "x: 16-byte aligned, ldx=%lld a multiple of 8 in [K, 2^22]",
                (long long)ldx);
    MOE_REQUIRE(!dx || operand_ok(W, ldw, K), MOE_ERR_SHAPE, "W: 16-byte aligned, ldw=%lld a multiple of 8 in [K, 2^22]",
                (long long)ldw);
    const BackwardWs w = backward_ws(T, N, K);
    MOE_REQUIRE((ws && aligned16(ws)) || !w.total, MOE_ERR_NULL, "ws is NULL or not 16-byte aligned");
    MOE_REQUIRE(ws_bytes >= w.total, MOE_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, w.total);
    uint8_t* wp = (uint8_t*)ws;
    void* gws = wp + w.gemm;
    const size_t gwb = ws_bytes - w.gemm;

    const bool own = needs_dz(dy_type, N, act);
    const int64_t ldz = own ? round_up(N, 8) : N;
    const uint16_t* dz = own ? (const uint16_t*)(wp + w.dz) : (const uint16_t*)dy;
    float* part = (float*)(wp + w.part);
    DenseArgs gx = {}, gw = {};
    gx.vec = gw.vec = 1;  // K % 8 == 0 and dense outputs
    gx.ldo = gw.ldo = K;
    gx.a = gw.a = dz;
    gx.lda = gw.lda = ldz;
    // [T, N] x [N, K]
    gx.b = W;
    gx.ldb = ldw;
    gx.M = (int)T;
    gx.N = gx.b_cols = (int)K;
    gx.K = (int)N;
    gx.res = dx_add;
    gx.ldr = K;
    gx.out = dx;
    // [T, N]^T x [T, K]
    gw.b = x;
    gw.ldb = ldx;
    gw.M = (int)N;
    gw.N = gw.b_cols = (int)K;
    gw.K = (int)T;
    gw.a_cols = (int)ldz;
    gw.out = dW;
    const DenseArgs *px = dx ? &gx : nullptr, *pw = dW ? &gw : nullptr;

    const bool group = grouped(T, N, K, own, dx, dW, dbias);
    if (own || (dbias && !group)) {
        const int64_t ldp = round_up(N, 8);
        if (const int rc = dz_launch(dy, dy_type == MOE_SRC_F32, act == MOE_ACT_NONE ? nullptr : pre, act, T, N, ldp,
                                     own && (dx || dW) ? (uint16_t*)(wp + w.dz) : nullptr, dbias ? part : nullptr,
                                     group ? nullptr : dbias, stream))
            return rc;
    }
    if (group) {
        const ColSum sum = own ? ColSum{part, 1, ldz, colsum_parts(T), N, dbias, 0} : ColSum{dy, 0, N, T, N, dbias, 0};
        return dense_group_launch(px, pw, nullptr, &sum, dbias ? 1 : 0, stream);
    }
    // A dx of 64 MB and more that is mostly written (a short sum) is stored past the
    // caches where dW follows, whose x then stays there.  Over seven sizes from 8192 x 4096
    // to 65536 x 1024 and 32768 x 7168, N = 64, 128, 256, both gradients take 0.86 to 1.01
    // times as long (one 1.12) and a step with its forward 0.84 to 1.00 (16384 x 7168 over
    // 256: 206 -> 202 and 279 -> 256 us); N = 512 and more, 32 MB and less: 0.97 to 1.13.
    gx.past = dW && N <= 256 && T * K >= 1 << 25;
    if (dx)
        if (const int rc = dense_launch(gx, OP_KC, OP_KS, EPI_LINEAR, gws, gwb, stream)) return rc;
    if (dW)
        if (const int rc = dense_launch(gw, OP_KS, OP_KS, EPI_LINEAR, gws, gwb, stream)) return rc;
    return MOE_OK;
}
