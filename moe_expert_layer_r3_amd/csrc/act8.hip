// Activations kept in 8 bits between the forward and the backward pass: rows in
// blocks of 128 columns, one fp32 scale each.  Both directions are bound by the
// bytes they move (3 per value and 1/32 more for the scales).
#include "dense_gemm.hpp"

namespace moe {

// 16 lanes take a block of a row, 8 columns each; a wave takes the same block of
// four consecutive rows, so its four scales are neighbours in memory.
__global__ __launch_bounds__(256) void act_save_kernel(const uint16_t* src, int64_t ld, int64_t rows, int64_t cols,
                                                       int64_t nb, int8_t* q, float* s) {
    const int lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);  // (row quad, block), block fastest
    const int64_t quad = unit / nb, blk = unit - quad * nb;
    const int64_t r = quad * 4 + (lane >> 4), c = blk * 128 + (lane & 15) * 8;
    const bool on = r < rows && c < cols;
    u32x4 w = {0u, 0u, 0u, 0u};
    if (on) w = *reinterpret_cast<const u32x4*>(src + r * ld + c);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = umax(mx, abs_bits(v[i]));
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) mx = umax(mx, (uint32_t)__shfl_xor((int)mx, o));
    if (r >= rows) return;
    const Keep8 k = keep8_scale(mx);
    if ((lane & 15) == 0) s[blk * rows + r] = k.s;
    if (!on) return;
    int t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = keep8_code(v[i], k.inv);
    *reinterpret_cast<v2u*>(q + r * cols + c) =
        v2u{pack_s8x4(t[0], t[1], t[2], t[3]), pack_s8x4(t[4], t[5], t[6], t[7])};
}

__global__ __launch_bounds__(256) void act_restore_kernel(const int8_t* q, const float* s, int64_t rows, int64_t cols,
                                                          int64_t nb, uint16_t* dst) {
    const int lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t quad = unit / nb, blk = unit - quad * nb;
    const int64_t r = quad * 4 + (lane >> 4), c = blk * 128 + (lane & 15) * 8;
    if (r >= rows || c >= cols) return;
    const float sc = s[blk * rows + r];
    const v2u w = *reinterpret_cast<const v2u*>(q + r * cols + c);
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = i < 2 ? w.x : w.y;
        o[i] = cvt_bf16x2(s8_of(x, (2 * i) & 3) * sc, s8_of(x, (2 * i + 1) & 3) * sc);
    }
    *reinterpret_cast<u32x4*>(dst + r * cols + c) = o;
}

namespace {
int check(int64_t rows, int64_t cols) {
    MOE_REQUIRE(rows >= 0 && rows <= (1 << 30), MOE_ERR_SHAPE, "rows=%lld outside [0, 2^30]", (long long)rows);
    MOE_REQUIRE(cols >= 8 && cols <= (1 << 20) && cols % 8 == 0, MOE_ERR_SHAPE, "cols=%lld: a multiple of 8 up to 2^20",
                (long long)cols);
    MOE_REQUIRE((rows + 3) / 4 * ((cols + 127) / 128) < (1ll << 31), MOE_ERR_SHAPE, "rows x cols too large");
    return MOE_OK;
}
}  // namespace

}  // namespace moe

using namespace moe;

extern "C" int moe_act_save(const uint16_t* src, int64_t ld, int64_t rows, int64_t cols, int8_t* q, float* s,
                            hipStream_t stream) {
    clear_error();
    if (const int rc = check(rows, cols)) return rc;
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(src && q && s, MOE_ERR_NULL, "src, q or s is NULL");
    MOE_REQUIRE(ld >= cols && ld <= (1 << 22) && ld % 8 == 0, MOE_ERR_SHAPE, "ld=%lld: a multiple of 8 in [cols, 2^22]",
                (long long)ld);
    MOE_REQUIRE(aligned16(src) && aligned16(q), MOE_ERR_SHAPE, "src and q: 16-byte aligned");
    const int64_t nb = (cols + 127) / 128, units = (rows + 3) / 4 * nb;
    act_save_kernel<<<dim3((unsigned)((units + 3) / 4)), dim3(256), 0, stream>>>(src, ld, rows, cols, nb, q, s);
    MOE_LAUNCH_CHECK("act_save_kernel");
    return MOE_OK;
}

extern "C" int moe_act_restore(const int8_t* q, const float* s, int64_t rows, int64_t cols, uint16_t* dst,
                               hipStream_t stream) {
    clear_error();
    if (const int rc = check(rows, cols)) return rc;
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(q && s && dst, MOE_ERR_NULL, "q, s or dst is NULL");
    MOE_REQUIRE(aligned16(dst) && aligned16(q), MOE_ERR_SHAPE, "q and dst: 16-byte aligned");
    const int64_t nb = (cols + 127) / 128, units = (rows + 3) / 4 * nb;
    act_restore_kernel<<<dim3((unsigned)((units + 3) / 4)), dim3(256), 0, stream>>>(q, s, rows, cols, nb, dst);
    MOE_LAUNCH_CHECK("act_restore_kernel");
    return MOE_OK;
}
