// Activations kept in 8 bits between the forward and the backward pass: rows in
// blocks of 128 columns, one fp32 scale each.  Both directions are bound by the
// bytes they move (3 per value and 1/32 more for the scales): 16384 x 7168 is saved
// in 66.8 us (5.3 TB/s) and restored in 62.2 us (5.7 TB/s).
#include "dense_gemm.hpp"

namespace moe {

constexpr int64_t MAX_X = 1 << 20;  // blocks in x: a launch's x takes less than 2^32 threads
__device__ __forceinline__ int64_t wave_unit() {
    return ((int64_t)blockIdx.y * MAX_X + blockIdx.x) * 4 + (threadIdx.x >> 6);
}

// A wave takes four rows of four blocks (512 columns): 16 lanes to a block, 8
// columns each, all four rows' loads in flight, 1 KB of a row per load; a block's four
// scales are neighbours in memory.
__global__ __launch_bounds__(256) void act_save_kernel(const uint16_t* src, int64_t ld, int64_t rows, int64_t cols,
                                                       int64_t units, int8_t* q, float* s) {
    const int lane = threadIdx.x & 63;
    const int64_t unit = wave_unit();  // (row quad, 512 columns), columns fastest
    const int64_t quad = unit / units, blk = (unit - quad * units) * 4 + (lane >> 4);
    const int64_t r0 = quad * 4, c = blk * 128 + (lane & 15) * 8;
    if (r0 >= rows) return;  // the whole wave
    const bool on = c < cols;
    u32x4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = u32x4{0u, 0u, 0u, 0u};
        if (on) w[i] = *reinterpret_cast<const u32x4*>(src + min(r0 + i, rows - 1) * ld + c);
    }
    float sc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16_lo(w[i][j]);
            v[2 * j + 1] = bf16_hi(w[i][j]);
        }
        uint32_t mx = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = umax(mx, abs_bits(v[j]));
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) mx = umax(mx, (uint32_t)__shfl_xor((int)mx, o));
        const Keep8 k = keep8_scale(mx);
        sc[i] = k.s;
        if (!on || r0 + i >= rows) continue;
        int t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = keep8_code(v[j], k.inv);
        *reinterpret_cast<v2u*>(q + (r0 + i) * cols + c) =
            v2u{pack_s8x4(t[0], t[1], t[2], t[3]), pack_s8x4(t[4], t[5], t[6], t[7])};
    }
    if ((lane & 15) != 0 || !on) return;
    float* p = s + blk * rows + r0;
    if ((rows & 3) == 0) {
        *reinterpret_cast<v4f*>(p) = v4f{sc[0], sc[1], sc[2], sc[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r0 + i < rows) p[i] = sc[i];
    }
}

__global__ __launch_bounds__(256) void act_restore_kernel(const int8_t* q, const float* s, int64_t rows, int64_t cols,
                                                          int64_t units, uint16_t* dst) {
    const int lane = threadIdx.x & 63;
    const int64_t unit = wave_unit();
    const int64_t quad = unit / units, blk = (unit - quad * units) * 4 + (lane >> 4);
    const int64_t r0 = quad * 4, c = blk * 128 + (lane & 15) * 8;
    if (r0 >= rows || c >= cols) return;
    v2u w[4];
    float sc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = min(r0 + i, rows - 1);
        w[i] = *reinterpret_cast<const v2u*>(q + r * cols + c);
        sc[i] = s[blk * rows + r];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (r0 + i >= rows) return;
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t x = j < 2 ? w[i].x : w[i].y;
            o[j] = cvt_bf16x2(s8_of(x, (2 * j) & 3) * sc[i], s8_of(x, (2 * j + 1) & 3) * sc[i]);
        }
        *reinterpret_cast<u32x4*>(dst + (r0 + i) * cols + c) = o;
    }
}

namespace {
int check(int64_t rows, int64_t cols) {
    MOE_REQUIRE(rows >= 0 && rows <= (1 << 30), MOE_ERR_SHAPE, "rows=%lld outside [0, 2^30]", (long long)rows);
    MOE_REQUIRE(cols >= 8 && cols <= (1 << 20) && cols % 8 == 0, MOE_ERR_SHAPE, "cols=%lld: a multiple of 8 up to 2^20",
                (long long)cols);
    MOE_REQUIRE((rows + 3) / 4 * ((cols + 511) / 512) < (1ll << 36), MOE_ERR_SHAPE, "rows x cols too large");
    return MOE_OK;
}
dim3 grid(int64_t waves) {
    const int64_t b = (waves + 3) / 4;
    return dim3((unsigned)(b < MAX_X ? b : MAX_X), (unsigned)((b + MAX_X - 1) / MAX_X));
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
    MOE_REQUIRE(aligned16(src) && aligned16(q) && aligned16(s), MOE_ERR_SHAPE, "src, q and s: 16-byte aligned");
    const int64_t units = (cols + 511) / 512, waves = (rows + 3) / 4 * units;
    act_save_kernel<<<grid(waves), dim3(256), 0, stream>>>(src, ld, rows, cols, units, q, s);
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
    const int64_t units = (cols + 511) / 512, waves = (rows + 3) / 4 * units;
    act_restore_kernel<<<grid(waves), dim3(256), 0, stream>>>(q, s, rows, cols, units, dst);
    MOE_LAUNCH_CHECK("act_restore_kernel");
    return MOE_OK;
}
