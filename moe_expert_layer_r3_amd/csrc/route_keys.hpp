// Keys in routing order (value descending, then id ascending) and the sorting
// networks over them, shared by the routing kernels.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int MAXK = 16;

// Selection key of (logit x, expert e): one 64-bit integer whose order is the
// routing order (value descending, then id ascending), so a pick is a plain
// unsigned max and every key of a row is distinct.
//   high word: the float's bits mapped monotonically to unsigned (negative
//              values bit-inverted, positive ones with the sign bit set); x is
//              canonicalised by adding +0 first, so -0 and +0 share a key and
//              fall back to the id order, as IEEE comparison has them equal;
//              NaN takes 1, below every number (NaN sorts last)
//   low word : ~e, larger for the lower id
// Key 0 means "no candidate" (a lane slot past E).  Because the picks come out
// in strictly descending key order, the values still available in a round are
// exactly those below the previous pick: no per-value taken flags.
__device__ __forceinline__ uint64_t route_key(float x, int e) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    uint32_t hi = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    if (x != x) hi = 1u;
    return ((uint64_t)hi << 32) | (uint32_t)~e;
}
__device__ __forceinline__ float route_key_value(uint64_t key) {
    const uint32_t hi = (uint32_t)(key >> 32);
    return __uint_as_float((hi & 0x80000000u) ? (hi & 0x7FFFFFFFu) : ~hi);
}
__device__ __forceinline__ int route_key_id(uint64_t key) { return (int)~(uint32_t)key; }

// A key moved across the 16-lane row by a DPP pattern (no LDS trip).
template <int CTRL>
__device__ __forceinline__ uint64_t dpp_key(uint64_t v) {
    const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, 0xF, 0xF, true);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, 0xF, 0xF, true);
    return ((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo;
}
__device__ __forceinline__ uint64_t umax64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// The same routing order as a double.  For ord = the high word of route_key
// (the float's order-preserving bits, NaN -> 1) the 64-bit pattern
// 2^62 + ord * 2^30 + (1023 - e) is a positive, normal, finite IEEE double
// (its exponent field is 0x400 + the top ten bits of ord, at most 0x7FE
// because no non-NaN float maps above 0xFF800000), and such doubles order as
// their bit patterns do: by ord, then by the lower id.  A compare-exchange is
// then one v_max_f64 and one v_min_f64, with no lane mask and no select.
// 0.0 marks "no candidate" and sits below every key.  Needs e < 1024.
__device__ __forceinline__ double route_dkey(float x, int e) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    uint32_t ord = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    ord = x != x ? 1u : ord;
    const uint32_t hi = __builtin_amdgcn_alignbit(1u, ord, 2);  // 0x40000000 | ord >> 2
    const uint32_t lo = (ord << 30) | (uint32_t)(1023 - e);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ uint32_t route_dkey_ord(double d) {
    const uint64_t b = __builtin_bit_cast(uint64_t, d);
    return ((uint32_t)(b >> 32) << 2) | ((uint32_t)b >> 30);
}
__device__ __forceinline__ int route_dkey_id(double d) {
    return 1023 - (int)((uint32_t)__builtin_bit_cast(uint64_t, d) & 0x3FFu);
}
__device__ __forceinline__ float route_ord_value(uint32_t ord) {
    return __uint_as_float((ord & 0x80000000u) ? (ord & 0x7FFFFFFFu) : ~ord);
}

__device__ __forceinline__ void dce(double& a, double& b) {
    const double x = a, y = b;
    a = __builtin_fmax(x, y);
    b = __builtin_fmin(x, y);
}

// Eight keys sorted descending: Batcher's odd-even merge sort (19 exchanges).
__device__ __forceinline__ void dsort8(double* k) {
#pragma unroll
    for (int p = 1; p < 8; p <<= 1)
#pragma unroll
        for (int q = p; q >= 1; q >>= 1)
#pragma unroll
            for (int j = q % p; j <= 7 - q; j += 2 * q)
#pragma unroll
                for (int i = 0; i <= (q - 1 < 7 - j - q ? q - 1 : 7 - j - q); ++i)
                    if ((i + j) / (2 * p) == (i + j + q) / (2 * p)) dce(k[i + j], k[i + j + q]);
}

// The eight largest of two descending runs of eight, descending: the
// elementwise max of a and b reversed holds exactly the top eight of the
// union as a bitonic sequence, which three half-cleaner stages sort.
__device__ __forceinline__ void dmerge8(double* a, const double* b) {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = __builtin_fmax(a[i], b[7 - i]);
#pragma unroll
    for (int s = 4; s >= 1; s >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((i & s) == 0) dce(a[i], a[i + s]);
}

template <int CTRL>
__device__ __forceinline__ double dpp_dkey(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, true);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(double, ((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}

}  // namespace moe
