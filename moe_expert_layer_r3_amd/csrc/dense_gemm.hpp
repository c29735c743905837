// bf16 matrix products on gfx950 MFMA with fused epilogues: the shared parts of
// linear.hip and gated_ffn.hip.
//
//   C[m, n] = sum_k A(m, k) B(n, k)
//
// Each operand is stored either with k contiguous ("KC": A [M, K]) or with k as
// the row index ("KS": A [K, M]), so that forward (KC, KC), data-gradient (KC,
// KS) and weight-gradient (KS, KS) products read every matrix as it lies in
// memory; no transposed copy is made.
#pragma once

#include "mfma_common.hpp"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int DBK = 64;  // K step: 128 bytes of a KC row, 64 rows of a KS matrix

// EPI_PLAIN: EPI_LINEAR's common form (bf16 out = C + bias + residual; N and the
// strides multiples of 8);
// EPI_DGATE8: EPI_DGATE from the 8-bit [G, U]; EPI_GATE8: EPI_GATE with the 8-bit
// save, which needs whole 128-column blocks (the kernels read `save`: EPI_GATE)
enum { EPI_LINEAR = 0, EPI_PART = 1, EPI_GATE = 2, EPI_DGATE = 3, EPI_PLAIN = 4, EPI_DGATE8 = 5, EPI_GATE8 = 6 };
constexpr bool is_dgate(int epi) { return epi == EPI_DGATE || epi == EPI_DGATE8; }

struct DenseArgs {
    const uint16_t* a;  // KC [M, lda] / KS [K, lda]
    const uint16_t* b;  // KC [N, ldb] / KS [K, ldb]
    int64_t lda, ldb;
    int M, N, K;     // EPI_GATE: N = 2f, the B rows are [G; U]
    int a_cols, b_cols;  // KS operands: columns that may be read (a multiple of 8, >= M / N)
    int mt, nt;      // tiles along M and N
    int ksteps;      // K steps of one split
    // EPI_LINEAR
    const uint16_t* bias;  // [N]
    const uint16_t* res;   // [M, ldr]
    int64_t ldr;
    void* out;             // [M, ldo] bf16 / fp32
    int64_t ldo;
    uint16_t* pre;         // [M, N] bf16
    int act, out_f32, vec;  // vec: N, strides and pointers allow four elements at a time
    int past;               // 256-column tiles of EPI_PLAIN store past the caches
    // EPI_PART: part[split][m][part_ld]
    float* part;
    int64_t part_ld;
    // EPI_GATE / EPI_DGATE
    int f, save;
    uint16_t* h;    // [M, f]
    void* gu;       // [M, 2f] bf16 or int8 codes
    float* gu_s;    // [2f/128, M]
    uint16_t* dgu;  // [M, 2f]
};

// ---------------------------------------------------------------- activations
// act(z) and act'(z) of four values; `act` is uniform.  sigmoid from the hardware
// exp2 and reciprocal (about 1 ulp each).
// Phi(z): the complementary function keeps its relative accuracy for z << 0, where
// 1 + erf(z / sqrt 2) would cancel.
__device__ __forceinline__ float gelu_cdf(float z) { return 0.5f * erfcf(z * -0.70710678118654752f); }
__device__ __forceinline__ float relu(float z) { return z > 0.f ? z : (z == z ? 0.f : z); }  // NaN stays NaN
__device__ __forceinline__ void act_value4(int act, const float* z, float* v) {
    switch (act) {
        case MOE_ACT_RELU:
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = relu(z[i]);
            return;
        case MOE_ACT_SILU:
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = silu(z[i]);
            return;
        case MOE_ACT_GELU:
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = z[i] * gelu_cdf(z[i]);
            return;
        case MOE_ACT_SIGMOID:
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = sigmoid_fast(z[i]);
            return;
        default:
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = z[i];
    }
}
__device__ __forceinline__ void act_both4(int act, const float* z, float* v, float* slope) {
    switch (act) {
        case MOE_ACT_RELU:
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = relu(z[i]);
                slope[i] = z[i] > 0.f ? 1.f : 0.f;
            }
            return;
        case MOE_ACT_SILU:
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float s = sigmoid_fast(z[i]);
                v[i] = z[i] * s;
                slope[i] = s + v[i] * (1.f - s);
            }
            return;
        case MOE_ACT_GELU:
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float c = gelu_cdf(z[i]);
                v[i] = z[i] * c;
                slope[i] = c + z[i] * __builtin_amdgcn_exp2f(-0.72134752044448170f * z[i] * z[i]) * 0.39894228040143268f;
            }
            return;
        case MOE_ACT_SIGMOID:
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // s(z) s(-z) from e = exp(-|z|), without 1 - s, which cancels for z >> 0
                const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * __builtin_fabsf(z[i]));
                const float r = __builtin_amdgcn_rcpf(1.f + e);
                v[i] = z[i] < 0.f ? e * r : r;
                slope[i] = e * r * r;
            }
            return;
        default:
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = z[i];
                slope[i] = 1.f;
            }
    }
}

// ---------------------------------------------------------------- 8-bit blocks
// Scale of an 8-bit block from the largest |v| as a bit pattern (taken with an
// unsigned maximum, so a NaN wins over every number): s = a / 127 and the
// factor 127 / a, both correctly rounded.
struct Keep8 {
    float s, inv;
};
__device__ __forceinline__ Keep8 keep8_scale(uint32_t amax_bits) {
    const float lo = 7.888609052210118e-31f;  // 2^-100
    float a = __uint_as_float(amax_bits);
    if (a < lo) a = lo;  // false for NaN
    return Keep8{a / 127.f, 127.f / a};
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
// |v * inv| <= 127 (1 + 2^-23), which rounds to at most 127; NaN converts to 0
// and is restored as NaN through the scale
__device__ __forceinline__ int keep8_code(float v, float inv) { return (int)__builtin_rintf(v * inv); }
__device__ __forceinline__ uint32_t pack_s8x4(int a, int b, int c, int d) {
    return (uint32_t)(a & 0xFF) | ((uint32_t)(b & 0xFF) << 8) | ((uint32_t)(c & 0xFF) << 16) | ((uint32_t)d << 24);
}
__device__ __forceinline__ float s8_of(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

// ---------------------------------------------------------------- operand moves
// 16 bytes per lane, global -> LDS (lane l to LDS m0 + 16 l), through a buffer
// descriptor: a lane whose offset is OOB reads nothing and writes zeros, which
// is how row, column and K tails are filled.
constexpr uint32_t OOB = 0x80000000u;
__device__ __forceinline__ u32x4 buf_desc(const void* base) {
    const uint64_t p = (uint64_t)(uintptr_t)base;
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(p >> 32) & 0xFFFFu)), 0x7FFFFFF0u,
                 0x00020000u};
}
// Two 1 KB segments to adjacent LDS (lds, lds + 1024).  The waits that the
// compiler cannot insert around inline assembly are part of it: five states
// between a vector instruction's write of a descriptor SGPR (v_readfirstlane) and
// the load that reads it, one between a write of M0 and the load.
__device__ __forceinline__ void dma16b2(const u32x4& desc, uint32_t voff0, uint32_t voff1, uint32_t lds) {
    asm volatile(
        "s_nop 4\n\t"
        "buffer_load_dwordx4 %1, %3, 0 offen lds\n\t"
        "s_add_u32 m0, m0, 0x400\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %2, %3, 0 offen lds"
        : "+{m0}"(lds)
        : "v"(voff0), "v"(voff1), "s"(desc)
        : "memory", "scc");
}

// Transposing LDS read: the 16 lanes of a group supply 4 K rows x 16 columns
// (lane i: row i / 4, columns 4 (i % 4) .. + 3) and lane i receives column i's
// four K values.
template <int OFF>
__device__ __forceinline__ v2u lds_tr16(uint32_t addr) {
    typedef __attribute__((address_space(3))) s16x4* ptr;
    return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(uintptr_t)(addr + OFF)));
}

__device__ __forceinline__ v4f mfma_bf16(const u32x4& a, const u32x4& b, const v4f& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// LDS images of one operand's K step, R rows (KC) or columns (KS):
//   KC: row r at 128 r; its eight 16-byte chunks c at c ^ (r & 7).
//   KS: per 128 columns a 16 KB image, K row k at 256 k; its sixteen chunks c
//       at c ^ 2 f(k), f(k) = (k & 3) | (k >> 3 & 1) << 2: the eight K rows a
//       half-wave reads of one 16-column fragment fall on distinct banks.
// One 1 KB segment (one DMA instruction) is 8 KC rows or 4 K rows.
struct KcLane {
    uint32_t off;  // this lane's byte offset in a segment
    uint32_t row, k;  // its row in a segment, its first K value
    __device__ __forceinline__ KcLane(int lane, int64_t ld) {
        row = (uint32_t)lane >> 3;
        const uint32_t c = ((uint32_t)lane & 7) ^ row;
        k = c * 8;
        off = row * (uint32_t)(ld * 2) + c * 16;
    }
};
__device__ __forceinline__ uint32_t ks_f(uint32_t k) { return (k & 3) | ((k >> 3 & 1) << 2); }

// KC fragment of 16 rows from row r0 (a multiple of 16), K values 32 s + 8 g ..
// + 7 (g = lane / 16): the byte offset of this lane for s = 0; s = 1 is it ^ 64.
__device__ __forceinline__ uint32_t kc_frag(int lane, int r0) {
    const uint32_t r = (uint32_t)(r0 + (lane & 15));
    return r * 128 + ((((uint32_t)lane >> 4) ^ (r & 7)) << 4);
}
// KS fragment of 16 columns (16-column group c16 of the image): this lane's byte
// offset for K values 8 g .. + 3; + 1024 the next four, + 8192 per s.
__device__ __forceinline__ uint32_t ks_frag(int lane, int c16) {
    const uint32_t l15 = (uint32_t)lane & 15;
    const uint32_t k = ((uint32_t)lane >> 4) * 8 + (l15 >> 2);
    return k * 256 + (((uint32_t)c16 ^ ks_f(k)) << 5) + (l15 & 3) * 8;
}

// The same in images of 64 columns: K row k at 128 k, its eight chunks c at
// c ^ 2 f64(k); + 512 the next four K values, + 4096 per s.
__device__ __forceinline__ uint32_t ks_f64(uint32_t k) { return (k >> 1 & 1) | ((k >> 3 & 1) << 1); }
__device__ __forceinline__ uint32_t ks_frag64(int lane, int c16) {
    const uint32_t l15 = (uint32_t)lane & 15;
    const uint32_t k = ((uint32_t)lane >> 4) * 8 + (l15 >> 2);
    return k * 128 + (((uint32_t)c16 ^ ks_f64(k)) << 5) + (l15 & 3) * 8;
}

// ---------------------------------------------------------------- epilogues
__device__ __forceinline__ void load_bf16x4(const uint16_t* p, float* v) {
    const v2u w = *reinterpret_cast<const v2u*>(p);
    v[0] = bf16_lo(w.x);
    v[1] = bf16_hi(w.x);
    v[2] = bf16_lo(w.y);
    v[3] = bf16_hi(w.y);
}
__device__ __forceinline__ v2u pack_bf16x4(float a, float b, float c, float d) {
    return v2u{cvt_bf16x2(a, b), cvt_bf16x2(c, d)};
}

// What the epilogue of C[m, n .. n + 3] reads from memory, loaded ahead of its use.
// Loads are not predicated (places past the matrix read its last row or first
// columns instead), so that a batch of them is in flight at a time.
template <int EPI>
struct EpiIn {
    v2u a = {0u, 0u}, b = {0u, 0u};  // residual; saved G, U
    float sa = 0.f, sb = 0.f;        // their 8-bit scales
    __device__ __forceinline__ void load(const DenseArgs& g, int64_t m, int n) {
        if (m >= g.M) m = g.M - 1;
        if constexpr (is_dgate(EPI)) {
            if (n >= g.f) n = 0;
            const int64_t row = m * (2 * (int64_t)g.f);
            if constexpr (EPI == EPI_DGATE8) {
                const int64_t blk = n >> 7, nb = g.f >> 7;
                sa = g.gu_s[blk * g.M + m];
                sb = g.gu_s[(nb + blk) * g.M + m];
                a.x = *reinterpret_cast<const uint32_t*>((const int8_t*)g.gu + row + n);
                b.x = *reinterpret_cast<const uint32_t*>((const int8_t*)g.gu + row + g.f + n);
            } else {
                a = *reinterpret_cast<const v2u*>((const uint16_t*)g.gu + row + n);
                b = *reinterpret_cast<const v2u*>((const uint16_t*)g.gu + row + g.f + n);
            }
        } else if constexpr (EPI == EPI_PLAIN || EPI == EPI_LINEAR) {
            if (!g.res) return;
            const uint16_t* p = g.res + m * g.ldr;
            if (EPI == EPI_PLAIN || g.vec) {
                a = *reinterpret_cast<const v2u*>(p + (n < g.N ? n : 0));
            } else {
                const int last = g.N - 1;
                a.x = p[min(n, last)] | (uint32_t)p[min(n + 1, last)] << 16;
                a.y = p[min(n + 2, last)] | (uint32_t)p[min(n + 3, last)] << 16;
            }
        }
    }
};
// The biases of columns n .. n + 3 (a thread's columns are the same for all its rows)
template <int EPI>
struct EpiBias {
    v4f a = {0.f, 0.f, 0.f, 0.f}, b = {0.f, 0.f, 0.f, 0.f};  // EPI_GATE: of G and U
    __device__ __forceinline__ void load(const DenseArgs& g, int n) {
        if constexpr (EPI == EPI_LINEAR || EPI == EPI_PLAIN || EPI == EPI_GATE) {
            if (!g.bias) return;
            float t[4];
            if constexpr (EPI == EPI_GATE) {
                if (n >= g.f) return;
                load_bf16x4(g.bias + n, t);
                a = v4f{t[0], t[1], t[2], t[3]};
                load_bf16x4(g.bias + g.f + n, t);
                b = v4f{t[0], t[1], t[2], t[3]};
            } else if (EPI == EPI_PLAIN || g.vec) {
                if (n >= g.N) return;
                load_bf16x4(g.bias + n, t);
                a = v4f{t[0], t[1], t[2], t[3]};
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = bf16_to_f32(g.bias[min(n + i, g.N - 1)]);
            }
        }
    }
};
__device__ __forceinline__ void unpack_bf16x4(v2u w, float* v) {
    v[0] = bf16_lo(w.x);
    v[1] = bf16_hi(w.x);
    v[2] = bf16_lo(w.y);
    v[3] = bf16_hi(w.y);
}

// EPI_LINEAR for C[m, n .. n + 3], m < M, n < N
__device__ __forceinline__ void epi_linear(const DenseArgs& g, int64_t m, int n, v4f c, const EpiIn<EPI_LINEAR>& in,
                                           const EpiBias<EPI_LINEAR>& bias) {
    const int left = g.N - n;
    c += bias.a;
    float v[4] = {c.x, c.y, c.z, c.w}, t[4];
    if (g.pre) {
        uint16_t* p = g.pre + m * g.N + n;
        const v2u w = pack_bf16x4(v[0], v[1], v[2], v[3]);
        if (g.vec) {
            *reinterpret_cast<v2u*>(p) = w;
        } else {
            p[0] = (uint16_t)w.x;
            if (left > 1) p[1] = (uint16_t)(w.x >> 16);
            if (left > 2) p[2] = (uint16_t)w.y;
            if (left > 3) p[3] = (uint16_t)(w.y >> 16);
        }
    }
    act_value4(g.act, v, v);
    if (g.res) {
        unpack_bf16x4(in.a, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += t[i];
    }
    if (g.out_f32) {
        float* p = (float*)g.out + m * g.ldo + n;
        if (g.vec) {
            *reinterpret_cast<v4f*>(p) = v4f{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < left) p[i] = v[i];
        }
    } else {
        uint16_t* p = (uint16_t*)g.out + m * g.ldo + n;
        const v2u w = pack_bf16x4(v[0], v[1], v[2], v[3]);
        if (g.vec) {
            *reinterpret_cast<v2u*>(p) = w;
        } else {
            p[0] = (uint16_t)w.x;
            if (left > 1) p[1] = (uint16_t)(w.x >> 16);
            if (left > 2) p[2] = (uint16_t)w.y;
            if (left > 3) p[3] = (uint16_t)(w.y >> 16);
        }
    }
}

// EPI_PLAIN for C[m, n .. n + 3], m < M, n < N
__device__ __forceinline__ void epi_plain(const DenseArgs& g, int64_t m, int n, v4f c, const EpiIn<EPI_PLAIN>& in,
                                          const EpiBias<EPI_PLAIN>& bias) {
    float t[4];
    c += bias.a;
    if (g.res) {
        unpack_bf16x4(in.a, t);
        c += v4f{t[0], t[1], t[2], t[3]};
    }
    uint16_t* p = (uint16_t*)g.out + m * g.ldo;
    *reinterpret_cast<v2u*>(p + n) = pack_bf16x4(c.x, c.y, c.z, c.w);
}

// EPI_DGATE for dh[m, n .. n + 3], m < M, n < f (f % 8 == 0): [dG, dU] and h from
// the saved G, U, rounded to bf16 as operands of the products behind (a second bf16
// term of the rest would double those)
template <int EPI>
__device__ __forceinline__ void epi_dgate(const DenseArgs& g, int64_t m, int n, v4f dh, const EpiIn<EPI>& in) {
    float G[4], U[4];
    if constexpr (EPI == EPI_DGATE8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            G[i] = s8_of(in.a.x, i) * in.sa;
            U[i] = s8_of(in.b.x, i) * in.sb;
        }
    } else {
        unpack_bf16x4(in.a, G);
        unpack_bf16x4(in.b, U);
    }
    float dG[4], dU[4], h[4], v[4], sl[4];
    act_both4(g.act, G, v, sl);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        dG[i] = dh[i] * U[i] * sl[i];
        dU[i] = dh[i] * v[i];
        h[i] = v[i] * U[i];
    }
    uint16_t* p = g.dgu + m * (2 * (int64_t)g.f);
    *reinterpret_cast<v2u*>(p + n) = pack_bf16x4(dG[0], dG[1], dG[2], dG[3]);
    *reinterpret_cast<v2u*>(p + g.f + n) = pack_bf16x4(dU[0], dU[1], dU[2], dU[3]);
    if (g.h) *reinterpret_cast<v2u*>(g.h + m * (int64_t)g.f + n) = pack_bf16x4(h[0], h[1], h[2], h[3]);
}

// EPI_GATE for the sums G, U[m, n .. n + 3]; `on`: m < M and n < f.  With the 8-bit
// save (f % 128 == 0) 32 adjacent lanes hold one 128-column block of a row, and
// every lane of a wave calls.  h is rounded to bf16, the operand of y's product.
__device__ __forceinline__ void epi_gate(const DenseArgs& g, int64_t m, int n, v4f G, v4f U,
                                         const EpiBias<EPI_GATE>& bias, bool on) {
    G += bias.a;
    U += bias.b;
    if (g.save == MOE_SAVE_INT8) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const v4f v = w ? U : G;
            uint32_t mx = umax(umax(abs_bits(v.x), abs_bits(v.y)), umax(abs_bits(v.z), abs_bits(v.w)));
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) mx = umax(mx, (uint32_t)__shfl_xor((int)mx, o));
            const Keep8 k = keep8_scale(mx);
            if (on) {
                if ((threadIdx.x & 31) == 0) g.gu_s[((int64_t)(w * (g.f >> 7)) + (n >> 7)) * g.M + m] = k.s;
                *reinterpret_cast<uint32_t*>((int8_t*)g.gu + m * (2 * (int64_t)g.f) + (int64_t)w * g.f + n) =
                    pack_s8x4(keep8_code(v.x, k.inv), keep8_code(v.y, k.inv), keep8_code(v.z, k.inv),
                              keep8_code(v.w, k.inv));
            }
        }
    }
    if (!on) return;
    const float z[4] = {G.x, G.y, G.z, G.w};
    float h[4];
    act_value4(g.act, z, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] *= U[i];
    *reinterpret_cast<v2u*>(g.h + m * g.f + n) = pack_bf16x4(h[0], h[1], h[2], h[3]);
    if (g.save == MOE_SAVE_BF16) {
        uint16_t* p = (uint16_t*)g.gu + m * (2 * (int64_t)g.f) + n;
        *reinterpret_cast<v2u*>(p) = pack_bf16x4(G[0], G[1], G[2], G[3]);
        *reinterpret_cast<v2u*>(p + g.f) = pack_bf16x4(U[0], U[1], U[2], U[3]);
    }
}

// EPI_GATE without the 8-bit save for G, U[m, n] and [m, n + 1] (m < M, n < f)
__device__ __forceinline__ void epi_gate2(const DenseArgs& g, int64_t m, int n, v4f G, v4f U) {
    if (g.bias) {
        G.x += bf16_to_f32(g.bias[n]);
        G.y += bf16_to_f32(g.bias[n + 1]);
        U.x += bf16_to_f32(g.bias[g.f + n]);
        U.y += bf16_to_f32(g.bias[g.f + n + 1]);
    }
    const float z[4] = {G.x, G.y, 0.f, 0.f};
    float h[4];
    act_value4(g.act, z, h);
    *reinterpret_cast<uint32_t*>(g.h + m * g.f + n) = cvt_bf16x2(h[0] * U.x, h[1] * U.y);
    if (g.save == MOE_SAVE_BF16) {
        uint16_t* p = (uint16_t*)g.gu + m * (2 * (int64_t)g.f) + n;
        *reinterpret_cast<uint32_t*>(p) = cvt_bf16x2(G.x, G.y);
        *reinterpret_cast<uint32_t*>(p + g.f) = cvt_bf16x2(U.x, U.y);
    }
}

// ---------------------------------------------------------------- host side
// A product: fills in tiles, splits and workspace use and launches it (and, for
// a split K, the sum of the pieces with the epilogue).
enum { OP_KC = 0, OP_KS = 1 };
int dense_launch(DenseArgs g, int la, int lb, int epi, void* ws, size_t ws_bytes, hipStream_t stream);
// dense_thin.hip: products of few rows with both operands K-contiguous
int dense_thin_launch(const DenseArgs& g, int epi, hipStream_t stream);
constexpr int THIN_ROWS = 4, SLAB_ROWS = 128;
int dense_slab_launch(const DenseArgs& g, int splits, hipStream_t stream);
// fp32 workspace of a product with M x N results and K summands
size_t dense_ws(int64_t M, int64_t N, int64_t K, int la, int lb, int epi);

// column sums of a [T, Na] and b [T, Nb] (bf16, dense, Na, Nb % 4 == 0) as bf16,
// each skipped if its output is NULL; part: fp32 workspace of colsum_ws bytes for
// each of the two
size_t colsum_ws(int64_t T, int64_t N);
int colsum_launch(const uint16_t* a, int64_t Na, uint16_t* out_a, const uint16_t* b, int64_t Nb, uint16_t* out_b,
                  int64_t T, float* part, hipStream_t stream);
// A small problem's gradients in one launch: a data gradient (KC, KS), weight
// gradients (KS, KS), each NULL if not wanted, and column sums
struct ColSum {
    const void* src;  // [rows, ld], bf16 or fp32
    int f32;
    int64_t ld, rows, N;
    uint16_t* out;  // [N]
    int blocks;     // of 32 columns (filled in by the launch)
};
struct DenseGroup {
    DenseArgs dx, dw[2];
    ColSum sums[2];
    int tiles[3];
};
// (looks at M, N, K only; sum_rows: rows of the column sums, 0 without them)
bool dense_group_pays(const DenseArgs* dx, const DenseArgs* dw0, const DenseArgs* dw1, int64_t sum_rows);
int dense_group_launch(const DenseArgs* dx, const DenseArgs* dw0, const DenseArgs* dw1, const ColSum* sums, int nsums,
                       hipStream_t stream);

// dz = dy * act'(pre) [T, ldz] bf16 (dz may be NULL) and its column sums: part
// [colsum_parts(T), ldz] fp32 those of chunks of rows (may be NULL), dbias their
// sums (may be NULL); dy [T, N] dense, ldz = N rounded up to 8
int colsum_parts(int64_t T);
int dz_launch(const void* dy, int dy_f32, const uint16_t* pre, int act, int64_t T, int64_t N, int64_t ldz, uint16_t* dz,
              float* part, uint16_t* dbias, hipStream_t stream);

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
// fill of n bf16 (or other 2-byte) zeros by a kernel (memset nodes stay out of graphs)
int zero16_launch(uint16_t* p, int64_t n, hipStream_t stream);

}  // namespace moe
