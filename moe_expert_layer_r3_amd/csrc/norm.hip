// The norms around the layer: in front of it (moe_norm), and behind it together
// with the gate, the scaled residual sum and the next layer's norm (moe_join), and
// their gradients.
#include <type_traits>

#include "common.hpp"

namespace moe {
namespace {

constexpr int NT = 256;  // threads of a workgroup

struct JoinArgs {
    const uint16_t* y;  // NULL: a norm of r alone
    int64_t ldy;
    const void* r;
    int64_t ldr;
    const void *w_post, *gate, *w_pre;
    int gate_kind, gate_act;
    bool w_f32, gate_f32;
    float r_scale, y_scale, eps;
    int64_t T, d;
    void* r_out;
    uint16_t* h;
    float *rstd_post, *rstd_pre;
    float part, parts;  // set by the launch: see square_of
};

struct JoinGradArgs {
    const void* d_out;
    const uint16_t* dh;
    const uint16_t* y;
    int64_t ldy;
    const void* r_out;
    int64_t ldr;  // of r_out (moe_norm_backward: of x)
    const void *w_post, *gate, *w_pre;
    int gate_kind, gate_act;
    bool w_f32, gate_f32;
    float r_scale, y_scale;
    const float *rstd_post, *rstd_pre;
    int64_t T, d;
    void* dr;
    uint16_t* dy;
    void* dgate;                             // per token or element
    float *part_pre, *part_y;  // partial sums over the tokens, NULL: not wanted
};

typedef unsigned int u4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));

// eight values from element i (a multiple of 8)
__device__ __forceinline__ void load8(float (&v)[8], const void* p, int64_t i, bool f32) {
    if (f32) {
        const f4* q = reinterpret_cast<const f4*>(static_cast<const float*>(p) + i);
        const f4 a = q[0], b = q[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    } else {
        const u4 a = *reinterpret_cast<const u4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16_lo(a[j]);
            v[2 * j + 1] = bf16_hi(a[j]);
        }
    }
}
__device__ __forceinline__ void store8(void* p, int64_t i, bool f32, const float (&v)[8]) {
    if (f32) {
        f4* q = reinterpret_cast<f4*>(static_cast<float*>(p) + i);
        q[0] = f4{v[0], v[1], v[2], v[3]};
        q[1] = f4{v[4], v[5], v[6], v[7]};
    } else {
        *reinterpret_cast<u4*>(static_cast<uint16_t*>(p) + i) =
            u4{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7])};
    }
}
// a value as it is stored
__device__ __forceinline__ float stored(float v, bool f32) { return f32 ? v : bf16_to_f32(f32_to_bf16(v)); }
__device__ __forceinline__ float load1(const void* p, int64_t i, bool f32) {
    return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ void store1(void* p, int64_t i, bool f32, float v) {
    if (f32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16(v);
}

// Gate and its slope, for the gradients. The exponential of -|x| serves both, without
// cancellation: e / (1 + e)^2 is the slope on either side. exp2 and reciprocal of the
// hardware, the product's rounding and a Newton step made good: 4 roundings' worth off,
// half the instructions of expf and a division. Beyond |x| = 128 e is 0, as it is from 88 on
// (exp2 gives no values below 2^-126); stopped there, the product's rounding stays a number
// for infinite x too. A NaN goes through.
struct Gate {
    float value, slope;
};
__device__ __forceinline__ Gate gate_of(float x, int act) {
    if (act != MOE_ACT_SIGMOID) return {x, 1.0f};
    float n = -fabsf(x);
    n = n < -128.f ? -128.f : n;
    const float t = n * 1.4426950408889634f;
    const float lost = fmaf(n, 1.4426950408889634f, -t) + n * 1.9259629911266175e-8f;  // of the product, and of log2 e
    const float e0 = __builtin_amdgcn_exp2f(t), e = fmaf(e0, lost * 0.6931471805599453f, e0);
    const float d = 1.0f + e, r = __builtin_amdgcn_rcpf(d), q = fmaf(fmaf(-d, r, 1.0f), r, r);
    return {x >= 0.f ? q : e * q, e * q * q};
}
__device__ __forceinline__ float gate_value(float x, int act) {
    return act == MOE_ACT_SIGMOID ? 1.0f / (1.0f + expf(-x)) : x;
}
__device__ __forceinline__ float gate_slope(float x, int act) { return gate_of(x, act).slope; }

// Squares are taken of values times part = 2^-n, 4^n >= d, and their sum divided by
// parts = d 4^-n: it then passes fp32's range where the mean itself does, not d times before.
// (Powers of two: nothing is rounded but squares that are subnormal then, next to which even an
// eps of 1e-28 is large.)
__device__ __forceinline__ float square_of(float v, float part) {
    const float q = v * part;
    return q * q;
}

// Sum over the workgroup, the same in every thread; `slot` alternates so that one
// barrier does.
__device__ __forceinline__ float block_sum(float v, float (*lds)[NT / 64], int& slot) {
    v = group_sum<64>(v);
    if ((threadIdx.x & 63) == 0) lds[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) s += lds[slot][i];
    slot ^= 1;
    return s;
}

// r_out of one element, each operation rounded as it is written: r_out is stored in as few
// as eight bits, and where it lies next to the border of two of them, the same
// operations give the same one.
__device__ __forceinline__ float joined(float r, float y, float rho, float w, float g, float r_scale, float y_scale) {
#pragma clang fp contract(off)
    return r_scale * r + y_scale * (g * (y * rho * w));
}

// eight gate values of row t, columns c ...
__device__ __forceinline__ void gate8(float (&g)[8], const void* gate, int kind, bool f32, int64_t t, int64_t c, int64_t d) {
    if (kind == MOE_GATE_CHANNEL) load8(g, gate, c, f32);
    else if (kind == MOE_GATE_FULL) load8(g, gate, t * d + c, f32);
    else {
        const float v = kind == MOE_GATE_TOKEN ? load1(gate, t, f32) : 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = v;
    }
}

// Rows of more than 16384 columns: one workgroup per row, the row read again for each
// sum, from the caches. 4096 rows of 16400, gate per channel: 191 us, of 107 at the rate of
// a large copy; what a thread does in turn between barriers bounds it.
template <bool RF32>
__global__ __launch_bounds__(NT) void join_kernel(JoinArgs a) {
    __shared__ float lds[2][NT / 64];
    int slot = 0;
    const int64_t d = a.d;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const uint16_t* y = a.y ? a.y + t * a.ldy : nullptr;
        float rho_y = 1.0f;
        if (y && a.w_post) {
            float s = 0.f;
            for (int64_t c = threadIdx.x * 8; c < d; c += NT * 8) {
                float v[8];
                load8(v, y, c, false);
#pragma unroll
                for (int j = 0; j < 8; ++j) s += square_of(v[j], a.part);
            }
            rho_y = 1.0f / sqrtf(block_sum(s, lds, slot) / a.parts + a.eps);
            if (a.rstd_post && threadIdx.x == 0) a.rstd_post[t] = rho_y;
        }
        const void* r = RF32 ? (const void*)(static_cast<const float*>(a.r) + t * a.ldr)
                             : (const void*)(static_cast<const uint16_t*>(a.r) + t * a.ldr);
        float s = 0.f;
        for (int64_t c = threadIdx.x * 8; c < d; c += NT * 8) {
            float rv[8];
            load8(rv, r, c, RF32);
            if (y) {
                float v[8], g[8], w[8];
                load8(v, y, c, false);
                gate8(g, a.gate, a.gate_kind, a.gate_f32, t, c, d);
                if (a.w_post) load8(w, a.w_post, c, a.w_f32);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    rv[j] = joined(rv[j], v[j], rho_y, a.w_post ? w[j] : 1.0f, gate_value(g[j], a.gate_act), a.r_scale,
                                   a.y_scale);
                store8(a.r_out, t * d + c, RF32, rv);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s += square_of(stored(rv[j], RF32), a.part);
        }
        if (!a.w_pre) continue;
        const float rho = 1.0f / sqrtf(block_sum(s, lds, slot) / a.parts + a.eps);
        if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[t] = rho;
        for (int64_t c = threadIdx.x * 8; c < d; c += NT * 8) {
            float rv[8], w[8];
            if (y) load8(rv, a.r_out, t * d + c, RF32);
            else load8(rv, r, c, RF32);
            load8(w, a.w_pre, c, a.w_f32);
#pragma unroll
            for (int j = 0; j < 8; ++j) rv[j] = rv[j] * rho * w[j];
            store8(a.h, t * d + c, false, rv);
        }
    }
}

// Their gradients; what is summed over the tokens goes into the workgroup's own row of
// the partial sums, in memory: 526 us where the copy rate allows 161. Two such sums are read and
// written for every row, 16 bytes a column next to the operands' 12, and the row is read three
// times, for the means in turn.
template <bool RF32>
__global__ __launch_bounds__(NT) void join_backward_kernel(JoinGradArgs a) {
    __shared__ float lds[2][NT / 64];
    int slot = 0;
    const int64_t d = a.d;
    bool first = true;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, first = false) {
        const uint16_t* y = a.y ? a.y + t * a.ldy : nullptr;
        const void* r = RF32 ? (const void*)(static_cast<const float*>(a.r_out) + t * a.ldr)
                             : (const void*)(static_cast<const uint16_t*>(a.r_out) + t * a.ldr);
        const float rho = a.w_pre ? a.rstd_pre[t] : 0.f;
        const float rho_y = y && a.w_post ? a.rstd_post[t] : 1.f;
        float mean = 0.f;
        if (a.w_pre) {
            float s = 0.f;
            for (int64_t c = threadIdx.x * 8; c < d; c += NT * 8) {
                float dh[8], w[8], rv[8];
                load8(dh, a.dh, t * d + c, false);
                load8(w, a.w_pre, c, a.w_f32);
                load8(rv, r, c, RF32);
#pragma unroll
                for (int j = 0; j < 8; ++j) s += dh[j] * w[j] * (rv[j] * rho);
            }
            mean = block_sum(s, lds, slot) / (float)d;
        }
        // D of eight columns; dh * r_out * rho of them
        auto total = [&](int64_t c, float (&D)[8], float (&e)[8]) {
            if (a.d_out) load8(D, a.d_out, t * d + c, RF32);
            else
                for (int j = 0; j < 8; ++j) D[j] = 0.f;
            if (!a.w_pre) return;
            float dh[8], w[8], rv[8];
            load8(dh, a.dh, t * d + c, false);
            load8(w, a.w_pre, c, a.w_f32);
            load8(rv, r, c, RF32);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float rh = rv[j] * rho;
                D[j] += rho * (dh[j] * w[j] - rh * mean);
                e[j] = dh[j] * rh;
            }
        };
        float sn = 0.f, sg = 0.f;
        const bool token = y && a.gate_kind == MOE_GATE_TOKEN;
        if (y && (a.w_post || token)) {
            for (int64_t c = threadIdx.x * 8; c < d; c += NT * 8) {
                float D[8], e[8], v[8], g[8], w[8];
                total(c, D, e);
                load8(v, y, c, false);
                gate8(g, a.gate, a.gate_kind, a.gate_f32, t, c, d);
                if (a.w_post) load8(w, a.w_post, c, a.w_f32);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float n = a.w_post ? v[j] * rho_y * w[j] : v[j], dz = a.y_scale * D[j];
                    sg += dz * n;
                    sn += dz * gate_of(g[j], a.gate_act).value * n;   // dn * w_post * y * rho_y
                }
            }
            if (a.w_post) sn = block_sum(sn, lds, slot) / (float)d;
            if (token) {
                sg = block_sum(sg, lds, slot);
                if (a.dgate && threadIdx.x == 0)
                    store1(a.dgate, t, a.gate_f32, sg * gate_slope(load1(a.gate, t, a.gate_f32), a.gate_act));
            }
        }
        const int64_t base = (int64_t)blockIdx.x * d;
        auto add8 = [&](float* p, int64_t c, const float (&v)[8]) {
            float o[8];
            if (first)
                for (int j = 0; j < 8; ++j) o[j] = 0.f;
            else load8(o, p, base + c, true);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] += v[j];
            store8(p, base + c, true, o);
        };
        for (int64_t c = threadIdx.x * 8; c < d; c += NT * 8) {
            float D[8], e[8], o[8];
            total(c, D, e);
            if (a.part_pre) add8(a.part_pre, c, e);
            if (a.dr) {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = a.r_scale * D[j];
                store8(a.dr, t * d + c, RF32, o);
            }
            if (!y) continue;
            float v[8], g[8], w[8], dg[8], p[8];
            load8(v, y, c, false);
            gate8(g, a.gate, a.gate_kind, a.gate_f32, t, c, d);
            if (a.w_post) load8(w, a.w_post, c, a.w_f32);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float yh = v[j] * rho_y, n = a.w_post ? yh * w[j] : v[j];
                const float dz = a.y_scale * D[j], dn = dz * gate_of(g[j], a.gate_act).value;
                dg[j] = dz * n;
                p[j] = (a.gate_kind == MOE_GATE_CHANNEL ? dz : dn) * yh;
                o[j] = a.w_post ? rho_y * (dn * w[j] - yh * sn) : dn;
            }
            if (a.dy) store8(a.dy, t * d + c, false, o);
            if (a.part_y) add8(a.part_y, c, p);
            if (a.gate_kind == MOE_GATE_FULL && a.dgate) {
#pragma unroll
                for (int j = 0; j < 8; ++j) dg[j] *= gate_slope(g[j], a.gate_act);
                store8(a.dgate, t * d + c, a.gate_f32, dg);
            }
        }
    }
}

// ---------------------------------------------------------------- rows in registers
//
// A team holds a row: every thread one chunk of eight columns, the same columns in
// every row, so that weights and column sums stay in its registers. Rows of up to
// 512 columns: teams of L lanes (a power of two) of a wave, no barriers; longer
// ones: a workgroup of up to 1024 threads, one barrier per sum. The next row's loads
// go out before this row's sums are waited for. (512 columns in a workgroup of one wave
// instead: gradients of 16384 rows 32.1 against 32.8 us, of 1237 rows of 320 12.4 against 11.7;
// 256 columns, 16384 rows: forward 14.4 against 10.9, gradients 27.8 against 22.3.)
//
// Bound by memory where there are many rows: 16384 rows of 7168, y, r and both outputs in
// bf16, take 190 us (4.9 TB/s; a large copy reaches 5.0), a norm alone of 4096 rows 19 us.
// Few rows are bound by the latency of a row's chain of load, sum, barrier, store: 64 rows
// of 8192 6.4 us.

// Sum over aligned groups of L lanes (a power of two up to 64), in every lane.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float swap16_add(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float swap32_add(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
template <int N>
__device__ __forceinline__ void lanes_sum(float (&v)[N], int L) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (L > 1) v[i] = dpp_add<0xB1>(v[i]);    // lane xor 1
        if (L > 2) v[i] = dpp_add<0x4E>(v[i]);    // lane xor 2
        if (L > 4) v[i] = dpp_add<0x141>(v[i]);   // mirrored in 8
        if (L > 8) v[i] = dpp_add<0x140>(v[i]);   // mirrored in 16
        if (L > 16) v[i] = swap16_add(v[i]);
        if (L > 32) v[i] = swap32_add(v[i]);
    }
}
// Sums over the team, in every thread; lds alternates between calls.
template <bool WAVE, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int L, float (*lds)[16][4], int& slot) {
    if constexpr (WAVE) {
        lanes_sum(v, L);
    } else {
        lanes_sum(v, 64);
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 15, waves = blockDim.x >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) lds[slot][wave][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lane < waves ? lds[slot][lane][i] : 0.f;
        lanes_sum(v, 16);
        slot ^= 1;
    }
}

// eight columns as they lie in memory
template <bool F32>
struct Chunk {
    u4 q[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        const u4* s = reinterpret_cast<const u4*>(static_cast<const char*>(p) + i * (F32 ? 4 : 2));
#pragma unroll
        for (int k = 0; k < (F32 ? 2 : 1); ++k) q[k] = s[k];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < (F32 ? 2 : 1); ++k) q[k] = u4{0u, 0u, 0u, 0u};
    }
    // keeps the values packed over this point: unpacked ones are made anew behind it
    __device__ __forceinline__ void pin() {
#pragma unroll
        for (int k = 0; k < (F32 ? 2 : 1); ++k) asm volatile("" : "+v"(q[k]));
    }
    __device__ __forceinline__ void put(const float (&v)[8]) {  // values that are of the type
#pragma unroll
        for (int j = 0; j < (F32 ? 8 : 4); ++j) {
            if constexpr (F32) q[j >> 2][j & 3] = __float_as_uint(v[j]);
            else q[0][j] = cvt_bf16x2(v[2 * j], v[2 * j + 1]);
        }
    }
    __device__ __forceinline__ float operator[](int j) const {
        if constexpr (F32) return __uint_as_float(q[j >> 2][j & 3]);
        else return (j & 1) ? bf16_hi(q[0][j >> 1]) : bf16_lo(q[0][j >> 1]);
    }
};

struct Team {
    int64_t row, rows;  // first row, and how many teams there are
    int64_t c;          // first column
    bool on;            // the thread has columns
};
template <bool WAVE>
__device__ __forceinline__ Team team_of(int64_t d, int L) {
    if constexpr (WAVE) {
        const int lane = threadIdx.x & 63, per = 64 / L;
        const int64_t wave = (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
        const int64_t c = (lane & (L - 1)) * 8;
        return {wave * per + lane / L, (int64_t)gridDim.x * (blockDim.x >> 6) * per, c, c < d};
    } else {
        const int64_t c = (int64_t)threadIdx.x * 8;
        return {blockIdx.x, gridDim.x, c, c < d};
    }
}

// eight exponentials at once would not fit the registers
__device__ __forceinline__ void two_at_a_time(int j) {
    if (j & 1) __builtin_amdgcn_sched_barrier(0);
}

enum { FULL_NONE = 0, FULL_BF16 = 1, FULL_F32 = 2 };  // a gate per element, and its type

// Y: with y, else a norm of r alone. Waves of one workgroup run rows of their own in
// the WAVE form; a team without a row left computes on the last one and stores nothing.
template <bool RF32, bool Y, int FULL, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void join_rows_kernel(JoinArgs a, int L) {
    __shared__ float lds[2][16][4];
    int slot = 0;
    const int64_t d = a.d;
    const Team tm = team_of<WAVE>(d, L);
    float wp[8], gc[8], wn[8];  // weights of y's norm, a channel's gate, weights of the next norm
#pragma unroll
    for (int j = 0; j < 8; ++j) wp[j] = gc[j] = 1.0f, wn[j] = 0.f;
    if (tm.on) {
        if (Y && a.w_post) load8(wp, a.w_post, tm.c, a.w_f32);
        if (Y && a.gate_kind == MOE_GATE_CHANNEL) {
            load8(gc, a.gate, tm.c, a.gate_f32);
#pragma unroll
            for (int j = 0; j < 8; ++j) gc[j] = gate_value(gc[j], a.gate_act);
        }
        if (a.w_pre) load8(wn, a.w_pre, tm.c, a.w_f32);
    }
    Chunk<false> y, y1;
    Chunk<RF32> r, r1;
    Chunk<FULL == FULL_F32> g, g1;
    y1.zero(), r1.zero(), g1.zero();
    auto fetch = [&](int64_t t) {
        if (!tm.on) return;
        r1.load(a.r, t * a.ldr + tm.c);
        if constexpr (Y) y1.load(a.y, t * a.ldy + tm.c);
        if constexpr (FULL != FULL_NONE) g1.load(a.gate, t * d + tm.c);
    };
    // the WAVE form's teams of one wave go round together
    const int64_t last = a.T - 1;
    fetch(tm.row < a.T ? tm.row : last);
    for (int64_t t0 = WAVE ? tm.row & ~(int64_t)(64 / L - 1) : tm.row; t0 < a.T; t0 += tm.rows) {
        const int64_t t = WAVE ? t0 + (tm.row & (64 / L - 1)) : t0;
        const bool live = !WAVE || t < a.T;
        y = y1, r = r1, g = g1;
        if (t0 + tm.rows < a.T) fetch(t + tm.rows < a.T ? t + tm.rows : last);
        float rv[8];
        if constexpr (Y) {
            float rho_y = 1.0f;
            if (a.w_post) {
                float s[1] = {0.f};
#pragma unroll
                for (int j = 0; j < 8; ++j) s[0] += square_of(y[j], a.part);
                team_sum<WAVE>(s, L, lds, slot);
                rho_y = 1.0f / sqrtf(s[0] / a.parts + a.eps);
                if (a.rstd_post && live && tm.c == 0) a.rstd_post[t] = rho_y;
            }
            float gt = 1.0f;
            if (a.gate_kind == MOE_GATE_TOKEN) gt = gate_value(load1(a.gate, live ? t : last, a.gate_f32), a.gate_act);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float f = FULL != FULL_NONE ? gate_value(g[j], a.gate_act) : gc[j];
                if (a.gate_kind == MOE_GATE_TOKEN) f = gt;
                rv[j] = stored(joined(r[j], y[j], rho_y, wp[j], f, a.r_scale, a.y_scale), RF32);
            }
            if (live && tm.on) store8(a.r_out, t * d + tm.c, RF32, rv);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) rv[j] = r[j];
        }
        if (!a.w_pre) continue;
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] += square_of(rv[j], a.part);
        team_sum<WAVE>(s, L, lds, slot);
        const float rho = 1.0f / sqrtf(s[0] / a.parts + a.eps);
        if (live && tm.on) {
            if (a.rstd_pre && tm.c == 0) a.rstd_pre[t] = rho;
#pragma unroll
            for (int j = 0; j < 8; ++j) rv[j] = rv[j] * rho * wn[j];
            store8(a.h, t * d + tm.c, false, rv);
        }
    }
}

// The gradients. With z = g n and a = dh w_pre the mean that dy's norm needs,
//     sum D z = sum d_out z + rho (sum a z - mean(a rh) sum rh z),
// comes from sums that do not wait for mean(a rh): one round of four sums per row.
// Sums over the tokens: dh rh, and D g yh (a channel's gate, the same for all of
// them, is put in at the end).
// MOST: threads of a workgroup at most. With a gate per element the next row's chunks fit
// the registers up to 512.
// 16384 rows of 7168, bf16: 263 us of reading and writing six operands (5.4 TB/s), memory-bound;
// four sums in four rounds would add three barriers to every row.
template <bool RF32, bool Y, int FULL, bool WAVE, int MOST>
__global__ __launch_bounds__(MOST) void join_rows_backward_kernel(JoinGradArgs a, int L) {
    constexpr bool AHEAD = FULL == FULL_NONE || MOST <= 512;
    __shared__ float lds[2][16][4];
    int slot = 0;
    const int64_t d = a.d;
    const Team tm = team_of<WAVE>(d, L);
    float wz[8], wn[8];  // of y: the norm's weight, a channel's gate; of the next norm
#pragma unroll
    for (int j = 0; j < 8; ++j) wz[j] = 1.0f, wn[j] = 0.f;
    if (tm.on) {
        float v[8];
        if (Y && a.w_post) load8(wz, a.w_post, tm.c, a.w_f32);
        if (Y && a.gate_kind == MOE_GATE_CHANNEL) {
            load8(v, a.gate, tm.c, a.gate_f32);
#pragma unroll
            for (int j = 0; j < 8; ++j) wz[j] *= gate_value(v[j], a.gate_act);
        }
        if (a.w_pre) load8(wn, a.w_pre, tm.c, a.w_f32);
    }
    float acc_n[8], acc_y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc_n[j] = acc_y[j] = 0.f;
    Chunk<false> y, y1, h, h1;
    Chunk<RF32> r, r1, o, o1;
    Chunk<FULL == FULL_F32> g, g1;
    y1.zero(), h1.zero(), r1.zero(), o1.zero(), g1.zero();
    auto fetch = [&](int64_t t) {
        if (!tm.on) return;
        if (a.w_pre) {
            h1.load(a.dh, t * d + tm.c);
            r1.load(a.r_out, t * a.ldr + tm.c);
        }
        if (a.d_out) o1.load(a.d_out, t * d + tm.c);
        if constexpr (Y) y1.load(a.y, t * a.ldy + tm.c);
        if constexpr (FULL != FULL_NONE) g1.load(a.gate, t * d + tm.c);
    };
    const int64_t last = a.T - 1;
    if constexpr (AHEAD) fetch(tm.row < a.T ? tm.row : last);
    for (int64_t t0 = WAVE ? tm.row & ~(int64_t)(64 / L - 1) : tm.row; t0 < a.T; t0 += tm.rows) {
        const int64_t t = WAVE ? t0 + (tm.row & (64 / L - 1)) : t0;
        const bool live = !WAVE || t < a.T;
        const int64_t tt = live ? t : last;
        if constexpr (!AHEAD) fetch(tt);
        y = y1, h = h1, r = r1, o = o1, g = g1;
        if constexpr (AHEAD)
            if (t0 + tm.rows < a.T) fetch(t + tm.rows < a.T ? t + tm.rows : last);
        const float rho = a.w_pre ? a.rstd_pre[tt] : 0.f;
        const float rho_y = Y && a.w_post ? a.rstd_post[tt] : 1.f;
        float gt = 1.f, gs = 0.f;
        if (Y && a.gate_kind == MOE_GATE_TOKEN) {
            const float v = load1(a.gate, tt, a.gate_f32);
            gt = gate_value(v, a.gate_act);
            gs = gate_slope(v, a.gate_act);
        }
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float aj = h[j] * wn[j], rh = r[j] * rho;
            s[0] += aj * rh;
            if constexpr (Y) {
                float z = y[j] * rho_y * wz[j];
                if constexpr (FULL != FULL_NONE) z *= gate_of(g[j], a.gate_act).value;
                s[1] += o[j] * z;
                s[2] += aj * z;
                s[3] += rh * z;
                if constexpr (FULL != FULL_NONE && MOST > 512) two_at_a_time(j);
            }
        }
        if constexpr (Y) {
            team_sum<WAVE>(s, L, lds, slot);
        } else {
            float s1[1] = {s[0]};
            team_sum<WAVE>(s1, L, lds, slot);
            s[0] = s1[0];
        }
        y.pin(), h.pin(), r.pin(), o.pin(), g.pin();
        const float mean = s[0] / (float)d;
        float sn = 0.f;
        if constexpr (Y) {
            const float sum = a.y_scale * (s[1] + rho * (s[2] - mean * s[3]));
            if (a.gate_kind == MOE_GATE_TOKEN && a.dgate && live && tm.c == 0) store1(a.dgate, t, a.gate_f32, sum * gs);
            sn = sum * gt / (float)d;
        }
        if (!live || !tm.on) continue;
        float dr[8], dy[8], dg[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float rh = r[j] * rho, D = o[j] + rho * (h[j] * wn[j] - rh * mean);
            acc_n[j] += h[j] * rh;
            dr[j] = a.r_scale * D;
            if constexpr (Y) {
                const float yh = y[j] * rho_y, dz = a.y_scale * D;
                float q = dz * gt;
                if constexpr (FULL != FULL_NONE) {
                    const Gate f = gate_of(g[j], a.gate_act);
                    q *= f.value;
                    dg[j] = dz * (yh * wz[j]) * f.slope;
                }
                acc_y[j] += q * yh;
                dy[j] = a.w_post ? rho_y * (q * wz[j] - yh * sn) : q * wz[j];
                if constexpr (FULL != FULL_NONE && MOST > 512) two_at_a_time(j);
            }
        }
        if (a.dr) store8(a.dr, t * d + tm.c, RF32, dr);
        if constexpr (Y) {
            if (a.dy) store8(a.dy, t * d + tm.c, false, dy);
            if constexpr (FULL != FULL_NONE)
                if (a.dgate) store8(a.dgate, t * d + tm.c, FULL == FULL_F32, dg);
        }
    }
    // one partial row per workgroup or wave
    int64_t part = blockIdx.x;
    if constexpr (WAVE) {
        part = (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
        for (int m = L; m < 64; m <<= 1)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                acc_n[j] += __shfl_xor(acc_n[j], m);
                acc_y[j] += __shfl_xor(acc_y[j], m);
            }
        if ((threadIdx.x & 63) >= L) return;
    }
    if (!tm.on) return;
    if (a.part_pre) store8(a.part_pre, part * d + tm.c, true, acc_n);
    if (Y && a.part_y) store8(a.part_y, part * d + tm.c, true, acc_y);
}

// Rows of 8200 to 16384 columns: a workgroup of 1024 threads, two chunks to a thread,
// 8192 columns apart. What else would need registers lies in LDS, a thread's own values in
// places of its own (no barriers): a channel's gate; for the gradients y's weights and one
// of the column sums. The other weights come from the caches for each row. 4096 rows of
// 16384, gate per channel: forward 115 us, gradients 175 (copy rate 107 and 161); 8200 columns
// 65 and 97, by the re-reading kernels 80 and 257.
constexpr int LONG = 2, LONG_STEP = 8192;
// a thread's own eight values in LDS
typedef f4 Own8[2][1024];
__device__ __forceinline__ void put_own(Own8& p, const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) p[i][threadIdx.x] = f4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
}
__device__ __forceinline__ void get_own(float (&v)[8], const Own8& p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = p[j >> 2][threadIdx.x][j & 3];
}
template <bool RF32, bool Y, int FULL>
__global__ __launch_bounds__(1024) void join_long_kernel(JoinArgs a) {
    __shared__ float lds[2][16][4];
    int slot = 0;
    const int64_t d = a.d, c0 = (int64_t)threadIdx.x * 8;
    __shared__ Own8 channel[Y && FULL == FULL_NONE ? LONG : 1];  // a channel's gate
    if (Y && FULL == FULL_NONE && a.gate_kind != MOE_GATE_TOKEN) {
#pragma unroll
        for (int k = 0; k < LONG; ++k) {
            const int64_t c = c0 + k * LONG_STEP;
            if (c >= d) continue;
            float v[8];
            gate8(v, a.gate, a.gate_kind, a.gate_f32, 0, c, d);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = gate_value(v[j], a.gate_act);
            put_own(channel[k], v);
        }
    }
    Chunk<false> y[LONG], y1[LONG];
    Chunk<RF32> r[LONG], r1[LONG];
    Chunk<FULL == FULL_F32> g[LONG], g1[LONG];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int k = 0; k < LONG; ++k) {
            const int64_t c = c0 + k * LONG_STEP;
            if (c >= d) continue;
            if constexpr (Y) y1[k].load(a.y, t * a.ldy + c);
            r1[k].load(a.r, t * a.ldr + c);
            if constexpr (FULL != FULL_NONE) g1[k].load(a.gate, t * d + c);
        }
    };
#pragma unroll
    for (int k = 0; k < LONG; ++k) y1[k].zero(), r1[k].zero(), g1[k].zero();
    if (blockIdx.x < a.T) fetch(blockIdx.x);
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
#pragma unroll
        for (int k = 0; k < LONG; ++k) y[k] = y1[k], r[k] = r1[k], g[k] = g1[k];
        if (t + gridDim.x < a.T) fetch(t + gridDim.x);
        if constexpr (Y) {
            float rho_y = 1.0f;
            if (a.w_post) {
                float s[1] = {0.f};
#pragma unroll
                for (int k = 0; k < LONG; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[0] += square_of(y[k][j], a.part);
                team_sum<false>(s, 64, lds, slot);
                rho_y = 1.0f / sqrtf(s[0] / a.parts + a.eps);
                if (a.rstd_post && threadIdx.x == 0) a.rstd_post[t] = rho_y;
            }
            float gt = 1.0f;
            if (a.gate_kind == MOE_GATE_TOKEN) gt = gate_value(load1(a.gate, t, a.gate_f32), a.gate_act);
#pragma unroll
            for (int k = 0; k < LONG; ++k) {
                const int64_t c = c0 + k * LONG_STEP;
                if (c >= d) continue;
                float w[8], f[8], rv[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 1.0f;
                if (a.w_post) load8(w, a.w_post, c, a.w_f32);
                if (FULL == FULL_NONE && a.gate_kind != MOE_GATE_TOKEN) get_own(f, channel[k]);
                else
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = FULL != FULL_NONE ? gate_value(g[k][j], a.gate_act) : gt;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    rv[j] = stored(joined(r[k][j], y[k][j], rho_y, w[j], f[j], a.r_scale, a.y_scale), RF32);
                store8(a.r_out, t * d + c, RF32, rv);
                r[k].put(rv);
            }
        }
        if (!a.w_pre) continue;
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < LONG; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += square_of(r[k][j], a.part);
        team_sum<false>(s, 64, lds, slot);
        const float rho = 1.0f / sqrtf(s[0] / a.parts + a.eps);
        if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[t] = rho;
#pragma unroll
        for (int k = 0; k < LONG; ++k) {
            const int64_t c = c0 + k * LONG_STEP;
            if (c >= d) continue;
            float w[8];
            load8(w, a.w_pre, c, a.w_f32);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = r[k][j] * rho * w[j];
            store8(a.h, t * d + c, false, w);
        }
    }
}

// Their gradients, with the sums of join_rows_backward_kernel.
template <bool RF32, bool Y, int FULL>
__global__ __launch_bounds__(1024) void join_long_backward_kernel(JoinGradArgs a) {
    __shared__ float lds[2][16][4];
    int slot = 0;
    const int64_t d = a.d, c0 = (int64_t)threadIdx.x * 8;
    // a thread's column sums: dh rh, and D g yh; of y: the norm's weights, a channel's gate
    float acc_n[LONG][8];
    __shared__ Own8 acc_y[Y ? LONG : 1], of_y[Y ? LONG : 1];
#pragma unroll
    for (int k = 0; k < LONG; ++k) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc_n[k][j] = 0.f;
        if constexpr (Y) {
            const int64_t c = c0 + k * LONG_STEP;
            put_own(acc_y[k], acc_n[k]);
            if (c >= d) continue;
            float w[8], v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = v[j] = 1.0f;
            if (a.w_post) load8(w, a.w_post, c, a.w_f32);
            if (FULL == FULL_NONE && a.gate_kind == MOE_GATE_CHANNEL) load8(v, a.gate, c, a.gate_f32);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] *= a.gate_kind == MOE_GATE_CHANNEL ? gate_of(v[j], a.gate_act).value : 1.0f;
            put_own(of_y[k], w);
        }
    }
    Chunk<false> y[LONG], h[LONG];
    Chunk<RF32> r[LONG], o[LONG];
    Chunk<FULL == FULL_F32> g[LONG];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
#pragma unroll
        for (int k = 0; k < LONG; ++k) {
            const int64_t c = c0 + k * LONG_STEP;
            y[k].zero(), h[k].zero(), r[k].zero(), o[k].zero(), g[k].zero();
            if (c >= d) continue;
            if (a.w_pre) {
                h[k].load(a.dh, t * d + c);
                r[k].load(a.r_out, t * a.ldr + c);
            }
            if (a.d_out) o[k].load(a.d_out, t * d + c);
            if constexpr (Y) y[k].load(a.y, t * a.ldy + c);
            if constexpr (FULL != FULL_NONE) g[k].load(a.gate, t * d + c);
        }
        const float rho = a.w_pre ? a.rstd_pre[t] : 0.f;
        const float rho_y = Y && a.w_post ? a.rstd_post[t] : 1.f;
        Gate gt = {1.f, 0.f};
        if (Y && a.gate_kind == MOE_GATE_TOKEN) gt = gate_of(load1(a.gate, t, a.gate_f32), a.gate_act);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < LONG; ++k) {
            const int64_t c = c0 + k * LONG_STEP;
            if (c >= d) continue;
            __builtin_amdgcn_sched_barrier(0);
            float wn[8], wz[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) wn[j] = 0.f;
            if (a.w_pre) load8(wn, a.w_pre, c, a.w_f32);
            if constexpr (Y) get_own(wz, of_y[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float aj = h[k][j] * wn[j], rh = r[k][j] * rho;
                s[0] += aj * rh;
                if constexpr (Y) {
                    float z = y[k][j] * rho_y * wz[j];
                    if constexpr (FULL != FULL_NONE) z *= gate_of(g[k][j], a.gate_act).value;
                    s[1] += o[k][j] * z;
                    s[2] += aj * z;
                    s[3] += rh * z;
                }
                two_at_a_time(j);
            }
        }
        team_sum<false>(s, 64, lds, slot);
#pragma unroll
        for (int k = 0; k < LONG; ++k) y[k].pin(), h[k].pin(), r[k].pin(), o[k].pin(), g[k].pin();
        const float mean = s[0] / (float)d;
        float sn = 0.f;
        if constexpr (Y) {
            const float sum = a.y_scale * (s[1] + rho * (s[2] - mean * s[3]));
            if (a.gate_kind == MOE_GATE_TOKEN && a.dgate && threadIdx.x == 0) store1(a.dgate, t, a.gate_f32, sum * gt.slope);
            sn = sum * gt.value / (float)d;
        }
#pragma unroll
        for (int k = 0; k < LONG; ++k) {
            const int64_t c = c0 + k * LONG_STEP;
            if (c >= d) continue;
            __builtin_amdgcn_sched_barrier(0);
            float wn[8], wz[8], dr[8], dy[8], dg[8], ey[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) wn[j] = 0.f;
            if (a.w_pre) load8(wn, a.w_pre, c, a.w_f32);
            if constexpr (Y) get_own(wz, of_y[k]), get_own(ey, acc_y[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float rh = r[k][j] * rho, D = o[k][j] + rho * (h[k][j] * wn[j] - rh * mean);
                acc_n[k][j] += h[k][j] * rh;
                dr[j] = a.r_scale * D;
                if constexpr (Y) {
                    const float yh = y[k][j] * rho_y, dz = a.y_scale * D;
                    float q = dz * gt.value;
                    if constexpr (FULL != FULL_NONE) {
                        const Gate f = gate_of(g[k][j], a.gate_act);
                        q *= f.value;
                        dg[j] = dz * (yh * wz[j]) * f.slope;
                    }
                    ey[j] += q * yh;
                    dy[j] = a.w_post ? rho_y * (q * wz[j] - yh * sn) : q * wz[j];
                }
                two_at_a_time(j);
            }
            if constexpr (Y) put_own(acc_y[k], ey);
            if (a.dr) store8(a.dr, t * d + c, RF32, dr);
            if constexpr (Y) {
                if (a.dy) store8(a.dy, t * d + c, false, dy);
                if constexpr (FULL != FULL_NONE)
                    if (a.dgate) store8(a.dgate, t * d + c, FULL == FULL_F32, dg);
            }
        }
    }
    const int64_t part = blockIdx.x;
#pragma unroll
    for (int k = 0; k < LONG; ++k) {
        const int64_t c = c0 + k * LONG_STEP;
        if (c >= d) continue;
        if (a.part_pre) store8(a.part_pre, part * d + c, true, acc_n[k]);
        if constexpr (Y) {
            float v[8];
            get_own(v, acc_y[k]);
            if (a.part_y) store8(a.part_y, part * d + c, true, v);
        }
    }
}

// The columns' sums over the partial rows, in a fixed order; then dw_pre, or dw_post and
// a channel's dgate, which share one sum q: dw_post = g q, dgate = w_post slope(gate) q.
// COLS columns to a workgroup of 1024 threads, the others over the rows: 64, or 16
// where 64 would leave half the compute units without work (100000 x 64, 4096 partial rows: the
// backward pass 29.7 -> 23.7 us; 1024 x 7168, with whole cache lines of 64: 25.5 against 28.5).
struct ColumnSums {
    const float *pre, *y;
    int64_t rows, d;
    void *dw_pre, *dw_post, *dgate;
    const void *w_post, *gate;
    bool w_f32, gate_f32, channel;
    int act;
};
template <int COLS>
__global__ __launch_bounds__(1024) void column_sums_kernel(ColumnSums a) {
    __shared__ float lds[16][COLS];
    const int col = threadIdx.x % COLS;
    const int64_t c = (int64_t)blockIdx.x * COLS + col;
    const bool of_y = a.pre == nullptr || blockIdx.y == 1;
    const float* p = (of_y ? a.y : a.pre) + (c < a.d ? c : a.d - 1);
    float s = 0.f;
#pragma unroll 8
    for (int64_t i = threadIdx.x / COLS; i < a.rows; i += 1024 / COLS) s += p[i * a.d];
#pragma unroll
    for (int m = COLS; m < 64; m <<= 1) s += __shfl_xor(s, m);
    if ((threadIdx.x & 63) < COLS) lds[threadIdx.x >> 6][col] = s;
    __syncthreads();
    if (threadIdx.x >= COLS || c >= a.d) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += lds[i][col];
    if (!of_y) {
        store1(a.dw_pre, c, a.w_f32, s);
        return;
    }
    const float g = a.channel ? load1(a.gate, c, a.gate_f32) : 0.f;
    if (a.dw_post) store1(a.dw_post, c, a.w_f32, a.channel ? s * gate_value(g, a.act) : s);
    if (a.dgate) {
        if (a.w_post) s *= load1(a.w_post, c, a.w_f32);
        store1(a.dgate, c, a.gate_f32, s * gate_slope(g, a.act));
    }
}

// zeros for the gradients of weights and of a channel's gate without tokens
__global__ __launch_bounds__(256) void zero_columns_kernel(void* a, void* b, void* g, int64_t d, bool w_f32, bool gate_f32) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= d) return;
    if (a) store1(a, c, w_f32, 0.f);
    if (b) store1(b, c, w_f32, 0.f);
    if (g) store1(g, c, gate_f32, 0.f);
}

// ---------------------------------------------------------------- host
constexpr int64_t MAX_D = 1 << 20, MAX_LD = 1 << 22, MAX_T = 1 << 30;

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
bool type_ok(int32_t t) { return t == MOE_SRC_F32 || t == MOE_SRC_BF16; }
bool finite(float v) { return v - v == 0.f; }
bool ld_ok(int64_t ld, int64_t d) { return ld >= d && ld <= MAX_LD && ld % 8 == 0; }

int check_rows(const char* what, int64_t T, int64_t d) {
    MOE_REQUIRE(T >= 0 && T <= MAX_T, MOE_ERR_SHAPE, "%s: T=%lld outside [0, 2^30]", what, (long long)T);
    MOE_REQUIRE(d >= 8 && d <= MAX_D && d % 8 == 0, MOE_ERR_SHAPE, "%s: d=%lld: a multiple of 8 up to 2^20", what,
                (long long)d);
    return MOE_OK;
}
int check_gate(const char* what, int32_t kind, int32_t type, int32_t act, const void* gate, int64_t T) {
    MOE_REQUIRE(kind >= MOE_GATE_NONE && kind <= MOE_GATE_FULL, MOE_ERR_UNSUPPORTED, "%s: gate kind %d", what, kind);
    if (kind == MOE_GATE_NONE) return MOE_OK;
    MOE_REQUIRE(type_ok(type), MOE_ERR_UNSUPPORTED, "%s: gate type %d", what, type);
    MOE_REQUIRE(act == MOE_ACT_NONE || act == MOE_ACT_SIGMOID, MOE_ERR_UNSUPPORTED, "%s: gate activation %d", what, act);
    MOE_REQUIRE(gate || T == 0, MOE_ERR_NULL, "%s: NULL gate", what);
    MOE_REQUIRE(kind == MOE_GATE_TOKEN || aligned16(gate), MOE_ERR_SHAPE, "%s: gate: 16-byte aligned", what);
    return MOE_OK;
}

// How a launch takes rows of d columns: in registers up to 8192 (a chunk of eight to
// each of up to 1024 threads) and 16384 (two chunks), read again for each sum beyond.
// (4096 rows of 8192: forward 52 us in registers, 72 read again; gradients 88 and 227.)
constexpr int64_t MAX_ROW = 8192, MAX_LONG = LONG * LONG_STEP;
struct Shape {
    int L, threads, per;  // lanes of a team in a wave (0: a workgroup to a row); rows of a workgroup at a time
};
Shape shape_of(int64_t d) {
    if (d > MAX_ROW) return {0, d > MAX_LONG ? NT : 1024, 1};
    const int chunks = (int)(d / 8);
    if (chunks > 64) return {0, (chunks + 63) / 64 * 64, 1};
    int L = 1;
    while (L < chunks) L <<= 1;
    return {L, 256, 4 * (64 / L)};
}
// workgroups of a backward launch: enough to fill the compute units, but four rows at
// least to each where there are more rows than units, for the partial sums' sake
// (2048 x 2048: 21.2 us, one row at least 22.8, sixteen 22.5; a norm's 12.4, 16.3, 13.5)
int64_t backward_blocks(int64_t T, int64_t d) {
    const Shape s = shape_of(d);
    const int64_t cus = num_cus(), units = (T + s.per - 1) / s.per;
    int64_t n = cus * (1024 / s.threads);
    const int64_t most = units / 4 > cus ? units / 4 : cus;
    n = n < most ? n : most;
    if (d > MAX_LONG) n = n < (1 << 27) / d ? n : (1 << 27) / d;
    return units < n ? units : n;
}
int64_t partial_rows(int64_t T, int64_t d) { return backward_blocks(T, d) * (shape_of(d).L ? 4 : 1); }
size_t backward_bytes(int64_t T, int64_t d, int sums) { return (size_t)partial_rows(T, d) * d * sums * sizeof(float); }

// f(Y, FULL as integral constants)
template <typename F>
void with_gate(bool y, int32_t kind, bool f32, F&& f) {
    if (!y) f(std::false_type{}, std::integral_constant<int, FULL_NONE>{});
    else if (kind != MOE_GATE_FULL) f(std::true_type{}, std::integral_constant<int, FULL_NONE>{});
    else if (f32) f(std::true_type{}, std::integral_constant<int, FULL_F32>{});
    else f(std::true_type{}, std::integral_constant<int, FULL_BF16>{});
}

template <bool RF32>
void launch_join(const JoinArgs& a, hipStream_t stream) {
    const Shape s = shape_of(a.d);
    const int64_t units = (a.T + s.per - 1) / s.per, most = (int64_t)num_cus() * (2048 / s.threads);
    const dim3 grid((unsigned)(units < most ? units : most)), block(s.threads);
    if (a.d > MAX_LONG) {
        join_kernel<RF32><<<grid, block, 0, stream>>>(a);
        return;
    }
    with_gate(a.y != nullptr, a.gate_kind, a.gate_f32, [&](auto y, auto full) {
        if (a.d > MAX_ROW) join_long_kernel<RF32, y.value, full.value><<<grid, block, 0, stream>>>(a);
        else if (s.L) join_rows_kernel<RF32, y.value, full.value, true><<<grid, block, 0, stream>>>(a, s.L);
        else join_rows_kernel<RF32, y.value, full.value, false><<<grid, block, 0, stream>>>(a, s.L);
    });
}
template <bool RF32>
void launch_join_backward(const JoinGradArgs& a, hipStream_t stream) {
    const Shape s = shape_of(a.d);
    const dim3 grid((unsigned)backward_blocks(a.T, a.d)), block(s.threads);
    if (a.d > MAX_LONG) {
        join_backward_kernel<RF32><<<grid, block, 0, stream>>>(a);
        return;
    }
    with_gate(a.y != nullptr, a.gate_kind, a.gate_f32, [&](auto y, auto full) {
        if (a.d > MAX_ROW) {
            join_long_backward_kernel<RF32, y.value, full.value><<<grid, block, 0, stream>>>(a);
            return;
        }
        if (s.L) {
            join_rows_backward_kernel<RF32, y.value, full.value, true, 256><<<grid, block, 0, stream>>>(a, s.L);
            return;
        }
        if constexpr (full.value != FULL_NONE) {
            if (s.threads <= 512) {
                join_rows_backward_kernel<RF32, y.value, full.value, false, 512><<<grid, block, 0, stream>>>(a, s.L);
                return;
            }
        }
        join_rows_backward_kernel<RF32, y.value, full.value, false, 1024><<<grid, block, 0, stream>>>(a, s.L);
    });
}

int launch_forward(JoinArgs a, bool r_f32, hipStream_t stream) {
    a.part = 1.0f;
    for (a.parts = (float)a.d; a.parts > 1.0f; a.parts *= 0.25f) a.part *= 0.5f;
    if (r_f32) launch_join<true>(a, stream);
    else launch_join<false>(a, stream);
    MOE_LAUNCH_CHECK("join_rows_kernel");
    return MOE_OK;
}

// dw_gate: of a gate per channel
int launch_backward(JoinGradArgs a, bool r_f32, void* dw_post, void* dw_pre, void* dw_gate, void* ws, hipStream_t stream) {
    if (a.T == 0) {
        if (!dw_post && !dw_pre && !dw_gate) return MOE_OK;
        zero_columns_kernel<<<dim3((unsigned)((a.d + 255) / 256)), dim3(256), 0, stream>>>(dw_post, dw_pre, dw_gate, a.d,
                                                                                           a.w_f32, a.gate_f32);
        MOE_LAUNCH_CHECK("zero_columns_kernel");
        return MOE_OK;
    }
    const int64_t rows = partial_rows(a.T, a.d);
    float* p = static_cast<float*>(ws);
    int n = 0;
    if (dw_pre) a.part_pre = p + rows * a.d * n++;
    if (dw_post || dw_gate) a.part_y = p + rows * a.d * n++;
    if (r_f32) launch_join_backward<true>(a, stream);
    else launch_join_backward<false>(a, stream);
    MOE_LAUNCH_CHECK("join_rows_backward_kernel");
    if (n == 0) return MOE_OK;
    const ColumnSums s = {a.part_pre, a.part_y, rows, a.d, dw_pre, dw_post, dw_gate, a.w_post, a.gate, a.w_f32, a.gate_f32,
                          a.gate_kind == MOE_GATE_CHANNEL, a.gate_act};
    const int64_t tiles = (a.d + 63) / 64;
    if (tiles * n >= num_cus() / 2)
        column_sums_kernel<64><<<dim3((unsigned)tiles, n), dim3(1024), 0, stream>>>(s);
    else
        column_sums_kernel<16><<<dim3((unsigned)((a.d + 15) / 16), n), dim3(1024), 0, stream>>>(s);
    MOE_LAUNCH_CHECK("column_sums_kernel");
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_norm(const void* x, int32_t x_type, int64_t ldx, const void* w, int32_t w_type, int64_t T, int64_t d,
                        float eps, uint16_t* h, float* rstd, hipStream_t stream) {
    clear_error();
    if (const int rc = check_rows("norm", T, d)) return rc;
    MOE_REQUIRE(type_ok(x_type) && type_ok(w_type), MOE_ERR_UNSUPPORTED, "norm: x type %d, w type %d", x_type, w_type);
    MOE_REQUIRE(eps > 0.f && finite(eps), MOE_ERR_SHAPE, "norm: eps must be positive and finite");
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(x && w && h, MOE_ERR_NULL, "norm: NULL x, w or h");
    MOE_REQUIRE(ld_ok(ldx, d), MOE_ERR_SHAPE, "norm: ldx=%lld: a multiple of 8 in [d, 2^22]", (long long)ldx);
    MOE_REQUIRE(aligned16(x) && aligned16(w) && aligned16(h), MOE_ERR_SHAPE, "norm: x, w and h: 16-byte aligned");
    JoinArgs a = {};
    a.r = x;
    a.ldr = ldx;
    a.w_pre = w;
    a.w_f32 = w_type == MOE_SRC_F32;
    a.eps = eps;
    a.T = T;
    a.d = d;
    a.h = h;
    a.rstd_pre = rstd;
    return launch_forward(a, x_type == MOE_SRC_F32, stream);
}

extern "C" int moe_norm_backward_workspace(int64_t T, int64_t d, size_t* bytes) {
    clear_error();
    MOE_REQUIRE(bytes, MOE_ERR_NULL, "norm_backward_workspace: NULL bytes");
    if (const int rc = check_rows("norm_backward_workspace", T, d)) return rc;
    *bytes = backward_bytes(T, d, 1);
    return MOE_OK;
}

extern "C" int moe_norm_backward(const uint16_t* dh, const void* x, int32_t x_type, int64_t ldx, const void* w,
                                 int32_t w_type, const float* rstd, const void* dx_add, int64_t T, int64_t d, void* dx,
                                 void* dw, void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    if (const int rc = check_rows("norm_backward", T, d)) return rc;
    MOE_REQUIRE(type_ok(x_type) && type_ok(w_type), MOE_ERR_UNSUPPORTED, "norm_backward: x type %d, w type %d", x_type,
                w_type);
    if (T > 0) {
        MOE_REQUIRE(dh && x && w && rstd, MOE_ERR_NULL, "norm_backward: NULL dh, x, w or rstd");
        MOE_REQUIRE(ld_ok(ldx, d), MOE_ERR_SHAPE, "norm_backward: ldx=%lld: a multiple of 8 in [d, 2^22]", (long long)ldx);
        MOE_REQUIRE(aligned16(dh) && aligned16(x) && aligned16(w) && aligned16(dx_add) && aligned16(dx), MOE_ERR_SHAPE,
                    "norm_backward: dh, x, w, dx_add and dx: 16-byte aligned");
    }
    MOE_REQUIRE(aligned16(dw) && aligned16(ws), MOE_ERR_SHAPE, "norm_backward: dw and ws: 16-byte aligned");
    if (dw && T > 0) {
        MOE_REQUIRE(ws, MOE_ERR_NULL, "norm_backward: NULL ws");
        MOE_REQUIRE(ws_bytes >= backward_bytes(T, d, 1), MOE_ERR_WORKSPACE, "norm_backward: workspace of %zu bytes, %zu needed",
                    ws_bytes, backward_bytes(T, d, 1));
    }
    if (!dx && !dw) return MOE_OK;
    JoinGradArgs a = {};
    a.d_out = dx_add;
    a.dh = dh;
    a.r_out = x;
    a.ldr = ldx;
    a.w_pre = w;
    a.w_f32 = w_type == MOE_SRC_F32;
    a.r_scale = 1.0f;
    a.rstd_pre = rstd;
    a.T = T;
    a.d = d;
    a.dr = dx;
    return launch_backward(a, x_type == MOE_SRC_F32, nullptr, dw, nullptr, ws, stream);
}

extern "C" int moe_join(const uint16_t* y, int64_t ldy, const void* r, int32_t r_type, int64_t ldr, const void* w_post,
                        const void* gate, int32_t gate_kind, int32_t gate_type, int32_t gate_act, float r_scale,
                        float y_scale, const void* w_pre, int32_t w_type, int64_t T, int64_t d, float eps, void* r_out,
                        uint16_t* h, float* rstd_post, float* rstd_pre, hipStream_t stream) {
    clear_error();
    if (const int rc = check_rows("join", T, d)) return rc;
    MOE_REQUIRE(type_ok(r_type) && type_ok(w_type), MOE_ERR_UNSUPPORTED, "join: r type %d, w type %d", r_type, w_type);
    if (const int rc = check_gate("join", gate_kind, gate_type, gate_act, gate, T)) return rc;
    MOE_REQUIRE(eps > 0.f && finite(eps), MOE_ERR_SHAPE, "join: eps must be positive and finite");
    MOE_REQUIRE(finite(r_scale) && finite(y_scale), MOE_ERR_SHAPE, "join: r_scale and y_scale must be finite");
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(y && r && r_out, MOE_ERR_NULL, "join: NULL y, r or r_out");
    MOE_REQUIRE(!w_pre || h, MOE_ERR_NULL, "join: NULL h");
    MOE_REQUIRE(ld_ok(ldy, d) && ld_ok(ldr, d), MOE_ERR_SHAPE, "join: ldy=%lld, ldr=%lld: multiples of 8 in [d, 2^22]",
                (long long)ldy, (long long)ldr);
    MOE_REQUIRE(r_out != r || ldr == d, MOE_ERR_SHAPE, "join: r_out is r's memory, but its rows lie apart");
    MOE_REQUIRE(aligned16(y) && aligned16(r) && aligned16(w_post) && aligned16(w_pre) && aligned16(r_out) && aligned16(h),
                MOE_ERR_SHAPE, "join: y, r, weights, r_out and h: 16-byte aligned");
    JoinArgs a = {y, ldy, r, ldr, w_post, gate, w_pre, gate_kind, gate_kind == MOE_GATE_NONE ? MOE_ACT_NONE : gate_act,
                  w_type == MOE_SRC_F32, gate_type == MOE_SRC_F32, r_scale, y_scale, eps, T, d, r_out, h, rstd_post, rstd_pre};
    return launch_forward(a, r_type == MOE_SRC_F32, stream);
}

extern "C" int moe_join_backward_workspace(int64_t T, int64_t d, size_t* bytes) {
    clear_error();
    MOE_REQUIRE(bytes, MOE_ERR_NULL, "join_backward_workspace: NULL bytes");
    if (const int rc = check_rows("join_backward_workspace", T, d)) return rc;
    *bytes = backward_bytes(T, d, 2);
    return MOE_OK;
}

extern "C" int moe_join_backward(const void* d_out, const uint16_t* dh, const uint16_t* y, int64_t ldy, const void* r_out,
                                 int32_t r_type, const void* w_post, const void* gate, int32_t gate_kind, int32_t gate_type,
                                 int32_t gate_act, float r_scale, float y_scale, const void* w_pre, int32_t w_type,
                                 const float* rstd_post, const float* rstd_pre, int64_t T, int64_t d, void* dr, uint16_t* dy,
                                 void* dw_post, void* dw_pre, void* dgate, void* ws, size_t ws_bytes, hipStream_t stream) {
    clear_error();
    if (const int rc = check_rows("join_backward", T, d)) return rc;
    MOE_REQUIRE(type_ok(r_type) && type_ok(w_type), MOE_ERR_UNSUPPORTED, "join_backward: r type %d, w type %d", r_type, w_type);
    if (const int rc = check_gate("join_backward", gate_kind, gate_type, gate_act, gate, T)) return rc;
    MOE_REQUIRE(finite(r_scale) && finite(y_scale), MOE_ERR_SHAPE, "join_backward: r_scale and y_scale must be finite");
    MOE_REQUIRE(w_post || !dw_post, MOE_ERR_NULL, "join_backward: dw_post without w_post");
    MOE_REQUIRE(w_pre || !dw_pre, MOE_ERR_NULL, "join_backward: dw_pre without w_pre");
    MOE_REQUIRE(gate_kind != MOE_GATE_NONE || !dgate, MOE_ERR_NULL, "join_backward: dgate without a gate");
    const int sums = (dw_pre != nullptr) + (dw_post || (dgate && gate_kind == MOE_GATE_CHANNEL));
    if (T > 0) {
        MOE_REQUIRE(y && (d_out || dh), MOE_ERR_NULL, "join_backward: NULL y, or neither d_out nor dh");
        MOE_REQUIRE((w_pre != nullptr) == (dh != nullptr), MOE_ERR_NULL, "join_backward: dh goes with w_pre");
        MOE_REQUIRE(!w_pre || (r_out && rstd_pre), MOE_ERR_NULL, "join_backward: NULL r_out or rstd_pre");
        MOE_REQUIRE(!w_post || rstd_post, MOE_ERR_NULL, "join_backward: NULL rstd_post");
        MOE_REQUIRE(ld_ok(ldy, d), MOE_ERR_SHAPE, "join_backward: ldy=%lld: a multiple of 8 in [d, 2^22]", (long long)ldy);
        MOE_REQUIRE(aligned16(d_out) && aligned16(dh) && aligned16(y) && aligned16(r_out) && aligned16(w_post) &&
                        aligned16(w_pre) && aligned16(dr) && aligned16(dy),
                    MOE_ERR_SHAPE, "join_backward: operands and gradients: 16-byte aligned");
        if (sums) {
            MOE_REQUIRE(ws, MOE_ERR_NULL, "join_backward: NULL ws");
            MOE_REQUIRE(ws_bytes >= backward_bytes(T, d, sums), MOE_ERR_WORKSPACE,
                        "join_backward: workspace of %zu bytes, %zu needed", ws_bytes, backward_bytes(T, d, sums));
        }
    }
    MOE_REQUIRE(aligned16(dw_post) && aligned16(dw_pre) && aligned16(ws) && (gate_kind == MOE_GATE_TOKEN || aligned16(dgate)),
                MOE_ERR_SHAPE, "join_backward: weights' gradients, dgate and ws: 16-byte aligned");
    if (!dr && !dy && !dw_post && !dw_pre && !dgate) return MOE_OK;
    JoinGradArgs a = {};
    a.d_out = d_out;
    a.dh = dh;
    a.y = y;
    a.ldy = ldy;
    a.r_out = r_out;
    a.ldr = d;
    a.w_post = w_post;
    a.gate = gate;
    a.w_pre = w_pre;
    a.gate_kind = gate_kind;
    a.gate_act = gate_kind == MOE_GATE_NONE ? MOE_ACT_NONE : gate_act;
    a.w_f32 = w_type == MOE_SRC_F32;
    a.gate_f32 = gate_type == MOE_SRC_F32;
    a.r_scale = r_scale;
    a.y_scale = y_scale;
    a.rstd_post = rstd_post;
    a.rstd_pre = rstd_pre;
    a.T = T;
    a.d = d;
    a.dr = dr;
    a.dy = dy;
    a.dgate = gate_kind == MOE_GATE_CHANNEL ? nullptr : dgate;
    return launch_backward(a, r_type == MOE_SRC_F32, dw_post, dw_pre, gate_kind == MOE_GATE_CHANNEL ? dgate : nullptr, ws,
                           stream);
}
