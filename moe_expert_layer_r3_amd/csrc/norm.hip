// The norms around the layer: in front of it (moe_norm), and behind it together
// with the gate, the scaled residual sum and the next layer's norm (moe_join), and
// their gradients.
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
    float *part_post, *part_pre, *part_gate;  // [gridDim.x, d] each, NULL: not wanted
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

__device__ __forceinline__ float sigmoid32(float x) { return 1.0f / (1.0f + expf(-x)); }
// gate and its slope
__device__ __forceinline__ float gate_value(float x, int act) { return act == MOE_ACT_SIGMOID ? sigmoid32(x) : x; }
__device__ __forceinline__ float gate_slope(float x, int act) {
    return act == MOE_ACT_SIGMOID ? sigmoid32(x) * sigmoid32(-x) : 1.0f;
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

// One workgroup per row, the row read again for each sum.
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
                for (int j = 0; j < 8; ++j) s += v[j] * v[j];
            }
            rho_y = 1.0f / sqrtf(block_sum(s, lds, slot) / (float)d + a.eps);
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
                for (int j = 0; j < 8; ++j) {
                    const float n = a.w_post ? v[j] * rho_y * w[j] : v[j];
                    rv[j] = a.r_scale * rv[j] + a.y_scale * (gate_value(g[j], a.gate_act) * n);
                }
                store8(a.r_out, t * d + c, RF32, rv);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float q = stored(rv[j], RF32);
                s += q * q;
            }
        }
        if (!a.w_pre) continue;
        const float rho = 1.0f / sqrtf(block_sum(s, lds, slot) / (float)d + a.eps);
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

// One workgroup per row, the row read again for each sum; what is summed over the
// tokens goes into the workgroup's own row of the partial sums.
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
                    sn += dz * gate_value(g[j], a.gate_act) * n;   // dn * w_post * y * rho_y
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
                const float dz = a.y_scale * D[j], dn = dz * gate_value(g[j], a.gate_act);
                dg[j] = dz * n;
                p[j] = dn * yh;
                o[j] = a.w_post ? rho_y * (dn * w[j] - yh * sn) : dn;
            }
            if (a.dy) store8(a.dy, t * d + c, false, o);
            if (a.part_post) add8(a.part_post, c, p);
            if (a.part_gate) add8(a.part_gate, c, dg);
            if (a.gate_kind == MOE_GATE_FULL && a.dgate) {
#pragma unroll
                for (int j = 0; j < 8; ++j) dg[j] *= gate_slope(g[j], a.gate_act);
                store8(a.dgate, t * d + c, a.gate_f32, dg);
            }
        }
    }
}

// Sums of the partial rows, in order, 64 columns to a wave and 4 waves to the rows.
struct ColumnSum {
    const float* part;
    void* out;
    bool f32;
    const void* gate;  // != NULL: times the slope of the gate's activation
    bool gate_f32;
    int act;
};
struct ColumnSums {
    ColumnSum s[3];
    int64_t rows, d;
};
__global__ __launch_bounds__(256) void column_sums_kernel(ColumnSums a) {
    __shared__ float lds[4][64];
    const ColumnSum q = a.s[blockIdx.y];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.f;
    if (c < a.d)
        for (int64_t i = wave; i < a.rows; i += 4) s += q.part[i * a.d + c];
    lds[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= a.d) return;
    s = (lds[0][lane] + lds[1][lane]) + (lds[2][lane] + lds[3][lane]);
    if (q.gate) s *= gate_slope(load1(q.gate, c, q.gate_f32), q.act);
    store1(q.out, c, q.f32, s);
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

// workgroups of a backward launch, each with its partial sums: twice the compute
// units, fewer where the partial sums would pass 2^27 elements
int64_t backward_blocks(int64_t T, int64_t d) {
    int64_t n = 2 * (int64_t)num_cus();
    n = n < (1 << 27) / d ? n : (1 << 27) / d;
    return T < n ? T : n;
}
size_t backward_bytes(int64_t T, int64_t d, int sums) { return (size_t)backward_blocks(T, d) * d * sums * sizeof(float); }

dim3 row_grid(int64_t T) { return dim3((unsigned)(T < (1 << 22) ? T : 1 << 22)); }


// the weights' gradients from the partial sums (T == 0: zeros)
int launch_column_sums(ColumnSums& s, int n, hipStream_t stream) {
    if (n == 0) return MOE_OK;
    column_sums_kernel<<<dim3((unsigned)((s.d + 63) / 64), n), dim3(256), 0, stream>>>(s);
    MOE_LAUNCH_CHECK("column_sums_kernel");
    return MOE_OK;
}

int launch_backward(JoinGradArgs a, bool r_f32, void* dw_post, void* dw_pre, void* dw_gate, void* ws, hipStream_t stream) {
    const int64_t nb = backward_blocks(a.T, a.d);
    ColumnSums s = {};
    s.rows = nb;
    s.d = a.d;
    int n = 0;
    float* p = static_cast<float*>(ws);
    auto want = [&](void* out, bool f32, const void* gate, float** part) {
        if (!out) return;
        s.s[n++] = {p, out, f32, gate, a.gate_f32, a.gate_act};
        *part = p;
        p += nb * a.d;
    };
    want(dw_post, a.w_f32, nullptr, &a.part_post);
    want(dw_pre, a.w_f32, nullptr, &a.part_pre);
    want(dw_gate, a.gate_f32, a.gate, &a.part_gate);
    if (a.T > 0) {
        if (r_f32) join_backward_kernel<true><<<dim3((unsigned)nb), dim3(NT), 0, stream>>>(a);
        else join_backward_kernel<false><<<dim3((unsigned)nb), dim3(NT), 0, stream>>>(a);
        MOE_LAUNCH_CHECK("join_backward_kernel");
    } else {
        for (int i = 0; i < n; ++i) s.s[i].gate = nullptr;
    }
    return launch_column_sums(s, n, stream);
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
    if (x_type == MOE_SRC_F32) join_kernel<true><<<row_grid(T), dim3(NT), 0, stream>>>(a);
    else join_kernel<false><<<row_grid(T), dim3(NT), 0, stream>>>(a);
    MOE_LAUNCH_CHECK("join_kernel");
    return MOE_OK;
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
    if (r_type == MOE_SRC_F32) join_kernel<true><<<row_grid(T), dim3(NT), 0, stream>>>(a);
    else join_kernel<false><<<row_grid(T), dim3(NT), 0, stream>>>(a);
    MOE_LAUNCH_CHECK("join_kernel");
    return MOE_OK;
}

extern "C" int moe_join_backward_workspace(int64_t T, int64_t d, size_t* bytes) {
    clear_error();
    MOE_REQUIRE(bytes, MOE_ERR_NULL, "join_backward_workspace: NULL bytes");
    if (const int rc = check_rows("join_backward_workspace", T, d)) return rc;
    *bytes = backward_bytes(T, d, 3);
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
    const int sums = (dw_post != nullptr) + (dw_pre != nullptr) + (dgate && gate_kind == MOE_GATE_CHANNEL);
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
