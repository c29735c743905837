// Routing by scores: the choice of experts from softmax or sigmoid scores with a
// balance bias and groups, its replay from a record, its gradient, and the update
// of the bias.
#include "common.hpp"
#include "gate_parts.hpp"
#include "route_keys.hpp"

namespace moe {
namespace {

constexpr int MAX_E = 1024;

struct ScoreArgs {
    const void* logits;
    const float* bias;
    int64_t T;
    int E, k, groups, top_groups, group_top;
    float scale;
    int32_t* ids;
    float* w;
    int32_t* load;
    int32_t* rec;  // of this layer and first token
    int64_t rec_stride;
};

// ---------------------------------------------------------------- logits
template <bool F32>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
    if constexpr (F32) return static_cast<const float*>(p)[i];
    else return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}
// -inf and the type's lowest value mask an expert
template <bool F32>
__device__ __forceinline__ bool is_masked(float l) {
    return l <= (F32 ? -3.402823466e38f : -3.389531389e38f);
}
__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// Maximum and sum of exponentials of a row that a wave holds, masked experts left
// out. A NaN anywhere makes the sum NaN (fmaxf passes over it, exp does not).
struct RowStat {
    double m, inv;
};
template <bool F32, int VPL>
__device__ __forceinline__ RowStat row_stat(const float (&l)[VPL], int lane, int E) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (lane + 64 * i < E && !is_masked<F32>(l[i])) m = fmaxf(m, l[i]);
    m = group_max<64>(m);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (lane + 64 * i < E && !is_masked<F32>(l[i])) sum += exp((double)l[i] - (double)m);
    sum = wave_sum64(sum);
    return {(double)m, sum == 0.0 ? 0.0 : 1.0 / sum};
}
template <bool F32, bool SIGMOID>
__device__ __forceinline__ double score(float l, RowStat st) {
    if (is_masked<F32>(l)) return 0.0;
    if constexpr (SIGMOID) return sigmoid64(l);
    else return exp((double)l - st.m) * st.inv;
}

// Weights of the chosen experts: lane j < k of a group of WIDTH lanes has logit l
// (masked: the expert has no weight) and, without renorm, score s. Sums go in
// ascending slot order.
template <bool F32, bool SIGMOID, bool RENORM, int WIDTH>
__device__ __forceinline__ double share(float l, double s, int lane, int k) {
    if constexpr (!RENORM) return s;
    if constexpr (!SIGMOID) {
        float m = lane < k && !is_masked<F32>(l) ? l : -INFINITY;
        m = group_max<WIDTH>(m);
        s = is_masked<F32>(l) ? 0.0 : exp((double)l - (double)m);
    }
    double sum = 0.0;
    for (int j = 0; j < k; ++j) sum += __shfl(s, j, WIDTH);
    return sum == 0.0 ? 0.0 : s / sum;
}

// ---------------------------------------------------------------- choice

// One wave per token: lane l holds experts l, l + 64, ...; k rounds of a wave-wide
// maximum over the keys of the groups that stay.
template <bool F32, bool SIGMOID, bool RENORM, int VPL>
__global__ __launch_bounds__(256) void score_topk_kernel(ScoreArgs a) {
    __shared__ float group_c[4][64 * VPL];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int E = a.E, k = a.k;
    for (int64_t row0 = (int64_t)blockIdx.x * 4; row0 < a.T; row0 += (int64_t)gridDim.x * 4) {
        const int64_t row = row0 + wave;
        const bool live = row < a.T;
        const int64_t base = (live ? row : 0) * E;
        float l[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 64 * i;
            l[i] = e < E ? logit<F32>(a.logits, base + e) : 0.f;
        }
        RowStat st = {0.0, 0.0};
        if constexpr (!SIGMOID) st = row_stat<F32, VPL>(l, lane, E);
        uint64_t key[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 64 * i;
            key[i] = 0ull;
            if (e < E) {
                float c = (float)score<F32, SIGMOID>(l[i], st);
                if (a.bias) c += a.bias[e];
                if (is_masked<F32>(l[i])) c = -INFINITY;
                key[i] = route_key(c, e);
                group_c[wave][e] = c == c ? c : -INFINITY;
            }
        }
        if (a.groups > 1) {
            __syncthreads();
            // 64 / GP lanes to a group, GP the power of two that holds the groups
            int gp = 1;
            while (gp < a.groups) gp <<= 1;
            const int lpg = 64 / gp, S = E / a.groups;
            const int g = lane / lpg, sub = lane % lpg;
            float t1 = -INFINITY, t2 = -INFINITY;
            if (g < a.groups) {
                for (int i = sub; i < S; i += lpg) {
                    const float v = group_c[wave][g * S + i];
                    t2 = fmaxf(t2, fminf(t1, v));
                    t1 = fmaxf(t1, v);
                }
            }
            for (int m = 1; m < lpg; m <<= 1) {
                const float o1 = __shfl_xor(t1, m), o2 = __shfl_xor(t2, m);
                t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
                t1 = fmaxf(t1, o1);
            }
            const float v = a.group_top == 2 && t2 > -INFINITY ? t1 + t2 : t1;
            int ahead = 0;
            for (int o = 0; o < a.groups; ++o) {
                const float ov = __shfl(v, o * lpg);
                ahead += (ov > v) | ((ov == v) & (o < g));
            }
            const uint64_t stay = __ballot(g < a.groups && ahead < a.top_groups);
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int e = lane + 64 * i;
                if (e < E && !((stay >> (e / S * lpg)) & 1ull)) key[i] = 0ull;
            }
            __syncthreads();  // the next row's values
        }
        uint64_t thr = ~0ull, mine = 0ull;
        for (int s = 0; s < k; ++s) {
            uint64_t b = 0ull;
#pragma unroll
            for (int i = 0; i < VPL; ++i) b = (key[i] < thr && key[i] > b) ? key[i] : b;
#pragma unroll
            for (int m = 32; m >= 1; m >>= 1) {
                const uint64_t o = __shfl_xor(b, m);
                b = o > b ? o : b;
            }
            thr = b;
            if (lane == s) mine = b;
        }
        const int id = lane < k ? route_key_id(mine) : 0;
        const float ls = logit<F32>(a.logits, base + id);
        const double h = share<F32, SIGMOID, RENORM, 64>(ls, score<F32, SIGMOID>(ls, st), lane, k);
        if (live && lane < k) {
            a.ids[row * k + lane] = id;
            a.w[row * k + lane] = (float)((double)a.scale * h);
            if (a.rec) a.rec[(int64_t)lane * a.rec_stride + row] = id;
            if (a.load) atomicAdd(a.load + id, 1);
        }
    }
}

// ---------------------------------------------------------------- replay

// 16 lanes per token where the chosen logits alone decide its weights.
template <bool F32, bool SIGMOID, bool RENORM>
__global__ __launch_bounds__(256) void score_replay_kernel(ScoreArgs a, int32_t* status) {
    const int lane = threadIdx.x & 15, E = a.E, k = a.k;
    for (int64_t row0 = (int64_t)blockIdx.x * 16; row0 < a.T; row0 += (int64_t)gridDim.x * 16) {
        const int64_t row = row0 + (threadIdx.x >> 4);
        const bool live = row < a.T;
        const int64_t t = live ? row : 0;
        const int id = lane < k ? a.rec[(int64_t)lane * a.rec_stride + t] : 0;
        int bad = lane < k && (id < 0 || id >= E), dup = 0;
        for (int j = 0; j < k; ++j) {
            const int o = __shfl(id, j, 16);
            dup |= lane < k && j < lane && o == id;
        }
#pragma unroll
        for (int m = 8; m >= 1; m >>= 1) {
            bad |= __shfl_xor(bad, m, 16);
            dup |= __shfl_xor(dup, m, 16);
        }
        const float l = logit<F32>(a.logits, t * E + (bad ? 0 : id));
        const double h = share<F32, SIGMOID, RENORM, 16>(l, score<F32, SIGMOID>(l, RowStat{0.0, 0.0}), lane, k);
        if (live && lane < k) {
            a.ids[row * k + lane] = id;
            a.w[row * k + lane] = bad ? 0.f : (float)((double)a.scale * h);
        }
        const int flags = (bad ? MOE_FLAG_BAD_ID : 0) | (dup ? MOE_FLAG_DUP_ID : 0);
        if (live && lane == 0 && flags && status) atomicOr(status, flags);
    }
}

// One wave per token where the whole row does (softmax without renorm).
template <bool F32, int VPL>
__global__ __launch_bounds__(256) void score_replay_row_kernel(ScoreArgs a, int32_t* status) {
    const int lane = threadIdx.x & 63, E = a.E, k = a.k;
    const int64_t step = (int64_t)gridDim.x * 4;
    for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < a.T; row += step) {
        float l[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 64 * i;
            l[i] = e < E ? logit<F32>(a.logits, row * E + e) : 0.f;
        }
        const RowStat st = row_stat<F32, VPL>(l, lane, E);
        const int id = lane < k ? a.rec[(int64_t)lane * a.rec_stride + row] : 0;
        const bool bad = __ballot(lane < k && (id < 0 || id >= E)) != 0;
        bool dup = false;
        for (int j = 0; j < k; ++j) {
            const int o = __shfl(id, j);
            dup |= lane < k && j < lane && o == id;
        }
        dup = __ballot(dup) != 0;
        if (lane < k) {
            const float ls = logit<F32>(a.logits, row * E + (bad ? 0 : id));
            a.ids[row * k + lane] = id;
            a.w[row * k + lane] = bad ? 0.f : (float)((double)a.scale * score<F32, false>(ls, st));
        }
        const int flags = (bad ? MOE_FLAG_BAD_ID : 0) | (dup ? MOE_FLAG_DUP_ID : 0);
        if (lane == 0 && flags && status) atomicOr(status, flags);
    }
}

// ---------------------------------------------------------------- gradient

struct ScoreGradArgs {
    const float* d_w;  // or the partials and where each pair's row is
    const float* part;
    const int32_t* pair_row;
    int ngroups;
    const void* logits;
    const int32_t* ids;
    int64_t T;
    int E, k;
    float scale;
    float* d_gate;
    void* d_logits;
};

// One wave per token: the first k lanes have a slot each; every lane then writes
// its elements of the row, each the sum of the slots that hold its expert.
template <bool F32, bool SIGMOID, bool RENORM, bool PARTS, int VPL>
__global__ __launch_bounds__(256) void score_backward_kernel(ScoreGradArgs a) {
    const int lane = threadIdx.x & 63, E = a.E, k = a.k;
    const int64_t step = (int64_t)gridDim.x * 4;
    for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < a.T; row += step) {
        float dw = 0.f;
        if constexpr (PARTS) {
            if (lane < k) {
                const int r = a.pair_row[row * k + lane];
                if (r >= 0)
                    for (int g = 0; g < a.ngroups; ++g) dw += a.part[(int64_t)r * MOE_GATE_PARTS + g];
                a.d_gate[row * k + lane] = dw;
            }
        } else if (lane < k) {
            dw = a.d_w[row * k + lane];
        }
        const int id = lane < k ? a.ids[row * k + lane] : 0;
        const bool bad = __ballot(lane < k && (id < 0 || id >= E)) != 0;
        float l[VPL];
        RowStat st = {0.0, 0.0};
        if constexpr (!SIGMOID && !RENORM) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int e = lane + 64 * i;
                l[i] = e < E ? logit<F32>(a.logits, row * E + e) : 0.f;
            }
            st = row_stat<F32, VPL>(l, lane, E);
        }
        const float ls = logit<F32>(a.logits, row * E + (bad ? 0 : id));
        const double s = score<F32, SIGMOID>(ls, st);
        const double h = share<F32, SIGMOID, RENORM, 64>(ls, s, lane, k);
        double dot = 0.0;
        if constexpr (RENORM || !SIGMOID) {
            const double p = h * (double)dw;
            for (int j = 0; j < k; ++j) dot += __shfl(p, j);
        }
        // a slot's gradient of its own logit (softmax without renorm: before the row's part)
        double c = (double)a.scale * h * ((double)dw - (RENORM ? dot : 0.0));
        if constexpr (SIGMOID) c = is_masked<F32>(ls) ? 0.0 : c * sigmoid64(-(double)ls);
        if (lane >= k || bad) c = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 64 * i;
            double acc = 0.0;
            for (int j = 0; j < k; ++j) {
                const int o = __shfl(id, j);
                const double oc = __shfl(c, j);
                if (o == e) acc += oc;
            }
            if constexpr (!SIGMOID && !RENORM) {
                if (!bad && e < E) acc -= score<F32, false>(l[i], st) * (double)a.scale * dot;
            }
            if (e < E) {
                if constexpr (F32) static_cast<float*>(a.d_logits)[row * E + e] = (float)acc;
                else static_cast<uint16_t*>(a.d_logits)[row * E + e] = (uint16_t)f32_to_bf16((float)acc);
            }
        }
    }
}

// ---------------------------------------------------------------- bias

__global__ __launch_bounds__(1024) void balance_bias_kernel(int32_t* load, const float* bias, int E, float step, int clear,
                                                            float* out) {
    __shared__ int64_t part[16];
    const int e = threadIdx.x;
    const int64_t n = e < E ? load[e] : 0;
    int64_t sum = n;
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) sum += __shfl_xor(sum, m);
    if ((e & 63) == 0) part[e >> 6] = sum;
    __syncthreads();
    int64_t total = 0;
    for (int i = 0; i < 16; ++i) total += part[i];
    if (e >= E) return;
    const int64_t own = n * E;
    out[e] = bias[e] + (total > own ? step : total < own ? -step : 0.f);
    if (clear) load[e] = 0;
}

// ---------------------------------------------------------------- host
int check_scored(const char* what, int64_t T, int32_t E, int32_t k, int32_t type, int32_t score, float scale) {
    MOE_REQUIRE(type == MOE_SRC_F32 || type == MOE_SRC_BF16, MOE_ERR_UNSUPPORTED, "%s: logits type %d", what, type);
    MOE_REQUIRE(score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID, MOE_ERR_UNSUPPORTED, "%s: score %d", what, score);
    MOE_REQUIRE(T >= 0 && T <= (1 << 30), MOE_ERR_SHAPE, "%s: T=%lld outside [0, 2^30]", what, (long long)T);
    MOE_REQUIRE(E >= 1 && E <= MAX_E, MOE_ERR_SHAPE, "%s: E=%d outside [1, 1024]", what, E);
    MOE_REQUIRE(k >= 1 && k <= MAXK && k <= E, MOE_ERR_SHAPE, "%s: k=%d outside [1, min(16, E)]", what, k);
    MOE_REQUIRE(scale - scale == 0.f, MOE_ERR_SHAPE, "%s: scale is not finite", what);
    return MOE_OK;
}
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
dim3 row_blocks(int64_t T, int per) {
    const int64_t n = (T + per - 1) / per, most = 1 << 20;
    return dim3((unsigned)(n < most ? n : most));
}

// f(F32, SIGMOID, RENORM as integral constants)
template <typename F>
void with_forms(int32_t type, int32_t score, int32_t renorm, F&& f) {
    auto renorm_of = [&](auto t, auto s) {
        if (renorm) f(t, s, std::true_type{});
        else f(t, s, std::false_type{});
    };
    auto score_of = [&](auto t) {
        if (score == MOE_SCORE_SIGMOID) renorm_of(t, std::true_type{});
        else renorm_of(t, std::false_type{});
    };
    if (type == MOE_SRC_F32) score_of(std::true_type{});
    else score_of(std::false_type{});
}
// f(values per lane that hold E experts in 64 lanes)
template <typename F>
void with_vpl(int E, F&& f) {
    if (E <= 64) f(std::integral_constant<int, 1>{});
    else if (E <= 256) f(std::integral_constant<int, 4>{});
    else f(std::integral_constant<int, 16>{});
}

int launch_backward(ScoreGradArgs a, int32_t type, int32_t score, int32_t renorm, bool parts, hipStream_t stream) {
    with_forms(type, score, renorm, [&](auto t, auto s, auto r) {
        with_vpl(a.E, [&](auto v) {
            if (parts)
                score_backward_kernel<t.value, s.value, r.value, true, v.value><<<row_blocks(a.T, 4), 256, 0, stream>>>(a);
            else
                score_backward_kernel<t.value, s.value, r.value, false, v.value><<<row_blocks(a.T, 4), 256, 0, stream>>>(a);
        });
    });
    MOE_LAUNCH_CHECK("score_backward_kernel");
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_route_scored(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t k, int32_t score,
                                const float* bias, int32_t groups, int32_t top_groups, int32_t group_top, int32_t renorm,
                                float scale, int32_t* ids, float* w, int32_t* load, int32_t* rec, int32_t n_layers,
                                int64_t seq_len, int32_t layer, int64_t s0, hipStream_t stream) {
    clear_error();
    if (const int rc = check_scored("route_scored", T, E, k, logits_type, score, scale)) return rc;
    MOE_REQUIRE(groups >= 1 && groups <= 64 && E % groups == 0, MOE_ERR_SHAPE,
                "route_scored: groups=%d: 1 to 64 that divide E=%d", groups, E);
    MOE_REQUIRE(top_groups >= 1 && top_groups <= groups && k <= top_groups * (E / groups), MOE_ERR_SHAPE,
                "route_scored: top_groups=%d: up to groups=%d, holding at least k=%d experts", top_groups, groups, k);
    MOE_REQUIRE(group_top == 1 || group_top == 2, MOE_ERR_SHAPE, "route_scored: group_top=%d: 1 or 2", group_top);
    if (rec) {
        MOE_REQUIRE(n_layers >= 1 && layer >= 0 && layer < n_layers, MOE_ERR_SHAPE,
                    "route_scored: layer %d outside [0, %d)", layer, n_layers);
        MOE_REQUIRE(s0 >= 0 && seq_len >= T && s0 <= seq_len - T, MOE_ERR_SHAPE,
                    "route_scored: tokens [%lld, %lld + T) outside seq_len %lld", (long long)s0, (long long)s0,
                    (long long)seq_len);
    }
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(logits && ids && w, MOE_ERR_NULL, "route_scored: NULL logits/ids/w");
    MOE_REQUIRE(aligned16(logits), MOE_ERR_SHAPE, "route_scored: logits: 16-byte aligned");
    ScoreArgs a = {logits, bias, T, E, k, groups, top_groups == groups ? 1 : top_groups, group_top, scale, ids, w, load,
                   rec ? rec + (int64_t)layer * k * seq_len + s0 : nullptr, seq_len};
    if (top_groups == groups) a.groups = 1;  // every group stays
    with_forms(logits_type, score, renorm, [&](auto t, auto s, auto r) {
        with_vpl(E, [&](auto v) {
            score_topk_kernel<t.value, s.value, r.value, v.value><<<row_blocks(T, 4), 256, 0, stream>>>(a);
        });
    });
    MOE_LAUNCH_CHECK("score_topk_kernel");
    return MOE_OK;
}

extern "C" int moe_replay_scored(const int32_t* rec, int32_t n_layers, int32_t k, int64_t seq_len, int32_t layer,
                                 int64_t s0, int64_t T, const void* logits, int32_t logits_type, int32_t E, int32_t score,
                                 int32_t renorm, float scale, int32_t* ids, float* w, int32_t* dev_status,
                                 hipStream_t stream) {
    clear_error();
    if (const int rc = check_scored("replay_scored", T, E, k, logits_type, score, scale)) return rc;
    MOE_REQUIRE(n_layers >= 1 && layer >= 0 && layer < n_layers, MOE_ERR_SHAPE, "replay_scored: layer %d outside [0, %d)",
                layer, n_layers);
    MOE_REQUIRE(s0 >= 0 && seq_len >= T && s0 <= seq_len - T, MOE_ERR_SHAPE,
                "replay_scored: tokens [%lld, %lld + T) outside seq_len %lld", (long long)s0, (long long)s0,
                (long long)seq_len);
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(rec && logits && ids && w, MOE_ERR_NULL, "replay_scored: NULL rec/logits/ids/w");
    MOE_REQUIRE(aligned16(logits), MOE_ERR_SHAPE, "replay_scored: logits: 16-byte aligned");
    ScoreArgs a = {};
    a.logits = logits;
    a.T = T;
    a.E = E;
    a.k = k;
    a.scale = scale;
    a.ids = ids;
    a.w = w;
    a.rec = const_cast<int32_t*>(rec) + (int64_t)layer * k * seq_len + s0;
    a.rec_stride = seq_len;
    with_forms(logits_type, score, renorm, [&](auto t, auto s, auto r) {
        if constexpr (!s.value && !r.value)
            with_vpl(E, [&](auto v) {
                score_replay_row_kernel<t.value, v.value><<<row_blocks(T, 4), 256, 0, stream>>>(a, dev_status);
            });
        else
            score_replay_kernel<t.value, s.value, r.value><<<row_blocks(T, 16), 256, 0, stream>>>(a, dev_status);
    });
    MOE_LAUNCH_CHECK("score_replay_kernel");
    return MOE_OK;
}

extern "C" int moe_route_scored_backward(const float* d_w, const void* logits, int32_t logits_type, const int32_t* ids,
                                         int64_t T, int32_t k, int32_t E, int32_t score, int32_t renorm, float scale,
                                         void* d_logits, hipStream_t stream) {
    clear_error();
    if (const int rc = check_scored("route_scored_backward", T, E, k, logits_type, score, scale)) return rc;
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(d_w && logits && ids && d_logits, MOE_ERR_NULL, "route_scored_backward: NULL argument");
    MOE_REQUIRE(aligned16(logits) && aligned16(d_logits), MOE_ERR_SHAPE,
                "route_scored_backward: logits and d_logits: 16-byte aligned");
    return launch_backward({d_w, nullptr, nullptr, 0, logits, ids, T, E, k, scale, nullptr, d_logits}, logits_type, score,
                           renorm, false, stream);
}

extern "C" int moe_route_scored_backward_parts(const float* gate_part, const int32_t* pair_row, int64_t row_cap, int32_t d,
                                               const void* logits, int32_t logits_type, const int32_t* ids, int64_t T,
                                               int32_t k, int32_t E, int32_t score, int32_t renorm, float scale,
                                               float* d_gate, void* d_logits, hipStream_t stream) {
    clear_error();
    if (const int rc = check_scored("route_scored_backward_parts", T, E, k, logits_type, score, scale)) return rc;
    MOE_REQUIRE(d > 0 && d % 128 == 0, MOE_ERR_SHAPE, "route_scored_backward_parts: d=%d must be a multiple of 128", d);
    MOE_REQUIRE(row_cap >= 0, MOE_ERR_SHAPE, "route_scored_backward_parts: bad row_cap");
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(pair_row && logits && ids && d_gate && d_logits && (row_cap == 0 || gate_part), MOE_ERR_NULL,
                "route_scored_backward_parts: NULL argument");
    MOE_REQUIRE(aligned16(logits) && aligned16(d_logits), MOE_ERR_SHAPE,
                "route_scored_backward_parts: logits and d_logits: 16-byte aligned");
    return launch_backward({nullptr, gate_part, pair_row, gate_groups(d), logits, ids, T, E, k, scale, d_gate, d_logits},
                           logits_type, score, renorm, true, stream);
}

extern "C" int moe_balance_bias(int32_t* load, const float* bias, int32_t E, float step, int32_t clear, float* bias_out,
                                hipStream_t stream) {
    clear_error();
    MOE_REQUIRE(E >= 1 && E <= MAX_E, MOE_ERR_SHAPE, "balance_bias: E=%d outside [1, 1024]", E);
    MOE_REQUIRE(step - step == 0.f, MOE_ERR_SHAPE, "balance_bias: step is not finite");
    MOE_REQUIRE(load && bias && bias_out, MOE_ERR_NULL, "balance_bias: NULL load/bias/bias_out");
    balance_bias_kernel<<<dim3(1), dim3(1024), 0, stream>>>(load, bias, E, step, clear, bias_out);
    MOE_LAUNCH_CHECK("balance_bias_kernel");
    return MOE_OK;
}
