// Routing by scores: the choice of experts from softmax or sigmoid scores with a
// balance bias and groups, its replay from a record, its gradient, and the update
// of the bias.
#include <type_traits>

#include "common.hpp"
#include "gate_parts.hpp"
#include "route_keys.hpp"

namespace moe {
namespace {

constexpr int MAX_E = 1024;
constexpr float LOW = -3.402823466e38f;  // below every number that counts

struct ScoreArgs {
    const void* logits;
    const float* bias;
    int64_t T;
    int E, k, groups, top_groups, group_top;
    bool renorm;
    float scale;
    int lds_wave, lds_row;     // floats of LDS for each wave, and for each of its rows
    int inv_S;                 // ceil(2^22 / (E / groups)): e * inv_S >> 22 is e's group
    int group_bits, lpr_bits;  // logarithms of the power of two that holds the groups, and of a row's lanes
    int spread;                // a group's lanes start at its four group * spread mod 8
    int32_t* ids;
    float* w;
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

// For weights and gradients, which are rounded to 32 bits: exp(x), x <= 0, from a polynomial of
// degree 10, 1 + r + r^2 g(r) with g interpolated at the Chebyshev nodes of
// [-ln 2 / 2, ln 2 / 2] (off by 2^-49 of itself; Taylor's of that degree would be by 2^-41, which
// shows where a gradient is a difference), a reciprocal from the hardware's and two Newton
// steps (2^-50): a third of the instructions of the exact ones.
__device__ __forceinline__ double exp_poly(double r) {
    double p = 2.761379556582631e-07;
    p = __builtin_fma(p, r, 2.7625102018960324e-06);
    p = __builtin_fma(p, r, 2.4801536409043718e-05);
    p = __builtin_fma(p, r, 0.0001984120875696787);
    p = __builtin_fma(p, r, 0.0013888888905871355);
    p = __builtin_fma(p, r, 0.008333333353717168);
    p = __builtin_fma(p, r, 0.041666666666651364);
    p = __builtin_fma(p, r, 0.16666666666648303);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_fma(p, r, 1.0);
}
__device__ __forceinline__ double exp_near(double x) {
    const double n = __builtin_rint(x * 1.4426950408889634);
    const double r = __builtin_fma(-n, 2.319046813846300e-17, __builtin_fma(-n, 0.6931471805599453, x));
    // (a far x: r is up to 2^-53 |x|, the polynomial below 2^760, and the result 0)
    return __builtin_amdgcn_ldexp(exp_poly(r), (int)__builtin_fmax(n, -2000.0));
}
// The same for a row's sum, in three operations less: the whole number comes from adding 1.5 2^52
// (in its lowest bits), ln 2 is one constant (off by 2^-55 of itself, 2^-50 of a term at x = -30),
// and x stops at -800, where terms are 0 next to the largest one's 1. For rows of
// finite or masked logits alone: a NaN does not go through. Times 2^UP, whose exponent comes with
// the whole number.
template <int UP = 0>
__device__ __forceinline__ double exp_term(double x) {
    constexpr double whole = 6755399441055744.0 + UP;
    x = __builtin_fmax(x, -800.0);
    const double t = __builtin_fma(x, 1.4426950408889634, whole);
    const int n = (int)(uint32_t)__builtin_bit_cast(uint64_t, t);
    return __builtin_amdgcn_ldexp(exp_poly(__builtin_fma(whole - t, 0.6931471805599453, x)), n);
}
__device__ __forceinline__ double inverse_near(double x) {  // of a number from 1 to 2
    double y = __builtin_amdgcn_rcp(x);
    y = __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
    return __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
}
// From exp(-|l|), so that no reciprocal leaves the normal range; 0 where exp(-l) passes the
// largest double (at 709.7827 as a float), as it makes 1 / (1 + exp(-l)) in 64 bits.
__device__ __forceinline__ double sigmoid_near(float l) {
    const float far = fabsf(l);
    const double e = exp_near((double)(far >= 709.7827f ? -1000.f : -far)), q = inverse_near(1.0 + e);
    return (l < 0.f ? e : 1.0) * q;
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// A value of the lane that a butterfly step over LPR lanes pairs this one with.
template <int CTRL>
__device__ __forceinline__ float dpp32(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int STEP>
__device__ __forceinline__ float partner(float v) {
    if constexpr (STEP == 0) return dpp32<0xB1>(v);         // lane xor 1
    else if constexpr (STEP == 1) return dpp32<0x4E>(v);    // lane xor 2
    else if constexpr (STEP == 2) return dpp32<0x141>(v);   // mirrored in 8
    else if constexpr (STEP == 3) return dpp32<0x140>(v);   // mirrored in 16
    else return __shfl_xor(v, 16);
}
template <int STEP>
__device__ __forceinline__ double partner(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const float lo = partner<STEP>(__uint_as_float((uint32_t)b)), hi = partner<STEP>(__uint_as_float((uint32_t)(b >> 32)));
    return __builtin_bit_cast(double, ((uint64_t)__float_as_uint(hi) << 32) | __float_as_uint(lo));
}
template <int LPR, typename T, typename F>
__device__ __forceinline__ T team_reduce(T v, F&& f) {
    v = f(v, partner<0>(v));
    v = f(v, partner<1>(v));
    v = f(v, partner<2>(v));
    if constexpr (LPR >= 16) v = f(v, partner<3>(v));
    if constexpr (LPR >= 32) v = f(v, partner<4>(v));
    return v;
}
template <int LPR, typename T>
__device__ __forceinline__ T team_sum(T v) {
    return team_reduce<LPR>(v, [](T x, T y) { return x + y; });
}
template <int LPR>
__device__ __forceinline__ float team_max(float v) {
    return team_reduce<LPR>(v, [](float x, float y) { return fmaxf(x, y); });
}

// exp by the hardware's exp2: off by (2 |x| + 3) 2^-24 of itself at most (the
// difference x, its product and exp2 are rounded).
__device__ __forceinline__ float exp32(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

// Maximum and sum of exponentials of a row that a wave holds, masked experts left
// out. A NaN anywhere makes the sum NaN (fmaxf passes over it, exp does not).
// EXACT: for the choice, which is defined by these values. Otherwise the terms are
// exp_near's, for weights and gradients: the same terms in every kernel, added in 64 bits in an
// order that goes by the lanes that hold a row, so that a weight made by two kernels can
// differ where it lies next to the border of two fp32 values.
struct RowStat {
    double m, inv;
};
template <bool F32, bool EXACT, int VPL>
__device__ __forceinline__ RowStat row_stat(const float (&l)[VPL], int lane, int E) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (lane + 64 * i < E && !is_masked<F32>(l[i])) m = fmaxf(m, l[i]);
    m = group_max<64>(m);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (lane + 64 * i < E && !is_masked<F32>(l[i])) {
            if constexpr (EXACT) sum += exp((double)l[i] - (double)m);
            else sum += exp_near((double)l[i] - (double)m);
        }
    sum = wave_sum64(sum);
    return {(double)m, sum == 0.0 ? 0.0 : 1.0 / sum};
}
template <bool F32, bool SIGMOID, bool EXACT = false>
__device__ __forceinline__ double score(float l, RowStat st) {
    if (is_masked<F32>(l)) return 0.0;
    if constexpr (SIGMOID) return EXACT ? sigmoid64(l) : sigmoid_near(l);
    else return (EXACT ? exp((double)l - st.m) : exp_near((double)l - st.m)) * st.inv;
}

// Weights of the chosen experts: lane j < k of a group of WIDTH lanes has logit l
// (masked: the expert has no weight) and, without renorm, score s. The sum is a
// butterfly over eight or sixteen lanes, zeros past the k-th: the same wherever the
// slots stand in lanes of their own.
template <bool F32, bool SIGMOID, int WIDTH>
__device__ __forceinline__ double share(float l, double s, int lane, int k, bool renorm) {
    if (!renorm) return s;
    if constexpr (!SIGMOID) {
        float m = lane < k && !is_masked<F32>(l) ? l : -INFINITY;
        m = team_max<WIDTH>(m);
        s = is_masked<F32>(l) ? 0.0 : exp_near((double)l - (double)m);
    }
    const double sum = team_sum<WIDTH>(lane < k ? s : 0.0);
    return sum == 0.0 ? 0.0 : s / sum;
}

// Accesses of a wave's own LDS region before this point are done before those behind it.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------- choice

// Sorting networks over keys as doubles: one v_max_f64 and one v_min_f64 an exchange
// (written out: the compiler would make each key canonical first, which they are).
__device__ __forceinline__ double kmax(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ double kmin(double a, double b) {
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
// the largest over the wave, in every lane
__device__ __forceinline__ double wave_kmax(double v) {
    v = kmax(v, partner<0>(v));
    v = kmax(v, partner<1>(v));
    v = kmax(v, partner<2>(v));
    v = kmax(v, partner<3>(v));
    uint64_t b = __builtin_bit_cast(uint64_t, v);
    auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
    auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
    v = kmax(__builtin_bit_cast(double, ((uint64_t)hi[0] << 32) | lo[0]), __builtin_bit_cast(double, ((uint64_t)hi[1] << 32) | lo[1]));
    b = __builtin_bit_cast(uint64_t, v);
    lo = __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false);
    hi = __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
    return kmax(__builtin_bit_cast(double, ((uint64_t)hi[0] << 32) | lo[0]), __builtin_bit_cast(double, ((uint64_t)hi[1] << 32) | lo[1]));
}

// One row by a whole wave, as it is defined: scores in 64 bits, rounded. Lane l holds
// experts l, l + 64, ...; k rounds of a wave-wide maximum over the keys of the groups
// that stay, as doubles (route_dkey). lds: E floats of this wave. Rare where the kernel below calls it, and a
// function of its own so that its registers are not the caller's. Bound by its chain: k
// rounds of a maximum over 64 lanes, 64-bit exponentials in front: 5.3 us for one row of 256.
typedef const __attribute__((address_space(4))) ScoreArgs* KernelArgs;
typedef __attribute__((address_space(3))) float* LdsFloats;
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
    return ((uint64_t)hi << 32) | lo;
}
template <bool F32, bool SIGMOID, int VPL>
__device__ __attribute__((noinline)) void choose_exactly(KernelArgs args, int64_t row_, LdsFloats lds) {
    const __attribute__((address_space(4))) ScoreArgs& a = *(KernelArgs)uniform((uint64_t)args);
    const int64_t row = (int64_t)uniform((uint64_t)row_);
    const int lane = threadIdx.x & 63, E = a.E, k = a.k;
    const int64_t base = row * E;
    float l[VPL], bias[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = logit<F32>(a.logits, base + min(lane + 64 * i, E - 1));
#pragma unroll
    for (int i = 0; i < VPL; ++i) bias[i] = a.bias ? a.bias[min(lane + 64 * i, E - 1)] : 0.f;
    RowStat st = {0.0, 0.0};
    if constexpr (!SIGMOID) st = row_stat<F32, true, VPL>(l, lane, E);
    double key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 64 * i;
        key[i] = 0.0;
        if (e < E) {
            float c = (float)score<F32, SIGMOID, true>(l[i], st);
            if (a.bias) c += bias[i];
            if (is_masked<F32>(l[i])) c = -INFINITY;
            key[i] = route_dkey(c, e);
            if (a.groups > 1) lds[e] = c == c ? c : -INFINITY;
        }
    }
    if (a.groups > 1) {
        wave_sync();
        // 64 / GP lanes to a group, GP the power of two that holds the groups
        const int shift = 6 - a.group_bits, lpg = 1 << shift, S = E / a.groups;
        const int g = lane >> shift, sub = lane & (lpg - 1);
        float t1 = -INFINITY, t2 = -INFINITY;
        if (g < a.groups) {
#pragma unroll 4
            for (int i = sub; i < S; i += lpg) {
                const float v = lds[g * S + i];
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
#pragma unroll 8
        for (int o = 0; o < a.groups; ++o) {
            const float ov = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), o << shift));
            ahead += (ov > v) | ((ov == v) & (o < g));
        }
        const uint64_t stay = __ballot(g < a.groups && ahead < a.top_groups);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 64 * i;
            if (e < E && !((stay >> ((uint32_t)e * (uint32_t)a.inv_S >> 22 << shift)) & 1ull)) key[i] = 0.0;
        }
        wave_sync();  // the next row's values
    }
    double thr = INFINITY, mine = 0.0;
    for (int s = 0; s < k; ++s) {
        double b = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) b = key[i] < thr ? kmax(key[i], b) : b;
        thr = wave_kmax(b);
        if (lane == s) mine = thr;
    }
    const int id = lane < k ? route_dkey_id(mine) : 0;
    const float ls = logit<F32>(a.logits, base + id);
    if constexpr (!SIGMOID)
        if (!a.renorm) st = row_stat<F32, false, VPL>(l, lane, E);
    const double h = share<F32, SIGMOID, 16>(ls, score<F32, SIGMOID>(ls, st), lane, k, a.renorm);
    if (lane < k) {
        a.ids[row * k + lane] = id;
        a.w[row * k + lane] = (float)((double)a.scale * h);
        if (a.rec) a.rec[(int64_t)lane * a.rec_stride + row] = id;
    }
}

__device__ __forceinline__ KernelArgs kernel_args() { return (KernelArgs)__builtin_amdgcn_kernarg_segment_ptr(); }

// Every row exactly: more groups that count than 32 lanes hold, less than four experts, or few rows
// of many picks or groups.
template <bool F32, bool SIGMOID, int VPL>
__global__ __launch_bounds__(256) void score_topk_exact_kernel(ScoreArgs a) {
    extern __shared__ float lds_all[];
    const int wave = threadIdx.x >> 6;
    for (int64_t row = (int64_t)blockIdx.x * 4 + wave; row < a.T; row += (int64_t)gridDim.x * 4)
        choose_exactly<F32, SIGMOID, VPL>(kernel_args(), row, (LdsFloats)(lds_all + wave * a.lds_wave));
}

__device__ __forceinline__ void exchange(double& a, double& b) {
    const double x = a, y = b;
    a = kmax(x, y);
    b = kmin(x, y);
}
template <int N>
__device__ __forceinline__ void sort_bitonic(double* k) {  // descending
#pragma unroll
    for (int s = N / 2; s >= 1; s >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((i & s) == 0) exchange(k[i], k[i + s]);
}
template <int N>
__device__ __forceinline__ void sort_keys(double* k) {  // Batcher's odd-even merge sort
#pragma unroll
    for (int p = 1; p < N; p <<= 1)
#pragma unroll
        for (int q = p; q >= 1; q >>= 1)
#pragma unroll
            for (int j = q % p; j <= N - 1 - q; j += 2 * q)
#pragma unroll
                for (int i = 0; i <= (q - 1 < N - 1 - j - q ? q - 1 : N - 1 - j - q); ++i)
                    if ((i + j) / (2 * p) == (i + j + q) / (2 * p)) exchange(k[i + j], k[i + j + q]);
}
// the N largest of two descending runs of N
template <int N>
__device__ __forceinline__ void merge_keys(double* a, const double* b) {
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = kmax(a[i], b[N - 1 - i]);
    sort_bitonic<N>(a);
}
template <int STEP, int KT>
__device__ __forceinline__ void merge_partner(double* g) {
    double o[KT];
#pragma unroll
    for (int i = 0; i < KT; ++i) o[i] = partner<STEP>(g[i]);
    merge_keys<KT>(g, o);
}

// Two distances, u = 2^-24 and the hardware's exp2 and reciprocal good to 2 u, that
// decide what order 32 bits are certain of.
constexpr float U = 5.9604644775390625e-8f;
// Logits at least this far apart, the larger one l: their scores, exact, differ by more
// than two roundings to 32 bits (a softmax score by a factor exp(l - l'), a sigmoid one by
// 1 + (1 - s)(l - l'), 1 - s = 1 / (1 + exp(l))). Where scores leave the normal
// range, infinite: nothing is certain there.
template <bool SIGMOID>
__device__ __forceinline__ float logit_margin(float l, float top) {
    if constexpr (SIGMOID) return l < -80.f ? INFINITY : 8.f * U * (1.0f + exp32(l));
    else return l < top - 60.f || top == -LOW ? INFINITY : 8.f * U;
}
// c' = s' + bias at least this far apart, s' scores up to s_max. Each side: s' is off by
// s (1 - s) (2 + 3/2 |l|) u + 3 u s <= 3.2 u (sigmoid: exp2 and its argument, the sum, the
// reciprocal) or s (2 |l - m| + 2 ln E + 10) u <= 25 u s_max (softmax: s |l - m| <= s_max / e),
// the definition's by u / 2, and both sums by u |c|.
template <bool SIGMOID>
__device__ __forceinline__ float choice_margin(float c, float s_max) {
    return (SIGMOID ? 8.f * U : 64.f * U * s_max) + 4.f * U * fabsf(c);
}
// The same for groups' sums of two, size = |c| + |c| of them: their own sum is rounded too.
template <bool SIGMOID>
__device__ __forceinline__ float choice_group_margin(float size, float s_max) {
    return (SIGMOID ? 16.f * U : 128.f * U * s_max) + 12.f * U * size;
}
// A group's two scores s' without a bias, relative to their sum: off by (1 - s) |l| u 3/2 + 6 u
// or (2 |l - m| + 2 ln E + 10) u each, |l| up to 80, and one more rounding. Tiny sums, infinite.
template <bool SIGMOID>
__device__ __forceinline__ float group_margin(float v) {
    return v < 1e-30f ? INFINITY : (SIGMOID ? 400.f : 512.f) * U * v;
}

// Four neighbouring values, from any element on.
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t h4u __attribute__((ext_vector_type(2), aligned(2)));
template <bool F32>
__device__ __forceinline__ void load4(float* v, const void* p) {
    if constexpr (F32) {
        const f4u q = *static_cast<const f4u*>(p);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
        const h4u q = *static_cast<const h4u*>(p);
        v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
    }
}
// v[i] = v[i + n] for n = 1 to 3, as far as there are any
__device__ __forceinline__ void shift4(float* v, int n) {
    const float a = v[1], b = v[2], c = v[3];
    v[0] = n == 1 ? a : n == 2 ? b : n == 3 ? c : v[0];
    v[1] = n == 1 ? b : n == 2 ? c : v[1];
    v[2] = n == 1 ? c : v[2];
}

// fmaxf makes its arguments canonical first; these are
__device__ __forceinline__ float max_of_numbers(float a, float b) {
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// LPR lanes to a row, VPL logits to a lane (4 neighbours in every 4 LPR), k <= KT.
//
// The choice is defined by scores that are rounded from 64 bits, but 32 bits decide
// nearly every row. With a bias the experts are ordered by c' = s' + bias from the
// hardware's exp2 and reciprocal, without one by their logits (which no rounding
// touches: equal logits have equal scores, and the id decides). A row is certain if
// its groups, its k picks among themselves and the last pick and every expert
// behind it are the margins above apart. Where only picks, and one expert behind
// them, come nearer, these few are ordered anew (sigmoid scores with a bias: one row in
// 1000 of 256 experts); other rows are chosen anew by the whole wave.
// Keys: c' or the logit as a double with the id in the bits that 32-bit values leave
// zero. VL of a lane's values come to that: all, or, where the groups that stay hold at
// most half the experts, those of them alone. A lane passes on its 8 largest; one
// whose last passed key comes near the last pick makes the row uncertain.
//
// Bound by vector instructions (80% of the cycles), not by memory: 131072 rows of 256, sigmoid,
// bias, 4 of 8 groups, take 45 us, of which reading 128 MiB needs 27; one wave per row and
// 64-bit scores took 228. Softmax without groups: 37 us renormalised, 57 with the row's sum in
// 64 bits for weights that are not (51 with 32-bit terms, which made them up to 2 ln E + 3 roundings
// off). Lanes of a row: as few as hold its groups and logits, since every step of the merge is
// done by all of them. The picks' logits are read again for their weights, from memory: 59 of the
// 194 MB that are fetched (the next rows' have taken their place in L2).
// Rows that 32 bits do not decide cost a wave each: 16384 (131072) of 256 equal logits with a bias
// 37 (207) us, of a softmax with one logit 15 in front and a bias of zero 46 (262).
template <bool F32, bool SIGMOID, bool BIAS, int LPR, int VPL, int VL, int KT>
__global__ __launch_bounds__(256, LPR == 32 ? 3 : 4) void score_topk_kernel(ScoreArgs a) {
    extern __shared__ float lds_all[];
    constexpr int ROWS = 64 / LPR, LK = 8, N4 = VPL / 4, L4 = VL / 4;
    constexpr uint64_t TEAM = (1ull << LPR) - 1;
    const int lane = threadIdx.x & 63, team = lane / LPR;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int E = a.E, k = a.k, S = a.E / a.groups;
    float* lds = lds_all + wave * a.lds_wave;
    const bool quads = (S & 3) == 0;  // groups of whole fours
    int p = lane & (LPR - 1);
    // where a lane's fours of the groups that stay are: the how manieth such group, five bits each
    uint32_t group_of[(L4 + 5) / 6];
    if (VL < VPL || a.groups > 1) {
#pragma unroll
        for (int i = 0; i < (L4 + 5) / 6; ++i) group_of[i] = 0;
#pragma unroll
        for (int j = 0; j < L4; ++j)
            group_of[j / 6] |= ((uint32_t)(4 * LPR * j + 4 * p) * (uint32_t)a.inv_S >> 22 & 31u) << (5 * (j % 6));
    }
    const int64_t step = (int64_t)gridDim.x * 4 * ROWS;
    float c[VPL];
    // the logits of a team's row from a wave's first row on
    auto source = [&](int64_t row0) { return static_cast<const char*>(a.logits) + row0 * E * (F32 ? 4 : 2); };
    auto offset = [&](int64_t row0) { return (uint32_t)(row0 + team < a.T ? team * E : 0); };
    auto fetch = [&](int64_t row0) {
        const char* src = source(row0);
        const uint32_t base = offset(row0);
#pragma unroll
        for (int j = 0; j < N4; ++j)
            load4<F32>(c + 4 * j, src + (base + (uint32_t)min(4 * LPR * j + 4 * p, E - 4)) * (F32 ? 4u : 2u));
    };
    const int64_t first = ((int64_t)blockIdx.x * 4 + wave) * ROWS;
    if (first < a.T) fetch(first);
    float* bias = lds_all + 4 * a.lds_wave;
    if constexpr (BIAS) {
        for (int e = threadIdx.x; e < LPR * VPL; e += 256) bias[e] = e < E ? a.bias[e] : 0.f;
        __syncthreads();
    }
    for (int64_t row0 = first; row0 < a.T; row0 += step) {
        // what follows from this is made anew for each row: it would not fit the registers
        asm volatile("" : "+v"(p));
        const int64_t row = row0 + team;
        const bool live = row < a.T;
        if (VL == VPL && row0 != first) fetch(row0);
        if (E & 3) {
            // a row's last four, read from three before its end at most
#pragma unroll
            for (int j = 0; j < N4; ++j) shift4(c + 4 * j, 4 * LPR * j + 4 * p - (E - 4));
        }
        if (E < LPR * VPL) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) c[i] = 4 * LPR * (i >> 2) + 4 * p + (i & 3) < E ? c[i] : LOW;
        }
        // LOW for masked experts (and none); a NaN stays one for now
        float least = c[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) least = fminf(least, c[i]);
        const bool some_masked = __ballot(is_masked<F32>(least)) != 0;
        if (some_masked) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) c[i] = is_masked<F32>(c[i]) ? LOW : c[i];
        }
        bool unsure = false;
        float m = 0.f, s_max = 1.f;
        double sum = 1.0;
        if constexpr (!SIGMOID) {
            m = c[0];
#pragma unroll
            for (int i = 1; i < VPL; ++i) m = __builtin_elementwise_maximum(m, c[i]);
            m = team_reduce<LPR>(m, [](float x, float y) { return __builtin_elementwise_maximum(x, y); });
            // one NaN or infinity is in every score of its row
            unsure = !(m < INFINITY);
            m = unsure ? 0.f : m;
            if (!a.renorm) {
                // the weights' sum too (a row with nothing left: all terms 0)
                const double top = m == LOW ? 0.0 : (double)m;
                sum = 0.0;
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    sum += exp_term((double)c[i] - top);
                    if (i % 8 == 7) __builtin_amdgcn_sched_barrier(0);
                }
            } else if (BIAS) {
                sum = 0.0;
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    sum += c[i] == LOW ? 0.0 : (double)exp32(c[i] - m);
                    if (i % 8 == 7) __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (BIAS || !a.renorm) {
                sum = team_sum<LPR>(sum);
                s_max = sum == 0.0 ? 0.f : 1.0f / (float)sum;
            }
        }
        // score of a logit, 0 of LOW
        auto score32 = [&](float l) {
            if constexpr (SIGMOID) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l * -1.4426950408889634f));
            else return exp32(l - m) * s_max;
        };
        if constexpr (BIAS) {
            auto add_bias = [&](auto masked) {
#pragma unroll
                for (int j = 0; j < N4; ++j) {
                    const float4 q = *reinterpret_cast<const float4*>(bias + 4 * LPR * j + 4 * p);
                    const float b[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float v = __builtin_amdgcn_fmed3f(score32(c[4 * j + i]) + b[i], LOW, -LOW);
                        if constexpr (masked.value) c[4 * j + i] = c[4 * j + i] == LOW ? LOW : v;
                        else c[4 * j + i] = v;
                    }
                }
            };
            if (some_masked) add_bias(std::true_type{});
            else add_bias(std::false_type{});
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) c[i] = __builtin_amdgcn_fmed3f(c[i], LOW, -LOW) + 0.0f;  // (-0 is 0)
        }
        float v_of[VL];   // the values that are picked from, and the first id of each four
        int id_of[L4];
#pragma unroll
        for (int j = 0; j < L4; ++j) id_of[j] = 4 * LPR * j + 4 * p;
        if (VL < VPL || a.groups > 1) {
            // each group's largest two by lanes of their own, through LDS
            const bool sums = a.group_top == 2;
            const bool scores = !BIAS && sums;
            float* mine = lds + team * a.lds_row;
#pragma unroll
            for (int j = 0; j < N4; ++j) {
                const int e = 4 * LPR * j + 4 * p;
                if (LPR * VPL == E || e < E)
                    *reinterpret_cast<float4*>(mine + e) = float4{c[4 * j], c[4 * j + 1], c[4 * j + 2], c[4 * j + 3]};
            }
            if (VL < VPL && row0 + step < a.T) fetch(row0 + step);  // all that is needed of these is in LDS now
            wave_sync();
            const int shift = a.lpr_bits - a.group_bits;
            const int lpg = 1 << shift, g = p >> shift, sub = p & (lpg - 1);
            float t1 = LOW, t2 = LOW;
            auto take = [&](float v) {
                if (scores) v = v == LOW ? LOW : score32(v);
                t2 = __builtin_amdgcn_fmed3f(t1, t2, v);
                t1 = max_of_numbers(t1, v);
            };
            if (g < a.groups) {
                const float* q = mine + g * S;
                if (quads) {
                    // the lanes start at fours of their own: on different banks
                    const int n = S >> 2;
                    int i = sub + ((g * a.spread & 7) << shift);
                    i = i < n ? i : sub;
#pragma unroll 4
                    for (int x = sub; x < n; x += lpg) {
                        const float4 v = *reinterpret_cast<const float4*>(q + 4 * i);
                        take(v.x), take(v.y), take(v.z), take(v.w);
                        i += lpg;
                        i = i < n ? i : sub;
                    }
                } else {
                    for (int i = sub; i < S; i += lpg) take(q[i]);
                }
            }
            for (int x = 1; x < lpg; x <<= 1) {
                const float o1 = __shfl_xor(t1, x), o2 = __shfl_xor(t2, x);
                t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
                t1 = fmaxf(t1, o1);
            }
            const float v = sums && t2 > LOW ? t1 + t2 : t1;
            int ahead = 0;
            for (int o = 0; o < a.groups; ++o) {
                const float ov = __shfl(v, o << shift, LPR);
                ahead += (ov > v) | ((ov == v) & (o < g));
            }
            const bool stays = g < a.groups && ahead < a.top_groups;
            const float last = -team_max<LPR>(stays ? -v : LOW);
            const float next = team_max<LPR>(g < a.groups && !stays ? v : LOW);
            const float size = team_max<LPR>(
                BIAS && (v == last || v == next) ? (t1 > LOW ? fabsf(t1) : 0.f) + (t2 > LOW ? fabsf(t2) : 0.f) : 0.f);
            const float far = BIAS ? choice_group_margin<SIGMOID>(size, s_max)
                                   : scores ? group_margin<SIGMOID>(last) : logit_margin<SIGMOID>(last, m);
            // (equal logits are equal, and the lower group stays)
            unsure |= !(last - next > far || (!BIAS && !sums && last == next && last > 0.5f * LOW));
            const uint32_t stay = (uint32_t)(__ballot(stays) >> (team * LPR));
            if (VL < VPL || quads) {
                // the fours of the groups that stay, in order; which group is the o-th of them, by a table
                int* table = reinterpret_cast<int*>(mine + a.lds_row - 32);
                if (stays && sub == 0) table[__popc(stay & ((1u << p) - 1u)) >> shift] = g;
                wave_sync();
                const int n = a.top_groups * S;
#pragma unroll
                for (int j = 0; j < L4; ++j) {
                    const int x = 4 * LPR * j + 4 * p;
                    const int o = (int)(group_of[j / 6] >> (5 * (j % 6)) & 31u);
                    const int off = (int)__umul24(o, S);
                    id_of[j] = x < n ? (int)__umul24(table[x < n ? o : 0], S) + (x - off) : 0;
                }
#pragma unroll
                for (int j = 0; j < L4; ++j) {
                    const float4 q = *reinterpret_cast<const float4*>(mine + id_of[j]);
                    v_of[4 * j] = q.x, v_of[4 * j + 1] = q.y, v_of[4 * j + 2] = q.z, v_of[4 * j + 3] = q.w;
                }
#pragma unroll
                for (int j = 0; j < L4; ++j) {
                    const bool in = 4 * LPR * j + 4 * p < n;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v_of[4 * j + i] = in ? v_of[4 * j + i] : LOW;
                }
            } else {
#pragma unroll
                for (int i = 0; i < VL; ++i) {
                    const int e = 4 * LPR * (i >> 2) + 4 * p + (i & 3);
                    const bool in = (stay >> (((uint32_t)e * (uint32_t)a.inv_S >> 22 << shift) & 31u)) & 1u;
                    v_of[i] = in && e < E ? c[i] : LOW;
                }
            }
            wave_sync();  // the next row's values
        } else {
#pragma unroll
            for (int i = 0; i < VL; ++i) v_of[i] = c[i];
        }
        // the lane's LK largest keys, run by run
        double key[LK];
#pragma unroll
        for (int r = 0; r < VL; r += LK) {
            double run[LK];
#pragma unroll
            for (int i = 0; i < LK; ++i) {
                const uint64_t b = __builtin_bit_cast(uint64_t, (double)v_of[r + i]);
                uint32_t id = (uint32_t)id_of[(r + i) >> 2] | (uint32_t)(i & 3);
                // by the logit: the lower id's key is the larger one, of positive and of negative values
                if constexpr (!BIAS) id ^= ~((int32_t)(b >> 32) >> 31) & 1023;
                run[i] = __builtin_bit_cast(double, b | id);
            }
            sort_keys<LK>(run);
            if (r == 0) {
#pragma unroll
                for (int i = 0; i < LK; ++i) key[i] = run[i];
            } else {
                merge_keys<LK>(key, run);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        double top[KT];
        if constexpr (KT == LK) {
#pragma unroll
            for (int i = 0; i < LK; ++i) top[i] = kmax(key[i], partner<0>(key[LK - 1 - i]));
            sort_bitonic<LK>(top);
        } else {
            // both lanes' passed keys whole: the larger and the smaller half of a bitonic run
#pragma unroll
            for (int i = 0; i < LK; ++i) {
                const double o = partner<0>(key[LK - 1 - i]);
                top[i] = kmax(key[i], o);
                top[KT - LK + i] = kmin(key[i], o);
            }
            sort_bitonic<LK>(top);
            sort_bitonic<LK>(top + KT - LK);
        }
        merge_partner<1, KT>(top);
        merge_partner<2, KT>(top);
        if constexpr (LPR >= 16) merge_partner<3, KT>(top);
        if constexpr (LPR >= 32) merge_partner<4, KT>(top);
        // lane j has pick j
        double mine = top[0];
#pragma unroll
        for (int i = 1; i < KT; ++i) mine = p == i ? top[i] : mine;
        const float v = (float)mine;
        int id = (int)((uint32_t)__builtin_bit_cast(uint64_t, mine) & 1023u);
        if constexpr (!BIAS) id ^= ~((int32_t)(__builtin_bit_cast(uint64_t, mine) >> 32) >> 31) & 1023;
        float l = logit<F32>(source(row0) + (offset(row0) + (uint32_t)(id < E ? id : 0)) * (F32 ? 4u : 2u), 0);
        const float margin = BIAS ? choice_margin<SIGMOID>(v, s_max) : logit_margin<SIGMOID>(v, m);
        const float next = dpp32<0x101>(v), next_margin = dpp32<0x101>(margin);  // of lane + 1 in its 16
        bool mixed = p < k - 1 && !(v - next > fmaxf(margin, next_margin) || (!BIAS && v == next));
        if (p == k - 1) unsure |= !(v > 0.5f * LOW);
        const float last = __shfl(v, k - 1, LPR), bar = last - __shfl(margin, k - 1, LPR);
        const double last_key = __shfl(mine, k - 1, LPR);
        // the experts that are not picks and come near the last one
        int behind = 0;
        double best = -INFINITY;
#pragma unroll
        for (int i = 0; i < LK; ++i) {
            const float x = (float)key[i];
            const bool near = !(x < bar) && key[i] < last_key && (BIAS || x != last);
            behind += near;
            best = near ? kmax(best, key[i]) : best;
            // (what the lane did not pass on comes behind its last key)
            if (VL > LK && i == LK - 1) unsure |= !(x < bar);
        }
        if constexpr (SIGMOID && BIAS) {
            // The picks and one expert near the last of them: ordered anew by their exact c.
            behind = (int)team_sum<LPR>((float)behind);
            unsure |= behind > 1;
            mixed |= behind == 1;
            mixed = ((__ballot(mixed && !unsure && live) >> (team * LPR)) & TEAM) != 0;
            if (__ballot(mixed)) {
                best = team_reduce<LPR>(best, [](double x, double y) { return kmax(x, y); });
                const int id9 = behind ? (int)((uint32_t)__builtin_bit_cast(uint64_t, best) & 1023u) : 0;
                const float l9 = logit<F32>(source(row0) + (offset(row0) + (uint32_t)id9) * (F32 ? 4u : 2u), 0);
                const float c = (float)sigmoid64((double)l) + bias[id], c9 = (float)sigmoid64((double)l9) + bias[id9];
                int rank = behind && (c9 > c || (c9 == c && id9 < id)), rank9 = 0;
                for (int q = 0; q < k; ++q) {
                    const float cq = __shfl(c, q, LPR);
                    const int iq = __shfl(id, q, LPR);
                    rank += cq > c || (cq == c && iq < id);
                    rank9 += cq > c9 || (cq == c9 && iq < id9);
                }
                int pick = rank9 == p ? id9 : id;
                for (int q = 0; q < k; ++q) {
                    const int rq = __shfl(rank, q, LPR), iq = __shfl(id, q, LPR);
                    pick = rq == p ? iq : pick;
                }
                if (mixed && p < k) {
                    id = pick;
                    l = logit<F32>(source(row0) + (offset(row0) + (uint32_t)id) * (F32 ? 4u : 2u), 0);
                }
            }
        } else {
            unsure |= mixed || behind;
        }
        const uint64_t unsure_all = __ballot(unsure && live);
        if (live && !((unsure_all >> (team * LPR)) & TEAM)) {
            RowStat st = {(double)m, 0.0};
            if constexpr (!SIGMOID) st.inv = sum == 0.0 ? 0.0 : 1.0 / sum;
            const double s = a.renorm && !SIGMOID ? 0.0 : score<F32, SIGMOID>(l, st);
            const double h = share<F32, SIGMOID, (LPR < 16 ? LPR : 16)>(l, s, p, k, a.renorm);
            if (p < k) {
                a.ids[row * k + p] = id;
                a.w[row * k + p] = (float)((double)a.scale * h);
                if (a.rec) a.rec[(int64_t)p * a.rec_stride + row] = id;
            }
        }
        if (unsure_all == 0) continue;
#pragma unroll 1
        for (int t = 0; t < ROWS; ++t)
            if ((unsure_all >> (t * LPR)) & TEAM)
                choose_exactly<F32, SIGMOID, (LPR * VPL + 63) / 64>(kernel_args(), row0 + t, (LdsFloats)lds);
    }
}

// load[e] += how often e stands in ids, counted in LDS first: atomics to one kilobyte
// of memory go one after the other (all 131072 straight to memory took 100 us). 16384 ids to
// a workgroup, all on their way at once.
typedef int i4u __attribute__((ext_vector_type(4), aligned(4)));
__global__ __launch_bounds__(1024) void score_load_kernel(const int32_t* ids, int64_t n, int E, int32_t* load) {
    __shared__ int32_t count[MAX_E];
    for (int e = threadIdx.x; e < E; e += 1024) count[e] = 0;
    __syncthreads();
    for (int64_t i0 = (int64_t)blockIdx.x * 16384; i0 < n; i0 += (int64_t)gridDim.x * 16384) {
        i4u q[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t i = i0 + r * 4096 + threadIdx.x * 4;
            q[r] = i4u{-1, -1, -1, -1};
            if (i + 4 <= n) q[r] = *reinterpret_cast<const i4u*>(ids + i);
            else
                for (int j = 0; j < 3; ++j)
                    if (i + j < n) q[r][j] = ids[i + j];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (q[r][j] >= 0) atomicAdd(&count[q[r][j]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 1024)
        if (count[e]) atomicAdd(load + e, count[e]);
}

// ---------------------------------------------------------------- replay

// 16 lanes per token where the chosen logits alone decide its weights: k of a row's logits
// are read, scattered. Bound by 64-bit exponentials and latency: 16384 tokens, k = 8: 5.1 us.
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
        const double h = share<F32, SIGMOID, 16>(l, score<F32, SIGMOID>(l, RowStat{0.0, 0.0}), lane, k, RENORM);
        if (live && lane < k) {
            a.ids[row * k + lane] = id;
            a.w[row * k + lane] = bad ? 0.f : (float)((double)a.scale * h);
        }
        const int flags = (bad ? MOE_FLAG_BAD_ID : 0) | (dup ? MOE_FLAG_DUP_ID : 0);
        if (live && lane == 0 && flags && status) atomicOr(status, flags);
    }
}

// A row that 16 lanes hold: lane p the logits 64 j + 4 p + i, and its softmax. KEEP: l is
// afterwards 2^UP exp(l - m), rounded once to 32 bits, in which 2^UP keeps the normal range down to
// scores of 2^-150 (and a gradient made from it has room for values up to 2^104).
template <bool F32, int VPL, bool KEEP = false>
struct Row16 {
    static constexpr int UP = KEEP ? 24 : 0;
    float l[VPL];
    RowStat st;
    bool odd;        // a NaN or infinity is in every score that is not masked: KEEP says which of the lane's
    uint64_t there;  // are not, and l is 0
    __device__ __forceinline__ void fetch(const void* logits, int64_t row, int E, int p) {
        const char* src = static_cast<const char*>(logits) + row * E * (F32 ? 4 : 2);
        if (VPL > 4 || E >= 4) {
#pragma unroll
            for (int j = 0; j < VPL / 4; ++j)
                load4<F32>(l + 4 * j, src + (uint32_t)min(64 * j + 4 * p, E - 4) * (F32 ? 4u : 2u));
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) l[i] = logit<F32>(src, min(64 * (i >> 2) + 4 * p + (i & 3), E - 1));
        }
    }
    __device__ __forceinline__ void sums(int E, int p) {
        if ((VPL > 4 || E >= 4) && (E & 3)) {
#pragma unroll
            for (int j = 0; j < VPL / 4; ++j) shift4(l + 4 * j, 64 * j + 4 * p - (E - 4));
        }
        if (E < 16 * VPL) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) l[i] = 64 * (i >> 2) + 4 * p + (i & 3) < E ? l[i] : LOW;
        }
        // LOW for masked experts; m is NaN where a logit is
        float least = l[0], m = l[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) {
            least = fminf(least, l[i]);
            m = __builtin_elementwise_maximum(m, l[i]);
        }
        m = team_reduce<16>(m, [](float x, float y) { return __builtin_elementwise_maximum(x, y); });
        if (__ballot(is_masked<F32>(least))) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) l[i] = is_masked<F32>(l[i]) ? LOW : l[i];
            m = is_masked<F32>(m) ? LOW : m;
        }
        const double top = m == LOW ? 0.0 : (double)m;  // (a row with nothing left: all terms 0)
        odd = !(m < INFINITY);
        if (KEEP && __ballot(odd)) {
            there = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i) there |= (uint64_t)(l[i] != LOW) << i;
        }
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const double e = exp_term<UP>((double)l[i] - top);
            sum += e;
            if constexpr (KEEP) {
                l[i] = (float)e;
                asm volatile("" : "+v"(l[i]));  // (here, in the logit's register)
            }
            if ((KEEP || VPL > 32) && i % 8 == 7) __builtin_amdgcn_sched_barrier(0);  // (more would not fit the registers)
        }
        sum = team_sum<16>(sum);
        if (odd) sum = NAN;
        st = {(double)m, m == LOW ? 0.0 : (double)(1 << UP) / sum};
    }
};

// 16 lanes per token where the whole row does (softmax without renorm). 16384 tokens of 256
// experts (16 MiB, 3.4 us of reading) take 7.5 us: one round of four waves to a SIMD, whose loads
// come back at about the same time, and then 18 64-bit operations for each logit (7.0 with
// 32-bit exponentials).
template <bool F32, int VPL>
__global__ __launch_bounds__(256) void score_replay_row_kernel(ScoreArgs a, int32_t* status) {
    const int lane = threadIdx.x & 15, E = a.E, k = a.k;
    for (int64_t row0 = (int64_t)blockIdx.x * 16; row0 < a.T; row0 += (int64_t)gridDim.x * 16) {
        const int64_t row = row0 + (threadIdx.x >> 4);
        const bool live = row < a.T;
        const int64_t t = live ? row : row0;
        int p = lane;
        asm volatile("" : "+v"(p));  // (what follows from it is made where it is used: most waves have one round)
        Row16<F32, VPL> r;
        r.fetch(a.logits, t, E, p);
        const int id = lane < k ? a.rec[(int64_t)lane * a.rec_stride + t] : 0;
        int bad = lane < k && (id < 0 || id >= E), dup = 0;
        for (int j = 0; j < k; ++j) {
            const int o = __shfl(id, j, 16);
            dup |= lane < k && j < lane && o == id;
        }
        bad = ((__ballot(bad) >> (threadIdx.x & 48)) & 0xFFFF) != 0;
        dup = ((__ballot(dup) >> (threadIdx.x & 48)) & 0xFFFF) != 0;
        const float ls = logit<F32>(a.logits, t * E + (bad ? 0 : id));  // on its way during the sums
        r.sums(E, p);
        if (live && lane < k) {
            a.ids[row * k + lane] = id;
            a.w[row * k + lane] = bad ? 0.f : (float)((double)a.scale * score<F32, false>(ls, r.st));
        }
        const int flags = (bad ? MOE_FLAG_BAD_ID : 0) | (dup ? MOE_FLAG_DUP_ID : 0);
        if (live && lane == 0 && flags && status) atomicOr(status, flags);
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
    int lds_wave;  // floats of LDS for each wave
};

// 16 lanes per token, four tokens to a wave: lane j < k has slot j; the slots' values go
// into the rows' place in LDS, from which whole rows are written. In the whole-row form
// they are the brackets of s_e (scale d_w - scale dot), made in 64 bits: for a row of one large score
// the two terms are nearly equal. Brackets, 1 / sum and exponentials are rounded to 32 bits each
// and multiplied there: 5 2^-24 of a gradient. Bound by the latency of one round of waves, in
// which the stores wait for ids, their logits and exponentials: 16384 tokens of 256 experts,
// fp32, 7.4 us (writing them 3.4), and 9.0 with the whole row's gradient (reading and writing 6.7).
template <bool F32, bool SIGMOID, bool RENORM, bool PARTS, int VPL>
__global__ __launch_bounds__(256) void score_backward_kernel(ScoreGradArgs a) {
    constexpr bool WHOLE = !SIGMOID && !RENORM;
    extern __shared__ float lds_all[];
    const int lane = threadIdx.x & 63, team = lane >> 4, E = a.E, k = a.k;
    int p = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int EP = WHOLE ? (E + 3) & ~3 : E;  // a row's floats in LDS
    float* lds = lds_all + wave * a.lds_wave;
    float* mine = lds + team * EP;
    const int64_t step = (int64_t)gridDim.x * 16;
    for (int64_t row0 = ((int64_t)blockIdx.x * 4 + wave) * 4; row0 < a.T; row0 += step) {
        const int64_t row = row0 + team;
        const bool live = row < a.T;
        const int64_t t = live ? row : row0;
        Row16<F32, VPL, true> r;
        r.st = {0.0, 0.0};
        if constexpr (WHOLE) {
            asm volatile("" : "+v"(p));  // (what follows from it is made where it is used: most waves have one round)
            r.fetch(a.logits, t, E, p);
        }
        const int id = p < k ? a.ids[t * k + p] : 0;
        float dw = 0.f;
        if constexpr (PARTS) {
            if (p < k) {
                const int r = a.pair_row[t * k + p];
                if (r >= 0) {
                    const float* q = a.part + (int64_t)r * MOE_GATE_PARTS;
                    for (int g = 0; g < a.ngroups; ++g) dw += q[g];
                }
                if (live) a.d_gate[row * k + p] = dw;
            }
        } else if (p < k) {
            dw = a.d_w[t * k + p];
        }
        // zeros to the rows' place
        if constexpr (!WHOLE)
            for (int i = 4 * lane; i < 4 * EP; i += 256) *reinterpret_cast<float4*>(lds + i) = float4{0.f, 0.f, 0.f, 0.f};
        const bool outside = p < k && (id < 0 || id >= E);
        const bool bad = ((__ballot(outside) >> (16 * team)) & 0xFFFF) != 0;
        const float ls = logit<F32>(a.logits, t * E + (bad ? 0 : id));
        if constexpr (WHOLE) {
            r.sums(E, p);
            asm volatile("" : "+v"(p));  // (its columns are not kept over the sums)
        }
        const double s = score<F32, SIGMOID>(ls, r.st);
        const double h = share<F32, SIGMOID, 16>(ls, s, p, k, RENORM);
        double dot = 0.0;
        if constexpr (RENORM || WHOLE) dot = team_sum<16>(p < k ? h * (double)dw : 0.0);
        // the slot's gradient of its own logit; WHOLE: of its score, -scale dot that of every other
        const double all = WHOLE ? (double)a.scale * dot : 0.0;
        if constexpr (WHOLE) {
            const float v = bad ? 0.f : (float)-all;
#pragma unroll
            for (int j = 0; j < VPL / 4; ++j)
                if (64 * j + 4 * p < E) *reinterpret_cast<float4*>(mine + 64 * j + 4 * p) = float4{v, v, v, v};
        }
        double c = WHOLE ? (double)a.scale * (double)dw : (double)a.scale * h * ((double)dw - (RENORM ? dot : 0.0));
        if constexpr (SIGMOID) c *= sigmoid_near(-ls);
        if (!WHOLE && is_masked<F32>(ls)) c = 0.0;  // (next to a chosen NaN too)
        wave_sync();
        const bool on = p < k && !bad;
        if (on) reinterpret_cast<int*>(mine)[id] = p;
        wave_sync();
        // an expert in several slots (a record may have that): each of them writes the sum
        if (__ballot(on && reinterpret_cast<int*>(mine)[id] != p)) {
            double sum = 0.0;
            for (int j = 0; j < k; ++j) {
                const int o = __shfl(id, j, 16);
                const double oc = __shfl(c, j, 16);
                sum += o == id ? oc : 0.0;
            }
            c = sum;
        }
        wave_sync();
        if (on) mine[id] = (float)(c - all);
        wave_sync();
        if constexpr (WHOLE) {
            const float inv = bad ? 0.f : (float)r.st.inv;
            char* out = static_cast<char*>(a.d_logits) + t * E * (F32 ? 4 : 2);
#pragma unroll
            for (int j = 0; j < VPL / 4; ++j) {
                const int e = 64 * j + 4 * p;
                if (!live || e >= E) continue;
                const float4 q = *reinterpret_cast<const float4*>(mine + e);
                float v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = r.l[4 * j + i] * (inv * v[i]) * (1.0f / (1 << r.UP));
                if (e + 4 <= E) {
                    if constexpr (F32) *reinterpret_cast<f4u*>(out + e * 4) = f4u{v[0], v[1], v[2], v[3]};
                    else *reinterpret_cast<h4u*>(out + e * 2) = h4u{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
                } else {
                    for (int i = 0; i < E - e; ++i) {
                        if constexpr (F32) reinterpret_cast<float*>(out)[e + i] = v[i];
                        else reinterpret_cast<uint16_t*>(out)[e + i] = (uint16_t)f32_to_bf16(v[i]);
                    }
                }
            }
            if (__ballot(live && r.odd && !bad)) {
#pragma unroll 1
                for (int i = 0; i < VPL; ++i) {
                    const int e = 64 * (i >> 2) + 4 * p + (i & 3);
                    const float v = (r.there >> i) & 1 ? NAN : 0.f;
                    if (!live || !r.odd || bad || e >= E) continue;
                    if constexpr (F32) reinterpret_cast<float*>(out)[e] = v;
                    else reinterpret_cast<uint16_t*>(out)[e] = (uint16_t)f32_to_bf16(v);
                }
            }
        } else {
            // the four rows are one piece of memory, from a multiple of four elements on
            const int n = (int)(a.T - row0 < 4 ? a.T - row0 : 4) * E;
            char* out = static_cast<char*>(a.d_logits) + row0 * E * (F32 ? 4 : 2);
            for (int i = 4 * lane; i < n; i += 256) {
                const float4 q = *reinterpret_cast<const float4*>(lds + i);
                if (i + 4 <= n) {
                    if constexpr (F32) *reinterpret_cast<float4*>(out + i * 4) = q;
                    else *reinterpret_cast<uint2*>(out + i * 2) = uint2{cvt_bf16x2(q.x, q.y), cvt_bf16x2(q.z, q.w)};
                } else {
                    const float v[4] = {q.x, q.y, q.z, q.w};
                    for (int j = 0; j < n - i; ++j) {
                        if constexpr (F32) reinterpret_cast<float*>(out)[i + j] = v[j];
                        else reinterpret_cast<uint16_t*>(out)[i + j] = (uint16_t)f32_to_bf16(v[j]);
                    }
                }
            }
        }
        wave_sync();  // the next rows' zeros
    }
}

// ---------------------------------------------------------------- bias

// bias + step sign(mean - load), the mean as an exact comparison of integers:
// total against load E. One workgroup, bound by a launch's latency (1.9 us).
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

// f(values per lane that hold E experts in 16 lanes)
template <typename F>
void with_row16(int E, F&& f) {
    if (E <= 64) f(std::integral_constant<int, 4>{});
    else if (E <= 256) f(std::integral_constant<int, 16>{});
    else if (E <= 512) f(std::integral_constant<int, 32>{});
    else f(std::integral_constant<int, 64>{});
}

template <bool F32, bool SIGMOID, int LPR, int VPL, int KT>
void launch_topk(ScoreArgs a, hipStream_t stream) {
    constexpr int ROWS = 64 / LPR;
    a.lpr_bits = LPR == 8 ? 3 : LPR == 16 ? 4 : 5;
    const int S = a.E / a.groups;
    bool half = false;  // the groups that stay hold at most half of what the lanes can
    if (a.groups > 1) {
        // a row's values and 32 more for its table, rows half the 64 banks apart
        a.lds_row = (a.E + 3) / 4 * 4 + 32;
        a.lds_row += (96 - a.lds_row % 64) % 64;
        a.lds_wave = ROWS * a.lds_row;
        half = S % 4 == 0 && a.top_groups * S <= LPR * VPL / 2;
    }
    // as many workgroups as run at once: each has its next rows' logits on their way
    const int64_t blocks = (a.T + 4 * ROWS - 1) / (4 * ROWS), most = 4 * (int64_t)num_cus();
    const dim3 grid((unsigned)(blocks < most ? blocks : most));
    const size_t lds = ((size_t)a.lds_wave * 4 + (a.bias ? LPR * VPL : 0)) * sizeof(float);
    auto go = [&](auto vl) {
        if (a.bias) score_topk_kernel<F32, SIGMOID, true, LPR, VPL, vl.value, KT><<<grid, 256, lds, stream>>>(a);
        else score_topk_kernel<F32, SIGMOID, false, LPR, VPL, vl.value, KT><<<grid, 256, lds, stream>>>(a);
    };
    if constexpr (VPL >= 16) {
        if (half) {
            go(std::integral_constant<int, VPL / 2>{});
            return;
        }
    }
    go(std::integral_constant<int, VPL>{});
}

// The lanes of a row hold its logits, and its groups one each at least.
template <bool F32, bool SIGMOID>
void launch_choice_of(ScoreArgs a, hipStream_t stream) {
    const int E = a.E, G = a.groups;
    const int S = E / G;
    a.inv_S = ((1 << 22) + S - 1) / S;
    while ((1 << a.group_bits) < G) ++a.group_bits;
    // groups a multiple of 32 floats apart would read the same banks
    a.spread = S % 32 == 0;
    // A whole wave to a row, and to all of it exactly, where that is no slower than 16 lanes or 32:
    // up to 1024 rows of 129 to 256 experts that need 16 picks or more than 8 groups (1024 rows, k = 16:
    // 6.0 us against 7.8, 32 groups 7.1 against 8.5; one row 5.4 against 4.6).
    const bool few_lanes = G <= 8 && a.k <= 8;
    // Up to 32 rows for each compute unit lanes are plenty, and twice as many to a row shorten what
    // they do in turn (one row of 256 experts, no groups, 5.9 -> 4.0 us; 2048 rows 6.4 -> 4.5; 8192 7.3 -> 5.8;
    // 512 experts 5.2 -> 4.0, 6.9 -> 4.7, 10.1 -> 8.6); more rows lose by it (32768: 14 -> 17 us, 31 -> 36).
    const bool wide = a.T <= 32 * (int64_t)num_cus();
    if (G > 32 || E < 4 || (E > 128 && E <= 256 && a.T <= 1024 && !few_lanes)) {
        a.lds_wave = E;
        with_vpl(E, [&](auto v) {
            score_topk_exact_kernel<F32, SIGMOID, v.value>
                <<<row_blocks(a.T, 4), 256, (size_t)a.lds_wave * 4 * sizeof(float), stream>>>(a);
        });
    } else if (few_lanes && E <= 256) {
        if (E <= 64) launch_topk<F32, SIGMOID, 8, 8, 8>(a, stream);
        else if (E <= 128) launch_topk<F32, SIGMOID, 8, 16, 8>(a, stream);
        else if (wide) launch_topk<F32, SIGMOID, 16, 16, 8>(a, stream);
        else launch_topk<F32, SIGMOID, 8, 32, 8>(a, stream);
    } else if (G <= 16 && E <= 512) {
        if (E <= 128) launch_topk<F32, SIGMOID, 16, 8, 16>(a, stream);
        else if (E <= 256) launch_topk<F32, SIGMOID, 16, 16, 16>(a, stream);
        else if (a.k <= 8 && wide) launch_topk<F32, SIGMOID, 32, 16, 8>(a, stream);
        else if (a.k <= 8) launch_topk<F32, SIGMOID, 16, 32, 8>(a, stream);
        else launch_topk<F32, SIGMOID, 16, 32, 16>(a, stream);
    } else {
        if (a.k <= 8) launch_topk<F32, SIGMOID, 32, 32, 8>(a, stream);
        else launch_topk<F32, SIGMOID, 32, 32, 16>(a, stream);
    }
}
void launch_choice(const ScoreArgs& a, int32_t type, int32_t score, hipStream_t stream) {
    const bool sig = score == MOE_SCORE_SIGMOID;
    if (type == MOE_SRC_F32) {
        if (sig) launch_choice_of<true, true>(a, stream);
        else launch_choice_of<true, false>(a, stream);
    } else {
        if (sig) launch_choice_of<false, true>(a, stream);
        else launch_choice_of<false, false>(a, stream);
    }
}

int launch_backward(ScoreGradArgs a, int32_t type, int32_t score, int32_t renorm, bool parts, hipStream_t stream) {
    a.lds_wave = 4 * ((a.E + 3) / 4 * 4);
    const dim3 grid = row_blocks(a.T, 16);
    const size_t lds = (size_t)a.lds_wave * 4 * sizeof(float);
    with_forms(type, score, renorm, [&](auto t, auto s, auto r) {
        auto go = [&](auto v) {
            if (parts) score_backward_kernel<t.value, s.value, r.value, true, v.value><<<grid, 256, lds, stream>>>(a);
            else score_backward_kernel<t.value, s.value, r.value, false, v.value><<<grid, 256, lds, stream>>>(a);
        };
        if constexpr (!s.value && !r.value) with_row16(a.E, go);
        else go(std::integral_constant<int, 4>{});
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
    ScoreArgs a = {};
    a.logits = logits;
    a.bias = bias;
    a.T = T;
    a.E = E;
    a.k = k;
    a.groups = top_groups == groups ? 1 : groups;  // every group stays
    a.top_groups = top_groups;
    a.group_top = group_top;
    a.renorm = renorm != 0;
    a.scale = scale;
    a.ids = ids;
    a.w = w;
    a.rec = rec ? rec + (int64_t)layer * k * seq_len + s0 : nullptr;
    a.rec_stride = seq_len;
    launch_choice(a, logits_type, score, stream);
    MOE_LAUNCH_CHECK("score_topk_kernel");
    if (load) {
        const int64_t n = T * k, blocks = (n + 16383) / 16384;
        score_load_kernel<<<dim3((unsigned)(blocks < 32 ? blocks : 32)), dim3(1024), 0, stream>>>(ids, n, E, load);
        MOE_LAUNCH_CHECK("score_load_kernel");
    }
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
            with_row16(E, [&](auto v) {
                score_replay_row_kernel<t.value, v.value><<<row_blocks(T, 16), 256, 0, stream>>>(a, dev_status);
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
    return launch_backward({d_w, nullptr, nullptr, 0, logits, ids, T, E, k, scale, nullptr, d_logits, 0}, logits_type, score,
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
    return launch_backward({nullptr, gate_part, pair_row, gate_groups(d), logits, ids, T, E, k, scale, d_gate, d_logits, 0},
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
