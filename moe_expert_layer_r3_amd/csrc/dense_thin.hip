// Products with few rows (decoded tokens): C[m, n] = sum_k x[m, k] W[n, k], M <= 64.
//
// Bound by the bytes of W, each read once: a workgroup owns 16 NB rows of W and its
// NW waves split K, so that W goes from memory straight into MFMA operands (16
// bytes per lane, 64 adjacent bytes of 16 rows per load) with U steps of 32 always
// in flight per wave, and no workspace or second launch is needed: the waves'
// fp32 sums are added in order through LDS and the epilogue runs on them.  x is
// re-read by every workgroup from L2; NB = 2 halves that where M > 16.
#include "dense_gemm.hpp"

namespace moe {

template <int MT, int NB, int NW, int EPI>
__global__ __launch_bounds__(NW * 64) void dense_thin_kernel(DenseArgs g) {
    constexpr int U = MT + NB <= 3 ? 8 : 4;
    constexpr bool GATE = EPI == EPI_GATE;
    __shared__ v4f red[NW][NB * MT][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l15 = lane & 15, gk = (lane >> 4) * 8;
    const int n0 = blockIdx.x * NB * (GATE ? 8 : 16);

    // epilogue operands early: their latency hides behind the product
    const int fr = tid >> 6, em = (fr % MT) * 16 + l15;
    const int en = n0 + fr / MT * (GATE ? 8 : 16) + (lane >> 4) * 4;
    const bool mine = fr < NB * MT;
    EpiIn<EPI> in;
    if (mine) in.load(g, em, en);

    // rows past the matrix read its last row: their results are not stored
    const uint16_t *px[MT], *pw[NB];
#pragma unroll
    for (int m = 0; m < MT; ++m) px[m] = g.a + (int64_t)min(m * 16 + l15, g.M - 1) * g.lda;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        int64_t row;
        if constexpr (GATE) {  // eight G rows, then the eight U rows of the same h columns
            row = min(n0 + b * 8 + (l15 & 7), g.f - 1) + (l15 >= 8 ? g.f : 0);
        } else {
            row = min(n0 + b * 16 + l15, g.N - 1);
        }
        pw[b] = g.b + row * g.ldb;
    }
    const int steps = (g.K + 31) / 32, per = (steps + NW - 1) / NW;
    const int s0 = wave * per, n = min(per, steps - s0);  // n may be <= 0
    const bool tail = (g.K & 31) != 0;

    v4f acc[NB][MT];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[b][m] = v4f{0.f, 0.f, 0.f, 0.f};

    u32x4 fx[U][MT], fw[U][NB];
    auto load = [&](int u, int s) {
        int k = (s0 + s) * 32 + gk;
        if (k >= g.K) k = 0;  // multiplied as zero below
#pragma unroll
        for (int b = 0; b < NB; ++b) fw[u][b] = *reinterpret_cast<const u32x4*>(pw[b] + k);
#pragma unroll
        for (int m = 0; m < MT; ++m) fx[u][m] = *reinterpret_cast<const u32x4*>(px[m] + k);
    };
    auto mul = [&](int u, int s) {
        if (tail && (s0 + s) * 32 + gk >= g.K) {
            const u32x4 z = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int b = 0; b < NB; ++b) fw[u][b] = z;
#pragma unroll
            for (int m = 0; m < MT; ++m) fx[u][m] = z;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[b][m] = mfma_bf16(fw[u][b], fx[u][m], acc[b][m]);
    };
    if (n > 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) load(u, min(u, n - 1));
        int s = 0;
        for (; s + U < n; s += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                mul(u, s + u);
                load(u, min(s + U + u, n - 1));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s + u < n) mul(u, s + u);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int m = 0; m < MT; ++m) red[wave][b * MT + m][lane] = acc[b][m];
    __syncthreads();
    if (!mine) return;
    auto sum = [&](int l) {
        v4f s = red[0][fr][l];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += red[w][fr][l];
        return s;
    };
    if constexpr (GATE) {  // lanes 0-31 hold G, lanes 32-63 U of the same columns
        if (lane >= 32) return;
        const v4f G = sum(lane), U4 = sum(lane + 32);
        epi_gate(g, em, en, G, U4, em < g.M && en < g.f);
    } else {
        const v4f s = sum(lane);
        if (em >= g.M || en >= g.N) return;
        if constexpr (EPI == EPI_PLAIN)
            epi_plain(g, em, en, s, in);
        else
            epi_linear(g, em, en, s, in);
    }
}

namespace {
template <int MT, int NB, int NW, int EPI>
int launch(const DenseArgs& g, hipStream_t stream) {
    const int per = NB * (EPI == EPI_GATE ? 8 : 16), cols = EPI == EPI_GATE ? g.f : g.N;
    dense_thin_kernel<MT, NB, NW, EPI><<<dim3((unsigned)((cols + per - 1) / per)), dim3(NW * 64), 0, stream>>>(g);
    MOE_LAUNCH_CHECK("dense_thin_kernel");
    return MOE_OK;
}
template <int EPI>
int launch_rows(const DenseArgs& g, hipStream_t stream) {
    const int mt = (g.M + 15) / 16, tiles = g.N / 16;
    // few rows of W: one 16-row group per workgroup, K over 16 waves
    if (tiles < 192) {
        if (mt == 1) return launch<1, 1, 16, EPI>(g, stream);
        if (mt == 2) return launch<2, 1, 16, EPI>(g, stream);
        return launch<4, 1, 16, EPI>(g, stream);
    }
    if (mt == 1) return launch<1, 1, 8, EPI>(g, stream);
    if (mt == 2) return launch<2, 2, 8, EPI>(g, stream);
    return launch<4, 2, 8, EPI>(g, stream);
}
}  // namespace

bool dense_is_thin(int64_t M, int epi, int save) {
    return M <= THIN_ROWS && (epi == EPI_LINEAR || epi == EPI_PLAIN || (epi == EPI_GATE && save != MOE_SAVE_INT8));
}

int dense_thin_launch(const DenseArgs& g, int epi, hipStream_t stream) {
    if (epi == EPI_GATE) return launch_rows<EPI_GATE>(g, stream);
    if (epi == EPI_PLAIN) return launch_rows<EPI_PLAIN>(g, stream);
    return launch_rows<EPI_LINEAR>(g, stream);
}

}  // namespace moe
