// bf16 matrix products with fused epilogues (dense_gemm.hpp): the kernels and
// the choice between them.
#include "dense_gemm.hpp"

namespace moe {

// Tile index of a workgroup: XCD x runs a contiguous eighth of the tiles, which
// go m fastest inside groups of 8 m-tiles, so that the tiles an XCD runs side by
// side share few A and B tiles in its L2.
__device__ __forceinline__ void dense_tile(const DenseArgs& g, int& mt, int& nt, int& split) {
    const int per = g.mt * g.nt;
    const int t0 = (int)xcd_tile(blockIdx.x, gridDim.x);
    split = t0 / per;
    const int t = t0 - split * per;
    constexpr int GM = 8;
    const int grp = t / (GM * g.nt);
    const int gm = min(GM, g.mt - grp * GM);
    const int in = t - grp * GM * g.nt;
    nt = in / gm;
    mt = grp * GM + in - nt * gm;
}

// ---------------------------------------------------------------- 64 x 64 wave tiles
// WM x WN waves of 64 x 64, K steps of 64 double-buffered in LDS: while a step is
// multiplied the next one is on its way.
template <int WM, int WN, int LA, int LB, int EPI>
__global__ __launch_bounds__(WM * WN * 64) void dense_kernel(DenseArgs g) {
    constexpr int BM = WM * 64, BN = WN * 64, NW = WM * WN;
    constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
    constexpr int ASEG = BM / 8 / NW, BSEG = BN / 8 / NW;
    static_assert(LA == OP_KC || BM % 128 == 0, "KS images are 128 columns wide");
    static_assert(LB == OP_KC || BN % 128 == 0, "KS images are 128 columns wide");
    static_assert(EPI != EPI_GATE || (WN == 4 && LB == OP_KC), "gated tiles pair 128 G with 128 U columns");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * STAGE];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    int mt, nt, split;
    dense_tile(g, mt, nt, split);
    const int64_t m0 = (int64_t)mt * BM;
    const int n0 = nt * (EPI == EPI_GATE ? 128 : BN);
    const int ks0 = split * g.ksteps;
    const int ks1 = min(ks0 + g.ksteps, (g.K + DBK - 1) / DBK);
    const uint32_t sbase = __builtin_amdgcn_readfirstlane(lds_addr(smem));

    // this wave's DMA segments: first row (KC) or K row and image (KS)
    uint32_t va[ASEG], vb[BSEG], ka[ASEG], kb[BSEG];  // byte offsets and K indices
    const uint8_t *pa, *pb;
    if constexpr (LA == OP_KC) {
        const KcLane l(lane, g.lda);
        const int64_t r0 = m0 + wave * ASEG * 8;
        pa = (const uint8_t*)(g.a + r0 * g.lda) + (int64_t)ks0 * 128;
#pragma unroll
        for (int i = 0; i < ASEG; ++i) {
            va[i] = r0 + 8 * i + l.row < g.M ? l.off + (uint32_t)(8 * i * g.lda * 2) : OOB;
            ka[i] = l.k;
        }
    } else {
        const int img = wave * ASEG / 16, k0 = (wave * ASEG % 16) * 4;
        const int64_t c0 = m0 + img * 128;
        pa = (const uint8_t*)(g.a + c0) + (int64_t)ks0 * DBK * g.lda * 2;
#pragma unroll
        for (int i = 0; i < ASEG; ++i) {
            const uint32_t k = k0 + 4 * i + (lane >> 4), c = (lane & 15) ^ (2 * ks_f(k));
            va[i] = c0 + c * 8 < g.a_cols ? k * (uint32_t)(g.lda * 2) + c * 16 : OOB;
            ka[i] = k;
        }
    }
    if constexpr (LB == OP_KC) {
        const KcLane l(lane, g.ldb);
        const int q = wave * BSEG * 8;  // first LDS row
        int64_t r0 = n0 + q;
        int64_t lim = g.N;
        if constexpr (EPI == EPI_GATE) {
            r0 = n0 + (q & 127) + (q >= 128 ? g.f : 0);
            lim = q >= 128 ? 2 * (int64_t)g.f : g.f;
        }
        pb = (const uint8_t*)(g.b + r0 * g.ldb) + (int64_t)ks0 * 128;
#pragma unroll
        for (int i = 0; i < BSEG; ++i) {
            vb[i] = r0 + 8 * i + l.row < lim ? l.off + (uint32_t)(8 * i * g.ldb * 2) : OOB;
            kb[i] = l.k;
        }
    } else {
        const int img = wave * BSEG / 16, k0 = (wave * BSEG % 16) * 4;
        const int64_t c0 = n0 + img * 128;
        pb = (const uint8_t*)(g.b + c0) + (int64_t)ks0 * DBK * g.ldb * 2;
#pragma unroll
        for (int i = 0; i < BSEG; ++i) {
            const uint32_t k = k0 + 4 * i + (lane >> 4), c = (lane & 15) ^ (2 * ks_f(k));
            vb[i] = c0 + c * 8 < g.b_cols ? k * (uint32_t)(g.ldb * 2) + c * 16 : OOB;
            kb[i] = k;
        }
    }
    const int64_t step_a = LA == OP_KC ? 128 : (int64_t)DBK * g.lda * 2;
    const int64_t step_b = LB == OP_KC ? 128 : (int64_t)DBK * g.ldb * 2;
    auto issue = [&](int st, int ks) {
        const uint32_t left = (uint32_t)(g.K - ks * DBK);
        const u32x4 da = buf_desc(pa), db = buf_desc(pb);
        const uint32_t sA = sbase + st * STAGE + wave * ASEG * 1024;
        const uint32_t sB = sbase + st * STAGE + A_BYTES + wave * BSEG * 1024;
#pragma unroll
        for (int i = 0; i < ASEG; ++i) dma16b(da, ka[i] < left ? va[i] : OOB, sA + i * 1024);
#pragma unroll
        for (int i = 0; i < BSEG; ++i) dma16b(db, kb[i] < left ? vb[i] : OOB, sB + i * 1024);
        pa += step_a;
        pb += step_b;
    };

    // fragment read offsets
    uint32_t ra[4], rb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (LA == OP_KC)
            ra[i] = kc_frag(lane, wm * 64 + i * 16);
        else
            ra[i] = (wm >> 1) * 16384 + ks_frag(lane, (wm & 1) * 4 + i);
        if constexpr (EPI == EPI_GATE)
            rb[i] = A_BYTES + kc_frag(lane, (i >> 1) * 128 + wn * 32 + (i & 1) * 16);
        else if constexpr (LB == OP_KC)
            rb[i] = A_BYTES + kc_frag(lane, wn * 64 + i * 16);
        else
            rb[i] = A_BYTES + (wn >> 1) * 16384 + ks_frag(lane, (wn & 1) * 4 + i);
    }
    auto frag = [&](auto layout, uint32_t addr, int s) {
        if constexpr (decltype(layout)::value == OP_KC) {
            return lds16<0>(addr ^ (s * 64));
        } else {
            const v2u lo = lds_tr16<0>(addr + s * 8192), hi = lds_tr16<1024>(addr + s * 8192);
            return u32x4{lo.x, lo.y, hi.x, hi.y};
        }
    };

    v4f acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    issue(0, ks0);
    for (int ks = ks0; ks < ks1; ++ks) {
        const int st = (ks - ks0) & 1;
        if (ks + 1 < ks1) {
            issue(st ^ 1, ks + 1);
            wait_vmcnt<ASEG + BSEG>();
        } else {
            wait_vmcnt<0>();
        }
        phase_barrier();
        uint32_t sX = sbase + st * STAGE;
        pin(sX);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            u32x4 fa[4], fb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // KC offsets are added before the s flip: stages are 1 KB aligned
                fa[i] = frag(std::integral_constant<int, LA>{}, sX + ra[i], s);
                fb[i] = frag(std::integral_constant<int, LB>{}, sX + rb[i], s);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = mfma_bf16(fb[j], fa[i], acc[i][j]);
        }
        wait_lgkm0();
        phase_barrier();  // every wave has read this stage: the next issue may overwrite it
    }

    // ---- epilogue: this lane holds C[m][n .. n + 3]
    const int l15 = lane & 15, g4 = (lane >> 4) * 4;
    if constexpr (EPI == EPI_GATE) {
        const int nb = n0 + wn * 32 + g4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) add_gate_bias(g, nb + j * 16, acc[i][j], acc[i][j + 2]);
        if (g.save == MOE_SAVE_INT8) {
            uint32_t* rowmax = reinterpret_cast<uint32_t*>(smem);  // [4 waves][2][BM]
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint32_t mx = 0;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) mx = umax(mx, abs_bits(acc[i][2 * w + j][r]));
                    mx = umax(mx, (uint32_t)__shfl_xor((int)mx, 16));
                    mx = umax(mx, (uint32_t)__shfl_xor((int)mx, 32));
                    if (lane < 16) rowmax[(wn * 2 + w) * BM + wm * 64 + i * 16 + l15] = mx;
                }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = wm * 64 + i * 16 + l15;
                const int64_t m = m0 + r;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint32_t mx = 0;
#pragma unroll
                    for (int v = 0; v < 4; ++v) mx = umax(mx, rowmax[(v * 2 + w) * BM + r]);
                    const Keep8 k = keep8_scale(mx);
                    if (m >= g.M) continue;
                    if (wn == 0 && lane < 16) g.gu_s[((int64_t)(w * (g.f >> 7)) + nt) * g.M + m] = k.s;
                    int8_t* q = (int8_t*)g.gu + m * (2 * (int64_t)g.f) + (int64_t)w * g.f + nb;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const v4f v = acc[i][2 * w + j];
                        *reinterpret_cast<uint32_t*>(q + j * 16) =
                            pack_s8x4(keep8_code(v.x, k.inv), keep8_code(v.y, k.inv), keep8_code(v.z, k.inv),
                                      keep8_code(v.w, k.inv));
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + wm * 64 + i * 16 + l15;
            if (m >= g.M) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j) epi_gate(g, m, nb + j * 16, acc[i][j], acc[i][j + 2]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + wm * 64 + i * 16 + l15;
            if (m >= g.M) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + wn * 64 + j * 16 + g4;
                if constexpr (EPI == EPI_LINEAR)
                    epi_linear(g, m, n, acc[i][j]);
                else if constexpr (EPI == EPI_DGATE)
                    epi_dgate(g, m, n, acc[i][j]);
                else if (n < g.part_ld)
                    *reinterpret_cast<v4f*>(g.part + ((int64_t)split * g.M + m) * g.part_ld + n) = acc[i][j];
            }
        }
    }
}

// ---------------------------------------------------------------- split K: sum and epilogue
// One thread per four columns; the pieces are added in order.
template <int EPI>
__global__ __launch_bounds__(256) void dense_sum_kernel(DenseArgs g, int splits) {
    const int cols = EPI == EPI_GATE ? g.f : (int)g.part_ld;
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = idx / (cols / 4);
    const int n = (int)(idx - m * (cols / 4)) * 4;
    const bool on = m < g.M;
    const int64_t plane = (int64_t)g.M * g.part_ld;
    auto sum = [&](int col) {
        v4f s = {0.f, 0.f, 0.f, 0.f};
        if (on) {
            const float* p = g.part + m * g.part_ld + col;
            for (int i = 0; i < splits; ++i) s += *reinterpret_cast<const v4f*>(p + i * plane);
        }
        return s;
    };
    if constexpr (EPI == EPI_GATE) {
        v4f G = sum(n), U = sum(g.f + n);
        if (on) add_gate_bias(g, n, G, U);
        if (g.save == MOE_SAVE_INT8) {
            // f % 128 == 0: 32 lanes hold one block of a row
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
        if (on) epi_gate(g, m, n, G, U);
    } else {
        if (!on) return;
        const v4f s = sum(n);
        if constexpr (EPI == EPI_DGATE)
            epi_dgate(g, m, n, s);
        else
            epi_linear(g, m, n, s);
    }
}

// ---------------------------------------------------------------- host side
namespace {
struct Shape {
    int64_t mt, nt;
    int bm, bn;  // bn: columns of C (h columns for EPI_GATE)
    int splits, ksteps;
};
// Tiles and K splits of an M x N product over K.  A product with fewer tiles
// than two per compute unit is split along K, each piece at least 8 K steps.
Shape dense_shape(int64_t M, int64_t N, int64_t K, int epi) {
    Shape s;
    const int64_t cols = epi == EPI_GATE ? N / 2 : N;
    s.bm = epi == EPI_GATE ? 64 : 128;
    s.bn = 128;
    s.mt = (M + s.bm - 1) / s.bm;
    s.nt = (cols + s.bn - 1) / s.bn;
    const int64_t steps = (K + DBK - 1) / DBK;
    const int64_t want = 2 * num_cus();
    int64_t sp = 1;
    // pieces go through 128 x 128 tiles
    const int64_t tiles = (M + 127) / 128 * ((N + 127) / 128);
    if (tiles * 2 <= want) sp = want / tiles;
    if (sp > steps / 8) sp = steps / 8;
    if (sp > 32) sp = 32;
    if (sp < 1) sp = 1;
    s.ksteps = (int)((steps + sp - 1) / sp);
    s.splits = (int)((steps + s.ksteps - 1) / s.ksteps);
    if (s.splits > 1) {
        s.bm = 128;
        s.mt = (M + 127) / 128;
        s.nt = (N + 127) / 128;
    }
    return s;
}
template <int WM, int WN, int LA, int LB, int EPI>
int launch_one(const DenseArgs& g, int splits, hipStream_t stream) {
    const int64_t grid = (int64_t)g.mt * g.nt * splits;
    dense_kernel<WM, WN, LA, LB, EPI><<<dim3((unsigned)grid), dim3(WM * WN * 64), 0, stream>>>(g);
    MOE_LAUNCH_CHECK("dense_kernel");
    return MOE_OK;
}
template <int EPI>
int launch_sum(const DenseArgs& g, int splits, hipStream_t stream) {
    const int64_t cols = EPI == EPI_GATE ? g.f : g.part_ld;
    const int64_t blocks = ((int64_t)g.M * (cols / 4) + 255) / 256;
    dense_sum_kernel<EPI><<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(g, splits);
    MOE_LAUNCH_CHECK("dense_sum_kernel");
    return MOE_OK;
}
template <int EPI>
int launch_layout(const DenseArgs& g, int la, int lb, int splits, hipStream_t stream) {
    if (la == OP_KC && lb == OP_KC) return launch_one<2, 2, OP_KC, OP_KC, EPI>(g, splits, stream);
    if (la == OP_KC) return launch_one<2, 2, OP_KC, OP_KS, EPI>(g, splits, stream);
    return launch_one<2, 2, OP_KS, OP_KS, EPI>(g, splits, stream);
}
}  // namespace

size_t dense_ws(int64_t M, int64_t N, int64_t K, int epi) {
    if (M <= 0 || N <= 0 || K <= 0) return 0;  // T = 0
    const Shape s = dense_shape(M, N, K, epi);
    return s.splits > 1 ? (size_t)s.splits * M * round_up(N, 4) * 4 : 0;
}

int dense_launch(DenseArgs g, int la, int lb, int epi, void* ws, size_t ws_bytes, hipStream_t stream) {
    const Shape s = dense_shape(g.M, g.N, g.K, epi);
    MOE_REQUIRE(s.mt * s.nt * s.splits < (1ll << 31), MOE_ERR_SHAPE, "product of %d x %d has too many tiles", g.M, g.N);
    g.mt = (int)s.mt;
    g.nt = (int)s.nt;
    g.ksteps = s.ksteps;
    if (s.splits > 1) {
        MOE_REQUIRE(ws && ws_bytes >= dense_ws(g.M, g.N, g.K, epi), MOE_ERR_WORKSPACE, "workspace too small");
        g.part = (float*)ws;
        g.part_ld = round_up(g.N, 4);
        const int rc = launch_layout<EPI_PART>(g, la, lb, s.splits, stream);
        if (rc != MOE_OK) return rc;
        if (epi == EPI_GATE) return launch_sum<EPI_GATE>(g, s.splits, stream);
        if (epi == EPI_DGATE) return launch_sum<EPI_DGATE>(g, s.splits, stream);
        return launch_sum<EPI_LINEAR>(g, s.splits, stream);
    }
    if (epi == EPI_GATE) return launch_one<1, 4, OP_KC, OP_KC, EPI_GATE>(g, 1, stream);
    if (epi == EPI_DGATE) return launch_one<2, 2, OP_KC, OP_KS, EPI_DGATE>(g, 1, stream);
    return launch_layout<EPI_LINEAR>(g, la, lb, 1, stream);
}

// ---------------------------------------------------------------- column sums, zeros
namespace {
constexpr int CS_ROWS = 64;  // least rows of one partial sum
int64_t colsum_chunks(int64_t T) {
    int64_t c = (T + CS_ROWS - 1) / CS_ROWS;
    return c > 256 ? 256 : (c < 1 ? 1 : c);
}
}  // namespace

// Partial column sums (fp32) of src over a chunk of rows: a wave takes 256
// columns, the four waves every fourth row.
__global__ __launch_bounds__(256) void colsum_kernel(const uint16_t* src, int64_t ld, int64_t T, int64_t N,
                                                     int64_t rows, float* part) {
    __shared__ float sm[4][256];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t n = (int64_t)blockIdx.x * 256 + lane * 4;
    const int64_t t1 = min((int64_t)(blockIdx.y + 1) * rows, T);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (n < N) {
        for (int64_t t = (int64_t)blockIdx.y * rows + w; t < t1; t += 4) {
            float v[4];
            load_bf16x4(src + t * ld + n, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += v[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sm[w][lane * 4 + i] = s[i];
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c < N)
        part[blockIdx.y * N + c] =
            (sm[0][threadIdx.x] + sm[1][threadIdx.x]) + (sm[2][threadIdx.x] + sm[3][threadIdx.x]);
}

// out[n] = bf16 of the chunks' sums, added in order
__global__ __launch_bounds__(256) void colsum_finish_kernel(const float* part, int chunks, int64_t ld, int64_t N,
                                                            uint16_t* out) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    float s = 0.f;
    for (int c = 0; c < chunks; ++c) s += part[c * ld + n];
    out[n] = (uint16_t)cvt_bf16x2(s, 0.f);
}

__global__ __launch_bounds__(256) void zero16_kernel(uint16_t* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

size_t colsum_ws(int64_t T, int64_t N) { return (size_t)colsum_chunks(T) * N * 4; }

int colsum_finish(const float* part, int chunks, int64_t ld, int64_t N, uint16_t* out, hipStream_t stream) {
    colsum_finish_kernel<<<dim3((unsigned)((N + 255) / 256)), dim3(256), 0, stream>>>(part, chunks, ld, N, out);
    MOE_LAUNCH_CHECK("colsum_finish_kernel");
    return MOE_OK;
}

int colsum_launch(const uint16_t* src, int64_t ld, int64_t T, int64_t N, uint16_t* out, float* part,
                  hipStream_t stream) {
    const int chunks = (int)colsum_chunks(T);
    const int64_t rows = (T + chunks - 1) / chunks;
    colsum_kernel<<<dim3((unsigned)((N + 255) / 256), chunks), dim3(256), 0, stream>>>(src, ld, T, N, rows, part);
    MOE_LAUNCH_CHECK("colsum_kernel");
    return colsum_finish(part, chunks, N, N, out, stream);
}

int zero16_launch(uint16_t* p, int64_t n, hipStream_t stream) {
    const int64_t blocks = (n + 255) / 256;
    zero16_kernel<<<dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream>>>(p, n);
    MOE_LAUNCH_CHECK("zero16_kernel");
    return MOE_OK;
}

// dz = dy * act'(pre) of moe_linear_backward: bf16 rows of stride ldz (columns
// past N zero) and, if part is given, fp32 column sums over chunks of rows
// (summed before the rounding).  One thread per four columns of a row.
__global__ __launch_bounds__(256) void dz_kernel(const void* dy, int dy_f32, const uint16_t* pre, int act, int64_t T,
                                                 int64_t N, int64_t ldz, int64_t rows, uint16_t* dz, float* part) {
    __shared__ float sm[4][256];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t n = (int64_t)blockIdx.x * 256 + lane * 4;
    const int64_t t1 = min((int64_t)(blockIdx.y + 1) * rows, T);
    const bool vec = (N & 3) == 0;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (n < ldz) {
        for (int64_t t = (int64_t)blockIdx.y * rows + w; t < t1; t += 4) {
            float v[4] = {0.f, 0.f, 0.f, 0.f}, p[4] = {0.f, 0.f, 0.f, 0.f};
            const int64_t at = t * N + n;
            if (vec) {
                if (n < N) {
                    if (dy_f32) {
                        const v4f q = *reinterpret_cast<const v4f*>((const float*)dy + at);
                        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
                    } else {
                        load_bf16x4((const uint16_t*)dy + at, v);
                    }
                    if (pre) load_bf16x4(pre + at, p);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < N) {
                        v[i] = dy_f32 ? ((const float*)dy)[at + i] : bf16_to_f32(((const uint16_t*)dy)[at + i]);
                        if (pre) p[i] = bf16_to_f32(pre[at + i]);
                    }
            }
            if (act != MOE_ACT_NONE) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float val, sl;
                    act_both(act, p[i], val, sl);
                    v[i] *= sl;
                }
            }
            if (dz) *reinterpret_cast<v2u*>(dz + t * ldz + n) = pack_bf16x4(v[0], v[1], v[2], v[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += v[i];
        }
    }
    if (!part) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) sm[w][lane * 4 + i] = s[i];
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c < ldz)
        part[blockIdx.y * ldz + c] =
            (sm[0][threadIdx.x] + sm[1][threadIdx.x]) + (sm[2][threadIdx.x] + sm[3][threadIdx.x]);
}

int dz_launch(const void* dy, int dy_f32, const uint16_t* pre, int act, int64_t T, int64_t N, int64_t ldz, uint16_t* dz,
              float* part, uint16_t* dbias, hipStream_t stream) {
    const int chunks = (int)colsum_chunks(T);
    const int64_t rows = (T + chunks - 1) / chunks;
    dz_kernel<<<dim3((unsigned)((ldz + 255) / 256), chunks), dim3(256), 0, stream>>>(
        dy, dy_f32, pre, act, T, N, ldz, rows, dz, dbias ? part : nullptr);
    MOE_LAUNCH_CHECK("dz_kernel");
    return dbias ? colsum_finish(part, chunks, ldz, N, dbias, stream) : MOE_OK;
}

}  // namespace moe
