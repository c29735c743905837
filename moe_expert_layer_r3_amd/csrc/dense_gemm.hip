// bf16 matrix products with fused epilogues (dense_gemm.hpp): the kernels and
// the choice between them.
#include "dense_gemm.hpp"

namespace moe {

// Tile index of a workgroup: XCD x runs a contiguous eighth of the tiles, which
// go m fastest inside groups of 8 m-tiles, so that the tiles an XCD runs side by
// side share few A and B tiles in its L2.
__device__ __forceinline__ void dense_tile(const DenseArgs& g, int bid, int tiles, int& mt, int& nt, int& split) {
    const int per = g.mt * g.nt;
    const int t0 = (int)xcd_tile(bid, tiles);
    split = t0 / per;
    const int t = t0 - split * per;
    constexpr int GM = 8;
    const int grp = t / (GM * g.nt);
    const int gm = min(GM, g.mt - grp * GM);
    const int in = t - grp * GM * g.nt;
    // uniform values, kept in SGPRs so that operand addresses are scalar arithmetic
    split = __builtin_amdgcn_readfirstlane(split);
    nt = __builtin_amdgcn_readfirstlane(in / gm);
    mt = __builtin_amdgcn_readfirstlane(grp * GM + in - nt * gm);
}

// v4f of four columns of a row of bf16 or fp32, zeros past its end; at: the first
// one's index, left: the row's columns from there (it may be none); VEC: rows are of
// whole fours.  What is past the end is read from the row's last columns and dropped:
// branches would split a loop's loads (dz of 203 x 1001: 6.6 us with them, 4.6 without).
template <bool F32, bool VEC>
__device__ __forceinline__ v4f load4(const void* src, int64_t at, int left) {
    float v[4];
    if constexpr (VEC) {
        const int64_t a = at + min(0, left - 4);
        if constexpr (F32) {
            const v4f w = *reinterpret_cast<const v4f*>((const float*)src + a);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = w[i];
        } else {
            load_bf16x4((const uint16_t*)src + a, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t a = at + min(i, left - 1);
            v[i] = F32 ? ((const float*)src)[a] : bf16_to_f32(((const uint16_t*)src)[a]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < left ? v[i] : 0.f;
    return v4f{v[0], v[1], v[2], v[3]};
}

// Epilogue of ROWS x COLS fp32 results that the workgroup has put into LDS: rows
// leave in order, 16 bytes of LDS (four columns) per thread and step, so that
// global accesses are whole lines and the element-wise code exists once (written
// out for every accumulator register it is too long to be unrolled).
// 16-byte chunk c of row r lies at c ^ (r & 15), which spreads the 16 rows that a
// wave's accumulators write together over the banks.
__device__ __forceinline__ uint32_t stage_at(int cols, int r, int c) { return (uint32_t)(r * cols * 4 + ((c ^ (r & 15)) << 4)); }

template <int EPI, int ROWS, int COLS, int THREADS>
struct TileEpilogue {
    static constexpr int PER_ROW = (EPI == EPI_GATE ? COLS / 2 : COLS) / 4, STEPS = ROWS * PER_ROW / THREADS;
    // What the steps read from memory is loaded a batch ahead (the first one before
    // the results are staged).  The loop stays rolled: its code is long.
    static constexpr bool READS = EPI == EPI_LINEAR || is_dgate(EPI) || EPI == EPI_PLAIN;
    static constexpr int BATCH = EPI == EPI_PLAIN && STEPS % 8 == 0 ? 8 : STEPS < 4 ? STEPS : 4;
    static_assert(STEPS % BATCH == 0, "whole batches");
    EpiIn<EPI> in[READS ? BATCH : 1];
    EpiBias<EPI> bias;
    // this thread's first row; where a wave takes one row, a scalar
    static __device__ __forceinline__ int first_row() {
        const int r = threadIdx.x / PER_ROW;
        return PER_ROW % 64 == 0 ? __builtin_amdgcn_readfirstlane(r) : r;
    }
    __device__ __forceinline__ void load(const DenseArgs& g, int64_t m0, int n0, int s = 0) {
        if (s == 0) bias.load(g, n0 + threadIdx.x % PER_ROW * 4);
        if constexpr (READS) {
            const int c = threadIdx.x % PER_ROW, r0 = first_row();
#pragma unroll
            for (int i = 0; i < BATCH; ++i) in[i].load(g, m0 + (s + i) * (THREADS / PER_ROW) + r0, n0 + c * 4);
        }
    }
    __device__ __forceinline__ void step(const DenseArgs& g, const uint8_t* sm, int64_t m0, int n0, int split, int s,
                                         const EpiIn<EPI>& in) {
        const int c = threadIdx.x % PER_ROW, r = s * (THREADS / PER_ROW) + first_row();
        const int n = n0 + c * 4;
        const int64_t m = m0 + r;
        const v4f v = *reinterpret_cast<const v4f*>(sm + stage_at(COLS, r, c));
        if constexpr (EPI == EPI_GATE) {
            const v4f u = *reinterpret_cast<const v4f*>(sm + stage_at(COLS, r, c + PER_ROW));
            epi_gate(g, m, n, v, u, bias, m < g.M && n < g.f);
        } else if constexpr (EPI == EPI_LINEAR) {
            if (m < g.M && n < g.N) epi_linear(g, m, n, v, in, bias);
        } else if constexpr (EPI == EPI_PLAIN) {
            if (m < g.M && n < g.N) epi_plain(g, m, n, v, in, bias);
        } else if constexpr (is_dgate(EPI)) {
            if (m < g.M && n < g.f) epi_dgate(g, m, n, v, in);
        } else {
            if (m < g.M && n < g.part_ld)
                *reinterpret_cast<v4f*>(g.part + ((int64_t)split * g.M + m) * g.part_ld + n) = v;
        }
    }
    __device__ __forceinline__ void run(const DenseArgs& g, const uint8_t* sm, int64_t m0, int n0, int split) {
#pragma unroll 1
        for (int s = 0; s < STEPS; s += BATCH) {
            TileEpilogue next;
            next.bias = bias;
            if (READS && s + BATCH < STEPS) next.load(g, m0, n0, s + BATCH);
#pragma unroll
            for (int i = 0; i < BATCH; ++i) step(g, sm, m0, n0, split, s + i, in[READS ? i : 0]);
            *this = next;
        }
    }
};

// ---------------------------------------------------------------- 64 x 64 wave tiles
// WM x WN waves of 64 x 64, K steps of 64 double-buffered in LDS: while a step is
// multiplied the next one is on its way.  Two workgroups per compute unit hide each
// other's barriers: 12000 x 600 over 1200 in 29 us (0.60 PFLOP/s; 128 x 256 tiles 39 us,
// whose last round is emptier).  Bound by the wait for the LDS DMA, which one step of
// look-ahead does not cover.
template <int WM, int WN, int LA, int LB, int EPI>
__global__ __launch_bounds__(WM * WN * 64) void dense_kernel(DenseArgs g) {
    constexpr int BM = WM * 64, BN = WN * 64, NW = WM * WN;
    constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
    constexpr int ASEG = BM / 8 / NW, BSEG = BN / 8 / NW;
    static_assert(ASEG % 2 == 0 && BSEG % 2 == 0, "segments move in pairs");
    static_assert(LA == OP_KC || BM % 128 == 0, "KS images are 128 columns wide");
    static_assert(LB == OP_KC || BN % 128 == 0, "KS images are 128 columns wide");
    static_assert(EPI != EPI_GATE || (WN == 4 && LB == OP_KC), "gated tiles pair 128 G with 128 U columns");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * STAGE];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    int mt, nt, split;
    dense_tile(g, blockIdx.x, gridDim.x, mt, nt, split);
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
        for (int i = 0; i < ASEG; i += 2)
            dma16b2(da, ka[i] < left ? va[i] : OOB, ka[i + 1] < left ? va[i + 1] : OOB, sA + i * 1024);
#pragma unroll
        for (int i = 0; i < BSEG; i += 2)
            dma16b2(db, kb[i] < left ? vb[i] : OOB, kb[i + 1] < left ? vb[i + 1] : OOB, sB + i * 1024);
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

    // ---- epilogue: this lane holds C[m][n .. n + 3]; the K loop's last barrier freed LDS
    const int l15 = lane & 15, g4 = lane >> 4;
    TileEpilogue<EPI, BM, BN, NW * 64> epi;
    epi.load(g, m0, n0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = EPI == EPI_GATE ? (j >> 1) * 128 + wn * 32 + (j & 1) * 16 : wn * 64 + j * 16;
            *reinterpret_cast<v4f*>(smem + stage_at(BN, wm * 64 + i * 16 + l15, col / 4 + g4)) = acc[i][j];
        }
    __syncthreads();
    epi.run(g, smem, m0, n0, split);
}

// ---------------------------------------------------------------- 64 x 64 tiles
// Small problems, where a K loop's time is its loads' latency: four waves of 32 x 32,
// a ring of five K steps in LDS (80 KB, two workgroups per compute unit), four of
// them in flight while one is multiplied, one barrier per step.  1237 x 688 over 1032
// takes 7.8 us (0.22 PFLOP/s): its 17 steps are 3.7 us, launch, first loads and
// epilogue the rest.
constexpr int RING = 5, SMALL_STAGE = 16384;  // A, B: 64 rows (columns) of a step
template <int LA, int LB, int EPI>
__device__ __forceinline__ void small_tile(const DenseArgs& g, int bid, int tiles, uint8_t* smem) {
    constexpr int STAGE = SMALL_STAGE, HALF = STAGE / 2;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    int mt, nt, split;
    dense_tile(g, bid, tiles, mt, nt, split);
    const int64_t m0 = (int64_t)mt * 64;
    const int n0 = nt * (EPI == EPI_GATE ? 32 : 64);
    const int ks0 = split * g.ksteps;
    const int ks1 = min(ks0 + g.ksteps, (g.K + DBK - 1) / DBK);
    const int kend = min(g.K, ks1 * DBK);
    const uint32_t sbase = __builtin_amdgcn_readfirstlane(lds_addr(smem));

    // DMA: wave w moves segments 2w, 2w + 1 of both operands: KC rows 16w .. + 15, KS
    // K rows 16w .. + 15
    uint32_t va[2], vb[2];
    const uint8_t *pa, *pb;
    const KcLane la(lane, g.lda), lb(lane, g.ldb);
    const uint32_t kseg = wave * 16 + (lane >> 3);  // KS: K row of segment 2w, + 8 of 2w + 1
    auto ks_off = [&](int i, int64_t c0, int cols, int64_t ld) {
        const uint32_t k = kseg + 8 * i, c = (lane & 7) ^ (2 * ks_f64(k));
        return c0 + c * 8 < cols ? k * (uint32_t)(ld * 2) + c * 16 : OOB;
    };
    if constexpr (LA == OP_KC) {
        const int64_t r0 = m0 + wave * 16;
        pa = (const uint8_t*)(g.a + r0 * g.lda);
#pragma unroll
        for (int i = 0; i < 2; ++i) va[i] = r0 + 8 * i + la.row < g.M ? la.off + (uint32_t)(8 * i * g.lda * 2) : OOB;
    } else {
        pa = (const uint8_t*)(g.a + m0);
#pragma unroll
        for (int i = 0; i < 2; ++i) va[i] = ks_off(i, m0, g.a_cols, g.lda);
    }
    if constexpr (LB == OP_KC) {
        int64_t r0 = n0 + wave * 16, lim = g.N;
        if constexpr (EPI == EPI_GATE) {  // 32 G rows, then the 32 U rows of the same h columns
            r0 = n0 + (wave & 1) * 16 + (wave >> 1) * (int64_t)g.f;
            lim = (wave >> 1) ? 2 * (int64_t)g.f : g.f;
        }
        pb = (const uint8_t*)(g.b + r0 * g.ldb);
#pragma unroll
        for (int i = 0; i < 2; ++i) vb[i] = r0 + 8 * i + lb.row < lim ? lb.off + (uint32_t)(8 * i * g.ldb * 2) : OOB;
    } else {
        pb = (const uint8_t*)(g.b + n0);
#pragma unroll
        for (int i = 0; i < 2; ++i) vb[i] = ks_off(i, n0, g.b_cols, g.ldb);
    }
    const int64_t step_a = LA == OP_KC ? 128 : (int64_t)DBK * g.lda * 2;
    const int64_t step_b = LB == OP_KC ? 128 : (int64_t)DBK * g.ldb * 2;
    // steps past the end fill zeros without reading memory
    auto issue = [&](int slot, int ks) {
        const int left = kend - ks * DBK;
        const u32x4 da = buf_desc(pa + ks * step_a), db = buf_desc(pb + ks * step_b);
        const uint32_t s = sbase + slot * STAGE + wave * 2048;
        const int a0 = LA == OP_KC ? (int)la.k : (int)kseg, a1 = LA == OP_KC ? a0 : a0 + 8;
        const int b0 = LB == OP_KC ? (int)lb.k : (int)kseg, b1 = LB == OP_KC ? b0 : b0 + 8;
        dma16b2(da, a0 < left ? va[0] : OOB, a1 < left ? va[1] : OOB, s);
        dma16b2(db, b0 < left ? vb[0] : OOB, b1 < left ? vb[1] : OOB, s + HALF);
    };

    uint32_t ra[2], rb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        ra[i] = LA == OP_KC ? kc_frag(lane, wm * 32 + i * 16) : ks_frag64(lane, wm * 2 + i);
        const int c = EPI == EPI_GATE ? i * 32 + wn * 16 : wn * 32 + i * 16;
        rb[i] = HALF + (LB == OP_KC ? kc_frag(lane, c) : ks_frag64(lane, c / 16));
    }
    auto frag = [&](auto layout, uint32_t addr, auto sc) {
        constexpr int s = decltype(sc)::value;
        if constexpr (decltype(layout)::value == OP_KC) {
            return lds16<0>(addr ^ (s * 64));
        } else {
            const v2u lo = lds_tr16<s * 4096>(addr), hi = lds_tr16<s * 4096 + 512>(addr);
            return u32x4{lo.x, lo.y, hi.x, hi.y};
        }
    };
    v4f acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

#pragma unroll
    for (int i = 0; i < RING - 1; ++i) issue(i, ks0 + i);
    int slot = 0;
    for (int ks = ks0; ks < ks1; ++ks) {
        wait_vmcnt<(RING - 2) * 4>();  // this step has landed; the next three are in flight
        wait_lgkm0();
        phase_barrier();  // for every wave, which has also read the previous step
        uint32_t base = sbase + slot * STAGE;
        pin(base);
        u32x4 fa[2][2], fb[2][2];
        static_for<0, 2>([&](auto sc) {
            constexpr int s = decltype(sc)::value;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i][s] = frag(std::integral_constant<int, LA>{}, base + ra[i], sc);
                fb[i][s] = frag(std::integral_constant<int, LB>{}, base + rb[i], sc);
            }
        });
        // the DMA goes out while the fragments are on their way
        issue(slot == 0 ? RING - 1 : slot - 1, ks + RING - 1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = mfma_bf16(fb[j][s], fa[i][s], acc[i][j]);
        slot = slot == RING - 1 ? 0 : slot + 1;
    }
    wait_lgkm0();
    wait_vmcnt<0>();  // the fills past the end have landed
    phase_barrier();

    const int l15 = lane & 15, g4 = lane >> 4;
    TileEpilogue<EPI, 64, 64, 256> epi;
    epi.load(g, m0, n0);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = EPI == EPI_GATE ? j * 32 + wn * 16 : wn * 32 + j * 16;
            *reinterpret_cast<v4f*>(smem + stage_at(64, wm * 32 + i * 16 + l15, col / 4 + g4)) = acc[i][j];
        }
    __syncthreads();
    epi.run(g, smem, m0, n0, split);
}
template <int LA, int LB, int EPI>
__global__ __launch_bounds__(256) void dense_small_kernel(DenseArgs g) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[RING * SMALL_STAGE];
    small_tile<LA, LB, EPI>(g, blockIdx.x, gridDim.x, smem);
}

// Column sums of 32 columns over all rows, as bf16: 8 threads to a row (four columns
// each), 32 rows at a time and eight such loads in flight, added in a fixed order.
template <bool F32, bool VEC>
__device__ __forceinline__ v4f colsum_rows(const ColSum& c, int64_t n, int q) {
    constexpr int R = 8;
    v4f s = {0.f, 0.f, 0.f, 0.f};
    const int left = (int)(c.N - n);
    if (left <= 0) return s;
    for (int64_t t = q; t < c.rows; t += 32 * R) {
        v4f v[R];
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] = load4<F32, VEC>(c.src, min(t + 32 * i, c.rows - 1) * c.ld + n, left);
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (t + 32 * i < c.rows) s += v[i];
    }
    return s;
}
__device__ __forceinline__ void colsum_block(const ColSum& c, int block, uint8_t* smem) {
    float* sm = reinterpret_cast<float*>(smem);  // [32 rows][32 columns]
    const int64_t n = (int64_t)block * 32 + (threadIdx.x & 7) * 4;
    const int q = threadIdx.x >> 3;
    const bool vec = (c.N & 3) == 0;
    const v4f s = c.f32 ? (vec ? colsum_rows<true, true>(c, n, q) : colsum_rows<true, false>(c, n, q))
                        : (vec ? colsum_rows<false, true>(c, n, q) : colsum_rows<false, false>(c, n, q));
#pragma unroll
    for (int i = 0; i < 4; ++i) sm[q * 32 + (threadIdx.x & 7) * 4 + i] = s[i];
    __syncthreads();
    const int64_t m = (int64_t)block * 32 + threadIdx.x;
    if (threadIdx.x < 32 && m < c.N) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += sm[i * 32 + threadIdx.x];
        c.out[m] = (uint16_t)cvt_bf16x2(v, 0.f);
    }
}

// A small problem's gradients in one launch: up to two weight gradients, column
// sums, the data gradient; the longest sums over K first.  None of them fills the
// compute units by itself, and each launch has a few us of its own: the backward of
// a 1032 -> 344 gated block takes 25.7 -> 15.6 us at 64 rows and 45.2 -> 30.0 at 1237
// (5 launches -> 1 behind dG, dU), of a 1024 -> 256 linear layer 12.0 -> 8.5 at 1000
// rows.  Bound by launch and load latency below 200 rows, by the LDS DMA of 64 x 64
// tiles above.  A ring of three or four steps (three workgroups per unit) is no faster.
__global__ __launch_bounds__(256) void dense_group_kernel(DenseGroup g) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[RING * SMALL_STAGE];
    int b = blockIdx.x;
    if (b < g.tiles[1]) {
        small_tile<OP_KS, OP_KS, EPI_PLAIN>(g.dw[0], b, g.tiles[1], smem);
        return;
    }
    b -= g.tiles[1];
    if (b < g.tiles[2]) {
        small_tile<OP_KS, OP_KS, EPI_PLAIN>(g.dw[1], b, g.tiles[2], smem);
        return;
    }
    b -= g.tiles[2];
    if (b < g.sums[0].blocks) return colsum_block(g.sums[0], b, smem);
    b -= g.sums[0].blocks;
    if (b < g.sums[1].blocks) return colsum_block(g.sums[1], b, smem);
    b -= g.sums[1].blocks;
    small_tile<OP_KC, OP_KS, EPI_PLAIN>(g.dx, b, g.tiles[0], smem);
}

// ---------------------------------------------------------------- 256 x 256 tiles
// Eight waves as 2 (M) x 4 (N); a wave owns, of each 128-row half of A and each
// 128-column half of B, 64 rows x 32 columns.  A K step of 64 is two phases of 32
// MFMAs (one half of A against both halves of B), and the two waves of a SIMD (one
// of each M half) run one half-phase apart: while one multiplies, the other reads
// its next fragments from LDS and issues its share of the DMA, so the matrix core
// sees MFMAs throughout.  Barriers separate the half-phases.
//
//   phase   fragments read              multiplies     DMA issued (2 per wave and half)
//     0     A0, B1 of step k             A0 x B0, B1    A1 of step k + 1, B0 of step k + 2
//     1     A1 of step k, B0 of k + 1    A1 x B0, B1    A0, B1 of step k + 2
//
// so that both phases read 12 fragments and issue four instructions per wave.
// Two LDS stages of 64 KB.  A wave's reads are complete before the barrier that
// ends its reading half-phase, so what phase p read is refilled in phase p + 1; a
// refill is awaited (vmcnt(8): those of the last two phases stay in flight) one
// phase before it is read, ahead of a barrier.  Steps past the end fill zeros
// without reading memory, so the counts hold to the last step.
//
// Workgroups are persistent (one per compute unit).  At the end of a tile the DMA of
// the next one's first steps goes out before the results leave, straight from the
// accumulators (DIRECT): lanes trade 16-column pieces (permlane16_swap) so that
// each holds 8 adjacent columns.  The general
// epilogues, too long to be written out for every register, go through LDS.
//
// HM = 1: 128 x 256 tiles, for products with too few 256 x 256 ones.  A K step is
// then one phase (16 fragments read, 32 MFMAs, 6 DMA instructions) and LDS holds
// three stages of 48 KB, so the DMA still runs two steps ahead.
//
// 16384 x 4096 over 7168 (gated, [G, U] saved) takes 654 us, 1.47 PFLOP/s; 16384 x 7168
// over 2048 with a residual 408 us, as a data gradient over 4096 680 us (1.41), 4096 x
// 7168 over 16384 as a weight gradient 699 us (1.38); another card is 7% slower on all.
// The clock is 1.6 to 1.8 GHz under that load (power); the matrix cores are busy 76%
// of the cycles in the first, 57, 67 and 61% in the others; tiles' ends take the rest.
//
// act: the activation of the gated epilogues at compile time (-1: at run time).
constexpr bool is_direct(int epi, int act) {
    return epi == EPI_PLAIN || epi == EPI_PART || ((epi == EPI_GATE || is_dgate(epi)) && act >= 0);
}

// A lane's results after the swap: 8 adjacent columns from n
__device__ __forceinline__ void swap_cols(v4f& a, v4f& b) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        uint32_t x = __float_as_uint(a[r]), y = __float_as_uint(b[r]);
        swap16(x, y);
        a[r] = __uint_as_float(x);
        b[r] = __uint_as_float(y);
    }
}
__device__ __forceinline__ u32x4 pack_bf16x8(const v4f& a, const v4f& b) {
    return u32x4{cvt_bf16x2(a.x, a.y), cvt_bf16x2(a.z, a.w), cvt_bf16x2(b.x, b.y), cvt_bf16x2(b.z, b.w)};
}
__device__ __forceinline__ void unpack_bf16x8(const u32x4& w, v4f& a, v4f& b) {
    a = v4f{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
    b = v4f{bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
}

template <int HM, int LA, int LB, int EPI, int ACT>
__global__ __launch_bounds__(512, 1) void dense_wide_kernel(DenseArgs g, int tiles) {
    constexpr int HALF = 16384, STAGE = (HM + 2) * HALF, BOFF = HM * HALF, STAGES = HM == 2 ? 2 : 3;
    constexpr bool GATE = EPI == EPI_GATE, DIRECT = is_direct(EPI, ACT);
    static_assert(!GATE || LB == OP_KC, "gated tiles pair 128 G with 128 U rows of W13");
    // A wave's 32 columns of half b of B begin at wn WSTEP + b HSTEP: 64 adjacent
    // columns for KC operands, whose rows may be dealt at will; a KS operand's 128
    // columns of a half stay adjacent (64-byte pieces of its rows cost 5%)
    constexpr int WSTEP = LB == OP_KC && !GATE ? 64 : 32, HSTEP = LB == OP_KC && !GATE ? 32 : 128;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[STAGES * STAGE];
    // EPI_GATE with the 8-bit save: row maxima [wave column][G, U][row]
    __shared__ uint32_t rowmax[GATE && DIRECT ? 4 : 1][2][HM * 128];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int l15 = lane & 15, g4 = lane >> 4;
    const uint32_t sbase = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    const int64_t step_a = LA == OP_KC ? 128 : (int64_t)DBK * g.lda * 2;
    const int64_t step_b = LB == OP_KC ? 128 : (int64_t)DBK * g.ldb * 2;

    // ---- the current tile
    int64_t m0 = 0;
    int n0 = 0, split = 0, ks0 = 0, ks1 = 0, kend = 0;
    // DMA: wave w moves segments 2w, 2w + 1 of every half: KC rows 16w .. + 15 (one
    // K chunk per lane), KS K rows 8w .. + 7
    uint32_t va[HM][2], vb[2][2];
    const uint8_t *pa[HM], *pb[2];
    const KcLane la(lane, g.lda), lb(lane, g.ldb);
    const uint32_t kseg = wave * 8 + (lane >> 4);  // KS: K row of segment 0, + 4 of segment 1
    auto setup = [&](int t) {
        int mt, nt;
        dense_tile(g, t, tiles, mt, nt, split);
        m0 = (int64_t)mt * (HM * 128);
        n0 = nt * (GATE ? 128 : 256);
        ks0 = split * g.ksteps;
        ks1 = min(ks0 + g.ksteps, (g.K + DBK - 1) / DBK);
        kend = min(g.K, ks1 * DBK);
#pragma unroll
        for (int h = 0; h < HM; ++h) {
            if constexpr (LA == OP_KC) {
                const int64_t r0 = m0 + h * 128 + wave * 16;
                pa[h] = (const uint8_t*)(g.a + r0 * g.lda);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    va[h][i] = r0 + 8 * i + la.row < g.M ? la.off + (uint32_t)(8 * i * g.lda * 2) : OOB;
            } else {
                const int64_t c0 = m0 + h * 128;
                pa[h] = (const uint8_t*)(g.a + c0);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t k = kseg + 4 * i, c = (lane & 15) ^ (2 * ks_f(k));
                    va[h][i] = c0 + c * 8 < g.a_cols ? k * (uint32_t)(g.lda * 2) + c * 16 : OOB;
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // (EPI_GATE: half 0 is G, half 1 U)
            if constexpr (LB == OP_KC) {
                const int64_t r0 = GATE ? (int64_t)h * g.f + n0 + wave * 16
                                        : n0 + (wave >> 1) * WSTEP + h * HSTEP + (wave & 1) * 16;
                const int64_t lim = GATE ? (int64_t)(h + 1) * g.f : g.N;
                pb[h] = (const uint8_t*)(g.b + r0 * g.ldb);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    vb[h][i] = r0 + 8 * i + lb.row < lim ? lb.off + (uint32_t)(8 * i * g.ldb * 2) : OOB;
            } else {
                const int64_t c0 = n0 + h * 128;
                pb[h] = (const uint8_t*)(g.b + c0);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t k = kseg + 4 * i, c = (lane & 15) ^ (2 * ks_f(k));
                    vb[h][i] = c0 + c * 8 < g.b_cols ? k * (uint32_t)(g.ldb * 2) + c * 16 : OOB;
                }
            }
        }
    };
    // half h of A (B) of K step ks into stage st
    auto issue_a = [&](int st, int h, int ks) {
        const int left = kend - ks * DBK;
        const u32x4 d = buf_desc(pa[h] + ks * step_a);
        const uint32_t s = sbase + st * STAGE + h * HALF + wave * 2048;
        const int k0 = LA == OP_KC ? (int)la.k : (int)kseg, k1 = LA == OP_KC ? (int)la.k : (int)kseg + 4;
        dma16b2(d, k0 < left ? va[h][0] : OOB, k1 < left ? va[h][1] : OOB, s);
    };
    auto issue_b = [&](int st, int h, int ks) {
        const int left = kend - ks * DBK;
        const u32x4 d = buf_desc(pb[h] + ks * step_b);
        const uint32_t s = sbase + st * STAGE + BOFF + h * HALF + wave * 2048;
        const int k0 = LB == OP_KC ? (int)lb.k : (int)kseg, k1 = LB == OP_KC ? (int)lb.k : (int)kseg + 4;
        dma16b2(d, k0 < left ? vb[h][0] : OOB, k1 < left ? vb[h][1] : OOB, s);
    };

    // fragment read offsets in a half.  KC: 16-row subtiles are 2048 apart, the
    // two K halves of a step one bit (64) apart.  KS: per subtile, K halves 8192
    // apart.
    uint32_t ra[4], rb[2];
    if constexpr (LA == OP_KC) {
        ra[0] = kc_frag(lane, wm * 64);
        ra[1] = ra[0] ^ 64;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) ra[i] = ks_frag(lane, wm * 4 + i);
    }
    if constexpr (LB == OP_KC) {
        rb[0] = BOFF + kc_frag(lane, wn * 32);
        rb[1] = rb[0] ^ 64;
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) rb[j] = BOFF + ks_frag(lane, wn * 2 + j);
    }
    // [subtile][K half]; B: half 0 of even and odd steps (HM = 1: of the step), half 1
    u32x4 fa[4][2], fb[3][2][2];
    auto read_a = [&](auto off_c, uint32_t base) {
        constexpr int OFF = decltype(off_c)::value;
        static_for<0, 4>([&](auto ic) {
            constexpr int i = decltype(ic)::value;
            if constexpr (LA == OP_KC) {
                fa[i][0] = lds16<OFF + i * 2048>(base + ra[0]);
                fa[i][1] = lds16<OFF + i * 2048>(base + ra[1]);
            } else {
                static_for<0, 2>([&](auto sc) {
                    constexpr int s = decltype(sc)::value;
                    const v2u lo = lds_tr16<OFF + s * 8192>(base + ra[i]), hi = lds_tr16<OFF + s * 8192 + 1024>(base + ra[i]);
                    fa[i][s] = u32x4{lo.x, lo.y, hi.x, hi.y};
                });
            }
        });
    };
    auto read_b = [&](auto off_c, auto hc, uint32_t base) {
        constexpr int OFF = decltype(off_c)::value, h = decltype(hc)::value;  // h: index in fb
        static_for<0, 2>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            if constexpr (LB == OP_KC) {
                fb[h][j][0] = lds16<OFF + j * 2048>(base + rb[0]);
                fb[h][j][1] = lds16<OFF + j * 2048>(base + rb[1]);
            } else {
                static_for<0, 2>([&](auto sc) {
                    constexpr int s = decltype(sc)::value;
                    const v2u lo = lds_tr16<OFF + s * 8192>(base + rb[j]), hi = lds_tr16<OFF + s * 8192 + 1024>(base + rb[j]);
                    fb[h][j][s] = u32x4{lo.x, lo.y, hi.x, hi.y};
                });
            }
        });
    };

    v4f acc[HM][2][4][2];
    auto multiply = [&](auto ac, auto st_c) {
        constexpr int a = decltype(ac)::value, st = decltype(st_c)::value;
        wait_lgkm0();
        phase_barrier();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[a][b][i][j] = mfma_bf16(fb[b ? 2 : st][j][s], fa[i][s], acc[a][b][i][j]);
        __builtin_amdgcn_s_setprio(0);
        phase_barrier();
    };
    constexpr std::integral_constant<int, 0> c0;
    constexpr std::integral_constant<int, 1> c1;
    constexpr std::integral_constant<int, 2> c2;
    constexpr std::integral_constant<int, HALF> half1;
    // `wait`: not in a tile's first step, whose operands have landed before it begins
    [[maybe_unused]] auto kstep = [&](auto st_c, int ks, bool wait) {
        constexpr int st = decltype(st_c)::value;
        constexpr std::integral_constant<int, st ^ 1> other;
        uint32_t base = sbase + st * STAGE, next = sbase + (st ^ 1) * STAGE;
        pin(base);
        read_a(c0, base);
        read_b(half1, c2, base);
        issue_b(st, 0, ks + 2);
        issue_a(st ^ 1, HM - 1, ks + 1);
        if (wait) wait_vmcnt<8>();  // A1 of this step, B0 of the next
        multiply(c0, st_c);
        pin(base);
        pin(next);
        read_a(half1, base);
        read_b(c0, other, next);
        issue_a(st, 0, ks + 2);
        issue_b(st, 1, ks + 2);
        if (wait) wait_vmcnt<8>();  // A0, B1 of the next step
        multiply(std::integral_constant<int, HM - 1>{}, st_c);
    };
    // HM = 1: step ks from stage st, refilling the stage of the step before
    auto kstep1 = [&](int st, int ks, bool wait) {
        uint32_t base = sbase + st * STAGE;
        pin(base);
        read_a(c0, base);
        read_b(c0, c0, base);
        read_b(half1, c2, base);
        const int refill = st == 0 ? 2 : st - 1;
        issue_a(refill, 0, ks + 2);
        issue_b(refill, 0, ks + 2);
        issue_b(refill, 1, ks + 2);
        if (wait) wait_vmcnt<6>();  // the next step
        multiply(c0, c0);
    };

    // ---- results straight from the accumulators.  Every store comes after
    // wait_vmcnt<0>: the next tile's first steps, issued before, have then landed, and
    // no wait of its first step has to wait for the stores.
    auto leave = [&](int64_t m0, int n0, int split) {
        const int coff = ((g4 & 1) << 4) | ((g4 & 2) << 2);  // a lane's 8 columns after swap_cols
        auto row = [&](int u) { return m0 + (u >> 2) * 128 + wm * 64 + (u & 3) * 16 + l15; };  // u: 4 a + i
        if constexpr (EPI == EPI_PART) {
            wait_vmcnt<0>();
            static_for<0, HM * 4>([&](auto uc) {
                constexpr int u = decltype(uc)::value;
                const int64_t m = row(u);
                float* p = g.part + ((int64_t)split * g.M + m) * g.part_ld;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int n = n0 + wn * WSTEP + b * HSTEP + j * 16 + g4 * 4;
                        if (m < g.M && n < g.part_ld) *reinterpret_cast<v4f*>(p + n) = acc[u >> 2][b][u & 3][j];
                    }
            });
        } else if constexpr (EPI == EPI_PLAIN) {
            u32x4 r[HM * 4][2];
            const int n = n0 + wn * WSTEP + coff;
            const bool on[2] = {n < g.N, n + HSTEP < g.N};
            // (loaded here: between the stores each load would wait for those before it;
            // gradients have none)
            constexpr bool BIAS = LA == OP_KC && LB == OP_KC;
            u32x4 bias[2] = {};
            if (BIAS && g.bias) {
#pragma unroll
                for (int b = 0; b < 2; ++b) bias[b] = *reinterpret_cast<const u32x4*>(g.bias + (on[b] ? n + b * HSTEP : 0));
            }
            if (g.res) {
                static_for<0, HM * 4>([&](auto uc) {
                    constexpr int u = decltype(uc)::value;
                    const int64_t m = min(row(u), (int64_t)g.M - 1);
                    const uint16_t* p = g.res + m * g.ldr;
#pragma unroll
                    for (int b = 0; b < 2; ++b) r[u][b] = *reinterpret_cast<const u32x4*>(p + (on[b] ? n + b * HSTEP : 0));
                });
            }
            wait_vmcnt<0>();
            static_for<0, HM * 4>([&](auto uc) {
                constexpr int u = decltype(uc)::value;
                const int64_t m = row(u);
                uint16_t* p = (uint16_t*)g.out + m * g.ldo;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    v4f v0 = acc[u >> 2][b][u & 3][0], v1 = acc[u >> 2][b][u & 3][1];
                    swap_cols(v0, v1);
                    if (BIAS && g.bias) {
                        v4f t0, t1;
                        unpack_bf16x8(bias[b], t0, t1);
                        v0 += t0;
                        v1 += t1;
                    }
                    if (g.res) {
                        v4f t0, t1;
                        unpack_bf16x8(r[u][b], t0, t1);
                        v0 += t0;
                        v1 += t1;
                    }
                    if (m < g.M && on[b]) {
                        u32x4* q = reinterpret_cast<u32x4*>(p + n + b * HSTEP);
                        const u32x4 w = pack_bf16x8(v0, v1);
                        if (g.past) {  // (the asm keeps the compiler from making one plain store of the two)
                            asm volatile("");
                            __builtin_nontemporal_store(w, q);
                            asm volatile("");
                        } else {
                            *q = w;
                        }
                    }
                }
            });
        } else if constexpr (EPI == EPI_GATE) {
            const int nj = n0 + wn * 32 + g4 * 4, n = n0 + wn * 32 + coff;
            if (g.bias) {
                EpiBias<EPI_GATE> bias[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) bias[j].load(g, nj + j * 16);
                static_for<0, HM * 4>([&](auto uc) {
                    constexpr int u = decltype(uc)::value;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        acc[u >> 2][0][u & 3][j] += bias[j].a;
                        acc[u >> 2][1][u & 3][j] += bias[j].b;
                    }
                });
            }
            if (g.save == MOE_SAVE_INT8) {
                static_for<0, HM * 4>([&](auto uc) {
                    constexpr int u = decltype(uc)::value;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        uint32_t mx = 0;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int q = 0; q < 4; ++q) mx = umax(mx, abs_bits(acc[u >> 2][w][u & 3][j][q]));
                        mx = umax(mx, (uint32_t)__shfl_xor((int)mx, 16));
                        mx = umax(mx, (uint32_t)__shfl_xor((int)mx, 32));
                        if (lane < 16) rowmax[wn][w][(u >> 2) * 128 + wm * 64 + (u & 3) * 16 + l15] = mx;
                    }
                });
                wait_lgkm0();
                phase_barrier();
            }
            wait_vmcnt<0>();
            const bool on = n < g.f;
            static_for<0, HM * 4>([&](auto uc) {
                constexpr int u = decltype(uc)::value;
                const int64_t m = row(u);
                const bool mine = on && m < g.M;
                const v4f G[2] = {acc[u >> 2][0][u & 3][0], acc[u >> 2][0][u & 3][1]};
                const v4f U[2] = {acc[u >> 2][1][u & 3][0], acc[u >> 2][1][u & 3][1]};
                if (g.save == MOE_SAVE_INT8) {
                    const int r = (u >> 2) * 128 + wm * 64 + (u & 3) * 16 + l15;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        uint32_t mx = rowmax[0][w][r];
#pragma unroll
                        for (int v = 1; v < 4; ++v) mx = umax(mx, rowmax[v][w][r]);
                        const Keep8 k = keep8_scale(mx);
                        if (wn == 0 && lane < 16 && m < g.M)
                            g.gu_s[((int64_t)(w * (g.f >> 7)) + (n0 >> 7)) * g.M + m] = k.s;
                        uint32_t q[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const v4f v = w ? U[j] : G[j];
                            q[j] = pack_s8x4(keep8_code(v.x, k.inv), keep8_code(v.y, k.inv), keep8_code(v.z, k.inv),
                                             keep8_code(v.w, k.inv));
                        }
                        swap16(q[0], q[1]);
                        if (mine)
                            *reinterpret_cast<v2u*>((int8_t*)g.gu + m * (2 * (int64_t)g.f) + (int64_t)w * g.f + n) =
                                v2u{q[0], q[1]};
                    }
                }
                auto put = [&](uint16_t* p, const v4f& a, const v4f& b) {
                    v2u x = pack_bf16x4(a.x, a.y, a.z, a.w), y = pack_bf16x4(b.x, b.y, b.z, b.w);
                    uint32_t x0 = x.x, x1 = x.y, y0 = y.x, y1 = y.y;
                    swap16(x0, y0);
                    swap16(x1, y1);
                    if (mine) *reinterpret_cast<u32x4*>(p) = u32x4{x0, x1, y0, y1};
                };
                if (g.save == MOE_SAVE_BF16) {
                    uint16_t* p = (uint16_t*)g.gu + m * (2 * (int64_t)g.f) + n;
                    put(p, G[0], G[1]);
                    put(p + g.f, U[0], U[1]);
                }
                v4f h[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float z[4] = {G[j].x, G[j].y, G[j].z, G[j].w};
                    float v[4];
                    act_value4(ACT, z, v);
                    h[j] = v4f{v[0], v[1], v[2], v[3]} * U[j];
                }
                put(g.h + m * (int64_t)g.f + n, h[0], h[1]);
            });
        } else {  // EPI_DGATE, EPI_DGATE8: four 16-row subtiles' loads in flight
            const int n = n0 + wn * WSTEP + coff;
            const bool on[2] = {n < g.f, n + HSTEP < g.f};
            constexpr bool I8 = EPI == EPI_DGATE8;
            u32x4 q[4][2][I8 ? 1 : 2];
            float sc[I8 ? 4 : 1][2][2];
            auto load = [&](auto uc) {
                constexpr int u = decltype(uc)::value, at = u & 3;
                const int64_t m = min(row(u), (int64_t)g.M - 1);
                const int64_t o = m * (2 * (int64_t)g.f);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int c = on[b] ? n + b * HSTEP : 0;
                    if constexpr (I8) {
                        const v2u x = *reinterpret_cast<const v2u*>((const int8_t*)g.gu + o + c);
                        const v2u y = *reinterpret_cast<const v2u*>((const int8_t*)g.gu + o + g.f + c);
                        q[at][b][0] = u32x4{x.x, x.y, y.x, y.y};
                        sc[at][b][0] = g.gu_s[(int64_t)(c >> 7) * g.M + m];
                        sc[at][b][1] = g.gu_s[(int64_t)((g.f >> 7) + (c >> 7)) * g.M + m];
                    } else {
                        q[at][b][0] = *reinterpret_cast<const u32x4*>((const uint16_t*)g.gu + o + c);
                        q[at][b][1] = *reinterpret_cast<const u32x4*>((const uint16_t*)g.gu + o + g.f + c);
                    }
                }
            };
            static_for<0, 4>([&](auto uc) { load(uc); });
            wait_vmcnt<0>();
            static_for<0, HM * 4>([&](auto uc) {
                constexpr int u = decltype(uc)::value, at = u & 3;
                const int64_t m = row(u);
                uint16_t* p = g.dgu + m * (2 * (int64_t)g.f) + n;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    v4f dh[2] = {acc[u >> 2][b][u & 3][0], acc[u >> 2][b][u & 3][1]};
                    swap_cols(dh[0], dh[1]);
                    v4f G[2], U[2], dG[2], dU[2], h[2];
                    if constexpr (I8) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                G[j][e] = s8_of(q[at][b][0][j], e) * sc[at][b][0];
                                U[j][e] = s8_of(q[at][b][0][2 + j], e) * sc[at][b][1];
                            }
                    } else {
                        unpack_bf16x8(q[at][b][0], G[0], G[1]);
                        unpack_bf16x8(q[at][b][1], U[0], U[1]);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float z[4] = {G[j].x, G[j].y, G[j].z, G[j].w};
                        float v[4], sl[4];
                        act_both4(ACT, z, v, sl);
                        const v4f vv = {v[0], v[1], v[2], v[3]}, ss = {sl[0], sl[1], sl[2], sl[3]};
                        dG[j] = dh[j] * U[j] * ss;
                        dU[j] = dh[j] * vv;
                        h[j] = vv * U[j];
                    }
                    if (m < g.M && on[b]) {
                        *reinterpret_cast<u32x4*>(p + b * HSTEP) = pack_bf16x8(dG[0], dG[1]);
                        *reinterpret_cast<u32x4*>(p + g.f + b * HSTEP) = pack_bf16x8(dU[0], dU[1]);
                        if (g.h)
                            *reinterpret_cast<u32x4*>(g.h + m * (int64_t)g.f + n + b * HSTEP) = pack_bf16x8(h[0], h[1]);
                    }
                }
                if constexpr (u + 4 < HM * 4) load(std::integral_constant<int, u + 4>{});
            });
        }
    };
    // ---- or through LDS, a 128-row half at a time
    auto leave_staged = [&](int64_t m0, int n0, int split) {
#pragma unroll
        for (int a = 0; a < HM; ++a) {
            TileEpilogue<EPI, 128, 256, 512> epi;
            epi.load(g, m0 + a * 128, n0);
            if (a) __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int c = (wn * WSTEP + b * HSTEP + j * 16) / 4;
                        *reinterpret_cast<v4f*>(smem + stage_at(256, wm * 64 + i * 16 + l15, c + g4)) = acc[a][b][i][j];
                    }
            __syncthreads();
            epi.run(g, smem, m0 + a * 128, n0, split);
        }
        __syncthreads();
    };

    bool have = false;  // acc holds a tile's results
    int64_t pm0 = 0;
    int pn0 = 0, psplit = 0;
    for (int t = blockIdx.x;; t += gridDim.x) {
        const bool more = t < tiles;
        if constexpr (!DIRECT) {
            if (have) leave_staged(pm0, pn0, psplit);
        }
        if (more) {
            setup(t);
            issue_b(0, 0, ks0);
            issue_a(0, 0, ks0);
            issue_b(0, 1, ks0);
            issue_b(1, 0, ks0 + 1);
            if constexpr (HM == 2) issue_a(0, 1, ks0);
            issue_a(1, 0, ks0 + 1);
            issue_b(1, 1, ks0 + 1);
        }
        if constexpr (DIRECT) {
            if (have) leave(pm0, pn0, psplit);
        }
        if (!more) break;
        if (!DIRECT || !have) wait_vmcnt<0>();
        phase_barrier();
        if constexpr (HM == 2) {
            uint32_t base = sbase;
            pin(base);
            read_b(c0, c0, base);
            wait_lgkm0();
            phase_barrier();
        }
#pragma unroll
        for (int a = 0; a < HM; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[a][b][i][j] = v4f{0.f, 0.f, 0.f, 0.f};
        if (wm == 1) phase_barrier();  // the second wave of each SIMD runs half a phase behind
        if constexpr (HM == 2) {
            for (int ks = ks0; ks < ks1; ks += 2) {
                kstep(c0, ks, ks > ks0);
                if (ks + 1 < ks1) kstep(c1, ks + 1, true);
            }
        } else {
            int st = 0;
            for (int ks = ks0; ks < ks1; ++ks) {
                kstep1(st, ks, ks > ks0);
                st = st == 2 ? 0 : st + 1;
            }
        }
        if (wm == 0) phase_barrier();
        // every wave has read the last step, and this wave's fills past the end (into
        // places only it refills) have landed: LDS may be refilled, or reused
        wait_vmcnt<0>();
        if constexpr (!DIRECT) phase_barrier();
        have = true;
        pm0 = m0;
        pn0 = n0;
        psplit = split;
    }
    wait_vmcnt<0>();
}

// ---------------------------------------------------------------- split K: sum and epilogue
// One thread per four columns; the pieces are added in order.  Bound by reading them
// (from the LLC, just written): two of 16384 x 256 into fp32 take 12 us, 4.2 TB/s.
template <int EPI>
__global__ __launch_bounds__(128) void dense_sum_kernel(DenseArgs g, int splits) {
    const int cols = EPI == EPI_GATE ? g.f : (int)g.part_ld;
    const int64_t idx = (int64_t)blockIdx.x * 128 + threadIdx.x;
    const int64_t m = idx / (cols / 4);
    const int n = (int)(idx - m * (cols / 4)) * 4;
    const bool on = m < g.M;
    const int64_t plane = (int64_t)g.M * g.part_ld;
    auto sum = [&](int col) {
        v4f s = {0.f, 0.f, 0.f, 0.f};
        if (on) {
            const float* p = g.part + m * g.part_ld + col;
            // eight loads in flight; past the last piece it is read again, not added
            for (int i = 0; i < splits; i += 8) {
                v4f t[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) t[j] = *reinterpret_cast<const v4f*>(p + min(i + j, splits - 1) * plane);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i + j < splits) s += t[j];
            }
        }
        return s;
    };
    EpiBias<EPI> bias;
    bias.load(g, n);
    if constexpr (EPI == EPI_GATE) {
        const v4f G = sum(n), U = sum(g.f + n);
        epi_gate(g, m, n, G, U, bias, on);
    } else {
        if (!on) return;
        EpiIn<EPI> in;
        in.load(g, m, n);
        const v4f s = sum(n);
        if constexpr (is_dgate(EPI))
            epi_dgate(g, m, n, s, in);
        else if constexpr (EPI == EPI_PLAIN)
            epi_plain(g, m, n, s, in, bias);
        else
            epi_linear(g, m, n, s, in, bias);
    }
}

// ---------------------------------------------------------------- host side
namespace {
enum Kind {
    THIN = MOE_DENSE_THIN,
    SLAB = MOE_DENSE_SLAB,
    SMALL = MOE_DENSE_SMALL,
    TILES = MOE_DENSE_TILES,
    HALF = MOE_DENSE_HALF,
    WIDE = MOE_DENSE_WIDE
};
struct Shape {
    Kind kind;
    int64_t mt, nt;
    int splits, ksteps;
    bool pieces;  // results go through the workspace and dense_sum_kernel
    double us;    // estimated
};
// K in at most `sp` pieces of at least `least` steps
void set_splits(Shape& s, int64_t K, int64_t sp, int64_t least) {
    const int64_t steps = (K + DBK - 1) / DBK;
    if (sp > steps / least) sp = steps / least;
    if (sp > 32) sp = 32;
    if (sp < 1) sp = 1;
    s.ksteps = (int)((steps + sp - 1) / sp);
    s.splits = (int)((steps + s.ksteps - 1) / s.ksteps);
}
// The kernel for an M x N product over K.  THIN (up to 4 rows) and SLAB (up to 128
// rows, K in pieces) go by the rows.  Of the tiled ones, each with K whole or in as
// many pieces as fill the compute units, the one with the least estimated time is
// taken:
//     rounds of tiles x K steps x time of a step + fixed
//         + the pieces' second launch (4 us) and traffic (8 bytes per result, 10 TB/s)
// with the steps' times measured on operands of 16 to 120 MB:
//   WIDE   256 x 256 tiles   1.45 us a step   2048 x 7168 over 4096: 96 us (HALF 123)
//   HALF   128 x 256         0.87             1024 x 7168 over 2048: 32 us (TILES 40)
//   TILES  128 x 128         1.05 (two of them on a compute unit; 0.75 alone)
//                                             12000 x 600 over 1200: 29 us (HALF 39)
//   SMALL  64 x 64           0.38 (two; 0.22 alone)
//                                             256 x 4096 over 7168: 29 us (TILES 31)
// The estimates are within 15% of the times over 50 shapes, and the choice within
// 10% of the best kernel's.
struct Tiling {
    Kind kind;
    int bm, bn, per_cu;      // tile, workgroups that share a compute unit
    double alone, shared, fixed;  // us per step (one, per_cu of them on a unit), us
    int least;               // K steps of a piece at least
};
constexpr Tiling TILINGS[] = {{WIDE, 256, 256, 1, 1.45, 1.45, 10., 8},
                              {HALF, 128, 256, 1, 0.87, 0.87, 7., 8},
                              {TILES, 128, 128, 2, 0.75, 1.05, 6., 8},
                              {SMALL, 64, 64, 2, 0.22, 0.38, 5., 8}};
Shape dense_shape(int64_t M, int64_t N, int64_t K, int la, int lb, int epi) {
    Shape s;
    const bool gate = epi == EPI_GATE || epi == EPI_GATE8;
    const int64_t cus = num_cus();
    s.splits = 1;
    s.ksteps = (int)((K + DBK - 1) / DBK);
    s.mt = 1;
    s.pieces = false;
    s.us = 0.;
    if (la == OP_KC && lb == OP_KC && M <= SLAB_ROWS) {
        s.kind = M <= THIN_ROWS && epi != EPI_GATE8 ? THIN : SLAB;
        s.nt = (N + 127) / 128;
        if (s.kind == SLAB) set_splits(s, K, cus / s.nt, 4);
        s.pieces = s.kind == SLAB;
        return s;
    }
    Shape best = s;
    double least = 1e30;
    for (const Tiling& t : TILINGS) {
        for (int64_t share = 0; share <= t.per_cu; ++share) {  // 0: K whole
            Shape c = s;
            c.kind = t.kind;
            // gated tiles hold half as many h columns (on TILES: 64 x 256 tiles of B rows)
            const bool paired = gate && share == 0;
            int64_t bm = t.bm, bn = paired ? t.bn / 2 : t.bn;
            if (paired && t.kind == TILES) bm = 64, bn = 128;
            c.mt = (M + bm - 1) / bm;
            c.nt = ((paired ? N / 2 : N) + bn - 1) / bn;
            const int64_t tiles = c.mt * c.nt;
            if (share) {
                set_splits(c, K, share * cus / tiles, t.least);
                if (c.splits < 2) continue;
                c.pieces = true;
            }
            // the 8-bit save takes whole 128-column blocks: in the sum of the pieces
            if (epi == EPI_GATE8 && t.kind == SMALL && !share) {
                c.nt = (N + 63) / 64;
                c.pieces = true;
            }
            const int64_t n = tiles * c.splits;
            // a launch takes less than 2^32 threads; HALF and WIDE are persistent
            if (t.per_cu > 1 && n >= (1 << 23)) continue;
            const double rounds = (double)((n + t.per_cu * cus - 1) / (t.per_cu * cus));
            double us = rounds * c.ksteps * (n <= cus ? t.alone : t.shared) + t.fixed;
            if (c.pieces) us += 4. + (double)c.splits * M * N * 8 / 1e7;
            if (us < least) {
                least = us;
                best = c;
                best.us = us;
            }
        }
    }
    return best;
}
template <int WM, int WN, int LA, int LB, int EPI>
int launch_one(const DenseArgs& g, int splits, hipStream_t stream) {
    const int64_t grid = (int64_t)g.mt * g.nt * splits;
    dense_kernel<WM, WN, LA, LB, EPI><<<dim3((unsigned)grid), dim3(WM * WN * 64), 0, stream>>>(g);
    MOE_LAUNCH_CHECK("dense_kernel");
    return MOE_OK;
}
template <int LA, int LB, int EPI>
int launch_small_one(const DenseArgs& g, int splits, hipStream_t stream) {
    dense_small_kernel<LA, LB, EPI><<<dim3((unsigned)(g.mt * g.nt * splits)), dim3(256), 0, stream>>>(g);
    MOE_LAUNCH_CHECK("dense_small_kernel");
    return MOE_OK;
}
template <int EPI>
int launch_small(const DenseArgs& g, int la, int lb, int splits, hipStream_t stream) {
    if (la == OP_KC && lb == OP_KC) return launch_small_one<OP_KC, OP_KC, EPI>(g, splits, stream);
    if (la == OP_KC) return launch_small_one<OP_KC, OP_KS, EPI>(g, splits, stream);
    return launch_small_one<OP_KS, OP_KS, EPI>(g, splits, stream);
}
template <int LA, int LB, int EPI, int ACT = -1, int HM = 2>
int launch_wide(const DenseArgs& g, int splits, hipStream_t stream) {
    const int tiles = g.mt * g.nt * splits, cus = num_cus() & ~7;
    const int grid = tiles < cus ? tiles : cus;
    dense_wide_kernel<HM, LA, LB, EPI, ACT><<<dim3((unsigned)grid), dim3(512), 0, stream>>>(g, tiles);
    MOE_LAUNCH_CHECK("dense_wide_kernel");
    return MOE_OK;
}
template <int EPI, int HM = 2>
int launch_wide_any(const DenseArgs& g, int la, int lb, int splits, hipStream_t stream) {
    if (la == OP_KC && lb == OP_KC) return launch_wide<OP_KC, OP_KC, EPI, -1, HM>(g, splits, stream);
    if (la == OP_KC) return launch_wide<OP_KC, OP_KS, EPI, -1, HM>(g, splits, stream);
    return launch_wide<OP_KS, OP_KS, EPI, -1, HM>(g, splits, stream);
}
// the gated epilogues: silu, the usual activation, is compiled in
template <int LB, int EPI, int HM = 2>
int launch_wide_act(const DenseArgs& g, hipStream_t stream) {
    if (g.act == MOE_ACT_SILU) return launch_wide<OP_KC, LB, EPI, MOE_ACT_SILU, HM>(g, 1, stream);
    return launch_wide<OP_KC, LB, EPI, -1, HM>(g, 1, stream);
}
template <int EPI>
int launch_sum(const DenseArgs& g, int splits, hipStream_t stream) {
    const int64_t cols = EPI == EPI_GATE ? g.f : g.part_ld;
    const int64_t blocks = ((int64_t)g.M * (cols / 4) + 127) / 128;
    dense_sum_kernel<EPI><<<dim3((unsigned)blocks), dim3(128), 0, stream>>>(g, splits);
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

size_t dense_ws(int64_t M, int64_t N, int64_t K, int la, int lb, int epi) {
    if (M <= 0 || N <= 0 || K <= 0) return 0;  // T = 0
    const Shape s = dense_shape(M, N, K, la, lb, epi);
    return s.pieces ? (size_t)s.splits * M * round_up(N, 4) * 4 : 0;
}

int dense_launch(DenseArgs g, int la, int lb, int epi, void* ws, size_t ws_bytes, hipStream_t stream) {
    if (epi == EPI_GATE && g.save == MOE_SAVE_INT8) epi = EPI_GATE8;
    const Shape s = dense_shape(g.M, g.N, g.K, la, lb, epi);
    if (epi == EPI_GATE8) epi = EPI_GATE;
    if (epi == EPI_DGATE && g.save == MOE_SAVE_INT8) epi = EPI_DGATE8;
    if (epi == EPI_LINEAR && g.vec && !g.out_f32 && !g.pre && g.act == MOE_ACT_NONE && g.N % 8 == 0 && g.ldo % 8 == 0 &&
        (!g.res || g.ldr % 8 == 0))
        epi = EPI_PLAIN;
    MOE_REQUIRE(s.mt * s.nt * s.splits < (1ll << 31), MOE_ERR_SHAPE, "product of %d x %d has too many tiles", g.M, g.N);
    g.mt = (int)s.mt;
    g.nt = (int)s.nt;
    g.ksteps = s.ksteps;
    if (s.kind == THIN) return dense_thin_launch(g, epi, stream);
    if (s.pieces) {
        MOE_REQUIRE(ws && aligned16(ws) && ws_bytes >= (size_t)s.splits * g.M * round_up(g.N, 4) * 4, MOE_ERR_WORKSPACE,
                    "workspace too small");
        g.part = (float*)ws;
        g.part_ld = round_up(g.N, 4);
        const int rc = s.kind == SLAB    ? dense_slab_launch(g, s.splits, stream)
                       : s.kind == SMALL ? launch_small<EPI_PART>(g, la, lb, s.splits, stream)
                       : s.kind == HALF  ? launch_wide_any<EPI_PART, 1>(g, la, lb, s.splits, stream)
                       : s.kind == WIDE  ? launch_wide_any<EPI_PART>(g, la, lb, s.splits, stream)
                                         : launch_layout<EPI_PART>(g, la, lb, s.splits, stream);
        if (rc != MOE_OK) return rc;
        if (epi == EPI_GATE) return launch_sum<EPI_GATE>(g, s.splits, stream);
        if (epi == EPI_DGATE) return launch_sum<EPI_DGATE>(g, s.splits, stream);
        if (epi == EPI_DGATE8) return launch_sum<EPI_DGATE8>(g, s.splits, stream);
        if (epi == EPI_PLAIN) return launch_sum<EPI_PLAIN>(g, s.splits, stream);
        return launch_sum<EPI_LINEAR>(g, s.splits, stream);
    }
    if (s.kind == SMALL) {
        if (epi == EPI_GATE) return launch_small_one<OP_KC, OP_KC, EPI_GATE>(g, 1, stream);
        if (epi == EPI_DGATE) return launch_small_one<OP_KC, OP_KS, EPI_DGATE>(g, 1, stream);
        if (epi == EPI_DGATE8) return launch_small_one<OP_KC, OP_KS, EPI_DGATE8>(g, 1, stream);
        if (epi == EPI_LINEAR) return launch_small_one<OP_KC, OP_KC, EPI_LINEAR>(g, 1, stream);
        return launch_small<EPI_PLAIN>(g, la, lb, 1, stream);
    }
    if (s.kind == HALF) {
        if (epi == EPI_GATE) return launch_wide_act<OP_KC, EPI_GATE, 1>(g, stream);
        if (epi == EPI_DGATE) return launch_wide_act<OP_KS, EPI_DGATE, 1>(g, stream);
        if (epi == EPI_DGATE8) return launch_wide_act<OP_KS, EPI_DGATE8, 1>(g, stream);
        if (epi == EPI_LINEAR) return launch_wide<OP_KC, OP_KC, EPI_LINEAR, -1, 1>(g, 1, stream);
        return launch_wide_any<EPI_PLAIN, 1>(g, la, lb, 1, stream);
    }
    if (s.kind == WIDE) {
        if (epi == EPI_GATE) return launch_wide_act<OP_KC, EPI_GATE>(g, stream);
        if (epi == EPI_DGATE) return launch_wide_act<OP_KS, EPI_DGATE>(g, stream);
        if (epi == EPI_DGATE8) return launch_wide_act<OP_KS, EPI_DGATE8>(g, stream);
        if (epi == EPI_LINEAR) return launch_wide<OP_KC, OP_KC, EPI_LINEAR>(g, 1, stream);
        // (data and weight gradients are always EPI_PLAIN)
        return launch_wide_any<EPI_PLAIN>(g, la, lb, 1, stream);
    }
    if (epi == EPI_GATE) return launch_one<1, 4, OP_KC, OP_KC, EPI_GATE>(g, 1, stream);
    if (epi == EPI_DGATE) return launch_one<2, 2, OP_KC, OP_KS, EPI_DGATE>(g, 1, stream);
    if (epi == EPI_DGATE8) return launch_one<2, 2, OP_KC, OP_KS, EPI_DGATE8>(g, 1, stream);
    if (epi == EPI_LINEAR) return launch_one<2, 2, OP_KC, OP_KC, EPI_LINEAR>(g, 1, stream);
    return launch_layout<EPI_PLAIN>(g, la, lb, 1, stream);
}

// The group is taken where its estimated time is less than the single products' and
// the column sums' two launches (4 us each).  A group's time: its longest sum over K,
// or all steps dealt to two workgroups per compute unit and half a longest one, or
// its column sums' rounds of 256 rows (0.45 to 0.66 us each: dx and dbias of 64 -> 64 at
// 16384 rows 31 us grouped and 13 alone, at 65536 171 and 19; a weight gradient is longer).
// Measured on 66 shapes: gated 2048 -> 512 at 2048 rows 54 us (alone 68), 4096 -> 512 at
// 4096 rows 201 (170); linear 7168 -> 256 at 203 rows 11.0 (12.4), at 2048 43.5 (36.8);
// the rule's choice is within 10% of the better one on 64 of them.
bool dense_group_pays(const DenseArgs* dx, const DenseArgs* dw0, const DenseArgs* dw1, int64_t sum_rows) {
    const DenseArgs* p[3] = {dx, dw0, dw1};
    const Tiling& t = TILINGS[3];
    double alone = sum_rows ? 8. : 0., steps = 0., longest = 0.;
    int n = 0;
    int64_t tiles = 0;
    for (int i = 0; i < 3; ++i) {
        if (!p[i]) continue;
        const DenseArgs& g = *p[i];
        const int64_t c = ((g.M + 63ll) / 64) * ((g.N + 63ll) / 64), ks = (g.K + DBK - 1) / DBK;
        alone += dense_shape(g.M, g.N, g.K, i == 0 ? OP_KC : OP_KS, OP_KS, EPI_PLAIN).us;
        steps += (double)c * ks;
        if (longest < ks) longest = (double)ks;
        tiles += c;
        ++n;
    }
    if (n + (sum_rows ? 1 : 0) < 2 || n == 0 || tiles >= (1 << 22)) return false;
    const int64_t cus = num_cus();
    const double step = tiles <= cus ? t.alone : t.shared;
    double us = steps / (t.per_cu * cus) * t.shared + longest * step / 2;
    if (us < longest * step) us = longest * step;
    const double sum_us = (double)((sum_rows + 255) / 256) * 0.5;
    if (us < sum_us) us = sum_us;
    return us + t.fixed < alone;
}

int dense_group_launch(const DenseArgs* dx, const DenseArgs* dw0, const DenseArgs* dw1, const ColSum* sums, int nsums,
                       hipStream_t stream) {
    const DenseArgs* p[3] = {dx, dw0, dw1};
    DenseGroup g = {};
    DenseArgs* q[3] = {&g.dx, &g.dw[0], &g.dw[1]};
    int64_t blocks = 0;
    for (int i = 0; i < 3; ++i) {
        if (!p[i]) continue;
        *q[i] = *p[i];
        q[i]->mt = (p[i]->M + 63) / 64;
        q[i]->nt = (p[i]->N + 63) / 64;
        q[i]->ksteps = (p[i]->K + DBK - 1) / DBK;
        g.tiles[i] = q[i]->mt * q[i]->nt;
        blocks += g.tiles[i];
    }
    for (int i = 0; i < nsums; ++i) {
        g.sums[i] = sums[i];
        g.sums[i].blocks = (int)((sums[i].N + 31) / 32);
        blocks += g.sums[i].blocks;
    }
    dense_group_kernel<<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(g);
    MOE_LAUNCH_CHECK("dense_group_kernel");
    return MOE_OK;
}

// ---------------------------------------------------------------- column sums, zeros
// Column sums in two launches: fp32 sums of chunks of rows, then the chunks'
// sums in a fixed order.  Bound by the bytes read; what matters is loads in
// flight: a wave takes 256 columns and CS_ROWS / 4 rows of a chunk, all loaded
// before the first is added.  dz and chunks of 16384 x 256 from fp32 take
// 8.2 us (3.1 TB/s; too short to reach more), the chunks' sums 6 us.
namespace {
constexpr int CS_ROWS = 8;  // rows of a chunk that are loaded at a time
struct Chunks {
    int n;
    int64_t rows;
};
// at most 1024 chunks, each a multiple of CS_ROWS rows
Chunks colsum_chunks(int64_t T) {
    int64_t rows = round_up((T + 1023) / 1024, CS_ROWS);
    if (rows < CS_ROWS) rows = CS_ROWS;
    const int64_t n = (T + rows - 1) / rows;
    return Chunks{(int)(n < 1 ? 1 : n), rows};
}
}  // namespace

// dz = dy * act'(pre) of moe_linear_backward: bf16 rows of stride ldz (columns
// past N zero) if dz is given, and fp32 column sums over chunks of rows (before
// the rounding) if part is given.  One thread per four columns of a row.
// dz is rounded, from fp32 dy too, since the products' operands are bf16: the rest as a
// second bf16 term would double the products, for results that are rounded to bf16
// themselves (they are about 1.4 times as far off as by that rounding alone).
struct DzArgs {
    const void* dy;
    int dy_f32;
    int64_t ld;
    const uint16_t* pre;  // [T, N]
    int64_t N, ldz;
    uint16_t* dz;   // [T, ldz]
    float* part;    // [chunks, ldz]
    uint16_t* out;  // [N]
    int blocks;     // of 256 columns
};
template <bool ACT, bool F32, bool VEC>
__global__ __launch_bounds__(256) void dz_kernel(DzArgs d0, DzArgs d1, int act, int64_t T, int64_t rows) {
    __shared__ float sm[4][256];
    const bool second = (int)blockIdx.x >= d0.blocks;
    const DzArgs& d = second ? d1 : d0;
    const int bx = blockIdx.x - (second ? d0.blocks : 0);
    const void* dy = d.dy;
    const int64_t ld = d.ld, N = d.N, ldz = d.ldz;
    const uint16_t* pre = d.pre;
    uint16_t* dz = d.dz;
    float* part = d.part;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t n = (int64_t)bx * 256 + lane * 4;
    const int64_t t0 = (int64_t)blockIdx.y * rows, t1 = min(t0 + rows, T);
    const int left = (int)(N - n);
    constexpr int R = CS_ROWS / 4;
    v4f s = {0.f, 0.f, 0.f, 0.f};
    if (n < ldz) {
        for (int64_t t = t0 + w; t < t1; t += CS_ROWS) {
            v4f v[R], p[ACT ? R : 1];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int64_t r = min(t + 4 * i, t1 - 1);
                v[i] = load4<F32, VEC>(dy, r * ld + n, left);
                if (ACT) p[i] = load4<false, VEC>(pre, r * N + n, left);
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (t + 4 * i >= t1) break;
                if (ACT) {
                    const float z[4] = {p[i].x, p[i].y, p[i].z, p[i].w};
                    float val[4], sl[4];
                    act_both4(act, z, val, sl);
                    v[i] *= v4f{sl[0], sl[1], sl[2], sl[3]};
                }
                if (dz)
                    *reinterpret_cast<v2u*>(dz + (t + 4 * i) * ldz + n) = pack_bf16x4(v[i].x, v[i].y, v[i].z, v[i].w);
                s += v[i];
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) sm[w][lane * 4 + i] = s[i];
    __syncthreads();
    const int64_t c = (int64_t)bx * 256 + threadIdx.x;
    if (c < ldz)
        part[blockIdx.y * ldz + c] =
            (sm[0][threadIdx.x] + sm[1][threadIdx.x]) + (sm[2][threadIdx.x] + sm[3][threadIdx.x]);
}

// out[n] = bf16 of the chunks' sums: 16 columns per block, 16 threads to a column
__global__ __launch_bounds__(256) void colsum_finish_kernel(DzArgs d0, DzArgs d1, int chunks) {
    __shared__ float sm[16][17];
    const int first = (int)((d0.N + 15) / 16);
    const bool second = (int)blockIdx.x >= first;
    const float* part = second ? d1.part : d0.part;
    uint16_t* out = second ? d1.out : d0.out;
    const int64_t ld = second ? d1.ldz : d0.ldz, N = second ? d1.N : d0.N;
    const int c = threadIdx.x & 15, q = threadIdx.x >> 4;
    const int64_t n = (int64_t)(blockIdx.x - (second ? first : 0)) * 16 + c;
    float s = 0.f;
    if (n < N) {
#pragma unroll 8
        for (int i = q; i < chunks; i += 16) s += part[i * ld + n];
    }
    sm[q][c] = s;
    __syncthreads();
    if (q == 0 && n < N) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += sm[i][c];
        out[n] = (uint16_t)cvt_bf16x2(s, 0.f);
    }
}

__global__ __launch_bounds__(256) void zero16_kernel(uint16_t* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

int colsum_parts(int64_t T) { return colsum_chunks(T).n; }
size_t colsum_ws(int64_t T, int64_t N) { return (size_t)colsum_chunks(T).n * N * 4; }

namespace {
using yes = std::true_type;
using no = std::false_type;
int dz_both(DzArgs d0, DzArgs d1, int act, int64_t T, hipStream_t stream) {
    const Chunks c = colsum_chunks(T);
    d0.blocks = (int)((d0.ldz + 255) / 256);
    d1.blocks = (int)((d1.ldz + 255) / 256);
    const dim3 grid((unsigned)(d0.blocks + d1.blocks), c.n);
    const bool vec = d0.N % 4 == 0;  // (d1: bf16 of a multiple of 8 columns, beside such a d0 without act)
    auto go = [&](auto act_c, auto f32_c, auto vec_c) {
        dz_kernel<decltype(act_c)::value, decltype(f32_c)::value, decltype(vec_c)::value>
            <<<grid, dim3(256), 0, stream>>>(d0, d1, act, T, c.rows);
    };
    auto pick = [&](auto act_c, auto f32_c) { vec ? go(act_c, f32_c, yes{}) : go(act_c, f32_c, no{}); };
    auto pick_f32 = [&](auto act_c) { d0.dy_f32 ? pick(act_c, yes{}) : pick(act_c, no{}); };
    act != MOE_ACT_NONE ? pick_f32(yes{}) : pick_f32(no{});
    MOE_LAUNCH_CHECK("dz_kernel");
    if (!d0.out) return MOE_OK;
    const int64_t blocks = (d0.N + 15) / 16 + (d1.N + 15) / 16;
    colsum_finish_kernel<<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(d0, d1, c.n);
    MOE_LAUNCH_CHECK("colsum_finish_kernel");
    return MOE_OK;
}
}  // namespace

int dz_launch(const void* dy, int dy_f32, const uint16_t* pre, int act, int64_t T, int64_t N, int64_t ldz, uint16_t* dz,
              float* part, uint16_t* dbias, hipStream_t stream) {
    const DzArgs d = {dy, dy_f32, N, pre, N, ldz, dz, part, dbias, 0};
    return dz_both(d, DzArgs{}, act, T, stream);
}

int colsum_launch(const uint16_t* a, int64_t Na, uint16_t* out_a, const uint16_t* b, int64_t Nb, uint16_t* out_b,
                  int64_t T, float* part, hipStream_t stream) {
    DzArgs d[2] = {};
    int n = 0;
    if (out_a) d[n++] = DzArgs{a, 0, Na, nullptr, Na, Na, nullptr, part, out_a, 0};
    if (out_b) d[n++] = DzArgs{b, 0, Nb, nullptr, Nb, Nb, nullptr, part + (out_a ? colsum_ws(T, Na) / 4 : 0), out_b, 0};
    return n ? dz_both(d[0], d[1], MOE_ACT_NONE, T, stream) : MOE_OK;
}

int zero16_launch(uint16_t* p, int64_t n, hipStream_t stream) {
    const int64_t blocks = (n + 255) / 256;
    zero16_kernel<<<dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream>>>(p, n);
    MOE_LAUNCH_CHECK("zero16_kernel");
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_dense_kernel(int64_t M, int64_t N, int64_t K, int32_t product, int32_t* kernel, int32_t* pieces) {
    clear_error();
    MOE_REQUIRE(kernel && pieces, MOE_ERR_NULL, "kernel or pieces is NULL");
    MOE_REQUIRE(product >= MOE_PRODUCT_FORWARD && product <= MOE_PRODUCT_GRADIENT, MOE_ERR_UNSUPPORTED,
                "unknown product %d", product);
    MOE_REQUIRE(M >= 1 && M <= (1 << 30) && N >= 1 && N <= (1 << 20) && K >= 1 && K <= (1 << 30), MOE_ERR_SHAPE,
                "M=%lld, N=%lld, K=%lld: at least 1, at most 2^30, 2^20 and 2^30", (long long)M, (long long)N, (long long)K);
    constexpr int EPIS[] = {EPI_LINEAR, EPI_GATE, EPI_GATE8, EPI_LINEAR};
    const int side = product == MOE_PRODUCT_GRADIENT ? OP_KS : OP_KC;
    const Shape s = dense_shape(M, N, K, OP_KC, side, EPIS[product]);
    *kernel = s.kind;
    *pieces = s.pieces ? s.splits : 0;
    return MOE_OK;
}
