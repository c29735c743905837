// Products with few rows (decoded tokens): C[m, n] = sum_k x[m, k] W[n, k], M <= 128.
// Bound by the bytes of W, each read once.
#include "dense_gemm.hpp"

namespace moe {

template <int EPI>
__device__ __forceinline__ void finish(const DenseArgs& g, int m, int n, v4f v) {
    if (n >= g.N) return;
    EpiIn<EPI> in;
    EpiBias<EPI> bias;
    in.load(g, m, n);
    bias.load(g, n);
    if constexpr (EPI == EPI_PLAIN)
        epi_plain(g, m, n, v, in, bias);
    else
        epi_linear(g, m, n, v, in, bias);
}

// dense_thin_kernel (up to 4 rows): a workgroup owns R rows of W and its NW waves
// split K, so that W goes from memory straight into MFMA operands with U loads
// always in flight per wave, and no workspace or second launch is needed: the
// waves' fp32 sums are added in order through LDS and the epilogue runs on them.
// An MFMA takes 16 rows of W.  With R = 4 they are 4 rows x 4 chunks of K, and
// likewise the 16 rows of x: of the products only those of equal chunks count.  A W
// of few rows is then spread over 4 times as many compute units (one alone streams
// about 20 GB/s): 256 rows of 7168 take 4.2 us, 10.7 us with R = 16.  Where R = 16
// fills the chip its fewer workgroups are ahead (7168 rows of 2048: 7.7 us, 3.8 TB/s,
// against 15.7 us; 4096 rows of 7168: 11.8 us, 5.0 TB/s).
template <int R, int NW, int EPI>
__global__ __launch_bounds__(NW * 64) void dense_thin_kernel(DenseArgs g) {
    static_assert(R == 4 || R == 16, "rows of W per workgroup");
    constexpr int U = R == 4 ? 4 : 8, C = 16 / R, STEP = 32 * C;  // K chunks and K values per step
    constexpr bool GATE = EPI == EPI_GATE;
    __shared__ v4f red[NW][R == 4 ? 4 : 64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l15 = lane & 15, r = l15 / C, chunk = l15 % C;  // W row (and x row) r, chunk
    const int gk = chunk * 32 + (lane >> 4) * 8;
    constexpr int COLS = GATE ? R / 2 : R;  // columns of the result per workgroup
    const int n0 = blockIdx.x * COLS;

    // rows past the matrix read its last row: their results are not stored
    const uint16_t* px = g.a + (int64_t)min(r, g.M - 1) * g.lda;
    int64_t row;
    if constexpr (GATE)  // G rows, then the U rows of the same h columns
        row = min(n0 + r % COLS, g.f - 1) + (r >= COLS ? g.f : 0);
    else
        row = min(n0 + r, g.N - 1);
    const uint16_t* pw = g.b + row * g.ldb;
    const int steps = (g.K + STEP - 1) / STEP, per = (steps + NW - 1) / NW;
    const int s0 = wave * per, n = min(per, steps - s0);  // n may be <= 0
    const bool tail = g.K % STEP != 0;

    v4f acc = {0.f, 0.f, 0.f, 0.f};
    u32x4 fx[U], fw[U];
    auto load = [&](int u, int s) {
        int k = (s0 + s) * STEP + gk;
        if (k >= g.K) k = 0;  // multiplied as zero below
        fw[u] = *reinterpret_cast<const u32x4*>(pw + k);
        fx[u] = *reinterpret_cast<const u32x4*>(px + k);
    };
    auto mul = [&](int u, int s) {
        if (tail && (s0 + s) * STEP + gk >= g.K) fw[u] = fx[u] = u32x4{0u, 0u, 0u, 0u};
        acc = mfma_bf16(fw[u], fx[u], acc);
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
    if constexpr (R == 4) {
        // acc[c] = (W row lane / 16, chunk c) x (x row-chunk lane % 16): this lane's
        // useful value is that of its x chunk; four lanes hold a result's chunks
        float v = chunk == 0 ? acc.x : chunk == 1 ? acc.y : chunk == 2 ? acc.z : acc.w;
        v += __shfl_xor(v, 1);
        v += __shfl_xor(v, 2);
        if (chunk == 0) reinterpret_cast<float*>(&red[wave][r])[lane >> 4] = v;  // [x row][W row]
        __syncthreads();
        if (tid >= g.M) return;
        v4f s = red[0][tid];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += red[w][tid];
        if constexpr (GATE) {
            if (n0 < g.f) epi_gate2(g, tid, n0, v4f{s.x, s.y, 0.f, 0.f}, v4f{s.z, s.w, 0.f, 0.f});
        } else {
            finish<EPI>(g, tid, n0, s);
        }
    } else {
        // acc[i] = W row 4 (lane / 16) + i, x row lane % 16
        red[wave][lane] = acc;
        __syncthreads();
        if (tid >= (GATE ? 32 : 64) || l15 >= g.M) return;
        auto sum = [&](int l) {
            v4f s = red[0][l];
#pragma unroll
            for (int w = 1; w < NW; ++w) s += red[w][l];
            return s;
        };
        const int n4 = n0 + (lane >> 4) * 4;
        if constexpr (GATE) {
            const v4f G = sum(lane), U4 = sum(lane + 32);  // G rows 0-7, U rows 8-15
            EpiBias<EPI_GATE> bias;
            bias.load(g, n4);
            epi_gate(g, l15, n4, G, U4, bias, n4 < g.f);
        } else {
            finish<EPI>(g, l15, n4, sum(lane));
        }
    }
}

// dense_slab_kernel (up to 128 rows): a workgroup takes 128 rows of W (16 per wave)
// and a range of K, in slabs of at most 128 KB of x, which it moves into LDS at once;
// then every wave streams its W rows into MFMA operands without synchronisation.  The
// fp32 sums of the K ranges go to the workspace (EPI_PART) and dense_sum_kernel
// adds them in order.  Against the kernel above, x passes through the texture path
// once per 128 W rows instead of once per 16, whose re-reads cost more than the
// second launch from 5 rows on (48 rows of x, 4096 rows of 7168: 16.4 us and 34.8 us;
// 16 rows of x: 14.5 and 16.0 us).
template <int MT>
__global__ __launch_bounds__(512) void dense_slab_kernel(DenseArgs g) {
    constexpr int U = 4;  // K steps of 64 in flight per wave (two loads each)
    constexpr int STEP = MT * 2048, SLAB = 131072, SLAB_STEPS = SLAB / STEP;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[SLAB];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int split = blockIdx.x / g.nt, nt = blockIdx.x - split * g.nt;
    const int l15 = lane & 15, gk = (lane >> 4) * 8;
    const uint32_t sbase = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    const int end = min((split + 1) * g.ksteps, (g.K + DBK - 1) / DBK);

    // W: rows past the matrix read its last row (their results are not stored)
    const int n0 = nt * 128 + wave * 16;
    const uint16_t* pw = g.b + (int64_t)min(n0 + l15, g.N - 1) * g.ldb;
    const KcLane xl(lane, g.lda);
    v4f acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = v4f{0.f, 0.f, 0.f, 0.f};

    for (int ks0 = split * g.ksteps; ks0 < end; ks0 += SLAB_STEPS) {
        const int n = min(SLAB_STEPS, end - ks0);
        u32x4 fw[U][2];
        auto load = [&](int u, int s) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                int k = (ks0 + s) * DBK + i * 32 + gk;
                if (k >= g.K) k = 0;  // multiplied as zero below
                fw[u][i] = *reinterpret_cast<const u32x4*>(pw + k);
            }
        };
        // x: K step s, 16-row group q (two 1 KB segments) by wave (s MT + q) % 8
        for (int j = wave; j < n * MT; j += 8) {
            const int s = j / MT, q = j - s * MT;
            const int k0 = (ks0 + s) * DBK;
            const u32x4 d = buf_desc((const uint8_t*)(g.a + (int64_t)q * 16 * g.lda + k0));
            const bool kok = (int)xl.k < g.K - k0;
            const int r = q * 16 + xl.row;
            dma16b2(d, kok && r < g.M ? xl.off : OOB, kok && r + 8 < g.M ? xl.off + (uint32_t)(16 * g.lda) : OOB,
                    sbase + s * STEP + q * 2048);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) load(u, min(u, n - 1));
        // loads complete in order: the 2 U younger ones may stay in flight (none of them
        // may be scheduled behind the wait)
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<U * 2>();
        phase_barrier();
        uint32_t base = sbase;
        pin(base);
        const uint32_t ra = base + kc_frag(lane, 0);
        const int klast = g.K - (ks0 + n - 1) * DBK;  // K values of the slab's last step
        auto mul = [&](int u, int s) {
            if (s == n - 1 && klast < DBK) {
                const u32x4 z = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (i * 32 + gk >= klast) fw[u][i] = z;
            }
            const uint32_t r = ra + s * STEP;
            static_for<0, MT>([&](auto mc) {
                constexpr int m = decltype(mc)::value;
                acc[m] = mfma_bf16(fw[u][0], lds16<m * 2048>(r), acc[m]);
                acc[m] = mfma_bf16(fw[u][1], lds16<m * 2048>(r ^ 64), acc[m]);
            });
        };
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
        // (also tells the compiler that the next slab's registers are free: it would
        // wait for the x slab before the first W loads otherwise)
        wait_vmcnt<0>();
        if (ks0 + SLAB_STEPS < end) {  // every wave has read the slab: the next one may overwrite it
            wait_lgkm0();
            phase_barrier();
        }
    }
    const int col = n0 + (lane >> 4) * 4;
    if (col >= g.part_ld) return;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int row = m * 16 + l15;
        if (row < g.M) *reinterpret_cast<v4f*>(g.part + ((int64_t)split * g.M + row) * g.part_ld + col) = acc[m];
    }
}

namespace {
template <int EPI>
int launch_thin(const DenseArgs& g, hipStream_t stream) {
    constexpr int half = EPI == EPI_GATE ? 2 : 1;
    const int cols = EPI == EPI_GATE ? g.f : g.N;
    const unsigned wide = (unsigned)((cols + 16 / half - 1) / (16 / half)), narrow = (unsigned)((cols + 4 / half - 1) / (4 / half));
    if (wide >= 192)
        dense_thin_kernel<16, 8, EPI><<<dim3(wide), dim3(512), 0, stream>>>(g);
    else
        dense_thin_kernel<4, 16, EPI><<<dim3(narrow), dim3(1024), 0, stream>>>(g);
    MOE_LAUNCH_CHECK("dense_thin_kernel");
    return MOE_OK;
}
}  // namespace

int dense_thin_launch(const DenseArgs& g, int epi, hipStream_t stream) {
    if (epi == EPI_GATE) return launch_thin<EPI_GATE>(g, stream);
    if (epi == EPI_PLAIN) return launch_thin<EPI_PLAIN>(g, stream);
    return launch_thin<EPI_LINEAR>(g, stream);
}

int dense_slab_launch(const DenseArgs& g, int splits, hipStream_t stream) {
    const dim3 grid((unsigned)(g.nt * splits));
    if (g.M <= 16)
        dense_slab_kernel<1><<<grid, dim3(512), 0, stream>>>(g);
    else if (g.M <= 32)
        dense_slab_kernel<2><<<grid, dim3(512), 0, stream>>>(g);
    else if (g.M <= 64)
        dense_slab_kernel<4><<<grid, dim3(512), 0, stream>>>(g);
    else
        dense_slab_kernel<8><<<grid, dim3(512), 0, stream>>>(g);
    MOE_LAUNCH_CHECK("dense_slab_kernel");
    return MOE_OK;
}

}  // namespace moe
