// nvfp4_grouped.cu -- matrix products grouped by expert with ragged sizes
// (nvfp4_grouped_mm) on the block-scaled FP4 tensor cores.
//
// out[r,:] = (A[r,:] B[e]^T) * S_dec(A, r) * S_dec(B, e) for the rows r of each
// expert e.  The weight is the MMA's M side (128 of its rows, one accumulator lane
// each) and the tokens its N side: an expert with few tokens then costs a
// narrow product (N down to 16) instead of a padded 128-row one.  With few tokens an
// expert the weights' bytes bound the kernel, with many the tensor cores.
//
// A CTA owns 128 weight rows times BT tokens of one expert.  The experts' sizes
// are known on the device only: the grid has the largest number of token tiles T
// rows in E groups can need (token tiles fastest, so that the CTAs of one weight
// tile run together), and each CTA finds its expert by a warp-wide scan of the
// offsets (CTAs past the last tile leave at once).
//   - warp 0: TMA of the code tiles (256 columns of K: 128 bytes a row, 128-byte
//     swizzle) and bulk copies of the weight's scale tiles, kStages slots deep;
//   - warp 1: per 64 columns, scale tiles to tensor memory and one tcgen05.mma;
//   - warps 4-7: the tokens' scales.  Groups start at any row, so their 128 x 4
//     tiles cannot be laid out ahead: thread i reads token i's 16 scale bytes of a
//     stage (some stages ahead, in registers) and writes them where the tile
//     wants them.  The same warps then read the accumulator and store.
// A tile's last columns may read the next group's rows (or, past T, zeros): those
// products are computed and not stored.  Every wait is bounded; a CTA whose wait
// runs out writes NaN to its tile.
#include "nvfp4_device.cuh"
#include "nvfp4_tensor.cuh"

namespace nvfp4 {
namespace {

constexpr int kGmThreads = 256;
constexpr int kGmRows = 128;                              // weight rows of a tile
constexpr int kGmStageK = 4;                              // 64-column MMA steps per stage
constexpr int kGmAhead = 4;                               // stages the token scales are read ahead

template <int BT>
struct GmShape {
    static constexpr int kStages = BT <= 32 ? 4 : 3;
    static constexpr int kSfbTiles = (BT + 127) / 128;    // 128-row scale tiles of the tokens
    static constexpr int kSlotW = kGmRows * 128, kSlotT = BT * 128;
    static constexpr int kSlotSfw = kGmStageK * 512, kSlotSft = kGmStageK * 512 * kSfbTiles;
    static constexpr int kSlot = kSlotW + kSlotT + kSlotSfw + kSlotSft;
    static constexpr int kSmem = kStages * kSlot + 1024;  // + alignment slack
    static constexpr int kSfCols = 4 + 4 * kSfbTiles;     // tensor-memory columns per step
    static constexpr int kCols = BT + kStages * kGmStageK * kSfCols;
    static constexpr int kTmem = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static constexpr int kSfWarps = BT >= 128 ? 4 : (BT + 31) / 32;   // warps that hold tokens' scales
};

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// token tile `slot` of the groups: its expert, first row and row count (0: none)
__device__ __forceinline__ void find_tile(const GroupedArgs& a, int64_t slot, int BT, int& expert, int64_t& row,
                                          int& rows) {
    const int lane = threadIdx.x & 31;
    expert = 0;
    row = 0;
    rows = 0;
    int64_t before = 0;                                   // tiles of the experts seen so far
    for (int64_t e0 = 0; e0 < a.E; e0 += 32) {
        const int64_t e = e0 + lane;
        int64_t lo = 0, n = 0;
        if (e < a.E) {
            lo = min(max(a.offsets[e], int64_t{0}), a.T);
            n = max(min(max(a.offsets[e + 1], int64_t{0}), a.T) - lo, int64_t{0});
        }
        const int64_t tiles = (n + BT - 1) / BT;
        int64_t upto = tiles;                             // inclusive scan over the lanes
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += u;
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, before + upto > slot);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int64_t first = before + __shfl_sync(0xFFFFFFFFu, upto - tiles, l);
            const int64_t at = (slot - first) * BT;
            expert = static_cast<int>(e0 + l);
            row = __shfl_sync(0xFFFFFFFFu, lo, l) + at;
            rows = static_cast<int>(min(__shfl_sync(0xFFFFFFFFu, n, l) - at, static_cast<int64_t>(BT)));
            return;
        }
        before += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
}

// the 16 scale bytes of token row `row` from step k0 on (zeros past its last step)
__device__ __forceinline__ uint4 token_scales(const GroupedArgs& a, int64_t row, int k0, int ksteps) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (k0 >= ksteps) return v;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(a.scales_a) + row * ksteps + k0;   // 4 bytes a step
    if (ksteps % 4 == 0) return __ldg(reinterpret_cast<const uint4*>(p));
    v.x = __ldg(p);
    if (k0 + 1 < ksteps) v.y = __ldg(p + 1);
    if (k0 + 2 < ksteps) v.z = __ldg(p + 2);
    if (k0 + 3 < ksteps) v.w = __ldg(p + 3);
    return v;
}

template <int BT, int ODT>
__global__ void __launch_bounds__(kGmThreads)
    k_grouped(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapT,
              const GroupedArgs a, int tiles) {
    using G = GmShape<BT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[G::kStages], empty[G::kStages], accb;
    __shared__ uint32_t tmem_base;
    __shared__ int timed_out;
    __shared__ float alpha[BT];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    int expert, rows;
    int64_t row0;
    find_tile(a, blockIdx.x % tiles, BT, expert, row0, rows);
    if (rows == 0) return;                                // the same for the whole CTA
    const int ntile = static_cast<int>(blockIdx.x) / tiles;
    const int n0 = ntile * kGmRows;
    const int ksteps = static_cast<int>(a.K / 64);
    const int nstages = (ksteps + kGmStageK - 1) / kGmStageK;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&tmem_base)),
                     "r"(G::kTmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        for (int i = 0; i < G::kStages; ++i) {
            mbar_init(&full[i], 1 + G::kSfWarps);         // the TMA's transactions and the scale warps
            mbar_init(&empty[i]);
        }
        mbar_init(&accb);
        timed_out = 0;
        asm volatile("fence.mbarrier_init.release.cluster;");
    }
    for (int i = tid; i < rows; i += kGmThreads) {
        float enc, da = 1.0f, db = 1.0f;
        if (a.gamax_a_mode != NVFP4_GAMAX_NONE)
            global_scales(a.gamax_a[a.gamax_a_mode == NVFP4_GAMAX_ROW_GIVEN ? row0 + i : 0], a.bound, enc, da);
        if (a.gamax_b) global_scales(a.gamax_b[expert], a.bound, enc, db);
        alpha[i] = mul_rn(da, db);
    }
    asm volatile("tcgen05.fence::before_thread_sync;");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;");
    const uint32_t tmem = tmem_base;

    if (tid == 0) {
        // ---- codes and the weight's scales ----
        const int wrow = expert * static_cast<int>(a.N) + n0;
        const uint8_t* sfw = a.scales_b + ((static_cast<int64_t>(expert) * ((a.N + 127) / 128) + ntile) * ksteps) * 512;
        for (int t = 0; t < nstages; ++t) {
            const int s = t % G::kStages;
            if (t >= G::kStages && !mbar_wait(&empty[s], static_cast<uint32_t>((t / G::kStages - 1) & 1))) {
                timed_out = 1;
                break;
            }
            const int k0 = t * kGmStageK;
            const int nk = min(ksteps - k0, kGmStageK);
            uint8_t* slot = smem + s * G::kSlot;
            mbar_expect_tx(&full[s], static_cast<uint32_t>(G::kSlotW + G::kSlotT + nk * 512));
            tma_2d(slot, &mapW, k0 * 32, wrow, &full[s]);
            tma_2d(slot + G::kSlotW, &mapT, k0 * 32, static_cast<int>(row0), &full[s]);
            bulk_copy(slot + G::kSlotW + G::kSlotT, sfw + static_cast<int64_t>(k0) * 512, nk * 512, &full[s]);
        }
    } else if (tid == 32) {
        // ---- products ----
        const uint32_t idesc = instr_desc(kGmRows, BT);
        for (int t = 0; t < nstages; ++t) {
            const int s = t % G::kStages;
            if (timed_out || !mbar_wait(&full[s], static_cast<uint32_t>((t / G::kStages) & 1))) {
                timed_out = 1;
                break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;");
            const uint32_t slot = smem_addr(smem) + s * G::kSlot;
            const uint32_t sf = slot + G::kSlotW + G::kSlotT;
            const uint64_t dw = smem_desc(slot, 16, 1024, 2), dt = smem_desc(slot + G::kSlotW, 16, 1024, 2);
            const uint64_t dsw = smem_desc(sf, 0, 128), dst = smem_desc(sf + G::kSlotSfw, 0, 128);
            const uint32_t c0 = tmem + BT + static_cast<uint32_t>(s * kGmStageK * G::kSfCols);
            const int nk = min(ksteps - t * kGmStageK, kGmStageK);
#pragma unroll
            for (int kk = 0; kk < kGmStageK; ++kk) {
                if (kk >= nk) break;
                const uint32_t c = c0 + kk * G::kSfCols;
                asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(c), "l"(dsw + kk * 32));
#pragma unroll
                for (int j = 0; j < G::kSfbTiles; ++j)
                    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(c + 4 + 4 * j),
                                 "l"(dst + (kk * G::kSfbTiles + j) * 32));
                mma_f4(tmem, dw + kk * 2, dt + kk * 2, idesc, c, c + 4, t + kk > 0 ? 1u : 0u);
            }
            asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                smem_addr(&empty[s])));
        }
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_addr(&accb)));
    } else if (warp >= 4 && warp < 4 + G::kSfWarps) {
        // ---- the tokens' scales: rows i and, of 256-token tiles, i + 128 ----
        const int i = tid - 128;
        uint4 v[kGmAhead][G::kSfbTiles];
        auto load = [&](int t, uint4* d) {
#pragma unroll
            for (int j = 0; j < G::kSfbTiles; ++j)
                d[j] = i + 128 * j < rows ? token_scales(a, row0 + i + 128 * j, t * kGmStageK, ksteps)
                                          : make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int u = 0; u < kGmAhead; ++u) load(u, v[u]);
        bool ok = true;
        for (int t0 = 0; t0 < nstages && ok; t0 += kGmAhead) {
#pragma unroll
            for (int u = 0; u < kGmAhead; ++u) {
                const int t = t0 + u;
                if (t >= nstages) break;
                const int s = t % G::kStages;
                if (t >= G::kStages && !mbar_wait(&empty[s], static_cast<uint32_t>((t / G::kStages - 1) & 1))) {
                    timed_out = 1;
                    ok = false;
                    break;
                }
                uint8_t* sf = smem + s * G::kSlot + G::kSlotW + G::kSlotT + G::kSlotSfw + (i % 32) * 16 + (i / 32) * 4;
#pragma unroll
                for (int j = 0; j < G::kSfbTiles; ++j) {
                    const uint32_t w[4] = {v[u][j].x, v[u][j].y, v[u][j].z, v[u][j].w};
#pragma unroll
                    for (int kk = 0; kk < kGmStageK; ++kk)
                        *reinterpret_cast<uint32_t*>(sf + (kk * G::kSfbTiles + j) * 512) = w[kk];
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
                load(t + kGmAhead, v[u]);
            }
        }
    }
    // ---- epilogue: warps 4-7 read their 32 accumulator lanes ----
    if (warp >= 4) {
        __syncwarp();
        if (!mbar_wait(&accb, 0)) timed_out = 1;
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;");
        const int64_t n = n0 + 32 * (warp - 4) + lane;
        const bool bad = timed_out != 0;
        for (int c0 = 0; c0 < rows; c0 += 16) {
            uint32_t v[16];
            asm volatile(
                "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                  "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                : "r"(tmem + (static_cast<uint32_t>(32 * (warp - 4)) << 16) + static_cast<uint32_t>(c0)));
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (c0 + i >= rows || n >= a.N) break;
                // no stage at all (K == 0): the accumulator was never written
                const float acc = nstages ? __uint_as_float(v[i]) : 0.0f;
                const float f = bad ? __int_as_float(0x7FC00000) : mul_rn(acc, alpha[c0 + i]);
                const int64_t o = (row0 + c0 + i) * a.N + n;
                if (ODT == NVFP4_F32) static_cast<float*>(a.out)[o] = f;
                else static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(f);
            }
        }
    }
    pdl_trigger();
    asm volatile("tcgen05.fence::before_thread_sync;");
    __syncthreads();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G::kTmem));
}

template <int BT, int ODT>
cudaError_t launch_grouped_t(const GroupedArgs& a, cudaStream_t s) {
    using G = GmShape<BT>;
    CUtensorMap mapW = {}, mapT = {};
    if (a.K > 0 && (!encode_codes_map(&mapW, a.codes_b, a.E * a.N, a.K, kGmRows) ||
                    !encode_codes_map(&mapT, a.codes_a, a.T, a.K, BT)))
        return cudaErrorInvalidValue;
    // each group's tiles: all full ones, and at most one partial one a group
    const int64_t tiles = a.T / BT + (a.E < a.T ? a.E : a.T);
    const int64_t blocks = tiles * ((a.N + kGmRows - 1) / kGmRows);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    static thread_local int configured_dev = -1;         // the attribute is per device
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_dev != dev) {
        const cudaError_t e =
            cudaFuncSetAttribute(k_grouped<BT, ODT>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
        if (e != cudaSuccess) return e;
        configured_dev = dev;
    }
    return launch_pdl(k_grouped<BT, ODT>, dim3(static_cast<unsigned>(blocks)), dim3(kGmThreads), G::kSmem, s, mapW,
                      mapT, a, static_cast<int>(tiles));
}

template <int BT>
cudaError_t launch_grouped_o(const GroupedArgs& a, cudaStream_t s) {
    return a.out_dtype == NVFP4_F32 ? launch_grouped_t<BT, NVFP4_F32>(a, s) : launch_grouped_t<BT, NVFP4_BF16>(a, s);
}

}  // namespace

int launch_grouped_mm(const GroupedArgs& a, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // tokens a tile: about twice the mean group, so that most groups are one tile
    const int64_t mean = (a.T + a.E - 1) / a.E;
    if (mean <= 8) return static_cast<int>(launch_grouped_o<16>(a, s));
    if (mean <= 16) return static_cast<int>(launch_grouped_o<32>(a, s));
    if (mean <= 32) return static_cast<int>(launch_grouped_o<64>(a, s));
    return static_cast<int>(launch_grouped_o<128>(a, s));
}

}  // namespace nvfp4
