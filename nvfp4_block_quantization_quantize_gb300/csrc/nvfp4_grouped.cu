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
// offsets (CTAs past the last tile only take part in its barriers).
//   - warp 0: TMA of the code tiles (256 columns of K: 128 bytes a row, 128-byte
//     swizzle) and bulk copies of the weight's scale tiles, kStages slots deep;
//   - warp 1: per 64 columns, scale tiles to tensor memory and one tcgen05.mma;
//   - warps 4-7: the tokens' scales.  Groups start at any row, so their 128 x 4
//     tiles cannot be laid out ahead: thread i reads token i's 16 scale bytes of a
//     stage (some stages ahead, in registers) and writes them where the tile
//     wants them;
//   - warps 2 and 3: the tokens' decode scales.  All warps then store the accumulator.
// Measured, in a graph of calls: 64 tokens on 64 experts of [2048, 4096] 27.9 us (5.8 TB/s), 2 of 8
// experts of [1024, 1024] 3.6 us, 1999 tokens on 13 experts of [1430, 2112] 12.0 us; one group
// of 64 tokens x [14336, 4096] 11.3 us, x [4096, 14336] 20.8 us (32 weight tiles for 152 SMs:
// K is not split).
// A tile's last columns may read the next group's rows (or, past T, zeros): those
// products are computed and not stored.  Every wait is bounded; a CTA whose wait
// runs out writes NaN to its tile.
#include <cmath>
#include <type_traits>

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
    static constexpr int kSlotW = kGmRows * 128, kSlotT = BT * 128;
    static constexpr int kSlotSfw = kGmStageK * 512, kSlotSft = kGmStageK * 512;
    static constexpr int kSlot = kSlotW + kSlotT + kSlotSfw + kSlotSft;
    static constexpr int kSmem = kStages * kSlot + 1024;  // + alignment slack
    static constexpr int kSfCols = 8;                     // tensor-memory columns per step: 4 of each side's scales
    static constexpr int kCols = BT + kStages * kGmStageK * kSfCols;
    static constexpr int kTmem = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static constexpr int kSfWarps = (BT + 31) / 32;       // warps that hold tokens' scales
    static_assert(BT <= 128, "one 128-row scale tile holds the tokens");
};

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// rows [lo, hi) of expert e, the offsets clamped to [0, T]
__device__ __forceinline__ void group_rows(const GroupedArgs& a, int e, int& lo, int& hi) {
    const long long* off = reinterpret_cast<const long long*>(a.offsets) + e;
    const long long T = a.T;
    lo = static_cast<int>(min(max(__ldg(off), 0LL), T));
    hi = max(static_cast<int>(min(max(__ldg(off + 1), 0LL), T)), lo);
}

// Token tile `slot` of the groups: its expert, first row and row count (0: past the
// last).  A whole warp calls it; T < 2^31, so 32 bits do.
__device__ __forceinline__ void find_tile(const GroupedArgs& a, int slot, int BT, int& expert, int& row, int& rows) {
    const int lane = threadIdx.x & 31;
    expert = 0;
    row = 0;
    rows = 0;
    int before = 0;                                       // tiles of the experts seen so far
    for (int e0 = 0; e0 < static_cast<int>(a.E); e0 += 32) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < a.E) group_rows(a, e, lo, hi);
        const int n = hi - lo;
        const int tiles = (n + BT - 1) / BT;
        int upto = tiles;                                 // inclusive scan over the lanes
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += u;
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, before + upto > slot);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int at = (slot - before - __shfl_sync(0xFFFFFFFFu, upto - tiles, l)) * BT;
            expert = e0 + l;
            row = __shfl_sync(0xFFFFFFFFu, lo, l) + at;
            rows = min(__shfl_sync(0xFFFFFFFFu, n, l) - at, BT);
            return;
        }
        before += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
}

// the 16 scale bytes of token row `row` from step k0 on (zeros past its last step)
__device__ __forceinline__ uint4 token_scales(const GroupedArgs& a, int row, int k0, int ksteps) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (k0 >= ksteps) return v;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(a.scales_a) + static_cast<int64_t>(row) * ksteps + k0;
    if (ksteps % 4 == 0) return __ldg(reinterpret_cast<const uint4*>(p));
    v.x = __ldg(p);
    if (k0 + 1 < ksteps) v.y = __ldg(p + 1);
    if (k0 + 2 < ksteps) v.z = __ldg(p + 2);
    if (k0 + 3 < ksteps) v.w = __ldg(p + 3);
    return v;
}

// 32 accumulator columns of this warp's 32 lanes, from the warp's tensor-memory address
__device__ __forceinline__ void load_columns(uint32_t from, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(from));
}

// Scales and stores them: token col + i of the tile (of `rows`, the first at row0 of out) for
// weight row nw + lane.  alpha: the tile's decode scales (readable up to col + 31).  bad: NaN
// instead.  bf16 rows that start on 16 bytes are turned in shared memory (2 KB at turn), so
// that four lanes store a token's 32 rows at 16 bytes each; else a lane stores its own row.
constexpr int kTurn = 32 * 64;

template <int ODT>
__device__ __forceinline__ void store_columns(const GroupedArgs& a, const uint32_t* v, const float* alpha, int col,
                                              int rows, int row0, int64_t nw, bool bad, uint8_t* turn, int lane) {
    float f[32];
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const float4 al = *reinterpret_cast<const float4*>(alpha + col + i);
        f[i] = mul_rn(__uint_as_float(v[i]), al.x);
        f[i + 1] = mul_rn(__uint_as_float(v[i + 1]), al.y);
        f[i + 2] = mul_rn(__uint_as_float(v[i + 2]), al.z);
        f[i + 3] = mul_rn(__uint_as_float(v[i + 3]), al.w);
    }
    if (bad) {
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = __int_as_float(0x7FC00000);
    }
    if (ODT == NVFP4_BF16 && a.N % 8 == 0 && !bad) {      // (bad: copies may still come into the stages)
        __syncwarp();                                     // the last turn is read
#pragma unroll
        for (int i = 0; i < 32; ++i)
            *reinterpret_cast<__nv_bfloat16*>(turn + i * 64 + lane * 2) = __float2bfloat16_rn(f[i]);
        __syncwarp();
        const int64_t n = nw + (lane & 3) * 8;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            const int token = col + i + lane / 4;
            const uint4 o = *reinterpret_cast<const uint4*>(turn + (i + lane / 4) * 64 + (lane & 3) * 16);
            if (token < rows && n < a.N)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<int64_t>(row0 + token) * a.N + n) = o;
        }
    } else if (nw + lane < a.N) {
        int64_t o = static_cast<int64_t>(row0 + col) * a.N + nw + lane;
#pragma unroll
        for (int i = 0; i < 32; ++i, o += a.N) {
            if (col + i >= rows) break;
            if (ODT == NVFP4_F32) static_cast<float*>(a.out)[o] = f[i];
            else static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(f[i]);
        }
    }
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
    __shared__ __align__(16) float alpha[BT < 32 ? 32 : BT];

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);               // the same for the whole warp, and known to be
    // what needs no input, while the kernel before may still run
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&tmem_base)),
                     "r"(G::kTmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 32) {
        for (int i = 0; i < G::kStages; ++i) {
            mbar_init(&full[i], 1 + G::kSfWarps);         // the TMA's transactions and the scale warps
            mbar_init(&empty[i]);
        }
        mbar_init(&accb);
        timed_out = 0;
        asm volatile("fence.mbarrier_init.release.cluster;");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&mapW)));
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&mapT)));
    }
    pdl_trigger();                                        // the next kernel waits for this one's end itself
    pdl_wait();
    int expert, row0, rows;
    find_tile(a, blockIdx.x % tiles, BT, expert, row0, rows);
    const int ntile = static_cast<int>(blockIdx.x) / tiles;
    const int n0 = ntile * kGmRows;
    const int ksteps = static_cast<int>(a.K / 64);
    // a tile past the last takes part in the barriers alone
    const int nstages = rows == 0 ? 0 : (ksteps + kGmStageK - 1) / kGmStageK;
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
            tma_2d(slot + G::kSlotW, &mapT, k0 * 32, row0, &full[s]);
            bulk_copy(slot + G::kSlotW + G::kSlotT, sfw + static_cast<int64_t>(k0) * 512, nk * 512, &full[s]);
        }
    } else if (warp == 1) {
        // ---- products (the whole warp issues, one lane's predicate guards) ----
        const uint32_t idesc = instr_desc(kGmRows, BT), el = elect_one();
        for (int t = 0; t < nstages; ++t) {
            const int s = t % G::kStages;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[s], static_cast<uint32_t>((t / G::kStages) & 1)))) {
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
                copy_scales_warp<1>(el, c, dsw + kk * 32);
                copy_scales_warp<1>(el, c + 4, dst + kk * 32);
                mma_f4_warp<1>(el, tmem, dw + kk * 2, dt + kk * 2, idesc, c, c + 4, t + kk > 0 ? 1u : 0u);
            }
            commit_warp<1>(el, &empty[s]);
        }
        commit_warp<1>(el, &accb);
    } else if (warp == 2 || warp == 3) {
        // ---- the tokens' decode scales ----
        for (int i = tid - 64; i < (BT < 32 ? 32 : BT); i += 64) {
            float enc, da = 1.0f, db = 1.0f;
            if (i < rows && a.gamax_a_mode != NVFP4_GAMAX_NONE)
                global_scales(a.gamax_a[a.gamax_a_mode == NVFP4_GAMAX_ROW_GIVEN ? row0 + i : 0], a.bound, enc, da);
            if (i < rows && a.gamax_b) global_scales(a.gamax_b[expert], a.bound, enc, db);
            alpha[i] = mul_rn(da, db);
        }
    } else if (warp >= 4 && warp < 4 + G::kSfWarps) {
        // ---- the tokens' scales: row i ----
        const int i = tid - 128;
        uint4 v[kGmAhead];
        auto load = [&](int t) {
            return i < rows ? token_scales(a, row0 + i, t * kGmStageK, ksteps) : make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int u = 0; u < kGmAhead; ++u) v[u] = load(u);
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
                const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                for (int kk = 0; kk < kGmStageK; ++kk) *reinterpret_cast<uint32_t*>(sf + kk * 512) = w[kk];
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
                v[u] = load(t + kGmAhead);
            }
        }
    }
    // ---- epilogue: every warp a quarter of the accumulator's lanes and every other 32 columns ----
    __syncwarp();
    if (!mbar_wait(&accb, 0)) timed_out = 1;
    __syncthreads();                                      // the decode scales are there, the stages free
    asm volatile("tcgen05.fence::after_thread_sync;");
    const bool bad = timed_out != 0;
    const int quad = warp & 3;
    for (int c0 = 32 * (warp >> 2); c0 < rows; c0 += 64) {
        uint32_t v[32];
        load_columns(tmem + (static_cast<uint32_t>(32 * quad) << 16) + static_cast<uint32_t>(c0), v);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        if (nstages == 0) {                               // K == 0: the accumulator was never written
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0;
        }
        store_columns<ODT>(a, v, alpha, c0, rows, row0, n0 + 32 * quad, bad, smem + warp * kTurn, lane);
    }
    asm volatile("tcgen05.fence::before_thread_sync;");
    __syncthreads();
    if (warp == 0) {
        if (bad) settle();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G::kTmem));
    }
}

// ---- many tokens an expert: pairs of SMs -------------------------------------------------------
// The same product with tcgen05 .cta_group::2: the two CTAs of a cluster share a tile of 256
// weight rows (128 each, and their accumulator lanes) times up to 192 tokens (each CTA
// stages half of them), so a CTA loads 28 KB of codes per 256 columns for 128 x 192 outputs
// instead of 32 KB for 128 x 128: a 128 x 128 tile wants about 140 bytes a clock per SM
// from L2 at the FP4 rate, more than it gives.  Two accumulators (2 x 192 of 512
// tensor-memory columns) let the stores of one tile overlap the products of the next;
// one persistent CTA per SM walks the tiles.
//   warp 0       TMA of the CTA's own half of a stage of 512 columns (one copy brings both its
//                256-column pieces of 128 bytes a row: a copy has a fixed cost), all of it
//                signalling the first CTA's barrier (a thread's own release to the other CTA
//                would cost about 0.9 us a stage, measured, against 0.4 us of products)
//   warp 1       in the first CTA: scale copies and MMAs for both
//   warps 2-9    accumulator to global memory
// The tokens' scales are laid out for the tiles by a kernel before (k_token_scales, into
// the caller's workspace).  The MMA's N is the tile's token count rounded up to 32, so a
// group's last tile costs what it needs.  A wait that runs out stops the CTA's roles; its
// unfinished tiles become NaN.
// Measured: 8192 tokens on 8 experts of [14336, 4096] 188 to 205 us, as calls and in a graph alike, by
// the card and its power (4.7 to 5.1 PFLOP/s; at 189 us tensor pipe 56 %, L2 61 % of their peaks).  With
// parts left out, on a card where the whole took 188: the copies alone 140 us (about the 86 bytes a clock
// an SM's TMA takes in at most), products with their scale copies alone 144, both without the stores 160.
constexpr int kGpStoreWarps = 8;                          // two for each quarter of the accumulator's lanes
constexpr int kGpThreads = 64 + 32 * kGpStoreWarps;
constexpr int kGpBT = 192;
constexpr int kGpStages = 3;
constexpr int kGpStageK = 2 * kGmStageK;                  // 64-column steps of a stage, in two halves
constexpr int kGpHalfW = 128 * 128, kGpHalfT = kGpBT / 2 * 128;              // codes of a half
constexpr int kGpSlotSfw = kGpStageK * 512, kGpSlotSft = kGpStageK * 1024;
constexpr int kGpSlot = 2 * (kGpHalfW + kGpHalfT) + kGpSlotSfw + kGpSlotSft;  // 68 KB
constexpr int kGpSmem = kGpStages * kGpSlot + kGpStoreWarps * kTurn + 1024;
constexpr int kGpGroups = 256;                            // experts whose places are kept in shared memory
constexpr uint32_t kGpColSf = 2 * kGpBT;                  // scales: two stages of 4 steps of 4 + 8 columns

// Tiles are walked in blocks of token tiles whose codes are about kBlockBytes, a block's token tiles
// fastest and then its weight tiles, so that what runs together shares tokens and weights and
// a block's tokens stay in L2.  Without blocks the weights of all experts run together: us without /
// with, 8192 tokens on 8 experts of [4096, 14336] 229 / 192, 16384 on 64 of [2048, 7168] 197 / 142, 8192 on 8
// of [14336, 4096] 193 / 190 (blocks of 1 MB to 4 MB 193 to 195, of 30 MB at K = 14336 197).  (Single-SM
// tiles go either way, so they are not cut: 64 experts 8192 x 2048 of K 7168 129 / 119, 32 experts 4096 x 2048 of
// K 4096 40 / 42; pairs take the first.)
constexpr int64_t kBlockBytes = 10 << 20;

unsigned block_tiles(const GroupedArgs& a, int64_t slots) {
    const int64_t n = kBlockBytes / (kGpBT * a.K / 2);
    return static_cast<unsigned>(n < 3 ? 3 : n > slots ? slots : n);
}

// token tile and weight tile of `tile`
__device__ __forceinline__ void place(unsigned tile, unsigned slots, unsigned wide, unsigned block, int& slot, int& ntile) {
    const unsigned b = tile / (block * wide), in = tile - b * (block * wide), n = min(block, slots - b * block);
    slot = static_cast<int>(b * block + in % n);
    ntile = static_cast<int>(in / n);
}

// token tiles of 192 rows, at most: all full ones, and one partial one a group
int64_t pair_slots(const GroupedArgs& a) { return a.T / kGpBT + (a.E < a.T ? a.E : a.T); }

// The token tiles' scales in the tensor cores' layout: tile (slot, step, half) of 512
// bytes at (slot * ksteps + step) * 2 + half, word (r % 32) * 4 + r / 32 of it row r's
// four bytes of the step.  One CTA a slot; a thread takes row tid, so that a row's
// bytes are read by one thread, 16 at a time.
__global__ void __launch_bounds__(256) k_token_scales(const GroupedArgs a, uint32_t* out) {
    pdl_trigger();                                        // the product waits for this kernel's end itself
    pdl_wait();
    int expert, row0, rows;
    find_tile(a, blockIdx.x, kGpBT, expert, row0, rows);
    const int ksteps = static_cast<int>(a.K / 64), i = threadIdx.x;
    if (rows == 0 || i >= (rows + 31) / 32 * 32) return;  // what the product copies but no stored column uses stays
    for (int k0 = blockIdx.y * 8; k0 < min(ksteps, static_cast<int>(blockIdx.y + 1) * 8); k0 += 4) {
        const uint4 v = i < rows ? token_scales(a, row0 + i, k0, ksteps) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t* o = out + ((static_cast<int64_t>(blockIdx.x) * ksteps + k0) * 2 + i / 128) * 128 + (i % 32) * 4 + i % 128 / 32;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k0 + k < ksteps) o[k * 256] = w[k];
    }
}

__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
    return r;
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// mbar_wait for arrivals from the other CTA of the pair
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity) {
    for (long it = 0; it < kWaitLimit; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return false;
}

// both of two barriers' phases (of the second unless skip), with the two polls under way together; a whole warp
// calls it and all its lanes get the same answer
__device__ __forceinline__ bool mbar_wait_both(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, bool skip) {
    for (long it = 0; it < kWaitLimit; ++it) {
        uint32_t x, y;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%2], %3;\n\t"
            "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 q, [%4], %5;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t"
            "selp.u32 %1, 1, 0, q;\n\t}"
            : "=r"(x), "=r"(y)
            : "r"(smem_addr(a)), "r"(pa), "r"(smem_addr(b)), "r"(pb)
            : "memory");
        if (__all_sync(0xFFFFFFFFu, x && (y || skip))) return true;
    }
    return false;
}

// TMA into this CTA's shared memory, signalling the barrier at cluster address bar (of either CTA)
__device__ __forceinline__ void tma_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_3d_pair(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// ---- a pair's bf16 output by TMA
// The accumulator is read in the layout of a product's fragments: word 16 hh + 4 j + 2 m + e of
// lane l is column 8 j + 2 (l % 4) + e of row 16 hh + 8 m + l / 4 (32 columns, the warp's 32 rows),
// so that a pair of words is a token pair of one weight row and a transposing stmatrix turns 8
// tokens x 32 rows at once: against two-byte stores of the 32x32b layout's rows a quarter of the
// shared memory's accesses (8192 tokens on 8 experts of
// [14336, 4096]: without stores 160 us, with those 202, by these 193; two warps' rows together,
// 128 bytes a token, gain nothing, stores by lanes from the same layout take 200).
__device__ __forceinline__ void load_fragments(uint32_t from, uint32_t* v) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh, v += 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
            "[%16];"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
              "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
            : "r"(from + (static_cast<uint32_t>(16 * hh) << 16)));
}

// the stores of this thread's groups are out of shared memory (ALL: are done)
template <bool ALL>
__device__ __forceinline__ void bulk_stores_wait() {
    if (ALL) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    else asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// store_columns for fragments: 32 tokens whole go out of shared memory (2 KB at turn, 64 bytes a token,
// 64-byte swizzle) by TMA, the last of a tile by lanes.
__device__ __forceinline__ void store_fragments(const GroupedArgs& a, const CUtensorMap* out, const uint32_t* v,
                                                const float* alpha, int col, int rows, int row0, int64_t nw, bool bad,
                                                uint8_t* turn, int lane) {
    if (nw >= a.N) return;
    if (lane == 0) bulk_stores_wait<false>();
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 al = *reinterpret_cast<const float2*>(alpha + col + 8 * j + 2 * (lane & 3));
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t* u = v + 16 * (q >> 1) + 4 * j + 2 * (q & 1);
            const __nv_bfloat162 b = __floats2bfloat162_rn(mul_rn(__uint_as_float(u[0]), al.x), mul_rn(__uint_as_float(u[1]), al.y));
            w[q] = bad ? 0x7FC07FC0u : *reinterpret_cast<const uint32_t*>(&b);
        }
        // lane l gives the place of token 8 j + l % 8's rows 8 (l / 8) to 8 (l / 8) + 7
        const int i = 8 * j + (lane & 7);
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                         smem_addr(turn + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4))),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
    }
    if (col + 32 <= rows) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                             reinterpret_cast<uint64_t>(out)),
                         "r"(static_cast<int>(nw)), "r"(row0 + col), "r"(smem_addr(turn))
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        return;
    }
    __syncwarp();
    const int64_t n = nw + (lane & 3) * 8;
#pragma unroll
    for (int i = lane / 4; i < 32; i += 8) {
        const uint4 o = *reinterpret_cast<const uint4*>(turn + i * 64 + (((lane & 3) ^ ((i >> 1) & 3)) << 4));
        if (col + i < rows && n < a.N)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<int64_t>(row0 + col + i) * a.N + n) = o;
    }
    __syncwarp();
}

template <int ODT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGpThreads, 1)
    k_grouped_pair(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapT,
                   const __grid_constant__ CUtensorMap mapW2, const __grid_constant__ CUtensorMap mapT2,
                   const __grid_constant__ CUtensorMap mapSW, const __grid_constant__ CUtensorMap mapST,
                   const __grid_constant__ CUtensorMap mapOut,
                   const GroupedArgs a, unsigned slots, unsigned all_tiles, unsigned block) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[kGpStages], done[2 * kGpStages], acc_full[2], acc_empty[2];
    __shared__ uint32_t tmem_base;
    __shared__ volatile int timed_out;
    __shared__ __align__(16) float alpha[2][kGpBT];
    __shared__ int tiles_to[kGpGroups], first_row[kGpGroups], end_row[kGpGroups];     // of each expert

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);               // the same for the whole warp, and known to be
    const int rank = static_cast<int>(blockIdx.x & 1);
    const unsigned pairs = gridDim.x / 2;
    const int ksteps = static_cast<int>(a.K / 64);
    const int nstages = (ksteps + kGpStageK - 1) / kGpStageK;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    if (tid == 32) {
        for (int i = 0; i < kGpStages; ++i) mbar_init(&full[i]);             // used in the first CTA: both CTAs' transactions
        for (int i = 0; i < 2 * kGpStages; ++i) mbar_init(&done[i]);         // the products of a stage's half
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i]);
            mbar_init(&acc_empty[i], 2 * kGpStoreWarps);  // of both CTAs
        }
        timed_out = 0;
        asm volatile("fence.mbarrier_init.release.cluster;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;");
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    asm volatile("tcgen05.fence::after_thread_sync;");
    const uint32_t tmem = __reduce_max_sync(0xFFFFFFFFu, tmem_base);      // in a uniform register, as tcgen05 operands are
    pdl_trigger();                                        // the next kernel waits for this one's end itself
    pdl_wait();

    // the experts' rows, and the token tiles up to each: what find_tile makes of the offsets, once
    const bool few = a.E <= kGpGroups;
    if (few) {
        for (int e = tid; e < a.E; e += kGpThreads) group_rows(a, e, first_row[e], end_row[e]);
        __syncthreads();
        if (warp == 0) {
            int before = 0;
            for (int e0 = 0; e0 < a.E; e0 += 32) {
                const int e = e0 + lane;
                int upto = e < a.E ? (end_row[e] - first_row[e] + kGpBT - 1) / kGpBT : 0;
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const int u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                    if (lane >= o) upto += u;
                }
                if (e < a.E) tiles_to[e] = before + upto;
                before += __shfl_sync(0xFFFFFFFFu, upto, 31);
            }
        }
        __syncthreads();
    }
    auto find = [&](int slot, int& expert, int& row0, int& rows) {
        if (!few) return find_tile(a, slot, kGpBT, expert, row0, rows);
        expert = row0 = rows = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, e0 + lane < a.E && tiles_to[e0 + lane] > slot);
            if (!hit) continue;
            expert = e0 + __ffs(hit) - 1;
            row0 = first_row[expert] + (slot - (expert ? tiles_to[expert - 1] : 0)) * kGpBT;
            rows = min(end_row[expert] - row0, kGpBT);
            return;
        }
    };
    int st = 0, it = 0;                                   // stages and (non-empty) tiles so far
    const unsigned wide = static_cast<unsigned>((a.N + 255) / 256);
    // one pass over the pair's tiles, the same in every role
    auto each_tile = [&](auto body) {
        for (unsigned tile = blockIdx.x / 2; tile < all_tiles; tile += pairs) {
            int slot, ntile, expert, row0, rows;
            place(tile, slots, wide, block, slot, ntile);
            find(slot, expert, row0, rows);
            // the same in all lanes; the reduction lets the compiler know
            rows = __reduce_max_sync(0xFFFFFFFFu, rows);
            if (rows == 0) continue;
            const int N = (rows + 31) / 32 * 32;
            if (!body(ntile, slot, expert, row0, rows, N)) return;
            ++it;
        }
    };
    if (warp == 0) {
        const int sf_tiles = static_cast<int>((a.N + 127) / 128);
        each_tile([&](int ntile, int slot, int expert, int row0, int, int N) {
            const int n0 = ntile * 256 + rank * 128;
            const int wrow = expert * static_cast<int>(a.N) + n0, trow = row0 + rank * (N / 2);
            // a pair's second half past N has no scale tile of its own: any one will do
            const int sfw = (expert * sf_tiles + min(n0 / 128, sf_tiles - 1)) * ksteps, sft = slot * ksteps * 2;
            for (int t = 0; t < nstages; ++t, ++st) {
                const int s = st % kGpStages;
                if (st >= kGpStages && !mbar_wait_cluster(&done[2 * s + 1], static_cast<uint32_t>((st / kGpStages - 1) & 1))) {
                    timed_out = 1;
                    return false;
                }
                if (lane == 0) {
                    const int k0 = t * kGpStageK;
                    uint8_t *dst = smem + s * kGpSlot, *dstT = dst + 2 * kGpHalfW, *sf = dstT + 2 * kGpHalfT;
                    const uint32_t bar = cluster_addr(&full[s], 0);
                    // both halves in one copy, but for a row's last, ragged piece
                    const bool ragged = ksteps % kGmStageK && k0 + kGpStageK > ksteps;
                    const int one = ragged && k0 + kGmStageK >= ksteps;      // that piece alone is there
                    if (rank == 0) mbar_expect_tx(&full[s], 2 * (kGpSlot - one * (kGpHalfW + kGpHalfT)));
                    if (!ragged) {
                        tma_3d_pair(dst, &mapW2, 0, wrow, k0 / kGmStageK, bar);
                        tma_3d_pair(dstT, &mapT2, 0, trow, k0 / kGmStageK, bar);
                    } else {
                        for (int h = 0; h < 2 - one; ++h) {
                            tma_2d_pair(dst + h * kGpHalfW, &mapW, (k0 + h * kGmStageK) * 32, wrow, bar);
                            tma_2d_pair(dstT + h * kGpHalfT, &mapT, (k0 + h * kGmStageK) * 32, trow, bar);
                        }
                    }
                    tma_2d_pair(sf, &mapSW, 0, sfw + k0, bar);
                    tma_2d_pair(sf + kGpSlotSfw, &mapST, 0, sft + 2 * k0, bar);
                }
                __syncwarp();
            }
            return true;
        });
    } else if (warp == 1 && rank == 0) {
        // Slots and phases are counted up, and every operand is the base plus a counter's multiple: what
        // the compiler can keep in uniform registers (division by the ring's length cannot) and issue fast.
        const uint32_t el = elect_one();
        const uint32_t sf0 = 2 * (kGpHalfW + kGpHalfT);
        const uint64_t dw0 = smem_desc(smem_addr(smem), 16, 1024, 2);
        const uint64_t dt0 = smem_desc(smem_addr(smem) + 2 * kGpHalfW, 16, 1024, 2);
        const uint64_t dsw0 = smem_desc(smem_addr(smem) + sf0, 0, 128);
        const uint64_t dst0 = smem_desc(smem_addr(smem) + sf0 + kGpSlotSfw, 0, 128);
        uint32_t s = 0, phase = 0;                        // of the stages
        bool first = true;
        each_tile([&](int, int, int, int, int, int N) {
            const uint32_t idesc = instr_desc(256, N);
            const int buf = it & 1;
            if (it >= 2 && !__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&acc_empty[buf], static_cast<uint32_t>((it / 2 - 1) & 1)))) {
                timed_out = 1;
                return false;
            }
            asm volatile("tcgen05.fence::after_thread_sync;");
            const uint32_t d = tmem + buf * kGpBT;
            // the steps of a half from the stage's offset `at` on (a branch between two issues costs about as much
            // as an issue, so whole halves and both kinds of tiles have code of their own)
            auto steps = [&](auto two, auto whole, uint64_t at, int half, uint32_t acc, int nk) {
                const uint64_t dw = dw0 + at + half * (kGpHalfW / 16), dt = dt0 + at + half * (kGpHalfT / 16);
                const uint64_t dsw = dsw0 + at + half * (kGpSlotSfw / 32), dst = dst0 + at + half * (kGpSlotSft / 32);
                const uint32_t c0 = tmem + kGpColSf + half * 48;
#pragma unroll
                for (int kk = 0; kk < kGmStageK; ++kk) {
                    if (!decltype(whole)::value && kk >= nk) break;
                    const uint32_t c = c0 + kk * 12;
                    copy_scales_warp<2>(el, c, dsw + kk * 32);
                    copy_scales_warp<2>(el, c + 4, dst + kk * 64);
                    if (decltype(two)::value) copy_scales_warp<2>(el, c + 8, dst + kk * 64 + 32);
                    mma_f4_warp<2>(el, d, dw + kk * 2, dt + kk * 2, idesc, c, c + 4, kk > 0 ? 1u : acc);
                }
            };
            auto k_loop = [&](auto two) {
                for (int k0 = 0; k0 < ksteps; k0 += kGpStageK) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        // The stage is there, and the products of the same half of the stage before are done: the
                        // scales' columns of two halves are used in turn, and a copy is not ordered behind earlier
                        // products that read what it overwrites.  The other half's products keep the pipe busy.
                        const uint32_t before = s ? s - 1 : kGpStages - 1;
                        if (!mbar_wait_both(&full[s], phase, &done[2 * before + half], s ? phase : phase ^ 1, first))
                            return false;
                        asm volatile("tcgen05.fence::after_thread_sync;");
                        const uint64_t at = s * (kGpSlot / 16);
                        const int nk = ksteps - k0 - half * kGmStageK;       // of a ragged stage's second half <= 0
                        const uint32_t acc = k0 + half > 0 ? 1u : 0u;
                        if (nk >= kGmStageK) steps(two, std::true_type{}, at, half, acc, nk);
                        else steps(two, std::false_type{}, at, half, acc, nk);
                        commit_warp<2>(el, &done[2 * s + half]);
                    }
                    first = false;
                    if (++s == kGpStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
                return true;
            };
            if (!__all_sync(0xFFFFFFFFu, N > 128 ? k_loop(std::true_type{}) : k_loop(std::false_type{}))) {
                timed_out = 1;
                return false;
            }
            commit_warp<2>(el, &acc_full[buf]);
            return true;
        });
    } else if (warp >= 2) {
        // a quarter of the accumulator's lanes, and columns 96 * part up to 96 more
        constexpr int kCols = kGpBT / (kGpStoreWarps / 4);
        const int quad = warp & 3, part = (warp - 2) / 4;
        const uint32_t from = tmem + (static_cast<uint32_t>(32 * quad) << 16) + static_cast<uint32_t>(part * kCols);
        uint8_t* turn = smem + kGpStages * kGpSlot + (warp - 2) * kTurn;
        const bool whole = ODT == NVFP4_BF16 && a.N % 8 == 0;                // rows of out start on 16 bytes
        each_tile([&](int ntile, int, int expert, int row0, int rows, int) {
            const int buf = it & 1;
            for (int i = tid - 64; i < kGpBT; i += 32 * kGpStoreWarps) {
                float enc, da = 1.0f, db = 1.0f;
                if (i < rows && a.gamax_a_mode != NVFP4_GAMAX_NONE)
                    global_scales(a.gamax_a[a.gamax_a_mode == NVFP4_GAMAX_ROW_GIVEN ? row0 + i : 0], a.bound, enc, da);
                if (a.gamax_b) global_scales(a.gamax_b[expert], a.bound, enc, db);
                alpha[buf][i] = mul_rn(da, db);
            }
            asm volatile("bar.sync 1, %0;" ::"n"(32 * kGpStoreWarps) : "memory");
            if (!timed_out && !mbar_wait_cluster(&acc_full[buf], static_cast<uint32_t>((it / 2) & 1))) timed_out = 1;
            __syncwarp();
            const bool bad = timed_out != 0;
            asm volatile("tcgen05.fence::after_thread_sync;");
            // all of the warp's columns first, so that the accumulator is free before anything is stored
            uint32_t v[kCols];
#pragma unroll
            for (int c = 0; c < kCols; c += 32)
                if (part * kCols + c < rows) {
                    if (whole) load_fragments(from + buf * kGpBT + static_cast<uint32_t>(c), v + c);
                    else load_columns(from + buf * kGpBT + static_cast<uint32_t>(c), v + c);
                }
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
            asm volatile("tcgen05.fence::before_thread_sync;");
            __syncwarp();
            if (lane == 0) {
                if (rank == 0) mbar_arrive(&acc_empty[buf]);
                else mbar_arrive_cluster(cluster_addr(&acc_empty[buf], 0));
            }
            const int64_t nw = static_cast<int64_t>(ntile) * 256 + rank * 128 + 32 * quad;     // the warp's first row
#pragma unroll
            for (int c = 0; c < kCols; c += 32) {
                const int col = part * kCols + c;
                if (col >= rows) break;
                if (whole) store_fragments(a, &mapOut, v + c, alpha[buf], col, rows, row0, nw, bad, turn, lane);
                else store_columns<ODT>(a, v + c, alpha[buf], col, rows, row0, nw, bad, turn, lane);
            }
            return true;
        });
        if (lane == 0) bulk_stores_wait<true>();
    }
    // neither CTA leaves while the other may still read its shared memory or arrive at its barriers
    __syncwarp();
    if (timed_out) settle();
    asm volatile("tcgen05.fence::before_thread_sync;");
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

template <int ODT>
cudaError_t launch_pair(const GroupedArgs& a, cudaStream_t s) {
    const int64_t slots = pair_slots(a), ksteps = a.K / 64;
    const int64_t tiles = slots * ((a.N + 255) / 256);
    if (tiles > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    CUtensorMap mapW = {}, mapT = {}, mapW2 = {}, mapT2 = {}, mapSW = {}, mapST = {}, mapOut = {};
    if (!encode_codes_map(&mapW, a.codes_b, a.E * a.N, a.K, 128) ||
        !encode_codes_map(&mapT, a.codes_a, a.T, a.K, kGpBT / 2) ||
        !encode_codes_map2(&mapW2, a.codes_b, a.E * a.N, a.K, 128) ||
        !encode_codes_map2(&mapT2, a.codes_a, a.T, a.K, kGpBT / 2) ||
        !encode_scales_map(&mapSW, a.scales_b, a.E * ((a.N + 127) / 128) * ksteps, kGpStageK) ||
        !encode_scales_map(&mapST, a.workspace, slots * ksteps * 2, 2 * kGpStageK) ||
        (ODT == NVFP4_BF16 && a.N % 8 == 0 && !encode_out_map(&mapOut, a.out, a.T, a.N)))
        return cudaErrorInvalidValue;
    static thread_local int configured_dev = -1;         // the attribute and the pairs are per device
    static thread_local int pairs_at_once = 0;            // an odd SM of a GPC has no partner
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_dev != dev) {
        cudaError_t e = cudaFuncSetAttribute(k_grouped_pair<ODT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGpSmem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(sm_count() / 2 * 2));
        cfg.blockDim = dim3(kGpThreads);
        cfg.dynamicSmemBytes = kGpSmem;
        if ((e = cudaOccupancyMaxActiveClusters(&pairs_at_once, k_grouped_pair<ODT>, &cfg)) != cudaSuccess) return e;
        if (pairs_at_once < 1) return cudaErrorInvalidConfiguration;
        configured_dev = dev;
    }
    const cudaError_t e = launch_pdl(k_token_scales, dim3(static_cast<unsigned>(slots), static_cast<unsigned>((ksteps + 7) / 8)),
                                     dim3(256), 0, s, a, reinterpret_cast<uint32_t*>(a.workspace));
    if (e != cudaSuccess) return e;
    const int64_t pairs = tiles < pairs_at_once ? tiles : pairs_at_once;
    return launch_pdl(k_grouped_pair<ODT>, dim3(static_cast<unsigned>(2 * pairs)), dim3(kGpThreads), kGpSmem, s, mapW,
                      mapT, mapW2, mapT2, mapSW, mapST, mapOut, a, static_cast<unsigned>(slots), static_cast<unsigned>(tiles), block_tiles(a, slots));
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

// Whether the call takes pairs of SMs (and a workspace): by a model of both, in us, on the
// tiles to be expected (a half-filled one a group; of a single group what it has).  A wave of
// pairs takes about 2.6 + 0.7 K / 1024 us and the call 10 more (the scales' layout, the first
// tiles' start and the last ones' end), a wave of 128 x 128 tiles, two CTAs an SM, 3.6 + 2 K / 1024
// and 3 more; neither is faster than its bytes at 5.2 and 4.8 TB/s.  The last wave counts half its share
// and half a whole one.  (Outputs are counted at two bytes, fp32 ones
// too: a path needs or needs no workspace by the sizes alone.)  On 28 shapes the choice costs at most 1.3 % of
// the faster path's time, but for one of 256 tokens x [4096, 4096] (11.1 / 12.0); us pairs / single: K 4096, 4
// experts 1024 x 14336 46 / 50, 2 experts 4096 x 4096 38 / 49, 8 experts 8192 x 14336 193 / 296, 16 experts
// 2048 x 4096 44 / 39; K 1024, 4 experts 8192 x 1024 19 / 13.
static bool takes_pairs(const GroupedArgs& a) {
    constexpr double kSms = 152;
    if (a.K <= 0 || a.E <= 0 || a.N <= 128 || a.T < 33 * a.E || a.K / 64 > 8 * 65535) return false;
    const double E = static_cast<double>(a.E), T = static_cast<double>(a.T), N = static_cast<double>(a.N);
    const double k = static_cast<double>(a.K) / 1024;
    const double mb = ((E * N + T) * static_cast<double>(a.K) * 0.5625 + T * N * 2) / 1e6;
    auto waves = [&](int rows, int cols, double at_once) {                   // of tiles of rows tokens x cols
        const double tiles = (a.E == 1 ? ceil(T / rows) : T / rows + 0.5 * E) * ceil(N / cols), w = tiles / at_once;
        return w <= 1 ? 1.0 : 0.5 * (w + ceil(w));
    };
    const double pairs = 10 + fmax(waves(kGpBT, 256, kSms / 2) * (2.6 + 0.7 * k), mb / 5.2);
    const double single = 3 + fmax(waves(128, 128, 2 * kSms) * (3.6 + 2 * k), mb / 4.8);
    return pairs < single;
}

int64_t grouped_workspace(const GroupedArgs& a) {
    return takes_pairs(a) ? pair_slots(a) * (a.K / 64) * 1024 : 0;
}

int launch_grouped_mm(const GroupedArgs& a, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (takes_pairs(a))
        return static_cast<int>(a.out_dtype == NVFP4_F32 ? launch_pair<NVFP4_F32>(a, s) : launch_pair<NVFP4_BF16>(a, s));
    // tokens a tile: about twice the mean group, so that most groups are one tile
    const int64_t mean = (a.T + a.E - 1) / a.E;
    if (mean <= 8) return static_cast<int>(launch_grouped_o<16>(a, s));
    if (mean <= 16) return static_cast<int>(launch_grouped_o<32>(a, s));
    if (mean <= 32) return static_cast<int>(launch_grouped_o<64>(a, s));
    return static_cast<int>(launch_grouped_o<128>(a, s));
}

}  // namespace nvfp4
