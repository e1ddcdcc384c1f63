// nvfp4_attend.cu -- attention of few queries a sequence over a paged NVFP4 cache
// (nvfp4_cache_attention): out = sum_j softmax_j(scale q . k_j) v_j.
//
// The G = Hq / Hkv heads that share a KV head, times a sequence's queries, are the rows
// of a group; every byte of the cache is used once for all of them, 4 D operations a row for
// 9/8 D bytes: with few rows the kernel is bound by memory.  The warp-level MMA takes
// decoded keys and values straight from registers.
//   - A key or value decodes exactly to f16 (q * dec(s): six significant bits).
//   - S^T = K Q^T as m16n8k16 with 16 tokens times 8 rows, so 8 rows fill the product.  The
//     order of a head's elements inside it is free as long as A and B agree: lane (r, c) takes D / 4
//     consecutive elements of tokens r and r + 8, whole 16-element blocks, from its tile.
//   - O^T = V^T P^T as m16n8k16 with 16 elements times 8 rows over 16 tokens.  Its A fragment pairs
//     tokens; two tokens' codes are interleaved four bits at a time before they are decoded.  P^T's
//     8 x 8 blocks are turned from S^T's layout by movmatrix.
//   - Online softmax: weights are made by a reference kBase below a maximum, so that small ones keep
//     their bits in f16; it is raised only when a weight would pass 2^15, which f16 holds, and
//     which a vote finds without exchanging maxima.
// Work is counted in tiles of 16 tokens of a group, over all groups of all sequences, and
// each warp takes an equal run of them, whatever the lengths: a warp finishes the groups that
// lie in its run by itself, those that are cut between the warps of a CTA are joined in shared memory at its
// end, and those cut between CTAs leave partial sums in the workspace, which k_join adds in
// order.  A warp works on pairs of tiles; its own ring of shared memory is filled by bulk copies,
// one or two a pair, that run ahead across groups.
// Measured: 64 sequences of 512 to 32768 keys, 8 KV heads of 128 and 64 query heads (655 MB), 131 us, 5.0 TB/s of the 6.7 of a
// copy; one sequence of 131072 keys (151 MB) 46 us, one of 200 6.4 us.  Bound by issue and latency: a pair of tiles takes some
// 650 instructions of a warp (half of them the decoding: a word of eight codes is 4 conversions), and with the registers for
// 16 warps an SM the slots are 61 % full, the ALUs 55 to 65 %.  Tiles alone instead of pairs took 228 us, divisions to
// find a tile's place 258, masks on every tile 187, runs shared by a CTA's warps 157.
#include <algorithm>

#include "nvfp4_attend.cuh"

namespace nvfp4 {
namespace {

constexpr int kWarps = 8;
constexpr int kMinTiles = 4;                              // a warp's run is not made shorter
static_assert(kGroupCost < kWarps * kMinTiles, "a CTA's run holds some of a group that is cut at its end");

template <int D, int NT>
constexpr int kStages = D == 64 ? 4 : D == 128 && NT == 1 ? 2 : D == 128 ? 4 : 2;      // pairs of tiles a warp's ring holds

// ---- who does what ------------------------------------------------------------------------------
template <int R>
struct Units {
    __device__ __forceinline__ static int64_t share(const AttendArgs& a, int64_t b) { return sequence<R>(a, b).units; }
};

template <int R>
struct Groups {
    __device__ __forceinline__ static int64_t share(const AttendArgs& a, int64_t b) { return sequence<R>(a, b).runs; }
};

// warps that take part
__device__ __forceinline__ int64_t parts_of(int64_t units, int64_t warps) {
    const int64_t most = (units + kMinTiles - 1) / kMinTiles;
    return most < warps ? most : warps;
}

// Where a warp's run starts: unit u, `in` units into a group of sequence b, which has `before` units ahead of it.
struct Start {
    int64_t u, b, before, group;
    Seq s;
    int in;
};

// The run that would start at unit x starts at x's group where x is not past the group's own cost.  Every lane of a
// warp calls it.
template <int R>
__device__ __forceinline__ Start run_start(const AttendArgs& a, const Shares<Units<R>>& shares, int64_t x) {
    Start t;
    shares.find(a, x, &t.b, &t.before);
    t.s = sequence<R>(a, t.b);
    const int64_t per = kGroupCost + t.s.tiles, from = x - t.before;
    t.group = quotient(from, per);
    t.in = static_cast<int>(from - t.group * per);
    if (t.in <= kGroupCost) x -= t.in, t.in = 0;
    t.u = x;
    return t;
}

// A place in a warp's run: a part of a group, tiles ta .. tb of the group's s.tiles.
struct Place {
    int64_t u, end;           // next unit, end of the run
    int64_t b, base;          // sequence of the unit before, units before it
    Seq s;
    int h, rt, ta, tb;        // the group's KV head and row tile
    bool more;                // there was a part

    // at the first part of the run from t to unit u1
    __device__ __forceinline__ void start(const AttendArgs& a, const Start& t, int64_t u1) {
        end = u1, b = t.b, base = t.before, s = t.s, more = t.u < u1;
        const int per = kGroupCost + s.tiles, to = static_cast<int>(min(static_cast<int64_t>(per), t.in + (u1 - t.u)));
        rt = static_cast<int>(quotient(t.group, a.cache.Hkv));
        h = static_cast<int>(t.group - static_cast<int64_t>(rt) * a.cache.Hkv);
        u = t.u + (to - t.in), ta = max(t.in - kGroupCost, 0), tb = to - kGroupCost;
    }

    // the next part; false at the end of the run
    template <int R>
    __device__ __forceinline__ bool next(const AttendArgs& a) {
        if (u >= end) return false;
        if (u < base + s.units) {                         // the sequence's next group
            if (++h == a.cache.Hkv) h = 0, ++rt;
        } else {
            do {
                base += s.units, ++b;
                s = sequence<R>(a, b);
            } while (u >= base + s.units);
            h = rt = 0;
        }
        const int to = static_cast<int>(min(static_cast<int64_t>(kGroupCost + s.tiles), end - u));
        u += to;
        ta = 0, tb = to - kGroupCost;
        return true;
    }
};

// ---- arithmetic ---------------------------------------------------------------------------------
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* x, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}

// an 8 x 8 matrix of 16-bit values, a row's pair a lane, turned
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// what f16 pair h leaves of lo and hi, `times` as large
__device__ __forceinline__ uint32_t rest_f16(uint32_t h, float lo, float hi, float times = 1.0f) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_f16(mul_rn(sub_rn(lo, v.x), times), mul_rn(sub_rn(hi, v.y), times));
}

// What the first f16 leaves of an fp32 query's weight (at most 2^3 of a weight up to 2^15, 2^-25 of one that is smaller than
// f16 holds) is rounded this many times as large, and its product divided by it: half a step is then 2^-36, not the 2^-25 at
// which f16 ends.
constexpr float kRestScale = 2048.0f;

// A part of a cut group, as a warp leaves it: the first part of its run lies in `sums`, the last in its ring.
struct Left {
    int64_t first, row0;      // the group's first unit (-1: none); its sequence's first query
    int n, h, rt, ta, tb, tiles;
};

// Shared memory: rings [kWarps][kStages][2 records], sums [kWarps][8 NT][D + 4], (max, sum)
// [kWarps][2][8 NT][2], barriers [kWarps][kStages], each warp's two places and two parts left.
template <int D, int NT>
struct Shape {
    static constexpr int R = 8 * NT;                      // rows of a group tile
    static constexpr int sum = R * (D + 4) * 4;           // a part's sums
    static constexpr int one = kStages<D, NT> * 2 * kRecord<D>;       // a warp's ring, which holds a part's sums at the end
    static_assert(one >= sum && sum % 128 == 0, "the last part's sums lie in the ring");
    static constexpr int ring = kWarps * one;
    static constexpr int sums = kWarps * sum;
    static constexpr int stats = kWarps * 2 * R * 2 * 4;
    static constexpr int bars = kWarps * kStages<D, NT> * 8;
    static constexpr int bytes = ring + sums + stats + bars + kWarps * 2 * (sizeof(Place) + sizeof(Left));
};

// F32: queries and weights enter the products as two f16 (a weight's second one kRestScale times as large), and a tile's sums
// are added in fp32
template <int D, int NT, bool F32>
__global__ void __launch_bounds__(kWarps * 32, D <= 128 && NT == 1 ? 2 : 1) k_attend(const AttendArgs a, int split) {
    using S = Shape<D, NT>;
    constexpr int R = S::R, kSteps = D / 16, kParts = F32 ? 2 : 1, kStage = kStages<D, NT>;
    constexpr int kUnits = D / 64;                        // 8-element words of V a lane takes per token
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* const ring = smem;
    float* const sums = reinterpret_cast<float*>(smem + S::ring);
    float* const stats = reinterpret_cast<float*>(smem + S::ring + S::sums);
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + S::ring + S::sums + S::stats);
    Place* const all_places = reinterpret_cast<Place*>(bars + kWarps * kStage);
    Left* const lefts = reinterpret_cast<Left*>(all_places + 2 * kWarps);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    if (lane < kStage) mbar_init(bars + warp * kStage + lane);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_trigger();
    pdl_wait();
    Place* const places = all_places + 2 * warp;
    Cut* const cut = split ? cuts<D, R>(a, gridDim.x) + blockIdx.x : nullptr;
    if (split && threadIdx.x == 0) cut->n = 0;
    int64_t units = 0;
    {                                                     // this warp's run
        Start t = {};
        int64_t end = 0;
        if (split) {
            const Shares<Units<R>> shares(a);
            units = shares.total;
            const int64_t warps = parts_of(units, static_cast<int64_t>(gridDim.x) * kWarps);
            const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
            if (i < warps) {
                t = run_start<R>(a, shares, quotient(units * i, warps));
                end = i + 1 < warps ? run_start<R>(a, shares, quotient(units * (i + 1), warps)).u : units;
            }
        } else {                                          // one group a CTA
            bool some;
            if (a.offsets) {
                const Shares<Groups<R>> shares(a);
                some = blockIdx.x < shares.total;
                if (some) {
                    shares.find(a, blockIdx.x, &t.b, &t.before);
                    t.s = sequence<R>(a, t.b);
                    t.group = blockIdx.x - t.before;
                }
            } else {                                      // every sequence has as many
                const uint32_t groups = (a.Hq / a.cache.Hkv + R - 1) / R * a.cache.Hkv;
                t.b = blockIdx.x / groups, t.group = blockIdx.x % groups;
                t.s = sequence<R>(a, t.b);
                some = t.s.n > 0;
            }
            if (some) {
                t.before = 0;
                const int64_t first = t.group * (kGroupCost + t.s.tiles);
                auto at = [&](int w) {                    // the first warp of those without a tile has the group's start
                    const int x = t.s.tiles * w / kWarps;
                    return w == kWarps ? kGroupCost + t.s.tiles : x > 0 ? kGroupCost + x : 0;
                };
                t.in = at(warp), t.u = first + t.in;
                end = first + at(warp + 1);
            }
        }
        if (lane == 0) {
            places[0].start(a, t, end);
            places[1] = places[0];
            lefts[2 * warp].first = lefts[2 * warp + 1].first = -1;
        }
    }
    __syncwarp();

    const int G = a.Hq / a.cache.Hkv, per_page = a.cache.page_size / 16;
    uint8_t* const my_ring = ring + warp * S::one;
    uint64_t* const my_bars = bars + warp * kStage;

    // ---- copies, kStage pairs of tiles ahead: the place of this warp's next pair and its pages.  Pages and tiles of a page
    // are counted along (a division a tile costs as much as decoding it)
    const int skip_pages = 2 / per_page, skip_tiles = 2 % per_page;
    const int64_t page_bytes = static_cast<int64_t>(a.cache.Hkv) * per_page * kRecord<D>;
    auto advance = [&](Place& p) {                        // one lane walks, all read
        __syncwarp();
        if (lane == 0) p.more = p.next<R>(a);
        __syncwarp();
        return p.more;
    };
    Place &ahead = places[0], &at = places[1];
    int ahead_left = 0, ahead_tile = 0;                   // tiles to the end of the part, tile of the page
    const int32_t* ahead_table = nullptr;                 // the page's place in the table
    const uint8_t* ahead_head = nullptr;                  // the head's first byte in page 0
    int32_t page_a = -1, page_b = -1;                     // pages of the two tiles
    uint32_t there = 0;                                   // tiles of stages that have a page, two bits a stage
    auto pages = [&]() {
        page_a = __ldg(ahead_table);
        page_b = ahead_tile + 1 < per_page || ahead_left < 2 ? page_a : __ldg(ahead_table + 1);
    };
    auto begin = [&]() {                                  // at the first pair of a part
        const int tile = ahead.s.t0 + ahead.ta, page = tile / per_page;
        ahead_tile = tile - page * per_page;
        ahead_table = a.pages + ahead.b * a.width + page;
        ahead_head = a.cache.data + static_cast<int64_t>(ahead.h) * per_page * kRecord<D>;
        pages();
    };
    auto seek = [&]() {                                   // to the next part that has a pair
        ahead_left = 0;
        while (advance(ahead)) {
            ahead_left = ahead.tb - ahead.ta;
            if (ahead_left > 0) break;
        }
        if (ahead_left > 0) begin();
    };
    auto issue = [&](int stage) {
        if (ahead_left <= 0) return;
        const bool is_a = page_a >= 0 && page_a < a.cache.pages;
        const bool is_b = ahead_left > 1 && page_b >= 0 && page_b < a.cache.pages;
        there = (there & ~(3u << 2 * stage)) | (is_a ? 1u : 0u) << 2 * stage | (is_b ? 2u : 0u) << 2 * stage;
        if (lane == 0) {
            uint8_t* const dst = my_ring + stage * 2 * kRecord<D>;
            uint64_t* const bar = my_bars + stage;
            const uint8_t* const src = ahead_head + page_a * page_bytes + static_cast<int64_t>(ahead_tile) * kRecord<D>;
            if (is_a && is_b && ahead_tile + 1 < per_page) {      // one piece of memory
                mbar_expect_tx(bar, 2 * kRecord<D>);
                bulk_copy(dst, src, 2 * kRecord<D>, bar);
            } else if (is_a || is_b) {
                mbar_expect_tx(bar, (is_a && is_b ? 2 : 1) * kRecord<D>);
                if (is_a) bulk_copy(dst, src, kRecord<D>, bar);
                if (is_b) bulk_copy(dst + kRecord<D>, ahead_head + page_b * page_bytes, kRecord<D>, bar);
            } else {                                      // no such page: nothing comes
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
            }
        }
        ahead_left -= 2;
        if (ahead_left <= 0) {
            seek();
            return;
        }
        ahead_table += skip_pages;
        ahead_tile += skip_tiles;
        if (ahead_tile >= per_page) ahead_tile -= per_page, ++ahead_table;
        pages();
    };
    bool some = ahead.more;
    if (some) {                                           // the first queries, while the pages and tiles are fetched
        const int row = min(ahead.rt * R + (NT == 1 ? r : lane >> 1), ahead.s.n * G - 1), size = a.dtype == NVFP4_BF16 ? 2 : 4;
        int query, head;
        split_row(ahead.s.n, G, row, &query, &head);
        const uint8_t* const q = static_cast<const uint8_t*>(a.q) + ((ahead.s.row0 + query) * a.q_stride +
                                                                     (static_cast<int64_t>(ahead.h) * G + head) * D) * size;
        for (int i = NT == 1 ? c : lane & 1; i < D * size / 128; i += NT == 1 ? 4 : 2)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(q + i * 128));
    }
    ahead_left = some ? ahead.tb - ahead.ta : 0;
    if (ahead_left > 0) begin();
    else if (some) seek();
    for (int i = 0; i < kStage; ++i) issue(i);

    int stage = 0;
    uint32_t phase = 0;
    bool lost = false;                                    // a wait ran out
    for (; some; some = advance(at)) {
        const int h = at.h, rt = at.rt, n = at.s.n;
        const int nrows = at.s.n * G, len = at.s.len, pos0 = len - at.s.n;
        const int64_t row0 = at.s.row0;

        // ---- queries: fragments, the factor of a row's logits, and the keys a row sees
        uint32_t qf[kParts][NT][kSteps][2];
        float factor[NT][2];
        int lo[NT][2], hi[NT][2];
        int all_lo = 0, all_hi = len;                   // keys that every row sees
        const GScale gk = [&] {
            GScale g{0.0f, 1.0f, 1.0f};
            if (a.cache.k_mode != NVFP4_GAMAX_NONE) {
                g.A = __ldg(a.cache.k_gamax + (a.cache.k_mode == NVFP4_GAMAX_ROW_GIVEN ? h : 0));
                global_scales(g.A, a.cache.bound, g.Senc, g.Sdec);
            }
            return g;
        }();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = min(rt * R + nt * 8 + r, nrows - 1);
            int query, head;
            split_row(n, G, row, &query, &head);
            const int64_t e = (row0 + query) * a.q_stride + (static_cast<int64_t>(h) * G + head) * D + c * (D / 4);
            float x[D / 4];
            if (a.dtype == NVFP4_BF16) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + e) + i);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
                        x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + e) + i);
                    x[4 * i] = u.x, x[4 * i + 1] = u.y, x[4 * i + 2] = u.z, x[4 * i + 3] = u.w;
                }
            }
            // a row scaled to at most 2^15 by a power of two (its exponent at least -112, so that this is a float)
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) top = max_nd(top, fabsf(x[i]));
            top = max_nd(top, __shfl_xor_sync(kFullMask, top, 1));
            top = max_nd(top, __shfl_xor_sync(kFullMask, top, 2));
            const int ex = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -112), 126) - 14;
            const float down = power_of_two(-ex), mine = power_of_two(ex);
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float x0 = mul_rn(x[4 * i + 2 * k], down), x1 = mul_rn(x[4 * i + 2 * k + 1], down);
                    qf[0][nt][i][k] = pack_f16(x0, x1);
                    if (F32) qf[kParts - 1][nt][i][k] = rest_f16(qf[0][nt][i][k], x0, x1);
                }
            // this lane's columns of S^T: rows 2c and 2c + 1
            const float dec = mul_rn(mul_rn(a.scale, kLog2e), gk.Sdec);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                factor[nt][k] = mul_rn(__shfl_sync(kFullMask, mine, (2 * c + k) * 4), dec);
                split_row(n, G, min(rt * R + nt * 8 + 2 * c + k, nrows - 1), &query, &head);
                const int p = pos0 + query;
                hi[nt][k] = a.causal ? min(len, max(p + 1, 0)) : len;
                lo[nt][k] = a.window > 0 ? max(0, p - a.window + 1) : 0;
            }
        }
        int first, last, head;                            // queries of the first and the last row
        split_row(n, G, rt * R, &first, &head);
        split_row(n, G, min(rt * R + R, nrows) - 1, &last, &head);
        if (a.causal) all_hi = min(len, max(pos0 + first + 1, 0));
        if (a.window > 0) all_lo = max(0, pos0 + last - a.window + 1);
        const int seen_lo = a.window > 0 ? max(0, pos0 + first - a.window + 1) : 0;

        float o[NT][kSteps][4], top[NT][2], den[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
            top[nt][0] = top[nt][1] = kLowest;
            den[nt][0] = den[nt][1] = 0.0f;
        }

        int left = at.tb - at.ta, j0 = (at.s.t0 + at.ta) * 16;
        for (; left > 0; left -= 2, j0 += 32) {
            if (!lost) lost = !__all_sync(kFullMask, mbar_wait(my_bars + stage, phase));
            const uint32_t have = there >> 2 * stage & 3u;
            if (have && !lost) {
                const uint8_t* rec = my_ring + stage * 2 * kRecord<D>;
                // S^T: MMA rows r and r + 8 are tokens (r >> 1) + 4 (r & 1) and 8 more, so that rows 2c and 2c + 1
                // (the pairs of the second product) are tokens c and c + 4
                const int tok = (r >> 1) + 4 * (r & 1);
                float sc[2][NT][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) sc[e][nt][0] = sc[e][nt][1] = sc[e][nt][2] = sc[e][nt][3] = 0.0f;
                    uint32_t kw[2][D / 32], ks[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint8_t* p = rec + e * kRecord<D> + (tok + 8 * k) * (D / 2) + c * (D / 8);
                        if constexpr (D == 64) {
                            const uint2 u = *reinterpret_cast<const uint2*>(p);
                            kw[k][0] = u.x, kw[k][1] = u.y;
                        } else {
#pragma unroll
                            for (int i = 0; i < D / 128; ++i) {
                                const uint4 u = reinterpret_cast<const uint4*>(p)[i];
                                kw[k][4 * i] = u.x, kw[k][4 * i + 1] = u.y, kw[k][4 * i + 2] = u.z, kw[k][4 * i + 3] = u.w;
                            }
                        }
                        const uint8_t* q = rec + e * kRecord<D> + 8 * D + (tok + 8 * k) * (D / 16) + c * (D / 64);
                        ks[k] = D == 64 ? *q : D == 128 ? *reinterpret_cast<const uint16_t*>(q) : *reinterpret_cast<const uint32_t*>(q);
                    }
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) {            // blocks of 16 of this lane
                        uint32_t x[2][8];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t u = e4m3_pair(i < 2 ? ks[k] : ks[k] >> 16);
                            const uint32_t sp = __byte_perm(u, u, i & 1 ? 0x3232 : 0x1010);
                            decode4(kw[k][2 * i], sp, x[k]);
                            decode4(kw[k][2 * i + 1], sp, x[k] + 4);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {             // steps of 4 elements a lane
                            const uint32_t f[4] = {x[0][2 * j], x[1][2 * j], x[0][2 * j + 1], x[1][2 * j + 1]};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int p = 0; p < kParts; ++p)
                                    mma_f16(sc[e][nt], f, qf[p][nt][4 * i + j][0], qf[p][nt][4 * i + j][1]);
                        }
                    }
                }
                const bool whole = have == 3u && j0 >= all_lo && j0 + 32 <= all_hi;
                // logits less the reference; that is raised where a weight would pass 2^kMost
                float w[2][NT][4];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[e][nt][k] = __fmaf_rn(sc[e][nt][k], factor[nt][k & 1], -top[nt][k & 1]);
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int j = j0 + 16 * e + tok + 8 * (k >> 1);
                                if (!(have >> e & 1) || j < lo[nt][k & 1] || j >= hi[nt][k & 1]) w[e][nt][k] = kNone;
                            }
                }
                bool high = false;
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k) high |= w[e][nt][k] > kMost;
                if (__any_sync(kFullMask, high)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float m = top[nt][k];
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int i = k; i < 4; i += 2)
                                    if (w[e][nt][i] > kNone)
                                        m = max_nd(m, __fsub_ru(__fmul_ru(sc[e][nt][i], factor[nt][k]), kBase));
                            m = max_nd(m, __shfl_xor_sync(kFullMask, m, 4));
                            m = max_nd(m, __shfl_xor_sync(kFullMask, m, 8));
                            m = max_nd(m, __shfl_xor_sync(kFullMask, m, 16));
                            const float less = exp2_approx(sub_rn(top[nt][k], m));
                            top[nt][k] = m;
                            den[nt][k] = mul_rn(den[nt][k], less);
#pragma unroll
                            for (int i = 0; i < kSteps; ++i) {
                                o[nt][i][k] = mul_rn(o[nt][i][k], less);
                                o[nt][i][k + 2] = mul_rn(o[nt][i][k + 2], less);
                            }
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int i = k; i < 4; i += 2)
                                    if (!(w[e][nt][i] <= kNone)) w[e][nt][i] = __fmaf_rn(sc[e][nt][i], factor[nt][k], -m);
                        }
                }
                uint32_t pf[2][kParts][NT][2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            w[e][nt][k] = exp2_approx(w[e][nt][k]);
                            den[nt][k & 1] = add_rn(den[nt][k & 1], w[e][nt][k]);
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t u = pack_f16(w[e][nt][2 * k], w[e][nt][2 * k + 1]);
                            pf[e][0][nt][k] = turn8x8(u);
                            if (F32) pf[e][kParts - 1][nt][k] = turn8x8(rest_f16(u, w[e][nt][2 * k], w[e][nt][2 * k + 1], kRestScale));
                        }
                    }
                // O^T: this lane's tokens are c, c + 4, c + 8 and c + 12, its words of 8 elements r * kUnits ..
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint8_t* vrec = rec + e * kRecord<D> + 9 * D;
                    uint32_t vw[4][kUnits], vs[4][(kUnits + 1) / 2];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int tk = c + 4 * k;
                        const uint8_t* p = vrec + tk * (D / 2) + r * kUnits * 4;
                        if constexpr (kUnits == 1) {
                            vw[k][0] = *reinterpret_cast<const uint32_t*>(p);
                        } else if constexpr (kUnits == 2) {
                            const uint2 u = *reinterpret_cast<const uint2*>(p);
                            vw[k][0] = u.x, vw[k][1] = u.y;
                        } else {
                            const uint4 u = *reinterpret_cast<const uint4*>(p);
                            vw[k][0] = u.x, vw[k][1] = u.y, vw[k][2] = u.z, vw[k][3] = u.w;
                        }
#pragma unroll
                        for (int i = 0; i < (kUnits + 1) / 2; ++i) vs[k][i] = vrec[8 * D + tk * (D / 16) + r * kUnits / 2 + i];
                    }
                    if (!whole) {                         // what no row sees was perhaps never written
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int i = 0; i < (kUnits + 1) / 2; ++i) {
                                const int j = j0 + 16 * e + c + 4 * k;
                                if (!(have >> e & 1) || j < seen_lo || j >= len) vs[k][i] = 0;
                            }
                    }
#pragma unroll
                    for (int i = 0; i < kUnits; ++i) {
                        // two tokens' codes of one element to a byte (multiplied, not shifted: the ALU has enough to do)
                        const uint32_t s01 = e4m3_pair(vs[1][i / 2] * 256u + vs[0][i / 2]);
                        const uint32_t s23 = e4m3_pair(vs[3][i / 2] * 256u + vs[2][i / 2]);
                        constexpr uint32_t kLow = 0x0F0F0F0Fu;
                        uint32_t even01[4], odd01[4], even23[4], odd23[4];
                        decode4((vw[0][i] & kLow) | ((vw[1][i] * 16u) & ~kLow), s01, even01);
                        decode4(((vw[0][i] >> 4) & kLow) | (vw[1][i] & ~kLow), s01, odd01);
                        decode4((vw[2][i] & kLow) | ((vw[3][i] * 16u) & ~kLow), s23, even23);
                        decode4(((vw[2][i] >> 4) & kLow) | (vw[3][i] & ~kLow), s23, odd23);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t f[4] = {even01[j], odd01[j], even23[j], odd23[j]};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if (F32) {
                                    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f}, rest[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                    mma_f16(part, f, pf[e][0][nt][0], pf[e][0][nt][1]);
                                    mma_f16(rest, f, pf[e][kParts - 1][nt][0], pf[e][kParts - 1][nt][1]);
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        o[nt][4 * i + j][k] = add_rn(o[nt][4 * i + j][k], __fmaf_rn(rest[k], 1.0f / kRestScale, part[k]));
                                } else {
                                    mma_f16(o[nt][4 * i + j], f, pf[e][0][nt][0], pf[e][0][nt][1]);
                                }
                            }
                        }
                    }
                }
            }
            __syncwarp();                                 // the pair is read
            if (!lost) issue(stage);
            if (++stage == kStage) stage = 0, phase ^= 1;
        }

        // ---- the end of the part: a whole group is written, what is cut is left for the CTA's end
        const bool complete = at.ta == 0 && at.tb == at.s.tiles;
        const int place = at.u >= at.end && at.ta == 0 ? 1 : 0;       // the run's last part, which it did not start amid
        __syncwarp();                                     // the last part's sums go into the ring: its copies are in and read
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int q = nt * 8 + 2 * c + k;
                float l = den[nt][k];
                l = add_rn(l, __shfl_xor_sync(kFullMask, l, 4));
                l = add_rn(l, __shfl_xor_sync(kFullMask, l, 8));
                l = add_rn(l, __shfl_xor_sync(kFullMask, l, 16));
                if (lost) l = __int_as_float(0x7FC00000);
                // elements (r kUnits + i) * 8 + 2 j (and + 1) of row q
                if (complete) {
                    const int row = rt * R + q;
                    if (row < nrows) {
                        int query, hd;
                        split_row(n, G, row, &query, &hd);
                        const Finish f(a, h * G + hd, h, top[nt][k], l);
                        const int64_t token = row0 + query;
#pragma unroll
                        for (int i = 0; i < kSteps / 2; ++i) {
                            float v[4] = {o[nt][2 * i][k], o[nt][2 * i][k + 2], o[nt][2 * i + 1][k], o[nt][2 * i + 1][k + 2]};
                            f.store(a, token, h * G + hd, r * kUnits * 8 + 4 * i, v);
                        }
                    }
                } else {
                    float* const st = stats + (2 * warp + place) * R * 2;
                    if (r == 0) st[2 * q] = top[nt][k], st[2 * q + 1] = l;
                    float* const to = place ? reinterpret_cast<float*>(my_ring) : sums + warp * (S::sum / 4);
                    float4* dst = reinterpret_cast<float4*>(to + q * (D + 4) + r * kUnits * 8);
#pragma unroll
                    for (int i = 0; i < kSteps / 2; ++i)
                        dst[i] = make_float4(o[nt][2 * i][k], o[nt][2 * i][k + 2], o[nt][2 * i + 1][k], o[nt][2 * i + 1][k + 2]);
                }
            }
        if (!complete && lane == 0) {
            Left& x = lefts[2 * warp + place];
            x.row0 = row0, x.n = n, x.h = h, x.rt = rt, x.ta = at.ta, x.tb = at.tb, x.tiles = at.s.tiles;
            x.first = at.base + (static_cast<int64_t>(rt) * a.cache.Hkv + h) * (kGroupCost + at.s.tiles);
        }
    }
    if (lost) settle();

    // ---- the parts that this CTA's warps left, joined in their order
    __syncthreads();
    static_assert(2 * kWarps <= 32, "a lane for each part");
    const int64_t mine = lane < 2 * kWarps ? lefts[lane].first : -1;
    const unsigned parts = __ballot_sync(kFullMask, mine >= 0);
    const unsigned below = parts & ((1u << lane) - 1u);
    const int64_t previous = __shfl_sync(kFullMask, mine, below ? 31 - __clz(below) : 0);
    unsigned firsts = __ballot_sync(kFullMask, mine >= 0 && (!below || previous != mine));
    while (firsts) {
        const int i = __ffs(firsts) - 1;
        firsts &= firsts - 1;
        const unsigned group = parts & ~((1u << i) - 1u) & (firsts ? (1u << (__ffs(firsts) - 1)) - 1u : ~0u);      // its parts
        const Left x = lefts[i];
        const int tb = lefts[31 - __clz(group)].tb;
        const bool complete = x.ta == 0 && tb == x.tiles;
        const int rows = min(R, x.n * G - x.rt * R);
        if (threadIdx.x == 0 && x.ta > 0 && !complete) {  // cut at this CTA's start; the first such cut of the group?
            const int64_t warps = parts_of(units, static_cast<int64_t>(gridDim.x) * kWarps);
            const int64_t g1 = x.first + kGroupCost + x.tiles;
            if (quotient(units * (static_cast<int64_t>(blockIdx.x) - 1) * kWarps, warps) <= x.first + kGroupCost)
                *cut = Cut{x.row0, x.n, x.h, x.rt, static_cast<int>(quotient(g1 * warps - 1, units) / kWarps)};
        }
        float* const part = reinterpret_cast<float*>(a.workspace) +
                            (static_cast<int64_t>(blockIdx.x) * 2 + (x.ta > 0 ? 0 : 1)) * kPart<D, R>;
        for (int y = threadIdx.x; y < R * (D / 4); y += kWarps * 32) {
            const int q = y / (D / 4), d = y % (D / 4) * 4;
            if (q >= rows) continue;
            float m = kLowest, l = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < 2 * kWarps; ++k)
                if (group >> k & 1) m = max_nd(m, stats[(k * R + q) * 2]);
#pragma unroll
            for (int k = 0; k < 2 * kWarps; ++k) {
                if (!(group >> k & 1)) continue;
                const float2 st = *reinterpret_cast<const float2*>(stats + (k * R + q) * 2);
                const float f = exp2_approx(sub_rn(st.x, m));
                l = __fmaf_rn(st.y, f, l);
                const float* from = k & 1 ? reinterpret_cast<const float*>(ring + (k >> 1) * S::one) : sums + (k >> 1) * (S::sum / 4);
                const float4 u = *reinterpret_cast<const float4*>(from + q * (D + 4) + d);
                v[0] = __fmaf_rn(u.x, f, v[0]), v[1] = __fmaf_rn(u.y, f, v[1]);
                v[2] = __fmaf_rn(u.z, f, v[2]), v[3] = __fmaf_rn(u.w, f, v[3]);
            }
            if (complete) {
                int query, head;
                split_row(x.n, G, x.rt * R + q, &query, &head);
                Finish(a, x.h * G + head, x.h, m, l).store(a, x.row0 + query, x.h * G + head, d, v);
            } else {
                *reinterpret_cast<float4*>(part + q * D + d) = make_float4(v[0], v[1], v[2], v[3]);
                if (d == 0) part[R * D + 2 * q] = m, part[R * D + 2 * q + 1] = l;
            }
        }
    }
}

// ---- launches -----------------------------------------------------------------------------------
// Row tiles of 16 where the cache is then decoded fewer times for all rows: a tile of 16 takes about 1.6 times as long as one
// of 8 (16 sequences of 8192 keys, 8 KV heads of 128: 16 rows 57 us and 67 in tiles of 8; 24 rows 95 and 94; 8 rows 54
// and 42).  Not for the widest heads or fp32, whose fragments fill the registers.
bool two_tiles(const AttendArgs& a) {
    const int64_t rows = (a.T * (a.Hq / a.cache.Hkv) + a.B - 1) / a.B;      // of a sequence, in the mean
    return a.dtype == NVFP4_BF16 && a.cache.D <= 128 && (rows + 15) / 16 * 8 < (rows + 7) / 8 * 5;
}

// Keys up to which a group is not cut, but has a CTA of its own and no k_join after it: 1020 keys of one sequence 10.3 us,
// cut 11.7, of 32 sequences 13.9 and 20.5; 1200 keys 11.5 and 11.7, 16.0 and 22.5; 1300 keys 12.6 and 11.7 (8 KV heads of 128,
// bf16).  Heads of 512 bytes and more take longer a tile, so that few groups (up to half of the CTAs that run at once with
// heads of 256, an eighth of twice as many with 128) are cut earlier: of fp32 128, 1020 keys of one sequence take 13.4 and 13.4,
// 1060 14.8 and 13.4, of 8 16.4 and 17.6, of 32 21.7 and 26.1; of bf16 256 1020 keys 14.0 and 14.0, 1060 14.6 and 14.1, of
// 16 15.4 and 18.9; of fp32 256 760 keys 16.0 and 16.9, 900 18.4 and 17.0, of 16 19.1 and 23.1.  Not
// where there are more groups than kWaves times the CTAs that run at once: equal runs then keep all busy (8 KV heads of 128: 64
// sequences of 1020 keys 26.5 us uncut, 29.7 cut, 256 of 1024 114 and 82; 1000 of 100 keys 499 and 89).
constexpr int kSmall = 1200, kWaves = 2;

int small_keys(const AttendArgs& a, int64_t runs, int64_t at_once) {
    const int bytes = a.cache.D * (a.dtype == NVFP4_F32 ? 4 : 2);
    if (bytes <= 256 || runs > at_once / (a.cache.D <= 128 ? 8 : 2)) return kSmall;
    return bytes <= 512 ? 1024 : 768;
}

int64_t runs_bound(const AttendArgs& a, int R) {          // groups, at most
    const int64_t G = a.Hq / a.cache.Hkv;
    const int64_t tiles = a.ragged ? a.T * G / R + a.B : a.B * ((G + R - 1) / R);
    return tiles * a.cache.Hkv;
}

// CTAs of k_attend; *split: whether runs may cut groups
int64_t grid_of(const AttendArgs& a, int R, int* split) {
    int64_t cap = a.width * a.cache.page_size;            // keys of a group, at most
    if (a.window > 0) cap = std::min<int64_t>(cap, a.window + (a.ragged ? a.T : 1));
    const int64_t runs = runs_bound(a, R);
    const int64_t at_once = static_cast<int64_t>(sm_count()) * (a.cache.D <= 128 && R == 8 ? 2 : 1);
    *split = cap > small_keys(a, runs, at_once) || runs > kWaves * at_once;
    return *split ? at_once : runs;
}

template <int D, int NT, bool F32>
cudaError_t launch_t(const AttendArgs& a, cudaStream_t s) {
    using S = Shape<D, NT>;
    auto* kernel = k_attend<D, NT, F32>;
    static thread_local int dev_of = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev_of != dev) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::bytes);
        if (e != cudaSuccess) return e;
        dev_of = dev;
    }
    int split;
    const int64_t grid = grid_of(a, S::R, &split);
    cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kWarps * 32), S::bytes, s, a, split);
    if (e == cudaSuccess && split) e = launch_join<D, S::R>(a, static_cast<int>(grid), s);
    return e;
}

template <int D>
cudaError_t launch_d(const AttendArgs& a, cudaStream_t s) {
    if (a.dtype == NVFP4_F32) return launch_t<D, 1, true>(a, s);
    if constexpr (D <= 128)
        if (two_tiles(a)) return launch_t<D, 2, false>(a, s);
    return launch_t<D, 1, false>(a, s);
}

// whether k_attend_many may take a sequence
bool may_have_many(const AttendArgs& a) {
    return a.dtype == NVFP4_BF16 && a.cache.D <= 128 &&
           is_many((a.ragged ? a.T : 1) * (a.Hq / a.cache.Hkv), a.width * a.cache.page_size);
}

}  // namespace

int64_t attend_workspace(const AttendArgs& a) {           // both kernels', one after the other
    const int R = two_tiles(a) ? 16 : 8;
    int split;
    const int64_t grid = grid_of(a, R, &split);
    const int64_t few = split ? grid * (2 * R * (a.cache.D + 2) * 4 + static_cast<int64_t>(sizeof(Cut))) : 0;
    const int64_t many = may_have_many(a) ? attend_many_workspace(a) : 0;
    return few > many ? few : many;
}

int launch_attend(const AttendArgs& given, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    AttendArgs a = given;
    const bool many = may_have_many(a);
    a.take = many ? kTakeFew : kTakeAll;
    cudaError_t e = a.cache.D == 64 ? launch_d<64>(a, s) : a.cache.D == 128 ? launch_d<128>(a, s) : launch_d<256>(a, s);
    if (e == cudaSuccess && many) {
        a.take = kTakeMany;
        e = launch_attend_many(a, s);
    }
    return static_cast<int>(e);
}

}  // namespace nvfp4
