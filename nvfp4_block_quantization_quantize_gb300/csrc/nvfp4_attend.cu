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
//   - Online softmax: a row's maximum is raised only when a weight would pass 2^8 (f16 holds
//     2^15), which a vote finds without exchanging maxima.
// Work is counted in tiles of 16 tokens of a group, over all groups of all sequences, and
// each CTA takes an equal run of them, whatever the lengths: a group that runs across CTAs
// leaves its partial sums in the workspace, and k_join adds them in order.  A warp takes
// every kWarps-th pair of tiles of its CTA's run; its own ring of shared memory is filled by bulk
// copies, one or two a pair, that run ahead across groups.
#include "nvfp4_block.cuh"
#include "nvfp4_tensor.cuh"

namespace nvfp4 {
namespace {

constexpr int kWarps = 8;
constexpr int kMinTiles = 2 * kWarps;                     // tiles below which a CTA's run is not cut further
constexpr float kLowest = -3.4028234663852886e38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNone = -__builtin_huge_valf();          // a masked logit
constexpr float kSlack = 8.0f;                            // a weight may reach 2^8 before the maximum is raised

template <int D>
constexpr int kRecord = 18 * D;                           // bytes of a tile
template <int D, int NT>
constexpr int kStages = D == 64 ? 4 : D == 128 && NT == 1 ? 2 : D == 128 ? 4 : 2;      // pairs of tiles a warp's ring holds

// ---- who does what ------------------------------------------------------------------------------
// A sequence's share of the work.
struct Seq {
    int64_t row0;             // its first query
    int n, len;               // queries, keys
    int t0, tiles;            // tiles of 16 keys that some query sees
    int runs;                 // row tiles times KV heads: groups
    int64_t units;            // runs * max(tiles, 1): a group that sees nothing is a unit too
};

template <int R>
__device__ __forceinline__ Seq sequence(const AttendArgs& a, int64_t b) {
    Seq s;
    int64_t end;
    if (a.offsets) {
        s.row0 = min(max(__ldg(a.offsets + b), int64_t{0}), a.T);
        end = min(max(__ldg(a.offsets + b + 1), int64_t{0}), a.T);
    } else {
        s.row0 = b;
        end = b + 1;
    }
    s.n = end > s.row0 ? static_cast<int>(end - s.row0) : 0;
    const int64_t cap = a.width * a.cache.page_size;
    s.len = static_cast<int>(min(max(__ldg(a.lengths + b), int64_t{0}), cap));
    const int first = a.window > 0 ? max(0, s.len - s.n + 1 - a.window) : 0;
    s.t0 = first / 16;
    s.tiles = max(0, (s.len + 15) / 16 - s.t0);
    const int G = a.Hq / a.cache.Hkv;
    const int64_t rows = static_cast<int64_t>(s.n) * G;
    s.runs = static_cast<int>((rows + R - 1) / R) * a.cache.Hkv;
    s.units = static_cast<int64_t>(s.runs) * max(s.tiles, 1);
    return s;
}

// Sum of all sequences' units, and the sequence that unit x lies in with the units before it; GROUPS: with a group
// for a unit.  Every lane of a warp calls them.
template <int R>
__device__ __forceinline__ int64_t total_units(const AttendArgs& a) {
    const int lane = threadIdx.x & 31;
    int64_t sum = 0;
    for (int64_t b = lane; b < a.B; b += 32) sum += sequence<R>(a, b).units;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
    return sum;
}

template <int R, bool GROUPS>
__device__ __forceinline__ bool find_unit(const AttendArgs& a, int64_t x, int64_t* seq, int64_t* before) {
    const int lane = threadIdx.x & 31;
    int64_t base = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += 32) {
        const int64_t b = b0 + lane;
        int64_t u = 0;
        if (b < a.B) {
            const Seq q = sequence<R>(a, b);
            u = GROUPS ? q.runs : q.units;
        }
        int64_t s = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(kFullMask, s, o);
            if (lane >= o) s += v;
        }
        const unsigned has = __ballot_sync(kFullMask, base + s > x);
        if (has) {
            const int l = __ffs(has) - 1;
            *seq = b0 + l;
            *before = base + __shfl_sync(kFullMask, s - u, l);
            return true;
        }
        base += __shfl_sync(kFullMask, s, 31);
    }
    return false;
}

// CTAs that take part, and the first unit of CTA i
__device__ __forceinline__ int64_t parts_of(int64_t units, int64_t ctas) {
    const int64_t most = (units + kMinTiles - 1) / kMinTiles;
    return most < ctas ? most : ctas;
}

// A place in a CTA's run: a part [ta, tb) of a group's tiles.
struct Place {
    int64_t u, end;           // next unit, end of the run
    int64_t b, base;          // sequence of the unit before, units before it
    Seq s;
    int group, ta, tb;        // of the current part: tiles ta .. tb of the group's s.tiles
    bool known;               // s belongs to b
    bool more;                // there was a part

    __device__ __forceinline__ void start(int64_t u0, int64_t u1, int64_t b0, int64_t before) {
        u = u0, end = u1, b = b0, base = before, known = false;
    }

    // the next part; false at the end of the run
    template <int R>
    __device__ __forceinline__ bool next(const AttendArgs& a) {
        if (u >= end) return false;
        while (true) {
            if (!known) s = sequence<R>(a, b);
            known = true;
            if (u < base + s.units) break;
            base += s.units;
            ++b;
            known = false;
        }
        const int per = max(s.tiles, 1);
        const int64_t x = u - base;
        group = static_cast<int>(x / per);
        ta = static_cast<int>(x - static_cast<int64_t>(group) * per);
        tb = static_cast<int>(min(static_cast<int64_t>(per), ta + (end - u)));
        u += tb - ta;
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

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t e4m3_pair(uint32_t bytes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(bytes)));
    return h;
}

// a word's four code bytes as f16 pairs times the pair s
__device__ __forceinline__ void decode4(uint32_t w, uint32_t s, uint32_t* h) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = mul_f16x2(h[i], s);
}

// an 8 x 8 matrix of 16-bit values, a row's pair a lane, turned
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ float exp2_approx(float x) {   // 2 ulp
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// what f16 pair h leaves of lo and hi
__device__ __forceinline__ uint32_t rest_f16(uint32_t h, float lo, float hi) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_f16(sub_rn(lo, v.x), sub_rn(hi, v.y));
}

__device__ __forceinline__ float power_of_two(int e) {    // e in [-126, 127]
    return __int_as_float((e + 127) << 23);
}

// 4 elements of a row from its sums v, its maximum m (of logits times log2 e) and denominator l
__device__ __forceinline__ void finish_row(const AttendArgs& a, int64_t token, int head, int h, int d, float m, float l,
                                           float* v) {
    if (a.sinks) {
        const float sink = mul_rn(__ldg(a.sinks + head), kLog2e), top = max_nd(m, sink), f = exp2_approx(sub_rn(m, top));
        l = __fmaf_rn(l, f, exp2_approx(sub_rn(sink, top)));
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = mul_rn(v[k], f);
        m = top;
    }
    float enc, dec = 1.0f;
    if (a.cache.v_mode != NVFP4_GAMAX_NONE)
        global_scales(__ldg(a.cache.v_gamax + (a.cache.v_mode == NVFP4_GAMAX_ROW_GIVEN ? h : 0)), a.cache.bound, enc, dec);
    const float by = l == 0.0f ? 0.0f : div_rn(dec, l);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = mul_rn(v[k], by);
    const int64_t at = (token * a.Hq + head) * a.cache.D + d;
    if (a.out_dtype == NVFP4_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v[0], v[1]), y = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
    if (a.lse && d == 0)
        a.lse[token * a.Hq + head] = l == 0.0f ? __int_as_float(0xFF800000) : mul_rn(add_rn(m, log2f(l)), kLn2);
}

// Shared memory: rings [kWarps][kStages][2 records], sums [kWarps][8 NT][D + 4], (max, sum)
// [kWarps][8 NT][2], barriers [kWarps][kStages], the run found, each warp's two places.
template <int D, int NT>
struct Shape {
    static constexpr int R = 8 * NT;                      // rows of a group tile
    static constexpr int ring = kWarps * kStages<D, NT> * 2 * kRecord<D>;
    static constexpr int sums = kWarps * R * (D + 4) * 4;
    static constexpr int stats = kWarps * R * 2 * 4;
    static constexpr int bytes = ring + sums + stats + kWarps * kStages<D, NT> * 8 + 32 + kWarps * 2 * sizeof(Place);
};

// a partial result of a CTA: R rows of D sums, then R pairs (maximum, denominator)
template <int D, int NT>
constexpr int64_t kPart = 8 * NT * (D + 2);

// F32: queries and weights enter the products as two f16, and a tile's sums are added in fp32
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
    int64_t* const found = reinterpret_cast<int64_t*>(bars + kWarps * kStage);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    if (threadIdx.x < kWarps * kStage) mbar_init(bars + threadIdx.x);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_trigger();
    pdl_wait();
    if (warp == 0) {                                      // this CTA's run of units: [u0, u1), `before` ahead of sequence b
        int64_t u0 = 0, u1 = 0, b = 0, before = 0;
        if (split) {
            const int64_t units = total_units<R>(a), ctas = parts_of(units, gridDim.x), i = blockIdx.x;
            if (i < ctas) {
                u0 = units * i / ctas, u1 = units * (i + 1) / ctas;
                find_unit<R, false>(a, u0, &b, &before);
            }
        } else if (find_unit<R, true>(a, blockIdx.x, &b, &before)) {      // one group
            const int per = max(sequence<R>(a, b).tiles, 1);
            u0 = (blockIdx.x - before) * per, u1 = u0 + per, before = 0;
        }
        if (lane == 0) found[0] = u0, found[1] = u1, found[2] = b, found[3] = before;
    }
    __syncthreads();
    const int64_t u0 = found[0], u1 = found[1];
    if (u0 >= u1) return;

    const int G = a.Hq / a.cache.Hkv, per_page = a.cache.page_size / 16;
    uint8_t* const my_ring = ring + warp * kStage * 2 * kRecord<D>;
    uint64_t* const my_bars = bars + warp * kStage;
    Place* const places = reinterpret_cast<Place*>(found + 4) + 2 * warp;

    // ---- copies, kStage pairs of tiles ahead: the place of this warp's next pair and its pages.  Pages and tiles of a page
    // are counted along (a division a tile costs as much as decoding it)
    const int skip_pages = 2 * kWarps / per_page, skip_tiles = 2 * kWarps % per_page;
    const int64_t page_bytes = static_cast<int64_t>(a.cache.Hkv) * per_page * kRecord<D>;
    if (lane < 2) places[lane].start(u0, u1, found[2], found[3]);
    auto advance = [&](Place& p) {                        // one lane walks, all read
        __syncwarp();
        if (lane == 0) p.more = p.next<R>(a);
        __syncwarp();
        return p.more;
    };
    Place& ahead = places[0];
    int ahead_left = 0, ahead_tile = 0;                   // tiles to the end of the part, tile of the page
    const int32_t* ahead_table = nullptr;                 // the page's place in the table
    const uint8_t* ahead_head = nullptr;                  // the head's first byte in page 0
    int32_t page_a = -1, page_b = -1;                     // pages of the two tiles
    uint32_t there = 0;                                   // tiles of stages that have a page, two bits a stage
    auto pages = [&]() {
        page_a = __ldg(ahead_table);
        page_b = ahead_tile + 1 < per_page || ahead_left < 2 ? page_a : __ldg(ahead_table + 1);
    };
    auto seek = [&]() {                                   // to the first pair of this warp in the next part that has one
        ahead_left = 0;
        while (advance(ahead)) {
            ahead_left = ahead.s.tiles > 0 ? ahead.tb - ahead.ta - 2 * warp : 0;
            if (ahead_left > 0) break;
        }
        if (ahead_left <= 0) return;
        const int tile = ahead.s.t0 + ahead.ta + 2 * warp, page = tile / per_page;
        ahead_tile = tile - page * per_page;
        ahead_table = a.pages + ahead.b * a.width + page;
        ahead_head = a.cache.data + static_cast<int64_t>(ahead.group % a.cache.Hkv) * per_page * kRecord<D>;
        pages();
    };
    auto issue = [&](int stage) {
        if (ahead_left <= 0) return;
        const bool is_a = page_a >= 0 && page_a < a.cache.pages;
        const bool is_b = ahead_left > 1 && page_b >= 0 && page_b < a.cache.pages;
        there = (there & ~(3u << 2 * stage)) | (is_a ? 1u : 0u) << 2 * stage | (is_b ? 2u : 0u) << 2 * stage;
        if (lane == 0) {
            uint8_t* const dst = my_ring + stage * 2 * kRecord<D>;
            uint64_t* const bar = my_bars + stage;
            const uint8_t* const src = ahead_head + page_a * page_bytes + ahead_tile * kRecord<D>;
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
        ahead_left -= 2 * kWarps;
        if (ahead_left <= 0) {
            seek();
            return;
        }
        ahead_table += skip_pages;
        ahead_tile += skip_tiles;
        if (ahead_tile >= per_page) ahead_tile -= per_page, ++ahead_table;
        pages();
    };
    seek();
    for (int i = 0; i < kStage; ++i) issue(i);

    int stage = 0;
    uint32_t phase = 0;
    bool lost = false;                                    // a wait ran out
    Place& at = places[1];
    while (advance(at)) {
        const int h = at.group % a.cache.Hkv, rt = at.group / a.cache.Hkv;
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
            const int64_t e = (row0 + row / G) * a.q_stride + (static_cast<int64_t>(h) * G + row % G) * D + c * (D / 4);
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
                const int qrow = min(rt * R + nt * 8 + 2 * c + k, nrows - 1), p = pos0 + qrow / G;
                hi[nt][k] = a.causal ? min(len, max(p + 1, 0)) : len;
                lo[nt][k] = a.window > 0 ? max(0, p - a.window + 1) : 0;
            }
        }
        {
            const int first = rt * R / G, last = min(rt * R + R, nrows) - 1;
            if (a.causal) all_hi = min(len, max(pos0 + first + 1, 0));
            if (a.window > 0) all_lo = max(0, pos0 + last / G - a.window + 1);
        }
        const int seen_lo = a.window > 0 ? max(0, pos0 + rt * R / G - a.window + 1) : 0;

        float o[NT][kSteps][4], top[NT][2], den[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
            top[nt][0] = top[nt][1] = kLowest;
            den[nt][0] = den[nt][1] = 0.0f;
        }

        int left = at.s.tiles > 0 ? at.tb - at.ta - 2 * warp : 0, j0 = (at.s.t0 + at.ta + 2 * warp) * 16;
        for (; left > 0; left -= 2 * kWarps, j0 += 2 * kWarps * 16) {
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
                // logits less the maximum; that is raised where a weight would pass 2^kSlack
                float w[2][NT][4];
                bool high = false;
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            w[e][nt][k] = __fmaf_rn(sc[e][nt][k], factor[nt][k & 1], -top[nt][k & 1]);
                            if (!whole) {
                                const int j = j0 + 16 * e + tok + 8 * (k >> 1);
                                if (!(have >> e & 1) || j < lo[nt][k & 1] || j >= hi[nt][k & 1]) w[e][nt][k] = kNone;
                            }
                            high |= w[e][nt][k] > kSlack;
                        }
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
                                    if (w[e][nt][i] > kNone) m = max_nd(m, mul_rn(sc[e][nt][i], factor[nt][k]));
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
                            if (F32) pf[e][kParts - 1][nt][k] = turn8x8(rest_f16(u, w[e][nt][2 * k], w[e][nt][2 * k + 1]));
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
                        for (int i = 0; i < (kUnits + 1) / 2; ++i) {
                            vs[k][i] = vrec[8 * D + tk * (D / 16) + r * kUnits / 2 + i];
                            // what no row sees was perhaps never written
                            const int j = j0 + 16 * e + tk;
                            if (!whole && (!(have >> e & 1) || j < seen_lo || j >= len)) vs[k][i] = 0;
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
                                    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                                    for (int p = kParts - 1; p >= 0; --p) mma_f16(part, f, pf[e][p][nt][0], pf[e][p][nt][1]);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) o[nt][4 * i + j][k] = add_rn(o[nt][4 * i + j][k], part[k]);
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

        // ---- the warps' sums of this part, joined in the order of the warps
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
                if (r == 0) {
                    stats[(warp * R + q) * 2] = top[nt][k];
                    stats[(warp * R + q) * 2 + 1] = l;
                }
                // elements (r kUnits + i) * 8 + 2 j (and + 1) of row q
                float4* dst = reinterpret_cast<float4*>(sums + (warp * R + q) * (D + 4) + r * kUnits * 8);
#pragma unroll
                for (int i = 0; i < kSteps / 2; ++i)
                    dst[i] = make_float4(o[nt][2 * i][k], o[nt][2 * i][k + 2], o[nt][2 * i + 1][k], o[nt][2 * i + 1][k + 2]);
            }
        __syncthreads();
        const int used = at.s.tiles > 0 ? min(kWarps, (at.tb - at.ta + 1) / 2) : 0;
        const bool complete = at.ta == 0 && at.tb == max(at.s.tiles, 1);
        const int rows = min(R, nrows - rt * R);
        float* const part = reinterpret_cast<float*>(a.workspace) +
                            (static_cast<int64_t>(blockIdx.x) * 2 + (at.ta > 0 ? 0 : 1)) * kPart<D, NT>;
        for (int x = threadIdx.x; x < R * (D / 4); x += kWarps * 32) {
            const int q = x / (D / 4), d = x % (D / 4) * 4;
            if (q >= rows) continue;
            float m = kLowest, l = 0.0f;
            for (int w = 0; w < used; ++w) m = max_nd(m, stats[(w * R + q) * 2]);
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int w = 0; w < used; ++w) {
                const float f = exp2_approx(sub_rn(stats[(w * R + q) * 2], m));
                l = __fmaf_rn(stats[(w * R + q) * 2 + 1], f, l);
                const float4 u = *reinterpret_cast<const float4*>(sums + (w * R + q) * (D + 4) + d);
                v[0] = __fmaf_rn(u.x, f, v[0]), v[1] = __fmaf_rn(u.y, f, v[1]);
                v[2] = __fmaf_rn(u.z, f, v[2]), v[3] = __fmaf_rn(u.w, f, v[3]);
            }
            if (complete) {
                const int row = rt * R + q;
                finish_row(a, row0 + row / G, h * G + row % G, h, d, m, l, v);
            } else {
                *reinterpret_cast<float4*>(part + q * D + d) = make_float4(v[0], v[1], v[2], v[3]);
                if (d == 0) part[R * D + 2 * q] = m, part[R * D + 2 * q + 1] = l;
            }
        }
        __syncthreads();
    }
    if (lost) settle();
}

// A group that several CTAs took parts of, joined in their order: CTA i joins it if the i-th run is the second
// that holds some of it.
template <int D, int NT>
__global__ void __launch_bounds__(256) k_join(const AttendArgs a, int ctas_max) {
    constexpr int R = 8 * NT;
    __shared__ int64_t found[3];
    pdl_trigger();
    pdl_wait();
    if (threadIdx.x < 32) {
        const int64_t units = total_units<R>(a), ctas = parts_of(units, ctas_max), i = blockIdx.x + 1;
        int64_t b = 0, before = 0;
        if (i < ctas) find_unit<R, false>(a, units * i / ctas, &b, &before);
        if (threadIdx.x == 0) found[0] = i < ctas ? units : 0, found[1] = b, found[2] = before;
    }
    __syncthreads();
    const int64_t units = found[0];
    if (units == 0) return;
    const int64_t ctas = parts_of(units, ctas_max), i = blockIdx.x + 1;
    const int64_t x = units * i / ctas;                   // where run i starts
    const Seq s = sequence<R>(a, found[1]);
    const int per = max(s.tiles, 1);
    const int group = static_cast<int>((x - found[2]) / per);
    const int64_t g0 = found[2] + static_cast<int64_t>(group) * per, g1 = g0 + per;
    if (x == g0 || units * (i - 1) / ctas > g0) return;   // not cut here, or joined by an earlier CTA
    const int64_t last = (g1 * ctas - 1) / units;         // the run that holds unit g1 - 1
    const int G = a.Hq / a.cache.Hkv, h = group % a.cache.Hkv, rt = group / a.cache.Hkv;
    const int rows = min(R, s.n * G - rt * R);
    // run i - 1 has the group's first tiles as its last part, the others as their first
    const float* ws = reinterpret_cast<const float*>(a.workspace);
    auto part = [&](int64_t run) { return ws + (run * 2 + (run == i - 1 ? 1 : 0)) * kPart<D, NT>; };
    for (int y = threadIdx.x; y < R * (D / 4); y += 256) {
        const int q = y / (D / 4), d = y % (D / 4) * 4;
        if (q >= rows) continue;
        float m = kLowest, l = 0.0f;
#pragma unroll 16
        for (int64_t run = i - 1; run <= last; ++run) m = max_nd(m, part(run)[R * D + 2 * q]);
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (int64_t run = i - 1; run <= last; ++run) {
            const float* p = part(run);
            const float2 st = *reinterpret_cast<const float2*>(p + R * D + 2 * q);
            const float f = exp2_approx(sub_rn(st.x, m));
            l = __fmaf_rn(st.y, f, l);
            const float4 u = *reinterpret_cast<const float4*>(p + q * D + d);
            v[0] = __fmaf_rn(u.x, f, v[0]), v[1] = __fmaf_rn(u.y, f, v[1]);
            v[2] = __fmaf_rn(u.z, f, v[2]), v[3] = __fmaf_rn(u.w, f, v[3]);
        }
        const int row = rt * R + q;
        finish_row(a, s.row0 + row / G, h * G + row % G, h, d, m, l, v);
    }
}

// ---- launches -----------------------------------------------------------------------------------
// Row tiles of 16 where groups of 8 rows would be read more than once (the cache is then decoded
// once for both), but not for the widest heads or fp32, whose fragments fill the registers.
bool two_tiles(const AttendArgs& a) {
    const int64_t rows = (a.T * (a.Hq / a.cache.Hkv) + a.B - 1) / a.B;      // of a sequence, in the mean
    return a.dtype == NVFP4_BF16 && a.cache.D <= 128 && rows > 8;
}

constexpr int kSmall = 512;                               // keys up to which a group is not cut

int64_t runs_bound(const AttendArgs& a, int R) {          // groups, at most
    const int64_t G = a.Hq / a.cache.Hkv;
    const int64_t tiles = a.offsets ? a.T * G / R + a.B : a.B * ((G + R - 1) / R);
    return tiles * a.cache.Hkv;
}

// CTAs of k_attend; *split: whether runs may cut groups
int64_t grid_of(const AttendArgs& a, int R, int* split) {
    const int64_t cap = a.width * a.cache.page_size;
    const int64_t runs = runs_bound(a, R);
    *split = cap > kSmall || runs > (int64_t{1} << 20);
    return *split ? static_cast<int64_t>(sm_count()) * 2 : runs;
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
    if (e == cudaSuccess && split && grid > 1)
        e = launch_pdl(k_join<D, NT>, dim3(static_cast<unsigned>(grid - 1)), dim3(256), 0, s, a, static_cast<int>(grid));
    return e;
}

template <int D>
cudaError_t launch_d(const AttendArgs& a, cudaStream_t s) {
    if (a.dtype == NVFP4_F32) return launch_t<D, 1, true>(a, s);
    if constexpr (D <= 128)
        if (two_tiles(a)) return launch_t<D, 2, false>(a, s);
    return launch_t<D, 1, false>(a, s);
}

}  // namespace

int64_t attend_workspace(const AttendArgs& a) {
    const int R = two_tiles(a) ? 16 : 8;
    int split;
    const int64_t grid = grid_of(a, R, &split);
    return split ? grid * 2 * R * (a.cache.D + 2) * 4 : 0;
}

int launch_attend(const AttendArgs& a, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return static_cast<int>(a.cache.D == 64 ? launch_d<64>(a, s) : a.cache.D == 128 ? launch_d<128>(a, s) : launch_d<256>(a, s));
}

}  // namespace nvfp4
