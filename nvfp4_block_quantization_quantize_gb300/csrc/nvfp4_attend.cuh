// nvfp4_attend.cuh -- what the kernels of nvfp4_cache_attention share: sequences and the
// work they make, decoding of codes, the end of an output row.
#pragma once

#include "nvfp4_block.cuh"
#include "nvfp4_tensor.cuh"

namespace nvfp4 {
namespace {

constexpr float kLowest = -3.4028234663852886e38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNone = -__builtin_huge_valf();          // a masked logit
// k_attend's weights are 2^(a logit - the row's reference), which stands kBase below the largest logit when it is set and is
// raised before a weight passes 2^kMost (f16 holds it).  From 2^-14 down f16 has a fixed step of 2^-24: 2^-35 of the largest
// weight.  64 ragged sequences take 129.7 us with a base of 0 or 7, 130.4 with 11, 131.6 with 13 (raised more often).
constexpr float kBase = 11.0f, kMost = 15.0f;
// What a group costs besides its tiles (its queries, its end), in tiles: the first units of every group.  A run is not
// cut inside them.  64 ragged sequences took 138 us with 2, 133 with 6 and with 12, 135 with 20.
constexpr int kGroupCost = 8;

template <int D>
constexpr int kRecord = 18 * D;                           // bytes of a tile

// ---- who does what ------------------------------------------------------------------------------
// Sequences that the tensor-memory kernel (k_attend_many) takes: of 48 rows and more (8 sequences of 8192 keys, 8 KV heads of
// 128, the other kernel's launch with each: 48 rows 74 us there and 86 by the warp-level kernel, 32 rows 74 and 65, 96 rows 75
// and 144), unless they are so short that its start costs more than its rate gains (600 keys, 4 KV heads, 64 rows: 38 us
// there and 20).
constexpr int kManyRows = 48;
constexpr int64_t kManyWork = int64_t{1} << 18;           // rows times keys

enum Take { kTakeAll, kTakeFew, kTakeMany };

__host__ __device__ __forceinline__ bool is_many(int64_t rows, int64_t keys) { return rows >= kManyRows && rows * keys >= kManyWork; }

// A sequence's share of the work.
struct Seq {
    int64_t row0;             // its first query
    int n, len;               // queries, keys
    int t0, tiles;            // tiles of 16 keys that some query sees
    int runs;                 // row tiles times KV heads: groups
    int64_t units;            // runs * (kGroupCost + tiles)
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
    if (a.take != kTakeAll && is_many(rows, s.len) != (a.take == kTakeMany)) s.n = 0;      // the other kernel's
    s.runs = s.n ? static_cast<int>((rows + R - 1) / R) * a.cache.Hkv : 0;
    s.units = static_cast<int64_t>(s.runs) * (kGroupCost + s.tiles);
    return s;
}

// x / y of values that mostly fit in 32 bits (the 64-bit division costs a third of a microsecond)
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    if ((x | y) >> 32 == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return x / y;
}

__device__ __forceinline__ int64_t scan_add(int64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(kFullMask, v, o);
        if ((threadIdx.x & 31) >= o) v += u;
    }
    return v;
}

// The sequences' shares of the work, F::share(a, b), added up.  A warp holds it: each lane the sequences lane, lane + 32, ..;
// the first 32 stay in registers.
template <class F>
struct Shares {
    int64_t first, upto;      // this lane's first sequence's share; that of the first sequences up to it
    int64_t total;

    __device__ __forceinline__ static int64_t share(const AttendArgs& a, int64_t b) { return b < a.B ? F::share(a, b) : 0; }

    __device__ __forceinline__ explicit Shares(const AttendArgs& a) {
        const int lane = threadIdx.x & 31;
        first = share(a, lane);
        upto = scan_add(first);
        total = __shfl_sync(kFullMask, upto, 31);
        if (a.B > 32) {
            int64_t sum = 0;
            for (int64_t b = lane + 32; b < a.B; b += 32) sum += share(a, b);
            total += __shfl_sync(kFullMask, scan_add(sum), 31);
        }
    }

    // the sequence that unit x < total lies in, and the units before it
    __device__ __forceinline__ void find(const AttendArgs& a, int64_t x, int64_t* seq, int64_t* before) const {
        int64_t base = 0, own = first, s = upto;
        for (int64_t b0 = 0;; b0 += 32) {
            const unsigned has = __ballot_sync(kFullMask, base + s > x);
            if (has || b0 + 32 >= a.B) {
                const int l = has ? __ffs(has) - 1 : 0;
                *seq = b0 + l;
                *before = base + __shfl_sync(kFullMask, s - own, l);
                return;
            }
            base += __shfl_sync(kFullMask, s, 31);
            own = share(a, b0 + 32 + (threadIdx.x & 31));
            s = scan_add(own);
        }
    }
};

// the query and the head of a row of a sequence's KV head
__device__ __forceinline__ void split_row(int n, int G, int row, int* query, int* head) {
    *query = n == 1 ? 0 : row / G;
    *head = row - *query * G;
}

// ---- arithmetic ---------------------------------------------------------------------------------
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

__device__ __forceinline__ float exp2_approx(float x) {   // 2 ulp
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float power_of_two(int e) {    // e in [-126, 127]
    return __int_as_float((e + 127) << 23);
}

// A row's end: its sums times `by` are its output; m its maximum (of logits times log2 e), l its denominator.
struct Finish {
    float by, lse;

    __device__ __forceinline__ Finish(const AttendArgs& a, int head, int h, float m, float l) {
        float enc, dec = 1.0f, f = 1.0f;
        if (a.sinks) {
            const float sink = mul_rn(__ldg(a.sinks + head), kLog2e), top = max_nd(m, sink);
            f = exp2_approx(sub_rn(m, top));
            l = __fmaf_rn(l, f, exp2_approx(sub_rn(sink, top)));
            m = top;
        }
        if (a.cache.v_mode != NVFP4_GAMAX_NONE)
            global_scales(__ldg(a.cache.v_gamax + (a.cache.v_mode == NVFP4_GAMAX_ROW_GIVEN ? h : 0)), a.cache.bound, enc, dec);
        by = l == 0.0f ? 0.0f : mul_rn(f, div_rn(dec, l));
        lse = 0.0f;
        if (a.lse) lse = l == 0.0f ? __int_as_float(0xFF800000) : mul_rn(add_rn(m, log2f(l)), kLn2);
    }

    // 4 elements from element d
    __device__ __forceinline__ void store(const AttendArgs& a, int64_t token, int head, int d, float* v) const {
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
        if (a.lse && d == 0) a.lse[token * a.Hq + head] = lse;
    }
};

// What k_join is to do for a CTA: the group that its run starts amid, if the CTA before has its first
// tiles, which the CTAs up to `last` took parts of.
struct Cut {
    int64_t row0;             // the sequence's first query
    int n, h, rt, last;       // its queries (0: nothing to do); the group's KV head and row tile
};

// a partial result of a CTA: R rows of D sums, then R pairs (maximum, denominator)
template <int D, int R>
constexpr int64_t kPart = R * (D + 2);

// the workspace: two partial results a CTA, then a Cut each
template <int D, int R>
__device__ __forceinline__ Cut* cuts(const AttendArgs& a, int64_t ctas) {
    return reinterpret_cast<Cut*>(reinterpret_cast<float*>(a.workspace) + ctas * 2 * kPart<D, R>);
}

// A group that several CTAs took parts of, joined: 8 rows a CTA, kSub warps a row, each of which adds every kSub-th part in
// their order; the first then adds the warps' sums in theirs.  Bound by latency: a long sequence alone makes 38 parts a
// group, which four warps read in three turns (one warp a row took 10 us of a 47 us call); with 256 rows a group
// most CTAs have nothing to do, and small ones end sooner.  Of 131072 keys' 45 us it takes 9, elsewhere 3 to 4.
template <int R>
constexpr int kSub = R <= 16 ? 4 : 1;

template <int D, int R>
__global__ void __launch_bounds__(256 * kSub<R>) k_join(const AttendArgs a, int ctas) {
    constexpr int S = kSub<R>, kCols = (D + 127) / 128, kBatch = S > 1 ? 4 : 2;      // float4 columns a lane; parts loaded together
    constexpr int kStep = D < 128 ? D / 4 : 32;           // lanes that have columns
    __shared__ float sums[S > 1 ? 8 * S : 1][S > 1 ? D + 2 : 1];
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % S;
    const Cut cut = cuts<D, R>(a, ctas)[i];
    if (cut.n == 0) return;
    const int G = a.Hq / a.cache.Hkv, rows = min(R, cut.n * G - cut.rt * R), runs = cut.last - i + 2;
    const int q = blockIdx.y * 8 + warp / S;
    if (S == 1 && q >= rows) return;
    // CTA i - 1 has the group's first tiles as its last part, the others as their first
    const float* const ws = reinterpret_cast<const float*>(a.workspace);
    auto part = [&](int run) { return ws + (static_cast<int64_t>(i - 1 + run) * 2 + (run == 0 ? 1 : 0)) * kPart<D, R>; };
    float m = kLowest, l = 0.0f, v[kCols][4] = {};
    auto add = [&](float pm, float pl, const float4* u) {
        const float top = max_nd(m, pm), f = exp2_approx(sub_rn(m, top)), g = exp2_approx(sub_rn(pm, top));
        m = top, l = __fmaf_rn(l, f, mul_rn(pl, g));
#pragma unroll
        for (int x = 0; x < kCols; ++x) {
            v[x][0] = __fmaf_rn(v[x][0], f, mul_rn(u[x].x, g)), v[x][1] = __fmaf_rn(v[x][1], f, mul_rn(u[x].y, g));
            v[x][2] = __fmaf_rn(v[x][2], f, mul_rn(u[x].z, g)), v[x][3] = __fmaf_rn(v[x][3], f, mul_rn(u[x].w, g));
        }
    };
    if (q < rows) {
        for (int first = sub; first < runs; first += S * kBatch) {
            float2 st[kBatch];
            float4 u[kBatch][kCols];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int run = first + k * S;
                st[k] = make_float2(kLowest, 0.0f);
                if (run < runs) st[k] = *reinterpret_cast<const float2*>(part(run) + R * D + 2 * q);
#pragma unroll
                for (int x = 0; x < kCols; ++x) {
                    u[k][x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (run < runs && lane < kStep) u[k][x] = reinterpret_cast<const float4*>(part(run) + q * D)[x * 32 + lane];
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) add(st[k].x, st[k].y, u[k]);
        }
        if (S > 1 && sub > 0) {
            float* const mine = sums[warp % (8 * S)];
#pragma unroll
            for (int x = 0; x < kCols; ++x)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (lane < kStep) mine[(x * 4 + k) * kStep + lane] = v[x][k];
            if (lane == 0) mine[D] = m, mine[D + 1] = l;
        }
    }
    if (S > 1) {
        __syncthreads();
        if (sub > 0 || q >= rows) return;
        for (int w = 1; w < S; ++w) {
            const float* const other = sums[(warp + w) % (8 * S)];
            float4 u[kCols];
#pragma unroll
            for (int x = 0; x < kCols; ++x) {
                float y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = lane < kStep ? other[(x * 4 + k) * kStep + lane] : 0.0f;
                u[x] = make_float4(y[0], y[1], y[2], y[3]);
            }
            add(other[D], other[D + 1], u);
        }
    }
    int query, head;
    split_row(cut.n, G, cut.rt * R + q, &query, &head);
    const Finish end(a, cut.h * G + head, cut.h, m, l);
#pragma unroll
    for (int x = 0; x < kCols; ++x)
        if (lane < kStep) end.store(a, cut.row0 + query, cut.h * G + head, (x * 32 + lane) * 4, v[x]);
}

template <int D, int R>
cudaError_t launch_join(const AttendArgs& a, int ctas, cudaStream_t s) {
    if (ctas < 2) return cudaSuccess;
    return launch_pdl(k_join<D, R>, dim3(static_cast<unsigned>(ctas - 1), R / 8), dim3(256 * kSub<R>), 0, s, a, ctas);
}

}  // namespace

// the kernel of many queries a sequence
cudaError_t launch_attend_many(const AttendArgs& a, cudaStream_t s);
int64_t attend_many_workspace(const AttendArgs& a);

}  // namespace nvfp4
