// nvfp4_mv.cu -- the product of at most 16 tokens with an NVFP4 weight
// (nvfp4_mv): out[m,n] = S_dec(n) * sum_k x[m,k] * (q[n,k] * dec(s[n,k/16])).
//
// Every weight byte is used once for at most 16 tokens, so the weight's 9/16
// byte per element is the floor and the kernel is bound by memory; tcgen05 would
// not help (its 128-row tiles would want the decoded weights staged through
// shared memory), the warp-level MMA takes them straight from registers.
//   - A weight decodes exactly to f16: q * dec(s) has at most 6 significant bits
//     and lies in [2^-10, 2688].
//   - x is scaled per token and warp by a power of two to at most 2^15 and held
//     in shared memory as f16, in the order the MMA's B fragments are read.  An fp32
//     x is hi + 2^-11 lo (22 bits), and the two have sums of their own until a chain's
//     end: with lo unscaled an element would lose bits from 2^-15 of the largest on
//     (f16 ends at 2^-24), so it does from 2^-27 on.
//   - m16n8k16: 16 weight rows times 8 tokens.  The order of k inside a product
//     is free as long as A and B agree, so lane (g, t) of a warp takes whole
//     blocks: 16 * VB consecutive weights of rows g and g + 8, one 8 * VB-byte
//     load and VB scale bytes a row, for 4 * VB products (a chunk: 64 * VB columns).
//   - A chain of at most 16 products starts from zero and is added to an fp32 sum,
//     so the tensor core's own accumulation stays short.
// A CTA has 8 warps: WK parts of its columns times WR groups of 16 weight rows.  Its x
// is staged once; then each warp walks down row tiles with kAhead chunks of weights in
// flight (registers; the loads run on across tiles).  Per tile the WK warps of a row
// group add their sums through shared memory.  Where the columns are too many for one
// CTA, or the rows too few for all SMs, the CTAs of a cluster split the columns and
// their sums meet through distributed shared memory at the end: no workspace, no
// atomics, every sum in a fixed order.
//
// Measured, in a graph of calls: 4 tokens x [65536, 8192] 53.5 us (5.7 TB/s, 0.84 of the copy
// rate; without its products the structure takes 51.5 us, without the scale bytes too 45.5),
// 1 token x [14336, 4096] 8.6 us (3.8 TB/s), [1024, 1024] 2.35 us; 8 MXFP8 tokens x [4096, 14336]
// 12.0 us, 13 fp32 tokens x [5003, 2064] 10.75 us.
//
// VB is 4 where rows of codes are whole 32-byte sectors (K % 64 == 0, codes 32-byte
// aligned): one 256-bit and one 32-bit load per row and 256 columns.  Otherwise 1.
#include <cooperative_groups.h>

#include "nvfp4_block.cuh"

namespace nvfp4 {
namespace {

namespace cg = cooperative_groups;

constexpr int kMvWarps = 8;
constexpr int kMvMaxCluster = 8;
constexpr int kMvMaxTiles = 16;                           // row tiles per cluster with sums kept to the end

template <int VB>
constexpr int kAhead = VB == 4 ? 2 : 4;                   // chunks of weights in flight per warp
template <int VB>
constexpr int kStep = 4 / VB;                             // chunks in the 256 columns a warp stages at once
constexpr int kMvCtas = 2;                                // CTAs an SM holds
constexpr int kMvMaxX = 72 * 1024;                        // x's share of a CTA's shared memory

// how the work is cut, chosen by the host
struct MvPlan {
    int S;                    // CTAs of a cluster (parts of the columns)
    int WK;                   // warps a CTA splits its columns among; the others take further rows
    int tiles;                // tiles of 16 * (8 / WK) rows per cluster
    int cpw;                  // chunks per warp and round, a multiple of kStep
    int rounds;               // rounds of S * WK * cpw chunks over K
};

// bytes of a token's part of x (n chunks): its cells, and half a bank row more so
// that two tokens' fragment reads do not meet in a bank
template <int XT, int VB>
__host__ __device__ constexpr int x_stride(int n) {
    return n * 128 * VB * (XT == NVFP4_X_F32 ? 2 : 1) + 64;
}

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the first product of a chain: c = a b
__device__ __forceinline__ void mma_f16_first(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// a word's eight weights, scaled, as four f16 pairs (s holds the block's scale twice).  The four-byte
// unpack, which e2m1_decode_byte avoids, reads right here: tests compare the products of every variant of
// the kernel bit for bit.
__device__ __forceinline__ void weights8(uint32_t w, uint32_t s, uint32_t* h) {
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

__device__ __forceinline__ uint32_t e4m3_pair(uint32_t bytes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(bytes)));
    return h;
}

// VB scale bytes -> f16 pairs, each holding one scale twice
template <int VB>
__device__ __forceinline__ void scale_pairs(uint32_t bytes, uint32_t* s) {
#pragma unroll
    for (int i = 0; i < VB; i += 2) {
        const uint32_t h = e4m3_pair(bytes >> (8 * i));
        s[i] = __byte_perm(h, h, 0x1010);
        if (VB > 1) s[(i + 1) % VB] = __byte_perm(h, h, 0x3232);
    }
}

// VB blocks' codes (8 bytes each), streamed past L1, and their scale bytes
template <int VB>
__device__ __forceinline__ void load_blocks(const uint8_t* codes, const uint8_t* scales, uint32_t* w, uint32_t& s) {
    if constexpr (VB == 4) {
        asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(codes));
        s = __ldg(reinterpret_cast<const uint32_t*>(scales));
    } else {
        asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(codes));
        s = __ldg(scales);
    }
}

// ---- staging of x -----------------------------------------------------------------------------
// The n chunks of columns from k0 of one part, every token: first copied as they are
// into the token's part of shared memory (MXFP8 into its second half), then converted
// in place, 256 columns at a time, to cells of 16 bytes: cell (chunk, j, part, t) holds
// the 8 f16 values of columns chunk * 64 VB + t * 16 VB + 8 j, part 0 being hi and 1 lo.
// The part's WR warps take the tokens in turn.
template <int XT>
constexpr int kXSize = XT == NVFP4_X_F32 ? 4 : XT == NVFP4_X_BF16 ? 2 : 1;

template <int XT, int VB>
__device__ __forceinline__ int raw_offset(int n) {
    return XT == NVFP4_X_MXFP8 ? n * 64 * VB : 0;
}

template <int XT, int VB>
__device__ __forceinline__ void copy_x(const MvArgs& a, uint8_t* xs, int64_t k0, int n, int wr, int WR, int lane) {
    const int64_t left = a.K - k0;
    const int cols = static_cast<int>(left < n * 64 * VB ? (left > 0 ? left : 0) : n * 64 * VB);
    const uint8_t* src = static_cast<const uint8_t*>(a.x) + k0 * kXSize<XT>;
    for (int m = wr; m < a.M; m += WR) {
        uint8_t* dst = xs + m * x_stride<XT, VB>(n) + raw_offset<XT, VB>(n);
        const uint8_t* row = src + static_cast<int64_t>(m) * a.K * kXSize<XT>;
        for (int i = lane; i < cols * kXSize<XT> / 16; i += 32) cp_async16(dst + 16 * i, row + 16 * i);
    }
    cp_async_commit();
}

__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}

// 2^e as a float, e >= -149
__device__ __forceinline__ float power_of_two(int e) {
    return e >= -126 ? __int_as_float((e + 127) << 23) : __int_as_float(1 << (e + 149));
}

// 2^e twice, as f16 pairs' bits whose product it is (e in [-38, 30]): f16 itself ends at 2^15
// and 2^-24.  An E4M3 value times the first is exact (a multiple of 2^-23, at most 2^15 for those
// that end within f16's range), so that the second makes the only rounding.
__device__ __forceinline__ uint2 power_of_two_f16(int e) {
    const int first = min(max(e, -14), 15), rest = e - first;
    return make_uint2(static_cast<uint32_t>(first + 15) * (0x00010001u << 10),
                      rest >= -14 ? static_cast<uint32_t>(rest + 15) * (0x00010001u << 10) : 0x00010001u << (rest + 24));
}

// 8 columns as four f16 pairs: the raw ones at r scaled by f.x, an fp32's bits, or by the f16 pairs
// f.x and f.y (MXFP8)
template <int XT, int P>
__device__ __forceinline__ void convert8(const uint8_t* r, uint2 f, uint32_t (*h)[4]) {
    if (XT == NVFP4_X_MXFP8) {
        const uint2 u = *reinterpret_cast<const uint2*>(r);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            h[0][q] = mul_f16x2(mul_f16x2(e4m3_pair((q < 2 ? u.x : u.y) >> (16 * (q & 1))), f.x), f.y);
        return;
    }
    float v[8];
    if (XT == NVFP4_X_F32) {
        const float4* p = reinterpret_cast<const float4*>(r);
        const float4 u = p[0], w = p[1];
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w, v[4] = w.x, v[5] = w.y, v[6] = w.z, v[7] = w.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(r);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = __uint_as_float(w[q] << 16);
            v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
        }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float x0 = mul_rn(v[2 * q], __uint_as_float(f.x)), x1 = mul_rn(v[2 * q + 1], __uint_as_float(f.x));
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const __half2 o = __floats2half2_rn(x0, x1);
            h[p][q] = *reinterpret_cast<const uint32_t*>(&o);
            // what hi leaves, times 2^11 (at most hi's own size); an infinite hi (an infinity of x) leaves nothing
            const float2 b = __half22float2(o);
            x0 = isinf(b.x) ? 0.0f : mul_rn(sub_rn(x0, b.x), 2048.0f);
            x1 = isinf(b.y) ? 0.0f : mul_rn(sub_rn(x1, b.y), 2048.0f);
        }
    }
}

// largest magnitude (its bits) of 8 raw columns, NaN dropped
template <int XT>
__device__ __forceinline__ uint32_t top8(const uint8_t* r) {
    if (XT == NVFP4_X_F32) {
        const float4* p = reinterpret_cast<const float4*>(r);
        const float4 u = p[0], w = p[1];
        const float m0 = max_nd(max_nd(fabsf(u.x), fabsf(u.y)), max_nd(fabsf(u.z), fabsf(u.w)));
        const float m1 = max_nd(max_nd(fabsf(w.x), fabsf(w.y)), max_nd(fabsf(w.z), fabsf(w.w)));
        return __float_as_uint(max_nd(max_nd(m0, m1), 0.0f));
    }
    const uint4 u = *reinterpret_cast<const uint4*>(r);
    uint32_t p = absmax_bf16x2(absmax_bf16x2(0u, u.x), u.y);
    p = absmax_bf16x2(absmax_bf16x2(p, u.z), u.w);
    return max(p << 16, p & 0xFFFF0000u);
}

// largest magnitude of 16 E4M3 codes, as its 7 bits (NaN: the largest)
__device__ __forceinline__ uint32_t top_code(uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t lo = 0, hi = 0;                              // of even and odd bytes, two each
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo = __vmaxu2(lo, w[i] & 0x007F007Fu);
        hi = __vmaxu2(hi, (w[i] >> 8) & 0x007F007Fu);
    }
    const uint32_t m = __vmaxu2(lo, hi);
    return max(m & 0xFFFFu, m >> 16);
}

// Converts the copied columns of tokens wr, wr + WR, ..; up[m]: what that token's sums are to
// be multiplied by.  sb: the tokens' E8M0 bytes of these columns, sb_stride apart.
template <int XT, int VB>
__device__ __forceinline__ void convert_x(const MvArgs& a, uint8_t* xs, float* up, const uint8_t* sb, int sb_stride,
                                          int64_t k0, int n, int wr, int WR, int lane) {
    constexpr int P = XT == NVFP4_X_F32 ? 2 : 1;
    constexpr int kPiece = 8 * kXSize<XT>;                // bytes of 8 raw columns
    const int steps = n / kStep<VB>;
    const int64_t left = a.K - k0;
    const int pieces = static_cast<int>(left < steps * 256 ? (left > 0 ? left : 0) : steps * 256) / 8;
    for (int m = wr; m < a.M; m += WR) {
        uint8_t* cells = xs + m * x_stride<XT, VB>(n);
        const uint8_t* raw = cells + raw_offset<XT, VB>(n);
        uint32_t top = 0;
        if (XT == NVFP4_X_MXFP8) {
            // the largest exponent of a value: scale byte + 9 + the exponent of the largest code c of its columns (c / 8 - 7,
            // below that of its three bits), at least 1; a group of zeros, whose scale may be any, has none
            for (int i = lane; i * 2 < pieces; i += 32) {
                const uint32_t b = sb[m * sb_stride + i / 2], c = top_code(*reinterpret_cast<const uint4*>(raw + 16 * i));
                if (c != 0 && b != 255) top = max(top, b + (c < 8 ? 31 - __clz(c) : 2 + (c >> 3)));
            }
        } else {
            for (int i = lane; i < pieces; i += 32) top = max(top, top8<XT>(raw + kPiece * i));
        }
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        // scaled to at most 2^15: x by 2^(14 - e), e its exponent (at least -112, so that this is a
        // float); an E4M3 element of scale byte b by 2^(b + 23 - top) (above 23: of zeros)
        const int e = XT == NVFP4_X_MXFP8 ? static_cast<int>(max(top, 1u)) - 9 - 127 - 14
                                          : max(static_cast<int>(top >> 23) - 127, -112) - 14;
        if (lane == 0) up[m] = power_of_two(e);
        const float down = XT == NVFP4_X_MXFP8 ? 0.0f : power_of_two(-e);
#pragma unroll 2
        for (int s = 0; s < steps; ++s) {
            const int i = s * 32 + lane;                  // piece of 8 columns
            uint2 f = make_uint2(__float_as_uint(down), 0u);
            if (XT == NVFP4_X_MXFP8) {
                const int b = i < pieces ? sb[m * sb_stride + i / 4] : 0;
                f = power_of_two_f16(min(max(b - 127 - e, -38), 23));
                if (b == 255) f.x = 0x7FFF7FFFu;          // NaN
            }
            uint32_t h[P][4];
            convert8<XT, P>(raw + kPiece * i, f, h);
            __syncwarp();                                 // all of the step is read
            const int j = i % (2 * VB), t = i / (2 * VB) % 4, chunk = i / (8 * VB);
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<uint4*>(cells + (((chunk * 2 * VB + j) * P + p) * 4 + t) * 16) =
                    i < pieces ? make_uint4(h[p][0], h[p][1], h[p][2], h[p][3]) : make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
    }
}

// decode scale of weight row n (any n without a per-row amax)
__device__ __forceinline__ float decode(const MvArgs& a, int64_t n) {
    float enc, dec = 1.0f;
    if (a.gamax_mode != NVFP4_GAMAX_NONE)
        global_scales(a.gamax[a.gamax_mode == NVFP4_GAMAX_ROW_GIVEN ? n : 0], a.bound, enc, dec);
    return dec;
}

__device__ __forceinline__ void store_out(const MvArgs& a, int m, int64_t n, float v, float dec) {
    v = mul_rn(v, dec);
    const int64_t o = static_cast<int64_t>(m) * a.N + n;
    if (a.out_dtype == NVFP4_F32) static_cast<float*>(a.out)[o] = v;
    else static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
}

template <int NT>
constexpr int kMvRow = 8 * NT * 16;                       // floats of a warp's tile of sums

// Dynamic shared memory: x [WK][M][x_stride(cpw)]; an MXFP8 x's scale bytes [WK][M][2 VB cpw];
// then the sums kept to the end [tiles][WR][M][16] when the columns are split.  Lane groups
// past the last token read its values, and their columns are not stored.  Rows past N and
// blocks past K read the last ones again: such rows are not stored, such blocks meet zeros of x.
template <int XT, int NT, int VB>
__global__ void __launch_bounds__(32 * kMvWarps, kMvCtas) k_mv(const MvArgs a, const MvPlan p) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int P = XT == NVFP4_X_F32 ? 2 : 1;
    constexpr int kChain = VB == 1 ? 2 : 8;               // words of a row whose products form a chain: at most 16
    __shared__ float red[2][kMvWarps][kMvRow<NT>];        // [token][row] of each warp, two tiles in turn
    __shared__ float up[kMvWarps][16];                    // of each part of the columns
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = p.S > 1 ? static_cast<int>(cluster.block_rank()) : 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int WR = kMvWarps / p.WK, wk = warp % p.WK, wr = warp / p.WK;
    const int g = lane >> 2, t = lane & 3;
    const int bpr = a.K / 16;
    const int all_chunks = (bpr + 4 * VB - 1) / (4 * VB);
    const int tile0 = static_cast<int>(blockIdx.x / p.S) * p.tiles;
    const int ntiles = min(p.tiles, (a.N + 16 * WR - 1) / (16 * WR) - tile0);
    const int stride = x_stride<XT, VB>(p.cpw);
    const int sb_stride = XT == NVFP4_X_MXFP8 ? 2 * VB * p.cpw : 0;
    uint8_t* xs = smem + static_cast<size_t>(wk) * a.M * stride;
    uint8_t* sb = smem + static_cast<size_t>(p.WK) * a.M * stride + wk * a.M * sb_stride;
    float* kept = reinterpret_cast<float*>(smem + static_cast<size_t>(p.WK) * a.M * (stride + sb_stride));
    const uint8_t* frag[NT];                              // this lane's fragments of its tokens
#pragma unroll
    for (int q = 0; q < NT; ++q) frag[q] = xs + min(q * 8 + g, a.M - 1) * stride + t * 16;
    const bool keep = p.S > 1 || p.rounds > 1;
    int turn = 0;                                         // of red, over all tiles and rounds
    pdl_trigger();                                        // the next kernel waits for this one's end itself
    pdl_wait();

    for (int round = 0; round < p.rounds; ++round) {
        const int chunk0 = ((round * p.S + rank) * p.WK + wk) * p.cpw;
        const int n = min(max(all_chunks - chunk0, 0), p.cpw);          // this warp's chunks
        const int total = ntiles * n;
        const int64_t k0 = static_cast<int64_t>(chunk0) * 64 * VB;
        if (round) __syncthreads();                       // the previous round's x is no longer read
        copy_x<XT, VB>(a, xs, k0, p.cpw, wr, WR, lane);
        if (XT == NVFP4_X_MXFP8) {
            const int64_t groups = (static_cast<int64_t>(a.K) + 31) / 32, first = k0 / 32;
            for (int m = wr; m < a.M; m += WR) {
                const uint8_t* src = a.x_scales + m * groups + first;
                uint8_t* dst = sb + m * sb_stride;
                if (groups % 4 == 0) {                    // whole words, with x's copies
                    for (int i = 4 * lane; i < sb_stride; i += 128)
                        if (first + i < groups) cp_async4(dst + i, src + i);
                } else {
                    for (int i = lane; i < sb_stride; i += 32)
                        if (first + i < groups) dst[i] = __ldg(src + i);
                }
            }
            cp_async_commit();
        }
        // loads run kAhead chunks ahead of the products, on into the next tiles
        uint32_t w[kAhead<VB>][2][2 * VB], sc[kAhead<VB>][2];
        // (pointers to the lane's blocks of rows g and g + 8 in the warp's first chunk, and bytes from there)
        int lt = 0, lc = 0;
        const uint8_t *c0, *c1, *s0, *s1;
        const int first_blk = (chunk0 * 4 + t) * VB, most_blk = bpr - VB - first_blk;
        auto rows = [&] {
            const int row = ((tile0 + lt) * WR + wr) * 16 + g;
            const int64_t r0 = static_cast<int64_t>(min(row, a.N - 1)) * bpr + first_blk;
            const int64_t r1 = static_cast<int64_t>(min(row + 8, a.N - 1)) * bpr + first_blk;
            s0 = a.scales + r0, s1 = a.scales + r1;
            c0 = a.codes + r0 * 8, c1 = a.codes + r1 * 8;
        };
        rows();
        auto load = [&](int u) {
            if (lt >= ntiles || n == 0) return;
            const int blk = min(lc * 4 * VB, most_blk);
            load_blocks<VB>(c0 + blk * 8, s0 + blk, w[u][0], sc[u][0]);
            load_blocks<VB>(c1 + blk * 8, s1 + blk, w[u][1], sc[u][1]);
            if (++lc == n) {
                lc = 0;
                ++lt;
                rows();
            }
        };
#pragma unroll
        for (int u = 0; u < kAhead<VB>; ++u) load(u);
        cp_async_wait<0>();
        __syncwarp();
        convert_x<XT, VB>(a, xs, up[wk], sb, sb_stride, k0, p.cpw, wr, WR, lane);
        __syncthreads();
        // without a per-row amax the decode scale is known here; with one, its row's is fetched ahead
        const bool per_row = a.gamax_mode == NVFP4_GAMAX_ROW_GIVEN;
        const float dec_all = per_row || keep ? 1.0f : decode(a, 0);
        float acc[NT][4];
        int c = 0, tile = 0;
        auto clear = [&](float (*f)[4]) {
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) f[q][i] = 0.0f;
        };
        // A row group's sums of a tile, added in the order of its WK warps by the threads of (token, row);
        // the warps take turns at being the first of those (few tokens need one warp only).
        auto end_tile = [&] {
            float* r = red[turn][warp];
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = q * 8 + 2 * t + (i & 1);
                    if (m < a.M) r[m * 16 + g + 8 * (i >> 1)] = mul_rn(acc[q][i], up[wk][m]);
                }
            const int from = ((wk + tile) & (p.WK - 1)) * 32 + lane;
            const int64_t row = static_cast<int64_t>((tile0 + tile) * WR + wr) * 16 + (lane & 15);
            const float dec = per_row && !keep && from < a.M * 16 && row < a.N ? decode(a, row) : dec_all;
            // by number, one barrier a row group: its warps come here from different steps of the loop below
            asm volatile("bar.sync %0, %1;" ::"r"(1 + wr), "r"(32 * p.WK) : "memory");
            for (int i = from; i < a.M * 16; i += 32 * p.WK) {
                float v = 0.0f;
#pragma unroll
                for (int q = 0; q < kMvWarps; ++q)
                    if (q < p.WK) v = add_rn(v, red[turn][wr * p.WK + q][i]);
                if (keep) {
                    float* k = kept + (tile * WR + wr) * a.M * 16 + i;
                    *k = round ? add_rn(*k, v) : v;
                } else if (row < a.N) {
                    store_out(a, i >> 4, row, v, dec);
                }
            }
            clear(acc);
            c = 0;
            ++tile;
            turn ^= 1;
        };
        clear(acc);
        for (int i0 = 0; i0 < total; i0 += kAhead<VB>) {
#pragma unroll
            for (int u = 0; u < kAhead<VB>; ++u) {
                if (i0 + u >= total) break;
                uint32_t s[2][VB];
                scale_pairs<VB>(sc[u][0], s[0]);
                scale_pairs<VB>(sc[u][1], s[1]);
                const int at = c * (128 * VB * P);
                float d[P][NT][4];
#pragma unroll
                for (int j = 0; j < 2 * VB; ++j) {        // word j of each row: two products
                    uint32_t A[2][4];
                    weights8(w[u][0][j], s[0][j / 2], A[0]);
                    weights8(w[u][1][j], s[1][j / 2], A[1]);
#pragma unroll
                    for (int q = 0; q < NT; ++q)
#pragma unroll
                        for (int h = 0; h < P; ++h) {
                            const uint4 b = *reinterpret_cast<const uint4*>(frag[q] + at + (j * P + h) * 64);
                            if (j % kChain == 0)
                                mma_f16_first(d[h][q], A[0][0], A[1][0], A[0][1], A[1][1], b.x, b.y);
                            else
                                mma_f16(d[h][q], A[0][0], A[1][0], A[0][1], A[1][1], b.x, b.y);
                            mma_f16(d[h][q], A[0][2], A[1][2], A[0][3], A[1][3], b.z, b.w);
                        }
                    if (j % kChain == kChain - 1)         // the chains' end
#pragma unroll
                        for (int q = 0; q < NT; ++q)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[q][i] = add_rn(acc[q][i], P == 2 ? __fmaf_rn(d[P - 1][q][i], 0x1p-11f, d[0][q][i]) : d[0][q][i]);
                }
                load(u);
                if (++c == n) end_tile();
            }
        }
        while (tile < ntiles) end_tile();                 // a warp with no columns takes part with zeros
    }
    if (keep) {
        // the parts of the columns, added in rank order (read from the CTAs that have them: sending them to
        // the one that adds them up, with one barrier less, took 2 us longer)
        if (p.S > 1) cluster.sync();
        else __syncthreads();
        for (int i = rank * blockDim.x + tid; i < ntiles * WR * a.M * 16; i += p.S * blockDim.x) {
            const int64_t row = (static_cast<int64_t>(tile0) * WR + i / (a.M * 16)) * 16 + (i & 15);
            if (row >= a.N) continue;
            const float dec = decode(a, row);
            float v = kept[i];
            if (p.S > 1) {
                float part[kMvMaxCluster];                // loaded together: a remote load takes long
#pragma unroll
                for (int q = 0; q < kMvMaxCluster; ++q) part[q] = q < p.S ? *cluster.map_shared_rank(kept + i, q) : 0.0f;
                v = part[0];
#pragma unroll
                for (int q = 1; q < kMvMaxCluster; ++q) v = q < p.S ? add_rn(v, part[q]) : v;
            }
            store_out(a, i / 16 % a.M, row, v, dec);
        }
        if (p.S > 1) cluster.sync();                      // kept is read by the whole cluster
    }
}

// The cut whose longest row of CTAs takes the least time, in the time of a warp's chunk of
// 256 columns: S parts of the columns over a cluster and WK over a CTA's warps (what does
// not fit a CTA's shared memory takes more rounds), the row tiles spread over the clusters
// that run at once.  A tile's end costs about half a chunk, a cluster's two barriers about
// two, staging about one per 2 KB of a CTA's x.
template <int XT, int VB>
MvPlan plan_mv(const MvArgs& a) {
    const int64_t chunks = (static_cast<int64_t>(a.K) + 64 * VB - 1) / (64 * VB);
    const int64_t rows = (static_cast<int64_t>(a.N) + 15) / 16;
    MvPlan best = {};
    double least = -1.0;
    for (int S = 1; S <= kMvMaxCluster; ++S)
        for (int WK = 1; WK <= kMvWarps; WK *= 2) {
            if (S * WK > 1 && static_cast<int64_t>(S * WK - 1) >= chunks) continue;      // a part without columns
            const int most = ((kMvMaxX / (WK * a.M) - 64) / (x_stride<XT, VB>(1) - 64)) / kStep<VB> * kStep<VB>;
            if (most < 1) continue;
            const int WR = kMvWarps / WK;
            int64_t cpw = (chunks + S * WK - 1) / (S * WK);
            const int64_t rounds = (cpw + most - 1) / most;
            cpw = ((cpw + rounds - 1) / rounds + kStep<VB> - 1) / kStep<VB> * kStep<VB>;
            const int64_t row_tiles = (rows + WR - 1) / WR;
            const int64_t clusters = static_cast<int64_t>(kMvCtas) * sm_count() / S;
            int64_t tiles = (row_tiles + clusters - 1) / clusters;
            if ((S > 1 || rounds > 1) && tiles * WR > kMvMaxTiles) tiles = kMvMaxTiles / WR;
            const int64_t waves = ((row_tiles + tiles - 1) / tiles + clusters - 1) / clusters;
            const double chunk = VB / 4.0;
            const double stage = static_cast<double>(rounds) * WK * a.M * x_stride<XT, VB>(static_cast<int>(cpw)) / 2048;
            const double time = waves * (tiles * rounds * (cpw * chunk + 0.5) + stage / kMvWarps + (S > 1 ? 2 : 0));
            if (least < 0 || time < least) {
                least = time;
                best = MvPlan{S, WK, static_cast<int>(tiles), static_cast<int>(cpw), static_cast<int>(rounds)};
            }
        }
    return best;
}

template <int XT, int NT, int VB>
cudaError_t launch_mv_t(const MvArgs& a, cudaStream_t s) {
    const MvPlan p = plan_mv<XT, VB>(a);
    const int64_t WR = kMvWarps / p.WK;
    const int64_t blocks = ((static_cast<int64_t>(a.N) + 16 * WR - 1) / (16 * WR) + p.tiles - 1) / p.tiles * p.S;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const size_t sb = XT == NVFP4_X_MXFP8 ? 2 * VB * p.cpw : 0;
    const size_t smem = static_cast<size_t>(p.WK) * a.M * (x_stride<XT, VB>(p.cpw) + sb) +
                        (p.S > 1 || p.rounds > 1 ? p.tiles * WR * a.M * 64 : 0);
    static thread_local int configured_dev = -1;         // the attribute is per device
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_dev != dev) {
        const cudaError_t e = cudaFuncSetAttribute(k_mv<XT, NT, VB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kMvMaxX + kMvMaxX / 32 + kMvMaxTiles * 16 * 64);
        if (e != cudaSuccess) return e;
        configured_dev = dev;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(32 * kMvWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_mv<XT, NT, VB>, a, p);
}

template <int XT>
cudaError_t launch_mv_x(const MvArgs& a, cudaStream_t s) {
    if (a.K % 64 == 0 && reinterpret_cast<uintptr_t>(a.codes) % 32 == 0)
        return a.M <= 8 ? launch_mv_t<XT, 1, 4>(a, s) : launch_mv_t<XT, 2, 4>(a, s);
    return a.M <= 8 ? launch_mv_t<XT, 1, 1>(a, s) : launch_mv_t<XT, 2, 1>(a, s);
}

}  // namespace

int launch_mv(const MvArgs& a, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (a.x_type) {
        case NVFP4_X_F32: return static_cast<int>(launch_mv_x<NVFP4_X_F32>(a, s));
        case NVFP4_X_BF16: return static_cast<int>(launch_mv_x<NVFP4_X_BF16>(a, s));
        default: return static_cast<int>(launch_mv_x<NVFP4_X_MXFP8>(a, s));
    }
}

}  // namespace nvfp4
