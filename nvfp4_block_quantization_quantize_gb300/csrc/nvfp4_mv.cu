// nvfp4_mv.cu -- the product of at most 16 tokens with an NVFP4 weight
// (nvfp4_mv): out[m,n] = S_dec(n) * sum_k x[m,k] * (q[n,k] * dec(s[n,k/16])).
//
// Every weight byte is used once for at most 16 tokens, so the weight's 9/16
// byte per element is the floor and the kernel is bound by memory; tcgen05 would
// not help (its 128-row tiles would want the decoded weights staged through
// shared memory), the warp-level MMA takes them straight from registers.
//   - A weight decodes exactly to f16: q * dec(s) has at most 6 significant bits
//     and lies in [2^-10, 2688].
//   - x is scaled per token and K-slice by a power of two to at most 2^15 and
//     held in shared memory as f16 (an fp32 x as hi + lo, 22 bits), in the order
//     the MMA's B fragments are read.
//   - m16n8k16: 16 weight rows times 8 tokens.  The order of k inside a product
//     is free as long as A and B agree, so lane (g, t) of a warp takes whole
//     blocks: 16 * VB consecutive weights of rows g and g + 8, one 8 * VB-byte
//     load and VB scale bytes a row, for 4 * VB products.
//   - A chain of products starts from zero every 64 * VB columns and is added to
//     an fp32 sum, so the tensor core's own accumulation stays short.
// A CTA has W warps of 16 rows each over one slice of K (8 chunks of 64 * VB);
// each warp issues all the slice's loads at once.  The CTAs of a cluster take the
// slices of the same rows in turn and add their partial sums through distributed
// shared memory in rank order: no workspace, no atomics, the same bits each run.
#include <cooperative_groups.h>

#include "nvfp4_block.cuh"

namespace nvfp4 {
namespace {

namespace cg = cooperative_groups;

constexpr int kMvChunks = 8;                              // chunks of 64 * VB columns per slice
constexpr int kMvMaxCluster = 8;

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// a code byte's two weights, scaled (s holds the block's scale twice)
__device__ __forceinline__ uint32_t weight2(uint32_t w, int byte, uint32_t s) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(e2m1_decode_byte(w, byte)), "r"(s));
    return r;
}

// VB scale bytes -> f16 pairs, each holding one scale twice
template <int VB>
__device__ __forceinline__ void scale_pairs(uint32_t bytes, uint32_t* s) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(bytes)));
    s[0] = __byte_perm(h, h, 0x1010);
    if (VB == 2) s[VB - 1] = __byte_perm(h, h, 0x3232);
}

// VB blocks' codes (8 bytes each) streamed past L1, and their scale bytes
template <int VB>
__device__ __forceinline__ void load_blocks(const uint8_t* codes, const uint8_t* scales, int64_t blk, bool in,
                                            uint32_t* w, uint32_t& s) {
#pragma unroll
    for (int i = 0; i < 2 * VB; ++i) w[i] = 0;
    s = 0;
    if (!in) return;
    if (VB == 2) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2 * VB - 2]), "=r"(w[2 * VB - 1])
                     : "l"(codes + blk * 8));
        s = __ldg(reinterpret_cast<const uint16_t*>(scales + blk));
    } else {
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1])
                     : "l"(codes + blk * 8));
        s = __ldg(scales + blk);
    }
}

// 8 elements of x as fp32; columns past K are zero
template <int XT>
__device__ __forceinline__ void load_x8(const MvArgs& a, int64_t m, int k, float* v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (k >= a.K) return;                       // K % 16 == 0: a piece of 8 is whole or absent
    const int64_t e = m * a.K + k;
    if (XT == NVFP4_X_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + e);
        const float4 u = __ldg(p), w = __ldg(p + 1);
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w, v[4] = w.x, v[5] = w.y, v[6] = w.z, v[7] = w.w;
    } else if (XT == NVFP4_X_BF16) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + e));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + e));
        const uint32_t w[2] = {u.x, u.y};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            e4m3_decode2(w[i >> 1] >> (16 * (i & 1)), w[i >> 1] >> (16 * (i & 1) + 8), v[2 * i], v[2 * i + 1]);
    }
}

// One token's slice of x (columns k0 .. k0 + 512 * VB - 1) to shared memory by
// one warp: cell (chunk, j, part, token, t) of 16 bytes holds the 8 f16 values of
// columns chunk * 64 VB + t * 16 VB + 8 j of token's part (hi or lo).  Returns the
// exponent the token's sums are to be scaled by.
template <int XT, int VB>
__device__ __forceinline__ int stage_x(const MvArgs& a, uint4* xs, int Mp, int m, int k0, int lane) {
    constexpr int P = XT == NVFP4_X_F32 ? 2 : 1;
    constexpr int N8 = 2 * VB;                            // pieces of 8 columns per lane: 512 VB / 8 / 32
    float v[N8][8];
    int ex;
#pragma unroll
    for (int i = 0; i < N8; ++i) load_x8<XT>(a, m, k0 + (lane + 32 * i) * 8, v[i]);
    if (XT == NVFP4_X_MXFP8) {
        // value = e4m3 * 2^(b - 127); scaled by 2^(6 - top) with top the largest b: at most 448 * 64
        const int groups = (a.K + 31) / 32;
        int b[N8], top = 0;
#pragma unroll
        for (int i = 0; i < N8; ++i) {
            const int k = k0 + (lane + 32 * i) * 8;
            b[i] = k < a.K ? a.x_scales[static_cast<int64_t>(m) * groups + k / 32] : 0;
            if (b[i] != 255) top = max(top, b[i]);
        }
        top = __reduce_max_sync(0xFFFFFFFFu, top);
#pragma unroll
        for (int i = 0; i < N8; ++i) {
            const int f = 127 + 6 + b[i] - top;           // the factor's exponent field
            const float s = b[i] == 255 ? __int_as_float(0x7FC00000) : f > 0 ? __int_as_float(f << 23) : 0.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) v[i][q] = mul_rn(v[i][q], s);
        }
        ex = top - 127 - 6;
    } else {
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < N8; ++i)
#pragma unroll
            for (int q = 0; q < 8; ++q) mx = max_nd(mx, fabsf(v[i][q]));
        // exponent of the maximum, at least -112 so that 2^(14 - e) is a float
        const int e = max(static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(mx)) >> 23) - 127, -112);
        const float s = __int_as_float((127 + 14 - e) << 23);
#pragma unroll
        for (int i = 0; i < N8; ++i)
#pragma unroll
            for (int q = 0; q < 8; ++q) v[i][q] = mul_rn(v[i][q], s);
        ex = e - 14;
    }
#pragma unroll
    for (int i = 0; i < N8; ++i) {
        const int piece = lane + 32 * i;                  // columns 8 * piece of the slice
        const int chunk = piece / (8 * VB), t = piece / (2 * VB) % 4, j = piece % (2 * VB);
        uint4* cell = xs + (((chunk * 2 * VB + j) * P) * Mp + m) * 4 + t;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const __half2 h = __floats2half2_rn(v[i][2 * q], v[i][2 * q + 1]);
                w[q] = *reinterpret_cast<const uint32_t*>(&h);
                if (P == 2 && p == 0) {
                    // what hi leaves; an infinite hi (an infinity of x) leaves nothing
                    const float2 f = __half22float2(h);
                    v[i][2 * q] = isinf(f.x) ? 0.0f : sub_rn(v[i][2 * q], f.x);
                    v[i][2 * q + 1] = isinf(f.y) ? 0.0f : sub_rn(v[i][2 * q + 1], f.y);
                }
            }
            cell[p * Mp * 4] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    return ex;
}

// grid.x = cluster size * row blocks; a cluster's CTAs share W * 16 rows.
// Mp: M rounded up to a power of two (a lane group past it reads another token's
// values, and its columns are not stored).
template <int XT, int NT, int VB>
__global__ void __launch_bounds__(256) k_mv(const MvArgs a, int Mp) {
    extern __shared__ uint4 xs[];
    constexpr int P = XT == NVFP4_X_F32 ? 2 : 1;
    constexpr int kSlice = kMvChunks * 64 * VB;
    __shared__ float part[8 * 16 * 16];                   // [token][row]: W * 16 rows of at most 16 tokens
    __shared__ int ex[16];
    pdl_wait();
    const cg::cluster_group cluster = cg::this_cluster();
    const int S = cluster.num_blocks(), rank = cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = blockDim.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int R = W * 16;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / S) * R;
    const int64_t r = row0 + warp * 16 + g;
    const int64_t bpr = a.K / 16;
    const int slices = (a.K + kSlice - 1) / kSlice;
    float tot[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[n][i] = 0.0f;

    for (int sl = rank; sl < slices; sl += S) {
        const int k0 = sl * kSlice;
        uint32_t w[kMvChunks][2][2 * VB], sc[kMvChunks][2];
#pragma unroll
        for (int c = 0; c < kMvChunks; ++c) {
            const int64_t blk = k0 / 16 + (c * 4 + t) * VB;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                load_blocks<VB>(a.codes, a.scales, (r + 8 * h) * bpr + blk, r + 8 * h < a.N && blk < bpr, w[c][h],
                                sc[c][h]);
        }
        __syncthreads();                                  // the previous slice's x is no longer read
        for (int m = warp; m < a.M; m += W) {
            const int e = stage_x<XT, VB>(a, xs, Mp, m, k0, lane);
            if (lane == 0) ex[m] = e;
        }
        __syncthreads();
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
#pragma unroll
        for (int c = 0; c < kMvChunks; ++c) {
            if (k0 + c * 64 * VB >= a.K) break;
            uint32_t s[2][VB];
            scale_pairs<VB>(sc[c][0], s[0]);
            scale_pairs<VB>(sc[c][1], s[1]);
            float d[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) d[n][i] = 0.0f;
#pragma unroll
            for (int j = 0; j < 2 * VB; ++j) {            // word j of each row: two products
                uint32_t A[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) A[h][i] = weight2(w[c][h][j], i, s[h][j / 2]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const int tok = (n * 8 + g) & (Mp - 1);
                        const uint4 b = xs[(((c * 2 * VB + j) * P + p) * Mp + tok) * 4 + t];
                        mma_f16(d[n], A[0][0], A[1][0], A[0][1], A[1][1], b.x, b.y);
                        mma_f16(d[n], A[0][2], A[1][2], A[0][3], A[1][3], b.z, b.w);
                    }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] = add_rn(acc[n][i], d[n][i]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = n * 8 + 2 * t + (i & 1);
                if (m < a.M) tot[n][i] = add_rn(tot[n][i], ldexpf(acc[n][i], ex[m]));
            }
    }
    // the cluster's partial sums, added in rank order
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = n * 8 + 2 * t + (i & 1);
            if (m < a.M) part[m * R + warp * 16 + g + 8 * (i >> 1)] = tot[n][i];
        }
    cluster.sync();
    for (int i = rank * blockDim.x + tid; i < a.M * R; i += S * blockDim.x) {
        const int m = i / R;
        const int64_t n = row0 + i % R;
        if (n >= a.N) continue;
        float v = 0.0f;
        for (int q = 0; q < S; ++q) v = add_rn(v, *cluster.map_shared_rank(part + i, q));
        if (a.gamax_mode != NVFP4_GAMAX_NONE) {
            float enc, dec;
            global_scales(a.gamax[a.gamax_mode == NVFP4_GAMAX_ROW_GIVEN ? n : 0], a.bound, enc, dec);
            v = mul_rn(v, dec);
        }
        const int64_t o = static_cast<int64_t>(m) * a.N + n;
        if (a.out_dtype == NVFP4_F32) static_cast<float*>(a.out)[o] = v;
        else static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
    }
    cluster.sync();                                       // part is read by the whole cluster
    pdl_trigger();
}

template <int XT, int NT, int VB>
cudaError_t launch_mv_t(const MvArgs& a, cudaStream_t s) {
    constexpr int kSlice = kMvChunks * 64 * VB;
    constexpr int P = XT == NVFP4_X_F32 ? 2 : 1;
    int Mp = 1;
    while (Mp < a.M) Mp *= 2;
    const size_t smem = static_cast<size_t>(Mp) * kSlice * 2 * P;
    const int slices = (a.K + kSlice - 1) / kSlice;
    // the fewest rounds of at most kMvMaxCluster slices, in equal parts
    const int rounds = (slices + kMvMaxCluster - 1) / kMvMaxCluster;
    const int S = (slices + rounds - 1) / rounds;
    // whole 8-warp CTAs when they fill the SMs, else fewer warps each
    int W = 8;
    while (W > 1 && (static_cast<int64_t>(a.N) + 16 * W - 1) / (16 * W) * S < 2 * sm_count()) W /= 2;
    const int64_t blocks = (static_cast<int64_t>(a.N) + 16 * W - 1) / (16 * W) * S;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    static thread_local int configured_dev = -1;         // the attribute is per device
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_dev != dev) {
        const cudaError_t e = cudaFuncSetAttribute(k_mv<XT, NT, VB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   16 * kSlice * 2 * P);
        if (e != cudaSuccess) return e;
        configured_dev = dev;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(32 * W);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_mv<XT, NT, VB>, a, Mp);
}

template <int XT>
cudaError_t launch_mv_x(const MvArgs& a, cudaStream_t s) {
    if (a.K % 32 == 0) return a.M <= 8 ? launch_mv_t<XT, 1, 2>(a, s) : launch_mv_t<XT, 2, 2>(a, s);
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
