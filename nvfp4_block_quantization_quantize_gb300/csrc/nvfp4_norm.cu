// nvfp4_norm.cu -- residual addition, root-mean-square norm and quantization
// of its output in one pass (nvfp4_rmsnorm).
//
// Per row, fp32: h = x + hidden, y = (h * rsqrt(mean(h^2) + eps)) * weight, then y to
// NVFP4 (e2m1 codes, one E4M3 scale per 16) or MXFP8 (E4M3 elements, one E8M0
// scale per 32).  Each element is read once and each result written once, about
// ten operations an element: the kernel is bound by memory (by latency for a few
// rows).  A row belongs to one CTA: a thread holds C blocks of 16 elements in
// registers from the load to the stores, so nothing is read twice; rows longer
// than the registers hold (C == 0) are read a second time instead.
#include "nvfp4_block.cuh"

namespace nvfp4 {
namespace {

constexpr int kNormMaxThreads = 1024;

// 16 elements of memory this kernel may also write (the hidden state in place):
// a plain load, not the read-only path
template <int DT>
__device__ __forceinline__ void load16_rw(const void* base, int64_t elem0, float* y) {
    if (DT == NVFP4_BF16) lds16<DT>(static_cast<const uint16_t*>(base) + elem0, y);
    else lds16<DT>(static_cast<const float*>(base) + elem0, y);
}

template <int DT>
__device__ __forceinline__ void store16(void* base, int64_t elem0, const float* y) {
    if (DT == NVFP4_BF16) store16_bf16(static_cast<uint16_t*>(base), elem0, y);
    else store16_f32(static_cast<float*>(base), elem0, y);
}

// h = x + hidden of the 16 elements from elem0
template <int DT>
__device__ __forceinline__ void load_h(const NormArgs& a, int64_t elem0, float* h) {
    load16<DT>(a.x, elem0, h);
    if (a.hidden) {
        float r[16];
        load16_rw<DT>(a.hidden, elem0, r);
        add16(h, r);
    }
}

// y = (h * rstd) * weight of the 16 elements from column col
__device__ __forceinline__ void normed(const NormArgs& a, int64_t col, float rstd, const float* h, float* y) {
    float w[16];
    if (!a.weight) {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = mul_rn(h[i], rstd);
        return;
    }
    if (a.weight_dtype == NVFP4_BF16) load16<NVFP4_BF16>(a.weight, col, w);
    else load16<NVFP4_F32>(a.weight, col, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = mul_rn(mul_rn(h[i], rstd), w[i]);
}

// sum or maximum over a row's threads (whole warps); s has one float per warp of
// the CTA, and every thread of the CTA calls it
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* s) {
    const int warps = blockDim.x >> 5, tid = threadIdx.x;
    float* row = s + threadIdx.y * warps;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = MAX ? max_nd(v, u) : add_rn(v, u);
    }
    if (warps == 1) return v;
    if ((tid & 31) == 0) row[tid >> 5] = v;
    __syncthreads();
    v = (tid & 31) < warps ? row[tid & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = MAX ? max_nd(v, u) : add_rn(v, u);
    }
    return v;
}

// E8M0 exponent of a group amax: the least e >= -127 with b <= 448 * 2^e, 448 =
// 1.75 * 2^8 (b an infinity: 120, whose elements then saturate)
__device__ __forceinline__ int e8m0_exponent(float b) {
    const uint32_t u = __float_as_uint(b);
    const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, -127), 120);
}

// Quantize and store the 16 elements y of row `row`, block `blk` of bpr.  MXFP8:
// the even and odd thread of a pair hold a group's two halves (a group past the
// row's end holds zeros); every thread of the warp calls it, `live` ones store.
template <int FMT>
__device__ __forceinline__ void quantize16(const NormArgs& a, int64_t row, int64_t blk, int64_t bpr, bool live,
                                           const GScale& g, const float* y) {
    const float own = absmax16(y);
    if (FMT == NVFP4_FMT_MXFP8) {
        const float b = max_nd(own, __shfl_xor_sync(0xFFFFFFFFu, own, 1));
        if (!live) return;
        const int e = e8m0_exponent(b);
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);    // 2^-e, -e in [-120, 127]
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t c0, c1, c2, c3;
            e4m3_encode2(mul_rn(y[4 * i], inv), mul_rn(y[4 * i + 1], inv), c0, c1);
            e4m3_encode2(mul_rn(y[4 * i + 2], inv), mul_rn(y[4 * i + 3], inv), c2, c3);
            w[i] = c0 | (c1 << 8) | (c2 << 16) | (c3 << 24);
        }
        *reinterpret_cast<uint4*>(a.codes + (row * bpr + blk) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        if (!(blk & 1)) a.scales[row * ((bpr + 1) >> 1) + (blk >> 1)] = static_cast<uint8_t>(e + 127);
    } else {
        if (!live) return;
        const uint32_t sf = e4m3_encode(min_nd(block_s6f<true>(own, g.Senc), 448.0f));
        const float D = mul_rn(e4m3_decode(sf), g.Sdec);
        uint32_t w0, w1;
        float q[1];
        PhiloxKeys none;                            // nearest rounding draws nothing
        encode_plain16<NVFP4_RTN>(y, D, own, 0, none, w0, w1, nullptr, sf, q, false);
        *reinterpret_cast<uint2*>(a.codes + (row * bpr + blk) * 8) = make_uint2(w0, w1);
        a.scales[row * bpr + blk] = static_cast<uint8_t>(sf);
    }
}

// blockDim (threads per row, rows per CTA); C blocks of 16 per thread held in
// registers, or C == 0 with the row read twice
template <int DT, int C, int FMT>
__global__ void __launch_bounds__(kNormMaxThreads) k_rmsnorm(const NormArgs a) {
    __shared__ float ssum[32], smax[32];
    pdl_wait();
    const int64_t bpr = a.K / 16;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool in = row < a.M;
    const int64_t T = blockDim.x;
    // threads of a pair stay together: every thread makes the same number of steps
    const int64_t steps = C ? C : (bpr + T - 1) / T;
    float h[C ? C : 1][16];
    float sum = 0.0f;
    auto load = [&](int64_t c, float* v) {
        const int64_t blk = threadIdx.x + c * T;
        if (in && blk < bpr) load_h<DT>(a, (row * bpr + blk) * 16, v);
        else
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    };
    auto square = [&](const float* v) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s = __fmaf_rn(v[i], v[i], s);
        sum = add_rn(sum, s);
    };
    if constexpr (C) {
#pragma unroll
        for (int c = 0; c < C; ++c) load(c, h[c]);
#pragma unroll
        for (int c = 0; c < C; ++c) square(h[c]);
    } else {
        for (int64_t c = 0; c < steps; ++c) {
            load(c, h[0]);
            square(h[0]);
        }
    }
    const float mean = div_rn(row_reduce<false>(sum, ssum), static_cast<float>(a.K));
    const float rstd = div_rn(1.0f, __fsqrt_rn(add_rn(mean, a.eps)));
    GScale g{0.0f, 1.0f, 1.0f};
    if (FMT == NVFP4_FMT_NVFP4 && a.codes && a.gamax_mode != NVFP4_GAMAX_NONE) {
        if (a.gamax_mode == NVFP4_GAMAX_ROW) {
            float m = 0.0f;
            auto rowmax = [&](int64_t c, const float* v) {
                const int64_t blk = threadIdx.x + c * T;
                if (!in || blk >= bpr) return;
                float y[16];
                normed(a, blk * 16, rstd, v, y);
                m = max_nd(m, absmax16(y));
            };
            if constexpr (C) {
#pragma unroll
                for (int c = 0; c < C; ++c) rowmax(c, h[c]);
            } else {
                for (int64_t c = 0; c < steps; ++c) {
                    load(c, h[0]);
                    rowmax(c, h[0]);
                }
            }
            g.A = row_reduce<true>(m, smax);
            if (in && threadIdx.x == 0) a.gamax[row] = g.A;
        } else if (in) {
            g.A = a.gamax[a.gamax_mode == NVFP4_GAMAX_ROW_GIVEN ? row : 0];
        }
        global_scales(g.A, a.bound, g.Senc, g.Sdec);
    }
    auto finish = [&](int64_t c, const float* v) {
        const int64_t blk = threadIdx.x + c * T;
        const bool live = in && blk < bpr;
        float y[16];
        if (live) {
            if (a.hidden_out) store16<DT>(a.hidden_out, (row * bpr + blk) * 16, v);
            normed(a, blk * 16, rstd, v, y);
            if (a.out) store16<DT>(a.out, (row * bpr + blk) * 16, y);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = 0.0f;
        }
        if (a.codes) quantize16<FMT>(a, row, blk, bpr, live, g, y);
    };
    if constexpr (C) {
#pragma unroll
        for (int c = 0; c < C; ++c) finish(c, h[c]);
    } else {
        for (int64_t c = 0; c < steps; ++c) {
            load(c, h[0]);
            finish(c, h[0]);
        }
    }
    pdl_trigger();
}

template <int DT, int FMT>
cudaError_t launch_c(const NormArgs& a, int C, dim3 grid, dim3 block, cudaStream_t s) {
    switch (C) {
        case 1: return launch_pdl(k_rmsnorm<DT, 1, FMT>, grid, block, 0, s, a);
        case 2: return launch_pdl(k_rmsnorm<DT, 2, FMT>, grid, block, 0, s, a);
        default: return launch_pdl(k_rmsnorm<DT, 0, FMT>, grid, block, 0, s, a);
    }
}

}  // namespace

int launch_rmsnorm(const NormArgs& a, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t bpr = a.K / 16;
    const int C = bpr <= kNormMaxThreads ? 1 : bpr <= 2 * kNormMaxThreads ? 2 : 0;
    int T = kNormMaxThreads;
    if (C) T = static_cast<int>(((bpr + C - 1) / C + 31) / 32 * 32);
    const int rows = T >= 256 ? 1 : 256 / T;
    const int64_t blocks = (a.M + rows - 1) / rows;
    if (blocks > 0x7FFFFFFF) return static_cast<int>(cudaErrorInvalidConfiguration);
    const dim3 grid(static_cast<unsigned>(blocks)), block(static_cast<unsigned>(T), static_cast<unsigned>(rows));
    const bool bf = a.dtype == NVFP4_BF16, mx = a.format == NVFP4_FMT_MXFP8;
    cudaError_t e;
    if (bf) e = mx ? launch_c<NVFP4_BF16, NVFP4_FMT_MXFP8>(a, C, grid, block, s)
                   : launch_c<NVFP4_BF16, NVFP4_FMT_NVFP4>(a, C, grid, block, s);
    else e = mx ? launch_c<NVFP4_F32, NVFP4_FMT_MXFP8>(a, C, grid, block, s)
                : launch_c<NVFP4_F32, NVFP4_FMT_NVFP4>(a, C, grid, block, s);
    return static_cast<int>(e);
}

}  // namespace nvfp4
