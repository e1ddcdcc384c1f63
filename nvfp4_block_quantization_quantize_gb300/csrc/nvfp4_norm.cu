// nvfp4_norm.cu -- residual addition, root-mean-square norm and quantization
// of its output in one pass (nvfp4_rmsnorm).
//
// Per row, fp32: h = x + hidden, y = (h * rsqrt(mean(h^2) + eps)) * weight, then y to
// NVFP4 (e2m1 codes, one E4M3 scale per 16) or MXFP8 (E4M3 elements, one E8M0
// scale per 32).  Each element is read once and each result written once, about
// ten operations an element: the kernel is bound by memory (by latency for a few
// rows).  A row belongs to one CTA: a thread holds a block of 16 elements in
// registers from the load to the stores, so nothing is read twice; rows of over
// 1024 blocks are read a second time instead.
// Measured, in a graph of calls: 16384 x 4096 bf16 with the residual, MXFP8 out, 73 us (6.45 TB/s,
// 0.95 of the copy rate), NVFP4 out 79 us, with row amaxes 108 us (y is made twice, and the row
// reduced twice); 1 x 4096 2.2 us; 2048 x 20480 79 us (read twice), with the residual 87.
#include "nvfp4_block.cuh"

namespace nvfp4 {
namespace {

constexpr int kNormMaxThreads = 1024;

// 32 bytes of memory.  W: the address is 32-byte aligned (one 256-bit access: a warp's
// 16-element blocks of bf16 are then one contiguous piece).  RO: through the read-only
// path; the hidden state, which this kernel may write in place, is not.
template <bool W, bool RO>
__device__ __forceinline__ void load32(const void* p, uint32_t* w) {
    if constexpr (W) {
        if constexpr (RO)
            asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                         : "l"(p));
        else
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                         : "l"(p)
                         : "memory");
    } else {
        const uint4* q = static_cast<const uint4*>(p);
        const uint4 a = RO ? __ldg(q) : q[0], b = RO ? __ldg(q + 1) : q[1];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
}

template <bool W>
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
    if constexpr (W)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    else {
        uint4* q = static_cast<uint4*>(p);
        q[0] = make_uint4(w[0], w[1], w[2], w[3]);
        q[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// 16 elements from element elem0, as they are (8 words of bf16, 16 of fp32)
template <int DT>
constexpr int kWords = DT == NVFP4_BF16 ? 8 : 16;

template <int DT, bool W, bool RO>
__device__ __forceinline__ void load_raw(const void* base, int64_t elem0, uint32_t* w) {
    const uint8_t* p = static_cast<const uint8_t*>(base) + elem0 * (DT == NVFP4_BF16 ? 2 : 4);
    load32<W, RO>(p, w);
    if (DT == NVFP4_F32) load32<W, RO>(p + 32, w + kWords<DT> - 8);
}

template <int DT>
__device__ __forceinline__ void widen(const uint32_t* w, float* y) {
#pragma unroll
    for (int i = 0; i < kWords<DT>; ++i) {
        if (DT == NVFP4_BF16) {
            y[2 * i] = __uint_as_float(w[i] << 16);
            y[(2 * i + 1) % 16] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            y[i] = __uint_as_float(w[i]);
        }
    }
}

template <int DT, bool W>
__device__ __forceinline__ void store16(void* base, int64_t elem0, const float* y) {
    uint8_t* p = static_cast<uint8_t*>(base) + elem0 * (DT == NVFP4_BF16 ? 2 : 4);
    uint32_t w[kWords<DT>];
#pragma unroll
    for (int i = 0; i < kWords<DT>; ++i) {
        if (DT == NVFP4_BF16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[(2 * i + 1) % 16]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        } else {
            w[i] = __float_as_uint(y[i]);
        }
    }
    store32<W>(p, w);
    if (DT == NVFP4_F32) store32<W>(p + 32, w + kWords<DT> - 8);
}

// x (+ hidden) of 16 elements as loaded
template <int DT>
struct Raw {
    uint32_t x[kWords<DT>], r[kWords<DT>];
};

template <int DT, bool W>
__device__ __forceinline__ void load_block(const NormArgs& a, int64_t elem0, Raw<DT>& raw) {
    load_raw<DT, W, true>(a.x, elem0, raw.x);
    if (a.hidden) load_raw<DT, W, false>(a.hidden, elem0, raw.r);
}

// h = x + hidden
template <int DT>
__device__ __forceinline__ void sum_block(const NormArgs& a, const Raw<DT>& raw, float* h) {
    widen<DT>(raw.x, h);
    if (a.hidden) {
        float r[16];
        widen<DT>(raw.r, r);
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

// blockDim (threads per row, rows per CTA).  C == 1: a thread holds its block of 16 in
// registers; the CTA walks down the rows, the next row's loads under way while the present
// one is reduced and stored.  C == 0: a thread walks along a row, which is read a second
// time.  W: every row starts on 32 bytes.  MAXT: rows of at most 512 threads have the
// registers to hold the next row in fp32 too, as one CTA an SM (4096 x 7168: 32 us, two
// CTAs that spill 38 us, without the next row 56 us); bf16 is held to 64, for three and more
// (16384 x 4096 with hidden: 73 us; with 104 registers and fewer CTAs 77 us).
template <int DT, int C, int FMT, bool W, int MAXT>
__global__ void __launch_bounds__(MAXT, DT == NVFP4_BF16 && MAXT == 512 ? 2 : 1) k_rmsnorm(const NormArgs a) {
    __shared__ float ssum[2][32], smax[2][32];
    pdl_trigger();                                        // the next kernel waits for this one's end itself
    pdl_wait();
    const int64_t bpr = a.K / 16;
    const int64_t T = blockDim.x;
    const int64_t hop = static_cast<int64_t>(gridDim.x) * blockDim.y;
    int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    // threads of a pair stay together: every thread makes the same number of steps
    const int64_t steps = C ? 1 : (bpr + T - 1) / T;
    constexpr bool kAhead = C == 1 && (DT == NVFP4_BF16 || MAXT == 512);     // fp32 of 1024 threads would spill
    Raw<DT> raw;
    auto load = [&](int64_t r, int64_t c) {
        const int64_t blk = threadIdx.x + c * T;
        if (r < a.M && blk < bpr) load_block<DT, W>(a, (r * bpr + blk) * 16, raw);
    };
    auto value = [&](int64_t r, int64_t c, float* h) {
        if (r < a.M && threadIdx.x + c * T < bpr) sum_block<DT>(a, raw, h);
        else
#pragma unroll
            for (int i = 0; i < 16; ++i) h[i] = 0.0f;
    };
    if (kAhead) load(row, 0);
    int turn = 0;                                         // of the reductions' slots
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.y; first < a.M; first += hop, row += hop, turn ^= 1) {
        const bool in = row < a.M;
        float h[16], sum = 0.0f;
        for (int64_t c = 0; c < steps; ++c) {
            if (!kAhead) load(row, c);
            value(row, c, h);
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) s = __fmaf_rn(h[i], h[i], s);
            sum = add_rn(sum, s);
        }
        if (kAhead) load(row + hop, 0);
        const float mean = div_rn(row_reduce<false>(sum, ssum[turn]), static_cast<float>(a.K));
        const float rstd = div_rn(1.0f, __fsqrt_rn(add_rn(mean, a.eps)));
        GScale g{0.0f, 1.0f, 1.0f};
        if (FMT == NVFP4_FMT_NVFP4 && a.codes && a.gamax_mode != NVFP4_GAMAX_NONE) {
            if (a.gamax_mode == NVFP4_GAMAX_ROW) {
                float m = 0.0f;
                for (int64_t c = 0; c < steps; ++c) {
                    const int64_t blk = threadIdx.x + c * T;
                    if (!C) {
                        load(row, c);
                        value(row, c, h);
                    }
                    if (!in || blk >= bpr) continue;
                    float y[16];
                    normed(a, blk * 16, rstd, h, y);
                    m = max_nd(m, absmax16(y));
                }
                g.A = row_reduce<true>(m, smax[turn]);
                if (in && threadIdx.x == 0) a.gamax[row] = g.A;
            } else if (in) {
                g.A = a.gamax[a.gamax_mode == NVFP4_GAMAX_ROW_GIVEN ? row : 0];
            }
            global_scales(g.A, a.bound, g.Senc, g.Sdec);
        }
        for (int64_t c = 0; c < steps; ++c) {
            const int64_t blk = threadIdx.x + c * T;
            if (!C) {
                load(row, c);
                value(row, c, h);
            }
            const bool live = in && blk < bpr;
            float y[16];
            if (live) {
                if (a.hidden_out) store16<DT, W>(a.hidden_out, (row * bpr + blk) * 16, h);
                normed(a, blk * 16, rstd, h, y);
                if (a.out) store16<DT, W>(a.out, (row * bpr + blk) * 16, y);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = 0.0f;
            }
            if (a.codes) quantize16<FMT>(a, row, blk, bpr, live, g, y);
        }
    }
}

template <int DT, int FMT, bool W>
cudaError_t launch_norm_t(const NormArgs& a, cudaStream_t s) {
    const int64_t bpr = a.K / 16;
    const bool whole = bpr <= kNormMaxThreads;
    const int T = whole ? static_cast<int>((bpr + 31) / 32 * 32) : kNormMaxThreads;
    const int rows = T >= 256 ? 1 : 256 / T;
    auto* kernel = T * rows <= 512 ? k_rmsnorm<DT, 1, FMT, W, 512>
                   : whole         ? k_rmsnorm<DT, 1, FMT, W, kNormMaxThreads>
                                   : k_rmsnorm<DT, 0, FMT, W, kNormMaxThreads>;
    // as many CTAs as run at once, found once per device, variant and CTA size (8 of 32 .. 256 threads a
    // row have 256 a CTA; above, one size each)
    static thread_local int dev_of = -1, at_once[2][33];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev_of != dev) {
        for (auto& v : at_once)
            for (int& n : v) n = 0;
        dev_of = dev;
    }
    int& n = at_once[whole][T * rows / 32];
    if (n == 0) {
        int per_sm = 0;
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, T * rows, 0);
        if (e != cudaSuccess) return e;
        n = (per_sm < 1 ? 1 : per_sm) * sm_count();
    }
    const int64_t blocks = (a.M + rows - 1) / rows;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks < n ? blocks : n)), dim3(T, rows), 0, s, a);
}

template <int DT, int FMT>
cudaError_t launch_norm_w(const NormArgs& a, cudaStream_t s) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.hidden) |
                           reinterpret_cast<uintptr_t>(a.hidden_out) | reinterpret_cast<uintptr_t>(a.out);
    return bits % 32 == 0 ? launch_norm_t<DT, FMT, true>(a, s) : launch_norm_t<DT, FMT, false>(a, s);
}

}  // namespace

int launch_rmsnorm(const NormArgs& a, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool mx = a.format == NVFP4_FMT_MXFP8;
    if (a.dtype == NVFP4_BF16)
        return static_cast<int>(mx ? launch_norm_w<NVFP4_BF16, NVFP4_FMT_MXFP8>(a, s)
                                   : launch_norm_w<NVFP4_BF16, NVFP4_FMT_NVFP4>(a, s));
    return static_cast<int>(mx ? launch_norm_w<NVFP4_F32, NVFP4_FMT_MXFP8>(a, s)
                               : launch_norm_w<NVFP4_F32, NVFP4_FMT_NVFP4>(a, s));
}

}  // namespace nvfp4
