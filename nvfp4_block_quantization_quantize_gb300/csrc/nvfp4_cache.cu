// nvfp4_cache.cu -- the heads of new tokens on their way to attention: norms of
// queries and keys, their rotation, and keys and values quantized into a paged NVFP4
// cache (nvfp4_qk_norm_rope, nvfp4_cache_write), and the cache read back
// (nvfp4_cache_read).
//
// Per head of D elements, fp32: y = x * rsqrt(mean(x^2) + eps) * w, then pairs (a, b) of
// its first rotary_dim elements turn to m (a cos t - b sin t, b cos t + a sin t), t = 2 pi *
// position * phase / 2^64.  The phase is a whole number of 2^-64 turns, so position * phase wraps
// exactly where whole turns drop out: a far position loses nothing (the angle's error is the
// phase's rounding times the position, 2^-65 turns each).  Of the turn left whole quarters drop out exactly too, and
// the rest is rounded to fp32: sines and cosines next to zero keep their relative accuracy.
// Each element is read once and written once, ten to twenty operations each:
// bound by memory, by latency for a few tokens.
//   - A thread holds 16 elements of a head: 8 pairs.  With the pairs' halves apart (half layout) they
//     are 8 elements of each half, else 16 in a row, so that no pair crosses threads.
//   - A group of 4 to 32 threads holds a head; a warp takes heads of one token, so that the 8
//     angles of a thread serve all of them, and loads the next while it works on one.
//   - A block of 16 to quantize is a thread's own, or (half layout) made by exchanging 8 elements with the
//     neighbouring thread: the even one quantizes the first half's block, the odd one the second's.
#include "nvfp4_block.cuh"

namespace nvfp4 {
namespace {

constexpr int kHeadsThreads = 256;

// 8 elements from element e, as they are
template <int DT>
constexpr int kRaw8 = DT == NVFP4_BF16 ? 4 : 8;

template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t e, uint32_t* w) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + e * (DT == NVFP4_BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < kRaw8<DT> / 4; ++i) {
        const uint4 u = __ldg(p + i);
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
}

template <int DT>
__device__ __forceinline__ void widen8(const uint32_t* w, float* y) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (DT == NVFP4_BF16) y[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        else y[i] = __uint_as_float(w[i % kRaw8<DT>]);
    }
}

template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t e, const float* y) {
    uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(base) + e * (DT == NVFP4_BF16 ? 2 : 4));
    uint32_t w[kRaw8<DT>];
#pragma unroll
    for (int i = 0; i < kRaw8<DT>; ++i) {
        if (DT == NVFP4_BF16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i % 8], y[(2 * i + 1) % 8]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        } else {
            w[i] = __float_as_uint(y[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kRaw8<DT> / 4; ++i) p[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

__device__ __forceinline__ void load_weight8(const void* base, int dtype, int e, float* y) {
    uint32_t w[8];
    if (dtype == NVFP4_BF16) {
        load8<NVFP4_BF16>(base, e, w);
        widen8<NVFP4_BF16>(w, y);
    } else {
        load8<NVFP4_F32>(base, e, w);
        widen8<NVFP4_F32>(w, y);
    }
}

// amax of KV head h (1 without a global scale, whose encode and decode scales are 1)
__device__ __forceinline__ GScale head_scale(int mode, const float* gamax, int h, float bound) {
    GScale g{0.0f, 1.0f, 1.0f};
    if (mode != NVFP4_GAMAX_NONE) {
        g.A = __ldg(gamax + (mode == NVFP4_GAMAX_ROW_GIVEN ? h : 0));
        global_scales(g.A, bound, g.Senc, g.Sdec);
    }
    return g;
}

// Where a slot lies: its page's first byte plus its tile's place there, for head 0 (null: there is no such slot), and its row
// of the tile.
struct Place {
    uint8_t* tile;
    int row;
};

__device__ __forceinline__ Place place_of(const CacheArgs& c, int64_t s) {
    if (s < 0 || s >= c.pages * c.page_size) return {nullptr, 0};
    int64_t page;                                         // (a 64-bit division costs more than a block's quantization)
    if (s >> 31 == 0) page = static_cast<uint32_t>(s) / static_cast<uint32_t>(c.page_size);
    else page = s / c.page_size;
    const int in = static_cast<int>(s - page * c.page_size);
    return {c.data + (page * c.Hkv * (c.page_size / 16) + in / 16) * (18 * c.D), in % 16};
}

__device__ __forceinline__ int64_t head_bytes(const CacheArgs& c) { return static_cast<int64_t>(c.page_size / 16) * (18 * c.D); }

// 16 elements from element e of the row that slot s is, as nvfp4_quantize quantizes them
__device__ __forceinline__ void quantize_into(uint8_t* part, int row, int D, int e, const GScale& g, const float* y) {
    const float own = absmax16(y);
    const uint32_t sf = e4m3_encode(min_nd(block_s6f<true>(own, g.Senc), 448.0f));
    const float d = mul_rn(e4m3_decode(sf), g.Sdec);
    uint32_t w0, w1;
    float none[1];
    PhiloxKeys keys;                                        // nearest rounding draws nothing
    encode_plain16<NVFP4_RTN>(y, d, own, 0, keys, w0, w1, nullptr, sf, none, false);
    *reinterpret_cast<uint2*>(part + row * (D / 2) + e / 2) = make_uint2(w0, w1);
    part[8 * D + row * (D / 16) + e / 16] = static_cast<uint8_t>(sf);
}

// L threads a head.  A token's heads (q, k, then v when they go to the cache) are cut into
// `chunks` of `per` heads, one a warp.  TURN: norms and rotation, of pairs half the rotated elements apart (HALF) or of
// neighbours; CACHE: k and v go to the cache.
// Registers for as many warps as keep memory busy: 64 a thread without a cache or a turn (bf16), 80 with both.
// Measured, 16384 bf16 tokens: 32 + 8 heads of 128 turned 65 us, 5.2 TB/s (201 us with the layout read at run time); 8 + 8 heads
// quantized and read back 40 us for the two kernels (a thread a block in k_cache_read, its place found for each: 67 us).
enum Turn { kNoTurn, kHalf, kNeighbours };

template <int DT, int L, Turn TURN, bool CACHE>
__global__ void __launch_bounds__(kHeadsThreads, DT == NVFP4_BF16 && !(TURN != kNoTurn && CACHE) ? 4 : 3) k_heads(const HeadsArgs a, int chunks, int per) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, t = lane % L, sub = lane / L;
    const uint32_t warp = blockIdx.x * (kHeadsThreads / 32) + (threadIdx.x >> 5);      // (several chunks: few tokens)
    const int64_t token = warp / static_cast<uint32_t>(chunks);
    if (token >= a.T) return;                               // whole warps
    const int first = static_cast<int>(warp % static_cast<uint32_t>(chunks)) * per;
    const int nq = a.q ? a.Hq : 0, total = nq + (a.k ? a.Hkv : 0) + (a.v ? a.Hkv : 0);
    const int end = min(first + per, total);
    const bool live = t < a.D / 16;
    const bool turned = TURN != kNoTurn && t < a.rotary_dim / 16;
    const bool apart = TURN == kHalf && turned;
    const int half = a.rotary_dim / 2;

    float cs[8], sn[8];
    if (TURN != kNoTurn && turned && first < nq + a.Hkv) {
        const uint64_t pos = static_cast<uint64_t>(__ldg(a.positions + token));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t turn = pos * __ldg(reinterpret_cast<const unsigned long long*>(a.phases) + 8 * t + i);
            // whole quarters of a turn drop out exactly; what is left, at most 1/8 turn, in fp32: its nearest whole number of 2^32
            // and the rest of that, each rounded by 2^-24 at most (a conversion of 64 bits takes longer: a token 3.08 us)
            const uint64_t quarter = (turn + (1ull << 61)) >> 62, left = turn - (quarter << 62);
            const float high = static_cast<float>(static_cast<int32_t>((left + 0x80000000ull) >> 32));
            const float low = static_cast<float>(static_cast<int32_t>(left));
            float s0, c0;
            sincospif(mul_rn(__fmaf_rn(high, 4294967296.0f, low), 1.0842021724855044e-19f), &s0, &c0);      // 2^-63: in half turns
            const float sine = quarter & 1 ? c0 : s0, cosine = quarter & 1 ? s0 : c0;
            const uint32_t q = static_cast<uint32_t>(quarter);
            const uint32_t sine_down = q << 30 & 0x80000000u, cosine_down = (q + 1) << 30 & 0x80000000u;      // their sign bits
            cs[i] = mul_rn(__uint_as_float(__float_as_uint(cosine) ^ cosine_down), a.magnitude);
            sn[i] = mul_rn(__uint_as_float(__float_as_uint(sine) ^ sine_down), a.magnitude);
        }
    }
    Place place{nullptr, 0};
    if (CACHE) place = place_of(a.cache, __ldg(a.slots + token));

    // Where a thread's elements of a head lie: e0 .. e0 + 7 and e1 .. e1 + 7 (v has no pairs).  A token's heads are one
    // after the other.
    const int e0_qk = apart ? 8 * t : 16 * t, e1_qk = apart ? half + 8 * t : 16 * t + 8;
    constexpr int kSize = DT == NVFP4_BF16 ? 2 : 4;
    const uint8_t* const q_in = static_cast<const uint8_t*>(a.q) + token * a.q_stride * kSize;
    const uint8_t* const k_in = static_cast<const uint8_t*>(a.k) + token * a.k_stride * kSize;
    const uint8_t* const v_in = static_cast<const uint8_t*>(a.v) + token * a.v_stride * kSize;
    const int nk = nq + (a.k ? a.Hkv : 0);                // the first head of v
    uint32_t raw[2 * kRaw8<DT>];
    auto load = [&](int j) {
        if (j >= end || !live) return;
        const bool is_v = CACHE && j >= nk;
        const uint8_t* const head = j < nq ? q_in + j * a.D * kSize : is_v ? v_in + (j - nk) * a.D * kSize : k_in + (j - nq) * a.D * kSize;
        load8<DT>(head, is_v ? 16 * t : e0_qk, raw);
        load8<DT>(head, is_v ? 16 * t + 8 : e1_qk, raw + kRaw8<DT>);
    };
    load(first + sub);
    for (int j0 = first; j0 < end; j0 += 32 / L) {
        const int j = j0 + sub;
        const bool in = j < end && live;
        const bool is_q = j < nq, is_v = CACHE && j >= nk;
        const int e0 = is_v ? 16 * t : e0_qk, e1 = is_v ? 16 * t + 8 : e1_qk;
        float y[16];
        if (in) {
            widen8<DT>(raw, y);
            widen8<DT>(raw + kRaw8<DT>, y + 8);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = 0.0f;
        }
        load(j + 32 / L);
        if (TURN != kNoTurn && a.q_weight) {                // the sums of all of the warp's heads
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) s = __fmaf_rn(y[i], y[i], s);
#pragma unroll
            for (int o = L / 2; o; o >>= 1) s = add_rn(s, __shfl_xor_sync(kFullMask, s, o));
            if (!is_v && in) {
                const void* const weight = is_q ? a.q_weight : a.k_weight;
                const float rstd = __frsqrt_rn(add_rn(div_rn(s, static_cast<float>(a.D)), a.eps));
                float w[8];
                load_weight8(weight, a.weight_dtype, e0, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = mul_rn(mul_rn(y[i], rstd), w[i]);
                load_weight8(weight, a.weight_dtype, e1, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i + 8] = mul_rn(mul_rn(y[i + 8], rstd), w[i]);
            }
        }
        if (TURN != kNoTurn && turned && !is_v) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                constexpr bool kApart = TURN == kHalf;
                const int p = kApart ? i : 2 * i, q = kApart ? i + 8 : 2 * i + 1;
                const float u = y[p], v = y[q];
                y[p] = __fmaf_rn(u, cs[i], -mul_rn(v, sn[i]));
                y[q] = __fmaf_rn(v, cs[i], mul_rn(u, sn[i]));
            }
        }
        if (in && (is_q || !CACHE)) {
            uint8_t* const out = static_cast<uint8_t*>(is_q ? a.q_out : a.k_out) +
                                 (token * (is_q ? a.Hq : a.Hkv) + (is_q ? j : j - nq)) * a.D * kSize;
            store8<DT>(out, e0, y);
            store8<DT>(out, e1, y + 8);
        }
        if (CACHE) {
            int e = e0;
            const int h = j - (is_v ? nk : nq);
            if (TURN == kHalf) {       // blocks of 16 from two neighbours' halves
                const bool odd = t & 1;
                float got[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) got[i] = __shfl_xor_sync(kFullMask, odd ? y[i] : y[i + 8], 1);
                if (apart && !is_v) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        y[i] = odd ? got[i] : y[i];
                        y[i + 8] = odd ? y[i + 8] : got[i];
                    }
                    e = odd ? half + 8 * (t - 1) : 8 * t;
                }
            }
            if (in && !is_q && place.tile) {
                uint8_t* const tile = place.tile + h * head_bytes(a.cache);
                const GScale g = is_v ? head_scale(a.cache.v_mode, a.cache.v_gamax, h, a.cache.bound)
                                      : head_scale(a.cache.k_mode, a.cache.k_gamax, h, a.cache.bound);
                quantize_into(tile + (is_v ? 9 * a.D : 0), place.row, a.D, e, g, y);
            }
        }
    }
}

// A warp takes part of a slot's blocks of 16 elements, keys first, then values, a thread a block: 8 bytes of codes and a
// scale to 16 values (zeros where there is no such slot): bound by memory.  LG: log2 of the blocks of a head.
template <int ODT, int LG>
__global__ void __launch_bounds__(256) k_cache_read(const CacheReadArgs a, int chunks) {
    pdl_trigger();
    pdl_wait();
    const CacheArgs& c = a.cache;
    const uint32_t warp = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t token = warp / static_cast<uint32_t>(chunks);
    if (token >= a.T) return;
    const int chunk = static_cast<int>(warp % static_cast<uint32_t>(chunks)), half = c.Hkv << LG;
    const Place place = place_of(c, __ldg(a.slots + token));
    const bool wide = (reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) % 32 == 0;
    for (int i = chunk * 32 + (threadIdx.x & 31); i < 2 * half; i += chunks * 32) {
        const bool is_v = i >= half;
        const int x = is_v ? i - half : i, h = x >> LG, grp = x & ((1 << LG) - 1);
        void* const out = is_v ? a.v : a.k;
        if (!out) continue;
        float y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = 0.0f;
        if (place.tile) {
            const uint8_t* part = place.tile + h * head_bytes(c) + (is_v ? 9 * c.D : 0);
            const uint2 w = *reinterpret_cast<const uint2*>(part + place.row * (c.D / 2) + grp * 8);
            const float d = e4m3_decode(part[8 * c.D + (place.row << LG) + grp]);
            const GScale g = is_v ? head_scale(c.v_mode, c.v_gamax, h, c.bound) : head_scale(c.k_mode, c.k_gamax, h, c.bound);
            dequant16<true>(w.x, w.y, d, g.Sdec, y);
        }
        uint8_t* const to = static_cast<uint8_t*>(out) + (token * half + x) * (ODT == NVFP4_BF16 ? 32 : 64);
        uint32_t w[ODT == NVFP4_BF16 ? 8 : 16];
        if (ODT == NVFP4_BF16) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&v);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j % (ODT == NVFP4_BF16 ? 8 : 16)] = __float_as_uint(y[j]);
        }
#pragma unroll
        for (int j = 0; j < (ODT == NVFP4_BF16 ? 8 : 16); j += 8) store32(to + 4 * j, w + j, wide);
    }
}

template <int DT>
cudaError_t launch_heads_t(const HeadsArgs& a, cudaStream_t s) {
    const int groups = a.D / 16, L = groups <= 4 ? 4 : groups <= 8 ? 8 : groups <= 16 ? 16 : 32;
    const int total = (a.q ? a.Hq : 0) + (a.k ? a.Hkv : 0) + (a.v ? a.Hkv : 0), step = 32 / L;
    // few tokens: a warp takes one round of heads, so that all run at once
    const int rounds = (total + step - 1) / step;
    const int64_t warps = static_cast<int64_t>(sm_count()) * 16;
    int64_t chunks = a.T >= warps ? 1 : (warps + a.T - 1) / a.T;
    if (chunks > rounds) chunks = rounds;
    const int per = (rounds + static_cast<int>(chunks) - 1) / static_cast<int>(chunks) * step;
    chunks = (total + per - 1) / per;
    const int64_t blocks = (a.T * chunks + kHeadsThreads / 32 - 1) / (kHeadsThreads / 32);
    const bool cache = a.slots != nullptr;
    const dim3 grid(static_cast<unsigned>(blocks));
    const int n = static_cast<int>(chunks);
    auto go = [&](auto* kernel) { return launch_pdl(kernel, grid, dim3(kHeadsThreads), 0, s, a, n, per); };
    const bool apart = a.layout == NVFP4_ROPE_HALF;         // (norms alone: whichever)
    if (!a.q && !a.positions && !a.k_weight && cache)       // nvfp4_cache_write
        return L == 4 ? go(k_heads<DT, 4, kNoTurn, true>) : L == 8 ? go(k_heads<DT, 8, kNoTurn, true>) : go(k_heads<DT, 16, kNoTurn, true>);
    if (cache && apart) return L == 4 ? go(k_heads<DT, 4, kHalf, true>) : L == 8 ? go(k_heads<DT, 8, kHalf, true>) : go(k_heads<DT, 16, kHalf, true>);
    if (cache)
        return L == 4 ? go(k_heads<DT, 4, kNeighbours, true>) : L == 8 ? go(k_heads<DT, 8, kNeighbours, true>) : go(k_heads<DT, 16, kNeighbours, true>);
    if (apart)
        return L == 4 ? go(k_heads<DT, 4, kHalf, false>) : L == 8 ? go(k_heads<DT, 8, kHalf, false>)
               : L == 16 ? go(k_heads<DT, 16, kHalf, false>) : go(k_heads<DT, 32, kHalf, false>);
    return L == 4 ? go(k_heads<DT, 4, kNeighbours, false>) : L == 8 ? go(k_heads<DT, 8, kNeighbours, false>)
           : L == 16 ? go(k_heads<DT, 16, kNeighbours, false>) : go(k_heads<DT, 32, kNeighbours, false>);
}

}  // namespace

int launch_heads(const HeadsArgs& a, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return static_cast<int>(a.dtype == NVFP4_BF16 ? launch_heads_t<NVFP4_BF16>(a, s) : launch_heads_t<NVFP4_F32>(a, s));
}

int launch_cache_read(const CacheReadArgs& a, void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // few slots: a warp takes one round of blocks, so that all run at once
    const int rounds = (2 * a.cache.Hkv * (a.cache.D / 16) + 31) / 32;
    const int64_t warps = static_cast<int64_t>(sm_count()) * 32;
    int64_t chunks = a.T >= warps ? 1 : (warps + a.T - 1) / a.T;
    if (chunks > rounds) chunks = rounds;
    const dim3 grid(static_cast<unsigned>((a.T * chunks + 7) / 8));
    auto go = [&](auto* kernel) { return static_cast<int>(launch_pdl(kernel, grid, dim3(256), 0, s, a, static_cast<int>(chunks))); };
    if (a.out_dtype == NVFP4_BF16)
        return a.cache.D == 64 ? go(k_cache_read<NVFP4_BF16, 2>) : a.cache.D == 128 ? go(k_cache_read<NVFP4_BF16, 3>) : go(k_cache_read<NVFP4_BF16, 4>);
    return a.cache.D == 64 ? go(k_cache_read<NVFP4_F32, 2>) : a.cache.D == 128 ? go(k_cache_read<NVFP4_F32, 3>) : go(k_cache_read<NVFP4_F32, 4>);
}

}  // namespace nvfp4
