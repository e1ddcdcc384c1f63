// nvfp4_tensor.cuh -- the tcgen05 / TMA building blocks the FP4 products share:
// shared-memory and instruction descriptors of tcgen05.mma .kind::mxf4nvf4,
// mbarriers with bounded waits, TMA and bulk copies, the code matrices' maps.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "nvfp4_params.h"

namespace nvfp4 {

constexpr long kWaitLimit = 1L << 22;                     // try_wait rounds before giving up

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// shared-memory matrix descriptor, K-major: lbo = byte step between core
// matrices along K, sbo = between 8-row groups along M/N; layout 0 = no
// swizzle (core matrices of 8 rows x 16 bytes), 2 = 128-byte swizzle (rows
// of 128 bytes, 8-row atoms of 1 KB, 1 KB-aligned)
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t layout = 0) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32;
    d |= 1ull << 46;                                      // descriptor version for sm_100 family
    d |= static_cast<uint64_t>(layout & 7u) << 61;        // base offset 0
    return d;
}

// instruction descriptor for .kind::mxf4nvf4: A and B e2m1 (format 1), both
// K-major, E4M3 scales, scale-factor ids 0, N >> 3 and M >> 4
__device__ __forceinline__ uint32_t instr_desc(int M, int N) {
    uint32_t d = 0;
    d |= 1u << 7;                                         // A format: e2m1
    d |= 1u << 10;                                        // B format: e2m1
    d |= static_cast<uint32_t>(N >> 3) << 17;
    d |= static_cast<uint32_t>(M >> 4) << 24;
    return d;
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t arrivals = 1) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(arrivals));
}

__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity) {
    for (long it = 0; it < kWaitLimit; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return false;
}

// A CTA one of whose waits ran out calls this before it ends: the copies it has issued take microseconds, and are
// in after the millisecond this sleeps.
__device__ __forceinline__ void settle() {
    for (int i = 0; i < 1024; ++i) __nanosleep(1000);
}

// decode scale S_dec = 1 / min(6 * bound / A, FLT_MAX) of a per-tensor amax
// (1 without one, and when A is not a positive finite number)
__device__ __forceinline__ float decode_scale(const float* gamax, float bound) {
    if (!gamax) return 1.0f;
    const float A = *gamax;
    const float enc = (!(A > 0.0f) || isinf(A)) ? 1.0f : fminf(__fdiv_rn(__fmul_rn(6.0f, bound), A), 3.4028234663852886e+38f);
    return __fdiv_rn(1.0f, enc);
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void mma_f4(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc));
}

// ---- issue by a whole warp ---------------------------------------------------------------------
// The forms above are issued by one thread under a branch; the compiler then moves
// each operand to a uniform register per instruction, and issuing costs about 45
// clocks an instruction (measured: 128 x 128 x 64 products with two scale copies
// each take 134 clocks apart instead of 92).  Here the whole warp comes along with
// the same operands and one elected lane's predicate guards the instruction.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}

// CG: CTAs of the product (1, or the 2 SMs of a pair: M up to 256)
template <int CG>
__device__ __forceinline__ void mma_f4_warp(uint32_t el, uint32_t d, uint64_t da, uint64_t db, uint32_t idesc,
                                            uint32_t sfa, uint32_t sfb, uint32_t acc) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "setp.ne.b32 q, %7, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(da), "l"(db), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc), "r"(el));
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "setp.ne.b32 q, %7, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(da), "l"(db), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc), "r"(el));
}

// a 512-byte scale tile to four tensor-memory columns
template <int CG>
__device__ __forceinline__ void copy_scales_warp(uint32_t el, uint32_t col, uint64_t desc) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(col), "l"(desc), "r"(el));
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(col), "l"(desc), "r"(el));
}

// arrive on bar (with CG == 2 in both CTAs of the pair) when the products issued so far are done
template <int CG>
__device__ __forceinline__ void commit_warp(uint32_t el, uint64_t* bar) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
            "r"(el)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}" ::"r"(
                smem_addr(bar)),
            "r"(el), "h"(static_cast<uint16_t>(3))
            : "memory");
}

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    if (!encode) {
        cudaDriverEntryPointQueryResult q;
        PFN_cuTensorMapEncodeTiled_v12000 f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", reinterpret_cast<void**>(&f), 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            encode = f;
    }
    return encode;
}

// 2D map of a [rows, K/2]-byte code matrix, boxes of box_rows x 128 bytes, 128-byte swizzle
inline bool encode_codes_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t K, int box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
    const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the same with two neighbouring pieces of 128 bytes of each row a box ([2][box_rows][128], each
// piece swizzled as above); the columns past the last whole piece are left out
inline bool encode_codes_map2(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t K, int box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return false;
    const cuuint64_t pieces = K < 256 ? 1 : static_cast<cuuint64_t>(K / 256);
    const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(rows), pieces};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(K / 2), 128};
    const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(box_rows), 2};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(codes), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2D map of a bf16 output [rows, N], N % 8 == 0: boxes of 32 rows x 32 columns, 64-byte swizzle
inline bool encode_out_map(CUtensorMap* map, void* out, int64_t rows, int64_t N) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(N) * 2};
    const cuuint32_t box[2] = {32, 32};
    const cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// 2D map of `tiles` 512-byte scale tiles, boxes of box_tiles of them
inline bool encode_scales_map(CUtensorMap* map, const uint8_t* scales, int64_t tiles, int box_tiles) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return false;
    const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(tiles)};
    const cuuint64_t strides[1] = {512};
    const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_tiles)};
    const cuuint32_t estr[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(scales), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace nvfp4
