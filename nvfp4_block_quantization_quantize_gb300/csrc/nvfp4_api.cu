// nvfp4_api.cu -- the C ABI declared in include/nvfp4.h.
//
// Host side only: argument checks (nothing is enqueued when one fails), the
// optional global-amax pass, and the choice of kernel.  No allocation, no
// synchronization; everything runs on the caller's stream.
#include <cstdarg>
#include <cstdio>
#include <cstdint>

#include <cuda_runtime.h>

#include "nvfp4_params.h"

namespace {

thread_local char g_msg[512] = "";

int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
    va_end(ap);
    return code;
}

int cuda_fail(int err, const char* what) {
    return fail(NVFP4_ECUDA, "%s: %s", what, cudaGetErrorString(static_cast<cudaError_t>(err)));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_ptr(const void* p, const char* name, bool required, uintptr_t align = 16) {
    if (!p) return required ? fail(NVFP4_EINVAL, "%s must not be NULL", name) : NVFP4_OK;
    if (!aligned(p, align)) return fail(NVFP4_EINVAL, "%s must be %d-byte aligned", name, int(align));
    return NVFP4_OK;
}

int check_shape(int64_t M, int64_t K) {
    if (M < 0 || K < 0) return fail(NVFP4_EINVAL, "M and K must be >= 0 (got %lld, %lld)",
                                    (long long)M, (long long)K);
    if (K % 16 != 0) return fail(NVFP4_EINVAL, "K must be a multiple of 16 (got %lld)", (long long)K);
    if (K > 0 && M > INT64_MAX / 4 / K) return fail(NVFP4_EINVAL, "M*K is too large");
    if (M >= (int64_t{1} << 35) || K >= (int64_t{1} << 35))
        return fail(NVFP4_EINVAL, "M and K must each be below 2^35");
    return NVFP4_OK;
}

// A buffer of a call, for check_apart.
struct Buffer {
    const void* p;            // null = not given
    uint64_t bytes;
    const char* name;
};

bool overlap(const Buffer& a, const Buffer& b) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.p), q = reinterpret_cast<uintptr_t>(b.p);
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    return p <= q ? q - p < a.bytes : p - q < b.bytes;
}

// No output shares a byte with an input or another output: CTAs read their inputs while
// others store, and through the read-only path.
template <int NO, int NI>
int check_apart(const Buffer (&outs)[NO], const Buffer (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (const Buffer& in : ins)
            if (overlap(outs[i], in)) return fail(NVFP4_EINVAL, "%s must not overlap %s", outs[i].name, in.name);
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return fail(NVFP4_EINVAL, "%s must not overlap %s", outs[i].name, outs[j].name);
    }
    return NVFP4_OK;
}

bool is_row_mode(int g) { return g == NVFP4_GAMAX_ROW || g == NVFP4_GAMAX_ROW_GIVEN; }

// Largest K with a columnwise output: 65535 CTA columns of 256 (1x16 row-owner
// kernel; the tile kernels cover 512 columns per CTA column).
constexpr int64_t kMaxColwiseK = 65535LL * 256;

// Checks shared by quantize and qdq.
int check_quant(const void* x, int64_t M, int64_t K, int dtype, int block, int rounding,
                const float* residual, int gamax_mode, const float* gamax, int err_mode,
                float bound, bool colwise) {
    int rc = check_shape(M, K);
    if (rc) return rc;
    if (dtype != NVFP4_F32 && dtype != NVFP4_BF16) return fail(NVFP4_EINVAL, "bad dtype %d", dtype);
    if (block != NVFP4_BLOCK_1X16 && block != NVFP4_BLOCK_16X16) return fail(NVFP4_EINVAL, "bad block %d", block);
    if (rounding != NVFP4_RTN && rounding != NVFP4_SR && rounding != NVFP4_RTN_STD)
        return fail(NVFP4_EINVAL, "bad rounding %d", rounding);
    if (gamax_mode < NVFP4_GAMAX_NONE || gamax_mode > NVFP4_GAMAX_ROW_GIVEN)
        return fail(NVFP4_EINVAL, "bad gamax_mode %d", gamax_mode);
    if (err_mode < NVFP4_ERR_NONE || err_mode > NVFP4_ERR_MSE) return fail(NVFP4_EINVAL, "bad err_mode %d", err_mode);
    if (!(bound > 0.0f && bound <= 448.0f)) return fail(NVFP4_EINVAL, "scale_bound must be in (0, 448]");
    if ((block == NVFP4_BLOCK_16X16 || colwise) && M % 16 != 0)
        return fail(NVFP4_EINVAL, "16x16 blocks and columnwise output need M %% 16 == 0");
    if (is_row_mode(gamax_mode) && (block == NVFP4_BLOCK_16X16 || colwise))
        return fail(NVFP4_EINVAL, "per-row global scales allow 1x16 rowwise output only");
    if (err_mode != NVFP4_ERR_NONE) {
        if (rounding != NVFP4_RTN)
            return fail(NVFP4_EINVAL, "four-over-six is round-to-nearest with its own scale association only");
        if (residual) return fail(NVFP4_EINVAL, "four-over-six takes no residual");
        if (gamax_mode == NVFP4_GAMAX_NONE) return fail(NVFP4_EINVAL, "four-over-six needs a global amax");
        if (bound != 256.0f && bound != 448.0f) return fail(NVFP4_EINVAL, "four-over-six bound must be 256 or 448");
    }
    if (colwise && residual) return fail(NVFP4_EINVAL, "columnwise output takes no residual");
    if (colwise && K > kMaxColwiseK)            // the columnwise kernels' grid spans K along y
        return fail(NVFP4_EINVAL, "columnwise output needs K <= %lld", static_cast<long long>(kMaxColwiseK));
    const bool any = M > 0 && K > 0;
    if ((rc = check_ptr(x, "x", any))) return rc;
    if ((rc = check_ptr(residual, "residual", false))) return rc;
    if ((rc = check_ptr(gamax, "gamax", gamax_mode != NVFP4_GAMAX_NONE && (any || gamax_mode == NVFP4_GAMAX_TENSOR ||
                                                                        (gamax_mode == NVFP4_GAMAX_ROW && M > 0)), 4)))
        return rc;
    return NVFP4_OK;
}

// The amax pass (TENSOR / ROW) then the quantize kernel with the amax given.
int run_quant(nvfp4::QuantArgs a, float* gamax, void* stream) {
    int err;
    a.pk = nvfp4::philox_keys(a.seed, a.step);
    if (a.gamax_mode == NVFP4_GAMAX_TENSOR || a.gamax_mode == NVFP4_GAMAX_ROW) {
        err = nvfp4::launch_amax(a.x, a.M, a.K, a.dtype, a.residual, a.gamax_mode, gamax, stream);
        if (err) return cuda_fail(err, "amax launch");
        a.gamax_mode = a.gamax_mode == NVFP4_GAMAX_TENSOR ? NVFP4_GAMAX_TENSOR_GIVEN : NVFP4_GAMAX_ROW_GIVEN;
    }
    if (a.M == 0 || a.K == 0) return NVFP4_OK;
    err = a.codes_col ? nvfp4::launch_quantize_tiles(a, stream) : nvfp4::launch_quantize_rows(a, stream);
    if (err) return cuda_fail(err, "quantize launch");
    return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_quantize(const void* x, int64_t M, int64_t K, int dtype, int block, int rounding,
                   float* residual, uint64_t seed, uint64_t step, int64_t row_offset,
                   int gamax_mode, float* gamax, int err_mode, float scale_bound,
                   uint8_t* codes, uint8_t* scales, uint8_t* codes_col, uint8_t* scales_col,
                   cudaStream_t stream) {
    g_msg[0] = '\0';
    if ((codes_col == nullptr) != (scales_col == nullptr))
        return fail(NVFP4_EINVAL, "give both codes_col and scales_col, or neither");
    const bool colwise = codes_col != nullptr;
    int rc = check_quant(x, M, K, dtype, block, rounding, residual, gamax_mode, gamax, err_mode,
                         scale_bound, colwise);
    if (rc) return rc;
    const bool any = M > 0 && K > 0;
    if ((rc = check_ptr(codes, "codes", any))) return rc;
    if ((rc = check_ptr(scales, "scales", any))) return rc;
    if ((rc = check_ptr(codes_col, "codes_col", false))) return rc;
    if ((rc = check_ptr(scales_col, "scales_col", false))) return rc;
    nvfp4::QuantArgs a{x, M, K, dtype, block, rounding, residual, seed, step, row_offset,
                       gamax_mode, gamax, err_mode, scale_bound, codes, scales, codes_col,
                       scales_col, nullptr};
    return run_quant(a, gamax, stream);
}

int nvfp4_qdq(const void* x, int64_t M, int64_t K, int dtype, int block, int rounding,
              float* residual, uint64_t seed, uint64_t step, int64_t row_offset,
              int gamax_mode, float* gamax, int err_mode, float scale_bound,
              uint8_t* codes, uint8_t* scales, void* out_bf16, cudaStream_t stream) {
    g_msg[0] = '\0';
    int rc = check_quant(x, M, K, dtype, block, rounding, residual, gamax_mode, gamax, err_mode,
                         scale_bound, false);
    if (rc) return rc;
    const bool any = M > 0 && K > 0;
    if ((rc = check_ptr(codes, "codes", false))) return rc;
    if ((rc = check_ptr(scales, "scales", false))) return rc;
    if ((rc = check_ptr(out_bf16, "out_bf16", any))) return rc;
    nvfp4::QuantArgs a{x, M, K, dtype, block, rounding, residual, seed, step, row_offset,
                       gamax_mode, gamax, err_mode, scale_bound, codes, scales, nullptr, nullptr,
                       static_cast<uint16_t*>(out_bf16)};
    return run_quant(a, gamax, stream);
}

int nvfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K,
                     int gamax_mode, const float* gamax, float scale_bound, void* out,
                     int out_dtype, cudaStream_t stream) {
    g_msg[0] = '\0';
    int rc = check_shape(M, K);
    if (rc) return rc;
    if (gamax_mode < NVFP4_GAMAX_NONE || gamax_mode > NVFP4_GAMAX_ROW_GIVEN)
        return fail(NVFP4_EINVAL, "bad gamax_mode %d", gamax_mode);
    if (out_dtype != NVFP4_F32 && out_dtype != NVFP4_BF16) return fail(NVFP4_EINVAL, "bad out_dtype %d", out_dtype);
    if (!(scale_bound > 0.0f && scale_bound <= 448.0f)) return fail(NVFP4_EINVAL, "scale_bound must be in (0, 448]");
    const bool any = M > 0 && K > 0;
    if ((rc = check_ptr(codes, "codes", any))) return rc;
    if ((rc = check_ptr(scales, "scales", any))) return rc;
    if ((rc = check_ptr(out, "out", any))) return rc;
    if ((rc = check_ptr(gamax, "gamax", any && gamax_mode != NVFP4_GAMAX_NONE, 4))) return rc;
    nvfp4::DequantArgs a{codes, scales, M, K, gamax_mode, gamax, scale_bound, out, out_dtype};
    const int err = nvfp4::launch_dequantize(a, stream);
    if (err) return cuda_fail(err, "dequantize launch");
    return NVFP4_OK;
}

int nvfp4_amax(const void* x, int64_t M, int64_t K, int dtype, const float* residual, int mode,
               float* out, cudaStream_t stream) {
    g_msg[0] = '\0';
    int rc = check_shape(M, K);
    if (rc) return rc;
    if (dtype != NVFP4_F32 && dtype != NVFP4_BF16) return fail(NVFP4_EINVAL, "bad dtype %d", dtype);
    if (mode != NVFP4_GAMAX_TENSOR && mode != NVFP4_GAMAX_ROW)
        return fail(NVFP4_EINVAL, "amax mode must be NVFP4_GAMAX_TENSOR or NVFP4_GAMAX_ROW");
    const bool any = M > 0 && K > 0;
    if ((rc = check_ptr(x, "x", any))) return rc;
    if ((rc = check_ptr(residual, "residual", false))) return rc;
    if ((rc = check_ptr(out, "out", mode == NVFP4_GAMAX_TENSOR || M > 0, 4))) return rc;
    const int err = nvfp4::launch_amax(x, M, K, dtype, residual, mode, out, stream);
    if (err) return cuda_fail(err, "amax launch");
    return NVFP4_OK;
}

int nvfp4_scales_to_mma(const uint8_t* scales, int64_t rows, int64_t cols, uint8_t* out, cudaStream_t stream) {
    g_msg[0] = '\0';
    if (rows < 0 || cols < 0) return fail(NVFP4_EINVAL, "rows and cols must be >= 0");
    const bool any = rows > 0 && cols > 0;
    int rc;
    if ((rc = check_ptr(scales, "scales", any, 1))) return rc;
    if ((rc = check_ptr(out, "out", any, 4))) return rc;
    if (!any) return NVFP4_OK;
    const int err = nvfp4::launch_scales_mma(scales, rows, cols, out, stream);
    if (err) return cuda_fail(err, "scale layout launch");
    return NVFP4_OK;
}

int nvfp4_mm(const uint8_t* codes_a, const uint8_t* scales_a, const uint8_t* codes_b, const uint8_t* scales_b,
             int64_t M, int64_t N, int64_t K, const float* gamax_a, const float* gamax_b, float scale_bound,
             void* out, int out_dtype, cudaStream_t stream) {
    g_msg[0] = '\0';
    if (M < 0 || N < 0 || K < 0) return fail(NVFP4_EINVAL, "M, N and K must be >= 0");
    if (M % 128 || N % 128 || K % 64)
        return fail(NVFP4_EINVAL, "nvfp4_mm needs M %% 128 == 0, N %% 128 == 0 and K %% 64 == 0");
    if (out_dtype != NVFP4_F32 && out_dtype != NVFP4_BF16) return fail(NVFP4_EINVAL, "bad out_dtype %d", out_dtype);
    if (!(scale_bound > 0.0f && scale_bound <= 448.0f)) return fail(NVFP4_EINVAL, "scale_bound must be in (0, 448]");
    const bool any = M > 0 && N > 0;
    const bool anyk = any && K > 0;
    int rc;
    if ((rc = check_ptr(codes_a, "codes_a", anyk))) return rc;
    if ((rc = check_ptr(scales_a, "scales_a", anyk))) return rc;
    if ((rc = check_ptr(codes_b, "codes_b", anyk))) return rc;
    if ((rc = check_ptr(scales_b, "scales_b", anyk))) return rc;
    if ((rc = check_ptr(gamax_a, "gamax_a", false, 4))) return rc;
    if ((rc = check_ptr(gamax_b, "gamax_b", false, 4))) return rc;
    if ((rc = check_ptr(out, "out", any))) return rc;
    if (!any) return NVFP4_OK;
    if (K == 0) {
        const size_t bytes = static_cast<size_t>(M) * static_cast<size_t>(N) * (out_dtype == NVFP4_F32 ? 4 : 2);
        const int err = static_cast<int>(cudaMemsetAsync(out, 0, bytes, static_cast<cudaStream_t>(stream)));
        return err ? cuda_fail(err, "mm zero fill") : NVFP4_OK;
    }
    const int err = nvfp4::launch_mm(codes_a, scales_a, codes_b, scales_b, M, N, K, gamax_a, gamax_b, scale_bound,
                                     out, out_dtype, stream);
    if (err) return cuda_fail(err, "mm launch");
    return NVFP4_OK;
}

int nvfp4_global_scales(const float* gamax, int64_t n, float scale_bound, float* s_enc, float* s_dec,
                        cudaStream_t stream) {
    g_msg[0] = '\0';
    if (n < 0) return fail(NVFP4_EINVAL, "n must be >= 0");
    if (!(scale_bound > 0.0f && scale_bound <= 448.0f)) return fail(NVFP4_EINVAL, "scale_bound must be in (0, 448]");
    int rc;
    if ((rc = check_ptr(gamax, "gamax", n > 0, 4))) return rc;
    if ((rc = check_ptr(s_enc, "s_enc", false, 4))) return rc;
    if ((rc = check_ptr(s_dec, "s_dec", false, 4))) return rc;
    if (n > 0 && !s_enc && !s_dec) return fail(NVFP4_EINVAL, "give s_enc, s_dec or both");
    const int err = nvfp4::launch_global_scales(gamax, n, scale_bound, s_enc, s_dec, stream);
    if (err) return cuda_fail(err, "global scales launch");
    return NVFP4_OK;
}

int nvfp4_rmsnorm(const void* x, const void* hidden, int64_t M, int64_t K, int dtype, const void* weight,
                  int weight_dtype, float eps, void* hidden_out, void* out, int format, int gamax_mode,
                  float* gamax, float scale_bound, uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
    g_msg[0] = '\0';
    int rc = check_shape(M, K);
    if (rc) return rc;
    if (dtype != NVFP4_F32 && dtype != NVFP4_BF16) return fail(NVFP4_EINVAL, "bad dtype %d", dtype);
    if (weight_dtype != NVFP4_F32 && weight_dtype != NVFP4_BF16)
        return fail(NVFP4_EINVAL, "bad weight_dtype %d", weight_dtype);
    if (!(eps >= 0.0f && eps <= 3.4028234663852886e+38f)) return fail(NVFP4_EINVAL, "eps must be >= 0 and finite");
    if (format != NVFP4_FMT_NVFP4 && format != NVFP4_FMT_MXFP8) return fail(NVFP4_EINVAL, "bad format %d", format);
    if (gamax_mode < NVFP4_GAMAX_NONE || gamax_mode > NVFP4_GAMAX_ROW_GIVEN)
        return fail(NVFP4_EINVAL, "bad gamax_mode %d", gamax_mode);
    if (gamax_mode == NVFP4_GAMAX_TENSOR)
        return fail(NVFP4_EINVAL, "the norm quantizes in one pass: give the tensor amax, or use a per-row one");
    if (format == NVFP4_FMT_MXFP8 && gamax_mode != NVFP4_GAMAX_NONE)
        return fail(NVFP4_EINVAL, "NVFP4_FMT_MXFP8 has no global scale");
    if (!(scale_bound > 0.0f && scale_bound <= 448.0f)) return fail(NVFP4_EINVAL, "scale_bound must be in (0, 448]");
    if ((codes == nullptr) != (scales == nullptr)) return fail(NVFP4_EINVAL, "give both codes and scales, or neither");
    const bool any = M > 0 && K > 0;
    if (any && !codes && gamax_mode != NVFP4_GAMAX_NONE)
        return fail(NVFP4_EINVAL, "a gamax_mode needs codes and scales");
    if (any && !codes && !out && !hidden_out) return fail(NVFP4_EINVAL, "no output is given");
    if ((hidden == nullptr) != (hidden_out == nullptr))
        return fail(NVFP4_EINVAL, "give both hidden and hidden_out, or neither");
    if ((rc = check_ptr(x, "x", any))) return rc;
    if ((rc = check_ptr(hidden, "hidden", false))) return rc;
    if ((rc = check_ptr(weight, "weight", false))) return rc;
    if ((rc = check_ptr(hidden_out, "hidden_out", false))) return rc;
    if ((rc = check_ptr(out, "out", false))) return rc;
    if ((rc = check_ptr(codes, "codes", false))) return rc;
    if ((rc = check_ptr(scales, "scales", false))) return rc;
    if ((rc = check_ptr(gamax, "gamax", gamax_mode != NVFP4_GAMAX_NONE && M > 0, 4))) return rc;
    if (M == 0) return NVFP4_OK;
    if (K == 0) {                               // an empty row's amax is +0
        if (gamax_mode != NVFP4_GAMAX_ROW) return NVFP4_OK;
        const int err = static_cast<int>(cudaMemsetAsync(gamax, 0, static_cast<size_t>(M) * 4, stream));
        return err ? cuda_fail(err, "norm zero fill") : NVFP4_OK;
    }
    const uint64_t m = M, k = K, full = m * k * (dtype == NVFP4_F32 ? 4 : 2);
    const bool mx = format == NVFP4_FMT_MXFP8;
    const uint64_t amax = gamax_mode == NVFP4_GAMAX_NONE ? 0 : gamax_mode == NVFP4_GAMAX_TENSOR_GIVEN ? 4 : m * 4;
    const bool row = gamax_mode == NVFP4_GAMAX_ROW;       // gamax is written
    const Buffer outs[] = {{hidden_out, full, "hidden_out"},
                           {out, full, "out"},
                           {codes, mx ? m * k : m * (k / 2), "codes"},
                           {scales, m * (mx ? (k + 31) / 32 : k / 16), "scales"},
                           {gamax, row ? amax : 0, "gamax"}};
    const Buffer ins[] = {{x, full, "x"},
                          {hidden, hidden == hidden_out ? 0 : full, "hidden"},      // updated in place: an output alone
                          {weight, k * (weight_dtype == NVFP4_F32 ? 4 : 2), "weight"},
                          {gamax, row ? 0 : amax, "gamax"}};
    if ((rc = check_apart(outs, ins))) return rc;
    const nvfp4::NormArgs a{x, hidden, M, K, dtype, weight, weight_dtype, eps, hidden_out, out, format, gamax_mode,
                            gamax, scale_bound, codes, scales};
    const int err = nvfp4::launch_rmsnorm(a, stream);
    if (err) return cuda_fail(err, "norm launch");
    return NVFP4_OK;
}

int nvfp4_mv(const void* x, const uint8_t* x_scales, int x_type, const uint8_t* codes, const uint8_t* scales,
             int64_t M, int64_t N, int64_t K, int gamax_mode, const float* gamax, float scale_bound, void* out,
             int out_dtype, cudaStream_t stream) {
    g_msg[0] = '\0';
    if (M < 0 || N < 0 || K < 0) return fail(NVFP4_EINVAL, "M, N and K must be >= 0");
    if (M > 16) return fail(NVFP4_EINVAL, "nvfp4_mv takes at most 16 rows of x (got %lld)", (long long)M);
    if (K % 16) return fail(NVFP4_EINVAL, "K must be a multiple of 16 (got %lld)", (long long)K);
    if (N >= (int64_t{1} << 30) || K >= (int64_t{1} << 30)) return fail(NVFP4_EINVAL, "N and K must be below 2^30");
    if (x_type < NVFP4_X_F32 || x_type > NVFP4_X_MXFP8) return fail(NVFP4_EINVAL, "bad x_type %d", x_type);
    if (out_dtype != NVFP4_F32 && out_dtype != NVFP4_BF16) return fail(NVFP4_EINVAL, "bad out_dtype %d", out_dtype);
    if (gamax_mode != NVFP4_GAMAX_NONE && gamax_mode != NVFP4_GAMAX_TENSOR_GIVEN &&
        gamax_mode != NVFP4_GAMAX_ROW_GIVEN)
        return fail(NVFP4_EINVAL, "gamax_mode must be NONE, TENSOR_GIVEN or ROW_GIVEN (got %d)", gamax_mode);
    if (!(scale_bound > 0.0f && scale_bound <= 448.0f)) return fail(NVFP4_EINVAL, "scale_bound must be in (0, 448]");
    if ((x_type == NVFP4_X_MXFP8) != (x_scales != nullptr) && M > 0 && K > 0)
        return fail(NVFP4_EINVAL, "x_scales go with an MXFP8 x");
    const bool any = M > 0 && N > 0;
    const bool anyk = any && K > 0;
    int rc;
    if ((rc = check_ptr(x, "x", anyk))) return rc;
    if ((rc = check_ptr(x_scales, "x_scales", false))) return rc;
    if ((rc = check_ptr(codes, "codes", anyk))) return rc;
    if ((rc = check_ptr(scales, "scales", anyk))) return rc;
    if ((rc = check_ptr(gamax, "gamax", any && gamax_mode != NVFP4_GAMAX_NONE, 4))) return rc;
    if ((rc = check_ptr(out, "out", any))) return rc;
    if (!any) return NVFP4_OK;
    const uint64_t m = M, n = N, k = K;
    const Buffer outs[] = {{out, m * n * (out_dtype == NVFP4_F32 ? 4 : 2), "out"}};
    const Buffer ins[] = {{x, m * k * (x_type == NVFP4_X_F32 ? 4 : x_type == NVFP4_X_BF16 ? 2 : 1), "x"},
                          {x_scales, x_type == NVFP4_X_MXFP8 ? m * ((k + 31) / 32) : 0, "x_scales"},
                          {codes, n * (k / 2), "codes"},
                          {scales, n * (k / 16), "scales"},
                          {gamax, gamax_mode == NVFP4_GAMAX_NONE ? 0 : gamax_mode == NVFP4_GAMAX_ROW_GIVEN ? n * 4 : 4, "gamax"}};
    if ((rc = check_apart(outs, ins))) return rc;
    if (K == 0) {
        const size_t bytes = static_cast<size_t>(M) * static_cast<size_t>(N) * (out_dtype == NVFP4_F32 ? 4 : 2);
        const int err = static_cast<int>(cudaMemsetAsync(out, 0, bytes, stream));
        return err ? cuda_fail(err, "mv zero fill") : NVFP4_OK;
    }
    const nvfp4::MvArgs a{x, x_scales, x_type, codes, scales, static_cast<int>(M), static_cast<int>(N),
                          static_cast<int>(K), gamax_mode, gamax, scale_bound, out, out_dtype};
    const int err = nvfp4::launch_mv(a, stream);
    if (err) return cuda_fail(err, "mv launch");
    return NVFP4_OK;
}

int64_t nvfp4_grouped_mm_workspace(int64_t E, int64_t T, int64_t N, int64_t K) {
    constexpr int64_t kMax = int64_t{1} << 30;
    if (E <= 0 || T <= 0 || N <= 0 || K <= 0 || E >= kMax || T >= kMax || N >= kMax || K >= kMax) return 0;
    nvfp4::GroupedArgs a = {};
    a.E = E, a.T = T, a.N = N, a.K = K;
    return nvfp4::grouped_workspace(a);
}

int nvfp4_grouped_mm(const uint8_t* codes_a, const uint8_t* scales_a, const int64_t* offsets,
                     const uint8_t* codes_b, const uint8_t* scales_b, int64_t E, int64_t T, int64_t N, int64_t K,
                     int gamax_a_mode, const float* gamax_a, const float* gamax_b, float scale_bound, void* out,
                     int out_dtype, uint8_t* workspace, int64_t workspace_bytes, cudaStream_t stream) {
    g_msg[0] = '\0';
    constexpr int64_t kMax = int64_t{1} << 30;
    if (E < 0 || T < 0 || N < 0 || K < 0) return fail(NVFP4_EINVAL, "E, T, N and K must be >= 0");
    if (K % 64) return fail(NVFP4_EINVAL, "nvfp4_grouped_mm needs K %% 64 == 0 (got %lld)", (long long)K);
    if (E >= kMax || T >= kMax || N >= kMax || K >= kMax || (N > 0 && E > (kMax - 1) / N))
        return fail(NVFP4_EINVAL, "E * N, T and K must be below 2^30");
    if (out_dtype != NVFP4_F32 && out_dtype != NVFP4_BF16) return fail(NVFP4_EINVAL, "bad out_dtype %d", out_dtype);
    if (gamax_a_mode != NVFP4_GAMAX_NONE && gamax_a_mode != NVFP4_GAMAX_TENSOR_GIVEN &&
        gamax_a_mode != NVFP4_GAMAX_ROW_GIVEN)
        return fail(NVFP4_EINVAL, "gamax_a_mode must be NONE, TENSOR_GIVEN or ROW_GIVEN (got %d)", gamax_a_mode);
    if (!(scale_bound > 0.0f && scale_bound <= 448.0f)) return fail(NVFP4_EINVAL, "scale_bound must be in (0, 448]");
    const bool any = E > 0 && T > 0 && N > 0;
    const bool anyk = any && K > 0;
    int rc;
    if ((rc = check_ptr(codes_a, "codes_a", anyk))) return rc;
    if ((rc = check_ptr(scales_a, "scales_a", anyk))) return rc;
    if ((rc = check_ptr(offsets, "offsets", any, 8))) return rc;
    if ((rc = check_ptr(codes_b, "codes_b", anyk))) return rc;
    if ((rc = check_ptr(scales_b, "scales_b", anyk))) return rc;
    if ((rc = check_ptr(gamax_a, "gamax_a", any && gamax_a_mode != NVFP4_GAMAX_NONE, 4))) return rc;
    if ((rc = check_ptr(gamax_b, "gamax_b", false, 4))) return rc;
    if ((rc = check_ptr(out, "out", any))) return rc;
    if (!any) return NVFP4_OK;
    const nvfp4::GroupedArgs a{codes_a, scales_a, offsets, codes_b, scales_b, E, T, N, K, gamax_a_mode, gamax_a,
                               gamax_b, scale_bound, out, out_dtype, workspace};
    const int64_t need = nvfp4::grouped_workspace(a);
    if (workspace_bytes < need)
        return fail(NVFP4_EINVAL, "the workspace needs %lld bytes (got %lld)", (long long)need, (long long)workspace_bytes);
    if ((rc = check_ptr(workspace, "workspace", need > 0))) return rc;
    const uint64_t e = E, t = T, n = N, k = K;
    const Buffer outs[] = {{out, t * n * (out_dtype == NVFP4_F32 ? 4 : 2), "out"}, {workspace, static_cast<uint64_t>(need), "workspace"}};
    const Buffer ins[] = {{codes_a, t * (k / 2), "codes_a"},
                          {scales_a, t * (k / 16), "scales_a"},
                          {offsets, (e + 1) * 8, "offsets"},
                          {codes_b, e * n * (k / 2), "codes_b"},
                          {scales_b, e * ((n + 127) / 128 * 128) * (k / 16), "scales_b"},      // at most 2^63
                          {gamax_a, gamax_a_mode == NVFP4_GAMAX_NONE ? 0 : gamax_a_mode == NVFP4_GAMAX_ROW_GIVEN ? t * 4 : 4, "gamax_a"},
                          {gamax_b, e * 4, "gamax_b"}};
    if ((rc = check_apart(outs, ins))) return rc;
    const int err = nvfp4::launch_grouped_mm(a, stream);
    if (err) return cuda_fail(err, "grouped mm launch");
    return NVFP4_OK;
}

// the sizes and scales of a cache (its pointer is checked by the call); *n: its bytes
static int check_cache(int64_t pages, int64_t page_size, int64_t Hkv, int64_t D, int64_t T, int k_mode,
                       const float* k_gamax, int v_mode, const float* v_gamax, float scale_bound, uint64_t* n) {
    constexpr int64_t kMax = int64_t{1} << 30, kHeads = 1 << 15;
    if (pages < 0 || T < 0 || Hkv < 0) return fail(NVFP4_EINVAL, "pages, T and Hkv must be >= 0");
    if (pages >= kMax || T >= kMax || Hkv >= kHeads) return fail(NVFP4_EINVAL, "pages and T must be below 2^30, Hkv below 2^15");
    if (D != 64 && D != 128 && D != 256) return fail(NVFP4_EINVAL, "a cache's D must be 64, 128 or 256 (got %lld)", (long long)D);
    if (page_size <= 0 || page_size % 16 || page_size >= kMax)
        return fail(NVFP4_EINVAL, "page_size must be a multiple of 16 (got %lld)", (long long)page_size);
    // pages * Hkv * page_size * D below 2^62
    if (pages > 0 && Hkv > 0 && page_size > (int64_t{1} << 62) / pages / Hkv / D) return fail(NVFP4_EINVAL, "the cache is too large");
    for (const int m : {k_mode, v_mode})
        if (m != NVFP4_GAMAX_NONE && m != NVFP4_GAMAX_TENSOR_GIVEN && m != NVFP4_GAMAX_ROW_GIVEN)
            return fail(NVFP4_EINVAL, "k_mode and v_mode must be NONE, TENSOR_GIVEN or ROW_GIVEN (got %d)", m);
    if (!(scale_bound > 0.0f && scale_bound <= 448.0f)) return fail(NVFP4_EINVAL, "scale_bound must be in (0, 448]");
    int rc;
    if ((rc = check_ptr(k_gamax, "k_gamax", k_mode != NVFP4_GAMAX_NONE, 4))) return rc;
    if ((rc = check_ptr(v_gamax, "v_gamax", v_mode != NVFP4_GAMAX_NONE, 4))) return rc;
    *n = static_cast<uint64_t>(pages) * static_cast<uint64_t>(Hkv) * static_cast<uint64_t>(page_size / 16) * static_cast<uint64_t>(18 * D);
    return NVFP4_OK;
}

static uint64_t gamax_bytes(int mode, int64_t Hkv) {
    return mode == NVFP4_GAMAX_NONE ? 0 : mode == NVFP4_GAMAX_TENSOR_GIVEN ? 4 : static_cast<uint64_t>(Hkv) * 4;
}

// a token's heads are contiguous, tokens `stride` elements apart: whole 16 bytes
static int check_stride(int64_t stride, int size, const char* name) {
    if (stride < 0 || stride >= int64_t{1} << 32 || stride * size % 16)
        return fail(NVFP4_EINVAL, "%s must be >= 0, below 2^32 and of whole 16 bytes (got %lld elements)", name, (long long)stride);
    return NVFP4_OK;
}

static uint64_t strided_bytes(int64_t T, int64_t stride, int64_t H, int64_t D, int size) {
    return T == 0 || H == 0 ? 0 : (static_cast<uint64_t>(T - 1) * static_cast<uint64_t>(stride) + static_cast<uint64_t>(H) * static_cast<uint64_t>(D)) * size;
}

static int run_heads(const nvfp4::HeadsArgs& a, uint64_t cache_bytes, cudaStream_t stream) {
    const int size = a.dtype == NVFP4_F32 ? 4 : 2;
    int rc;
    const uint64_t t = a.T, row = static_cast<uint64_t>(a.D) * size;
    const Buffer outs[] = {{a.q_out, t * a.Hq * row, "q_out"}, {a.k_out, t * a.Hkv * row, "k_out"}, {a.cache.data, cache_bytes, "cache"}};
    const uint64_t w = static_cast<uint64_t>(a.D) * (a.weight_dtype == NVFP4_F32 ? 4 : 2);
    const Buffer ins[] = {{a.q, strided_bytes(a.T, a.q_stride, a.Hq, a.D, size), "q"},
                          {a.k, strided_bytes(a.T, a.k_stride, a.Hkv, a.D, size), "k"},
                          {a.v, strided_bytes(a.T, a.v_stride, a.Hkv, a.D, size), "v"},
                          {a.q_weight, w, "q_weight"},
                          {a.k_weight, w, "k_weight"},
                          {a.positions, t * 8, "positions"},
                          {a.phases, static_cast<uint64_t>(a.rotary_dim) * 4, "phases"},
                          {a.slots, t * 8, "slots"},
                          {a.cache.k_gamax, gamax_bytes(a.cache.k_mode, a.Hkv), "k_gamax"},
                          {a.cache.v_gamax, gamax_bytes(a.cache.v_mode, a.Hkv), "v_gamax"}};
    if ((rc = check_apart(outs, ins))) return rc;
    const int err = nvfp4::launch_heads(a, stream);
    return err ? cuda_fail(err, "heads launch") : NVFP4_OK;
}

int nvfp4_qk_norm_rope(const void* q, const void* k, const void* v, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                       int64_t q_stride, int64_t k_stride, int64_t v_stride, int dtype, const void* q_weight,
                       const void* k_weight, int weight_dtype, float eps, const int64_t* positions,
                       const uint64_t* phases, int64_t rotary_dim, int layout, float magnitude, void* q_out, void* k_out,
                       uint8_t* cache, int64_t pages, int64_t page_size, const int64_t* slots, int k_mode,
                       const float* k_gamax, int v_mode, const float* v_gamax, float scale_bound, cudaStream_t stream) {
    g_msg[0] = '\0';
    constexpr int64_t kMax = int64_t{1} << 30, kHeads = 1 << 15;
    const bool cached = slots != nullptr;
    int rc;
    uint64_t bytes = 0;
    if (T < 0 || Hq < 0 || Hkv < 0 || T >= kMax || Hq >= kHeads || Hkv >= kHeads)
        return fail(NVFP4_EINVAL, "T must be in [0, 2^30), Hq and Hkv in [0, 2^15)");
    if (D <= 0 || D % 16 || D > 512) return fail(NVFP4_EINVAL, "D must be a multiple of 16 up to 512 (got %lld)", (long long)D);
    if (dtype != NVFP4_F32 && dtype != NVFP4_BF16) return fail(NVFP4_EINVAL, "bad dtype %d", dtype);
    if (weight_dtype != NVFP4_F32 && weight_dtype != NVFP4_BF16) return fail(NVFP4_EINVAL, "bad weight_dtype %d", weight_dtype);
    if (!(eps >= 0.0f && eps <= 3.4028234663852886e+38f)) return fail(NVFP4_EINVAL, "eps must be >= 0 and finite");
    if (!(magnitude >= -3.4028234663852886e+38f && magnitude <= 3.4028234663852886e+38f))
        return fail(NVFP4_EINVAL, "magnitude must be finite");
    if (layout != NVFP4_ROPE_HALF && layout != NVFP4_ROPE_INTERLEAVED) return fail(NVFP4_EINVAL, "bad layout %d", layout);
    if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 16)
        return fail(NVFP4_EINVAL, "rotary_dim must be a multiple of 16 up to D (got %lld)", (long long)rotary_dim);
    if ((q_weight == nullptr) != (k_weight == nullptr)) return fail(NVFP4_EINVAL, "give both q_weight and k_weight, or neither");
    // (a cache without pages has no memory: every slot lies outside it)
    if ((cached ? cache == nullptr && pages != 0 : cache != nullptr) || cached != (v != nullptr) || cached == (k_out != nullptr)) {
        if (T > 0 && Hkv > 0) return fail(NVFP4_EINVAL, "give v, cache and slots and no k_out, or k_out and none of them");
    }
    if (cached) {
        if (layout == NVFP4_ROPE_HALF && rotary_dim % 32)
            return fail(NVFP4_EINVAL, "with a cache and halves apart rotary_dim must be a multiple of 32 (got %lld)", (long long)rotary_dim);
        if ((rc = check_cache(pages, page_size, Hkv, D, T, k_mode, k_gamax, v_mode, v_gamax, scale_bound, &bytes))) return rc;
    }
    const int size = dtype == NVFP4_F32 ? 4 : 2;
    if ((rc = check_stride(q_stride, size, "q_stride"))) return rc;
    if ((rc = check_stride(k_stride, size, "k_stride"))) return rc;
    if ((rc = check_stride(v_stride, size, "v_stride"))) return rc;
    const bool turned = rotary_dim > 0 && T > 0;
    if ((rc = check_ptr(q, "q", T > 0 && Hq > 0))) return rc;
    if ((rc = check_ptr(k, "k", T > 0 && Hkv > 0))) return rc;
    if ((rc = check_ptr(v, "v", false))) return rc;
    if ((rc = check_ptr(q_weight, "q_weight", false))) return rc;
    if ((rc = check_ptr(k_weight, "k_weight", false))) return rc;
    if ((rc = check_ptr(positions, "positions", turned, 8))) return rc;
    if ((rc = check_ptr(phases, "phases", turned, 8))) return rc;
    if ((rc = check_ptr(q_out, "q_out", T > 0 && Hq > 0))) return rc;
    if ((rc = check_ptr(k_out, "k_out", false))) return rc;
    if ((rc = check_ptr(cache, "cache", false))) return rc;
    if ((rc = check_ptr(slots, "slots", false, 8))) return rc;
    if (T == 0 || Hq + Hkv == 0) return NVFP4_OK;
    nvfp4::HeadsArgs a = {};
    a.q = Hq > 0 ? q : nullptr, a.k = Hkv > 0 ? k : nullptr, a.v = Hkv > 0 && cached ? v : nullptr;
    a.T = T, a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.Hq = static_cast<int>(Hq), a.Hkv = static_cast<int>(Hkv), a.D = static_cast<int>(D), a.dtype = dtype;
    a.q_weight = q_weight, a.k_weight = k_weight, a.weight_dtype = weight_dtype, a.eps = eps;
    a.rotary_dim = static_cast<int>(rotary_dim), a.layout = layout, a.magnitude = magnitude;
    if (turned) a.positions = positions, a.phases = phases;
    a.q_out = q_out, a.k_out = cached ? nullptr : k_out, a.slots = slots;
    if (cached)
        a.cache = {cache, pages, static_cast<int>(page_size), a.Hkv, a.D, k_mode, v_mode, k_gamax, v_gamax, scale_bound};
    return run_heads(a, bytes, stream);
}

int nvfp4_cache_write(const void* k, const void* v, int64_t T, int64_t Hkv, int64_t D, int64_t k_stride,
                      int64_t v_stride, int dtype, uint8_t* cache, int64_t pages, int64_t page_size,
                      const int64_t* slots, int k_mode, const float* k_gamax, int v_mode, const float* v_gamax,
                      float scale_bound, cudaStream_t stream) {
    g_msg[0] = '\0';
    uint64_t bytes = 0;
    int rc = check_cache(pages, page_size, Hkv, D, T, k_mode, k_gamax, v_mode, v_gamax, scale_bound, &bytes);
    if (rc) return rc;
    if (dtype != NVFP4_F32 && dtype != NVFP4_BF16) return fail(NVFP4_EINVAL, "bad dtype %d", dtype);
    const int size = dtype == NVFP4_F32 ? 4 : 2;
    if ((rc = check_stride(k_stride, size, "k_stride"))) return rc;
    if ((rc = check_stride(v_stride, size, "v_stride"))) return rc;
    const bool any = T > 0 && Hkv > 0;
    if ((rc = check_ptr(k, "k", any))) return rc;
    if ((rc = check_ptr(v, "v", any))) return rc;
    if ((rc = check_ptr(slots, "slots", any, 8))) return rc;
    if ((rc = check_ptr(cache, "cache", any && pages > 0))) return rc;
    if (!any || pages == 0) return NVFP4_OK;
    nvfp4::HeadsArgs a = {};
    a.k = k, a.v = v, a.T = T, a.k_stride = k_stride, a.v_stride = v_stride;
    a.Hkv = static_cast<int>(Hkv), a.D = static_cast<int>(D), a.dtype = dtype, a.weight_dtype = dtype;
    a.slots = slots;
    a.cache = {cache, pages, static_cast<int>(page_size), a.Hkv, a.D, k_mode, v_mode, k_gamax, v_gamax, scale_bound};
    return run_heads(a, bytes, stream);
}

int nvfp4_cache_read(const uint8_t* cache, int64_t pages, int64_t page_size, int64_t Hkv, int64_t D,
                     const int64_t* slots, int64_t T, int k_mode, const float* k_gamax, int v_mode,
                     const float* v_gamax, float scale_bound, void* k, void* v, int out_dtype, cudaStream_t stream) {
    g_msg[0] = '\0';
    uint64_t bytes = 0;
    int rc = check_cache(pages, page_size, Hkv, D, T, k_mode, k_gamax, v_mode, v_gamax, scale_bound, &bytes);
    if (rc) return rc;
    if (out_dtype != NVFP4_F32 && out_dtype != NVFP4_BF16) return fail(NVFP4_EINVAL, "bad out_dtype %d", out_dtype);
    const bool any = T > 0 && Hkv > 0;
    if ((rc = check_ptr(cache, "cache", any && pages > 0))) return rc;
    if ((rc = check_ptr(slots, "slots", any, 8))) return rc;
    if ((rc = check_ptr(k, "k", any && !v))) return rc;
    if ((rc = check_ptr(v, "v", false))) return rc;
    if (!any) return NVFP4_OK;
    const uint64_t out = static_cast<uint64_t>(T) * Hkv * D * (out_dtype == NVFP4_F32 ? 4 : 2);
    const Buffer outs[] = {{k, out, "k"}, {v, out, "v"}};
    const Buffer ins[] = {{cache, bytes, "cache"},
                          {slots, static_cast<uint64_t>(T) * 8, "slots"},
                          {k_gamax, gamax_bytes(k_mode, Hkv), "k_gamax"},
                          {v_gamax, gamax_bytes(v_mode, Hkv), "v_gamax"}};
    if ((rc = check_apart(outs, ins))) return rc;
    nvfp4::CacheReadArgs a = {};
    a.cache = {const_cast<uint8_t*>(cache), pages, static_cast<int>(page_size), static_cast<int>(Hkv), static_cast<int>(D),
               k_mode, v_mode, k_gamax, v_gamax, scale_bound};
    a.slots = slots, a.T = T, a.k = k, a.v = v, a.out_dtype = out_dtype;
    const int err = nvfp4::launch_cache_read(a, stream);
    return err ? cuda_fail(err, "cache read launch") : NVFP4_OK;
}

// the sizes that fix an attention's kernels and workspace; false where there is nothing to do or they are out of range
static bool attend_sizes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t width, int64_t page_size,
                         int dtype, int ragged, nvfp4::AttendArgs* a) {
    constexpr int64_t kMax = int64_t{1} << 30, kHeads = 1 << 15;
    if (T <= 0 || Hq <= 0 || Hkv <= 0 || B <= 0 || T >= kMax || Hq >= kHeads || Hkv >= kHeads || B >= kMax || Hq % Hkv ||
        (D != 64 && D != 128 && D != 256) || width < 0 || page_size <= 0 || page_size % 16 || page_size >= kMax ||
        width >= kMax / page_size)
        return false;
    a->T = T, a->Hq = static_cast<int>(Hq), a->B = B, a->width = width, a->dtype = dtype, a->ragged = ragged;
    a->cache.Hkv = static_cast<int>(Hkv), a->cache.D = static_cast<int>(D), a->cache.page_size = static_cast<int>(page_size);
    return true;
}

int64_t nvfp4_cache_attention_workspace(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t width,
                                        int64_t page_size, int dtype, int ragged) {
    nvfp4::AttendArgs a = {};
    return attend_sizes(T, Hq, Hkv, D, B, width, page_size, dtype, ragged, &a) ? nvfp4::attend_workspace(a) : 0;
}

int nvfp4_cache_attention(const void* q, int64_t T, int64_t Hq, int64_t q_stride, int dtype, const uint8_t* cache,
                          int64_t pages, int64_t page_size, int64_t Hkv, int64_t D, const int32_t* page_table,
                          int64_t B, int64_t width, const int64_t* lengths, const int64_t* offsets, int k_mode,
                          const float* k_gamax, int v_mode, const float* v_gamax, float scale_bound, float scale,
                          int causal, int64_t window, const float* sinks, void* out, int out_dtype, float* lse,
                          uint8_t* workspace, int64_t workspace_bytes, cudaStream_t stream) {
    g_msg[0] = '\0';
    constexpr int64_t kMax = int64_t{1} << 30, kHeads = 1 << 15;
    uint64_t bytes = 0;
    int rc = check_cache(pages, page_size, Hkv, D, T, k_mode, k_gamax, v_mode, v_gamax, scale_bound, &bytes);
    if (rc) return rc;
    if (dtype != NVFP4_F32 && dtype != NVFP4_BF16) return fail(NVFP4_EINVAL, "bad dtype %d", dtype);
    if (out_dtype != NVFP4_F32 && out_dtype != NVFP4_BF16) return fail(NVFP4_EINVAL, "bad out_dtype %d", out_dtype);
    if (Hq < 0 || Hq >= kHeads) return fail(NVFP4_EINVAL, "Hq must be in [0, 2^15)");
    if (Hkv == 0 ? Hq != 0 : Hq % Hkv) return fail(NVFP4_EINVAL, "Hq must be a multiple of Hkv");
    if (B < 0 || B >= kMax) return fail(NVFP4_EINVAL, "B must be in [0, 2^30)");
    if (width < 0 || width >= kMax / page_size) return fail(NVFP4_EINVAL, "width * page_size must be in [0, 2^30)");
    if (T * (Hkv > 0 ? Hq / Hkv : 0) >= kMax) return fail(NVFP4_EINVAL, "T * Hq / Hkv must be below 2^30");
    if (!offsets && T != B) return fail(NVFP4_EINVAL, "without offsets a sequence has one query: T must be B");
    if (causal != 0 && causal != 1) return fail(NVFP4_EINVAL, "causal must be 0 or 1 (got %d)", causal);
    if (window < 0) return fail(NVFP4_EINVAL, "window must be >= 0");
    if (!(scale >= -3.4028234663852886e+38f && scale <= 3.4028234663852886e+38f)) return fail(NVFP4_EINVAL, "scale must be finite");
    if ((rc = check_stride(q_stride, dtype == NVFP4_F32 ? 4 : 2, "q_stride"))) return rc;
    const bool any = T > 0 && Hq > 0 && B > 0;
    const bool keys = any && width > 0 && pages > 0;
    if ((rc = check_ptr(q, "q", any))) return rc;
    if ((rc = check_ptr(cache, "cache", keys))) return rc;
    if ((rc = check_ptr(page_table, "page_table", any && width > 0, 4))) return rc;
    if ((rc = check_ptr(lengths, "lengths", any, 8))) return rc;
    if ((rc = check_ptr(offsets, "offsets", false, 8))) return rc;
    if ((rc = check_ptr(sinks, "sinks", false, 4))) return rc;
    if ((rc = check_ptr(out, "out", any))) return rc;
    if ((rc = check_ptr(lse, "lse", false, 4))) return rc;
    nvfp4::AttendArgs a = {};
    if (!any || !attend_sizes(T, Hq, Hkv, D, B, width, page_size, dtype, offsets != nullptr, &a)) return NVFP4_OK;
    const int64_t need = nvfp4::attend_workspace(a);
    if (workspace_bytes < need)
        return fail(NVFP4_EINVAL, "the workspace needs %lld bytes (got %lld)", (long long)need, (long long)workspace_bytes);
    if ((rc = check_ptr(workspace, "workspace", need > 0))) return rc;
    const uint64_t heads = static_cast<uint64_t>(T) * static_cast<uint64_t>(Hq);
    const Buffer outs[] = {{out, heads * D * (out_dtype == NVFP4_F32 ? 4 : 2), "out"},
                           {lse, heads * 4, "lse"},
                           {workspace, static_cast<uint64_t>(need), "workspace"}};
    const Buffer ins[] = {{q, strided_bytes(T, q_stride, Hq, D, dtype == NVFP4_F32 ? 4 : 2), "q"},
                          {cache, bytes, "cache"},
                          {page_table, static_cast<uint64_t>(B) * static_cast<uint64_t>(width) * 4, "page_table"},
                          {lengths, static_cast<uint64_t>(B) * 8, "lengths"},
                          {offsets, static_cast<uint64_t>(B + 1) * 8, "offsets"},
                          {k_gamax, gamax_bytes(k_mode, Hkv), "k_gamax"},
                          {v_gamax, gamax_bytes(v_mode, Hkv), "v_gamax"},
                          {sinks, static_cast<uint64_t>(Hq) * 4, "sinks"}};
    if ((rc = check_apart(outs, ins))) return rc;
    a.q = q, a.q_stride = q_stride;
    a.cache = {const_cast<uint8_t*>(cache), cache ? pages : 0, a.cache.page_size, a.cache.Hkv, a.cache.D, k_mode, v_mode, k_gamax, v_gamax, scale_bound};
    a.pages = page_table, a.lengths = lengths, a.offsets = offsets, a.scale = scale, a.causal = causal;
    a.window = static_cast<int>(window < kMax ? window : kMax), a.sinks = sinks;
    a.out = out, a.out_dtype = out_dtype, a.lse = lse, a.workspace = workspace;
    const int err = nvfp4::launch_attend(a, stream);
    return err ? cuda_fail(err, "attention launch") : NVFP4_OK;
}

int nvfp4_probe_divide(const float* a, const float* b, float* out, int64_t n, cudaStream_t stream) {
    g_msg[0] = '\0';
    if (n < 0) return fail(NVFP4_EINVAL, "n must be >= 0");
    int rc;
    if ((rc = check_ptr(a, "a", n > 0, 4))) return rc;
    if ((rc = check_ptr(b, "b", n > 0, 4))) return rc;
    if ((rc = check_ptr(out, "out", n > 0, 4))) return rc;
    const int err = nvfp4::launch_probe_divide(a, b, out, n, stream);
    if (err) return cuda_fail(err, "probe launch");
    return NVFP4_OK;
}

int nvfp4_probe_sub_f16(const uint32_t* q, const float* v, float* out, int64_t n, cudaStream_t stream) {
    g_msg[0] = '\0';
    if (n < 0) return fail(NVFP4_EINVAL, "n must be >= 0");
    int rc;
    if ((rc = check_ptr(q, "q", n > 0, 4))) return rc;
    if ((rc = check_ptr(v, "v", n > 0, 4))) return rc;
    if ((rc = check_ptr(out, "out", n > 0, 4))) return rc;
    const int err = nvfp4::launch_probe_sub_f16(q, v, out, n, stream);
    if (err) return cuda_fail(err, "probe launch");
    return NVFP4_OK;
}

int nvfp4_probe_e2m1(uint32_t first, int64_t n, uint8_t* out, cudaStream_t stream) {
    g_msg[0] = '\0';
    if (n < 0 || n > (int64_t{1} << 32)) return fail(NVFP4_EINVAL, "n must be in [0, 2^32]");
    if (static_cast<uint64_t>(first) + static_cast<uint64_t>(n) > (uint64_t{1} << 32))
        return fail(NVFP4_EINVAL, "first + n must not pass 2^32");
    int rc;
    if ((rc = check_ptr(out, "out", n > 0, 4))) return rc;
    const int err = nvfp4::launch_probe_e2m1(first, n, out, stream);
    if (err) return cuda_fail(err, "probe launch");
    return NVFP4_OK;
}

const char* nvfp4_last_error(void) { return g_msg; }

int nvfp4_abi_version(void) { return 100; }

}  // extern "C"
