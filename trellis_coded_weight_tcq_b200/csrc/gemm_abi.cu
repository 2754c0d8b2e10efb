// gemm_abi.cu -- C entry points of the batched products and the 8-bit checkpoints:
// host-side checks, workspace layout and launches.  Like every entry point, they
// neither allocate nor synchronise nor keep anything between calls.
#include <stdint.h>

#include "codes.cuh"
#include "gemm.cuh"

using namespace tcq;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;  // rows, columns and tokens

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

bool valid_x(tcq_xdtype t) { return t == TCQ_X_F16 || t == TCQ_X_BF16; }
bool valid_q8(tcq_q8 f) { return f == TCQ_Q8_INT8 || f == TCQ_Q8_E4M3; }
bool valid_act(tcq_activation a) { return a >= TCQ_ACT_NONE && a <= TCQ_ACT_GELU_TANH; }

bool valid_dim(int64_t v) { return v >= 0 && v <= kMaxDim; }

// a [n, cols] array of 16-bit rows: its stride reaches the next row without overlap
bool valid_rows(const void* p, int64_t ld, int64_t cols) { return p && aligned(p, 2) && ld >= cols && ld <= 2 * kMaxDim; }

bool direct(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

int sms()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

tcq_status check_matrix(tcq_dtype dt, int L, int k, int T, int64_t rows, int64_t cols)
{
    if (!valid_dim(rows) || !valid_dim(cols)) return TCQ_ERR_INVALID_ARG;
    if (dt != TCQ_F32 && dt != TCQ_F16 && dt != TCQ_MAD) return TCQ_ERR_INVALID_ARG;
    if (k < 1 || k > TCQ_MAX_K || L < k || L > TCQ_MAX_L || T < 1 || T > TCQ_MAX_T || T % 4 != 0)
        return TCQ_ERR_UNSUPPORTED;
    if (dt == TCQ_F32 && L >= 15) return TCQ_ERR_UNSUPPORTED;  // the table lives in shared memory
    if (cols % T != 0) return TCQ_ERR_INVALID_ARG;
    if ((unsigned long long)rows * (unsigned long long)cols > (1ull << 42)) return TCQ_ERR_INVALID_ARG;
    return TCQ_OK;
}

bool matrix_pointers(const uint32_t* bits, const uint32_t* start, const float* scale, const void* cb, tcq_dtype dt)
{
    return bits && start && aligned(bits, 4) && aligned(start, 4) && (!scale || aligned(scale, 4)) &&
           (dt == TCQ_MAD || (cb && aligned(cb, dt == TCQ_F16 ? 2 : 4)));
}

int code_mode(tcq_dtype dt) { return dt == TCQ_F16 ? 1 : dt == TCQ_MAD ? kMadCodebook : 0; }

CodedMatrix matrix(const uint32_t* bits, const uint32_t* start, const float* scale, const void* cb, tcq_dtype dt, int L,
                   int k, int T, int64_t rows, int64_t cols)
{
    return {bits, start, scale, cb, code_mode(dt), L, k, T,
            tcq_words_per_block(k, T), rows, cols};
}

// Large bfloat16 batches multiply in bfloat16, the operands a bfloat16 layer has anyway: the
// weights are rounded to 8 bits of precision, which leaves the result off by about as much
// again as its own rounding to bfloat16 (2.4e-3 of its norm in all against 1.7e-3 with
// 11-bit weights), and saves the pass that scales the activations to binary16 rows and some
// of the multipliers' power.  Measured with 8 / with 11 bits, 14336 x 4096, in long runs: 4096
// tokens forward 416 / 454 us, input gradient 422 / 494; 512 tokens 95 / 106 and 96 / 108;
// 257 tokens 91 / 101 and 90 / 99.  Up to 256 tokens, where the matrix is mostly decoded
// inside the product, the pass takes a few microseconds, and the weights keep 11 bits.
bool bf16_operands(tcq_xdtype xdtype, int64_t n) { return xdtype == TCQ_X_BF16 && n > 256; }

// Whether weights are stored over a power of two of their table (powers.cuh): a binary32
// table's entries may be of any size; binary16 ones without scales are stored exactly as
// they are, and the computed code's lie below 2 (powers_of).
bool table_power_wanted(tcq_dtype dt, const float* scale) { return dt == TCQ_F32 || (dt == TCQ_F16 && scale); }

// Workspace of a product: the binary16 matrix, its row powers and its table's, the
// binary16 activations (rows of `inner` elements) and theirs.
struct GemmSpace {
    size_t row_pow2, row_exponents, table_top, x, x_pow2, partial, total;
};

// `weights`: bytes of the binary16 matrix; `partial`: of the sums of a reduction's pieces
GemmSpace gemm_space(size_t weights, int64_t rows, int64_t n, int64_t inner, size_t partial)
{
    GemmSpace s;
    s.row_pow2 = align256(weights);
    s.row_exponents = s.row_pow2 + align256((size_t)rows * 4);
    s.table_top = s.row_exponents + align256((size_t)rows);
    s.x = s.table_top + 256;
    s.x_pow2 = s.x + align256((size_t)n * round_up(inner, 8) * 2);
    s.partial = s.x_pow2 + align256((size_t)n * 4);
    s.total = s.partial + align256(partial);
    return s;
}

size_t matrix16_bytes(int64_t rows, int64_t cols) { return (size_t)rows * round_up(cols, 8) * 2; }

GemmSpace forward_space(tcq_dtype dt, int L, int T, int64_t rows, int64_t cols, int64_t n, int num_sms)
{
    if (fused_shape(T, rows, cols, n))
        return gemm_space(0, rows, n, cols, fused_partial_bytes(code_mode(dt), L, rows, cols, n, num_sms));
    return gemm_space(matrix16_bytes(rows, cols), rows, n, cols, gemm_partial_bytes(n, rows, cols, num_sms));
}

GemmSpace dgrad_space(int64_t rows, int64_t cols, int64_t n, int num_sms)
{
    return gemm_space(matrix16_bytes(rows, cols), rows, n, rows, gemm_partial_bytes(n, cols, rows, num_sms));
}

// The checkpoint's values, a copy of dZ (where TMA cannot read it), the pieces' sums.
struct WgradSpace {
    size_t dz, partial, total;
};

WgradSpace wgrad_space(int64_t rows, int64_t cols, int64_t n, int num_sms)
{
    WgradSpace s;
    s.dz = align256((size_t)n * round_up(cols, 8) * 2);
    s.partial = s.dz + align256((size_t)n * round_up(rows, 8) * 2);
    s.total = s.partial + align256(gemm_partial_bytes(rows, cols, n, num_sms));
    return s;
}

Epilogue plain_epilogue(void* out, int64_t ldo)
{
    Epilogue e = {};
    e.out = out;
    e.ldo = ldo;
    return e;
}

tcq_status status(cudaError_t e) { return e == cudaSuccess ? TCQ_OK : TCQ_ERR_CUDA; }

}  // namespace

extern "C" {

size_t tcq_gemm_workspace_bytes(int L, int k, int T, int64_t rows, int64_t cols, int64_t n, tcq_dtype cb_dtype)
{
    if (check_matrix(cb_dtype, L, k, T, rows, cols) != TCQ_OK || !valid_dim(n) || n == 0 || rows == 0 || cols == 0)
        return 0;
    const int num_sms = sms();
    return forward_space(cb_dtype, L, T, rows, cols, n, num_sms > 0 ? num_sms : 148).total;
}

tcq_status tcq_gemm(const uint32_t* bits, const uint32_t* start_state, const float* scale, const void* codebook,
                    tcq_dtype cb_dtype, int L, int k, int T, int64_t rows, int64_t cols, const void* x,
                    tcq_xdtype xdtype, int64_t ldx, int64_t n, const float* bias, tcq_activation act,
                    const void* residual, int64_t ldr, void* y, int64_t ldy, uint8_t* z_codes, uint8_t* z_scales,
                    tcq_q8 z_format, void* workspace, size_t workspace_bytes, tcq_stream_t stream)
{
    const tcq_status shape = check_matrix(cb_dtype, L, k, T, rows, cols);
    if (shape != TCQ_OK) return shape;
    if (!valid_dim(n) || !valid_x(xdtype) || !valid_act(act) || !valid_q8(z_format)) return TCQ_ERR_INVALID_ARG;
    if (n == 0 || rows == 0) return TCQ_OK;
    if (cols == 0 || !matrix_pointers(bits, start_state, scale, codebook, cb_dtype) || !valid_rows(x, ldx, cols) ||
        !valid_rows(y, ldy, rows) || (residual && !valid_rows(residual, ldr, rows)) || (bias && !aligned(bias, 4)) ||
        (z_codes == nullptr) != (z_scales == nullptr))
        return TCQ_ERR_INVALID_ARG;
    const int num_sms = sms();
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const CodedMatrix w = matrix(bits, start_state, scale, codebook, cb_dtype, L, k, T, rows, cols);
    if (n == 1 && !z_codes) {
        if (num_sms <= 0) return TCQ_ERR_CUDA;
        GemvLayerArgs g;
        static_cast<GemvArgs&>(g) = {w.bits, w.start_state, w.scale, w.cb, w.cb_f16, L, k, T, w.W, rows, cols, nullptr,
                                     nullptr};
        g.x16 = x;
        g.x_vec = aligned(x, 8);
        g.e = plain_epilogue(y, ldy);
        g.e.bias = bias;
        g.e.act = act;
        g.e.residual = residual;
        return status(launch_gemv_layer(g, xdtype, num_sms, st));
    }
    if (!workspace || !aligned(workspace, 256)) return TCQ_ERR_INVALID_ARG;
    const GemmSpace sp = forward_space(cb_dtype, L, T, rows, cols, n, num_sms > 0 ? num_sms : 148);
    if (workspace_bytes < sp.total) return TCQ_ERR_WORKSPACE;
    if (num_sms <= 0) return TCQ_ERR_CUDA;
    unsigned int* err = device_error_word(st);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    float* row_pow2 = reinterpret_cast<float*>(ws + sp.row_pow2);
    float* x_pow2 = reinterpret_cast<float*>(ws + sp.x_pow2);
    float* partial = reinterpret_cast<float*>(ws + sp.partial);
    uint32_t* table_top = table_power_wanted(cb_dtype, scale) ? reinterpret_cast<uint32_t*>(ws + sp.table_top) : nullptr;
    const int64_t ldw = round_up(cols, 8);

    const bool fused = fused_shape(T, rows, cols, n);
    GemmProblem p = {x, ldx, ws, ldw, n, rows, cols, 0, xdtype};
    Epilogue ep = plain_epilogue(y, ldy);
    // binary16 rows that TMA can read are used where they are
    const bool scaled = xdtype != TCQ_X_F16 || !direct(x, ldx);
    ScaleRows sx;
    if (scaled) {
        sx.x = x;
        sx.xdtype = xdtype;
        sx.ldx = ldx;
        sx.n = n;
        sx.cols = cols;
        sx.out = ws + sp.x;
        sx.ldo = ldw;
        sx.row_pow2 = x_pow2;
        p.a = ws + sp.x;
        p.lda = ldw;
        ep.row_scale = x_pow2;
    }
    cudaError_t e = cudaSuccess;
    if (bf16_operands(xdtype, n)) {
        e = launch_decode_bf16(w, ws, ldw, num_sms, st);
        if (e == cudaSuccess && !direct(x, ldx)) e = launch_copy16(x, ldx, n, cols, ws + sp.x, ldw, num_sms, st);
        p.fmt = 1;
        if (direct(x, ldx)) {
            p.a = x;
            p.lda = ldx;
        }
        ep.row_scale = nullptr;
        scale = nullptr;  // in the weights
        table_top = nullptr;
    } else if (fused) {
        // a binary32 table's power is found by the product
        if (scaled || scale) e = launch_prepare(sx, powers_of(w, row_pow2, nullptr, w.cb_f16 ? table_top : nullptr), st);
    } else {
        e = launch_decode16(w, ws, ldw, row_pow2, nullptr, table_top, num_sms, st);
        sx.early = true;
        if (e == cudaSuccess && scaled) e = launch_prepare(sx, {}, st);
    }
    if (e != cudaSuccess) return TCQ_ERR_CUDA;
    ep.col_scale = scale ? row_pow2 : nullptr;
    ep.table_top = table_top;
    ep.bias = bias;
    ep.residual = residual;
    ep.ldr = ldr;
    ep.act = act;
    ep.z_codes = z_codes;
    ep.z_scales = z_scales;
    ep.z_format = z_format;
    if (fused) {
        WeightPowers powers;
        powers.row = ep.col_scale;
        powers.staged = table_top && !w.cb_f16;
        if (powers.staged)
            powers.table_out = table_top;
        else
            powers.table = table_top;
        return status(launch_gemm_fused(w, p.a, p.lda, n, xdtype, powers, partial, ep, num_sms, err, scaled || scale, st));
    }
    return status(launch_gemm_tc(kGemmForward, p, ep, partial, num_sms, err, st));
}

size_t tcq_gemm_dgrad_workspace_bytes(int L, int k, int T, int64_t rows, int64_t cols, int64_t n, tcq_dtype cb_dtype)
{
    if (check_matrix(cb_dtype, L, k, T, rows, cols) != TCQ_OK || !valid_dim(n) || n == 0 || rows == 0 || cols == 0)
        return 0;
    const int num_sms = sms();
    return dgrad_space(rows, cols, n, num_sms > 0 ? num_sms : 148).total;
}

tcq_status tcq_gemm_dgrad(const uint32_t* bits, const uint32_t* start_state, const float* scale, const void* codebook,
                          tcq_dtype cb_dtype, int L, int k, int T, int64_t rows, int64_t cols, const void* dz,
                          tcq_xdtype xdtype, int64_t lddz, int64_t n, void* dx, int64_t lddx, void* workspace,
                          size_t workspace_bytes, tcq_stream_t stream)
{
    const tcq_status shape = check_matrix(cb_dtype, L, k, T, rows, cols);
    if (shape != TCQ_OK) return shape;
    if (!valid_dim(n) || !valid_x(xdtype)) return TCQ_ERR_INVALID_ARG;
    if (n == 0 || cols == 0) return TCQ_OK;
    if (!valid_rows(dx, lddx, cols)) return TCQ_ERR_INVALID_ARG;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) return status(cudaMemset2DAsync(dx, (size_t)lddx * 2, 0, (size_t)cols * 2, (size_t)n, st));
    if (!matrix_pointers(bits, start_state, scale, codebook, cb_dtype) || !valid_rows(dz, lddz, rows) || !workspace ||
        !aligned(workspace, 256))
        return TCQ_ERR_INVALID_ARG;
    const int num_sms = sms();
    const GemmSpace sp = dgrad_space(rows, cols, n, num_sms > 0 ? num_sms : 148);
    if (workspace_bytes < sp.total) return TCQ_ERR_WORKSPACE;
    if (num_sms <= 0) return TCQ_ERR_CUDA;
    unsigned int* err = device_error_word(st);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    float* row_pow2 = reinterpret_cast<float*>(ws + sp.row_pow2);
    float* x_pow2 = reinterpret_cast<float*>(ws + sp.x_pow2);
    float* partial = reinterpret_cast<float*>(ws + sp.partial);
    const CodedMatrix w = matrix(bits, start_state, scale, codebook, cb_dtype, L, k, T, rows, cols);
    const int64_t ldw = round_up(cols, 8);

    uint8_t* row_exponents = ws + sp.row_exponents;
    uint32_t* table_top = table_power_wanted(cb_dtype, scale) ? reinterpret_cast<uint32_t*>(ws + sp.table_top) : nullptr;
    GemmProblem p = {dz, lddz, ws, ldw, n, cols, rows, 0, xdtype};
    Epilogue ep = plain_epilogue(dx, lddx);
    if (bf16_operands(xdtype, n)) {
        cudaError_t e = launch_decode_bf16(w, ws, ldw, num_sms, st);
        if (e == cudaSuccess && !direct(dz, lddz)) {
            p.a = ws + sp.x;
            p.lda = round_up(rows, 8);
            e = launch_copy16(dz, lddz, n, rows, ws + sp.x, p.lda, num_sms, st);
        }
        if (e != cudaSuccess) return TCQ_ERR_CUDA;
        p.fmt = 1;
        return status(launch_gemm_tc(kGemmDgrad, p, ep, partial, num_sms, err, st));
    }
    cudaError_t e = launch_decode16(w, ws, ldw, row_pow2, row_exponents, table_top, num_sms, st);
    if (e != cudaSuccess) return TCQ_ERR_CUDA;
    // W's rows run along the reduction: their powers go with dZ's columns, and the table's
    // with them; without scales the epilogue multiplies it in
    if (!scale) ep.table_top = table_top;
    if (xdtype != TCQ_X_F16 || scale || !direct(dz, lddz)) {
        const int64_t ldz = round_up(rows, 8);
        ScaleRows sx;
        sx.x = dz;
        sx.xdtype = xdtype;
        sx.ldx = lddz;
        sx.n = n;
        sx.cols = rows;
        sx.col_exponents = scale ? row_exponents : nullptr;
        sx.table_top = scale ? table_top : nullptr;
        sx.out = ws + sp.x;
        sx.ldo = ldz;
        sx.row_pow2 = x_pow2;
        sx.early = true;
        e = launch_prepare(sx, {}, st);
        if (e != cudaSuccess) return TCQ_ERR_CUDA;
        p.a = ws + sp.x;
        p.lda = ldz;
        ep.row_scale = x_pow2;
    }
    return status(launch_gemm_tc(kGemmDgrad, p, ep, partial, num_sms, err, st));
}

size_t tcq_wgrad8_workspace_bytes(int64_t rows, int64_t cols, int64_t n)
{
    if (!valid_dim(rows) || !valid_dim(cols) || !valid_dim(n) || n == 0 || rows == 0 || cols == 0) return 0;
    const int num_sms = sms();
    return wgrad_space(rows, cols, n, num_sms > 0 ? num_sms : 148).total;
}

tcq_status tcq_wgrad8(const void* dz, tcq_xdtype xdtype, int64_t lddz, const uint8_t* x_codes, const uint8_t* x_scales,
                      tcq_q8 x_format, int64_t n, int64_t rows, int64_t cols, float* dw, int64_t lddw, int accumulate,
                      void* workspace, size_t workspace_bytes, tcq_stream_t stream)
{
    if (!valid_dim(n) || !valid_dim(rows) || !valid_dim(cols) || !valid_x(xdtype) || !valid_q8(x_format))
        return TCQ_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return TCQ_OK;
    if (!dw || !aligned(dw, 4) || lddw < cols || lddw > 2 * kMaxDim) return TCQ_ERR_INVALID_ARG;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (n == 0) {
        if (accumulate) return TCQ_OK;
        return status(cudaMemset2DAsync(dw, (size_t)lddw * 4, 0, (size_t)cols * 4, (size_t)rows, st));
    }
    if (!valid_rows(dz, lddz, rows) || !x_codes || !x_scales || !workspace || !aligned(workspace, 256))
        return TCQ_ERR_INVALID_ARG;
    const int num_sms = sms();
    const WgradSpace sp = wgrad_space(rows, cols, n, num_sms > 0 ? num_sms : 148);
    if (workspace_bytes < sp.total) return TCQ_ERR_WORKSPACE;
    if (num_sms <= 0) return TCQ_ERR_CUDA;
    unsigned int* err = device_error_word(st);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    const int64_t ldq = round_up(cols, 8);
    cudaError_t e = launch_unpack8(x_codes, x_scales, x_format, n, cols, ws, xdtype, ldq, num_sms, st);
    if (e != cudaSuccess) return TCQ_ERR_CUDA;
    GemmProblem p = {dz, lddz, ws, ldq, rows, cols, n, xdtype == TCQ_X_BF16 ? 1 : 0, xdtype};
    if (!direct(dz, lddz)) {
        unsigned char* copy = ws + sp.dz;
        const int64_t ldz = round_up(rows, 8);
        e = launch_copy16(dz, lddz, n, rows, copy, ldz, num_sms, st);
        if (e != cudaSuccess) return TCQ_ERR_CUDA;
        p.a = copy;
        p.lda = ldz;
    }
    Epilogue ep = plain_epilogue(dw, lddw);
    ep.accumulate = accumulate != 0;
    return status(launch_gemm_tc(kGemmWgrad, p, ep, reinterpret_cast<float*>(ws + sp.partial), num_sms, err, st));
}

tcq_status tcq_pack8(const void* x, tcq_xdtype xdtype, int64_t ldx, int64_t n, int64_t cols, tcq_q8 format,
                     uint8_t* codes, uint8_t* scales, tcq_stream_t stream)
{
    if (!valid_dim(n) || !valid_dim(cols) || !valid_x(xdtype) || !valid_q8(format)) return TCQ_ERR_INVALID_ARG;
    if (n == 0 || cols == 0) return TCQ_OK;
    if (!valid_rows(x, ldx, cols) || !codes || !scales) return TCQ_ERR_INVALID_ARG;
    const int num_sms = sms();
    if (num_sms <= 0) return TCQ_ERR_CUDA;
    return status(launch_pack8(x, xdtype, ldx, n, cols, format, codes, scales, num_sms,
                               reinterpret_cast<cudaStream_t>(stream)));
}

tcq_status tcq_unpack8(const uint8_t* codes, const uint8_t* scales, tcq_q8 format, int64_t n, int64_t cols, void* x,
                       tcq_xdtype xdtype, int64_t ldx, tcq_stream_t stream)
{
    if (!valid_dim(n) || !valid_dim(cols) || !valid_x(xdtype) || !valid_q8(format)) return TCQ_ERR_INVALID_ARG;
    if (n == 0 || cols == 0) return TCQ_OK;
    if (!valid_rows(x, ldx, cols) || !codes || !scales) return TCQ_ERR_INVALID_ARG;
    const int num_sms = sms();
    if (num_sms <= 0) return TCQ_ERR_CUDA;
    return status(launch_unpack8(codes, scales, format, n, cols, x, xdtype, ldx, num_sms,
                                 reinterpret_cast<cudaStream_t>(stream)));
}

size_t tcq_act_grad8_workspace_bytes(int64_t n, int64_t rows)
{
    if (!valid_dim(n) || !valid_dim(rows) || n == 0 || rows == 0) return 0;
    return align256((size_t)act_grad8_splits(n, rows) * rows * 4);
}

tcq_status tcq_act_grad8(const void* dy, tcq_xdtype xdtype, int64_t lddy, const uint8_t* z_codes,
                         const uint8_t* z_scales, tcq_q8 z_format, tcq_activation act, int64_t n, int64_t rows, void* dz,
                         int64_t lddz, float* dbias, void* workspace, size_t workspace_bytes, tcq_stream_t stream)
{
    if (!valid_dim(n) || !valid_dim(rows) || !valid_x(xdtype) || !valid_q8(z_format) || !valid_act(act))
        return TCQ_ERR_INVALID_ARG;
    if (rows == 0) return TCQ_OK;
    if (dbias && !aligned(dbias, 4)) return TCQ_ERR_INVALID_ARG;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (n == 0) return dbias ? status(cudaMemsetAsync(dbias, 0, (size_t)rows * 4, st)) : TCQ_OK;
    if (!valid_rows(dy, lddy, rows) || !valid_rows(dz, lddz, rows) ||
        (act != TCQ_ACT_NONE && (!z_codes || !z_scales)))
        return TCQ_ERR_INVALID_ARG;
    if (dbias) {
        if (!workspace || !aligned(workspace, 256)) return TCQ_ERR_INVALID_ARG;
        if (workspace_bytes < tcq_act_grad8_workspace_bytes(n, rows)) return TCQ_ERR_WORKSPACE;
    }
    ActGradArgs a = {dy, lddy, z_codes, z_scales, act, n, rows, dz, lddz,
                     dbias ? static_cast<float*>(workspace) : nullptr, dbias, act_grad8_splits(n, rows)};
    return status(launch_act_grad8(a, xdtype, z_format, st));
}

}  // extern "C"
