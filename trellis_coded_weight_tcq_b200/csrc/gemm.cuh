// gemm.cuh -- internal launch interface of the batched products with a
// trellis-coded matrix, their gradients and the 8-bit checkpoints.
#pragma once

#include "codes.cuh"
#include "common.cuh"

namespace tcq {

// A trellis-coded matrix (tcq_gemv's layout).
struct CodedMatrix {
    const uint32_t* bits;
    const uint32_t* start_state;
    const float* scale;  // [rows * cols / T] or nullptr
    const void* cb;
    int cb_f16;          // 0 binary32 table, 1 binary16 table, kMadCodebook computed
    int L, K, T, W;
    long long rows, cols;
};

// What happens to a product before it is stored.
struct Epilogue {
    const float* row_scale;  // power of two per output row, or nullptr
    const float* col_scale;  // power of two per output column, or nullptr
    const uint32_t* table_top;  // the table's power (table_power), in all outputs, or nullptr
    const float* bias;       // per output column, or nullptr
    const void* residual;    // output type, or nullptr
    long long ldr;
    void* out;
    long long ldo;
    int act;
    uint8_t* z_codes;        // [m, n] contiguous, or nullptr
    uint8_t* z_scales;       // [m, ceil(n / 32)]
    int z_format;
    int accumulate;          // fp32 outputs: add to what is there
};

// One token of the forward product (gemv.cu): the matrix-vector kernels on a 16-bit
// vector, weights in fp32, with the epilogue's bias, activation and residual.
struct GemvLayerArgs : GemvArgs {
    const void* x16;
    bool x_vec;  // 8-byte aligned
    Epilogue e;
};
cudaError_t launch_gemv_layer(const GemvLayerArgs& a, int xdtype, int num_sms, cudaStream_t stream);

enum GemmKind { kGemmForward = 0, kGemmDgrad = 1, kGemmWgrad = 2 };

// out[m, n] = epilogue(sum_k a b), 16-bit operands (fmt 0 binary16, 1 bfloat16):
//   forward  a [m, k] row-major, b [n, k] row-major
//   dgrad    a [m, k] row-major, b [k, n] row-major
//   wgrad    a [k, m] row-major, b [k, n] row-major, fp32 out
// Leading dimensions in elements, multiples of 8; bases 16-byte aligned.
struct GemmProblem {
    const void* a;
    long long lda;
    const void* b;
    long long ldb;
    long long m, n, k;
    int fmt;
    int xdtype;  // output type of forward and dgrad
};

// Workspace of a product with few tiles, whose reduction is cut into pieces (0: none).
size_t gemm_partial_bytes(long long m, long long n, long long k, int num_sms);
cudaError_t launch_gemm_tc(GemmKind kind, const GemmProblem& p, const Epilogue& e, float* partial, int num_sms,
                           unsigned int* err, cudaStream_t stream);

// The powers that a weight is stored over; nullptr: 1.
struct WeightPowers {
    const float* row = nullptr;       // per row
    const uint32_t* table = nullptr;  // of a binary16 table (table_power)
    // of a binary32 table, small enough that every CTA finds it from its own copy: `staged`,
    // and where to leave it for the epilogue, or nullptr
    bool staged = false;
    uint32_t* table_out = nullptr;
};

// W as binary16 [rows, ldw], each weight over its row's power of two (row_pow2[r] and its
// exponent field row_exponents[r], or nullptr; written when the matrix has scales) and
// over the table's (table_top, written unless it is nullptr: with row_exponents before this
// launch, else by it or before it).
cudaError_t launch_decode16(const CodedMatrix& w, void* out, long long ldw, float* row_pow2, uint8_t* row_exponents,
                            uint32_t* table_top, int num_sms, cudaStream_t stream);

// W as bfloat16, each weight scale * codeword rounded once.
cudaError_t launch_decode_bf16(const CodedMatrix& w, void* out, long long ldw, int num_sms, cudaStream_t stream);

// x [n, cols] as binary16 rows over a power of two each (row_pow2[n]).  col_exponents (or
// nullptr, 8-byte aligned): fp32 exponent fields of powers of two that multiply the
// columns first, each with the power of table_top (or nullptr).  `early`: the launch before it in the stream is one of this call's
// (launch_decode16), which it may run beside; the exponents may then be those of the row
// powers that launch_decode16 read.
struct ScaleRows {
    const void* x = nullptr;
    int xdtype = TCQ_X_F16;
    long long ldx = 0, n = 0, cols = 0;
    const uint8_t* col_exponents = nullptr;
    const uint32_t* table_top = nullptr;
    void* out = nullptr;
    long long ldo = 0;
    float* row_pow2 = nullptr;
    bool early = false;
    bool vec = false;  // set by the launch: rows that 16-byte loads can read
};

// out[r] for the rows of a coded matrix, per_row scales each: the least power of two
// above the largest finite |scale|, times 2^-down, and its exponent field (or nullptr).  table_top
// [kTableParts], unless nullptr: the largest finite magnitudes of the table's parts.
struct RowPowers {
    const float* scale = nullptr;
    long long rows = 0;
    int per_row = 0, down = 0;
    float* out = nullptr;
    uint8_t* exponents = nullptr;
    const void* table = nullptr;
    int table_f16 = 0, table_log2 = 0;
    uint32_t* table_top = nullptr;
};

// What to ask for the powers of a matrix, those of its rows where it has scales.
inline RowPowers powers_of(const CodedMatrix& w, float* row_pow2, uint8_t* row_exponents, uint32_t* table_top)
{
    RowPowers p;
    if (w.scale) {
        p.scale = w.scale;
        p.rows = w.rows;
        p.per_row = (int)(w.cols / w.T);
        // the computed code's numbers are below 2: its part of the power is known
        p.down = w.cb_f16 == kMadCodebook ? 14 : 0;
        p.out = row_pow2;
        p.exponents = row_exponents;
    }
    p.table = w.cb;
    p.table_f16 = w.cb_f16;
    p.table_log2 = w.L;
    p.table_top = table_top;
    return p;
}

// Any of them (n == 0, rows == 0, no table_top: not wanted), in one launch.
cudaError_t launch_prepare(ScaleRows a, RowPowers p, cudaStream_t stream);

// 16-bit rows copied to another stride, beside the launch before it in the stream (one of
// this call's that neither reads nor writes these rows).
cudaError_t launch_copy16(const void* x, long long ldx, long long n, long long cols, void* out, long long ldo,
                          int num_sms, cudaStream_t stream);

// The forward product with the decoding inside it, for small batches (fused_shape):
// x binary16 [n, cols] (ldx a multiple of 8, 16-byte aligned).  `early`: the launch
// before it in the stream is one of this call's, which it may start beside.
bool fused_shape(int T, long long rows, long long cols, long long n);
size_t fused_partial_bytes(int cb_f16, int L, long long rows, long long cols, long long n, int num_sms);
cudaError_t launch_gemm_fused(const CodedMatrix& w, const void* x, long long ldx, long long n, int xdtype,
                              const WeightPowers& powers, float* partial, const Epilogue& e, int num_sms, unsigned int* err,
                              bool early, cudaStream_t stream);

cudaError_t launch_pack8(const void* x, int xdtype, long long ldx, long long n, long long cols, int format,
                         uint8_t* codes, uint8_t* scales, int num_sms, cudaStream_t stream);
cudaError_t launch_unpack8(const uint8_t* codes, const uint8_t* scales, int format, long long n, long long cols,
                           void* x, int xdtype, long long ldx, int num_sms, cudaStream_t stream);

struct ActGradArgs {
    const void* dy;
    long long lddy;
    const uint8_t* z_codes;
    const uint8_t* z_scales;
    int act;
    long long n, rows;
    void* dz;
    long long lddz;
    float* partial;  // [splits, rows], or nullptr: no dbias
    float* dbias;
    int splits;      // row ranges
};
int act_grad8_splits(long long n, long long rows);
cudaError_t launch_act_grad8(const ActGradArgs& a, int xdtype, int format, cudaStream_t stream);

}  // namespace tcq
