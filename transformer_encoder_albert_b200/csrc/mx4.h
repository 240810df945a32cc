// mx4.h -- launchers of the microscaled 4-bit kernels (internal to the .so).
#pragma once
#include "kernels.h"

namespace albert {

// ------------------------------------------------------ microscaled 4-bit path --
// Element types of rows (mirror include/albert.h) and the storage of 4-bit rows:
// mx4.cuh.  nv: nvfp4 (blocks of 16, E4M3 scales times tensor_scale), else mxfp4
// (blocks of 32, E8M0 scales; tensor_scale unused).
enum ElemType : int { kElemBf16 = 0, kElemF32 = 1, kElemF16 = 5 };

struct Mx4QuantArgs {
    const void *x;          // [rows, cols], rows ld elements apart
    int type;               // ElemType
    long long ld;
    int rows, cols;
    bool nv;
    float tensor_scale;
    uint8_t *codes, *scales;
    const int *n_rows;      // device: rows that hold data (<= rows), or nullptr
    const int *status;      // device status word: non-zero skips the work; or nullptr
    int trigger;            // see GemmArgs
};
struct Mx4NormArgs {
    Mx4QuantArgs q;         // x: the rows to normalize; codes, scales: of the normalized rows
    const float *gamma, *beta;
    float eps;
    void *y;                // normalized rows in x's type, or nullptr
    long long ld_y;
};
cudaError_t launch_mx4_quant(const Mx4QuantArgs &a, cudaStream_t s, bool pdl);
cudaError_t launch_mx4_dequant(const uint8_t *codes, const uint8_t *scales, int rows, int cols, bool nv,
                               float tensor_scale, void *out, int type, long long ld, cudaStream_t s);
cudaError_t launch_mx4_norm(const Mx4NormArgs &a, cudaStream_t s, bool pdl);
// *out = bits of the largest |x| as fp32.
cudaError_t launch_amax_bf16(const bf16 *x, size_t n, unsigned *out, cudaStream_t s);

// y = alpha * (A W^T) + bias, GELU_tanh if gelu, + residual; rounded once to out_type,
// or quantized (q, q_scales) from its fp32 value.
struct Mx4GemmArgs {
    const uint8_t *a, *a_scales, *w, *w_scales;
    int M, N, K;
    bool nv;
    float alpha;            // product of the two tensor scales
    const float *bias;      // [N] or nullptr
    int gelu;
    const void *res;        // [M, N] of out_type, or nullptr (as with a 4-bit result)
    long long ld_res;
    void *out;              // nullptr: 4-bit result
    int out_type;
    long long ld_out;
    uint8_t *q, *q_scales;
    float q_ts;
    const int *n_rows;      // device row count (<= M) or nullptr
    int *status;            // device status word: an expired wait is recorded there
    int check_status;       // non-zero: a status already recorded skips the work
    int trigger;
    unsigned long long wait_ns;
    int withhold_loads;     // see GemmArgs
};
// Tensor maps of the products' operands and results.
// Map of a byte row-major [rows, cols] tensor with a {box_cols, box_rows} box.
int make_tmap_u8(CUtensorMap *tm, const void *base, uint64_t rows, uint64_t cols, uint32_t box_cols, uint32_t box_rows,
                 bool swizzle128);
// Map of [rows, cols] 16-bit elements, rows ld elements apart, with a 32x32 box and the
// 64-byte swizzle.
int make_tmap_tile16(CUtensorMap *tm, const void *base, int type, uint64_t rows, uint64_t cols, uint64_t ld);

cudaError_t launch_mx4_gemm(const Mx4GemmArgs &a, int num_sms, cudaStream_t s, bool pdl);

// The same for at most kMx4MaxTokens rows, which it quantizes itself
// when x is given (then a, a_scales are unused): one launch, no workspace.
constexpr int kMx4MaxTokens = 32;
struct Mx4TokArgs : Mx4GemmArgs {
    const void *x;          // [M, K] rows of x_type, or nullptr: a, a_scales
    int x_type;
    long long ld_x;
    float x_ts;
    int vec_x;              // the rows are 16-byte aligned
};
cudaError_t launch_mx4_tokens(const Mx4TokArgs &a, int num_sms, cudaStream_t s);

}  // namespace albert
