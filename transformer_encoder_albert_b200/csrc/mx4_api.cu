// mx4_api.cu -- the C entries of the microscaled 4-bit operators (include/albert.h):
// checks of their arguments and their launches.
#include <atomic>
#include <cmath>
#include <mutex>

#include "albert.h"
#include "mx4.cuh"
#include "mx4.h"

using namespace albert;

namespace {

// Status word of the linear layers' bounded waits, one per device, and where a query puts
// what it has taken from it: in one step, so that no status recorded meanwhile is lost.
__device__ int g_mx4_status, g_mx4_taken;
__global__ void take_status() { g_mx4_taken = atomicExch(&g_mx4_status, 0); }

constexpr int kMaxCols = 1 << 24, kMaxRows = 1 << 30;
constexpr float kMinScale = 7.888609052210118e-31f, kMaxScale = 1.2676506002282294e30f;  // 2^-100, 2^100

bool is_format(int fmt) { return fmt == ALBERT_MXFP4 || fmt == ALBERT_NVFP4; }
bool is_type(int t) { return t == ALBERT_BF16 || t == ALBERT_FP32 || t == ALBERT_FP16; }
int elem_size(int t) { return t == ALBERT_FP32 ? 4 : 2; }
bool scale_ok(int fmt, float ts) { return fmt == ALBERT_MXFP4 || (ts >= kMinScale && ts <= kMaxScale); }
bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool cols_ok(int c) { return c >= 1 && c <= kMaxCols; }
bool rows_ok(int r) { return r >= 0 && r <= kMaxRows; }

size_t scales_bytes(int rows, int cols, bool nv) {
    return (size_t)((rows + 127) / 128) * mx4_stages(cols) * (nv ? 4 : 2) * kMx4TileBytes;
}
size_t codes_bytes(int rows, int cols) { return (size_t)rows * mx4_code_pitch(cols); }
size_t up16(size_t n) { return (n + 15) / 16 * 16; }

int status_of(cudaError_t e) { return e == cudaSuccess ? ALBERT_OK : ALBERT_ERR_CUDA; }

// SM count and status word of the current device, looked up once per device.
cudaError_t device_info(int &sms, int *&status) {
    static std::atomic<int> known_sms[64];
    static std::atomic<int *> known_status[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (status = known_status[dev].load(std::memory_order_acquire)) != nullptr) {
        sms = known_sms[dev].load(std::memory_order_relaxed);
        return cudaSuccess;
    }
    void *p = nullptr;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaGetSymbolAddress(&p, g_mx4_status);
    if (e != cudaSuccess) return e;
    status = static_cast<int *>(p);
    if (dev < 64) {
        known_sms[dev].store(sms, std::memory_order_relaxed);
        known_status[dev].store(status, std::memory_order_release);
    }
    return cudaSuccess;
}

// Checks shared by the entries that write a 4-bit tensor from rows of x.
int check_rows(const void *x, int x_type, long long ld, int rows, int cols, int fmt, float ts, const void *codes,
               const void *scales) {
    if (!rows_ok(rows) || !cols_ok(cols) || ld < cols) return ALBERT_ERR_SHAPE;
    if (!is_format(fmt) || !is_type(x_type) || !scale_ok(fmt, ts)) return ALBERT_ERR_CONFIG;
    if (!aligned(x, elem_size(x_type)) || !aligned(codes, 16) || !aligned(scales, 16)) return ALBERT_ERR_CONFIG;
    return ALBERT_OK;
}

// Whether any of the rows at a (wa bytes each, la apart) shares a byte with any of those at b.
bool rows_overlap(const void *a, long long la, long long wa, const void *b, long long lb, long long wb, int rows) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    if (pa + (rows - 1) * la + wa <= pb || pb + (rows - 1) * lb + wb <= pa) return false;
    for (int i = 0; i < rows; ++i)
        for (int j = 0; j < rows; ++j)
            if (pa + i * la < pb + j * lb + wb && pb + j * lb < pa + i * la + wa) return true;
    return false;
}

// The linear layer; wait_ns, withhold: as in GemmArgs.
int linear(const albert_mx4_linear_args *p, void *stream, unsigned long long wait_ns, int withhold) {
    if (!p) return ALBERT_ERR_NULL;
    if (!rows_ok(p->rows) || !cols_ok(p->n) || !cols_ok(p->k)) return ALBERT_ERR_SHAPE;
    if (p->rows == 0) return ALBERT_OK;
    if (!p->w_codes || !p->w_scales) return ALBERT_ERR_NULL;
    if (!p->x && (!p->a_codes || !p->a_scales)) return ALBERT_ERR_NULL;
    if (!p->out && (!p->q_codes || !p->q_scales)) return ALBERT_ERR_NULL;
    const size_t ws = p->x ? albert_mx4_linear_workspace_bytes(p->rows, p->k, p->fmt) : 0;
    if (ws && !p->workspace) return ALBERT_ERR_NULL;
    if (p->x && p->ld_x < p->k) return ALBERT_ERR_SHAPE;
    if (p->out && p->ld_out < p->n) return ALBERT_ERR_SHAPE;
    if (p->residual && p->ld_residual < p->n) return ALBERT_ERR_SHAPE;
    if (!is_format(p->fmt) || (p->x && !is_type(p->x_type)) || ((p->out || p->residual) && !is_type(p->out_type)))
        return ALBERT_ERR_CONFIG;
    if (!scale_ok(p->fmt, p->x_scale) || !scale_ok(p->fmt, p->w_scale) || (!p->out && !scale_ok(p->fmt, p->q_scale)))
        return ALBERT_ERR_CONFIG;
    if (!aligned(p->w_codes, 16) || !aligned(p->w_scales, 16) || !aligned(p->bias, 4) ||
        (p->x ? !aligned(p->x, elem_size(p->x_type)) : !aligned(p->a_codes, 16) || !aligned(p->a_scales, 16)) ||
        (ws && !aligned(p->workspace, 16)) || (p->residual && !aligned(p->residual, elem_size(p->out_type))) ||
        (p->out ? !aligned(p->out, elem_size(p->out_type)) : !aligned(p->q_codes, 16) || !aligned(p->q_scales, 16)))
        return ALBERT_ERR_CONFIG;
    if (p->gelu != 0 && p->gelu != 1) return ALBERT_ERR_CONFIG;
    if (p->residual && !p->out) return ALBERT_ERR_CONFIG;
    // (a CTA of the few-row kernel may write its columns while another still reads x)
    if (p->rows <= kMx4MaxTokens && p->x && p->out) {
        const long long ex = elem_size(p->x_type), eo = elem_size(p->out_type);
        if (rows_overlap(p->x, p->ld_x * ex, p->k * ex, p->out, p->ld_out * eo, p->n * eo, p->rows)) return ALBERT_ERR_CONFIG;
    }
    // the product of the tensor scales multiplies the fp32 sum: far from fp32's limits
    if (p->fmt == ALBERT_NVFP4 && !(p->x_scale * p->w_scale >= kMinScale && p->x_scale * p->w_scale <= kMaxScale))
        return ALBERT_ERR_CONFIG;

    const bool nv = p->fmt == ALBERT_NVFP4;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms = 0;
    int *status = nullptr;
    cudaError_t e = device_info(sms, status);
    if (e != cudaSuccess) return ALBERT_ERR_CUDA;
    Mx4TokArgs g{};
    g.w = static_cast<const uint8_t *>(p->w_codes);
    g.w_scales = static_cast<const uint8_t *>(p->w_scales);
    g.M = p->rows; g.N = p->n; g.K = p->k;
    g.nv = nv;
    g.alpha = nv ? p->x_scale * p->w_scale : 1.0f;
    g.bias = p->bias;
    g.gelu = p->gelu;
    g.res = p->residual; g.ld_res = p->ld_residual;
    g.out = p->out; g.out_type = p->out_type; g.ld_out = p->ld_out;
    if (!p->out) {
        g.q = static_cast<uint8_t *>(p->q_codes);
        g.q_scales = static_cast<uint8_t *>(p->q_scales);
        g.q_ts = nv ? p->q_scale : 1.0f;
    }
    g.status = status;
    g.wait_ns = wait_ns;
    g.withhold_loads = withhold;
    g.a = static_cast<const uint8_t *>(p->a_codes);
    g.a_scales = static_cast<const uint8_t *>(p->a_scales);
    if (p->rows <= kMx4MaxTokens) {
        g.x = p->x;
        g.x_type = p->x_type;
        g.ld_x = p->ld_x;
        g.x_ts = nv ? p->x_scale : 1.0f;
        g.vec_x = aligned(p->x, 16) && p->ld_x * elem_size(p->x_type) % 16 == 0;
        return status_of(launch_mx4_tokens(g, sms, s));
    }
    if (p->x) {
        Mx4QuantArgs q{};
        q.x = p->x; q.type = p->x_type; q.ld = p->ld_x; q.rows = p->rows; q.cols = p->k;
        q.nv = nv;
        q.tensor_scale = nv ? p->x_scale : 1.0f;
        q.codes = static_cast<uint8_t *>(p->workspace);
        q.scales = q.codes + up16(codes_bytes(p->rows, p->k));
        // (its grid is resident at once, so the product's CTAs only take SMs it has left)
        q.trigger = 1;
        if ((e = launch_mx4_quant(q, s, false)) != cudaSuccess) return ALBERT_ERR_CUDA;
        g.a = q.codes;
        g.a_scales = q.scales;
    }
    return status_of(launch_mx4_gemm(g, sms, s, p->x != nullptr));
}

}  // namespace

extern "C" {

size_t albert_mx4_codes_bytes(int rows, int cols) { return rows < 1 || !rows_ok(rows) || !cols_ok(cols) ? 0 : codes_bytes(rows, cols); }

size_t albert_mx4_scales_bytes(int rows, int cols, int fmt) {
    return rows < 1 || !rows_ok(rows) || !cols_ok(cols) || !is_format(fmt) ? 0 : scales_bytes(rows, cols, fmt == ALBERT_NVFP4);
}

int albert_mx4_quantize(const void *x, int x_type, long long ld_x, int rows, int cols, int fmt, float tensor_scale,
                        void *codes, void *scales, void *stream) {
    if (rows == 0 && cols_ok(cols)) return ALBERT_OK;
    if (!x || !codes || !scales) return ALBERT_ERR_NULL;
    if (int rc = check_rows(x, x_type, ld_x, rows, cols, fmt, tensor_scale, codes, scales)) return rc;
    Mx4QuantArgs a{};
    a.x = x; a.type = x_type; a.ld = ld_x; a.rows = rows; a.cols = cols;
    a.nv = fmt == ALBERT_NVFP4;
    a.tensor_scale = a.nv ? tensor_scale : 1.0f;
    a.codes = static_cast<uint8_t *>(codes);
    a.scales = static_cast<uint8_t *>(scales);
    return status_of(launch_mx4_quant(a, static_cast<cudaStream_t>(stream), false));
}

int albert_mx4_dequantize(const void *codes, const void *scales, int rows, int cols, int fmt, float tensor_scale,
                          void *out, int out_type, long long ld_out, void *stream) {
    if (rows == 0 && cols_ok(cols)) return ALBERT_OK;
    if (!codes || !scales || !out) return ALBERT_ERR_NULL;
    if (int rc = check_rows(out, out_type, ld_out, rows, cols, fmt, tensor_scale, codes, scales)) return rc;
    const bool nv = fmt == ALBERT_NVFP4;
    return status_of(launch_mx4_dequant(static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), rows,
                                        cols, nv, nv ? tensor_scale : 1.0f, out, out_type, ld_out,
                                        static_cast<cudaStream_t>(stream)));
}

int albert_mx4_layer_norm(const void *x, int x_type, long long ld_x, const float *gamma, const float *beta, float eps,
                          int rows, int cols, int fmt, float tensor_scale, void *y, long long ld_y, void *codes,
                          void *scales, void *stream) {
    if (rows == 0 && cols_ok(cols)) return ALBERT_OK;
    if (!x || !gamma || !beta || !codes || !scales) return ALBERT_ERR_NULL;
    if (int rc = check_rows(x, x_type, ld_x, rows, cols, fmt, tensor_scale, codes, scales)) return rc;
    if (y && ld_y < cols) return ALBERT_ERR_SHAPE;
    if (!(eps >= 0.f) || !std::isfinite(eps) || (y && !aligned(y, elem_size(x_type))) || !aligned(gamma, 4) ||
        !aligned(beta, 4))
        return ALBERT_ERR_CONFIG;
    Mx4NormArgs a{};
    a.q.x = x; a.q.type = x_type; a.q.ld = ld_x; a.q.rows = rows; a.q.cols = cols;
    a.q.nv = fmt == ALBERT_NVFP4;
    a.q.tensor_scale = a.q.nv ? tensor_scale : 1.0f;
    a.q.codes = static_cast<uint8_t *>(codes);
    a.q.scales = static_cast<uint8_t *>(scales);
    a.gamma = gamma; a.beta = beta; a.eps = eps; a.y = y; a.ld_y = ld_y;
    return status_of(launch_mx4_norm(a, static_cast<cudaStream_t>(stream), false));
}

size_t albert_mx4_linear_workspace_bytes(int rows, int k, int fmt) {
    if (rows < 1 || !rows_ok(rows) || !cols_ok(k) || !is_format(fmt) || rows <= kMx4MaxTokens) return 0;
    return up16(codes_bytes(rows, k)) + scales_bytes(rows, k, fmt == ALBERT_NVFP4);
}

int albert_mx4_linear(const albert_mx4_linear_args *p, void *stream) { return linear(p, stream, 0, 0); }

int albert_test_mx4_linear_stall(const albert_mx4_linear_args *p, long long wait_ns, void *stream) {
    return wait_ns < 1 ? ALBERT_ERR_CONFIG : linear(p, stream, (unsigned long long)wait_ns, 1);
}

int albert_mx4_get_status(void *stream) {
    static std::mutex one;  // (queries of one device share the word they are taken to)
    int st = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return ALBERT_ERR_CUDA;
    const std::lock_guard<std::mutex> hold(one);
    take_status<<<1, 1, 0, s>>>();
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyFromSymbolAsync(&st, g_mx4_taken, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return ALBERT_ERR_CUDA;
    return st;
}

}  // extern "C"
