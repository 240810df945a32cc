// mx4_quant.cu -- rows to microscaled 4-bit values and back, and LayerNorm with
// a 4-bit result.
//
// Quantizing reads every value once and writes 1/2 byte plus the block's scale
// for it: bound by memory.  A warp takes 256 columns (eight per lane, one 16-byte
// load of 16-bit values) of the four rows r, r+32, r+64, r+96 of a 128-row scale
// tile: four loads in flight per lane, and the four rows' scale words of a tile
// are 16 adjacent bytes.
#include <type_traits>

#include "kernels.h"
#include "mx4.cuh"
#include "sm100_ptx.cuh"

namespace albert {
namespace {

constexpr int kQWarps = 8;

// 4-byte address of the scale word of (row, tile) -- four blocks of one row.
__device__ __forceinline__ size_t scale_word_offset(int row, int tile, int row_tiles) {
    return ((size_t)(row >> 7) * row_tiles + tile) * kMx4TileBytes + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

template <typename T, bool NV>
__global__ void __launch_bounds__(32 * kQWarps)
mx4_quant_kernel(const T *__restrict__ x, long long ld, int rows, int cols, const int *n_rows, float ts, float six_ts,
                 uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, int vec, long long items, const int *status,
                 int trigger) {
    if (trigger) griddep_launch_dependents();
    griddep_wait();
    if (status && *reinterpret_cast<const volatile int *>(status) != 0) return;
    const int lane = threadIdx.x & 31;
    int nr = n_rows ? *reinterpret_cast<const volatile int *>(n_rows) : rows;
    nr = nr < rows ? nr : rows;
    const int chunks = mx4_stages(cols), pitch = mx4_code_pitch(cols);
    const int row_tiles = chunks * Mx4<NV>::kStageTiles;
    // item = (128-row tile, row r of 32, 256-column chunk), chunks innermost
    for (long long it = (long long)blockIdx.x * kQWarps + (threadIdx.x >> 5); it < items;
         it += (long long)gridDim.x * kQWarps) {
        const int chunk = (int)(it % chunks);
        const long long rr = it / chunks;
        const int row0 = (int)(rr >> 5) * 128 + (int)(rr & 31);
        const int col = chunk * kMx4StageCols + lane * 8;
        const int n = cols - col;
        float v[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = row0 + 32 * i;
            load8<T>(x + (size_t)row * ld + col, row < nr ? (n > 0 ? n : 0) : 0, vec != 0, v[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = row0 + 32 * i;
            uint32_t word;
            const uint32_t q = mx4_warp_quant<NV>(v[i], ts, six_ts, lane, word);
            if (row < nr && col / 2 < pitch) *reinterpret_cast<uint32_t *>(codes + (size_t)row * pitch + col / 2) = q;
            constexpr int kTileLanes = Mx4<NV>::kTileCols / 8;
            if (lane % kTileLanes == 0)  // (rows past the end: scale 0, so that a tile is always whole)
                *reinterpret_cast<uint32_t *>(scales + scale_word_offset(row, chunk * Mx4<NV>::kStageTiles + lane / kTileLanes,
                                                                         row_tiles)) = word;
        }
    }
}

template <typename T, bool NV>
__global__ void __launch_bounds__(32 * kQWarps)
mx4_dequant_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int rows, int cols, float ts,
                   T *__restrict__ out, long long ld, int vec, long long items) {
    const int lane = threadIdx.x & 31;
    const int chunks = mx4_stages(cols), pitch = mx4_code_pitch(cols);
    const int row_tiles = chunks * Mx4<NV>::kStageTiles;
    for (long long it = (long long)blockIdx.x * kQWarps + (threadIdx.x >> 5); it < items;
         it += (long long)gridDim.x * kQWarps) {
        const int chunk = (int)(it % chunks);
        const long long rr = it / chunks;
        const int row0 = (int)(rr >> 5) * 128 + (int)(rr & 31);
        const int col = chunk * kMx4StageCols + lane * 8;
        const int n = cols - col;
        uint32_t q[4] = {}, sb[4] = {};
        if (n > 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = row0 + 32 * i;
                if (row >= rows) continue;
                q[i] = __ldg(reinterpret_cast<const uint32_t *>(codes + (size_t)row * pitch + col / 2));
                const int blk = col / Mx4<NV>::kBlock;
                sb[i] = __ldg(scales + scale_word_offset(row, blk >> 2, row_tiles) + (blk & 3));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = row0 + 32 * i;
                if (row >= rows) continue;
                const float s = mx4_scale_value<NV>(sb[i]);
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[j] = __fmul_rn(e2m1_value((q[i] >> (4 * j)) & 15u), s);  // exact
                    if (NV) v[j] = __fmul_rn(v[j], ts);
                }
                store8<T>(out + (size_t)row * ld + col, n, vec != 0, v);
            }
        }
    }
}

// LayerNorm of a row in fp32 (mean, then the mean square of the differences, both
// over the row's values held in registers or read again), y in the input's type,
// and the 4-bit form of the fp32 result.  One CTA per row.
__device__ __forceinline__ float block_sum(float v, float *red, int warps) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += red[i];
    return s;
}

template <typename T, bool NV>
__global__ void __launch_bounds__(32 * kQWarps)
mx4_norm_kernel(const T *__restrict__ x, long long ld, const float *__restrict__ gamma, const float *__restrict__ beta,
                float eps, int rows, int cols, const int *n_rows, float ts, float six_ts, T *__restrict__ y, long long ld_y,
                uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, int vec, int vec_y, int vec_g,
                const int *status, int trigger) {
    __shared__ float red[kQWarps];
    if (trigger) griddep_launch_dependents();
    griddep_wait();
    if (status && *reinterpret_cast<const volatile int *>(status) != 0) return;
    int nr = n_rows ? *reinterpret_cast<const volatile int *>(n_rows) : rows;
    nr = nr < rows ? nr : rows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunks = mx4_stages(cols), pitch = mx4_code_pitch(cols);
    const int row_tiles = chunks * Mx4<NV>::kStageTiles;
    for (int row = blockIdx.x; row < nr; row += gridDim.x) {
        const T *src = x + (size_t)row * ld;
        float sum = 0.f;
        for (int c = warp; c < chunks; c += kQWarps) {
            const int col = c * kMx4StageCols + lane * 8, n = cols - col > 0 ? cols - col : 0;
            float v[8];
            load8<T>(src + col, n, vec != 0, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[i];
        }
        const float mean = block_sum(sum, red, kQWarps) / (float)cols;
        float sq = 0.f;
        for (int c = warp; c < chunks; c += kQWarps) {
            const int col = c * kMx4StageCols + lane * 8, n = cols - col > 0 ? cols - col : 0;
            float v[8];
            load8<T>(src + col, n, vec != 0, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = i < n ? v[i] - mean : 0.f;
                sq = fmaf(d, d, sq);
            }
        }
        const float rstd = rsqrtf(block_sum(sq, red, kQWarps) / (float)cols + eps);
        for (int c = warp; c < chunks; c += kQWarps) {
            const int col = c * kMx4StageCols + lane * 8, n = cols - col > 0 ? cols - col : 0;
            float v[8], g[8], b[8];
            load8<T>(src + col, n, vec != 0, v);
            load8<float>(gamma + col, n, vec_g != 0, g);
            load8<float>(beta + col, n, vec_g != 0, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? fmaf((v[i] - mean) * rstd, g[i], b[i]) : 0.f;
            if (y) store8<T>(y + (size_t)row * ld_y + col, n, vec_y != 0, v);
            uint32_t word;
            const uint32_t q = mx4_warp_quant<NV>(v, ts, six_ts, lane, word);
            if (col / 2 < pitch) *reinterpret_cast<uint32_t *>(codes + (size_t)row * pitch + col / 2) = q;
            constexpr int kTileLanes = Mx4<NV>::kTileCols / 8;
            if (lane % kTileLanes == 0)
                *reinterpret_cast<uint32_t *>(scales + scale_word_offset(row, c * Mx4<NV>::kStageTiles + lane / kTileLanes,
                                                                         row_tiles)) = word;
        }
    }
}

// CTAs of `kernel` that are resident at once, at most `need`.
template <typename K>
cudaError_t resident_grid(K kernel, long long need, int &blocks) {
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, 32 * kQWarps, 0);
    const long long cap = (long long)(per_sm > 0 ? per_sm : 1) * sms;
    blocks = (int)(need < cap ? need : cap);
    return e;
}

inline bool aligned16(const void *p, long long ld, int elem) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * elem) % 16 == 0;
}

template <typename T, bool NV>
cudaError_t quant_typed(const Mx4QuantArgs &a, cudaStream_t s, bool pdl) {
    const long long items = (long long)((a.rows + 127) / 128) * 32 * mx4_stages(a.cols);
    int blocks = 0;
    cudaError_t e = resident_grid(mx4_quant_kernel<T, NV>, (items + kQWarps - 1) / kQWarps, blocks);
    if (e != cudaSuccess) return e;
    const int vec = aligned16(a.x, a.ld, sizeof(T));
    const float six = 6.0f * a.tensor_scale;
    if (pdl)
        return launch_pdl(mx4_quant_kernel<T, NV>, dim3(blocks), dim3(32 * kQWarps), 0, s, static_cast<const T *>(a.x),
                          a.ld, a.rows, a.cols, a.n_rows, a.tensor_scale, six, a.codes, a.scales, vec, items, a.status,
                          a.trigger);
    mx4_quant_kernel<T, NV><<<blocks, 32 * kQWarps, 0, s>>>(static_cast<const T *>(a.x), a.ld, a.rows, a.cols, a.n_rows,
                                                            a.tensor_scale, six, a.codes, a.scales, vec, items, a.status,
                                                            a.trigger);
    return cudaGetLastError();
}

template <typename T, bool NV>
cudaError_t dequant_typed(const uint8_t *codes, const uint8_t *scales, int rows, int cols, float ts, void *out,
                          long long ld, cudaStream_t s) {
    const long long items = (long long)((rows + 127) / 128) * 32 * mx4_stages(cols);
    int blocks = 0;
    cudaError_t e = resident_grid(mx4_dequant_kernel<T, NV>, (items + kQWarps - 1) / kQWarps, blocks);
    if (e != cudaSuccess) return e;
    mx4_dequant_kernel<T, NV><<<blocks, 32 * kQWarps, 0, s>>>(codes, scales, rows, cols, ts, static_cast<T *>(out), ld,
                                                              aligned16(out, ld, sizeof(T)), items);
    return cudaGetLastError();
}

template <typename T, bool NV>
cudaError_t norm_typed(const Mx4NormArgs &a, cudaStream_t s, bool pdl) {
    int blocks = 0;
    cudaError_t e = resident_grid(mx4_norm_kernel<T, NV>, a.q.rows, blocks);
    if (e != cudaSuccess) return e;
    const int vec = aligned16(a.q.x, a.q.ld, sizeof(T)), vec_y = aligned16(a.y, a.ld_y, sizeof(T));
    const int vec_g = aligned16(a.gamma, 4, 4) && aligned16(a.beta, 4, 4);
    const float six = 6.0f * a.q.tensor_scale;
    if (pdl)
        return launch_pdl(mx4_norm_kernel<T, NV>, dim3(blocks), dim3(32 * kQWarps), 0, s, static_cast<const T *>(a.q.x),
                          a.q.ld, a.gamma, a.beta, a.eps, a.q.rows, a.q.cols, a.q.n_rows, a.q.tensor_scale, six,
                          static_cast<T *>(a.y), a.ld_y, a.q.codes, a.q.scales, vec, vec_y, vec_g, a.q.status, a.q.trigger);
    mx4_norm_kernel<T, NV><<<blocks, 32 * kQWarps, 0, s>>>(
        static_cast<const T *>(a.q.x), a.q.ld, a.gamma, a.beta, a.eps, a.q.rows, a.q.cols, a.q.n_rows, a.q.tensor_scale,
        six, static_cast<T *>(a.y), a.ld_y, a.q.codes, a.q.scales, vec, vec_y, vec_g, a.q.status, a.q.trigger);
    return cudaGetLastError();
}

}  // namespace

#define MX4_BY_TYPE(fn, type, nv, ...)                                                        \
    do {                                                                                      \
        switch (type) {                                                                       \
            case kElemBf16: return (nv) ? fn<bf16, true>(__VA_ARGS__) : fn<bf16, false>(__VA_ARGS__);     \
            case kElemF16: return (nv) ? fn<__half, true>(__VA_ARGS__) : fn<__half, false>(__VA_ARGS__);  \
            case kElemF32: return (nv) ? fn<float, true>(__VA_ARGS__) : fn<float, false>(__VA_ARGS__);    \
        }                                                                                     \
        return cudaErrorInvalidValue;                                                         \
    } while (0)

cudaError_t launch_mx4_quant(const Mx4QuantArgs &a, cudaStream_t s, bool pdl) {
    if (a.rows < 1) return cudaSuccess;
    MX4_BY_TYPE(quant_typed, a.type, a.nv, a, s, pdl);
}
cudaError_t launch_mx4_dequant(const uint8_t *codes, const uint8_t *scales, int rows, int cols, bool nv, float ts,
                               void *out, int type, long long ld, cudaStream_t s) {
    if (rows < 1) return cudaSuccess;
    MX4_BY_TYPE(dequant_typed, type, nv, codes, scales, rows, cols, ts, out, ld, s);
}
cudaError_t launch_mx4_norm(const Mx4NormArgs &a, cudaStream_t s, bool pdl) {
    if (a.q.rows < 1) return cudaSuccess;
    MX4_BY_TYPE(norm_typed, a.q.type, a.q.nv, a, s, pdl);
}

}  // namespace albert
