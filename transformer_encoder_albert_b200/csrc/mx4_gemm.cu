// mx4_gemm.cu -- the linear layer on microscaled 4-bit operands.
//
// First form: 64x64 tiles, operands read back to fp32 in shared memory, fp32
// products and sums on the CUDA cores.
#include <type_traits>

#include "kernels.h"
#include "mx4.cuh"
#include "sm100_ptx.cuh"

namespace albert {
namespace {

constexpr int TM = 64, TN = 64, TK = 32;

__device__ __forceinline__ float load_elem(const void *p, int type, size_t i) {
    if (type == kElemF32) return static_cast<const float *>(p)[i];
    if (type == kElemF16) return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const bf16 *>(p)[i]);
}
__device__ __forceinline__ void store_elem(void *p, int type, size_t i, float v) {
    if (type == kElemF32) static_cast<float *>(p)[i] = v;
    else if (type == kElemF16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<bf16 *>(p)[i] = __float2bfloat16_rn(v);
}

template <bool NV>
__device__ __forceinline__ float read_value(const uint8_t *codes, const uint8_t *scales, int rows, int K, int row, int k) {
    if (row >= rows || k >= K) return 0.f;
    const uint8_t c = codes[(size_t)row * mx4_code_pitch(K) + k / 2];
    const int blk = k / Mx4<NV>::kBlock, tiles = mx4_stages(K) * Mx4<NV>::kStageTiles;
    const uint8_t sb = scales[((size_t)(row >> 7) * tiles + (blk >> 2)) * kMx4TileBytes + (row & 31) * 16 +
                              ((row >> 5) & 3) * 4 + (blk & 3)];
    return e2m1_value((k & 1) ? c >> 4 : c & 15) * mx4_scale_value<NV>(sb);
}

template <bool NV>
__global__ void __launch_bounds__(256) mx4_gemm_kernel(const Mx4GemmArgs p) {
    __shared__ float sa[TM][TK + 1], sb[TN][TK + 1];
    __shared__ float st[TM][TN + 1];
    if (p.trigger) griddep_launch_dependents();
    griddep_wait();
    if (p.check_status && *reinterpret_cast<const volatile int *>(p.status) != 0) return;
    int nr = p.n_rows ? *reinterpret_cast<const volatile int *>(p.n_rows) : p.M;
    nr = nr < p.M ? nr : p.M;
    const int m0 = blockIdx.y * TM, n0 = blockIdx.x * TN, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    if (m0 >= nr) return;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += TK) {
        for (int i = threadIdx.x; i < TM * TK; i += 256) {
            sa[i / TK][i % TK] = read_value<NV>(p.a, p.a_scales, nr, p.K, m0 + i / TK, k0 + i % TK);
            sb[i / TK][i % TK] = read_value<NV>(p.w, p.w_scales, p.N, p.K, n0 + i / TK, k0 + i % TK);
        }
        __syncthreads();
        for (int k = 0; k < TK; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[ty * 4 + i][k], sb[tx * 4 + j][k], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int row = m0 + ty * 4 + i, col = n0 + tx * 4 + j;
            float v = 0.f;
            if (row < nr && col < p.N) {
                v = p.alpha * acc[i][j] + (p.bias ? p.bias[col] : 0.f);
                if (p.gelu) v = v / (1.0f + __expf(-1.5957691216057308f * (v + 0.044715f * v * v * v)));
                if (p.res) v += load_elem(p.res, p.out_type, (size_t)row * p.ld_res + col);
                if (p.out) store_elem(p.out, p.out_type, (size_t)row * p.ld_out + col, v);
            }
            st[ty * 4 + i][tx * 4 + j] = v;
        }
    if (!p.q) return;
    __syncthreads();
    constexpr int kB = Mx4<NV>::kBlock, kPer = TN / kB;
    const int tiles = mx4_stages(p.N) * Mx4<NV>::kStageTiles, pitch = mx4_code_pitch(p.N);
    for (int i = threadIdx.x; i < TM * kPer; i += 256) {
        const int r = i / kPer, row = m0 + r, c0 = (i % kPer) * kB, blk = (n0 + c0) / kB;
        if (row >= nr || (n0 + c0) / 2 >= pitch) continue;
        uint32_t m = 0;
        for (int j = 0; j < kB; ++j) m = umax(m, abs_bits(st[r][c0 + j]));
        const Mx4Scale s = mx4_block_scale<NV>(m, p.q_ts, 6.0f * p.q_ts);
        for (int j = 0; j < kB; j += 8) {
            float y[8];
            for (int e = 0; e < 8; ++e) y[e] = __fmul_rn(st[r][c0 + j + e], s.mul);
            *reinterpret_cast<uint32_t *>(p.q + (size_t)row * pitch + (n0 + c0 + j) / 2) = s.zero ? 0u : cvt_e2m1x8(y);
        }
        p.q_scales[((size_t)(row >> 7) * tiles + (blk >> 2)) * kMx4TileBytes + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
                   (blk & 3)] = (uint8_t)s.byte;
    }
    // the scale bytes between the last block and the end of the row's tiles are 0
    const int last = (pitch * 2) / kB, all = tiles * 4;
    if (blockIdx.x == gridDim.x - 1)
        for (int i = threadIdx.x; i < TM * (all - last); i += 256) {
            const int row = m0 + i / (all - last), blk = last + i % (all - last);
            if (row < nr)
                p.q_scales[((size_t)(row >> 7) * tiles + (blk >> 2)) * kMx4TileBytes + (row & 31) * 16 +
                           ((row >> 5) & 3) * 4 + (blk & 3)] = 0;
        }
}

}  // namespace

cudaError_t launch_mx4_gemm(const Mx4GemmArgs &a, int num_sms, cudaStream_t s, bool pdl) {
    (void)num_sms;
    if (a.M < 1) return cudaSuccess;
    const dim3 grid((a.N + TN - 1) / TN, (a.M + TM - 1) / TM);
    if (pdl) return launch_pdl(a.nv ? mx4_gemm_kernel<true> : mx4_gemm_kernel<false>, grid, dim3(256), 0, s, a);
    if (a.nv) mx4_gemm_kernel<true><<<grid, 256, 0, s>>>(a);
    else mx4_gemm_kernel<false><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace albert
