// mx4_quant.cu -- rows to microscaled 4-bit values and back, and LayerNorm with
// a 4-bit result.
//
// Quantizing reads every value once and writes 1/2 byte plus the block's scale for
// it, so memory is its floor; what it came down to was instructions (106 per lane and
// eight values at first, 65% of the issue slots).  Here a lane takes 16 consecutive
// values (one 32-byte load of 16-bit values), which halves the work per block scale
// and leaves one shuffle (mxfp4) or none (nvfp4) for it; 16-bit magnitudes are
// compared two at a time; whole chunks take a path without bounds.  A half-warp
// covers 256 columns of a row, a warp the rows r and r + 32 of a 128-row scale tile,
// and the next such pair's loads are in flight while one is converted.
#include <algorithm>
#include <type_traits>

#include "mx4.cuh"
#include "mx4.h"
#include "sm100_ptx.cuh"

namespace albert {
namespace {

constexpr int kQWarps = 8;

// 4-byte address of the scale word of (row, tile) -- four blocks of one row.
__device__ __forceinline__ size_t scale_word_offset(int row, int tile, int row_tiles) {
    return ((size_t)(row >> 7) * row_tiles + tile) * kMx4TileBytes + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// The scale bytes of the rows between the last and the end of its tile are 0, as the quantiser
// leaves them: equal calls leave equal tiles.  By all threads of the grid; a thread takes the
// four rows that share 16 bytes of a tile.
__device__ __forceinline__ void zero_past_rows(uint8_t *scales, int rows, int row_tiles) {
    const int in_tile = rows & 127;
    if (rows <= 0 || in_tile == 0) return;
    uint8_t *last = scales + (size_t)(rows >> 7) * row_tiles * kMx4TileBytes;
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < row_tiles * 32; i += gridDim.x * blockDim.x) {
        const int r = i & 31;
        uint32_t *word = reinterpret_cast<uint32_t *>(last + (size_t)i * 16);
        if (r >= in_tile) {
            *reinterpret_cast<uint4 *>(word) = make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int q = 1; q < 4; ++q)
                if (r + 32 * q >= in_tile) word[q] = 0;
        }
    }
}

// A warp's walk over (row pair, chunk) items with a grid stride, chunks innermost:
// one division at the start, none per item.  Pair g is the rows 128 (g / 64) +
// 64 (g / 32 % 2) + g % 32 and the row 32 below.
struct Walk {
    int chunk, chunks, dc;
    int pair, dp;  // (rows <= 2^30: pairs, and a step past them, fit)
    __device__ __forceinline__ Walk(int chunks_, int first, int stride) : chunks(chunks_) {
        pair = first / chunks_;
        chunk = first - pair * chunks_;
        dp = stride / chunks_;
        dc = stride - dp * chunks_;
    }
    __device__ __forceinline__ void next() {
        chunk += dc;
        pair += dp;
        if (chunk >= chunks) {
            chunk -= chunks;
            ++pair;
        }
    }
    __device__ __forceinline__ int row0() const { return (pair >> 6) * 128 + ((pair >> 5) & 1) * 64 + (pair & 31); }
};

__device__ __forceinline__ void ld_global_v8(const void *p, uint32_t *w) {
    asm("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p));
}
__device__ __forceinline__ void ld_cached_v8(const float *p, float (&v)[8]) {
    asm("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]) : "l"(p));
}
__device__ __forceinline__ void st_global_v8(void *p, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}

// Sixteen consecutive values as stored: 8 words, or 16 for fp32.  vec: 2 = p is 32-byte
// aligned, 1 = 16-byte, 0 = neither.
template <typename T>
struct Raw16 {
    Raw8<T> h[2];
};
template <typename T>
__device__ __forceinline__ Raw16<T> load_raw16(const T *p, int n, int vec) {
    Raw16<T> r;
    if (vec == 2 && n >= 16) {
        if constexpr (sizeof(T) == 4) {
            ld_global_v8(p, r.h[0].w);
            ld_global_v8(p + 8, r.h[1].w);
        } else {
            uint32_t w[8];
            ld_global_v8(p, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r.h[0].w[i] = w[i];
                r.h[1].w[i] = w[4 + i];
            }
        }
    } else {
        r.h[0] = load_raw8<T>(p, n, vec != 0);
        r.h[1] = load_raw8<T>(p + 8, n - 8, vec != 0);
    }
    return r;
}

// Rows that are aligned to their type only (an odd row stride): a warp moves 256 columns of
// one row in consecutive 4-byte words, aligned down for 16-bit types, and hands them over
// through shared memory -- one value per access cost a lane 16 loads or stores 32 bytes
// apart (8192 x 1001 bf16: quantised in 11.9 us, 9.3 now; read back in 54, 7.1 now).
template <typename T>
constexpr int kSegWords = sizeof(T) == 4 ? 256 : 132;  // (16-bit: 129, up to a multiple of 16 bytes)
template <typename T>
struct Seg {  // as loaded: nothing waits for the values before they are staged
    uint32_t w[sizeof(T) == 4 ? 8 : 4];
    unsigned short edge;  // (16-bit) lane 0: the first value if its word starts before the row; lane 1: a last one alone in its word
};
// 1 if a 16-bit row starts in the upper half of a 4-byte word.
template <typename T>
__device__ __forceinline__ int seg_shift(const T *p) {
    return sizeof(T) == 4 ? 0 : (int)(reinterpret_cast<uintptr_t>(p) >> 1) & 1;
}
// The first n (at most 256) values at src; the others are 0.
template <typename T>
__device__ __forceinline__ Seg<T> seg_load(const T *src, int n, int lane) {
    Seg<T> r = {};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane + 32 * i < n) r.w[i] = __ldg(reinterpret_cast<const uint32_t *>(src) + lane + 32 * i);
    } else {
        n = n < kMx4StageCols ? n : kMx4StageCols;
        const int s = seg_shift(src);
        const uint32_t *words = reinterpret_cast<const uint32_t *>(src - s);  // word o: values 2 o - s, 2 o - s + 1
        const unsigned short *halves = reinterpret_cast<const unsigned short *>(src);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int o = lane + 32 * i;
            if (2 * o >= s && 2 * o - s + 1 < n) r.w[i] = __ldg(words + o);
        }
        const int alone = lane == 0 ? (s ? 0 : -1) : lane == 1 && (n - 1 + s) % 2 == 0 ? n - 1 : -1;
        if (alone >= 0 && alone < n) r.edge = __ldg(halves + alone);
    }
    return r;
}
// To shared memory, word by word (s, n: as loaded).
template <typename T>
__device__ __forceinline__ void seg_stage(uint32_t *sw, const Seg<T> &r, int s, int n, int lane) {
#pragma unroll
    for (int i = 0; i < (sizeof(T) == 4 ? 8 : 4); ++i) sw[lane + 32 * i] = r.w[i];
    if constexpr (sizeof(T) == 2) {
        n = n < kMx4StageCols ? n : kMx4StageCols;
        if (lane == 0) sw[128] = 0;
        __syncwarp();
        unsigned short *halves = reinterpret_cast<unsigned short *>(sw);
        if (lane == 0 && s && n > 0) halves[1] = r.edge;
        if (lane == 1 && n > 0 && (n - 1 + s) % 2 == 0) halves[n - 1 + s] = r.edge;
    }
}
// NW words of values from value `first` (even) on, of a staged row with shift s.
template <typename T, int NW>
__device__ __forceinline__ void seg_read(const uint32_t *sw, int s, int first, uint32_t (&out)[NW]) {
    const uint32_t *p = sw + first * (int)sizeof(T) / 4;
#pragma unroll
    for (int i = 0; i < NW; i += 4) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p + i);
        out[i] = q.x;
        out[i + 1] = q.y;
        out[i + 2] = q.z;
        out[i + 3] = q.w;
    }
    if (sizeof(T) == 2 && s) {
        const uint32_t end = p[NW];
#pragma unroll
        for (int i = 0; i < NW; ++i) out[i] = __funnelshift_r(out[i], i + 1 < NW ? out[i + 1] : end, 16);
    }
}
// n (at most 256) values from sw, value 0 in the lower half of its first word, to dst.
template <typename T>
__device__ __forceinline__ void seg_store(T *dst, int n, const uint32_t *sw, int lane) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane + 32 * i < n) reinterpret_cast<uint32_t *>(dst)[lane + 32 * i] = sw[lane + 32 * i];
    } else {
        n = n < kMx4StageCols ? n : kMx4StageCols;
        const int s = seg_shift(dst);
        uint32_t *words = reinterpret_cast<uint32_t *>(dst - s);  // as in seg_load
        unsigned short *halves = reinterpret_cast<unsigned short *>(dst);
        if (s) {
            const uint32_t first = sw[0];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int o = lane + 32 * i;
                if (o > 0 && 2 * o < n) words[o] = __funnelshift_r(sw[o - 1], sw[o], 16);
            }
            if (lane == 0 && n > 0) halves[0] = (unsigned short)first;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int o = lane + 32 * i;
                if (2 * o + 1 < n) words[o] = sw[o];
            }
        }
        if (lane == 1 && n > 0 && (n - 1 + s) % 2 == 0) halves[n - 1] = (unsigned short)(s ? sw[(n - 1) / 2] >> 16 : sw[(n - 1) / 2]);
    }
}

template <typename T, bool NV, bool SEGS>  // SEGS: rows that are not 16-byte aligned
__global__ void __launch_bounds__(32 * kQWarps)
mx4_quant_kernel(const T *__restrict__ x, long long ld, int rows, int cols, const int *n_rows, float ts,
                 uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, int vec, int pairs, const int *status,
                 int trigger) {
    __shared__ uint4 seg4[SEGS ? kQWarps * 2 * kSegWords<T> / 4 : 1];
    uint32_t *seg = reinterpret_cast<uint32_t *>(seg4) + (SEGS ? (threadIdx.x >> 5) * 2 * kSegWords<T> : 0);
    if (trigger) griddep_launch_dependents();
    griddep_wait();
    const Mx4Ts tsc = mx4_ts(ts);
    if (status && *reinterpret_cast<const volatile int *>(status) != 0) return;
    const int lane = threadIdx.x & 31, sub = lane & 15, lower = lane >> 4;  // lower: the row 32 below
    int nr = n_rows ? *reinterpret_cast<const volatile int *>(n_rows) : rows;
    nr = nr < rows ? nr : rows;
    const int chunks = mx4_stages(cols), pitch = mx4_code_pitch(cols);
    const int row_tiles = chunks * Mx4<NV>::kStageTiles;
    Walk w(chunks, blockIdx.x * kQWarps + (threadIdx.x >> 5), gridDim.x * kQWarps);
    struct Segs {
        Seg<T> h[2];
    };
    using Raw = std::conditional_t<SEGS, Segs, Raw16<T>>;
    auto load = [&]() -> Raw {
        if constexpr (SEGS) {
            Raw r;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = w.row0() + 32 * h, col = w.chunk * kMx4StageCols;
                r.h[h] = seg_load<T>(x + (size_t)row * ld + col, w.pair < pairs && row < nr ? cols - col : 0, lane);
            }
            return r;
        } else {
            const int row = w.row0() + 32 * lower, col = w.chunk * kMx4StageCols + sub * 16;
            return load_raw16<T>(x + (size_t)row * ld + col, w.pair < pairs && row < nr ? cols - col : 0, vec);
        }
    };
    auto store = [&](const Raw &raw, int row0, int chunk) {
        const int row = row0 + 32 * lower, col = chunk * kMx4StageCols + sub * 16;
        Raw16<T> r;
        if constexpr (SEGS) {
            constexpr int kHalf = 2 * sizeof(T);  // words of eight values
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int y = row0 + 32 * h;
                seg_stage<T>(seg + h * kSegWords<T>, raw.h[h], seg_shift(x + (size_t)y * ld),
                             y < nr ? cols - chunk * kMx4StageCols : 0, lane);
            }
            __syncwarp();
            uint32_t t[2 * kHalf];
            seg_read<T>(seg + lower * kSegWords<T>, seg_shift(x + (size_t)row * ld), sub * 16, t);
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
                r.h[0].w[i] = t[i];
                r.h[1].w[i] = t[kHalf + i];
            }
        } else {
            r = raw;
        }
        uint32_t m;
        if constexpr (sizeof(T) == 4) {
            m = umax(raw8_amax<T>(r.h[0]), raw8_amax<T>(r.h[1]));
        } else {
            uint32_t m2 = r.h[0].w[0] & 0x7fff7fffu;
#pragma unroll
            for (int i = 1; i < 8; ++i) m2 = umax_x2(m2, r.h[i >> 2].w[i & 3] & 0x7fff7fffu);
            m = umax(m2 & 0xffffu, m2 >> 16);
        }
        if constexpr (!NV) m = umax(m, __shfl_xor_sync(0xffffffffu, m, 1));  // a block is two lanes
        const Mx4Scale s = mx4_block_scale<NV>(amax_f32_bits<T>(m), tsc);
        const uint64_t mul2 = f2_make(s.mul, s.mul);
        uint32_t q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
            raw8_values<T>(r.h[h], v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = f2_split(f2_mul(f2_make(v[2 * i], v[2 * i + 1]), mul2));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
            q[h] = s.zero ? 0u : cvt_e2m1x8(v);
        }
        // the lanes of a tile put their scale bytes together
        constexpr int kLanes = NV ? 1 : 2, kTileLanes = 4 * kLanes;
        uint32_t word = s.byte << (8 * ((sub / kLanes) & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, kLanes);
        word |= __shfl_xor_sync(0xffffffffu, word, 2 * kLanes);
        if (row < nr && col / 2 < pitch)
            *reinterpret_cast<uint2 *>(codes + (size_t)row * pitch + col / 2) = make_uint2(q[0], q[1]);
        if (sub % kTileLanes == 0)  // (rows past the end: scale 0, so that a tile is always whole)
            *reinterpret_cast<uint32_t *>(scales + scale_word_offset(row, chunk * Mx4<NV>::kStageTiles + sub / kTileLanes,
                                                                     row_tiles)) = word;
    };
    // the next item's rows load while the current ones are converted
    Raw a = load(), b;
    while (w.pair < pairs) {
        int row0 = w.row0(), chunk = w.chunk;
        w.next();
        b = load();
        store(a, row0, chunk);
        if (w.pair >= pairs) break;
        row0 = w.row0();
        chunk = w.chunk;
        w.next();
        a = load();
        store(b, row0, chunk);
    }
}

template <typename T, bool NV, bool SEGS>
__global__ void __launch_bounds__(32 * kQWarps)
mx4_dequant_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int rows, int cols, float ts,
                   T *__restrict__ out, long long ld, int vec, int pairs) {
    __shared__ uint4 seg4[SEGS ? kQWarps * 2 * kSegWords<T> / 4 : 1];
    uint32_t *seg = reinterpret_cast<uint32_t *>(seg4) + (SEGS ? (threadIdx.x >> 5) * 2 * kSegWords<T> : 0);
    const int lane = threadIdx.x & 31, sub = lane & 15, lower = lane >> 4;
    const int chunks = mx4_stages(cols), pitch = mx4_code_pitch(cols);
    const int row_tiles = chunks * Mx4<NV>::kStageTiles;
    Walk w(chunks, blockIdx.x * kQWarps + (threadIdx.x >> 5), gridDim.x * kQWarps);
    auto load = [&](uint2 &q, uint32_t &sb) {
        const int row = w.row0() + 32 * lower, col = w.chunk * kMx4StageCols + sub * 16, blk = col / Mx4<NV>::kBlock;
        q = make_uint2(0, 0);
        sb = 0;
        if (w.pair < pairs && row < rows && col < cols) {
            q = __ldg(reinterpret_cast<const uint2 *>(codes + (size_t)row * pitch + col / 2));
            sb = __ldg(scales + scale_word_offset(row, blk >> 2, row_tiles) + (blk & 3));
        }
    };
    auto store = [&](uint2 q, uint32_t sb, int row0, int chunk) {
        const int row = row0 + 32 * lower, col = chunk * kMx4StageCols + sub * 16, n = cols - col;
        if (!SEGS && (row >= rows || n <= 0)) return;
        const float s = mx4_scale_value<NV>(sb);
        float v[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            e2m1x8_values(h ? q.y : q.x, v[h]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[h][j] = __fmul_rn(v[h][j], s);  // exact
                if (NV) v[h][j] = __fmul_rn(v[h][j], ts);
            }
        }
        T *dst = out + (size_t)row * ld + col;
        if constexpr (SEGS) {
            uint32_t *mine = seg + lower * kSegWords<T> + sub * 4 * sizeof(T);
            __syncwarp();
            store8<T>(reinterpret_cast<T *>(mine), 8, true, v[0]);
            store8<T>(reinterpret_cast<T *>(mine) + 8, 8, true, v[1]);
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = row0 + 32 * h, c = chunk * kMx4StageCols;
                if (r < rows) seg_store<T>(out + (size_t)r * ld + c, cols - c, seg + h * kSegWords<T>, lane);
            }
        } else if (vec == 2 && n >= 16) {
            if constexpr (sizeof(T) == 4) {
                st_global_v8(dst, reinterpret_cast<const uint32_t *>(v[0]));
                st_global_v8(dst + 8, reinterpret_cast<const uint32_t *>(v[1]));
            } else {
                uint32_t o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = pack_x2<T>(v[j >> 2][2 * (j & 3)], v[j >> 2][2 * (j & 3) + 1]);
                st_global_v8(dst, o);
            }
        } else {
            store8<T>(dst, n, vec != 0, v[0]);
            store8<T>(dst + 8, n - 8, vec != 0, v[1]);
        }
    };
    uint2 qa, qb;
    uint32_t sa, sb;
    load(qa, sa);
    while (w.pair < pairs) {
        int row0 = w.row0(), chunk = w.chunk;
        w.next();
        load(qb, sb);
        store(qa, sa, row0, chunk);
        if (w.pair >= pairs) break;
        row0 = w.row0();
        chunk = w.chunk;
        w.next();
        load(qa, sa);
        store(qb, sb, row0, chunk);
    }
}

// LayerNorm, one warp per row of at most 256 NCH columns: the row stays in registers
// (one read), the sums by shuffles, the next row's loads in flight meanwhile.  fp32
// statistics in two passes; the 4-bit form is taken of the fp32 result, y is its rounding to
// x's type.  The first pass's mean m0 carries the rounding of its sum, which outweighs the
// row's own spread where that is small beside the mean (rows of one value: y was off by up
// to 1).  So the second pass sums the differences d = x - m0 beside their squares:
//   e = sum(d) / n, variance = sum(d^2) / n - e^2, y = (d - e) rstd gamma + beta,
// which holds for any m0 near the mean.  It costs an addition per pair and its shuffles
// (12301 x 768 bf16 in mxfp4: 9.1 us, 8.6 without).
// The warp's sum of a in lanes 0..15, of b in lanes 16..31: six shuffles for two sums' ten.
__device__ __forceinline__ float warp_sums(float a, float b, int lane) {
    const bool upper = lane & 16;
    float s = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
// From the means of d^2 and of d: rstd, and -e rstd.  (A variance below 0 is rounding; NaN and
// infinity stay.)
__device__ __forceinline__ float2 norm_factors(float mean_sq, float e, float eps) {
    const float var = mean_sq < __int_as_float(0x7f800000) ? fmaf(-e, e, mean_sq) : mean_sq;
    const float rstd = rsqrtf((var < 0.f ? 0.f : var) + eps);
    return make_float2(rstd, -e * rstd);
}

template <typename T, bool NV, int NCH>
__global__ void __launch_bounds__(32 * kQWarps)
mx4_norm_warp_kernel(const T *__restrict__ x, long long ld, const float *__restrict__ gamma,
                     const float *__restrict__ beta, float eps, int rows, int cols, const int *n_rows, float ts,
                     T *__restrict__ y, long long ld_y, uint8_t *__restrict__ codes,
                     uint8_t *__restrict__ scales, int vec, int vec_y, int vec_g, const int *status, int trigger) {
    if (trigger) griddep_launch_dependents();
    griddep_wait();
    const Mx4Ts tsc = mx4_ts(ts);
    if (status && *reinterpret_cast<const volatile int *>(status) != 0) return;
    int nr = n_rows ? *reinterpret_cast<const volatile int *>(n_rows) : rows;
    nr = nr < rows ? nr : rows;
    const int lane = threadIdx.x & 31, stride = gridDim.x * kQWarps;
    const int chunks = mx4_stages(cols), pitch = mx4_code_pitch(cols);
    const int row_tiles = chunks * Mx4<NV>::kStageTiles;
    int row = blockIdx.x * kQWarps + (threadIdx.x >> 5);
    Raw8<T> raw[NCH];
    auto load = [&](int r) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int col = c * kMx4StageCols + lane * 8;
            raw[c] = load_raw8<T>(x + (size_t)r * ld + col, r < nr ? cols - col : 0, vec != 0);
        }
    };
    // One row.  WHOLE: all 256 NCH columns exist, so nothing is masked.
    auto one_row = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        uint64_t v[NCH][4];  // fp32 pairs
        uint64_t s2 = f2_make(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            float f[8];
            raw8_values<T>(raw[c], f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[c][i] = f2_make(f[2 * i], f[2 * i + 1]);
                s2 = f2_add(s2, v[c][i]);
            }
        }
        if (row + stride < nr) load(row + stride);
        const float2 sf = f2_split(s2);
        float sum = sf.x + sf.y;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float mean = sum / (float)cols;
        const uint64_t nmean2 = f2_make(-mean, -mean);
        uint64_t q2 = f2_make(0.f, 0.f), e2 = q2;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int n = cols - c * kMx4StageCols - lane * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[c][i] = f2_add(v[c][i], nmean2);
                if (!WHOLE) {
                    const float2 d = f2_split(v[c][i]);
                    v[c][i] = f2_make(2 * i < n ? d.x : 0.f, 2 * i + 1 < n ? d.y : 0.f);
                }
                q2 = f2_fma(v[c][i], v[c][i], q2);
                e2 = f2_add(e2, v[c][i]);
            }
        }
        const float2 qf = f2_split(q2), ef = f2_split(e2);
        float sq = qf.x + qf.y, sd = ef.x + ef.y;
        const float s = warp_sums(sq, sd, lane), t = __shfl_xor_sync(0xffffffffu, s, 16);
        const float2 k = norm_factors((lane & 16 ? t : s) / (float)cols, (lane & 16 ? s : t) / (float)cols, eps);
        const uint64_t rstd2 = f2_make(k.x, k.x), off2 = f2_make(k.y, k.y);
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            if (!WHOLE && c >= chunks) break;
            const int col = c * kMx4StageCols + lane * 8, n = cols - col;
            float g[8], b[8], u[8];
            if (WHOLE) {  // (one 32-byte access a lane: two of 16 bytes cost L1 twice the lines)
                ld_cached_v8(gamma + col, g);
                ld_cached_v8(beta + col, b);
            } else {
                load8<float>(gamma + col, n, vec_g != 0, g);
                load8<float>(beta + col, n, vec_g != 0, b);  // (0 past the end, and so the result)
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = f2_split(f2_fma(f2_fma(v[c][i], rstd2, off2), f2_make(g[2 * i], g[2 * i + 1]), f2_make(b[2 * i], b[2 * i + 1])));
                u[2 * i] = f.x;
                u[2 * i + 1] = f.y;
            }
            if (!WHOLE) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i >= n) u[i] = 0.f;  // (not NaN, where the row's statistics are)
            }
            float m = fmax3_abs_nan(u[0], u[1], u[2]);
            m = fmax3_abs_nan(m, u[3], u[4]);
            m = fmax3_abs_nan(m, u[5], fmax3_abs_nan(u[6], u[7], 0.f));
            if (y) store8<T>(y + (size_t)row * ld_y + col, WHOLE ? 8 : n, WHOLE || vec_y != 0, u);
            uint32_t word;
            const uint32_t q = mx4_warp_quant<NV>(u, abs_bits(m), tsc, lane, word);
            if (WHOLE || col / 2 < pitch) *reinterpret_cast<uint32_t *>(codes + (size_t)row * pitch + col / 2) = q;
            constexpr int kTileLanes = Mx4<NV>::kTileCols / 8;
            if (lane % kTileLanes == 0)
                *reinterpret_cast<uint32_t *>(scales + scale_word_offset(row, c * Mx4<NV>::kStageTiles + lane / kTileLanes,
                                                                         row_tiles)) = word;
        }
    };
    if (row < nr) load(row);
    zero_past_rows(scales, nr, row_tiles);
    const bool whole = cols == NCH * kMx4StageCols && vec && vec_g == 2 && (!y || vec_y);
    if (whole)
        for (; row < nr; row += stride) one_row(std::true_type{});
    else
        for (; row < nr; row += stride) one_row(std::false_type{});
}

// The same with one CTA of W warps per row, for rows of at most 512 W columns: a lane has
// sixteen consecutive columns (per row and warp the sums, the scales and the addresses cost
// about as much as eight columns' arithmetic), the parameters stay in registers and the
// next row's values load while this one's sums are joined.  WORDS: rows that are not
// 16-byte aligned, or of a width that is no multiple of 8, come and go by words.  What
// bounds it over many rows is instructions: 8192 rows of 1000, 2048, 4096 bf16 columns take
// 9.1, 15.9 and 35.6 us (eight columns a lane: 10.7, 20.9, 43; in the kernel for wider rows
// 25, 33, 58), of 1001 by words 16.8 (by values, in that kernel, 30).
template <int W>
__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    if constexpr (W == 2) return red[0] + red[1];
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
        const float4 r = reinterpret_cast<const float4 *>(red)[i];
        s.x += r.x;
        s.y += r.y;
        s.z += r.z;
        s.w += r.w;
    }
    return (s.x + s.y) + (s.z + s.w);
}
// Two sums at once.
template <int W>
__device__ __forceinline__ float2 block_sums(float a, float b, float *red) {
    const float v = warp_sums(a, b, threadIdx.x & 31);
    if ((threadIdx.x & 15) == 0) red[threadIdx.x >> 4] = v;
    __syncthreads();
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        const float4 r = reinterpret_cast<const float4 *>(red)[i];
        s.x += r.x;
        s.y += r.y;
        s.z += r.z;
        s.w += r.w;
    }
    return make_float2(s.x + s.z, s.y + s.w);
}

template <typename T, bool NV, int W, bool WORDS>
__global__ void __launch_bounds__(32 * W)
mx4_norm_cta_kernel(const T *__restrict__ x, long long ld, const float *__restrict__ gamma,
                    const float *__restrict__ beta, float eps, int rows, int cols, const int *n_rows, float ts,
                    T *__restrict__ y, long long ld_y, uint8_t *__restrict__ codes,
                    uint8_t *__restrict__ scales, int vec, int vec_y, int vec_g, const int *status, int trigger) {
    // one for each barrier of a row: its second one separates its first from the next row's
    __shared__ __align__(16) float red[W];
    __shared__ __align__(16) float red2[2 * W];
    __shared__ uint4 seg4[WORDS ? W * 2 * kSegWords<T> / 4 : 1];
    uint32_t *seg = reinterpret_cast<uint32_t *>(seg4) + (WORDS ? (threadIdx.x >> 5) * 2 * kSegWords<T> : 0);
    if (trigger) griddep_launch_dependents();
    griddep_wait();
    const Mx4Ts tsc = mx4_ts(ts);
    if (status && *reinterpret_cast<const volatile int *>(status) != 0) return;
    int nr = n_rows ? *reinterpret_cast<const volatile int *>(n_rows) : rows;
    nr = nr < rows ? nr : rows;
    const int lane = threadIdx.x & 31;
    const int chunks = mx4_stages(cols), pitch = mx4_code_pitch(cols);
    const int row_tiles = chunks * Mx4<NV>::kStageTiles;
    // (a division per sum cost a twentieth; the mean's rounding is made good below, the
    // variance's is half a unit of rstd)
    const float inv_cols = 1.0f / (float)cols;
    const int col = threadIdx.x * 16, n = cols - col;  // aligned rows: n is 0 or less, 8, or more
    const int col0 = (threadIdx.x >> 5) * 512;
    constexpr int kLanes = NV ? 1 : 2, kTileLanes = 4 * kLanes;  // lanes of a block, of a scale tile
    uint64_t g[8], b[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float t[8] = {}, u[8] = {};
        if constexpr (WORDS) {
            load8<float>(gamma + col + 8 * h, n - 8 * h, vec_g != 0, t);
            load8<float>(beta + col + 8 * h, n - 8 * h, vec_g != 0, u);
        } else if (n > 8 * h) {
            ld_cached_v8(gamma + col + 8 * h, t);
            ld_cached_v8(beta + col + 8 * h, u);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            g[4 * h + i] = f2_make(t[2 * i], t[2 * i + 1]);
            b[4 * h + i] = f2_make(u[2 * i], u[2 * i + 1]);
        }
    }
    struct Segs {
        Seg<T> h[2];
    };
    using Raw = std::conditional_t<WORDS, Segs, Raw16<T>>;
    auto load = [&](int row) -> Raw {
        Raw r = {};
        if constexpr (WORDS) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                r.h[h] = seg_load<T>(x + (size_t)row * ld + col0 + 256 * h, row < nr ? cols - col0 - 256 * h : 0, lane);
            return r;
        } else {  // (no path by values: it would hold up the one warp that has the row's end, and with it the rest)
            const T *src = x + (size_t)row * ld + col;
            if (row >= nr || n <= 0) return r;
            if (vec == 2 && n > 8) return load_raw16<T>(src, 16, 2);
            r.h[0] = load_raw8<T>(src, 8, true);
            if (n > 8) r.h[1] = load_raw8<T>(src + 8, 8, true);
            return r;
        }
    };
    int row = blockIdx.x;
    Raw raw = load(row);
    zero_past_rows(scales, nr, row_tiles);
    for (; row < nr; row += gridDim.x) {
        Raw16<T> own;
        if constexpr (WORDS) {
            constexpr int kHalf = 2 * sizeof(T);  // words of eight values
            uint32_t w[2 * kHalf];
            __syncwarp();
            const int shift = seg_shift(x + (size_t)row * ld);
            seg_stage<T>(seg, raw.h[0], shift, cols - col0, lane);
            seg_stage<T>(seg + kSegWords<T>, raw.h[1], shift, cols - col0 - 256, lane);
            __syncwarp();
            seg_read<T>(seg + (lane >> 4) * kSegWords<T>, shift, (lane & 15) * 16, w);
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
                own.h[0].w[i] = w[i];
                own.h[1].w[i] = w[kHalf + i];
            }
        } else {
            own = raw;
        }
        uint64_t v[8];
        uint64_t s2 = f2_make(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[8];
            raw8_values<T>(own.h[h], f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[4 * h + i] = f2_make(f[2 * i], f[2 * i + 1]);
                s2 = f2_add(s2, v[4 * h + i]);
            }
        }
        raw = load(row + gridDim.x);
        const float2 sf = f2_split(s2);
        const float mean = block_sum<W>(sf.x + sf.y, red) * inv_cols;
        const uint64_t nmean2 = f2_make(-mean, -mean);
        float sq = 0.f, sd = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint64_t q2 = f2_make(0.f, 0.f), e2 = q2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[4 * h + i] = f2_add(v[4 * h + i], nmean2);
                if constexpr (WORDS) {
                    const float2 d = f2_split(v[4 * h + i]);
                    v[4 * h + i] = f2_make(8 * h + 2 * i < n ? d.x : 0.f, 8 * h + 2 * i + 1 < n ? d.y : 0.f);
                }
                q2 = f2_fma(v[4 * h + i], v[4 * h + i], q2);
                e2 = f2_add(e2, v[4 * h + i]);
            }
            const float2 qf = f2_split(q2), ef = f2_split(e2);
            sq += WORDS || n > 8 * h ? qf.x + qf.y : 0.f;
            sd += WORDS || n > 8 * h ? ef.x + ef.y : 0.f;
        }
        const float2 sums = block_sums<W>(sq, sd, red2);
        const float2 k = norm_factors(sums.x * inv_cols, sums.y * inv_cols, eps);
        const uint64_t rstd2 = f2_make(k.x, k.x), off2 = f2_make(k.y, k.y);
        if (col0 >= cols) continue;  // (the whole warp)
        float u[16];
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 w = f2_split(f2_fma(f2_fma(v[i], rstd2, off2), g[i], b[i]));
            u[2 * i] = n > (WORDS ? 2 * i : 8 * (i >> 2)) ? w.x : 0.f;
            u[2 * i + 1] = n > (WORDS ? 2 * i + 1 : 8 * (i >> 2)) ? w.y : 0.f;
            m = fmax3_abs_nan(m, u[2 * i], u[2 * i + 1]);
        }
        if (WORDS && y) {  // (the staged row has been read: two barriers ago)
            T *mine = reinterpret_cast<T *>(seg + (lane >> 4) * kSegWords<T>) + (lane & 15) * 16;
            store8<T>(mine, 8, true, *reinterpret_cast<const float (*)[8]>(u));
            store8<T>(mine + 8, 8, true, *reinterpret_cast<const float (*)[8]>(u + 8));
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h)
                seg_store<T>(y + (size_t)row * ld_y + col0 + 256 * h, cols - col0 - 256 * h, seg + h * kSegWords<T>, lane);
        } else if (y && n > 0) {
            T *dst = y + (size_t)row * ld_y + col;
            if (vec_y == 2 && n > 8) {
                if constexpr (sizeof(T) == 4) {
                    st_global_v8(dst, reinterpret_cast<const uint32_t *>(u));
                    st_global_v8(dst + 8, reinterpret_cast<const uint32_t *>(u + 8));
                } else {
                    uint32_t o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = pack_x2<T>(u[2 * i], u[2 * i + 1]);
                    st_global_v8(dst, o);
                }
            } else {
                store8<T>(dst, 8, true, *reinterpret_cast<const float (*)[8]>(u));
                if (n > 8) store8<T>(dst + 8, 8, true, *reinterpret_cast<const float (*)[8]>(u + 8));
            }
        }
        uint32_t bits = abs_bits(m);
        if constexpr (!NV) bits = umax(bits, __shfl_xor_sync(0xffffffffu, bits, 1));
        const Mx4Scale s = mx4_block_scale<NV>(bits, tsc);
        const uint64_t mul2 = f2_make(s.mul, s.mul);
        uint32_t q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float z[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = f2_split(f2_mul(f2_make(u[8 * h + 2 * i], u[8 * h + 2 * i + 1]), mul2));
                z[2 * i] = f.x;
                z[2 * i + 1] = f.y;
            }
            q[h] = s.zero ? 0u : cvt_e2m1x8(z);
        }
        uint32_t word = s.byte << (8 * ((lane / kLanes) & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, kLanes);
        word |= __shfl_xor_sync(0xffffffffu, word, 2 * kLanes);
        if (col / 2 < pitch) *reinterpret_cast<uint2 *>(codes + (size_t)row * pitch + col / 2) = make_uint2(q[0], q[1]);
        if (lane % kTileLanes == 0 && col < chunks * kMx4StageCols)
            *reinterpret_cast<uint32_t *>(scales + scale_word_offset(row, col / Mx4<NV>::kTileCols, row_tiles)) = word;
    }
}

// Wider rows: one CTA per row, each warp holds four of the row's chunks (every eighth);
// chunks beyond those are read again in each pass (from L1 or L2).  2000 rows of 8200 bf16
// columns take 24 us in mxfp4, 29 in nvfp4.
template <typename T, bool NV>
__global__ void __launch_bounds__(32 * kQWarps, sizeof(T) == 4 ? 2 : NV ? 3 : 4)  // (nvfp4: two CTAs per SM took 36 us)
mx4_norm_wide_kernel(const T *__restrict__ x, long long ld, const float *__restrict__ gamma,
                     const float *__restrict__ beta, float eps, int rows, int cols, const int *n_rows, float ts,
                     T *__restrict__ y, long long ld_y, uint8_t *__restrict__ codes,
                     uint8_t *__restrict__ scales, int vec, int vec_y, int vec_g, const int *status, int trigger) {
    constexpr int W = kQWarps, HELD = 4;
    __shared__ __align__(16) float red[W];  // as above
    __shared__ __align__(16) float red2[2 * W];
    if (trigger) griddep_launch_dependents();
    griddep_wait();
    const Mx4Ts tsc = mx4_ts(ts);
    if (status && *reinterpret_cast<const volatile int *>(status) != 0) return;
    int nr = n_rows ? *reinterpret_cast<const volatile int *>(n_rows) : rows;
    nr = nr < rows ? nr : rows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunks = mx4_stages(cols), pitch = mx4_code_pitch(cols);
    const int row_tiles = chunks * Mx4<NV>::kStageTiles;
    constexpr int kTileLanes = Mx4<NV>::kTileCols / 8;
    zero_past_rows(scales, nr, row_tiles);
    for (int row = blockIdx.x; row < nr; row += gridDim.x) {
        const T *src = x + (size_t)row * ld;
        Raw8<T> raw[HELD];
#pragma unroll
        for (int h = 0; h < HELD; ++h) {
            const int col = (warp + h * W) * kMx4StageCols + lane * 8;
            raw[h] = load_raw8<T>(src + col, cols - col, vec != 0);
        }
        // f(chunk, first column, columns left, values): held chunks, then the others
        auto each = [&](auto f) {
            float v[8];
#pragma unroll
            for (int h = 0; h < HELD; ++h) {
                const int c = warp + h * W, col = c * kMx4StageCols + lane * 8;
                if (c >= chunks) break;
                raw8_values<T>(raw[h], v);
                f(c, col, cols - col, v);
            }
            for (int c = warp + HELD * W; c < chunks; c += W) {
                const int col = c * kMx4StageCols + lane * 8;
                load8<T>(src + col, cols - col, vec != 0, v);
                f(c, col, cols - col, v);
            }
        };
        float sum = 0.f;
        each([&](int, int, int, const float (&v)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[i];
        });
        const float mean = block_sum<W>(sum, red) / (float)cols;
        float sq = 0.f, sd = 0.f;
        each([&](int, int, int n, const float (&v)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = i < n ? v[i] - mean : 0.f;
                sq = fmaf(d, d, sq);
                sd += d;
            }
        });
        const float2 sums = block_sums<W>(sq, sd, red2);
        const float2 k = norm_factors(sums.x / (float)cols, sums.y / (float)cols, eps);
        each([&](int c, int col, int n, float (&v)[8]) {
            float g[8], b[8];
            load8<float>(gamma + col, n, vec_g != 0, g);
            load8<float>(beta + col, n, vec_g != 0, b);
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = i < n ? fmaf(fmaf(v[i] - mean, k.x, k.y), g[i], b[i]) : 0.f;
                m = umax(m, abs_bits(v[i]));
            }
            if (y) store8<T>(y + (size_t)row * ld_y + col, n, vec_y != 0, v);
            uint32_t word;
            const uint32_t q = mx4_warp_quant<NV>(v, m, tsc, lane, word);
            if (col / 2 < pitch) *reinterpret_cast<uint32_t *>(codes + (size_t)row * pitch + col / 2) = q;
            if (lane % kTileLanes == 0)
                *reinterpret_cast<uint32_t *>(scales + scale_word_offset(row, c * Mx4<NV>::kStageTiles + lane / kTileLanes,
                                                                         row_tiles)) = word;
        });
    }
}

// (weights, once per handle: no need to be fast)
__global__ void amax_bf16_kernel(const bf16 *__restrict__ x, size_t n, unsigned *out) {
    uint32_t m = 0;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x)
        m = umax(m, abs_bits(__bfloat162float(x[i])));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) atomicMax(out, m);
}

// CTAs of `kernel` that are resident at once (asked once per device), at most `need`.
template <typename K>
cudaError_t resident_grid(K kernel, std::atomic<int> (&cached)[64], long long need, int &blocks, int warps = kQWarps) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int cap = dev < 64 ? cached[dev].load(std::memory_order_acquire) : 0;
    if (cap == 0) {
        int sms = 0, per_sm = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, 32 * warps, 0);
        if (e != cudaSuccess) return e;
        cap = (per_sm > 0 ? per_sm : 1) * sms;
        if (dev < 64) cached[dev].store(cap, std::memory_order_release);
    }
    blocks = (int)(need < cap ? need : cap);
    return cudaSuccess;
}

// One call for both kinds of launch (pdl: as launch_pdl).
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), int blocks, int warps, cudaStream_t s, bool pdl, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(32 * warps);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

inline bool aligned16(const void *p, long long ld, int elem) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * elem) % 16 == 0;
}

inline int vec_width(const void *p, long long ld, int elem) {
    return (reinterpret_cast<uintptr_t>(p) & 31) == 0 && (ld * elem) % 32 == 0 ? 2 : aligned16(p, ld, elem) ? 1 : 0;
}

template <typename T, bool NV, bool SEGS>
cudaError_t quant_launch(const Mx4QuantArgs &a, int vec, cudaStream_t s, bool pdl) {
    // (all row pairs of the last tile, whose scale bytes are written whole)
    const int pairs = (a.rows + 127) / 128 * 64;
    const long long items = (long long)pairs * mx4_stages(a.cols);
    static std::atomic<int> cached[64];
    int blocks = 0;
    auto kernel = mx4_quant_kernel<T, NV, SEGS>;
    cudaError_t e = resident_grid(kernel, cached, (items + kQWarps - 1) / kQWarps, blocks);
    if (e != cudaSuccess) return e;
    return launch(kernel, blocks, kQWarps, s, pdl, static_cast<const T *>(a.x), a.ld, a.rows, a.cols, a.n_rows,
                  a.tensor_scale, a.codes, a.scales, vec, pairs, a.status, a.trigger);
}
template <typename T, bool NV>
cudaError_t quant_typed(const Mx4QuantArgs &a, cudaStream_t s, bool pdl) {
    const int vec = vec_width(a.x, a.ld, sizeof(T));
    return vec ? quant_launch<T, NV, false>(a, vec, s, pdl) : quant_launch<T, NV, true>(a, vec, s, pdl);
}

template <typename T, bool NV, bool SEGS>
cudaError_t dequant_launch(const uint8_t *codes, const uint8_t *scales, int rows, int cols, float ts, T *out, long long ld,
                           int vec, cudaStream_t s) {
    const int pairs = (rows + 127) / 128 * 64;
    const long long items = (long long)pairs * mx4_stages(cols);
    static std::atomic<int> cached[64];
    int blocks = 0;
    auto kernel = mx4_dequant_kernel<T, NV, SEGS>;
    cudaError_t e = resident_grid(kernel, cached, (items + kQWarps - 1) / kQWarps, blocks);
    if (e != cudaSuccess) return e;
    return launch(kernel, blocks, kQWarps, s, false, codes, scales, rows, cols, ts, out, ld, vec, pairs);
}
template <typename T, bool NV>
cudaError_t dequant_typed(const uint8_t *codes, const uint8_t *scales, int rows, int cols, float ts, void *out,
                          long long ld, cudaStream_t s) {
    const int vec = vec_width(out, ld, sizeof(T));
    return vec ? dequant_launch<T, NV, false>(codes, scales, rows, cols, ts, static_cast<T *>(out), ld, vec, s)
               : dequant_launch<T, NV, true>(codes, scales, rows, cols, ts, static_cast<T *>(out), ld, vec, s);
}

// Whether rows of x and of y are 16-byte aligned.
template <typename T>
bool norm_aligned(const Mx4NormArgs &a) {
    return aligned16(a.q.x, a.q.ld, sizeof(T)) && (!a.y || aligned16(a.y, a.ld_y, sizeof(T)));
}

template <typename T, bool NV, typename K>
cudaError_t norm_launch(K kernel, std::atomic<int> (&cached)[64], int rows_per_cta, int warps, const Mx4NormArgs &a, cudaStream_t s,
                        bool pdl) {
    int blocks = 0;
    // (few rows: CTAs without one too, so that a thread zeroes 16 bytes of the last tiles at the
    // most; one row of 8192 in nvfp4 took 4.8 us with its own CTA writing all 64 KB)
    const int row_tiles = mx4_stages(a.q.cols) * Mx4<NV>::kStageTiles;
    const int need = std::max((a.q.rows + rows_per_cta - 1) / rows_per_cta, (row_tiles + warps - 1) / warps);
    cudaError_t e = resident_grid(kernel, cached, need, blocks, warps);
    if (e != cudaSuccess) return e;
    const int vec = vec_width(a.q.x, a.q.ld, sizeof(T)), vec_y = vec_width(a.y, a.ld_y, sizeof(T));
    const int vec_g = std::min(vec_width(a.gamma, 8, 4), vec_width(a.beta, 8, 4));
    return launch(kernel, blocks, warps, s, pdl, static_cast<const T *>(a.q.x), a.q.ld, a.gamma, a.beta, a.eps, a.q.rows,
                  a.q.cols, a.q.n_rows, a.q.tensor_scale, static_cast<T *>(a.y), a.ld_y, a.q.codes, a.q.scales, vec, vec_y,
                  vec_g, a.q.status, a.q.trigger);
}

template <typename T, bool NV, int W, bool WORDS>
cudaError_t norm_rows(const Mx4NormArgs &a, cudaStream_t s, bool pdl) {
    static std::atomic<int> cached[64];
    return norm_launch<T, NV>(mx4_norm_cta_kernel<T, NV, W, WORDS>, cached, 1, W, a, s, pdl);
}
template <typename T, bool NV, int W>
cudaError_t norm_width(const Mx4NormArgs &a, cudaStream_t s, bool pdl) {
    const bool words = a.q.cols % 8 || !norm_aligned<T>(a) || vec_width(a.gamma, 8, 4) != 2 || vec_width(a.beta, 8, 4) != 2;
    return words ? norm_rows<T, NV, W, true>(a, s, pdl) : norm_rows<T, NV, W, false>(a, s, pdl);
}

template <typename T, bool NV>
cudaError_t norm_typed(const Mx4NormArgs &a, cudaStream_t s, bool pdl) {
    // A warp per row once the rows fill the machine's warps several times over; a CTA per
    // row for few rows (5 rows of 1000: 4.4 us against 7.9), for rows a warp cannot hold
    // in half its registers, and for rows without alignment (8192 x 767: 16.9 us against
    // 21); both sides of the other widths at the kernel above.
    static std::atomic<int> c1[64], c3[64], wide[64];
    if (a.q.cols <= 256) return norm_launch<T, NV>(mx4_norm_warp_kernel<T, NV, 1>, c1, kQWarps, kQWarps, a, s, pdl);
    if (a.q.cols <= 768 && a.q.rows >= 512 && norm_aligned<T>(a))
        return norm_launch<T, NV>(mx4_norm_warp_kernel<T, NV, 3>, c3, kQWarps, kQWarps, a, s, pdl);
    if (a.q.cols <= 1024) return norm_width<T, NV, 2>(a, s, pdl);
    if (a.q.cols <= 2048) return norm_width<T, NV, 4>(a, s, pdl);
    if (a.q.cols <= 4096) return norm_width<T, NV, 8>(a, s, pdl);
    if (a.q.cols <= 8192) return norm_width<T, NV, 16>(a, s, pdl);
    return norm_launch<T, NV>(mx4_norm_wide_kernel<T, NV>, wide, 1, kQWarps, a, s, pdl);
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
cudaError_t launch_amax_bf16(const bf16 *x, size_t n, unsigned *out, cudaStream_t s) {
    cudaError_t e = cudaMemsetAsync(out, 0, sizeof(unsigned), s);
    if (e != cudaSuccess) return e;
    amax_bf16_kernel<<<256, 256, 0, s>>>(x, n, out);
    return cudaGetLastError();
}
cudaError_t launch_mx4_norm(const Mx4NormArgs &a, cudaStream_t s, bool pdl) {
    if (a.q.rows < 1) return cudaSuccess;
    MX4_BY_TYPE(norm_typed, a.q.type, a.q.nv, a, s, pdl);
}

}  // namespace albert
