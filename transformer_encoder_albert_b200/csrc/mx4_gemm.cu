// mx4_gemm.cu -- the linear layer on microscaled 4-bit operands, many rows.
//
// z = alpha A W^T + bias, tanh-GELU, + residual; A [M, K] and W [N, K] as E2M1
// codes with block scales (mx4.cuh), the products and the multiplication by both
// scales on tcgen05 (kind::mxf4 / mxf4nvf4, block_scale), sums in fp32.
//
// Persistent, one CTA per SM, warp-specialized:
//   warp 0      : TMA producer: per stage 256 columns of A and W (128-byte rows,
//                 128-byte swizzle) and their scale tiles (512 bytes per 128 rows and
//                 four blocks, plain); the whole warp in step, one elected lane issues
//                 (117 cycles a stage; one lane inside a branch needed 374);
//   warp 1      : issues four products of K = 64 per stage;
//   warp 2      : issues the copies of the scale tiles to tensor memory, ahead of the
//                 products (6 or 12 copies per stage at about 26 cycles each would cost
//                 the products' warp more than half their time);
//   warps 4..19 : epilogue, four warps per lane quadrant, each every fourth 32-column
//                 chunk (a chunk is some 190 dependent instructions: with two warps per
//                 quadrant it took 1330 cycles, and K = 768 only gives a tile 1536);
//                 16-bit rows leave through a swizzled staging tile by TMA, their residual
//                 tiles arrive by TMA a chunk ahead; fp32 and rows that are not 16-byte
//                 aligned go a column per lane.
// Two tile shapes:
//   * a CTA pair per 256x256 tile (cta_group::2): each CTA stages 128 rows of A and of
//     W and the scales of its A rows and of all W rows.  Two 256-column accumulators
//     would fill tensor memory; they overlap by 96 columns, which leaves 96 for the
//     scales.  The epilogue's first chunks cover the overlap, so the next tile's
//     products start once those are in registers.
//   * one CTA per 128x128 tile, two separate accumulators, for work that would leave
//     pairs idle.
// Tensor memory holds four scale units (a stage of mxfp4, half a stage of nvfp4, 24
// columns on pairs).  A unit's columns are written again only after the products that
// read them have completed: their stage's empty barrier, or the commit in its middle.
// (With two whole stages of nvfp4 the copies waited for products: the step took 8192^3, the
// product alone, from 219 to 217 us.)
// What bounds it: at K = 768 the epilogue (18797 x 2304: 24.6 us, 86.6 MB of results alone
// are 13 at the copy rate); at 8192^3 the main loop, which takes 654 (mxfp4) and 705 (nvfp4)
// cycles a stage where the nominal rate is 512, at the 1.6 GHz that the power cap leaves; 190
// and 203 us.  Which wait those cycles go to has not been found: a library product of the same
// operands took 176 us under the same cap.
// Every wait is bounded; see the bf16 GEMM.
#include <type_traits>

#include "mx4.cuh"
#include "mx4.h"
#include "mx4_ptx.cuh"

namespace albert {
namespace {

// What the epilogue leaves (a kernel each: its code stays short).
enum class Result { k16Bit, k16BitRes, kF32, k4Bit };  // (Res: + residual)

constexpr int kEpiWarps = 16, kEpi0 = 4;  // epilogue warps, the first of them
constexpr int kThreads = 32 * (kEpi0 + kEpiWarps);
constexpr int kTile = 2048;               // a staging tile: 32 rows of 64 bytes
constexpr int kRowsBytes = 128 * 128;  // 128 rows x 256 columns of codes

template <bool NV, bool PAIR, Result OUT>
struct Plan {
    static constexpr int TN = PAIR ? 256 : 128;              // columns of a tile
    static constexpr int UM = PAIR ? 256 : 128;              // rows of a tile
    static constexpr int ST = Mx4<NV>::kStageTiles;          // scale tiles per 128 rows and stage
    static constexpr int SFA = ST * kMx4TileBytes;
    static constexpr int SFB = (TN / 128) * SFA;
    static constexpr int STAGE = 2 * kRowsBytes + SFA + SFB;  // bytes per CTA and stage
    static constexpr int STG = (OUT == Result::k4Bit ? 0 : OUT == Result::k16Bit ? 1 : 2) * kTile;  // per epilogue warp
    static constexpr int BIAS = OUT == Result::k4Bit ? 64 : 32;  // biases per epilogue warp
    // As many stages as fit beside the staging tiles, at most six: a fifth takes 8192^3 from
    // 197 to 190 us (mxfp4) and 18797 rows of 2048 -> 768 from 17.6 to 17.1.
    static constexpr int ROOM = (232448 - 64 - 1024 - 512 - kEpiWarps * (STG + 4 * BIAS)) / STAGE;
    static constexpr int NST = ROOM < 6 ? ROOM : 6;
    static constexpr int ACC1 = PAIR ? 160 : 128;            // first column of the second accumulator
    static constexpr int SFCOL = PAIR ? 416 : 256;           // first scale column
    static constexpr int UNITS = ST / 2;                     // scale units per stage: two tiles of each 128 rows
    static constexpr int SFUNIT = 8 * (1 + TN / 128);        // scale columns per unit
    static constexpr int SFR = 4;                            // units in tensor memory
    static constexpr int PER = TN / 128;                     // 32-column chunks per epilogue warp
    static constexpr int SMEM = 1024 + NST * STAGE + kEpiWarps * (STG + 4 * BIAS) + 512;
    static_assert(SFCOL + SFR * SFUNIT <= 512, "tensor memory columns");
    static_assert(SMEM + 64 <= 232448, "shared memory per CTA, the wait limit included");
    static_assert(NST >= 4, "stages");
    static_assert((2 * NST + 12 + kEpiWarps) * 8 + 32 <= 512, "barriers");
};

// Walk over a CTA's tiles, unit u = tile (u / n_sub, u % n_sub), by additions.
struct TileWalk {
    int u, m, n, step, dm, dn, n_sub;
    __device__ __forceinline__ TileWalk(int first, int step_, int n_sub_) : u(first), step(step_), n_sub(n_sub_) {
        m = first / n_sub_;
        n = first - m * n_sub_;
        dm = step_ / n_sub_;
        dn = step_ - dm * n_sub_;
    }
    __device__ __forceinline__ void next() {
        u += step;
        m += dm;
        n += dn;
        if (n >= n_sub) {
            n -= n_sub;
            ++m;
        }
    }
};

struct Ctrl {
    uint64_t *full, *empty, *sfull, *half, *tfull, *tfree, *drain, *sdrain, *rbar;
    uint32_t *tmem_slot;
    volatile int *abort_flag;
    int *misc;
};

// Byte offset of 16-byte chunk q of row r in a 32x32 16-bit tile stored with the TMA
// 64-byte swizzle.
__device__ __forceinline__ uint32_t stg_off(int r, int q) {
    return (uint32_t)(r * 64 + ((q ^ ((r >> 1) & 3)) << 4));
}
__device__ __forceinline__ void st_shared_u4(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_u16(uint32_t a, uint16_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u1(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint16_t ld_shared_u16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}

// Four bytes to shared memory, without registers in between; and all of this thread's.
__device__ __forceinline__ void copy4_async(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// tma_store_2d of the lane whose predicate holds, without a branch.
__device__ __forceinline__ void tma_store_if(bool on, const void *tmap, uint32_t src, int x, int y) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
                 "@q cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\t}"
                 ::"l"(tmap), "r"(src), "r"(x), "r"(y), "r"((uint32_t)on) : "memory");
}

// v += row `lane` of a 16-bit 32x32 tile.
__device__ __forceinline__ void add_tile16(uint32_t tile, int lane, bool f16, float (&v)[32]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 w = ld_shared_u4(tile + stg_off(lane, q));
        const uint32_t w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = f16 ? unpack_x2<__half>(w4[e]) : unpack_x2<bf16>(w4[e]);
            v[8 * q + 2 * e] += f.x;
            v[8 * q + 2 * e + 1] += f.y;
        }
    }
}

template <bool NV, bool PAIR, Result OUT>
__global__ void __launch_bounds__(kThreads, 1)
mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmRes, const Mx4GemmArgs p,
                int n_sub, int tma_out, int tma_res) {
    using P = Plan<NV, PAIR, OUT>;
    constexpr bool QOUT = OUT == Result::k4Bit, f32 = OUT == Result::kF32, RES = OUT == Result::k16BitRes;
    constexpr int NST = P::NST, TN = P::TN, ST = P::ST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sA = base, *sB = sA + NST * kRowsBytes, *sSA = sB + NST * kRowsBytes, *sSB = sSA + NST * P::SFA;
    uint8_t *sStg = sSB + NST * P::SFB;  // (a multiple of 1024 from base: the stages and scale tiles are)
    float *sBias = reinterpret_cast<float *>(sStg + kEpiWarps * P::STG);
    uint64_t *bars = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(sBias) + kEpiWarps * 4 * P::BIAS);
    Ctrl c;
    c.full = bars;
    c.empty = bars + NST;
    c.sfull = bars + 2 * NST;
    c.half = bars + 2 * NST + 4;
    c.tfull = bars + 2 * NST + 6;
    c.tfree = bars + 2 * NST + 8;
    c.drain = bars + 2 * NST + 10;
    c.sdrain = bars + 2 * NST + 11;
    c.rbar = bars + 2 * NST + 12;
    uint32_t *u32 = reinterpret_cast<uint32_t *>(bars + 2 * NST + 12 + kEpiWarps);
    c.tmem_slot = u32;
    c.abort_flag = reinterpret_cast<volatile int *>(u32 + 1);
    c.misc = reinterpret_cast<int *>(u32 + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0;
    const int slot = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    const int nslots = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;

    if (p.trigger) griddep_launch_dependents();
    if (threadIdx.x == 0) {
        *c.abort_flag = 0;
        wait_limit_init(p.wait_ns);
        for (int i = 0; i < NST; ++i) {
            mbar_init(smem_u32(&c.full[i]), 1);
            mbar_init(smem_u32(&c.empty[i]), 1);
        }
        for (int i = 0; i < P::SFR; ++i) mbar_init(smem_u32(&c.sfull[i]), 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&c.half[i]), 1);
            mbar_init(smem_u32(&c.tfull[i]), 1);
            mbar_init(smem_u32(&c.tfree[i]), (PAIR ? 2 : 1) * kEpiWarps);
        }
        mbar_init(smem_u32(c.drain), 1);
        mbar_init(smem_u32(c.sdrain), 1);
        for (int i = 0; i < kEpiWarps; ++i) mbar_init(smem_u32(&c.rbar[i]), 1);
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
        prefetch_tmap(&tmSA);
        prefetch_tmap(&tmSB);
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(smem_u32(c.tmem_slot), 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(c.tmem_slot), 512);
            tmem_relinquish();
        }
    }
    griddep_wait();
    if (threadIdx.x == 0) {
        c.misc[0] = p.n_rows ? *reinterpret_cast<const volatile int *>(p.n_rows) : p.M;
        c.misc[1] = p.check_status ? *reinterpret_cast<const volatile int *>(p.status) : 0;
    }
    tc_fence_before();
    if (PAIR) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *c.tmem_slot;

    const bool skip = c.misc[1] != 0 || c.misc[0] < 0 || c.misc[0] > p.M;
    const int n_rows = skip ? 0 : c.misc[0];
    const int m_blocks = (n_rows + P::UM - 1) / P::UM;
    const int units = m_blocks * n_sub;  // (the host has checked that they and a step past them fit)
    const int kblocks = mx4_stages(p.K);

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer --
        // (the whole warp in step here too)
        const uint32_t leader = elect_leader();
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        const int loaded = p.withhold_loads ? 0 : units;
        for (TileWalk w(slot, nslots, n_sub); w.u < loaded && ok; w.next()) {
            // scale maps: rows of 256 bytes, a stage of one 128-row tile is 2 ST of them
            const int ma = w.m * (P::UM / 128) + (int)rank, nb = w.n * TN + (int)rank * 128;
            int ya = ma * kblocks * 2 * ST, yb = w.n * (TN / 128) * kblocks * 2 * ST;
            for (int kb = 0; kb < kblocks; ++kb, ya += 2 * ST, yb += 2 * ST) {
                if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&c.empty[stage]), phase ^ 1, c.abort_flag))) {
                    ok = false;
                    break;
                }
                const uint32_t full = smem_u32(c.full) + 8 * stage;
                const uint32_t fb = PAIR ? mapa_shared(full, 0) : full;
                if (leader && rank == 0) mbar_arrive_expect_tx(full, (PAIR ? 2 : 1) * P::STAGE);
                __syncwarp();
                const uint32_t fs = smem_u32(sSB) + stage * P::SFB;
                tma_load_elected<PAIR>(leader, smem_u32(sA) + stage * kRowsBytes, &tmA, fb, kb * 128, ma * 128);
                tma_load_elected<PAIR>(leader, smem_u32(sB) + stage * kRowsBytes, &tmB, fb, kb * 128, nb);
                tma_load_elected<PAIR>(leader, smem_u32(sSA) + stage * P::SFA, &tmSA, fb, 0, ya);
                tma_load_elected<PAIR>(leader, fs, &tmSB, fb, 0, yb);
                if (PAIR) tma_load_elected<PAIR>(leader, fs + P::SFA, &tmSB, fb, 0, yb + kblocks * 2 * ST);
                ++issued;
                if (++stage == NST) { stage = 0; phase ^= 1; }
            }
        }
        // The last loads of each slot (rank 1's land on rank 0's barriers too): where a wait has run
        // out in another warp nobody else sees them land, and the CTAs' memory must outlast them.
        if (rank == 0) {
            for (int i = 0; i < NST && i < issued; ++i) {
                if (--stage < 0) { stage = NST - 1; phase ^= 1; }
                mbar_wait_drain(smem_u32(&c.full[stage]), phase);
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------------------- MMA issuer --
        // (the whole warp walks the loop in step, one elected lane issues)
        if (rank == 0) {
            const uint32_t leader = elect_leader();
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, c.abort_flag)) != 0;
            };
            const uint64_t da0 = sw128_kmajor_desc(smem_u32(sA)), db0 = sw128_kmajor_desc(smem_u32(sB));
            uint32_t stage = 0, t = 0;  // t: tiles issued by this CTA
            uint32_t it = 0;                       // stages consumed
            bool ok = true;
            for (int u = slot; u < units && ok; u += nslots, ++t) {
                if (PAIR) {
                    // the previous tile's columns of the overlap have been read
                    if (t >= 1 && !wait(&c.tfree[(t - 1) & 1], ((t - 1) >> 1) & 1)) break;
                } else {
                    if (t >= 2 && !wait(&c.tfree[t & 1], ((t - 2) >> 1) & 1)) break;
                }
                const uint32_t d = tmem + (t & 1) * P::ACC1;
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    // (a descriptor's address field counts 16 bytes: a product's 32 bytes of K are 2)
                    const uint64_t da = da0 + stage * (kRowsBytes >> 4), db = db0 + stage * (kRowsBytes >> 4);
                    const int left = p.K - kb * kMx4StageCols;
#pragma unroll
                    for (int h = 0; h < P::UNITS; ++h) {
                        // scales in tensor memory, operands in shared memory: the scale warp, which has
                        // waited for the stage, arrives on the same barrier as its copies
                        const uint32_t j = it * P::UNITS + h;
                        if (!wait(&c.sfull[j % P::SFR], (j / P::SFR) & 1)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t ca = tmem + P::SFCOL + (j % P::SFR) * P::SFUNIT, cb = ca + 8;
                        auto product = [&](int i, uint32_t who, uint32_t acc) {
                            const int g = NV ? i : i >> 1, k = h * (4 / P::UNITS) + i;
                            umma_mx4<NV, PAIR>(who, d, da + 2 * k, db + 2 * k, idesc_mx4<NV>(P::UM, TN, NV ? 0 : 2 * (k & 1)),
                                               ca + 4 * g, cb + g * (TN / 128) * 4, acc);
                        };
                        if (left > 3 * 64) {
#pragma unroll
                            for (int i = 0; i < 4 / P::UNITS; ++i) product(i, leader, h + i != 0 || kb != 0);
                        } else {  // products past the last column are left out
#pragma unroll
                            for (int i = 0; i < 4 / P::UNITS; ++i)
                                product(i, (h * (4 / P::UNITS) + i) * 64 < left ? leader : 0u, h + i != 0 || kb != 0);
                        }
                        if (h + 1 < P::UNITS) umma_commit_elected<PAIR>(leader, smem_u32(&c.half[it & 1]), 1);
                    }
                    if (!ok) break;
                    umma_commit_elected<PAIR>(leader, smem_u32(c.empty) + 8 * stage, 3);
                    if (++stage == NST) stage = 0;
                }
                if (!ok) break;
                umma_commit_elected<PAIR>(leader, smem_u32(&c.tfull[t & 1]), 3);
            }
            umma_commit_elected<PAIR>(leader, smem_u32(c.drain), 1);
            mbar_wait_drain(smem_u32(c.drain), 0);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------- scale copies --
        if (rank == 0) {
            const uint32_t leader = elect_leader();
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, c.abort_flag)) != 0;
            };
            const uint64_t da0 = scale_tile_desc(smem_u32(sSA)), db0 = scale_tile_desc(smem_u32(sSB));
            uint32_t stage = 0, phase = 0, it = 0;
            uint32_t es = 0, eph = 0;  // stage and phase of the stage whose scale columns come free next
            bool ok = true;
            for (int u = slot; u < units && ok; u += nslots) {
                for (int kb = 0; kb < kblocks; ++kb, ++it) {
                    if (!wait(&c.full[stage], phase)) { ok = false; break; }
                    const uint64_t da = da0 + stage * (P::SFA >> 4), db = db0 + stage * (P::SFB >> 4);
#pragma unroll
                    for (int h = 0; h < P::UNITS; ++h) {
                        // the products that read these columns four units ago have completed (with four
                        // stages of one unit each, the full stage tells)
                        constexpr uint32_t kAgo = P::SFR / P::UNITS;  // in stages
                        if ((P::UNITS == 2 || NST > P::SFR) && it >= kAgo) {
                            if (h + 1 < P::UNITS) {
                                if (!wait(&c.half[it & 1], ((it - 2) >> 1) & 1)) { ok = false; break; }
                            } else {
                                if (!wait(&c.empty[es], eph)) { ok = false; break; }
                                if (++es == NST) { es = 0; eph ^= 1; }
                            }
                        }
                        tc_fence_after();
                        const uint32_t j = it * P::UNITS + h;
                        const uint32_t ca = tmem + P::SFCOL + (j % P::SFR) * P::SFUNIT, cb = ca + 8;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int g = 2 * h + i;
                            tmem_cp_scales<PAIR>(leader, ca + 4 * i, da + g * (kMx4TileBytes >> 4));
#pragma unroll
                            for (int b = 0; b < TN / 128; ++b)
                                tmem_cp_scales<PAIR>(leader, cb + (i * (TN / 128) + b) * 4,
                                                     db + ((b * P::SFA + g * kMx4TileBytes) >> 4));
                        }
                        umma_commit_elected<PAIR>(leader, smem_u32(&c.sfull[j % P::SFR]), 1);
                        if (lane == 0) mbar_arrive(smem_u32(&c.sfull[j % P::SFR]));
                    }
                    if (!ok) break;
                    if (++stage == NST) { stage = 0; phase ^= 1; }
                }
            }
            umma_commit_elected<PAIR>(leader, smem_u32(c.sdrain), 1);
            mbar_wait_drain(smem_u32(c.sdrain), 0);
        }
    } else if (warp >= kEpi0) {
        // ---------------------------------------------------------- epilogue --
        constexpr int PER = P::PER;
        const int ew = warp - kEpi0, quad = warp & 3, part = ew >> 2;
        float *bias_s = sBias + ew * P::BIAS;  // one or two chunks' biases
        const uint32_t stg = smem_u32(sStg + ew * P::STG), rbar = smem_u32(&c.rbar[ew]);
        const bool res = RES || (f32 && p.res != nullptr);
        uint32_t t = 0, rph = 0, chunks = 0;
        bool res_pending = false;
        // this warp's i-th chunk of a tile: the first accumulator of a pair is read from its
        // upper end, the second from its lower end, so that the overlap comes first
        auto chunk_of = [&](uint32_t tt, int i) { return (PAIR && (tt & 1) == 0) ? (TN / 32 - 1 - part) - 4 * i : part + 4 * i; };
        // residual tiles use the second staging tile, results the first
        auto res_issue = [&](const TileWalk &w, uint32_t tt, int i) {
            if (lane == 0) {
                mbar_arrive_expect_tx(rbar, kTile);
                tma_load_2d(stg + kTile, &tmRes, rbar, w.n * TN + chunk_of(tt, i) * 32,
                            w.m * P::UM + (int)rank * 128 + quad * 32);
            }
            res_pending = true;
        };
        // fp32: two tiles of 16 columns; a lane copies its column of the residual rows, which are in
        // place before the chunk's sums are (loaded on use, a few rows at a time, they made
        // 8192 x 2304 x 1024 take 49 us instead of 42)
        const uint32_t col_at = stg + (lane >> 4) * kTile + (lane & 3) * 4;
        const int col_q = (lane >> 2) & 3;
        auto res32_issue = [&](const TileWalk &w, uint32_t tt, int i) {
            const int col = w.n * TN + chunk_of(tt, i) * 32 + lane, r0 = w.m * P::UM + (int)rank * 128 + quad * 32;
            if (col >= p.N) return;
            const uint32_t *src = static_cast<const uint32_t *>(p.res) + (size_t)r0 * p.ld_res + col;
            const int rows = n_rows - r0 < 32 ? n_rows - r0 : 32;
#pragma unroll 8
            for (int y = 0; y < rows; ++y) copy4_async(col_at + stg_off(y, col_q), src + (size_t)y * p.ld_res);
        };
        auto bias_load = [&](const TileWalk &w, uint32_t tt, int i) {
            const int col = w.n * TN + chunk_of(tt, i) * 32 + lane;
            return (p.bias && col < p.N) ? __ldg(p.bias + col) : 0.f;
        };
        const Mx4Ts q_ts = mx4_ts(p.q_ts);
        float bnext = 0.f;
        TileWalk w(slot, nslots, n_sub), wn = w;  // this tile, the next
        if (w.u < units) {
            bnext = bias_load(w, 0, 0);
            if (RES && tma_res) res_issue(w, 0, 0);
            if (f32 && res) res32_issue(w, 0, 0);
        }
        bool ok = true;
        for (; w.u < units && ok; w = wn, ++t) {
            wn.next();
            const int m = w.m, n = w.n;
            const int row0 = m * P::UM + (int)rank * 128 + quad * 32, row = row0 + lane;
            const bool row_ok = row < n_rows;
            bool got = mbar_wait(smem_u32(&c.tfull[t & 1]), (t >> 1) & 1, c.abort_flag);
            if (!__all_sync(0xffffffffu, got)) break;
            tc_fence_after();
            const uint32_t tb = tmem + ((uint32_t)(quad * 32) << 16) + (t & 1) * P::ACC1;
#pragma unroll 1
            for (int i = 0; i < PER; ++i, ++chunks) {
                const int ch = chunk_of(t, i);
                uint32_t r[32];
                tmem_ld32(tb + ch * 32, r);
                float *bs = bias_s + (P::BIAS == 64 ? (chunks & 1) * 32 : 0);  // (its readers have passed a __syncwarp since)
                bs[lane] = bnext;
                tmem_ld_wait();
                if (i == 0) tc_fence_before();
                __syncwarp();
                if (i == 0 && lane == 0) {
                    // pair: the overlap is in registers; else: the whole accumulator is
                    if (PAIR) mbar_arrive_cluster(mapa_shared(smem_u32(&c.tfree[t & 1]), 0));
                    else mbar_arrive(smem_u32(&c.tfree[t & 1]));
                }
                if (i + 1 < PER) bnext = bias_load(w, t, i + 1);
                else if (wn.u < units) bnext = bias_load(wn, t + 1, 0);
                const int col0 = n * TN + ch * 32;
                const int left = p.N - col0;  // columns of this chunk that exist
                uint64_t v2[16];  // columns col0 + 2j, col0 + 2j + 1
                const uint64_t alpha2 = f2_make(p.alpha, p.alpha);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float4 b = *reinterpret_cast<const float4 *>(bs + 4 * q);
                    v2[2 * q] = f2_fma(alpha2, f2_make_u(r[4 * q], r[4 * q + 1]), f2_make(b.x, b.y));
                    v2[2 * q + 1] = f2_fma(alpha2, f2_make_u(r[4 * q + 2], r[4 * q + 3]), f2_make(b.z, b.w));
                }
                if (p.gelu) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v2[j] = gelu_f2(v2[j]);
                }
                float v[32];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 f = f2_split(v2[j]);
                    v[2 * j] = f.x;
                    v[2 * j + 1] = f.y;
                }
                if constexpr (QOUT) {
                    constexpr int kB = Mx4<NV>::kBlock, kNB = 32 / kB;
                    const int pitch = mx4_code_pitch(p.N), tiles = mx4_stages(p.N) * ST;
                    uint32_t bytes = 0, q[4] = {};
                    if (left < 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j >= left) v[j] = 0.f;
                    }
#pragma unroll
                    for (int b = 0; b < kNB; ++b) {
                        float mx = fabsf(v[b * kB]);
#pragma unroll
                        for (int j = 1; j + 1 < kB; j += 2) mx = fmax3_abs_nan(mx, v[b * kB + j], v[b * kB + j + 1]);
                        mx = fmax3_abs_nan(mx, v[b * kB + kB - 1], 0.f);
                        const Mx4Scale s = mx4_block_scale<NV>(abs_bits(mx), q_ts);
                        const uint64_t mul2 = f2_make(s.mul, s.mul);
                        bytes |= s.byte << (8 * b);
#pragma unroll
                        for (int j = 0; j < kB; j += 8) {
                            float y[8];
#pragma unroll
                            for (int e = 0; e < 8; e += 2) {
                                const float2 f = f2_split(f2_mul(f2_make(v[b * kB + j + e], v[b * kB + j + e + 1]), mul2));
                                y[e] = f.x;
                                y[e + 1] = f.y;
                            }
                            q[(b * kB + j) / 8] = s.zero ? 0u : cvt_e2m1x8(y);
                        }
                    }
                    // (rows past the last: scale 0 to the end of their tile, as the quantiser leaves them)
                    if (row < (n_rows + 127) / 128 * 128) {
                        if (row_ok && col0 / 2 < pitch)
                            *reinterpret_cast<uint4 *>(p.q + (size_t)row * pitch + col0 / 2) = make_uint4(q[0], q[1], q[2], q[3]);
                        const int blk = col0 / kB;
                        uint8_t *sp = p.q_scales + ((size_t)(row >> 7) * tiles + (blk >> 2)) * kMx4TileBytes + (row & 31) * 16 +
                                      ((row >> 5) & 3) * 4 + (blk & 3);
                        if (!row_ok) bytes = 0;
                        if (NV) *reinterpret_cast<uint16_t *>(sp) = (uint16_t)bytes;
                        else *sp = (uint8_t)bytes;
                    }
                } else {
                    const int rows = n_rows - row0 < 32 ? n_rows - row0 : 32;  // of this warp's 32 that exist
                    if constexpr (f32) {
                        // through the warp's own 4 KB; a column per lane to and from global memory
                        __syncwarp();
                        if (res) {
                            copy_async_wait();
                            __syncwarp();
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const uint4 x = ld_shared_u4(stg + (q >> 2) * kTile + stg_off(lane, q & 3));
                                v[4 * q] += __uint_as_float(x.x);
                                v[4 * q + 1] += __uint_as_float(x.y);
                                v[4 * q + 2] += __uint_as_float(x.z);
                                v[4 * q + 3] += __uint_as_float(x.w);
                            }
                        }
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            st_shared_u4(stg + (q >> 2) * kTile + stg_off(lane, q & 3),
                                         make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                                    __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3])));
                        __syncwarp();
                        if (lane < left) {
                            uint32_t *dst = static_cast<uint32_t *>(p.out) + (size_t)row0 * p.ld_out + col0 + lane;
#pragma unroll 8
                            for (int y = 0; y < rows; ++y) dst[(size_t)y * p.ld_out] = ld_shared_u1(col_at + stg_off(y, col_q));
                        }
                        if (res) {
                            __syncwarp();
                            if (i + 1 < PER) res32_issue(w, t, i + 1);
                            else if (wn.u < units) res32_issue(wn, t + 1, 0);
                        }
                    } else {
                        // a 16-bit 32x32 tile
                        const bool f16 = p.out_type == kElemF16;
                        const uint32_t rtile = stg + kTile, tile = stg;
                        if constexpr (RES) {
                            if (tma_res) {
                                bool rok = mbar_wait(rbar, rph, c.abort_flag);
                                if (!__all_sync(0xffffffffu, rok)) { ok = false; break; }
                                rph ^= 1;
                                res_pending = false;
                            } else {  // (rows that are not 16-byte aligned: a column per lane)
                                __syncwarp();
                                if (lane < left) {
                                    const unsigned short *src =
                                        static_cast<const unsigned short *>(p.res) + (size_t)row0 * p.ld_res + col0 + lane;
                                    const uint32_t at = rtile + (lane & 7) * 2;
#pragma unroll 8
                                    for (int y = 0; y < rows; ++y)
                                        st_shared_u16(at + stg_off(y, lane >> 3), src[(size_t)y * p.ld_res]);
                                }
                                __syncwarp();
                            }
                            add_tile16(rtile, lane, f16, v);
                            __syncwarp();
                            if (tma_res) {
                                if (i + 1 < PER) res_issue(w, t, i + 1);
                                else if (wn.u < units) res_issue(wn, t + 1, 0);
                            }
                        }
                        uint32_t o[16];
                        if (f16) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = pack_x2<__half>(v[2 * j], v[2 * j + 1]);
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = pack_x2<bf16>(v[2 * j], v[2 * j + 1]);
                        }
                        // the store that last used this tile has read it (lane 0 has the stores, the
                        // other lanes empty groups: no branch)
                        bulk_wait_read0();
                        __syncwarp();
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            st_shared_u4(tile + stg_off(lane, q), make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]));
                        // by TMA unless rows past the last one would be written, or columns: a store's
                        // end is cut off at 16 bytes, and what lies between is written as 0
                        if (tma_out && (row0 + 32 <= n_rows || n_rows == p.M) && (left >= 32 || tma_out > 1)) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            tma_store_if(lane == 0 && left > 0 && row0 < n_rows, &tmOut, tile, col0, row0);
                            bulk_commit();
                        } else {
                            __syncwarp();
                            if (lane < left) {
                                unsigned short *dst = static_cast<unsigned short *>(p.out) + (size_t)row0 * p.ld_out + col0 + lane;
                                const uint32_t at = tile + (lane & 7) * 2;
                                for (int y = 0; y < rows; ++y)
                                    dst[(size_t)y * p.ld_out] = ld_shared_u16(at + stg_off(y, lane >> 3));
                            }
                            __syncwarp();
                        }
                    }
                }
            }
        }
        // outstanding copies finish before the CTA's shared memory goes away
        if (lane == 0) bulk_wait0();
        if (f32) copy_async_wait();
        if (res_pending && lane == 0) mbar_wait_drain(rbar, rph);
        __syncwarp();
    }
    tc_fence_before();
    if (PAIR) cluster_sync();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *c.abort_flag) set_status(p.status, kStatusTimeout);
}

template <bool NV, bool PAIR, Result OUT>
cudaError_t configure() {
    static std::atomic<unsigned long long> done{0};
    return ensure_smem_attr(reinterpret_cast<const void *>(mx4_gemm_kernel<NV, PAIR, OUT>), Plan<NV, PAIR, OUT>::SMEM, done);
}

template <bool NV, bool PAIR, Result OUT>
cudaError_t launch_tile(const Mx4GemmArgs &a, int num_sms, cudaStream_t s, bool pdl) {
    using P = Plan<NV, PAIR, OUT>;
    CUtensorMap tmA, tmB, tmSA, tmSB;
    const int pitch = mx4_code_pitch(a.K), stages = mx4_stages(a.K);
    const uint64_t ta = (uint64_t)((a.M + 127) / 128) * stages * P::ST, tb = (uint64_t)((a.N + 127) / 128) * stages * P::ST;
    if (make_tmap_u8(&tmA, a.a, a.M, pitch, 128, 128, true) || make_tmap_u8(&tmB, a.w, a.N, pitch, 128, 128, true) ||
        make_tmap_u8(&tmSA, a.a_scales, 2 * ta, 256, 256, 2 * P::ST, false) ||
        make_tmap_u8(&tmSB, a.w_scales, 2 * tb, 256, 256, 2 * P::ST, false))
        return cudaErrorInvalidValue;
    cudaError_t e = configure<NV, PAIR, OUT>();
    if (e != cudaSuccess) return e;
    // a 4-bit result's scale tiles reach to a multiple of 256 columns
    const int n_sub = ((OUT == Result::k4Bit ? mx4_stages(a.N) * kMx4StageCols : a.N) + P::TN - 1) / P::TN;
    const long long units = (long long)((a.M + P::UM - 1) / P::UM) * n_sub;
    if (units > 0x7fffff00LL - num_sms) return cudaErrorInvalidValue;
    const int slots = PAIR ? num_sms / 2 : num_sms;
    const int grid = (PAIR ? 2 : 1) * (int)(units < slots ? units : slots);
    const int es = a.out_type == kElemF32 ? 4 : 2;
    auto ok16 = [&](const void *q, long long ld) { return q && (reinterpret_cast<uintptr_t>(q) & 15) == 0 && ld * es % 16 == 0; };
    CUtensorMap tmOut = tmA, tmRes = tmA;
    const int tma_res = ok16(a.res, a.ld_res) && a.out_type != kElemF32;
    // (2: a row's end is a multiple of 16 bytes too)
    const int tma_out = ok16(a.out, a.ld_out) && a.out_type != kElemF32 ? (a.N % 8 == 0 ? 2 : 1) : 0;
    if ((tma_out && make_tmap_tile16(&tmOut, a.out, a.out_type, a.M, a.N, a.ld_out)) ||
        (tma_res && make_tmap_tile16(&tmRes, a.res, a.out_type, a.M, a.N, a.ld_res)))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (PAIR) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = 2;
        attr[na].val.clusterDim.y = 1;
        attr[na++].val.clusterDim.z = 1;
    }
    if (pdl) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see launch_pdl
        attr[na++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = P::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = na;
    return cudaLaunchKernelEx(&cfg, mx4_gemm_kernel<NV, PAIR, OUT>, tmA, tmB, tmSA, tmSB, tmOut, tmRes, a, n_sub, tma_out,
                              tma_res);
}

template <bool NV, Result OUT>
cudaError_t launch_fmt(const Mx4GemmArgs &a, int num_sms, cudaStream_t s, bool pdl) {
    // The cheaper of the two shapes by their waves: measured in both formats over 64..9000 rows,
    // N 768..4096, K 768..4096 (stages 3, 8, 16), a launch takes about 4.4 us + waves (0.36 +
    // 0.33 stages) on single 128x128 tiles and 5.4 us + waves (1.05 + 0.35 stages) on pairs'
    // 256x256 tiles (mxfp4: 3000x2304x4096 19.8 against 17.8; 4096x2304x768 9.2 against 10.0,
    // where the rule is wrong by most, it takes the pairs; 1500x4096x4096 19.2 against 17.7).
    const int stages = mx4_stages(a.K);
    const long long single = (long long)((a.M + 127) / 128) * ((a.N + 127) / 128);
    const long long pair = (long long)((a.M + 255) / 256) * ((a.N + 255) / 256);
    const long long waves1 = (single + num_sms - 1) / num_sms, waves2 = (pair + num_sms / 2 - 1) / (num_sms / 2);
    if (540 + waves2 * (105 + 35 * stages) < 440 + waves1 * (36 + 33 * stages))
        return launch_tile<NV, true, OUT>(a, num_sms, s, pdl);
    return launch_tile<NV, false, OUT>(a, num_sms, s, pdl);
}

}  // namespace

cudaError_t launch_mx4_gemm(const Mx4GemmArgs &a, int num_sms, cudaStream_t s, bool pdl) {
    if (a.M < 1) return cudaSuccess;
    switch (a.q ? Result::k4Bit : a.out_type == kElemF32 ? Result::kF32 : a.res ? Result::k16BitRes : Result::k16Bit) {
        case Result::k4Bit:
            return a.nv ? launch_fmt<true, Result::k4Bit>(a, num_sms, s, pdl) : launch_fmt<false, Result::k4Bit>(a, num_sms, s, pdl);
        case Result::kF32:
            return a.nv ? launch_fmt<true, Result::kF32>(a, num_sms, s, pdl) : launch_fmt<false, Result::kF32>(a, num_sms, s, pdl);
        case Result::k16BitRes:
            return a.nv ? launch_fmt<true, Result::k16BitRes>(a, num_sms, s, pdl) : launch_fmt<false, Result::k16BitRes>(a, num_sms, s, pdl);
        case Result::k16Bit:
            return a.nv ? launch_fmt<true, Result::k16Bit>(a, num_sms, s, pdl) : launch_fmt<false, Result::k16Bit>(a, num_sms, s, pdl);
    }
    return cudaErrorInvalidValue;
}

}  // namespace albert
