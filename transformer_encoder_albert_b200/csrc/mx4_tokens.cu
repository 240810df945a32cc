// mx4_tokens.cu -- the linear layer on 4-bit operands for a few rows (tokens): one
// launch that quantizes the rows itself and is bound by reading the weights.
//
// The operands change places: 128 rows of W (features) are the product's M, the
// tokens its N, so a 128x256 block of codes (16 KB) and its scales feed four
// products whose cost does not matter.  A CTA holds one 128-feature tile and a slice
// of K; a cluster of up to 8 CTAs shares a tile's K when the tiles alone would leave
// SMs without work, and adds the partial sums over distributed shared memory in rank
// order (no atomics, the same bits every time, no workspace).
//   warp 0      : TMA ring of weight stages (all in flight before any product);
//   warp 14     : copies a stage's scales to tensor memory.  A ring stage has scale
//                 columns of its own there, so the stage's barrier guards them too;
//   warp 1      : products;
//   warps 2..13 : quantize (or copy) the tokens into a stage's second operand, then the
//                 epilogue.
// Rows of the token operand past the last token are never written: they only reach
// result columns that nobody reads.
#include <type_traits>

#include "mx4.cuh"
#include "mx4.h"
#include "mx4_ptx.cuh"

namespace albert {
namespace {

constexpr int kWorkers = 12;  // two per stage of a full ring (one left 16 tokens at 2.5 TB/s of weights)
constexpr int kTokThreads = 32 * (3 + kWorkers);
constexpr int kWBytes = 128 * 128;   // codes of a weight stage
constexpr int kMaxRing = 6;            // at most kWorkers
constexpr int kMaxCluster = 8;

template <bool NV, int NT>
struct TokPlan {
    static constexpr int ST = Mx4<NV>::kStageTiles;
    static constexpr int RING = kWBytes + ST * kMx4TileBytes;           // bytes of a stage's weights
    static constexpr int TOK = NT * 128 + ST * kMx4TileBytes;           // and of its tokens
    static constexpr int SFCOLS = 8 * ST;                               // scale columns of a ring stage
    static constexpr int COLS = NT + kMaxRing * SFCOLS <= 128 ? 128 : 256;
    static_assert(NT + kMaxRing * SFCOLS <= 256, "tensor memory columns");
    // CTAs of a cluster wait for one another, so none may hold tensor memory that keeps
    // another from starting: a CTA takes at least its columns' share of an SM's shared
    // memory (228 KB for 512 columns, 1 KB of each CTA's being the system's), and what
    // fits an SM by shared memory also fits it by tensor memory.
    static constexpr int kLeast = 233472 / 512 * COLS - 1024 - 64;
    static int smem(int ring) {
        const int n = 1024 + ring * (RING + TOK) + NT * 128 * 4 + 512;
        return n > kLeast ? n : kLeast;
    }
};

__device__ __forceinline__ float ld_dsmem_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_u2(uint32_t a, uint2 v) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ void st_shared_u1(uint32_t a, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
// Rows r0 .. r0 + 2 PAIRS - 1 of a 256-column stage of the tokens, by a warp: a
// half-warp per row, 16 columns a lane; the row pairs' loads and chains of dependent
// instructions overlap (rows past the last read as 0 and are not stored).
template <typename T, int PAIRS>
struct TokenRows {
    Raw8<T> a[PAIRS], b[PAIRS];
    __device__ __forceinline__ void load(const Mx4TokArgs &p, int r0, int kb, int lane) {
        const int col = kb * kMx4StageCols + (lane & 15) * 16;
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const int row = r0 + 2 * i + (lane >> 4);
            const T *src = static_cast<const T *>(p.x) + (size_t)row * p.ld_x + col;
            const int n = row < p.M ? p.K - col : 0;
            a[i] = load_raw8<T>(src, n, p.vec_x != 0);
            b[i] = load_raw8<T>(src + 8, n - 8, p.vec_x != 0);
        }
    }
    template <bool NV>
    __device__ __forceinline__ void quantize(const Mx4TokArgs &p, int r0, uint32_t codes, uint32_t scales, int lane) const {
        const int sub = lane & 15;
        const Mx4Ts ts = mx4_ts(p.x_ts);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const int row = r0 + 2 * i + (lane >> 4);
            uint32_t m = umax(raw8_amax<T>(a[i]), raw8_amax<T>(b[i]));
            if constexpr (!NV) m = umax(m, __shfl_xor_sync(0xffffffffu, m, 1));
            const Mx4Scale s = mx4_block_scale<NV>(amax_f32_bits<T>(m), ts);
            float v[8], u[8];
            raw8_values<T>(a[i], v);
            raw8_values<T>(b[i], u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = __fmul_rn(v[e], s.mul);
                u[e] = __fmul_rn(u[e], s.mul);
            }
            const uint2 q = s.zero ? make_uint2(0, 0) : make_uint2(cvt_e2m1x8(v), cvt_e2m1x8(u));
            constexpr int kLanes = NV ? 1 : 2, kTileLanes = 4 * kLanes;
            uint32_t word = s.byte << (8 * ((sub / kLanes) & 3));
            word |= __shfl_xor_sync(0xffffffffu, word, kLanes);
            word |= __shfl_xor_sync(0xffffffffu, word, 2 * kLanes);
            if (row < p.M) {
                // 128-byte rows with the 128-byte swizzle (16-byte chunk index XOR row % 8)
                st_shared_u2(codes + row * 128 + (((sub >> 1) ^ (row & 7)) << 4) + (sub & 1) * 8, q);
                if (sub % kTileLanes == 0) st_shared_u1(scales + (sub / kTileLanes) * kMx4TileBytes + row * 16, word);
            }
        }
    }
};

// A warp's stages i = first, first + ring, ... of the tokens.  The first rows of the
// next stage load while the current one is converted and while its slot is still being
// read: reading them after the wait left each stage to the latency of L2.
template <typename T, bool NV, int PAIRS, typename Slot>
__device__ __forceinline__ void feed_tokens(const Mx4TokArgs &p, int first, int kb0, int nkb, int ring, int part, int parts,
                                            int lane, Slot slot) {
    TokenRows<T, PAIRS> now, next;
    const int own = part * 2 * PAIRS, step = parts * 2 * PAIRS;  // this warp's rows of a stage
    if (first < nkb) next.load(p, own, kb0 + first, lane);
    for (int i = first; i < nkb; i += ring) {
        now = next;
        if (i + ring < nkb) next.load(p, own, kb0 + i + ring, lane);
        uint32_t codes, scales;
        if (!slot.take(codes, scales)) return;
        if (own < p.M) now.template quantize<NV>(p, own, codes, scales, lane);
        for (int r0 = own + step; r0 < p.M; r0 += step) {
            now.load(p, r0, kb0 + i, lane);
            now.template quantize<NV>(p, r0, codes, scales, lane);
        }
        slot.give();
    }
}
// No more row pairs per warp than the tokens need: a chain of four pairs takes about
// 1.5 us, of one 0.5 us.
template <typename T, bool NV, typename Slot>
__device__ __forceinline__ void feed_any(const Mx4TokArgs &p, int first, int kb0, int nkb, int ring, int part, int parts,
                                         int lane, Slot slot) {
    if (p.M <= 2 * parts) feed_tokens<T, NV, 1>(p, first, kb0, nkb, ring, part, parts, lane, slot);
    else if (p.M <= 4 * parts || sizeof(T) == 4) feed_tokens<T, NV, 2>(p, first, kb0, nkb, ring, part, parts, lane, slot);
    else feed_tokens<T, NV, 4>(p, first, kb0, nkb, ring, part, parts, lane, slot);
}

template <bool NV>
__device__ __forceinline__ void stage_packed(const Mx4TokArgs &p, int kb, int first, int step, uint32_t codes,
                                             uint32_t scales, int lane) {
    constexpr int ST = Mx4<NV>::kStageTiles;
    const int sub = lane & 15, half = lane >> 4, pitch = mx4_code_pitch(p.K), byte = kb * 128 + sub * 8;
    for (int r0 = first; r0 < p.M; r0 += step) {
        const int row = r0 + half;
        if (row >= p.M) continue;
        uint2 q = make_uint2(0, 0);
        if (byte < pitch) q = __ldg(reinterpret_cast<const uint2 *>(p.a + (size_t)row * pitch + byte));
        st_shared_u2(codes + row * 128 + (((sub >> 1) ^ (row & 7)) << 4) + (sub & 1) * 8, q);
        if (sub < ST)  // (rows below 32: the first words of the tile's lanes)
            st_shared_u1(scales + sub * kMx4TileBytes + row * 16,
                         __ldg(reinterpret_cast<const uint32_t *>(p.a_scales + ((size_t)kb * ST + sub) * kMx4TileBytes + row * 16)));
    }
}

template <bool NV, int NT>
__global__ void __launch_bounds__(kTokThreads)
mx4_tokens_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmSW, const Mx4TokArgs p,
                  int ring, int nclu, int stream_w) {
    using P = TokPlan<NV, NT>;
    constexpr int ST = P::ST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sW = base, *sT = sW + ring * kWBytes;                              // codes: weights, tokens
    uint8_t *sSW = sT + ring * NT * 128, *sST = sSW + ring * ST * kMx4TileBytes;  // scale tiles
    float *sum = reinterpret_cast<float *>(sST + ring * ST * kMx4TileBytes);      // [NT][128] partial sums
    uint64_t *bars = reinterpret_cast<uint64_t *>(sum + NT * 128);
    uint64_t *full = bars, *empty = bars + kMaxRing, *ready = bars + 2 * kMaxRing, *scaled = bars + 3 * kMaxRing, *done = bars + 4 * kMaxRing;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = nclu > 1 ? cluster_ctarank() : 0;
    const int tile = (int)(blockIdx.x / nclu);
    const int stages = mx4_stages(p.K);
    const int kb0 = (int)((long long)stages * rank / nclu), kb1 = (int)((long long)stages * (rank + 1) / nclu);
    const int nkb = kb1 - kb0;  // >= 1

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        wait_limit_init(p.wait_ns);
        for (int i = 0; i < ring; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), 1);
            mbar_init(smem_u32(&ready[i]), 32 * (kWorkers / ring));
            mbar_init(smem_u32(&scaled[i]), 2);
        }
        mbar_init(smem_u32(done), 2);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), P::COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t once = policy_evict_first();
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            for (int kb = p.withhold_loads ? kb1 : kb0; kb < kb1; ++kb) {
                if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1, abort_flag)) break;
                const uint32_t fb = smem_u32(&full[stage]);
                mbar_arrive_expect_tx(fb, P::RING);
                if (stream_w)
                    tma_load_2d_hint(smem_u32(sW) + stage * kWBytes, &tmW, fb, kb * 128, tile * 128, once);
                else
                    tma_load_2d(smem_u32(sW) + stage * kWBytes, &tmW, fb, kb * 128, tile * 128);
                tma_load_2d(smem_u32(sSW) + stage * ST * kMx4TileBytes, &tmSW, fb, 0, (tile * stages + kb) * 2 * ST);
                ++issued;
                if (++stage == ring) { stage = 0; phase ^= 1; }
            }
            // (the last of each slot: a wait that ran out in another warp leaves nobody else to see
            // them land, and the CTA's memory must outlast them)
            for (int i = 0; i < ring && i < issued; ++i) {
                if (--stage < 0) { stage = ring - 1; phase ^= 1; }
                mbar_wait_drain(smem_u32(&full[stage]), phase);
            }
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2 + kWorkers) {
        const uint32_t leader = elect_leader();
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag)) != 0;
        };
        uint32_t stage = 0, phase = 0;
        for (int i = 0; i < nkb; ++i) {
            const uint32_t ca = tmem + NT + stage * P::SFCOLS, cb = ca + 4 * ST;
            if (warp == 1) {
                // the scale warp, which has waited for the stage's operands, arrives here too
                if (!wait(&scaled[stage], phase)) break;
                tc_fence_after();
                const uint32_t w0 = smem_u32(sW) + stage * kWBytes, t0 = smem_u32(sT) + stage * NT * 128;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int g = NV ? k : k >> 1;
                    umma_mx4<NV, false>(leader, tmem, sw128_kmajor_desc(w0 + k * 32), sw128_kmajor_desc(t0 + k * 32),
                                        idesc_mx4<NV>(128, NT, NV ? 0 : 2 * (k & 1)), ca + 4 * g, cb + 4 * g, (i | k) != 0);
                }
                umma_commit_elected<false>(leader, smem_u32(empty) + 8 * stage, 0);
            } else {
                if (!wait(&full[stage], phase) || !wait(&ready[stage], phase)) break;
                tc_fence_after();
                const uint32_t fw = smem_u32(sSW) + stage * ST * kMx4TileBytes, ft = smem_u32(sST) + stage * ST * kMx4TileBytes;
#pragma unroll
                for (int g = 0; g < ST; ++g) {
                    tmem_cp_scales<false>(leader, ca + 4 * g, scale_tile_desc(fw + g * kMx4TileBytes));
                    tmem_cp_scales<false>(leader, cb + 4 * g, scale_tile_desc(ft + g * kMx4TileBytes));
                }
                umma_commit_elected<false>(leader, smem_u32(scaled) + 8 * stage, 0);
                if (lane == 0) mbar_arrive(smem_u32(scaled) + 8 * stage);
            }
            if (++stage == (uint32_t)ring) { stage = 0; phase ^= 1; }
        }
        // (after a wait that ran out too: what was issued before it must complete)
        umma_commit_elected<false>(leader, smem_u32(done), 0);
    } else {
        // ------------------------------------------------------------ tokens --
        const int wk = warp - 2;
        // a warp fills the same ring stage every time, so that it never waits for a phase two
        // ahead of the barrier's; where the ring is short, several warps share a stage's rows
        const int own = wk % ring, part = wk / ring, parts = kWorkers / ring;
        struct Slot {
            uint32_t codes, scales, empty, ready, phase;
            volatile int *abort_flag;
            __device__ bool take(uint32_t &c, uint32_t &s) {
                c = codes;
                s = scales;
                const bool ok = __all_sync(0xffffffffu, mbar_wait(empty, phase, abort_flag));
                phase ^= 1;
                return ok;
            }
            __device__ void give() {
                fence_proxy_async_smem();  // the products read this through the async proxy
                mbar_arrive(ready);
            }
        } sl{smem_u32(sT) + own * NT * 128, smem_u32(sST) + own * ST * kMx4TileBytes, smem_u32(&empty[own]),
             smem_u32(&ready[own]), 1, abort_flag};
        if (part < parts) {
            if (!p.x) {
                for (int i = own; i < nkb; i += ring) {
                    uint32_t codes, scales;
                    if (!sl.take(codes, scales)) break;
                    stage_packed<NV>(p, kb0 + i, 2 * part, 2 * parts, codes, scales, lane);
                    sl.give();
                }
            } else if (p.x_type == kElemF32) {
                feed_any<float, NV>(p, own, kb0, nkb, ring, part, parts, lane, sl);
            } else if (p.x_type == kElemF16) {
                feed_any<__half, NV>(p, own, kb0, nkb, ring, part, parts, lane, sl);
            } else {
                feed_any<bf16, NV>(p, own, kb0, nkb, ring, part, parts, lane, sl);
            }
        }
    }
    // ------------------------------------------------------------- epilogue --
    // Every product has completed, or a wait has run out somewhere in this CTA; then what is in
    // flight still ends before tensor memory is read or freed and the CTA's memory goes away.
    const bool got = mbar_wait(smem_u32(done), 0, abort_flag);
    if (!got) mbar_wait_drain(smem_u32(done), 0);
    const bool ok = __syncthreads_and(got && *abort_flag == 0) != 0;
    tc_fence_after();
    if (warp >= 2 && warp < 6) {
        // lane quadrant warp % 4: feature 32 (warp % 4) + lane
        const int quad = warp & 3;
        uint32_t r[32];
        tmem_ld32(tmem + ((uint32_t)(quad * 32) << 16), r);  // (columns past NT: not read below)
        tmem_ld_wait();
#pragma unroll
        for (int t = 0; t < NT; ++t) sum[t * 128 + quad * 32 + lane] = __uint_as_float(r[t]);
    }
    tc_fence_before();
    if (nclu > 1) cluster_sync();
    else __syncthreads();
    if (warp >= 2 && warp < 2 + kWorkers && ok) {
        const int wk = warp - 2, f = (wk & 3) * 32 + lane, feat = tile * 128 + f;
        const float bias = p.bias && feat < p.N ? __ldg(p.bias + feat) : 0.f;
        const uint32_t own = smem_u32(sum);
        const Mx4Ts q_ts = mx4_ts(p.q_ts);
        if (!p.out) {  // scale bytes of the rows past the last token, to the end of their tile
            constexpr int kTiles = 128 / Mx4<NV>::kTileCols;
            for (int i = threadIdx.x - 64 + (int)rank * 32 * kWorkers; i < 128 * kTiles; i += 32 * kWorkers * nclu) {
                const int r = i & 127;
                if (r >= p.M)
                    *reinterpret_cast<uint32_t *>(p.q_scales + (size_t)(tile * kTiles + (i >> 7)) * kMx4TileBytes + (r & 31) * 16 +
                                                  (r >> 5) * 4) = 0;
            }
        }
        // this CTA's tokens: rank, rank + nclu, ..., the groups of four warps in turn
        for (int t = (int)rank + (wk >> 2) * nclu; t < p.M; t += kWorkers / 4 * nclu) {
            float acc = 0.f;
            if (nclu == 1) {
                acc = sum[t * 128 + f];
            } else {
                for (int c = 0; c < nclu; ++c) acc += ld_dsmem_f32(mapa_shared(own + (t * 128 + f) * 4, c));
            }
            float v = fmaf(p.alpha, acc, bias);
            if (p.gelu) v = f2_split(gelu_f2(f2_make(v, 0.f))).x;
            if (p.out) {
                if (feat < p.N) {
                    const size_t ro = (size_t)t * p.ld_res + feat, oo = (size_t)t * p.ld_out + feat;
                    if (p.out_type == kElemF32) {
                        if (p.res) v += static_cast<const float *>(p.res)[ro];
                        static_cast<float *>(p.out)[oo] = v;
                    } else if (p.out_type == kElemF16) {
                        if (p.res) v += __half2float(static_cast<const __half *>(p.res)[ro]);
                        static_cast<__half *>(p.out)[oo] = __float2half_rn(v);
                    } else {
                        if (p.res) v += __bfloat162float(static_cast<const bf16 *>(p.res)[ro]);
                        static_cast<bf16 *>(p.out)[oo] = __float2bfloat16_rn(v);
                    }
                }
            } else {
                // 4-bit result: a warp's 32 features are one block (mxfp4) or two (nvfp4)
                if (feat >= p.N) v = 0.f;
                uint32_t m = abs_bits(v);
#pragma unroll
                for (int o = 1; o < Mx4<NV>::kBlock; o <<= 1) m = umax(m, __shfl_xor_sync(0xffffffffu, m, o));
                const Mx4Scale s = mx4_block_scale<NV>(m, q_ts);
                float y[8];
                y[0] = __fmul_rn(v, s.mul);
#pragma unroll
                for (int j = 1; j < 8; ++j) y[j] = __shfl_down_sync(0xffffffffu, y[0], j);
                const uint32_t q = s.zero ? 0u : cvt_e2m1x8(y);
                const int pitch = mx4_code_pitch(p.N);
                if ((lane & 7) == 0 && feat / 2 < pitch) *reinterpret_cast<uint32_t *>(p.q + (size_t)t * pitch + feat / 2) = q;
                if (lane % Mx4<NV>::kBlock == 0) {
                    // (token t < 32: row t of the first row tile)
                    const int blk = feat / Mx4<NV>::kBlock;
                    p.q_scales[(size_t)(blk >> 2) * kMx4TileBytes + t * 16 + (blk & 3)] = (uint8_t)s.byte;
                }
            }
        }
    }
    // a peer may still read this CTA's partial sums
    if (nclu > 1) cluster_sync();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, P::COLS);
    }
    if (threadIdx.x == 0 && *abort_flag) set_status(p.status, kStatusTimeout);
}

template <bool NV, int NT>
cudaError_t launch_tok(const Mx4TokArgs &a, int num_sms, cudaStream_t s) {
    using P = TokPlan<NV, NT>;
    const int stages = mx4_stages(a.K), pitch = mx4_code_pitch(a.K);
    // a 4-bit result's scale tiles reach to a multiple of 256 columns
    const int tiles = ((a.out ? a.N : mx4_stages(a.N) * kMx4StageCols) + 127) / 128;
    // as many CTAs per tile as there are SMs for, stages of K, and the portable cluster size
    int nclu = tiles < num_sms ? num_sms / tiles : 1;
    nclu = nclu < stages ? nclu : stages;
    nclu = nclu < kMaxCluster ? nclu : kMaxCluster;
    const int slice = (stages + nclu - 1) / nclu;
    const int ring = slice < kMaxRing ? slice : kMaxRing;
    CUtensorMap tmW, tmSW;
    const uint64_t st = (uint64_t)((a.N + 127) / 128) * stages * P::ST;
    if (make_tmap_u8(&tmW, a.w, a.N, pitch, 128, 128, true) || make_tmap_u8(&tmSW, a.w_scales, 2 * st, 256, 256, 2 * P::ST, false))
        return cudaErrorInvalidValue;
    // A matrix of more than a quarter of L2 (126 MB) does not last there until its next use,
    // behind the layers in between: it passes through (16384 x 8192: 18.0 us against 19.2);
    // a smaller one stays.
    const int stream_w = (long long)a.N * pitch > 32ll << 20;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(mx4_tokens_kernel<NV, NT>), P::smem(kMaxRing), done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = nclu;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(tiles * nclu);
    cfg.blockDim = dim3(kTokThreads);
    cfg.dynamicSmemBytes = P::smem(ring);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = nclu > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, mx4_tokens_kernel<NV, NT>, tmW, tmSW, a, ring, nclu, stream_w);
}

}  // namespace

cudaError_t launch_mx4_tokens(const Mx4TokArgs &a, int num_sms, cudaStream_t s) {
    if (a.M < 1) return cudaSuccess;
    if (a.M <= 16) return a.nv ? launch_tok<true, 16>(a, num_sms, s) : launch_tok<false, 16>(a, num_sms, s);
    return a.nv ? launch_tok<true, 32>(a, num_sms, s) : launch_tok<false, 32>(a, num_sms, s);
}

}  // namespace albert
