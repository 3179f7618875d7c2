// Dense product of FP8_B128 operands (bloomery issue page, s.3 "Kernel
// dispatch": the FP8 release's block-scaled matrices; s.2: ReLU^2):
//
//   z[m,n]   = sum_b sx[m,b] * sw[n,b] * sum_{k in block b} qx[m,k] qw[n,k]
//   out[m,n] = bf16(z) or bf16(relu(z)^2)
//
// E4M3 codes, one fp32 scale per 128 values along K of each row of either
// operand, fp32 sums.  Two kernels by the number of rows M:
//
//  - M <= 16: a weight stream.  Every CTA owns an equal share of the N weight
//    rows over the whole of K (weight_stream.cuh); eight warps split K and add
//    their sums once.  Bound: HBM bytes and the launch.
//  - above: tcgen05 tiles of 128 rows of x by BN rows of w.  A 128-byte K
//    stage is one scale block, so its product goes to a TMEM slot of its own
//    and the epilogue warps, which hold the tile's fp32 sums in registers, add
//    it times both scales while the tensor core fills the next slot.  Two
//    operations of fp32 per value and block take as long as the tensor core's
//    own work (512 cycles of an SM for 128 x 256 x 128), and the registers
//    that TMEM values arrive in do not pair up for the two-wide instructions
//    without a move each: the sums bound large products.
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "weight_stream.cuh"

namespace moe {

struct LinearArgs {
    const uint8_t* xq;    // [M][Kp]
    const float* xs;      // [M][kb]
    const uint8_t* wq;    // [N][Kp]
    const float* ws;      // [N][kb]
    uint16_t* out;        // [M][N]
    int64_t M;
    int N, Kp, kb;
    int relu2;
};

__device__ __forceinline__ float lin_act(float z, int relu2) {
    return relu2 ? (z <= 0.0f ? 0.0f : __fmul_rn(z, z)) : z;   // a NaN stays one
}

// ----------------------------------------------------------------------------- few rows

struct LinearFewArgs {
    LinearArgs l;
    FwShare share;
    int chunks;         // of a weight row
    int slot_bytes, n_stages;
};

struct LinearFewMaps {
    CUtensorMap w[2];   // boxes of share.rows weight rows, and of one less
};

// MT tiles of 16 weight rows per unit, TT of 8 rows of x.
template <int MT, int TT>
__global__ void __launch_bounds__(FW_THREADS, 1)
    linear_few_kernel(const __grid_constant__ LinearFewMaps maps, LinearFewArgs a, DevCtx ctx) {
    extern __shared__ __align__(1024) uint8_t lf_smem[];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    FwRed red;
    red.buf = reinterpret_cast<float*>(lf_smem + (size_t)FW_WARPS * a.n_stages * a.slot_bytes);
    FwRings rings;
    rings.base = lf_smem;
    rings.full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(red.buf) + FwRed::bytes(a.share.units));
    rings.empty = rings.full + FW_WARPS * FW_MAX_STAGES;
    rings.slot_bytes = a.slot_bytes;
    rings.n = a.n_stages;
    uint64_t* rbar = rings.full + FwRings::kBarBytes / 8;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(rbar + 1);
    red.bar = smem_u32(rbar);
    red.turn = 0;
    if (tid == 0) {
        rings.init();
        mbar_init(smem_u32(rbar), FW_WARPS);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.w[0]);
    }
    __syncthreads();
    pdl_enter();

    const LinearArgs& l = a.l;
    const int n_units = gridDim.x * a.share.units;
    auto unit_row = [&](int u) { return (int)((int64_t)u * l.N / n_units); };
    if (warp >= FW_WARPS) {   // producers: a lane fills ring w, every eighth chunk of each unit
        fw_producer_regs();
        const uint64_t policy = l2_policy_evict_first();
        const bool mine = fw_put_lane();
        const int w = mine ? fw_put_ring() : 0;
        FwPut put(rings, w);
        int unit = -1, k = 0, n0 = 0, n = 0;
        auto next_unit = [&]() {
            k = w;
            do {
                if (++unit == a.share.units || k >= a.chunks) return false;
                const int u = blockIdx.x * a.share.units + unit;
                n0 = unit_row(u);
                n = unit_row(u + 1) - n0;
            } while (n <= 0);
            return true;
        };
        const bool active = mine && next_unit();
        auto step = [&]() {
            put.fill(&maps.w[a.share.rows - n], k * FW_CHUNK, n0, n * FW_CHUNK, policy);
            k += FW_WARPS;
            return k < a.chunks || next_unit();
        };
        if (!fw_produce(put, active, step, ctx, abort_flag)) fw_settle();
        return;
    }

    fw_consumer_regs();
    FwTake ring(rings, warp);
    const int g = lane / 4, q = lane % 4;
    const int M = (int)l.M;
    FwSide<TT> side;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int row = min(t * 8 + g, M - 1);
        side.act[t] = l.xq + (int64_t)row * l.Kp + q * 16;
    }
    side.xs = l.xs + (int64_t)min(lane, M - 1) * l.kb;
    for (int un = 0; un < a.share.units; ++un) {
        const int u = blockIdx.x * a.share.units + un;
        const int n0 = unit_row(u), n = unit_row(u + 1) - n0;
        FwAcc<MT, TT> acc;
        acc.clear();
        if (n > 0 && warp < a.chunks) {
            side.ws = l.ws + (int64_t)(n0 + min(lane, n - 1)) * l.kb;
            FwActs<TT> v;
            fw_fetch(v, side, warp * FW_CHUNK, l.Kp);
            for (int k = warp; k < a.chunks;) {
                if (!ring.wait(ctx, abort_flag)) return fw_settle();
                fw_mul(acc, ring.data(), n, v);
                ring.release();
                k += FW_WARPS;
                if (k < a.chunks) fw_fetch(v, side, k * FW_CHUNK, l.Kp);
            }
        }
        float* mine = red.mine(warp);
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int r = 0; r < MT + 1; ++r)   // rows g + 8 r
                    mine[(t * 8 + 2 * q + c) * FW_ROWS + g + 8 * r] = acc.d[r / 2][t][c + 2 * (r % 2)];
        if (!red.exchange(ctx, abort_flag)) return fw_settle();
        for (int j = tid; j < n * M; j += 32 * FW_WARPS) {
            const int t = j / n, row = j - t * n;
            const float z = red.sum(t, row);
            l.out[(int64_t)t * l.N + n0 + row] = __bfloat16_as_ushort(__float2bfloat16_rn(lin_act(z, l.relu2)));
        }
    }
}

// ----------------------------------------------------------------------------- tiles

constexpr int LT_BM = 128;              // rows of x per tile (TMEM lanes)
constexpr int LT_KB = 128;              // bytes of K per stage: one scale block
constexpr int LT_EPI = 8;               // epilogue warps: two per TMEM lane quadrant
constexpr int LT_THREADS = 32 * (4 + LT_EPI);
constexpr int LT_MMA = 2;               // threads that issue products: the issue of one stage takes one thread
                                        // about as long as the tensor core's work for a narrow tile (410 to 480 cycles,
                                        // in a branch of one lane; from a converged warp it was not measured)
constexpr int LT_SC = 8;                // blocks of K of a scale slot: whole pairs of stages
constexpr int LT_SS = 2;                // slots of the scale ring
constexpr int LT_MAX_STAGES = 8;

template <int BN>
struct LtShape {
    // TMEM holds the products of two pairs of stages: taken two at a time, the waits, counters and
    // branches of a stage's sums cost half as much (they took as many instructions as the sums)
    static constexpr int kSlots = 2;
    static constexpr int kTmem = 2 * kSlots * BN;                         // columns
    static constexpr int kStage = (LT_BM + BN) * LT_KB;
    // a scale slot is [LT_SC][kLd] floats; 4 words over a multiple of 32, so that the copies of 4 rows by
    // 8 blocks meet 32 banks
    static constexpr int kLd = LT_BM + BN + 4;
    static constexpr int kScale = LT_SC * kLd * 4;
    static constexpr int kCols = BN / 2;                               // columns of an epilogue warp
};

struct LinearTileArgs {
    LinearArgs l;
    int m_tiles, n_tiles;
    int n_stages;
};

struct LinearMaps {
    CUtensorMap x, w;
};

__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// 16 TMEM lanes by 32 columns: v[4 j + 2 i + e] is row lane / 4 + 8 i, column 8 j + 2 (lane % 4) + e.  So a
// thread meets a quarter of the columns: with a row per thread each of them reads every column's scale,
// and those reads (four cycles of shared memory for 16 bytes, however few addresses) took 1.2k cycles of
// a stage of 128 x 256.  The wait names the registers, so that nothing reads them before it.
// Two loads of eight registers: one of sixteen leaves the sums more moves to make (194 against 187 us at
// 4096 x 10752 x 2688), four of four as well (196).
__device__ __forceinline__ void lt_tmem_ld(uint32_t taddr, uint32_t (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; i += 8)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]),
                       "=r"(v[i + 6]), "=r"(v[i + 7])
                     : "r"(taddr + 2 * i));
}
__device__ __forceinline__ void lt_tmem_wait(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                   "+r"(v[15]));
}

// The four lanes of a quad hold one row's words of four 16-byte pieces, word l of each in lane l;
// afterwards lane l holds piece l.
__device__ __forceinline__ void lt_transpose(uint32_t (&p)[4], int l) {
#pragma unroll
    for (int d = 1; d <= 2; d *= 2) {
        const bool hi = l & d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & d) continue;
            const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? p[i] : p[i + d], d);
            if (hi) p[i] = got;
            else p[i + d] = got;
        }
    }
}

// Every lane looks for itself, and only a wait that is not over takes the slow way: one lane's look and a
// shuffle of what it saw cost each stage of a warp more than its sums.
__device__ __forceinline__ bool lt_wait(uint32_t bar, uint32_t parity, const DevCtx& ctx, volatile int* abort) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return mbar_wait_warp(bar, parity, ctx, abort);
}

// A warp's wait for something thousands of cycles away.
__device__ __forceinline__ bool lt_wait_long(uint32_t bar, uint32_t parity, const DevCtx& ctx, volatile int* abort) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (globaltimer() - t0 > ctx.timeout_ns) {
            record_error(ctx.err, MOE_ETIMEOUT);
            *abort = 1;
            return false;
        }
        __nanosleep(500);
    }
    return true;
}

// Persistent over the tiles, the row tiles of one weight tile first.  Warp 0 loads the codes (TMA), warps
// 1 and 3 issue the products of the ring's even and odd slots (by turns within a tile, a slot's uses could be
// the other thread's, and the parity of full that of the use two back), warp 2 copies the scales, the others
// sum and store.
template <int BN>
__global__ void __launch_bounds__(LT_THREADS, 1)
    linear_tile_kernel(const __grid_constant__ LinearMaps maps, LinearTileArgs a, DevCtx ctx) {
    using S = LtShape<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const int NS = a.n_stages;
    uint8_t* scales = smem + (size_t)NS * S::kStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + LT_SS * S::kScale);
    uint64_t* empty = full + LT_MAX_STAGES;
    uint64_t* pfull = empty + LT_MAX_STAGES;
    uint64_t* pempty = pfull + S::kSlots;
    uint64_t* sfull = pempty + S::kSlots;
    uint64_t* sempty = sfull + LT_SS;
    uint64_t* drain = sempty + LT_SS;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(drain + LT_MMA);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + LT_MMA) + 1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const LinearArgs& l = a.l;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int p = 0; p < S::kSlots; ++p) {
            mbar_init(smem_u32(&pfull[p]), LT_MMA);
            mbar_init(smem_u32(&pempty[p]), LT_EPI);
        }
        for (int s = 0; s < LT_SS; ++s) {
            mbar_init(smem_u32(&sfull[s]), 1);
            mbar_init(smem_u32(&sempty[s]), LT_EPI);
        }
        for (int m = 0; m < LT_MMA; ++m) mbar_init(smem_u32(drain + m), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.x);
        tma_prefetch_desc(&maps.w);
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_holder), S::kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    pdl_enter();

    const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles;
    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = l2_policy_evict_last();
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const int m0 = (int)(t % a.m_tiles) * LT_BM, n0 = (int)(t / a.m_tiles) * BN;
                for (int ks = 0; ks < l.kb; ++ks) {
                    if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, ctx, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = smem_u32(&full[stage]);
                    mbar_arrive_expect_tx(fb, S::kStage);
                    const uint32_t dst = smem_u32(smem + (size_t)stage * S::kStage);
                    tma_load_2d(dst, &maps.x, fb, ks * LT_KB, m0, pol);
                    tma_load_2d(dst + LT_BM * LT_KB, &maps.w, fb, ks * LT_KB, n0, pol);
                    if (++stage == NS) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok || *abort_flag) {   // copies in flight land before the block may end
                const uint64_t t0 = globaltimer();
                while (globaltimer() - t0 < 200000ull) __nanosleep(1000);
            }
        }
    } else if (warp == 2) {
        // A read takes 8 neighbouring blocks of 4 rows: the rows of the scale matrices are not aligned to
        // more than 4 bytes, and 32 rows at a time would touch 32 lines.  Through registers: as 4-byte
        // asynchronous copies they took 180 cycles each, 17k for the 8 blocks of a tile of 128 x 256, and
        // held up the shared memory reads of the sums on the same scheduler.
        const int kk = lane % LT_SC, r0 = lane / LT_SC;
        int ss = 0;
        uint32_t sph = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const int64_t m0 = (t % a.m_tiles) * LT_BM;
            const int n0 = (int)(t / a.m_tiles) * BN;
            for (int ks = 0; ks < l.kb; ks += LT_SC) {
                const bool in_k = ks + kk < l.kb;
                float* sd = reinterpret_cast<float*>(scales + ss * S::kScale) + kk * S::kLd + r0;
                const float* xs = l.xs + (m0 + r0) * l.kb + ks + kk;
                const float* ws = l.ws + (int64_t)(n0 + r0) * l.kb + ks + kk;
                const int step = 4 * l.kb, mx = in_k ? (int)min((int64_t)LT_BM, l.M - m0) : 0;
                const int mw = in_k ? min(BN, l.N - n0) : 0;
                if (!__all_sync(0xffffffffu, lt_wait_long(smem_u32(&sempty[ss]), sph ^ 1u, ctx, abort_flag))) {
                    ok = false;
                    break;
                }
                // A tile of 64 columns has an SM for itself and little to wait for: all reads under way at once.
                // Else 16 (4096 x 10752 x 2688: 206 us; with 8 of them 210, and with all of a slot's 208, in the
                // way of the sums' reads of shared memory).
                if constexpr (BN == 64) {
                    float vx[LT_BM / 4], vw[BN / 4];
#pragma unroll
                    for (int i = 0; i < LT_BM / 4; ++i) vx[i] = r0 + 4 * i < mx ? xs[i * step] : 0.0f;
#pragma unroll
                    for (int i = 0; i < BN / 4; ++i) vw[i] = r0 + 4 * i < mw ? ws[i * step] : 0.0f;
#pragma unroll
                    for (int i = 0; i < LT_BM / 4; ++i) sd[4 * i] = vx[i];
#pragma unroll
                    for (int i = 0; i < BN / 4; ++i) sd[LT_BM + 4 * i] = vw[i];
                } else {
                    static_assert(LT_BM % 64 == 0 && BN % 64 == 0, "whole copies");
                    auto copy = [&](float* to, const float* from, int rows) {   // 64 rows
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = r0 + 4 * i < rows ? from[i * step] : 0.0f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) to[4 * i] = v[i];
                    };
#pragma unroll
                    for (int r = 0; r < LT_BM; r += 64) copy(sd + r, xs + r / 4 * step, mx - r);
#pragma unroll
                    for (int r = 0; r < BN; r += 64) copy(sd + LT_BM + r, ws + r / 4 * step, mw - r);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sfull[ss]));
                if (++ss == LT_SS) {
                    ss = 0;
                    sph ^= 1u;
                }
            }
        }
    } else if (warp < 4) {
        if (lane == 0) {
            const uint32_t idesc = make_idesc(0u, LT_BM, BN);
            const int m = warp == 3;
            int stage = 0, ps = 0;
            uint32_t phase = 0, pph = 0;
            bool ok = true, issued = false;
            for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                for (int ks = 0; ks < l.kb; ++ks) {
                    const bool last = ks == l.kb - 1;
                    if (stage % LT_MMA == m) {
                        if (!mbar_wait(smem_u32(&full[stage]), phase, ctx, abort_flag) ||
                            !mbar_wait(smem_u32(&pempty[ps]), pph ^ 1u, ctx, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t xa = smem_u32(smem + (size_t)stage * S::kStage);
                        const uint64_t xd = sw128_desc(xa), wd = sw128_desc(xa + LT_BM * LT_KB);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)   // the block's sum: the slot is overwritten first
                            mma_ss<true>(tmem_base + (2 * ps + ks % 2) * BN, xd + 2 * kk, wd + 2 * kk, idesc,
                                         kk != 0 ? 1u : 0u);
                        issued = true;
                        mma_commit(smem_u32(&empty[stage]));
                        mma_commit(smem_u32(&pfull[ps]));
                    } else if (last && ks % 2 == 0) {   // a pair of one: nothing to add to it
                        if (!mbar_wait(smem_u32(&pempty[ps]), pph ^ 1u, ctx, abort_flag)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive(smem_u32(&pfull[ps]));
                    }
                    if (++stage == NS) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if ((ks % 2 == 1 || last) && ++ps == S::kSlots) {
                        ps = 0;
                        pph ^= 1u;
                    }
                }
            }
            if ((!ok || *abort_flag) && issued) {
                mma_commit(smem_u32(drain + m));
                mbar_wait_drain(smem_u32(drain + m), 0, ctx.timeout_ns);
            }
        }
    } else {
        const int quad = warp & 3;                        // TMEM lanes 32 quad ..
        const int c0 = (warp - 4) / 4 * S::kCols;         // columns c0 .. c0 + kCols
        constexpr int NC = S::kCols / 32;
        const int q = lane % 4, r0 = quad * 32 + lane / 4;
        const uint32_t tq = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)c0;
        int ps = 0, ss = 0;
        uint32_t pph = 0, sph = 0;
        bool ok = true;
        uint32_t v[2][16];   // the next values come while these are summed
        for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const int64_t m = (t % a.m_tiles) * LT_BM + r0;
            const int n0 = (int)(t / a.m_tiles) * BN + c0;
            uint64_t acc[4][NC * 4];   // rows r0 + 8 i, columns 8 j + 2 q and the next
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < NC * 4; ++j) acc[i][j] = 0;
            ok = lt_wait(smem_u32(&sfull[ss]), sph, ctx, abort_flag) && lt_wait(smem_u32(&pfull[ps]), pph, ctx, abort_flag);
            if (!ok) break;
            tc_fence_after();
            lt_tmem_ld(tq + 2 * ps * BN, v[0]);
            for (int ks = 0, kk = 0; ks < l.kb; ks += 2) {
                const bool two = ks + 1 < l.kb;
                // the sums of one stage, the last of its pair or not
                auto add = [&](int sub, bool end) {
                    const float* sc = reinterpret_cast<const float*>(scales + ss * S::kScale) + (kk + sub) * S::kLd;
                    const uint32_t ta = tq + (2 * ps + sub) * BN;
                    uint64_t sx[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) sx[i] = f2_pack(sc[r0 + 8 * i], sc[r0 + 8 * i]);
                    const float* sw = sc + LT_BM + c0 + 2 * q;
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        uint64_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint64_t*>(sw + c * 32 + j * 8);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {   // lanes 0 .. 15, 16 .. 31 of the quadrant
                            uint32_t(&p)[16] = v[h];
                            lt_tmem_wait(p);
                            if (h == 0) lt_tmem_ld(ta + (16u << 16) + c * 32, v[1]);
                            else if (c + 1 < NC) lt_tmem_ld(ta + (c + 1) * 32, v[0]);
                            else if (!end) lt_tmem_ld(ta + BN, v[0]);
                            else {   // the last read of the pair: free it, go on to the next
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(smem_u32(&pempty[ps]));
                                if (++ps == S::kSlots) {
                                    ps = 0;
                                    pph ^= 1u;
                                }
                                if (ks + 2 < l.kb) {
                                    ok = lt_wait(smem_u32(&pfull[ps]), pph, ctx, abort_flag);
                                    if (!ok) return;
                                    tc_fence_after();
                                    lt_tmem_ld(tq + 2 * ps * BN, v[0]);
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const uint64_t pp = f2_pack(__uint_as_float(p[4 * j + 2 * i]),
                                                                __uint_as_float(p[4 * j + 2 * i + 1]));
                                    uint64_t& s = acc[2 * h + i][4 * c + j];
                                    s = f2_fma(f2_mul(pp, w[j]), sx[2 * h + i], s);
                                }
                        }
                    }
                };
                if (two) {
                    add(0, false);
                    add(1, true);
                } else {
                    add(0, true);
                }
                if (!ok) break;
                kk += 2;
                if (kk == LT_SC || ks + 2 >= l.kb) {
                    kk = 0;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sempty[ss]));
                    if (++ss == LT_SS) {
                        ss = 0;
                        sph ^= 1u;
                    }
                    if (ks + 2 < l.kb) {
                        ok = lt_wait(smem_u32(&sfull[ss]), sph, ctx, abort_flag);
                        if (!ok) break;
                    }
                }
            }
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float lo, hi;
                        f2_unpack(acc[i][4 * c + j], lo, hi);
                        const __nv_bfloat162 b = __floats2bfloat162_rn(lin_act(lo, l.relu2), lin_act(hi, l.relu2));
                        w[j] = *reinterpret_cast<const uint32_t*>(&b);
                    }
                    lt_transpose(w, q);   // now 8 columns in a row, a quad 64 bytes
                    const int n = n0 + c * 32 + q * 8;
                    if (m + 8 * i < l.M && n < l.N)   // N is a multiple of 16
                        *reinterpret_cast<uint4*>(l.out + (m + 8 * i) * l.N + n) = make_uint4(w[0], w[1], w[2], w[3]);
                }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, S::kTmem);
    }
}

// ----------------------------------------------------------------------------- host

typedef CUresult (*FwEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static FwEncodeFn fw_encode_fn() {
    static const FwEncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<FwEncodeFn>(p) : nullptr;
    }();
    return fn;
}

bool fw_map(CUtensorMap* m, const void* base, int64_t rows, int64_t bytes, int64_t ld, int chunk, int box_rows) {
    const FwEncodeFn fn = fw_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)bytes / 4, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {(cuuint32_t)chunk / 4, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MT, int TT>
static cudaError_t launch_linear_few(LinearFewArgs& a, int num_sms, const DevCtx& ctx, cudaStream_t stream) {
    LinearFewMaps maps = {};
    for (int i = 0; i < 2 && a.share.rows > i; ++i)
        if (!fw_map(&maps.w[i], a.l.wq, a.l.N, a.l.Kp, a.l.Kp, FW_CHUNK, a.share.rows - i)) return cudaErrorInvalidValue;
    const size_t fixed = FwRed::bytes(a.share.units) + FwRings::kBarBytes + 8 + 16;
    a.n_stages = (int)std::min<size_t>(FW_MAX_STAGES, (kMaxSmem - fixed) / FW_WARPS / a.slot_bytes);
    const size_t smem = (size_t)FW_WARPS * a.n_stages * a.slot_bytes + fixed;
    auto k = linear_few_kernel<MT, TT>;
    cudaError_t e = allow_smem(k);
    if (e != cudaSuccess) return e;
    return launch_k(k, dim3(num_sms), dim3(FW_THREADS), smem, stream, maps, a, ctx);
}

template <int BN>
static cudaError_t launch_linear_tiles(const LinearArgs& l, int num_sms, const DevCtx& ctx, cudaStream_t stream) {
    using S = LtShape<BN>;
    LinearMaps maps;
    if (!make_map_u8_b128(&maps.x, l.xq, l.M, l.Kp, LT_BM) || !make_map_u8_b128(&maps.w, l.wq, l.N, l.Kp, BN))
        return cudaErrorInvalidValue;
    LinearTileArgs a = {};
    a.l = l;
    a.m_tiles = (int)((l.M + LT_BM - 1) / LT_BM);
    a.n_tiles = (l.N + BN - 1) / BN;
    const size_t fixed = 1024 + LT_SS * S::kScale + (2 * LT_MAX_STAGES + 2 * S::kSlots + 2 * LT_SS + LT_MMA) * 8 + 16;
    a.n_stages = (int)std::min<size_t>(LT_MAX_STAGES, (kMaxSmem - fixed) / S::kStage);
    a.n_stages -= a.n_stages % LT_MMA;   // each slot has one issuer
    const size_t smem = (size_t)a.n_stages * S::kStage + fixed;
    auto k = linear_tile_kernel<BN>;
    cudaError_t e = allow_smem(k);
    if (e != cudaSuccess) return e;
    const int64_t grid = std::min<int64_t>((int64_t)a.m_tiles * a.n_tiles, num_sms);
    return launch_k(k, dim3((unsigned)grid), dim3(LT_THREADS), smem, stream, maps, a, ctx);
}

static cudaError_t launch_linear(const LinearArgs& l, int num_sms, const DevCtx& ctx, cudaStream_t stream) {
    if (l.M <= kFewMaxTokens) {
        LinearFewArgs a = {};
        a.l = l;
        a.chunks = (l.Kp + FW_CHUNK - 1) / FW_CHUNK;
        a.share = fw_share(l.N, num_sms);
        a.slot_bytes = (a.share.rows * FW_CHUNK + 127) / 128 * 128;
        // as many matrix tiles as there are rows for: 1856 weight rows (13 per SM) of 2688 against one row of x
        // in 3.9 us with one, 4.2 with two; two tiles of x for one of M <= 8 would double the instructions
        if (a.share.rows <= 16)
            return l.M <= 8 ? launch_linear_few<1, 1>(a, num_sms, ctx, stream)
                            : launch_linear_few<1, 2>(a, num_sms, ctx, stream);
        return l.M <= 8 ? launch_linear_few<2, 1>(a, num_sms, ctx, stream)
                        : launch_linear_few<2, 2>(a, num_sms, ctx, stream);
    }
    // 64 columns while every tile has an SM of its own, else 128 (us, 64 against 128 columns):
    //   tiles of 64     42: 64 x 2688 x 1856   8.5, 10.6      84: 256 x 2688 x 1856   8.8, 11.2
    //                  145: 577 x 1856 x 2688 10.6, 13.7     168: 64 x 10752 x 2688  18.1, 14.3
    //                  336: 1024 x 2688 x 1856 19.5, 19.1    672: 2048 x 2688 x 1856 30.5, 26.9
    // (32 columns: 8.9 at 64 x 2688 x 1856, 12.9 at 256.)
    const int64_t mt = (l.M + LT_BM - 1) / LT_BM;
    if (mt * ((l.N + 63) / 64) <= num_sms) return launch_linear_tiles<64>(l, num_sms, ctx, stream);
    return launch_linear_tiles<128>(l, num_sms, ctx, stream);
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_linear_fp8_b128(int64_t M, int32_t N, int32_t K, const uint8_t* x_codes, const float* x_scales,
                               const uint8_t* w_codes, const float* w_scales, int32_t act, void* out, void* stream) {
    if (M < 0 || M >= ((int64_t)1 << 31) - 128 || N < 16 || N > (1 << 20) || N % 16 != 0 || K < 16 || K > 65536 ||
        K % 16 != 0)
        return MOE_EINVAL;
    if (act != MOE_ACT_NONE && act != MOE_ACT_RELU2) return MOE_EINVAL;
    if (M == 0) return MOE_OK;
    auto al = [](const void* p, uintptr_t n) { return p && reinterpret_cast<uintptr_t>(p) % n == 0; };
    if (!al(x_codes, 16) || !al(w_codes, 16) || !al(out, 16) || !al(x_scales, 4) || !al(w_scales, 4))
        return MOE_EINVAL;
    const int64_t kb = (K + 127) / 128, out_bytes = M * N * 2;
    if (overlap(out, out_bytes, x_codes, M * kb * 128) || overlap(out, out_bytes, x_scales, M * kb * 4) ||
        overlap(out, out_bytes, w_codes, N * kb * 128) || overlap(out, out_bytes, w_scales, N * kb * 4))
        return MOE_EINVAL;
    DevCtx ctx;
    int sms = 0;
    const moe_status s = internal_device(&ctx, &sms);
    if (s != MOE_OK) return s;
    LinearArgs l = {};
    l.xq = x_codes;
    l.xs = x_scales;
    l.wq = w_codes;
    l.ws = w_scales;
    l.out = static_cast<uint16_t*>(out);
    l.M = M;
    l.N = N;
    l.kb = (K + 127) / 128;
    l.Kp = l.kb * 128;
    l.relu2 = act == MOE_ACT_RELU2;
    return launch_linear(l, sms, ctx, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ECUDA;
}

}  // extern "C"
