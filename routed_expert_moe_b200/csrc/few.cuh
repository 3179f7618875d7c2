// Weight streaming for a few tokens: the parts that the few-token layer
// (few.cu) and the few-row dense product (linear_b128.cu) share.
//
// A weight row is read once from HBM and meets at most 16 activation rows, so
// the work is a stream: 2 * 16 operations per weight at most, far below what
// the tensor cores take at HBM's rate.  Each of a CTA's eight consumer warps
// has a ring in shared memory of its own.  A lane of one of four producer
// warps fills it (one TMA box, 16 to 24 rows of a chunk of K, per stage; with
// one producer warp the issue of the boxes bounds the stream).  A consumer
// fetches the activations that go with its next stage into registers, waits
// for the weights, multiplies with warp-level matrix instructions (weights as
// the 16-row operand, tokens as the 8-column one) and hands the slot back.  No consumer waits for another within a stream.  tcgen05 would need
// 128 weight rows per instruction; boxes of 16 to 24 rows let every SM stream
// the same number of bytes.
//
// Copying row by row instead (untiled bulk copies) costs a fixed 32 cycles of
// an SM's copy engine per row: 4.6 TB/s at 512 bytes per row, against 7.0 with
// boxes.  Consumers that fill their rings themselves spend 500 cycles a stage
// on it.
//
// Lane (g, q) = (lane / 4, lane % 4) of a warp reads 16 bytes at
// 64 * segment + 16 * q of weight rows 16 m + g and 16 m + g + 8 and of token
// g's activations: the matrix instruction's K index is assigned to those bytes
// in the same order on both sides, so no value moves between lanes.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int FW_WARPS = 8;                   // consumer warps
constexpr int FW_PROD = 4;                    // producer warps: one issues a box every 220 cycles at best
constexpr int FW_THREADS = 32 * (FW_WARPS + FW_PROD);
constexpr int FW_SEG = 64;                    // bytes of a row that one matrix step takes
constexpr int FW_ROWS = 24;                   // weight rows per stage at most
constexpr int FW_MAX_STAGES = 6;              // of one warp's ring
constexpr int FW_SMEM = 227 * 1024;           // shared memory a block may use

// Segments per stage.  Seven: an odd number puts the rows of a stage, 448 bytes apart, into
// alternating halves of the banks.  Formats with a scale per 128 bytes take whole blocks.
constexpr int fw_segs(bool block) { return block ? 6 : 7; }

// Registers: a block of 12 warps starts with 168 per thread.  The consumers' operands need more, the
// producers' few: 8 warps x 32 x 216 + 4 x 32 x 64 = 63488 of the 64512 that the block holds.
__device__ __forceinline__ void fw_consumer_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 216;"); }
__device__ __forceinline__ void fw_producer_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 64;"); }
static_assert(FW_WARPS % 4 == 0 && FW_PROD % 4 == 0, "whole warpgroups");
static_assert(32 * (FW_WARPS * 216 + FW_PROD * 64) <= 32 * (FW_WARPS + FW_PROD) * 168, "registers of the block");

// How a weight row of `bytes` bytes is cut into chunks (the last one may reach past the row: zeros).
struct FwCut {
    int bytes;    // of a row
    int chunk;    // bytes per stage
    int n;        // chunks per row
};
inline FwCut fw_cut(int bytes, bool block) {
    FwCut c;
    c.bytes = bytes;
    c.chunk = fw_segs(block) * FW_SEG;
    c.n = (bytes + c.chunk - 1) / c.chunk;
    return c;
}

// D (16 weight rows x 8 tokens, fp32) += A (16 x 16 values) * B (8 x 16 values), bf16 or fp16 operands
// (volatile: it must stay where the whole warp is converged).  E4M3 operands are converted to fp16,
// which holds them exactly: the warp-level E4M3 instruction takes 24 cycles of a scheduler here,
// against 8 for the fp16 one.
template <bool BF16>
__device__ __forceinline__ void fw_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four E4M3 codes as two pairs of fp16 values.
__device__ __forceinline__ void fw_half4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}

// The rings' barriers and slots in shared memory, [warp][slot].
struct FwRings {
    uint8_t* base;
    uint64_t* full;      // one arrival (the producer's) and the box's bytes
    uint64_t* empty;     // one arrival (the consumer's)
    int slot_bytes, n;

    static constexpr size_t kBarBytes = 2 * FW_WARPS * FW_MAX_STAGES * sizeof(uint64_t);
    __device__ __forceinline__ void init() const {   // one thread
        for (int i = 0; i < FW_WARPS * FW_MAX_STAGES; ++i) {
            mbar_init(smem_u32(full + i), 1);
            mbar_init(smem_u32(empty + i), 1);
        }
    }
};

// Consumer side of ring `warp`.
struct FwTake {
    const uint8_t* base;
    uint32_t full, empty;
    int slot_bytes, n, slot;
    uint32_t parity;

    __device__ __forceinline__ FwTake(const FwRings& r, int warp)
        : base(r.base + (size_t)warp * r.n * r.slot_bytes),
          full(smem_u32(r.full + warp * FW_MAX_STAGES)),
          empty(smem_u32(r.empty + warp * FW_MAX_STAGES)),
          slot_bytes(r.slot_bytes),
          n(r.n),
          slot(0),
          parity(0) {}
    // Waits for the next slot.  Every lane looks at the barrier, so that data that is there already
    // costs one look.
    __device__ __forceinline__ bool wait(const DevCtx& ctx, volatile int* abort) {
        const uint32_t bar = full + 8 * slot;
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        return mbar_wait_warp(bar, parity, ctx, abort) && __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
    }
    __device__ __forceinline__ const uint8_t* data() const { return base + slot * slot_bytes; }
    // Every lane has read the slot: hands it back.
    __device__ __forceinline__ void release() {
        __syncwarp();
        if (threadIdx.x % 32 == 0) mbar_arrive(empty + 8 * slot);
        if (++slot == n) {
            slot = 0;
            parity ^= 1u;
        }
    }
};

// Producer side of one ring: one lane of a producer warp each.
struct FwPut {
    uint8_t* base;
    uint32_t full, empty;
    int slot_bytes, n, slot;
    uint32_t parity;

    __device__ __forceinline__ FwPut(const FwRings& r, int warp)
        : base(r.base + (size_t)warp * r.n * r.slot_bytes),
          full(smem_u32(r.full + warp * FW_MAX_STAGES)),
          empty(smem_u32(r.empty + warp * FW_MAX_STAGES)),
          slot_bytes(r.slot_bytes),
          n(r.n),
          slot(0),
          parity(1) {}
    __device__ __forceinline__ bool ready() const {   // no wait
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(empty + 8 * slot), "r"(parity)
            : "memory");
        return ok != 0;
    }
    __device__ __forceinline__ void next() {
        if (++slot == n) {
            slot = 0;
            parity ^= 1u;
        }
    }
    // Starts the copy of a box of `bytes` bytes at byte x of row y into the next slot.
    __device__ __forceinline__ void fill(const CUtensorMap* map, int x, int y, uint32_t bytes, uint64_t policy) {
        const uint32_t bar = full + 8 * slot;
        mbar_arrive_expect_tx(bar, bytes);
        tma_load_2d(smem_u32(base) + slot * slot_bytes, map, bar, x / 4, y, policy);
        next();
    }
    // Hands over an empty slot (the consumer looks at what stands beside it).
    __device__ __forceinline__ void mark() {
        mbar_arrive(full + 8 * slot);
        next();
    }
};

// A producer warp's ring, by lane: those of lanes 0 and 1.
__device__ __forceinline__ int fw_put_ring() { return threadIdx.x / 32 - FW_WARPS + FW_PROD * (threadIdx.x % 32); }
__device__ __forceinline__ bool fw_put_lane() { return threadIdx.x % 32 < FW_WARPS / FW_PROD; }

// A producer warp's loop: step() fills one stage of this lane's ring, false once there is none left.
// A lane looks for a free slot without waiting, so that one slow ring does not hold up the others.
// Ends (false) when no ring made progress for the time limit or a consumer gave up.
template <typename Step>
__device__ __forceinline__ bool fw_produce(FwPut& put, bool active, const Step& step, const DevCtx& ctx,
                                           volatile int* abort) {
    uint64_t t0 = globaltimer();
    uint32_t idle = 0;
    while (__any_sync(0xffffffffu, active)) {
        bool moved = false;
        if (active && put.ready()) {
            active = step();
            moved = true;
        }
        if (__any_sync(0xffffffffu, moved)) {
            idle = 0;
            continue;
        }
        if ((++idle & 63u) == 0) {
            if (idle == 64) t0 = globaltimer();
            bool stop = *abort != 0;
            if (globaltimer() - t0 > ctx.timeout_ns) {
                record_error(ctx.err, MOE_ETIMEOUT);
                *abort = 1;
                stop = true;
            }
            if (__any_sync(0xffffffffu, stop)) return false;
        }
    }
    return true;
}

// How a stream's operands are held: weights in bf16 (activations too), or in E4M3 with activations as
// E4M3 codes or as fp16 values; BLOCK: a scale per 128 weights of a row, BLOCK_ACT: of the activations.
template <bool BF16_, bool CODES_, bool BLOCK_, bool BLOCK_ACT_>
struct FwFmt {
    static constexpr bool BF16 = BF16_, CODES = CODES_, BLOCK = BLOCK_, BLOCK_ACT = BLOCK_ACT_;
    static constexpr int SEGS = fw_segs(BLOCK);
    static constexpr int AB = BF16 || CODES ? 16 : 32;   // bytes of activations that go with 16 of weights
    static constexpr int AV = AB / 16;                   // loads for them
};

// What goes with the weights of N segments, in registers: the activations of this lane's NT columns
// (g + 8 nt), the scales of weight row `lane` and of column `lane`, handed round by shuffles.  A stage's
// first batch is fetched while the warp still waits for its weights.
template <typename F, int N, int NT>
struct FwActs {
    static constexpr int KB = F::BLOCK ? N / 2 : 1;
    static_assert(!F::BLOCK || N % 2 == 0, "whole blocks");
    uint4 x[N][NT][F::AV];
    float ws[KB];
    float xs[F::BLOCK_ACT ? KB : 1];
};

// Where they come from: from the start of a K row on (activations: this lane's first bytes).  A column
// without a token, like a row past the tile, repeats another one and is not used.
template <int NT>
struct FwSide {
    const uint8_t* act[NT];
    const float* ws;        // of weight row `lane`
    const float* xs;        // of column `lane`
};

// The batch from weight byte c0 on; the activation rows go with row_bytes weight bytes (zeros past
// them; weights may be padded).
template <typename F, int N, int NT>
__device__ __forceinline__ void fw_fetch(FwActs<F, N, NT>& v, const FwSide<NT>& side, int c0, int row_bytes) {
    const int q16 = (threadIdx.x % 4) * 16;
    const bool full = c0 + N * FW_SEG <= row_bytes;
    if (full) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint8_t* p = side.act[t] + c0 * F::AV;
#pragma unroll
            for (int s = 0; s < N; ++s)
#pragma unroll
                for (int j = 0; j < F::AV; ++j)
                    v.x[s][t][j] = *reinterpret_cast<const uint4*>(p + s * FW_SEG * F::AV + j * 16);
        }
    } else {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint8_t* p = side.act[t] + c0 * F::AV;
#pragma unroll
            for (int s = 0; s < N; ++s)
#pragma unroll
                for (int j = 0; j < F::AV; ++j) {
                    v.x[s][t][j] = make_uint4(0, 0, 0, 0);
                    if (c0 + s * FW_SEG + q16 < row_bytes)
                        v.x[s][t][j] = *reinterpret_cast<const uint4*>(p + s * FW_SEG * F::AV + j * 16);
                }
        }
    }
    if constexpr (F::BLOCK) {
#pragma unroll
        for (int b = 0; b < FwActs<F, N, NT>::KB; ++b) {
            const bool in = full || c0 + b * 128 < row_bytes;
            v.ws[b] = in ? __ldg(side.ws + c0 / 128 + b) : 0.0f;
            if constexpr (F::BLOCK_ACT) v.xs[b] = in ? __ldg(side.xs + c0 / 128 + b) : 0.0f;
        }
    }
}

// The running sums of 16 MT weight rows x 8 NT columns.  j: weight row 16 mt + g + 8 * (j / 2), column
// 8 nt + 2 q + j % 2.  A matrix instruction takes 21 cycles and a scheduler starts one every 8, so
// small tiles keep two chains of sums.
template <int MT, int NT>
struct FwAcc {
    static constexpr int kChains = MT * NT >= 4 ? 1 : 2;
    float d[kChains][MT][NT][4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int c = 0; c < kChains; ++c)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) d[c][mt][nt][j] = 0.0f;
    }
    __device__ __forceinline__ float sum(int mt, int nt, int j) const {
        return kChains == 1 ? d[0][mt][nt][j] : d[0][mt][nt][j] + d[kChains - 1][mt][nt][j];
    }
};

// 4 bytes (step j of 4) of weights of rows g (w0) and g + 8 (w1) of every tile times the activations that
// go with them: a quarter of 16 bytes of E4M3, or (even j) half of 16 bytes of bf16.
template <typename F, int MT, int NT>
__device__ __forceinline__ void fw_step(float (&d)[MT][NT][4], const uint4 (&x)[NT][F::AV], const uint4 (&w0)[MT],
                                        const uint4 (&w1)[MT], int j) {
    if constexpr (F::BF16) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint4 u = w0[mt], v = w1[mt], b = x[nt][0];
                if (j == 0) fw_mma<true>(d[mt][nt], u.x, v.x, u.y, v.y, b.x, b.y);
                if (j == 2) fw_mma<true>(d[mt][nt], u.z, v.z, u.w, v.w, b.z, b.w);
            }
    } else {
        uint32_t b[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint4 c = x[nt][F::CODES ? 0 : j / 2];
            if constexpr (F::CODES) {
                fw_half4(j == 0 ? c.x : j == 1 ? c.y : j == 2 ? c.z : c.w, b[nt][0], b[nt][1]);
            } else {
                b[nt][0] = j % 2 == 0 ? c.x : c.z;
                b[nt][1] = j % 2 == 0 ? c.y : c.w;
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const uint4 u = w0[mt], v = w1[mt];
            uint32_t a0, a1, a2, a3;
            fw_half4(j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w, a0, a2);
            fw_half4(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w, a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) fw_mma<false>(d[mt][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
        }
    }
}

// A batch of N segments from byte b of the slot's rows: `rows` weight rows (at most 16 MT) times the
// activations.
template <typename F, int N, int MT, int NT>
__device__ __forceinline__ void fw_mul(FwAcc<MT, NT>& acc, const uint8_t* slot, int b, int rows, const FwActs<F, N, NT>& v) {
    constexpr int C = FwAcc<MT, NT>::kChains;
    const int lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
    const uint8_t *r0[MT], *r1[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {   // rows past the last repeat it: their results are not used
        r0[mt] = slot + min(mt * 16 + g, rows - 1) * (F::SEGS * FW_SEG) + b + q * 16;
        r1[mt] = slot + min(mt * 16 + g + 8, rows - 1) * (F::SEGS * FW_SEG) + b + q * 16;
    }
    float part[C][MT][NT][4];
#pragma unroll
    for (int s = 0; s < N; ++s) {
        uint4 w0[MT], w1[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            w0[mt] = *reinterpret_cast<const uint4*>(r0[mt] + s * FW_SEG);
            w1[mt] = *reinterpret_cast<const uint4*>(r1[mt] + s * FW_SEG);
        }
        if constexpr (F::BLOCK) {
            if (s % 2 == 0) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 4; ++j) part[c][mt][nt][j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) fw_step<F, MT, NT>(part[j % C], v.x[s], w0, w1, j);
            if (s % 2 == 1) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const float s0 = __shfl_sync(0xffffffffu, v.ws[s / 2], mt * 16 + g);
                    const float s1 = __shfl_sync(0xffffffffu, v.ws[s / 2], mt * 16 + g + 8);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float x0 = 1.0f, x1 = 1.0f;
                        if constexpr (F::BLOCK_ACT) {
                            x0 = __shfl_sync(0xffffffffu, v.xs[s / 2], nt * 8 + 2 * q);
                            x1 = __shfl_sync(0xffffffffu, v.xs[s / 2], nt * 8 + 2 * q + 1);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float sc = j / 2 ? s1 : s0;
                            if constexpr (F::BLOCK_ACT) sc *= j % 2 ? x1 : x0;
                            float p = part[0][mt][nt][j];
                            if constexpr (C == 2) p += part[C - 1][mt][nt][j];
                            acc.d[0][mt][nt][j] = __fmaf_rn(sc, p, acc.d[0][mt][nt][j]);
                        }
                    }
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; j += F::BF16 ? 2 : 1)
                fw_step<F, MT, NT>(acc.d[(F::BF16 ? j / 2 : j) % C], v.x[s], w0, w1, j);
        }
    }
}

// The other way round, for bf16 activations that come in two parts: 16 rows of activations (two sets of
// eight, FwActs' columns) times 8 NT weight rows.  The low parts ride in the operand's second half, and
// the 17 to 24 weight rows of a unit are three tiles of eight instead of two of 16: six instructions a
// segment against eight (layer of 16 tokens: 241 against 283 us).
template <int NT>
struct FwAccT {
    float d[2][NT][4];   // j: activation row g (+ 8 * (j / 2)), weight row 8 nt + 2 q + j % 2
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) d[0][nt][j] = d[1][nt][j] = 0.0f;
    }
    __device__ __forceinline__ float sum(int nt, int j) const { return d[0][nt][j] + d[1][nt][j]; }
};
template <typename F, int N, int NT>
__device__ __forceinline__ void fw_mul_t(FwAccT<NT>& acc, const uint8_t* slot, int rows, const FwActs<F, N, 2>& v) {
    static_assert(F::BF16, "bf16 in two parts");
    const int lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        if (nt * 8 >= rows) break;
        // rows past the last repeat it: their results are not used
        const uint8_t* r = slot + min(nt * 8 + g, rows - 1) * (F::SEGS * FW_SEG) + q * 16;
#pragma unroll
        for (int s = 0; s < N; ++s) {
            const uint4 a = v.x[s][0][0], b = v.x[s][1][0], w = *reinterpret_cast<const uint4*>(r + s * FW_SEG);
            fw_mma<true>(acc.d[0][nt], a.x, b.x, a.y, b.y, w.x, w.y);
            fw_mma<true>(acc.d[1][nt], a.z, b.z, a.w, b.w, w.z, w.w);
        }
    }
}

// Segments fetched together (registers: two columns of fp16 take twice the room of one).
template <typename F, int NT>
constexpr int fw_batch() {
    return NT == 2 && F::AV == 2 ? (F::BLOCK ? 2 : 1) : F::SEGS;
}
// A whole stage, whose first batch has been fetched.
template <typename F, int MT, int NT>
__device__ __forceinline__ void fw_mul_stage(FwAcc<MT, NT>& acc, const uint8_t* slot, int rows, int c0, int row_bytes,
                                             const FwSide<NT>& side, FwActs<F, fw_batch<F, NT>(), NT>& v) {
    constexpr int N = fw_batch<F, NT>();
    static_assert(F::SEGS % N == 0, "whole batches");
    fw_mul(acc, slot, 0, rows, v);
#pragma unroll 1
    for (int s = N; s < F::SEGS; s += N) {
        fw_fetch(v, side, c0 + s * FW_SEG, row_bytes);
        fw_mul(acc, slot, s * FW_SEG, rows, v);
    }
}

// The pairs (list entry i, chunk k) of a stream that fall to warp w.  The chunks rotate over the warps
// from one expert to the next, so that a short last chunk does not always fall to the same warp; the
// rotation goes by the expert's number, so that a token's sums do not hang on the experts that others
// brought into the list.
struct FwPairs {
    int i, k;
    __device__ __forceinline__ void seek(const int* list, int n_list, int n_chunks, int w) {
        for (; i < n_list; ++i) {
            k = (w - list[i] * (n_chunks | 1)) & (FW_WARPS - 1);
            if (k < n_chunks) return;
        }
    }
    __device__ __forceinline__ void step(const int* list, int n_list, int n_chunks, int w) {
        k += FW_WARPS;
        if (k < n_chunks) return;
        ++i;
        seek(list, n_list, n_chunks, w);
    }
};

// The warps' partial sums of one unit, [warp][token][row], and their exchange.  Two buffers take
// turns (one is enough for a single unit), so that one barrier per unit (bounded: every warp arrives,
// then waits for all) orders both the reads after the writes and the next unit's writes after the reads.
struct FwRed {
    static constexpr int kWarp = 16 * FW_ROWS;
    static constexpr int kFloats = FW_WARPS * kWarp;
    static constexpr size_t bytes(int units) { return (units > 1 ? 2 : 1) * kFloats * sizeof(float); }
    float* buf;          // [2][kFloats], or [1] for a single unit
    uint32_t bar;        // mbarrier of FW_WARPS arrivals
    int turn;

    __device__ __forceinline__ float* mine(int warp) const { return buf + (turn & 1) * kFloats + warp * kWarp; }
    __device__ __forceinline__ bool exchange(const DevCtx& ctx, volatile int* abort) {
        __syncwarp();
        if (threadIdx.x % 32 == 0) mbar_arrive(bar);
        const bool ok = mbar_wait_warp(bar, turn & 1, ctx, abort);
        ++turn;
        return ok;
    }
    // after exchange(): element (token, row) over the warps, in order
    __device__ __forceinline__ float sum(int token, int row) const {
        const float* b = buf + ((turn & 1) ^ 1) * kFloats + token * FW_ROWS + row;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < FW_WARPS; ++w) s += b[w * kWarp];
        return s;
    }
};

// Copies in flight land before the block may end (after a wait has given up).
__device__ __forceinline__ void fw_settle() {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) __nanosleep(1000);
}

// How n output rows are shared: units of `rows` or `rows` - 1 rows, so many per CTA; a unit's warps
// split K.
struct FwShare {
    int units;     // per CTA
    int rows;      // per unit at most
};
inline FwShare fw_share(int n, int num_sms) {
    FwShare s;
    const int share = (n + num_sms - 1) / num_sms;
    s.units = (share + FW_ROWS - 1) / FW_ROWS;
    s.rows = (share + s.units - 1) / s.units;
    return s;
}

// Map of a row-major matrix of rows of `bytes` bytes, `ld` bytes apart, box `chunk` bytes x box_rows
// rows (no swizzle; 4-byte elements, so that a box row may hold up to 1 KB).
bool fw_map(CUtensorMap* m, const void* base, int64_t rows, int64_t bytes, int64_t ld, int chunk, int box_rows);

}  // namespace moe
