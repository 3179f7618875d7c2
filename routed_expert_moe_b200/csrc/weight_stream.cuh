// Weight streaming for a few rows: the parts of the FP8_B128 product of at most
// 16 rows (linear_b128.cu).
//
// A weight row is read once from HBM and meets at most 16 activation rows, so
// the work is a stream.  Each of a CTA's eight consumer warps has a ring in
// shared memory of its own.  A lane of one of four producer warps fills it
// (one TMA box, up to 24 rows of a chunk of K, per stage; with one producer
// warp the issue of the boxes bounds the stream).  A consumer fetches the
// activations that go with its next stage into registers, waits for the
// weights, multiplies with warp-level matrix instructions (weights as the
// 16-row operand, tokens as the 8-column one) and hands the slot back.  No
// consumer waits for another within a stream.  tcgen05 would need 128 weight
// rows per instruction, 15 units for 1856 rows; boxes of as many rows as an SM's
// share (13 of 1856; several units of at most 24 beyond that) let every SM
// stream the same number of bytes.
//
// Copying row by row instead (untiled bulk copies) costs a fixed 32 cycles of
// an SM's copy engine per row: 4.6 TB/s at 512 bytes per row, against 7.0 with
// boxes.  Consumers that fill their rings themselves spend 500 cycles a stage
// on it.
//
// Device times, launch included: 1856 rows of 2688 in 3.9 us for one token,
// 5.1 for 16; 10752 rows of 2688 in 12.3 for eight (2.4 TB/s), where a CTA has
// four units one after the other and each converts its codes to fp16 (fetching
// the next unit's activations before the warps' sums are joined: 13.0).
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

// Segments per stage: whole blocks of 128, one scale each.  Six, chunks of 384 bytes, are seven chunks of a
// row of 2688 and five of 1920, one for each warp at most; where they are nine or more, some warps work twice
// while others wait, and eight segments are a little faster (us, for 4 / 6 / 8 segments; M x N x K):
//   1 x 1856 x 2688  4.1 / 3.9 / 4.0     16 x 1856 x 2688  4.7 / 4.5 / 4.7     8 x 10752 x 2688  14.3 / 12.4 / 13.0
//   1 x 2688 x 1920  4.0 / 4.0 / 4.2      1 x 1856 x 3200  4.3 / 4.4 / 4.2      8 x 5376 x 3200   8.5 /  8.9 /  8.3
//   1 x 1856 x 4096  4.6 / 4.8 / 4.4
constexpr int FW_SEGS = 6;
constexpr int FW_CHUNK = FW_SEGS * FW_SEG;    // bytes of a row per stage

// Registers: a block of 12 warps starts with 168 per thread.  The consumers' operands need more, the
// producers' few: 8 warps x 32 x 216 + 4 x 32 x 64 = 63488 of the 64512 that the block holds.
__device__ __forceinline__ void fw_consumer_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 216;"); }
__device__ __forceinline__ void fw_producer_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 64;"); }
static_assert(FW_WARPS % 4 == 0 && FW_PROD % 4 == 0, "whole warpgroups");
static_assert(32 * (FW_WARPS * 216 + FW_PROD * 64) <= 32 * (FW_WARPS + FW_PROD) * 168, "registers of the block");

// D (16 weight rows x 8 tokens, fp32) += A (16 x 16 values) * B (8 x 16 values) (volatile: it must stay
// where the whole warp is converged).  The E4M3 operands are converted to fp16, which holds them exactly:
// the warp-level E4M3 instruction takes 24 cycles of a scheduler here, against 8 for the fp16 one.
__device__ __forceinline__ void fw_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
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

// What goes with the weights of a stage, in registers: the activations of this lane's NT columns
// (g + 8 nt), the scales of weight row `lane` and of column `lane`, handed round by shuffles.  They are
// fetched while the warp still waits for its weights.
template <int NT>
struct FwActs {
    static constexpr int KB = FW_SEGS / 2;
    uint4 x[FW_SEGS][NT];
    float ws[KB], xs[KB];
};

// Where they come from: from the start of a K row on (activations: this lane's first bytes).  A column
// without a token, like a row past the tile, repeats another one and is not used.
template <int NT>
struct FwSide {
    const uint8_t* act[NT];
    const float* ws;        // of weight row `lane`
    const float* xs;        // of column `lane`
};

// Those of byte c0 on, zeros past the row's row_bytes.
template <int NT>
__device__ __forceinline__ void fw_fetch(FwActs<NT>& v, const FwSide<NT>& side, int c0, int row_bytes) {
    const int q16 = (threadIdx.x % 4) * 16;
    const bool full = c0 + FW_CHUNK <= row_bytes;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const uint8_t* p = side.act[t] + c0;
        if (full) {
#pragma unroll
            for (int s = 0; s < FW_SEGS; ++s) v.x[s][t] = *reinterpret_cast<const uint4*>(p + s * FW_SEG);
        } else {
#pragma unroll
            for (int s = 0; s < FW_SEGS; ++s) {
                v.x[s][t] = make_uint4(0, 0, 0, 0);
                if (c0 + s * FW_SEG + q16 < row_bytes) v.x[s][t] = *reinterpret_cast<const uint4*>(p + s * FW_SEG);
            }
        }
    }
#pragma unroll
    for (int b = 0; b < FwActs<NT>::KB; ++b) {
        const bool in = full || c0 + b * 128 < row_bytes;
        v.ws[b] = in ? side.ws[c0 / 128 + b] : 0.0f;
        v.xs[b] = in ? side.xs[c0 / 128 + b] : 0.0f;
    }
}

// The running sums of 16 MT weight rows x 8 NT columns.  j: weight row 16 mt + g + 8 * (j / 2), column
// 8 nt + 2 q + j % 2.  A matrix instruction takes 21 cycles and a scheduler starts one every 8, so small
// tiles sum a block in two chains.
template <int MT, int NT>
struct FwAcc {
    static constexpr int kChains = MT * NT >= 4 ? 1 : 2;
    float d[MT][NT][4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) d[mt][nt][j] = 0.0f;
    }
};

// 4 bytes (step j of 4) of weights of rows g (w0) and g + 8 (w1) of every tile times the activations that
// go with them.
template <int MT, int NT>
__device__ __forceinline__ void fw_step(float (&d)[MT][NT][4], const uint4 (&x)[NT], const uint4 (&w0)[MT],
                                        const uint4 (&w1)[MT], int j) {
    auto word = [j](const uint4& c) { return j == 0 ? c.x : j == 1 ? c.y : j == 2 ? c.z : c.w; };
    uint32_t b[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) fw_half4(word(x[nt]), b[nt][0], b[nt][1]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        uint32_t a0, a1, a2, a3;
        fw_half4(word(w0[mt]), a0, a2);
        fw_half4(word(w1[mt]), a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) fw_mma(d[mt][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
    }
}

// A stage: `rows` weight rows (at most 16 MT) times the activations.
template <int MT, int NT>
__device__ __forceinline__ void fw_mul(FwAcc<MT, NT>& acc, const uint8_t* slot, int rows, const FwActs<NT>& v) {
    constexpr int C = FwAcc<MT, NT>::kChains;
    const int lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
    const uint8_t *r0[MT], *r1[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {   // rows past the last repeat it: their results are not used
        r0[mt] = slot + min(mt * 16 + g, rows - 1) * FW_CHUNK + q * 16;
        r1[mt] = slot + min(mt * 16 + g + 8, rows - 1) * FW_CHUNK + q * 16;
    }
#pragma unroll
    for (int b = 0; b < FW_SEGS / 2; ++b) {
        float part[C][MT][NT][4];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) part[c][mt][nt][j] = 0.0f;
#pragma unroll
        for (int s = 2 * b; s < 2 * b + 2; ++s) {
            uint4 w0[MT], w1[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                w0[mt] = *reinterpret_cast<const uint4*>(r0[mt] + s * FW_SEG);
                w1[mt] = *reinterpret_cast<const uint4*>(r1[mt] + s * FW_SEG);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) fw_step<MT, NT>(part[j % C], v.x[s], w0, w1, j);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const float s0 = __shfl_sync(0xffffffffu, v.ws[b], mt * 16 + g);
            const float s1 = __shfl_sync(0xffffffffu, v.ws[b], mt * 16 + g + 8);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float x0 = __shfl_sync(0xffffffffu, v.xs[b], nt * 8 + 2 * q);
                const float x1 = __shfl_sync(0xffffffffu, v.xs[b], nt * 8 + 2 * q + 1);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float p = part[0][mt][nt][j];
                    if constexpr (C == 2) p += part[C - 1][mt][nt][j];
                    float& d = acc.d[mt][nt][j];
                    d = __fmaf_rn((j / 2 ? s1 : s0) * (j % 2 ? x1 : x0), p, d);
                }
            }
        }
    }
}

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
// split K.  (Units of at most 16 rows, one tile each, where a CTA has more than FW_ROWS: 16384 rows of 8192 in
// 44 us against 39.5.)
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
