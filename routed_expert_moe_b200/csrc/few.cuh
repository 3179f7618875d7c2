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
// for the weights, multiplies with warp-level matrix instructions (tokens as
// the 16-row operand, weight rows as the 8-column one) and hands the slot
// back.  No consumer waits for another within a stream.  tcgen05 would need
// 128 weight rows per instruction; boxes of 16 to 24 rows let every SM stream
// the same number of bytes.
//
// Copying row by row instead (untiled bulk copies) costs a fixed 32 cycles of
// an SM's copy engine per row: 4.6 TB/s at 512 bytes per row, against 7.0 with
// boxes.  Consumers that fill their rings themselves spend 500 cycles a stage
// on it.
//
// Lane (g, q) = (lane / 4, lane % 4) of a warp reads 16 bytes at
// 64 * segment + 16 * q of weight rows g, g + 8, g + 16 and of tokens g and g + 8:
// the matrix instruction's K index is assigned to those bytes in the same
// order on both sides, so no value moves between lanes.
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

// Segments per stage.  Five: an odd number puts the rows of a stage, 320 bytes apart, into
// alternating halves of the banks.  Formats with a scale per 128 bytes take whole blocks.
constexpr int fw_segs(bool block) { return block ? 6 : 5; }

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

// D (16 tokens x 8 weight rows, fp32) += A (16 x 16 values) * B (8 x 16 values), bf16 or fp16 operands
// (volatile: it must stay where the whole warp is converged).  E4M3 operands are converted to fp16,
// which holds them exactly: the warp-level E4M3 instruction takes 24 cycles of a scheduler here,
// against 8 for the fp16 one, and would convert the activations again for every eight weight rows.
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

// What goes with the weights of N segments, in registers: the two activation rows that this lane
// supplies (rows g and g + 8 of the 16-row operand; TWO: they differ), the scales of one weight row
// (row `lane`, handed round by shuffles) and of the two activation rows.  The first batch of a stage is
// fetched while the warp still waits for its weights.
template <typename F, int N, bool TWO>
struct FwActs {
    static constexpr int KB = F::BLOCK ? N / 2 : 1;
    static_assert(!F::BLOCK || N % 2 == 0, "whole blocks");
    uint4 x[N][TWO ? 2 : 1][F::AV];
    float ws[KB];
    float xs[F::BLOCK_ACT ? KB : 1][TWO ? 2 : 1];
};

// Where they come from: from the start of a K row on (activation rows: this lane's first bytes).  A token
// slot without a token, like a row past the tile, repeats another one and is not used.
struct FwSide {
    const uint8_t* act[2];
    const float* ws;        // of weight row `lane`
    const float* xs[2];
};

// The batch from weight byte c0 on; the activation rows go with row_bytes weight bytes (zeros past
// them; weights may be padded).
template <typename F, int N, bool TWO>
__device__ __forceinline__ void fw_fetch(FwActs<F, N, TWO>& v, const FwSide& side, int c0, int row_bytes) {
    const int q16 = (threadIdx.x % 4) * 16;
    const bool full = c0 + N * FW_SEG <= row_bytes;
    if (full) {
#pragma unroll
        for (int t = 0; t < (TWO ? 2 : 1); ++t) {
            const uint8_t* p = side.act[t] + c0 * F::AV;
#pragma unroll
            for (int s = 0; s < N; ++s)
#pragma unroll
                for (int j = 0; j < F::AV; ++j)
                    v.x[s][t][j] = *reinterpret_cast<const uint4*>(p + s * FW_SEG * F::AV + j * 16);
        }
    } else {
#pragma unroll
        for (int t = 0; t < (TWO ? 2 : 1); ++t) {
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
        for (int b = 0; b < FwActs<F, N, TWO>::KB; ++b) {
            const bool in = full || c0 + b * 128 < row_bytes;
            v.ws[b] = in ? __ldg(side.ws + c0 / 128 + b) : 0.0f;
            if constexpr (F::BLOCK_ACT) {
#pragma unroll
                for (int t = 0; t < (TWO ? 2 : 1); ++t) v.xs[b][t] = in ? __ldg(side.xs[t] + c0 / 128 + b) : 0.0f;
            }
        }
    }
}

// The running sums of 16 activation rows x 8 NT weight rows, in two chains that do not wait for one
// another.  j: activation row g (+ 8 * (j / 2)), weight row 8 nt + 2 q + j % 2.
template <int NT>
struct FwAcc {
    float d[2][NT][4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) d[0][nt][j] = d[1][nt][j] = 0.0f;
    }
    __device__ __forceinline__ float sum(int nt, int j) const { return d[0][nt][j] + d[1][nt][j]; }
};

// 16 bytes of weights of one row times the activations that go with them.
template <typename F, bool TWO>
__device__ __forceinline__ void fw_step(float (&d0)[4], float (&d1)[4], const uint4 (&x)[TWO ? 2 : 1][F::AV],
                                        const uint4& w) {
    if constexpr (F::BF16) {
        const uint4 a = x[0][0], b = x[TWO ? 1 : 0][0];
        fw_mma<true>(d0, a.x, b.x, a.y, b.y, w.x, w.y);
        fw_mma<true>(d1, a.z, b.z, a.w, b.w, w.z, w.w);
    } else {
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t b0, b1, a[2][2];
            fw_half4(ww[j], b0, b1);
#pragma unroll
            for (int t = 0; t < (TWO ? 2 : 1); ++t) {
                if constexpr (F::CODES) {
                    const uint4 c = x[t][0];
                    fw_half4(j == 0 ? c.x : j == 1 ? c.y : j == 2 ? c.z : c.w, a[t][0], a[t][1]);
                } else {
                    const uint4 c = x[t][j / 2];
                    a[t][0] = j % 2 == 0 ? c.x : c.z;
                    a[t][1] = j % 2 == 0 ? c.y : c.w;
                }
            }
            fw_mma<false>(j % 2 ? d1 : d0, a[0][0], a[TWO ? 1 : 0][0], a[0][1], a[TWO ? 1 : 0][1], b0, b1);
        }
    }
}

// A batch of N segments from byte b of the slot's rows: `rows` weight rows (at most 8 NT; tiles of eight
// past them are skipped) times the activations.
template <typename F, int N, bool TWO, int NT>
__device__ __forceinline__ void fw_mul(FwAcc<NT>& acc, const uint8_t* slot, int b, int rows, const FwActs<F, N, TWO>& v) {
    const int lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        if (nt * 8 >= rows) break;
        // rows past the last repeat it: their results are not used
        const uint8_t* r = slot + min(nt * 8 + g, rows - 1) * (F::SEGS * FW_SEG) + b + q * 16;
        float part[2][4];
#pragma unroll
        for (int s = 0; s < N; ++s) {
            const uint4 w = *reinterpret_cast<const uint4*>(r + s * FW_SEG);
            if constexpr (F::BLOCK) {
                if (s % 2 == 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) part[0][j] = part[1][j] = 0.0f;
                }
                fw_step<F, TWO>(part[0], part[1], v.x[s], w);
                if (s % 2 == 1) {
                    const float s0 = __shfl_sync(0xffffffffu, v.ws[s / 2], nt * 8 + 2 * q);
                    const float s1 = __shfl_sync(0xffffffffu, v.ws[s / 2], nt * 8 + 2 * q + 1);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float sc = j % 2 ? s1 : s0;
                        if constexpr (F::BLOCK_ACT) sc *= v.xs[s / 2][TWO ? j / 2 : 0];
                        float& d = acc.d[s / 2 % 2][nt][j];
                        d = __fmaf_rn(sc, part[0][j] + part[1][j], d);
                    }
                }
            } else {
                fw_step<F, TWO>(acc.d[0][nt], acc.d[1][nt], v.x[s], w);
            }
        }
    }
}

// The batches of a stage after the first (registers: two activation rows of fp16 take twice the room).
template <typename F, bool TWO>
constexpr int fw_batch() {
    return TWO && F::AV == 2 ? (F::BLOCK ? 2 : 1) : F::SEGS;
}
template <typename F, bool TWO, int NT>
__device__ __forceinline__ void fw_mul_stage(FwAcc<NT>& acc, const uint8_t* slot, int rows, int c0, int row_bytes,
                                             const FwSide& side, FwActs<F, fw_batch<F, TWO>(), TWO>& v) {
    constexpr int N = fw_batch<F, TWO>();
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
