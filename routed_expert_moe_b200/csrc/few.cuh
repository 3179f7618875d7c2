// Weight streaming for a few tokens: the parts that the few-token layer
// (few.cu) and the few-row dense product (linear_b128.cu) share.
//
// A weight row is read once from HBM and meets at most 16 activation rows, so
// the work is a stream: 2 * 16 operations per weight at most, far below what
// the tensor cores take at HBM's rate.  Each of a CTA's eight warps runs a
// pipeline of its own: its lane 0 copies the next rows' chunk of K into the
// warp's ring in shared memory (one untiled bulk copy per row), the warp waits
// on that copy's barrier, multiplies with warp-level matrix instructions
// (weights as the 16-row operand, tokens as the 8-column one), and refills the
// slot it has read.  No warp waits for another within a stream.  tcgen05 would
// need 128 weight rows per instruction; here a warp takes 9 or 10, which lets
// every SM stream the same number of bytes.
//
// Lane (g, q) = (lane / 4, lane % 4) of a warp reads 16 bytes at
// 64 * segment + 16 * q of weight rows g and g + 8 and of token g's
// activations: the matrix instruction's K index is assigned to those bytes in
// the same order on both sides, so no value moves between lanes.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int FW_WARPS = 8;
constexpr int FW_THREADS = 32 * FW_WARPS;
constexpr int FW_SEG = 64;                    // bytes of a row that one matrix step takes
constexpr int FW_CHUNK = 768;                 // bytes of a row per stage at most
constexpr int FW_GROUP = 4;                   // segments whose activations are loaded together
constexpr int FW_ROWS = 16;                   // weight rows per stage at most
constexpr int FW_MAX_STAGES = 7;              // of one warp's ring
constexpr int FW_SMEM = 227 * 1024;           // shared memory a block may use

// How a weight row of `bytes` bytes is cut into chunks of whole units: segments, or scale blocks.
struct FwCut {
    int bytes;    // of a row
    int chunk;    // bytes per stage; the last one may be shorter
    int n;        // chunks per row
};
inline FwCut fw_cut(int bytes, int unit) {
    FwCut c;
    c.bytes = bytes;
    const int n = (bytes + FW_CHUNK - 1) / FW_CHUNK;
    c.chunk = ((bytes + n - 1) / n + unit - 1) / unit * unit;
    c.n = (bytes + c.chunk - 1) / c.chunk;
    return c;
}
// Distance between two rows of a stage: 64 bytes modulo 128, so that the two rows that eight
// neighbouring lanes read lie in different banks.
inline int fw_row_stride(int chunk) { return chunk % 128 == 64 ? chunk : chunk + 64; }

__device__ __forceinline__ void fw_bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                             uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
        ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(policy) : "memory");
}

__device__ __forceinline__ uint4 fw_lds(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// D (16 x 8, fp32) += A (16 rows x 32 bytes) * B (8 columns x 32 bytes): bf16 or E4M3 operands.
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
            "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One warp's ring.
struct FwRing {
    uint32_t base;       // slots
    uint32_t bars;       // one mbarrier per slot (8 bytes each)
    int slot_bytes, stride, n;
    int put, take;       // next slot to fill, to read
    uint32_t parity;     // of the next slot to read
    uint64_t policy;

    // Starts the copy of `rows` rows of `bytes` bytes, ld bytes apart.  Whole warp, converged; every
    // lane has finished reading the slot.
    __device__ __forceinline__ void fill(const uint8_t* src, int64_t ld, int rows, uint32_t bytes) {
        if (threadIdx.x % 32 == 0) {
            const uint32_t bar = bars + 8 * put;
            uint32_t dst = base + put * slot_bytes;
            mbar_arrive_expect_tx(bar, bytes * rows);
            for (int r = 0; r < rows; ++r, dst += stride, src += ld) fw_bulk_load(dst, src, bytes, bar, policy);
        }
        if (++put == n) put = 0;
    }
    // Waits for the next slot; returns its address in `slot`.
    __device__ __forceinline__ bool wait(uint32_t& slot, const DevCtx& ctx, volatile int* abort) {
        slot = base + take * slot_bytes;
        return mbar_wait_warp(bars + 8 * take, parity, ctx, abort);
    }
    __device__ __forceinline__ void next() {
        if (++take == n) {
            take = 0;
            parity ^= 1u;
        }
    }
};

// A lane's activations and block scales for FW_GROUP segments.
template <int NT, bool SPLIT, bool BLOCK, bool BLOCK_ACT>
struct FwActs {
    uint4 b[FW_GROUP][NT];                        // 16 bytes of token g + 8 * nt
    uint4 lo[SPLIT ? FW_GROUP : 1][NT];           // low parts (SPLIT: an activation is the sum of two bf16)
    float ws[BLOCK ? FW_GROUP / 2 : 1][2];        // scale of weight rows g, g + 8 per 128-byte block
    float xs[BLOCK_ACT ? FW_GROUP / 2 : 1][NT][2];   // scale of tokens 8 nt + 2 q, + 1 per block
};

// A lane's rows of activations: its tokens g + 8 * nt (+ 16 q bytes), zeros for a token that is not there.
template <int NT>
struct FwRows {
    const uint8_t* p[NT];
    bool on[NT];
};
__device__ __forceinline__ uint4 fw_ld16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

// Fetches FW_GROUP segments from byte c0 of the rows on.  `n_seg` of them are in the stage; rows hold
// `row_bytes` bytes (a row may end inside the last one).  lo: distance to the low parts.
template <int NT, bool SPLIT, bool BLOCK, bool BLOCK_ACT>
__device__ __forceinline__ void fw_load(FwActs<NT, SPLIT, BLOCK, BLOCK_ACT>& v, const FwRows<NT>& r, int c0, int n_seg,
                                        int row_bytes, int64_t lo) {
    const int q16 = (threadIdx.x % 4) * 16;
    const bool whole = n_seg >= FW_GROUP && c0 + FW_GROUP * FW_SEG <= row_bytes;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int s = 0; s < FW_GROUP; ++s) {
            v.b[s][nt] = make_uint4(0, 0, 0, 0);
            if constexpr (SPLIT) v.lo[s][nt] = make_uint4(0, 0, 0, 0);
        }
        if (r.on[nt]) {
            if (whole) {
#pragma unroll
                for (int s = 0; s < FW_GROUP; ++s) {
                    v.b[s][nt] = fw_ld16(r.p[nt] + c0 + s * FW_SEG);
                    if constexpr (SPLIT) v.lo[s][nt] = fw_ld16(r.p[nt] + lo + c0 + s * FW_SEG);
                }
            } else {
#pragma unroll
                for (int s = 0; s < FW_GROUP; ++s)
                    if (s < n_seg && c0 + s * FW_SEG + q16 < row_bytes) {
                        v.b[s][nt] = fw_ld16(r.p[nt] + c0 + s * FW_SEG);
                        if constexpr (SPLIT) v.lo[s][nt] = fw_ld16(r.p[nt] + lo + c0 + s * FW_SEG);
                    }
            }
        }
    }
}

// One group of segments seg0 .. of a stage: weight rows g and g + 8 at r0 and r1 (this lane's 16
// bytes of segment 0), `left` bytes of the row remain from the chunk's start.
template <bool BF16, int NT, bool SPLIT, bool BLOCK, bool BLOCK_ACT>
__device__ __forceinline__ void fw_group(float (&acc)[NT][4], uint32_t r0, uint32_t r1, int seg0, int n_seg, int left,
                                         const FwActs<NT, SPLIT, BLOCK, BLOCK_ACT>& v) {
    const int q16 = (threadIdx.x % 4) * 16;
#pragma unroll
    for (int s = 0; s < FW_GROUP; s += 2) {
        if (seg0 + s >= n_seg) break;
        float part[NT][4] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int seg = seg0 + s + h;
            if (seg >= n_seg) break;
            uint4 a0 = fw_lds(r0 + seg * FW_SEG), a1 = fw_lds(r1 + seg * FW_SEG);
            if (seg * FW_SEG + FW_SEG > left) {   // the row ends inside the segment
                if (seg * FW_SEG + q16 >= left) a0 = a1 = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float(&d)[4] = BLOCK ? part[nt] : acc[nt];
                const uint4 b = v.b[s + h][nt];
                fw_mma<BF16>(d, a0.x, a1.x, a0.y, a1.y, b.x, b.y);
                fw_mma<BF16>(d, a0.z, a1.z, a0.w, a1.w, b.z, b.w);
                if constexpr (SPLIT) {
                    const uint4 l = v.lo[s + h][nt];
                    fw_mma<BF16>(d, a0.x, a1.x, a0.y, a1.y, l.x, l.y);
                    fw_mma<BF16>(d, a0.z, a1.z, a0.w, a1.w, l.z, l.w);
                }
            }
        }
        if constexpr (BLOCK) {   // the two segments are one block of 128
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float sc = v.ws[s / 2][c / 2];
                    if constexpr (BLOCK_ACT) sc *= v.xs[s / 2][nt][c % 2];
                    acc[nt][c] = __fmaf_rn(sc, part[nt][c], acc[nt][c]);
                }
        }
    }
}

// One stage: load(v, seg0, n) fetches the activations of a group (n segments of the stage from seg0); the first group's are under way while the
// warp waits for the weights, the next group's while one is multiplied.
template <bool BF16, int NT, bool SPLIT, bool BLOCK, bool BLOCK_ACT, typename Load>
__device__ __forceinline__ bool fw_stage(float (&acc)[NT][4], FwRing& ring, int rows, int bytes, const Load& load,
                                         const DevCtx& ctx, volatile int* abort) {
    const int lane = threadIdx.x % 32, g = lane / 4, q16 = (lane % 4) * 16;
    const int n_seg = (bytes + FW_SEG - 1) / FW_SEG;
    FwActs<NT, SPLIT, BLOCK, BLOCK_ACT> v0, v1;
    load(v0, 0, n_seg);
    uint32_t slot;
    if (!ring.wait(slot, ctx, abort)) return false;
    // rows past the tile repeat its last one: their products are not used
    const uint32_t r0 = slot + min(g, rows - 1) * ring.stride + q16, r1 = slot + min(g + 8, rows - 1) * ring.stride + q16;
#pragma unroll
    for (int s = 0; s < FW_CHUNK / FW_SEG; s += 2 * FW_GROUP) {
        if (s + FW_GROUP < n_seg) load(v1, s + FW_GROUP, n_seg - s - FW_GROUP);
        fw_group<BF16, NT, SPLIT, BLOCK, BLOCK_ACT>(acc, r0, r1, s, n_seg, bytes, v0);
        if (s + 2 * FW_GROUP < n_seg) load(v0, s + 2 * FW_GROUP, n_seg - s - 2 * FW_GROUP);
        if (s + FW_GROUP < n_seg)
            fw_group<BF16, NT, SPLIT, BLOCK, BLOCK_ACT>(acc, r0, r1, s + FW_GROUP, n_seg, bytes, v1);
    }
    ring.next();
    __syncwarp();   // every lane has read the slot: the caller may fill it again
    return true;
}

// The pairs (expert i, chunk k) of a stream of n_list x n_chunks that fall to warp w of n_w (a power
// of two).  The chunks rotate over the warps from one expert to the next, so that a short last chunk
// does not always fall to the same warp.
struct FwPairs {
    int i, k;
    __device__ __forceinline__ void seek(int n_list, int n_chunks, int w, int n_w) {   // from expert i's first
        for (; i < n_list; ++i) {
            k = (w - i * (n_chunks | 1)) & (n_w - 1);
            if (k < n_chunks) return;
        }
    }
    __device__ __forceinline__ void step(int n_list, int n_chunks, int w, int n_w) {
        k += n_w;
        if (k < n_chunks) return;
        ++i;
        seek(n_list, n_chunks, w, n_w);
    }
};

// The warps' partial sums of one tile, [warp][row][token].  Two buffers take turns, so that one
// barrier per tile (bounded: every warp arrives, then waits for all eight) orders both the reads after
// the writes and the next writes after the reads.
template <int NT>
struct FwRed {
    static constexpr int kWarp = FW_ROWS * NT * 8;
    static constexpr int kFloats = FW_WARPS * kWarp;
    float* buf;          // [2][kFloats]
    uint32_t bar;        // mbarrier of FW_WARPS arrivals
    int turn;

    __device__ __forceinline__ bool exchange(const float (&acc)[NT][4], int warp, const DevCtx& ctx,
                                             volatile int* abort) {
        const int lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
        float* b = buf + (turn & 1) * kFloats + warp * kWarp;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float* p = b + g * NT * 8 + nt * 8 + 2 * q;
            *reinterpret_cast<float2*>(p) = make_float2(acc[nt][0], acc[nt][1]);
            *reinterpret_cast<float2*>(p + 8 * NT * 8) = make_float2(acc[nt][2], acc[nt][3]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
        const bool ok = mbar_wait_warp(bar, turn & 1, ctx, abort);
        ++turn;
        return ok;
    }
    // after exchange(): element (row, token) over warps w0 .. w0 + n_w, in order
    __device__ __forceinline__ float sum(int row, int token, int w0, int n_w) const {
        const float* b = buf + ((turn & 1) ^ 1) * kFloats + w0 * kWarp + row * NT * 8 + token;
        float s = 0.0f;
        for (int w = 0; w < n_w; ++w) s += b[w * kWarp];
        return s;
    }
};

// Copies in flight land before the block may end (after a wait has given up).
__device__ __forceinline__ void fw_settle() {
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) __nanosleep(1000);
}

// A unit of output rows is shared by the CTA's warps: one group of eight warps that split K (up to 16
// rows) or two groups of four.
struct FwShare {
    int units;     // per CTA
    int groups;    // 1 or 2
    int rows;      // per group at most
};
inline FwShare fw_share(int n, int num_sms) {
    FwShare s;
    const int share = (n + num_sms - 1) / num_sms;
    s.units = (share + 2 * FW_ROWS - 1) / (2 * FW_ROWS);
    const int per = (share + s.units - 1) / s.units;
    s.groups = per > FW_ROWS ? 2 : 1;
    s.rows = (per + s.groups - 1) / s.groups;
    return s;
}

}  // namespace moe
