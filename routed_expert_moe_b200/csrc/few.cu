// The whole routed-MoE layer for 1 to 16 tokens in two launches (bloomery
// issue page, s.2 "Checkpoint facts" and s.3 "Existing owners and gaps";
// audio.cpp model page, "CPU weight offload": router, expert products and
// routing weights):
//
//   l[t,e] = x[t] . Wr[e] (+ b[e])      fixed point, every product rounded to 2^-40, summed exactly
//   S_t, w = the K largest (ties to the lower index), softmax over them
//   h[t,e] = relu(W_up[e] x[t])^2       out[t] = sum_e w[t,e] W_down[e] h[t,e] (+ shared) (+ residual)
//
// 1. few_router_kernel: one block per expert computes its exact logits for all tokens (few enough
//    tokens that the exact sum costs less than an approximate one with a bound and a second pass);
//    further blocks quantise x.  It zeroes the second kernel's counters.
// 2. few_layer_kernel, persistent, one CTA of eight warps per SM: every CTA ranks the logits itself
//    (the same integers give the same choice everywhere), lists the touched experts, and then its
//    consumer warps stream weights (few.cuh): up pieces (16 rows of one expert, claimed for single warps),
//    then the CTA's share of the output rows through all touched experts, so that the weighted sum
//    over experts, the residual and the one rounding happen in the CTA that holds them.  The
//    ring of a warp without further up pieces takes down weights while the last pieces report.
//
// Up pieces are claimed from a counter, so those that a warp waits for belong to warps that run and
// that wait for nothing; no CTA needs another to be resident, and every wait is bounded.
//
// Bound: HBM bytes of the touched experts' weights.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "few.cuh"

namespace moe {

constexpr int FEW_RT = 256;          // threads of the router kernel

// ----------------------------------------------------------------------------- router

struct FewRouterArgs {
    const uint16_t* x;
    const uint16_t* wr;
    const float* bias;
    int T, H, E;
    long long* logits;   // [T][E], units of 2^-40
    __half* xq;          // values of x's E4M3 codes [T][H], or null
    float x_scale;
    int* counters;       // [2]: piece claims, piece reports
};

// The E4M3 codes (nearest-even, saturating) of two quotients, as a pair of fp16 values.
__device__ __forceinline__ uint32_t few_code_values(float a, float b) {
    const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    uint32_t lo, hi;
    fw_half4(c, lo, hi);
    return lo;
}

__global__ void __launch_bounds__(FEW_RT) few_router_kernel(FewRouterArgs a, DevCtx ctx) {
    pdl_enter();
    __shared__ long long s_l[kFewMaxTokens][8];
    __shared__ float s_x[kFewMaxTokens][8], s_w[8];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int nv = a.H / 8;
    if ((int)blockIdx.x >= a.E) {   // one token's E4M3 codes, as values
        const int t = blockIdx.x - a.E;
        const uint4* xr = reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.H);
        for (int v = tid; v < nv; v += FEW_RT) {
            const uint4 p = xr[v];
            const uint32_t w[4] = {p.x, p.y, p.z, p.w};
            uint32_t c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                c[j] = few_code_values(__fdiv_rn(__uint_as_float(w[j] << 16), a.x_scale),
                                       __fdiv_rn(__uint_as_float(w[j] & 0xFFFF0000u), a.x_scale));
            reinterpret_cast<uint4*>(a.xq + (int64_t)t * a.H)[v] = make_uint4(c[0], c[1], c[2], c[3]);
        }
        return;
    }
    const int e = blockIdx.x;
    if (e == 0 && tid < 2) a.counters[tid] = 0;
    // a warp takes one token over 1 / parts of H
    const int parts = a.T == 1 ? 8 : a.T == 2 ? 4 : a.T <= 4 ? 2 : 1;
    const int part = warp % parts;
    const uint4* wv = reinterpret_cast<const uint4*>(a.wr + (int64_t)e * a.H);
    for (int t = warp / parts; t < a.T; t += 8 / parts) {
        const uint4* xv = reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.H);
        long long acc = 0;
        float xs = 0.0f, ws = 0.0f;
#pragma unroll 4
        for (int v = part * 32 + lane; v < nv; v += 32 * parts) {
            const uint4 p = xv[v], r = wv[v];
            const uint32_t pp[4] = {p.x, p.y, p.z, p.w}, rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float f = __uint_as_float((j & 1) ? (pp[j / 2] & 0xFFFF0000u) : (pp[j / 2] << 16));
                const float h = __uint_as_float((j & 1) ? (rr[j / 2] & 0xFFFF0000u) : (rr[j / 2] << 16));
                acc += __float2ll_rn(__fmul_rn(__fmul_rn(f, h), 0x1p40f));   // the product is exact
                xs = __fmaf_rn(f, f, xs);
                ws = __fmaf_rn(h, h, ws);
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            acc += __shfl_xor_sync(0xffffffffu, acc, off);
            xs += __shfl_xor_sync(0xffffffffu, xs, off);
            ws += __shfl_xor_sync(0xffffffffu, ws, off);
        }
        if (lane == 0) {
            s_l[t][part] = acc;
            s_x[t][part] = xs;
            if (t == 0) s_w[part] = ws;
        }
    }
    __syncthreads();
    if (tid < a.T) {
        long long l = 0;
        float xs = 0.0f, ws = 0.0f;
        for (int p = 0; p < parts; ++p) {
            l += s_l[tid][p];
            xs += s_x[tid][p];
            ws += s_w[p];
        }
        // the domain of exactness, as in the other routers: upper bounds of the norms below 2^22
        const double infl = 1.0 + (double)(a.H + 64) * 0x1p-23;
        const float b = a.bias ? a.bias[e] : 0.0f;
        if (!(sqrt((double)xs * infl) * sqrt((double)ws * infl) < 0x1p22) || !(fabsf(b) < 0x1p21f))
            record_error(ctx.err, MOE_ERANGE);
        if (a.bias) l += __float2ll_rn(__fmul_rn(b, 0x1p40f));
        a.logits[(int64_t)tid * a.E + e] = l;
    }
}

// ----------------------------------------------------------------------------- layer

struct FewArgs {
    const uint16_t* x;
    const uint16_t* residual;   // or null
    uint16_t* out;
    int32_t* topk_idx;          // or null
    float* topk_w;              // or null
    const long long* logits;
    const uint8_t* act;         // up operand rows [T][H]: x, or the fp16 values of its E4M3 codes
    const float* su;            // E4M3: [E]; B128: [E][F][kbu]
    const float* sd;            // E4M3: [E]; B128: [E][H][kbd]
    float x_scale, h_scale;
    uint8_t* h;                 // [rows][F]: bf16 high parts and then low parts, or fp16 values of E4M3 codes
    int64_t h_lo;               // bf16: bytes from a high part to its low part
    int* counters;
    int T, H, E, K, F, ns;
    FwCut up, down;
    FwShare share;              // of the output rows
    int slot_bytes, n_stages;
    int n_list_max;
    int first;                  // pieces that a CTA claims at the start
    int hold;                   // test hook: up piece 0 never reports
};

// Weight matrices: rows of W_up in boxes of 16; rows of W_down in boxes of share.rows and one less;
// the same of the shared expert.
struct FewMaps {
    CUtensorMap up, down[2], up_s, down_s[2];
};

constexpr int FEW_PIECE = 16;   // rows of an up piece (F is a multiple of 16)

// shared memory after the rings: reduction buffers | wt [n][16] f32 | rowi [n][16] u16 | tok [n][16] u8 |
// lst_e [n] i32 | lst_n [n] i32 | emask [256] i32 | slot [256] i32 | sel_w [16][16] f32 | sel_e [16][16] i32 |
// barriers | piece of each slot | flags
__host__ __device__ inline size_t few_table_bytes(int n_list) {
    return (size_t)n_list * (64 + 32 + 16 + 8) + 16 + 4 * 1024 + FwRings::kBarBytes + 8 +
           FW_WARPS * FW_MAX_STAGES * 4 + 16;
}

// The K best experts of one token (one warp): by logit, ties to the lower index; lane k returns the
// k-th.  A 64-bit maximum as three 32-bit warp reductions: high word (signed), low word, index.
__device__ __forceinline__ void few_select(const long long* row, int E, int K, int lane, int& my_e, float& my_w) {
    long long key[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = lane + 32 * j;
        key[j] = e < E ? __ldcg(row + e) : 0;
    }
    uint32_t taken = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (lane + 32 * j >= E) taken |= 1u << j;
    long long my_l = 0, first = 0;
    my_e = 0;
    for (int k = 0; k < K; ++k) {
        long long best = LLONG_MIN;
        int bj = -1;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (!((taken >> j) & 1u) && (bj < 0 || key[j] > best)) {
                best = key[j];
                bj = j;
            }
        const int hi = bj < 0 ? INT_MIN : (int)(best >> 32);
        const int mhi = __reduce_max_sync(0xffffffffu, hi);
        const bool in1 = bj >= 0 && hi == mhi;
        const unsigned lo = in1 ? (unsigned)best : 0u;
        const unsigned mlo = __reduce_max_sync(0xffffffffu, lo);
        const bool in2 = in1 && lo == mlo;
        const unsigned e = in2 ? (unsigned)(lane + 32 * bj) : 0xFFFFFFFFu;
        const unsigned me = __reduce_min_sync(0xffffffffu, e);
        if (in2 && e == me) taken |= 1u << bj;
        const long long l = ((long long)mhi << 32) | mlo;
        if (k == 0) first = l;
        if (lane == k) {
            my_e = (int)me;
            my_l = l;
        }
    }
    const float ex = lane < K ? expf((float)((double)(my_l - first) * 0x1p-40)) : 0.0f;
    float z = 0.0f;
    for (int k = 0; k < K; ++k) z += __shfl_sync(0xffffffffu, ex, k);
    my_w = ex / z;
}

template <int FMT>
using FewFmt = FwFmt<FMT == MOE_BF16, false, FMT == MOE_FP8_B128, false>;

// One up piece: 16 rows of a list entry with at most 8 TT tokens.
template <int FMT, int TT>
__device__ __forceinline__ bool few_up(const FewArgs& a, FwTake& ring, int e, int f, int n_tok, const uint16_t* rowi,
                                       const uint8_t* tok, const DevCtx& ctx, volatile int* abort) {
    using F = FewFmt<FMT>;
    constexpr bool BF16 = F::BF16, BLOCK = F::BLOCK;
    const int lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
    const int row_bytes = BF16 ? 2 * a.H : a.H;
    FwSide<TT> side;
#pragma unroll
    for (int t = 0; t < TT; ++t) side.act[t] = a.act + (int64_t)tok[min(t * 8 + g, n_tok - 1)] * a.H * 2 + q * F::AB;
    if constexpr (BLOCK) side.ws = a.su + ((int64_t)e * a.F + f + lane % FEW_PIECE) * (a.up.bytes / 128);
    FwAcc<1, TT> acc;
    acc.clear();
    FwActs<F, fw_batch<F, TT>(), TT> v;
    fw_fetch(v, side, 0, row_bytes);
    for (int c0 = 0; c0 < a.up.bytes;) {
        if (!ring.wait(ctx, abort)) return false;
        fw_mul_stage(acc, ring.data(), FEW_PIECE, c0, row_bytes, side, v);
        ring.release();
        c0 += a.up.chunk;
        if (c0 < a.up.bytes) fw_fetch(v, side, c0, row_bytes);
    }
    const float sc = BF16 ? 1.0f : BLOCK ? a.x_scale : __fmul_rn(a.su[e], a.x_scale);
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int s = t * 8 + 2 * q + j % 2;
            if (s >= n_tok) continue;
            const int64_t o = (int64_t)rowi[s] * a.F + f + g + 8 * (j / 2);
            float z = acc.sum(0, t, j);
            if constexpr (!BF16) z = __fmul_rn(z, sc);
            const float h = z <= 0.0f ? 0.0f : __fmul_rn(z, z);   // a NaN stays one
            if constexpr (BF16) {
                // h as the sum of two bf16, 16 bits of it: one alone would add a second rounding of the
                // output's size
                const __nv_bfloat16 hi = __float2bfloat16_rn(h);
                const float top = __bfloat162float(hi);
                reinterpret_cast<__nv_bfloat16*>(a.h)[o] = hi;
                reinterpret_cast<__nv_bfloat16*>(a.h + a.h_lo)[o] =
                    __float2bfloat16_rn(top < __uint_as_float(0x7f800000u) ? __fsub_rn(h, top) : 0.0f);
            } else {
                reinterpret_cast<uint16_t*>(a.h)[o] = (uint16_t)few_code_values(__fdiv_rn(h, a.h_scale), 0.0f);
            }
        }
    return true;
}

// One warp's part of n output rows from d0 on, through its pairs of all list entries: the weighted sums
// tot [token][row] (shared memory, this warp's).
template <int FMT>
struct FewDown {
    using F = FewFmt<FMT>;
    static constexpr bool BF16 = F::BF16, BLOCK = F::BLOCK;
    const FewArgs& a;
    FwTake& ring;
    const int *lst_e, *lst_n;
    const uint16_t* rowi;
    const uint8_t* tok;
    const float* wt;
    int n_list, warp, d0, n;
    float* tot;
    const DevCtx& ctx;
    volatile int* abort;

    // Entry i: the activations of its first 8 TT token slots (bf16, TT 1: high and low parts), weight scales
    template <int NT>
    __device__ __forceinline__ void point(FwSide<NT>& side, int i, bool parts) const {
        const int lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
        const int last = lst_n[i] - 1;
        side.act[0] = a.h + (int64_t)rowi[i * 16 + min(g, last)] * a.F * 2 + q * F::AB;
        if constexpr (NT == 2)
            side.act[1] = parts ? side.act[0] + a.h_lo : a.h + (int64_t)rowi[i * 16 + min(8 + g, last)] * a.F * 2 + q * F::AB;
        if constexpr (BLOCK) side.ws = a.sd + ((int64_t)lst_e[i] * a.H + d0 + min(lane, n - 1)) * (a.down.bytes / 128);
    }
    // The running sums of one entry and a stage of them
    template <int NT>
    struct Acc {
        typename std::conditional<BF16, FwAccT<3>, FwAcc<2, NT>>::type s;
    };
    template <int NT>
    __device__ __forceinline__ void mul(Acc<NT>& acc, int c0, int row_bytes, const FwSide<NT>& side,
                                        FwActs<F, fw_batch<F, NT>(), NT>& v) const {
        if constexpr (BF16) fw_mul_t(acc.s, ring.data(), n, v);
        else fw_mul_stage(acc.s, ring.data(), n, c0, row_bytes, side, v);
    }
    // Weighted sums of entry i, for the tokens routed to it only
    template <int NT>
    __device__ __forceinline__ void add(const Acc<NT>& acc, int i, bool parts) const {
        const int lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
        if constexpr (BF16) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int s = t * 8 + g;
                if (s >= lst_n[i] || (t == 1 && parts)) continue;
                const float w = wt[i * 16 + s];
#pragma unroll
                for (int nt = 0; nt < 3; ++nt) {
                    float2* p = reinterpret_cast<float2*>(tot + tok[i * 16 + s] * FW_ROWS + nt * 8 + 2 * q);
                    float y0 = acc.s.sum(nt, 2 * t), y1 = acc.s.sum(nt, 2 * t + 1);
                    if (parts) {
                        y0 += acc.s.sum(nt, 2);
                        y1 += acc.s.sum(nt, 3);
                    }
                    const float2 v = *p;
                    *p = make_float2(__fmaf_rn(w, y0, v.x), __fmaf_rn(w, y1, v.y));
                }
            }
        } else {
            const float sc = FMT == MOE_FP8_E4M3 ? a.sd[lst_e[i]] : 1.0f;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int s = t * 8 + 2 * q + c;
                    if (s >= lst_n[i]) continue;
                    const float w = wt[i * 16 + s] * sc;
                    float* p = tot + tok[i * 16 + s] * FW_ROWS + g;
#pragma unroll
                    for (int r = 0; r < 3; ++r)   // rows g + 8 r
                        p[8 * r] = __fmaf_rn(w, acc.s.sum(r / 2, t, c + 2 * (r % 2)), p[8 * r]);
                }
        }
        __syncwarp();
    }
    // An entry with more than eight tokens
    __device__ __forceinline__ bool wide(FwPairs& pr) {
        const int i = pr.i, row_bytes = BF16 ? 2 * a.F : a.F;
        FwSide<2> hi, lo;
        point<2>(hi, i, false);
        if constexpr (BF16) {
            lo.act[0] = hi.act[0] + a.h_lo;
            lo.act[1] = hi.act[1] + a.h_lo;
        }
        Acc<2> acc;
        acc.s.clear();
        do {
            const int c0 = pr.k * a.down.chunk;
            FwActs<F, fw_batch<F, 2>(), 2> v;
            fw_fetch(v, hi, c0, row_bytes);
            if (!ring.wait(ctx, abort)) return false;
            mul(acc, c0, row_bytes, hi, v);
            if constexpr (BF16) {
                fw_fetch(v, lo, c0, row_bytes);
                mul(acc, c0, row_bytes, lo, v);
            }
            ring.release();
            pr.step(lst_e, n_list, a.down.n, warp);
        } while (pr.i == i);
        add(acc, i, false);
        return true;
    }
    __device__ __forceinline__ bool run() {
        constexpr int NT = BF16 ? 2 : 1;   // high and low parts
        const int row_bytes = BF16 ? 2 * a.F : a.F;
        FwPairs pr{0, 0};
        pr.seek(lst_e, n_list, a.down.n, warp);
        bool fetched = false;
        FwSide<NT> side;
        FwActs<F, fw_batch<F, NT>(), NT> v;
        while (pr.i < n_list) {
            const int i = pr.i;
            if (lst_n[i] > 8) {
                if (!wide(pr)) return false;
                continue;
            }
            if (!fetched) {
                point<NT>(side, i, true);
                fw_fetch(v, side, pr.k * a.down.chunk, row_bytes);
            }
            Acc<NT> acc;
            acc.s.clear();
            do {
                if (!ring.wait(ctx, abort)) return false;
                mul(acc, pr.k * a.down.chunk, row_bytes, side, v);
                ring.release();
                // the next pair's activations, of this entry or the next
                pr.step(lst_e, n_list, a.down.n, warp);
                fetched = pr.i < n_list && lst_n[pr.i] <= 8;
                if (fetched) {
                    if (pr.i != i) point<NT>(side, pr.i, true);
                    fw_fetch(v, side, pr.k * a.down.chunk, row_bytes);
                }
            } while (pr.i == i);
            add(acc, i, true);
        }
        return true;
    }
};

template <int FMT>
__global__ void __launch_bounds__(FW_THREADS, 1)
    few_layer_kernel(const __grid_constant__ FewMaps maps, const __grid_constant__ FewArgs a, DevCtx ctx) {
    constexpr int ES = FMT == MOE_BF16 ? 2 : 1;
    extern __shared__ __align__(1024) uint8_t few_smem[];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    uint8_t* p = few_smem + (size_t)FW_WARPS * a.n_stages * a.slot_bytes;
    FwRed red;
    red.buf = reinterpret_cast<float*>(p);
    p += FwRed::bytes(a.share.units);
    float* wt = reinterpret_cast<float*>(p);
    p += (size_t)a.n_list_max * 64;
    uint16_t* rowi = reinterpret_cast<uint16_t*>(p);
    p += (size_t)a.n_list_max * 32;
    uint8_t* tok = p;
    p += (size_t)a.n_list_max * 16;
    int* lst_e = reinterpret_cast<int*>(p);
    int* lst_n = lst_e + a.n_list_max;
    p += ((size_t)a.n_list_max * 8 + 15) / 16 * 16;
    int* emask = reinterpret_cast<int*>(p);
    p += 1024;
    int* eslot = reinterpret_cast<int*>(p);
    p += 1024;
    float(*sel_w)[16] = reinterpret_cast<float(*)[16]>(p);
    p += 1024;
    int(*sel_e)[16] = reinterpret_cast<int(*)[16]>(p);
    p += 1024;
    FwRings rings;
    rings.base = few_smem;
    rings.full = reinterpret_cast<uint64_t*>(p);
    rings.empty = rings.full + FW_WARPS * FW_MAX_STAGES;
    rings.slot_bytes = a.slot_bytes;
    rings.n = a.n_stages;
    uint64_t* rbar = rings.full + FwRings::kBarBytes / 8;
    volatile int* slot_piece = reinterpret_cast<volatile int*>(rbar + 1);   // [warp][slot]
    volatile int* abort_flag = slot_piece + FW_WARPS * FW_MAX_STAGES;
    int* n_touched = const_cast<int*>(abort_flag) + 1;
    int* first_piece = n_touched + 1;
    red.bar = smem_u32(rbar);
    red.turn = 0;

    if (tid == 0) {
        rings.init();
        mbar_init(smem_u32(rbar), FW_WARPS);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.up);
        tma_prefetch_desc(&maps.down[0]);
        tma_prefetch_desc(&maps.down[1]);
    }
    for (int i = tid; i < 256; i += FW_THREADS) emask[i] = 0;
    __syncthreads();
    pdl_enter();

    // The CTA's first pieces: an equal share for every CTA of those that there are at least (K experts'),
    // claimed together; single claims would let the CTAs that start first take more than others.
    if (tid == 32 * FW_WARPS) *first_piece = a.first > 0 ? atomicAdd(a.counters, a.first) : 0;

    // ---- the routing, the same in every CTA
    for (int t = warp; t < a.T; t += FW_WARPS + FW_PROD) {
        int e;
        float w;
        few_select(a.logits + (int64_t)t * a.E, a.E, a.K, lane, e, w);
        if (lane < a.K) {
            sel_e[t][lane] = e;
            sel_w[t][lane] = w;
            atomicOr(&emask[e], 1 << t);
            if (blockIdx.x == 0) {
                if (a.topk_idx) a.topk_idx[t * a.K + lane] = e;
                if (a.topk_w) a.topk_w[t * a.K + lane] = w;
            }
        }
    }
    __syncthreads();
    if (warp == 0) {   // the touched experts, ascending, then the shared expert's chunks
        int n = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int mask = e < a.E ? emask[e] : 0;
            const uint32_t m = __ballot_sync(0xffffffffu, mask != 0);
            if (mask) {
                const int i = n + __popc(m & ((1u << lane) - 1u));
                eslot[e] = i;
                lst_e[i] = e;
                lst_n[i] = __popc(mask);
            }
            n += __popc(m);
        }
        if (lane < a.ns) {
            lst_e[n + lane] = a.E + lane;
            lst_n[n + lane] = a.T;
        }
        if (lane == 0) *n_touched = n;
    }
    __syncthreads();
    const int n_routed = *n_touched, n_list = n_routed + a.ns;
    // each list entry's tokens, ascending, with the row of h and the weight that go with them
    for (int i = tid; i < a.T * (a.K + a.ns); i += FW_THREADS) {
        const int t = i % a.T, k = i / a.T;
        int s, row;
        float w;
        if (k < a.K) {
            const int e = sel_e[t][k];
            s = eslot[e] * 16 + __popc(emask[e] & ((1 << t) - 1));
            row = t * a.K + k;
            w = sel_w[t][k];
        } else {
            s = (n_routed + k - a.K) * 16 + t;
            row = a.T * a.K + (k - a.K) * a.T + t;
            w = 1.0f;
        }
        rowi[s] = (uint16_t)row;
        tok[s] = (uint8_t)t;
        wt[s] = w;
    }
    __syncthreads();

    // ---- work
    const int per = a.F / FEW_PIECE, n_pieces = n_list * per;   // pieces of one expert, of all
    const int n_units = gridDim.x * a.share.units;
    auto unit_row = [&](int u) { return (int)((int64_t)u * a.H / n_units); };

    if (warp >= FW_WARPS) {
        // ---- producers: a lane fills ring w stage by stage, its pieces and then its pairs of every unit
        fw_producer_regs();
        const uint64_t policy = l2_policy_evict_first();
        const bool active = fw_put_lane();
        const int w = active ? fw_put_ring() : 0;
        FwPut put(rings, w);
        volatile int* my_piece = slot_piece + w * FW_MAX_STAGES;
        int y = 0, x = a.up.bytes, n = 0, piece = 0;   // the rows and the byte to fill next
        // the rings past the CTA's first share start with a claim of their own as far as there is one
        // for every CTA's
        int claim = w < a.first ? *first_piece + w : n_pieces;
        if (active && w >= a.first && (w - a.first) * (int)gridDim.x < n_pieces - a.first * (int)gridDim.x)
            claim = atomicAdd(a.counters, 1);
        int unit = -1;                                 // output unit (-1: still in pieces)
        const CUtensorMap* map = nullptr;
        FwPairs pr{0, 0};
        auto next_unit = [&]() {   // to the next output unit with something for this ring
            do {
                if (++unit == a.share.units) return false;
                const int u = blockIdx.x * a.share.units + unit;
                y = unit_row(u);
                n = unit_row(u + 1) - y;
                pr.i = 0;
                pr.seek(lst_e, n_list, a.down.n, w);
            } while (n <= 0 || pr.i >= n_list);
            return true;
        };
        auto step = [&]() {
            if (unit < 0) {
                if (x >= a.up.bytes) {
                    piece = claim;
                    if (piece >= n_pieces) {   // the consumer's sign that there is no further piece
                        my_piece[put.slot] = n_pieces;
                        put.mark();
                        return next_unit();
                    }
                    const int i = piece / per, e = lst_e[i], f = (piece - i * per) * FEW_PIECE;
                    x = 0;
                    map = e < a.E ? &maps.up : &maps.up_s;
                    y = (e < a.E ? e : e - a.E) * a.F + f;
                }
                my_piece[put.slot] = piece;
                put.fill(map, x, y, FEW_PIECE * a.up.chunk, policy);
                x += a.up.chunk;
                // the next piece is claimed one stage before it is needed
                if (x >= a.up.bytes) claim = atomicAdd(a.counters, 1);
                return true;
            }
            const int e = lst_e[pr.i], one_less = a.share.rows - n;   // 0 or 1
            // chunk j of the shared expert: columns from j F on (past j's end: the next chunk's weights,
            // which meet activations of zero)
            if (e < a.E)
                put.fill(&maps.down[one_less], pr.k * a.down.chunk, e * a.H + y, n * a.down.chunk, policy);
            else
                put.fill(&maps.down_s[one_less], (e - a.E) * a.F * ES + pr.k * a.down.chunk, y, n * a.down.chunk, policy);
            pr.step(lst_e, n_list, a.down.n, w);
            return pr.i < n_list || next_unit();
        };
        if (!fw_produce(put, active, step, ctx, abort_flag)) fw_settle();
        return;
    }

    // ---- consumers: pieces
    fw_consumer_regs();
    FwTake ring(rings, warp);
    while (true) {
        if (!ring.wait(ctx, abort_flag)) return fw_settle();
        const int piece = slot_piece[warp * FW_MAX_STAGES + ring.slot];
        if (piece >= n_pieces) {
            ring.release();
            break;
        }
        const int i = piece / per, f = (piece - i * per) * FEW_PIECE;
        const int n_tok = lst_n[i];
        const bool ok = n_tok <= 8
                            ? few_up<FMT, 1>(a, ring, lst_e[i], f, n_tok, rowi + i * 16, tok + i * 16, ctx, abort_flag)
                            : few_up<FMT, 2>(a, ring, lst_e[i], f, n_tok, rowi + i * 16, tok + i * 16, ctx, abort_flag);
        if (!ok) return fw_settle();
        __syncwarp();
        if (lane == 0 && !(a.hold && piece == 0)) {
            __threadfence();
            red_release_add(a.counters + 1, 1);
        }
    }

    // ---- output rows, once every piece has reported
    {
        int good = 1;
        if (lane == 0) good = wait_count(a.counters + 1, n_pieces, ctx, abort_flag) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, good, 0)) return fw_settle();
        __syncwarp();
    }
    for (int un = 0; un < a.share.units; ++un) {
        const int u = blockIdx.x * a.share.units + un;
        const int d0 = unit_row(u), n = unit_row(u + 1) - d0;
        float* tot = red.mine(warp);
        for (int j = lane; j < FwRed::kWarp; j += 32) tot[j] = 0.0f;
        __syncwarp();
        if (n > 0) {
            FewDown<FMT> down{a, ring, lst_e, lst_n, rowi, tok, wt, n_list, warp, d0, n, tot, ctx, abort_flag};
            if (!down.run()) return fw_settle();
        }
        if (!red.exchange(ctx, abort_flag)) return fw_settle();
        for (int j = tid; j < n * a.T; j += 32 * FW_WARPS) {
            const int t = j / n, row = j - t * n;
            float o = red.sum(t, row);
            if constexpr (FMT != MOE_BF16) o = __fmul_rn(o, a.h_scale);
            const int64_t at = (int64_t)t * a.H + d0 + row;
            if (a.residual) o = __fadd_rn(o, bf16_bits_to_float(a.residual[at]));
            a.out[at] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
        }
    }
}

// ----------------------------------------------------------------------------- host

static int few_row_bytes(int K, int dtype) { return dtype == MOE_BF16 ? 2 * K : dtype == MOE_FP8_B128 ? (K + 127) / 128 * 128 : K; }

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

template <int FMT>
static cudaError_t launch_layer(const FewMaps& maps, FewArgs& a, int num_sms, const DevCtx& ctx, cudaStream_t stream) {
    const size_t fixed = FwRed::bytes(a.share.units) + few_table_bytes(a.n_list_max);
    a.n_stages = (int)std::min<size_t>(FW_MAX_STAGES, (FW_SMEM - fixed) / FW_WARPS / a.slot_bytes);
    const size_t smem = (size_t)FW_WARPS * a.n_stages * a.slot_bytes + fixed;
    auto k = few_layer_kernel<FMT>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_k(k, dim3(num_sms), dim3(FW_THREADS), smem, stream, maps, a, ctx);
}

cudaError_t launch_few(const moe_dims* d, const uint16_t* x, const uint16_t* wr, const float* bias, const void* w_up,
                       const void* w_down, const void* w_up_s, const void* w_down_s, const moe_fp8_scales* sc,
                       const uint16_t* residual, uint16_t* out, int32_t* idx, float* w, const FewWs& ws, int hold,
                       int num_sms, const DevCtx& ctx, cudaStream_t stream) {
    const bool fp8 = d->expert_dtype != MOE_BF16;
    FewRouterArgs r = {};
    r.x = x;
    r.wr = wr;
    r.bias = bias;
    r.T = (int)d->T;
    r.H = d->H;
    r.E = d->E;
    r.logits = ws.logits;
    r.xq = fp8 ? reinterpret_cast<__half*>(ws.xq) : nullptr;
    r.x_scale = fp8 ? sc->x_scale : 1.0f;
    r.counters = ws.counters;
    cudaError_t e = launch_k(few_router_kernel, dim3(d->E + (fp8 ? r.T : 0)), dim3(FEW_RT), 0, stream, r, ctx);
    if (e != cudaSuccess) return e;

    FewArgs a = {};
    a.x = x;
    a.residual = residual;
    a.out = out;
    a.topk_idx = idx;
    a.topk_w = w;
    a.logits = ws.logits;
    a.act = fp8 ? ws.xq : reinterpret_cast<const uint8_t*>(x);
    a.first = std::min((d->K + d->Fs / d->F) * (d->F / FEW_PIECE) / num_sms, FW_WARPS);
    a.su = fp8 ? sc->w_up_scale : nullptr;
    a.sd = fp8 ? sc->w_down_scale : nullptr;
    a.x_scale = fp8 ? sc->x_scale : 1.0f;
    a.h_scale = fp8 ? sc->h_scale : 1.0f;
    a.ns = d->Fs / d->F;
    a.h = ws.h;
    a.h_lo = d->T * (int64_t)(d->K + a.ns) * d->F * 2;
    a.counters = ws.counters;
    a.T = r.T;
    a.H = d->H;
    a.E = d->E;
    a.K = d->K;
    a.F = d->F;
    const bool block = d->expert_dtype == MOE_FP8_B128;
    a.up = fw_cut(few_row_bytes(d->H, d->expert_dtype), block);
    a.down = fw_cut(few_row_bytes(d->F, d->expert_dtype), block);
    a.share = fw_share(d->H, num_sms);
    a.slot_bytes = (std::max(a.share.rows, FEW_PIECE) * a.up.chunk + 127) / 128 * 128;
    FewMaps maps = {};
    const int ns = a.ns;
    bool ok = fw_map(&maps.up, w_up, (int64_t)d->E * d->F, a.up.bytes, a.up.bytes, a.up.chunk, FEW_PIECE);
    if (ns > 0) ok = ok && fw_map(&maps.up_s, w_up_s, (int64_t)ns * d->F, a.up.bytes, a.up.bytes, a.up.chunk, FEW_PIECE);
    for (int i = 0; i < 2 && a.share.rows > i; ++i)
        ok = ok && fw_map(&maps.down[i], w_down, (int64_t)d->E * d->H, a.down.bytes, a.down.bytes, a.down.chunk,
                          a.share.rows - i);
    for (int i = 0; i < 2 && ns > 0 && a.share.rows > i; ++i)
        ok = ok && fw_map(&maps.down_s[i], w_down_s, d->H, (int64_t)d->Fs * 2, (int64_t)d->Fs * 2, a.down.chunk,
                          a.share.rows - i);
    if (!ok) return cudaErrorInvalidValue;
    a.n_list_max = (int)std::min<int64_t>(d->E, d->T * d->K) + a.ns;
    a.hold = hold;
    switch (d->expert_dtype) {
        case MOE_BF16: return launch_layer<MOE_BF16>(maps, a, num_sms, ctx, stream);
        case MOE_FP8_E4M3: return launch_layer<MOE_FP8_E4M3>(maps, a, num_sms, ctx, stream);
        default: return launch_layer<MOE_FP8_B128>(maps, a, num_sms, ctx, stream);
    }
}

}  // namespace moe
