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
//    further blocks write the E4M3 codes of x.  It zeroes the second kernel's counters.
// 2. few_layer_kernel, persistent, one CTA of eight warps per SM: every CTA ranks the logits itself
//    (the same integers give the same choice everywhere), lists the touched experts, and then its
//    warps stream weights (few.cuh): up pieces (9 or 10 rows of one expert, claimed by single warps),
//    then the CTA's share of the output rows through all touched experts, so that the weighted sum
//    over experts, the residual and the one rounding happen in the CTA that holds them.  A warp
//    without further up pieces fills its ring with down weights while the last pieces report.
//
// Up pieces are claimed from a counter, so those that a warp waits for belong to warps that run and
// that wait for nothing; no CTA needs another to be resident, and every wait is bounded.
//
// Bound: HBM bytes of the touched experts' weights.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "few.cuh"

namespace moe {

constexpr int FEW_RT = 256;          // threads of the router kernel
constexpr int FEW_PQ = 8;            // claimed pieces of a warp: its ring's, and the next one
static_assert(FEW_PQ > FW_MAX_STAGES, "a piece has one stage at least");
constexpr int FEW_ABSENT = 0xFFFF;   // token not routed to the expert

// ----------------------------------------------------------------------------- router

struct FewRouterArgs {
    const uint16_t* x;
    const uint16_t* wr;
    const float* bias;
    int T, H, E;
    long long* logits;   // [T][E], units of 2^-40
    uint8_t* xq;         // E4M3 codes of x [T][H], or null
    float x_scale;
    int* counters;       // [2]: piece claims, piece reports
};

__global__ void __launch_bounds__(FEW_RT) few_router_kernel(FewRouterArgs a, DevCtx ctx) {
    pdl_enter();
    __shared__ long long s_l[kFewMaxTokens][8];
    __shared__ float s_x[kFewMaxTokens][8], s_w[8];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int nv = a.H / 8;
    if ((int)blockIdx.x >= a.E) {   // E4M3 codes of one token
        const int t = blockIdx.x - a.E;
        const uint4* xr = reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.H);
        for (int v = tid; v < nv; v += FEW_RT) {
            const uint4 p = xr[v];
            const uint32_t w[4] = {p.x, p.y, p.z, p.w};
            uint32_t c[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float f = __uint_as_float((j & 1) ? (w[j / 2] & 0xFFFF0000u) : (w[j / 2] << 16));
                c[j / 4] |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(f, a.x_scale), __NV_SATFINITE, __NV_E4M3)
                            << (8 * (j % 4));
            }
            reinterpret_cast<uint2*>(a.xq + (int64_t)t * a.H)[v] = make_uint2(c[0], c[1]);
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
    const uint8_t* act;         // up operand rows: x, or its E4M3 codes
    const uint8_t* w_up;
    const uint8_t* w_down;
    const uint8_t* w_up_s;      // shared expert (bf16): [ns F][H]
    const uint8_t* w_down_s;    // [H][ns F]
    const float* su;            // E4M3: [E]; B128: [E][F][kbu]
    const float* sd;            // E4M3: [E]; B128: [E][H][kbd]
    float x_scale, h_scale;
    uint8_t* h;                 // bf16: high parts [rows][F] then low parts; else codes [rows][F]
    int64_t h_lo;               // bf16: bytes from a high part to its low part
    int* counters;
    int T, H, E, K, F, ns;
    FwCut up, down;
    FwShare share;              // of the output rows; its `rows` also bound an up piece
    int stride, slot_bytes, n_stages;
    int n_list_max;
    int hold;                   // test hook: up piece 0 never reports
};

// shared memory after the rings: reduction buffers | wt [n][16] f32 | lst_e [n] i32 | rowi [n][16] u16 |
// emask [256] i32 | slot [256] i32 | sel_w [16][16] f32 | sel_e [16][16] i32 | barriers | piece queues | flags
__host__ __device__ inline size_t few_table_bytes(int n_list) {
    return (size_t)n_list * (64 + 4 + 32) + 16 + 4 * 1024 + (FW_WARPS * FW_MAX_STAGES + 1) * 8 + FW_WARPS * FEW_PQ * 4 +
           16;
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

template <int FMT, int NT>
__global__ void __launch_bounds__(FW_THREADS, 1) few_layer_kernel(FewArgs a, DevCtx ctx) {
    constexpr bool BF16 = FMT == MOE_BF16, BLOCK = FMT == MOE_FP8_B128;
    constexpr int ES = BF16 ? 2 : 1;
    extern __shared__ __align__(1024) uint8_t few_smem[];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    uint8_t* p = few_smem + (size_t)FW_WARPS * a.n_stages * a.slot_bytes;
    FwRed<NT> red;
    red.buf = reinterpret_cast<float*>(p);
    p += 2 * FwRed<NT>::kFloats * sizeof(float);
    float* wt = reinterpret_cast<float*>(p);
    p += (size_t)a.n_list_max * 64;
    uint16_t* rowi = reinterpret_cast<uint16_t*>(p);
    p += (size_t)a.n_list_max * 32;
    int* lst_e = reinterpret_cast<int*>(p);
    p += ((size_t)a.n_list_max * 4 + 15) / 16 * 16;
    int* emask = reinterpret_cast<int*>(p);
    p += 1024;
    int* eslot = reinterpret_cast<int*>(p);
    p += 1024;
    float(*sel_w)[16] = reinterpret_cast<float(*)[16]>(p);
    p += 1024;
    int(*sel_e)[16] = reinterpret_cast<int(*)[16]>(p);
    p += 1024;
    uint64_t* bars = reinterpret_cast<uint64_t*>(p);
    uint64_t* rbar = bars + FW_WARPS * FW_MAX_STAGES;
    int* pieces = reinterpret_cast<int*>(rbar + 1) + warp * FEW_PQ;
    volatile int* abort_flag = reinterpret_cast<int*>(rbar + 1) + FW_WARPS * FEW_PQ;
    int* n_touched = const_cast<int*>(abort_flag) + 1;
    red.bar = smem_u32(rbar);
    red.turn = 0;
    FwRing ring;
    ring.base = smem_u32(few_smem) + warp * a.n_stages * a.slot_bytes;
    ring.bars = smem_u32(bars + warp * FW_MAX_STAGES);
    ring.slot_bytes = a.slot_bytes;
    ring.stride = a.stride;
    ring.n = a.n_stages;
    ring.put = ring.take = 0;
    ring.parity = 0;
    ring.policy = l2_policy_evict_first();

    if (lane == 0)
        for (int s = 0; s < a.n_stages; ++s) mbar_init(ring.bars + 8 * s, 1);
    if (tid == 0) {
        mbar_init(smem_u32(rbar), FW_WARPS);
        *abort_flag = 0;
    }
    if (lane == 0) fence_mbar_init();
    for (int i = tid; i < 256; i += FW_THREADS) emask[i] = 0;
    __syncthreads();
    pdl_enter();

    // ---- the routing, the same in every CTA
    for (int t = warp; t < a.T; t += FW_WARPS) {
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
    if (warp == 0) {   // the touched experts, ascending
        int n = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const bool on = e < a.E && emask[e] != 0;
            const uint32_t m = __ballot_sync(0xffffffffu, on);
            if (on) {
                const int i = n + __popc(m & ((1u << lane) - 1u));
                eslot[e] = i;
                lst_e[i] = e;
            }
            n += __popc(m);
        }
        if (lane < a.ns) lst_e[n + lane] = a.E + lane;
        if (lane == 0) *n_touched = n;
    }
    __syncthreads();
    const int n_routed = *n_touched, n_list = n_routed + a.ns;
    for (int i = tid; i < n_list * 16; i += FW_THREADS) {
        const int j = i / 16 - n_routed, t = i % 16;   // j >= 0: chunk j of the shared expert, every token
        const bool on = j >= 0 && t < a.T;
        rowi[i] = (uint16_t)(on ? a.T * a.K + j * a.T + t : FEW_ABSENT);
        wt[i] = on ? 1.0f : 0.0f;
    }
    __syncthreads();
    for (int i = tid; i < a.T * a.K; i += FW_THREADS) {
        const int t = i / a.K, k = i % a.K;
        const int s = eslot[sel_e[t][k]] * 16 + t;
        rowi[s] = (uint16_t)i;
        wt[s] = sel_w[t][k];
    }
    __syncthreads();

    // ---- work: each expert's F rows in `per` equal pieces, as many pieces in all as fill a whole
    // number of rounds over the grid's warps
    const int n_warps = gridDim.x * FW_WARPS;
    const int rounds = (int)(((int64_t)n_list * a.F + (int64_t)n_warps * a.share.rows - 1) / ((int64_t)n_warps * a.share.rows));
    const int per = min(a.F, max(rounds * n_warps / n_list, (a.F + a.share.rows - 1) / a.share.rows));
    const int n_pieces = n_list * per;
    auto piece_row = [&](int j) { return (int)((int64_t)j * a.F / per); };
    // output rows: unit u's group starts at
    const int n_groups = gridDim.x * a.share.units * a.share.groups;
    const int my_group = warp * a.share.groups / FW_WARPS, gw = FW_WARPS / a.share.groups, wk = warp % gw;
    auto group_row = [&](int u, int grp) { return (int)((int64_t)(u * a.share.groups + grp) * a.H / n_groups); };

    // ---- filling the ring, stage by stage: this warp's up pieces, then its pairs of every unit
    const uint8_t* f_src = nullptr;      // the rows being filled, ld apart
    int64_t f_ld = 0;
    int f_n = 0, f_k = a.up.n;           // their number, and the next chunk
    int f_queue = 0, claim = 0;          // pieces queued so far; the next piece (lane 0)
    int f_unit = -1, f_d0 = 0;           // the output unit being filled (-1: still in up pieces), its first row
    FwPairs f_pair{0, 0};
    int f_i = -1;                        // the expert that f_src belongs to
    if (lane == 0) claim = atomicAdd(a.counters, 1);
    auto next_unit = [&]() {
        ++f_unit;
        f_i = -1;
        f_pair.i = 0;
        f_pair.seek(n_list, a.down.n, wk, gw);
        const int u = blockIdx.x * a.share.units + f_unit;
        f_d0 = group_row(u, my_group);
        f_n = group_row(u, my_group + 1) - f_d0;
    };
    auto fill_next = [&]() {
        if (f_unit < 0) {
            if (f_k == a.up.n) {
                const int piece = __shfl_sync(0xffffffffu, claim, 0);
                if (lane == 0) pieces[f_queue % FEW_PQ] = piece;
                ++f_queue;
                __syncwarp();
                if (piece < n_pieces) {
                    const int i = piece / per, j = piece - i * per, f = piece_row(j);
                    f_n = piece_row(j + 1) - f;
                    f_k = 0;
                    const int e = lst_e[i];
                    f_src = e < a.E ? a.w_up + ((int64_t)e * a.F + f) * a.up.bytes
                                    : a.w_up_s + ((int64_t)(e - a.E) * a.F + f) * a.up.bytes;
                } else {
                    next_unit();
                }
            }
            if (f_unit < 0) {
                ring.fill(f_src + f_k * a.up.chunk, a.up.bytes, f_n,
                          (uint32_t)min(a.up.chunk, a.up.bytes - f_k * a.up.chunk));
                // the next piece is claimed one stage before it is needed
                if (++f_k == a.up.n && lane == 0) claim = atomicAdd(a.counters, 1);
                return;
            }
        }
        while (f_unit < a.share.units) {
            if (f_pair.i < n_list && f_n > 0) {
                if (f_pair.i != f_i) {
                    f_i = f_pair.i;
                    const int e = lst_e[f_i];
                    f_ld = e < a.E ? (int64_t)a.down.bytes : (int64_t)a.ns * a.F * ES;
                    f_src = e < a.E ? a.w_down + ((int64_t)e * a.H + f_d0) * f_ld
                                    : a.w_down_s + (int64_t)f_d0 * f_ld + (int64_t)(e - a.E) * a.F * ES;
                }
                ring.fill(f_src + f_pair.k * a.down.chunk, f_ld, f_n,
                          (uint32_t)min(a.down.chunk, a.down.bytes - f_pair.k * a.down.chunk));
                f_pair.step(n_list, a.down.n, wk, gw);
                return;
            }
            next_unit();
        }
    };
    for (int s = 0; s < a.n_stages; ++s) fill_next();

    const int g = lane / 4, q = lane % 4;
    // ---- up pieces
    for (int c_queue = 0;; ++c_queue) {
        const int piece = pieces[c_queue % FEW_PQ];
        if (piece >= n_pieces) break;
        const int i = piece / per, f = piece_row(piece % per), n = piece_row(piece % per + 1) - f;
        const int e = lst_e[i];
        FwRows<NT> act;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            act.on[nt] = rowi[i * 16 + nt * 8 + g] != FEW_ABSENT;
            act.p[nt] = a.act + (int64_t)(nt * 8 + g) * a.H * ES + q * 16;
        }
        const int kb = a.up.bytes / 128;
        const float* ws0 = BLOCK ? a.su + ((int64_t)e * a.F + f + min(g, n - 1)) * kb : nullptr;
        const float* ws1 = BLOCK ? a.su + ((int64_t)e * a.F + f + min(g + 8, n - 1)) * kb : nullptr;
        float acc[NT][4] = {};
        for (int k = 0; k < a.up.n; ++k) {
            const int c0 = k * a.up.chunk, bytes = min(a.up.chunk, a.up.bytes - c0);
            auto load = [&](auto& v, int seg0, int n_seg) {
                const int off = c0 + seg0 * FW_SEG;
                fw_load(v, act, off, n_seg, a.H * ES, 0);
                if constexpr (BLOCK) {
#pragma unroll
                    for (int s = 0; s < FW_GROUP / 2; ++s)
                        if (2 * s < n_seg) {
                            v.ws[s][0] = __ldg(ws0 + off / 128 + s);
                            v.ws[s][1] = __ldg(ws1 + off / 128 + s);
                        }
                }
            };
            if (!fw_stage<BF16, NT, false, BLOCK, false>(acc, ring, n, bytes, load, ctx, abort_flag)) return fw_settle();
            fill_next();
        }
        const float sc = BF16 ? 1.0f : BLOCK ? a.x_scale : __fmul_rn(a.su[e], a.x_scale);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int row = g + 8 * (c / 2);
                const int hr = rowi[i * 16 + nt * 8 + 2 * q + c % 2];
                if (hr == FEW_ABSENT || row >= n) continue;
                float z = acc[nt][c];
                if constexpr (!BF16) z = __fmul_rn(z, sc);
                const float h = z <= 0.0f ? 0.0f : __fmul_rn(z, z);   // a NaN stays one
                const int64_t o = (int64_t)hr * a.F + f + row;
                if constexpr (BF16) {
                    // h as the sum of two bf16, 16 bits of it: one alone would add a second rounding
                    // of the output's size
                    const __nv_bfloat16 hi = __float2bfloat16_rn(h);
                    const float top = __bfloat162float(hi);
                    reinterpret_cast<__nv_bfloat16*>(a.h)[o] = hi;
                    reinterpret_cast<__nv_bfloat16*>(a.h + a.h_lo)[o] =
                        __float2bfloat16_rn(top < __uint_as_float(0x7f800000u) ? __fsub_rn(h, top) : 0.0f);
                } else {
                    a.h[o] = (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(h, a.h_scale), __NV_SATFINITE, __NV_E4M3);
                }
            }
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
    const int kb = a.down.bytes / 128;
    for (int un = 0; un < a.share.units; ++un) {
        const int u = blockIdx.x * a.share.units + un;
        const int d0 = group_row(u, my_group), n = group_row(u, my_group + 1) - d0;
        float tot[NT][4] = {};
        FwPairs pr{0, 0};
        pr.seek(n_list, a.down.n, wk, gw);
        while (n > 0 && pr.i < n_list) {
            const int i = pr.i, e = lst_e[i];
            FwRows<NT> act;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = rowi[i * 16 + nt * 8 + g];
                act.on[nt] = r != FEW_ABSENT;
                act.p[nt] = a.h + (int64_t)r * a.F * ES + q * 16;
            }
            const float* ws0 = BLOCK ? a.sd + ((int64_t)e * a.H + d0 + min(g, n - 1)) * kb : nullptr;
            const float* ws1 = BLOCK ? a.sd + ((int64_t)e * a.H + d0 + min(g + 8, n - 1)) * kb : nullptr;
            float acc[NT][4] = {};
            for (; pr.i == i; pr.step(n_list, a.down.n, wk, gw)) {
                const int c0 = pr.k * a.down.chunk, bytes = min(a.down.chunk, a.down.bytes - c0);
                auto load = [&](auto& v, int seg0, int n_seg) {
                    const int off = c0 + seg0 * FW_SEG;
                    fw_load(v, act, off, n_seg, a.F * ES, a.h_lo);
                    if constexpr (BLOCK) {
#pragma unroll
                        for (int s = 0; s < FW_GROUP / 2; ++s)
                            if (2 * s < n_seg) {
                                v.ws[s][0] = __ldg(ws0 + off / 128 + s);
                                v.ws[s][1] = __ldg(ws1 + off / 128 + s);
                            }
                    }
                };
                if (!fw_stage<BF16, NT, BF16, BLOCK, false>(acc, ring, n, bytes, load, ctx, abort_flag))
                    return fw_settle();
                fill_next();
            }
            // this warp's part of the expert's output, weighted, for the tokens routed to it only
            // (another expert's infinity must not reach a token as 0 * inf)
            const float sc = FMT == MOE_FP8_E4M3 ? a.sd[e] : 1.0f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int t = i * 16 + nt * 8 + 2 * q + c;
                    if (rowi[t] == FEW_ABSENT) continue;
                    const float w = wt[t] * sc;
                    tot[nt][c] = __fmaf_rn(w, acc[nt][c], tot[nt][c]);
                    tot[nt][c + 2] = __fmaf_rn(w, acc[nt][c + 2], tot[nt][c + 2]);
                }
        }
        if (!red.exchange(tot, warp, ctx, abort_flag)) return fw_settle();
        const int r0 = group_row(u, 0), rows = group_row(u, a.share.groups) - r0;
        const int half = group_row(u, 1) - r0;   // rows of the first group
        for (int j = tid; j < rows * a.T; j += FW_THREADS) {
            const int t = j / rows, row = j - t * rows;
            float o = row < half ? red.sum(row, t, 0, gw) : red.sum(row - half, t, gw, gw);
            if constexpr (!BF16) o = __fmul_rn(o, a.h_scale);
            const int64_t at = (int64_t)t * a.H + r0 + row;
            if (a.residual) o = __fadd_rn(o, bf16_bits_to_float(a.residual[at]));
            a.out[at] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
        }
    }
}

// ----------------------------------------------------------------------------- host

static int few_row_bytes(int K, int dtype) { return dtype == MOE_BF16 ? 2 * K : dtype == MOE_FP8_B128 ? (K + 127) / 128 * 128 : K; }

template <int FMT, int NT>
static cudaError_t launch_layer(FewArgs& a, int num_sms, const DevCtx& ctx, cudaStream_t stream) {
    const size_t fixed = 2 * FwRed<NT>::kFloats * sizeof(float) + few_table_bytes(a.n_list_max);
    a.n_stages = (int)std::min<size_t>(FW_MAX_STAGES, (FW_SMEM - fixed) / FW_WARPS / a.slot_bytes);
    const size_t smem = (size_t)FW_WARPS * a.n_stages * a.slot_bytes + fixed;
    auto k = few_layer_kernel<FMT, NT>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_k(k, dim3(num_sms), dim3(FW_THREADS), smem, stream, a, ctx);
}

template <int FMT>
static cudaError_t launch_fmt(FewArgs& a, int num_sms, const DevCtx& ctx, cudaStream_t stream) {
    return a.T <= 8 ? launch_layer<FMT, 1>(a, num_sms, ctx, stream) : launch_layer<FMT, 2>(a, num_sms, ctx, stream);
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
    r.xq = fp8 ? ws.xq : nullptr;
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
    a.w_up = static_cast<const uint8_t*>(w_up);
    a.w_down = static_cast<const uint8_t*>(w_down);
    a.w_up_s = static_cast<const uint8_t*>(w_up_s);
    a.w_down_s = static_cast<const uint8_t*>(w_down_s);
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
    const int unit = d->expert_dtype == MOE_FP8_B128 ? 128 : FW_SEG;
    a.up = fw_cut(few_row_bytes(d->H, d->expert_dtype), unit);
    a.down = fw_cut(few_row_bytes(d->F, d->expert_dtype), unit);
    a.share = fw_share(d->H, num_sms);
    a.share.rows = std::max(a.share.rows, 8);   // a narrow output still leaves up pieces of eight rows
    a.stride = fw_row_stride(std::max(a.up.chunk, a.down.chunk));
    a.slot_bytes = a.share.rows * a.stride;
    a.n_list_max = (int)std::min<int64_t>(d->E, d->T * d->K) + a.ns;
    a.hold = hold;
    switch (d->expert_dtype) {
        case MOE_BF16: return launch_fmt<MOE_BF16>(a, num_sms, ctx, stream);
        case MOE_FP8_E4M3: return launch_fmt<MOE_FP8_E4M3>(a, num_sms, ctx, stream);
        default: return launch_fmt<MOE_FP8_B128>(a, num_sms, ctx, stream);
    }
}

}  // namespace moe
