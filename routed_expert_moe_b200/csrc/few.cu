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
// 2. few_layer_kernel, persistent, one CTA per SM: every CTA ranks the logits itself (the same
//    integers give the same choice everywhere) and lists the touched experts; then the CTAs claim units
//    of 128 weight rows (up units of all entries, then down units) from a counter and multiply them on
//    the tensor cores: weights as the 128-row operand through a TMA ring, the tokens as 16 columns.
//      up:   columns are all T tokens (x itself, no gather); the epilogue keeps those that the entry has
//      down: columns are the entry's rows of h (the rows that follow, of other entries, are not used)
//    A down unit waits until its entry's up units have reported.  The warp that finishes the last
//    entry of 32 output rows sums them over the experts, with the residual, in one rounding.
//
// Units are claimed in list order, so those that a unit waits for belong to CTAs that run; no CTA
// needs another to be resident, and every wait is bounded.
//
// Bound: HBM bytes of the touched experts' weights, at one to three tokens the fixed steps around them:
// two launches, the choice of experts (3 us), units that are one SM's work alone.  128-row
// units leave SMs without work at one or two tokens (87 up units at one token of the full sizes), which
// costs little: a load-only kernel takes 12.3 us for those 60 MB (bf16) and 8.2 for 30 MB (E4M3), launch
// included, on 74, 87, 126 and 148 SMs alike.  Units of 64 rows while there are few were slower (bf16, 3
// tokens: 92 against 72 us): a stage of half the weights takes the same products.
//
// H = 2688, E = 128, K = 6, F = 1856, us, against moe_forward, and what the touched weights take at the
// rate of a copy (experts chosen nearly evenly: 68 of 128 by 16 tokens):
//   tokens       1                   4                   8                     16
//   bf16    40 / 53 / 19        83 / 96 / 69       139 / 145 / 129       223 / 219 / 214
//   E4M3    36 / 42 /  9        52 / 65 / 35        83 /  90 /  64       127 / 128 / 107
//   B128    37 / 45 / 10        56 / 71 / 36        86 /  97 /  68       131 / 135 / 112
#include <algorithm>
#include <climits>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int FEW_RT = 512;          // threads of the router kernel
constexpr int FEW_RW = FEW_RT / 32;

// ----------------------------------------------------------------------------- router

struct FewRouterArgs {
    const uint16_t* x;
    const uint16_t* wr;
    const float* bias;
    int T, H, E;
    long long* logits;   // [T][E], units of 2^-40
    uint8_t* xq;         // E4M3 codes of x [T][H], or null
    float x_scale;
    int* counters;       // of the second kernel: zeroed here
    int n_counters;
};

__global__ void __launch_bounds__(FEW_RT) few_router_kernel(FewRouterArgs a, DevCtx ctx) {
    pdl_enter();
    __shared__ long long s_l[kFewMaxTokens][FEW_RW];
    __shared__ float s_x[kFewMaxTokens][FEW_RW], s_w[FEW_RW];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int nv = a.H / 8;
    if ((int)blockIdx.x >= a.E) {   // one token's E4M3 codes
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
    for (int i = e * FEW_RT + tid; i < a.n_counters; i += a.E * FEW_RT) a.counters[i] = 0;
    // a warp takes one token over 1 / parts of H
    const int parts = a.T == 1 ? 16 : a.T == 2 ? 8 : a.T <= 4 ? 4 : a.T <= 8 ? 2 : 1;
    const int part = warp % parts, t = warp / parts;
    const uint4* wv = reinterpret_cast<const uint4*>(a.wr + (int64_t)e * a.H);
    if (t < a.T) {
        const uint4* xv = reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.H);
        long long acc = 0;
        float xs = 0.0f, ws = 0.0f, big = 0.0f;
        // A product p, |p| < 32, as two integers by fp32 additions alone (a conversion to 64 bits takes
        // 16 times as long): adding kHi rounds it to the grid 2^-17, what is left over is exact and at
        // most 2^-18, and adding kLo rounds that to the grid 2^-40, ties to even like the sum of both,
        // since the first part is an even multiple of 2^-40.  The bits of the two sums count grid steps
        // from those of the constants.
        constexpr float kHi = 96.0f, kLo = 1.5f * 0x1p-17f;
        constexpr int B = 4;   // vectors whose loads are under way together
        for (int v0 = part * 32 + lane; v0 < nv; v0 += 32 * parts * B) {
            uint4 pv[B], rv[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int v = v0 + 32 * parts * b;
                pv[b] = rv[b] = make_uint4(0, 0, 0, 0);
                if (v < nv) {
                    pv[b] = xv[v];
                    rv[b] = wv[v];
                }
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const uint32_t pp[4] = {pv[b].x, pv[b].y, pv[b].z, pv[b].w}, rr[4] = {rv[b].x, rv[b].y, rv[b].z, rv[b].w};
                uint32_t n_hi = 0, n_lo = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float f = __uint_as_float((j & 1) ? (pp[j / 2] & 0xFFFF0000u) : (pp[j / 2] << 16));
                    const float h = __uint_as_float((j & 1) ? (rr[j / 2] & 0xFFFF0000u) : (rr[j / 2] << 16));
                    const float p = __fmul_rn(f, h);   // exact
                    const float hi = __fadd_rn(p, kHi);
                    const float lo = __fadd_rn(__fsub_rn(p, __fsub_rn(hi, kHi)), kLo);
                    n_hi += __float_as_uint(hi);
                    n_lo += __float_as_uint(lo);
                    big = fmaxf(big, fabsf(p));
                    xs = __fmaf_rn(f, f, xs);
                    ws = __fmaf_rn(h, h, ws);
                }
                acc += ((long long)(int)(n_hi - 8u * __float_as_uint(kHi)) << 23) + (int)(n_lo - 8u * __float_as_uint(kLo));
            }
        }
        if (!__all_sync(0xffffffffu, big < 32.0f && xs < 3.0e38f && ws < 3.0e38f)) {
            // a product outside the range of the two roundings above
            acc = 0;
            for (int v = part * 32 + lane; v < nv; v += 32 * parts) {
                const uint4 p4 = xv[v], r4 = wv[v];
                const uint32_t pp[4] = {p4.x, p4.y, p4.z, p4.w}, rr[4] = {r4.x, r4.y, r4.z, r4.w};
                for (int j = 0; j < 8; ++j) {
                    const float f = __uint_as_float((j & 1) ? (pp[j / 2] & 0xFFFF0000u) : (pp[j / 2] << 16));
                    const float h = __uint_as_float((j & 1) ? (rr[j / 2] & 0xFFFF0000u) : (rr[j / 2] << 16));
                    acc += __float2ll_rn(__fmul_rn(__fmul_rn(f, h), 0x1p40f));
                }
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

constexpr int FL_THREADS = 384;     // weights, two of products, columns, two sets of four of the epilogue; all route
constexpr int FL_MMA = 2;           // warps that issue products: of the even and of the odd stages
constexpr int FL_BM = 128;          // weight rows per unit
constexpr int FL_KB = 128;          // bytes of K per stage (E4M3: one scale block)
constexpr int FL_A = FL_BM * FL_KB;
constexpr int FL_N = 16;            // token columns
constexpr int FL_B = FL_N * FL_KB;
constexpr int FL_UQ = 4;            // unit queue slots
constexpr int FL_MAX_STAGES = 12;
// Bytes of each shared matrix that are fetched into L2 while the routing is found.
constexpr int64_t kFewWarmBytes = (int64_t)24 << 20;
static_assert(kFewMaxTokens == FL_N, "a token per column");

template <int FMT>
struct FlShape {
    static constexpr bool BF16 = FMT == MOE_BF16, BLOCK = FMT == MOE_FP8_B128;
    static constexpr int kStage = FL_A + (BF16 ? 2 : 1) * FL_B;   // bf16: low parts of h beside the high ones
    // TMEM results: of a scale block, of a unit.  Each is kept as several sums: instructions that add to
    // the same columns wait for one another, and the two issuing threads are not ordered.  bf16: 32
    // columns each, the second 16 for the low parts of h.
    static constexpr int kCols = BF16 ? 2 * FL_N : FL_N;
    static constexpr int kSums = BLOCK ? 2 : 2 * FL_MMA;
    static constexpr int kSlots = BLOCK ? 8 : 1;   // of each set of epilogue warps
    static constexpr int kTmem = 2 * kSlots * kSums * kCols;
};

// Weights in boxes of 128 and of 64 rows (the last rows of an expert), tokens and h in boxes of 16.
struct FewMaps {
    CUtensorMap up128, up64, down128, down64, ups128, ups64, downs128, downs64, x, h;
};

struct FewArgs {
    const uint16_t* residual;   // or null
    uint16_t* out;
    int32_t* topk_idx;          // or null
    float* topk_w;              // or null
    const long long* logits;
    const float* su;            // E4M3: [E]; B128: [E][F][k_up]
    const float* sd;            // E4M3: [E]; B128: [E][H][k_down]
    float x_scale, h_scale;
    uint8_t* h;                 // [rows][F] in list order: E4M3 codes; bf16 high parts, then all low parts
    float* y;                   // [T*K + ns*T][H]: expert outputs of assignment t*K + k, then shared chunks
    int* counters;              // claim | reports per entry [n_list_max] | entries done per 32 output rows
    const uint8_t* warm[2];     // shared expert: weights to fetch into L2 while the routing is found
    int64_t warm_bytes;         // of each
    int T, H, E, K, F, ns;
    int k_up, k_down;           // stages per unit
    int m_up, m_down;           // units per entry
    int n_stages, n_list_max;
    int hold;                   // test hook: the first up unit never reports
};

// shared memory after the ring: barriers | queue, flags | lst_e, lst_mask, lst_off [n] i32 | rowi [n][16] u16 |
// emask, eslot [256] i32 | sel_w [16][16] f32 | sel_e [16][16] i32
__host__ __device__ inline size_t few_table_bytes(int n_list) {
    return (2 * FL_MAX_STAGES + 2 * 16 + FL_MMA + 2 * FL_UQ) * 8 + (FL_UQ + 4) * 4 + (size_t)n_list * (3 * 4 + 32) + 4 * 1024 + 16;
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

__device__ __forceinline__ void fl_ld16(uint32_t taddr, uint32_t (&v)[FL_N]) {   // no wait
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

// This lane's row of a result: its sums added up, for a down unit of bf16 with those of the low parts.
// one: a unit of a single stage, whose other sums were not written.
template <int FMT>
__device__ __forceinline__ void fl_read(uint32_t addr, bool down, bool one, float (&z)[FL_N]) {
    using S = FlShape<FMT>;
    uint32_t p[S::kSums][FL_N];
#pragma unroll
    for (int s = 0; s < S::kSums; ++s) fl_ld16(addr + s * S::kCols, p[s]);
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int c = 0; c < FL_N; ++c) {
        z[c] = __uint_as_float(p[0][c]);
#pragma unroll
        for (int s = 1; s < S::kSums; ++s)
            if (s < 2 || !one) z[c] += __uint_as_float(p[s][c]);
    }
    if (S::BF16 && down) {
#pragma unroll
        for (int s = 0; s < S::kSums; ++s) fl_ld16(addr + s * S::kCols + FL_N, p[s]);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int c = 0; c < FL_N; ++c)
#pragma unroll
            for (int s = 0; s < S::kSums; ++s)
                if (s < 2 || !one) z[c] += __uint_as_float(p[s][c]);
    }
}

// out[t][r .. r + 3] for t = t0, t0 + 4, ..: the weighted sum over the experts in the order of the token's
// choice, the shared chunks, the residual, one rounding.  What this takes is reads of L2 one after the
// other, so eight terms of two tokens are under way together.
__device__ __forceinline__ void fl_combine(const FewArgs& a, const float (*sel_w)[16], int r, int t0) {
    if (r >= a.H) return;   // H is a multiple of 16
    constexpr int KB = 8;
    const int terms = a.K + a.ns;
    for (; t0 < a.T; t0 += 8) {
        float4 o[2] = {};
        for (int k0 = 0; k0 < terms; k0 += KB) {
            float4 v[2][KB];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    const int t = t0 + 4 * i, k = k0 + j;
                    const int64_t row = k < a.K ? (int64_t)t * a.K + k : (int64_t)a.T * k + t;
                    if (t < a.T && k < terms) v[i][j] = __ldcg(reinterpret_cast<const float4*>(a.y + row * a.H + r));
                }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    const int t = t0 + 4 * i, k = k0 + j;
                    if (t >= a.T || k >= terms) continue;
                    const float w = k < a.K ? sel_w[t][k] : 1.0f;
                    o[i].x = __fmaf_rn(w, v[i][j].x, o[i].x);
                    o[i].y = __fmaf_rn(w, v[i][j].y, o[i].y);
                    o[i].z = __fmaf_rn(w, v[i][j].z, o[i].z);
                    o[i].w = __fmaf_rn(w, v[i][j].w, o[i].w);
                }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = t0 + 4 * i;
            if (t >= a.T) continue;
            const int64_t at = (int64_t)t * a.H + r;
            if (a.residual) {
                const uint2 s = *reinterpret_cast<const uint2*>(a.residual + at);
                o[i].x = __fadd_rn(o[i].x, __uint_as_float(s.x << 16));
                o[i].y = __fadd_rn(o[i].y, __uint_as_float(s.x & 0xFFFF0000u));
                o[i].z = __fadd_rn(o[i].z, __uint_as_float(s.y << 16));
                o[i].w = __fadd_rn(o[i].w, __uint_as_float(s.y & 0xFFFF0000u));
            }
            const __nv_bfloat162 lo = __floats2bfloat162_rn(o[i].x, o[i].y), hi = __floats2bfloat162_rn(o[i].z, o[i].w);
            *reinterpret_cast<uint2*>(a.out + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
    }
}

// The stage of K that a unit begins with.  Every CTA reads the same columns (x, or one entry's rows of
// h): in step, all of them would ask one L2 slice for the same lines.  It goes by expert and block alone,
// so that a row's sum does not hang on the batch.
__device__ __forceinline__ int fl_first(int e, int blk, int k_stages) { return (e * 5 + blk * 11) % k_stages; }

template <int FMT>
__global__ void __launch_bounds__(FL_THREADS, 1)
    few_layer_kernel(const __grid_constant__ FewMaps maps, const __grid_constant__ FewArgs a, DevCtx ctx) {
    using S = FlShape<FMT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const int NS = a.n_stages;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + (size_t)NS * S::kStage);
    uint64_t* empty = full + FL_MAX_STAGES;
    uint64_t* rfull = empty + FL_MAX_STAGES;   // TMEM results
    uint64_t* rempty = rfull + 16;
    uint64_t* drain = rempty + 16;
    uint64_t* uq_full = drain + FL_MMA;
    uint64_t* uq_empty = uq_full + FL_UQ;
    volatile int* uq = reinterpret_cast<volatile int*>(uq_empty + FL_UQ);
    volatile int* abort_flag = uq + FL_UQ;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(const_cast<int*>(abort_flag + 1));
    int* n_touched = reinterpret_cast<int*>(tmem_holder + 1);
    float(*sel_w)[16] = reinterpret_cast<float(*)[16]>(n_touched + 2);
    int(*sel_e)[16] = reinterpret_cast<int(*)[16]>(sel_w + 16);
    int* emask = &sel_e[16][0];
    int* eslot = emask + 256;
    int* lst_e = eslot + 256;
    int* lst_mask = lst_e + a.n_list_max;
    int* lst_off = lst_mask + a.n_list_max;
    uint16_t* rowi = reinterpret_cast<uint16_t*>(lst_off + a.n_list_max);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int p = 0; p < 2 * S::kSlots; ++p) {
            mbar_init(smem_u32(&rfull[p]), S::BLOCK ? 1 : FL_MMA);
            mbar_init(smem_u32(&rempty[p]), 4);
        }
        for (int m = 0; m < FL_MMA; ++m) mbar_init(smem_u32(drain + m), 1);
        for (int q = 0; q < FL_UQ; ++q) {
            mbar_init(smem_u32(&uq_full[q]), 1);
            mbar_init(smem_u32(&uq_empty[q]), 1 + FL_MMA + 8);   // columns, products, epilogue warps
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.up128);
        tma_prefetch_desc(&maps.down128);
        tma_prefetch_desc(&maps.x);
        tma_prefetch_desc(&maps.h);
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_holder), S::kTmem);
    if (warp == 2 && a.warm_bytes > 0) {
        // weights are inputs that no kernel before this one writes, and a prefetch changes no data
        constexpr int64_t piece = 16 * 1024;
        const int64_t n = (a.warm_bytes + piece - 1) / piece;
        for (int64_t i = (int64_t)blockIdx.x * 32 + lane; i < 2 * n; i += (int64_t)gridDim.x * 32) {
            const int64_t off = (i >= n ? i - n : i) * piece;
            bulk_prefetch_l2(a.warm[i >= n] + off, (uint32_t)min(piece, a.warm_bytes - off));
        }
    }
    for (int i = tid; i < 256; i += FL_THREADS) emask[i] = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    pdl_enter();

    // ---- the routing, the same in every CTA: a warp per token
    for (int t = warp; t < a.T; t += FL_THREADS / 32) {
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
        int n = 0, off = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int mask = e < a.E ? emask[e] : 0;
            const uint32_t m = __ballot_sync(0xffffffffu, mask != 0);
            int pre = __popc(mask);   // rows of h before this expert's: an inclusive scan
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, pre, d);
                if (lane >= d) pre += v;
            }
            if (mask) {
                const int i = n + __popc(m & ((1u << lane) - 1u));
                eslot[e] = i;
                lst_e[i] = e;
                lst_mask[i] = mask;
                lst_off[i] = off + pre - __popc(mask);
            }
            off += __shfl_sync(0xffffffffu, pre, 31);
            n += __popc(m);
        }
        if (lane < a.ns) {
            lst_e[n + lane] = a.E + lane;
            lst_mask[n + lane] = (1 << a.T) - 1;
            lst_off[n + lane] = a.T * (a.K + lane);
        }
        if (lane == 0) *n_touched = n;
    }
    __syncthreads();
    const int n_routed = *n_touched, n_list = n_routed + a.ns;
    const int rows = a.T * (a.K + a.ns);
    // each entry's rows of y, in the order of its tokens
    for (int i = tid; i < rows; i += FL_THREADS) {
        const int t = i % a.T, k = i / a.T;
        const int e = k < a.K ? sel_e[t][k] : 0;
        const int s = k < a.K ? eslot[e] * 16 + __popc(emask[e] & ((1 << t) - 1)) : (n_routed + k - a.K) * 16 + t;
        rowi[s] = (uint16_t)(k < a.K ? t * a.K + k : a.T * k + t);
    }
    __syncthreads();

    const int n_up = n_list * a.m_up, n_units = n_up + n_list * a.m_down;
    int* done = a.counters + 1;                  // per entry: epilogue warps of up units
    int* summed = done + a.n_list_max;           // per 32 output rows: entries whose product is stored

    // A consumer's next unit from the queue (single thread)
    auto next_unit = [&](int& qs, uint32_t& qph, int& u) {
        if (!mbar_wait(smem_u32(&uq_full[qs]), qph, ctx, abort_flag)) return false;
        u = uq[qs];
        mbar_arrive(smem_u32(&uq_empty[qs]));
        if (++qs == FL_UQ) {
            qs = 0;
            qph ^= 1u;
        }
        return u >= 0;
    };
    auto settle = [&]() {   // copies in flight land before the block may end
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 200000ull) __nanosleep(1000);
    };

    if (warp == 0) {
        // ---------------------------------------------------------------- units and their weights
        if (lane == 0) {
            const uint64_t policy = l2_policy_evict_first();
            int stage = 0, qs = 0;
            uint32_t phase = 0, qph = 0;
            bool ok = true;
            int claim = atomicAdd(a.counters, 1);
            while (ok) {
                const int u = claim < n_units ? claim : -1;
                if (!mbar_wait(smem_u32(&uq_empty[qs]), qph ^ 1u, ctx, abort_flag)) {
                    ok = false;
                    break;
                }
                uq[qs] = u;
                mbar_arrive(smem_u32(&uq_full[qs]));
                if (++qs == FL_UQ) {
                    qs = 0;
                    qph ^= 1u;
                }
                if (u < 0) break;
                const bool up = u < n_up;
                const int v = up ? u : u - n_up, mb = up ? a.m_up : a.m_down;
                const int i = v / mb, blk = v - i * mb, r0 = blk * FL_BM, e = lst_e[i], n_out = up ? a.F : a.H;
                const int k_stages = up ? a.k_up : a.k_down;
                const bool whole = n_out - r0 > 64, shd = e >= a.E;
                const CUtensorMap* map = up ? (shd ? (whole ? &maps.ups128 : &maps.ups64) : (whole ? &maps.up128 : &maps.up64))
                                            : (shd ? (whole ? &maps.downs128 : &maps.downs64)
                                                   : (whole ? &maps.down128 : &maps.down64));
                // shared chunk j: rows j F .. of its up matrix, columns j F .. of its down matrix (past the
                // chunk's end the next one's weights meet columns of zeros)
                const int y = shd ? (up ? (e - a.E) * a.F + r0 : r0) : e * n_out + r0;
                const int x0 = shd && !up ? (e - a.E) * a.F * 2 : 0;
                // bytes of the stage: these rows and the columns that the other producer loads
                const uint32_t bytes = (whole ? FL_A : FL_A / 2) + (S::BF16 && !up ? 2 : 1) * FL_B;
                // the next unit is claimed a few stages before it is needed, so that the CTAs end together
                const int claim_at = max(0, k_stages - 4);
                int k = fl_first(e, blk, k_stages);
                for (int ks = 0; ks < k_stages; ++ks) {
                    if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, ctx, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = smem_u32(&full[stage]);
                    mbar_arrive_expect_tx(fb, bytes);
                    tma_load_2d(smem_u32(smem + (size_t)stage * S::kStage), map, fb, x0 + k * FL_KB, y, policy);
                    if (++k == k_stages) k = 0;
                    if (++stage == NS) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (ks == claim_at) claim = atomicAdd(a.counters, 1);
                }
            }
            if (!ok) settle();
        }
    } else if (warp == 6) {
        // ---------------------------------------------------------------- the units' columns: tokens or h
        // A thread of its own: the weights of a down unit load while this one waits for its entry.
        if (lane == 0) {
            const uint64_t policy = l2_policy_evict_last();
            int stage = 0, qs = 0, u;
            uint32_t phase = 0, qph = 0;
            bool ok = true;
            while (ok && next_unit(qs, qph, u)) {
                const bool up = u < n_up;
                const int v = up ? u : u - n_up, mb = up ? a.m_up : a.m_down;
                const int i = v / mb, blk = v - i * mb, k_stages = up ? a.k_up : a.k_down;
                const int y = up ? 0 : lst_off[i];
                const CUtensorMap* map = up ? &maps.x : &maps.h;
                if (!up) {
                    ok = wait_count(done + i, 4 * a.m_up, ctx, abort_flag);
                    if (!ok) break;
                    fence_proxy_async_global();
                }
                int k = fl_first(lst_e[i], blk, k_stages);
                for (int ks = 0; ks < k_stages; ++ks) {
                    if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, ctx, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = smem_u32(&full[stage]), dst = smem_u32(smem + (size_t)stage * S::kStage) + FL_A;
                    tma_load_2d(dst, map, fb, k * FL_KB, y, policy);
                    if (S::BF16 && !up) tma_load_2d(dst + FL_B, map, fb, k * FL_KB, rows + y, policy);
                    if (++k == k_stages) k = 0;
                    if (++stage == NS) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok || *abort_flag) settle();
        }
    } else if (warp == 1 || warp == 7) {
        // ---------------------------------------------------------------- products
        // The issue of a stage's four instructions takes one thread about as long as the stage's share
        // of HBM (320 to 400 cycles, in a branch of one lane as here; from a converged warp it was not measured):
        // two threads take turns, one with the even slots of the ring and one with the odd ones.
        // (By turns within a unit, a slot's uses could be the other thread's, and the parity of full that of the
        // use two back.)
        if (lane == 0) {
            const int m = warp == 7;
            int stage = 0, qs = 0, slot = 0, other = S::kSlots, u;
            uint32_t phase = 0, qph = 0, sph = 0, other_ph = 0;
            bool ok = true, issued = false;
            for (int end = S::kSlots; ok && next_unit(qs, qph, u); end = 3 * S::kSlots - end) {
                const bool up = u < n_up;
                const int k_stages = up ? a.k_up : a.k_down;
                const uint32_t idesc = make_idesc(S::BF16 ? 1u : 0u, FL_BM, S::BF16 && !up ? 2 * FL_N : FL_N);
                if (!S::BLOCK && !mbar_wait(smem_u32(&rempty[slot]), sph ^ 1u, ctx, abort_flag)) {
                    ok = false;
                    break;
                }
                for (int ks = 0; ks < k_stages; ++ks) {
                    if (stage % FL_MMA == m) {
                        if (!mbar_wait(smem_u32(&full[stage]), phase, ctx, abort_flag) ||
                            (S::BLOCK && !mbar_wait(smem_u32(&rempty[slot]), sph ^ 1u, ctx, abort_flag))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t wa = smem_u32(smem + (size_t)stage * S::kStage);
                        const uint64_t wd = sw128_desc(wa), bd = sw128_desc(wa + FL_A);
                        const uint32_t d = tmem_base + (uint32_t)((slot * S::kSums + (S::BLOCK ? 0 : 2 * (ks % FL_MMA))) * S::kCols);
                        const uint32_t first = S::BLOCK || ks < FL_MMA ? 0u : 1u;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)   // 32 bytes of K each (the descriptors count 16)
                            mma_ss<!S::BF16>(d + (kk % 2) * S::kCols, wd + 2 * kk, bd + 2 * kk, idesc,
                                             kk >= 2 ? 1u : first);
                        issued = true;
                        mma_commit(smem_u32(&empty[stage]));
                        if (S::BLOCK) mma_commit(smem_u32(&rfull[slot]));
                    }
                    if (++stage == NS) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (S::BLOCK || ks == k_stages - 1) {
                        if (!S::BLOCK) mma_commit(smem_u32(&rfull[slot]));
                        if (++slot == end) {
                            slot = end - S::kSlots;
                            sph ^= 1u;
                        }
                    }
                }
                // the next unit is the other set's
                const int s = slot;
                slot = other;
                other = s;
                const uint32_t p = sph;
                sph = other_ph;
                other_ph = p;
            }
            if ((!ok || *abort_flag) && issued) {   // every MMA issued so far ends before TMEM is released
                mma_commit(smem_u32(drain + m));
                mbar_wait_drain(smem_u32(drain + m), 0, ctx.timeout_ns);
            }
        }
    } else {
        // ---------------------------------------------------------------- epilogue: a lane per weight row
        // Two sets of four warps take turns: the stores, fences and counters at a unit's end take about
        // as long as the reads of its sums.
        const int q = warp & 3;   // TMEM lanes 32 q ..
        const int set = warp >= 8, first_slot = set * S::kSlots;   // its own slots
        bool mine = set;
        const uint32_t t_lane = tmem_base + ((uint32_t)(q * 32) << 16);
        int qs = 0, slot = first_slot;
        uint32_t qph = 0, sph = 0;
        bool ok = true;
        while (ok) {
            if (!mbar_wait_warp(smem_u32(&uq_full[qs]), qph, ctx, abort_flag)) break;
            const int u = uq[qs];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&uq_empty[qs]));
            if (++qs == FL_UQ) {
                qs = 0;
                qph ^= 1u;
            }
            if (u < 0) break;
            const bool up = u < n_up;
            mine = !mine;
            if (!mine) continue;
            const int v = up ? u : u - n_up, mb = up ? a.m_up : a.m_down;
            const int i = v / mb, blk = v - i * mb, e = lst_e[i], n_out = up ? a.F : a.H;
            const int row = blk * FL_BM + q * 32 + lane;
            const bool in = row < n_out;
            float z[FL_N];
            if constexpr (S::BLOCK) {
                const int kb = up ? a.k_up : a.k_down;
                const float* ws = (up ? a.su : a.sd) + ((int64_t)e * n_out + (in ? row : 0)) * kb;
#pragma unroll
                for (int c = 0; c < FL_N; ++c) z[c] = 0.0f;
                // two blocks ahead: the acquires and fences of other warps empty L1, so each may come from L2
                // (11 tokens: 107 us, 111 with one block ahead)
                int b = fl_first(e, blk, kb);
                auto scale = [&]() {
                    const float s = ws[b];
                    if (++b == kb) b = 0;
                    return s;
                };
                float sw = scale(), sw1 = scale();
                for (int ks = 0; ks < kb; ++ks) {
                    const float sw2 = scale();
                    if (!mbar_wait_warp(smem_u32(&rfull[slot]), sph, ctx, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    float p[FL_N];
                    fl_read<FMT>(t_lane + (uint32_t)(slot * S::kSums * S::kCols), false, false, p);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&rempty[slot]));
                    if (++slot == first_slot + S::kSlots) {
                        slot = first_slot;
                        sph ^= 1u;
                    }
#pragma unroll
                    for (int c = 0; c < FL_N; ++c) z[c] = __fmaf_rn(sw, p[c], z[c]);
                    sw = sw1;
                    sw1 = sw2;
                }
                if (!ok) break;
            } else {
                if (!mbar_wait_warp(smem_u32(&rfull[slot]), sph, ctx, abort_flag)) break;
                tc_fence_after();
                fl_read<FMT>(t_lane + (uint32_t)(slot * S::kSums * S::kCols), !up, (up ? a.k_up : a.k_down) == 1, z);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&rempty[slot]));
                if (++slot == first_slot + S::kSlots) {
                    slot = first_slot;
                    sph ^= 1u;
                }
            }
            const int mask = lst_mask[i];
            if (up) {
                // columns are tokens; the entry's keep their order in its rows of h
                const float sc = S::BF16 ? 1.0f : S::BLOCK ? a.x_scale : __fmul_rn(a.su[e], a.x_scale);
                const int64_t o0 = (int64_t)lst_off[i] * a.F + row;
                int c = 0;
#pragma unroll
                for (int t = 0; t < FL_N; ++t) {
                    if (!((mask >> t) & 1)) continue;
                    const int64_t o = o0 + (int64_t)c * a.F;
                    ++c;
                    if (!in) continue;
                    float zz = z[t];
                    if constexpr (!S::BF16) zz = __fmul_rn(zz, sc);
                    const float h = zz <= 0.0f ? 0.0f : __fmul_rn(zz, zz);   // a NaN stays one
                    if constexpr (S::BF16) {
                        // h as the sum of two bf16, 16 bits of it: one alone would add a second rounding
                        // of the output's size
                        const __nv_bfloat16 hi = __float2bfloat16_rn(h);
                        const float top = __bfloat162float(hi);
                        __nv_bfloat16* hp = reinterpret_cast<__nv_bfloat16*>(a.h) + o;
                        hp[0] = hi;
                        hp[(int64_t)rows * a.F] =
                            __float2bfloat16_rn(top < __uint_as_float(0x7f800000u) ? __fsub_rn(h, top) : 0.0f);
                    } else {
                        a.h[o] = (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(h, a.h_scale), __NV_SATFINITE, __NV_E4M3);
                    }
                }
                // for the TMA loads of h: every lane's stores, then the warp's report
                fence_proxy_async_global();
                __syncwarp();
                if (lane == 0 && !(a.hold && u == 0)) red_release_add(done + i, 1);
            } else {
                const float sc = S::BF16 ? 1.0f : S::BLOCK ? a.h_scale : __fmul_rn(a.sd[e], a.h_scale);
                const int n_tok = __popc(mask);
#pragma unroll
                for (int c = 0; c < FL_N; ++c)
                    if (c < n_tok && in) {
                        float y = z[c];
                        if constexpr (!S::BF16) y = __fmul_rn(y, sc);
                        __stcg(a.y + (int64_t)rowi[i * 16 + c] * a.H + row, y);
                    }
                // the last entry's warp for these 32 rows sums them
                __syncwarp();
                int last = 0;
                if (lane == 0) {
                    __threadfence();
                    last = atomicAdd(summed + blk * 4 + q, 1) == n_list - 1;
                    __threadfence();
                }
                __syncwarp();   // the other lanes read too, and the shuffle orders no memory
                if (__shfl_sync(0xffffffffu, last, 0))
                    fl_combine(a, sel_w, blk * FL_BM + q * 32 + lane % 8 * 4, lane / 8);
                __syncwarp();
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

static int few_row_bytes(int K, int dtype) {
    return dtype == MOE_BF16 ? 2 * K : dtype == MOE_FP8_B128 ? (K + 127) / 128 * 128 : K;
}

int few_counters(const moe_dims* d) {
    const int64_t n_list = std::min<int64_t>(d->E, d->T * d->K) + d->Fs / d->F;
    return (int)(1 + n_list + 4 * ((d->H + FL_BM - 1) / FL_BM));
}

template <int FMT>
static cudaError_t launch_layer(const FewMaps& maps, FewArgs& a, int num_sms, const DevCtx& ctx, cudaStream_t stream) {
    using S = FlShape<FMT>;
    const size_t fixed = 1024 + few_table_bytes(a.n_list_max);
    a.n_stages = (int)std::min<size_t>(FL_MAX_STAGES, (kMaxSmem - fixed) / S::kStage);
    a.n_stages -= a.n_stages % FL_MMA;   // each slot has one issuer
    const size_t smem = (size_t)a.n_stages * S::kStage + fixed;
    auto k = few_layer_kernel<FMT>;
    cudaError_t e = allow_smem(k);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.n_list_max * (a.m_up + a.m_down);
    return launch_k(k, dim3((unsigned)std::min<int64_t>(units, num_sms)), dim3(FL_THREADS), smem, stream, maps, a, ctx);
}

cudaError_t launch_few(const moe_dims* d, const uint16_t* x, const uint16_t* wr, const float* bias, const void* w_up,
                       const void* w_down, const void* w_up_s, const void* w_down_s, const moe_fp8_scales* sc,
                       const uint16_t* residual, uint16_t* out, int32_t* idx, float* w, const FewWs& ws, int hold,
                       int num_sms, const DevCtx& ctx, cudaStream_t stream) {
    const bool fp8 = d->expert_dtype != MOE_BF16;
    const int T = (int)d->T, ns = d->Fs / d->F, rows = T * (d->K + ns);
    FewArgs a = {};
    a.residual = residual;
    a.out = out;
    a.topk_idx = idx;
    a.topk_w = w;
    a.logits = ws.logits;
    a.su = fp8 ? sc->w_up_scale : nullptr;
    a.sd = fp8 ? sc->w_down_scale : nullptr;
    a.x_scale = fp8 ? sc->x_scale : 1.0f;
    a.h_scale = fp8 ? sc->h_scale : 1.0f;
    a.h = ws.h;
    a.y = ws.y;
    a.counters = ws.counters;
    a.T = T;
    a.H = d->H;
    a.E = d->E;
    a.K = d->K;
    a.F = d->F;
    a.ns = ns;
    a.m_up = (d->F + FL_BM - 1) / FL_BM;
    a.m_down = (d->H + FL_BM - 1) / FL_BM;
    a.n_list_max = (int)std::min<int64_t>(d->E, d->T * d->K) + ns;
    a.hold = hold;
    const int ub = few_row_bytes(d->H, d->expert_dtype), db = few_row_bytes(d->F, d->expert_dtype);
    const int es = fp8 ? 1 : 2;
    a.k_up = (ub + FL_KB - 1) / FL_KB;
    a.k_down = (db + FL_KB - 1) / FL_KB;
    FewMaps maps = {};
    const int64_t ur = (int64_t)d->E * d->F, dr = (int64_t)d->E * d->H;
    // a box of 64 rows serves the last rows of an expert when 64 or fewer are left
    const bool u64 = d->F % FL_BM > 0 && d->F % FL_BM <= 64, d64 = d->H % FL_BM > 0 && d->H % FL_BM <= 64;
    bool ok = make_map_u8_b128(&maps.up128, w_up, ur, ub, 128) && make_map_u8_b128(&maps.down128, w_down, dr, db, 128) &&
              make_map_u8_b128(&maps.x, fp8 ? static_cast<const void*>(ws.xq) : x, T, (int64_t)d->H * es, FL_N) &&
              make_map_u8_b128(&maps.h, ws.h, (int64_t)rows * es, (int64_t)d->F * es, FL_N);
    if (u64) ok = ok && make_map_u8_b128(&maps.up64, w_up, ur, ub, 64);
    if (d64) ok = ok && make_map_u8_b128(&maps.down64, w_down, dr, db, 64);
    if (ns > 0) {
        ok = ok && make_map_u8_b128(&maps.ups128, w_up_s, d->Fs, ub, 128) &&
             make_map_u8_b128(&maps.downs128, w_down_s, d->H, (int64_t)d->Fs * 2, 128);
        if (u64) ok = ok && make_map_u8_b128(&maps.ups64, w_up_s, d->Fs, ub, 64);
        if (d64) ok = ok && make_map_u8_b128(&maps.downs64, w_down_s, d->H, (int64_t)d->Fs * 2, 64);
        a.warm[0] = static_cast<const uint8_t*>(w_up_s);
        a.warm[1] = static_cast<const uint8_t*>(w_down_s);
        a.warm_bytes = std::min<int64_t>((int64_t)d->Fs * d->H * 2, kFewWarmBytes);
    }
    if (!ok) return cudaErrorInvalidValue;

    FewRouterArgs r = {};
    r.x = x;
    r.wr = wr;
    r.bias = bias;
    r.T = T;
    r.H = d->H;
    r.E = d->E;
    r.logits = ws.logits;
    r.xq = fp8 ? ws.xq : nullptr;
    r.x_scale = a.x_scale;
    r.counters = ws.counters;
    r.n_counters = few_counters(d);
    const cudaError_t e = launch_k(few_router_kernel, dim3(d->E + (fp8 ? T : 0)), dim3(FEW_RT), 0, stream, r, ctx);
    if (e != cudaSuccess) return e;
    switch (d->expert_dtype) {
        case MOE_BF16: return launch_layer<MOE_BF16>(maps, a, num_sms, ctx, stream);
        case MOE_FP8_E4M3: return launch_layer<MOE_FP8_E4M3>(maps, a, num_sms, ctx, stream);
        default: return launch_layer<MOE_FP8_B128>(maps, a, num_sms, ctx, stream);
    }
}

}  // namespace moe
