// The norms between two blocks of the decoder, in one pass over the rows
// (bloomery issue page, s.2: a hybrid decoder of pre-norm blocks; audio.cpp
// model page, "Q4_K, Q3_K and Q2_K expert profiles": the model's normalisation).
//
//   n[t]  = y[t] / sqrt(mean(y[t]^2) + eps) * gain_post            norm after a block
//   x'[t] = x[t] + alpha * gate (*) n[t]                           gate, residual scale, residual sum
//   u[t]  = x'[t] / sqrt(mean(x'[t]^2) + eps) * gain_pre           norm before the next block
//   codes, scales: u[t] as FP8_B128 (one fp32 scale amax / 448 per 128 values)
//
// Everything between the bf16 inputs and the one rounding of each output is
// fp32: u and the codes come from the unrounded x', the codes from the
// unrounded u.  A row is read once and stays in registers between its two
// sums of squares.
//
// Bound: HBM bytes (about 8 bytes and 12 operations per value), latency at a
// few rows.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

struct NormArgs {
    const uint16_t* y;          // block output (POST)
    const uint16_t* gain_post;  // [H] or null (POST)
    const uint16_t* gate;       // [H] or [T][H] or null (POST)
    int64_t gate_ld;            // 0: one row for all tokens; H: a row per token
    const uint16_t* x;          // residual stream
    const uint16_t* gain_pre;   // [H] or null
    uint16_t* x_out;            // POST
    uint16_t* u;                // or null
    uint8_t* codes;             // [T][Kp] or null
    float* scales;              // [T][Kp / 128]
    int64_t T;
    int H;
    float eps, alpha;
};

__device__ __forceinline__ void nm_unpack(const uint4& q, float (&f)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 nm_pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum over the block, the same bits in every thread: a butterfly in each warp, then the warps' sums
// in warp order.  red: one float per warp, a buffer of its own per call between two barriers.
__device__ __forceinline__ float nm_block_sum(float v, float* red, int n_warps) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (n_warps == 1) return v;
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < n_warps; ++i) s += red[i];
    return s;
}

// A block per row at a time (grid-stride); thread i of its n holds the row's 16-byte vectors i + j * n,
// j < VPT.
template <int VPT, int MAXT, bool POST, bool CODES>
__global__ void __launch_bounds__(MAXT, 1024 / MAXT) norm_kernel(NormArgs a) {
    pdl_enter();
    __shared__ float red[2][2][32];   // [row parity][sum][warp]
    const int nv = a.H / 8;
    const int kb = (a.H + 127) / 128;
    const int i0 = threadIdx.x, n = blockDim.x;
    int par = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, par ^= 1) {
        uint4 xq[VPT];
        const uint4* xr = reinterpret_cast<const uint4*>(a.x + t * a.H);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = i0 + j * n;
            xq[j] = v < nv ? xr[v] : make_uint4(0, 0, 0, 0);
        }
        float f[VPT][8];
        if constexpr (POST) {
            const uint4* yr = reinterpret_cast<const uint4*>(a.y + t * a.H);
            uint4 yq[VPT];
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = i0 + j * n;
                yq[j] = v < nv ? yr[v] : make_uint4(0, 0, 0, 0);
            }
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                float y[8];
                nm_unpack(yq[j], y);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = __fmaf_rn(y[i], y[i], ss);
            }
            ss = nm_block_sum(ss, red[par][0], n / 32);
            const float r = __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)a.H), a.eps));
            uint4* xo = reinterpret_cast<uint4*>(a.x_out + t * a.H);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = i0 + j * n;
                float p[8], xx[8];
                nm_unpack(yq[j], f[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[j][i] *= r;
                if (v < nv) {
                    if (a.gain_post) {
                        nm_unpack(reinterpret_cast<const uint4*>(a.gain_post)[v], p);
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[j][i] *= p[i];
                    }
                    if (a.gate) {
                        nm_unpack(reinterpret_cast<const uint4*>(a.gate + t * a.gate_ld)[v], p);
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[j][i] *= p[i];
                    }
                    nm_unpack(xq[j], xx);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[j][i] = __fmaf_rn(a.alpha, f[j][i], xx[i]);
                    xo[v] = nm_pack(f[j]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[j][i] = 0.0f;   // also where the row's r is not finite
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < VPT; ++j) nm_unpack(xq[j], f[j]);
        }
        if (!a.u && !CODES) continue;
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __fmaf_rn(f[j][i], f[j][i], ss);
        ss = nm_block_sum(ss, red[par][1], n / 32);
        const float r = __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)a.H), a.eps));
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = i0 + j * n;
#pragma unroll
            for (int i = 0; i < 8; ++i) f[j][i] = v < nv ? f[j][i] * r : 0.0f;
            if (a.gain_pre && v < nv) {
                float p[8];
                nm_unpack(reinterpret_cast<const uint4*>(a.gain_pre)[v], p);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[j][i] *= p[i];
            }
            if (a.u && v < nv) reinterpret_cast<uint4*>(a.u + t * a.H)[v] = nm_pack(f[j]);
        }
        if constexpr (CODES) {
            // a block of 128 values is 16 neighbouring lanes (vectors past the row are zero)
            float m[VPT];
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                m[j] = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m[j] = fmaxf(m[j], fabsf(f[j][i]));
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1)
#pragma unroll
                for (int j = 0; j < VPT; ++j) m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], off));
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = i0 + j * n;
                // Not below the smallest normal number, so that 1 / s is finite.  A product with it is
                // within 2^-23 of the quotient, next to half a step of the codes, 2^-4; a quotient per
                // value took longer than the bytes.
                const float s = m[j] > 0.0f ? fmaxf(__fdiv_rn(m[j], 448.0f), 0x1p-126f) : 1.0f;
                const float is = __frcp_rn(s);
                if (v < kb * 16) {
                    uint32_t c[2] = {0, 0};
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        c[i / 4] |= (uint32_t)__nv_cvt_float2_to_fp8x2(
                                        make_float2(__fmul_rn(f[j][i], is), __fmul_rn(f[j][i + 1], is)),
                                        __NV_SATFINITE, __NV_E4M3)
                                    << (8 * (i % 4));
                    *reinterpret_cast<uint2*>(a.codes + (t * kb * 16 + v) * 8) = make_uint2(c[0], c[1]);
                    if (v % 16 == 0) a.scales[t * kb + v / 16] = s;
                }
            }
        }
    }
}

// ----------------------------------------------------------------------------- host

template <int VPT, int MAXT>
static cudaError_t launch_vpt(const NormArgs& a, int threads, int num_sms, cudaStream_t stream) {
    const bool post = a.y != nullptr, codes = a.codes != nullptr;
    void (*k)(NormArgs) = post ? (codes ? norm_kernel<VPT, MAXT, true, true> : norm_kernel<VPT, MAXT, true, false>)
                               : (codes ? norm_kernel<VPT, MAXT, false, true> : norm_kernel<VPT, MAXT, false, false>);
    // a row for each block, up to a grid that only takes time to launch: with as many blocks as fit, each
    // with several rows, a row's loads wait for the stores of the one before (pre, 16384 rows: 32 -> 40 us)
    const int64_t grid = std::min<int64_t>(a.T, 1024 * num_sms);
    return launch_k(k, dim3((unsigned)grid), dim3((unsigned)threads), 0, stream, a);
}

static cudaError_t launch_norm(const NormArgs& a, int num_sms, cudaStream_t stream) {
    // vectors of a row, a whole number of 128-value blocks
    const int nv = (a.H + 127) / 128 * 16;
    // With three rows or more for every SM, several small blocks of an SM work at once, and a thread has
    // three or four vectors of each input under way; with fewer, a vector per thread has the least latency.
    // Device times, H = 2688 (one vector against three), prenorm to u and postnorm to x', u:
    //   T = 296    2.7 against 3.1 us,   4.3 against  5.7
    //   T = 577    4.3 against 3.5,      7.6 against  6.6
    //   T = 16384   58 against  32,      153 against   81       (a warp per row: 35, 117)
    // What bounds the large ones is how many loads an SM has under way, so 1024 threads fit on it (64
    // registers each): with 768, postnorm took 93 us.  prenorm to codes (39 us, 21 at the rate of a copy)
    // is held up by the shuffles of its maxima, done for all vectors together (one after the other: 43);
    // warp reductions for them took longer.
    // The price of 64 registers: postnorm spills 40 to 80 bytes a thread in the forms of four vectors (8 in
    // that of three with codes) and 460 to 630 in that of eight, which prenorm spills from as well (52, with
    // codes 284).  Three vectors exist for 128 threads alone, the class of H = 2688: just above 4096 and 8192
    // values a little more than half of the vector slots hold data.
    if (a.T >= 3 * num_sms) {
        const int w = (nv + 127) / 128;
        if (w <= 2) return launch_vpt<2, 128>(a, 128, num_sms, stream);
        if (w <= 3) return launch_vpt<3, 128>(a, 128, num_sms, stream);
        if (w <= 4) return launch_vpt<4, 128>(a, 128, num_sms, stream);
        if (w <= 8) return launch_vpt<4, 256>(a, 256, num_sms, stream);
        if (w <= 16) return launch_vpt<4, 512>(a, 512, num_sms, stream);
    }
    auto threads = [&](int vpt) { return ((nv + vpt - 1) / vpt + 31) / 32 * 32; };
    if (nv <= 1024) return launch_vpt<1, 1024>(a, threads(1), num_sms, stream);
    if (nv <= 2048) return launch_vpt<2, 1024>(a, threads(2), num_sms, stream);
    if (nv <= 4096) return launch_vpt<4, 1024>(a, threads(4), num_sms, stream);
    return launch_vpt<8, 1024>(a, threads(8), num_sms, stream);
}

}  // namespace moe

using namespace moe;

namespace {
bool is_aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

moe_status run_norm(const NormArgs& a, void* stream) {
    DevCtx ctx;
    int sms = 0;
    const moe_status s = internal_device(&ctx, &sms);
    if (s != MOE_OK) return s;
    return launch_norm(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ECUDA;
}

moe_status check_norm(int64_t T, int32_t H, float eps) {
    if (T < 0 || T >= ((int64_t)1 << 31) || H < 16 || H > 65536 || H % 16 != 0) return MOE_EINVAL;
    return eps >= 0.0f && eps < 3.4e38f ? MOE_OK : MOE_EINVAL;
}

bool codes_ok(const uint8_t* codes, const float* scales) {
    return !codes == !scales && is_aligned(codes, 16) && is_aligned(scales, 4);
}

// A row of bf16 outputs may replace the row of inputs that it is made of; nothing else may be shared.
bool buffers_ok(const NormArgs& a) {
    const int64_t row = (int64_t)a.H * 2, act = a.T * row, kb = (a.H + 127) / 128;
    const bool per_token = a.gate_ld != 0;
    const struct {
        const void* p;
        int64_t n;
        bool rows;   // [T][H] bf16
    } out[4] = {{a.x_out, act, true}, {a.u, act, true}, {a.codes, a.T * kb * 128, false}, {a.scales, a.T * kb * 4, false}},
      in[5] = {{a.x, act, true}, {a.y, act, true}, {a.gate, per_token ? act : row, per_token},
               {a.gain_post, row, false}, {a.gain_pre, row, false}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 5; ++j)
            if (!(out[i].rows && in[j].rows && out[i].p == in[j].p) && overlap(out[i].p, out[i].n, in[j].p, in[j].n))
                return false;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return false;
    }
    return true;
}
}  // namespace

extern "C" {

moe_status moe_prenorm(int64_t T, int32_t H, float eps, const void* x, const void* gain, void* u, uint8_t* codes,
                       float* scales, void* stream) {
    const moe_status s = check_norm(T, H, eps);
    if (s != MOE_OK) return s;
    if (T == 0) return MOE_OK;
    if (!x || (!u && !codes) || !codes_ok(codes, scales)) return MOE_EINVAL;
    if (!is_aligned(x, 16) || !is_aligned(gain, 16) || !is_aligned(u, 16)) return MOE_EINVAL;
    NormArgs a = {};
    a.x = static_cast<const uint16_t*>(x);
    a.gain_pre = static_cast<const uint16_t*>(gain);
    a.u = static_cast<uint16_t*>(u);
    a.codes = codes;
    a.scales = scales;
    a.T = T;
    a.H = H;
    a.eps = eps;
    if (!buffers_ok(a)) return MOE_EINVAL;
    return run_norm(a, stream);
}

moe_status moe_postnorm(int64_t T, int32_t H, float eps, float alpha, const void* y, const void* gain,
                        const void* gate, int64_t gate_ld, const void* x, void* x_out, const void* next_gain, void* u,
                        uint8_t* codes, float* scales, void* stream) {
    const moe_status s = check_norm(T, H, eps);
    if (s != MOE_OK) return s;
    if (!(alpha > -3.4e38f && alpha < 3.4e38f)) return MOE_EINVAL;
    if (gate && gate_ld != 0 && gate_ld != H) return MOE_EINVAL;
    if (T == 0) return MOE_OK;
    if (!y || !x || !x_out || !codes_ok(codes, scales)) return MOE_EINVAL;
    if (!is_aligned(y, 16) || !is_aligned(gain, 16) || !is_aligned(gate, 16) || !is_aligned(x, 16) ||
        !is_aligned(x_out, 16) || !is_aligned(next_gain, 16) || !is_aligned(u, 16))
        return MOE_EINVAL;
    NormArgs a = {};
    a.y = static_cast<const uint16_t*>(y);
    a.gain_post = static_cast<const uint16_t*>(gain);
    a.gate = static_cast<const uint16_t*>(gate);
    a.gate_ld = gate_ld;
    a.x = static_cast<const uint16_t*>(x);
    a.gain_pre = static_cast<const uint16_t*>(next_gain);
    a.x_out = static_cast<uint16_t*>(x_out);
    a.u = static_cast<uint16_t*>(u);
    a.codes = codes;
    a.scales = scales;
    a.T = T;
    a.H = H;
    a.eps = eps;
    a.alpha = alpha;
    if (!buffers_ok(a)) return MOE_EINVAL;
    return run_norm(a, stream);
}

}  // extern "C"
