// filter_math.cuh -- the arithmetic of tempered, truncated distributions that
// the sampler and the filtered policy statistics share.
//
// A row z[0..V) with temperature t has x_v = (z_v - M)/t, M = max z, and
// weights e_v = e^(x_v).  Tokens are ordered by (logit descending, index
// ascending); top-k, top-p and min-p each keep a prefix of that order, so the
// kept set is a prefix as well and is named by its last element, the cut
// (tau, i):  v is kept  <=>  z_v > tau  or  (z_v == tau and v <= i).
//
// Which token ends a nucleus, and which one a uniform u falls on, are
// comparisons of partial sums of e with a share of the whole sum.  So that
// such a decision does not hang on the rounding of a sum, weights are formed
// to about 2^-46 relative and summed as 64-bit integers: integer sums are
// exact and do not depend on their order, hence on the batch or the launch.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace pstat {

constexpr int64_t kFilterMaxV = PSTAT_FILTER_MAX_V;
constexpr float kFilterTempMin = 1.f / 1048576.f;  // 2^-20
constexpr float kFilterTempMax = 1048576.f;        // 2^20

// 2^(-j/64), j = 0..63, each as an unevaluated sum of two floats.
struct ExpTable {
    float2 v[64];
};

// Order-preserving map: a smaller key is a larger logit.  -0 and +0 are one
// value (x + 0 turns -0 into +0).  -inf has the largest key of all.
__device__ __forceinline__ uint32_t desc_key(float z) {
    const uint32_t b = __float_as_uint(z + 0.f);
    return ~(b ^ (uint32_t)(((int32_t)b >> 31) | (int32_t)0x80000000));
}
__device__ __forceinline__ float key_logit(uint32_t dk) {
    const uint32_t a = ~dk;
    return __uint_as_float((a & 0x80000000u) ? (a ^ 0x80000000u) : ~a);
}
constexpr uint32_t kKeyNegInf = 0xFF800000u;  // desc_key(-inf)

// log2(e)/t as an unevaluated sum of two floats: the quotient and the
// division's exact remainder over t.
struct TempScale {
    float ch, cl;
};
__device__ __forceinline__ TempScale temp_scale(float t) {
    constexpr float kH = 1.4426950408889634f;
    constexpr float kL = (float)(1.4426950408889634074 - (double)kH);
    TempScale s;
    s.ch = __fdiv_rn(kH, t);
    s.cl = __fdiv_rn(fmaf(-s.ch, t, kH) + kL, t);
    return s;
}

// round(2^k e^((z - M)/t)) to about 2^-46 relative, 0 where e^((z-M)/t) is
// below 2^-63.  With y = (M - z) log2(e)/t in double-float arithmetic, write
// y = j/64 + r, |r| <= 2^-7 (plus the low part); then 2^-y = 2^-(j/64) 2^-r:
// the first factor from the table and a power of two, the second from
// e^-s = 1 - s + s^2/2 - s^3/6 + s^4/24 - s^5/120, s = r ln 2 <= 2^-7.5,
// whose next term s^6/720 is below 2^-54.  The first two terms are carried in
// double-float, the others (below 2^-24) in fp32.  z = M gives 2^k exactly.
__device__ __forceinline__ uint64_t fixed_weight(float z, float M, TempScale c, int k,
                                                 const float2* __restrict__ table) {
    const float dh = M - z;
    if (!(dh * c.ch < 63.f)) return 0;
    const float bb = dh - M;
    const float dl = (M - (dh - bb)) - (z + bb);  // exact remainder of M - z
    // (rounding intrinsics where a product's own rounding error is used: the
    // compiler may not fuse those into a later addition)
    const float y0 = __fmul_rn(dh, c.ch);
    const float y1 = fmaf(dh, c.ch, -y0) + fmaf(dh, c.cl, dl * c.ch);
    const int j = __float2int_rn(y0 * 64.f);
    const float r0 = fmaf((float)j, -0.015625f, y0);  // exact
    const float rh = r0 + y1;
    const float rb = rh - r0;
    const float rl = (r0 - (rh - rb)) + (y1 - rb);
    constexpr float kLn2H = 0.69314718055994531f;
    constexpr float kLn2L = (float)(0.69314718055994530942 - (double)kLn2H);
    const float sh = __fmul_rn(rh, kLn2H);
    const float sl = fmaf(rh, kLn2H, -sh) + fmaf(rh, kLn2L, rl * kLn2H);
    const float p = __fmul_rn(sh, sh);
    const float pe = fmaf(2.f * sh, sl, fmaf(sh, sh, -p));
    const float q = p * sh * fmaf(sh, fmaf(sh, -1.f / 120.f, 1.f / 24.f), -1.f / 6.f);
    const float ah = fmaf(p, 0.5f, -sh);
    const float al = fmaf(p, 0.5f, -__fadd_rn(ah, sh)) + (q + fmaf(0.5f, pe, -sl));
    const float2 tb = table[j & 63];
    const float ph = __fmul_rn(tb.x, ah);
    const float pl = fmaf(tb.x, ah, -ph) + fmaf(tb.x, al, tb.y * ah);
    const float eh = tb.x + ph;
    const float el = (ph - (eh - tb.x)) + (tb.y + pl);
    const float scale = __int_as_float((127 + k - (j >> 6)) << 23);
    return (uint64_t)(__float2ll_rn(eh * scale) + __float2ll_rn(el * scale));
}

// Binary digits after the point of the fixed weights of a row whose sum is
// below 2^b: the sum of all of them stays below 2^62.
__device__ __forceinline__ int fixed_scale(float sum_upper) {
    const int b = (int)(__float_as_uint(sum_upper) >> 23) - 127 + 1;  // sum_upper < 2^b
    return 61 - b;
}

// ln(S 2^-k) for a sum S >= 2^k of fixed weights.  Near 1 the logarithm is
// taken of the exact excess, so that it keeps its relative precision.
__device__ __forceinline__ float fixed_log(uint64_t S, int k) {
    const float inv = __int_as_float((127 - k) << 23);
    const uint64_t one = 1ull << k;
    if (S < 2 * one) return log1pf((float)(S - one) * inv);
    return logf((float)S * inv);
}

}  // namespace pstat
