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
// to 2^-45 + 2^-44.5 |x| relative and summed as 64-bit integers: integer sums are
// exact and do not depend on their order, hence on the batch or the launch.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "chunk_math.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace pstat {

constexpr int64_t kFilterMaxV = PSTAT_FILTER_MAX_V;
constexpr float kFilterTempMin = 1.f / 1048576.f;  // 2^-20
constexpr float kFilterTempMax = 1048576.f;        // 2^20

// 2^(-j/64), j = 0..63, each as an unevaluated sum of two floats.
__device__ const float2 kExp2Table[64] = {
    {0x1p+0f, 0x0p+0f}, {0x1.fa7c18p-1f, 0x1.9e90d8p-29f},
    {0x1.f50766p-1f, -0x1.246ebp-27f}, {0x1.efa1bep-1f, 0x1.cc2b44p-26f},
    {0x1.ea4afap-1f, 0x1.52486cp-28f}, {0x1.e502eep-1f, 0x1.e2cffep-27f},
    {0x1.dfc974p-1f, -0x1.908c94p-26f}, {0x1.da9e6p-1f, 0x1.ed9942p-28f},
    {0x1.d5818ep-1f, -0x1.822dbcp-28f}, {0x1.d072d4p-1f, 0x1.40f13p-26f},
    {0x1.cb720ep-1f, -0x1.8837ccp-28f}, {0x1.c67f12p-1f, 0x1.cafa2ap-26f},
    {0x1.c199bep-1f, -0x1.3d56b2p-28f}, {0x1.bcc1eap-1f, -0x1.f687c6p-26f},
    {0x1.b7f77p-1f, -0x1.a09438p-26f}, {0x1.b33a2cp-1f, -0x1.ec3a82p-27f},
    {0x1.ae89fap-1f, -0x1.a94b14p-27f}, {0x1.a9e6b6p-1f, -0x1.50c048p-26f},
    {0x1.a5503cp-1f, -0x1.b83b54p-26f}, {0x1.a0c668p-1f, -0x1.2886a6p-27f},
    {0x1.9c4918p-1f, 0x1.51f848p-28f}, {0x1.97d82ap-1f, -0x1.0d8d84p-32f},
    {0x1.93737cp-1f, -0x1.e64744p-26f}, {0x1.8f1aeap-1f, -0x1.baa232p-27f},
    {0x1.8ace54p-1f, 0x1.15506ep-28f}, {0x1.868d9ap-1f, -0x1.2edb44p-27f},
    {0x1.82589ap-1f, -0x1.accc7cp-27f}, {0x1.7e2f34p-1f, -0x1.261634p-26f},
    {0x1.7a1148p-1f, -0x1.829fdp-26f}, {0x1.75feb6p-1f, -0x1.37b306p-26f},
    {0x1.71f75ep-1f, 0x1.1d8beep-26f}, {0x1.6dfb24p-1f, -0x1.cd72e8p-28f},
    {0x1.6a09e6p-1f, 0x1.9fcef4p-27f}, {0x1.662388p-1f, 0x1.2a9112p-28f},
    {0x1.6247ecp-1f, -0x1.f8b55p-26f}, {0x1.5e76f2p-1f, -0x1.4a5bd6p-26f},
    {0x1.5ab07ep-1f, -0x1.5bd5ecp-28f}, {0x1.56f474p-1f, -0x1.295b04p-26f},
    {0x1.5342b6p-1f, -0x1.2c561p-26f}, {0x1.4f9b28p-1f, -0x1.2c5a6cp-26f},
    {0x1.4bfdaep-1f, -0x1.593abcp-26f}, {0x1.486a2cp-1f, -0x1.47d866p-26f},
    {0x1.44e086p-1f, 0x1.8624b4p-31f}, {0x1.4160a2p-1f, 0x1.f72e2ap-29f},
    {0x1.3dea64p-1f, 0x1.824684p-26f}, {0x1.3a7db4p-1f, -0x1.634c02p-26f},
    {0x1.371a74p-1f, -0x1.18aac6p-26f}, {0x1.33c08cp-1f, -0x1.b37d2p-26f},
    {0x1.306fep-1f, 0x1.4636e2p-26f}, {0x1.2d285ap-1f, 0x1.b900c2p-27f},
    {0x1.29e9ep-1f, -0x1.5c0424p-26f}, {0x1.26b456p-1f, 0x1.789f38p-27f},
    {0x1.2387a6p-1f, 0x1.ceac48p-26f}, {0x1.2063b8p-1f, 0x1.0c519ap-26f},
    {0x1.1d4874p-1f, -0x1.d2e8cap-26f}, {0x1.1a35bep-1f, 0x1.6df96ep-26f},
    {0x1.172b84p-1f, -0x1.c15742p-28f}, {0x1.1429aap-1f, 0x1.d525bcp-26f},
    {0x1.11301ep-1f, -0x1.fdb496p-26f}, {0x1.0e3ec4p-1f, -0x1.a585ccp-26f},
    {0x1.0b5586p-1f, 0x1.9f3122p-26f}, {0x1.087452p-1f, -0x1.e2990ep-27f},
    {0x1.059b0ep-1f, -0x1.9d4f52p-26f}, {0x1.02c9a4p-1f, -0x1.887fap-29f},
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

// a - b, as one packed FMA.
__device__ __forceinline__ uint64_t f2_set(float v) { return f2_pack(v, v); }
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) {
    return f2_fma(b, f2_set(-1.f), a);
}
__device__ __forceinline__ uint64_t f2_neg(uint64_t v) { return v ^ 0x8000000080000000ull; }

// round(2^k e^((z - M)/t)) of two logits, k <= 60; 0 where that is far below 1.
// With y = (M - z) log2(e)/t in double-float arithmetic, write y = j/64 + r, |r| <=
// 2^-7 (plus the low part); then 2^-y = 2^-(j/64) 2^-r: the first factor from the
// table and a power of two, the second from e^-s = 1 - s + s^2/2 - s^3/6 + s^4/24 -
// s^5/120, s = r ln 2 <= 2^-7.5, whose next term s^6/720 is below 2^-54.  The first
// two terms are carried in double-float, the others (below 2^-24) in fp32.  z = M
// gives 2^k exactly.  (A table-driven exponential, as in Tang, ACM TOMS 15, 1989.)
// Before the rounding to whole numbers the relative error is at most 2^-45 (the terms
// in fp32 and the low word's roundings) + 2^-44.5 |x|: y is off by 10.5 x 2^-48 of itself,
// from the scale's low part and from four roundings of its own.  Measured, at
// temperatures of 0.3 to 1.3: 2^-46.1 for |x| below 1, 2^-45.1 to 3, 2^-43.4 to 7,
// 2^-42.8 to 21.
// Packed arithmetic on both: a pass that weighs a whole row is bound by issued
// instructions, of which this takes about 80 for a pair and scalar arithmetic
// over 100 for each.
__device__ __forceinline__ void fixed_weights(float z0, float z1, float M, TempScale c, int k,
                                              const float2* __restrict__ table, uint64_t& w0,
                                              uint64_t& w1) {
    const float limit = (float)(k + 2);
    float d0 = M - z0, d1 = M - z1;
    const bool far0 = !(d0 * c.ch < limit), far1 = !(d1 * c.ch < limit);
    if (far0) {  // selects
        d0 = 0.f;
        z0 = M;
    }
    if (far1) {
        d1 = 0.f;
        z1 = M;
    }
    const uint64_t Mp = f2_set(M), ch = f2_set(c.ch);
    const uint64_t z = f2_pack(z0, z1), dh = f2_pack(d0, d1);
    const uint64_t bb = f2_sub(dh, Mp);
    const uint64_t dl = f2_sub(f2_sub(Mp, f2_sub(dh, bb)), f2_add(z, bb));  // rest of M - z
    const uint64_t y0 = f2_mul(dh, ch);
    const uint64_t y1 = f2_add(f2_fma(dh, ch, f2_neg(y0)), f2_fma(dh, f2_set(c.cl), f2_mul(dl, ch)));
    float ja, jb;
    f2_unpack(f2_mul(y0, f2_set(64.f)), ja, jb);
    const int j0 = __float2int_rn(ja), j1 = __float2int_rn(jb);
    const uint64_t r0 = f2_fma(f2_pack((float)j0, (float)j1), f2_set(-0.015625f), y0);  // exact
    const uint64_t rh = f2_add(r0, y1);
    const uint64_t rb = f2_sub(rh, r0);
    const uint64_t rl = f2_add(f2_sub(r0, f2_sub(rh, rb)), f2_sub(y1, rb));
    constexpr float kLn2H = 0.69314718055994531f;
    constexpr float kLn2L = (float)(0.69314718055994530942 - (double)kLn2H);
    const uint64_t lh = f2_set(kLn2H);
    const uint64_t sh = f2_mul(rh, lh), nsh = f2_neg(sh);
    const uint64_t sl = f2_add(f2_fma(rh, lh, nsh), f2_fma(rh, f2_set(kLn2L), f2_mul(rl, lh)));
    const uint64_t p = f2_mul(sh, sh);
    const uint64_t pe = f2_fma(f2_add(sh, sh), sl, f2_fma(sh, sh, f2_neg(p)));
    const uint64_t q =
        f2_mul(f2_mul(p, sh), f2_fma(sh, f2_fma(sh, f2_set(-1.f / 120.f), f2_set(1.f / 24.f)),
                                     f2_set(-1.f / 6.f)));
    const uint64_t half = f2_set(0.5f);
    const uint64_t ah = f2_fma(p, half, nsh);
    const uint64_t al = f2_add(f2_fma(p, half, f2_neg(f2_add(ah, sh))),
                               f2_add(q, f2_sub(f2_mul(half, pe), sl)));
    const float2 t0 = table[j0 & 63], t1 = table[j1 & 63];
    const uint64_t th = f2_pack(t0.x, t1.x), tl = f2_pack(t0.y, t1.y);
    const uint64_t ph = f2_mul(th, ah);
    const uint64_t pl = f2_add(f2_fma(th, ah, f2_neg(ph)), f2_fma(th, al, f2_mul(tl, ah)));
    const uint64_t eh = f2_add(th, ph);
    const uint64_t el = f2_add(f2_sub(ph, f2_sub(eh, th)), f2_add(tl, pl));
    // (eh + el) 2^54 as an integer, eh >= 1/2 being a multiple of 2^-24 and el
    // below 2^-23, then rounded to k - n digits: conversions to 64-bit integers
    // run at a sixteenth of the rate of 32-bit ones.
    float a0, a1, b0, b1;
    f2_unpack(f2_mul(eh, f2_set(16777216.f)), a0, a1);
    f2_unpack(f2_mul(el, f2_set(18014398509481984.f)), b0, b1);
    auto fixed = [&](float a, float b, int j, bool far) -> uint64_t {
        const int64_t m = ((int64_t)__float2int_rn(a) << 30) + __float2int_rn(b);
        const int drop = 60 - k + (j >> 6);  // in [0, 62]
        const uint64_t w = (((uint64_t)m << 6) + ((1ull << drop) >> 1)) >> drop;
        return far ? 0 : w;
    };
    w0 = fixed(a0, b0, j0, far0);
    w1 = fixed(a1, b1, j1, far1);
}
__device__ __forceinline__ uint64_t fixed_weight(float z, float M, TempScale c, int k,
                                                 const float2* __restrict__ table) {
    uint64_t w, same;
    fixed_weights(z, z, M, c, k, table, w, same);
    return w;
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

// ---------------------------------------------------------------------------
// fp32 statistics of one chunk (PSTAT_CHUNK_* columns, 16 vectors of 16 bytes
// per lane), at the temperature's scale c = ch:
//   m = max z,  m2 = RN(m c),  delta = m c - m2 (exact),
//   a_i = RN(z_i c - m2),  s = sum 2^a_i,  u = sum 2^a_i a_i  (base 2),
// the form of chunk_math.cuh with c for log2(e).  Moving a chunk to the row
// maximum M multiplies by 2^((m - M) c - delta).  Where m c is so large that
// delta could weigh in the exponent, a_i = (z_i - m) c and delta = 0.
// -inf logits give 2^-inf = 0; only u needs them kept out (0 times -inf), so a
// chunk whose u comes out NaN is summed again with a_i held above -1024.
// A NaN or +inf logit makes the record's m NaN.
// ---------------------------------------------------------------------------
struct ChunkRecord {
    float m, s, u, delta;
};

__device__ __forceinline__ uint32_t bf2_max_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float warp_max_nan(float m) {
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(m));
    return r;
}

// Slot -> registers: lane L takes the 16 neighbouring vectors from 16 L, in an
// order turned by L so that the lanes of a quarter warp meet no bank twice;
// vectors past the chunk's end read as -inf.
template <typename E>
__device__ __forceinline__ void load_lane_run(const void* buf, int len, int lane,
                                              uint4 (&q)[kVecPerLane]) {
    const uint4* v = reinterpret_cast<const uint4*>(buf) + kVecPerLane * lane;
    constexpr int kVec = Elem<E>::kVec;
    const int nvec = (len + kVec - 1) / kVec - kVecPerLane * lane;
    if (len == Elem<E>::kChunk) {
#pragma unroll
        for (int j = 0; j < kVecPerLane; ++j) q[j] = v[(j + lane) & (kVecPerLane - 1)];
    } else {
#pragma unroll
        for (int j = 0; j < kVecPerLane; ++j) {
            const int at = (j + lane) & (kVecPerLane - 1);
            q[j] = at < nvec ? v[at] : Elem<E>::neg_inf_vec();
        }
    }
}

// The 16 bytes from byte `shift` (below 16, a multiple of 2) of two vectors.
__device__ __forceinline__ uint4 shift_vectors(const uint4& lo, const uint4& hi, uint32_t shift) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (shift & 8)
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    if (shift & 4)
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    if (shift & 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// load_lane_run of a chunk that starts `shift` bytes into the slot; the same
// vectors in the same places, so the same bits come out of them.
template <typename E>
__device__ __forceinline__ void load_lane_run_shifted(const void* buf, uint32_t shift, int len,
                                                      int lane, uint4 (&q)[kVecPerLane]) {
    const uint4* v = reinterpret_cast<const uint4*>(buf) + kVecPerLane * lane;
    constexpr int kVec = Elem<E>::kVec;
    const int nvec = (len + kVec - 1) / kVec - kVecPerLane * lane;
#pragma unroll
    for (int j = 0; j < kVecPerLane; ++j) {
        const int at = (j + lane) & (kVecPerLane - 1);
        q[j] = at < nvec ? shift_vectors(v[at], v[at + 1], shift) : Elem<E>::neg_inf_vec();
    }
}

// Maximum of one lane's vectors: the maximum of its group of columns.
__device__ __forceinline__ float lane_max(const uint4 (&q)[kVecPerLane], uint16_t*) {
    uint32_t a0 = q[0].x, a1 = q[0].y, a2 = q[0].z, a3 = q[0].w;
#pragma unroll
    for (int j = 1; j < kVecPerLane; ++j) {
        a0 = bf2_max_nan(a0, q[j].x);
        a1 = bf2_max_nan(a1, q[j].y);
        a2 = bf2_max_nan(a2, q[j].z);
        a3 = bf2_max_nan(a3, q[j].w);
    }
    const uint32_t a = bf2_max_nan(bf2_max_nan(a0, a1), bf2_max_nan(a2, a3));
    return max_nan(bf2_lo(a), bf2_hi(a));
}
__device__ __forceinline__ float lane_max(const uint4 (&q)[kVecPerLane], float*) {
    float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
    for (int j = 0; j < kVecPerLane; ++j) {
        a0 = max_nan(a0, max_nan(__uint_as_float(q[j].x), __uint_as_float(q[j].y)));
        a1 = max_nan(a1, max_nan(__uint_as_float(q[j].z), __uint_as_float(q[j].w)));
    }
    return max_nan(a0, a1);
}

// Pairs of floats of one 16-byte vector.
__device__ __forceinline__ void vector_pairs(const uint4& q, uint64_t (&p)[4], uint16_t*) {
    p[0] = f2_pack(bf2_lo(q.x), bf2_hi(q.x));
    p[1] = f2_pack(bf2_lo(q.y), bf2_hi(q.y));
    p[2] = f2_pack(bf2_lo(q.z), bf2_hi(q.z));
    p[3] = f2_pack(bf2_lo(q.w), bf2_hi(q.w));
}
__device__ __forceinline__ void vector_pairs(const uint4& q, uint64_t (&p)[2], float*) {
    p[0] = f2_pack(__uint_as_float(q.x), __uint_as_float(q.y));
    p[1] = f2_pack(__uint_as_float(q.z), __uint_as_float(q.w));
}

// kDirect: a = (z - m) c; else a = z c - m2.  kFloor: a >= -1024.
template <typename E, bool kU, bool kDirect, bool kFloor>
__device__ __forceinline__ void chunk_sums(const uint4 (&q)[kVecPerLane], float m, float c,
                                           float m2, float& s_out, float& u_out) {
    constexpr int kPairs = 8 / sizeof(E);
    const uint64_t cc = f2_pack(c, c), nm2 = f2_pack(-m2, -m2), nm = f2_pack(-m, -m);
    uint64_t s[kPairs], u[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) s[i] = u[i] = 0;
#pragma unroll
    for (int j = 0; j < kVecPerLane; ++j) {
        uint64_t z[kPairs];
        vector_pairs(q[j], z, (E*)nullptr);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            uint64_t a = kDirect ? f2_mul(f2_add(z[i], nm), cc) : f2_fma(z[i], cc, nm2);
            float a0, a1;
            f2_unpack(a, a0, a1);
            if (kFloor) {
                a0 = fmaxf(a0, -1024.f);
                a1 = fmaxf(a1, -1024.f);
                a = f2_pack(a0, a1);
            }
            const uint64_t e = f2_pack(ex2_approx(a0), ex2_approx(a1));
            s[i] = f2_add(s[i], e);
            if (kU) u[i] = f2_fma(e, a, u[i]);
        }
    }
    float st[kPairs], ut[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        st[i] = hsum2(s[i]);
        ut[i] = hsum2(u[i]);
    }
#pragma unroll
    for (int w = kPairs / 2; w; w >>= 1)
#pragma unroll
        for (int i = 0; i < w; ++i) {
            st[i] += st[i + w];
            ut[i] += ut[i + w];
        }
    float ss = st[0], uu = ut[0];
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
        if (kU) uu += __shfl_xor_sync(0xFFFFFFFFu, uu, off);
    }
    s_out = ss;
    u_out = kU ? uu : 0.f;
}

template <typename E, bool kU>
__device__ __forceinline__ ChunkRecord chunk_record(const uint4 (&q)[kVecPerLane], float lane_m,
                                                    float c) {
    const float m = warp_max_nan(lane_m);
    if (m == -INFINITY) return {m, 0.f, 0.f, 0.f};
    if (!(m < INFINITY)) return {NAN, 0.f, 0.f, 0.f};
    const float m2 = __fmul_rn(m, c);
    const float delta = fmaf(m, c, -m2);
    ChunkRecord r = {m, 0.f, 0.f, delta};
    if (fabsf(delta) <= 4.f) {  // false where m c overflows
        chunk_sums<E, kU, false, false>(q, m, c, m2, r.s, r.u);
        if (kU && r.u != r.u) chunk_sums<E, kU, false, true>(q, m, c, m2, r.s, r.u);
    } else {
        chunk_sums<E, kU, true, kU>(q, m, c, m2, r.s, r.u);
        r.delta = 0.f;
    }
    return r;
}

// Relative error of a sum of those records, and of its parts, against the
// exact sum: in units of 2^-24, ex2 4, the rounding of a (|a| + 4) ln 2 with a
// mass-weighted mean |a| of at most log2 V = 20, that of c half as much, 17
// for a lane's sums, 3 for its tree, 5 for the lanes, and 12 for the move to M
// and the fold: below 64, so 2^-18.  Measured errors are two orders smaller.
constexpr float kSumError = 1.f / 262144.f;

// The row's (M, S, U base 2) from its records, by one warp, every lane alike;
// NaN M where a record is bad, -inf where every logit is masked.
__device__ __forceinline__ float3 fold_records(const float4* rec, int n, float c,
                                               int lane) {
    // The usual rows have at most 64 chunks: both of a lane's records are loaded
    // before either is used.
    const float4 none = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    const float4 r0 = lane < n ? rec[lane] : none;
    const float4 r1 = lane + 32 < n ? rec[lane + 32] : none;
    float M = max_nan(r0.x, r1.x);
    for (int i = lane + 64; i < n; i += 32) M = max_nan(M, rec[i].x);
    M = warp_max_nan(M);
    float S = 0.f, U = 0.f;
    if (M > -INFINITY) {
        auto add = [&](const float4& r) {
            if (r.x == -INFINITY) return;
            const float a = fmaf(r.x - M, c, -r.w);
            const float f = exp2f(a);
            S = fmaf(r.y, f, S);
            U = fmaf(f, fmaf(fmaxf(a, -1024.f), r.y, r.z), U);
        };
        add(r0);
        add(r1);
        for (int i = lane + 64; i < n; i += 32) add(rec[i]);
#pragma unroll
        for (int off = 16; off; off >>= 1) {
            S += __shfl_xor_sync(0xFFFFFFFFu, S, off);
            U += __shfl_xor_sync(0xFFFFFFFFu, U, off);
        }
    }
    return make_float3(M, S, U);
}

}  // namespace pstat
