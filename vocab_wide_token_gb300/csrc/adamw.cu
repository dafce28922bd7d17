// adamw.cu -- an AdamW step over a list of tensors, with moments of 32 or 8 bits.
//
//   g' = f g,  f = min(1, max_norm / norm)
//   m  = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// One read and one write of everything, so bound by HBM: 28 bytes an element in fp32,
// 10 with bf16 parameters and gradients and 8-bit moments.  There the instructions weigh
// more than the bytes: 10 bytes at 6.7 TB/s leave an SM about 55 instructions for each
// element, and decoding, drawing (18), encoding and the step are 85, or 64 rounded to nearest.
// 60 million elements, with bf16 parameters and gradients unless said otherwise:
//   32-bit moments  203 us drawn, 6.5 TB/s; 191 to nearest; all in fp32 241 us, 7.0 TB/s
//   8-bit moments   171 us drawn, 3.5 TB/s; 124 us to nearest, 4.9 TB/s; fp32 drawn 153 us
// Codes of zero and values below the least code cost more, up to 30 us where nearly every
// block has some.
// A tensor with an address off 16 bytes goes element by element (step_block): 353 us to nearest
// and 488 drawn with 32-bit moments, 501 and 546 with 8-bit ones.
//
// 8-bit moments.  Codes of three bits of mantissa under an exponent that reaches a fixed
// number of binary orders below the largest of a block of 128: 4 bits and a sign for m
// (14 orders), 5 bits for v (30 orders, as v is a square).  A code is the upper bits of
// the fp32 number less the block's base, so that coding takes an addition and a shift.
// v moves by 1 - b2, a thousandth, in a step, and a step of its codes is an eighth: rounded
// to nearest it would stand still.  So a value is rounded up with the probability of
// its distance from the code below (by a hash of seed, tensor and element: the same call
// gives the same bits), and the mean moves as it should.  A v above zero never gets
// the code of zero, since its root divides the step.
//
// m and v are formed by the products and sums above, each rounded once to fp32 (no fused
// multiply-add), so the code of a value does not hang on the compiler.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <memory>
#include <new>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace pstat {
namespace {

constexpr int kAdThreads = 256;
constexpr int kAdBlock = 128;                   // elements that share an exponent: a warp's
constexpr int kAdUnit = 4096;                   // elements of one tensor, a CTA's turn
constexpr int kAdUnitSmall = 512;               // of one with 8-bit moments, a warp's
constexpr int kAdCtas = 2;                      // per SM
// Most CTAs for each SM of the forms that HBM alone bounds, whose reads and writes then come
// in turns: 60 million fp32 elements 242 us (260 with kAdCtas), the 8-bit moments' values 91 us
// (105 with 8).  A drawn step takes longer with more CTAs: 214 us, 202 with kAdCtas.
constexpr int kAdTurns = 64;
constexpr int kAdBatch = 600;                   // tensors of one launch (they travel as its arguments)
constexpr int kDepthM = 14, kDepthV = 30;       // binary orders below a block's largest

struct AdTensor {
    void* p;
    const void* g;
    void* m;
    void* v;
    int64_t n;
    uint32_t first_unit;
    uint32_t place;  // in the list
};
template <int N>
struct AdBatch {
    int count;
    uint32_t units;
    AdTensor t[N];
};

struct AdOptions {
    double lr, beta1, beta2, weight_decay;
    int64_t step;
    const float* lr_at;  // device values that take the place of the numbers, or null
    const int64_t* step_at;
    const int64_t* seed_at;
    const float* norm;
    float eps, max_norm;
    float decay, size, root;  // AdScalars', where neither lr nor the step lies on the device
    uint64_t seed;
    int random;
    int* dev_error;
};

// What the elements need of the options.
struct AdScalars {
    float b1, c1, b2, c2, eps, factor, decay, size, root;
    float rest;  // of the gradients' factor: 1, or a power of two (see scalars_of)
    uint32_t seed_key;
    int skip;        // bits of PSTAT_DEV_* for which nothing is done
    bool small_eps;  // the roots of subnormal numbers weigh against eps (see updated)
    bool tiny_eps;   // eps itself is no divisor for reciprocals that flush small ones
};

// 32 bits that are as good as random, from a counter under a key: two rounds of
// multiplications by odd constants (the fractions of the roots of 2 and 3) and shifts,
// with the key before and between them.  Each half is even over counters, keys and
// neighbours, so that a moment's mean is kept; the halves of one word (the draws of an
// element's two moments) depend on one another: a bit agrees in 36 to 64 of a hundred.
__device__ __forceinline__ uint32_t mix32(uint32_t x, uint32_t key) {
    x ^= key;
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x += key;
    x *= 0xBB67AE85u;
    return x ^ (x >> 16);
}

__host__ __device__ inline void corrections(double lr, double weight_decay, double beta1, double beta2, double t,
                                            float& decay, float& size, float& root) {
    decay = (float)(1.0 - lr * weight_decay);
    size = (float)(lr / (1.0 - pow(beta1, t)));
    root = (float)(1.0 / sqrt(1.0 - pow(beta2, t)));
}

__device__ AdScalars scalars_of(const AdOptions& o) {
    AdScalars s;
    s.b1 = (float)o.beta1;
    s.c1 = (float)(1.0 - o.beta1);
    s.b2 = (float)o.beta2;
    s.c2 = (float)(1.0 - o.beta2);
    s.eps = o.eps;
    s.decay = o.decay;
    s.size = o.size;
    s.root = o.root;
    s.skip = 0;
    if (o.lr_at || o.step_at) {
        const double lr = o.lr_at ? (double)*after_wait(o.lr_at) : o.lr;
        const double t = (double)(o.step_at ? *after_wait(o.step_at) : o.step);
        if (!(lr >= 0.0 && lr < INFINITY) || t < 1.0) s.skip |= PSTAT_DEV_BAD_PARAM;  // as the host's
        corrections(lr, o.weight_decay, o.beta1, o.beta2, t, s.decay, s.size, s.root);
    }
    s.small_eps = !(s.eps >= 0x1p-41f * s.root);
    s.tiny_eps = !(s.eps >= 0x1p-60f);
    s.factor = s.rest = 1.f;
    if (o.norm) {
        const float norm = *after_wait(o.norm);
        if (!(norm < INFINITY)) s.skip |= PSTAT_DEV_NONFINITE;
        if (norm > o.max_norm) s.factor = __fdiv_rn(o.max_norm, norm);
        // A factor below the normal numbers (max_norm < 4) has lost bits, while what it scales, up to
        // 2^128, comes out as a normal number: 2^125 times as large it keeps them.
        if (s.factor < 0x1p-126f) {
            s.factor = __fdiv_rn(__fmul_rn(o.max_norm, 0x1p125f), norm);
            s.rest = 0x1p-125f;
        }
    }
    const uint64_t seed = o.seed_at ? (uint64_t)*after_wait(o.seed_at) : o.seed;
    s.seed_key = mix32((uint32_t)(seed >> 32) ^ mix32((uint32_t)seed, 0x9E3779B9u), 0x3C6EF372u);
    return s;
}

__device__ __forceinline__ void unpack4(const uint2& q, float (&x)[4]) {
    x[0] = bf2_lo(q.x), x[1] = bf2_hi(q.x), x[2] = bf2_lo(q.y), x[3] = bf2_hi(q.y);
}
__device__ __forceinline__ void unpack4(const uint4& q, float (&x)[4]) {
    x[0] = __uint_as_float(q.x), x[1] = __uint_as_float(q.y);
    x[2] = __uint_as_float(q.z), x[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ float load1(const void* at, int64_t i, bool bf16) {
    return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(at)[i] << 16)
                : static_cast<const float*>(at)[i];
}

// The 8-bit codes of a block's elements: their exponent base, from the largest.
__device__ __forceinline__ int code_base(uint32_t top, int depth) { return max(((int)top - depth) * 8, 0); }

__device__ __forceinline__ float decode_m(uint32_t code, int base) {
    const uint32_t c = code & 127u;
    uint32_t b = c ? (uint32_t)((int)c + base) << 20 : 0u;
    if (c == 127u) b = 0x7FFFFFFFu;
    return __uint_as_float(b | (code & 128u) << 24);
}
__device__ __forceinline__ float decode_v(uint32_t code, int base) {
    const uint32_t b = code ? (uint32_t)((int)code + base) << 20 : 0u;
    return __uint_as_float(code == 255u ? 0x7FFFFFFFu : b);
}
// `draw`: 20 bits; the value is rounded up where its rest and the draw reach 2^20.
__device__ __forceinline__ uint32_t encode_m(float x, int base, uint32_t draw) {
    const uint32_t bits = __float_as_uint(x), a = bits & 0x7FFFFFFFu;
    int c = (int)((a + draw) >> 20) - base;
    if ((int)(a >> 20) - base < 1) {  // below the least value: that, with its probability, or zero
        const float least = __uint_as_float((uint32_t)(base + 1) << 20);
        c = fabsf(x) > least * ((float)draw * 0x1p-20f);
    }
    if (a >= 0x7F800000u) c = 127;
    return (uint32_t)c | (bits >> 24 & 128u);
}
__device__ __forceinline__ uint32_t encode_v(float x, int base, uint32_t draw) {
    const uint32_t a = __float_as_uint(x) & 0x7FFFFFFFu;
    int c = (int)((a + draw) >> 20) - base;
    if ((int)(a >> 20) - base < 1) c = a ? 1 : 0;
    return a >= 0x7F800000u ? 255u : (uint32_t)c;
}
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t a = __float_as_uint(x) & 0x7FFFFFFFu;
    return a < 0x7F800000u ? a : 0u;
}

// kAny: the factor may have a rest.
template <bool kAny>
__device__ __forceinline__ void moments(float g, const AdScalars& s, float& m, float& v) {
    const float x = kAny ? __fmul_rn(__fmul_rn(g, s.factor), s.rest) : __fmul_rn(g, s.factor);
    m = __fadd_rn(__fmul_rn(m, s.b1), __fmul_rn(x, s.c1));
    v = __fadd_rn(__fmul_rn(v, s.b2), __fmul_rn(__fmul_rn(x, x), s.c2));
}
// The root and the quotient are approximations of 2^-22: the step they give is a small
// part of the parameter, or all of one that was zero.  A root that flushes subnormal numbers drops
// up to 2^-63, which s.root multiplies: where eps is at least 2^22 times that, it is 2^-22 of the
// divisor.  Of a smaller eps (1e-15 at the first step with beta2 = 0.999: 0.3%) those numbers
// are scaled to normal ones first, and divisors as small likewise; others have the same bits
// either way.
__device__ __forceinline__ float updated_fast(float p, float m, float v, const AdScalars& s) {
    float root, step;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(v));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(step) : "f"(fmaf(root, s.root, s.eps)));
    return fmaf(-s.size, step * m, p * s.decay);
}
__device__ __forceinline__ float updated(float p, float m, float v, const AdScalars& s) {
    if (!s.small_eps) return updated_fast(p, m, v, s);
    const bool low = v < 0x1p-126f;
    float root, step;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(low ? v * 0x1p64f : v));
    if (low) root *= 0x1p-32f;
    const float divisor = fmaf(root, s.root, s.eps), scale = divisor < 0x1p-100f ? 0x1p100f : 1.f;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(step) : "f"(divisor * scale));
    return fmaf(-s.size, step * m * scale, p * s.decay);
}
// Two parameters to bf16; the draws' upper 16 bits are used.  kAny: they may be NaN.
template <bool kRandom, bool kAny>
__device__ __forceinline__ uint32_t to_bf16(float x, float y, uint32_t draw_x, uint32_t draw_y) {
    if (!kRandom) return bf2_pack_rn(x, y);
    uint32_t a = __float_as_uint(x) + (draw_x >> 16), b = __float_as_uint(y) + (draw_y >> 16);
    if (kAny && x != x) a = 0x7FC00000u;
    if (kAny && y != y) b = 0x7FC00000u;
    return __byte_perm(a, b, 0x7632);
}

// One tensor's addresses and keys, for the blocks of a unit.
struct AdView {
    void* p;
    const void* g;
    void* m;
    void* v;
    int64_t n;
    uint32_t key, key_p;
};
__device__ __forceinline__ AdView view_of(const AdTensor& at, const AdScalars& s) {
    const uint32_t key = mix32(s.seed_key ^ at.place, 0xDAA66D2Bu);
    return {at.p, after_wait(at.g), at.m, at.v, at.n, key, key ^ 0xA54FF53Au};
}
__device__ __forceinline__ uint32_t draw_of(const AdView& t, int64_t k) {
    return mix32((uint32_t)k, t.key + (uint32_t)(k >> 32) * 0x9E3779B9u);
}

// A block of 128 elements by a warp, whatever its alignment, size and values: element
// 128 b + 32 e + lane is a lane's e-th.
template <bool kBf16P, bool kBf16G, bool kSmall, bool kRandom>
__device__ __noinline__ void step_block(const AdView t, const AdScalars* shared, int64_t b) {
    const int lane = threadIdx.x & 31;
    const AdScalars s = *shared;
    uint8_t *m8 = static_cast<uint8_t*>(t.m), *v8 = static_cast<uint8_t*>(t.v);
    float *m32 = static_cast<float*>(t.m), *v32 = static_cast<float*>(t.v);
    int bm = 0, bv = 0;
    if (kSmall) {
        bm = code_base(m8[t.n + b], kDepthM);
        bv = code_base(v8[t.n + b], kDepthV);
    }
    float xp[4], xm[4], xv[4];
    uint32_t top_m = 0, top_v = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t k = b * kAdBlock + 32 * e + lane;
        const bool in = k < t.n;
        xp[e] = in ? load1(t.p, k, kBf16P) : 0.f;
        const float xg = in ? load1(t.g, k, kBf16G) : 0.f;
        if (kSmall) {
            xm[e] = decode_m(in ? m8[k] : 0u, bm);
            xv[e] = decode_v(in ? v8[k] : 0u, bv);
        } else {
            xm[e] = in ? m32[k] : 0.f;
            xv[e] = in ? v32[k] : 0.f;
        }
        moments<true>(xg, s, xm[e], xv[e]);
        xp[e] = updated(xp[e], xm[e], xv[e], s);
        top_m = max(top_m, finite_bits(xm[e]));
        top_v = max(top_v, finite_bits(xv[e]));
    }
    if (kSmall) {
        top_m = __reduce_max_sync(0xFFFFFFFFu, top_m) >> 23;
        top_v = __reduce_max_sync(0xFFFFFFFFu, top_v) >> 23;
        bm = code_base(top_m, kDepthM);
        bv = code_base(top_v, kDepthV);
        __syncwarp();  // every lane has read the old exponents
        if (lane == 0) {
            m8[t.n + b] = (uint8_t)top_m;
            v8[t.n + b] = (uint8_t)top_v;
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t k = b * kAdBlock + 32 * e + lane;
        if (k >= t.n) continue;
        const uint32_t h = kRandom ? draw_of(t, k) : 0x80008000u;  // nearest: half a step
        if (kBf16P)
            static_cast<uint16_t*>(t.p)[k] =
                (uint16_t)(to_bf16<kRandom, true>(xp[e], 0.f, kRandom ? mix32(h, t.key_p) : 0u, 0u) & 0xFFFFu);
        else
            static_cast<float*>(t.p)[k] = xp[e];
        if (kSmall) {
            const uint32_t low = kRandom ? 8u : 0u;
            m8[k] = (uint8_t)encode_m(xm[e], bm, h >> 16 << 4 | low);
            v8[k] = (uint8_t)encode_v(xv[e], bv, (h & 0xFFFFu) << 4 | low);
        } else {
            m32[k] = xm[e];
            v32[k] = xv[e];
        }
    }
}

// Copies 16 bytes to shared memory in the background, or none.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// A byte as a word that nothing has to be done with when it comes.
__device__ __forceinline__ uint32_t load_byte(const uint8_t* at) {
    uint32_t x;
    asm volatile("ld.global.u8 %0, [%1];" : "=r"(x) : "l"(at) : "memory");
    return x;
}
constexpr uint32_t kTopsSet = 1u << 16;  // beside a block's new exponents
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A warp's ring in shared memory, for 8-bit moments: stages of two neighbouring blocks each,
// their parameters, gradients, codes of m and codes of v.  What a lane holds for blocks on their
// way is then no register.
template <bool kBf16P, bool kBf16G>
struct AdRing {
    static constexpr int kBlocks = 2;
    static constexpr int kP = kAdBlock * (kBf16P ? 2 : 4), kG = kAdBlock * (kBf16G ? 2 : 4);  // bytes of a block
    static constexpr int kAtG = kBlocks * kP, kAtM = kAtG + kBlocks * kG, kAtV = kAtM + kBlocks * kAdBlock;
    static constexpr int kBytes = kAtV + kBlocks * kAdBlock;
    static constexpr int kStages = kBytes * 3 * (kAdThreads / 32) < 48 * 1024 ? 3 : 2;

    template <int kBytes>
    static __device__ __forceinline__ void copy(uint32_t dst, const char* src) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int at = 0; at < kBytes; at += 512)
            if (kBytes - at >= 512 || 16 * lane < kBytes - at) copy16(dst + at + 16 * lane, src + at + 16 * lane);
    }
    // The blocks from b on.
    static __device__ __forceinline__ void load(uint32_t stage, const AdView& t, int64_t b) {
        copy<kBlocks * kP>(stage, static_cast<const char*>(t.p) + b * kP);
        copy<kBlocks * kG>(stage + kAtG, static_cast<const char*>(t.g) + b * kG);
        copy<kBlocks * kAdBlock>(stage + kAtM, static_cast<const char*>(t.m) + b * kAdBlock);
        copy<kBlocks * kAdBlock>(stage + kAtV, static_cast<const char*>(t.v) + b * kAdBlock);
    }
};

// Blocks b and b + 1 with 8-bit moments, from a stage: element 128 b + 4 lane + e is a lane's
// e-th of block b.  Both go through each phase together, whose reductions and votes then
// overlap.  What is rare takes a branch of its own that the warp goes through together: codes
// of zero, values below the least code.  Where a code or a result is an infinity or NaN, or
// a root needs more care (small_eps), nothing is stored, for step_block: false.  `exponents`
// has lane b % 32's in its lower byte (m) and the next (v), and the new ones come out in the
// same way.
//   decoding   bits = (code << 20) + (base << 20)
//   encoding   the code is bits 20.. of bits + draw - (base << 20), which 16 times as large
//              is the upper byte
template <bool kBf16P, bool kBf16G, bool kRandom>
__device__ __forceinline__ bool step_small(const uint8_t* stage, uint32_t exponents, const AdView& t,
                                           const AdScalars& s, int64_t b, uint32_t& tops) {
    using Ring = AdRing<kBf16P, kBf16G>;
    using P = typename std::conditional<kBf16P, uint2, uint4>::type;
    using G = typename std::conditional<kBf16G, uint2, uint4>::type;
    constexpr int kN = Ring::kBlocks;
    const int lane = threadIdx.x & 31;
    const int64_t i = b * kAdBlock + 4 * lane;
    float xm[kN][4], xv[kN][4];
    uint32_t zeros = 0, nans = 0;
    uint32_t cm[kN], cv[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        cm[j] = *reinterpret_cast<const uint32_t*>(stage + Ring::kAtM + j * kAdBlock + 4 * lane);
        cv[j] = *reinterpret_cast<const uint32_t*>(stage + Ring::kAtV + j * kAdBlock + 4 * lane);
        const uint32_t top = __shfl_sync(0xFFFFFFFFu, exponents, ((int)b + j) & 31);
        const uint32_t Bm = (uint32_t)code_base(top & 255u, kDepthM) << 20;
        const uint32_t Bv = (uint32_t)code_base(top >> 8, kDepthV) << 20;
        const uint32_t w = cm[j] & 0x7F7F7F7Fu;
        // a byte of 127 (m) or 255 (v), and a byte of 0
        nans |= (w + 0x01010101u) | ((~cv[j] - 0x01010101u) & cv[j]);
        zeros |= (w - 0x01010101u) | ((cv[j] - 0x01010101u) & ~cv[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t a = __byte_perm(w, 0, 0x4440 + e), c = __byte_perm(cv[j], 0, 0x4440 + e);
            const uint32_t sign = (cm[j] << (24 - 8 * e)) & 0x80000000u;
            xm[j][e] = __uint_as_float(a * 0x100000u + Bm | sign);
            xv[j][e] = __uint_as_float(c * 0x100000u + Bv);
        }
    }
    if (__any_sync(0xFFFFFFFFu, zeros & 0x80808080u)) {
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!(cm[j] & 0x7Fu << (8 * e))) xm[j][e] = __uint_as_float(__float_as_uint(xm[j][e]) & 0x80000000u);
                if (!(cv[j] & 0xFFu << (8 * e))) xv[j][e] = 0.f;
            }
    }
    const uint32_t key = t.key + (uint32_t)(i >> 32) * 0x9E3779B9u;  // of both: b is even
    uint32_t h[kN][4], top_m[kN], top_v[kN];
    uint2 out_p[kN];
    float4 out_f[kN];
    float lost = 0.f;  // a NaN where a parameter is not finite
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        float xp[4], xg[4];
        uint32_t d[4] = {};
        unpack4(*reinterpret_cast<const P*>(stage + j * Ring::kP + (int)sizeof(P) * lane), xp);
        unpack4(*reinterpret_cast<const G*>(stage + Ring::kAtG + j * Ring::kG + (int)sizeof(G) * lane), xg);
        top_m[j] = top_v[j] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            moments<false>(xg[e], s, xm[j][e], xv[j][e]);
            top_m[j] = max(top_m[j], __float_as_uint(xm[j][e]) & 0x7FFFFFFFu);
            top_v[j] = max(top_v[j], __float_as_uint(xv[j][e]));  // no less than +0, or a NaN, which may have a sign
            xp[e] = updated_fast(xp[e], xm[j][e], xv[j][e], s);
            if (kBf16P && kRandom) lost = fmaf(xp[e], 0.f, lost);
            h[j][e] = kRandom ? mix32((uint32_t)i + j * kAdBlock + e, key) : 0u;
            if (kBf16P && kRandom) d[e] = mix32(h[j][e], t.key_p);
        }
        if (kBf16P)
            out_p[j] = make_uint2(to_bf16<kRandom, false>(xp[0], xp[1], d[0], d[1]),
                                  to_bf16<kRandom, false>(xp[2], xp[3], d[2], d[3]));
        else
            out_f[j] = make_float4(xp[0], xp[1], xp[2], xp[3]);
    }
    bool whole = true;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        top_m[j] = __reduce_max_sync(0xFFFFFFFFu, top_m[j]);
        top_v[j] = __reduce_max_sync(0xFFFFFFFFu, top_v[j]);
        whole = whole && top_m[j] < 0x7F800000u && top_v[j] < 0x7F800000u;
    }
    if (s.small_eps)
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)  // above zero, below 2^-126
                whole = whole && __float_as_uint(xv[j][e]) - 1u >= 0x7FFFFFu;
    if (__any_sync(0xFFFFFFFFu, !whole || (nans & 0x80808080u) || lost != lost)) return false;
    uint32_t ym[kN][4], yv[kN][4];
    bool low = false;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        top_m[j] >>= 23;
        top_v[j] >>= 23;
        const uint32_t Bm = (uint32_t)code_base(top_m[j], kDepthM) << 20;
        const uint32_t Bv = (uint32_t)code_base(top_v[j], kDepthV) << 20;
        const uint32_t half = kRandom ? 8u : 0x80000u;
        uint32_t least_m = 0xFFFFFFFFu, least_v = 0xFFFFFFFFu;
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // a draw is 16 bits, times 16, and a half of that
            const uint32_t m = __float_as_uint(xm[j][e]), a = m & 0x7FFFFFFFu, v = __float_as_uint(xv[j][e]);
            least_m = min(least_m, a);
            least_v = min(least_v, v);
            ym[j][e] = a * 16u + (half - Bm) * 16u + (kRandom ? __byte_perm(h[j][e], 0, 0x4324) : 0u);
            yv[j][e] = v * 16u + (half - Bv) * 16u + (kRandom ? __byte_perm(h[j][e], 0, 0x4104) : 0u);
            ym[j][e] |= m & 0x80000000u;
        }
        low = low || least_m < Bm + (1u << 20) || least_v < Bv + (1u << 20);
    }
    if (__any_sync(0xFFFFFFFFu, low)) {
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            const uint32_t least_m = ((uint32_t)code_base(top_m[j], kDepthM) << 20) + (1u << 20);
            const uint32_t least_v = ((uint32_t)code_base(top_v[j], kDepthV) << 20) + (1u << 20);
            // Nine eighths of a power of two, or 2^-129: this product and that with a draw are
            // exact, as encode_m's are.
            const float unit = __uint_as_float(least_m) * 0x1p-20f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t draw = kRandom ? (h[j][e] >> 12 & 0xFFFF0u) | 8u : 0x80000u;
                if ((__float_as_uint(xm[j][e]) & 0x7FFFFFFFu) < least_m)
                    ym[j][e] = (__float_as_uint(xm[j][e]) & 0x80000000u) |
                               (fabsf(xm[j][e]) > unit * (float)draw ? 1u << 24 : 0u);
                if (__float_as_uint(xv[j][e]) < least_v) yv[j][e] = xv[j][e] != 0.f ? 1u << 24 : 0u;
            }
        }
    }
    uint8_t *m8 = static_cast<uint8_t*>(t.m), *v8 = static_cast<uint8_t*>(t.v);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        const int64_t at = i + j * kAdBlock;
        if (kBf16P)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(t.p) + at) = out_p[j];
        else
            *reinterpret_cast<float4*>(static_cast<float*>(t.p) + at) = out_f[j];
        *reinterpret_cast<uint32_t*>(m8 + at) = __byte_perm(__byte_perm(ym[j][0], ym[j][1], 0x0073),
                                                            __byte_perm(ym[j][2], ym[j][3], 0x0073), 0x5410);
        *reinterpret_cast<uint32_t*>(v8 + at) = __byte_perm(__byte_perm(yv[j][0], yv[j][1], 0x0073),
                                                            __byte_perm(yv[j][2], yv[j][3], 0x0073), 0x5410);
    }
#pragma unroll
    for (int j = 0; j < kN; ++j)
        if (lane == (((int)b + j) & 31)) tops = top_m[j] | top_v[j] << 8 | kTopsSet;
    return true;
}

// Two whole blocks with 32-bit moments from b on, as above; all loads come before the first use.
template <bool kBf16P, bool kBf16G, bool kRandom>
__device__ __forceinline__ void step_wide(const AdView& t, const AdScalars& s, int64_t b) {
    using P = typename std::conditional<kBf16P, uint2, uint4>::type;
    using G = typename std::conditional<kBf16G, uint2, uint4>::type;
    float *m32 = static_cast<float*>(t.m), *v32 = static_cast<float*>(t.v);
    P rp[2];
    G rg[2];
    uint4 rm[2], rv[2];
    const int64_t i0 = b * kAdBlock + 4 * (threadIdx.x & 31);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t i = i0 + j * kAdBlock;
        rp[j] = *reinterpret_cast<const P*>(static_cast<const char*>(t.p) + i * (kBf16P ? 2 : 4));
        rg[j] = *reinterpret_cast<const G*>(static_cast<const char*>(t.g) + i * (kBf16G ? 2 : 4));
        rm[j] = *reinterpret_cast<const uint4*>(m32 + i);
        rv[j] = *reinterpret_cast<const uint4*>(v32 + i);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t i = i0 + j * kAdBlock;
        float xp[4], xg[4], xm[4], xv[4];
        uint32_t d[4] = {};
        unpack4(rp[j], xp);
        unpack4(rg[j], xg);
        unpack4(rm[j], xm);
        unpack4(rv[j], xv);
        const uint32_t key = t.key + (uint32_t)(i >> 32) * 0x9E3779B9u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            moments<false>(xg[e], s, xm[e], xv[e]);
            xp[e] = updated(xp[e], xm[e], xv[e], s);
            if (kBf16P && kRandom) d[e] = mix32(mix32((uint32_t)i + e, key), t.key_p);
        }
        if (kBf16P)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(t.p) + i) = make_uint2(
                to_bf16<kRandom, true>(xp[0], xp[1], d[0], d[1]), to_bf16<kRandom, true>(xp[2], xp[3], d[2], d[3]));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(t.p) + i) = make_float4(xp[0], xp[1], xp[2], xp[3]);
        *reinterpret_cast<float4*>(m32 + i) = make_float4(xm[0], xm[1], xm[2], xm[3]);
        *reinterpret_cast<float4*>(v32 + i) = make_float4(xv[0], xv[1], xv[2], xv[3]);
    }
}

// A warp's units [u0, u1) of a tensor with 8-bit moments: neighbouring blocks, so that the warp
// reads and writes the exponents of 32 blocks at once.  (Written a byte at a time by all warps
// of a CTA, which read others of the same 32 bytes meanwhile, they held it up: 60 million
// bf16 elements in 218 us, 171 so.)
template <bool kBf16P, bool kBf16G, bool kRandom>
__device__ __forceinline__ void step_small_units(const AdTensor& at, uint32_t u0, uint32_t u1, const AdScalars& s,
                                                 const AdScalars* shared, uint8_t* ring) {
    using Ring = AdRing<kBf16P, kBf16G>;
    constexpr int kPerUnit = kAdUnitSmall / kAdBlock, kAhead = Ring::kStages - 1;
    static_assert(kPerUnit % Ring::kBlocks == 0 && Ring::kBlocks == 2, "");
    const int lane = threadIdx.x & 31;
    const AdView t = view_of(at, s);
    const bool quick = ((reinterpret_cast<uintptr_t>(t.p) | reinterpret_cast<uintptr_t>(t.g) |
                         reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v)) &
                        15u) == 0 &&
                       !s.tiny_eps && s.rest == 1.f;
    int64_t b = (int64_t)(u0 - at.first_unit) * kPerUnit;
    const int64_t blocks = min((t.n + kAdBlock - 1) / kAdBlock, (int64_t)(u1 - at.first_unit) * kPerUnit);
    const int64_t end = quick ? min(blocks, t.n / kAdBlock - 1) : b;  // up to here there are two whole blocks
    uint8_t *em = static_cast<uint8_t*>(t.m) + t.n, *ev = static_cast<uint8_t*>(t.v) + t.n;
    const int64_t last = t.n / kAdBlock - 1;
    const uint32_t ring_at = smem_u32(ring);
    int64_t chunk = b >> 5;
    uint32_t tops = 0, exponents = 0, next_m = 0, next_v = 0;
    if (b < end) {
        const int64_t k = min(chunk * 32 + lane, last), l = min(k + 32, last);
        exponents = load_byte(em + k) | load_byte(ev + k) << 8;
        next_m = load_byte(em + l);
        next_v = load_byte(ev + l);
    }
    while (true) {
        __syncwarp();  // the ring has been read
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (b + 2 * k < end) Ring::load(ring_at + k * Ring::kBytes, t, b + 2 * k);
            copies_commit();
        }
        int stage = 0, fill = kAhead;
        bool done = true;
#pragma unroll 1
        for (; b < end; b += 2) {
            if (b >> 5 != chunk) {
                chunk = b >> 5;
                exponents = next_m | next_v << 8;
                const int64_t l = min(chunk * 32 + 32 + lane, last);
                next_m = load_byte(em + l);
                next_v = load_byte(ev + l);
            }
            copies_wait<kAhead - 1>();
            __syncwarp();  // all lanes' copies are there, and all have read the stage before
            if (b + 2 * kAhead < end) Ring::load(ring_at + fill * Ring::kBytes, t, b + 2 * kAhead);
            copies_commit();
            done = step_small<kBf16P, kBf16G, kRandom>(ring + stage * Ring::kBytes, exponents, t, s, b, tops);
            if (!done) break;
            stage = stage + 1 == Ring::kStages ? 0 : stage + 1;
            fill = fill + 1 == Ring::kStages ? 0 : fill + 1;
            if ((b & 31) == 30 || b + 2 >= end) {
                if (tops & kTopsSet) {
                    em[chunk * 32 + lane] = (uint8_t)tops;
                    ev[chunk * 32 + lane] = (uint8_t)(tops >> 8);
                }
                tops = 0;
            }
        }
        copies_wait<0>();
        if (done) break;
        // Blocks that step_block does; what it writes of the exponents stays.
        step_block<kBf16P, kBf16G, true, kRandom>(t, shared, b);
        step_block<kBf16P, kBf16G, true, kRandom>(t, shared, b + 1);
        if (((b & 31) == 30 || b + 2 >= end) && (tops & kTopsSet)) {
            em[chunk * 32 + lane] = (uint8_t)tops;
            ev[chunk * 32 + lane] = (uint8_t)(tops >> 8);
        }
        if ((b & 31) == 30) tops = 0;
        b += 2;
    }
    for (; b < blocks; ++b) step_block<kBf16P, kBf16G, true, kRandom>(t, shared, b);
}

// A CTA's units [u0, u1) of a tensor with 32-bit moments: a warp takes two neighbouring blocks
// every 16.
template <bool kBf16P, bool kBf16G, bool kRandom>
__device__ __forceinline__ void step_wide_units(const AdTensor& at, uint32_t u0, uint32_t u1, const AdScalars& s,
                                                const AdScalars* shared) {
    constexpr int kPerUnit = kAdUnit / kAdBlock, kTurn = kAdThreads / 32 * 2;
    static_assert(kPerUnit % kTurn == 0, "");
    const AdView t = view_of(at, s);
    const bool quick =
        ((reinterpret_cast<uintptr_t>(t.p) & (kBf16P ? 7u : 15u)) |
         (reinterpret_cast<uintptr_t>(t.g) & (kBf16G ? 7u : 15u)) |
         ((reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v)) & 15u)) == 0 &&
        s.rest == 1.f;
    int64_t b = (int64_t)(u0 - at.first_unit) * kPerUnit + (threadIdx.x >> 5) * 2;
    const int64_t blocks = min((t.n + kAdBlock - 1) / kAdBlock, (int64_t)(u1 - at.first_unit) * kPerUnit);
    const int64_t end = quick ? min(blocks, t.n / kAdBlock - 1) : 0;  // up to here there are two whole blocks
#pragma unroll 1
    for (; b < end; b += kTurn) step_wide<kBf16P, kBf16G, kRandom>(t, s, b);
    for (; b < blocks; b += kTurn)
        for (int64_t k = b; k < min(b + 2, blocks); ++k) step_block<kBf16P, kBf16G, false, kRandom>(t, shared, k);
}

template <int N>
__device__ __forceinline__ int ad_tensor_of(const AdBatch<N>& g, uint32_t u) {
    int lo = 0, hi = g.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (g.t[mid].first_unit <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// One kind of tensors to a launch, so that each has the registers that it needs.
template <int N, bool kBf16P, bool kBf16G, bool kSmall, bool kRandom>
__global__ void __launch_bounds__(kAdThreads, kBf16P && !kSmall && !kRandom ? 3 : kAdCtas)
    adamw_kernel(const __grid_constant__ AdBatch<N> b, const __grid_constant__ AdOptions o) {
    using Ring = AdRing<kBf16P, kBf16G>;
    __shared__ AdScalars shared;
    __shared__ __align__(16) uint8_t rings[kSmall ? kAdThreads / 32 * Ring::kStages * Ring::kBytes : 16];
    uint8_t* ring = kSmall ? rings + (threadIdx.x >> 5) * Ring::kStages * Ring::kBytes : nullptr;
    // units go to CTAs in turn, those of 8-bit moments to warps
    const uint32_t parts = kSmall ? gridDim.x * (kAdThreads / 32) : gridDim.x;
    const uint32_t part = kSmall ? blockIdx.x * (kAdThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    const uint32_t u0 = (uint32_t)((uint64_t)b.units * part / parts);
    const uint32_t u1 = (uint32_t)((uint64_t)b.units * (part + 1) / parts);
    grid_wait();
    if (threadIdx.x == 0) {
        shared = scalars_of(o);
        if (shared.skip && blockIdx.x == 0 && o.dev_error) atomicOr(o.dev_error, shared.skip);
    }
    __syncthreads();
    const AdScalars s = shared;
    if (s.skip || u0 == u1) return;
    int i = ad_tensor_of(b, u0);
    for (uint32_t u = u0; u < u1; ++i) {
        const uint32_t end = i + 1 < b.count ? min(u1, b.t[i + 1].first_unit) : u1;
        if (kSmall)
            step_small_units<kBf16P, kBf16G, kRandom>(b.t[i], u, end, s, &shared, ring);
        else
            step_wide_units<kBf16P, kBf16G, kRandom>(b.t[i], u, end, s, &shared);
        u = end;
    }
}

// The values that 8-bit moments stand for.  Here a tensor's p and g are the outputs.
template <int N>
__global__ void __launch_bounds__(kAdThreads) adamw_moments_kernel(const __grid_constant__ AdBatch<N> b) {
    const uint32_t u0 = (uint32_t)((uint64_t)b.units * blockIdx.x / gridDim.x);
    const uint32_t u1 = (uint32_t)((uint64_t)b.units * (blockIdx.x + 1) / gridDim.x);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int i = ad_tensor_of(b, u0);
    grid_wait();
    for (uint32_t u = u0; u < u1; ++u) {
        while (i + 1 < b.count && b.t[i + 1].first_unit <= u) ++i;
        const AdTensor& t = b.t[i];
        const uint8_t* m = static_cast<const uint8_t*>(after_wait(t.m));
        const uint8_t* v = static_cast<const uint8_t*>(after_wait(t.v));
        float* om = static_cast<float*>(t.p);
        float* ov = static_cast<float*>(const_cast<void*>(t.g));
        const bool aligned = ((reinterpret_cast<uintptr_t>(om) | reinterpret_cast<uintptr_t>(ov)) & 15u) == 0 &&
                             ((reinterpret_cast<uintptr_t>(m) | reinterpret_cast<uintptr_t>(v)) & 3u) == 0;
        const int64_t b0 = (int64_t)(u - t.first_unit) * (kAdUnit / kAdBlock);
        constexpr int kRows = kAdUnit / kAdBlock / (kAdThreads / 32);  // blocks of a warp
        const int64_t k0 = b0 + warp * kRows;
        if (aligned && (k0 + kRows) * kAdBlock <= t.n) {
            uint32_t cm[kRows], cv[kRows], em[kRows], ev[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                cm[r] = *reinterpret_cast<const uint32_t*>(m + (k0 + r) * kAdBlock + 4 * lane);
                cv[r] = *reinterpret_cast<const uint32_t*>(v + (k0 + r) * kAdBlock + 4 * lane);
                em[r] = m[t.n + k0 + r];
                ev[r] = v[t.n + k0 + r];
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int bm = code_base(em[r], kDepthM), bv = code_base(ev[r], kDepthV);
                const int64_t e0 = (k0 + r) * kAdBlock + 4 * lane;
                *reinterpret_cast<float4*>(om + e0) =
                    make_float4(decode_m(cm[r] & 255u, bm), decode_m(cm[r] >> 8 & 255u, bm),
                                decode_m(cm[r] >> 16 & 255u, bm), decode_m(cm[r] >> 24, bm));
                *reinterpret_cast<float4*>(ov + e0) =
                    make_float4(decode_v(cv[r] & 255u, bv), decode_v(cv[r] >> 8 & 255u, bv),
                                decode_v(cv[r] >> 16 & 255u, bv), decode_v(cv[r] >> 24, bv));
            }
        } else {
            for (int64_t k = k0; k < k0 + kRows && k * kAdBlock < t.n; ++k) {
                const int bm = code_base(m[t.n + k], kDepthM), bv = code_base(v[t.n + k], kDepthV);
                for (int64_t e = k * kAdBlock + lane; e < min(t.n, (k + 1) * kAdBlock); e += 32) {
                    om[e] = decode_m(m[e], bm);
                    ov[e] = decode_v(v[e], bv);
                }
            }
        }
    }
}

struct Span {
    uintptr_t from, to;
    bool written;
};
// Whether something written overlaps anything else of the call.
int spans_overlap(Span* s, int64_t n) {
    const auto before = [](const Span& a, const Span& b) { return a.from < b.from; };
    if (!std::is_sorted(s, s + n, before)) std::sort(s, s + n, before);
    uintptr_t end_any = 0, end_written = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (s[i].from < (s[i].written ? end_any : end_written)) return PSTAT_ERR_PARAM;
        end_any = std::max(end_any, s[i].to);
        if (s[i].written) end_written = std::max(end_written, s[i].to);
    }
    return PSTAT_OK;
}

int64_t state_bytes(int64_t n, int bits) { return bits == 8 ? n + (n + kAdBlock - 1) / kAdBlock : 4 * n; }
int64_t type_bytes(int dtype) { return dtype == PSTAT_BF16 ? 2 : 4; }
bool at_least(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
Span span_of(const void* p, int64_t bytes, bool written) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + (uintptr_t)bytes, written};
}

int check_adamw(const pstat_adamw_tensor* tensors, int64_t n) {
    if (n < 0 || n > PSTAT_ADAMW_MAX_TENSORS) return PSTAT_ERR_SHAPE;
    if (n > 0 && !tensors) return PSTAT_ERR_NULLPTR;
    for (int64_t i = 0; i < n; ++i) {
        const pstat_adamw_tensor& t = tensors[i];
        if ((t.param_dtype != PSTAT_F32 && t.param_dtype != PSTAT_BF16) ||
            (t.grad_dtype != PSTAT_F32 && t.grad_dtype != PSTAT_BF16) || (t.bits != 8 && t.bits != 32))
            return PSTAT_ERR_DTYPE;
        if (t.n < 0 || t.n > PSTAT_GRAD_MAX_ELEMENTS) return PSTAT_ERR_SHAPE;
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return PSTAT_ERR_NULLPTR;
        const uintptr_t state = t.bits == 8 ? 1 : 4;
        if (!at_least(t.param, type_bytes(t.param_dtype)) || !at_least(t.grad, type_bytes(t.grad_dtype)) ||
            !at_least(t.exp_avg, state) || !at_least(t.exp_avg_sq, state))
            return PSTAT_ERR_ALIGN;
    }
    if (n == 0) return PSTAT_OK;
    std::unique_ptr<Span[]> spans(new (std::nothrow) Span[4 * n]);
    if (!spans) return PSTAT_ERR_WORKSPACE;
    int64_t k = 0;
    for (int64_t i = 0; i < n; ++i) {
        const pstat_adamw_tensor& t = tensors[i];
        if (t.n == 0) continue;
        spans[k++] = span_of(t.param, t.n * type_bytes(t.param_dtype), true);
        spans[k++] = span_of(t.grad, t.n * type_bytes(t.grad_dtype), false);
        spans[k++] = span_of(t.exp_avg, state_bytes(t.n, t.bits), true);
        spans[k++] = span_of(t.exp_avg_sq, state_bytes(t.n, t.bits), true);
    }
    return spans_overlap(spans.get(), k);
}

int check_options(const pstat_adamw_options* o) {
    if (!o) return PSTAT_ERR_NULLPTR;
    // the bounds also refuse NaN
    if (!o->lr_at && !(o->lr >= 0.0 && o->lr < INFINITY)) return PSTAT_ERR_PARAM;
    if (!o->step_at && o->step < 1) return PSTAT_ERR_PARAM;
    if (!(o->beta1 >= 0.0 && o->beta1 < 1.0) || !(o->beta2 >= 0.0 && o->beta2 < 1.0)) return PSTAT_ERR_PARAM;
    if (!(o->eps >= 0.0 && o->eps < INFINITY) || !(o->weight_decay >= 0.0 && o->weight_decay < INFINITY))
        return PSTAT_ERR_PARAM;
    if (o->norm && !(o->max_norm >= 0.f)) return PSTAT_ERR_PARAM;
    if (!at_least(o->lr_at, 4) || !at_least(o->step_at, 8) || !at_least(o->seed_at, 8) || !at_least(o->norm, 4))
        return PSTAT_ERR_ALIGN;
    return PSTAT_OK;
}

// Appends a tensor to a batch; false when it is full or its units pass 32 bits.
template <int N>
bool add_tensor(AdBatch<N>& b, uint64_t& units, const AdTensor& t, int unit) {
    const uint64_t add = (uint64_t)((t.n + unit - 1) / unit);
    if (b.count == N || units + add > 0xFFFFFFFFull) return false;
    b.t[b.count] = t;
    b.t[b.count++].first_unit = (uint32_t)units;
    units += add;
    b.units = (uint32_t)units;
    return true;
}

unsigned grid_of(uint32_t units, int per_sm, const DeviceInfo& dev) {
    const uint32_t most = (uint32_t)dev.sm_count * per_sm;
    return units < most ? units : most;
}

// Bit 0: bf16 parameter, 1: bf16 gradient, 2: 8-bit moments.
uint32_t kind_of(const pstat_adamw_tensor& t) {
    return (t.param_dtype == PSTAT_BF16 ? 1u : 0u) | (t.grad_dtype == PSTAT_BF16 ? 2u : 0u) | (t.bits == 8 ? 4u : 0u);
}

template <int N, uint32_t kKind, bool kRandom>
int run_kind(const pstat_adamw_tensor* tensors, int64_t n, const AdOptions& o, const DeviceInfo& dev,
             cudaStream_t st) {
    constexpr bool kSmall = (kKind & 4u) != 0;
    AdBatch<N> b;
    for (int64_t i = 0; i < n;) {
        b.count = 0;
        b.units = 0;
        uint64_t units = 0;
        for (; i < n; ++i) {
            const pstat_adamw_tensor& t = tensors[i];
            if (t.n == 0 || kind_of(t) != kKind) continue;
            if (!add_tensor(b, units, {t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.n, 0u, (uint32_t)i},
                            kSmall ? kAdUnitSmall : kAdUnit))
                break;
        }
        // Many short CTAs where starting one costs little: no draws' keys, and no powers of the betas.
        const int turns = kSmall || kRandom || o.lr_at || o.step_at ? kAdCtas : kAdTurns;
        const uint32_t ctas = kSmall ? (b.units - 1) / (kAdThreads / 32) + 1 : b.units;
        if (b.count && launch_behind(adamw_kernel<N, (kKind & 1u) != 0, (kKind & 2u) != 0, kSmall, kRandom>,
                                     grid_of(ctas, turns, dev), kAdThreads, 0, st, 1, b, o) != cudaSuccess)
            return PSTAT_ERR_CUDA;
    }
    return PSTAT_OK;
}

template <int N>
int run_adamw(const pstat_adamw_tensor* tensors, int64_t n, const AdOptions& o, const DeviceInfo& dev,
              cudaStream_t st) {
    uint32_t present = 0;
    for (int64_t i = 0; i < n; ++i)
        if (tensors[i].n) present |= 1u << kind_of(tensors[i]);
    for (uint32_t kind = 0; kind < 8; ++kind) {
        if (!(present >> kind & 1u)) continue;
        int rc = PSTAT_OK;
        // draws are for what is held in fewer than 32 bits
        switch (kind | (o.random && (kind & 5u) ? 8u : 0u)) {
            case 0: rc = run_kind<N, 0, false>(tensors, n, o, dev, st); break;
            case 1: rc = run_kind<N, 1, false>(tensors, n, o, dev, st); break;
            case 2: rc = run_kind<N, 2, false>(tensors, n, o, dev, st); break;
            case 3: rc = run_kind<N, 3, false>(tensors, n, o, dev, st); break;
            case 4: rc = run_kind<N, 4, false>(tensors, n, o, dev, st); break;
            case 5: rc = run_kind<N, 5, false>(tensors, n, o, dev, st); break;
            case 6: rc = run_kind<N, 6, false>(tensors, n, o, dev, st); break;
            case 7: rc = run_kind<N, 7, false>(tensors, n, o, dev, st); break;
            case 9: rc = run_kind<N, 1, true>(tensors, n, o, dev, st); break;
            case 11: rc = run_kind<N, 3, true>(tensors, n, o, dev, st); break;
            case 12: rc = run_kind<N, 4, true>(tensors, n, o, dev, st); break;
            case 13: rc = run_kind<N, 5, true>(tensors, n, o, dev, st); break;
            case 14: rc = run_kind<N, 6, true>(tensors, n, o, dev, st); break;
            default: rc = run_kind<N, 7, true>(tensors, n, o, dev, st); break;
        }
        if (rc != PSTAT_OK) return rc;
    }
    return PSTAT_OK;
}

template <int N>
int run_moments(const pstat_adamw_moment* list, int64_t n, const DeviceInfo& dev, cudaStream_t st) {
    AdBatch<N> b;
    for (int64_t i = 0; i < n;) {
        b.count = 0;
        b.units = 0;
        uint64_t units = 0;
        for (; i < n; ++i) {
            const pstat_adamw_moment& t = list[i];
            if (t.n == 0) continue;
            if (!add_tensor(b, units, {t.out_avg, t.out_avg_sq, const_cast<void*>(t.exp_avg),
                                       const_cast<void*>(t.exp_avg_sq), t.n, 0u, (uint32_t)i},
                            kAdUnit))
                break;
        }
        if (b.count &&
            launch_behind(adamw_moments_kernel<N>, grid_of(b.units, kAdTurns, dev), kAdThreads, 0, st, 1, b) != cudaSuccess)
            return PSTAT_ERR_CUDA;
    }
    return PSTAT_OK;
}

}  // namespace
}  // namespace pstat

using namespace pstat;

extern "C" {

int pstat_adamw_step(const pstat_adamw_tensor* tensors, int64_t n_tensors, const pstat_adamw_options* options,
                     int* dev_error, pstat_stream_t stream) {
    int rc = check_options(options);
    if (rc != PSTAT_OK) return rc;
    rc = check_adamw(tensors, n_tensors);
    if (rc != PSTAT_OK || n_tensors == 0) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != PSTAT_OK) return rc;
    const pstat_adamw_options& p = *options;
    AdOptions o = {p.lr, p.beta1, p.beta2, p.weight_decay, p.step, p.lr_at, p.step_at, p.seed_at, p.norm,
                   (float)p.eps, p.max_norm, 0.f, 0.f, 0.f, p.seed, p.random, dev_error};
    if (!p.lr_at && !p.step_at)
        corrections(p.lr, p.weight_decay, p.beta1, p.beta2, (double)p.step, o.decay, o.size, o.root);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return n_tensors <= 32 ? run_adamw<32>(tensors, n_tensors, o, dev, st)
                           : run_adamw<kAdBatch>(tensors, n_tensors, o, dev, st);
}

int pstat_adamw_moments(const pstat_adamw_moment* list, int64_t n, pstat_stream_t stream) {
    if (n < 0 || n > PSTAT_ADAMW_MAX_TENSORS) return PSTAT_ERR_SHAPE;
    if (n == 0) return PSTAT_OK;
    if (!list) return PSTAT_ERR_NULLPTR;
    std::unique_ptr<Span[]> spans(new (std::nothrow) Span[4 * n]);
    if (!spans) return PSTAT_ERR_WORKSPACE;
    int64_t k = 0;
    for (int64_t i = 0; i < n; ++i) {
        const pstat_adamw_moment& t = list[i];
        if (t.n < 0 || t.n > PSTAT_GRAD_MAX_ELEMENTS) return PSTAT_ERR_SHAPE;
        if (t.n == 0) continue;
        if (!t.exp_avg || !t.exp_avg_sq || !t.out_avg || !t.out_avg_sq) return PSTAT_ERR_NULLPTR;
        if (!at_least(t.out_avg, 4) || !at_least(t.out_avg_sq, 4)) return PSTAT_ERR_ALIGN;
        spans[k++] = span_of(t.exp_avg, state_bytes(t.n, 8), false);
        spans[k++] = span_of(t.exp_avg_sq, state_bytes(t.n, 8), false);
        spans[k++] = span_of(t.out_avg, 4 * t.n, true);
        spans[k++] = span_of(t.out_avg_sq, 4 * t.n, true);
    }
    int rc = spans_overlap(spans.get(), k);
    if (rc != PSTAT_OK) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != PSTAT_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return n <= 32 ? run_moments<32>(list, n, dev, st) : run_moments<kAdBatch>(list, n, dev, st);
}

}  // extern "C"
