// adamw.cu -- an AdamW step over a list of tensors, with moments of 32 or 8 bits.
//
//   g' = f g,  f = min(1, max_norm / norm)
//   m  = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// One read and one write of everything, so bound by HBM: 28 bytes an element in fp32,
// 10 with bf16 parameters and gradients and 8-bit moments.  There the instructions weigh
// as much as the bytes: 10 bytes at 6.7 TB/s leave an SM about 55 instructions for
// each element, and decoding, drawing, encoding and the step take most of them.
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

#include "internal.h"
#include "ptx.cuh"

namespace pstat {
namespace {

constexpr int kAdThreads = 256;
constexpr int kAdBlock = 128;                   // elements that share an exponent: a warp's
constexpr int kAdUnit = 4096;                   // elements of one tensor, a CTA's turn
constexpr int kAdCtas = 2;                      // per SM
constexpr int kAdBatch = 600;                   // tensors of one launch (they travel as its arguments)
constexpr int kDepthM = 14, kDepthV = 30;       // binary orders below a block's largest

struct AdTensor {
    void* p;
    const void* g;
    void* m;
    void* v;
    int64_t n;
    uint32_t first_unit;
    uint32_t kind;  // bit 0: bf16 parameter, 1: bf16 gradient, 2: 8-bit moments; from bit 3: place in the list
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
    uint32_t seed_key;
    bool skip;
};

// 32 bits that are as good as random, from a counter under a key: two rounds of
// multiplications by odd constants (the fractions of the roots of 2 and 3) and shifts,
// with the key before and between them.
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
    if (o.lr_at || o.step_at) {
        const double lr = o.lr_at ? (double)*after_wait(o.lr_at) : o.lr;
        const double t = (double)(o.step_at ? *after_wait(o.step_at) : o.step);
        corrections(lr, o.weight_decay, o.beta1, o.beta2, t, s.decay, s.size, s.root);
    }
    s.factor = 1.f;
    s.skip = false;
    if (o.norm) {
        const float norm = *after_wait(o.norm);
        if (!(norm < INFINITY)) s.skip = true;
        if (norm > o.max_norm) s.factor = __fdiv_rn(o.max_norm, norm);
    }
    const uint64_t seed = o.seed_at ? (uint64_t)*after_wait(o.seed_at) : o.seed;
    s.seed_key = mix32((uint32_t)(seed >> 32) ^ mix32((uint32_t)seed, 0x9E3779B9u), 0x3C6EF372u);
    return s;
}

// Four neighbouring elements of one lane, or four that are 32 apart.
__device__ __forceinline__ void load4(const void* at, int64_t i, bool bf16, float (&x)[4]) {
    if (bf16) {
        const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(at) + i);
        x[0] = bf2_lo(q.x), x[1] = bf2_hi(q.x), x[2] = bf2_lo(q.y), x[3] = bf2_hi(q.y);
    } else {
        const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(at) + i);
        x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
    }
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

__device__ __forceinline__ void moments(float g, const AdScalars& s, float& m, float& v) {
    const float x = __fmul_rn(g, s.factor);
    m = __fadd_rn(__fmul_rn(m, s.b1), __fmul_rn(x, s.c1));
    v = __fadd_rn(__fmul_rn(v, s.b2), __fmul_rn(__fmul_rn(x, x), s.c2));
}
__device__ __forceinline__ float approx_sqrt(float x) {
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The root and the quotient are approximations of 2^-22: the step they give is a small
// part of the parameter, or all of one that was zero.
__device__ __forceinline__ float updated(float p, float m, float v, const AdScalars& s) {
    const float step = __fdividef(m, fmaf(approx_sqrt(v), s.root, s.eps));
    return fmaf(-s.size, step, p * s.decay);
}
__device__ __forceinline__ uint16_t to_bf16(float x, uint32_t draw, bool random) {
    if (random && x == x) return (uint16_t)((__float_as_uint(x) + draw) >> 16);
    return (uint16_t)(bf2_pack_rn(x, 0.f) & 0xFFFFu);
}

// One warp's blocks of 128 elements of a unit, kRows of them at a time.
template <bool kBf16P, bool kBf16G, bool kSmall>
__device__ __forceinline__ void step_unit(const AdTensor& t, uint32_t u, const AdScalars& s, bool random) {
    constexpr int kRows = kSmall ? 4 : 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const void* g = after_wait(t.g);
    void* p = t.p;
    const int64_t n = t.n;
    uint8_t* m8 = static_cast<uint8_t*>(t.m);
    uint8_t* v8 = static_cast<uint8_t*>(t.v);
    float* m32 = static_cast<float*>(t.m);
    float* v32 = static_cast<float*>(t.v);
    const uint32_t key = mix32(s.seed_key ^ (t.kind >> 3), 0xDAA66D2Bu);
    const uint32_t key_p = key ^ 0xA54FF53Au;
    const bool aligned = ((reinterpret_cast<uintptr_t>(p) & (kBf16P ? 7u : 15u)) |
                          (reinterpret_cast<uintptr_t>(g) & (kBf16G ? 7u : 15u)) |
                          ((reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v)) &
                           (kSmall ? 3u : 15u))) == 0;
    const int64_t b0 = (int64_t)(u - t.first_unit) * (kAdUnit / kAdBlock);
#pragma unroll 1
    for (int r = warp * kRows; r < kAdUnit / kAdBlock; r += kAdThreads / 32 * kRows) {
        if ((b0 + r) * kAdBlock >= n) break;
        float xp[kRows][4], xg[kRows][4], xm[kRows][4], xv[kRows][4];
        uint32_t cm[kRows], cv[kRows];
        uint8_t em[kRows], ev[kRows];
        const bool whole = aligned && (b0 + r + kRows) * kAdBlock <= n;
        const int stride = whole ? 1 : 32;
        const int first = whole ? 4 * lane : lane;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const int64_t i = (b0 + r + j) * kAdBlock + first;
            if (whole) {
                load4(p, i, kBf16P, xp[j]);
                load4(g, i, kBf16G, xg[j]);
                if (kSmall) {
                    cm[j] = *reinterpret_cast<const uint32_t*>(m8 + i);
                    cv[j] = *reinterpret_cast<const uint32_t*>(v8 + i);
                } else {
                    load4(m32, i, false, xm[j]);
                    load4(v32, i, false, xv[j]);
                }
            } else {
                cm[j] = cv[j] = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int64_t k = i + e * 32;
                    const bool in = k < n;
                    xp[j][e] = in ? load1(p, k, kBf16P) : 0.f;
                    xg[j][e] = in ? load1(g, k, kBf16G) : 0.f;
                    if (kSmall) {
                        cm[j] |= in ? (uint32_t)m8[k] << (8 * e) : 0u;
                        cv[j] |= in ? (uint32_t)v8[k] << (8 * e) : 0u;
                    } else {
                        xm[j][e] = in ? m32[k] : 0.f;
                        xv[j][e] = in ? v32[k] : 0.f;
                    }
                }
            }
            if (kSmall) {
                const bool in = (b0 + r + j) * kAdBlock < n;
                em[j] = in ? m8[n + b0 + r + j] : 0;
                ev[j] = in ? v8[n + b0 + r + j] : 0;
            }
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const int64_t i = (b0 + r + j) * kAdBlock + first;
            if (kSmall) {
                const int bm = code_base(em[j], kDepthM), bv = code_base(ev[j], kDepthV);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    xm[j][e] = decode_m(cm[j] >> (8 * e) & 255u, bm);
                    xv[j][e] = decode_v(cv[j] >> (8 * e) & 255u, bv);
                }
            }
            uint32_t top_m = 0, top_v = 0;
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                moments(xg[j][e], s, xm[j][e], xv[j][e]);
                xp[j][e] = updated(xp[j][e], xm[j][e], xv[j][e], s);
                if (kSmall) {
                    top_m = max(top_m, finite_bits(xm[j][e]));
                    top_v = max(top_v, finite_bits(xv[j][e]));
                }
                const int64_t k = i + e * stride;
                h[e] = 0x80008000u;
                if (random && (kSmall || kBf16P))
                    h[e] = mix32((uint32_t)k, key + (uint32_t)(k >> 32) * 0x9E3779B9u);
            }
            uint32_t out_m = 0, out_v = 0;
            if (kSmall) {
                top_m = __reduce_max_sync(0xFFFFFFFFu, top_m) >> 23;
                top_v = __reduce_max_sync(0xFFFFFFFFu, top_v) >> 23;
                const int bm = code_base(top_m, kDepthM), bv = code_base(top_v, kDepthV);
                const uint32_t low = random ? 8u : 0u;  // nearest: half a step
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    out_m |= encode_m(xm[j][e], bm, h[e] >> 16 << 4 | low) << (8 * e);
                    out_v |= encode_v(xv[j][e], bv, (h[e] & 0xFFFFu) << 4 | low) << (8 * e);
                }
                if (lane == 0 && (b0 + r + j) * kAdBlock < n) {
                    m8[n + b0 + r + j] = (uint8_t)top_m;
                    v8[n + b0 + r + j] = (uint8_t)top_v;
                }
            }
            uint16_t q[4];
            if (kBf16P) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    q[e] = to_bf16(xp[j][e], random ? mix32(h[e], key_p) >> 16 : 0u, random);
            }
            if (whole) {
                if (kBf16P)
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
                        make_uint2(q[0] | (uint32_t)q[1] << 16, q[2] | (uint32_t)q[3] << 16);
                else
                    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) =
                        make_float4(xp[j][0], xp[j][1], xp[j][2], xp[j][3]);
                if (kSmall) {
                    *reinterpret_cast<uint32_t*>(m8 + i) = out_m;
                    *reinterpret_cast<uint32_t*>(v8 + i) = out_v;
                } else {
                    *reinterpret_cast<float4*>(m32 + i) = make_float4(xm[j][0], xm[j][1], xm[j][2], xm[j][3]);
                    *reinterpret_cast<float4*>(v32 + i) = make_float4(xv[j][0], xv[j][1], xv[j][2], xv[j][3]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int64_t k = i + e * 32;
                    if (k >= n) continue;
                    if (kBf16P)
                        static_cast<uint16_t*>(p)[k] = q[e];
                    else
                        static_cast<float*>(p)[k] = xp[j][e];
                    if (kSmall) {
                        m8[k] = (uint8_t)(out_m >> (8 * e));
                        v8[k] = (uint8_t)(out_v >> (8 * e));
                    } else {
                        m32[k] = xm[j][e];
                        v32[k] = xv[j][e];
                    }
                }
            }
        }
    }
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

template <int N>
__global__ void __launch_bounds__(kAdThreads, kAdCtas)
    adamw_kernel(const __grid_constant__ AdBatch<N> b, const __grid_constant__ AdOptions o) {
    __shared__ AdScalars shared;
    const uint32_t u0 = (uint32_t)((uint64_t)b.units * blockIdx.x / gridDim.x);
    const uint32_t u1 = (uint32_t)((uint64_t)b.units * (blockIdx.x + 1) / gridDim.x);
    int i = ad_tensor_of(b, u0);
    grid_wait();
    if (threadIdx.x == 0) {
        shared = scalars_of(o);
        if (shared.skip && blockIdx.x == 0 && o.dev_error) atomicOr(o.dev_error, PSTAT_DEV_NONFINITE);
    }
    __syncthreads();
    const AdScalars s = shared;
    if (s.skip) return;
    for (uint32_t u = u0; u < u1; ++u) {
        while (i + 1 < b.count && b.t[i + 1].first_unit <= u) ++i;
        const AdTensor& t = b.t[i];
        const bool random = o.random != 0;
        switch (t.kind & 7u) {
            case 0: step_unit<false, false, false>(t, u, s, random); break;
            case 1: step_unit<true, false, false>(t, u, s, random); break;
            case 2: step_unit<false, true, false>(t, u, s, random); break;
            case 3: step_unit<true, true, false>(t, u, s, random); break;
            case 4: step_unit<false, false, true>(t, u, s, random); break;
            case 5: step_unit<true, false, true>(t, u, s, random); break;
            case 6: step_unit<false, true, true>(t, u, s, random); break;
            default: step_unit<true, true, true>(t, u, s, random); break;
        }
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
#pragma unroll
        for (int r = 0; r < kAdUnit / kAdBlock / (kAdThreads / 32); ++r) {
            const int64_t k = b0 + r * (kAdThreads / 32) + warp, e0 = k * kAdBlock;
            if (e0 >= t.n) break;
            const int bm = code_base(m[t.n + k], kDepthM), bv = code_base(v[t.n + k], kDepthV);
            if (aligned && e0 + kAdBlock <= t.n) {
                const uint32_t cm = *reinterpret_cast<const uint32_t*>(m + e0 + 4 * lane);
                const uint32_t cv = *reinterpret_cast<const uint32_t*>(v + e0 + 4 * lane);
                *reinterpret_cast<float4*>(om + e0 + 4 * lane) =
                    make_float4(decode_m(cm & 255u, bm), decode_m(cm >> 8 & 255u, bm),
                                decode_m(cm >> 16 & 255u, bm), decode_m(cm >> 24, bm));
                *reinterpret_cast<float4*>(ov + e0 + 4 * lane) =
                    make_float4(decode_v(cv & 255u, bv), decode_v(cv >> 8 & 255u, bv),
                                decode_v(cv >> 16 & 255u, bv), decode_v(cv >> 24, bv));
            } else {
                for (int64_t e = e0 + lane; e < min(t.n, e0 + kAdBlock); e += 32) {
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
bool add_tensor(AdBatch<N>& b, uint64_t& units, const AdTensor& t) {
    const uint64_t add = (uint64_t)((t.n + kAdUnit - 1) / kAdUnit);
    if (b.count == N || units + add > 0xFFFFFFFFull) return false;
    b.t[b.count] = t;
    b.t[b.count++].first_unit = (uint32_t)units;
    units += add;
    b.units = (uint32_t)units;
    return true;
}

unsigned grid_of(uint32_t units, const DeviceInfo& dev) {
    const uint32_t most = (uint32_t)dev.sm_count * kAdCtas;
    return units < most ? units : most;
}

template <int N>
int run_adamw(const pstat_adamw_tensor* tensors, int64_t n, const AdOptions& o, const DeviceInfo& dev,
              cudaStream_t st) {
    AdBatch<N> b;
    for (int64_t i = 0; i < n;) {
        b.count = 0;
        b.units = 0;
        uint64_t units = 0;
        for (; i < n; ++i) {
            const pstat_adamw_tensor& t = tensors[i];
            if (t.n == 0) continue;
            const uint32_t kind = (t.param_dtype == PSTAT_BF16 ? 1u : 0u) | (t.grad_dtype == PSTAT_BF16 ? 2u : 0u) |
                                  (t.bits == 8 ? 4u : 0u) | (uint32_t)i << 3;
            if (!add_tensor(b, units, {t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.n, 0u, kind})) break;
        }
        if (b.count &&
            launch_behind(adamw_kernel<N>, grid_of(b.units, dev), kAdThreads, 0, st, 1, b, o) != cudaSuccess)
            return PSTAT_ERR_CUDA;
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
                                       const_cast<void*>(t.exp_avg_sq), t.n, 0u, 0u}))
                break;
        }
        if (b.count &&
            launch_behind(adamw_moments_kernel<N>, grid_of(b.units, dev), kAdThreads, 0, st, 1, b) != cudaSuccess)
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
