// fp8.cu -- a head in 8-bit floating point: matrices in e4m3 with a scale for each run of
// 128 columns (of a row, or of 128 rows), and the logits of hidden states so given.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace pstat {
namespace {

constexpr int kF8Block = 128;

// ---------------------------------------------------------------------------
// Quantising.  A scale is the least power of two with max|x| <= 448 s: dividing by it is
// exact, so that an element is rounded once and its code is the nearest whatever
// the order of operations.  (max|x| / 448 itself would use the last bit of range, but
// e4m3 is a floating-point type, whose relative step does not depend on it.)
// A thread takes 8 neighbouring columns of every 16th row of a CTA's rows; all its loads
// are in flight before the first is used.  Bound by HBM.
// ---------------------------------------------------------------------------
constexpr int kQuThreads = 256;
constexpr int kQuRows = 64;  // rows of a CTA where each has its own scale

template <typename E>
__device__ __forceinline__ void load8(const E* row, int64_t col, int64_t K, bool vector, float (&x)[8]);
template <>
__device__ __forceinline__ void load8(const uint16_t* row, int64_t col, int64_t K, bool vector, float (&x)[8]) {
    if (vector && col + 8 <= K) {
        const uint4 q = *reinterpret_cast<const uint4*>(row + col);
        x[0] = bf2_lo(q.x), x[1] = bf2_hi(q.x), x[2] = bf2_lo(q.y), x[3] = bf2_hi(q.y);
        x[4] = bf2_lo(q.z), x[5] = bf2_hi(q.z), x[6] = bf2_lo(q.w), x[7] = bf2_hi(q.w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = col + i < K ? __uint_as_float((uint32_t)row[col + i] << 16) : 0.f;
    }
}
template <>
__device__ __forceinline__ void load8(const float* row, int64_t col, int64_t K, bool vector, float (&x)[8]) {
    if (vector && col + 8 <= K) {
        const float4 a = *reinterpret_cast<const float4*>(row + col);
        const float4 b = *reinterpret_cast<const float4*>(row + col + 4);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = col + i < K ? row[col + i] : 0.f;
    }
}

// The exponent field of a block's scale from the bits of its largest magnitude; 0 for
// a block that is not finite.
__device__ __forceinline__ uint32_t scale_field(uint32_t top) {
    if (top >= 0x7F800000u) return 0;
    if (top == 0) return 127;
    return (uint32_t)max((int)((top + 0x1FFFFFu) >> 23) - 8, 1);  // 448 = 1.75 x 2^8
}
__device__ __forceinline__ float scale_of(uint32_t field) {
    return field ? __uint_as_float(field << 23) : NAN;
}
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store8(uint8_t* q, int64_t col, int64_t K, bool vector, const float (&x)[8],
                                       uint32_t field) {
    const float inverse = field ? __uint_as_float((254u - field) << 23) : 0.f;
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        w[h] = field ? e4m3_pair(x[4 * h] * inverse, x[4 * h + 1] * inverse) |
                           e4m3_pair(x[4 * h + 2] * inverse, x[4 * h + 3] * inverse) << 16
                     : 0u;
    if (vector && col + 8 <= K) {
        *reinterpret_cast<uint2*>(q + col) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < K) q[col + i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
}

template <typename E, bool kTall>
__global__ void __launch_bounds__(kQuThreads)
    quantize_kernel(const void* x_at, int64_t T, int64_t K, int64_t ld, uint8_t* q, float* scale, int64_t scale_row,
                    int64_t scale_col, uint32_t col_blocks, int* dev_error) {
    constexpr int kIter = (kTall ? kF8Block : kQuRows) / 16;
    __shared__ uint32_t warp_top[kQuThreads / 32];
    grid_wait();
    const E* x = static_cast<const E*>(after_wait(x_at));
    const uint32_t cb = blockIdx.x % col_blocks;
    const int64_t rb = blockIdx.x / col_blocks;
    const int64_t r0 = rb * (kIter * 16) + threadIdx.x / 16;
    const int64_t col = (int64_t)cb * kF8Block + threadIdx.x % 16 * 8;
    const bool in_vec = ((reinterpret_cast<uintptr_t>(x) | (uintptr_t)(ld * (int64_t)sizeof(E))) & 15u) == 0;
    const bool out_vec = ((reinterpret_cast<uintptr_t>(q) | (uintptr_t)K) & 7u) == 0;
    float v[kIter][8];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int64_t r = r0 + 16 * i;
        load8<E>(x + (r < T ? r : 0) * ld, r < T ? col : K, K, in_vec, v[i]);
    }
    uint32_t top[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        top[i] = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top[i] = max(top[i], __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
    }
    bool lost = false;
    if (kTall) {
        uint32_t all = 0;
#pragma unroll
        for (int i = 0; i < kIter; ++i) all = max(all, top[i]);
        all = __reduce_max_sync(0xFFFFFFFFu, all);
        if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = all;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kQuThreads / 32; ++w) all = max(all, warp_top[w]);
        const uint32_t field = scale_field(all);
        if (threadIdx.x == 0) scale[rb * scale_row + cb * scale_col] = scale_of(field);
        lost = field == 0;
#pragma unroll
        for (int i = 0; i < kIter; ++i)
            if (r0 + 16 * i < T) store8(q + (r0 + 16 * i) * K, col, K, out_vec, v[i], field);
    } else {
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
#pragma unroll
            for (int m = 8; m; m /= 2) top[i] = max(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], m));
            const int64_t r = r0 + 16 * i;
            if (r >= T) continue;
            const uint32_t field = scale_field(top[i]);
            if (threadIdx.x % 16 == 0) scale[r * scale_row + cb * scale_col] = scale_of(field);
            lost |= field == 0;
            store8(q + r * K, col, K, out_vec, v[i], field);
        }
    }
    if (lost && dev_error && threadIdx.x % 16 == 0) atomicOr(dev_error, PSTAT_DEV_NONFINITE);
}

// ---------------------------------------------------------------------------
// Logits.  out[t, v] = sum_j f_j sum_k q[t, k] W[v, k], f_j = S[v / 128, j] s[t, j], j the blocks
// of 128 columns k.  Each block's product goes to a tensor-memory accumulator of its own,
// from where the epilogue adds it, times its scales, to sums in registers; blocks in
// ascending order and one CTA to a tile, so that a logit's bits depend on its row alone
// and not on the tile that it falls in.
//   warp 0    copies tiles of W and q into a ring of stages (TMA, 128-byte swizzle)
//   warp 1    issues tcgen05.mma (M 128, K 32), four to a block
//   warps 2.. a thread adds up one lane of the accumulator for up to 64 columns
// Two shapes of tile:
//   up to 128 tokens  128 rows of W are M, the tokens N (16, 32, 64 or 128): few tokens cost
//              few columns.  Bound by the one pass over W.
//   beyond     128 tokens are M, 256 rows of W N.  A thread's factor is one number to a
//              block, where with tokens as columns it is one for each column, read
//              from shared memory.  Bound by the tensor cores and the epilogue that
//              keeps up with them: 128 x 256 sums every 512 cycles.
// The epilogue's loads from tensor memory take their time whatever their size, so many
// warps with few columns each take turns: with 8 warps of 128 columns 2048 x 40,000
// logits ran at a tenth of the tensor cores' rate.
// All waits are bounded; on a timeout the CTA drains what is in flight and ends.
// ---------------------------------------------------------------------------
constexpr uint64_t kF8WaitNs = 2000000000ull;
constexpr int kF8M = 128;

template <int kN>
struct F8Tile {
    static constexpr bool kTokenLanes = kN == 256;
    static constexpr int kCols = kTokenLanes ? 64 : kN < 32 ? kN : 32;  // of an epilogue warp
    static constexpr int kEpiWarps = 4 * (kN / kCols);
    static constexpr int kFirstEpi = kTokenLanes ? 4 : 2;  // a warpgroup, for setmaxnreg
    static constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
    static constexpr uint32_t kABytes = kF8M * kF8Block;
    static constexpr uint32_t kBBytes = kN * kF8Block;
    static constexpr int kStages = kN == 256 ? 4 : kN == 128 ? 6 : kN == 64 ? 8 : kN == 32 ? 10 : 11;
    static constexpr int kBufs = kN == 256 ? 2 : 4;  // accumulators
    static constexpr uint32_t kTmemCols = kN * kBufs;
    static constexpr uint32_t kA = 0;
    static constexpr uint32_t kB = kA + kStages * kABytes;
    static constexpr uint32_t kScale = kB + kStages * kBBytes;  // [warps][2][kCols] floats
    static constexpr uint32_t kBars = kScale + (kTokenLanes ? 0 : kEpiWarps * 2 * kCols * 4);
    static constexpr uint32_t kNumBars = 2 * kStages + 2 * kBufs + 1;
    static constexpr uint32_t kSlot = kBars + kNumBars * 8;
    static constexpr uint32_t kBytes = kSlot + 16 + 1024;  // + alignment slack
    static_assert(kBytes <= 227 * 1024 && kTmemCols >= 32 && kTmemCols <= 512, "");
};

struct F8Args {
    CUtensorMap lanes, columns;  // the operands that are M and N
    const float* W_scale;
    const float* q_scale;
    int64_t scale_row, scale_col;
    int64_t ld_out;
    void* out;
    int T, V;
    int blocks;      // of 128 along K
    int row_blocks;  // of W_scale
    int t_tiles;     // tiles along the tokens, the quick index
    uint32_t tiles;
    bool vector;     // rows of logits start on 16 bytes
    int* dev_error;
};

// Registers of the wide tile's threads: launched with kLaunchRegs each, the first warpgroup
// keeps few and the epilogue takes more, its 64 sums, two loads in flight and the rest.
constexpr int kLaunchRegs = 96, kRoleRegs = 24, kEpiRegs = 112;
static_assert(128 * kRoleRegs + 512 * kEpiRegs <= 640 * kLaunchRegs, "the split fits what was launched");

template <typename O>
__device__ __forceinline__ void put(O* out, float x) {
    if constexpr (sizeof(O) == 4)
        *out = x;
    else
        *out = (uint16_t)(bf2_pack_rn(x, 0.f) & 0xFFFFu);
}

// One row on; opaque, so that the addresses of all rows are not formed at once, at two
// registers each.
template <typename O>
__device__ __forceinline__ O* next_row(O* at, int64_t ld) {
    return after_wait(at + ld);
}

// 16 registers of 32 lanes: in either half of the lanes, the 16 x 16 values lane by register
// turned to register by lane.
__device__ __forceinline__ void transpose16(float (&x)[16], int lane) {
#pragma unroll
    for (int d = 8; d; d /= 2)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i & d) continue;
            const bool high = (lane & d) != 0;
            const float got = __shfl_xor_sync(0xFFFFFFFFu, high ? x[i] : x[i + d], d);
            if (high)
                x[i] = got;
            else
                x[i + d] = got;
        }
}

template <int kN, typename O>
__global__ void __launch_bounds__(F8Tile<kN>::kThreads, 1)
    fp8_logits_kernel(const __grid_constant__ F8Args a) {
    using C = F8Tile<kN>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);
    uint64_t* empty = full + C::kStages;
    uint64_t* tfull = empty + C::kStages;
    uint64_t* tempty = tfull + C::kBufs;
    uint64_t* drain = tempty + C::kBufs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kSlot);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < C::kBufs; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], C::kEpiWarps);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        prefetch_tensormap(&a.lanes);
        prefetch_tensormap(&a.columns);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    bool failed = false;
    grid_wait();

    if (warp < C::kFirstEpi) {
    if (C::kTokenLanes) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_w = a.t_tiles == 1 ? policy_evict_first() : policy_evict_normal();
            const uint64_t pol_q = policy_evict_last();
            uint32_t it = 0;
            for (uint32_t u = blockIdx.x; u < a.tiles && !failed; u += gridDim.x) {
                const int tt = (int)(u % (uint32_t)a.t_tiles), vt = (int)(u / (uint32_t)a.t_tiles);
                const int m0 = (C::kTokenLanes ? tt : vt) * kF8M, n0 = (C::kTokenLanes ? vt : tt) * kN;
                for (int j = 0; j < a.blocks; ++j, ++it) {
                    const int s = it % C::kStages;
                    if (!mbar_wait_bounded(&empty[s], ((it / C::kStages) & 1u) ^ 1u, kF8WaitNs)) {
                        failed = true;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[s], C::kABytes + C::kBBytes);
                    tma_load_2d(smem + C::kA + s * C::kABytes, &a.lanes, j * kF8Block, m0, &full[s],
                                C::kTokenLanes ? pol_q : pol_w);
                    tma_load_2d(smem + C::kB + s * C::kBBytes, &a.columns, j * kF8Block, n0, &full[s],
                                C::kTokenLanes ? pol_w : pol_q);
                }
            }
            // every copy has landed before the CTA ends
            for (uint32_t k = 0; k < (uint32_t)C::kStages && k < it; ++k) {
                const uint32_t i = it - 1 - k;
                if (!mbar_wait_bounded(&full[i % C::kStages], (i / C::kStages) & 1u, kF8WaitNs)) failed = true;
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3_f32(kF8M, kN);
            uint32_t it = 0;
            for (uint32_t u = blockIdx.x; u < a.tiles && !failed; u += gridDim.x) {
                for (int j = 0; j < a.blocks; ++j, ++it) {
                    const uint32_t b = it % C::kBufs;
                    const int s = it % C::kStages;
                    if (!mbar_wait_bounded(&tempty[b], ((it / C::kBufs) & 1u) ^ 1u, kF8WaitNs) ||
                        !mbar_wait_bounded(&full[s], (it / C::kStages) & 1u, kF8WaitNs)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t a_at = smem_u32(smem + C::kA + s * C::kABytes);
                    const uint32_t b_at = smem_u32(smem + C::kB + s * C::kBBytes);
#pragma unroll
                    for (int k = 0; k < kF8Block / 32; ++k)
                        umma_f8(tmem + b * kN, sdesc_kmajor_sw128(a_at + 32 * k), sdesc_kmajor_sw128(b_at + 32 * k),
                                idesc, k != 0);
                    umma_commit(&empty[s]);
                    umma_commit(&tfull[b]);
                }
            }
            umma_commit(drain);
            if (!mbar_wait_bounded(drain, 0, kF8WaitNs)) failed = true;
        }
    }
    } else {
        if (C::kTokenLanes) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        constexpr int kCols = C::kCols;
        const int e = warp - C::kFirstEpi, quarter = warp & 3, part = e / 4;
        const int c0 = part * kCols;
        const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + c0;
        float* scales = reinterpret_cast<float*>(smem + C::kScale) + e * 2 * kCols;
        const float* W_scale = after_wait(a.W_scale);
        const float* q_scale = after_wait(a.q_scale);
        // After a timeout no wait is made and nothing is written, but the sums run to their
        // end: a way out of their loop would cost every sum a register of its own.
        auto wait_full = [&](uint32_t i) {
            if (!failed) {
                const bool ok = mbar_wait_bounded(&tfull[i % C::kBufs], (i / C::kBufs) & 1u, kF8WaitNs);
                failed = !__all_sync(0xFFFFFFFFu, ok);
            }
            tc_fence_after_sync();
        };
        uint32_t it = 0;
        for (uint32_t u = blockIdx.x; u < a.tiles && !failed; u += gridDim.x) {
            const int tt = (int)(u % (uint32_t)a.t_tiles), vt = (int)(u / (uint32_t)a.t_tiles);
            // tokens: of this lane, or of this warp's columns (a lane fetches one column's)
            const int t = C::kTokenLanes ? tt * kF8M + quarter * 32 + lane : tt * kN + c0 + lane;
            const int v = C::kTokenLanes ? vt * kN + c0 : vt * kF8M + quarter * 32 + lane;
            const bool mine = t < a.T && (C::kTokenLanes || lane < kCols);
            const float* qs = q_scale + (mine ? t * a.scale_row : 0);
            const int vb = C::kTokenLanes ? min(v / kF8Block, a.row_blocks - 1) : vt;
            const float* ws = W_scale + (int64_t)vb * a.blocks;
            float next = (mine ? qs[0] : 0.f), next_w = ws[0];
            uint64_t acc[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) acc[i] = 0;
            if constexpr (C::kTokenLanes) {
#pragma unroll 1
                for (int j = 0; j < a.blocks; ++j, ++it) {
                    const float f = __fmul_rn(next, next_w);
                    const uint64_t ff = f2_pack(f, f);
                    if (j + 1 < a.blocks) {
                        qs += a.scale_col;
                        next = mine ? *qs : 0.f;
                        next_w = *++ws;
                    }
                    const uint32_t b = it % C::kBufs;
                    wait_full(it);
#pragma unroll
                    for (int c = 0; c < kCols / 32; ++c) {
                        uint32_t r[32];
                        tmem_load(taddr + b * kN + c * 32, r);
                        tmem_ld_wait();
                        if (c == kCols / 32 - 1) {
                            tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&tempty[b]);
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            uint64_t& y = acc[(c * 32 + i) / 2];
                            y = f2_fma(f2_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), ff, y);
                        }
                    }
                }
            } else {
                for (int j = 0; j < a.blocks; ++j, ++it) {
                    float* fs = scales + (j & 1) * kCols;
                    if (lane < kCols) fs[lane] = __fmul_rn(next, next_w);
                    if (j + 1 < a.blocks) {
                        qs += a.scale_col;
                        next = mine ? *qs : 0.f;
                        next_w = *++ws;
                    }
                    const uint32_t b = it % C::kBufs;
                    wait_full(it);  // and the scales are written
                    uint32_t r[kCols];
                    tmem_load(taddr + b * kN, r);
                    tmem_ld_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tempty[b]);
#pragma unroll
                    for (int i = 0; i < kCols; i += 4) {
                        const float4 s = *reinterpret_cast<const float4*>(fs + i);
                        uint64_t &y0 = acc[i / 2], &y1 = acc[i / 2 + 1];
                        y0 = f2_fma(f2_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), f2_pack(s.x, s.y), y0);
                        y1 = f2_fma(f2_pack(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])), f2_pack(s.z, s.w),
                                    y1);
                    }
                }
            }
            if (failed) break;
            O* out = static_cast<O*>(a.out);
            if constexpr (!C::kTokenLanes) {
                // lanes write neighbouring logits of one token after another
                const int n = min(kCols, a.T - (tt * kN + c0));
                if (v < a.V) {
                    O* at = out + (int64_t)(tt * kN + c0) * a.ld_out + v;
#pragma unroll
                    for (int i = 0; i < kCols; ++i, at = next_row(at, a.ld_out)) {
                        float x, y;
                        f2_unpack(acc[i / 2], x, y);
                        if (i < n) put(at, i & 1 ? y : x);
                    }
                }
            } else if (a.vector && v + kCols <= a.V) {
                // a lane writes its token's logits, 16 bytes at a time
                constexpr int kVec = 16 / sizeof(O);
                uint4* row = reinterpret_cast<uint4*>(out + t * a.ld_out + v);
                if (t < a.T) {
#pragma unroll
                    for (int i = 0; i < kCols / kVec; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            float x, y;
                            f2_unpack(acc[(i * kVec + h * (kVec / 4)) / 2], x, y);
                            w[h] = kVec == 8 ? bf2_pack_rn(x, y) : __float_as_uint(h & 1 ? y : x);
                        }
                        row[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            } else {
                // rows at any alignment: turned, so that lanes write neighbouring logits
#pragma unroll
                for (int c = 0; c < kCols / 16; ++c) {
                    float x[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i) f2_unpack(acc[c * 8 + i], x[2 * i], x[2 * i + 1]);
                    transpose16(x, lane);
                    const int col = v + c * 16 + (lane & 15);
                    const int t0 = tt * kF8M + quarter * 32 + (lane & 16);
                    O* at = out + (int64_t)t0 * a.ld_out + col;
                    const int n = col < a.V ? min(16, a.T - t0) : 0;
#pragma unroll
                    for (int i = 0; i < 16; ++i, at = next_row(at, a.ld_out))
                        if (i < n) put(at, x[i]);
                }
            }
        }
    }
    if (failed && a.dev_error) atomicOr(a.dev_error, PSTAT_DEV_TIMEOUT);
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <int kN, typename O>
cudaError_t launch_logits(F8Args a, const void* q, const void* W, int64_t K, const DeviceInfo& dev, cudaStream_t st) {
    using C = F8Tile<kN>;
    static ContextSeen configured;
    const cudaError_t e = ensure_smem_optin(reinterpret_cast<const void*>(fp8_logits_kernel<kN, O>), (int)C::kBytes,
                                            configured);
    if (e != cudaSuccess) return e;
    if (C::kTokenLanes) {  // a warp that asks for registers that are not there waits for ever
        static std::atomic<int> regs{0};
        if (!regs) {
            cudaFuncAttributes attr;
            const cudaError_t f = cudaFuncGetAttributes(&attr, fp8_logits_kernel<kN, O>);
            if (f != cudaSuccess) return f;
            regs = attr.numRegs;
        }
        if (regs != kLaunchRegs) return cudaErrorInvalidKernelImage;
    }
    const int64_t t_tile = C::kTokenLanes ? kF8M : kN, v_tile = C::kTokenLanes ? kN : kF8M;
    a.t_tiles = (int)((a.T + t_tile - 1) / t_tile);
    const int64_t tiles = (a.V + v_tile - 1) / v_tile * a.t_tiles;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    a.tiles = (uint32_t)tiles;
    if (!make_byte_map(C::kTokenLanes ? &a.lanes : &a.columns, q, a.T, K, K, (int)t_tile) ||
        !make_byte_map(C::kTokenLanes ? &a.columns : &a.lanes, W, a.V, K, K, (int)v_tile))
        return cudaErrorInvalidValue;
    const int64_t grid = a.tiles < dev.sm_count ? a.tiles : dev.sm_count;
    return launch_behind(fp8_logits_kernel<kN, O>, (unsigned)grid, C::kThreads, C::kBytes, st, 1, a);
}

template <typename O>
cudaError_t launch_logits_of(const F8Args& a, const void* q, const void* W, int64_t K, const DeviceInfo& dev,
                             cudaStream_t st) {
    if (a.T <= 16) return launch_logits<16, O>(a, q, W, K, dev, st);
    if (a.T <= 32) return launch_logits<32, O>(a, q, W, K, dev, st);
    if (a.T <= 64) return launch_logits<64, O>(a, q, W, K, dev, st);
    if (a.T <= 128) return launch_logits<128, O>(a, q, W, K, dev, st);
    return launch_logits<256, O>(a, q, W, K, dev, st);
}

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace pstat

using namespace pstat;

extern "C" {

int pstat_fp8_quantize(const void* x, pstat_dtype dt, int64_t T, int64_t K, int64_t ld, int rows, void* out_q,
                       float* out_scale, int64_t scale_row, int64_t scale_col, int* dev_error,
                       pstat_stream_t stream) {
    if (dt != PSTAT_F32 && dt != PSTAT_BF16) return PSTAT_ERR_DTYPE;
    if (T < 0 || K < 1 || ld < K || K > INT32_MAX || T > INT32_MAX || (rows != 1 && rows != kF8Block))
        return PSTAT_ERR_SHAPE;
    if (T == 0) return PSTAT_OK;
    if (!x || !out_q || !out_scale) return PSTAT_ERR_NULLPTR;
    if (!aligned_to(x, dt == PSTAT_BF16 ? 2 : 4) || !aligned_to(out_scale, 4)) return PSTAT_ERR_ALIGN;
    const int64_t cols = (K + kF8Block - 1) / kF8Block;
    const int64_t row_blocks = rows == 1 ? (T + kQuRows - 1) / kQuRows : (T + kF8Block - 1) / kF8Block;
    if (scale_row < 1 || scale_col < 1 || cols * row_blocks > INT32_MAX) return PSTAT_ERR_SHAPE;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != PSTAT_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)(cols * row_blocks);
    auto launch = [&](auto kernel) {
        return launch_behind(kernel, grid, kQuThreads, 0, st, 1, x, T, K, ld, static_cast<uint8_t*>(out_q), out_scale,
                             scale_row, scale_col, (uint32_t)cols, dev_error);
    };
    const cudaError_t e =
        rows == 1 ? (dt == PSTAT_BF16 ? launch(quantize_kernel<uint16_t, false>) : launch(quantize_kernel<float, false>))
                  : (dt == PSTAT_BF16 ? launch(quantize_kernel<uint16_t, true>) : launch(quantize_kernel<float, true>));
    return e == cudaSuccess ? PSTAT_OK : PSTAT_ERR_CUDA;
}

int pstat_fp8_logits(const void* q, const float* q_scale, int64_t scale_row, int64_t scale_col, const void* W,
                     const float* W_scale, int64_t T, int64_t V, int64_t K, void* out, pstat_dtype out_dt,
                     int64_t ld_out, int* dev_error, pstat_stream_t stream) {
    if (out_dt != PSTAT_F32 && out_dt != PSTAT_BF16) return PSTAT_ERR_DTYPE;
    if (T < 0 || V < 1 || K < 16 || K % 16 || K > (1 << 24) || ld_out < V || T > INT32_MAX / 2 || V > INT32_MAX / 2 ||
        scale_row < 0 || scale_col < 0)
        return PSTAT_ERR_SHAPE;
    if (T == 0) return PSTAT_OK;
    if (!q || !q_scale || !W || !W_scale || !out) return PSTAT_ERR_NULLPTR;
    if (!aligned_to(q, 16) || !aligned_to(W, 16) || !aligned_to(q_scale, 4) || !aligned_to(W_scale, 4) ||
        !aligned_to(out, out_dt == PSTAT_BF16 ? 2 : 4))
        return PSTAT_ERR_ALIGN;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != PSTAT_OK) return rc;
    F8Args a = {};
    a.W_scale = W_scale;
    a.q_scale = q_scale;
    a.scale_row = scale_row;
    a.scale_col = scale_col;
    a.T = (int)T;
    a.V = (int)V;
    a.ld_out = ld_out;
    a.out = out;
    a.blocks = (int)((K + kF8Block - 1) / kF8Block);
    a.row_blocks = (int)((V + kF8Block - 1) / kF8Block);
    a.vector = aligned_to(out, 16) && ld_out % (out_dt == PSTAT_BF16 ? 8 : 4) == 0;
    a.dev_error = dev_error;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = out_dt == PSTAT_BF16 ? launch_logits_of<uint16_t>(a, q, W, K, dev, st)
                                               : launch_logits_of<float>(a, q, W, K, dev, st);
    return e == cudaSuccess ? PSTAT_OK : PSTAT_ERR_CUDA;
}

}  // extern "C"
