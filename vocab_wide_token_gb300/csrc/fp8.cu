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
constexpr int64_t kF8MaxStride = (int64_t)1 << 31;  // of scales: products with counts fit

// ---------------------------------------------------------------------------
// Quantising.  A scale is the least power of two with max|x| <= 448 s: dividing by it is
// exact, so that an element is rounded once and its code is the nearest whatever
// the order of operations.  (max|x| / 448 itself would use the last bit of range, but
// e4m3 is a floating-point type, whose relative step does not depend on it.)
// A thread takes 8 neighbouring columns of every 16th row of a CTA's rows; all its loads
// are in flight before the first is used.  Bound by HBM: 60,000 x 4096 bf16 by 128 x 128 in 114
// us, 6.4 TB/s, by rows 127 us, 5.8 (with 32 or 128 rows to a CTA 142); 151,936 x 4096 274 us.
// ---------------------------------------------------------------------------
constexpr int kQuThreads = 256;
constexpr int kQuRows = 64;  // rows of a CTA where each has its own scale

// 8 neighbouring columns, from an address on 16 bytes.
__device__ __forceinline__ void load8(const uint16_t* at, float (&x)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(at);
    x[0] = bf2_lo(q.x), x[1] = bf2_hi(q.x), x[2] = bf2_lo(q.y), x[3] = bf2_hi(q.y);
    x[4] = bf2_lo(q.z), x[5] = bf2_hi(q.z), x[6] = bf2_lo(q.w), x[7] = bf2_hi(q.w);
}
__device__ __forceinline__ void load8(const float* at, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(at)[0], b = reinterpret_cast<const float4*>(at)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float widen(float x) { return x; }

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

struct QuArgs {
    const void* x;
    int64_t T, K, ld;
    void* q;
    float* scale;
    int64_t scale_row, scale_col;
    uint32_t col_blocks;
    int* dev_error;
};

template <typename E, bool kTall>
__global__ void __launch_bounds__(kQuThreads)
    quantize_kernel(const __grid_constant__ QuArgs a) {
    constexpr int kIter = (kTall ? kF8Block : kQuRows) / 16;
    __shared__ uint32_t warp_top[kQuThreads / 32];
    grid_wait();
    const E* x = static_cast<const E*>(after_wait(a.x));
    uint8_t* q = static_cast<uint8_t*>(a.q);
    float* scale = a.scale;
    const int64_t T = a.T, K = a.K, ld = a.ld, scale_row = a.scale_row, scale_col = a.scale_col;
    const uint32_t col_blocks = a.col_blocks;
    int* dev_error = a.dev_error;
    const uint32_t cb = blockIdx.x % col_blocks;
    const int64_t rb = blockIdx.x / col_blocks;
    const int64_t r0 = rb * (kIter * 16) + threadIdx.x / 16;
    const int64_t col = (int64_t)cb * kF8Block + threadIdx.x % 16 * 8;
    const bool in_vec = ((reinterpret_cast<uintptr_t>(x) | (uintptr_t)(ld * (int64_t)sizeof(E))) & 15u) == 0;
    const bool out_vec = ((reinterpret_cast<uintptr_t>(q) | (uintptr_t)K) & 7u) == 0;
    float v[kIter][8];
    // One way for all rows of the CTA: a test between two loads would keep the second waiting.
    if (in_vec && (cb + 1) * (int64_t)kF8Block <= K && (rb + 1) * (int64_t)(kIter * 16) <= T) {
#pragma unroll
        for (int i = 0; i < kIter; ++i) load8(x + (r0 + 16 * i) * ld + col, v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int64_t r = r0 + 16 * i;
            const E* at = x + r * ld + col;
            if (in_vec && r < T && col + 8 <= K)
                load8(at, v[i]);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = r < T && col + e < K ? widen(at[e]) : 0.f;
        }
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

template <typename E, bool kTall>
cudaError_t launch_quantize(const QuArgs& a, unsigned grid, cudaStream_t st) {
    return launch_behind(quantize_kernel<E, kTall>, grid, kQuThreads, 0, st, 1, a);
}

// ---------------------------------------------------------------------------
// Logits.  out[t, v] = sum_j f_j sum_k q[t, k] W[v, k], f_j = S[v / 128, j] s[t, j], j the blocks
// of 128 columns k.  Each block's product goes to a tensor-memory accumulator of its own,
// from where the epilogue adds it, times its scales, to sums in registers; blocks in
// ascending order and one CTA to a logit, so that its bits depend on its row alone and not
// on the tile that it falls in.
//   warp 0    copies tiles of W and q into a ring of stages (TMA, 128-byte swizzle)
//   warp 1    issues tcgen05.mma (K 32), four to a block
//   the others  a thread adds up one lane of the accumulator for up to 32 columns (narrow tiles)
//               or 128 (wide ones)
// Up to 128 tokens (narrow tiles) 128 rows of W are M and the tokens N (16, 32, 64 or 128): few
// tokens cost few columns.  Bound by the one pass over W.
// Beyond (wide tiles) 256 tokens are M, 256 rows of W N, by a pair of CTAs (cta_group::2) that
// hold 128 rows of either operand each.  A thread's factor is one number to a block, where
// with tokens as columns it is one for each column, read from shared memory.  The pair is
// for the operands' way from L2: an SM takes in 32 KB for every 128 x 256 x 128 products,
// alone 48 KB.  8 epilogue warps with 128 columns each: with 16 of 64 the instructions of
// waiting and handing on, four warps' on each scheduler, bound it (2048 x 60,000 x 4096 in
// 454 us; 373 so).  4096 x 151,936 x 4096 takes 1.84 to 1.90 ms, 2.7 to 2.8 PFLOP/s (one call
// after another, which the power limit slows, 2.0 ms with the quantising): two accumulators of 256
// columns fill tensor memory, and a block's products (512 cycles), their way to the epilogue,
// its loads and its word back to the issuing CTA take 1,500 to 1,600 for two blocks.
// All waits are bounded; on a timeout a CTA drains what is in flight and ends.
// ---------------------------------------------------------------------------
constexpr long long kF8Wait = 4000000000ll;  // cycles, about two seconds
constexpr int kF8M = 128;

struct F8Args {
    CUtensorMap lanes, columns;  // the operands that are M and N
    CUtensorMap logits;          // wide tiles, `vector`
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

template <int kN>
struct F8Narrow {
    static constexpr int kCols = kN < 32 ? kN : 32;  // of an epilogue warp
    static constexpr int kEpiWarps = 4 * (kN / kCols);
    static constexpr int kThreads = 64 + 32 * kEpiWarps;
    static constexpr uint32_t kABytes = kF8M * kF8Block;
    static constexpr uint32_t kBBytes = kN * kF8Block;
    static constexpr int kStages = kN == 128 ? 6 : kN == 64 ? 8 : kN == 32 ? 10 : 11;
    static constexpr int kBufs = 4;  // accumulators
    static constexpr uint32_t kTmemCols = kN * kBufs;
    static constexpr uint32_t kA = 0;
    static constexpr uint32_t kB = kA + kStages * kABytes;
    static constexpr uint32_t kScale = kB + kStages * kBBytes;  // [warps][2][kCols] floats
    static constexpr uint32_t kBars = kScale + kEpiWarps * 2 * kCols * 4;
    static constexpr uint32_t kNumBars = 2 * kStages + 2 * kBufs + 1;
    static constexpr uint32_t kSlot = kBars + kNumBars * 8;
    static constexpr uint32_t kBytes = kSlot + 16 + 1024;  // + alignment slack
    static_assert(kBytes <= 227 * 1024 && kTmemCols >= 32 && kTmemCols <= 512, "");
};

template <int kN, typename O>
__global__ void __launch_bounds__(F8Narrow<kN>::kThreads, 1)
    fp8_narrow_kernel(const __grid_constant__ F8Args a) {
    using C = F8Narrow<kN>;
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

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_w = policy_evict_first(), pol_q = policy_evict_last();
            uint32_t it = 0;
            for (uint32_t u = blockIdx.x; u < a.tiles && !failed; u += gridDim.x) {
                for (int j = 0; j < a.blocks; ++j, ++it) {
                    const int s = it % C::kStages;
                    if (!mbar_wait_cycles(&empty[s], ((it / C::kStages) & 1u) ^ 1u, kF8Wait)) {
                        failed = true;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[s], C::kABytes + C::kBBytes);
                    tma_load_2d(smem + C::kA + s * C::kABytes, &a.lanes, j * kF8Block, (int)u * kF8M, &full[s], pol_w);
                    tma_load_2d(smem + C::kB + s * C::kBBytes, &a.columns, j * kF8Block, 0, &full[s], pol_q);
                }
            }
            // every copy has landed before the CTA ends
            for (uint32_t k = 0; k < (uint32_t)C::kStages && k < it; ++k) {
                const uint32_t i = it - 1 - k;
                if (!mbar_wait_cycles(&full[i % C::kStages], (i / C::kStages) & 1u, kF8Wait)) failed = true;
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
                    if (!mbar_wait_cycles(&tempty[b], ((it / C::kBufs) & 1u) ^ 1u, kF8Wait) ||
                        !mbar_wait_cycles(&full[s], (it / C::kStages) & 1u, kF8Wait)) {
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
            if (!mbar_wait_cycles(drain, 0, kF8Wait)) failed = true;
        }
    } else {
        constexpr int kCols = C::kCols;
        const int e = warp - 2, quarter = warp & 3, c0 = e / 4 * kCols;
        const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + c0;
        float* scales = reinterpret_cast<float*>(smem + C::kScale) + e * 2 * kCols;
        const float* W_scale = after_wait(a.W_scale);
        const float* q_scale = after_wait(a.q_scale);
        const bool mine = c0 + lane < a.T && lane < kCols;  // whether a lane fetches a column's scales
        uint32_t it = 0;
        for (uint32_t u = blockIdx.x; u < a.tiles && !failed; u += gridDim.x) {
            const float* qs = q_scale + (mine ? (c0 + lane) * a.scale_row : 0);
            const float* ws = W_scale + (int64_t)u * a.blocks;
            float next = mine ? *qs : 0.f, next_w = *ws;
            uint64_t acc[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) acc[i] = 0;
            // After a timeout no wait is made and nothing is written, but the sums run to
            // their end: a way out of their loop would cost every sum a register of its own.
            for (int j = 0; j < a.blocks; ++j, ++it) {
                // The halves take turns over all tiles: a lane that is ahead writes one only after
                // the next block's __syncwarp, when every lane has read what it held.
                float* fs = scales + (it & 1) * kCols;
                if (lane < kCols) fs[lane] = __fmul_rn(next, next_w);
                if (j + 1 < a.blocks) {
                    qs += a.scale_col;
                    next = mine ? *qs : 0.f;
                    next_w = *++ws;
                }
                const uint32_t b = it % C::kBufs;
                __syncwarp();  // the scales are written
                if (!failed) {
                    const bool ok = mbar_wait_cycles(&tfull[b], (it / C::kBufs) & 1u, kF8Wait);
                    failed = !__all_sync(0xFFFFFFFFu, ok);
                }
                tc_fence_after_sync();
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
                    y1 = f2_fma(f2_pack(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])), f2_pack(s.z, s.w), y1);
                }
            }
            if (failed) break;
            // lanes write neighbouring logits of one token after another
            const int v = (int)u * kF8M + quarter * 32 + lane, n = min(kCols, a.T - c0);
            if (v < a.V) {
                O* at = static_cast<O*>(a.out) + c0 * a.ld_out + v;
#pragma unroll
                for (int i = 0; i < kCols; ++i, at = next_row(at, a.ld_out)) {
                    float x, y;
                    f2_unpack(acc[i / 2], x, y);
                    if (i < n) put(at, i & 1 ? y : x);
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

struct F8Wide {
    static constexpr int kN = 256;
    static constexpr int kCols = 128;  // of an epilogue warp
    static constexpr int kEpiWarps = 8;
    static constexpr int kFirstEpi = 4;  // warps of the other roles: a warpgroup, for setmaxnreg
    static constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
    static constexpr uint32_t kOperand = 128 * kF8Block;  // bytes of a stage's A, and of its half of B
    static constexpr int kStages = 5;
    static constexpr int kBufs = 2;
    static constexpr uint32_t kTmemCols = kN * kBufs;
    static constexpr uint32_t kA = 0;
    static constexpr uint32_t kB = kA + kStages * kOperand;
    static constexpr uint32_t kStage = kB + kStages * kOperand;  // of the logits: [warps][2][32 rows][128 bytes]
    static constexpr uint32_t kWarpStage = 2 * 32 * 128;
    static constexpr uint32_t kBars = kStage + kEpiWarps * kWarpStage;
    static constexpr uint32_t kNumBars = 2 * kStages + 2 * kBufs + 1;
    static constexpr uint32_t kSlot = kBars + kNumBars * 8;
    static constexpr uint32_t kBytes = kSlot + 16 + 1024;
    static_assert(kBytes <= 227 * 1024 && kTmemCols == 512, "");
    // Registers: launched with kLaunchRegs a thread; the first warpgroup keeps few, and the
    // epilogue takes more for its 128 sums, 64 loaded values and the rest.  (With 24 for the
    // roles the compiler moved every loaded value once: 412 us in place of 373.)
    static constexpr int kLaunchRegs = 168, kRoleRegs = 40, kEpiRegs = 232;
    static_assert(32 * kFirstEpi * kRoleRegs + 32 * kEpiWarps * kEpiRegs <= kThreads * kLaunchRegs,
                  "the split fits what was launched");
};

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

template <typename O>
__global__ void __launch_bounds__(F8Wide::kThreads, 1) fp8_wide_kernel(const __grid_constant__ F8Args a) {
    using C = F8Wide;
    constexpr int kN = C::kN;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);  // alike in both CTAs
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);  // the even CTA's are used
    uint64_t* empty = full + C::kStages;
    uint64_t* tfull = empty + C::kStages;
    uint64_t* tempty = tfull + C::kBufs;  // the even CTA's are used
    uint64_t* drain = tempty + C::kBufs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kSlot);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t first = blockIdx.x / 2, step = gridDim.x / 2;  // pairs
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < C::kBufs; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * C::kEpiWarps);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        prefetch_tensormap(&a.lanes);
        prefetch_tensormap(&a.columns);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, C::kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are set up, and their tensor memory is there
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    bool failed = false;
    grid_wait();

    if (warp < C::kFirstEpi) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRoleRegs));
        if (warp == 0 && lane == 0) {
            const uint64_t pol_w = a.t_tiles == 1 ? policy_evict_first() : policy_evict_normal();
            const uint64_t pol_q = policy_evict_last();
            uint32_t it = 0;
            for (uint32_t u = first; u < a.tiles && !failed; u += step) {
                const int t0 = (int)(u % (uint32_t)a.t_tiles) * 2 * kF8M + (int)rank * kF8M;
                const int v0 = (int)(u / (uint32_t)a.t_tiles) * kN + (int)rank * (kN / 2);
                for (int j = 0; j < a.blocks; ++j, ++it) {
                    const int s = it % C::kStages;
                    if (!mbar_wait_cycles(&empty[s], ((it / C::kStages) & 1u) ^ 1u, kF8Wait)) {
                        failed = true;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 4 * C::kOperand);  // both CTAs' copies
                    const uint32_t bar = cluster_address(&full[s], 0);
                    tma_load_2d_pair(smem + C::kA + s * C::kOperand, &a.lanes, j * kF8Block, t0, bar, pol_q);
                    tma_load_2d_pair(smem + C::kB + s * C::kOperand, &a.columns, j * kF8Block, v0, bar, pol_w);
                }
            }
            // Every copy has landed before the pair ends: the even CTA's barriers count both's.
            if (rank == 0) {
                for (uint32_t k = 0; k < (uint32_t)C::kStages && k < it; ++k) {
                    const uint32_t i = it - 1 - k;
                    if (!mbar_wait_cycles(&full[i % C::kStages], (i / C::kStages) & 1u, kF8Wait)) failed = true;
                }
            }
            // The MMAs have released every stage: their arrivals here are the last thing that the
            // even CTA sends before the pair's end.
            for (uint32_t k = 0; k < (uint32_t)C::kStages && k < it && !failed; ++k) {
                const uint32_t i = it - 1 - k;
                if (!mbar_wait_cycles(&empty[i % C::kStages], (i / C::kStages) & 1u, kF8Wait)) failed = true;
            }
            if (failed) {  // the CTAs may have stopped at different copies: time to land
                const uint64_t now = global_ns();
                while (global_ns() - now < 10000000ull) {
                }
            }
        } else if (warp == 1 && lane == 0 && rank == 0) {
            constexpr uint32_t idesc = idesc_e4m3_f32(2 * kF8M, kN);
            uint32_t it = 0;
            for (uint32_t u = first; u < a.tiles && !failed; u += step) {
                for (int j = 0; j < a.blocks; ++j, ++it) {
                    const uint32_t b = it % C::kBufs;
                    const int s = it % C::kStages;
                    if (!mbar_wait_cycles(&tempty[b], ((it / C::kBufs) & 1u) ^ 1u, kF8Wait) ||
                        !mbar_wait_cycles(&full[s], (it / C::kStages) & 1u, kF8Wait)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint64_t a_at = sdesc_kmajor_sw128(smem_u32(smem + C::kA + s * C::kOperand));
                    const uint64_t b_at = sdesc_kmajor_sw128(smem_u32(smem + C::kB + s * C::kOperand));
#pragma unroll
                    for (int k = 0; k < kF8Block / 32; ++k)  // 32 bytes on: 2 in the descriptor's units
                        umma_f8_pair(tmem + b * kN, a_at + 2 * k, b_at + 2 * k, idesc, k != 0);
                    umma_commit_pair(&empty[s]);
                    umma_commit_pair(&tfull[b]);
                }
            }
            umma_commit_even(drain);
            if (!mbar_wait_cycles(drain, 0, kF8Wait)) failed = true;
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kEpiRegs));
        constexpr int kCols = C::kCols;
        const int e = warp - C::kFirstEpi, quarter = warp & 3, c0 = e / 4 * kCols;
        const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + c0;
        uint8_t* stage = smem + C::kStage + e * C::kWarpStage;
        uint32_t it = 0;
        for (uint32_t u = first; u < a.tiles && !failed; u += step) {
            const int t = (int)(u % (uint32_t)a.t_tiles) * 2 * kF8M + (int)rank * kF8M + quarter * 32 + lane;
            const int v = (int)(u / (uint32_t)a.t_tiles) * kN + c0;
            const float* qs = after_wait(a.q_scale) + (t < a.T ? t * a.scale_row : 0);
            const float* ws =
                after_wait(a.W_scale) + (int64_t)min(v / kF8Block, a.row_blocks - 1) * a.blocks;
            float next = *qs, next_w = *ws;
            uint64_t acc[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) acc[i] = 0;
#pragma unroll 1
            for (int j = 0; j < a.blocks; ++j, ++it) {  // to its end, as in the narrow tiles
                const float f = __fmul_rn(next, next_w);
                const uint64_t ff = f2_pack(f, f);
                if (j + 1 < a.blocks) {
                    qs += a.scale_col;
                    next = *qs;
                    next_w = *++ws;
                }
                const uint32_t b = it % C::kBufs;
                failed |= !mbar_wait_cycles(&tfull[b], (it / C::kBufs) & 1u, failed ? 0 : kF8Wait);
                __syncwarp();
                tc_fence_after_sync();
#pragma unroll
                for (int c = 0; c < kCols / 64; ++c) {
                    uint32_t r[64];
                    tmem_load(taddr + b * kN + c * 64, r);
                    tmem_ld_wait();
                    if (c == kCols / 64 - 1) {
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(cluster_address(&tempty[b], 0));
                    }
#pragma unroll
                    for (int i = 0; i < 64; i += 2) {
                        uint64_t& y = acc[(c * 64 + i) / 2];
                        y = f2_fma(f2_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), ff, y);
                    }
                }
            }
            failed = __any_sync(0xFFFFFFFFu, failed);
            if (failed) break;
            if (a.vector) {
                // 128 bytes of each of the warp's rows at a time, by way of shared memory, into
                // whole lines by TMA; it cuts off what lies past T or V.
                constexpr int kPer = 128 / sizeof(O);
#pragma unroll
                for (int h = 0; h < kCols / kPer; ++h) {
                    uint8_t* at = stage + (h & 1) * 32 * 128;
                    if (lane == 0) bulk_wait_group_read<1>();  // the store before the last has read its half
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float x, y;
                            if constexpr (sizeof(O) == 2) {
                                f2_unpack(acc[h * 32 + i * 4 + q], x, y);
                                w[q] = bf2_pack_rn(x, y);
                            } else {
                                f2_unpack(acc[h * 16 + i * 2 + q / 2], x, y);
                                w[q] = __float_as_uint(q & 1 ? y : x);
                            }
                        }
                        *reinterpret_cast<uint4*>(at + lane * 128 + ((i ^ (lane & 7)) * 16)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    const int col = v + h * kPer;
                    if (lane == 0) {
                        if (col < a.V && t < a.T) tma_store_2d(&a.logits, col * (int)sizeof(O), t, at);
                        bulk_commit_group();
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
                    const int col = v + c * 16 + (lane & 15), row = t - lane + (lane & 16);
                    O* at = static_cast<O*>(a.out) + (int64_t)row * a.ld_out + col;
                    const int n = col < a.V ? min(16, a.T - row) : 0;
#pragma unroll
                    for (int i = 0; i < 16; ++i, at = next_row(at, a.ld_out))
                        if (i < n) put(at, x[i]);
                }
            }
        }
        if (lane == 0) bulk_wait_group<0>();
        __syncwarp();
    }
    if (failed && a.dev_error) atomicOr(a.dev_error, PSTAT_DEV_TIMEOUT);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // neither CTA's memory is in use by the other any more
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, C::kTmemCols);
    }
}

template <int kN, typename O>
cudaError_t launch_narrow(F8Args a, const void* q, const void* W, int64_t K, const DeviceInfo& dev, cudaStream_t st) {
    using C = F8Narrow<kN>;
    static ContextSeen configured;
    const cudaError_t e = ensure_smem_optin(reinterpret_cast<const void*>(fp8_narrow_kernel<kN, O>), (int)C::kBytes,
                                            configured);
    if (e != cudaSuccess) return e;
    a.tiles = (uint32_t)((a.V + kF8M - 1) / kF8M);
    if (!make_byte_map(&a.columns, q, a.T, K, K, kN) || !make_byte_map(&a.lanes, W, a.V, K, K, kF8M))
        return cudaErrorInvalidValue;
    const unsigned grid = a.tiles < (uint32_t)dev.sm_count ? a.tiles : (unsigned)dev.sm_count;
    return launch_behind(fp8_narrow_kernel<kN, O>, grid, C::kThreads, C::kBytes, st, 1, a);
}

template <typename O>
cudaError_t launch_wide(F8Args a, const void* q, const void* W, int64_t K, const DeviceInfo& dev, cudaStream_t st) {
    using C = F8Wide;
    static ContextSeen configured;
    const cudaError_t e =
        ensure_smem_optin(reinterpret_cast<const void*>(fp8_wide_kernel<O>), (int)C::kBytes, configured);
    if (e != cudaSuccess) return e;
    // A warp that asks for registers that were not launched waits for ever.
    static std::atomic<int> regs{0};
    if (!regs) {
        cudaFuncAttributes attr;
        const cudaError_t f = cudaFuncGetAttributes(&attr, fp8_wide_kernel<O>);
        if (f != cudaSuccess) return f;
        regs = attr.numRegs;
    }
    if (regs != C::kLaunchRegs) return cudaErrorInvalidKernelImage;
    a.t_tiles = (a.T + 2 * kF8M - 1) / (2 * kF8M);
    const int64_t tiles = (int64_t)((a.V + C::kN - 1) / C::kN) * a.t_tiles;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    a.tiles = (uint32_t)tiles;
    a.vector = a.vector && (int64_t)a.V * (int)sizeof(O) <= INT32_MAX;
    if (!make_byte_map(&a.lanes, q, a.T, K, K, kF8M) || !make_byte_map(&a.columns, W, a.V, K, K, C::kN / 2) ||
        (a.vector && !make_byte_map(&a.logits, a.out, a.T, (int64_t)a.V * sizeof(O), a.ld_out * sizeof(O), 32)))
        return cudaErrorInvalidValue;
    const int64_t pairs = tiles < dev.sm_count / 2 ? tiles : dev.sm_count / 2;
    return launch_behind(fp8_wide_kernel<O>, (unsigned)(2 * pairs), C::kThreads, C::kBytes, st, 2, a);
}

// The narrowest tile that holds the tokens.  151,936 x 4096, us: up to 32 tokens 94 (tiles for 128
// take 108 to 152, wide ones 116 to 172), 64 tokens 96 (108, 117), 128 tokens 110 (wide 121).
template <typename O>
cudaError_t launch_logits_of(const F8Args& a, const void* q, const void* W, int64_t K, const DeviceInfo& dev,
                             cudaStream_t st) {
    if (a.T <= 16) return launch_narrow<16, O>(a, q, W, K, dev, st);
    if (a.T <= 32) return launch_narrow<32, O>(a, q, W, K, dev, st);
    if (a.T <= 64) return launch_narrow<64, O>(a, q, W, K, dev, st);
    if (a.T <= 128) return launch_narrow<128, O>(a, q, W, K, dev, st);
    return launch_wide<O>(a, q, W, K, dev, st);
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
    if (scale_row < 1 || scale_col < 1 || scale_row > kF8MaxStride || scale_col > kF8MaxStride ||
        cols * row_blocks > INT32_MAX)
        return PSTAT_ERR_SHAPE;
    const int64_t scale_rows = (T + rows - 1) / rows;  // two scales in one place?
    if (scale_row <= (cols - 1) * scale_col && scale_col <= (scale_rows - 1) * scale_row)
        return PSTAT_ERR_SHAPE;
    const int64_t x_bytes = extent_bytes(T, ld, K, dt == PSTAT_BF16 ? 2 : 4);
    const int64_t scale_bytes = extent_bytes(scale_rows, scale_row, (cols - 1) * scale_col + 1, 4);
    if (ranges_meet(out_q, T * K, x, x_bytes) || ranges_meet(out_scale, scale_bytes, x, x_bytes) ||
        ranges_meet(out_q, T * K, out_scale, scale_bytes))
        return PSTAT_ERR_PARAM;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != PSTAT_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const QuArgs a = {x, T, K, ld, out_q, out_scale, scale_row, scale_col, (uint32_t)cols, dev_error};
    const unsigned grid = (unsigned)(cols * row_blocks);
    cudaError_t e;
    if (rows == 1)
        e = dt == PSTAT_BF16 ? launch_quantize<uint16_t, false>(a, grid, st) : launch_quantize<float, false>(a, grid, st);
    else
        e = dt == PSTAT_BF16 ? launch_quantize<uint16_t, true>(a, grid, st) : launch_quantize<float, true>(a, grid, st);
    return e == cudaSuccess ? PSTAT_OK : PSTAT_ERR_CUDA;
}

int pstat_fp8_logits(const void* q, const float* q_scale, int64_t scale_row, int64_t scale_col, const void* W,
                     const float* W_scale, int64_t T, int64_t V, int64_t K, void* out, pstat_dtype out_dt,
                     int64_t ld_out, int* dev_error, pstat_stream_t stream) {
    if (out_dt != PSTAT_F32 && out_dt != PSTAT_BF16) return PSTAT_ERR_DTYPE;
    if (T < 0 || V < 1 || K < 16 || K % 16 || K > (1 << 24) || ld_out < V || T > INT32_MAX / 2 || V > INT32_MAX / 2 ||
        scale_row < 0 || scale_col < 0 || scale_row > kF8MaxStride || scale_col > kF8MaxStride)
        return PSTAT_ERR_SHAPE;
    if (T == 0) return PSTAT_OK;
    if (!q || !q_scale || !W || !W_scale || !out) return PSTAT_ERR_NULLPTR;
    if (!aligned_to(q, 16) || !aligned_to(W, 16) || !aligned_to(q_scale, 4) || !aligned_to(W_scale, 4) ||
        !aligned_to(out, out_dt == PSTAT_BF16 ? 2 : 4))
        return PSTAT_ERR_ALIGN;
    const int64_t cols = (K + kF8Block - 1) / kF8Block;
    const int64_t out_bytes = extent_bytes(T, ld_out, V, out_dt == PSTAT_BF16 ? 2 : 4);
    if (ranges_meet(out, out_bytes, q, T * K) || ranges_meet(out, out_bytes, W, V * K) ||
        ranges_meet(out, out_bytes, q_scale, extent_bytes(T, scale_row, (cols - 1) * scale_col + 1, 4)) ||
        ranges_meet(out, out_bytes, W_scale, (V + kF8Block - 1) / kF8Block * cols * 4))
        return PSTAT_ERR_PARAM;
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
