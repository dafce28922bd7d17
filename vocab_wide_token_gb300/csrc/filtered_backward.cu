// filtered_backward.cu -- the logits' gradient of the filtered policy statistics
// (sampling.cu has their forward).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "sampling.cuh"

namespace pstat {
namespace {

// ---------------------------------------------------------------------------
// Gradient: dz_v = (w/t)(1[v = y] - kept_v e_v/S), elementwise, one read and
// one write of a row: bound by HBM.  Each thread keeps kAhead groups of columns in
// flight as raw 16-byte vectors; a group is one 16-byte vector of the gradient
// (of two, 32 bytes apart between lanes, 512 x 151,936 fp32 zeros took 73 us, and
// take 47 us).  A group without a logit of at least tau (all
// but a few, once a filter cuts) is written as zeros without an exponential.
// A row is taken from the first column whose gradient is on 16 bytes.  Where its
// logit is not (kShift: odd strides or vocabularies), the groups are shifted out
// of the aligned vectors around them, which lie inside the row; 512 rows of
// 151,937 bf16 columns out of a stride of 151,944 took 89 us column by column.
// ---------------------------------------------------------------------------
constexpr int kFgThreads = 256;

// Groups that a thread has in flight (2048 x 151,936 bf16 with a nucleus: 3 groups
// 207 us, 4 201, 5 213, 6 248: registers), and how often: few blocks leave a tail,
// many repeat the row's set-up (1024 rows of fp32: 1 192 us, 2 180, 4 184; 2048 of
// bf16: 2 214, 4 201, 10 199, but 64 rows 10.2, 9.7 and 14.4).  fp32 logits with a bf16
// gradient take the bf16 figures: 512 rows 72 us, with an fp32 gradient 91, floors 69
// and 92.
constexpr int kAhead = 4;
template <typename Eout>
constexpr int kBlockCols = kFgThreads * kAhead * (16 / (int)sizeof(Eout)) * (sizeof(Eout) == 2 ? 4 : 2);

__device__ __forceinline__ void store_group(uint16_t* p, const float (&g)[8]) {
    Store8<uint16_t>::run(p, g);
}
__device__ __forceinline__ void store_group(float* p, const float (&g)[4]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(g[0], g[1], g[2], g[3]));
}

template <typename Ein, typename Eout, bool kShift>
__global__ void __launch_bounds__(kFgThreads)
    filtered_backward_kernel(const Ein* logits, int64_t V, int64_t ld, const int64_t* labels,
                             int64_t ignore_index, const float* weights, const float2* rowstats,
                             const float* cut_logit, const int64_t* cut_index, float temperature,
                             const float* temperatures, Eout* out, int64_t ld_out, int segs,
                             int* dev_error) {
    grid_wait();
    logits = after_wait(logits);
    labels = after_wait(labels);
    weights = after_wait(weights);
    rowstats = after_wait(rowstats);  // the finish kernel before this one may just have written them
    cut_logit = after_wait(cut_logit);
    cut_index = after_wait(cut_index);
    temperatures = after_wait(temperatures);
    const int64_t t = blockIdx.x / segs;
    const int seg = (int)(blockIdx.x - t * segs);
    const Ein* zin = logits + t * ld;
    Eout* zout = out + t * ld_out;
    const int64_t y = labels ? labels[t] : ignore_index;
    const float w = weights ? weights[t] : 1.f;
    const float temp = temperatures ? temperatures[t] : temperature;
    const float2 rs = rowstats[t];
    const float tau = cut_logit[t];
    const int64_t last = cut_index[t];
    int mode = 2;  // 0: zero row, 1: NaN row, 2: compute
    if (y == ignore_index || w == 0.f) {
        mode = 0;
    } else if (!(temp >= kFilterTempMin && temp <= kFilterTempMax) || y < 0 || y >= V ||
               !(rs.x > -INFINITY) || !(rs.y == rs.y)) {
        mode = 1;
        if (seg == 0 && threadIdx.x == 0 && dev_error)
            atomicOr(dev_error, (y < 0 || y >= V) ? PSTAT_DEV_BAD_LABEL
                                : !(temp >= kFilterTempMin && temp <= kFilterTempMax)
                                    ? PSTAT_DEV_BAD_PARAM
                                    : PSTAT_DEV_EMPTY_ROW);
    } else {
        const float zy = Elem<Ein>::to_float(zin[y]);
        // a masked label is never kept, not even where nothing is filtered
        if (!(zy > -INFINITY && (zy > tau || (zy == tau && y <= last)))) mode = 0;
    }
    const float M = rs.x;
    float c = 0.f, K = 0.f, g = 0.f;
    if (mode == 2) {
        c = kLog2e / temp;
        K = exp2f(-rs.y * kLog2e);  // 1 / S
        g = w / temp;
    }
    const float ngK = -g * K;
    const float fill = mode == 1 ? NAN : 0.f;
    // Column y is kept, so its gradient is g (1 - p_y), as -g expm1(ln p_y): near
    // p_y = 1 the difference itself would be lost (ln S keeps the precision of S - 1).
    auto gradient = [&](float z, int64_t col) {
        if (col == y) return -g * expm1f((z - M) / temp - rs.y);
        const bool kept = z > tau || (z == tau && col <= last);
        return kept ? ex2_approx((z - M) * c) * ngK : 0.f;
    };
    auto scalar = [&](int64_t c0, int64_t c1) {
        for (int64_t col = c0 + threadIdx.x; col < c1; col += kFgThreads)
            zout[col] = out_cast(mode == 2 ? gradient(Elem<Ein>::to_float(zin[col]), col) : fill, zout);
    };

    constexpr int kCols = 16 / (int)sizeof(Eout);           // columns of a group
    constexpr int kVecs = kCols * (int)sizeof(Ein) / 16;  // vectors of logits of a group
    const int out_off = (int)((reinterpret_cast<uintptr_t>(zout) & 15u) / sizeof(Eout));
    int64_t head = out_off ? kCols - out_off : 0;
    uint32_t shift = 0;
    int64_t behind = 0;  // columns that the last group's vectors hold behind it
    if (kShift) {
        shift = (uint32_t)(reinterpret_cast<uintptr_t>(zin + head) & 15u);
        if (head * sizeof(Ein) < shift) head += kCols;
        if (shift) behind = (16 - shift) / sizeof(Ein);
    }
    if (head + behind > V) return scalar(V * seg / segs, V * (seg + 1) / segs);
    const int64_t groups = (V - head - behind) / kCols;
    const int64_t g0 = groups * seg / segs, g1 = groups * (seg + 1) / segs;
    if (seg == 0) scalar(0, head);
    if (seg == segs - 1) scalar(head + groups * kCols, V);
    const uint4* vin =
        reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(zin + head) - shift);
    Eout* vout = zout + head;

    constexpr int kLoads = kVecs + (kShift ? 1 : 0);
    for (int64_t base = g0; base < g1; base += (int64_t)kFgThreads * kAhead) {
        uint4 raw[kAhead][kLoads];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t i = base + k * kFgThreads + threadIdx.x;
            if (i < g1 && mode == 2) {
                const uint4* src = vin + i * kVecs;
#pragma unroll
                for (int h = 0; h < kVecs; ++h) raw[k][h] = __ldcs(src + h);
                if (kShift) raw[k][kLoads - 1] = shift ? __ldcs(src + kVecs) : make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t i = base + k * kFgThreads + threadIdx.x;
            if (i >= g1) continue;
            float o[kCols];
            bool any = false;
            float x[kCols];
            if (mode == 2) {
                constexpr int kPer = kCols / kVecs;
#pragma unroll
                for (int h = 0; h < kVecs; ++h) {
                    float part[kPer];
                    RowReader<Ein>::unpack(
                        kShift ? shift_vectors(raw[k][h], raw[k][kShift ? h + 1 : h], shift)
                               : raw[k][h],
                        part);
#pragma unroll
                    for (int e = 0; e < kPer; ++e) x[h * kPer + e] = part[e];
                }
#pragma unroll
                for (int e = 0; e < kCols; ++e) any |= x[e] >= tau;
            }
            if (any) {
                const int64_t col = head + i * kCols;
#pragma unroll
                for (int e = 0; e < kCols; ++e) o[e] = ex2_approx((x[e] - M) * c) * ngK;
                // the few groups that the cut or the label falls into
                if (tau > -INFINITY || (y >= col && y < col + kCols)) {
#pragma unroll
                    for (int e = 0; e < kCols; ++e) o[e] = gradient(x[e], col + e);
                }
            } else {
#pragma unroll
                for (int e = 0; e < kCols; ++e) o[e] = fill;
            }
            store_group(vout + i * kCols, o);
        }
    }
}

template <typename Ein, typename Eout>
cudaError_t launch_filtered_backward(const void* logits, int64_t T, int64_t V, int64_t ld,
                                     const int64_t* labels, int64_t ignore_index,
                                     const float* weights, const float* rowstats,
                                     const float* cut_logit, const int64_t* cut_index,
                                     float temperature, const float* temperatures, void* out,
                                     int64_t ld_out, int* dev_error, cudaStream_t stream) {
    // Whether the first column whose gradient is on 16 bytes has its logit there as
    // well, in every row: a boundary of either comes round within 8 rows.
    bool shift = false;
    for (int64_t t = 0; t < T && t < 8; ++t) {
        const uintptr_t zin = reinterpret_cast<uintptr_t>(logits) + (uintptr_t)(t * ld) * sizeof(Ein);
        const uintptr_t zout = reinterpret_cast<uintptr_t>(out) + (uintptr_t)(t * ld_out) * sizeof(Eout);
        const uintptr_t head = ((16 - (zout & 15u)) & 15u) / sizeof(Eout);
        shift |= ((zin + head * sizeof(Ein)) & 15u) != 0;
    }
    const int64_t segs = (V + kBlockCols<Eout> - 1) / kBlockCols<Eout>;
    const auto kernel = shift ? filtered_backward_kernel<Ein, Eout, true>
                              : filtered_backward_kernel<Ein, Eout, false>;
    return launch_behind(kernel, (unsigned)(T * segs), kFgThreads, 0, stream, 1,
                         static_cast<const Ein*>(logits), V, ld, labels, ignore_index, weights,
                         reinterpret_cast<const float2*>(rowstats), cut_logit, cut_index, temperature,
                         temperatures, static_cast<Eout*>(out), ld_out, (int)segs, dev_error);
}

}  // namespace
}  // namespace pstat

using namespace pstat;

extern "C" int pstat_filtered_backward(const void* logits, pstat_dtype dt, int64_t T, int64_t V, int64_t ld,
                            const int64_t* labels, int64_t ignore_index, const float* weights,
                            const float* rowstats, const float* cut_logit,
                            const int64_t* cut_index, float temperature,
                            const float* temperatures, void* out_dlogits, pstat_dtype out_dt,
                            int64_t ld_out, int* dev_error, pstat_stream_t stream) {
    if ((dt != PSTAT_F32 && dt != PSTAT_BF16) || (out_dt != PSTAT_F32 && out_dt != PSTAT_BF16) ||
        (dt == PSTAT_BF16 && out_dt == PSTAT_F32))
        return PSTAT_ERR_DTYPE;
    if (T < 0 || V < 1 || ld < V || ld_out < V || V > kFilterMaxV || T > PSTAT_FILTER_MAX_T)
        return PSTAT_ERR_SHAPE;
    if (!temperatures && !(temperature >= kFilterTempMin && temperature <= kFilterTempMax))
        return PSTAT_ERR_PARAM;
    if (T == 0) return PSTAT_OK;
    if (!logits || !rowstats || !cut_logit || !cut_index || !out_dlogits) return PSTAT_ERR_NULLPTR;
    if (!aligned(logits, dt == PSTAT_BF16 ? 2 : 4) ||
        !aligned(out_dlogits, out_dt == PSTAT_BF16 ? 2 : 4) || !aligned(labels, 8) ||
        !aligned(weights, 4) || !aligned(rowstats, 8) || !aligned(cut_logit, 4) ||
        !aligned(cut_index, 8) || !aligned(temperatures, 4))
        return PSTAT_ERR_ALIGN;
    // Every block of a row reads the label's logit, so the gradient cannot go
    // where the logits are.
    const uintptr_t in = reinterpret_cast<uintptr_t>(logits), out = reinterpret_cast<uintptr_t>(out_dlogits);
    const uintptr_t in_bytes = (uintptr_t)((T - 1) * ld + V) * (dt == PSTAT_BF16 ? 2 : 4);
    const uintptr_t out_bytes = (uintptr_t)((T - 1) * ld_out + V) * (out_dt == PSTAT_BF16 ? 2 : 4);
    if (in < out + out_bytes && out < in + in_bytes) return PSTAT_ERR_PARAM;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != PSTAT_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const auto run = dt == PSTAT_BF16         ? launch_filtered_backward<uint16_t, uint16_t>
                     : out_dt == PSTAT_BF16 ? launch_filtered_backward<float, uint16_t>
                                            : launch_filtered_backward<float, float>;
    return run(logits, T, V, ld, labels, ignore_index, weights, rowstats, cut_logit, cut_index,
               temperature, temperatures, out_dlogits, ld_out, dev_error, st) == cudaSuccess
               ? PSTAT_OK
               : PSTAT_ERR_CUDA;
}
