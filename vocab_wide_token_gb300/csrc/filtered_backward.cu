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
// one write of a row: bound by HBM.  Each thread keeps kU 8-column groups in
// flight as raw 16-byte vectors.  A group without a logit of at least tau (all
// but a few, once a filter cuts) is written as zeros without an exponential.
// A row whose start is not on 16 bytes is taken from its first column that is,
// when input and output agree on which that is, and column by column else.
// ---------------------------------------------------------------------------
constexpr int kFgThreads = 256;

template <typename Ein, typename Eout>
__global__ void __launch_bounds__(kFgThreads)
    filtered_backward_kernel(const Ein* __restrict__ logits, int64_t V, int64_t ld,
                             const int64_t* __restrict__ labels, int64_t ignore_index,
                             const float* __restrict__ weights,
                             const float2* __restrict__ rowstats,
                             const float* __restrict__ cut_logit,
                             const int64_t* __restrict__ cut_index, float temperature,
                             const float* __restrict__ temperatures, Eout* __restrict__ out,
                             int64_t ld_out, int segs, int* __restrict__ dev_error) {
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
    // p_y = 1 the difference itself would be lost.
    auto gradient = [&](float z, int64_t col) {
        if (col == y) return -g * expm1f((z - M) / temp - rs.y);
        const bool kept = z > tau || (z == tau && col <= last);
        return kept ? ex2_approx((z - M) * c) * ngK : 0.f;
    };
    auto scalar = [&](int64_t c0, int64_t c1) {
        for (int64_t col = c0 + threadIdx.x; col < c1; col += kFgThreads)
            zout[col] = out_cast(mode == 2 ? gradient(Elem<Ein>::to_float(zin[col]), col) : fill, zout);
    };

    // Columns before the first 16-byte boundary of both rows, -1 if there is none.
    const int in_off = (int)((reinterpret_cast<uintptr_t>(zin) & 15u) / sizeof(Ein));
    const int out_off = (int)((reinterpret_cast<uintptr_t>(zout) & 15u) / sizeof(Eout));
    int head = -1;
    for (int h = 0; h < 8; ++h)
        if (((in_off + h) * sizeof(Ein)) % 16 == 0 && ((out_off + h) * sizeof(Eout)) % 16 == 0) {
            head = h;
            break;
        }
    if (head < 0 || head > V) return scalar(V * seg / segs, V * (seg + 1) / segs);
    const int64_t groups = (V - head) >> 3;
    const int64_t g0 = groups * seg / segs, g1 = groups * (seg + 1) / segs;
    if (seg == 0) scalar(0, head);
    if (seg == segs - 1) scalar(head + (groups << 3), V);
    const Ein* vin = zin + head;
    Eout* vout = zout + head;

    constexpr int kVecs = (int)sizeof(Ein) / 2;  // 16-byte vectors per group
    constexpr int kU = kVecs == 1 ? 6 : 4;
    for (int64_t base = g0; base < g1; base += (int64_t)kFgThreads * kU) {
        uint4 raw[kU][kVecs];
#pragma unroll
        for (int k = 0; k < kU; ++k) {
            const int64_t i = base + k * kFgThreads + threadIdx.x;
            if (i < g1 && mode == 2) {
                const uint4* src = reinterpret_cast<const uint4*>(vin + (i << 3));
#pragma unroll
                for (int h = 0; h < kVecs; ++h) raw[k][h] = __ldcs(src + h);
            }
        }
#pragma unroll
        for (int k = 0; k < kU; ++k) {
            const int64_t i = base + k * kFgThreads + threadIdx.x;
            if (i >= g1) continue;
            float o[8];
            bool any = false;
            float x[8];
            if (mode == 2) {
                constexpr int kPer = 8 / kVecs;
#pragma unroll
                for (int h = 0; h < kVecs; ++h) {
                    float part[kPer];
                    RowReader<Ein>::unpack(raw[k][h], part);
#pragma unroll
                    for (int e = 0; e < kPer; ++e) x[h * kPer + e] = part[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) any |= x[e] >= tau;
            }
            if (any) {
                const int64_t col = head + (i << 3);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = ex2_approx((x[e] - M) * c) * ngK;
                // the few groups that the cut or the label falls into
                if (tau > -INFINITY || (y >= col && y < col + 8)) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = gradient(x[e], col + e);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = fill;
            }
            Store8<Eout>::run(vout + (i << 3), o);
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
    int64_t segs = V / 32768;
    if (segs < 1) segs = 1;
    filtered_backward_kernel<Ein, Eout><<<(unsigned)(T * segs), kFgThreads, 0, stream>>>(
        static_cast<const Ein*>(logits), V, ld, labels, ignore_index, weights,
        reinterpret_cast<const float2*>(rowstats), cut_logit, cut_index, temperature, temperatures,
        static_cast<Eout*>(out), ld_out, (int)segs, dev_error);
    return cudaGetLastError();
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
