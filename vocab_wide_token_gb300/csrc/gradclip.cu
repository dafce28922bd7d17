// gradclip.cu -- the global L2 norm of a list of gradient tensors and their
// scaling by min(1, max_norm / norm).  Bound by HBM, one read for the norm, one read
// and one write for the scaling: 2.76 GB of fp32 in 383 us (7.2 TB/s) and 870 us
// (6.4 TB/s).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <memory>
#include <new>

#include "internal.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace pstat {
namespace {

constexpr int kGnThreads = 256;
constexpr int kGnUnroll = 8;                // 16-byte vectors in flight per thread
constexpr int64_t kUnitBytes = (int64_t)kGnThreads * kGnUnroll * 16;  // 32 KiB of one tensor
constexpr int kMaxBlocks = 2048;            // partial sums
constexpr int kNormCtas = 6;                // CTAs per SM, all resident
// The scaling holds 8 vectors per thread as well as their addresses: with 6 CTAs it
// spills (45 us for 110 MB where 4 take 37), and a grid of 6 for 4 resident ones runs
// one and a half waves (42 us).
constexpr int kScaleCtas = 4;
constexpr int kTeam = 16;                   // CTAs of a cluster (beyond the portable 8)
constexpr int kBatch = 800;                 // tensors of one launch (they travel as its arguments)

struct GradTensor {
    const void* in;
    void* out;
    int64_t n;
    uint32_t first_unit;
    uint32_t bf16;
};
template <int N>
struct GradBatch {
    int count;
    uint32_t units;
    GradTensor t[N];
};

__device__ __forceinline__ float elem(const void* p, int64_t i, bool bf16) {
    return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16)
                : static_cast<const float*>(p)[i];
}

// Whether an fp32 sum of squares stands: none of them can have overflowed or
// lost its low bits (squares below 2^-126 are below 2^-66 of a sum of 2^-60).
__device__ __forceinline__ bool in_range(float s) { return s > 8.6736174e-19f && s < 1.3292280e36f; }

// 16 bytes of elements, the k-th from v on, wherever v lies.
template <bool kBf16>
__device__ __forceinline__ uint4 vector_of(const void* v, int k, bool aligned) {
    if (aligned) return __ldcg(static_cast<const uint4*>(v) + k);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kBf16) {
            const uint16_t* p = static_cast<const uint16_t*>(v) + 8 * k + 2 * i;
            w[i] = p[0] | (uint32_t)p[1] << 16;
        } else {
            w[i] = static_cast<const uint32_t*>(v)[4 * k + i];
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The same elements in fp64: vectors `k`, `k + kGnThreads`, ... of `v` below
// `nv`.  Rare, so the vectors are loaded again rather than kept.
template <bool kBf16>
__device__ __noinline__ double wide_squares(const void* v, int k, int nv) {
    const bool aligned = (reinterpret_cast<uintptr_t>(v) & 15u) == 0;
    double d = 0.0;
    for (int j = 0; j < kGnUnroll && k < nv; ++j, k += kGnThreads) {
        const uint4 q = vector_of<kBf16>(v, k, aligned);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double lo = kBf16 ? bf2_lo(w[i]) : __uint_as_float(w[i]);
            const double hi = kBf16 ? bf2_hi(w[i]) : 0.f;
            d = fma(lo, lo, fma(hi, hi, d));
        }
    }
    return d;
}

// Adds the squares of a vector to four (two pairs of) sums.
template <bool kBf16>
__device__ __forceinline__ void add_squares(const uint4& q, uint64_t& s0, uint64_t& s1) {
    if (kBf16) {
        const uint64_t a = f2_pack(bf2_lo(q.x), bf2_hi(q.x));
        const uint64_t b = f2_pack(bf2_lo(q.y), bf2_hi(q.y));
        const uint64_t c = f2_pack(bf2_lo(q.z), bf2_hi(q.z));
        const uint64_t d = f2_pack(bf2_lo(q.w), bf2_hi(q.w));
        s0 = f2_fma(a, a, s0);
        s1 = f2_fma(b, b, s1);
        s0 = f2_fma(c, c, s0);
        s1 = f2_fma(d, d, s1);
    } else {
        const uint64_t a = f2_pack(__uint_as_float(q.x), __uint_as_float(q.y));
        const uint64_t b = f2_pack(__uint_as_float(q.z), __uint_as_float(q.w));
        s0 = f2_fma(a, a, s0);
        s1 = f2_fma(b, b, s1);
    }
}

// Sum of the squares of one thread's vectors of a unit.  In fp32, with one fp64
// addition for all of them: fp64 runs at about two operations per clock and SM.
// Vectors off 16 bytes are put together from their elements and added in the same
// order, so a tensor's bits do not depend on where it starts.  100 million elements:
// bf16 34 us, at an odd offset 52; fp32 61 and 78.
// The sum of up to 32 fp32 (64 bf16) squares in four fp32 sums is off by at most 10 (17:
// bf16 squares are exact, 15 of 16 additions round, and two join the sums) roundings of
// 2^-24, the norm by half of that and its own rounding: 6 x 2^-24, 9.5 x 2^-24 with bf16.
template <bool kBf16>
__device__ __forceinline__ double unit_squares(const void* v, int nv) {
    uint64_t s0 = 0, s1 = 0;
    uint32_t any = 0;
    if ((reinterpret_cast<uintptr_t>(v) & 15u) == 0) {
        uint4 q[kGnUnroll];
#pragma unroll
        for (int j = 0; j < kGnUnroll; ++j) {
            const int k = j * kGnThreads + (int)threadIdx.x;
            q[j] = k < nv ? vector_of<kBf16>(v, k, true) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < kGnUnroll; ++j) {
            any |= q[j].x | q[j].y | q[j].z | q[j].w;
            add_squares<kBf16>(q[j], s0, s1);
        }
    } else {
#pragma unroll 1
        for (int k = (int)threadIdx.x; k < nv; k += kGnThreads) {
            const uint4 q = vector_of<kBf16>(v, k, false);
            any |= q.x | q.y | q.z | q.w;
            add_squares<kBf16>(q, s0, s1);
        }
    }
    float x, y;
    f2_unpack(f2_add(s0, s1), x, y);
    const float s = x + y;
    if (in_range(s)) return (double)s;
    if (any == 0) return 0.0;
    return wide_squares<kBf16>(v, (int)threadIdx.x, nv);
}

// Fixed-order sum of one double per thread; the lanes of the first warp get it.
// Through shared memory: a warp's fp64 addition takes the SM's pipe 16 cycles, and
// this way a CTA makes 13 of them (with shuffles in every warp, 104: clipping 110 MB
// took 58 us with those and a square root in every thread, and takes 51).
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double all[kGnThreads];
    all[threadIdx.x] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x < 32) {
        for (int w = 0; w < kGnThreads; w += 32) s += all[w + (int)threadIdx.x];
#pragma unroll
        for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    }
    return s;
}

// Index of the tensor that holds unit u.  Bisected: the records are read one
// behind another from the launch's arguments, 300 of them in 5 us.
template <int N>
__device__ __forceinline__ int tensor_of(const GradBatch<N>& g, uint32_t u) {
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

// This thread's share of the squares of unit u, a unit of tensor t.
__device__ __forceinline__ double square_unit(const GradTensor& t, uint32_t u) {
    const bool bf16 = t.bf16;
    const void* in = after_wait(t.in);
    const int64_t per = kUnitBytes / (bf16 ? 2 : 4);
    const int64_t e0 = (int64_t)(u - t.first_unit) * per;
    const int64_t e1 = min(t.n, e0 + per);
    const int vec = bf16 ? 8 : 4;
    const int nv = (int)((e1 - e0) / vec);
    const void* v = static_cast<const char*>(in) + e0 * (bf16 ? 2 : 4);
    double sum = bf16 ? unit_squares<true>(v, nv) : unit_squares<false>(v, nv);
    for (int64_t k = e0 + (int64_t)nv * vec + threadIdx.x; k < e1; k += kGnThreads) {
        const double x = elem(in, k, bf16);
        sum = fma(x, x, sum);
    }
    return sum;
}

template <int N>
__global__ void __launch_bounds__(kGnThreads, kNormCtas)
    square_sums_kernel(const __grid_constant__ GradBatch<N> g, double* partial) {
    grid_wait();
    grid_launch_dependents();
    const uint32_t u0 = (uint32_t)((uint64_t)g.units * blockIdx.x / gridDim.x);
    const uint32_t u1 = (uint32_t)((uint64_t)g.units * (blockIdx.x + 1) / gridDim.x);
    double sum = 0.0;
    int i = tensor_of(g, u0);
    for (uint32_t u = u0; u < u1; ++u) {
        while (i + 1 < g.count && g.t[i + 1].first_unit <= u) ++i;
        sum += square_unit(g.t[i], u);
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// Every block that needs the norm adds the partial sums up itself, in the same
// order, so all of them hold the same bits (in the first warp).
__device__ __forceinline__ double total_of(const double* partial, int n) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kGnThreads) s += partial[i];
    return block_sum(s);
}

// What gradients are scaled by: factor, then rest, a power of two that is 1 unless
// max_norm / norm lies below the normal numbers.  There (max_norm < 4) the factor is
// 2^125 times as large, so that it keeps its 24 bits and no product overflows; an
// element of 1e37 clipped by a factor of 1e-45 is still a normal number.
struct Scale {
    float factor, rest;
    __device__ float operator()(float x) const { return x * factor * rest; }
};

// Norm and error bits, by one thread.
__device__ __forceinline__ Scale finish_norm(double total, float max_norm, bool write, float* out,
                                             int* dev_error) {
    const double norm = sqrt(total);
    const float f = (float)norm;
    const bool finite = f < INFINITY;
    if (write) {
        *out = f;
        if (!finite && dev_error) atomicOr(dev_error, PSTAT_DEV_NONFINITE);
    }
    if (!finite || norm <= (double)max_norm) return {1.f, 1.f};
    const double ratio = (double)max_norm / norm;
    return ratio < 0x1p-126 ? Scale{(float)(ratio * 0x1p125), 0x1p-125f} : Scale{(float)ratio, 1.f};
}

__global__ void __launch_bounds__(kGnThreads)
    norm_kernel(const double* partial, int n, float* out, int* dev_error) {
    grid_wait();
    partial = after_wait(partial);
    const double total = total_of(partial, n);
    if (threadIdx.x == 0) finish_norm(total, 0.f, true, out, dev_error);
}

__device__ __forceinline__ void scale_unit(const GradTensor& t, uint32_t u, const Scale scale) {
    const void* in = after_wait(t.in);
    void* out = t.out;
    const bool same = scale.factor == 1.f && scale.rest == 1.f;
    if (same && out == in) return;
    const bool bf16 = t.bf16;
    const int64_t per = kUnitBytes / (bf16 ? 2 : 4);
    const int64_t e0 = (int64_t)(u - t.first_unit) * per;
    const int64_t e1 = min(t.n, e0 + per);
    const int vec = bf16 ? 8 : 4;
    int64_t done = e0;
    if (((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0) {
        const int nv = (int)((e1 - e0) / vec);
        const int64_t off = e0 * (bf16 ? 2 : 4);
        const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(in) + off);
        uint4* o = reinterpret_cast<uint4*>(static_cast<char*>(out) + off);
        uint4 q[kGnUnroll];
#pragma unroll
        for (int j = 0; j < kGnUnroll; ++j) {
            const int k = j * kGnThreads + (int)threadIdx.x;
            if (k < nv) q[j] = __ldcs(v + k);
        }
#pragma unroll
        for (int j = 0; j < kGnUnroll; ++j) {
            const int k = j * kGnThreads + (int)threadIdx.x;
            if (k >= nv) continue;
            uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (same) continue;  // passed on bit for bit, NaNs included
                w[e] = bf16 ? bf2_pack_rn(scale(bf2_lo(w[e])), scale(bf2_hi(w[e])))
                            : __float_as_uint(scale(__uint_as_float(w[e])));
            }
            __stcs(o + k, make_uint4(w[0], w[1], w[2], w[3]));
        }
        done = e0 + (int64_t)nv * vec;
    }
    for (int64_t k = done + threadIdx.x; k < e1; k += kGnThreads) {
        if (bf16) {
            const uint16_t x = static_cast<const uint16_t*>(in)[k];
            static_cast<uint16_t*>(out)[k] =
                same ? x : (uint16_t)(bf2_pack_rn(scale(bf2_lo(x)), 0.f) & 0xFFFFu);
        } else {
            const uint32_t x = static_cast<const uint32_t*>(in)[k];
            static_cast<uint32_t*>(out)[k] =
                same ? x : __float_as_uint(scale(__uint_as_float(x)));
        }
    }
}

template <int N>
__global__ void __launch_bounds__(kGnThreads, kScaleCtas)
    scale_kernel(const __grid_constant__ GradBatch<N> g, const double* partial, int n,
                 float max_norm, float* out, int* dev_error) {
    __shared__ Scale s_scale;
    const uint32_t u0 = (uint32_t)((uint64_t)g.units * blockIdx.x / gridDim.x);
    const uint32_t u1 = (uint32_t)((uint64_t)g.units * (blockIdx.x + 1) / gridDim.x);
    int i = tensor_of(g, u1 - 1);
    grid_wait();
    partial = after_wait(partial);
    const double total = total_of(partial, n);
    if (threadIdx.x == 0) s_scale = finish_norm(total, max_norm, blockIdx.x == 0, out, dev_error);
    __syncthreads();
    const Scale scale = s_scale;
    // Backwards: what the norm read last is still in L2.
    for (uint32_t u = u1; u-- > u0;) {
        while (i > 0 && g.t[i].first_unit > u) --i;
        scale_unit(g.t[i], u, scale);
    }
}

// At most kTeam units: the norm and the scaling in one launch, by a cluster of
// one CTA per unit, whose CTAs hand each other their sums through shared memory.
// 16 units: norm 4.8 us against 5.5 by two launches, clipping 5.6 against 7.7 (and a
// launch less on the host, 2 us).  With two units per CTA the two launches win (32
// units: 8.0 against 5.5).
template <int N>
__global__ void __launch_bounds__(kGnThreads)
    few_units_kernel(const __grid_constant__ GradBatch<N> g, bool clip, float max_norm,
                     float* out, int* dev_error) {
    __shared__ double parts[kTeam];
    __shared__ Scale s_scale;
    const cg::cluster_group team = cg::this_cluster();
    const uint32_t rank = team.block_rank(), size = team.num_blocks();
    team.barrier_arrive();  // before a CTA's memory is written it has to have started
    grid_wait();
    const GradTensor& t = g.t[tensor_of(g, rank)];
    const double sum = block_sum(square_unit(t, rank));
    team.barrier_wait();
    if (threadIdx.x < size) *team.map_shared_rank(&parts[rank], threadIdx.x) = sum;
    team.sync();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (uint32_t r = 0; r < size; ++r) s += parts[r];
        s_scale = finish_norm(s, max_norm, rank == 0, out, dev_error);
    }
    if (!clip) return;
    __syncthreads();
    scale_unit(t, rank, s_scale);
}

int check_tensors(const pstat_tensor* tensors, int64_t n, bool outputs) {
    if (n < 0) return PSTAT_ERR_SHAPE;
    if (n > 0 && !tensors) return PSTAT_ERR_NULLPTR;
    for (int64_t i = 0; i < n; ++i) {
        const pstat_tensor& t = tensors[i];
        if (t.dtype != PSTAT_F32 && t.dtype != PSTAT_BF16) return PSTAT_ERR_DTYPE;
        if (t.n < 0 || t.n > PSTAT_GRAD_MAX_ELEMENTS) return PSTAT_ERR_SHAPE;
        if (t.n == 0) continue;
        if (!t.data || (outputs && !t.out)) return PSTAT_ERR_NULLPTR;
        const uintptr_t mask = t.dtype == PSTAT_BF16 ? 1 : 3;
        if ((reinterpret_cast<uintptr_t>(t.data) & mask) ||
            (outputs && (reinterpret_cast<uintptr_t>(t.out) & mask)))
            return PSTAT_ERR_ALIGN;
    }
    return PSTAT_OK;
}

// Whether an output overlaps another output, or another tensor that is read: the
// blocks that write it would race with those that use it.  (An output that is
// its own input is in place.)
struct Interval {
    uintptr_t from, to;
    bool out;
};
int check_overlap(const pstat_tensor* tensors, int64_t n) {
    std::unique_ptr<Interval[]> v(new (std::nothrow) Interval[2 * n]);
    if (!v) return PSTAT_ERR_WORKSPACE;
    int64_t m = 0;
    for (int64_t i = 0; i < n; ++i) {
        const pstat_tensor& t = tensors[i];
        if (t.n == 0) continue;
        const uintptr_t bytes = (uintptr_t)t.n * (t.dtype == PSTAT_BF16 ? 2 : 4);
        const uintptr_t in = reinterpret_cast<uintptr_t>(t.data), out = reinterpret_cast<uintptr_t>(t.out);
        v[m++] = {out, out + bytes, true};
        if (in != out) v[m++] = {in, in + bytes, false};
    }
    std::sort(v.get(), v.get() + m, [](const Interval& a, const Interval& b) { return a.from < b.from; });
    uintptr_t end_any = 0, end_out = 0;
    for (int64_t i = 0; i < m; ++i) {
        if (v[i].from < (v[i].out ? end_any : end_out)) return PSTAT_ERR_PARAM;
        end_any = std::max(end_any, v[i].to);
        if (v[i].out) end_out = std::max(end_out, v[i].to);
    }
    return PSTAT_OK;
}

// Fills the next batch from tensors[i..]; returns how many of them it covers.
template <int N>
int64_t fill(GradBatch<N>& g, const pstat_tensor* tensors, int64_t i, int64_t n) {
    g.count = 0;
    uint64_t units = 0;
    int64_t j = i;
    for (; j < n && g.count < N; ++j) {
        const pstat_tensor& t = tensors[j];
        if (t.n == 0) continue;
        const int64_t per = kUnitBytes / (t.dtype == PSTAT_BF16 ? 2 : 4);
        const uint64_t add = (uint64_t)((t.n + per - 1) / per);
        if (units + add > 0xFFFFFFFFull) break;
        g.t[g.count++] = {t.data, t.out, t.n, (uint32_t)units, t.dtype == PSTAT_BF16 ? 1u : 0u};
        units += add;
    }
    g.units = (uint32_t)units;
    return j - i;
}

int blocks_for(uint32_t units, int per_sm, const DeviceInfo& dev) {
    const uint32_t most = (uint32_t)(dev.sm_count * per_sm < kMaxBlocks ? dev.sm_count * per_sm : kMaxBlocks);
    return (int)(units < most ? units : most);
}

template <int N>
int run_norm(const pstat_tensor* tensors, int64_t n, bool clip, float max_norm, float* out_norm,
             double* partial, int64_t max_partials, int* dev_error, cudaStream_t st) {
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != PSTAT_OK) return rc;
    GradBatch<N> g;
    int n_partial = 0;
    for (int64_t i = 0; i < n;) {
        i += fill(g, tensors, i, n);
        if (g.units == 0) continue;
        if (n_partial == 0 && i == n && g.units <= (uint32_t)kTeam) {
            static ContextSeen cluster_set;
            if (ensure_large_cluster((const void*)few_units_kernel<N>, cluster_set) != cudaSuccess ||
                launch_behind(few_units_kernel<N>, g.units, kGnThreads, 0, st, g.units, g, clip,
                              max_norm, out_norm, dev_error) != cudaSuccess)
                return PSTAT_ERR_CUDA;
            return PSTAT_OK;
        }
        const int blocks = blocks_for(g.units, kNormCtas, dev);
        if (n_partial + blocks > max_partials) return PSTAT_ERR_WORKSPACE;
        if (launch_behind(square_sums_kernel<N>, (unsigned)blocks, kGnThreads, 0, st, 1, g,
                          partial + n_partial) != cudaSuccess)
            return PSTAT_ERR_CUDA;
        n_partial += blocks;
    }
    if (!clip || n_partial == 0) {
        if (launch_behind(norm_kernel, 1, kGnThreads, 0, st, 1, (const double*)partial, n_partial,
                          out_norm, dev_error) != cudaSuccess)
            return PSTAT_ERR_CUDA;
    } else {
        for (int64_t i = 0; i < n;) {
            i += fill(g, tensors, i, n);
            if (g.units == 0) continue;
            if (launch_behind(scale_kernel<N>, (unsigned)blocks_for(g.units, kScaleCtas, dev), kGnThreads, 0, st,
                              1, g, (const double*)partial, n_partial, max_norm, out_norm,
                              dev_error) != cudaSuccess)
                return PSTAT_ERR_CUDA;
        }
    }
    return cudaGetLastError() == cudaSuccess ? PSTAT_OK : PSTAT_ERR_CUDA;
}

int64_t max_launches(const pstat_tensor* tensors, int64_t n, int per) {
    // A batch ends when it is full or its unit index would pass 32 bits.
    uint64_t units = 0;
    for (int64_t i = 0; i < n; ++i) units += (uint64_t)(tensors[i].n / (kUnitBytes / 4) + 1);
    return (n + per - 1) / per + (int64_t)(units >> 31) + 1;
}

int norm_entry(const pstat_tensor* tensors, int64_t n, bool clip, float max_norm, float* out_norm,
               void* workspace, size_t ws_bytes, int* dev_error, pstat_stream_t stream) {
    int rc = check_tensors(tensors, n, clip);
    if (rc != PSTAT_OK) return rc;
    if (clip && !(max_norm >= 0.f)) return PSTAT_ERR_PARAM;
    if (clip && n > 0) {
        rc = check_overlap(tensors, n);
        if (rc != PSTAT_OK) return rc;
    }
    if (!out_norm) return PSTAT_ERR_NULLPTR;
    size_t need = 0;
    rc = pstat_grad_workspace_size(tensors, n, &need);
    if (rc != PSTAT_OK) return rc;
    if (!workspace || ws_bytes < need) return PSTAT_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 7u) || (reinterpret_cast<uintptr_t>(out_norm) & 3u))
        return PSTAT_ERR_ALIGN;
    double* partial = static_cast<double*>(workspace);
    const int64_t room = (int64_t)(ws_bytes / sizeof(double));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (n <= 32)
        return run_norm<32>(tensors, n, clip, max_norm, out_norm, partial, room, dev_error, st);
    return run_norm<kBatch>(tensors, n, clip, max_norm, out_norm, partial, room, dev_error, st);
}

}  // namespace
}  // namespace pstat

using namespace pstat;

extern "C" {

int pstat_grad_workspace_size(const pstat_tensor* tensors, int64_t n_tensors, size_t* bytes) {
    if (!bytes) return PSTAT_ERR_NULLPTR;
    const int rc = check_tensors(tensors, n_tensors, false);
    if (rc != PSTAT_OK) return rc;
    *bytes = (size_t)max_launches(tensors, n_tensors, n_tensors <= 32 ? 32 : kBatch) * kMaxBlocks *
             sizeof(double);
    return PSTAT_OK;
}

int pstat_grad_norm(const pstat_tensor* tensors, int64_t n_tensors, float* out_norm,
                    void* workspace, size_t ws_bytes, int* dev_error, pstat_stream_t stream) {
    return norm_entry(tensors, n_tensors, false, 0.f, out_norm, workspace, ws_bytes, dev_error,
                      stream);
}

int pstat_clip_grad_norm(const pstat_tensor* tensors, int64_t n_tensors, float max_norm,
                         float* out_norm, void* workspace, size_t ws_bytes, int* dev_error,
                         pstat_stream_t stream) {
    return norm_entry(tensors, n_tensors, true, max_norm, out_norm, workspace, ws_bytes, dev_error,
                      stream);
}

}  // extern "C"
