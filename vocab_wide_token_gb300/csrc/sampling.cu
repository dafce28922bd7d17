// sampling.cu -- drawing a token per row and the policy statistics of given
// labels under the tempered, truncated softmax (filter_math.cuh has the
// definitions).
//
//  filter_records_kernel  the only full read of the logits in the common case:
//                         per chunk the maximum and the tempered sums, per lane
//                         of a chunk the maximum of its columns (its group)
//  filter_finish_kernel   one CTA per row: from the records the whole sum, from
//                         the group maxima the few groups that can hold a kept
//                         token; reads those again, sorts what it finds and
//                         decides, where fp32 sums with their error bound do
//  filter_exact_kernel    the rows that were left: clusters of CTAs that go over
//                         the row again with exact sums
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "chunk_math.cuh"
#include "filter_math.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace pstat {
namespace {

constexpr int kExThreads = 512;
constexpr int kExWarps = kExThreads / 32;
constexpr int kBins = 2048;    // bins of one histogram level
constexpr int kCand = 2048;    // elements that are sorted at once
constexpr int kSpan = 4096;    // columns of one span of the index-order scan
constexpr int kMaxSpans = (int)(kFilterMaxV / kSpan);
static_assert(kBins % kExThreads == 0 && kCand % kExThreads == 0 && kSpan % kExThreads == 0, "");

struct FilterArgs {
    const void* logits;
    int64_t T, V, ld;
    int chunks;                 // of a row
    const float* uniform;       // sampling
    const int64_t* labels;      // statistics
    int64_t ignore_index;
    float temperature, top_p, min_p;
    int64_t top_k;
    const float* temperatures;  // per row, or null
    const int32_t* top_ks;
    const float* top_ps;
    const float* min_ps;
    int64_t* token;
    float* logprob;
    float* entropy;
    float2* rowstats;
    float* cut_logit;
    int64_t* cut_index;
    int* dev_error;
    // workspace
    float4* records;            // [T, chunks]
    void* group_max;            // [T, chunks, 32], the logits' type
    int* left_count;            // rows that the finish kernel leaves to the exact one
    int* left;                  // [T]
    ExpTable table;
};

// One row's settings.
struct RowSettings {
    float temp, top_p, min_p, u;
    int64_t top_k;
    bool greedy, valid, cut_k, cut_p, cut_m;
};
template <bool kSample>
__device__ __forceinline__ RowSettings row_settings(const FilterArgs& a, int64_t t) {
    RowSettings r;
    r.temp = a.temperatures ? a.temperatures[t] : a.temperature;
    r.top_p = a.top_ps ? a.top_ps[t] : a.top_p;
    r.min_p = a.min_ps ? a.min_ps[t] : a.min_p;
    r.top_k = a.top_ks ? a.top_ks[t] : a.top_k;
    r.u = kSample ? a.uniform[t] : 0.f;
    r.greedy = kSample && r.temp == 0.f;
    r.valid = (r.greedy || (r.temp >= kFilterTempMin && r.temp <= kFilterTempMax)) &&
              (r.top_p > 0.f && r.top_p <= 1.f) && (r.min_p >= 0.f && r.min_p <= 1.f) &&
              (r.u >= 0.f && r.u < 1.f);
    r.cut_k = r.top_k > 0 && r.top_k < a.V;
    r.cut_p = r.top_p < 1.f;
    r.cut_m = r.min_p > 0.f;
    return r;
}
// x >= ln(min_p)  <=>  z >= M + t ln(min_p), rounded up to a float.
__device__ __forceinline__ float min_p_logit(float M, const RowSettings& r) {
    return r.cut_m ? __double2float_ru((double)M + (double)r.temp * log((double)r.min_p))
                   : -INFINITY;
}

template <bool kSample>
__device__ void write_undefined(const FilterArgs& a, int64_t t, int err) {
    a.logprob[t] = NAN;
    if (kSample) {
        a.token[t] = -1;
    } else {
        a.entropy[t] = NAN;
        a.rowstats[t] = make_float2(NAN, NAN);
        a.cut_logit[t] = NAN;
        a.cut_index[t] = -1;
    }
    if (a.dev_error) atomicOr(a.dev_error, err);
}

__device__ __forceinline__ bool is_kept(float z, int64_t col, uint32_t cut_key, uint32_t cut_index) {
    const uint32_t dk = desc_key(z);
    return dk < cut_key || (dk == cut_key && (uint32_t)col <= cut_index);
}

// Statistics of one row from its cut, kept sum and entropy (one thread).
template <typename E>
__device__ void write_statistics(const FilterArgs& a, int64_t t, const E* row, float M, float lnS,
                                 float H, float temp, uint32_t cut_key, uint32_t cut_index) {
    int err = 0;
    float lp;
    const int64_t y = a.labels ? a.labels[t] : a.ignore_index;
    if (y == a.ignore_index) {
        lp = 0.f;
    } else if (y < 0 || y >= a.V) {
        lp = H = NAN;
        err = PSTAT_DEV_BAD_LABEL;
    } else {
        const float z = Elem<E>::to_float(row[y]);
        lp = is_kept(z, y, cut_key, cut_index) ? (z - M) / temp - lnS : -INFINITY;
    }
    a.logprob[t] = lp;
    a.entropy[t] = H;
    a.rowstats[t] = make_float2(M, lnS);
    a.cut_logit[t] = cut_key == 0xFFFFFFFFu ? -INFINITY : key_logit(cut_key);
    a.cut_index[t] = (int64_t)cut_index;
    if (err && a.dev_error) atomicOr(a.dev_error, err);
}

// ---------------------------------------------------------------------------
// Records.  The streaming scheme of the chunk statistics: every warp owns a
// ring of two 8 KB slots that bulk copies fill, takes a chunk out of its slot
// into registers (lane L: the 16-byte vectors L, L + 32, ...) and refills the
// slot at once.  The items (row, chunk) are split into one contiguous range per
// warp.  Lane L's maximum over its vectors is the maximum of group L of the
// chunk's columns.
// ---------------------------------------------------------------------------
template <typename E, bool kU>
__global__ void __launch_bounds__(kWarps * 32, 1)
    filter_records_kernel(const __grid_constant__ FilterArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int lane = threadIdx.x & 31;
    uint8_t* slots = smem + (size_t)warp * kStages * kSlotBytes;
    uint64_t* bars =
        reinterpret_cast<uint64_t*>(smem + (size_t)warps * kStages * kSlotBytes) + warp * kStages;
    constexpr int kChunk = Elem<E>::kChunk;
    const E* logits = static_cast<const E*>(a.logits);
    E* group_max = static_cast<E*>(a.group_max);
    const int V = (int)a.V, chunks = a.chunks;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.left_count = 0;

    const int64_t n_items = a.T * chunks;
    const int64_t gw = (int64_t)blockIdx.x * warps + warp;
    const int64_t nw = (int64_t)gridDim.x * warps;
    const int64_t i0 = n_items * gw / nw, i1 = n_items * (gw + 1) / nw;
    const int64_t n = i1 - i0;
    if (n <= 0) return;
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&bars[s], 1);
        fence_mbar_init();
    }
    __syncwarp();
    const uint64_t policy = policy_evict_normal();

    struct Item {
        int64_t t;
        int g;
    };
    auto next_item = [&](Item& it) {
        if (++it.g == chunks) {
            it.g = 0;
            ++it.t;
        }
    };
    auto locate = [&](const Item& it, const E*& src, int& len) -> bool {
        const int start = it.g * kChunk;
        len = min(kChunk, V - start);
        src = logits + it.t * a.ld + start;
        return ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) &&
               ((((size_t)len * sizeof(E)) & 15u) == 0);
    };
    auto issue = [&](const Item& it, int slot) {
        const E* src;
        int len;
        if (locate(it, src, len) && lane == 0) {
            const uint32_t bytes = (uint32_t)len * (uint32_t)sizeof(E);
            mbar_arrive_expect_tx(&bars[slot], bytes);
            bulk_g2s_hint(slots + (size_t)slot * kSlotBytes, src, bytes, &bars[slot], policy);
        }
    };
    auto scale_of = [&](int64_t t) {
        const float temp = a.temperatures ? a.temperatures[t] : a.temperature;
        return (temp >= kFilterTempMin && temp <= kFilterTempMax) ? temp_scale(temp).ch : kLog2e;
    };

    Item cur = {i0 / chunks, (int)(i0 % chunks)};
    Item ahead = cur;
    const int64_t prologue = n < kStages ? n : kStages;
    for (int64_t j = 0; j < prologue; ++j) {
        issue(ahead, (int)j);
        next_item(ahead);
    }
    uint32_t phase = 0;
    int64_t j = 0;
    bool timed_out = false;
    float c = scale_of(cur.t);
    for (; j < n; ++j) {
        const int slot = (int)(j % kStages);
        E* buf = reinterpret_cast<E*>(slots + (size_t)slot * kSlotBytes);
        const E* src;
        int len;
        if (locate(cur, src, len)) {
            bool ok = mbar_wait_bounded(&bars[slot], (phase >> slot) & 1u, kWaitLimitNs);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) {
                timed_out = true;
                break;
            }
            phase ^= 1u << slot;
        } else {
            constexpr int kVec = Elem<E>::kVec;
            const int padded = (len + kVec - 1) / kVec * kVec;
            for (int k = lane; k < padded; k += 32) buf[k] = (k < len) ? src[k] : Elem<E>::neg_inf();
            __syncwarp();
        }
        uint4 q[kVecPerLane];
        load_chunk_regs<E>(buf, len, lane, q);
        __syncwarp();
        fence_proxy_async_smem();  // our reads of the slot precede the next bulk write into it
        if (j + kStages < n) {
            issue(ahead, slot);
            next_item(ahead);
        }
        const float lm = lane_max(q, (E*)nullptr);
        const ChunkRecord r = chunk_record<E, kU>(q, lm, c);
        // exact: the maximum is one of the logits
        group_max[(i0 + j) * 32 + lane] = out_cast(lm, (E*)nullptr);
        if (lane == 0) a.records[i0 + j] = make_float4(r.m, r.s, r.u, r.delta);
        const int64_t t = cur.t;
        next_item(cur);
        if (cur.t != t && j + 1 < n) c = scale_of(cur.t);
    }
    if (timed_out) {
        if (lane == 0 && a.dev_error) atomicOr(a.dev_error, PSTAT_DEV_TIMEOUT);
        // The rows this warp leaves unfinished are undefined; copies still in
        // flight into this CTA's shared memory are drained before it ends.
        for (int64_t k = j; k < n; ++k)
            if (lane == 0) a.records[i0 + k] = make_float4(NAN, 0.f, 0.f, 0.f);
        const int64_t last = (j + kStages < n) ? j + kStages : n;
        for (int64_t k = j; k < last; ++k) {
            const int slot = (int)(k % kStages);
            const E* src;
            int len;
            if (locate(cur, src, len)) {
                mbar_wait_bounded(&bars[slot], (phase >> slot) & 1u, kWaitLimitNs);
                phase ^= 1u << slot;
            }
            next_item(cur);
        }
    }
}

// What one element selection found: the element (key, index), its rank in the
// order (1-based) and the mass up to and including it.
struct Selection {
    uint32_t key, index;
    uint32_t rank;
    uint64_t mass;
};

struct Histogram {
    uint32_t count[kBins];
    unsigned long long mass[kBins];
};

struct ExactShared {
    Histogram level0, level1;
    unsigned long long cand[kCand];
    unsigned long long span_mass[kMaxSpans];
    float span_u[kMaxSpans];
    float2 table[64];
    unsigned long long scratch[2 * kExWarps];
    // Team results, in the first CTA of a cluster.
    uint32_t n_min;
    uint32_t n_cand;
    uint32_t first;
    uint32_t first_kept;
    // Decisions that the first CTA announces.
    uint32_t klo, khi, n_in, count_before;
    uint64_t mass_before;
    Selection sel;
};

template <typename E>
struct RowReader;
template <>
struct RowReader<uint16_t> {
    static constexpr int kVec = 8;
    __device__ static void unpack(const uint4& q, float (&x)[8]) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf2_lo(w[i]);
            x[2 * i + 1] = bf2_hi(w[i]);
        }
    }
};
template <>
struct RowReader<float> {
    static constexpr int kVec = 4;
    __device__ static void unpack(const uint4& q, float (&x)[4]) {
        x[0] = __uint_as_float(q.x);
        x[1] = __uint_as_float(q.y);
        x[2] = __uint_as_float(q.z);
        x[3] = __uint_as_float(q.w);
    }
};

// Calls f(column, logit) for every column of a row, shared out over `n`
// threads of which this is thread `i`: whole 16-byte vectors between a head
// and a tail that are read one by one.
template <typename E, typename F>
__device__ __forceinline__ void for_each_logit(const E* row, int V, int i, int n, F f) {
    constexpr int kVec = RowReader<E>::kVec;
    const int skew = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(E));
    const int head = min(V, skew ? kVec - skew : 0);
    const int nv = (V - head) / kVec;
    const int tail = head + nv * kVec;
    if (i < head) f(i, Elem<E>::to_float(row[i]));
    const uint4* v = reinterpret_cast<const uint4*>(row + head);
    for (int j = i; j < nv; j += n) {
        float x[kVec];
        RowReader<E>::unpack(__ldg(v + j), x);
#pragma unroll
        for (int e = 0; e < kVec; ++e) f(head + j * kVec + e, x[e]);
    }
    for (int c = tail + i; c < V; c += n) f(c, Elem<E>::to_float(row[c]));
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// Exclusive sums of (a, b) over the threads of the CTA, in thread order.
template <int kThreads, typename T>
__device__ __forceinline__ void block_scan(unsigned long long* scratch, T a, T b, T& a_ex,
                                           T& b_ex) {
    static_assert(sizeof(T) <= 8, "");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T* wa = reinterpret_cast<T*>(scratch);
    T* wb = reinterpret_cast<T*>(scratch + kThreads / 32);
    T sa = a, sb = b;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T ta = __shfl_up_sync(0xFFFFFFFFu, sa, off);
        const T tb = __shfl_up_sync(0xFFFFFFFFu, sb, off);
        if (lane >= off) {
            sa += ta;
            sb += tb;
        }
    }
    if (lane == 31) {
        wa[warp] = sa;
        wb[warp] = sb;
    }
    __syncthreads();
    T oa = 0, ob = 0;
    for (int w = 0; w < warp; ++w) {
        oa += wa[w];
        ob += wb[w];
    }
    // exclusive sum of the lanes, without taking a back out of a sum
    T pa = __shfl_up_sync(0xFFFFFFFFu, sa, 1), pb = __shfl_up_sync(0xFFFFFFFFu, sb, 1);
    a_ex = lane ? oa + pa : oa;
    b_ex = lane ? ob + pb : ob;
    __syncthreads();
}

// Ascending bitonic sort of keys[0..n), padded in place to a power of two.
template <int kThreads>
__device__ __forceinline__ void sort_keys(unsigned long long* keys, int n) {
    int m = 2;
    while (m < n) m <<= 1;
    for (int i = n + threadIdx.x; i < m; i += kThreads) keys[i] = ~0ull;
    __syncthreads();
    for (int size = 2; size <= m; size <<= 1) {
        for (int stride = size >> 1; stride; stride >>= 1) {
            for (int p = threadIdx.x; p < m / 2; p += kThreads) {
                const int i = 2 * p - (p & (stride - 1));
                const unsigned long long a = keys[i], b = keys[i + stride];
                if ((a > b) == ((i & size) == 0)) {
                    keys[i] = b;
                    keys[i + stride] = a;
                }
            }
            __syncthreads();
        }
    }
}

// One row, worked on by the CTAs of a cluster (the team): passes over the row
// are shared out over all of them, decisions are taken in the first.
template <typename E>
struct Team {
    ExactShared& sm;        // this CTA's
    ExactShared& lead;      // the first CTA's
    cg::cluster_group cluster;
    const E* row;
    int V;
    int thread, threads;     // of the team
    bool first;              // this is the first CTA
    float M;
    TempScale c;
    int k;                   // digits of the fixed weights
    float bin_scale;

    template <typename F>
    __device__ void each(F f) const {
        for_each_logit(row, V, thread, threads, f);
    }
    __device__ uint64_t weight(float z) const { return fixed_weight(z, M, c, k, sm.table); }
    // Level-0 bins: equal steps of M - z, the last one open (the difference
    // and the product round monotonely, so bins are ranges of the order).
    __device__ int bin0(float z) const { return min(kBins - 1, __float2int_rd((M - z) * bin_scale)); }

    __device__ void clear(Histogram& h) const {
        for (int i = threadIdx.x; i < kBins; i += kExThreads) {
            h.count[i] = 0;
            h.mass[i] = 0;
        }
        __syncthreads();
    }
    // Adds every CTA's histogram to the first one's.
    __device__ void merge(Histogram ExactShared::*which) {
        cluster.sync();
        if (!first) {
            Histogram& mine = sm.*which;
            Histogram& all = lead.*which;
            for (int i = threadIdx.x; i < kBins; i += kExThreads) {
                if (mine.count[i]) atomicAdd(&all.count[i], mine.count[i]);
                if (mine.mass[i]) atomicAdd(&all.mass[i], mine.mass[i]);
            }
        }
        cluster.sync();
    }

    // First CTA: the bin in which the count reaches `want` (by_count) or the
    // mass reaches `target`; announces what lies before it and inside it.
    __device__ int pick_bin(const Histogram& h, bool by_count, uint32_t want, double target) {
        constexpr int kPer = kBins / kExThreads;
        const int b0 = threadIdx.x * kPer;
        uint64_t n = 0, w = 0;
        for (int i = 0; i < kPer; ++i) {
            n += h.count[b0 + i];
            w += h.mass[b0 + i];
        }
        uint64_t nb, wb;
        block_scan<kExThreads, uint64_t>(sm.scratch, n, w, nb, wb);
        nb += sm.count_before;
        wb += sm.mass_before;
        __syncthreads();
        for (int i = 0; i < kPer; ++i) {
            const uint64_t n1 = nb + h.count[b0 + i], w1 = wb + h.mass[b0 + i];
            const bool here = by_count ? (nb < want && want <= n1)
                                       : ((double)wb < target && (double)w1 >= target);
            if (here) {
                sm.count_before = (uint32_t)nb;
                sm.mass_before = wb;
                sm.n_in = h.count[b0 + i];
                sm.first = b0 + i;
            }
            nb = n1;
            wb = w1;
        }
        __syncthreads();
        return (int)sm.first;
    }

    // The element at which the count reaches `want`, or the mass `target`, in
    // the order of the finite logits; level0 holds all of them.  Bins are
    // narrowed until what is left can be sorted, or is one value.
    __device__ Selection select(bool by_count, uint32_t want, double target) {
        if (first) {
            if (threadIdx.x == 0) {
                sm.count_before = 0;
                sm.mass_before = 0;
            }
            __syncthreads();
            const int b = pick_bin(sm.level0, by_count, want, target);
            if (threadIdx.x < 2) {
                // Smallest key whose bin is >= b (thread 0) and > b (thread 1).
                const int edge = b + (int)threadIdx.x;
                uint32_t lo = desc_key(M), hi = kKeyNegInf;  // answer in [lo, hi]
                while (lo < hi) {
                    const uint32_t mid = lo + (hi - lo) / 2;
                    if (bin0(key_logit(mid)) >= edge)
                        hi = mid;
                    else
                        lo = mid + 1;
                }
                if (threadIdx.x == 0)
                    sm.klo = lo;
                else
                    sm.khi = b == kBins - 1 ? kKeyNegInf - 1 : lo - 1;
            }
        }
        cluster.sync();
        uint32_t klo = lead.klo, khi = lead.khi, n_in = lead.n_in;
        while (n_in > kCand && klo < khi) {
            int shift = 0;
            while (((khi - klo) >> shift) >= (uint32_t)kBins) ++shift;
            clear(sm.level1);
            each([&](int, float z) {
                const uint32_t dk = desc_key(z);
                if (dk >= klo && dk <= khi) {
                    const int b = (int)((dk - klo) >> shift);
                    atomicAdd(&sm.level1.count[b], 1u);
                    atomicAdd(&sm.level1.mass[b], (unsigned long long)weight(z));
                }
            });
            merge(&ExactShared::level1);
            if (first) {
                const uint32_t b = (uint32_t)pick_bin(sm.level1, by_count, want, target);
                if (threadIdx.x == 0) {
                    const uint32_t lo = klo + (b << shift);
                    sm.klo = lo;
                    sm.khi = min(khi, lo + ((1u << shift) - 1u));
                }
            }
            cluster.sync();
            klo = lead.klo;
            khi = lead.khi;
            n_in = lead.n_in;
        }
        if (n_in > kCand)
            select_tie(klo, by_count, want, target);
        else
            select_sorted(klo, khi, by_count, want, target);
        cluster.sync();
        return lead.sel;
    }

    // Few elements left: gather them into the first CTA, sort, scan.
    __device__ void select_sorted(uint32_t klo, uint32_t khi, bool by_count, uint32_t want,
                                  double target) {
        if (first && threadIdx.x == 0) sm.n_cand = 0;
        cluster.sync();
        each([&](int col, float z) {
            const uint32_t dk = desc_key(z);
            if (dk >= klo && dk <= khi) {
                const uint32_t at = atomicAdd(&lead.n_cand, 1u);
                if (at < (uint32_t)kCand)
                    lead.cand[at] = ((unsigned long long)dk << 32) | (uint32_t)col;
            }
        });
        cluster.sync();
        if (!first) return;
        const int n = min((int)sm.n_cand, kCand);
        sort_keys<kExThreads>(sm.cand, n);
        constexpr int kPer = kCand / kExThreads;
        const int i0 = threadIdx.x * kPer;
        uint64_t w[kPer], sum = 0;
        for (int i = 0; i < kPer; ++i) {
            w[i] = i0 + i < n ? weight(key_logit((uint32_t)(sm.cand[i0 + i] >> 32))) : 0;
            sum += w[i];
        }
        uint64_t wb, unused;
        block_scan<kExThreads, uint64_t>(sm.scratch, sum, 0, wb, unused);
        wb += sm.mass_before;
        const uint32_t before = sm.count_before;
        for (int i = 0; i < kPer && i0 + i < n; ++i) {
            const uint64_t w1 = wb + w[i];
            const uint32_t rank = before + i0 + i + 1;
            if (by_count ? rank == want : ((double)wb < target && (double)w1 >= target)) {
                const unsigned long long e = sm.cand[i0 + i];
                sm.sel = {(uint32_t)(e >> 32), (uint32_t)e, rank, w1};
            }
            wb = w1;
        }
    }

    // Many equal logits: how many of them are taken follows from their common
    // weight; the last one taken is found by counting them in index order.
    __device__ void select_tie(uint32_t key, bool by_count, uint32_t want, double target) {
        clear(sm.level1);
        each([&](int col, float z) {
            if (desc_key(z) == key) atomicAdd(&sm.level1.count[col / kSpan], 1u);
        });
        merge(&ExactShared::level1);
        if (!first) return;
        const uint64_t w = weight(key_logit(key));
        const uint32_t before = sm.count_before, n_in = sm.n_in;
        const uint64_t mass_before = sm.mass_before;
        uint32_t take;
        if (by_count) {
            take = want - before;
        } else {
            // smallest take >= 1 with mass_before + take w >= target
            uint32_t lo = 1, hi = n_in;
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo) / 2;
                if ((double)(mass_before + (uint64_t)mid * w) >= target)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            take = lo;
        }
        __syncthreads();
        const int spans = (V + kSpan - 1) / kSpan;
        uint64_t nb, unused;
        const uint64_t mine = (int)threadIdx.x < spans ? sm.level1.count[threadIdx.x] : 0;
        block_scan<kExThreads, uint64_t>(sm.scratch, mine, 0, nb, unused);
        if (nb < take && take <= nb + mine) {
            sm.first = threadIdx.x;
            sm.n_in = (uint32_t)nb;
        }
        __syncthreads();
        constexpr int kPer = kSpan / kExThreads;
        const int c0 = (int)sm.first * kSpan + threadIdx.x * kPer;
        const uint64_t skipped = sm.n_in;
        uint32_t hit = 0;
        for (int i = 0; i < kPer; ++i)
            if (c0 >= 0 && c0 + i < V && desc_key(Elem<E>::to_float(row[c0 + i])) == key) hit |= 1u << i;
        block_scan<kExThreads, uint64_t>(sm.scratch, __popc(hit), 0, nb, unused);
        nb += skipped;
        for (int i = 0; i < kPer; ++i) {
            if (!(hit >> i & 1u)) continue;
            if (++nb == take)
                sm.sel = {key, (uint32_t)(c0 + i), before + take, mass_before + (uint64_t)take * w};
        }
        __syncthreads();
    }
};

static_assert(kMaxSpans <= kExThreads && kMaxSpans <= kBins, "one thread per span");

// ---------------------------------------------------------------------------
// Finish: one CTA per row.
//
// Nothing filtered: the statistics follow from the records; a draw finds its
// chunk by the prefix sums of the chunks and its column by those of that
// chunk alone.  It stands when the target u S lies further than the sums' error
// bound from both ends of the column's interval.
//
// Filtered: a histogram of the group maxima over M - z gives a bin b such that
// the groups whose maximum lies in bins <= b are sure (top-k: k maxima, so at
// least k columns; min-p: the bin of its threshold) or likely (top-p: their
// maxima alone hold the mass) to hold all kept columns.  Only those groups are
// read again, and their columns in bins <= b sorted.  Their weights are exact;
// a nucleus is measured against the fp32 sum with its error bound (against an
// exact one after top-k), and the row is left to the exact kernel when the
// bound does not decide or the columns do not suffice.
// ---------------------------------------------------------------------------
constexpr int kFinThreads = 256;
constexpr int kFinBins = 1024;     // 64 binary orders of e, in steps of 1/16
constexpr int kFinCand = 1024;
constexpr int kFinGroups = 2048;
constexpr int kMaxChunks = (int)(kFilterMaxV / PSTAT_CHUNK_F32);

struct FinishShared {
    union {
        struct {
            uint32_t count[kFinBins];
            uint32_t mass[kFinBins];
        } hist;
        unsigned long long weight[kFinCand];  // inclusive sums
        float prefix[kMaxChunks];
    };
    unsigned long long cand[kFinCand];
    uint16_t group[kFinGroups];
    float2 table[64];
    unsigned long long scratch[2 * (kFinThreads / 32)];
    uint32_t n_group, n_cand, bin, found;
};
static_assert(kMaxChunks * 32 <= 65536, "group indices are 16 bits");

__device__ __forceinline__ void leave_row(const FilterArgs& a, int64_t t) {
    if (threadIdx.x == 0) a.left[atomicAdd(a.left_count, 1)] = (int)t;
}

// Reads kVec columns from `col` (a multiple of kVec) of a row; columns past V
// read as -inf.
template <typename E>
__device__ __forceinline__ void load_columns(const E* row, int col, int V,
                                             float (&x)[Elem<E>::kVec]) {
    constexpr int kVec = Elem<E>::kVec;
    const E* p = row + col;
    if (col + kVec <= V && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        RowReader<E>::unpack(__ldg(reinterpret_cast<const uint4*>(p)), x);
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            x[e] = col + e < V ? Elem<E>::to_float(p[e]) : -INFINITY;
    }
}

template <typename E>
__device__ void finish_greedy(const FilterArgs& a, int64_t t, const E* row, const float4* rec,
                              float M, FinishShared& sm) {
    constexpr int kChunk = Elem<E>::kChunk;
    if (threadIdx.x == 0) sm.bin = sm.found = 0xFFFFFFFFu;
    __syncthreads();
    for (int i = threadIdx.x; i < a.chunks; i += kFinThreads)
        if (rec[i].x == M) atomicMin(&sm.bin, (uint32_t)i);
    __syncthreads();
    const int c0 = (int)sm.bin * kChunk, c1 = min((int)a.V, c0 + kChunk);
    for (int col = c0 + threadIdx.x; col < c1; col += kFinThreads)
        if (Elem<E>::to_float(row[col]) == M) {
            atomicMin(&sm.found, (uint32_t)col);
            break;
        }
    __syncthreads();
    if (threadIdx.x == 0) {
        a.token[t] = (int64_t)sm.found;
        a.logprob[t] = 0.f;
    }
}

template <typename E>
__device__ void finish_draw(const FilterArgs& a, int64_t t, const E* row, const float4* rec,
                            float M, float c, const RowSettings& rs, float lnS,
                            FinishShared& sm) {
    const int lane = threadIdx.x & 31, n = a.chunks;
    if (threadIdx.x < 32) {
        float carry = 0.f;
        for (int i0 = 0; i0 < n; i0 += 32) {
            float w = 0.f;
            if (i0 + lane < n) {
                const float4 r = rec[i0 + lane];
                if (r.x > -INFINITY) w = r.y * exp2f(fmaf(r.x - M, c, -r.w));
            }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float o = __shfl_up_sync(0xFFFFFFFFu, w, off);
                if (lane >= off) w += o;
            }
            w += carry;
            if (i0 + lane < n) sm.prefix[i0 + lane] = w;
            carry = __shfl_sync(0xFFFFFFFFu, w, 31);
        }
        if (lane == 0) {
            sm.bin = 0xFFFFFFFFu;
            sm.found = 0;
        }
    }
    __syncthreads();
    const float total = sm.prefix[n - 1];
    const float target = rs.u * total;
    for (int i = threadIdx.x; i < n; i += kFinThreads)
        if (sm.prefix[i] > target && (i == 0 || sm.prefix[i - 1] <= target)) sm.bin = (uint32_t)i;
    __syncthreads();
    const int chunk = (int)sm.bin;
    if (chunk < 0 || chunk >= n) return leave_row(a, t);
    constexpr int kVec = Elem<E>::kVec, kPer = Elem<E>::kChunk / kFinThreads;
    const int col0 = chunk * Elem<E>::kChunk + threadIdx.x * kPer;
    float z[kPer], sum = 0.f;
#pragma unroll
    for (int v = 0; v < kPer / kVec; ++v) {
        float x[kVec];
        load_columns(row, col0 + v * kVec, (int)a.V, x);
#pragma unroll
        for (int e = 0; e < kVec; ++e) z[v * kVec + e] = x[e];
    }
    float ex[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        ex[e] = ex2_approx((z[e] - M) * c);
        sum += ex[e];
    }
    float before, unused;
    block_scan<kFinThreads, float>(sm.scratch, sum, 0.f, before, unused);
    float c0 = (chunk ? sm.prefix[chunk - 1] : 0.f) + before;
    const float room = kSumError * total;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const float c1 = c0 + ex[e];
        if (target - c0 > room && c1 - target > room) {  // one column at most
            a.token[t] = col0 + e;
            a.logprob[t] = (z[e] - M) / rs.temp - lnS;
            sm.found = 1;
        }
        c0 = c1;
    }
    __syncthreads();
    if (!sm.found) leave_row(a, t);
}

template <typename E, bool kSample>
__global__ void __launch_bounds__(kFinThreads)
    filter_finish_kernel(const __grid_constant__ FilterArgs a) {
    __shared__ FinishShared sm;
    const int64_t t = blockIdx.x;
    const int V = (int)a.V, lane = threadIdx.x & 31;
    const E* row = static_cast<const E*>(a.logits) + t * a.ld;
    const float4* rec = a.records + t * a.chunks;
    const RowSettings rs = row_settings<kSample>(a, t);
    if (!rs.valid) {
        if (threadIdx.x == 0) write_undefined<kSample>(a, t, PSTAT_DEV_BAD_PARAM);
        return;
    }
    const TempScale c = temp_scale(rs.greedy ? 1.f : rs.temp);
    const float3 st = fold_records(rec, a.chunks, c.ch, lane);
    const float M = st.x + 0.f, Sf = st.y;
    if (!(M > -INFINITY)) {
        if (threadIdx.x == 0) write_undefined<kSample>(a, t, PSTAT_DEV_EMPTY_ROW);
        return;
    }
    if (rs.greedy) return finish_greedy(a, t, row, rec, M, sm);
    if (!rs.cut_k && !rs.cut_p && !rs.cut_m) {
        const float lnS = logf(Sf);
        if (kSample) return finish_draw(a, t, row, rec, M, c.ch, rs, lnS, sm);
        if (threadIdx.x == 0)
            write_statistics(a, t, row, M, lnS, lnS - kLn2 * (st.z / Sf), rs.temp, 0xFFFFFFFFu,
                             (uint32_t)V - 1);
        return;
    }

    // ---- which groups are read again
    const bool by_mass = rs.cut_p && !rs.cut_k;
    const int k = rs.cut_k ? (int)rs.top_k : 0;
    if (threadIdx.x < 64) sm.table[threadIdx.x] = a.table.v[threadIdx.x];
    if (threadIdx.x == 0) {
        sm.n_group = sm.n_cand = 0;
        sm.bin = kFinBins;
    }
    const float bin_scale = c.ch * ((float)kFinBins / 64.f);
    auto bin_of = [&](float z) { return min(kFinBins - 1, __float2int_rd((M - z) * bin_scale)); };
    const E* gm = static_cast<const E*>(a.group_max) + t * a.chunks * 32;
    const int groups = a.chunks * 32;
    const float z_min = min_p_logit(M, rs);
    const int bin_m = rs.cut_m ? bin_of(z_min) : kFinBins;
    if (rs.cut_k || rs.cut_p) {
        for (int i = threadIdx.x; i < kFinBins; i += kFinThreads) sm.hist.count[i] = sm.hist.mass[i] = 0;
        __syncthreads();
        constexpr float kUnit = 131072.f;  // 2^17: the maxima of all groups stay below 2^32
        for (int i = threadIdx.x; i < groups; i += kFinThreads) {
            const float g = Elem<E>::to_float(gm[i]);
            if (g == -INFINITY) continue;
            const int b = bin_of(g);
            atomicAdd(&sm.hist.count[b], 1u);
            if (by_mass) atomicAdd(&sm.hist.mass[b], (uint32_t)(ex2_approx((g - M) * c.ch) * kUnit));
        }
        __syncthreads();
        constexpr int kPer = kFinBins / kFinThreads;
        const int b0 = threadIdx.x * kPer;
        uint32_t nc = 0, nm = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            nc += sm.hist.count[b0 + i];
            nm += sm.hist.mass[b0 + i];
        }
        uint32_t cb, mb;
        block_scan<kFinThreads, uint32_t>(sm.scratch, nc, nm, cb, mb);
        const float need = rs.top_p * Sf * kUnit;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint32_t c1 = cb + sm.hist.count[b0 + i], m1 = mb + sm.hist.mass[b0 + i];
            if (by_mass ? ((float)mb < need && (float)m1 >= need)
                        : (cb < (uint32_t)k && (uint32_t)k <= c1))
                sm.bin = b0 + i;
            cb = c1;
            mb = m1;
        }
    }
    __syncthreads();
    int b = (int)sm.bin;
    // top-p after top-k needs the whole top-k mass, so min-p may not shorten it
    if (!(rs.cut_k && rs.cut_p)) b = min(b, bin_m);
    if (b >= kFinBins - 1) return leave_row(a, t);

    // ---- gather
    for (int i = threadIdx.x; i < groups; i += kFinThreads)
        if (bin_of(Elem<E>::to_float(gm[i])) <= b) {
            const uint32_t at = atomicAdd(&sm.n_group, 1u);
            if (at < (uint32_t)kFinGroups) sm.group[at] = (uint16_t)i;
        }
    __syncthreads();
    const int n_group = (int)sm.n_group;
    if (n_group > kFinGroups) return leave_row(a, t);
    {
        constexpr int kVec = Elem<E>::kVec;
        const int j = threadIdx.x & 15;
        for (int gi = threadIdx.x >> 4; gi < n_group; gi += kFinThreads / 16) {
            const int g = sm.group[gi];
            const int col = (g >> 5) * Elem<E>::kChunk + ((g & 31) + 32 * j) * kVec;
            float x[kVec];
            load_columns(row, col, V, x);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                if (x[e] > -INFINITY && bin_of(x[e]) <= b) {
                    const uint32_t at = atomicAdd(&sm.n_cand, 1u);
                    if (at < (uint32_t)kFinCand)
                        sm.cand[at] = ((unsigned long long)desc_key(x[e]) << 32) | (uint32_t)(col + e);
                }
            }
        }
    }
    __syncthreads();
    const int n = (int)sm.n_cand;
    if (n > kFinCand) return leave_row(a, t);
    sort_keys<kFinThreads>(sm.cand, n);

    // ---- inclusive sums of the exact weights, in order
    const int scale = fixed_scale(Sf * (1.f + 2.f * kSumError));
    constexpr int kPer = kFinCand / kFinThreads;
    {
        uint64_t w[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = threadIdx.x * kPer + i;
            w[i] = at < n ? fixed_weight(key_logit((uint32_t)(sm.cand[at] >> 32)), M, c, scale, sm.table)
                          : 0;
            sum += w[i];
        }
        uint64_t wb, unused;
        block_scan<kFinThreads, uint64_t>(sm.scratch, sum, 0, wb, unused);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            wb += w[i];
            if (threadIdx.x * kPer + i < n) sm.weight[threadIdx.x * kPer + i] = wb;
        }
    }
    __syncthreads();

    // ---- how many are kept; n + 1 where a filter keeps all of these or more
    auto first_mass = [&](double target) {  // first i with weight[i] >= target, n if none
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if ((double)sm.weight[mid] >= target)
                hi = mid;
            else
                lo = mid + 1;
        }
        return lo;
    };
    int keep = n + 1;
    if (rs.cut_m) {
        const uint32_t km = desc_key(z_min);
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if ((uint32_t)(sm.cand[mid] >> 32) > km)
                hi = mid;
            else
                lo = mid + 1;
        }
        if (lo < n || b >= bin_m) keep = lo;
    }
    if (rs.cut_p) {
        if (rs.cut_k) {
            if (n < k) return leave_row(a, t);
            keep = min(keep, min(k, 1 + first_mass((double)rs.top_p * (double)sm.weight[k - 1])));
        } else {
            const double one = (double)(1ull << scale);
            const double target = (double)rs.top_p * (double)Sf * one;
            const int i0 = first_mass(target * (1.0 - (double)kSumError));
            const int i1 = first_mass(target * (1.0 + (double)kSumError));
            if (keep > i0) {  // else min-p ends before the nucleus can
                if (i0 != i1 || i0 == n) return leave_row(a, t);
                keep = i0 + 1;
            }
        }
    } else if (rs.cut_k && n >= k) {
        keep = min(keep, k);
    }
    if (keep > n) return leave_row(a, t);

    const uint64_t S = sm.weight[keep - 1];
    const float lnS = fixed_log(S, scale);
    if (!kSample) {
        float ux = 0.f;
        for (int i = threadIdx.x; i < keep; i += kFinThreads) {
            const uint64_t w = sm.weight[i] - (i ? sm.weight[i - 1] : 0);
            const float x = (key_logit((uint32_t)(sm.cand[i] >> 32)) - M) / rs.temp;
            if (w) ux = fmaf((float)w * __int_as_float((127 - scale) << 23), x, ux);
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) ux += __shfl_xor_sync(0xFFFFFFFFu, ux, off);
        float* part = reinterpret_cast<float*>(sm.scratch);
        if (lane == 0) part[threadIdx.x >> 5] = ux;
        __syncthreads();
        if (threadIdx.x == 0) {
            float U = 0.f;
            for (int w = 0; w < kFinThreads / 32; ++w) U += part[w];
            const unsigned long long cut = sm.cand[keep - 1];
            const float Sr = (float)S * __int_as_float((127 - scale) << 23);
            write_statistics(a, t, row, M, lnS, lnS - U / Sr, rs.temp, (uint32_t)(cut >> 32),
                             (uint32_t)cut);
        }
        return;
    }
    // ---- draw: the kept columns in index order
    __syncthreads();
    for (int i = threadIdx.x; i < keep; i += kFinThreads)
        sm.cand[i] = (sm.cand[i] << 32) | (uint32_t)i;
    sort_keys<kFinThreads>(sm.cand, keep);
    const double target = (double)rs.u * (double)S;
    uint64_t w[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int at = threadIdx.x * kPer + i;
        w[i] = 0;
        if (at < keep) {
            const uint32_t from = (uint32_t)sm.cand[at];
            w[i] = sm.weight[from] - (from ? sm.weight[from - 1] : 0);
        }
        sum += w[i];
    }
    uint64_t wb, unused;
    block_scan<kFinThreads, uint64_t>(sm.scratch, sum, 0, wb, unused);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int at = threadIdx.x * kPer + i;
        const uint64_t w1 = wb + w[i];
        // u = 0 takes the first kept column, however small its weight
        if (at < keep && (rs.u == 0.f ? at == 0 : ((double)wb <= target && (double)w1 > target))) {
            const int col = (int)(sm.cand[at] >> 32);
            a.token[t] = col;
            a.logprob[t] = (Elem<E>::to_float(row[col]) - M) / rs.temp - lnS;
        }
        wb = w1;
    }
}

// ---------------------------------------------------------------------------
// Exact: clusters of CTAs over the rows that were left, passes with exact sums.
// ---------------------------------------------------------------------------
template <typename E, bool kSample>
__device__ void exact_row(const FilterArgs& a, int64_t t, Team<E>& tm, ExactShared& sm,
                          ExactShared& lead, cg::cluster_group& cluster) {
    const int V = (int)a.V, lane = threadIdx.x & 31;
    const bool first = tm.first;
    const E* row = tm.row;
    const RowSettings rs = row_settings<kSample>(a, t);
    tm.c = temp_scale(rs.temp);
    const float3 st = fold_records(a.records + t * a.chunks, a.chunks, tm.c.ch, lane);
    const float M = st.x + 0.f;
    tm.M = M;
    tm.bin_scale = tm.c.ch * ((float)kBins / 64.f);
    tm.k = fixed_scale(st.y * (1.f + 2.f * kSumError));
    if (threadIdx.x == 0) {
        sm.n_min = 0;
        sm.first = sm.first_kept = 0xFFFFFFFFu;
    }
    cluster.sync();

    const float z_min = min_p_logit(M, rs);
    uint32_t cut_key = 0xFFFFFFFFu, cut_index = (uint32_t)V - 1;
    if (rs.cut_k || rs.cut_p || (rs.cut_m && !kSample)) {
        tm.clear(sm.level0);
        uint32_t n_min = 0;
        tm.each([&](int, float z) {
            if (z == -INFINITY) return;
            const int b = tm.bin0(z);
            atomicAdd(&sm.level0.count[b], 1u);
            const uint64_t w = tm.weight(z);
            if (w) atomicAdd(&sm.level0.mass[b], (unsigned long long)w);
            n_min += z >= z_min;
        });
        n_min = __reduce_add_sync(0xFFFFFFFFu, n_min);
        if (lane == 0) atomicAdd(&lead.n_min, n_min);
        tm.merge(&ExactShared::level0);
        if (first) {
            uint64_t n = 0, w = 0, nb, wb;
            for (int i = threadIdx.x; i < kBins; i += kExThreads) {
                n += sm.level0.count[i];
                w += sm.level0.mass[i];
            }
            block_scan<kExThreads, uint64_t>(sm.scratch, n, w, nb, wb);
            if (threadIdx.x == kExThreads - 1) {
                sm.sel.rank = (uint32_t)(nb + n);
                sm.sel.mass = wb + w;
            }
        }
        cluster.sync();
        const uint32_t n_finite = lead.sel.rank;
        uint64_t total = lead.sel.mass;
        const uint32_t n_keep_min = rs.cut_m ? lead.n_min : n_finite;
        cluster.sync();
        uint32_t want = rs.cut_k && rs.top_k < (int64_t)n_finite ? (uint32_t)rs.top_k : n_finite;
        Selection sel;
        bool have = false;
        if (rs.cut_p) {
            if (want < n_finite) total = tm.select(true, want, 0.0).mass;
            cluster.sync();
            sel = tm.select(false, 0, (double)rs.top_p * (double)total);
            want = sel.rank;
            have = n_keep_min >= want;
            cluster.sync();
        }
        if (!have) {
            sel = tm.select(true, min(want, n_keep_min), 0.0);
            cluster.sync();
        }
        cut_key = sel.key;
        cut_index = sel.index;
    } else if (rs.cut_m) {
        cut_key = desc_key(z_min);
    }

    // Kept mass (and sum of e x) of every span of the index order.
    const int spans = (V + kSpan - 1) / kSpan;
    uint32_t lowest = 0xFFFFFFFFu;
    for (int s = tm.thread >> 5; s < spans; s += tm.threads >> 5) {
        uint64_t w = 0;
        float ux = 0.f;
        const int c1 = min(V, (s + 1) * kSpan);
        for (int col = s * kSpan + lane; col < c1; col += 32) {
            const float z = Elem<E>::to_float(row[col]);
            if (is_kept(z, col, cut_key, cut_index)) {
                const uint64_t e = tm.weight(z);
                w += e;
                if (z > -INFINITY) lowest = min(lowest, (uint32_t)col);
                if (!kSample && e)
                    ux = fmaf((float)e * __int_as_float((127 - tm.k) << 23), (z - M) / rs.temp, ux);
            }
        }
        w = warp_sum(w);
        if (!kSample) {
#pragma unroll
            for (int off = 16; off; off >>= 1) ux += __shfl_xor_sync(0xFFFFFFFFu, ux, off);
        }
        if (lane == 0) {
            lead.span_mass[s] = w;
            if (!kSample) lead.span_u[s] = ux;
        }
    }
    if (kSample && rs.u == 0.f) {
        lowest = __reduce_min_sync(0xFFFFFFFFu, lowest);
        if (lane == 0) atomicMin(&lead.first_kept, lowest);
    }
    cluster.sync();
    if (!first) return;

    const uint64_t mine = (int)threadIdx.x < spans ? sm.span_mass[threadIdx.x] : 0;
    uint64_t before, unused;
    block_scan<kExThreads, uint64_t>(sm.scratch, mine, 0, before, unused);
    if (threadIdx.x == kExThreads - 1) sm.mass_before = before + mine;
    __syncthreads();
    const uint64_t S = sm.mass_before;
    const float lnS = fixed_log(S, tm.k);
    if (!kSample) {
        if (threadIdx.x == 0) {
            float U = 0.f;
            for (int s = 0; s < spans; ++s) U += sm.span_u[s];
            const float Sr = (float)S * __int_as_float((127 - tm.k) << 23);
            write_statistics(a, t, row, M, lnS, lnS - U / Sr, rs.temp, cut_key, cut_index);
        }
        return;
    }
    if (rs.u == 0.f) {  // the first kept column, however small its weight
        if (threadIdx.x == 0) {
            const uint32_t col = sm.first_kept;
            a.token[t] = col;
            a.logprob[t] = (Elem<E>::to_float(row[col]) - M) / rs.temp - lnS;
        }
        return;
    }
    const double target = (double)rs.u * (double)S;
    __syncthreads();
    if ((double)before <= target && (double)(before + mine) > target) {
        sm.first = threadIdx.x;
        sm.mass_before = before;
    }
    __syncthreads();
    constexpr int kPer = kSpan / kExThreads;
    const int c0 = (int)sm.first * kSpan + threadIdx.x * kPer;
    const uint64_t base = sm.mass_before;
    uint64_t w[kPer], sum = 0;
    for (int i = 0; i < kPer; ++i) {
        w[i] = 0;
        if (c0 >= 0 && c0 + i < V) {
            const float z = Elem<E>::to_float(row[c0 + i]);
            if (is_kept(z, c0 + i, cut_key, cut_index)) w[i] = tm.weight(z);
        }
        sum += w[i];
    }
    uint64_t wb;
    block_scan<kExThreads, uint64_t>(sm.scratch, sum, 0, wb, unused);
    wb += base;
    for (int i = 0; i < kPer; ++i) {
        const uint64_t w1 = wb + w[i];
        if (w[i] && (double)wb <= target && (double)w1 > target) {
            a.token[t] = c0 + i;
            a.logprob[t] = (Elem<E>::to_float(row[c0 + i]) - M) / rs.temp - lnS;
        }
        wb = w1;
    }
}

template <typename E, bool kSample>
__global__ void __launch_bounds__(kExThreads)
    filter_exact_kernel(const __grid_constant__ FilterArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    cg::cluster_group cluster = cg::this_cluster();
    ExactShared& sm = *reinterpret_cast<ExactShared*>(smem_raw);
    ExactShared& lead = *cluster.map_shared_rank(&sm, 0);
    const int team = (int)cluster.num_blocks();
    const int n = *a.left_count;
    if (threadIdx.x < 64) sm.table[threadIdx.x] = a.table.v[threadIdx.x];
    __syncthreads();
    for (int i = blockIdx.x / team; i < n; i += gridDim.x / team) {
        const int64_t t = a.left[i];
        Team<E> tm{sm, lead, cluster, static_cast<const E*>(a.logits) + t * a.ld, (int)a.V,
                   (int)(cluster.block_rank() * kExThreads + threadIdx.x), team * kExThreads,
                   cluster.block_rank() == 0, 0.f, {0.f, 0.f}, 0, 0.f};
        exact_row<E, kSample>(a, t, tm, sm, lead, cluster);
        cluster.sync();  // the next row writes what this one reads
    }
}

template <typename E, bool kSample>
cudaError_t launch_filter(const FilterArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
    static ContextSeen records_set, exact_set;
    const void* rec_fn = reinterpret_cast<const void*>(filter_records_kernel<E, !kSample>);
    const void* ex_fn = reinterpret_cast<const void*>(filter_exact_kernel<E, kSample>);
    cudaError_t e = ensure_smem_optin(rec_fn, (int)chunk_stats_smem_bytes(), records_set);
    if (e == cudaSuccess) e = ensure_smem_optin(ex_fn, (int)sizeof(ExactShared), exact_set);
    if (e != cudaSuccess) return e;

    // Few items are spread over as many SMs as there are, one warp each at first.
    const int64_t items = a.T * a.chunks;
    int64_t warps = (items + dev.sm_count - 1) / dev.sm_count;
    warps = warps < kWarps ? warps : kWarps;
    int64_t grid = (items + warps - 1) / warps;
    grid = grid < dev.sm_count ? grid : dev.sm_count;
    filter_records_kernel<E, !kSample><<<(unsigned)grid, (unsigned)warps * 32,
                                         (size_t)warps * kStages * (kSlotBytes + sizeof(uint64_t)),
                                         stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    filter_finish_kernel<E, kSample><<<(unsigned)a.T, kFinThreads, 0, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;

    int team = 1;
    while (team < 8 && a.V >= (int64_t)team * 8192) team *= 2;
    int64_t teams = (int64_t)dev.sm_count * 3 / team;
    if (teams > a.T) teams = a.T;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(teams * team));
    cfg.blockDim = dim3(kExThreads);
    cfg.dynamicSmemBytes = sizeof(ExactShared);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)team;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, filter_exact_kernel<E, kSample>, a);
}

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
    // Column y is kept, so its gradient is g (1 - p_y).
    auto gradient = [&](float z, int64_t col) {
        const float e = ex2_approx((z - M) * c);
        const bool kept = z > tau || (z == tau && col <= last);
        return col == y ? fmaf(-g, e * K, g) : kept ? e * ngK : 0.f;
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

ExpTable make_table() {
    ExpTable t;
    for (int j = 0; j < 64; ++j) {
        const double v = std::exp2(-j / 64.0);
        t.v[j].x = (float)v;
        t.v[j].y = (float)(v - (double)t.v[j].x);
    }
    return t;
}
const ExpTable& exp_table() {
    static const ExpTable t = make_table();
    return t;
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct FilterWorkspace {
    size_t group_max, left_count, left, total;  // records first
};
FilterWorkspace filter_workspace(int64_t T, int64_t V, pstat_dtype dt) {
    const int64_t chunk = dt == PSTAT_BF16 ? PSTAT_CHUNK_BF16 : PSTAT_CHUNK_F32;
    const size_t items = (size_t)T * (size_t)((V + chunk - 1) / chunk);
    FilterWorkspace w;
    w.group_max = align_up(items * kChunkRecordBytes, 256);
    w.left_count = align_up(w.group_max + items * 32 * (dt == PSTAT_BF16 ? 2 : 4), 256);
    w.left = w.left_count + 16;
    w.total = align_up(w.left + (size_t)T * sizeof(int), 256);
    return w;
}

int check_filters(const void* logits, pstat_dtype dt, int64_t T, int64_t V, int64_t ld,
                  const pstat_filters* f, bool zero_temperature) {
    if (dt != PSTAT_F32 && dt != PSTAT_BF16) return PSTAT_ERR_DTYPE;
    if (T < 0 || V < 1 || ld < V || V > kFilterMaxV || T > PSTAT_FILTER_MAX_T) return PSTAT_ERR_SHAPE;
    if (!f) return PSTAT_ERR_NULLPTR;
    if (!f->temperatures && !((zero_temperature && f->temperature == 0.f) ||
                              (f->temperature >= kFilterTempMin && f->temperature <= kFilterTempMax)))
        return PSTAT_ERR_PARAM;
    if (!f->top_ps && !(f->top_p > 0.f && f->top_p <= 1.f)) return PSTAT_ERR_PARAM;
    if (!f->min_ps && !(f->min_p >= 0.f && f->min_p <= 1.f)) return PSTAT_ERR_PARAM;
    if (T == 0) return PSTAT_OK;
    if (!logits) return PSTAT_ERR_NULLPTR;
    if (!aligned(logits, dt == PSTAT_BF16 ? 2 : 4) || !aligned(f->temperatures, 4) ||
        !aligned(f->top_ks, 4) || !aligned(f->top_ps, 4) || !aligned(f->min_ps, 4))
        return PSTAT_ERR_ALIGN;
    return PSTAT_OK;
}

int check_workspace(const void* workspace, size_t bytes, int64_t T, int64_t V, pstat_dtype dt) {
    if (!workspace || bytes < filter_workspace(T, V, dt).total) return PSTAT_ERR_WORKSPACE;
    return aligned(workspace, 16) ? PSTAT_OK : PSTAT_ERR_ALIGN;
}

FilterArgs filter_args(const void* logits, pstat_dtype dt, int64_t T, int64_t V, int64_t ld,
                       const pstat_filters* f, void* workspace, int* dev_error) {
    FilterArgs a = {};
    const FilterWorkspace w = filter_workspace(T, V, dt);
    char* ws = static_cast<char*>(workspace);
    const int64_t chunk = dt == PSTAT_BF16 ? PSTAT_CHUNK_BF16 : PSTAT_CHUNK_F32;
    a.chunks = (int)((V + chunk - 1) / chunk);
    a.records = reinterpret_cast<float4*>(ws);
    a.group_max = ws + w.group_max;
    a.left_count = reinterpret_cast<int*>(ws + w.left_count);
    a.left = reinterpret_cast<int*>(ws + w.left);
    a.logits = logits;
    a.T = T;
    a.V = V;
    a.ld = ld;
    a.temperature = f->temperature;
    a.top_k = f->top_k;
    a.top_p = f->top_p;
    a.min_p = f->min_p;
    a.temperatures = f->temperatures;
    a.top_ks = f->top_ks;
    a.top_ps = f->top_ps;
    a.min_ps = f->min_ps;
    a.dev_error = dev_error;
    a.table = exp_table();
    return a;
}

}  // namespace
}  // namespace pstat

using namespace pstat;

extern "C" {

int pstat_filter_workspace_size(int64_t T, int64_t V, pstat_dtype dt, size_t* bytes) {
    if (!bytes) return PSTAT_ERR_NULLPTR;
    if (dt != PSTAT_F32 && dt != PSTAT_BF16) return PSTAT_ERR_DTYPE;
    if (T < 0 || V < 1 || V > kFilterMaxV || T > PSTAT_FILTER_MAX_T) return PSTAT_ERR_SHAPE;
    *bytes = filter_workspace(T, V, dt).total;
    return PSTAT_OK;
}

int pstat_sample(const void* logits, pstat_dtype dt, int64_t T, int64_t V, int64_t ld,
                 const float* uniform, const pstat_filters* filters, int64_t* out_token,
                 float* out_logprob, void* workspace, size_t ws_bytes, int* dev_error,
                 pstat_stream_t stream) {
    int rc = check_filters(logits, dt, T, V, ld, filters, true);
    if (rc != PSTAT_OK || T == 0) return rc;
    if (!uniform || !out_token || !out_logprob) return PSTAT_ERR_NULLPTR;
    if (!aligned(uniform, 4) || !aligned(out_token, 8) || !aligned(out_logprob, 4))
        return PSTAT_ERR_ALIGN;
    rc = check_workspace(workspace, ws_bytes, T, V, dt);
    if (rc != PSTAT_OK) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != PSTAT_OK) return rc;
    FilterArgs a = filter_args(logits, dt, T, V, ld, filters, workspace, dev_error);
    a.uniform = uniform;
    a.token = out_token;
    a.logprob = out_logprob;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dt == PSTAT_BF16 ? launch_filter<uint16_t, true>(a, dev, st)
                                           : launch_filter<float, true>(a, dev, st);
    return e == cudaSuccess ? PSTAT_OK : PSTAT_ERR_CUDA;
}

int pstat_filtered_forward(const void* logits, pstat_dtype dt, int64_t T, int64_t V, int64_t ld,
                           const int64_t* labels, int64_t ignore_index,
                           const pstat_filters* filters, float* out_logprob, float* out_entropy,
                           float* out_rowstats, float* out_cut_logit, int64_t* out_cut_index,
                           void* workspace, size_t ws_bytes, int* dev_error,
                           pstat_stream_t stream) {
    int rc = check_filters(logits, dt, T, V, ld, filters, false);
    if (rc != PSTAT_OK || T == 0) return rc;
    if (!out_logprob || !out_entropy || !out_rowstats || !out_cut_logit || !out_cut_index)
        return PSTAT_ERR_NULLPTR;
    if (!aligned(labels, 8) || !aligned(out_logprob, 4) || !aligned(out_entropy, 4) ||
        !aligned(out_rowstats, 8) || !aligned(out_cut_logit, 4) || !aligned(out_cut_index, 8))
        return PSTAT_ERR_ALIGN;
    rc = check_workspace(workspace, ws_bytes, T, V, dt);
    if (rc != PSTAT_OK) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != PSTAT_OK) return rc;
    FilterArgs a = filter_args(logits, dt, T, V, ld, filters, workspace, dev_error);
    a.labels = labels;
    a.ignore_index = ignore_index;
    a.logprob = out_logprob;
    a.entropy = out_entropy;
    a.rowstats = reinterpret_cast<float2*>(out_rowstats);
    a.cut_logit = out_cut_logit;
    a.cut_index = out_cut_index;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dt == PSTAT_BF16 ? launch_filter<uint16_t, false>(a, dev, st)
                                           : launch_filter<float, false>(a, dev, st);
    return e == cudaSuccess ? PSTAT_OK : PSTAT_ERR_CUDA;
}

int pstat_filtered_backward(const void* logits, pstat_dtype dt, int64_t T, int64_t V, int64_t ld,
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

}  // extern "C"
