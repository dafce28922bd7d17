// sampling.cu -- drawing a token per row and the policy statistics of given
// labels under the tempered, truncated softmax (filter_math.cuh has the
// definitions).
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

constexpr int kFinThreads = 512;
constexpr int kFinWarps = kFinThreads / 32;
constexpr int kBins = 2048;    // bins of one histogram level
constexpr int kCand = 2048;    // elements that are sorted at once
constexpr int kSpan = 4096;    // columns of one span of the index-order scan
constexpr int kMaxSpans = (int)(kFilterMaxV / kSpan);
static_assert(kBins % kFinThreads == 0 && kCand % kFinThreads == 0 && kSpan % kFinThreads == 0, "");

struct FilterArgs {
    const void* logits;
    int64_t T, V, ld;
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
    ExpTable table;
};

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

struct FinishShared {
    Histogram level0, level1;
    unsigned long long cand[kCand];
    unsigned long long span_mass[kMaxSpans];
    float span_u[kMaxSpans];
    float2 table[64];
    unsigned long long warp_a[kFinWarps];
    unsigned long long warp_b[kFinWarps];
    // Team results, in the first CTA of a cluster.
    uint32_t max_key;  // smallest descending key
    uint32_t bad;
    uint32_t n_min;
    uint32_t n_cand;
    uint32_t first;
    float sum;
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
__device__ __forceinline__ void block_scan(FinishShared& sm, uint64_t a, uint64_t b, uint64_t& a_ex,
                                           uint64_t& b_ex) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t sa = a, sb = b;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint64_t ta = __shfl_up_sync(0xFFFFFFFFu, sa, off);
        const uint64_t tb = __shfl_up_sync(0xFFFFFFFFu, sb, off);
        if (lane >= off) {
            sa += ta;
            sb += tb;
        }
    }
    if (lane == 31) {
        sm.warp_a[warp] = sa;
        sm.warp_b[warp] = sb;
    }
    __syncthreads();
    uint64_t oa = 0, ob = 0;
    for (int w = 0; w < warp; ++w) {
        oa += sm.warp_a[w];
        ob += sm.warp_b[w];
    }
    a_ex = oa + sa - a;
    b_ex = ob + sb - b;
    __syncthreads();
}

// Ascending bitonic sort of the first n candidates (n <= kCand).
__device__ __forceinline__ void sort_candidates(FinishShared& sm, int n) {
    int m = 2;
    while (m < n) m <<= 1;
    for (int i = n + threadIdx.x; i < m; i += kFinThreads) sm.cand[i] = ~0ull;
    __syncthreads();
    for (int size = 2; size <= m; size <<= 1) {
        for (int stride = size >> 1; stride; stride >>= 1) {
            for (int p = threadIdx.x; p < m / 2; p += kFinThreads) {
                const int i = 2 * p - (p & (stride - 1));
                const unsigned long long a = sm.cand[i], b = sm.cand[i + stride];
                if ((a > b) == ((i & size) == 0)) {
                    sm.cand[i] = b;
                    sm.cand[i + stride] = a;
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
    FinishShared& sm;        // this CTA's
    FinishShared& lead;      // the first CTA's
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
        for (int i = threadIdx.x; i < kBins; i += kFinThreads) {
            h.count[i] = 0;
            h.mass[i] = 0;
        }
        __syncthreads();
    }
    // Adds every CTA's histogram to the first one's.
    __device__ void merge(Histogram FinishShared::*which) {
        cluster.sync();
        if (!first) {
            Histogram& mine = sm.*which;
            Histogram& all = lead.*which;
            for (int i = threadIdx.x; i < kBins; i += kFinThreads) {
                if (mine.count[i]) atomicAdd(&all.count[i], mine.count[i]);
                if (mine.mass[i]) atomicAdd(&all.mass[i], mine.mass[i]);
            }
        }
        cluster.sync();
    }

    // First CTA: the bin in which the count reaches `want` (by_count) or the
    // mass reaches `target`; announces what lies before it and inside it.
    __device__ int pick_bin(const Histogram& h, bool by_count, uint32_t want, double target) {
        constexpr int kPer = kBins / kFinThreads;
        const int b0 = threadIdx.x * kPer;
        uint64_t n = 0, w = 0;
        for (int i = 0; i < kPer; ++i) {
            n += h.count[b0 + i];
            w += h.mass[b0 + i];
        }
        uint64_t nb, wb;
        block_scan(sm, n, w, nb, wb);
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
            merge(&FinishShared::level1);
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
        sort_candidates(sm, n);
        constexpr int kPer = kCand / kFinThreads;
        const int i0 = threadIdx.x * kPer;
        uint64_t w[kPer], sum = 0;
        for (int i = 0; i < kPer; ++i) {
            w[i] = i0 + i < n ? weight(key_logit((uint32_t)(sm.cand[i0 + i] >> 32))) : 0;
            sum += w[i];
        }
        uint64_t wb, unused;
        block_scan(sm, sum, 0, wb, unused);
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
        merge(&FinishShared::level1);
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
        block_scan(sm, mine, 0, nb, unused);
        if (nb < take && take <= nb + mine) {
            sm.first = threadIdx.x;
            sm.n_in = (uint32_t)nb;
        }
        __syncthreads();
        constexpr int kPer = kSpan / kFinThreads;
        const int c0 = (int)sm.first * kSpan + threadIdx.x * kPer;
        const uint64_t skipped = sm.n_in;
        uint32_t hit = 0;
        for (int i = 0; i < kPer; ++i)
            if (c0 >= 0 && c0 + i < V && desc_key(Elem<E>::to_float(row[c0 + i])) == key) hit |= 1u << i;
        block_scan(sm, __popc(hit), 0, nb, unused);
        nb += skipped;
        for (int i = 0; i < kPer; ++i) {
            if (!(hit >> i & 1u)) continue;
            if (++nb == take)
                sm.sel = {key, (uint32_t)(c0 + i), before + take, mass_before + (uint64_t)take * w};
        }
        __syncthreads();
    }
};

static_assert(kMaxSpans <= kFinThreads && kMaxSpans <= kBins, "one thread per span");

template <typename E, bool kSample>
__device__ void write_undefined(const FilterArgs& a, int64_t t, int err) {
    if (kSample) {
        a.token[t] = -1;
        a.logprob[t] = NAN;
    } else {
        a.logprob[t] = NAN;
        a.entropy[t] = NAN;
        a.rowstats[t] = make_float2(NAN, NAN);
        a.cut_logit[t] = NAN;
        a.cut_index[t] = -1;
    }
    if (a.dev_error) atomicOr(a.dev_error, err);
}

template <typename E, bool kSample>
__global__ void __launch_bounds__(kFinThreads)
    filter_rows_kernel(const __grid_constant__ FilterArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    cg::cluster_group cluster = cg::this_cluster();
    FinishShared& sm = *reinterpret_cast<FinishShared*>(smem_raw);
    FinishShared& lead = *cluster.map_shared_rank(&sm, 0);
    const int team = (int)cluster.num_blocks();
    const int64_t t = blockIdx.x / team;
    const int V = (int)a.V;
    const E* row = static_cast<const E*>(a.logits) + t * a.ld;
    const bool first = cluster.block_rank() == 0;

    const float temp = a.temperatures ? a.temperatures[t] : a.temperature;
    const float top_p = a.top_ps ? a.top_ps[t] : a.top_p;
    const float min_p = a.min_ps ? a.min_ps[t] : a.min_p;
    const int64_t top_k = a.top_ks ? a.top_ks[t] : a.top_k;
    const float u = kSample ? a.uniform[t] : 0.f;
    const bool greedy = kSample && temp == 0.f;
    const bool valid = (greedy || (temp >= kFilterTempMin && temp <= kFilterTempMax)) &&
                       (top_p > 0.f && top_p <= 1.f) && (min_p >= 0.f && min_p <= 1.f) &&
                       (u >= 0.f && u < 1.f);
    if (!valid) {  // the same answer in every thread of the team
        if (first && threadIdx.x == 0) write_undefined<E, kSample>(a, t, PSTAT_DEV_BAD_PARAM);
        return;
    }
    if (threadIdx.x < 64) sm.table[threadIdx.x] = a.table.v[threadIdx.x];
    if (threadIdx.x == 0) {
        sm.max_key = 0xFFFFFFFFu;
        sm.bad = 0;
        sm.n_min = 0;
        sm.first = 0xFFFFFFFFu;
        sm.sum = 0.f;
    }
    cluster.sync();
    Team<E> tm{sm, lead, cluster, row, V,
               (int)(cluster.block_rank() * kFinThreads + threadIdx.x), team * kFinThreads, first,
               0.f, {0.f, 0.f}, 0, 0.f};

    // Maximum; NaN and +inf leave the row without a distribution.
    {
        uint32_t best = 0xFFFFFFFFu;
        bool bad = false;
        tm.each([&](int, float z) {
            bad |= !(z < INFINITY);
            best = min(best, desc_key(z));
        });
        best = __reduce_min_sync(0xFFFFFFFFu, best);
        const bool any = __any_sync(0xFFFFFFFFu, bad);
        if ((threadIdx.x & 31) == 0) {
            atomicMin(&lead.max_key, best);
            if (any) atomicOr(&lead.bad, 1u);
        }
    }
    cluster.sync();
    const uint32_t key_max = lead.max_key;
    if (lead.bad || key_max >= kKeyNegInf) {
        if (first && threadIdx.x == 0) write_undefined<E, kSample>(a, t, PSTAT_DEV_EMPTY_ROW);
        cluster.sync();  // the first CTA's shared memory stays until all have read it
        return;
    }
    const float M = key_logit(key_max);
    if (greedy) {
        uint32_t at = 0xFFFFFFFFu;
        tm.each([&](int col, float z) {
            if (z == M) at = min(at, (uint32_t)col);
        });
        at = __reduce_min_sync(0xFFFFFFFFu, at);
        if ((threadIdx.x & 31) == 0 && at != 0xFFFFFFFFu) atomicMin(&lead.first, at);
        cluster.sync();
        if (first && threadIdx.x == 0) {
            a.token[t] = sm.first;
            a.logprob[t] = 0.f;
        }
        return;
    }
    tm.M = M;
    tm.c = temp_scale(temp);
    tm.bin_scale = tm.c.ch * ((float)kBins / 64.f);
    // Any V weights of at most 1 sum to at most V.
    tm.k = fixed_scale((float)V);

    const bool cut_k = top_k > 0 && top_k < V;
    const bool cut_p = top_p < 1.f;
    const bool cut_m = min_p > 0.f;
    // x >= ln(min_p)  <=>  z >= M + t ln(min_p), rounded up to a float.
    const float z_min =
        cut_m ? __double2float_ru((double)M + (double)temp * log((double)min_p)) : -INFINITY;
    uint32_t cut_key = 0xFFFFFFFFu, cut_index = (uint32_t)V - 1;
    if (cut_k || cut_p || (cut_m && !kSample)) {
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
        if ((threadIdx.x & 31) == 0) atomicAdd(&lead.n_min, n_min);
        tm.merge(&FinishShared::level0);
        if (first) {
            uint64_t n = 0, w = 0, nb, wb;
            for (int i = threadIdx.x; i < kBins; i += kFinThreads) {
                n += sm.level0.count[i];
                w += sm.level0.mass[i];
            }
            block_scan(sm, n, w, nb, wb);
            if (threadIdx.x == kFinThreads - 1) {
                sm.sel.rank = (uint32_t)(nb + n);
                sm.sel.mass = wb + w;
            }
        }
        cluster.sync();
        const uint32_t n_finite = lead.sel.rank;
        uint64_t total = lead.sel.mass;
        const uint32_t n_keep_min = cut_m ? lead.n_min : n_finite;
        cluster.sync();
        uint32_t want = cut_k && top_k < (int64_t)n_finite ? (uint32_t)top_k : n_finite;
        Selection sel;
        bool have = false;
        if (cut_p) {
            if (want < n_finite) total = tm.select(true, want, 0.0).mass;
            cluster.sync();
            sel = tm.select(false, 0, (double)top_p * (double)total);
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
    } else if (cut_m) {
        cut_key = desc_key(z_min);
    }

    // Kept mass (and sum of e x) of every span of the index order.
    const int spans = (V + kSpan - 1) / kSpan;
    const int lane = threadIdx.x & 31;
    for (int s = tm.thread >> 5; s < spans; s += tm.threads >> 5) {
        uint64_t w = 0;
        float ux = 0.f;
        const int c1 = min(V, (s + 1) * kSpan);
        for (int col = s * kSpan + lane; col < c1; col += 32) {
            const float z = Elem<E>::to_float(row[col]);
            const uint32_t dk = desc_key(z);
            if (dk < cut_key || (dk == cut_key && (uint32_t)col <= cut_index)) {
                const uint64_t e = tm.weight(z);
                w += e;
                if (!kSample && e) {
                    const float x = (z - M) / temp;
                    ux = fmaf((float)e * __int_as_float((127 - tm.k) << 23), x, ux);
                }
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
    cluster.sync();
    if (!first) return;

    const uint64_t mine = (int)threadIdx.x < spans ? sm.span_mass[threadIdx.x] : 0;
    uint64_t before, unused;
    block_scan(sm, mine, 0, before, unused);
    if (threadIdx.x == kFinThreads - 1) sm.mass_before = before + mine;
    __syncthreads();
    const uint64_t S = sm.mass_before;
    const float lnS = fixed_log(S, tm.k);
    if (kSample) {
        const double target = (double)u * (double)S;
        __syncthreads();
        if ((double)before <= target && (double)(before + mine) > target) {
            sm.first = threadIdx.x;
            sm.mass_before = before;
        }
        __syncthreads();
        constexpr int kPer = kSpan / kFinThreads;
        const int c0 = (int)sm.first * kSpan + threadIdx.x * kPer;
        const uint64_t base = sm.mass_before;
        uint64_t w[kPer], sum = 0;
        for (int i = 0; i < kPer; ++i) {
            w[i] = 0;
            if (c0 >= 0 && c0 + i < V) {
                const float z = Elem<E>::to_float(row[c0 + i]);
                const uint32_t dk = desc_key(z);
                if (dk < cut_key || (dk == cut_key && (uint32_t)(c0 + i) <= cut_index))
                    w[i] = tm.weight(z);
            }
            sum += w[i];
        }
        uint64_t wb;
        block_scan(sm, sum, 0, wb, unused);
        wb += base;
        for (int i = 0; i < kPer; ++i) {
            const uint64_t w1 = wb + w[i];
            if (w[i] && (double)wb <= target && (double)w1 > target) {
                a.token[t] = c0 + i;
                a.logprob[t] = (Elem<E>::to_float(row[c0 + i]) - M) / temp - lnS;
            }
            wb = w1;
        }
    } else if (threadIdx.x == 0) {
        float U = 0.f;
        for (int s = 0; s < spans; ++s) U += sm.span_u[s];
        int err = 0;
        const float inv = __int_as_float((127 - tm.k) << 23);
        float H = lnS - U / ((float)S * inv), lp;
        const int64_t y = a.labels ? a.labels[t] : a.ignore_index;
        if (y == a.ignore_index) {
            lp = 0.f;
        } else if (y < 0 || y >= a.V) {
            lp = H = NAN;
            err = PSTAT_DEV_BAD_LABEL;
        } else {
            const float z = Elem<E>::to_float(row[y]);
            const uint32_t dk = desc_key(z);
            const bool kept = dk < cut_key || (dk == cut_key && (uint32_t)y <= cut_index);
            lp = kept ? (z - M) / temp - lnS : -INFINITY;
        }
        a.logprob[t] = lp;
        a.entropy[t] = H;
        a.rowstats[t] = make_float2(M, lnS);
        const bool all = cut_key == 0xFFFFFFFFu;
        a.cut_logit[t] = all ? -INFINITY : key_logit(cut_key);
        a.cut_index[t] = (int64_t)cut_index;
        if (err && a.dev_error) atomicOr(a.dev_error, err);
    }
}

template <typename E, bool kSample>
cudaError_t launch_filter(const FilterArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
    static ContextSeen configured;
    const void* fn = reinterpret_cast<const void*>(filter_rows_kernel<E, kSample>);
    const cudaError_t e = ensure_smem_optin(fn, (int)sizeof(FinishShared), configured);
    if (e != cudaSuccess) return e;
    int team = 1;
    while (team < 8 && a.T * team * 2 <= dev.sm_count && a.V >= (int64_t)team * 8192) team *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.T * team));
    cfg.blockDim = dim3(kFinThreads);
    cfg.dynamicSmemBytes = sizeof(FinishShared);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)team;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, filter_rows_kernel<E, kSample>, a);
}

// ---------------------------------------------------------------------------
// Gradient: dz_v = (w/t)(1[v = y] - kept_v e_v/S), elementwise.
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
    const int64_t c0 = V * seg / segs, c1 = V * (seg + 1) / segs;
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
    float c = 0.f, off = 0.f, g = 0.f;
    if (mode == 2) {
        c = kLog2e / temp;
        off = rs.y * kLog2e;
        g = w / temp;
    }
    const float fill = mode == 0 ? 0.f : NAN;
    for (int64_t col = c0 + threadIdx.x; col < c1; col += kFgThreads) {
        float v = fill;
        if (mode == 2) {
            const float z = Elem<Ein>::to_float(zin[col]);
            const bool kept = z > tau || (z == tau && col <= last);
            const float p = kept ? exp2f(fmaf(z - rs.x, c, -off)) : 0.f;
            v = col == y ? g * (1.f - p) : -(g * p);
            if (!kept) v = 0.f;
        }
        zout[col] = out_cast(v, zout);
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

FilterArgs filter_args(const void* logits, int64_t T, int64_t V, int64_t ld,
                       const pstat_filters* f, int* dev_error) {
    FilterArgs a = {};
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
    *bytes = 0;
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
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != PSTAT_OK) return rc;
    FilterArgs a = filter_args(logits, T, V, ld, filters, dev_error);
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
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != PSTAT_OK) return rc;
    FilterArgs a = filter_args(logits, T, V, ld, filters, dev_error);
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
