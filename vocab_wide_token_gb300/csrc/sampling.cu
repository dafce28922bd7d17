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
#include <type_traits>

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
constexpr int kSpan = 256;     // columns of one span of the index-order scan, a warp's
constexpr int kMaxSpans = (int)(kFilterMaxV / kSpan);
constexpr int kSpansPer = kMaxSpans / kExThreads;
static_assert(kBins % kExThreads == 0 && kMaxSpans % kExThreads == 0 && kSpan <= kExThreads, "");
constexpr int kMaxTeam = 16;

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
    grid_launch_dependents();

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

struct Histogram {
    uint32_t count[kBins];
    unsigned long long mass[kBins];
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

// Reads N times kVec columns from col[h] (multiples of kVec) of a row, all loads
// before the first use; columns past V read as -inf.
template <typename E, int N>
__device__ __forceinline__ void load_columns(const E* row, const int (&col)[N], int V,
                                             float (&x)[N][Elem<E>::kVec]) {
    constexpr int kVec = Elem<E>::kVec;
    if ((reinterpret_cast<uintptr_t>(row) & 15u) == 0) {
        uint4 q[N];
#pragma unroll
        for (int h = 0; h < N; ++h)
            q[h] = col[h] + kVec <= V ? __ldg(reinterpret_cast<const uint4*>(row + col[h]))
                                      : Elem<E>::neg_inf_vec();
#pragma unroll
        for (int h = 0; h < N; ++h) RowReader<E>::unpack(q[h], x[h]);
#pragma unroll
        for (int h = 0; h < N; ++h)
            if (col[h] < V && col[h] + kVec > V)  // the row's last, partial vector
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (col[h] + e < V) x[h][e] = Elem<E>::to_float(row[col[h] + e]);
    } else {
#pragma unroll
        for (int h = 0; h < N; ++h)
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                x[h][e] = col[h] + e < V ? Elem<E>::to_float(row[col[h] + e]) : -INFINITY;
    }
}

// *p += v in shared memory.  64-bit adds there are compare-and-swap loops, which
// crawl when lanes meet on one address; two 32-bit adds with the carry between
// them are not (nobody reads the sum before the next barrier).
__device__ __forceinline__ void add_wide(unsigned long long* p, uint64_t v) {
    uint32_t* half = reinterpret_cast<uint32_t*>(p);
    const uint32_t lo = (uint32_t)v, hi = (uint32_t)(v >> 32);
    const uint32_t old = atomicAdd(half, lo);
    const uint32_t carry = old + lo < old;
    if (hi + carry) atomicAdd(half + 1, hi + carry);
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
    // every warp scans the warps' totals, in the same order
    constexpr int kW = kThreads / 32;
    T ta = lane < kW ? wa[lane] : T(0), tb = lane < kW ? wb[lane] : T(0);
#pragma unroll
    for (int off = 1; off < kW; off <<= 1) {
        const T ua = __shfl_up_sync(0xFFFFFFFFu, ta, off);
        const T ub = __shfl_up_sync(0xFFFFFFFFu, tb, off);
        if (lane >= off) {
            ta += ua;
            tb += ub;
        }
    }
    const int prior = warp ? warp - 1 : 0;
    T oa = __shfl_sync(0xFFFFFFFFu, ta, prior), ob = __shfl_sync(0xFFFFFFFFu, tb, prior);
    if (warp == 0) oa = ob = T(0);
    // exclusive sum of the lanes, without taking a back out of a sum
    T pa = __shfl_up_sync(0xFFFFFFFFu, sa, 1), pb = __shfl_up_sync(0xFFFFFFFFu, sb, 1);
    a_ex = lane ? oa + pa : oa;
    b_ex = lane ? ob + pb : ob;
    __syncthreads();
}

// ---------------------------------------------------------------------------
// Selection in a list of (key, weight) in shared memory, by one CTA.
//
// The list is ordered by its keys (descending logit in the high word, column
// in the low one), or by the columns alone.  Among the keys in [kmin, kmax]
// this finds the one at which the count reaches `want`, or the mass `target`:
// histograms of the high word (or the column) narrow the range until few keys
// are left, or all that are left have one high word (then the columns are
// narrowed); each of those counts what lies before it.  Linear in the list,
// where sorting 2048 keys costs a block 66 synchronised steps.
// ---------------------------------------------------------------------------
struct Selected {
    unsigned long long key;
    uint32_t rank;  // 1-based
    uint64_t mass;  // up to and including it
};

constexpr int kListMembers = 128;
template <int kThreads>
struct ListShared {
    static constexpr int kBins = 1024;
    uint32_t count[kBins];
    unsigned long long mass[kBins];
    uint16_t member[kListMembers];
    uint32_t lo, n_in, n_member, count_before;
    unsigned long long mass_before;
    unsigned long long scratch[2 * (kThreads / 32)];
    Selected found;
};

template <int kThreads>
__device__ __noinline__ Selected list_select(ListShared<kThreads>& ls,
                                             const unsigned long long* keys,
                                             const unsigned long long* weights, int n,
                                             unsigned long long kmin, unsigned long long kmax,
                                             bool by_column, bool by_count, uint32_t want,
                                             uint64_t target, uint32_t count_before,
                                             uint64_t mass_before) {
    constexpr int kPer = ListShared<kThreads>::kBins / kThreads;
    uint32_t lo = by_column ? 0u : (uint32_t)(kmin >> 32);
    uint32_t hi = by_column ? (uint32_t)kFilterMaxV - 1 : (uint32_t)(kmax >> 32);
    uint32_t n_in = (uint32_t)n;  // keys in the range, at most
    auto inside = [&](unsigned long long key, uint32_t& p) {
        p = by_column ? (uint32_t)key : (uint32_t)(key >> 32);
        return key >= kmin && key <= kmax && p >= lo && p <= hi;
    };
    while (n_in > (uint32_t)kListMembers) {
        if (lo == hi) {  // equal logits: by their columns from here on
            if (!by_count) {
                for (int i = threadIdx.x; i < n; i += kThreads)
                    if ((uint32_t)(keys[i] >> 32) == lo) ls.mass[0] = weights[i];  // all alike
                __syncthreads();
                const uint64_t w = ls.mass[0];
                const uint64_t short_of = target - mass_before;
                want = count_before + (uint32_t)(w ? (short_of + w - 1) / w : n_in);
                by_count = true;
                __syncthreads();
            }
            kmin = kmin > ((unsigned long long)lo << 32) ? kmin : (unsigned long long)lo << 32;
            kmax = kmax < ((unsigned long long)lo << 32 | 0xFFFFFFFFu)
                       ? kmax
                       : ((unsigned long long)lo << 32 | 0xFFFFFFFFu);
            by_column = true;
            lo = 0;
            hi = (uint32_t)kFilterMaxV - 1;
        }
        int shift = 0;
        while (((hi - lo) >> shift) >= (uint32_t)ListShared<kThreads>::kBins) ++shift;
        for (int i = threadIdx.x; i < ListShared<kThreads>::kBins; i += kThreads)
            ls.count[i] = 0, ls.mass[i] = 0;
        if (threadIdx.x == 0) ls.n_in = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kThreads) {
            uint32_t p;
            if (inside(keys[i], p)) {
                atomicAdd(&ls.count[(p - lo) >> shift], 1u);
                if (weights[i]) add_wide(&ls.mass[(p - lo) >> shift], weights[i]);
            }
        }
        __syncthreads();
        const int b0 = threadIdx.x * kPer;
        uint64_t nc = 0, nm = 0;
        for (int i = 0; i < kPer; ++i) {
            nc += ls.count[b0 + i];
            nm += ls.mass[b0 + i];
        }
        uint64_t nb, wb;
        block_scan<kThreads, uint64_t>(ls.scratch, nc, nm, nb, wb);
        nb += count_before;
        wb += mass_before;
        for (int i = 0; i < kPer; ++i) {
            const uint64_t n1 = nb + ls.count[b0 + i], w1 = wb + ls.mass[b0 + i];
            if (by_count ? (nb < want && want <= n1) : (wb < target && w1 >= target)) {
                ls.lo = lo + ((uint32_t)(b0 + i) << shift);
                ls.n_in = ls.count[b0 + i];
                ls.count_before = (uint32_t)nb;
                ls.mass_before = wb;
            }
            nb = n1;
            wb = w1;
        }
        __syncthreads();
        if (ls.n_in == 0) break;  // nothing reaches it: the caller asked for too much
        lo = ls.lo;
        hi = min(hi, lo + ((1u << shift) - 1u));
        n_in = ls.n_in;
        count_before = ls.count_before;
        mass_before = ls.mass_before;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        ls.n_member = 0;
        ls.found = {~0ull, 0u, 0};
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        uint32_t p;
        if (inside(keys[i], p)) {
            const uint32_t at = atomicAdd(&ls.n_member, 1u);
            if (at < (uint32_t)kListMembers) ls.member[at] = (uint16_t)i;
        }
    }
    __syncthreads();
    // Two (four, in a CTA of 512) neighbouring lanes share a member.
    constexpr int kParts = kThreads / kListMembers;
    const int m = min((int)ls.n_member, kListMembers);
    const int item = (int)threadIdx.x / kParts;
    if ((int)(threadIdx.x & ~31u) / kParts < m) {
        const int me = ls.member[min(item, m - 1)];
        const unsigned long long mine = keys[me];
        uint32_t less = 0;
        uint64_t before = 0;
#pragma unroll 4
        for (int j = (int)threadIdx.x % kParts; j < m; j += kParts) {
            const int o = ls.member[j];
            const bool yes = by_column ? (uint32_t)keys[o] < (uint32_t)mine : keys[o] < mine;
            less += yes;
            before += yes ? weights[o] : 0;
        }
#pragma unroll
        for (int off = 1; off < kParts; off <<= 1) {
            less += __shfl_xor_sync(0xFFFFFFFFu, less, off);
            before += __shfl_xor_sync(0xFFFFFFFFu, before, off);
        }
        const uint32_t rank = count_before + less + 1;
        before += mass_before;
        const uint64_t after = before + weights[me];
        if (item < m && threadIdx.x % kParts == 0 &&
            (by_count ? rank == want : (before < target && after >= target)))
            ls.found = {mine, rank, after};
    }
    __syncthreads();
    const Selected found = ls.found;
    __syncthreads();
    return found;
}

// e x in units of 2^-44, x in fp32: every term is at most 1/e, so that they add
// up as integers, in any order.
__device__ __forceinline__ long long entropy_term(unsigned long long key, uint64_t w, float M,
                                                  float temp, int scale) {
    const float x = (key_logit((uint32_t)(key >> 32)) - M) / temp;
    const float e = (float)w * __int_as_float((127 - scale) << 23);
    return w ? __float2ll_rn(e * x * 1.7592186e13f) : 0;
}

// C >= p S in whole numbers; at least 1, so that a token is kept.
__device__ __forceinline__ uint64_t share_of(float p, uint64_t S) {
    const uint64_t target = __double2ull_ru((double)p * (double)S);
    return target ? target : 1;
}

struct ExactShared {
    uint32_t level0[kBins];
    Histogram level1;
    unsigned long long cand[kCand];
    unsigned long long weight[kCand];
    unsigned long long span_mass[kMaxSpans];
    float2 table[64];
    unsigned long long scratch[2 * kExWarps];
    ListShared<kExThreads> list;
    // Team results, in the first CTA of a cluster.
    unsigned long long part[kMaxTeam][4];
    unsigned long long sums[3][kExWarps];
    uint32_t n_cand;
    uint32_t first;
    uint32_t first_kept;
    // Decisions that the first CTA announces.
    uint32_t klo, khi, n_in, count_before, bin;
    unsigned long long mass_before, mass_in, total, offset, ux;
    Selected sel;
};

// One row, worked on by a team of CTAs: those of a cluster, or one CTA alone.
// Passes over the row are shared out over all of them, decisions are taken in
// the first.
template <typename E>
struct Team {
    ExactShared& sm;         // this CTA's
    ExactShared& lead;       // the first CTA's
    cg::cluster_group cluster;
    const E* row;
    int V;
    int thread, threads;     // of the team
    bool first, alone;
    bool entropy;            // the entropy's sum is wanted
    float M, temp;
    TempScale c;
    int k;                   // digits of the fixed weights
    float bin_scale;
    bool ties;               // the last selection ended among too many equal logits

    __device__ void sync() {
        if (alone)
            __syncthreads();
        else
            cluster.sync();
    }
    // f(span, this lane's first column of it, its logits): a warp goes through a
    // span of kSpan columns together, kVec neighbouring ones (twice, in fp32) to a
    // lane; columns past V are -inf.
    static constexpr int kLane = kSpan / 32;
    template <typename F>
    __device__ __forceinline__ void each_span(F f) const {
        constexpr int kVec = Elem<E>::kVec, kVecs = kLane / kVec;
        const int lane = thread & 31, warps = threads >> 5;
        for (int s = thread >> 5; s * kSpan < V; s += warps) {
            int col[kVecs];
            float part[kVecs][kVec], x[kLane];
#pragma unroll
            for (int h = 0; h < kVecs; ++h) col[h] = s * kSpan + lane * kLane + h * kVec;
            load_columns<E, kVecs>(row, col, V, part);
#pragma unroll
            for (int h = 0; h < kVecs; ++h)
#pragma unroll
                for (int e = 0; e < kVec; ++e) x[h * kVec + e] = part[h][e];
            f(s, col[0], x);
        }
    }
    __device__ uint64_t weight(float z) const { return fixed_weight(z, M, c, k, sm.table); }
    // Level-0 bins: equal steps of M - z, the last one open (the difference
    // and the product round monotonely, so bins are ranges of the order).
    __device__ int bin0(float z) const { return min(kBins - 1, __float2int_rd((M - z) * bin_scale)); }

    // Sums over the team of two or three values per thread: put() everywhere,
    // sync(), then get() in any CTA, by a whole warp.  The fourth slot is for
    // the candidates' number.
    template <int N>
    __device__ void put(const uint64_t (&v)[N]) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint64_t w = warp_sum(v[i]);
            if ((threadIdx.x & 31) == 0) sm.sums[i][threadIdx.x >> 5] = w;
        }
        __syncthreads();
        const int i = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (i < N) {
            const uint64_t all = warp_sum(lane < kExWarps ? sm.sums[i][lane] : 0);
            if (lane == 0) lead.part[thread / kExThreads][i] = all;
        }
    }
    __device__ uint64_t get(int which) const {
        const int lane = threadIdx.x & 31;
        return warp_sum(lane < threads / kExThreads ? lead.part[lane][which] : 0);
    }
    __device__ void clear(Histogram& h) const {
        for (int i = threadIdx.x; i < kBins; i += kExThreads) {
            h.count[i] = 0;
            h.mass[i] = 0;
        }
        __syncthreads();
    }
    // Adds every CTA's histogram (masses optional) to the first one's.
    __device__ void merge(const uint32_t* count, uint32_t* all_count,
                          const unsigned long long* mass = nullptr,
                          unsigned long long* all_mass = nullptr) {
        sync();
        if (!first)
            for (int i = threadIdx.x; i < kBins; i += kExThreads) {
                if (count[i]) atomicAdd(&all_count[i], count[i]);
                if (mass && mass[i]) add_wide(&all_mass[i], mass[i]);
            }
        sync();
    }

    // First CTA: the bin in which the count reaches `want` (by_count) or the
    // mass `target`; announces the count and mass before it and the count inside.
    __device__ int pick_bin(const uint32_t* count, const unsigned long long* mass, bool by_count,
                            uint32_t want, uint64_t target) {
        constexpr int kPer = kBins / kExThreads;
        const int b0 = threadIdx.x * kPer;
        uint64_t n = 0, w = 0;
        for (int i = 0; i < kPer; ++i) {
            n += count[b0 + i];
            w += mass ? mass[b0 + i] : 0;
        }
        uint64_t nb, wb;
        block_scan<kExThreads, uint64_t>(sm.scratch, n, w, nb, wb);
        nb += sm.count_before;
        wb += sm.mass_before;
        __syncthreads();
        for (int i = 0; i < kPer; ++i) {
            const uint64_t n1 = nb + count[b0 + i], w1 = wb + (mass ? mass[b0 + i] : 0);
            if (by_count ? (nb < want && want <= n1) : (wb < target && w1 >= target)) {
                sm.count_before = (uint32_t)nb;
                sm.mass_before = wb;
                sm.n_in = count[b0 + i];
                sm.first = b0 + i;
            }
            nb = n1;
            wb = w1;
        }
        __syncthreads();
        return (int)sm.first;
    }

    // First CTA: the last of the level-0 bins [lo, hi] before which the
    // estimated mass is below `target`.  A bin's mass is estimated by its count
    // times the weight of its middle (steps of 1/32 of a binary order: 1.1% of
    // it at most); `anchor`, if not negative, is a bin before which the mass is
    // known.  Announces the bin and its counts.
    __device__ int guess_bin(uint64_t target, int lo, int hi, int anchor, uint64_t known) {
        constexpr int kPer = kBins / kExThreads;
        const int b0 = threadIdx.x * kPer;
        const float one = __int_as_float((127 + k) << 23);
        uint64_t n = 0, w = 0, part[kPer];
        for (int i = 0; i < kPer; ++i) {
            n += sm.level0[b0 + i];
            const float mid = exp2f(-((float)(b0 + i) + 0.5f) * (64.f / kBins));
            part[i] = (uint64_t)((float)sm.level0[b0 + i] * mid * one);
            w += part[i];
        }
        uint64_t nb, wb;
        block_scan<kExThreads, uint64_t>(sm.scratch, n, w, nb, wb);
        if (threadIdx.x == 0) sm.first = (uint32_t)lo;
        uint64_t at = wb;
        for (int i = 0; i < kPer; ++i) {
            if (b0 + i == anchor) sm.offset = known - at;  // modulo 2^64
            at += part[i];
        }
        if (threadIdx.x == 0 && anchor < 0) sm.offset = 0;
        __syncthreads();
        at = wb + sm.offset;
        for (int i = 0; i < kPer; ++i) {
            if (b0 + i > lo && b0 + i <= hi && (int64_t)(at - target) < 0 && sm.level0[b0 + i])
                atomicMax(&sm.first, (uint32_t)(b0 + i));
            at += part[i];
        }
        __syncthreads();
        const int b = (int)sm.first;
        uint64_t before = nb;
        for (int i = 0; i < kPer; ++i) {
            if (b0 + i == b) {
                sm.count_before = (uint32_t)before;
                sm.n_in = sm.level0[b0 + i];
            }
            before += sm.level0[b0 + i];
        }
        __syncthreads();
        return b;
    }

    // First CTA: the keys of level-0 bin b.
    __device__ void bin_range(int b) {
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

    // One pass: the exact masses before and inside the keys [klo, khi], what lies
    // before by spans of the index order, and the elements inside, as far as
    // they fit; with `all` the mass of the whole row as well.
    __device__ __noinline__ void weigh_and_gather(uint32_t klo, uint32_t khi, bool all) {
        // Candidates are collected in each CTA and then moved to the first.
        if (threadIdx.x == 0) sm.n_cand = 0;
        __syncthreads();
        uint64_t outside = 0, inside = 0, ux = 0;
        // in registers: this function writes memory that could be *this
        const float M = this->M, temp = this->temp;
        const TempScale c = this->c;
        const int k = this->k;
        const bool entropy = this->entropy;
        const E* const row = this->row;
        ExactShared& lead = this->lead;
        const float2* const table = sm.table;
        auto weight = [&](float z) { return fixed_weight(z, M, c, k, table); };
        auto weights = [&](float z0, float z1, uint64_t& w0, uint64_t& w1) {
            fixed_weights(z0, z1, M, c, k, table, w0, w1);
        };
        each_span([&](int s, int col, const float (&x)[kLane]) {
            bool any = all;
#pragma unroll
            for (int e = 0; e < kLane; ++e) any |= desc_key(x[e]) <= khi;
            uint64_t before = 0;
            uint32_t hits = 0;
            if (__any_sync(0xFFFFFFFFu, any)) {
                uint64_t we[kLane];
#pragma unroll
                for (int e = 0; e < kLane; e += 2) weights(x[e], x[e + 1], we[e], we[e + 1]);
#pragma unroll
                for (int e = 0; e < kLane; ++e) {
                    const uint32_t dk = desc_key(x[e]);
                    const uint64_t w = we[e];
                    before += dk < klo ? w : 0;
                    outside += dk > khi ? w : 0;
                    hits |= (uint32_t)(dk >= klo && dk <= khi) << e;
                    if (entropy && dk < klo)
                        ux += (uint64_t)entropy_term((unsigned long long)dk << 32, w, M, temp, k);
                }
                before = warp_sum(before);
            }
            if ((threadIdx.x & 31) == 0) lead.span_mass[s] = before;
            if (hits) {
                uint32_t at = atomicAdd(&sm.n_cand, (uint32_t)__popc(hits));
#pragma unroll 1
                for (; hits; hits &= hits - 1, ++at) {
                    const int c = col + __ffs(hits) - 1;
                    const float z = Elem<E>::to_float(row[c]);
                    const uint64_t w = weight(z);
                    inside += w;
                    if (at < (uint32_t)kCand) {
                        sm.cand[at] = ((unsigned long long)desc_key(z) << 32) | (uint32_t)c;
                        sm.weight[at] = w;
                    }
                }
            }
        });
        put<3>({inside, outside, ux});
        if (threadIdx.x == 0) lead.part[thread / kExThreads][3] = sm.n_cand;
        sync();
        const int rank = thread / kExThreads;
        if (rank > 0) {
            uint32_t to = 0;
#pragma unroll
            for (int i = 0; i < kMaxTeam; ++i) to += i < rank ? (uint32_t)lead.part[i][3] : 0;
            const uint32_t mine = min(sm.n_cand, (uint32_t)kCand);
            for (uint32_t i = threadIdx.x; i < mine && to + i < (uint32_t)kCand; i += kExThreads) {
                lead.cand[to + i] = sm.cand[i];
                lead.weight[to + i] = sm.weight[i];
            }
        }
        if (first) {
            uint64_t before = 0;
            for (int i = threadIdx.x; i * kSpan < V; i += kExThreads) before += sm.span_mass[i];
            before = warp_sum(before);
            if ((threadIdx.x & 31) == 0) sm.scratch[threadIdx.x >> 5] = before;
            __syncthreads();
            if (threadIdx.x < 32) {
                before = warp_sum(threadIdx.x < kExWarps ? sm.scratch[threadIdx.x] : 0);
                const uint64_t in = get(0), out = get(1), sum = get(2), n = get(3);
                if (threadIdx.x == 0) {
                    sm.n_cand = (uint32_t)n;
                    sm.mass_before = before;
                    sm.mass_in = in;
                    sm.total = before + in + out;
                    sm.ux = sum;
                }
            }
        }
        sync();
    }

    // The element at which the count reaches `want`, or the mass `target`, in
    // the order of the finite logits, all of which level0 counts.  With `share`
    // the target is that share of the whole mass, which this takes as well;
    // `target` is then an estimate.  Afterwards, unless `ties`, the spans hold
    // the mass of what was kept.
    __device__ __noinline__ Selected select(bool by_count, uint32_t want, uint64_t target,
                                            float share = 0.f) {
        if (first) {
            if (threadIdx.x == 0) {
                sm.count_before = 0;
                sm.mass_before = 0;
            }
            __syncthreads();
            const int b = by_count ? pick_bin(sm.level0, nullptr, true, want, 0)
                                   : guess_bin(target, 0, kBins - 1, -1, 0);
            bin_range(b);
            if (threadIdx.x == 0) sm.bin = (uint32_t)b;
        }
        sync();
        uint32_t klo = lead.klo, khi = lead.khi, n_in = lead.n_in;
        int b = (int)lead.bin, lo = 0, hi = kBins - 1;
        weigh_and_gather(klo, khi, share > 0.f);
        if (!by_count) {
            if (share > 0.f) target = share_of(share, lead.total);
            // A guess that missed narrows the bins that are left, so this ends.
            while (true) {
                const uint64_t before = lead.mass_before, in = lead.mass_in;
                if (before >= target && b > lo)
                    hi = b - 1;
                else if (before + in < target && b < hi)
                    lo = b + 1;
                else
                    break;
                sync();
                if (first) {
                    const int anchor = b;
                    b = guess_bin(target, lo, hi, anchor, before);
                    bin_range(b);
                    if (threadIdx.x == 0) sm.bin = (uint32_t)b;
                }
                sync();
                klo = lead.klo;
                khi = lead.khi;
                n_in = lead.n_in;
                b = (int)lead.bin;
                weigh_and_gather(klo, khi, false);
            }
        }
        bool narrowed = false;
        while (n_in > kCand && klo < khi) {
            narrowed = true;
            int shift = 0;
            while (((khi - klo) >> shift) >= (uint32_t)kBins) ++shift;
            sync();
            clear(sm.level1);
            each_span([&](int, int col, const float (&x)[kLane]) {
                uint32_t hits = 0;
#pragma unroll
                for (int e = 0; e < kLane; ++e)
                    hits |= (uint32_t)(desc_key(x[e]) >= klo && desc_key(x[e]) <= khi) << e;
#pragma unroll 1
                for (; hits; hits &= hits - 1) {
                    const float z = Elem<E>::to_float(row[col + __ffs(hits) - 1]);
                    const uint32_t dk = desc_key(z);
                    {
                        const int i = (int)((dk - klo) >> shift);
                        atomicAdd(&sm.level1.count[i], 1u);
                        add_wide(&sm.level1.mass[i], weight(z));
                    }
                }
            });
            merge(sm.level1.count, lead.level1.count, sm.level1.mass, lead.level1.mass);
            if (first) {
                const uint32_t i = (uint32_t)pick_bin(sm.level1.count, sm.level1.mass, by_count,
                                                      want, target);
                if (threadIdx.x == 0) {
                    const uint32_t from = klo + (i << shift);
                    sm.klo = from;
                    sm.khi = min(khi, from + ((1u << shift) - 1u));
                }
            }
            sync();
            klo = lead.klo;
            khi = lead.khi;
            n_in = lead.n_in;
        }
        ties = n_in > kCand;
        if (ties) {
            sync();
            select_tie(klo, by_count, want, target);
        } else {
            if (narrowed) {
                sync();
                weigh_and_gather(klo, khi, false);
            }
            if (first) {
                const Selected f = list_select<kExThreads>(
                    sm.list, sm.cand, sm.weight, min((int)sm.n_cand, kCand),
                    (unsigned long long)klo << 32, (unsigned long long)khi << 32 | 0xFFFFFFFFu,
                    false, by_count, want, target, sm.count_before, sm.mass_before);
                if (threadIdx.x == 0) sm.sel = f;
                // what is kept of the candidates joins the spans
                for (int i = threadIdx.x; i < min((int)sm.n_cand, kCand); i += kExThreads) {
                    if (sm.cand[i] > f.key) continue;
                    const uint64_t w = sm.weight[i];
                    add_wide(&sm.span_mass[(uint32_t)sm.cand[i] / kSpan], w);
                    if (entropy)
                        add_wide(&sm.ux, (uint64_t)entropy_term(sm.cand[i], w, M, temp, k));
                }
            }
        }
        sync();
        const Selected found = lead.sel;
        sync();
        return found;
    }

    // Many equal logits: how many of them are taken follows from their common
    // weight; the last one taken is found by counting them in index order.
    __device__ void select_tie(uint32_t key, bool by_count, uint32_t want, uint64_t target) {
        each_span([&](int s, int, const float (&x)[kLane]) {
            uint32_t n = 0;
#pragma unroll
            for (int e = 0; e < kLane; ++e) n += desc_key(x[e]) == key;
            n = __reduce_add_sync(0xFFFFFFFFu, n);
            if ((threadIdx.x & 31) == 0) lead.span_mass[s] = n;
        });
        sync();
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
                if (mass_before + (uint64_t)mid * w >= target)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            take = lo;
        }
        __syncthreads();
        const int spans = (V + kSpan - 1) / kSpan;
        uint64_t nb, unused, mine = 0;
        for (int i = 0; i < kSpansPer; ++i) {
            const int s = kSpansPer * (int)threadIdx.x + i;
            mine += s < spans ? sm.span_mass[s] : 0;
        }
        block_scan<kExThreads, uint64_t>(sm.scratch, mine, 0, nb, unused);
        for (int i = 0; i < kSpansPer; ++i) {
            const int s = kSpansPer * (int)threadIdx.x + i;
            const uint64_t n = s < spans ? sm.span_mass[s] : 0;
            if (nb < take && take <= nb + n) {
                sm.first = (uint32_t)s;
                sm.n_in = (uint32_t)nb;
            }
            nb += n;
        }
        __syncthreads();
        const int c = (int)sm.first * kSpan + (int)threadIdx.x;
        const uint64_t skipped = sm.n_in;
        const bool hit = (int)threadIdx.x < kSpan && c >= 0 && c < V &&
                         desc_key(Elem<E>::to_float(row[c])) == key;
        block_scan<kExThreads, uint64_t>(sm.scratch, hit ? 1 : 0, 0, nb, unused);
        if (hit && skipped + nb + 1 == take)
            sm.sel = {(unsigned long long)key << 32 | (uint32_t)c, before + take,
                      mass_before + (uint64_t)take * w};
        __syncthreads();
    }
};

// ---------------------------------------------------------------------------
// Finish: one CTA per row.
//
// Nothing filtered: the statistics follow from the records; a draw finds its
// chunk by the prefix sums of the chunks and its column by those of that
// chunk alone.  It stands when the target u S lies further than the sums' error
// bound from both ends of the column's interval.
//
// Filtered: a histogram over M - z gives a bin b such that the columns in bins
// <= b are sure or likely to hold all kept ones: of the group maxima (top-k: k
// maxima, so at least k columns; top-p: their maxima alone hold the mass), of
// the columns themselves in a row short enough to be read twice at little
// cost, or simply the bin of min-p's threshold.  Only the groups whose maximum
// lies in those bins are read again.  What is found has exact weights; a
// nucleus is measured against the fp32 sum with its error bound (against an
// exact one after top-k), and the row is left to the exact kernel where the
// bound does not decide or the columns do not suffice.
//
// Up to one candidate per thread, every thread finds the rank and the mass
// before its own by comparing with all others: for the usual 50 to 100 that
// is a few hundred cycles, where a sort by a block needs 28 synchronised steps.
// Among more the cut and the draw are selected by histograms (list_select).
// ---------------------------------------------------------------------------
constexpr int kFinThreads = 256;
constexpr int kFinBins = 1024;     // 64 binary orders of e, in steps of 1/16
constexpr int kFinCand = 2048;
constexpr int kFinGroups = 2048;
constexpr int kFinAll = 1024;      // columns of a row that are all taken as candidates
constexpr int kFinShort = 16384;   // columns of a row whose histogram is of its columns
constexpr int kMaxChunks = (int)(kFilterMaxV / PSTAT_CHUNK_F32);

struct Candidate {
    unsigned long long key;  // (descending key, column)
    unsigned long long weight;
};

// What a row without filters needs.
struct DrawShared {
    float prefix[kMaxChunks];
    unsigned long long scratch[2 * (kFinThreads / 32)];
    uint32_t bin, found;
};

struct FinishShared {
    union {
        struct {
            uint32_t count[kFinBins];
            uint32_t mass[kFinBins];
        } hist;
        Candidate pair[kFinThreads];
        ListShared<kFinThreads> list;
        float prefix[kMaxChunks];
    };
    unsigned long long cand[kFinCand];
    union {
        unsigned long long weight[kFinCand];
        uint16_t group[kFinGroups];
    };
    float2 table[64];
    unsigned long long scratch[2 * (kFinThreads / 32)];
    unsigned long long target0, target1, total, sum, cut, draw, ux;
    uint32_t n_group, n_cand, bin, found, keep0, keep1;
};
static_assert(kMaxChunks * 32 <= 65536, "group indices are 16 bits");

__device__ __forceinline__ void leave_row(const FilterArgs& a, int64_t t) {
    if (threadIdx.x == 0) a.left[atomicAdd(a.left_count, 1)] = (int)t;
}

template <typename E, typename Shared>
__device__ void finish_greedy(const FilterArgs& a, int64_t t, const E* row, const float4* rec,
                              float M, Shared& sm) {
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

template <typename E, typename Shared>
__device__ void finish_draw(const FilterArgs& a, int64_t t, const E* row, const float4* rec,
                            float M, float c, const RowSettings& rs, float lnS, Shared& sm) {
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
    {
        int col[kPer / kVec];
        float x[kPer / kVec][kVec];
#pragma unroll
        for (int v = 0; v < kPer / kVec; ++v) col[v] = col0 + v * kVec;
        load_columns<E, kPer / kVec>(row, col, (int)a.V, x);
#pragma unroll
        for (int v = 0; v < kPer / kVec; ++v)
#pragma unroll
            for (int e = 0; e < kVec; ++e) z[v * kVec + e] = x[v][e];
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

// Calls f(group, maximum) for a row's groups, eight loads ahead.
template <typename E, typename F>
__device__ __forceinline__ void for_each_group(const E* __restrict__ gm, int groups, F f) {
    constexpr int kAhead = 8;
    for (int i0 = threadIdx.x; i0 < groups; i0 += kAhead * kFinThreads) {
        E g[kAhead];
#pragma unroll
        for (int h = 0; h < kAhead; ++h)
            g[h] = i0 + h * kFinThreads < groups ? gm[i0 + h * kFinThreads] : Elem<E>::neg_inf();
#pragma unroll
        for (int h = 0; h < kAhead; ++h)
            if (i0 + h * kFinThreads < groups) f(i0 + h * kFinThreads, Elem<E>::to_float(g[h]));
    }
}

// ln(min_p) t + M with the bounds of its fp32 error: the product of a logarithm
// of 2 ulp with t, and the sum.
struct MinP {
    float lo, hi;
};
__device__ __forceinline__ MinP min_p_bounds(float M, const RowSettings& rs) {
    if (!rs.cut_m) return {-INFINITY, -INFINITY};
    if (rs.min_p == 1.f) return {M, M};
    const float d = rs.temp * logf(rs.min_p);
    const float z = M + d;
    const float err = (fabsf(d) * 4.f + fabsf(z)) * 1.1920929e-7f;
    return {__fadd_rd(z, -err), fminf(M, __fadd_ru(z, err))};
}

struct FinishRow {
    int64_t t;
    RowSettings rs;
    float M, Sf;
    TempScale c;
    MinP mp;
    int k;         // top-k's, 0 if it does not cut
    int n;         // candidates
    bool all;      // they are all finite columns of the row
    bool all_min;  // they hold every column that min-p keeps
    int scale;     // digits of their weights
};

template <typename E, bool kSample>
__device__ __forceinline__ void write_token(const FilterArgs& a, const E* row, const FinishRow& r,
                                            uint32_t col, uint64_t S) {
    a.token[r.t] = (int64_t)col;
    a.logprob[r.t] = (Elem<E>::to_float(row[col]) - r.M) / r.rs.temp - fixed_log(S, r.scale);
}

template <typename E>
__device__ __forceinline__ void write_kept(const FilterArgs& a, const E* row, const FinishRow& r,
                                           unsigned long long cut, uint64_t S, long long ux) {
    const float lnS = fixed_log(S, r.scale);
    const float U = (float)ux * 5.6843419e-14f;  // 2^-44
    const float Sr = (float)S * __int_as_float((127 - r.scale) << 23);
    write_statistics(a, r.t, row, r.M, lnS, lnS - U / Sr, r.rs.temp, (uint32_t)(cut >> 32),
                     (uint32_t)cut);
}

// Targets of a nucleus that is measured against the fp32 sum: p S with the
// error bound taken off and added.
__device__ __forceinline__ void nucleus_targets(const FinishRow& r, FinishShared& sm) {
    const double target = (double)r.rs.top_p * (double)r.Sf * (double)(1ull << r.scale);
    sm.target0 = __double2ull_rd(target * (1.0 - (double)kSumError));
    sm.target1 = __double2ull_ru(target * (1.0 + (double)kSumError));
}

// Decides a row from at most kFinThreads candidates.
template <typename E, bool kSample>
__device__ __forceinline__ void finish_few(const FilterArgs& a, const E* row, const FinishRow& r,
                                           FinishShared& sm) {
    const int lane = threadIdx.x & 31, n = r.n;
    // `parts` neighbouring lanes share a candidate, each comparing it with its
    // share of the others.
    const int parts = n <= kFinThreads / 4 ? 4 : n <= kFinThreads / 2 ? 2 : 1;
    const int item = (int)threadIdx.x / parts, part = (int)threadIdx.x % parts;
    // (number, mass) of the candidates that `less` accepts
    auto count_before = [&](auto less, int& number, uint64_t& mass) {
        number = 0;
        mass = 0;
        if ((int)(threadIdx.x & ~31u) / parts < n) {
#pragma unroll 4
            for (int j = part; j < n; j += parts) {
                const Candidate o = sm.pair[j];
                const bool yes = less(o.key);
                number += yes;
                mass += yes ? o.weight : 0;
            }
            for (int off = 1; off < parts; off <<= 1) {
                number += __shfl_xor_sync(0xFFFFFFFFu, number, off);
                mass += __shfl_xor_sync(0xFFFFFFFFu, mass, off);
            }
        }
    };
    if ((int)threadIdx.x < n) {
        const unsigned long long mine = sm.cand[threadIdx.x];
        sm.pair[threadIdx.x] = {
            mine, fixed_weight(key_logit((uint32_t)(mine >> 32)), r.M, r.c, r.scale, sm.table)};
    }
    const bool whole = r.k > 0 || r.all;  // the whole mass is among the candidates'
    if (r.rs.cut_p && !whole && threadIdx.x == 0) nucleus_targets(r, sm);
    __syncthreads();
    const bool mine = item < n && part == 0;  // one thread speaks for a candidate
    const unsigned long long key = item < n ? sm.pair[item].key : ~0ull;
    const uint64_t w = item < n ? sm.pair[item].weight : 0;
    int rank;
    uint64_t before;
    count_before([&](unsigned long long o) { return o < key; }, rank, before);
    if (mine && rank == n - 1) sm.total = before + w;
    if (r.rs.cut_p && whole && mine && rank == (r.k > 0 && r.k < n ? r.k : n) - 1) {
        sm.target0 = sm.target1 = share_of(r.rs.top_p, before + w);
    }
    __syncthreads();
    // A column is kept when its rank, the mass before it and its logit pass
    // every filter; by the narrow and by the wide bounds.
    const float z = key_logit((uint32_t)(key >> 32));
    const bool in = mine && (r.k == 0 || rank < r.k);
    const int keep = __syncthreads_count(in && (!r.rs.cut_m || z >= r.mp.hi) &&
                                         (!r.rs.cut_p || before < sm.target0));
    const int most = __syncthreads_count(in && (!r.rs.cut_m || z >= r.mp.lo) &&
                                         (!r.rs.cut_p || before < sm.target1));
    // All candidates kept: then a filter must end here, or there are no others.
    const bool ends = keep < n || r.all || (r.k > 0 && r.k <= n) || r.all_min ||
                      (r.rs.cut_p && sm.total >= sm.target1);
    if (keep == 0 || keep != most || !ends) return leave_row(a, r.t);
    if (mine && rank == keep - 1) {
        sm.sum = before + w;
        sm.cut = key;
        if (kSample) sm.draw = __double2ull_rd((double)r.rs.u * (double)(before + w));
    }
    __syncthreads();
    const uint64_t S = sm.sum;
    const unsigned long long cut = sm.cut;
    if (!kSample) {
        const long long ux = (long long)warp_sum(
            mine && key <= cut ? (uint64_t)entropy_term(key, w, r.M, r.rs.temp, r.scale) : 0);
        if (lane == 0 && ux) add_wide(&sm.ux, (uint64_t)ux);
        __syncthreads();
        if (threadIdx.x == 0) write_kept(a, row, r, cut, S, (long long)sm.ux);
        return;
    }
    // The draw: the kept columns in index order.  u = 0 takes the first of
    // them, however small its weight.
    const uint32_t col = (uint32_t)key;
    int less;
    uint64_t mass;
    count_before([&](unsigned long long o) { return o <= cut && (uint32_t)o < col; }, less, mass);
    const uint64_t target = sm.draw;
    if (mine && key <= cut &&
        (r.rs.u == 0.f ? less == 0 : (mass <= target && mass + w > target)))
        write_token<E, kSample>(a, row, r, col, S);
}

// Decides a row from more candidates, by selections in their list.
template <typename E, bool kSample>
__device__ __noinline__ void finish_many(const FilterArgs& a, const E* row, const FinishRow& r,
                                         FinishShared& sm) {
    const int lane = threadIdx.x & 31, n = r.n;
    uint64_t total = 0;
    int n_hi = 0, n_lo = 0;  // columns that min-p keeps, by both bounds
    for (int i = threadIdx.x; i < n; i += kFinThreads) {
        const float z = key_logit((uint32_t)(sm.cand[i] >> 32));
        const uint64_t w = fixed_weight(z, r.M, r.c, r.scale, sm.table);
        sm.weight[i] = w;
        total += w;
        n_hi += z >= r.mp.hi;
        n_lo += z >= r.mp.lo;
    }
    total = warp_sum(total);
    n_hi = __reduce_add_sync(0xFFFFFFFFu, n_hi);
    n_lo = __reduce_add_sync(0xFFFFFFFFu, n_lo);
    if (lane == 0) {
        add_wide(&sm.total, total);
        atomicAdd(&sm.keep0, (uint32_t)n_hi);
        atomicAdd(&sm.keep1, (uint32_t)n_lo);
    }
    if (threadIdx.x == 0) nucleus_targets(r, sm);
    __syncthreads();
    total = sm.total;
    n_hi = (int)sm.keep0;
    n_lo = (int)sm.keep1;
    auto select = [&](bool by_count, uint32_t want, uint64_t target) {
        return list_select<kFinThreads>(sm.list, sm.cand, sm.weight, n, 0, ~0ull, false, by_count,
                                        want, target, 0, 0);
    };
    const bool whole = r.k > 0 || r.all;
    int keep = n + 1;  // n + 1: all of these, and perhaps more
    Selected end = {0, 0, 0};
    if (r.k > 0 && r.k <= n) {
        keep = r.k;
        end = select(true, (uint32_t)r.k, 0);
    }
    if (r.rs.cut_p) {
        uint64_t t0 = sm.target0, t1 = sm.target1;
        if (whole) {
            t0 = t1 = share_of(r.rs.top_p, keep <= n ? end.mass : total);
        }
        if (t0 == 0) return leave_row(a, r.t);
        if (total >= t0) {
            const Selected s = select(false, 0, t0);
            if (s.mass < t1) {
                // between the bounds, unless min-p ends before it
                if (!(r.rs.cut_m && n_lo < (int)s.rank)) return leave_row(a, r.t);
            } else if ((int)s.rank < keep) {
                keep = (int)s.rank;
                end = s;
            }
        }
    }
    if (r.rs.cut_m && n_hi < keep && n_hi != n_lo) return leave_row(a, r.t);
    if (r.rs.cut_m && n_lo < keep && (n_lo < n || r.all_min || r.all)) {
        keep = n_lo;
        end = select(true, (uint32_t)keep, 0);
    }
    if (keep > n && r.all) {
        keep = n;
        end = select(true, (uint32_t)n, 0);
    }
    if (keep > n || keep == 0 || (int)end.rank != keep) return leave_row(a, r.t);
    const uint64_t S = end.mass;
    const unsigned long long cut = end.key;
    if (!kSample) {
        long long ux = 0;
        for (int i = threadIdx.x; i < n; i += kFinThreads)
            if (sm.cand[i] <= cut)
                ux += entropy_term(sm.cand[i], sm.weight[i], r.M, r.rs.temp, r.scale);
        ux = (long long)warp_sum((uint64_t)ux);
        if (lane == 0 && ux) add_wide(&sm.ux, (uint64_t)ux);
        __syncthreads();
        if (threadIdx.x == 0) write_kept(a, row, r, cut, S, (long long)sm.ux);
        return;
    }
    const bool lowest = r.rs.u == 0.f;
    const Selected s = list_select<kFinThreads>(
        sm.list, sm.cand, sm.weight, n, 0, cut, true, lowest, 1,
        __double2ull_rd((double)r.rs.u * (double)S) + 1, 0, 0);
    if (threadIdx.x == 0) write_token<E, kSample>(a, row, r, (uint32_t)s.key, S);
}

// kFiltered: some row may have a filter; without, the kernel needs neither the
// registers nor the shared memory of the candidates.
template <typename E, bool kSample, bool kFiltered>
__global__ void __launch_bounds__(kFinThreads, kFiltered ? 4 : 6)
    filter_finish_kernel(const __grid_constant__ FilterArgs a) {
    __shared__ typename std::conditional<kFiltered, FinishShared, DrawShared>::type sm;
    constexpr int kVec = Elem<E>::kVec;
    const int64_t t = blockIdx.x;
    const int V = (int)a.V, lane = threadIdx.x & 31;
    const E* row = static_cast<const E*>(a.logits) + t * a.ld;
    const float4* rec = a.records + t * a.chunks;
    if constexpr (kFiltered) {
        for (int i = threadIdx.x; i < kFinBins; i += kFinThreads)
            sm.hist.count[i] = sm.hist.mass[i] = 0;
        if (threadIdx.x < 64) sm.table[threadIdx.x] = kExp2Table[threadIdx.x];
        if (threadIdx.x == 0) {
            sm.n_group = sm.n_cand = sm.keep0 = sm.keep1 = 0;
            sm.ux = sm.total = 0;
            sm.bin = kFinBins;
        }
    }
    FinishRow r;
    r.t = t;
    r.rs = row_settings<kSample>(a, t);
    const RowSettings& rs = r.rs;
    // Up to here only what the caller gave was read.  Every block waits, so that
    // this grid cannot complete before the records are.
    grid_wait();
    grid_launch_dependents();
    if (!rs.valid) {
        if (threadIdx.x == 0) write_undefined<kSample>(a, t, PSTAT_DEV_BAD_PARAM);
        return;
    }
    r.c = temp_scale(rs.greedy ? 1.f : rs.temp);
    const float3 st = fold_records(rec, a.chunks, r.c.ch, lane);
    const float M = r.M = st.x + 0.f, Sf = r.Sf = st.y;
    if (!(M > -INFINITY)) {
        if (threadIdx.x == 0) write_undefined<kSample>(a, t, PSTAT_DEV_EMPTY_ROW);
        return;
    }
    if (rs.greedy) return finish_greedy(a, t, row, rec, M, sm);
    if (!kFiltered || (!rs.cut_k && !rs.cut_p && !rs.cut_m)) {
        const float lnS = logf(Sf);
        if (kSample) {
            __syncthreads();  // the histogram's zeros share memory with the prefix sums
            return finish_draw(a, t, row, rec, M, r.c.ch, rs, lnS, sm);
        }
        if (threadIdx.x == 0)
            write_statistics(a, t, row, M, lnS, lnS - kLn2 * (st.z / Sf), rs.temp, 0xFFFFFFFFu,
                             (uint32_t)V - 1);
        return;
    }
    if constexpr (kFiltered) {

    r.k = rs.cut_k ? (int)rs.top_k : 0;
    r.mp = min_p_bounds(M, rs);
    r.all = V <= kFinAll;
    const float bin_scale = r.c.ch * ((float)kFinBins / 64.f);
    const float ch = r.c.ch;
    auto bin_of = [&](float z) { return min(kFinBins - 1, __float2int_rd((M - z) * bin_scale)); };
    const E* gm = static_cast<const E*>(a.group_max) + t * a.chunks * 32;
    const int groups = a.chunks * 32;
    const int bin_m = rs.cut_m ? bin_of(r.mp.lo) : kFinBins;
    // Columns up to this bin are gathered; the last bin is open.
    int b = kFinBins;
    __syncthreads();
    if (!r.all && (rs.cut_k || rs.cut_p)) {
        const bool by_mass = rs.cut_p && !rs.cut_k, short_row = V <= kFinShort;
        constexpr float kUnit = 131072.f;  // 2^17: of all groups together below 2^32
        auto add = [&](float z) {
            if (z == -INFINITY) return;
            const int i = bin_of(z);
            atomicAdd(&sm.hist.count[i], 1u);
            if (by_mass) atomicAdd(&sm.hist.mass[i], __float2uint_rn(ex2_approx((z - M) * ch) * kUnit));
        };
        if (short_row) {
            constexpr int kAhead = 2;
            for (int c0 = threadIdx.x * kVec; c0 < V; c0 += kAhead * kFinThreads * kVec) {
                int col[kAhead];
                float x[kAhead][kVec];
#pragma unroll
                for (int h = 0; h < kAhead; ++h) col[h] = c0 + h * kFinThreads * kVec;
                load_columns<E, kAhead>(row, col, V, x);
#pragma unroll
                for (int h = 0; h < kAhead; ++h)
#pragma unroll
                    for (int e = 0; e < kVec; ++e) add(x[h][e]);
            }
        } else {
            for_each_group(gm, groups, [&](int, float g) { add(g); });
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
        // a little more than the nucleus, so that roundings cannot fall short of it
        const float need = (rs.top_p + (1.f - rs.top_p) * 0.05f) * Sf * kUnit;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint32_t c1 = cb + sm.hist.count[b0 + i], m1 = mb + sm.hist.mass[b0 + i];
            if (by_mass ? ((float)mb < need && (float)m1 >= need)
                        : (cb < (uint32_t)r.k && (uint32_t)r.k <= c1))
                sm.bin = b0 + i;
            cb = c1;
            mb = m1;
        }
        __syncthreads();
        b = (int)sm.bin;
    }
    // top-p after top-k needs the whole top-k mass, so min-p may not shorten it
    if (!r.all) {
        if (!(rs.cut_k && rs.cut_p)) b = min(b, bin_m);
        if (b >= kFinBins - 1) return leave_row(a, t);
    }
    r.all_min = rs.cut_m && b >= bin_m;

    // ---- gather.  bin_of(z) <= b  <=>  (M - z) bin_scale < b + 1
    const float edge = r.all ? INFINITY : (float)(b + 1);
    int n_vec;  // vectors of kVec columns to look through
    if (r.all) {
        n_vec = (V + kVec - 1) / kVec;
    } else {
        for_each_group(gm, groups, [&](int i, float g) {
            if (g > -INFINITY && (M - g) * bin_scale < edge) {
                const uint32_t at = atomicAdd(&sm.n_group, 1u);
                if (at < (uint32_t)kFinGroups) sm.group[at] = (uint16_t)i;
            }
        });
        __syncthreads();
        const int n_group = (int)sm.n_group;
        if (n_group > kFinGroups) return leave_row(a, t);
        n_vec = n_group * kVecPerLane;
    }
    // One vector per thread, four ahead; what passes is rare, so it is picked
    // out of a bit mask and read again.
    constexpr int kAhead = 4;
    for (int i0 = threadIdx.x; i0 < n_vec; i0 += kAhead * kFinThreads) {
        float x[kAhead][kVec];
        int col[kAhead];
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
            const int i = i0 + h * kFinThreads;
            if (r.all) {
                col[h] = i * kVec;
            } else {
                const int g = sm.group[min(i, n_vec - 1) / kVecPerLane], j = i % kVecPerLane;
                col[h] = (g >> 5) * Elem<E>::kChunk + ((g & 31) + 32 * j) * kVec;
            }
            if (i >= n_vec) col[h] = V;
        }
        load_columns<E, kAhead>(row, col, V, x);
        uint32_t hits = 0;
#pragma unroll
        for (int h = 0; h < kAhead; ++h)
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                hits |= (uint32_t)(x[h][e] > -INFINITY && (r.all || (M - x[h][e]) * bin_scale < edge))
                        << (h * kVec + e);
        if (hits == 0) continue;
        uint32_t at = atomicAdd(&sm.n_cand, (uint32_t)__popc(hits));
#pragma unroll 1
        for (; hits; hits &= hits - 1, ++at) {
            const int bit = __ffs(hits) - 1, h = bit / kVec;
            const int c = (h == 0 ? col[0] : h == 1 ? col[1] : h == 2 ? col[2] : col[3]) + bit % kVec;
            if (at < (uint32_t)kFinCand)
                sm.cand[at] = ((unsigned long long)desc_key(Elem<E>::to_float(row[c])) << 32) |
                              (uint32_t)c;
        }
    }
    __syncthreads();
    r.n = (int)sm.n_cand;
    if (r.n > kFinCand || (rs.cut_p && r.k > r.n && !r.all)) return leave_row(a, t);
    r.scale = fixed_scale(Sf * (1.f + 2.f * kSumError));
    if (r.n <= kFinThreads)
        finish_few<E, kSample>(a, row, r, sm);
    else
        finish_many<E, kSample>(a, row, r, sm);

    }
}

// ---------------------------------------------------------------------------
// Exact: clusters of CTAs over the rows that were left, passes with exact sums.
// ---------------------------------------------------------------------------
template <typename E, bool kSample>
__device__ void exact_row(const FilterArgs& a, int64_t t, Team<E>& tm, ExactShared& sm,
                          ExactShared& lead) {
    const int V = (int)a.V, lane = threadIdx.x & 31;
    const bool first = tm.first;
    const E* row = tm.row;
    const RowSettings rs = row_settings<kSample>(a, t);
    tm.c = temp_scale(rs.temp);
    const float3 st = fold_records(a.records + t * a.chunks, a.chunks, tm.c.ch, lane);
    const float M = st.x + 0.f;
    tm.M = M;
    tm.temp = rs.temp;
    tm.bin_scale = tm.c.ch * ((float)kBins / 64.f);
    tm.k = fixed_scale(st.y * (1.f + 2.f * kSumError));
    if (threadIdx.x == 0) {
        sm.first = sm.first_kept = 0xFFFFFFFFu;
    }
    tm.sync();

    const float z_min = min_p_logit(M, rs);
    uint32_t cut_key = 0xFFFFFFFFu, cut_index = (uint32_t)V - 1;
    bool spans_ready = false;
    if (rs.cut_k || rs.cut_p || (rs.cut_m && !kSample)) {
        // Counts of the level-0 bins.
        for (int i = threadIdx.x; i < kBins; i += kExThreads) sm.level0[i] = 0;
        __syncthreads();
        uint32_t n_min = 0, n_fin = 0;
        tm.each_span([&](int, int, const float (&x)[Team<E>::kLane]) {
#pragma unroll
            for (int e = 0; e < Team<E>::kLane; ++e) {
                if (x[e] > -INFINITY) {
                    atomicAdd(&sm.level0[tm.bin0(x[e])], 1u);
                    n_min += x[e] >= z_min;
                    ++n_fin;
                }
            }
        });
        tm.template put<2>({n_min, n_fin});
        tm.merge(sm.level0, lead.level0);
        const uint32_t n_finite = (uint32_t)tm.get(1);
        const uint32_t n_keep_min = rs.cut_m ? (uint32_t)tm.get(0) : n_finite;
        tm.sync();
        uint32_t want = rs.cut_k && rs.top_k < (int64_t)n_finite ? (uint32_t)rs.top_k : n_finite;
        Selected sel;
        bool have = false;
        if (rs.cut_p) {
            if (want < n_finite) {
                const uint64_t total = tm.select(true, want, 0).mass;
                sel = tm.select(false, 0, share_of(rs.top_p, total));
            } else {
                const float about = rs.top_p * st.y * __int_as_float((127 + tm.k) << 23);
                sel = tm.select(false, 0, (uint64_t)about, rs.top_p);
            }
            want = sel.rank;
            have = n_keep_min >= want;
        }
        if (!have) sel = tm.select(true, min(want, n_keep_min), 0);
        spans_ready = !tm.ties;
        cut_key = (uint32_t)(sel.key >> 32);
        cut_index = (uint32_t)sel.key;
    } else if (rs.cut_m) {
        cut_key = desc_key(z_min);
    }

    // Kept mass of every span of the index order (and the sum of e x), where no
    // selection has left it.
    const int spans = (V + kSpan - 1) / kSpan;
    constexpr int kLane = Team<E>::kLane;
    if (!spans_ready) {
        uint64_t ux = 0;
        tm.each_span([&](int s, int col, const float (&x)[kLane]) {
            uint64_t w = 0, ws[kLane];
#pragma unroll
            for (int e = 0; e < kLane; e += 2)
                fixed_weights(x[e], x[e + 1], M, tm.c, tm.k, sm.table, ws[e], ws[e + 1]);
#pragma unroll
            for (int e = 0; e < kLane; ++e) {
                const uint64_t we = ws[e];
                const bool kept = is_kept(x[e], col + e, cut_key, cut_index);
                w += kept ? we : 0;
                if (!kSample && kept)
                    ux += (uint64_t)entropy_term((unsigned long long)desc_key(x[e]) << 32, we, M,
                                                 rs.temp, tm.k);
            }
            w = warp_sum(w);
            if (lane == 0) lead.span_mass[s] = w;
        });
        if (!kSample) tm.template put<3>({0, 0, ux});
    }
    if (kSample && rs.u == 0.f) {
        uint32_t lowest = 0xFFFFFFFFu;
        tm.each_span([&](int, int col, const float (&x)[kLane]) {
#pragma unroll
            for (int e = 0; e < kLane; ++e)
                if (x[e] > -INFINITY && is_kept(x[e], col + e, cut_key, cut_index))
                    lowest = min(lowest, (uint32_t)(col + e));
        });
        lowest = __reduce_min_sync(0xFFFFFFFFu, lowest);
        if (lane == 0) atomicMin(&lead.first_kept, lowest);
    }
    tm.sync();
    if (!first) return;

    uint64_t before, unused, mine = 0;
    for (int i = 0; i < kSpansPer; ++i) {
        const int s = kSpansPer * (int)threadIdx.x + i;
        mine += s < spans ? sm.span_mass[s] : 0;
    }
    block_scan<kExThreads, uint64_t>(sm.scratch, mine, 0, before, unused);
    if (threadIdx.x == kExThreads - 1) sm.mass_before = before + mine;
    if (threadIdx.x < 32 && !kSample && !spans_ready) {
        const uint64_t ux = tm.get(2);
        if (threadIdx.x == 0) sm.ux = ux;
    }
    __syncthreads();
    const uint64_t S = sm.mass_before;
    const float lnS = fixed_log(S, tm.k);
    if (!kSample) {
        if (threadIdx.x == 0) {
            const float U = (float)(long long)sm.ux * 5.6843419e-14f;  // 2^-44
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
    // C > u S in whole numbers
    const uint64_t target = __double2ull_rd((double)rs.u * (double)S);
    __syncthreads();
    for (int i = 0; i < kSpansPer; ++i) {
        const int s = kSpansPer * (int)threadIdx.x + i;
        const uint64_t w = s < spans ? sm.span_mass[s] : 0;
        if (before <= target && before + w > target) {
            sm.first = (uint32_t)s;
            sm.mass_before = before;
        }
        before += w;
    }
    __syncthreads();
    const int c = (int)sm.first * kSpan + (int)threadIdx.x;
    const uint64_t base = sm.mass_before;
    uint64_t w = 0;
    float z = 0.f;
    if ((int)threadIdx.x < kSpan && c >= 0 && c < V) {
        z = Elem<E>::to_float(row[c]);
        if (is_kept(z, c, cut_key, cut_index)) w = tm.weight(z);
    }
    uint64_t wb;
    block_scan<kExThreads, uint64_t>(sm.scratch, w, 0, wb, unused);
    wb += base;
    if (wb <= target && wb + w > target) {
        a.token[t] = c;
        a.logprob[t] = (z - M) / rs.temp - lnS;
    }
}

template <typename E, bool kSample>
__global__ void __launch_bounds__(kExThreads, 2)
    filter_exact_kernel(const __grid_constant__ FilterArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    cg::cluster_group cluster = cg::this_cluster();
    ExactShared& sm = *reinterpret_cast<ExactShared*>(smem_raw);
    ExactShared& lead = *cluster.map_shared_rank(&sm, 0);
    if (threadIdx.x < 64) sm.table[threadIdx.x] = kExp2Table[threadIdx.x];
    __syncthreads();
    grid_wait();
    const int n = *a.left_count;
    if (n == 0) return;
    // A cluster to a row, or, with more rows than a few for every cluster, a
    // CTA: what a team saves in a pass it loses again in synchronisation.
    const bool alone = n >= 4 * (int)(gridDim.x / cluster.num_blocks());
    const int team = alone ? 1 : (int)cluster.num_blocks();
    const int rank = alone ? 0 : (int)cluster.block_rank();
    for (int i = blockIdx.x / team; i < n; i += gridDim.x / team) {
        const int64_t t = a.left[i];
        Team<E> tm{sm, alone ? sm : lead, cluster, static_cast<const E*>(a.logits) + t * a.ld,
                   (int)a.V, rank * kExThreads + (int)threadIdx.x, team * kExThreads, rank == 0,
                   alone, !kSample, 0.f, 0.f, {0.f, 0.f}, 0, 0.f, false};
        exact_row<E, kSample>(a, t, tm, sm, tm.lead);
        tm.sync();  // the next row writes what this one reads
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
    const bool filtered = a.top_ks || a.top_ps || a.min_ps || (a.top_k > 0 && a.top_k < a.V) ||
                          a.top_p < 1.f || a.min_p > 0.f;
    e = launch_behind(filtered ? filter_finish_kernel<E, kSample, true>
                               : filter_finish_kernel<E, kSample, false>,
                      (unsigned)a.T, kFinThreads, 0, stream, 1, a);
    // Without filters only a draw can be left over.
    if (e != cudaSuccess || (!filtered && !kSample)) return e;
    // Large teams where few rows can be left over; 16 is beyond the portable size.
    static ContextSeen large_set;
    e = ensure_large_cluster(ex_fn, large_set);
    if (e != cudaSuccess) return e;
    const int most = a.T <= 64 ? kMaxTeam : kMaxTeam / 2;
    int team = 1;
    while (team < most && a.V >= (int64_t)team * 8192) team *= 2;
    int64_t teams = (int64_t)dev.sm_count * 2 / team;
    if (teams > a.T) teams = a.T;
    return launch_behind(filter_exact_kernel<E, kSample>, (unsigned)(teams * team), kExThreads,
                         sizeof(ExactShared), stream, (unsigned)team, a);
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
