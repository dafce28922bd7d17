// sampling.cuh -- what the kernels of the sampler and of the filtered policy
// statistics share: their arguments, a row's settings, column loads, block
// scans and selection in a list.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "chunk_math.cuh"
#include "filter_math.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace pstat {

inline bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct FilterArgs {
    const void* logits;
    int64_t T, V, ld;
    int chunks;                 // of a row
    bool stream_once;           // the logits do not stay in L2 anyway
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
// before the first use; columns past V read as -inf.  The logits are constant while
// the finish and the exact kernel live (the records kernel, whose blocks all wait
// before they let these start, comes between them and whatever wrote the logits).
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

// ln S of a row without filters, by every thread of a CTA.
//
// Where nearly all the mass lies on the maximum, S = 1 + X, an fp32 sum with that 1 in
// it keeps of X what exceeds 2^-24, and ln S, hence 1 - p of that token, its gradient,
// needs X itself.  So below 1 + 2^-6 (above, the sum's 2^-18 are 2^-12 of X) X is summed
// without the maximum's own term: from the records of the other chunks, and from the
// columns of the maximum's chunk, by vectors, warps of 32 vectors, and those in
// ascending order, so that a row gets the same bits from CTAs of any size.
// `scratch` holds 16 floats.  A draw from 2048 rows of 151,936 bf16 that are all like
// that takes 118 us, and took 113 with the logarithm of the fp32 sum.
constexpr float kPeaked = 1.015625f;
template <typename E, int kThreads>
__device__ __forceinline__ float unfiltered_log(const E* row, const float4* rec, int chunks, int V,
                                                float M, float S, float c, float* scratch) {
    if (S >= kPeaked) return logf(S);
    constexpr int kVec = Elem<E>::kVec, kVecs = Elem<E>::kChunk / kVec, kOwn = kVecs / kThreads;
    static_assert(kVecs == 512 && kOwn * kThreads == kVecs, "16 warps' sums");
    const int lane = threadIdx.x & 31;
    int top = -1;  // the maximum's chunk; with two of them S would be 2
    float others = 0.f;
    for (int i = lane; i < chunks; i += 32) {
        const float4 r = rec[i];
        if (r.x == M)
            top = i;
        else if (r.x > -INFINITY)
            others = fmaf(r.y, exp2f(fmaf(r.x - M, c, -r.w)), others);
    }
    top = max(__reduce_max_sync(0xFFFFFFFFu, top), 0);
#pragma unroll
    for (int off = 16; off; off >>= 1) others += __shfl_xor_sync(0xFFFFFFFFu, others, off);
    int col[kOwn];
    float x[kOwn][kVec];
#pragma unroll
    for (int h = 0; h < kOwn; ++h)
        col[h] = top * Elem<E>::kChunk + ((int)threadIdx.x + h * kThreads) * kVec;
    load_columns<E, kOwn>(row, col, V, x);
#pragma unroll
    for (int h = 0; h < kOwn; ++h) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < kVec; ++e) sum += x[h][e] == M ? 0.f : ex2_approx((x[h][e] - M) * c);
#pragma unroll
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
        if (lane == 0) scratch[((int)threadIdx.x + h * kThreads) >> 5] = sum;
    }
    __syncthreads();
    float X = others;
#pragma unroll
    for (int i = 0; i < kVecs / 32; ++i) X += scratch[i];
    __syncthreads();
    return log1pf(X);
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
// where sorting 2048 keys costs a block 66 synchronised steps.  `grain` low
// bits of the high word are alike in equal logits and say nothing else (16 of a
// bf16 logit's key).
// ---------------------------------------------------------------------------
struct Selected {
    unsigned long long key;
    uint32_t rank;  // 1-based
    uint64_t mass;  // up to and including it
};

// Low bits of a key that no two different logits of the type differ in.
template <typename E>
constexpr int kGrain = sizeof(E) == 2 ? 16 : 0;

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
                                             uint64_t mass_before, int grain) {
    constexpr int kPer = ListShared<kThreads>::kBins / kThreads;
    uint32_t lo = by_column ? 0u : (uint32_t)(kmin >> 32);
    uint32_t hi = by_column ? (uint32_t)kFilterMaxV - 1 : (uint32_t)(kmax >> 32);
    uint32_t n_in = (uint32_t)n;  // keys in the range, at most
    auto inside = [&](unsigned long long key, uint32_t& p) {
        p = by_column ? (uint32_t)key : (uint32_t)(key >> 32);
        return key >= kmin && key <= kmax && p >= lo && p <= hi;
    };
    while (n_in > (uint32_t)kListMembers) {
        if (!by_column && (lo >> grain) == (hi >> grain)) {
            // equal logits: by their columns from here on
            if (!by_count) {
                uint32_t p;
                for (int i = threadIdx.x; i < n; i += kThreads)
                    if (inside(keys[i], p)) ls.mass[0] = weights[i];  // all alike
                __syncthreads();
                const uint64_t w = ls.mass[0];
                const uint64_t short_of = target - mass_before;
                want = count_before + (uint32_t)(w ? (short_of + w - 1) / w : n_in);
                by_count = true;
                __syncthreads();
            }
            kmin = max(kmin, (unsigned long long)lo << 32);
            kmax = min(kmax, (unsigned long long)hi << 32 | 0xFFFFFFFFu);
            by_column = true;
            lo = 0;
            hi = (uint32_t)kFilterMaxV - 1;
        }
        // bins start on multiples of their width, so that one of 2^grain is one value
        int shift = by_column ? 0 : grain;
        while ((hi >> shift) - (lo >> shift) >= (uint32_t)ListShared<kThreads>::kBins) ++shift;
        lo = lo >> shift << shift;
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
    // Neighbouring lanes (four, in the exact kernel's CTA of 512) share a member.
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
    if (!w) return 0;
    // rn(v) by two 32-bit conversions (64-bit ones run at a sixteenth of the rate):
    // |v| < 2^43, the rest of v is exact, and what is taken off is even.
    const float v = e * x * 1.7592186e13f;
    const int hi = __float2int_rn(v * 0x1p-22f);
    return ((long long)hi << 22) + __float2int_rn(fmaf((float)hi, -0x1p22f, v));
}

// f S for a float f in [0, 1) and S < 2^62: the whole part, and whether there is
// a rest.  f = mant 2^-sh; the product is taken in 128 bits (fp64 runs at about
// two operations per clock and SM here, one conversion costs a thousand cycles).
__device__ __forceinline__ uint64_t part_of(float f, uint64_t S, bool& rest) {
    const uint32_t b = __float_as_uint(f), e = b >> 23;
    const uint64_t mant = (b & 0x7FFFFFu) | (e ? 0x800000u : 0u);
    const int sh = 150 - (int)(e ? e : 1u);  // in [24, 149]
    const uint64_t lo = S * mant, hi = __umul64hi(S, mant);
    if (sh < 64) {
        rest = (lo & ((1ull << sh) - 1)) != 0;
        return hi << (64 - sh) | lo >> sh;
    }
    rest = lo != 0 || (sh < 128 ? (hi & ((1ull << (sh - 64)) - 1)) != 0 : hi != 0);
    return sh < 128 ? hi >> (sh - 64) : 0;
}
// C >= p S  <=>  C >= share_of(p, S); at least 1, so that a token is kept.
__device__ __forceinline__ uint64_t share_of(float p, uint64_t S) {
    bool rest;
    const uint64_t t = part_of(p, S, rest);
    return max(t + rest, (uint64_t)1);
}
// C > u S  <=>  C > draw_of(u, S).
__device__ __forceinline__ uint64_t draw_of(float u, uint64_t S) {
    bool rest;
    return part_of(u, S, rest);
}

// The rows that the finish kernel left, behind it on the stream; `filtered`: some
// row may have a filter.
template <typename E, bool kSample>
cudaError_t launch_exact(const FilterArgs& a, bool filtered, const DeviceInfo& dev,
                         cudaStream_t stream);

}  // namespace pstat
