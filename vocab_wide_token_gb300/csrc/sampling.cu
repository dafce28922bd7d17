// sampling.cu -- drawing a token per row and the policy statistics of given
// labels under the tempered, truncated softmax (filter_math.cuh has the
// definitions).
//
//  filter_records_kernel  the only full read of the logits in the common case:
//                         per chunk the maximum and the tempered sums, per lane
//                         of a chunk the maximum of its columns (its group)
//  filter_finish_kernel   one CTA per row: from the records the whole sum, from
//                         the group maxima the few groups that can hold a kept
//                         token; reads those again and decides, where fp32 sums
//                         with their error bound do
//  filter_exact_kernel    (sampling_exact.cu) the rows that were left
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "sampling.cuh"

namespace pstat {
namespace {

// ---------------------------------------------------------------------------
// Records.  The streaming scheme of the chunk statistics: every warp owns a
// ring of two 8 KB slots that bulk copies fill, takes a chunk out of its slot
// into registers and refills the slot at once.  The items (row, chunk) are split
// into one contiguous range per warp.  Lane L holds the 256 bytes from 256 L of
// the chunk, and their maximum is the maximum of group L of its columns: a
// group that is read again is one run of memory (with the vectors L, L + 32, ...
// of the chunk statistics it is 16 half-used sectors, and drawing 1024 rows
// with top-k 50 spent 42 us on them).
// Bound by HBM: 2048 x 151,936 bf16 (622 MB) in 97 us, 6.4 TB/s.
// A chunk need not start or end on 16 bytes (odd vocabularies and strides): its
// aligned middle is copied to the place in the slot that has the same offset from
// a boundary, up to seven columns at either end are loaded by the lanes when the
// copy is issued, and the slot is read through a shift.
// ---------------------------------------------------------------------------
constexpr int kRecordSlot = kSlotBytes + 32;  // the offset, and the rest of the last vector

template <typename E, bool kU>
__global__ void __launch_bounds__(kWarps * 32, 1)
    filter_records_kernel(const __grid_constant__ FilterArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int lane = threadIdx.x & 31;
    uint8_t* slots = smem + (size_t)warp * kStages * kRecordSlot;
    uint64_t* bars =
        reinterpret_cast<uint64_t*>(smem + (size_t)warps * kStages * kRecordSlot) + warp * kStages;
    constexpr int kChunk = Elem<E>::kChunk;
    const E* logits = static_cast<const E*>(a.logits);
    E* group_max = static_cast<E*>(a.group_max);
    const int V = (int)a.V, chunks = a.chunks;
    grid_wait();  // the logits may be the previous kernel's, and so may the workspace
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.left_count = 0;
    grid_launch_dependents();

    const int64_t n_items = a.T * chunks;
    const int64_t gw = (int64_t)blockIdx.x * warps + warp;
    const int64_t nw = (int64_t)gridDim.x * warps;
    const int64_t i0 = n_items * gw / nw, i1 = n_items * (gw + 1) / nw;
    const int n = (int)(i1 - i0);
    if (n <= 0) return;
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&bars[s], 1);
        fence_mbar_init();
    }
    __syncwarp();
    const uint64_t policy = a.stream_once ? policy_evict_first() : policy_evict_normal();

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
    struct Span {
        const E* src;
        int len;
        uint32_t shift;  // of the start from a 16-byte boundary
        int head;        // columns before the next one
        uint32_t bytes;  // from there, to be copied
        // Lanes 0 to 7 have the columns before the copied ones, 8 to 15 those
        // behind them, 16 to 23 fill the last vector; -1: none.
        __device__ int edge(int lane) const {
            constexpr int kVec = Elem<E>::kVec;
            if (lane < 8) return lane < head ? lane : -1;
            const int col = lane < 16 ? head + (int)(bytes / sizeof(E)) + lane - 8 : len + lane - 16;
            return col < (lane < 16 ? len : lane < 24 ? (len + kVec - 1) / kVec * kVec : 0) ? col : -1;
        }
        __device__ bool ragged() const { return shift || (len * sizeof(E)) % 16; }
    };
    auto locate = [&](const Item& it) {
        Span p;
        const int start = it.g * kChunk;
        p.len = min(kChunk, V - start);
        p.src = logits + it.t * a.ld + start;
        p.shift = (uint32_t)(reinterpret_cast<uintptr_t>(p.src) & 15u);
        p.head = p.shift ? min(p.len, (int)((16 - p.shift) / sizeof(E))) : 0;
        p.bytes = (uint32_t)((p.len - p.head) * (int)sizeof(E)) & ~15u;
        return p;
    };
    static_assert(kStages == 2, "one register of edge columns for each slot");
    E edge0 = Elem<E>::neg_inf(), edge1 = edge0;
    auto issue = [&](const Item& it, int slot) {
        const Span p = locate(it);
        if (p.bytes && lane == 0) {
            mbar_arrive_expect_tx(&bars[slot], p.bytes);
            bulk_g2s_hint(slots + (size_t)slot * kRecordSlot + p.shift + p.head * sizeof(E),
                          p.src + p.head, p.bytes, &bars[slot], policy);
        }
        if (p.ragged()) {
            const int col = p.edge(lane);
            const E x = col >= 0 && col < p.len ? p.src[col] : Elem<E>::neg_inf();
            if (slot == 0)
                edge0 = x;
            else
                edge1 = x;
        }
    };
    auto scale_of = [&](int64_t t) {
        const float temp = a.temperatures ? a.temperatures[t] : a.temperature;
        return (temp >= kFilterTempMin && temp <= kFilterTempMax) ? temp_scale(temp).ch : kLog2e;
    };

    Item cur = {i0 / chunks, (int)(i0 % chunks)};
    Item ahead = cur;
    const int prologue = n < kStages ? n : kStages;
    for (int j = 0; j < prologue; ++j) {
        issue(ahead, j);
        next_item(ahead);
    }
    uint32_t phase = 0;
    int j = 0;
    bool timed_out = false;
    float c = scale_of(cur.t);
    for (; j < n; ++j) {
        const int slot = j % kStages;
        uint8_t* buf = slots + (size_t)slot * kRecordSlot;
        const Span p = locate(cur);
        if (p.bytes) {
            bool ok = mbar_wait_bounded(&bars[slot], (phase >> slot) & 1u, kWaitLimitNs);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) {
                timed_out = true;
                break;
            }
            phase ^= 1u << slot;
        }
        uint4 q[kVecPerLane];
        if (p.ragged()) {
            const int col = p.edge(lane);
            if (col >= 0)
                *reinterpret_cast<E*>(buf + p.shift + col * sizeof(E)) = slot == 0 ? edge0 : edge1;
            __syncwarp();
        }
        if (p.shift)
            load_lane_run_shifted<E>(buf, p.shift, p.len, lane, q);
        else
            load_lane_run<E>(buf, p.len, lane, q);
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
        for (int k = j; k < n; ++k)
            if (lane == 0) a.records[i0 + k] = make_float4(NAN, 0.f, 0.f, 0.f);
        const int last = (j + kStages < n) ? j + kStages : n;
        for (int k = j; k < last; ++k) {
            const int slot = k % kStages;
            if (locate(cur).bytes) {
                mbar_wait_bounded(&bars[slot], (phase >> slot) & 1u, kWaitLimitNs);
                phase ^= 1u << slot;
            }
            next_item(cur);
        }
    }
}

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
// cost, or simply the bin of min-p's threshold.  Of a longer row only the groups
// whose maximum lies in those bins are read again.  What is found has exact weights; a
// nucleus is measured against the fp32 sum with its error bound (against an
// exact one after top-k), and the row is left to the exact kernel where the
// bound does not decide or the columns do not suffice.
//
// Of up to 256 candidates every thread finds the rank and the mass before its own
// by comparing with all others: for the usual 50 to 100 that is a few hundred
// cycles, where a sort by a block needs 28 steps.  More are sorted.
// Bound by latency (records, maxima, columns, ranks, each behind the last): 7 us of a
// call's 11 for one row of V = 151,936 with top-k 50, 30 us for 2048 rows with a nucleus.
// ---------------------------------------------------------------------------
// Bins of M - z: 48 binary orders of e in steps of 1/16, then 510 in steps of 2 (at
// temperature 0.25 the 50th largest of 151,936 logits can be 2^-70 of the first:
// such rows took 95 us by way of the exact kernel, and take 18).
constexpr int kFinBins = 1024;
constexpr int kFineBins = 768;
constexpr float kBinsPerOrder = 16.f, kBinsPerStep = 32.f;
constexpr int kFinCand = 1024;
constexpr int kFinGroups = 2048;
constexpr int kFinShort = 16384;   // columns of a row whose histogram is of its columns
// Candidates that are compared all with all, one to a thread (1000 by 1024 threads
// take 110 us).
template <int kFinThreads>
constexpr int kFinFew = kFinThreads < 256 ? kFinThreads : 256;
constexpr int kMaxChunks = (int)(kFilterMaxV / PSTAT_CHUNK_F32);

struct Candidate {
    unsigned long long key;  // (descending key, column)
    unsigned long long weight;
};

// What a row without filters needs.
template <int kFinThreads>
struct DrawShared {
    float prefix[kMaxChunks];
    unsigned long long scratch[2 * (kFinThreads / 32)];
    uint32_t bin, found;
};

template <int kFinThreads>
struct FinishShared {
    union {
        struct {
            uint32_t count[kFinBins];
            uint32_t mass[kFinBins];
        } hist;
        Candidate pair[kFinFew<kFinThreads>];
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

// Calls f(group, maximum) for a row's groups, eight loads ahead.
template <typename E, int kFinThreads, typename F>
__device__ __forceinline__ void for_each_group(const E* gm, int groups, F f) {
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

// The first group with the row's maximum, and its first column there.
template <typename E, int kFinThreads, typename Shared>
__device__ void finish_greedy(const FilterArgs& a, int64_t t, const E* row, const E* gm, float M,
                              Shared& sm) {
    constexpr int kGroup = kVecPerLane * Elem<E>::kVec;
    static_assert(kGroup <= kFinThreads, "a thread per column of a group");
    if (threadIdx.x == 0) sm.bin = sm.found = 0xFFFFFFFFu;
    __syncthreads();
    for_each_group<E, kFinThreads>(gm, a.chunks * 32, [&](int i, float g) {
        if (g == M) atomicMin(&sm.bin, (uint32_t)i);
    });
    __syncthreads();
    const uint32_t col = sm.bin * kGroup + threadIdx.x;
    if (threadIdx.x < kGroup && col < (uint32_t)a.V && Elem<E>::to_float(row[col]) == M)
        atomicMin(&sm.found, col);
    __syncthreads();
    if (threadIdx.x == 0) {
        a.token[t] = (int64_t)sm.found;
        a.logprob[t] = 0.f;
    }
}

template <typename E, int kFinThreads, typename Shared>
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
    // Each thread sums its run of columns; the one whose run the target falls
    // into walks through it again.
    constexpr int kVec = Elem<E>::kVec, kChunk = Elem<E>::kChunk;
    constexpr int kPer = kChunk / kFinThreads < kVec ? kVec : kChunk / kFinThreads;
    constexpr int kAhead = kPer / kVec < 2 ? kPer / kVec : 2;
    static_assert(kPer % (kAhead * kVec) == 0, "whole vectors to a thread");
    const int own = (int)threadIdx.x * kPer, col0 = own < kChunk ? chunk * kChunk + own : (int)a.V;
    auto walk = [&](auto each) {
#pragma unroll 1
        for (int i = 0; i < kPer; i += kAhead * kVec) {
            int col[kAhead];
            float x[kAhead][kVec];
#pragma unroll
            for (int h = 0; h < kAhead; ++h) col[h] = col0 + i + h * kVec;
            load_columns<E, kAhead>(row, col, (int)a.V, x);
#pragma unroll
            for (int h = 0; h < kAhead; ++h)
#pragma unroll
                for (int e = 0; e < kVec; ++e) each(col[h] + e, x[h][e], ex2_approx((x[h][e] - M) * c));
        }
    };
    float sum = 0.f;
    walk([&](int, float, float e) { sum += e; });
    float before, unused;
    block_scan<kFinThreads, float>(sm.scratch, sum, 0.f, before, unused);
    float c0 = (chunk ? sm.prefix[chunk - 1] : 0.f) + before;
    if (c0 <= target && target < c0 + sum) {
        const float room = kSumError * total;
        walk([&](int col, float z, float e) {
            const float c1 = c0 + e;
            if (target - c0 > room && c1 - target > room) {  // one column at most
                a.token[t] = col;
                a.logprob[t] = (z - M) / rs.temp - lnS;
                sm.found = 1;
            }
            c0 = c1;
        });
    }
    __syncthreads();
    if (!sm.found) leave_row(a, t);
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
template <int kFinThreads>
__device__ __forceinline__ void nucleus_targets(const FinishRow& r, FinishShared<kFinThreads>& sm) {
    const uint64_t S = __float2ull_rn(r.Sf * __int_as_float((127 + r.scale) << 23));
    const uint64_t target = share_of(r.rs.top_p, S);
    static_assert(kSumError == 1.f / 262144.f, "2^-18");
    const uint64_t error = (target >> 18) + 2;
    sm.target0 = target > error ? target - error : 0;
    sm.target1 = target + error;
}

// Decides a row from at most kFinFew candidates.
template <typename E, bool kSample, int kFinThreads>
__device__ __forceinline__ void finish_few(const FilterArgs& a, const E* row, const FinishRow& r,
                                           FinishShared<kFinThreads>& sm) {
    const int lane = threadIdx.x & 31, n = r.n;
    // `parts` neighbouring lanes share a candidate, each comparing it with its
    // share of the others.
    const int parts = n <= kFinThreads / 8   ? 8
                      : n <= kFinThreads / 4 ? 4
                      : n <= kFinThreads / 2 ? 2
                                             : 1;
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
        if (kSample) sm.draw = draw_of(r.rs.u, before + w);
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

// Sorts n <= kFinCand keys; the places up to the next power of two, which it
// returns, are filled with the largest.  Bitonic, element t + r kFinThreads in
// register r of thread t: a pair is in one thread, in one warp (most steps), or met
// through shared memory.
template <int kFinThreads>
__device__ __noinline__ int block_sort(unsigned long long* key, int n) {
    constexpr int kRegs = kFinCand / kFinThreads;
    const int t = (int)threadIdx.x;
    int size = 64;
    while (size < n) size *= 2;
    unsigned long long v[kRegs];
#pragma unroll
    for (int r = 0; r < kRegs; ++r) v[r] = t + r * kFinThreads < n ? key[t + r * kFinThreads] : ~0ull;
    // This thread's element of the pair whose other element is `other`.
    auto meet = [&](int r, int run, int stride, unsigned long long other) {
        const bool low = !(t & stride), up = !((t + r * kFinThreads) & run);
        if ((other < v[r]) == (low == up)) v[r] = other;
    };
#pragma unroll 1
    for (int run = 2; run <= size; run *= 2)
#pragma unroll 1
        for (int stride = run / 2; stride > 0; stride /= 2) {
            if (stride >= kFinThreads) {
#pragma unroll
                for (int d = 1; d < kRegs; d *= 2)
                    if (stride == d * kFinThreads)
#pragma unroll
                        for (int r = 0; r < kRegs; ++r)
                            if (!(r & d) && ((v[r | d] < v[r]) == !((r * kFinThreads) & run))) {
                                const unsigned long long x = v[r];
                                v[r] = v[r | d];
                                v[r | d] = x;
                            }
            } else if (stride >= 32) {
                __syncthreads();
#pragma unroll
                for (int r = 0; r < kRegs; ++r)
                    if (r * kFinThreads < size) key[t + r * kFinThreads] = v[r];
                __syncthreads();
#pragma unroll
                for (int r = 0; r < kRegs; ++r)
                    if (r * kFinThreads < size)
                        meet(r, run, stride, key[(t ^ stride) + r * kFinThreads]);
            } else {
#pragma unroll
                for (int r = 0; r < kRegs; ++r)
                    if (r * kFinThreads < size)
                        meet(r, run, stride, __shfl_xor_sync(0xFFFFFFFFu, v[r], stride));
            }
        }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRegs; ++r)
        if (r * kFinThreads < size) key[t + r * kFinThreads] = v[r];
    __syncthreads();
    return size;
}

// Decides a row from more candidates: sorted, their ranks are their places and
// the mass before each is a prefix sum; the kept ones are sorted again by index
// for the draw.
template <typename E, bool kSample, int kFinThreads>
__device__ __noinline__ void finish_many(const FilterArgs& a, const E* row, const FinishRow& r,
                                         FinishShared<kFinThreads>& sm) {
    constexpr int kMost = kFinCand / kFinThreads;
    const int lane = threadIdx.x & 31, n = r.n;
    // neighbours, so many to a thread
    const int per = (block_sort<kFinThreads>(sm.cand, n) + kFinThreads - 1) / kFinThreads;
    const int i0 = (int)threadIdx.x * per;
    uint64_t sum = 0, before, unused;
    for (int i = i0; i < i0 + per; ++i) {
        const uint64_t w =
            i < n ? fixed_weight(key_logit((uint32_t)(sm.cand[i] >> 32)), r.M, r.c, r.scale, sm.table)
                  : 0;
        sm.weight[i] = w;
        sum += w;
    }
    block_scan<kFinThreads, uint64_t>(sm.scratch, sum, 0, before, unused);
    const bool whole = r.k > 0 || r.all;  // the whole mass is among the candidates'
    const int most_k = r.k > 0 && r.k < n ? r.k : n;
    if (r.rs.cut_p && !whole && threadIdx.x == 0) nucleus_targets(r, sm);
    uint64_t at = before;
    for (int i = i0; i < i0 + per; ++i) {
        at += sm.weight[i];
        if (i == n - 1) sm.total = at;
        if (r.rs.cut_p && whole && i == most_k - 1) sm.target0 = sm.target1 = share_of(r.rs.top_p, at);
    }
    __syncthreads();
    // How many pass every filter, by the narrow and by the wide bounds.
    int keep = 0, most = 0;
    at = before;
    for (int i = i0; i < i0 + per && i < most_k; ++i) {
        const float z = key_logit((uint32_t)(sm.cand[i] >> 32));
        keep += (!r.rs.cut_m || z >= r.mp.hi) && (!r.rs.cut_p || at < sm.target0);
        most += (!r.rs.cut_m || z >= r.mp.lo) && (!r.rs.cut_p || at < sm.target1);
        at += sm.weight[i];
    }
    keep = __reduce_add_sync(0xFFFFFFFFu, keep);
    most = __reduce_add_sync(0xFFFFFFFFu, most);
    if (lane == 0) {
        atomicAdd(&sm.keep0, (uint32_t)keep);
        atomicAdd(&sm.keep1, (uint32_t)most);
    }
    __syncthreads();
    keep = (int)sm.keep0;
    most = (int)sm.keep1;
    // All candidates kept: then a filter must end here, or there are no others.
    const bool ends = keep < n || r.all || (r.k > 0 && r.k <= n) || r.all_min ||
                      (r.rs.cut_p && sm.total >= sm.target1);
    if (keep == 0 || keep != most || !ends) return leave_row(a, r.t);
    at = before;
    uint64_t ux = 0;
    unsigned long long by_index[kMost];
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
        const int i = i0 + j;
        by_index[j] = ~0ull;
        if (j >= per || i >= keep) continue;
        const unsigned long long key = sm.cand[i];
        const uint64_t w = sm.weight[i];
        at += w;
        if (!kSample) ux += (uint64_t)entropy_term(key, w, r.M, r.rs.temp, r.scale);
        if (i == keep - 1) {
            sm.sum = at;
            sm.cut = key;
            if (kSample) sm.draw = draw_of(r.rs.u, at);
        }
        by_index[j] = key << 32 | (uint32_t)i;
    }
    if (!kSample) {
        ux = warp_sum(ux);
        if (lane == 0 && ux) add_wide(&sm.ux, ux);
        __syncthreads();
        if (threadIdx.x == 0) write_kept(a, row, r, sm.cut, sm.sum, (long long)sm.ux);
        return;
    }
    // The draw: the kept columns in index order.  u = 0 takes the first of
    // them, however small its weight.
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMost; ++j)
        if (j < per && i0 + j < keep) sm.cand[i0 + j] = by_index[j];
    __syncthreads();
    const int draws = (block_sort<kFinThreads>(sm.cand, keep) + kFinThreads - 1) / kFinThreads;
    const int d0 = (int)threadIdx.x * draws;
    sum = 0;
    for (int i = d0; i < d0 + draws && i < keep; ++i) sum += sm.weight[(uint32_t)sm.cand[i]];
    block_scan<kFinThreads, uint64_t>(sm.scratch, sum, 0, before, unused);
    const uint64_t target = sm.draw, S = sm.sum;
    at = before;
    for (int i = d0; i < d0 + draws && i < keep; ++i) {
        const uint64_t w = sm.weight[(uint32_t)sm.cand[i]];
        if (r.rs.u == 0.f ? i == 0 : (at <= target && at + w > target))
            write_token<E, kSample>(a, row, r, (uint32_t)(sm.cand[i] >> 32), S);
        at += w;
    }
}

// kFiltered: some row may have a filter; without, the kernel needs neither the
// registers nor the shared memory of the candidates.
template <typename E, bool kSample, bool kFiltered, int kFinThreads>
__global__ void __launch_bounds__(kFinThreads, (kFiltered ? 1024 : 1536) / kFinThreads)
    filter_finish_kernel(const __grid_constant__ FilterArgs a) {
    __shared__ typename std::conditional<kFiltered, FinishShared<kFinThreads>,
                                         DrawShared<kFinThreads>>::type sm;
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
    const E* gm = static_cast<const E*>(a.group_max) + t * a.chunks * 32;
    if (rs.greedy) return finish_greedy<E, kFinThreads>(a, t, row, gm, M, sm);
    if (!kFiltered || (!rs.cut_k && !rs.cut_p && !rs.cut_m)) {
        const float lnS = unfiltered_log<E, kFinThreads>(row, rec, a.chunks, V, M, Sf, r.c.ch,
                                                         reinterpret_cast<float*>(sm.scratch));
        if (kSample) {
            __syncthreads();  // the histogram's zeros share memory with the prefix sums
            return finish_draw<E, kFinThreads>(a, t, row, rec, M, r.c.ch, rs, lnS, sm);
        }
        if (threadIdx.x == 0)
            write_statistics(a, t, row, M, lnS, lnS - kLn2 * (st.z / Sf), rs.temp, 0xFFFFFFFFu,
                             (uint32_t)V - 1);
        return;
    }
    if constexpr (kFiltered) {

    r.k = rs.cut_k ? (int)rs.top_k : 0;
    r.mp = min_p_bounds(M, rs);
    const bool short_row = V <= kFinShort;
    r.all = V <= kFinFew<kFinThreads>;
    const float bin_scale = r.c.ch * kBinsPerOrder;
    const float ch = r.c.ch;
    auto bin_of = [&](float z) {
        const float y = (M - z) * bin_scale;
        if (y < (float)kFineBins) return __float2int_rd(y);
        // exact: both are multiples of the last place of y
        return kFineBins + min(kFinBins - 1 - kFineBins,
                               __float2int_rd((y - (float)kFineBins) * (1.f / kBinsPerStep)));
    };
    const int groups = a.chunks * 32;
    const int bin_m = rs.cut_m ? bin_of(r.mp.lo) : kFinBins;
    // Columns up to this bin are gathered; the last bin is open.
    int b = kFinBins, n_finite = V;
    __syncthreads();
    if (!r.all && (rs.cut_k || rs.cut_p)) {
        const bool by_mass = rs.cut_p && !rs.cut_k;
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
            for_each_group<E, kFinThreads>(gm, groups, [&](int, float g) { add(g); });
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
        if (threadIdx.x == kFinThreads - 1) sm.found = cb;
        __syncthreads();
        b = (int)sm.bin;
        n_finite = short_row ? (int)sm.found : V;
    }
    // top-p after top-k needs the whole top-k mass, so min-p may not shorten it
    if (!r.all) {
        if (!(rs.cut_k && rs.cut_p)) b = min(b, bin_m);
        if (b >= kFinBins - 1) {
            if (n_finite > kFinCand) return leave_row(a, t);
            r.all = true;
        }
    }
    r.all_min = rs.cut_m && b >= bin_m;

    // ---- gather.  bin_of(z) <= b  <=>  (M - z) bin_scale < edge
    const float edge = r.all          ? INFINITY
                       : b < kFineBins ? (float)(b + 1)
                                       : (float)kFineBins + (float)(b + 1 - kFineBins) * kBinsPerStep;
    const bool direct = r.all || short_row;  // every column, from L1 by now
    int n_vec;                               // vectors of kVec columns to look through
    if (direct) {
        n_vec = (V + kVec - 1) / kVec;
    } else {
        for_each_group<E, kFinThreads>(gm, groups, [&](int i, float g) {
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
            if (direct) {
                col[h] = i * kVec;
            } else {
                const int g = sm.group[min(i, n_vec - 1) / kVecPerLane], j = i % kVecPerLane;
                col[h] = ((g * kVecPerLane) + j) * kVec;  // 32 groups of 16 vectors are a chunk
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
    if (r.n <= kFinFew<kFinThreads>)
        finish_few<E, kSample, kFinThreads>(a, row, r, sm);
    else
        finish_many<E, kSample, kFinThreads>(a, row, r, sm);

    }
}

template <typename E, bool kU>
cudaError_t launch_records(const FilterArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
    static ContextSeen configured;
    const cudaError_t e =
        ensure_smem_optin(reinterpret_cast<const void*>(filter_records_kernel<E, kU>),
                          kWarps * kStages * (int)(kRecordSlot + sizeof(uint64_t)), configured);
    if (e != cudaSuccess) return e;
    // Few items are spread over as many SMs as there are, one warp each at first.
    const int64_t items = a.T * a.chunks;
    int64_t warps = (items + dev.sm_count - 1) / dev.sm_count;
    warps = warps < kWarps ? warps : kWarps;
    int64_t grid = (items + warps - 1) / warps;
    grid = grid < dev.sm_count ? grid : dev.sm_count;
    return launch_behind(filter_records_kernel<E, kU>, (unsigned)grid, (unsigned)warps * 32,
                         (size_t)warps * kStages * (kRecordSlot + sizeof(uint64_t)), stream, 1, a);
}

template <typename E, bool kSample>
cudaError_t launch_filter(FilterArgs a, const DeviceInfo& dev, cudaStream_t stream) {
    // A row without filters takes its entropy from the records; a filtered one
    // from what it keeps.  So sums of e x are formed unless every row is filtered.
    const bool every = (!a.top_ks && a.top_k > 0 && a.top_k < a.V) || (!a.top_ps && a.top_p < 1.f) ||
                       (!a.min_ps && a.min_p > 0.f);
    const bool some = every || a.top_ks || a.top_ps || a.min_ps;
    a.stream_once = a.T * a.V * (int64_t)sizeof(E) > dev.l2_bytes / 2;
    cudaError_t e = kSample || every ? launch_records<E, false>(a, dev, stream)
                                     : launch_records<E, true>(a, dev, stream);
    if (e != cudaSuccess) return e;
    // A row's time is mostly latency, so rows that are all resident at once get as
    // many threads as that leaves each; beyond, registers decide how many an SM holds.
    // 64 rows of V = 151,936, half of them with top-k 200: 256 threads 33 us, 512 25,
    // 1024 23, but then one row with top-k 50 takes 12 us in place of 11.
    const unsigned T = (unsigned)a.T;
    if (!some)
        e = launch_behind(filter_finish_kernel<E, kSample, false, 256>, T, 256, 0, stream, 1, a);
    else if (a.T <= 2 * dev.sm_count)
        e = launch_behind(filter_finish_kernel<E, kSample, true, 512>, T, 512, 0, stream, 1, a);
    else if (a.T <= 4 * dev.sm_count)
        e = launch_behind(filter_finish_kernel<E, kSample, true, 256>, T, 256, 0, stream, 1, a);
    else
        e = launch_behind(filter_finish_kernel<E, kSample, true, 128>, T, 128, 0, stream, 1, a);
    // Without filters only a draw can be left over.
    if (e != cudaSuccess || (!some && !kSample)) return e;
    return launch_exact<E, kSample>(a, some, dev, stream);
}

}  // namespace

cudaError_t launch_row_records(FilterArgs a, pstat_dtype dt, const DeviceInfo& dev,
                               cudaStream_t stream) {
    a.stream_once = a.T * a.V * (dt == PSTAT_BF16 ? 2 : 4) > dev.l2_bytes / 2;
    return dt == PSTAT_BF16 ? launch_records<uint16_t, false>(a, dev, stream)
                            : launch_records<float, false>(a, dev, stream);
}

namespace {

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

}  // extern "C"
