// beams.cu -- the next beams of a search over beams and vocabulary.
//
// Continuation (k, v) scores (z_kv - M_k) + d_k, d_k = score_k - ln S_k.  The records
// kernel of the sampler reads the logits once and leaves, per chunk, maximum and sum, and
// per 256 bytes of columns (a group) their maximum.  beam_finish_kernel, a CTA for a
// search, does the rest on those:
//
//   1. M_k and d_k from the records, a warp for each beam;
//   2. every thread takes a run of neighbouring groups (of all beams, in order) and its
//      best score.  The n best continuations lie in the n runs that are best by (score,
//      place): a run with n better ones before it has n continuations before its own;
//   3. for the same reason in the n best groups of those runs,
//   4. and those groups, n x 256 bytes, are read again for the n best of their columns.
//
// So at most n runs, groups and n x 128 columns are ever sorted, whatever the logits are
// (all equal, say), and ties go by place throughout.
//
// Scores are compared as pairs of floats, in 64-bit keys.  z - M is exact as a pair, so a
// row's offset, which its softmax does not depend on, costs no digits; the roundings of low
// words, in d and in adding it, are 2^-46 (|score| + 2 |score_k| + 28) at most (28 for ln S of
// 2^20 columns).  d_k also carries the error of the fp32 sum S.  Where two continuations of
// different beams lie closer than that, in or at the end of the list, the S of both beams is
// summed anew from exact weights (ln S to 2^-40, filter_math.cuh), and the choice is made
// again; scores of one beam differ by its logits alone and need none.
// Bound by the records, hence by HBM, for a batch of searches (64 of 16 beams over 151,936
// bf16 columns: 65 us, 311 MB at 4.8 TB/s, of which the records are 48 us); by latency for
// one (4 beams: 15 us, the records 5).  A search where two beams of 151,936 columns have to be
// summed anew takes 135 us more.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "sampling.cuh"

namespace pstat {
namespace {

constexpr int kBmKeep = PSTAT_BEAM_MAX_N;  // places of the list that is carried along
// Error of d_k: kSumError of S, and logf's of 1 ulp of at most ln 2^20 (2^-20).
constexpr float kBmError = 0x1.8p-18f;
static_assert(kBmError >= kSumError + 0x1p-20f, "");
static_assert(PSTAT_BEAM_MAX <= 64, "rows of a search in a 64-bit mask");

struct BeamArgs {
    FilterArgs f;  // logits, records, group maxima
    int beams, n;
    const float* scores;
    float* out_score;
    int64_t* out_parent;
    int64_t* out_token;
};

struct Entry {
    uint64_t key;  // 0: none
    uint32_t at;   // place: among ties the lower one comes first
};
__device__ __forceinline__ bool before(const Entry& a, const Entry& b) {
    return a.key > b.key || (a.key == b.key && a.at < b.at);
}

// A pair of floats, hi the sum of both rounded.
struct Pair {
    float hi, lo;
};
// a + b, exactly.
__device__ __forceinline__ Pair exact_sum(float a, float b) {
    const float s = __fadd_rn(a, b);
    const float t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
// a + b to about 2^-47 (|a| + |b|).
__device__ __forceinline__ Pair pair_sum(const Pair& a, const Pair& b) {
    const Pair s = exact_sum(a.hi, b.hi);
    const float l = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo));
    const float hi = __fadd_rn(s.hi, l);
    return {hi, __fsub_rn(l, __fsub_rn(hi, s.hi))};
}
// What the scores of a beam's continuations are formed from.
struct Base {
    Pair d;  // score - ln S
    float M;
};
__device__ __forceinline__ uint32_t ordered(float x) {  // ascending; +-0 alike
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ (uint32_t)(((int32_t)b >> 31) | (int32_t)0x80000000);
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
// 0 (no continuation) for what is masked, and for what lies below fp32's range: z - M of a mask
// of the type's lowest value can, and its sum with such a score.  The low words are NaN then,
// and so is the sum.
__device__ __forceinline__ uint64_t score_key(const Base& b, float z) {
    const Pair s = pair_sum(exact_sum(z, -b.M), b.d);
    if (!(s.hi > -INFINITY)) return 0;
    return (uint64_t)ordered(s.hi) << 32 | ordered(s.lo);
}
__device__ __forceinline__ Pair key_score(uint64_t key) {
    return {unordered((uint32_t)(key >> 32)), unordered((uint32_t)key)};
}
// a - b, which lie close.
__device__ __forceinline__ float pair_gap(uint64_t a, uint64_t b) {
    const Pair x = key_score(a), y = key_score(b);
    return (x.hi - y.hi) + (x.lo - y.lo);
}

template <int kThreads>
struct BeamShared {
    static constexpr int kNew = kThreads - kBmKeep;  // candidates of one round of sorting
    Base base[PSTAT_BEAM_MAX];
    float S[PSTAT_BEAM_MAX];
    uint64_t key[kThreads];
    uint32_t at[kThreads];
    Entry list[kBmKeep];       // what the last selection kept, best first
    uint32_t picked[kBmKeep];  // places of it
    uint64_t cand_key[kNew];
    uint32_t cand_at[kNew];
    int n_cand;
    int bad;
    unsigned long long doubtful;  // beams to be summed anew
    unsigned long long sum[kThreads / 32];
    float2 table[64];
};

__device__ __forceinline__ Entry shuffle_xor(const Entry& e, int m) {
    return {__shfl_xor_sync(0xFFFFFFFFu, e.key, m), __shfl_xor_sync(0xFFFFFFFFu, e.at, m)};
}
// One step of a bitonic sort among lanes: the better entry goes to the lower lane
// where `up` is set.
__device__ __forceinline__ void exchange(Entry& e, int m, bool up, int lane) {
    const Entry o = shuffle_xor(e, m);
    const bool low = (lane & m) == 0;
    if (before(o, e) == (low == up)) e = o;
}
__device__ __forceinline__ void warp_sort(Entry& e, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int m = size / 2; m; m /= 2) exchange(e, m, size == 32 || (lane & size) == 0, lane);
}

// The best `n` of the first `count` threads' entries, in order, in sm.list.  Up to 32: sorted
// warps whose lists of 32 are merged, two by two; beyond, all are sorted.
template <int kThreads>
__device__ __noinline__ void keep_best(BeamShared<kThreads>& sm, Entry e, int n, int count) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int warps = 1;
    while (warps * 32 < count) warps *= 2;
    if (warp < warps) warp_sort(e, lane);
    if (n <= 32) {
        if (warp < warps) {
            sm.key[threadIdx.x] = e.key;
            sm.at[threadIdx.x] = e.at;
        }
        for (int left = warps / 2; left; left /= 2) {
            __syncthreads();
            Entry a = {0, 0};
            if (warp < left) {
                const int i = 64 * warp + lane, j = 64 * warp + 63 - lane;
                a = {sm.key[i], sm.at[i]};
                const Entry b = {sm.key[j], sm.at[j]};
                if (before(b, a)) a = b;
#pragma unroll
                for (int m = 16; m; m /= 2) exchange(a, m, true, lane);
            }
            __syncthreads();
            if (warp < left) {
                sm.key[32 * warp + lane] = a.key;
                sm.at[32 * warp + lane] = a.at;
            }
        }
    } else {
        // Sorted warps alternate in direction from here on, as a bitonic sort wants them.
        const int total = warps * 32;
        if ((warp & 1) && warp < warps)
            e = {__shfl_sync(0xFFFFFFFFu, e.key, 31 - lane), __shfl_sync(0xFFFFFFFFu, e.at, 31 - lane)};
        for (int size = 64; size <= total; size *= 2) {
            const bool up = size == total || (threadIdx.x & size) == 0;
            for (int m = size / 2; m >= 32; m /= 2) {
                __syncthreads();
                sm.key[threadIdx.x] = e.key;
                sm.at[threadIdx.x] = e.at;
                __syncthreads();
                const int j = threadIdx.x ^ m;
                const Entry o = {sm.key[j], sm.at[j]};
                if (before(o, e) == (((threadIdx.x & m) == 0) == up)) e = o;
            }
            if (warp < warps)
#pragma unroll
                for (int m = 16; m; m /= 2) exchange(e, m, up, lane);
        }
        __syncthreads();
        sm.key[threadIdx.x] = e.key;
        sm.at[threadIdx.x] = e.at;
    }
    __syncthreads();
    if (threadIdx.x < kBmKeep) {
        const bool in = (int)threadIdx.x < n && (int)threadIdx.x < warps * 32;
        const Entry got = in ? Entry{sm.key[threadIdx.x], sm.at[threadIdx.x]} : Entry{0, 0xFFFFFFFFu};
        sm.list[threadIdx.x] = got;
        sm.picked[threadIdx.x] = got.key ? got.at : 0xFFFFFFFFu;
    }
    __syncthreads();
}

// The best n of `count` candidates in sm.list.  `visit(emit)` calls emit(entry, i) for
// all of them that this thread owns, i being the candidate's number; those that are not
// below `least` are gathered, and sorted at once where there is room, else by rounds.
template <int kThreads, typename Visit>
__device__ __forceinline__ void select_best(BeamShared<kThreads>& sm, int n, int count, uint64_t least, Visit visit) {
    constexpr int kNew = BeamShared<kThreads>::kNew;
    if (threadIdx.x == 0) sm.n_cand = 0;
    __syncthreads();
    const uint64_t floor = max(least, (uint64_t)1);
    visit([&](const Entry& e, int) {
        if (e.key < floor) return;
        const int at = atomicAdd(&sm.n_cand, 1);
        if (at < kNew) {
            sm.cand_key[at] = e.key;
            sm.cand_at[at] = e.at;
        }
    });
    __syncthreads();
    const int found = sm.n_cand;
    if (found <= kNew) {
        Entry e = {0, 0xFFFFFFFFu};
        if ((int)threadIdx.x < found) e = {sm.cand_key[threadIdx.x], sm.cand_at[threadIdx.x]};
        keep_best(sm, e, n, found);
        return;
    }
    // What `visit` reads of the list before (sm.picked) has to last through the rounds.
    Entry kept = {0, 0xFFFFFFFFu};
    const uint32_t picked = threadIdx.x < kBmKeep ? sm.picked[threadIdx.x] : 0u;
    for (int i0 = 0; i0 < count; i0 += kNew) {
        __syncthreads();
        if (threadIdx.x < kBmKeep) sm.picked[threadIdx.x] = picked;
        if ((int)threadIdx.x < kNew) sm.cand_key[threadIdx.x] = 0;
        __syncthreads();
        visit([&](const Entry& e, int i) {
            if (i >= i0 && i < i0 + kNew) {
                sm.cand_key[i - i0] = e.key;
                sm.cand_at[i - i0] = e.at;
            }
        });
        __syncthreads();
        Entry e = kept;
        if ((int)threadIdx.x < kNew)
            e = sm.cand_key[threadIdx.x] ? Entry{sm.cand_key[threadIdx.x], sm.cand_at[threadIdx.x]}
                                         : Entry{0, 0xFFFFFFFFu};
        keep_best(sm, e, n, kThreads);
        if ((int)threadIdx.x >= kNew) kept = sm.list[threadIdx.x - kNew];
    }
}

// ln S of a beam's row from exact weights: every thread of the CTA.
template <typename E, int kThreads>
__device__ __noinline__ void sum_anew(BeamShared<kThreads>& sm, const BeamArgs& a, const E* row, int k,
                                      float score) {
    const float M = sm.base[k].M;
    const int scale = fixed_scale(sm.S[k] * (1.f + 2.f * kSumError));
    const TempScale one = temp_scale(1.f);
    constexpr int kVec = Elem<E>::kVec;
    unsigned long long sum = 0;
    for (int c = (int)threadIdx.x * kVec; c < (int)a.f.V; c += kThreads * kVec) {
        const int col[1] = {c};
        float x[1][kVec];
        load_columns<E, 1>(row, col, (int)a.f.V, x);
#pragma unroll 1
        for (int e = 0; e < kVec; e += 2) {
            uint64_t w0, w1;
            fixed_weights(x[0][e], x[0][e + 1], M, one, scale, sm.table, w0, w1);
            sum += w0 + w1;
        }
    }
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) sm.sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0;
        for (int w = 0; w < kThreads / 32; ++w) sum += sm.sum[w];
        const double lnS = log((double)sum) - scale * 0.69314718055994530942;
        const float hi = (float)lnS;
        sm.base[k].d = pair_sum({score, 0.f}, {-hi, -(float)(lnS - (double)hi)});
    }
    __syncthreads();
}

template <typename E, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) beam_finish_kernel(const __grid_constant__ BeamArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    using Shared = BeamShared<kThreads>;
    Shared& sm = *reinterpret_cast<Shared*>(raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int beams = a.beams, n = a.n, V = (int)a.f.V, chunks = a.f.chunks;
    constexpr int kVec = Elem<E>::kVec;
    constexpr int kGroup = Elem<E>::kChunk / 32;  // columns
    const int64_t b = blockIdx.x, t0 = b * beams;
    if (threadIdx.x == 0) sm.bad = 0;
    if (threadIdx.x < 64) sm.table[threadIdx.x] = kExp2Table[threadIdx.x];
    __syncthreads();
    grid_wait();
    const float* scores = after_wait(a.scores) + t0;
    const float4* records = after_wait(a.f.records) + t0 * chunks;
    const E* maxima = static_cast<const E*>(after_wait(a.f.group_max)) + t0 * chunks * 32;
    const E* logits = static_cast<const E*>(after_wait(a.f.logits)) + t0 * a.f.ld;

    for (int k = warp; k < beams; k += kThreads / 32) {
        const float s = scores[k];
        const float3 r = fold_records(records + (int64_t)k * chunks, chunks, kLog2e, lane);
        if (lane == 0) {
            Pair d = {-INFINITY, 0.f};
            if (!(s < INFINITY))
                sm.bad = 1;
            else if (s > -INFINITY) {
                if (!(r.x < INFINITY))
                    sm.bad = 1;
                else if (r.x > -INFINITY)
                    d = exact_sum(s, -logf(r.y));
            }
            sm.base[k] = {d, r.x};
            sm.S[k] = r.y;
        }
    }
    __syncthreads();
    float* out_score = a.out_score + b * n;
    int64_t* out_parent = a.out_parent + b * n;
    int64_t* out_token = a.out_token + b * n;
    if (sm.bad) {
        if ((int)threadIdx.x < n) {
            out_score[threadIdx.x] = NAN;
            out_parent[threadIdx.x] = out_token[threadIdx.x] = -1;
        }
        if (threadIdx.x == 0 && a.f.dev_error) atomicOr(a.f.dev_error, PSTAT_DEV_EMPTY_ROW);
        return;
    }

    const int groups = chunks * 32;  // of a row
    const int total = beams * groups;
    const int run = ((total + kThreads - 1) / kThreads + 7) / 8 * 8;
    // The maxima of 8 groups from g, a multiple of 8: of one row, whose groups are a
    // multiple of 32.
    auto load8 = [&](int g, float (&x)[8]) {
        const uint4* p = reinterpret_cast<const uint4*>(maxima + g);
        if constexpr (sizeof(E) == 2) {
            RowReader<E>::unpack(p[0], x);
        } else {
            float y[4];
            RowReader<E>::unpack(p[0], y);
            x[0] = y[0], x[1] = y[1], x[2] = y[2], x[3] = y[3];
            RowReader<E>::unpack(p[1], y);
            x[4] = y[0], x[5] = y[1], x[6] = y[2], x[7] = y[3];
        }
    };
    const int g0 = min(total, (int)threadIdx.x * run), g1 = min(total, g0 + run), k0 = g0 / groups;
    // Calls f(maxima, their first group, beam) for this thread's run.
    auto each_of_run = [&](auto f) {
        int k = k0;
        for (int g = g0; g < g1; g += 8) {
            float x[8];
            load8(g, x);
            k += g >= (k + 1) * groups;
            f(x, g, k);
        }
    };
    constexpr int kVecs = kGroup / kVec;
    // Calls f(columns' logits, their first column, beam, candidate number) for this thread's
    // share of the picked groups.
    auto each_of_groups = [&](auto f) {
        for (int i = threadIdx.x; i < n * kVecs; i += kThreads) {
            const uint32_t g = sm.picked[i / kVecs];
            if (g == 0xFFFFFFFFu) continue;
            const int k = (int)g / groups;
            const int col[1] = {((int)g - k * groups) * kGroup + i % kVecs * kVec};
            if (col[0] >= V) continue;
            float x[1][kVec];
            load_columns<E, 1>(logits + (int64_t)k * a.f.ld, col, V, x);
            f(x[0], col[0], k, kVec * i);
        }
    };
    unsigned long long exact = 0;  // beams that were summed anew
    while (true) {
        Entry mine = {0, 0xFFFFFFFFu};
        each_of_run([&](const float(&x)[8], int, int k) {
            const float m = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                                  fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
            const uint64_t key = score_key(sm.base[k], m);
            if (key > mine.key) mine = {key, threadIdx.x};
        });
        keep_best(sm, mine, n, kThreads);
        // groups of those runs
        const int eights = run / 8;
        select_best(sm, n, n * run, sm.list[n - 1].key, [&](auto emit) {
            for (int i = threadIdx.x; i < n * eights; i += kThreads) {
                const uint32_t r = sm.picked[i / eights];
                const int g = r == 0xFFFFFFFFu ? total : (int)r * run + i % eights * 8;
                if (g >= total) continue;
                float x[8];
                load8(g, x);
                const Base c = sm.base[g / groups];
#pragma unroll
                for (int q = 0; q < 8; ++q) emit(Entry{score_key(c, x[q]), (uint32_t)(g + q)}, 8 * i + q);
            }
        });
        // columns of those groups, whose list is wanted again below
        const uint32_t picked = threadIdx.x < kBmKeep ? sm.picked[threadIdx.x] : 0u;
        select_best(sm, n, n * kGroup, sm.list[n - 1].key, [&](auto emit) {
            each_of_groups([&](const float(&x)[kVec], int col, int k, int i) {
#pragma unroll
                for (int q = 0; q < kVec; ++q)
                    emit(Entry{score_key(sm.base[k], x[q]), (uint32_t)(k * V + col + q)}, i + q);
            });
        });
        if (beams == 1) break;
        // Beams whose sums' errors could change the list.
        if (threadIdx.x == 0) sm.doubtful = 0;
        if (threadIdx.x < kBmKeep) sm.picked[threadIdx.x] = picked;
        __syncthreads();
        const uint64_t last = sm.list[n - 1].key;  // 0: every continuation is in the list
        constexpr float kTol = 2.f * kBmError;
        auto doubt = [&](unsigned long long rows_a, int row) {
            unsigned long long others = rows_a & ~(1ull << row);
            if (exact >> row & 1) others &= ~exact;
            if (others) atomicOr(&sm.doubtful, (others | 1ull << row) & ~exact);
        };
        if ((int)threadIdx.x + 1 < n) {
            const Entry x = sm.list[threadIdx.x], y = sm.list[threadIdx.x + 1];
            if (y.key && pair_gap(x.key, y.key) <= kTol) doubt(1ull << (x.at / (uint32_t)V), (int)(y.at / (uint32_t)V));
        }
        if (last) {
            unsigned long long border = 0;  // beams of the list's end
            for (int i = n - 1; i >= 0 && pair_gap(sm.list[i].key, last) <= kTol; --i)
                border |= 1ull << (sm.list[i].at / (uint32_t)V);
            auto outside = [&](uint64_t key, int row) {
                if (key && key <= last && pair_gap(last, key) <= kTol) doubt(border, row);
            };
            if (mine.key && (mine.key >= last || pair_gap(last, mine.key) <= kTol))
                each_of_run([&](const float(&x)[8], int, int k) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) outside(score_key(sm.base[k], x[q]), k);
                });
            each_of_groups([&](const float(&x)[kVec], int, int k, int) {
#pragma unroll
                for (int q = 0; q < kVec; ++q) outside(score_key(sm.base[k], x[q]), k);
            });
        }
        __syncthreads();
        const unsigned long long rows = sm.doubtful;
        __syncthreads();
        if (!rows) break;
        for (int k = 0; k < beams; ++k)
            if (rows >> k & 1) sum_anew<E>(sm, a, logits + (int64_t)k * a.f.ld, k, scores[k]);
        exact |= rows;
    }
    if ((int)threadIdx.x < n) {
        const Entry e = sm.list[threadIdx.x];
        out_score[threadIdx.x] = e.key ? key_score(e.key).hi : -INFINITY;
        out_parent[threadIdx.x] = e.key ? (int64_t)(e.at / (uint32_t)V) : -1;
        out_token[threadIdx.x] = e.key ? (int64_t)(e.at % (uint32_t)V) : -1;
    }
}

struct BeamWorkspace {
    size_t group_max, spare, total;  // records first
};
BeamWorkspace beam_workspace(int64_t T, int64_t V, pstat_dtype dt) {
    const int64_t chunk = dt == PSTAT_BF16 ? PSTAT_CHUNK_BF16 : PSTAT_CHUNK_F32;
    const size_t items = (size_t)T * (size_t)((V + chunk - 1) / chunk);
    BeamWorkspace w;
    w.group_max = align_up(items * kChunkRecordBytes, 256);
    w.spare = align_up(w.group_max + items * 32 * (dt == PSTAT_BF16 ? 2 : 4), 256);
    w.total = w.spare + 16;
    return w;
}

int check_beams(pstat_dtype dt, int64_t B, int64_t beams, int64_t V) {
    if (dt != PSTAT_F32 && dt != PSTAT_BF16) return PSTAT_ERR_DTYPE;
    if (B < 0 || beams < 1 || beams > PSTAT_BEAM_MAX || V < 1 || V > kFilterMaxV ||
        B > PSTAT_FILTER_MAX_T / beams)
        return PSTAT_ERR_SHAPE;
    return PSTAT_OK;
}

template <typename E, int kThreads>
cudaError_t launch_finish(const BeamArgs& a, unsigned B, cudaStream_t st) {
    static ContextSeen configured;
    const cudaError_t e = ensure_smem_optin(reinterpret_cast<const void*>(beam_finish_kernel<E, kThreads>),
                                            (int)sizeof(BeamShared<kThreads>), configured);
    if (e != cudaSuccess) return e;
    return launch_behind(beam_finish_kernel<E, kThreads>, B, kThreads, sizeof(BeamShared<kThreads>), st, 1, a);
}

// A search's time is latency: sorting the threads' best takes longer with more of them,
// reading the maxima with fewer.  Where 256 threads have 8 maxima each at most (and the
// list leaves room for its candidates) they take 13.0 us a call against 15.1 with 1024 (33
// searches, 3 beams of 10,007); with 64 searches of 8 beams of 152,064 it is 48 against 39.
template <typename E>
cudaError_t launch_finish_of(const BeamArgs& a, unsigned B, cudaStream_t st) {
    if (a.n <= 32 && (int64_t)a.beams * a.f.chunks * 32 <= 256 * 8) return launch_finish<E, 256>(a, B, st);
    return launch_finish<E, 1024>(a, B, st);
}

}  // namespace
}  // namespace pstat

using namespace pstat;

extern "C" {

int pstat_beam_workspace_size(int64_t B, int64_t beams, int64_t V, pstat_dtype dt, size_t* bytes) {
    if (!bytes) return PSTAT_ERR_NULLPTR;
    const int rc = check_beams(dt, B, beams, V);
    if (rc != PSTAT_OK) return rc;
    *bytes = beam_workspace(B * beams, V, dt).total;
    return PSTAT_OK;
}

int pstat_beam_select(const void* logits, pstat_dtype dt, int64_t B, int64_t beams, int64_t V, int64_t ld,
                      const float* scores, int64_t n, float* out_score, int64_t* out_parent,
                      int64_t* out_token, void* workspace, size_t ws_bytes, int* dev_error,
                      pstat_stream_t stream) {
    int rc = check_beams(dt, B, beams, V);
    if (rc != PSTAT_OK) return rc;
    if ((ld < V && ld != 0) || n < 1 || n > PSTAT_BEAM_MAX_N) return PSTAT_ERR_SHAPE;
    if (B == 0) return PSTAT_OK;
    if (!logits || !scores || !out_score || !out_parent || !out_token) return PSTAT_ERR_NULLPTR;
    if (!aligned(logits, dt == PSTAT_BF16 ? 2 : 4) || !aligned(scores, 4) || !aligned(out_score, 4) ||
        !aligned(out_parent, 8) || !aligned(out_token, 8))
        return PSTAT_ERR_ALIGN;
    const BeamWorkspace w = beam_workspace(B * beams, V, dt);
    if (!workspace || ws_bytes < w.total) return PSTAT_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return PSTAT_ERR_ALIGN;
    // A search's scores are read by the CTA that writes its results, before it writes them.
    const bool in_place = out_score == scores && n == beams;
    const struct {
        const void* p;
        int64_t bytes;
        bool written;
    } range[] = {{workspace, (int64_t)w.total, true},
                 {out_score, B * n * 4, true},
                 {out_parent, B * n * 8, true},
                 {out_token, B * n * 8, true},
                 {logits, extent_bytes(B * beams, ld, V, dt == PSTAT_BF16 ? 2 : 4), false},
                 {scores, in_place ? 0 : B * beams * 4, false}};
    for (int i = 0; i < 6; ++i)
        for (int j = i + 1; j < 6; ++j)
            if (range[i].written && ranges_meet(range[i].p, range[i].bytes, range[j].p, range[j].bytes))
                return PSTAT_ERR_PARAM;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != PSTAT_OK) return rc;
    char* ws = static_cast<char*>(workspace);
    BeamArgs a = {};
    a.f.logits = logits;
    a.f.T = B * beams;
    a.f.V = V;
    a.f.ld = ld;
    a.f.chunks = (int)((V + (dt == PSTAT_BF16 ? PSTAT_CHUNK_BF16 : PSTAT_CHUNK_F32) - 1) /
                       (dt == PSTAT_BF16 ? PSTAT_CHUNK_BF16 : PSTAT_CHUNK_F32));
    a.f.temperature = 1.f;
    a.f.records = reinterpret_cast<float4*>(ws);
    a.f.group_max = ws + w.group_max;
    a.f.left_count = reinterpret_cast<int*>(ws + w.spare);
    a.f.dev_error = dev_error;
    a.beams = (int)beams;
    a.n = (int)n;
    a.scores = scores;
    a.out_score = out_score;
    a.out_parent = out_parent;
    a.out_token = out_token;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_row_records(a.f, dt, dev, st);
    if (e != cudaSuccess) return PSTAT_ERR_CUDA;
    e = dt == PSTAT_BF16 ? launch_finish_of<uint16_t>(a, (unsigned)B, st)
                         : launch_finish_of<float>(a, (unsigned)B, st);
    return e == cudaSuccess ? PSTAT_OK : PSTAT_ERR_CUDA;
}

}  // extern "C"
