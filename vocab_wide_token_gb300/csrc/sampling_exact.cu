// sampling_exact.cu -- the rows of the sampler and of the filtered statistics
// that fp32 sums or a short list of candidates do not decide: nuclei of
// thousands of tokens, large top_k, draws close to a border, masses of equal
// logits.
//
// A cluster of CTAs (a team) goes over the row again.  Its first CTA, the
// leader, decides; the others wait for its commands, each a pass over the row
// shared out over the team.  A row with a nucleus takes two passes: one counts
// the logits in 2048 bins of M - z, one weighs every column exactly, by spans
// of the index order, and collects the columns of the bin that the cut is
// expected in.  A cluster barrier takes 1 to 2 thousand cycles and a pass over
// 151,936 columns by ten CTAs some 15 thousand, so decisions that only the leader
// needs stay with it.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "sampling.cuh"

namespace cg = cooperative_groups;

namespace pstat {
namespace {

constexpr int kExThreads = 512;
constexpr int kExWarps = kExThreads / 32;
constexpr int kBins = 2048;    // bins of one histogram level
constexpr int kCand = 2048;    // elements of a list
constexpr int kSpan = 256;     // columns of one span of the index order, a warp's
constexpr int kLane = kSpan / 32;
constexpr int kMaxSpans = (int)(kFilterMaxV / kSpan);
constexpr int kSpansPer = kMaxSpans / kExThreads;
// One CTA per SM: with two the CTAs of a few rows crowd on half of the SMs, and
// the registers do not suffice for the weights (8 flat rows of V = 151,936 with
// top_p = 0.9: 61 us a call, with one 43).  Ten CTAs a team, as two such teams fill the 20
// SMs of a processing cluster, where two of eight leave four idle (16 clusters of
// ten or thirty of five are resident, 14 of eight).
constexpr int kMaxTeam = 10;
// With kAlone rows or more for every cluster the CTAs take rows alone: what a
// team saves in a pass it loses again in synchronisation.  Flat rows of
// V = 151,936 with top_p = 0.9, a call with all by teams or all alone: 12 rows 44 /
// 150 us, 32 rows 148 / 148.
constexpr int kAlone = 2;
static_assert(kBins % kExThreads == 0 && kMaxSpans % kExThreads == 0 && kSpan <= kExThreads, "");

enum Op : uint32_t {
    kDone,       // the row is finished
    kCount,      // level-0 histogram; how many logits are finite, and pass min-p
    kWeigh,      // masses below, in and above the keys [lo, hi]; collect those inside
    kNarrow,     // histogram of the keys [lo, hi] in steps of 2^arg
    kTies,       // by spans, the logits with key lo
    kSpans,      // by spans, the mass of what the cut (lo, hi) keeps
    kLowest      // the first column that it keeps
};
struct Command {
    uint32_t op, lo, hi, arg;
};

struct ExactShared {
    uint32_t level0[kBins];
    uint32_t inside[kBins];  // where in the bin they lie, summed, in steps of 2^-11
    union {
        struct {
            uint32_t count[kBins];
            unsigned long long mass[kBins];
        };
        ListShared<kExThreads> list;
    };
    unsigned long long cand[kCand];
    unsigned long long weight[kCand];
    unsigned long long span[kMaxSpans];
    float2 table[64];
    unsigned long long scratch[2 * kExWarps];
    unsigned long long sums[3][kExWarps];
    unsigned long long part[kMaxTeam][3];  // the leader's: sums of every CTA
    Command command[2];                    // the leader's, by turns
    uint32_t n_cand, first, lowest, offset;
    uint32_t bin, n_in, count_before, klo, khi, edge;
    float z_min;
    unsigned long long mass_before, shift, wide;
    Selected sel;
};

template <typename E, bool kSample>
struct Team {
    ExactShared& sm;
    ExactShared& lead;  // the leader's
    const E* row;
    int V, rank, size;  // CTAs of the team; one alone needs no cluster
    uint32_t turn;      // commands so far
    RowSettings rs;
    float M, Sf, z_min, bin_scale;
    TempScale c;
    int k;              // digits of the fixed weights

    __device__ void sync() const {
        if (size == 1)
            __syncthreads();
        else
            cg::this_cluster().sync();
    }
    __device__ uint64_t weight(float z) const { return fixed_weight(z, M, c, k, sm.table); }
    // Level-0 bins: equal steps of M - z, the last one open (the difference
    // and the product round monotonely, so bins are ranges of the order).
    __device__ int bin0(float z) const { return min(kBins - 1, __float2int_rd((M - z) * bin_scale)); }

    // f(span, this lane's first column of it, its logits): a warp goes through
    // a span together, kLane neighbouring columns to a lane; columns past V are
    // -inf.
    template <typename F>
    __device__ __forceinline__ void each_span(F f) const {
        constexpr int kVec = Elem<E>::kVec, kVecs = kLane / kVec;
        const int lane = threadIdx.x & 31, warps = size * kExWarps;
        const bool even = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
        auto fetch = [&](int s, uint4 (&raw)[kVecs]) {
#pragma unroll
            for (int h = 0; h < kVecs; ++h) {
                const int col = s * kSpan + lane * kLane + h * kVec;
                if (even && col + kVec <= V) raw[h] = __ldg(reinterpret_cast<const uint4*>(row + col));
            }
        };
        int s = rank * kExWarps + ((int)threadIdx.x >> 5);
        uint4 next[kVecs];
        fetch(s, next);
        for (; s * kSpan < V; s += warps) {
            const int col0 = s * kSpan + lane * kLane;
            float x[kLane];
#pragma unroll
            for (int h = 0; h < kVecs; ++h) {
                float part[kVec];
                RowReader<E>::unpack(next[h], part);
#pragma unroll
                for (int e = 0; e < kVec; ++e) x[h * kVec + e] = part[e];
            }
            fetch(s + warps, next);
            if (!even || col0 + kLane > V) {
#pragma unroll
                for (int e = 0; e < kLane; ++e)
                    x[e] = col0 + e < V ? Elem<E>::to_float(row[col0 + e]) : -INFINITY;
            }
            f(s, col0, x);
        }
    }

    // Three values per thread, summed over the CTA into the leader's part[rank].
    __device__ void put(uint64_t v0, uint64_t v1, uint64_t v2) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        v0 = warp_sum(v0);
        v1 = warp_sum(v1);
        v2 = warp_sum(v2);
        if (lane == 0) {
            sm.sums[0][warp] = v0;
            sm.sums[1][warp] = v1;
            sm.sums[2][warp] = v2;
        }
        __syncthreads();
        if (warp < 3) {
            const uint64_t all = warp_sum(lane < kExWarps ? sm.sums[warp][lane] : 0);
            if (lane == 0) lead.part[rank][warp] = all;
        }
    }
    // Leader, after the pass: the team's sum, in every thread.
    __device__ uint64_t get(int which) const {
        const int lane = threadIdx.x & 31;
        return warp_sum(lane < size ? sm.part[lane][which] : 0);
    }

    // ---- passes, by every CTA of the team --------------------------------------
    __device__ __forceinline__ void pass_count() const {
        if (rank) {
            for (int i = threadIdx.x; i < kBins; i += kExThreads) sm.level0[i] = sm.inside[i] = 0;
            __syncthreads();
        }
        uint32_t n_min = 0, n_finite = 0;
        each_span([&](int, int, const float (&x)[kLane]) {
#pragma unroll
            for (int e = 0; e < kLane; ++e)
                if (x[e] > -INFINITY) {
                    const int b = bin0(x[e]);
                    const float in = (M - x[e]) * bin_scale - (float)b;
                    atomicAdd(&sm.level0[b], 1u);
                    atomicAdd(&sm.inside[b], (uint32_t)__float2int_rn(fminf(in, 1.f) * 2048.f));
                    n_min += x[e] >= z_min;
                    ++n_finite;
                }
        });
        put(n_finite, n_min, 0);
        if (rank)
            for (int i = threadIdx.x; i < kBins; i += kExThreads)
                if (sm.level0[i]) {
                    atomicAdd(&lead.level0[i], sm.level0[i]);
                    atomicAdd(&lead.inside[i], sm.inside[i]);
                }
    }

    __device__ __forceinline__ void pass_weigh(uint32_t klo, uint32_t khi, bool all) const {
        if (rank) {
            if (threadIdx.x == 0) sm.n_cand = 0;
            __syncthreads();
        }
        uint64_t total = 0, inside = 0, ux = 0;
        each_span([&](int s, int col, const float (&x)[kLane]) {
            bool any = all;
#pragma unroll
            for (int e = 0; e < kLane; ++e) any |= desc_key(x[e]) <= khi;
            uint64_t before = 0;
            uint32_t hits = 0;
            if (__any_sync(0xFFFFFFFFu, any)) {
#pragma unroll
                for (int e = 0; e < kLane; e += 2) {
                    uint64_t w[2];
                    fixed_weights(x[e], x[e + 1], M, c, k, sm.table, w[0], w[1]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t dk = desc_key(x[e + h]);
                        total += w[h];
                        before += dk < klo ? w[h] : 0;
                        const bool in = dk >= klo && dk <= khi;
                        inside += in ? w[h] : 0;
                        hits |= (uint32_t)in << (e + h);
                        if (!kSample && dk < klo)
                            ux += (uint64_t)entropy_term((unsigned long long)dk << 32, w[h], M, rs.temp, k);
                    }
                }
                before = warp_sum(before);
            }
            if ((threadIdx.x & 31) == 0) lead.span[s] = before;
            if (hits) {
                uint32_t at = atomicAdd(&sm.n_cand, (uint32_t)__popc(hits));
#pragma unroll 1
                for (; hits; hits &= hits - 1, ++at)
                    if (at < (uint32_t)kCand) {
                        const int c0 = col + __ffs(hits) - 1;
                        sm.cand[at] =
                            ((unsigned long long)desc_key(Elem<E>::to_float(row[c0])) << 32) | (uint32_t)c0;
                    }
            }
        });
        put(inside, total, ux);
        if (rank) {  // the leader's own candidates are in place
            if (threadIdx.x == 0) sm.offset = atomicAdd(&lead.n_cand, sm.n_cand);
            __syncthreads();
            const uint32_t n = min(sm.n_cand, (uint32_t)kCand), to = sm.offset;
            for (uint32_t i = threadIdx.x; i < n && to + i < (uint32_t)kCand; i += kExThreads)
                lead.cand[to + i] = sm.cand[i];
        }
    }

    __device__ __forceinline__ void pass_narrow(uint32_t klo, uint32_t khi, int shift) const {
        if (rank) {
            for (int i = threadIdx.x; i < kBins; i += kExThreads) sm.count[i] = 0, sm.mass[i] = 0;
            __syncthreads();
        }
        each_span([&](int, int col, const float (&x)[kLane]) {
            uint32_t hits = 0;
#pragma unroll
            for (int e = 0; e < kLane; ++e)
                hits |= (uint32_t)(desc_key(x[e]) >= klo && desc_key(x[e]) <= khi) << e;
#pragma unroll 1
            for (; hits; hits &= hits - 1) {
                const float z = Elem<E>::to_float(row[col + __ffs(hits) - 1]);
                const uint32_t i = (desc_key(z) - klo) >> shift;
                atomicAdd(&sm.count[i], 1u);
                add_wide(&sm.mass[i], weight(z));
            }
        });
        if (rank) {
            __syncthreads();
            for (int i = threadIdx.x; i < kBins; i += kExThreads)
                if (sm.count[i]) {
                    atomicAdd(&lead.count[i], sm.count[i]);
                    add_wide(&lead.mass[i], sm.mass[i]);
                }
        }
    }

    __device__ __forceinline__ void pass_ties(uint32_t key) const {
        each_span([&](int s, int, const float (&x)[kLane]) {
            uint32_t n = 0;
#pragma unroll
            for (int e = 0; e < kLane; ++e) n += desc_key(x[e]) == key;
            n = __reduce_add_sync(0xFFFFFFFFu, n);
            if ((threadIdx.x & 31) == 0) lead.span[s] = n;
        });
    }

    __device__ __forceinline__ void pass_spans(uint32_t cut_key, uint32_t cut_index) const {
        uint64_t ux = 0;
        each_span([&](int s, int col, const float (&x)[kLane]) {
            uint64_t sum = 0;
#pragma unroll
            for (int e = 0; e < kLane; e += 2) {
                uint64_t w[2];
                fixed_weights(x[e], x[e + 1], M, c, k, sm.table, w[0], w[1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool kept = is_kept(x[e + h], col + e + h, cut_key, cut_index);
                    sum += kept ? w[h] : 0;
                    if (!kSample && kept)
                        ux += (uint64_t)entropy_term((unsigned long long)desc_key(x[e + h]) << 32, w[h],
                                                     M, rs.temp, k);
                }
            }
            sum = warp_sum(sum);
            if ((threadIdx.x & 31) == 0) lead.span[s] = sum;
        });
        if (!kSample) put(0, 0, ux);
    }

    __device__ __forceinline__ void pass_lowest(uint32_t cut_key, uint32_t cut_index) const {
        uint32_t low = 0xFFFFFFFFu;
        each_span([&](int, int col, const float (&x)[kLane]) {
#pragma unroll
            for (int e = 0; e < kLane; ++e)
                if (x[e] > -INFINITY && is_kept(x[e], col + e, cut_key, cut_index))
                    low = min(low, (uint32_t)(col + e));
        });
        low = __reduce_min_sync(0xFFFFFFFFu, low);
        if ((threadIdx.x & 31) == 0) atomicMin(&lead.lowest, low);
    }

    // On a copy, which stays in registers: the passes write memory that could be
    // *this.
    __device__ __noinline__ void run(const Command cmd) const {
        const Team t = *this;
        switch (cmd.op) {
            case kCount: t.pass_count(); break;
            case kWeigh: t.pass_weigh(cmd.lo, cmd.hi, cmd.arg != 0); break;
            case kNarrow: t.pass_narrow(cmd.lo, cmd.hi, (int)cmd.arg); break;
            case kTies: t.pass_ties(cmd.lo); break;
            case kSpans: t.pass_spans(cmd.lo, cmd.hi); break;
            case kLowest: t.pass_lowest(cmd.lo, cmd.hi); break;
            default: break;
        }
    }

    // Everyone but the leader.  The commands alternate between two places, so
    // that the leader cannot overwrite one that is still being read.
    __device__ void follow() {
        while (true) {
            sync();
            const Command cmd = lead.command[turn++ & 1u];
            if (cmd.op == kDone) return;
            run(cmd);
            sync();
        }
    }

    // ---- the leader -------------------------------------------------------------
    __device__ void command(Op op, uint32_t lo = 0, uint32_t hi = 0, uint32_t arg = 0) {
        const Command cmd = {op, lo, hi, arg};
        // what the pass adds to
        if (op == kCount)
            for (int i = threadIdx.x; i < kBins; i += kExThreads) sm.level0[i] = sm.inside[i] = 0;
        if (op == kNarrow)
            for (int i = threadIdx.x; i < kBins; i += kExThreads) sm.count[i] = 0, sm.mass[i] = 0;
        if (threadIdx.x == 0) {
            if (op == kWeigh) sm.n_cand = 0;
            if (op == kLowest) sm.lowest = 0xFFFFFFFFu;
            sm.command[turn & 1u] = cmd;
        }
        ++turn;
        sync();
        if (op == kDone) return;
        run(cmd);
        sync();
    }

    // The bin in which the count reaches `want` (by_count) or the mass `target`;
    // what lies before it and inside, in sm.
    __device__ uint32_t pick_bin(const uint32_t* count, const unsigned long long* mass,
                                 bool by_count, uint32_t want, uint64_t target,
                                 uint32_t count_before, uint64_t mass_before) const {
        constexpr int kPer = kBins / kExThreads;
        const int b0 = threadIdx.x * kPer;
        uint64_t n = 0, w = 0;
        for (int i = 0; i < kPer; ++i) {
            n += count[b0 + i];
            w += mass ? mass[b0 + i] : 0;
        }
        uint64_t nb, wb;
        block_scan<kExThreads, uint64_t>(sm.scratch, n, w, nb, wb);
        nb += count_before;
        wb += mass_before;
        for (int i = 0; i < kPer; ++i) {
            const uint64_t n1 = nb + count[b0 + i], w1 = wb + (mass ? mass[b0 + i] : 0);
            if (by_count ? (nb < want && want <= n1) : (wb < target && w1 >= target)) {
                sm.bin = b0 + i;
                sm.n_in = count[b0 + i];
                sm.count_before = (uint32_t)nb;
                sm.mass_before = wb;
            }
            nb = n1;
            wb = w1;
        }
        __syncthreads();
        return sm.bin;
    }

    // Around the last of the level-0 bins [lo, hi] before which the estimated mass is
    // below `target`.  A bin's mass is estimated by its count times the weight
    // of its logits' mean (its middle alone is 1.1% off for the few that weigh
    // most, which made one guess in four miss; the mean 2^-15); `anchor`, if not negative, is a bin before which the mass is known.
    struct Bins {
        uint32_t first, last, count_before, n_in;
    };
    __device__ Bins guess_bins(uint64_t target, int lo, int hi, int anchor, uint64_t known) const {
        constexpr int kPer = kBins / kExThreads;
        const int b0 = threadIdx.x * kPer;
        const float one = __int_as_float((127 + k) << 23);
        uint64_t n = 0, w = 0, part[kPer];
        for (int i = 0; i < kPer; ++i) {
            n += sm.level0[b0 + i];
            const float count = (float)sm.level0[b0 + i];
            const float mean = count > 0.f ? (float)sm.inside[b0 + i] / (count * 2048.f) : 0.f;
            part[i] = (uint64_t)(count * exp2f(-((float)(b0 + i) + mean) * (64.f / kBins)) * one);
            w += part[i];
        }
        uint64_t nb, wb;
        block_scan<kExThreads, uint64_t>(sm.scratch, n, w, nb, wb);
        if (threadIdx.x == 0) {
            sm.bin = (uint32_t)lo;
            if (anchor < 0) sm.shift = 0;
        }
        uint64_t at = wb;
        for (int i = 0; i < kPer; ++i) {
            if (b0 + i == anchor) sm.shift = known - at;  // modulo 2^64
            at += part[i];
        }
        __syncthreads();
        at = wb + sm.shift;
        for (int i = 0; i < kPer; ++i) {
            if (b0 + i > lo && b0 + i <= hi && (int64_t)(at - target) < 0 && sm.level0[b0 + i])
                atomicMax(&sm.bin, (uint32_t)(b0 + i));
            at += part[i];
        }
        __syncthreads();
        const uint32_t b = sm.bin;
        at = wb + sm.shift;
        for (int i = 0; i < kPer; ++i) {
            if ((uint32_t)(b0 + i) == b) {
                sm.count_before = (uint32_t)nb;
                // where in its mass the target is expected: near the start, the end
                sm.edge = (target - at) * 8 < part[i] ? 1 : (target - at) * 8 > part[i] * 7 ? 2 : 0;
            }
            nb += sm.level0[b0 + i];
            at += part[i];
        }
        __syncthreads();
        // There the guess takes the neighbour in, as a miss costs a pass.
        Bins g = {b, b, sm.count_before, sm.level0[b]};
        const uint32_t edge = sm.edge;
        if (edge == 2 && (int)b < hi && g.n_in + sm.level0[b + 1] <= (uint32_t)kCand)
            g.n_in += sm.level0[++g.last];
        if (edge == 1 && (int)b > lo && g.n_in + sm.level0[b - 1] <= (uint32_t)kCand) {
            g.n_in += sm.level0[--g.first];
            g.count_before -= sm.level0[g.first];
        }
        return g;
    }

    // The keys of the level-0 bins [first, last], in sm.klo and sm.khi.
    __device__ void bin_range(uint32_t first, uint32_t last) const {
        if (threadIdx.x < 2) {
            // Smallest key whose bin is >= first (thread 0) and > last (thread 1):
            // near the key of M - edge/bin_scale, or wherever a bisection finds it.
            const int edge = (int)(threadIdx.x ? last + 1 : first);
            uint32_t lo = desc_key(M), hi = kKeyNegInf;  // answer in [lo, hi]
            const uint32_t near = desc_key(M - (float)edge / bin_scale);
            if (near > lo + 64 && near + 64 < hi) {
                if (bin0(key_logit(near - 64)) < edge) lo = near - 63;
                if (bin0(key_logit(near + 64)) >= edge) hi = near + 64;
            }
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
                sm.khi = last == kBins - 1 ? kKeyNegInf - 1 : lo - 1;
        }
        __syncthreads();
    }

    // Masses before and inside the keys [klo, khi] and of the whole row (if asked
    // for), the candidates inside with their weights.
    struct Weighed {
        uint64_t before, inside, total;
    };
    __device__ __noinline__ Weighed weigh(uint32_t klo, uint32_t khi, bool all) {
        command(kWeigh, klo, khi, all);
        uint64_t before = 0;
        for (int i = threadIdx.x; i * kSpan < V; i += kExThreads) before += sm.span[i];
        before = warp_sum(before);
        if ((threadIdx.x & 31) == 0) sm.scratch[threadIdx.x >> 5] = before;
        const int n = min((int)sm.n_cand, kCand);
        for (int i = threadIdx.x; i < n; i += kExThreads)
            sm.weight[i] = weight(key_logit((uint32_t)(sm.cand[i] >> 32)));
        __syncthreads();
        const int lane = threadIdx.x & 31;
        before = warp_sum(lane < kExWarps ? sm.scratch[lane] : 0);
        const uint64_t in = get(0), total = get(1);
        __syncthreads();
        return {before, in, total};
    }
    // The element at which the count reaches `want`, or the mass `target`, in
    // the order of the finite logits, all of which level0 counts.  With `share`
    // the target is that share of the whole mass, which this takes as well;
    // `target` is then an estimate.  Afterwards, unless `ties` says that too many
    // equal logits came in between, the spans hold the mass of what is kept and
    // `ux` its sum of e x.
    __device__ __noinline__ Selected select(bool by_count, uint32_t want, uint64_t target, float share,
                               bool& ties, uint64_t& ux) {
        Bins g;
        if (by_count) {
            const uint32_t b = pick_bin(sm.level0, nullptr, true, want, 0, 0, 0);
            g = {b, b, sm.count_before, sm.n_in};
        } else {
            g = guess_bins(target, 0, kBins - 1, -1, 0);
        }
        bin_range(g.first, g.last);
        uint32_t klo = sm.klo, khi = sm.khi;
        Weighed m = weigh(klo, khi, share > 0.f);
        if (!by_count) {
            if (share > 0.f) target = share_of(share, m.total);
            // A guess that missed narrows the bins that are left, so this ends.
            int lo = 0, hi = kBins - 1;
            while (true) {
                if (m.before >= target && (int)g.first > lo)
                    hi = (int)g.first - 1;
                else if (m.before + m.inside < target && (int)g.last < hi)
                    lo = (int)g.last + 1;
                else
                    break;
                g = guess_bins(target, lo, hi, (int)g.first, m.before);
                bin_range(g.first, g.last);
                klo = sm.klo;
                khi = sm.khi;
                m = weigh(klo, khi, false);
            }
        }
        uint32_t n_in = g.n_in, count_before = g.count_before;
        uint64_t mass_before = m.before;
        bool narrowed = false;
        // every round leaves 1/2048 of the keys at most
        for (int round = 0; round < 4 && n_in > (uint32_t)kCand &&
                            (klo >> kGrain<E>) != (khi >> kGrain<E>);
             ++round) {
            narrowed = true;
            int shift = 0;
            while (((khi - klo) >> shift) >= (uint32_t)kBins) ++shift;
            command(kNarrow, klo, khi, (uint32_t)shift);
            const uint32_t i =
                pick_bin(sm.count, sm.mass, by_count, want, target, count_before, mass_before);
            klo += i << shift;
            khi = min(khi, klo + ((1u << shift) - 1u));
            n_in = sm.n_in;
            count_before = sm.count_before;
            mass_before = sm.mass_before;
            __syncthreads();
        }
        ties = n_in > (uint32_t)kCand;
        if (ties) return select_tie(klo, by_count, want, target, n_in, count_before, mass_before);
        if (narrowed) {
            m = weigh(klo, khi, false);
            mass_before = m.before;
        }
        const int n = min((int)sm.n_cand, kCand);
        ux = get(2);
        const Selected f = list_select<kExThreads>(
            sm.list, sm.cand, sm.weight, n, (unsigned long long)klo << 32,
            (unsigned long long)khi << 32 | 0xFFFFFFFFu, false, by_count, want, target,
            count_before, mass_before, kGrain<E>);
        // what is kept of the candidates joins the spans
        if (threadIdx.x == 0) sm.wide = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kExThreads) {
            if (sm.cand[i] > f.key) continue;
            const uint64_t w = sm.weight[i];
            add_wide(&sm.span[(uint32_t)sm.cand[i] / kSpan], w);
            if (!kSample) add_wide(&sm.wide, (uint64_t)entropy_term(sm.cand[i], w, M, rs.temp, k));
        }
        __syncthreads();
        ux += sm.wide;
        __syncthreads();
        return f;
    }

    // Many equal logits: how many of them are taken follows from their common
    // weight; the last one taken is found by counting them in index order.
    __device__ Selected select_tie(uint32_t klo, bool by_count, uint32_t want, uint64_t target,
                                   uint32_t n_in, uint32_t count_before, uint64_t mass_before) {
        // The one key in [klo, khi]: a bf16 logit's ends in ones where it is not
        // negative, in zeros where it is.
        const uint32_t low = (1u << kGrain<E>) - 1u;
        const uint32_t key = klo & 0x80000000u ? klo & ~low : klo | low;
        command(kTies, key);
        const uint64_t w = weight(key_logit(key));
        uint32_t take = n_in;
        if (by_count)
            take = want - count_before;
        else if (w)
            take = (uint32_t)((target - mass_before + w - 1) / w);
        uint64_t n = 0, nb, unused;
        for (int i = 0; i < kSpansPer; ++i) {
            const int s = kSpansPer * (int)threadIdx.x + i;
            n += s * kSpan < V ? sm.span[s] : 0;
        }
        block_scan<kExThreads, uint64_t>(sm.scratch, n, 0, nb, unused);
        if (threadIdx.x == 0) sm.first = 0;
        __syncthreads();
        for (int i = 0; i < kSpansPer; ++i) {
            const int s = kSpansPer * (int)threadIdx.x + i;
            n = s * kSpan < V ? sm.span[s] : 0;
            if (nb < take && take <= nb + n) {
                sm.first = (uint32_t)s;
                sm.offset = (uint32_t)nb;
            }
            nb += n;
        }
        __syncthreads();
        const int col = (int)sm.first * kSpan + (int)threadIdx.x;
        const uint32_t skipped = sm.offset;
        const bool hit = (int)threadIdx.x < kSpan && col < V &&
                         desc_key(Elem<E>::to_float(row[col])) == key;
        block_scan<kExThreads, uint64_t>(sm.scratch, hit ? 1 : 0, 0, nb, unused);
        if (hit && skipped + nb + 1 == take)
            sm.sel = {(unsigned long long)key << 32 | (uint32_t)col, count_before + take,
                      mass_before + (uint64_t)take * w};
        __syncthreads();
        const Selected f = sm.sel;
        __syncthreads();
        return f;
    }
    __device__ void lead_row(const FilterArgs& a, int64_t t) {
        uint32_t cut_key = 0xFFFFFFFFu, cut_index = (uint32_t)V - 1;
        bool spans_ready = false;
        uint64_t ux = 0;
        if (rs.cut_k || rs.cut_p || (rs.cut_m && !kSample)) {
            command(kCount);
            const uint32_t n_finite = (uint32_t)get(0);
            const uint32_t n_min = rs.cut_m ? (uint32_t)get(1) : n_finite;
            uint32_t want = rs.cut_k && rs.top_k < (int64_t)n_finite ? (uint32_t)rs.top_k : n_finite;
            Selected sel;
            bool have = false, ties = false;
            if (rs.cut_p) {
                if (want < n_finite) {
                    const uint64_t total = select(true, want, 0, 0.f, ties, ux).mass;
                    sel = select(false, 0, share_of(rs.top_p, total), 0.f, ties, ux);
                } else {
                    const float about = rs.top_p * Sf * __int_as_float((127 + k) << 23);
                    sel = select(false, 0, (uint64_t)about, rs.top_p, ties, ux);
                }
                want = sel.rank;
                have = n_min >= want;
            }
            if (!have) sel = select(true, min(want, n_min), 0, 0.f, ties, ux);
            spans_ready = !ties;
            cut_key = (uint32_t)(sel.key >> 32);
            cut_index = (uint32_t)sel.key;
        } else if (rs.cut_m) {
            cut_key = desc_key(z_min);
        }
        if (!spans_ready) {
            command(kSpans, cut_key, cut_index);
            if (!kSample) ux = get(2);
        }
        if (kSample && rs.u == 0.f) command(kLowest, cut_key, cut_index);
        command(kDone);

        // From here on the leader is alone with the row.
        uint64_t mine = 0, before, unused;
        for (int i = 0; i < kSpansPer; ++i) {
            const int s = kSpansPer * (int)threadIdx.x + i;
            mine += s * kSpan < V ? sm.span[s] : 0;
        }
        block_scan<kExThreads, uint64_t>(sm.scratch, mine, 0, before, unused);
        if (threadIdx.x == kExThreads - 1) {
            const uint64_t S = before + mine;
            sm.mass_before = S;
            // C > u S in whole numbers
            sm.wide = kSample ? draw_of(rs.u, S) : 0;
        }
        if (threadIdx.x == 0) sm.first = 0;
        __syncthreads();
        const uint64_t S = sm.mass_before, target = sm.wide;
        // Without filters ln S is the finish kernel's, so that its bits do not hang
        // on which of the two decided the row.
        const bool cut = rs.cut_k || rs.cut_p || rs.cut_m;
        const float lnS = cut ? fixed_log(S, k)
                              : unfiltered_log<E, kExThreads>(row, a.records + t * a.chunks, a.chunks, V,
                                                              M, Sf, c.ch,
                                                              reinterpret_cast<float*>(sm.scratch));
        if (!kSample) {
            if (threadIdx.x == 0) {
                const float U = (float)(long long)ux * 5.6843419e-14f;  // 2^-44
                const float Sr = (float)S * __int_as_float((127 - k) << 23);
                write_statistics(a, t, row, M, lnS, lnS - U / Sr, rs.temp, cut_key, cut_index);
            }
            return;
        }
        if (rs.u == 0.f) {  // the first kept column, however small its weight
            if (threadIdx.x == 0) {
                const uint32_t col = min(sm.lowest, (uint32_t)V - 1);
                a.token[t] = col;
                a.logprob[t] = (Elem<E>::to_float(row[col]) - M) / rs.temp - lnS;
            }
            return;
        }
        __syncthreads();
        for (int i = 0; i < kSpansPer; ++i) {
            const int s = kSpansPer * (int)threadIdx.x + i;
            const uint64_t w = s * kSpan < V ? sm.span[s] : 0;
            if (before <= target && before + w > target) {
                sm.first = (uint32_t)s;
                sm.mass_before = before;
            }
            before += w;
        }
        __syncthreads();
        const int col = (int)sm.first * kSpan + (int)threadIdx.x;
        const uint64_t base = sm.mass_before;
        uint64_t w = 0;
        float z = 0.f;
        if ((int)threadIdx.x < kSpan && col < V) {
            z = Elem<E>::to_float(row[col]);
            if (is_kept(z, col, cut_key, cut_index)) w = weight(z);
        }
        uint64_t wb;
        block_scan<kExThreads, uint64_t>(sm.scratch, w, 0, wb, unused);
        wb += base;
        if (wb <= target && wb + w > target) {
            a.token[t] = col;
            a.logprob[t] = (z - M) / rs.temp - lnS;
        }
    }
};

template <typename E, bool kSample>
__global__ void __launch_bounds__(kExThreads, 1)
    filter_exact_kernel(const __grid_constant__ FilterArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    ExactShared& sm = *reinterpret_cast<ExactShared*>(smem_raw);
    cg::cluster_group cluster = cg::this_cluster();
    if (threadIdx.x < 64) sm.table[threadIdx.x] = kExp2Table[threadIdx.x];
    __syncthreads();
    grid_wait();
    const int n = *a.left_count;
    if (n == 0) return;
    const int clusters = (int)(gridDim.x / cluster.num_blocks());
    const int size = n >= kAlone * clusters ? 1 : (int)cluster.num_blocks();
    const int rank = size == 1 ? 0 : (int)cluster.block_rank();
    ExactShared& lead = size == 1 ? sm : *cluster.map_shared_rank(&sm, 0);
    uint32_t turn = 0;
    for (int i = blockIdx.x / size; i < n; i += gridDim.x / size) {
        const int64_t t = a.left[i];
        const RowSettings rs = row_settings<kSample>(a, t);
        const TempScale c = temp_scale(rs.temp);
        const float3 st = fold_records(a.records + t * a.chunks, a.chunks, c.ch, threadIdx.x & 31);
        const float M = st.x + 0.f;
        float z_min = -INFINITY;
        if (rs.cut_m) {  // in fp64, so by one thread
            if (threadIdx.x == 0) sm.z_min = min_p_logit(M, rs);
            __syncthreads();
            z_min = sm.z_min;
        }
        Team<E, kSample> team{sm, lead, static_cast<const E*>(a.logits) + t * a.ld, (int)a.V, rank,
                              size, turn, rs, M, st.y, z_min,
                              c.ch * ((float)kBins / 64.f), c,
                              fixed_scale(st.y * (1.f + 2.f * kSumError))};
        if (rank == 0)
            team.lead_row(a, t);
        else
            team.follow();
        turn = team.turn;
        __syncthreads();  // the next row writes what this one reads
    }
    if (size > 1) cluster.sync();  // the leaders' shared memory stays until all have read it
}

}  // namespace

template <typename E, bool kSample>
cudaError_t launch_exact(const FilterArgs& a, bool filtered, const DeviceInfo& dev,
                         cudaStream_t stream) {
    static ContextSeen smem_set, cluster_set;
    const void* fn = reinterpret_cast<const void*>(filter_exact_kernel<E, kSample>);
    cudaError_t e = ensure_smem_optin(fn, (int)sizeof(ExactShared), smem_set);
    if (e == cudaSuccess) e = ensure_large_cluster(fn, cluster_set);
    if (e != cudaSuccess) return e;
    // A row without filters takes one pass, over which synchronisation weighs
    // more; of many such rows more are worked on at once by smaller teams (28 of
    // 2048 rows: 25 us, by teams of ten 33).
    const int most = filtered || a.T <= 64 ? kMaxTeam : kMaxTeam / 2;
    const int64_t want = (a.V + 8191) / 8192;
    const int team = (int)(want < most ? want : most);
    int64_t teams = dev.sm_count / team;
    if (teams > a.T) teams = a.T;
    if (teams < 1) teams = 1;
    return launch_behind(filter_exact_kernel<E, kSample>, (unsigned)(teams * team), kExThreads,
                         sizeof(ExactShared), stream, (unsigned)team, a);
}

template cudaError_t launch_exact<uint16_t, true>(const FilterArgs&, bool, const DeviceInfo&,
                                                cudaStream_t);
template cudaError_t launch_exact<uint16_t, false>(const FilterArgs&, bool, const DeviceInfo&,
                                                cudaStream_t);
template cudaError_t launch_exact<float, true>(const FilterArgs&, bool, const DeviceInfo&,
                                                cudaStream_t);
template cudaError_t launch_exact<float, false>(const FilterArgs&, bool, const DeviceInfo&,
                                                cudaStream_t);

}  // namespace pstat
