// reorder.cu -- states of the beams follow the beams that a search chose.
//
// Row b K + i of every output becomes row b K' + parents[b, i] of its input.  Bound by
// HBM.  A thread owns a column of 16 bytes (or what alignment leaves of them) through all
// rows of a search.  In place it loads the column of every row's parent before it stores any,
// so that a permutation needs neither a second buffer nor an order; a row that is its own
// parent is neither read nor written.  Into other buffers it goes by rounds of 8 rows, and a
// parent of rows in several rounds is asked for in each.
//
// A warp's parents are one load, a lane each, and known before the first row is loaded: one by
// one they kept each row waiting for the last one's.  Many short CTAs, as what they read
// and write comes in turns.  Four caches of 128 rows x 8 x 1501 x 128 bf16 in place: 8 beams
// 325 us, 6.9 TB/s (430 row by row with 8 CTAs to an SM); 4 beams 350 (540), 16 beams 360
// (545), 32 beams 394 (490), 64 beams 505 (1,265).  Views whose rows or runs start off 16
// bytes move by what they start on: 8 x 1501 (of 1600) x 102 bf16, 4 bytes at a time, 734 us in
// place and 773 into other buffers, x 101, 2 bytes, 1,281 and 1,338, where HBM would do with 275
// and 307.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <memory>
#include <new>

#include "internal.h"
#include "ptx.cuh"

namespace pstat {
namespace {

constexpr int kReThreads = 256;
constexpr int kReTurns = 256;  // most CTAs for each SM
constexpr int kReBatch = 300;  // states of one launch (they travel as its arguments)

struct ReState {
    const char* in;
    char* out;
    int64_t in_row, out_row, in_seg, out_seg;  // strides in bytes
    uint32_t per_seg;                          // vectors of a run
    uint32_t columns;                          // of a row
    uint32_t units;                            // blocks of columns of a search
    uint32_t first_unit;
    uint32_t vec;                              // bytes of a vector
    uint32_t pad;
};
template <int N>
struct ReBatch {
    int count;
    uint32_t units;
    ReState s[N];
};

struct ReArgs {
    const int64_t* parents;
    int64_t B;
    int beams, out_beams;
    bool in_place;
    int* dev_error;
};

// One column of search b, of every lane that `has` one.  All lanes are here: lane l reads the
// l-th parent, and the others ask it for that.
template <typename V, int kRows, bool kClear>
__device__ __forceinline__ void move_column(const ReState& s, const ReArgs& a, const int64_t* parents,
                                            int64_t b, uint32_t col, bool has) {
    const int lane = threadIdx.x & 31;
    const uint32_t seg = col / s.per_seg, at = col - seg * s.per_seg;
    const char* in = after_wait(s.in) + b * a.beams * s.in_row + seg * s.in_seg + (int64_t)at * sizeof(V);
    char* out = s.out + b * a.out_beams * s.out_row + seg * s.out_seg + (int64_t)at * sizeof(V);
    for (int i0 = 0; i0 < a.out_beams; i0 += kRows) {  // once in place: kRows >= out_beams there
        constexpr int kWords = (kRows + 31) / 32;
        int from[kWords];  // -1: the row stays
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const int i = i0 + 32 * w + lane;
            const int64_t p = i < a.out_beams ? parents[i] : -1;
            from[w] = p >= 0 && p < a.beams && !(a.in_place && p == i) ? (int)p : -1;
        }
        int p[kRows];  // all before the first row's load
#pragma unroll
        for (int i = 0; i < kRows; ++i) p[i] = __shfl_sync(0xFFFFFFFFu, from[i / 32], i % 32) | (has ? 0 : -1);
        V x[kRows];
        uint64_t moved = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (p[i] >= 0) {
                moved |= 1ull << i;
                x[i] = *reinterpret_cast<const V*>(in + p[i] * s.in_row);
            }
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (moved >> i & 1) *reinterpret_cast<V*>(out + (int64_t)(i0 + i) * s.out_row) = x[i];
        if constexpr (kClear) {  // rare, and the same rows for all lanes
            static_assert(kRows <= 32, "");
            uint32_t none = __ballot_sync(0xFFFFFFFFu, from[0] < 0 && lane < kRows && i0 + lane < a.out_beams);
            for (; none; none &= none - 1)
                if (has) *reinterpret_cast<V*>(out + (int64_t)(i0 + __ffs(none) - 1) * s.out_row) = V();
        }
    }
}

// kRows: rows whose columns a thread holds at a time, as few as the search allows.  64 of 16
// bytes would be all its registers, so such searches move 8 bytes at a time.  kClear: rows
// without a parent become zeros, and are left as they are otherwise.
template <int N, int kRows, bool kClear>
__global__ void __launch_bounds__(kReThreads, kRows <= 8 ? 4 : kRows <= 16 ? 2 : 1)
    reorder_kernel(const __grid_constant__ ReBatch<N> g, const __grid_constant__ ReArgs a) {
    grid_wait();
    const int64_t* parents = after_wait(a.parents);
    if (blockIdx.x == 0 && a.dev_error) {
        bool bad = false;
        for (int64_t i = threadIdx.x; i < a.B * a.out_beams; i += kReThreads)
            bad |= parents[i] < -1 || parents[i] >= a.beams;
        if (bad) atomicOr(a.dev_error, PSTAT_DEV_BAD_PARAM);
    }
    for (uint32_t u = blockIdx.x; u < g.units; u += gridDim.x) {
        int lo = 0, hi = g.count - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (g.s[mid].first_unit <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        const ReState& s = g.s[lo];
        const uint32_t r = u - s.first_unit;
        const int64_t b = r / s.units;
        const uint32_t col = (r - (uint32_t)b * s.units) * kReThreads + threadIdx.x;
        const bool has = col < s.columns;
        const int64_t* p = parents + b * a.out_beams;
        switch (s.vec) {
            case 16:
                if constexpr (kRows <= 32) move_column<uint4, kRows, kClear>(s, a, p, b, has ? col : 0u, has);
                break;
            case 8:
                move_column<uint2, kRows, kClear>(s, a, p, b, has ? col : 0u, has);
                break;
            case 4: move_column<uint32_t, kRows, kClear>(s, a, p, b, has ? col : 0u, has); break;
            case 2: move_column<uint16_t, kRows, kClear>(s, a, p, b, has ? col : 0u, has); break;
            default: move_column<uint8_t, kRows, kClear>(s, a, p, b, has ? col : 0u, has); break;
        }
    }
}

// What a state covers in memory: rows of runs.
struct Extent {
    uintptr_t from;
    int64_t rows, row, segs, seg, bytes;
    bool written;
    int64_t row_extent() const { return (segs - 1) * seg + bytes; }
    uintptr_t to() const { return from + (uintptr_t)((rows - 1) * row + row_extent()); }
};
// Whether [a, a + na) and [b, b + nb) meet, all positions modulo `period`, na and nb <= period.
bool meet_modulo(uintptr_t a, int64_t na, uintptr_t b, int64_t nb, int64_t period) {
    const uintptr_t p = (uintptr_t)period;
    const uintptr_t ab = (b - a % p + p) % p;  // of b behind a (b >= a in memory is not needed)
    return ab < (uintptr_t)na || ab + (uintptr_t)nb > p;
}
// Whether a's runs miss b's in every period of a's run stride, which divides both row strides:
// b's taken one by one where they have that stride too, else all of a row of b.
bool apart_by_runs(const Extent& a, const Extent& b) {
    if (a.bytes > a.seg || a.row % a.seg || b.row % a.seg) return false;
    const int64_t nb = b.seg == a.seg ? b.bytes : b.row_extent();
    return nb <= a.seg && !meet_modulo(a.from, a.bytes, b.from, nb, a.seg);
}
// Whether two extents overlap.  Exact where they do not reach across each other; where they
// do, they are apart if their rows are (views side by side in the rows of one buffer)
// or their runs (views of a cache's heads), and taken for an overlap otherwise.
bool overlap(const Extent& a, const Extent& b) {
    if (a.to() <= b.from || b.to() <= a.from) return false;
    if (a.row == b.row && a.row_extent() <= a.row && b.row_extent() <= a.row &&
        !meet_modulo(a.from, a.row_extent(), b.from, b.row_extent(), a.row))
        return false;
    return !apart_by_runs(a, b) && !apart_by_runs(b, a);
}

constexpr int64_t kMaxStride = (int64_t)1 << 46;
constexpr uint64_t kMaxUnits = 0xF0000000ull;  // of a launch

// Bytes of the widest vector.  (64 rows of 16 bytes would be all of a thread's registers.)
uint32_t widest_of(bool in_place, int64_t out_beams) { return in_place && out_beams > 32 ? 8 : 16; }

// A state that is not empty as the kernel takes it, first_unit apart; false where its vectors do
// not count in 32 bits.
bool state_of(const pstat_beam_state& p, int64_t B, uint32_t widest, ReState* out) {
    ReState s = {static_cast<const char*>(p.data), static_cast<char*>(p.out), p.row_stride, p.out_row_stride,
                 p.seg_stride, p.out_seg_stride, 0, 0, 0, 0, 0, 0};
    int64_t segments = p.segments, bytes = p.seg_bytes;
    if (segments > 1 && p.seg_stride == bytes && p.out_seg_stride == bytes) bytes *= segments, segments = 1;
    if (segments == 1) s.in_seg = s.out_seg = 0;
    const uint64_t all = reinterpret_cast<uintptr_t>(p.data) | reinterpret_cast<uintptr_t>(p.out) |
                         (uint64_t)(s.in_row | s.out_row | s.in_seg | s.out_seg | bytes);
    const int shift = __builtin_ctzll(all | widest);
    s.vec = 1u << shift;
    const int64_t per_seg = bytes >> shift;
    if (per_seg > 0xFFFFFFFFll || segments * per_seg > 0xFFFFFFFFll - kReThreads) return false;
    s.per_seg = (uint32_t)per_seg;
    s.columns = (uint32_t)(segments * per_seg);
    s.units = (s.columns + kReThreads - 1) / kReThreads;
    *out = s;
    return (uint64_t)s.units * (uint64_t)B <= kMaxUnits;
}

int check_states(const pstat_beam_state* states, int64_t n, const int64_t* parents, int64_t B, int64_t beams,
                 int64_t out_beams, bool* in_place) {
    if (n < 0 || n > (1 << 20) || B < 0 || B > PSTAT_FILTER_MAX_T || beams < 1 || beams > PSTAT_BEAM_MAX ||
        out_beams < 1 || out_beams > PSTAT_BEAM_MAX_N)
        return PSTAT_ERR_SHAPE;
    if (n > 0 && !states) return PSTAT_ERR_NULLPTR;
    if (n == 0 || B == 0) return PSTAT_OK;
    if (!parents) return PSTAT_ERR_NULLPTR;
    if (reinterpret_cast<uintptr_t>(parents) & 7u) return PSTAT_ERR_ALIGN;
    std::unique_ptr<Extent[]> v(new (std::nothrow) Extent[2 * n + 1]);
    if (!v) return PSTAT_ERR_WORKSPACE;
    const int64_t parent_bytes = 8 * B * out_beams;
    v[0] = {reinterpret_cast<uintptr_t>(parents), 1, parent_bytes, 1, parent_bytes, parent_bytes, false};
    int64_t m = 1;
    bool first = true;
    for (int64_t i = 0; i < n; ++i) {
        const pstat_beam_state& s = states[i];
        if (s.segments < 0 || s.seg_bytes < 0 || s.segments > kMaxStride || s.seg_bytes > kMaxStride)
            return PSTAT_ERR_SHAPE;
        if (s.segments == 0 || s.seg_bytes == 0) continue;
        if (!s.data || !s.out) return PSTAT_ERR_NULLPTR;
        if (s.segments > kMaxStride / s.seg_bytes) return PSTAT_ERR_SHAPE;
        for (int64_t stride : {s.row_stride, s.out_row_stride, s.seg_stride, s.out_seg_stride})
            if (stride < 0 || stride > kMaxStride) return PSTAT_ERR_SHAPE;
        // runs of a row, and rows, must not overlap among themselves where they are written
        for (int64_t stride : {s.seg_stride, s.out_seg_stride})
            if (stride > 0 && s.segments - 1 > kMaxStride / stride) return PSTAT_ERR_SHAPE;
        if ((s.row_stride > 0 && B * beams - 1 > kMaxStride / s.row_stride) ||
            (s.out_row_stride > 0 && B * out_beams - 1 > kMaxStride / s.out_row_stride))
            return PSTAT_ERR_SHAPE;
        const int64_t out_extent = (s.segments - 1) * s.out_seg_stride + s.seg_bytes;
        const bool nested = (s.segments == 1 || s.out_seg_stride >= s.seg_bytes) && s.out_row_stride >= out_extent;
        const bool across = s.segments > 1 && s.out_row_stride >= s.seg_bytes &&
                            s.out_seg_stride >= (B * out_beams - 1) * s.out_row_stride + s.seg_bytes;
        if (B * out_beams > 1 ? !(nested || across) : (s.segments > 1 && s.out_seg_stride < s.seg_bytes))
            return PSTAT_ERR_SHAPE;
        const bool same = s.data == s.out;
        if (first) *in_place = same;
        first = false;
        if (same != *in_place) return PSTAT_ERR_PARAM;
        if (same && (beams != out_beams || s.row_stride != s.out_row_stride ||
                     (s.segments > 1 && s.seg_stride != s.out_seg_stride)))
            return PSTAT_ERR_PARAM;
        ReState taken;  // refused before any state is touched
        if (!state_of(s, B, widest_of(same, out_beams), &taken)) return PSTAT_ERR_SHAPE;
        const uintptr_t out = reinterpret_cast<uintptr_t>(s.out), in = reinterpret_cast<uintptr_t>(s.data);
        v[m++] = {out, B * out_beams, s.out_row_stride, s.segments, s.segments > 1 ? s.out_seg_stride : s.seg_bytes,
                  s.seg_bytes, true};
        if (!same)
            v[m++] = {in, B * beams, s.row_stride, s.segments, s.segments > 1 ? s.seg_stride : s.seg_bytes,
                      s.seg_bytes, false};
    }
    std::sort(v.get(), v.get() + m, [](const Extent& a, const Extent& b) { return a.from < b.from; });
    for (int64_t i = 0; i < m; ++i)
        for (int64_t j = i + 1; j < m && v[j].from < v[i].to(); ++j)
            if ((v[i].written || v[j].written) && overlap(v[i], v[j])) return PSTAT_ERR_PARAM;
    return PSTAT_OK;
}

template <int N, int kRows, bool kClear>
int run_rows(const pstat_beam_state* states, int64_t n, const ReArgs& a, const DeviceInfo& dev, cudaStream_t st) {
    const uint32_t widest = widest_of(a.in_place, a.out_beams);
    ReBatch<N> g;
    for (int64_t i = 0; i < n;) {
        g.count = 0;
        uint64_t units = 0;
        for (; i < n && g.count < N; ++i) {
            const pstat_beam_state& p = states[i];
            if (p.segments == 0 || p.seg_bytes == 0) continue;
            ReState s;
            if (!state_of(p, a.B, widest, &s)) return PSTAT_ERR_SHAPE;  // not after check_states
            const uint64_t add = (uint64_t)s.units * (uint64_t)a.B;
            if (units + add > kMaxUnits) break;
            s.first_unit = (uint32_t)units;
            units += add;
            g.s[g.count++] = s;
        }
        g.units = (uint32_t)units;
        if (!g.count) continue;
        const uint32_t most = (uint32_t)dev.sm_count * kReTurns;
        if (launch_behind(reorder_kernel<N, kRows, kClear>, g.units < most ? g.units : most, kReThreads, 0, st, 1, g,
                          a) != cudaSuccess)
            return PSTAT_ERR_CUDA;
    }
    return PSTAT_OK;
}

template <int kRows, bool kClear = false>
int run_states(const pstat_beam_state* states, int64_t n, const ReArgs& a, const DeviceInfo& dev, cudaStream_t st) {
    return n <= 16 ? run_rows<16, kRows, kClear>(states, n, a, dev, st)
                   : run_rows<kReBatch, kRows, kClear>(states, n, a, dev, st);
}

}  // namespace
}  // namespace pstat

using namespace pstat;

static int reorder(const pstat_beam_state* states, int64_t n_states, const int64_t* parents, int64_t B,
                   int64_t beams, int64_t out_beams, bool clear, int* dev_error, pstat_stream_t stream) {
    bool in_place = false;
    int rc = check_states(states, n_states, parents, B, beams, out_beams, &in_place);
    if (rc != PSTAT_OK) return rc;
    if (clear && in_place) return PSTAT_ERR_PARAM;
    if (n_states == 0 || B == 0) return PSTAT_OK;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != PSTAT_OK) return rc;
    const ReArgs a = {parents, B, (int)beams, (int)out_beams, in_place, dev_error};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (clear) return run_states<8, true>(states, n_states, a, dev, st);
    if (!in_place || out_beams <= 8) return run_states<8>(states, n_states, a, dev, st);
    if (out_beams <= 16) return run_states<16>(states, n_states, a, dev, st);
    if (out_beams <= 32) return run_states<32>(states, n_states, a, dev, st);
    return run_states<64>(states, n_states, a, dev, st);
}

extern "C" {

int pstat_beam_reorder(const pstat_beam_state* states, int64_t n_states, const int64_t* parents, int64_t B,
                       int64_t beams, int64_t out_beams, int* dev_error, pstat_stream_t stream) {
    return reorder(states, n_states, parents, B, beams, out_beams, false, dev_error, stream);
}

int pstat_beam_gather(const pstat_beam_state* states, int64_t n_states, const int64_t* parents, int64_t B,
                      int64_t beams, int64_t out_beams, int* dev_error, pstat_stream_t stream) {
    return reorder(states, n_states, parents, B, beams, out_beams, true, dev_error, stream);
}

}  // extern "C"
