// kv_rows.cuh — what attention of few query rows is made of, whichever way the
// cache holds its numbers (kv_rows.cu, kv4_rows.cu): the line of work and its
// pieces, query fragments, and the joining of what warps and CTAs have summed.
//
// An item is the rows (at most 16) of one sequence and key/value head. Decoding has few
// items and long key axes, so items are cut along the keys: the batch's work
// is one line of units of keys, items one after another, and each CTA of a
// resident grid takes an equal piece of it (a few whole items and a part of
// one at either end, whatever the sequences' lengths). An item that lies in
// several CTAs leaves one partial result for each in the workspace, and the
// CTA that comes last, by the item's counter, joins them in the order of the
// keys: no second launch, and the same bits whichever CTA is last. The counter
// is left at zero for the next call.
//
// The format, `F`, is a class of the cache's numbers for heads of up to F::kDim columns:
//   kWarps                       of a CTA
//   kSlice, kStages              keys of a warp's step, steps of its ring
//   kFixed                       units that an item's beginning and end count as, besides its keys
//   resident<NT>()               CTAs of an SM
//   kEarly                       launched so that it may begin as the kernel before it ends
//   kMergeInRing                 warps' rows meet in their rings
//   kUnits                       contributions have a unit of their own (else d is 0, and looked at nowhere)
//   Maps, Stage, Warp            its tensor maps, a step's memory, and what a warp keeps besides
//   look_up, fetch               where steps are, and asking for one
//   attend_slices                a warp's steps of a piece of work
#pragma once

#include <algorithm>
#include <atomic>
#include <cfloat>

#include "kv_attend.cuh"

namespace zc {
namespace kv {
namespace {

// Parts that are joined at a time, where there are more than twice as many: 57 parts of a long sequence at once made its
// call 58 us, in two steps 52; for 16 parts the second step costs what it saves.
constexpr int kGroup = 8;

template <int DP> struct Merge {  // 8 rows of a warp
    float o[8][DP + 4];
    float m[8], d[8], l[8];
};

// A part of an item: rows in units of 2^(m + d) (o) and 2^m (l).
template <int DP, int NT> struct Part {
    float o[8 * NT][DP];
    float m[8 * NT], d[8 * NT], l[8 * NT];
};

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
// The 8x8 matrix of halves whose rows the quads hold, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// Units of work of a sequence's items (the same for all of them).
template <class F> constexpr int kUnit = F::kWarps * F::kSlice;  // keys of a unit of work
template <class F> __device__ __forceinline__ uint32_t first_unit(const AttendArgs &a, const Seq &q) {
    const int pos = q.len - int(q.n);
    return a.window && pos >= int(a.window) ? uint32_t(pos - int(a.window) + 1) / kUnit<F> : 0;
}
template <class F> __device__ __forceinline__ uint32_t units_of(const AttendArgs &a, const Seq &q) {
    return max((uint32_t(q.len) + kUnit<F> - 1) / kUnit<F>, first_unit<F>(a, q) + 1) - first_unit<F>(a, q);
}
template <class F, int NT> __device__ __forceinline__ uint64_t work_of(const AttendArgs &a, const Seq &q) {
    return q.ok && q.n * a.group <= a.rows_most ? uint64_t((q.n * a.group + 8 * NT - 1) / (8 * NT)) * a.c.heads * (F::kFixed + units_of<F>(a, q)) : 0;
}

// A piece of work: units of item (seq, tile, h) on the line of work, and what
// this warp does of it.
struct Job {
    Seq seq;
    uint32_t tile, h;
    uint64_t w, upto, i0, i1;          // the piece [w, upto) of the item's keys [i0, i1)
    int all_lo, all_hi, x_lo, x_hi;    // keys seen by some row; by every row
    int first, steps;                  // this warp's slices: first, first + kWarps, ...
    __device__ __forceinline__ bool whole() const { return w == i0 && upto == i1; }
};

// The piece of work at w, whose sequence's work begins at `at` (both moved on).
template <class F, int NT>
__device__ __forceinline__ bool next_job(const AttendArgs &a, uint64_t &w, uint64_t w1, uint32_t &s, uint64_t &at, Job &job) {
    constexpr int kWarps = F::kWarps;
    while (w < w1) {
        const Seq seq = read_seq(a.b, s, a.d_status, a.c.tokens, false);
        const uint64_t work = work_of<F, NT>(a, seq);
        if (w >= at + work) {
            at += work;
            s++;
            continue;
        }
        const uint32_t units = F::kFixed + units_of<F>(a, seq);
        const uint64_t past = w - at;
        const uint32_t item = past >> 32 ? uint32_t(past / units) : uint32_t(past) / units;
        job.seq = seq;
        job.i1 = at + uint64_t(item + 1) * units;
        job.i0 = job.i1 - units + F::kFixed;
        job.w = max(w, job.i0);
        job.upto = min(w1, job.i1);
        w = job.upto;
        if (w <= job.i0) continue;  // (the CTA's work ends within the item's beginning, which belongs to the first keys' piece)
        job.tile = item / a.c.heads;
        job.h = item - job.tile * a.c.heads;
        const uint32_t row0 = job.tile * 8 * NT, n_rows = seq.n * a.group;
        bounds(a, seq, row0, job.all_lo, job.x_hi);
        bounds(a, seq, min(row0 + 8 * NT, n_rows) - 1, job.x_lo, job.all_hi);
        const int unit0 = int(first_unit<F>(a, seq) + uint32_t(job.w - job.i0)), warp = threadIdx.x >> 5;
        constexpr int kSlice = F::kSlice;
        const int end = min((job.all_hi + kSlice - 1) / kSlice, (unit0 + int(job.upto - job.w)) * kWarps);
        job.first = unit0 * kWarps + warp;
        if (job.first < job.all_lo / kSlice) job.first += (job.all_lo / kSlice - job.first + kWarps - 1) / kWarps * kWarps;
        job.steps = job.first < end ? (end - job.first + kWarps - 1) / kWarps : 0;
        return true;
    }
    return false;
}

// Looks up a piece's first steps and asks for the first of them. turn: the
// warp's slices before the piece.
template <class F>
__device__ __forceinline__ void begin(const AttendArgs &a, const typename F::Maps &maps, typename F::Warp &wp, typename F::Stage *ring, const Job &job, uint32_t turn) {
    constexpr int S = F::kStages;
    F::look_up(a, wp, job, 0);
    __syncwarp();
#pragma unroll 1
    for (int k = 0; k < S - 1; k++) F::fetch(a, maps, wp, ring, job, k, (turn + k) % S);
}

// After a wait was given up: waits (as long again) for the warp's slices [turn, turn + n) that are on their way.
template <class F> __device__ __forceinline__ void drain(const AttendArgs &a, typename F::Warp &wp, uint32_t turn, int n) {
    constexpr int S = F::kStages;
    for (int k = 0; k < min(S - 1, n); k++) bar_wait(&wp.full[(turn + k) % S], (turn + k) / S & 1, a.limit);
}

// All of the rows' work, as far as this warp's slices go.
template <int DP, int NT> struct Sums {
    float o[NT][DP / 16][4];
    // Of rows 2t, 2t + 1 of each tile: the scores' running maximum, how far above it the contributions' is,
    // 2^-d, and the weights' sums over this thread's keys (in units of 2^(m - kRaise)).
    float m[NT][2], d[NT][2], unit[NT][2], l[NT][2];
    uint32_t poison[NT][2];  // of this thread's columns: where a value that the row sees is NaN, and was taken out
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int i = 0; i < DP / 16; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) o[n][i][j] = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) m[n][e] = d[n][e] = kNone, unit[n][e] = l[n][e] = 0.0f, poison[n][e] = 0;
    }
};

// Query fragments: row g of each tile, columns [kRun t, kRun t + kRun) of a thread of a quad, exact in half by a power of
// two, and the scale of the scores of rows 2t, 2t + 1 of each tile.
template <int DP, int NT>
__device__ __forceinline__ void load_queries(const AttendArgs &a, const Job &job, uint32_t (&qf)[NT][DP / 16][2], float (&row_scale)[NT][2]) {
    constexpr int kRows = 8 * NT, kSteps = DP / 16, kRun = DP / 4;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t D = a.c.dim, h = job.h, row0 = job.tile * kRows, n_rows = job.seq.n * a.group;
    const Seq &seq = job.seq;
#pragma unroll
    for (int n = 0; n < NT; n++) {
        const uint32_t row = row0 + 8 * n + g;
        uint32_t w[kRun / 2];
#pragma unroll
        for (int i = 0; i < kRun / 8; i++) {
            uint4 v = make_uint4(0, 0, 0, 0);
            const uint32_t col = kRun * t + 8 * i;
            if (row < n_rows && col < D) {
                v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q.p) + row_at(a, a.q, seq, h, row) + col));
            }
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
        float scale = a.scale_log2;
        if (a.dtype == ZC_BF16) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < kRun / 2; i++) top = max(top, max(w[i] << 16 & 0x7FFF0000u, w[i] & 0x7FFF0000u));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            float up, down;
            row_powers(top, up, down);
            scale = a.scale_log2 * down;
#pragma unroll
            for (int i = 0; i < kRun / 2; i++) {
                const float2 f = unpack2<ZC_BF16>(w[i]);
                w[i] = half2_of(f.x * up, f.y * up);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; e++) row_scale[n][e] = __shfl_sync(0xFFFFFFFFu, scale, 4 * (2 * t + e));
#pragma unroll
        for (int i = 0; i < kSteps; i++) qf[n][i][0] = w[2 * i], qf[n][i][1] = w[2 * i + 1];
    }
}

// The warps' rows together, 8 at a time: into `part`, or finished.
template <int DP, int NT, int kWarps, bool kUnits, class At>
__device__ __forceinline__ void merge(const AttendArgs &a, const At &mg, const Job &job, Sums<DP, NT> &acc, Part<DP, NT> *part) {
    constexpr int kCols = DP / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    Merge<DP> &mine = mg(warp);
    const uint32_t n_rows = job.seq.n * a.group;
#pragma unroll
    for (int n = 0; n < NT; n++) {
        const uint32_t row0 = (job.tile * NT + n) * 8;
        if (n && row0 >= n_rows) break;
        if (n) __syncthreads();
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const int r = 2 * t + e;
            float l = acc.l[n][e];
#pragma unroll
            for (int d = 4; d < 32; d *= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
            l *= 1.0f / (1 << int(kRaise));
            if (acc.poison[n][e]) {
#pragma unroll
                for (int c = 0; c < kCols; c++)
                    if (acc.poison[n][e] >> c & 1) acc.o[n][c / 2][2 * (c & 1) + e] = NAN;
            }
            if (g == 0) mine.m[r] = acc.m[n][e], mine.l[r] = l;
            if (g == 0 && kUnits) mine.d[r] = acc.d[n][e];
#pragma unroll
            for (int c = 0; c < DP / 16; c += 2)
                *reinterpret_cast<float4 *>(&mine.o[r][kCols * g + 2 * c]) =
                    make_float4(acc.o[n][c][e], acc.o[n][c][2 + e], acc.o[n][c + 1][e], acc.o[n][c + 1][2 + e]);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < DP; i += 32 * kWarps) {
            const int r = i / (DP / 8), col = i % (DP / 8) * 8;
            if (row0 + r >= n_rows || col >= int(a.c.dim)) continue;
            float M = kNone, W = kNone, L = 0.0f, x[8] = {};
#pragma unroll
            for (int w = 0; w < kWarps; w++) M = fmaxf(M, mg(w).m[r]);
#pragma unroll
            for (int w = 0; w < kWarps; w++) W = kUnits ? fmaxf(W, above(mg(w).d[r], mg(w).m[r], M)) : M == kNone ? kNone : 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; w++) {
                const float by = ratio2(mg(w).m[r], M), f = kUnits ? ratio2(above(mg(w).d[r], mg(w).m[r], M), W) : by;
                L += mg(w).l[r] * by;
#pragma unroll
                for (int k = 0; k < 8; k++) x[k] += mg(w).o[r][col + k] * f;
            }
            if (part) {
                float4 *p = reinterpret_cast<float4 *>(&part->o[8 * n + r][col]);
                __stcg(p, make_float4(x[0], x[1], x[2], x[3]));
                __stcg(p + 1, make_float4(x[4], x[5], x[6], x[7]));
                if (col == 0) __stcg(&part->m[8 * n + r], M), __stcg(&part->l[8 * n + r], L);
                if (col == 0 && kUnits) __stcg(&part->d[8 * n + r], W);
            } else {
                emit(a, job.seq, job.h, row0 + r, col, x, M, W, L);
            }
        }
    }
}

// Parts of an item together: part i is in the first slot of CTA first + i, but
// the item's own first one (i = 0) in the second, where a piece that begins an
// item is. Joins parts i0, i0 + step, ... (n of them), into part i0 or, without
// `on`, into the finished rows.
// A thread takes 4 columns of a row and every ways-th part, kRun parts in
// flight together; the ways meet in shared memory.
template <int DP, int NT, int kThreads, bool kUnits>
__device__ __forceinline__ void join(const AttendArgs &a, uint8_t *smem, const Job &item, uint32_t first, uint32_t i0, uint32_t step,
                                     uint32_t n, bool on) {
    constexpr int kCols = DP / 4, kRun = 8;
    struct Way {
        float4 x;
        float m, d, l;
    };
    Way *met = reinterpret_cast<Way *>(smem);
    Part<DP, NT> *parts = static_cast<Part<DP, NT> *>(a.parts);
    auto part = [&](uint32_t i) -> Part<DP, NT> & { return parts[2 * (first + i) + (i ? 0 : 1)]; };
    const uint32_t row0 = item.tile * 8 * NT;
    const int rows = int(min(uint32_t(8 * NT), item.seq.n * a.group - row0)), D = int(a.c.dim);
    const int jobs = rows * kCols;                             // 4 columns of a row each
    const int ways = jobs >= kThreads ? 1 : kThreads / jobs;   // threads of a job
#pragma unroll 1
    for (int j0 = 0; j0 < jobs; j0 += kThreads) {
        const int job = ways == 1 ? j0 + int(threadIdx.x) : int(threadIdx.x) % jobs, way = ways == 1 ? 0 : int(threadIdx.x) / jobs;
        const int r = job / kCols, col = job % kCols * 4;
        const bool mine = job < jobs && way < ways && col < D;
        Way w = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), kNone, kNone, 0.0f};
        // brings w to the units (m, d)
        auto to_units = [&](float m, float d) {
            const float by = ratio2(w.m, m), f = kUnits ? ratio2(above(w.d, w.m, m), d) : by;
            w.l *= by;
            w.x.x *= f, w.x.y *= f, w.x.z *= f, w.x.w *= f;
            w.m = m, w.d = d;
        };
        auto add = [&](float4 x, float m, float d, float l) {
            const float by = ratio2(m, w.m), f = kUnits ? ratio2(above(d, m, w.m), w.d) : by;
            w.l += l * by;
            w.x.x += x.x * f, w.x.y += x.y * f, w.x.z += x.z * f, w.x.w += x.w * f;
        };
        if (mine) {
#pragma unroll 1
            for (uint32_t i = way; i < n; i += kRun * ways) {
                float4 x[kRun];
                float m[kRun], d[kRun], l[kRun];
#pragma unroll
                for (int k = 0; k < kRun; k++) {
                    const uint32_t of = i + k * ways;
                    const bool there = of < n;
                    const Part<DP, NT> &p = part(there ? i0 + of * step : i0);
                    x[k] = there ? __ldcg(reinterpret_cast<const float4 *>(&p.o[r][col])) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    m[k] = there ? __ldcg(&p.m[r]) : kNone, d[k] = there && kUnits ? __ldcg(&p.d[r]) : kNone, l[k] = there ? __ldcg(&p.l[r]) : 0.0f;
                }
                float m1 = w.m;
#pragma unroll
                for (int k = 0; k < kRun; k++) m1 = fmaxf(m1, m[k]);
                float d1 = kUnits ? above(w.d, w.m, m1) : m1 == kNone ? kNone : 0.0f;
#pragma unroll
                for (int k = 0; k < kRun; k++) d1 = kUnits ? fmaxf(d1, above(d[k], m[k], m1)) : d1;
                to_units(m1, d1);
#pragma unroll
                for (int k = 0; k < kRun; k++) add(x[k], m[k], d[k], l[k]);
            }
        }
        if (ways > 1) {
            met[threadIdx.x] = w;
            __syncthreads();
            if (way == 0)
#pragma unroll 1
                for (int k = 1; k < ways; k++) {
                    const Way v = met[threadIdx.x + k * jobs];
                    const float m1 = fmaxf(w.m, v.m);
                    to_units(m1, kUnits ? fmaxf(above(w.d, w.m, m1), above(v.d, v.m, m1)) : m1 == kNone ? kNone : 0.0f);
                    add(v.x, v.m, v.d, v.l);
                }
        }
        if (on) {
            __syncthreads();  // everyone has read part i0
            if (mine && way == 0) {
                Part<DP, NT> &p = part(i0);
                __stcg(reinterpret_cast<float4 *>(&p.o[r][col]), w.x);
                if (col == 0) __stcg(&p.m[r], w.m), __stcg(&p.l[r], w.l);
                if (col == 0 && kUnits) __stcg(&p.d[r], w.d);
            }
        } else if (mine && way == 0) {
            const float y[4] = {w.x.x, w.x.y, w.x.z, w.x.w};
            emit(a, item.seq, item.h, row0 + r, col, y, w.m, w.d, w.l);
        }
    }
}

// Whether this CTA is the last of n to come to a counter (which is left at zero then): what the others wrote before they
// came can be read.
__device__ __forceinline__ bool last_of(uint32_t *counter, uint32_t n, int &s_last) {
    __syncthreads();
    if (threadIdx.x == 0) {
        // releases what the CTA wrote (the barrier before it orders the other threads' writes) and acquires the others'
        uint32_t done;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(done) : "l"(counter) : "memory");
        if (done == n - 1) *counter = 0;
        s_last = done == n - 1;
    }
    __syncthreads();
    return s_last;
}

template <class F, int NT> constexpr size_t ring_bytes() { return sizeof(typename F::Stage) * F::kStages * F::kWarps; }
template <class F> constexpr size_t kJoinBytes = 32 * F::kWarps * 32;  // what join() takes
template <class F, int NT> constexpr size_t smem_bytes() {
    return ring_bytes<F, NT>() + (F::kMergeInRing ? sizeof(typename F::Stage) < kJoinBytes<F> ? kJoinBytes<F> : 0 : F::kWarps * sizeof(Merge<F::kDim>));
}

template <class F, int NT>
__global__ void __launch_bounds__(32 * F::kWarps, F::template resident<NT>()) rows_kernel(const __grid_constant__ AttendArgs a,
                                                                     const __grid_constant__ typename F::Maps maps) {
    using Warp = typename F::Warp;
    using Stage = typename F::Stage;
    constexpr int S = F::kStages, DP = F::kDim, kWarps = F::kWarps, kThreads = 32 * kWarps;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Warp s_warps[kWarps];
    __shared__ uint64_t s_warp[kWarps], s_at;
    __shared__ uint32_t s_seq;
    __shared__ int s_last;
    // Where warps' rows meet: behind the rings, or in the stage of each warp's ring that it has read last, which nothing is
    // asked for while its next piece begins.
    static_assert(!F::kMergeInRing || sizeof(Merge<DP>) <= sizeof(Stage), "a warp's rows do not fit a stage");
    static_assert(F::kMergeInRing || kWarps * sizeof(Merge<DP>) >= kJoinBytes<F>, "no room for joining");
    __shared__ uint32_t s_free[kWarps];
    auto mg = [&](int w) -> Merge<DP> & {
        if (F::kMergeInRing) return *reinterpret_cast<Merge<DP> *>(reinterpret_cast<Stage *>(smem) + w * S + s_free[w]);
        return reinterpret_cast<Merge<DP> *>(smem + ring_bytes<F, NT>())[w];
    };
    Part<DP, NT> *parts = reinterpret_cast<Part<DP, NT> *>(a.parts);
    const uint32_t B = a.c.tokens, cta = blockIdx.x;

    Warp &wp = s_warps[threadIdx.x / 32];
    Stage *ring = reinterpret_cast<Stage *>(smem) + threadIdx.x / 32 * S;
    if (threadIdx.x % 32 == 0) {
        for (int i = 0; i < S; i++) bar_init(&wp.full[i], 1);
        bar_init_done();
        prefetch_maps(maps);
    }

    if (F::kEarly) after_the_last();

    // The line of work, and this CTA's piece [w0, w1) of it.
    uint64_t mine = 0, sum, W;
    for (uint32_t s = threadIdx.x; s < a.b.n_seqs; s += kThreads) {
        const uint64_t work = work_of<F, NT>(a, read_seq(a.b, s, a.d_status, B, cta == 0));
        mine += work;
    }
    sum = block_scan<kWarps>(mine, s_warp, W);
    const uint64_t G = min(uint64_t(gridDim.x), W);  // no CTA between two that have work is without
    if (cta >= G) return;
    const uint64_t w0 = W * cta / G, w1 = W * (cta + 1) / G;
    uint64_t before = 0;
    for (uint32_t s0 = 0; s0 < a.b.n_seqs; s0 += kThreads) {
        if (a.b.n_seqs > kThreads) {  // more than one round: the sums above were not of single sequences
            const uint32_t s = s0 + threadIdx.x;
            mine = s < a.b.n_seqs ? work_of<F, NT>(a, read_seq(a.b, s, a.d_status, B, false)) : 0;
            uint64_t all;
            sum = before + block_scan<kWarps>(mine, s_warp, all);
            before += all;
        }
        if (mine && sum > w0 && sum - mine <= w0) s_seq = s0 + threadIdx.x, s_at = sum - mine;
        if (before > w0) break;
    }
    __syncthreads();
    uint32_t s = s_seq;
    uint64_t at = s_at, w = w0;  // where the sequence's work begins; where this CTA has got to

    uint32_t turn = 0;  // slices that this warp has asked for
    Job job, next;
    bool more = next_job<F, NT>(a, w, w1, s, at, job);
    if (more) begin<F>(a, maps, wp, ring, job, turn);  // (a CTA's work may be an item's beginning alone, which is another's)
    while (more) {
        Sums<DP, NT> acc;
        const bool ok = F::template attend_slices<NT>(a, maps, wp, ring, job, turn, acc);
        turn += uint32_t(job.steps);
        // The next piece's first slices are on their way while this one is finished.
        more = next_job<F, NT>(a, w, w1, s, at, next);
        if (more && ok) begin<F>(a, maps, wp, ring, next, turn);
        if (F::kMergeInRing && threadIdx.x % 32 == 0) s_free[threadIdx.x / 32] = (turn + S - 1) % S;
        if (__syncthreads_or(!ok)) {
            if (more && ok) drain<F>(a, wp, turn, next.steps);
            return;
        }
        const bool whole = job.whole();
        merge<DP, NT, kWarps, F::kUnits>(a, mg, job, acc, whole ? nullptr : parts + 2 * cta + (job.w == job.i0 ? 1 : 0));
        if (!whole) {
            // CTAs from that of the item's first unit to that of its last: unit u is CTA c's where
            // W c / G <= u < W (c + 1) / G, rounded down, so c = (u G + G - 1) / W
            const uint32_t c0 = uint32_t((job.i0 * G + G - 1) / W), c1 = uint32_t(((job.i1 - 1) * G + G - 1) / W);
            const uint32_t n = c1 - c0 + 1, mine = cta - c0;
            uint32_t *counter = a.counters + uint64_t(slot_of(job.seq.first, job.seq.s, a.group, 8 * NT, 1) + job.tile) * a.c.heads + job.h;
            uint8_t *space = F::kMergeInRing && sizeof(Stage) < kJoinBytes<F> ? smem + ring_bytes<F, NT>() : reinterpret_cast<uint8_t *>(&mg(0));
            // many parts: each kGroup of them first, by the last CTA of those, then what they make
            const uint32_t groups = n <= 2 * kGroup ? 1 : (n + kGroup - 1) / kGroup, g = groups == 1 ? 0 : mine / kGroup;
            uint32_t i0 = g * kGroup, step = 1, parts_of = groups == 1 ? n : min(uint32_t(kGroup), n - i0);
            uint32_t *first = groups == 1 ? counter : a.group_counters + 2 * (c0 + i0) + (g ? 0 : 1);
            bool on = groups > 1, go = last_of(first, parts_of, s_last);
#pragma unroll 1
            while (go) {
                join<DP, NT, kThreads, F::kUnits>(a, space, job, c0, i0, step, parts_of, on);
                go = on && last_of(counter, groups, s_last);
                i0 = 0, step = kGroup, parts_of = groups, on = false;
            }
        }
        if (F::kMergeInRing) {  // before a stage is asked for again
            fence_async();
            __syncthreads();
        }
        job = next;
    }
}

template <class F, int NT> int launch(const AttendArgs &a, uint32_t rows, cudaStream_t s) {
    static std::atomic<uint64_t> ready{0};  // devices whose kernel may use this much shared memory
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cuda_failed();
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(rows_kernel<F, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem_bytes<F, NT>())) != cudaSuccess)
            return cuda_failed();
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    typename F::Maps maps;
    const int st = make_maps(a.c, F::kDim, rows, maps);
    if (st != ZC_OK) return st;
    const uint32_t grid = uint32_t(sm_count() * F::template resident<NT>()), threads = 32 * F::kWarps;
    if (F::kEarly) return launch_early(rows_kernel<F, NT>, dim3(grid), threads, smem_bytes<F, NT>(), s, a, maps);
    rows_kernel<F, NT><<<grid, threads, smem_bytes<F, NT>(), s>>>(a, maps);
    return cudaGetLastError() == cudaSuccess ? ZC_OK : ZC_ECUDA;
}

} // namespace
} // namespace kv
} // namespace zc
