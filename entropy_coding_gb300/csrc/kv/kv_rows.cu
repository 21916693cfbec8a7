// kv_rows.cu — attention of few query rows over the 8-bit cache.
//
// A row is one query token and query head; the rows of a key/value head are
// its `group` query heads times the sequence's new tokens. With codes kc, vc
// and block scales ks, vs, over the keys j that row i sees:
//   s_ij = scale * ks_b(j) * (q_i . kc_j)
//   out_i = sum_j 2^(s_ij log2e - m) vs_b(j) vc_j / sum_j 2^(s_ij log2e - m)
//
// An item is the rows (at most 16) of one sequence and key/value head. Decoding has few
// items and long key axes, so items are cut along the keys: the batch's work
// is one line of 64-key units, items one after another, and each CTA of a
// resident grid takes an equal piece of it (a few whole items and a part of
// one at either end, whatever the sequences' lengths). An item that lies in
// several CTAs leaves one partial result for each in the workspace, and the
// CTA that comes last, by the item's counter, joins them in the order of the
// keys: no second launch, and the same bits whichever CTA is last. The counter
// is left at zero for the next call.
//
// A CTA has 4 warps; a warp takes 16 keys at a time, and both products run on
// mma.m16n8k16 with half operands and float accumulators, transposed: keys (or
// the output's columns) are the 16 and the query rows the 8, so that a decoding
// step's 4 or 8 rows of a head fill the tile. E4M3 codes are exact in half. A
// query row is exact in half too after it is multiplied by a power of two that
// brings its largest element to [2^14, 2^15) (what falls below 2^-24 then is
// 2^-38 of it). A row's weights w are rounded to half; they are kept in units
// of the row's running maximum of s + log2 vs (to a factor of 2^6), not of s
// alone, so that blocks whose scales differ by any factor keep their precision,
// and 2^9 above that unit: half keeps its 11 bits down to 2^-23 of the largest
// w vs. The sum of the weights is taken before that rounding, in units of the
// running maximum of s.
//
// Each warp streams its own keys and values through a ring of slices of 16
// rows in shared memory: one lane asks for two boxes a slice, and the warps
// meet only at an item's end. The boxes are swizzled, which spreads a
// fragment's reads over the banks. Within a row the columns are dealt to the
// threads of a quad in runs (the order of a product's inner index is free as
// long as both operands share it), so that fragments are read 16 bytes at a
// time.
//
// Measured on a GB300: the next tokens of 64 sequences of up to 8192 keys (8
// heads of 128, 4 query heads each), 558 MB of cache, in 98 us: 5.7 TB/s, 0.84
// of the copy rate. While slices stream, memory is the bound (a single long
// sequence's 268 MB go by in 37 us of the call's 52); the rest is the start (4
// us until the first slices are there), pieces' ends, and the joining of parts.
// The transposed products halved the tensor instructions for 4 rows (135 to 122
// us); fetching the next piece before the last is finished, 113 to 99.
#include <algorithm>
#include <atomic>
#include <cfloat>

#include "kv_attend.cuh"

namespace zc {
namespace kv {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kSlice = 16;              // keys of a warp's step
constexpr int kUnit = kWarps * kSlice;  // keys of a unit of work

// CTAs of an SM, as many as their registers allow, and slices of a ring, as
// many as fit the SM's shared memory then.
constexpr int kResident = 3;
// Parts that are joined at a time, where there are more than twice as many: 57 parts of a long sequence at once made its
// call 58 us, in two steps 52; for 16 parts the second step costs what it saves.
constexpr int kGroup = 8;
constexpr int stages(int dp) { return 3 * (128 / dp); }

template <int DP> struct Stage {
    uint8_t k[kSlice * DP];
    uint8_t v[kSlice * DP];
};

// What a warp keeps in shared memory besides its ring: the ring's barriers, and
// the blocks and scales of 64 of its steps, read 32 at a time.
constexpr int kAhead = 32;
template <int S> struct Warp {
    uint64_t full[S];
    int32_t block[2 * kAhead];
    float ks[2 * kAhead], vs[2 * kAhead];
};

template <int DP> struct Merge {  // 8 rows of each warp
    float o[kWarps][8][DP + 4];
    float m[kWarps][8], mw[kWarps][8], l[kWarps][8];
};

// A part of an item: rows in units of 2^mw (o) and 2^m (l).
template <int DP, int NT> struct Part {
    float o[8 * NT][DP];
    float m[8 * NT], mw[8 * NT], l[8 * NT];
};

template <int DP, int NT> constexpr size_t ring_bytes() { return sizeof(Stage<DP>) * stages(DP) * kWarps; }
template <int DP, int NT> constexpr size_t smem_bytes() { return ring_bytes<DP, NT>() + sizeof(Merge<DP>); }

__device__ __forceinline__ void cp4(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_of(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Where a box holds 16-byte chunk c of row r: the swizzle of the tensor maps.
template <int DP> __device__ __forceinline__ int chunk_at(int r, int c) {
    return r * DP + 16 * (c ^ (DP == 128 ? r & 7 : r >> 1 & 3));
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The 8x8 matrix of halves whose rows the quads hold, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// Units of work of a sequence's items (the same for all of them).
__device__ __forceinline__ uint32_t first_unit(const AttendArgs &a, const Seq &q) {
    const int pos = q.len - int(q.n);
    return a.window && pos >= int(a.window) ? uint32_t(pos - int(a.window) + 1) / kUnit : 0;
}
__device__ __forceinline__ uint32_t units_of(const AttendArgs &a, const Seq &q) {
    return max((uint32_t(q.len) + kUnit - 1) / kUnit, first_unit(a, q) + 1) - first_unit(a, q);
}
template <int NT> __device__ __forceinline__ uint64_t work_of(const AttendArgs &a, const Seq &q) {
    return q.ok && q.n * a.group <= a.rows_most ? uint64_t((q.n * a.group + 8 * NT - 1) / (8 * NT)) * a.c.heads * units_of(a, q) : 0;
}

// A piece of work: units of item (seq, tile, h) on the line of work, and what
// this warp does of it.
struct Job {
    Seq seq;
    uint32_t tile, h;
    uint64_t w, upto, i0, i1;          // the piece [w, upto) of the item's [i0, i1)
    int all_lo, all_hi, x_lo, x_hi;    // keys seen by some row; by every row
    int first, steps;                  // this warp's slices: first, first + kWarps, ...
    __device__ __forceinline__ bool whole() const { return w == i0 && upto == i1; }
};

// The piece of work at w, whose sequence's work begins at `at` (both moved on).
template <int NT>
__device__ __forceinline__ bool next_job(const AttendArgs &a, uint64_t &w, uint64_t w1, uint32_t &s, uint64_t &at, Job &job) {
    while (w < w1) {
        const Seq seq = read_seq(a.b, s, a.d_status, a.c.tokens, false);
        const uint64_t work = work_of<NT>(a, seq);
        if (w >= at + work) {
            at += work;
            s++;
            continue;
        }
        const uint32_t units = units_of(a, seq);
        const uint64_t past = w - at;
        const uint32_t item = past >> 32 ? uint32_t(past / units) : uint32_t(past) / units;
        job.seq = seq;
        job.i0 = at + item * units;
        job.i1 = job.i0 + units;
        job.w = w;
        job.upto = min(w1, job.i1);
        job.tile = item / a.c.heads;
        job.h = item - job.tile * a.c.heads;
        const uint32_t row0 = job.tile * 8 * NT, n_rows = seq.n * a.group;
        bounds(a, seq, row0, job.all_lo, job.x_hi);
        bounds(a, seq, min(row0 + 8 * NT, n_rows) - 1, job.x_lo, job.all_hi);
        const int unit0 = int(first_unit(a, seq) + uint32_t(w - job.i0)), warp = threadIdx.x >> 5;
        const int end = min((job.all_hi + kSlice - 1) / kSlice, (unit0 + int(job.upto - w)) * kWarps);
        job.first = unit0 * kWarps + warp;
        if (job.first < job.all_lo / kSlice) job.first += (job.all_lo / kSlice - job.first + kWarps - 1) / kWarps * kWarps;
        job.steps = job.first < end ? (end - job.first + kWarps - 1) / kWarps : 0;
        w = job.upto;
        return true;
    }
    return false;
}

// The blocks and scales of steps k0 .. k0 + 31, a step a lane. A block that is not there is read as block 0.
template <class Warp> __device__ __forceinline__ void look_up(const AttendArgs &a, Warp &wp, const Job &job, int k0) {
    const int k = k0 + (threadIdx.x & 31);
    if (k >= job.steps) return;
    const int64_t id = max(read_block(a.b, a.c, job.seq.s, block_of_16(a.c, uint32_t(job.first + k * kWarps)), a.d_status), int64_t(0));
    const int at = k & (2 * kAhead - 1);
    wp.block[at] = int32_t(id);
    cp4(&wp.ks[at], a.c.scale[0] + id * a.c.scale_stride + job.h);
    cp4(&wp.vs[at], a.c.scale[1] + id * a.c.scale_stride + job.h);
}

// Asks for step k's keys and values (one lane). Rows that nobody sees come along as they are.
template <int DP, class Warp>
__device__ __forceinline__ void fetch(const AttendArgs &a, const CodeMaps &maps, Warp &wp, Stage<DP> *ring, const Job &job, int k, uint32_t st) {
    if ((threadIdx.x & 31) == 0 && k < job.steps && !a.stall) {
        const uint32_t i = uint32_t(job.first + k * kWarps);
        const int row = int(job.h * a.c.tokens + i * kSlice - block_of_16(a.c, i) * a.c.tokens), id = wp.block[k & (2 * kAhead - 1)];
        bar_expect(&wp.full[st], sizeof(Stage<DP>));
        copy_box(ring[st].k, &maps.code[0], row, id, &wp.full[st]);
        copy_box(ring[st].v, &maps.code[1], row, id, &wp.full[st]);
    }
}

// Looks up a piece's first steps and asks for the first of them. turn: the
// warp's slices before the piece.
template <int DP, int S>
__device__ __forceinline__ void begin(const AttendArgs &a, const CodeMaps &maps, Warp<S> &wp, Stage<DP> *ring, const Job &job, uint32_t turn) {
    look_up(a, wp, job, 0);
    __syncwarp();
#pragma unroll 1
    for (int k = 0; k < S - 1; k++) fetch<DP>(a, maps, wp, ring, job, k, (turn + k) % S);
}

// After a wait was given up: waits (as long again) for the warp's slices [turn, turn + n) that are on their way.
template <int S> __device__ __forceinline__ void drain(const AttendArgs &a, Warp<S> &wp, uint32_t turn, int n) {
    for (int k = 0; k < min(S - 1, n); k++) bar_wait(&wp.full[(turn + k) % S], (turn + k) / S & 1, a.limit);
}

// All of the rows' work, as far as this warp's slices go.
template <int DP, int NT> struct Sums {
    float o[NT][DP / 16][4];
    // Of rows 2t, 2t + 1 of each tile: running maxima (the scores', and with the value scales),
    // 2^(m - mw), and the weights' sums over this thread's keys (in units of 2^(m - kRaise)).
    float m[NT][2], mw[NT][2], unit[NT][2], l[NT][2];
    uint32_t poison[NT][2];  // of this thread's columns: where a value that the row sees is NaN, and was taken out
};

template <int DP, int NT, int S>
__device__ __forceinline__ bool attend_slices(const AttendArgs &a, const CodeMaps &maps, Warp<S> &wp, Stage<DP> *ring, const Job &job,
                                              uint32_t turn, Sums<DP, NT> &acc) {
    constexpr int kRows = 8 * NT;
    constexpr int kSteps = DP / 16;      // inner steps of k q, and column tiles of the output
    constexpr int kRun = DP / 4;         // columns of q and k that a thread of a quad holds
    constexpr int kCols = DP / 8;        // columns of v that a thread's quad holds
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t D = a.c.dim, h = job.h;
    const Seq &seq = job.seq;
    const uint32_t row0 = job.tile * kRows, n_rows = seq.n * a.group;
    auto &o = acc.o;
    auto &m = acc.m;
    auto &mw = acc.mw;
    auto &unit = acc.unit;
    auto &l = acc.l;

    // Query fragments: row g of each tile, columns [kRun t, kRun t + kRun).
    uint32_t qf[NT][kSteps][2];
    float row_scale[NT][2];  // of rows 2t, 2t + 1 of each tile
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

#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
        for (int i = 0; i < kSteps; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) o[n][i][j] = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
        for (int e = 0; e < 2; e++) m[n][e] = mw[n][e] = kNone, unit[n][e] = l[n][e] = 0.0f, acc.poison[n][e] = 0;

    uint32_t st = turn % S, parity = turn / S & 1;  // of step k
    for (int k = 0; k < job.steps; k++) {
        if ((k & (kAhead - 1)) == 0) {
            cp_wait_all();
            __syncwarp();
            look_up(a, wp, job, k + kAhead);
        }
        if (!__all_sync(0xFFFFFFFFu, bar_wait(&wp.full[st], parity, a.limit))) {
            drain(a, wp, turn + k, job.steps - k);
            if (lane == 0) report(a.d_status, ZC_ETIMEOUT);
            return false;
        }
        // The stage before this one was read a step ago (the vote above comes after every lane's reads).
        fetch<DP>(a, maps, wp, ring, job, k + S - 1, st == 0 ? S - 1 : st - 1);
        Stage<DP> &sl = ring[st];
        if (++st == S) st = 0, parity ^= 1;
        const int key0 = (job.first + k * kWarps) * kSlice;
        const float ks = wp.ks[k & (2 * kAhead - 1)], vs = wp.vs[k & (2 * kAhead - 1)];

        // scores of 16 keys and the rows: c0, c1 are key g and rows 2t, 2t + 1, c2, c3 key g + 8
        // (two sums for a single tile: half the chain of dependent products)
        constexpr int kSums = NT == 1 ? 2 : 1;
        float part_sc[kSums][NT][4], sc[NT][4];
#pragma unroll
        for (int n = 0; n < kSums * NT; n++)
            part_sc[n / NT][n % NT][0] = part_sc[n / NT][n % NT][1] = part_sc[n / NT][n % NT][2] = part_sc[n / NT][n % NT][3] = 0.0f;
#pragma unroll
        for (int c = 0; c < kRun / 16; c++) {
            const uint4 v0 = *reinterpret_cast<const uint4 *>(&sl.k[chunk_at<DP>(g, kRun / 16 * t + c)]);
            const uint4 v1 = *reinterpret_cast<const uint4 *>(&sl.k[chunk_at<DP>(8 + g, kRun / 16 * t + c)]);
            const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
                uint32_t kf[4];
                e4m3x4_to_half2x2(w0[k], kf[0], kf[2]);
                e4m3x4_to_half2x2(w1[k], kf[1], kf[3]);
#pragma unroll
                for (int n = 0; n < NT; n++) mma(part_sc[k % kSums][n], kf, qf[n][4 * c + k][0], qf[n][4 * c + k][1]);
            }
        }
        const bool edge = key0 < job.x_lo || key0 + kSlice > job.x_hi;  // some row does not see all of it
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int j = 0; j < 4; j++)
                sc[n][j] = (kSums == 1 ? part_sc[0][n][j] : part_sc[0][n][j] + part_sc[kSums - 1][n][j]) * (row_scale[n][j & 1] * ks);
        if (edge) {
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    int lo, hi;
                    bounds(a, seq, min(row0 + 8 * n + 2 * t + e, n_rows - 1), lo, hi);
#pragma unroll
                    for (int j = 0; j < 2; j++)
                        if (key0 + g + 8 * j < lo || key0 + g + 8 * j >= hi) sc[n][2 * j + e] = kNone;
                }
        }
        // m and mw follow the maxima only once these are 2^kSlack and 2^kSlackW above them: after the first step a
        // rescaling is rare.
        const float lvs = __log2f(vs);
        bool grows = false;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float top = fmaxf(sc[n][e], sc[n][2 + e]);
                grows |= top > m[n][e] + kSlack || top + lvs > mw[n][e] + kSlackW;
            }
        if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
            for (int n = 0; n < NT; n++) {
                float down[2];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float top = fmaxf(sc[n][e], sc[n][2 + e]);
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                    const float m1 = fmaxf(m[n][e], top), w1 = fmaxf(mw[n][e], top + lvs);
                    l[n][e] *= ratio2(m[n][e], m1);
                    down[e] = ratio2(mw[n][e], w1);
                    m[n][e] = m1, mw[n][e] = w1;
                    unit[n][e] = w1 == kNone || m1 == kNone ? 0.0f : ex2(fminf(m1 - w1, 126.0f));
                }
#pragma unroll
                for (int c = 0; c < kSteps; c++)
                    o[n][c][0] *= down[0], o[n][c][1] *= down[1], o[n][c][2] *= down[0], o[n][c][3] *= down[1];
            }
        }
        // Weights p = 2^(s - m + kRaise), and in the output's units p * 2^(m + log2 vs - mw). (A block that is louder than
        // the unit by more than a float holds is hardly attended to: an infinite factor would make its weights of 0 NaN.)
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; n++) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float base = (m[n][e] == kNone ? 0.0f : m[n][e]) - kRaise, f = fminf(vs * unit[n][e], FLT_MAX);
                const float p0 = ex2(sc[n][e] - base), p1 = ex2(sc[n][2 + e] - base);
                l[n][e] += p0 + p1;
                w[e] = p0 * f, w[2 + e] = p1 * f;
            }
            pf[n][0] = transpose8(half2_of(w[0], w[1]));
            pf[n][1] = transpose8(half2_of(w[2], w[3]));
        }
        // Values: the thread's keys are 2t, 2t + 1, 2t + 8, 2t + 9, its columns [kCols g, kCols g + kCols).
        const int keys[4] = {2 * t, 2 * t + 1, 2 * t + 8, 2 * t + 9};
        if (edge) {
            // A row that does not see a key has weight 0 for it, but 0 * NaN is NaN: NaN codes are
            // taken out here and given to the rows that do see them.
            bool bad = false;
#pragma unroll 1
            for (int j = lane; j < kSlice * DP / 16; j += 32) {
                const uint4 v = *reinterpret_cast<const uint4 *>(&sl.v[16 * j]);
                bad |= any_nan(v.x) || any_nan(v.y) || any_nan(v.z) || any_nan(v.w);
            }
            if (__any_sync(0xFFFFFFFFu, bad)) {
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        int lo, hi;
                        bounds(a, seq, min(row0 + 8 * n + 2 * t + e, n_rows - 1), lo, hi);
#pragma unroll 1
                        for (int k = max(lo - key0, 0); k < min(hi - key0, kSlice); k++)
#pragma unroll 1
                            for (int c = 0; c < kCols; c++)
                                if ((sl.v[chunk_at<DP>(k, (kCols * g + c) / 16) + (kCols * g + c) % 16] & 0x7F) == 0x7F) acc.poison[n][e] |= 1u << c;
                    }
                __syncwarp();
#pragma unroll 1
                for (int j = lane; j < kSlice * DP; j += 32)
                    if ((sl.v[j] & 0x7F) == 0x7F) sl.v[j] = 0;
                fence_async();
                __syncwarp();
            }
        }
        uint32_t vw[4][kCols / 4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (kCols == 16) {
                const uint4 v = *reinterpret_cast<const uint4 *>(&sl.v[chunk_at<DP>(keys[j], g)]);
                vw[j][0] = v.x, vw[j][1] = v.y, vw[j][kCols / 4 - 2] = v.z, vw[j][kCols / 4 - 1] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2 *>(&sl.v[chunk_at<DP>(keys[j], g / 2) + 8 * (g & 1)]);
                vw[j][0] = v.x, vw[j][1] = v.y;
            }
        }
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {  // columns kCols g + c and + 1: rows g and g + 8 of the tile
            const uint32_t sel = (c & 3) | ((c & 3) + 4) << 4 | ((c & 3) + 1) << 8 | ((c & 3) + 5) << 12;
            const uint32_t b0 = __byte_perm(vw[0][c / 4], vw[1][c / 4], sel), b1 = __byte_perm(vw[2][c / 4], vw[3][c / 4], sel);
            uint32_t vf[4];
            e4m3x4_to_half2x2(b0, vf[0], vf[1]);
            e4m3x4_to_half2x2(b1, vf[2], vf[3]);
#pragma unroll
            for (int n = 0; n < NT; n++) mma(o[n][c / 2], vf, pf[n][0], pf[n][1]);
        }
    }

    return true;
}

// The warps' rows together, 8 at a time: into `part`, or finished.
template <int DP, int NT>
__device__ __forceinline__ void merge(const AttendArgs &a, Merge<DP> &mg, const Job &job, Sums<DP, NT> &acc, Part<DP, NT> *part) {
    constexpr int kCols = DP / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
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
            if (g == 0) mg.m[warp][r] = acc.m[n][e], mg.mw[warp][r] = acc.mw[n][e], mg.l[warp][r] = l;
#pragma unroll
            for (int c = 0; c < DP / 16; c += 2)
                *reinterpret_cast<float4 *>(&mg.o[warp][r][kCols * g + 2 * c]) =
                    make_float4(acc.o[n][c][e], acc.o[n][c][2 + e], acc.o[n][c + 1][e], acc.o[n][c + 1][2 + e]);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < DP; i += kThreads) {
            const int r = i / (DP / 8), col = i % (DP / 8) * 8;
            if (row0 + r >= n_rows || col >= int(a.c.dim)) continue;
            float M = kNone, W = kNone, L = 0.0f, x[8] = {};
#pragma unroll
            for (int w = 0; w < kWarps; w++) M = fmaxf(M, mg.m[w][r]), W = fmaxf(W, mg.mw[w][r]);
#pragma unroll
            for (int w = 0; w < kWarps; w++) {
                L += mg.l[w][r] * ratio2(mg.m[w][r], M);
                const float f = ratio2(mg.mw[w][r], W);
#pragma unroll
                for (int k = 0; k < 8; k++) x[k] += mg.o[w][r][col + k] * f;
            }
            if (part) {
                float4 *p = reinterpret_cast<float4 *>(&part->o[8 * n + r][col]);
                __stcg(p, make_float4(x[0], x[1], x[2], x[3]));
                __stcg(p + 1, make_float4(x[4], x[5], x[6], x[7]));
                if (col == 0) __stcg(&part->m[8 * n + r], M), __stcg(&part->mw[8 * n + r], W), __stcg(&part->l[8 * n + r], L);
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
template <int DP, int NT>
__device__ __forceinline__ void join(const AttendArgs &a, uint8_t *smem, const Job &item, uint32_t first, uint32_t i0, uint32_t step,
                                     uint32_t n, bool on) {
    constexpr int kCols = DP / 4, kRun = 8;
    struct Way {
        float4 x;
        float m, mw, l;
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
        // brings w to the units (m, mw)
        auto to_units = [&](float m, float mw) {
            const float f = ratio2(w.mw, mw);
            w.l *= ratio2(w.m, m);
            w.x.x *= f, w.x.y *= f, w.x.z *= f, w.x.w *= f;
            w.m = m, w.mw = mw;
        };
        auto add = [&](float4 x, float m, float mw, float l) {
            const float f = ratio2(mw, w.mw);
            w.l += l * ratio2(m, w.m);
            w.x.x += x.x * f, w.x.y += x.y * f, w.x.z += x.z * f, w.x.w += x.w * f;
        };
        if (mine) {
#pragma unroll 1
            for (uint32_t i = way; i < n; i += kRun * ways) {
                float4 x[kRun];
                float m[kRun], mw[kRun], l[kRun];
#pragma unroll
                for (int k = 0; k < kRun; k++) {
                    const uint32_t of = i + k * ways;
                    const bool there = of < n;
                    const Part<DP, NT> &p = part(there ? i0 + of * step : i0);
                    x[k] = there ? __ldcg(reinterpret_cast<const float4 *>(&p.o[r][col])) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    m[k] = there ? __ldcg(&p.m[r]) : kNone, mw[k] = there ? __ldcg(&p.mw[r]) : kNone, l[k] = there ? __ldcg(&p.l[r]) : 0.0f;
                }
                float m1 = w.m, w1 = w.mw;
#pragma unroll
                for (int k = 0; k < kRun; k++) m1 = fmaxf(m1, m[k]), w1 = fmaxf(w1, mw[k]);
                to_units(m1, w1);
#pragma unroll
                for (int k = 0; k < kRun; k++) add(x[k], m[k], mw[k], l[k]);
            }
        }
        if (ways > 1) {
            met[threadIdx.x] = w;
            __syncthreads();
            if (way == 0)
#pragma unroll 1
                for (int k = 1; k < ways; k++) {
                    const Way v = met[threadIdx.x + k * jobs];
                    to_units(fmaxf(w.m, v.m), fmaxf(w.mw, v.mw));
                    add(v.x, v.m, v.mw, v.l);
                }
        }
        if (on) {
            __syncthreads();  // everyone has read part i0
            if (mine && way == 0) {
                Part<DP, NT> &p = part(i0);
                __stcg(reinterpret_cast<float4 *>(&p.o[r][col]), w.x);
                if (col == 0) __stcg(&p.m[r], w.m), __stcg(&p.mw[r], w.mw), __stcg(&p.l[r], w.l);
            }
        } else if (mine && way == 0) {
            const float y[4] = {w.x.x, w.x.y, w.x.z, w.x.w};
            emit(a, item.seq, item.h, row0 + r, col, y, w.m, w.mw, w.l);
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

template <int DP, int NT>
__global__ void __launch_bounds__(kThreads, kResident) rows_kernel(const __grid_constant__ AttendArgs a,
                                                                     const __grid_constant__ CodeMaps maps) {
    constexpr int S = stages(DP);
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Warp<S> s_warps[kWarps];
    __shared__ uint64_t s_warp[kWarps], s_at;
    __shared__ uint32_t s_seq;
    __shared__ int s_last;
    Merge<DP> &mg = *reinterpret_cast<Merge<DP> *>(smem + ring_bytes<DP, NT>());
    Part<DP, NT> *parts = reinterpret_cast<Part<DP, NT> *>(a.parts);
    const uint32_t B = a.c.tokens, cta = blockIdx.x;

    Warp<S> &wp = s_warps[threadIdx.x / 32];
    Stage<DP> *ring = reinterpret_cast<Stage<DP> *>(smem) + threadIdx.x / 32 * S;
    if (threadIdx.x % 32 == 0) {
        for (int i = 0; i < S; i++) bar_init(&wp.full[i], 1);
        bar_init_done();
        prefetch_map(&maps.code[0]);
        prefetch_map(&maps.code[1]);
    }

    // The line of work, and this CTA's piece [w0, w1) of it.
    uint64_t mine = 0, sum, W;
    for (uint32_t s = threadIdx.x; s < a.b.n_seqs; s += kThreads) {
        const uint64_t work = work_of<NT>(a, read_seq(a.b, s, a.d_status, B, cta == 0));
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
            mine = s < a.b.n_seqs ? work_of<NT>(a, read_seq(a.b, s, a.d_status, B, false)) : 0;
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
    bool more = next_job<NT>(a, w, w1, s, at, job);
    begin<DP>(a, maps, wp, ring, job, turn);
    while (more) {
        Sums<DP, NT> acc;
        const bool ok = attend_slices<DP, NT>(a, maps, wp, ring, job, turn, acc);
        turn += uint32_t(job.steps);
        // The next piece's first slices are on their way while this one is finished.
        more = next_job<NT>(a, w, w1, s, at, next);
        if (more && ok) begin<DP>(a, maps, wp, ring, next, turn);
        if (__syncthreads_or(!ok)) {
            if (more && ok) drain(a, wp, turn, next.steps);
            return;
        }
        const bool whole = job.whole();
        merge<DP, NT>(a, mg, job, acc, whole ? nullptr : parts + 2 * cta + (job.w == job.i0 ? 1 : 0));
        if (!whole) {
            // CTAs from that of the item's first unit to that of its last: unit u is CTA c's where
            // W c / G <= u < W (c + 1) / G, rounded down, so c = (u G + G - 1) / W
            const uint32_t c0 = uint32_t((job.i0 * G + G - 1) / W), c1 = uint32_t(((job.i1 - 1) * G + G - 1) / W);
            const uint32_t n = c1 - c0 + 1, mine = cta - c0;
            uint32_t *counter = a.counters + uint64_t(slot_of(job.seq.first, job.seq.s, a.group, 8 * NT, 1) + job.tile) * a.c.heads + job.h;
            uint8_t *space = reinterpret_cast<uint8_t *>(&mg);
            // many parts: each kGroup of them first, by the last CTA of those, then what they make
            const uint32_t groups = n <= 2 * kGroup ? 1 : (n + kGroup - 1) / kGroup, g = groups == 1 ? 0 : mine / kGroup;
            uint32_t i0 = g * kGroup, step = 1, parts_of = groups == 1 ? n : min(uint32_t(kGroup), n - i0);
            uint32_t *first = groups == 1 ? counter : a.group_counters + 2 * (c0 + i0) + (g ? 0 : 1);
            bool on = groups > 1, go = last_of(first, parts_of, s_last);
#pragma unroll 1
            while (go) {
                join<DP, NT>(a, space, job, c0, i0, step, parts_of, on);
                go = on && last_of(counter, groups, s_last);
                i0 = 0, step = kGroup, parts_of = groups, on = false;
            }
        }
        job = next;
    }
}

template <int DP, int NT> int launch(const AttendArgs &a, cudaStream_t s) {
    static std::atomic<uint64_t> ready{0};  // devices whose kernel may use this much shared memory
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ZC_ECUDA;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(rows_kernel<DP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem_bytes<DP, NT>())) != cudaSuccess)
            return ZC_ECUDA;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    CodeMaps maps;
    const int st = make_maps(a.c, DP, kSlice, maps);
    if (st != ZC_OK) return st;
    rows_kernel<DP, NT><<<uint32_t(sm_count() * kResident), kThreads, smem_bytes<DP, NT>(), s>>>(a, maps);
    return cudaGetLastError() == cudaSuccess ? ZC_OK : ZC_ECUDA;
}

template <int NT> int launch_tiles_of(const AttendArgs &a, cudaStream_t s) {
    return a.c.dim <= 64 ? launch<64, NT>(a, s) : launch<128, NT>(a, s);
}

template <int NT> uint64_t part_bytes(uint32_t dim) {
    return uint64_t(sm_count()) * kResident * 2 * (dim <= 64 ? sizeof(Part<64, NT>) : sizeof(Part<128, NT>));
}

} // namespace

uint64_t rows_counters(const Batch &b, const Cache &c, uint32_t group) {
    return uint64_t(slot_of(b.total, b.n_seqs, group, 8, 1)) * c.heads;
}

uint64_t rows_group_counters() { return uint64_t(sm_count()) * kResident * 2; }

uint64_t rows_part_bytes(const Cache &c) { return part_bytes<2>(c.dim); }

// One tile of 8 rows or two: with two, 64 sequences of 4 rows take 135 us where one takes 100.
int launch_rows(const AttendArgs &a, cudaStream_t s) {
    return std::min<uint64_t>(uint64_t(a.b.most) * a.group, a.rows_most) <= 8 ? launch_tiles_of<1>(a, s) : launch_tiles_of<2>(a, s);
}

} // namespace kv
} // namespace zc
