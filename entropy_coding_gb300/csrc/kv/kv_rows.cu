// kv_rows.cu — attention of few query rows over the 8-bit cache.
//
// A row is one query token and query head; the rows of a key/value head are
// its `group` query heads times the sequence's new tokens. With codes kc, vc
// and block scales ks, vs, over the keys j that row i sees:
//   s_ij = scale * ks_b(j) * (q_i . kc_j)
//   out_i = sum_j 2^(s_ij log2e - m) vs_b(j) vc_j / sum_j 2^(s_ij log2e - m)
//
// The work is cut along the keys (kv_rows.cuh), in units of 64.
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
#include "kv_rows.cuh"

namespace zc {
namespace kv {
namespace {

constexpr int kAhead = 32;  // steps that are looked up at a time

template <int DP> struct Codes8 {
    static constexpr int kDim = DP, kWarps = 4, kSlice = 16;
    // CTAs of an SM, as many as their registers allow, and slices of a ring, as many as fit the SM's shared memory then.
    static constexpr int kResident = 3, kStages = 3 * (128 / DP);
    template <int NT> static constexpr int resident() { return kResident; }
    static constexpr bool kEarly = false;
    static constexpr bool kMergeInRing = false, kUnits = true;
    static constexpr uint32_t kFixed = 0;
    using Maps = CodeMaps;
    struct Stage {
        uint8_t k[kSlice * DP];
        uint8_t v[kSlice * DP];
    };
    // What a warp keeps in shared memory besides its ring: the ring's barriers, and the blocks and scales of 64 of its
    // steps, read 32 at a time.
    struct Warp {
        uint64_t full[kStages];
        int32_t block[2 * kAhead];
        float ks[2 * kAhead], vs[2 * kAhead];
    };
    static __device__ __forceinline__ void look_up(const AttendArgs &a, Warp &wp, const Job &job, int k0);
    static __device__ __forceinline__ void fetch(const AttendArgs &a, const CodeMaps &maps, Warp &wp, Stage *ring, const Job &job, int k, uint32_t st);
    template <int NT>
    static __device__ __forceinline__ bool attend_slices(const AttendArgs &a, const CodeMaps &maps, Warp &wp, Stage *ring, const Job &job,
                                                         uint32_t turn, Sums<DP, NT> &acc);
};

__device__ __forceinline__ void cp4(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_of(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Where a box holds 16-byte chunk c of row r: the swizzle of the tensor maps.
template <int DP> __device__ __forceinline__ int chunk_at(int r, int c) {
    return r * DP + 16 * (c ^ (DP == 128 ? r & 7 : r >> 1 & 3));
}

// The blocks and scales of steps k0 .. k0 + 31, a step a lane. A block that is not there is read as block 0.
template <int DP> __device__ __forceinline__ void Codes8<DP>::look_up(const AttendArgs &a, Warp &wp, const Job &job, int k0) {
    const int k = k0 + (threadIdx.x & 31);
    if (k >= job.steps) return;
    const int64_t id = max(read_block(a.b, a.c, job.seq.s, block_of_16(a.c, uint32_t(job.first + k * kWarps)), a.d_status), int64_t(0));
    const int at = k & (2 * kAhead - 1);
    wp.block[at] = int32_t(id);
    cp4(&wp.ks[at], a.c.scale[0] + id * a.c.scale_stride + job.h);
    cp4(&wp.vs[at], a.c.scale[1] + id * a.c.scale_stride + job.h);
}

// Asks for step k's keys and values (one lane). Rows that nobody sees come along as they are.
template <int DP>
__device__ __forceinline__ void Codes8<DP>::fetch(const AttendArgs &a, const CodeMaps &maps, Warp &wp, Stage *ring, const Job &job, int k, uint32_t st) {
    if ((threadIdx.x & 31) == 0 && k < job.steps && !a.stall) {
        const uint32_t i = uint32_t(job.first + k * kWarps);
        const int row = int(job.h * a.c.tokens + i * kSlice - block_of_16(a.c, i) * a.c.tokens), id = wp.block[k & (2 * kAhead - 1)];
        bar_expect(&wp.full[st], sizeof(Stage));
        copy_box(ring[st].k, &maps.code[0], row, id, &wp.full[st]);
        copy_box(ring[st].v, &maps.code[1], row, id, &wp.full[st]);
    }
}

template <int DP>
template <int NT>
__device__ __forceinline__ bool Codes8<DP>::attend_slices(const AttendArgs &a, const CodeMaps &maps, Warp &wp, Stage *ring, const Job &job,
                                                          uint32_t turn, Sums<DP, NT> &acc) {
    constexpr int kRows = 8 * NT, S = kStages;
    constexpr int kSteps = DP / 16;      // inner steps of k q, and column tiles of the output
    constexpr int kRun = DP / 4;         // columns of q and k that a thread of a quad holds
    constexpr int kCols = DP / 8;        // columns of v that a thread's quad holds
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const Seq &seq = job.seq;
    const uint32_t row0 = job.tile * kRows, n_rows = seq.n * a.group;
    auto &o = acc.o;
    auto &m = acc.m;
    auto &d = acc.d;
    auto &unit = acc.unit;
    auto &l = acc.l;

    // Query fragments: row g of each tile, columns [kRun t, kRun t + kRun).
    uint32_t qf[NT][kSteps][2];
    float row_scale[NT][2];  // of rows 2t, 2t + 1 of each tile
    load_queries<DP, NT>(a, job, qf, row_scale);
    acc.clear();

    uint32_t st = turn % S, parity = turn / S & 1;  // of step k
    for (int k = 0; k < job.steps; k++) {
        if ((k & (kAhead - 1)) == 0) {
            cp_wait_all();
            __syncwarp();
            look_up(a, wp, job, k + kAhead);
        }
        if (!__all_sync(0xFFFFFFFFu, bar_wait(&wp.full[st], parity, a.limit))) {
            drain<Codes8>(a, wp, turn + k, job.steps - k);
            if (lane == 0) report(a.d_status, ZC_ETIMEOUT);
            return false;
        }
        // The stage before this one was read a step ago (the vote above comes after every lane's reads).
        fetch(a, maps, wp, ring, job, k + S - 1, st == 0 ? S - 1 : st - 1);
        Stage &sl = ring[st];
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
                // (rounded here: what is subtracted below is the same number)
                sc[n][j] = __fmul_rn(kSums == 1 ? part_sc[0][n][j] : part_sc[0][n][j] + part_sc[kSums - 1][n][j], row_scale[n][j & 1] * ks);
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
        // m and m + d follow the maxima only once these are 2^kSlack and 2^kSlackW above them: after the first step a
        // rescaling is rare. (Scores are compared by their differences, which float32 holds however large they are.)
        const float lvs = __log2f(vs);
        bool grows = false;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float top = fmaxf(sc[n][e], sc[n][2 + e]);
                grows |= top - m[n][e] > kSlack || (top - m[n][e]) + lvs > d[n][e] + kSlackW;
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
                    const float m1 = fmaxf(m[n][e], top), was = above(d[n][e], m[n][e], m1);
                    const float d1 = fmaxf(was, above(lvs, top, m1));
                    l[n][e] *= ratio2(m[n][e], m1);
                    down[e] = ratio2(was, d1);
                    m[n][e] = m1, d[n][e] = d1;
                    unit[n][e] = d1 == kNone ? 0.0f : ex2(fminf(-d1, 126.0f));
                }
#pragma unroll
                for (int c = 0; c < kSteps; c++)
                    o[n][c][0] *= down[0], o[n][c][1] *= down[1], o[n][c][2] *= down[0], o[n][c][3] *= down[1];
            }
        }
        // Weights p = 2^(s - m + kRaise), and in the output's units p * 2^(log2 vs - d). (A block that is louder than
        // the unit by more than a float holds is hardly attended to: an infinite factor would make its weights of 0 NaN.)
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; n++) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float base = m[n][e] == kNone ? 0.0f : m[n][e], f = fminf(vs * unit[n][e], FLT_MAX);
                const float p0 = ex2((sc[n][e] - base) + kRaise), p1 = ex2((sc[n][2 + e] - base) + kRaise);
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

template <int NT> int launch_tiles_of(const AttendArgs &a, cudaStream_t s) {
    return a.c.dim <= 64 ? launch<Codes8<64>, NT>(a, 16, s) : launch<Codes8<128>, NT>(a, 16, s);
}

template <int NT> uint64_t part_bytes(uint32_t dim) {
    return uint64_t(sm_count()) * Codes8<128>::kResident * 2 * (dim <= 64 ? sizeof(Part<64, NT>) : sizeof(Part<128, NT>));
}

} // namespace

uint64_t rows_counters(const Batch &b, const Cache &c, uint32_t group) {
    return uint64_t(slot_of(b.total, b.n_seqs, group, 8, 1)) * c.heads;
}

uint64_t rows_group_counters() { return uint64_t(sm_count()) * Codes8<128>::kResident * 2; }

uint64_t rows_part_bytes(const Cache &c) { return part_bytes<2>(c.dim); }

// One tile of 8 rows or two: with two, 64 sequences of 4 rows take 135 us where one takes 100.
int launch_rows(const AttendArgs &a, cudaStream_t s) {
    return std::min<uint64_t>(uint64_t(a.b.most) * a.group, a.rows_most) <= 8 ? launch_tiles_of<1>(a, s) : launch_tiles_of<2>(a, s);
}

} // namespace kv
} // namespace zc
