// kv_tiles.cu — attention of many query rows (prompts, chunks of prompts,
// longer drafts) over the 8-bit cache, on the fifth-generation tensor cores.
//
// An item is up to 256 rows of one sequence and key/value head, in two tiles
// of 128 (a row is one query token and query head, as in kv_rows.cu). Over
// tiles of 128 keys, with codes kc, vc and block scales ks, vs:
//   S = Q Kc^T            128 x 128 x dim, half operands, float32 in tensor memory
//   s_ij = S_ij ks_b c_i  (c_i: the row's power of two and the softmax scale, log2)
//   w_ij = 2^(s_ij + log2 vs_b - mw_i + 9), rounded to half, back into tensor memory
//   O += W Vc             128 x dim x 128
//   l_i += sum_b (sum_{j in b} w_ij before rounding) 2^(mw_i - 9 - m_i - log2 vs_b)
// m_i and mw_i follow the row's maxima of s and of s + log2 vs (and may lag by
// 2^8 and 2^6), so O is in units of the largest contribution and l in units of
// the largest weight: block scales cost an exponent's bias for 16 columns, and no
// spread between them loses precision; half keeps its 11 bits down to 2^-23 of
// the largest w vs. A block whose scale is 2^69 below the unit adds less than
// 2^-60 of it and counts as 2^-69. out = O 2^(mw - 9 - m) / l.
//
// Work: as in kv_rows.cu, one line of key tiles over all items (an item's
// beginning and end count as 4 tiles), an equal piece for each of one CTA an SM; items cut by a piece's end leave partial
// results, which the last CTA of the item joins.
//
// A CTA is 16 warps in roles, which meet at barriers in shared memory:
//   warps 0-3, 4-7   a row a thread of the first and second tile: scores from
//                    tensor memory, weights back, the output's rescaling and end
//   warps 8-11       codes to halves, from the ring of code tiles to the ring of
//                    operand tiles, swizzled over 128 bytes as the products read them
//   warp 12          issues the products, as operands and weights come
//   warp 13          copies: 8 boxes of 16 keys a code tile, by block table
//   warp 14          one thread finds the CTA's pieces of work ahead of the others
//   warp 15          the first CTA's looks over the batch's counts and lengths
// While one tile's rows turn scores into weights, the other tile's products
// run: 4 products of 128 x 128 x 128 a key tile, 2048 clocks of the tensor
// cores.
//
// Measured on a GB300: an 8192-token prompt (32 query heads, 8 key/value heads
// of 128, causal) in 454 to 461 us, 1.2 PFLOP/s, 0.64 of the measured bfloat16 rate;
// 912 tokens of two sequences over 28384 keys in 185 us (1.15 PFLOP/s). The
// tensor cores are busy half of the time. A key tile takes 1.7 us where its
// products take 1.05: a row tile's chain of scores, weights (about 1.1 us: two
// passes over the scores, 128 exponentials a thread on a unit shared by two
// warps, and the conversions' instructions beside them) and its own products is
// longer than the other tile's products cover. The weights stand where the
// scores were, so that the next scores wait for these sums: with 128 columns of
// output, columns for both do not fit; with 64 they would (2 x 128 of scores, 2 x
// 64 of weights, 2 x 64 of sums), which this layout does not use. An item of one
// row tile leaves half of the row threads without work. Shared memory is the next limit: by its rate the products take 1536
// clocks of it a key tile, the conversion 768, the copies 256. An item's
// beginning and end take about 7 us (queries 1.6, output 3, the first scores and
// the last sums with nothing beside them), joining a cut item 10: 32 columns and
// 2 parts at a time, read whether they are there or not (16 columns, 4 parts and
// predicated reads: 25 us).
#include <atomic>

#include "kv_attend.cuh"

namespace zc {
namespace kv {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kTile = 128;              // rows of a tile, keys of a key tile
constexpr int kRows = 2 * kTile;        // rows of an item
constexpr int kBoxes = kTile / 16;      // boxes of a code tile
constexpr int kRaw = 3, kOps = 3;       // rings of code tiles and operand tiles (keys and values in turn)
// Units of work of an item besides its key tiles: its beginning and end. (An 8192-token prompt: 0 units 895 us, 2 units
// 590, 3 units 491, 4 units 453, 5 units 457; mixed lengths 68, 56, 52, 54 and 58: with fewer, the CTAs with many short
// items are last.)
constexpr uint32_t kFixed = 4;
constexpr int kJobs = 4;                // pieces of work that are known ahead
constexpr int kReaders = 8 + 4 + 1 + 1; // warps (and the products' thread) that read them
constexpr int kSlots = 8;               // key tiles whose scales are held: the copies run up to 3 ahead of the weights
constexpr uint32_t kColumns = 512;      // of tensor memory: S (and W in its place) 0, 128, O 256, 384

// Registers of a thread by warpgroup: two of rows, the conversion, the rest. What the groups take together is what the
// CTA was launched with, 128 for each of 512 threads; a sum above that would wait for registers for ever.
constexpr int kRowRegs = 160, kConvertRegs = 96, kOtherRegs = 96;
static_assert(2 * kRowRegs + kConvertRegs + kOtherRegs <= 4 * 128, "more registers than the CTA has");

struct Bars {
    uint64_t raw_full[kRaw], raw_empty[kRaw], op_full[kOps], op_empty[kOps], scale_full[kSlots];
    uint64_t q_full[2], s_full[2], p_full[2][2], o_full[2], rows, drained;
    uint64_t job_full[kJobs], job_empty[kJobs];
};

// A piece of work: key tiles of an item.
struct Job {
    Seq seq;
    uint32_t tile, h;
    int end;                         // no piece: the line's end
    int whole;                       // the piece is the whole item; else:
    uint32_t part;                   // where its partial result goes
    uint32_t c0, c1;                 // the CTAs that have the item's first and last units
    uint64_t counter;                // the item's
    int all_lo, all_hi, x_lo, x_hi;  // keys seen by some row; by every row
    int j0, n;                       // key tiles of the piece
    int tiles;                       // of 128 rows
    __device__ __forceinline__ bool edge(int j) const { return j * kTile < x_lo || (j + 1) * kTile > x_hi; }
};

template <int DP> struct Smem {
    uint8_t q[2][kTile * DP * 2];       // panels of 64 columns: 128-byte rows, swizzled
    uint8_t op[kOps][kTile * DP * 2];
    uint8_t raw[kRaw][kTile * DP];
    uint8_t out[8][32 * 64];            // a warp's rows, 32 columns at a time
    float ks[kSlots][kBoxes], lvs[kSlots][kBoxes];
    Bars bars;
    Job jobs[kJobs];
    uint64_t sums[kWarps], i0;
    uint32_t slot, seq, h, tmem;
    int last, poison;
};

// A part of an item, rows in units of 2^mw (o) and 2^m (l), for a row a thread.
template <int DP> struct Part {
    float4 o[DP / 4][kRows];
    float m[kRows], mw[kRows], l[kRows];
};

// ---------------------------------------------------------------------------
// Tensor memory and tensor cores

__device__ __forceinline__ void tm_load32(uint32_t at, float *x) {
    uint32_t *r = reinterpret_cast<uint32_t *>(x);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(at));
}
__device__ __forceinline__ void tm_store32(uint32_t at, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                   "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
                   "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
                   "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}
__device__ __forceinline__ void tm_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Keeps the uses of 32 loaded registers behind the wait before this: to the compiler they have their values from the load on.
__device__ __forceinline__ void tm_loaded(float *x) {
    asm volatile("" : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]), "+f"(x[8]),
                 "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]), "+f"(x[15]));
    asm volatile("" : "+f"(x[16]), "+f"(x[17]), "+f"(x[18]), "+f"(x[19]), "+f"(x[20]), "+f"(x[21]), "+f"(x[22]), "+f"(x[23]),
                 "+f"(x[24]), "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]), "+f"(x[29]), "+f"(x[30]), "+f"(x[31]));
}
__device__ __forceinline__ void tm_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Operand descriptors: 128-byte rows swizzled over 8-row atoms of 1024 bytes, atoms 1024 bytes apart. Of keys and
// queries the rows are rows and the inner index runs along them (the leading offset is not used); of values the inner
// index are the rows, and panels of 64 columns are `panel` bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t smem, uint32_t panel) {
    return uint64_t(smem >> 4 & 0x3FFF) | uint64_t(panel >> 4 & 0x3FFF) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 |
           uint64_t(2) << 61;
}
// Float32 sums of half products, 128 rows, n columns; the second operand's inner index along its rows or columns.
__host__ __device__ constexpr uint32_t product(uint32_t n, bool values) {
    return 1u << 4 | uint32_t(values) << 16 | n / 8 << 17 | 128u / 16 << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, uint32_t add) {
    asm volatile("{.reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;}" ::"r"(d), "l"(a),
                 "l"(b), "r"(kind), "r"(add) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, uint32_t add) {
    asm volatile("{.reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;}" ::"r"(d), "r"(a),
                 "l"(b), "r"(kind), "r"(add) : "memory");
}
// The barrier is arrived at when all products issued so far are done.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_of(bar)) : "memory");
}

__device__ __forceinline__ bool elected() {
    uint32_t p;
    asm volatile("{.reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p;}" : "=r"(p));
    return p;
}

template <int N> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void fma2(float &x, float &y, float a0, float a1, float b, float c) {  // x, y = a0 b + c, a1 b + c
    asm("{.reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %4}; mov.b64 c, {%5, %5}; fma.rn.f32x2 d, a, b, c; mov.b64 {%0, %1}, d;}"
        : "=f"(x), "=f"(y) : "f"(a0), "f"(a1), "f"(b), "f"(c));
}

// Where an operand tile holds 16-byte chunk c of row r.
__device__ __forceinline__ int panel_at(int r, int c) { return c / 8 * (kTile * 128) + r * 128 + 16 * (c % 8 ^ (r & 7)); }

__device__ __forceinline__ void add2(float &x, float &y, float a, float b) {  // x + a, y + b
    asm("{.reg .b64 c, d; mov.b64 c, {%0, %1}; mov.b64 d, {%2, %3}; add.rn.f32x2 c, c, d; mov.b64 {%0, %1}, c;}" : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}

// ---------------------------------------------------------------------------
// The line of work

// Work of an item of this slot (a sequence's run of 256 rows): kFixed units and one for each of its key tiles (or one);
// 0 if it is empty or not this kernel's.
__device__ __forceinline__ uint32_t units_of(const AttendArgs &a, const Seq &seq, uint32_t tile, Job &job) {
    const uint32_t n_rows = seq.n * a.group, row0 = tile * kRows;
    if (!seq.ok || n_rows <= a.rows_most || tile > (n_rows - 1) / kRows) return 0;
    job.seq = seq;
    job.tile = tile;
    bounds(a, seq, row0, job.all_lo, job.x_hi);
    bounds(a, seq, min(row0 + kRows, n_rows) - 1, job.x_lo, job.all_hi);
    job.tiles = n_rows - row0 > kTile ? 2 : 1;
    return kFixed + uint32_t(max((job.all_hi + kTile - 1) / kTile - job.all_lo / kTile, 1));
}

__device__ __forceinline__ uint32_t first_slot(const AttendArgs &a, uint32_t s) {
    return slot_of(tokens_before(a.b, s), s, a.group, kRows, 1);
}

// The sequence that slot u belongs to, by halving.
__device__ __forceinline__ uint32_t seq_of_slot(const AttendArgs &a, uint32_t u) {
    uint32_t lo = 0, hi = a.b.n_seqs;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (first_slot(a, mid) <= u) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Where the CTA has got to on the line. Where the counts fall, the slots that the walk passes need not be those that
// the line's length was taken from (a sequence is looked up by halving there): it ends with the slots and with the line.
struct Walk {
    uint64_t w, w1, i0;   // next work; the end; where the item begins
    uint64_t W, G;        // all work; the CTAs that share it
    uint32_t slot, s, h;  // the item
    uint32_t slots;       // of the batch
    __device__ __forceinline__ bool next(const AttendArgs &a, Job &job) {
        while (w < w1 && slot < slots) {
            const uint32_t units = units_of(a, read_seq(a.b, s, a.d_status, a.c.tokens, false), slot - first_slot(a, s), job);
            if (w >= i0 + units) {
                i0 += units;
                if (units && ++h < a.c.heads) continue;
                h = 0;
                slot++;
                while (s + 1 < a.b.n_seqs && first_slot(a, s + 1) <= slot) s++;
                continue;
            }
            const uint64_t first = i0 + kFixed, i1 = i0 + units, from = max(w, first), upto = min(w1, i1);
            if (i1 > W) return false;
            w = upto;
            if (upto <= first) continue;  // the piece ends within the item's beginning, which belongs to the first tile's piece
            job.h = h;
            job.j0 = job.all_lo / kTile + int(from - first);
            job.n = max(min(int(upto - from), (job.all_hi + kTile - 1) / kTile - job.j0), 0);
            job.whole = from == first && upto == i1;
            job.part = 2 * blockIdx.x + (from == first ? 1 : 0);
            if (!job.whole) {
                // CTA c has the units [W c / G, W (c + 1) / G), rounded down: unit u is CTA (u G + G - 1) / W's
                job.c0 = uint32_t((first * G + G - 1) / W);
                job.c1 = uint32_t(((i1 - 1) * G + G - 1) / W);
                job.counter = uint64_t(first_slot(a, s) + job.tile) * a.c.heads + h;
            }
            job.end = 0;
            return true;
        }
        return false;
    }
};

// ---------------------------------------------------------------------------
// Roles. Each returns false if a wait was given up.

// Finds the CTA's pieces of work ahead of the others (one thread).
template <int DP> __device__ __forceinline__ bool find_role(const AttendArgs &a, Smem<DP> &sm, Walk walk) {
    for (uint32_t k = 0;; k++) {
        Job job;
        const bool more = walk.next(a, job);
        if (!bar_wait(&sm.bars.job_empty[k % kJobs], (k / kJobs & 1) ^ 1, a.limit)) return false;
        job.end = !more;
        sm.jobs[k % kJobs] = job;
        bar_arrive(&sm.bars.job_full[k % kJobs]);
        if (!more) return true;
    }
}
template <int DP> __device__ __forceinline__ bool job_ready(Smem<DP> &sm, uint32_t k, long long limit) {
    return bar_wait(&sm.bars.job_full[k % kJobs], k / kJobs & 1, limit);
}
// A reader is done with piece k (a warp, or the products' thread).
template <int DP> __device__ __forceinline__ void job_done(Smem<DP> &sm, uint32_t k) { bar_arrive(&sm.bars.job_empty[k % kJobs]); }

template <int DP>
__device__ __forceinline__ bool copy_role(const AttendArgs &a, const CodeMaps &maps, Smem<DP> &sm) {
    const int lane = threadIdx.x & 31;
    uint32_t item = 0, tile = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; k++) {
        if (!(ok = __all_sync(0xFFFFFFFFu, job_ready(sm, k, a.limit)))) break;
        const Job &job = sm.jobs[k % kJobs];
        if (job.end) break;
        const int least = job.all_lo / 16, last = (job.all_hi - 1) / 16;  // boxes without a key that is seen hold others again
        for (int j = job.j0; j < job.j0 + job.n && ok; j++, tile++) {
            const int slot = tile % kSlots;
            int id = 0, row = 0;
            if (lane < kBoxes) {
                const uint32_t i = uint32_t(min(max(j * kBoxes + lane, least), last)), blk = block_of_16(a.c, i);
                id = int(max(read_block(a.b, a.c, job.seq.s, blk, a.d_status), int64_t(0)));
                row = int(job.h * a.c.tokens + i * 16 - blk * a.c.tokens);
                const int64_t at = id * a.c.scale_stride + job.h;
                sm.ks[slot][lane] = __ldg(a.c.scale[0] + at);
                sm.lvs[slot][lane] = __log2f(__ldg(a.c.scale[1] + at));
            }
            __syncwarp();
            if (lane == 0) bar_arrive(&sm.bars.scale_full[slot]);
#pragma unroll
            for (int kv = 0; kv < 2 && ok; kv++, item++) {
                if (a.stall) return true;
                const int r = item % kRaw;
                ok = __all_sync(0xFFFFFFFFu, bar_wait(&sm.bars.raw_empty[r], (item / kRaw & 1) ^ 1, a.limit));
                if (!ok) break;
                if (lane == 0) bar_expect(&sm.bars.raw_full[r], kTile * DP);
                __syncwarp();
                if (lane < kBoxes) copy_box(sm.raw[r] + lane * 16 * DP, &maps.code[kv], row, id, &sm.bars.raw_full[r]);
            }
        }
        __syncwarp();
        if (lane == 0) job_done(sm, k);
    }
    // The CTA outlives its copies, also those of a call that is given up.
    for (uint32_t k = item > kRaw ? item - kRaw : 0; k < item; k++) ok &= bar_wait(&sm.bars.raw_full[k % kRaw], k / kRaw & 1, a.limit);
    return ok;
}

template <int DP> __device__ __forceinline__ bool convert_role(Smem<DP> &sm, long long limit) {
    const int t = threadIdx.x - 256, lane = t & 31;
    uint32_t item = 0;
    for (uint32_t k = 0;; k++) {
        if (!__all_sync(0xFFFFFFFFu, job_ready(sm, k, limit))) return false;
        const Job &job = sm.jobs[k % kJobs];
        if (job.end) return true;
        for (int j = job.j0; j < job.j0 + job.n; j++)
#pragma unroll 1
            for (int kv = 0; kv < 2; kv++, item++) {
                const int r = item % kRaw, c = item % kOps;
                if (!__all_sync(0xFFFFFFFFu, bar_wait(&sm.bars.raw_full[r], item / kRaw & 1, limit) &&
                                                 bar_wait(&sm.bars.op_empty[c], (item / kOps & 1) ^ 1, limit)))
                    return false;
                // A row that does not see a key has weight 0 for it, but 0 * NaN is NaN: where some row does not see all
                // keys, NaN codes of values are taken out, and rows that see them get them at the end.
                const bool edge = kv && job.edge(j);
                constexpr int kChunks = DP / 16;
                // 8 lanes take 8 rows of one chunk: reads and writes of a quarter warp meet all banks
                auto chunk = [&](int i, int &row, int &ch) {
                    const int u = i * 128 + t;
                    row = u % 8 + u / (8 * kChunks) * 8, ch = u / 8 % kChunks;
                    return reinterpret_cast<uint4 *>(sm.raw[r] + row * DP + 16 * (ch ^ (DP == 128 ? row & 7 : row >> 1 & 3)));
                };
                int row, ch;
                if (edge) {
#pragma unroll 1
                    for (int i = 0; i < kTile * kChunks / 128; i++) {
                        uint32_t *w = reinterpret_cast<uint32_t *>(chunk(i, row, ch));
#pragma unroll 1
                        for (int k = 0; k < 4; k++) {
                            if (!any_nan(w[k])) continue;
                            w[k] &= ~__vcmpeq4(w[k] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                            if (j * kTile + row >= job.all_lo && j * kTile + row < job.all_hi) sm.poison = 1;
                        }
                    }
                }
                uint4 in[kTile * kChunks / 128];  // all reads first: the products' reads of shared memory go before them
#pragma unroll
                for (int i = 0; i < kTile * kChunks / 128; i++) in[i] = *chunk(i, row, ch);
#pragma unroll
                for (int i = 0; i < kTile * kChunks / 128; i++) {
                    const uint4 v = in[i];
                    chunk(i, row, ch);
                    uint4 lo, hi;
                    e4m3x4_to_half2x2(v.x, lo.x, lo.y);
                    e4m3x4_to_half2x2(v.y, lo.z, lo.w);
                    e4m3x4_to_half2x2(v.z, hi.x, hi.y);
                    e4m3x4_to_half2x2(v.w, hi.z, hi.w);
                    *reinterpret_cast<uint4 *>(sm.op[c] + panel_at(row, 2 * ch)) = lo;
                    *reinterpret_cast<uint4 *>(sm.op[c] + panel_at(row, 2 * ch + 1)) = hi;
                }
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(&sm.bars.raw_empty[r]), bar_arrive(&sm.bars.op_full[c]);
            }
        __syncwarp();
        if (lane == 0) job_done(sm, k);
    }
}

// A warp whose elected thread issues; the others keep its addresses uniform, as the products want them.
template <int DP> __device__ __forceinline__ bool product_role(Smem<DP> &sm, long long limit) {
    constexpr uint32_t kPanel = kTile * 128;
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, sm.tmem, 0);
    const bool one = elected();
    const uint64_t q0 = operand(smem_of(sm.q[0]), 0), k0 = operand(smem_of(sm.op[0]), 0), v0 = operand(smem_of(sm.op[0]), kPanel);
    constexpr uint32_t kQ = sizeof(sm.q[0]) >> 4, kOp = sizeof(sm.op[0]) >> 4;
    uint32_t item = 0, queries[2] = {0, 0}, weights[2] = {0, 0};
    auto scores = [&](int t, uint32_t c) {
        const uint64_t q = q0 + t * kQ, k = k0 + c * kOp;
        if (one) {
#pragma unroll
            for (int i = 0; i < DP / 16; i++) {  // 16 columns: 32 bytes on within a panel
                const uint32_t at = (i / 4 * kPanel + i % 4 * 32) >> 4;
                mma_ss(tm + t * 128, q + at, k + at, product(kTile, false), i > 0);
            }
        }
        __syncwarp();
    };
    // half of the key tile's sums: 64 keys
    auto sums = [&](int t, uint32_t c, int part, bool add) {
        const uint64_t v = v0 + c * kOp;
        if (one) {
#pragma unroll
            for (int i = 0; i < kTile / 32; i++) {  // 16 keys: 8 columns of weights, 16 rows of values
                const int at = part * (kTile / 32) + i;
                mma_ts(tm + 256 + t * 128, tm + t * 128 + 8 * at, v + (at * 16 * 128 >> 4), product(DP, true), add || i > 0);
            }
        }
        __syncwarp();
    };
    auto commit = [&](uint64_t *bar) {
        if (one) mma_commit(bar);
        __syncwarp();
    };
    auto wait = [&](uint64_t *bar, uint32_t parity) { return bool(__all_sync(0xFFFFFFFFu, bar_wait(bar, parity, limit))); };
    bool ok = true;
    for (uint32_t k = 0; ok; k++) {
        if (!(ok = __all_sync(0xFFFFFFFFu, job_ready(sm, k, limit)))) break;
        const Job &job = sm.jobs[k % kJobs];
        const int n = __shfl_sync(0xFFFFFFFFu, job.n, 0), tiles = __shfl_sync(0xFFFFFFFFu, job.tiles, 0);
        if (__shfl_sync(0xFFFFFFFFu, job.end, 0)) break;
        if (one) job_done(sm, k);
        if (!n) continue;
        ok = wait(&sm.bars.op_full[item % kOps], item / kOps & 1);
        for (int t = 0; t < tiles && ok; t++) {
            ok = wait(&sm.bars.q_full[t], queries[t]++ & 1);
            if (!ok) break;
            tm_after();
            scores(t, item % kOps);
            commit(&sm.bars.s_full[t]);
        }
        if (!ok) break;
        commit(&sm.bars.op_empty[item % kOps]);
        item++;
        for (int j = 0; j < n && ok; j++) {
            const uint32_t v = item, next = item + 1;
            item += j + 1 < n ? 2 : 1;
            ok = wait(&sm.bars.op_full[v % kOps], v / kOps & 1);
            for (int t = 0; t < tiles && ok; t++) {
                for (int part = 0; part < 2 && ok; part++) {
                    ok = wait(&sm.bars.p_full[t][part], weights[t] & 1);
                    if (!ok) break;
                    tm_after();
                    sums(t, v % kOps, part, j > 0 || part > 0);
                }
                if (!ok) break;
                weights[t]++;
                if (t == tiles - 1) commit(&sm.bars.op_empty[v % kOps]);
                if (j + 1 < n) {
                    if (t == 0) ok = wait(&sm.bars.op_full[next % kOps], next / kOps & 1);
                    if (!ok) break;
                    tm_after();
                    scores(t, next % kOps);
                    commit(&sm.bars.s_full[t]);
                    if (t == tiles - 1) commit(&sm.bars.op_empty[next % kOps]);
                } else {
                    commit(&sm.bars.o_full[t]);
                }
            }
        }
    }
    // Tensor memory is freed once the products are done, also those of a call that is given up.
    commit(&sm.bars.drained);
    return wait(&sm.bars.drained, 0) && ok;
}

// Columns [col, col + 32) of values that are NaN at keys that the row [lo, hi) sees, among the piece's key tiles where
// NaN was taken out; a bit a column.
__device__ __noinline__ uint32_t poisoned(const AttendArgs &a, const Job &job, int lo, int hi, int col) {
    uint32_t mask = 0;
#pragma unroll 1
    for (int j = job.j0; j < job.j0 + job.n; j++) {
        if (!job.edge(j)) continue;
#pragma unroll 1
        for (int key = max(j * kTile, lo); key < min((j + 1) * kTile, hi); key++) {
            const uint32_t blk = block_of_16(a.c, uint32_t(key) / 16);
            const int64_t id = max(read_block(a.b, a.c, job.seq.s, blk, a.d_status), int64_t(0));
            const uint8_t *v = a.c.code[1] + id * a.c.block_stride + (int64_t(job.h) * a.c.tokens + (key - blk * a.c.tokens)) * a.c.dim + col;
#pragma unroll 1
            for (int i = 0; i < min(32, int(a.c.dim) - col); i++)
                if ((__ldg(v + i) & 0x7F) == 0x7F) mask |= 1u << i;
        }
    }
    return mask;
}

// An item's parts together, by the 256 row threads: kCols columns of a row at a time, kRun parts in flight together.
// Apart from the loop over key tiles, whose registers are all taken.
template <int DP, int kCols, int kRun> __device__ __noinline__ void join_rows(const AttendArgs &a, const Job &job) {
    const Part<DP> *parts = static_cast<const Part<DP> *>(a.parts);
    const uint32_t c0 = job.c0, c1 = job.c1;
    // kCols columns of a row at a time, whichever rows there are
    const uint32_t rows = min(uint32_t(kRows), job.seq.n * a.group - job.tile * kRows), cols = a.c.dim;
#pragma unroll 1
    for (uint32_t u = threadIdx.x; u < rows * ((cols + kCols - 1) / kCols); u += 256) {
        const uint32_t r = u % rows, row = job.tile * kRows + r;
        const int i = int(u / rows) * kCols;
        float o[kCols / 16][16], M = kNone, W = kNone, L = 0.0f;
#pragma unroll
        for (int k = 0; k < kCols; k++) o[k / 16][k % 16] = 0.0f;
#pragma unroll 1
        for (uint32_t c = c0; c <= c1; c += kRun) {
            float4 v[kRun][kCols / 4];
            float pm[kRun], pw[kRun], pl[kRun];
#pragma unroll
            for (int n = 0; n < kRun; n++) {
                // the first part is in its CTA's second slot, the others in the first slots of the CTAs after it
                const uint32_t at = min(c + n, c1);
                const Part<DP> &p = parts[2 * at + (at == c0 ? 1 : 0)];
                pm[n] = __ldcg(&p.m[r]), pw[n] = __ldcg(&p.mw[r]), pl[n] = __ldcg(&p.l[r]);
#pragma unroll
                for (int k = 0; k < kCols / 4; k++) v[n][k] = __ldcg(&p.o[i / 4 + k][r]);
            }
#pragma unroll
            for (int n = 1; n < kRun; n++) {
                if (c + n > c1) {
                    pm[n] = pw[n] = kNone, pl[n] = 0.0f;
#pragma unroll
                    for (int k = 0; k < kCols / 4; k++) v[n][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
            }
            float m1 = M, w1 = W;
#pragma unroll
            for (int n = 0; n < kRun; n++) m1 = fmaxf(m1, pm[n]), w1 = fmaxf(w1, pw[n]);
            const float down = ratio2(W, w1);
            L *= ratio2(M, m1);
#pragma unroll
            for (int k = 0; k < kCols; k++) o[k / 16][k % 16] *= down;
#pragma unroll
            for (int n = 0; n < kRun; n++) {
                L += pl[n] * ratio2(pm[n], m1);
                const float f = ratio2(pw[n], w1);
#pragma unroll
                for (int k = 0; k < kCols / 4; k++) {
                    float *x = o[k / 4] + k % 4 * 4;
                    x[0] += v[n][k].x * f, x[1] += v[n][k].y * f, x[2] += v[n][k].z * f, x[3] += v[n][k].w * f;
                }
            }
            M = m1, W = w1;
        }
        const float by = row_factor(M, W, L);
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out.p) + row_at(a, a.out, job.seq, job.h, row) + i);
#pragma unroll
        for (int k = 0; k < kCols; k += 8) {
            const float *x = o[k / 16] + k % 16;
            if (i + k < int(cols))
                out[k / 8] = L == 0.0f ? make_uint4(0, 0, 0, 0) : make_uint4(pack_out(a, x[0] * by, x[1] * by), pack_out(a, x[2] * by, x[3] * by),
                                                                             pack_out(a, x[4] * by, x[5] * by), pack_out(a, x[6] * by, x[7] * by));
        }
        if (a.lse && i == 0) *lse_at(a, job.seq, job.h, row) = row_lse(M, L);
    }
}

// The lowest n bits (none for n < 0, all from 32 on).
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1; }

// The 256 row threads meet; false if that was given up.
__device__ __forceinline__ bool rows_meet(uint64_t *bar, uint32_t turn, long long limit) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) bar_arrive(bar);
    return __all_sync(0xFFFFFFFFu, bar_wait(bar, turn & 1, limit));
}

constexpr int kNoRow = -1;

// Asks for the warp's query rows of a piece, whole rows at a time (the tile's memory is not in use).
template <int DP> __device__ __forceinline__ void fetch_queries(const AttendArgs &a, Smem<DP> &sm, const Job &job) {
    constexpr int kLanes = DP / 8, kAtOnce = 32 / kLanes;  // lanes of a row, 16 bytes each
    const int r = threadIdx.x, half = r / kTile, lane = r & 31, ch = lane % kLanes;
    if (job.end || !job.n || half >= job.tiles) return;
    const uint32_t row = job.tile * kRows + r;
    const int64_t from = row < job.seq.n * a.group ? row_at(a, a.q, job.seq, job.h, row) : kNoRow;
#pragma unroll 4
    for (int i = 0; i < kLanes; i++) {
        const int of = i * kAtOnce + lane / kLanes;
        const int64_t at = __shfl_sync(0xFFFFFFFFu, from, of);
        const bool take = at != kNoRow && ch * 8 < int(a.c.dim);
        const uint32_t dst = smem_of(sm.q[half] + panel_at(r % kTile - lane + of, ch)), n = take ? 16 : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(static_cast<const uint16_t *>(a.q.p) + (take ? at + ch * 8 : 0)),
                     "r"(n) : "memory");
    }
}

// The row is there: exact in half by a power of two, with the sign of the scale. Returns the scale of its scores.
template <int DP> __device__ __forceinline__ float ready_query(const AttendArgs &a, Smem<DP> &sm) {
    const int r = threadIdx.x, half = r / kTile;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    const uint32_t sign = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
    float c = fabsf(a.scale_log2), up = 1.0f;
    if (a.dtype == ZC_BF16) {
        __nv_bfloat162 most = __float2bfloat162_rn(0.0f);
#pragma unroll
        for (int i = 0; i < DP / 8; i++) {
            const uint4 v = *reinterpret_cast<const uint4 *>(sm.q[half] + panel_at(r % kTile, i));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; k++) most = __hmax2_nan(most, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[k])));
        }
        float down;
        row_powers(__float_as_uint(fmaxf(__low2float(most), __high2float(most))), up, down);
        c *= down;
    }
    if (a.dtype == ZC_BF16 || sign) {
#pragma unroll 4
        for (int i = 0; i < DP / 8; i++) {
            uint4 *at = reinterpret_cast<uint4 *>(sm.q[half] + panel_at(r % kTile, i));
            const uint4 v = *at;
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if (a.dtype == ZC_BF16) {
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const float2 f = unpack2<ZC_BF16>(w[k]);
                    w[k] = half2_of(f.x * up, f.y * up);
                }
            }
            *at = make_uint4(w[0] ^ sign, w[1] ^ sign, w[2] ^ sign, w[3] ^ sign);
        }
    }
    fence_async();
    __syncwarp();
    if ((r & 31) == 0) bar_arrive(&sm.bars.q_full[half]);
    return c;
}

template <int DP>
__device__ __forceinline__ bool rows_role(const AttendArgs &a, Smem<DP> &sm) {
    Part<DP> *parts = reinterpret_cast<Part<DP> *>(a.parts);
    const int r = threadIdx.x, half = r / kTile;                 // row of the item; its tile
    const int lane = r & 31;
    const uint32_t lanes = uint32_t(r / 32 % 4 * 32) << 16;      // of tensor memory
    const uint32_t tmS = sm.tmem + half * 128 + lanes, tmO = sm.tmem + 256 + half * 128 + lanes;
    uint32_t tile = 0, scored = 0, summed = 0, met = 0;
    if (!__all_sync(0xFFFFFFFFu, job_ready(sm, 0, a.limit))) return false;
    fetch_queries(a, sm, sm.jobs[0]);
    for (uint32_t k = 0;; k++) {
        const Job &job = sm.jobs[k % kJobs], &next = sm.jobs[(k + 1) % kJobs];
        if (job.end) return true;
        const uint32_t row = job.tile * kRows + r, n_rows = job.seq.n * a.group;
        const bool mine = row < n_rows;
        const bool idle = !__any_sync(0xFFFFFFFFu, mine);  // a warp without rows: its weights may be anything
        int lo = 0, hi = 0;
        if (mine) bounds(a, job.seq, row, lo, hi);
        float m = kNone, mw = kNone, l = 0.0f;
        if (job.n && half >= job.tiles) tile += job.n;  // no rows in this tile
        if (job.n && half < job.tiles) {
            const float c = ready_query(a, sm);
            {
                for (int j = job.j0; j < job.j0 + job.n; j++, tile++, scored++) {
                    const int slot = tile % kSlots;
                    // A half that had no rows in the pieces before may be ahead of the copies by more than the ring of scales,
                    // where a wait for a phase tells nothing: its first scores come after their scales.
                    if (j == job.j0 && !__all_sync(0xFFFFFFFFu, bar_wait(&sm.bars.s_full[half], scored & 1, a.limit))) return false;
                    if (!__all_sync(0xFFFFFFFFu, bar_wait(&sm.bars.scale_full[slot], tile / kSlots & 1, a.limit))) return false;
                    float by[kBoxes], lvs[kBoxes];  // read early: the products keep shared memory busy
#pragma unroll
                    for (int b = 0; b < kBoxes; b += 4) {
                        const float4 u = *reinterpret_cast<const float4 *>(&sm.ks[slot][b]), v = *reinterpret_cast<const float4 *>(&sm.lvs[slot][b]);
                        by[b] = u.x, by[b + 1] = u.y, by[b + 2] = u.z, by[b + 3] = u.w;
                        lvs[b] = v.x, lvs[b + 1] = v.y, lvs[b + 2] = v.z, lvs[b + 3] = v.w;
                    }
                    const bool edge = job.edge(j);
#pragma unroll
                    for (int b = 0; b < kBoxes; b++) by[b] = fmaxf(c * by[b], 1e-37f);  // (0 * -infinity would be NaN)
                    if (!__all_sync(0xFFFFFFFFu, bar_wait(&sm.bars.s_full[half], scored & 1, a.limit))) return false;
                    if (idle) {
                        if (lane == 0) bar_arrive(&sm.bars.p_full[half][0]), bar_arrive(&sm.bars.p_full[half][1]);
                        continue;
                    }
                    tm_after();
                    const int from = lo - j * kTile, to = hi - j * kTile;
                    // 64 scores at a time, for their maxima and then for the weights: with all 128 in registers the loop spilled
                    // (drafts 27 us, with 64 25 us)
                    auto scores64 = [&](int part, float (&x)[64]) {
                        tm_load32(tmS + 64 * part, x);
                        tm_load32(tmS + 64 * part + 32, x + 32);
                        tm_wait_load();
                        tm_loaded(x);
                        tm_loaded(x + 32);
                        if (edge) {
#pragma unroll
                            for (int q = 0; q < 64; q += 32) {
                                const uint32_t seen = below(to - 64 * part - q) & ~below(from - 64 * part - q);
#pragma unroll
                                for (int i = 0; i < 32; i++) x[q + i] = seen >> i & 1 ? x[q + i] : kNone;
                            }
                        }
                    };
                    float top = kNone, topw = kNone;
                    float x[64];
#pragma unroll
                    for (int part = 1; part >= 0; part--) {
                        scores64(part, x);
#pragma unroll
                        for (int b = 0; b < 4; b++) {
                            float g = x[16 * b];
#pragma unroll
                            for (int i = 1; i < 16; i++) g = fmaxf(g, x[16 * b + i]);
                            g *= by[4 * part + b];
                            top = fmaxf(top, g);
                            topw = fmaxf(topw, g + lvs[4 * part + b]);
                        }
                    }
                    // As in kv_rows.cu: the maxima are followed once they have grown by 2^kSlack or 2^kSlackW.
                    const bool grows = top > m + kSlack || topw > mw + kSlackW;
                    if (__any_sync(0xFFFFFFFFu, grows)) {
                        float down = 1.0f;
                        if (grows) {
                            const float m1 = fmaxf(m, top), w1 = fmaxf(mw, topw);
                            l *= ratio2(m, m1);
                            down = ratio2(mw, w1);
                            m = m1, mw = w1;
                        }
                        // the last sums are done: the scores were issued after them
                        if (j > job.j0) {
#pragma unroll 1
                            for (int i = 0; i < DP; i += 32) {
                                float o[32];
                                tm_load32(tmO + i, o);
                                tm_wait_load();
                                tm_loaded(o);
#pragma unroll
                                for (int k = 0; k < 32; k++) o[k] *= down;
                                tm_store32(tmO + i, reinterpret_cast<uint32_t *>(o));
                            }
                        }
                    }
                    const float base = m == kNone ? 0.0f : m;
                    uint32_t *p = reinterpret_cast<uint32_t *>(x);
#pragma unroll
                    for (int part = 0; part < 2; part++) {  // the products start on the first 64 keys' weights
                        // (the weights take the columns of scores 0 to 63; those from 64 on are there until the next products)
                        if (part) scores64(1, x);
#pragma unroll
                        for (int b = 0; b < 4; b++) {
                            const float lf = fminf(fmaxf(lvs[4 * part + b] + (base - mw + kRaise), -60.0f), 126.0f);  // (mw = -infinity: every vs is 0)
                            const float bias = lf - base;
                            float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                float y0, y1;
                                fma2(y0, y1, x[16 * b + i], x[16 * b + i + 1], by[4 * part + b], bias);
                                y0 = ex2(y0), y1 = ex2(y1);
                                add2(sum0, sum1, y0, y1);
                                p[8 * b + i / 2] = half2_of(y0, y1);
                            }
                            l += (sum0 + sum1) * ex2(-lf);
                        }
                        tm_store32(tmS + 32 * part, p);
                        tm_wait_store();
                        tm_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive(&sm.bars.p_full[half][part]);
                    }
                }
                if (!__all_sync(0xFFFFFFFFu, bar_wait(&sm.bars.o_full[half], summed++ & 1, a.limit))) return false;
                tm_after();
            }
        }

        // The next piece's queries are on their way while this one is finished.
        if (!__all_sync(0xFFFFFFFFu, job_ready(sm, k + 1, a.limit))) return false;
        fetch_queries(a, sm, next);

        // The rows' ends: finished, or a part.
        const bool whole = job.whole;
        Part<DP> *part = parts + job.part;
        if (half < job.tiles) {
            const float by = row_factor(m, mw, l);
            const bool poison = job.n && *reinterpret_cast<volatile int *>(&sm.poison);
            const int64_t to = mine ? row_at(a, a.out, job.seq, job.h, row) : kNoRow;
            uint8_t *stage = sm.out[r / 32];
            // (all columns in flight: an 8192-token prompt in 452 us, 32 at a time in 476)
#pragma unroll
            for (int i = 0; i < DP; i += 32) {
                float o[32];
                if (job.n) {
                    tm_load32(tmO + i, o);
                    tm_wait_load();
                    tm_loaded(o);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; k++) o[k] = 0.0f;
                }
                if (poison && mine && i < int(a.c.dim)) {
                    const uint32_t mask = poisoned(a, job, lo, hi, i);
#pragma unroll
                    for (int k = 0; k < 32; k++)
                        if (mask >> k & 1) o[k] = NAN;
                }
                if (!whole) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4) __stcg(&part->o[(i + k) / 4][r], make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]));
                } else {
                    // through shared memory, so that a warp writes 64 bytes of each of 8 rows at a time
                    uint32_t w[16];
                    if (l == 0.0f) {
#pragma unroll
                        for (int k = 0; k < 16; k++) w[k] = 0;
                    } else if (a.dtype == ZC_BF16) {
#pragma unroll
                        for (int k = 0; k < 16; k++) w[k] = pack2<ZC_BF16>(o[2 * k] * by, o[2 * k + 1] * by);
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; k++) w[k] = pack2<ZC_FP16>(o[2 * k] * by, o[2 * k + 1] * by);
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        *reinterpret_cast<uint4 *>(stage + lane * 64 + 16 * (k ^ (lane >> 1 & 3))) =
                            make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const int of = 8 * k + lane / 4, ch = lane % 4;
                        const int64_t at = __shfl_sync(0xFFFFFFFFu, to, of);
                        const uint4 v = *reinterpret_cast<const uint4 *>(stage + of * 64 + 16 * (ch ^ (of >> 1 & 3)));
                        if (at != kNoRow && i + ch * 8 < int(a.c.dim))
                            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out.p) + at + i + ch * 8) = v;
                    }
                }
            }
            if (!whole) __stcg(&part->m[r], m), __stcg(&part->mw[r], mw), __stcg(&part->l[r], l);
            else if (mine && a.lse) *lse_at(a, job.seq, job.h, row) = row_lse(m, l);
            tm_before();
        }
        if (!whole) {
            if (!rows_meet(&sm.bars.rows, met++, a.limit)) return false;
            if (r == 0) {
                uint32_t *counter = a.counters + job.counter;
                uint32_t done;
                asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(done) : "l"(counter) : "memory");
                const bool last = done == job.c1 - job.c0;
                if (last) *counter = 0;
                sm.last = last;
            }
            if (!rows_meet(&sm.bars.rows, met++, a.limit)) return false;
            if (*reinterpret_cast<volatile int *>(&sm.last)) join_rows<DP, 32, 2>(a, job);
        }
        __syncwarp();
        if (lane == 0) job_done(sm, k);
    }
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) tiles_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CodeMaps maps) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Smem<DP> &sm = *reinterpret_cast<Smem<DP> *>(smem);
    const uint32_t cta = blockIdx.x;
    const int warp = threadIdx.x / 32;

    // The line of work, and this CTA's piece of it.
    const uint32_t slots = slot_of(a.b.total, a.b.n_seqs, a.group, kRows, 1);
    auto work_at = [&](uint32_t u, uint32_t &s, uint32_t &units) -> uint64_t {
        Job job;
        s = seq_of_slot(a, u);
        units = units_of(a, read_seq(a.b, s, a.d_status, a.c.tokens, false), u - first_slot(a, s), job);
        return uint64_t(units) * a.c.heads;
    };
    uint64_t mine = 0, sum, W;
    uint32_t s = 0, units = 0;
    for (uint32_t u = threadIdx.x; u < slots; u += kThreads) mine += work_at(u, s, units);
    sum = block_scan<kWarps>(mine, sm.sums, W);
    const uint64_t G = min(uint64_t(gridDim.x), W);  // no CTA between two that have work is without
    if (cta >= G) {
        if (cta == 0) report_batch(a.b, a.c.tokens, a.d_status, threadIdx.x, kThreads, false);
        return;
    }
    const uint64_t w0 = W * cta / G, w1 = W * (cta + 1) / G;
    uint64_t before = 0;
    for (uint32_t u0 = 0; u0 < slots; u0 += kThreads) {
        if (slots > kThreads) {  // more than one round: the sums above were not of single slots
            mine = u0 + threadIdx.x < slots ? work_at(u0 + threadIdx.x, s, units) : 0;
            uint64_t all;
            sum = before + block_scan<kWarps>(mine, sm.sums, all);
            before += all;
        }
        if (mine && sum > w0 && sum - mine <= w0) {
            sm.slot = u0 + threadIdx.x, sm.seq = s;
            sm.h = uint32_t((w0 - (sum - mine)) / units);
            sm.i0 = sum - mine + uint64_t(sm.h) * units;
        }
        if (before > w0) break;
    }
    if (threadIdx.x == 0) {
        Bars &b = sm.bars;
        for (int i = 0; i < kRaw; i++) bar_init(&b.raw_full[i], 1), bar_init(&b.raw_empty[i], 4);
        for (int i = 0; i < kOps; i++) bar_init(&b.op_full[i], 4), bar_init(&b.op_empty[i], 1);
        for (int i = 0; i < kSlots; i++) bar_init(&b.scale_full[i], 1);
        for (int i = 0; i < 2; i++) bar_init(&b.q_full[i], 4), bar_init(&b.s_full[i], 1), bar_init(&b.p_full[i][0], 4), bar_init(&b.p_full[i][1], 4), bar_init(&b.o_full[i], 1);
        for (int i = 0; i < kJobs; i++) bar_init(&b.job_full[i], 1), bar_init(&b.job_empty[i], kReaders);
        bar_init(&b.rows, 8);
        bar_init(&b.drained, 1);
        bar_init_done();
        prefetch_map(&maps.code[0]);
        prefetch_map(&maps.code[1]);
        sm.poison = 0;
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_of(&sm.tmem)), "r"(kColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tm_before();
    }
    __syncthreads();
    tm_after();
    
    bool ok = true;
    if (warp < 8) {
        more_registers<kRowRegs>();
        ok = rows_role<DP>(a, sm);
    } else if (warp < 12) {
        fewer_registers<kConvertRegs>();
        ok = convert_role<DP>(sm, a.limit);
    } else {
        fewer_registers<kOtherRegs>();
        if (warp == 12) ok = product_role<DP>(sm, a.limit);
        if (warp == 13) ok = copy_role<DP>(a, maps, sm);
        if (warp == 14 && threadIdx.x % 32 == 0) ok = find_role<DP>(a, sm, Walk{w0, w1, sm.i0, W, G, sm.slot, sm.seq, sm.h, slots});
        if (warp == 15 && cta == 0) report_batch(a.b, a.c.tokens, a.d_status, threadIdx.x % 32, 32, false);
    }
    if (!ok) report(a.d_status, ZC_ETIMEOUT);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    tm_before();
    __syncthreads();
    tm_after();
    if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sm.tmem), "r"(kColumns));
}

template <int DP> int launch(const AttendArgs &a, cudaStream_t s) {
    static std::atomic<uint64_t> ready{0};  // devices whose kernel may use this much shared memory
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ZC_ECUDA;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute(tiles_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(Smem<DP>))) != cudaSuccess)
            return ZC_ECUDA;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    CodeMaps maps;
    const int st = make_maps(a.c, DP, 16, maps);
    if (st != ZC_OK) return st;
    tiles_kernel<DP><<<uint32_t(sm_count()), kThreads, sizeof(Smem<DP>), s>>>(a, maps);
    return cudaGetLastError() == cudaSuccess ? ZC_OK : ZC_ECUDA;
}

} // namespace

uint64_t tiles_counters(const Batch &b, const Cache &c, uint32_t group) {
    return uint64_t(slot_of(b.total, b.n_seqs, group, kRows, 1)) * c.heads;
}

uint64_t tiles_part_bytes(const Cache &c) {
    return uint64_t(sm_count()) * 2 * (c.dim <= 64 ? sizeof(Part<64>) : sizeof(Part<128>));
}

int launch_tiles(const AttendArgs &a, cudaStream_t s) { return a.c.dim <= 64 ? launch<64>(a, s) : launch<128>(a, s); }

} // namespace kv
} // namespace zc
