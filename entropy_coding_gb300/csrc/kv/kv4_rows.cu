// kv4_rows.cu — attention of few query rows over the 4-bit cache.
//
// With codes kc, vc (E2M1) and a scale for every 16 columns of a row, over the
// keys j that row i sees:
//   k_j = kc_j ks_j, v_j = vc_j vs_j   (group by group; exact in half)
//   s_ij = scale * (q_i . k_j)
//   out_i = sum_j 2^(s_ij log2e - m) v_j / sum_j 2^(s_ij log2e - m)
//
// The work is cut along the keys (kv_rows.cuh), in units of 128. A warp takes 32
// keys at a time, in two halves of 16; both products are transposed and on
// mma.m16n8k16 as in kv_rows.cu, and query rows and weights are rounded as
// there, with no unit but that of the scores' maximum: values are whole numbers
// in half, whatever their scales. A code costs half a conversion (two codes to
// two halves) and half a product with its scale; codes of values are brought
// together by key before that, in nibbles, since a product's inner index runs
// along the keys.
//
// A step's codes come as a box of 32 rows (or two of 16), its scales as one of
// lines, a line for 16 rows. The order of keys in a score tile is free as long as
// their weights meet their values: it is chosen (`key_of`) so that reading a
// fragment of keys and one of values both meet all banks. Warps' rows meet, at a
// piece's end, in the steps of their rings that they have read last.
//
// Measured on a GB300: the next tokens of 64 sequences of up to 8192 keys (8
// heads of 128, 4 query heads each), 314 MB of cache, in 70 us: 4.5 TB/s, 0.66
// of the copy rate, where the 8-bit cache's 558 MB take 98; one token over 131072
// keys in 38. Bytes are not the bound here: with the steps' arithmetic left out
// the same copies take 58 us, of which 12 are the start, the pieces' ends and the
// joining. A step of 32 keys is about 660 instructions of a warp, 128 conversions and
// 128 products with scales among them, 190 of them for copies, waits and pieces'
// ends; conversions, half products and tensor-core products contend for issue
// (together at 0.5 instructions a clock, each alone at its unit's rate), so that
// neither more warps (4 CTAs an SM, or CTAs of 8, 12 or 16 warps) nor more steps in
// flight are faster. What was: an item's beginning and end counted as work (83.5
// to 73.2 us), boxes of 32 rows and scale lines by the tensor memory accelerator
// (90 to 84), beginning as the kernel in front of this one ends (73.2 to
// 70.4).
#include <cstddef>

#include "kv4_common.cuh"
#include "kv_rows.cuh"

namespace zc {
namespace kv {
namespace {

constexpr int kResidentMost = 3;

template <int DP> struct Codes4 {
    static constexpr int kDim = DP, kWarps = 4, kSlice = 32, kRow = DP / 2;
    static constexpr int kStages = 3 * (128 / DP);
    // CTAs of an SM: 3 hold the registers of one tile of rows (4 of fewer registers, with two steps of a ring each, take as
    // long), 2 those of two tiles (16 sequences of 16 rows: 23.7 us, with 3 and spilled registers 26.7).
    template <int NT> static constexpr int resident() { return NT == 1 ? 3 : 2; }
    static constexpr bool kEarly = true;
    static constexpr bool kMergeInRing = true, kUnits = false;
    // (64 sequences of up to 8192 keys: 0 units 83.5 us, with the CTAs that have many short items last, 2 units 74.4, 3 units
    // 73.8, 4 units 73.2, 6 units 73.9)
    static constexpr uint32_t kFixed = 4;
    struct Stage {
        uint8_t k[kSlice * kRow];
        uint8_t v[kSlice * kRow];
        uint8_t ks[2][kScaleLine], vs[2][kScaleLine];  // a line for each half's 16 rows, dim / 16 bytes a row
    };
    static_assert(sizeof(Stage) % 128 == 0 && offsetof(Stage, ks) % 128 == 0 && 16 * kRow % 128 == 0, "boxes begin on multiples of 128 bytes");
    static_assert(kStages - 1 <= 16 && sizeof(Stage) % (4 * DP) == 0, "boxes begin where their swizzle does");
    using Maps = CodeMaps4;
    // What a warp keeps in shared memory besides its ring: the ring's barriers, and where 32 of its steps are, looked up 16
    // at a time: a step's block and row in it, or those of its halves.
    static constexpr int kLook = 16;
    struct Warp {
        uint64_t full[kStages];
        int2 place[2 * kLook][2];
    };
    // Row 0 to 7 of a score tile's half: a key of 8. With rows of 64 bytes, swizzled over 64, the 8 lanes that read together
    // have two keys of different parity (of keys) or four whose 16-byte chunks lie apart (of values); with rows of 32 bytes
    // four keys that differ modulo 4 both times.
    static __device__ __forceinline__ int key_of(int r) { return int((DP == 128 ? 0x65742130u : 0x57463120u) >> 4 * r & 7); }
    static __device__ __forceinline__ void look_up(const AttendArgs &a, Warp &wp, const Job &job, int k0);
    static __device__ __forceinline__ void fetch(const AttendArgs &a, const CodeMaps4 &maps, Warp &wp, Stage *ring, const Job &job, int k, uint32_t st);
    template <int NT>
    static __device__ __forceinline__ bool attend_slices(const AttendArgs &a, const CodeMaps4 &maps, Warp &wp, Stage *ring, const Job &job,
                                                         uint32_t turn, Sums<DP, NT> &acc);
};

// Blocks of a multiple of 32 tokens hold a step's keys in one run of 32 rows; of others a step is two boxes of 16.
__device__ __forceinline__ bool in_halves(const AttendArgs &a) { return a.c.tokens % 32; }

// Where steps k0 .. k0 + 15 are, a half of a step a lane. A block that is not there is read as block 0, a half of which the
// rows see nothing as the nearest 16 keys that they do see.
template <int DP> __device__ __forceinline__ void Codes4<DP>::look_up(const AttendArgs &a, Warp &wp, const Job &job, int k0) {
    const int half = threadIdx.x & 1, k = k0 + (threadIdx.x & 31) / 2;
    if (k >= job.steps || (half && !in_halves(a))) return;
    uint32_t i = uint32_t(2 * (job.first + k * kWarps) + half);
    if (in_halves(a)) i = min(max(i, uint32_t(job.all_lo / 16)), uint32_t((job.all_hi - 1) / 16));
    const uint32_t blk = block_of_16(a.c, i);
    wp.place[k & (2 * kLook - 1)][half] = make_int2(int(max(read_block(a.b, a.c, job.seq.s, blk, a.d_status), int64_t(0))),
                                                    int(job.h * a.c.tokens + i * 16 - blk * a.c.tokens));
}

// Asks for step k's keys and values (one lane). Rows that nobody sees come along as they are.
template <int DP>
__device__ __forceinline__ void Codes4<DP>::fetch(const AttendArgs &a, const CodeMaps4 &maps, Warp &wp, Stage *ring, const Job &job, int k, uint32_t st) {
    if ((threadIdx.x & 31) == 0 && k < job.steps && !a.stall) {
        Stage &sl = ring[st];
        uint64_t *bar = &wp.full[st];
        bar_expect(bar, sizeof(Stage));
#pragma unroll 1
        for (int half = 0;; half++) {
            const int2 at = wp.place[k & (2 * kLook - 1)][half];
            copy_box(sl.k + half * 16 * kRow, &maps.code[0], at.y, at.x, bar);
            copy_box(sl.v + half * 16 * kRow, &maps.code[1], at.y, at.x, bar);
            copy_box(sl.ks[half], &maps.scale[0], at.y / 16, at.x, bar);
            copy_box(sl.vs[half], &maps.scale[1], at.y / 16, at.x, bar);
            if (half || !in_halves(a)) break;
        }
    }
}

// The low half of each byte of x, the high half of each of y.
__device__ __forceinline__ uint32_t low_halves(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(r) : "r"(x), "r"(y), "r"(0x0F0F0F0Fu));  // (x & m) | (y & ~m)
    return r;
}
template <int DP>
template <int NT>
__device__ __forceinline__ bool Codes4<DP>::attend_slices(const AttendArgs &a, const CodeMaps4 &maps, Warp &wp, Stage *ring, const Job &job,
                                                          uint32_t turn, Sums<DP, NT> &acc) {
    constexpr int kRows = 8 * NT, S = kStages;
    constexpr int kSteps = DP / 16;      // inner steps of k q, and column tiles of the output
    constexpr int kRun = DP / 4;         // columns of q and k that a thread of a quad holds
    constexpr int kCols = DP / 8;        // columns of v that a thread's quad holds
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const Seq &seq = job.seq;
    const uint32_t row0 = job.tile * kRows, n_rows = seq.n * a.group, groups = a.c.dim / 16;
    auto &o = acc.o;
    auto &l = acc.l;

    uint32_t qf[NT][kSteps][2];
    float row_scale[NT][2];  // of rows 2t, 2t + 1 of each tile
    load_queries<DP, NT>(a, job, qf, row_scale);
    // Scores stay products until their exponentials: a row's scale is positive for that, with its sign in the queries. (And
    // not 0, since a score that is left out is -infinity: 1e-37 of any product of half numbers is none.)
#pragma unroll
    for (int n = 0; n < NT; n++) {
#pragma unroll
        for (int i = 0; i < kSteps; i++)
#pragma unroll
            for (int j = 0; j < 2; j++) qf[n][i][j] ^= a.scale_log2 < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int e = 0; e < 2; e++) row_scale[n][e] = fmaxf(fabsf(row_scale[n][e]), 1e-37f);
    }
    acc.clear();
    // The largest product of a row and a key, as far as it was followed (or 0), and that from which on it is followed again.
    // A weight's exponent is a difference of products by the row's scale: of products close to one another that is exact,
    // however large they are. (One multiply-add of the product, its scale and the score's maximum is off by hundreds next to
    // a score of 10^9, and no faster.)
    float base[NT][2], most[NT][2];
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
        for (int e = 0; e < 2; e++) base[n][e] = 0.0f, most[n][e] = kNone;

    // This thread's keys of a half: key_of(g) and 8 more for scores, four for values; its groups of columns.
    const int key_g = key_of(g), key_v0 = key_of(2 * t), key_v1 = key_of(2 * t + 1);
    constexpr int kGroups = kRun / 16;   // of q and k
    const uint32_t kg0 = kGroups * t, vg = kCols * g / 16;
    uint32_t there[kGroups];             // brings a scale byte to both halves of a word; 0 behind the last column
#pragma unroll
    for (int i = 0; i < kGroups; i++) there[i] = kg0 + i < groups ? 0x00800080u : 0;

    uint32_t st = turn % S, parity = turn / S & 1;  // of step k
    for (int k = 0; k < job.steps; k++) {
        if ((k & (kLook - 1)) == 0) {
            __syncwarp();
            look_up(a, wp, job, k + kLook);
            __syncwarp();
        }
        if (!__all_sync(0xFFFFFFFFu, bar_wait(&wp.full[st], parity, a.limit))) {
            drain<Codes4>(a, wp, turn + k, job.steps - k);
            if (lane == 0) report(a.d_status, ZC_ETIMEOUT);
            return false;
        }
        // The stage before this one was read a step ago (the vote above comes after every lane's reads).
        fetch(a, maps, wp, ring, job, k + S - 1, st == 0 ? S - 1 : st - 1);
        Stage &sl = ring[st];
        if (++st == S) st = 0, parity ^= 1;
        const int key0 = (job.first + k * kWarps) * kSlice;
        // Scores of 2 x 16 keys and the rows: c0, c1 are key key_of(g) and rows 2t, 2t + 1, c2, c3 the key 8 on.
        float sc[2][NT][4];
#pragma unroll
        for (int half = 0; half < 2; half++) {
            uint32_t w[2][kRun / 8], s[2][kGroups];
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int r = key_g + 8 * j;
                const uint8_t *row = sl.k + (16 * half + r) * kRow;
                if (DP == 128) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(row + 16 * (t ^ (r >> 1 & 3)));
                    w[j][0] = v.x, w[j][1] = v.y, w[j][kRun / 8 - 2] = v.z, w[j][kRun / 8 - 1] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(row + 16 * (t >> 1 ^ (r >> 2 & 1)) + 8 * (t & 1));
                    w[j][0] = v.x, w[j][1] = v.y;
                }
#pragma unroll
                for (int i = 0; i < kGroups; i++) s[j][i] = sl.ks[half][r * groups + kg0 + i] * there[i];
            }
#pragma unroll
            for (int i = 0; i < kRun / 8; i++) {  // 8 columns: two inner steps
                uint32_t kf[2][4];
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    uint32_t h[4];
                    e2m1x8_to_half2x4(w[j][i], h[0], h[1], h[2], h[3]);
#pragma unroll
                    for (int x = 0; x < 4; x++) kf[x / 2][x % 2 * 2 + j] = mul_half2(h[x], s[j][i / 2]);
                }
#pragma unroll
                for (int x = 0; x < 2; x++)
#pragma unroll
                    for (int n = 0; n < NT; n++) {
                        if (i == 0 && x == 0) mma_first(sc[half][n], kf[x], qf[n][0][0], qf[n][0][1]);
                        else mma(sc[half][n], kf[x], qf[n][2 * i + x][0], qf[n][2 * i + x][1]);
                    }
            }
        }
        const bool edge = key0 < job.x_lo || key0 + kSlice > job.x_hi;  // some row does not see all of it
        if (edge) {
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    int lo, hi;
                    bounds(a, seq, min(row0 + 8 * n + 2 * t + e, n_rows - 1), lo, hi);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int key = key0 + key_g + 8 * j;
                        if (key < lo || key >= hi) sc[j / 2][n][j % 2 * 2 + e] = kNone;
                    }
                }
        }
        // The base follows the maximum only once that is 2^kSlackW above it: after the first step a rescaling is rare.
        bool grows = false;
        float top[NT][2];
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                top[n][e] = fmaxf(fmaxf(sc[0][n][e], sc[0][n][2 + e]), fmaxf(sc[1][n][e], sc[1][n][2 + e]));
                grows |= top[n][e] > most[n][e];
            }
        if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
            for (int n = 0; n < NT; n++) {
                float down[2];
#pragma unroll
                for (int e = 0; e < 2; e++) {
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) top[n][e] = fmaxf(top[n][e], __shfl_xor_sync(0xFFFFFFFFu, top[n][e], d));
                    const float was = most[n][e] == kNone ? kNone : base[n][e], now = fmaxf(was, top[n][e]);
                    down[e] = was == kNone ? 0.0f : ex2((was - now) * row_scale[n][e]);
                    l[n][e] *= down[e];
                    base[n][e] = now == kNone ? 0.0f : now;
                    most[n][e] = followed(now, row_scale[n][e]);
                }
#pragma unroll
                for (int c = 0; c < kSteps; c++)
                    o[n][c][0] *= down[0], o[n][c][1] *= down[1], o[n][c][2] *= down[0], o[n][c][3] *= down[1];
            }
        }
        // Weights 2^((product - base) scale + kRaise).
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int half = 0; half < 2; half++)
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const float2 past = add2(make_float2(sc[half][n][2 * j], sc[half][n][2 * j + 1]), make_float2(-base[n][0], -base[n][1]));
                    float2 p = fma2(past, make_float2(row_scale[n][0], row_scale[n][1]), both(kRaise));
                    p.x = ex2(p.x), p.y = ex2(p.y);
                    const float2 sum = add2(make_float2(l[n][0], l[n][1]), p);
                    l[n][0] = sum.x, l[n][1] = sum.y;
                    pf[half][n][j] = transpose8(half2_of(p.x, p.y));
                }
        if (edge) {
            // A row that does not see a key has weight 0 for it, but 0 times NaN (or an infinity) is NaN: scales that make
            // these are taken out here and given to the rows that do see them.
            bool bad = false;
#pragma unroll 1
            for (uint32_t j = lane; j < 2 * a.c.dim; j += 32) bad |= sl.vs[j / a.c.dim][j % a.c.dim] > kScaleMost;
            if (__any_sync(0xFFFFFFFFu, bad)) {
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        int lo, hi;
                        bounds(a, seq, min(row0 + 8 * n + 2 * t + e, n_rows - 1), lo, hi);
#pragma unroll 1
                        for (int j = max(lo - key0, 0); j < min(hi - key0, kSlice); j++)
                            if (vg < groups && sl.vs[j / 16][j % 16 * groups + vg] > kScaleMost) acc.poison[n][e] = (1u << kCols) - 1;
                    }
                __syncwarp();
#pragma unroll 1
                for (uint32_t j = lane; j < 2 * a.c.dim; j += 32)
                    if (sl.vs[j / a.c.dim][j % a.c.dim] > kScaleMost) sl.vs[j / a.c.dim][j % a.c.dim] = 0;
                fence_async();
                __syncwarp();
            }
        }
        // Values: the thread's keys are key_v0, key_v1 and these 8 on, its columns [kCols g, kCols g + kCols), of one group.
#pragma unroll
        for (int half = 0; half < 2; half++) {
            uint32_t w[4][kCols / 8], s[2];
            const uint8_t *sv = sl.vs[half] + vg;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int r = (j & 1 ? key_v1 : key_v0) + (j & 2 ? 8 : 0);
                const uint8_t *row = sl.v + (16 * half + r) * kRow;
                if (DP == 128) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(row + 16 * (g >> 1 ^ (r >> 1 & 3)) + 8 * (g & 1));
                    w[j][0] = v.x, w[j][kCols / 8 - 1] = v.y;
                } else {
                    w[j][0] = *reinterpret_cast<const uint32_t *>(row + 16 * (g >> 2 ^ (r >> 2 & 1)) + 4 * (g & 3));
                }
            }
            s[0] = sv[key_v0 * groups] * 0x80u + sv[key_v1 * groups] * 0x00800000u;
            s[1] = sv[(key_v0 + 8) * groups] * 0x80u + sv[(key_v1 + 8) * groups] * 0x00800000u;
#pragma unroll
            for (int i = 0; i < kCols / 8; i++) {
                // by key: even columns of two keys, and odd ones
                uint32_t vf[4][4];
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const uint32_t x = w[2 * j][i], y = w[2 * j + 1][i];
                    const uint32_t even = low_halves(x, y << 4), odd = low_halves(x >> 4, y);
                    uint32_t h[4];
                    e2m1x8_to_half2x4(even, h[0], h[1], h[2], h[3]);
#pragma unroll
                    for (int c = 0; c < 4; c++) vf[c][2 * j] = mul_half2(h[c], s[j]);
                    e2m1x8_to_half2x4(odd, h[0], h[1], h[2], h[3]);
#pragma unroll
                    for (int c = 0; c < 4; c++) vf[c][2 * j + 1] = mul_half2(h[c], s[j]);
                }
#pragma unroll
                for (int c = 0; c < 4; c++)  // columns 8 i + 2 c and + 1: rows g and g + 8 of the tile
#pragma unroll
                    for (int n = 0; n < NT; n++) mma(o[n][4 * i + c], vf[c], pf[half][n][0], pf[half][n][1]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
        for (int e = 0; e < 2; e++)
            if (most[n][e] != kNone) acc.m[n][e] = base[n][e] * row_scale[n][e];
    return true;
}

template <int NT> int launch_tiles_of(const AttendArgs &a, cudaStream_t s) {
    const uint32_t rows = a.c.tokens % 32 ? 16 : 32;
    return a.c.dim <= 64 ? launch<Codes4<64>, NT>(a, rows, s) : launch<Codes4<128>, NT>(a, rows, s);
}

} // namespace

uint64_t rows4_group_counters() { return uint64_t(sm_count()) * kResidentMost * 2; }

uint64_t rows4_part_bytes(const Cache &c) {
    return uint64_t(sm_count()) * kResidentMost * 2 * (c.dim <= 64 ? sizeof(Part<64, 2>) : sizeof(Part<128, 2>));
}

// One tile of 8 rows or two.
int launch_rows4(const AttendArgs &a, cudaStream_t s) {
    return std::min<uint64_t>(uint64_t(a.b.most) * a.group, a.rows_most) <= 8 ? launch_tiles_of<1>(a, s) : launch_tiles_of<2>(a, s);
}

} // namespace kv
} // namespace zc
