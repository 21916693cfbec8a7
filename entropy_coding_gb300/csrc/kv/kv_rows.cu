// kv_rows.cu — attention of few query rows over the 8-bit cache.
//
// A row is one query token and query head; the rows of a key/value head are
// its `group` query heads times the sequence's new tokens. With codes kc, vc
// and block scales ks, vs, over the keys j that row i sees:
//   s_ij = scale * ks_b(j) * (q_i . kc_j)
//   out_i = sum_j 2^(s_ij log2e - m) vs_b(j) vc_j / sum_j 2^(s_ij log2e - m)
//
// A CTA takes 16 rows, a warp 16 keys at a time, and both products run on
// mma.m16n8k16 with half operands and float accumulators. E4M3 codes are
// exact in half. A query row is exact in half too after it is multiplied by a
// power of two that brings its largest element to [2^14, 2^15) (what falls
// below 2^-24 then is 2^-38 of it). A row's weights w are rounded to half;
// they are kept in units of the row's running maximum of s + log2 vs, not of
// s alone, so that the largest contribution to the output is always 1 and
// blocks whose scales differ by any factor keep their precision. The sum of
// the weights is taken before that rounding, in units of the running maximum
// of s.
//
// Each warp streams its own keys and values through shared memory with
// cp.async, kStages slices of 16 rows deep, and the warps meet only at the
// end. Rows are padded by 16 bytes, which spreads a fragment's reads over the
// banks. Within a row the columns are dealt to the threads of a quad in runs
// (the order of a product's inner index is free as long as both operands
// share it), so that fragments are read 16 bytes at a time.
#include "kv_common.cuh"

namespace zc {
namespace kv {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kStages = 4;
constexpr int kRows = 16, kSlice = 16;  // rows of a CTA; keys of a warp's step
constexpr float kNone = -INFINITY;

template <int DP> struct Stage {
    uint8_t k[kSlice][DP + 16];
    uint8_t v[kSlice][DP + 16];
    float scale[4];  // ks, vs
};

template <int DP> struct Merge {  // over the stages, once the loop is done
    float o[kWarps][kRows][DP + 4];
    float m[kWarps][kRows], mw[kWarps][kRows], l[kWarps][kRows];
};

template <int DP> constexpr size_t smem_bytes() {
    return sizeof(Stage<DP>) * kStages * kWarps > sizeof(Merge<DP>) ? sizeof(Stage<DP>) * kStages * kWarps : sizeof(Merge<DP>);
}

__device__ __forceinline__ void cp16(void *dst, const void *src, bool take) {
    const uint32_t d = uint32_t(__cvta_generic_to_shared(dst)), n = take ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp4(void *dst, const void *src, bool take) {
    const uint32_t d = uint32_t(__cvta_generic_to_shared(dst)), n = take ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// 2^(a - b) with 2^(-inf - anything) = 0
__device__ __forceinline__ float ratio2(float a, float b) { return a == kNone ? 0.0f : ex2(a - b); }
// Whether one of the four codes is NaN (0x7F or 0xFF).
__device__ __forceinline__ bool any_nan(uint32_t v) { return __vcmpeq4(v & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0; }

template <int DT, int DP> __global__ void __launch_bounds__(kThreads, 3) rows_kernel(AttendArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int kSteps = DP / 16;      // inner steps of q k
    constexpr int kTiles = DP / 8;       // column tiles of the output
    constexpr int kRun = DP / 4;         // columns of q and k that a thread of a quad holds
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t h = blockIdx.y, D = a.c.dim, B = a.c.tokens;

    uint64_t tile;
    const uint32_t s = find_seq(a.b, blockIdx.x, a.group, kRows, 1, tile);
    const bool speak = threadIdx.x == 0 && tile == 0 && h == 0;
    const Seq seq = read_seq(a.b, s, a.d_status, B, speak);
    if (!seq.ok) return;
    const uint64_t row0 = tile * kRows, n_rows = uint64_t(seq.n) * a.group;
    if (row0 >= n_rows) return;

    // The keys that each of the thread's two rows sees: [lo, hi).
    const int64_t pos0 = int64_t(seq.len) - int64_t(seq.n);  // position of the sequence's first new token
    int lo[2], hi[2];
    bool row_ok[2];
    auto bounds = [&](uint64_t row, int &l, int &e) {
        const int64_t pos = pos0 + int64_t(row / a.group);
        e = int(a.causal ? max(pos + 1, int64_t(0)) : int64_t(seq.len));
        l = a.window ? int(max(pos - int64_t(a.window) + 1, int64_t(0))) : 0;
        if (l > e) l = e;
    };
#pragma unroll
    for (int r = 0; r < 2; r++) {
        const uint64_t row = row0 + g + 8 * r;
        row_ok[r] = row < n_rows;
        bounds(row_ok[r] ? row : n_rows - 1, lo[r], hi[r]);
    }
    int all_lo, all_hi, x_lo, x_hi;  // seen by some row; by every row
    bounds(row0, all_lo, x_hi);
    bounds(min(row0 + kRows, n_rows) - 1, x_lo, all_hi);

    // Query fragments: the thread's rows, columns [kRun t, kRun t + kRun).
    uint32_t qf[kSteps][4];
    float row_scale[2];
#pragma unroll
    for (int r = 0; r < 2; r++) {
        const uint64_t row = row0 + g + 8 * r;
        uint32_t w[kRun / 2];
#pragma unroll
        for (int i = 0; i < kRun / 8; i++) {
            uint4 v = make_uint4(0, 0, 0, 0);
            const uint32_t col = kRun * t + 8 * i;
            if (row_ok[r] && col < D) {
                const uint16_t *q = static_cast<const uint16_t *>(a.q.p) +
                                    (int64_t(seq.first) + int64_t(row / a.group)) * a.q.token +
                                    (int64_t(h) * a.group + int64_t(row % a.group)) * a.q.head + col;
                v = __ldg(reinterpret_cast<const uint4 *>(q));
            }
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
        row_scale[r] = a.scale_log2;
        if (DT == ZC_BF16) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < kRun / 2; i++) top = max(top, max(w[i] << 16 & 0x7FFF0000u, w[i] & 0x7FFF0000u));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            // 2^(14 - e) for the largest element's exponent e, within float's normal range
            const int field = min(max(127 + 14 - (int(top >> 23) - 127), 1), 253);
            const float up = __uint_as_float(uint32_t(field) << 23), down = __uint_as_float(uint32_t(254 - field) << 23);
            row_scale[r] = a.scale_log2 * down;
#pragma unroll
            for (int i = 0; i < kRun / 2; i++) {
                const float2 f = unpack2<DT>(w[i]);
                w[i] = half2_of(f.x * up, f.y * up);
            }
        }
#pragma unroll
        for (int i = 0; i < kSteps; i++) qf[i][r] = w[2 * i], qf[i][2 + r] = w[2 * i + 1];
    }

    Stage<DP> *stages = reinterpret_cast<Stage<DP> *>(smem) + warp * kStages;
    const int first = all_lo / kSlice + warp, end = (all_hi + kSlice - 1) / kSlice;  // slices of this warp: first, + kWarps, ...

    // Fetches slice i into stage st; rows outside the keys that someone sees, and
    // columns from D on, are zeros.
    auto fetch = [&](int i, int st) {
        if (i < end) {
            const int key0 = i * kSlice;
            const int64_t id = read_block(a.b, a.c, s, uint32_t(key0) / B, a.d_status);
            const uint32_t in_block = uint32_t(key0) % B;
            const int64_t base = max(id, int64_t(0)) * a.c.block_stride + (int64_t(h) * B + in_block) * D;
            constexpr int kChunks = DP / 16;
#pragma unroll
            for (int j = 0; j < kSlice * kChunks / 32; j++) {
                const int r = (j * 32 + lane) / kChunks, c = (j * 32 + lane) % kChunks * 16;
                const bool take = id >= 0 && key0 + r >= all_lo && key0 + r < all_hi && c < int(D);
                const int64_t off = take ? base + int64_t(r) * D + c : 0;
                cp16(&stages[st].k[r][c], a.c.code[0] + off, take);
                cp16(&stages[st].v[r][c], a.c.code[1] + off, take);
            }
            if (lane < 2) cp4(&stages[st].scale[lane], a.c.scale[lane] + max(id, int64_t(0)) * a.c.scale_stride + h, id >= 0);
        }
        cp_commit();
    };

    float o[kTiles][4];
#pragma unroll
    for (int i = 0; i < kTiles; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) o[i][j] = 0.0f;
    float m[2] = {kNone, kNone}, mw[2] = {kNone, kNone}, l[2] = {0.0f, 0.0f};

#pragma unroll
    for (int i = 0; i < kStages - 1; i++) fetch(first + i * kWarps, i);
    int st = 0;
    for (int i = first; i < end; i += kWarps) {
        cp_wait<kStages - 2>();
        __syncwarp();
        Stage<DP> &sl = stages[st];
        // scores of 16 rows and 16 keys
        float sc[2][4] = {};
#pragma unroll
        for (int n = 0; n < 2; n++) {
            uint32_t kw[kRun / 4];
#pragma unroll
            for (int c = 0; c < kRun / 16; c++) {
                const uint4 v = *reinterpret_cast<const uint4 *>(&sl.k[8 * n + g][kRun * t + 16 * c]);
                kw[4 * c] = v.x, kw[4 * c + 1] = v.y, kw[4 * c + 2] = v.z, kw[4 * c + 3] = v.w;
            }
#pragma unroll
            for (int c = 0; c < kSteps; c++)
                mma(sc[n], qf[c], e4m3x2_to_half2(uint16_t(kw[c])), e4m3x2_to_half2(uint16_t(kw[c] >> 16)));
        }
        const int key0 = i * kSlice;
        const bool edge = key0 < x_lo || key0 + kSlice > x_hi;  // some row does not see all of it
        const float ks = sl.scale[0], vs = sl.scale[1];
        float top[2] = {kNone, kNone};
#pragma unroll
        for (int n = 0; n < 2; n++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int r = j >> 1, key = key0 + 8 * n + 2 * t + (j & 1);
                float x = sc[n][j] * (row_scale[r] * ks);
                if (edge && (key < lo[r] || key >= hi[r])) x = kNone;
                sc[n][j] = x;
                top[r] = fmaxf(top[r], x);
            }
        const float lvs = __log2f(vs);
        float f[2], down[2];
#pragma unroll
        for (int r = 0; r < 2; r++) {
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 1));
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 2));
            const float m1 = fmaxf(m[r], top[r]), w1 = fmaxf(mw[r], top[r] + lvs);
            l[r] *= ratio2(m[r], m1);
            down[r] = ratio2(mw[r], w1);
            m[r] = m1, mw[r] = w1;
            // weights in the output's units: p * f, f = 2^(m + log2 vs - mw)
            f[r] = w1 == kNone || m1 == kNone ? 0.0f : vs * ex2(fminf(m1 - w1, 126.0f));
        }
        if (__any_sync(0xFFFFFFFFu, down[0] != 1.0f || down[1] != 1.0f)) {
#pragma unroll
            for (int c = 0; c < kTiles; c++) o[c][0] *= down[0], o[c][1] *= down[0], o[c][2] *= down[1], o[c][3] *= down[1];
        }
        uint32_t pf[4];
#pragma unroll
        for (int n = 0; n < 2; n++) {
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int r = j >> 1;
                p[j] = sc[n][j] == kNone ? 0.0f : ex2(sc[n][j] - m[r]);
                l[r] += p[j];
            }
            pf[2 * n] = half2_of(p[0] * f[0], p[1] * f[0]);
            pf[2 * n + 1] = half2_of(p[2] * f[1], p[3] * f[1]);
        }
        // Values: the thread's keys are 2t, 2t + 1, 2t + 8, 2t + 9, its columns [kTiles g, kTiles g + kTiles).
        const int keys[4] = {2 * t, 2 * t + 1, 2 * t + 8, 2 * t + 9};
        if (edge) {
            // A row that does not see a key has weight 0 for it, but 0 * NaN is NaN: NaN codes are
            // taken out here and given to the rows that do see them.
            bool bad = false;
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int c = 0; c < kTiles / 4; c++)
                    bad |= any_nan(*reinterpret_cast<const uint32_t *>(&sl.v[keys[j]][kTiles * g + 4 * c]));
            if (__any_sync(0xFFFFFFFFu, bad)) {
                for (int k = 0; k < kSlice; k++)
#pragma unroll
                    for (int c = 0; c < kTiles; c++)
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const int r = e >> 1, col = kTiles * (2 * t + (e & 1)) + c;
                            if ((sl.v[k][col] & 0x7F) == 0x7F && key0 + k >= lo[r] && key0 + k < hi[r]) o[c][e] = NAN;
                        }
                __syncwarp();
                for (int j = lane; j < kSlice * DP; j += 32)
                    if ((sl.v[j / DP][j % DP] & 0x7F) == 0x7F) sl.v[j / DP][j % DP] = 0;
                __syncwarp();
            }
        }
        uint32_t vw[4][kTiles / 4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (kTiles == 16) {
                const uint4 v = *reinterpret_cast<const uint4 *>(&sl.v[keys[j]][16 * g]);
                vw[j][0] = v.x, vw[j][1] = v.y, vw[j][kTiles / 4 - 2] = v.z, vw[j][kTiles / 4 - 1] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2 *>(&sl.v[keys[j]][8 * g]);
                vw[j][0] = v.x, vw[j][1] = v.y;
            }
        }
#pragma unroll
        for (int c = 0; c < kTiles; c++) {
            const uint32_t sel = (c & 3) | ((c & 3) + 4) << 4;  // byte c of two keys
            const uint32_t b0 = __byte_perm(vw[0][c / 4], vw[1][c / 4], sel), b1 = __byte_perm(vw[2][c / 4], vw[3][c / 4], sel);
            mma(o[c], pf, e4m3x2_to_half2(uint16_t(b0)), e4m3x2_to_half2(uint16_t(b1)));
        }
        __syncwarp();  // the stage before this one is free: it was read a step ago
        fetch(i + (kStages - 1) * kWarps, (st + kStages - 1) % kStages);
        st = (st + 1) % kStages;
    }
    cp_wait<0>();

    // The warps' rows together.
    __syncthreads();
    Merge<DP> &mg = *reinterpret_cast<Merge<DP> *>(smem);
#pragma unroll
    for (int r = 0; r < 2; r++) {
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
        if (t == 0) mg.m[warp][g + 8 * r] = m[r], mg.mw[warp][g + 8 * r] = mw[r], mg.l[warp][g + 8 * r] = l[r];
#pragma unroll
        for (int e = 0; e < 2; e++)
#pragma unroll
            for (int c = 0; c < kTiles; c++) mg.o[warp][g + 8 * r][kTiles * (2 * t + e) + c] = o[c][2 * r + e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * DP / 8; i += kThreads) {
        const int r = i / (DP / 8), col = i % (DP / 8) * 8;
        const uint64_t row = row0 + r;
        if (row >= n_rows || col >= int(D)) continue;
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
        // out = sum / L in the units of M; a row that sees no key is 0. (L is NaN where a score was.)
        const float by = L == 0.0f ? 0.0f : (W == kNone ? 0.0f : ex2(W - M)) / L;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; k++) w[k] = L == 0.0f ? 0u : pack2<DT>(x[2 * k] * by, x[2 * k + 1] * by);
        const int64_t token = int64_t(seq.first) + int64_t(row / a.group), head = int64_t(h) * a.group + int64_t(row % a.group);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out.p) + token * a.out.token + head * a.out.head + col) =
            make_uint4(w[0], w[1], w[2], w[3]);
        if (a.lse && col == 0)
            a.lse[token * a.heads + head] = L == 0.0f ? kNone : (M + log2f(L)) * 0.6931471805599453f;
    }
}

template <int DT, int DP> int launch(const AttendArgs &a, cudaStream_t s) {
    const uint64_t slots = slots_of(a.b.total, a.b.n_seqs, a.group, kRows, 1);
    if (slots > 0x7FFFFFFFull) return ZC_EINVAL;
    if (cudaFuncSetAttribute(rows_kernel<DT, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem_bytes<DP>())) != cudaSuccess)
        return ZC_ECUDA;
    rows_kernel<DT, DP><<<dim3(uint32_t(slots), a.c.heads), kThreads, smem_bytes<DP>(), s>>>(a);
    return cudaGetLastError() == cudaSuccess ? ZC_OK : ZC_ECUDA;
}

} // namespace

int launch_attend(int dtype, const AttendArgs &a, cudaStream_t s) {
    if (dtype == ZC_BF16) return a.c.dim <= 64 ? launch<ZC_BF16, 64>(a, s) : launch<ZC_BF16, 128>(a, s);
    return a.c.dim <= 64 ? launch<ZC_FP16, 64>(a, s) : launch<ZC_FP16, 128>(a, s);
}

} // namespace kv
} // namespace zc
