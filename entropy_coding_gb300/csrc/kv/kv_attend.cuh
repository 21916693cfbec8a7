// kv_attend.cuh — what the attention kernels share: arithmetic of weights,
// the keys that a row sees, sums over a CTA, and finished rows.
#pragma once

#include "kv_common.cuh"

namespace zc {
namespace kv {

constexpr float kNone = -INFINITY;
// How far (log2) the running maxima may lag behind: of the scores, and of the contributions.
constexpr float kSlack = 8.0f, kSlackW = 6.0f;
// The unit of the largest contribution stands for 2^kRaise in half: a weight of up to 2^(kRaise + kSlackW) = 2^15 is
// finite there, one above 2^-23 of the unit keeps half's 11 bits, and what a smaller one loses is below 2^-34 of the unit.
// That matters where one key has nearly all of a row's weight and a small value: the others' weights are the output then,
// and over 2^17 keys each of them is 2^-24 of the unit if they share a hundredth of the weight. (Following contributions
// more closely leaves room for a higher unit and costs rescalings: 16 sequences of 2 to 5 tokens take 24.8, 25.5 and 26.4
// us at 2^8 and 2^7, 2^6 and 2^9, 2^4 and 2^11, an 8192-token prompt 452, 454 and 456.)
constexpr float kRaise = 9.0f;
static_assert(kRaise + kSlackW <= 15.0f, "weights that half does not hold");

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

// The power of two that brings a bfloat16 row whose largest magnitude has these
// float bits to [2^14, 2^15), and its inverse, within float's normal range.
__device__ __forceinline__ void row_powers(uint32_t top, float &up, float &down) {
    const int field = min(max(127 + 14 - (int(top >> 23) - 127), 1), 253);
    up = __uint_as_float(uint32_t(field) << 23);
    down = __uint_as_float(uint32_t(254 - field) << 23);
}

// The keys [l, e) that a row sees.
__device__ __forceinline__ void bounds(const AttendArgs &a, const Seq &seq, uint32_t row, int &l, int &e) {
    const int pos = seq.len - int(seq.n) + int(row / a.group);  // (may be below 0: more new tokens than the sequence has)
    e = a.causal ? max(pos + 1, 0) : seq.len;
    l = a.window && pos >= int(a.window) ? pos - int(a.window) + 1 : 0;
    if (l > e) l = e;
}

// Where a row's query head is among the tensor's (q or out), in elements.
__device__ __forceinline__ int64_t row_at(const AttendArgs &a, const Rows &x, const Seq &seq, uint32_t h, uint32_t row) {
    const uint32_t token = row / a.group, head = row - token * a.group;
    return int64_t(seq.first + token) * x.token + int64_t(h * a.group + head) * x.head;
}
__device__ __forceinline__ float *lse_at(const AttendArgs &a, const Seq &seq, uint32_t h, uint32_t row) {
    const uint32_t token = row / a.group, head = row - token * a.group;
    return a.lse + int64_t(seq.first + token) * a.heads + h * a.group + head;
}

// Inclusive sum over the threads up to this one; `total`: over all of the CTA's kWarps warps.
template <int kWarps> __device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t *s_warp, uint64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v += u;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
        if (w < warp) v += s_warp[w];
        total += s_warp[w];
    }
    return v;
}

// Two numbers of the output's type.
__device__ __forceinline__ uint32_t pack_out(const AttendArgs &a, float x, float y) {
    return a.dtype == ZC_BF16 ? pack2<ZC_BF16>(x, y) : pack2<ZC_FP16>(x, y);
}

// A finished row is its sum (in units of 2^(W - kRaise)) by this factor: out = x / L in the units of M. A row that sees no
// key is 0, whatever x holds. (L is NaN where a score was. The power in two halves: neither leaves float's range where
// value scales are near its ends.)
__device__ __forceinline__ float row_factor(float M, float W, float L) {
    if (W == kNone) return 0.0f / L;
    const float half = 0.5f * (W - M - kRaise), x = ex2(half);
    return x * (x / L);
}
__device__ __forceinline__ float row_lse(float M, float L) { return L == 0.0f ? kNone : (M + log2f(L)) * 0.6931471805599453f; }

// n columns (a multiple of 4) of a finished row from `col` on.
template <int n>
__device__ __forceinline__ void emit(const AttendArgs &a, const Seq &seq, uint32_t h, uint32_t row, int col,
                                     const float (&x)[n], float M, float W, float L) {
    const float by = row_factor(M, W, L);
    uint16_t *o = static_cast<uint16_t *>(a.out.p) + row_at(a, a.out, seq, h, row) + col;
#pragma unroll
    for (int k = 0; k < n; k += 4)
        *reinterpret_cast<uint2 *>(o + k) = L == 0.0f ? make_uint2(0, 0) : make_uint2(pack_out(a, x[k] * by, x[k + 1] * by),
                                                                                      pack_out(a, x[k + 2] * by, x[k + 3] * by));
    if (a.lse && col == 0) *lse_at(a, seq, h, row) = row_lse(M, L);
}

} // namespace kv
} // namespace zc
