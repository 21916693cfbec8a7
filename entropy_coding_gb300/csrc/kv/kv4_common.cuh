// kv4_common.cuh — the 4-bit cache's numbers, pieces of rows in registers, and
// where packed tokens belong (kv4_write.cu, kv4_read.cu, kv_rotate.cu).
//
// A scale byte is bits 14 to 7 of a half: one shift makes the number of it. A
// code times a scale has at most 6 significant bits and lies between 2^-18 and
// 61440, so that half holds it exactly and one product of halves makes two
// numbers.
#pragma once

#include "kv_common.cuh"

namespace zc {
namespace kv {

constexpr uint32_t kScaleMost = 0xE2, kScaleNaN = 0xFF;  // 10240: 6 times that is still finite in half

// Heads that a CTA of a run of tokens does one after another: the run's places are looked up once for them, and the next
// head's numbers are on their way meanwhile; as many as leave 3 CTAs for 2 SMs. (133678 tokens of 8 heads read: 1 head 148
// us, 2 heads 118, 4 and 8 heads 111; 16978 tokens 20.1, 16.2, 15.9 and 14.9; 777 tokens 3.3, 3.9, 5.0 and 7.1; 32 tokens
// written and read back 5.6, 6.4, 8.3 and 12.2.)
inline uint32_t heads_of_a_cta(uint32_t runs, uint32_t heads) {
    const uint64_t most = uint64_t(runs) * heads * 2 / (3 * uint64_t(sm_count()));
    if (most <= 1) return 1;
    const uint32_t groups = most >= heads ? 1 : uint32_t((heads + most - 1) / most);
    return (heads + groups - 1) / groups;
}

#ifdef __CUDACC__

// Eight codes (columns in order from the low half of the low byte on) to eight halves.
__device__ __forceinline__ void e2m1x8_to_half2x4(uint32_t v, uint32_t &h0, uint32_t &h1, uint32_t &h2, uint32_t &h3) {
    asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4; cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b; "
        "cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d;}"
        : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3) : "r"(v));
}
// Eight floats to eight codes, to nearest even, saturating at +-6.
__device__ __forceinline__ uint32_t floatx8_to_e2m1(const float2 *x) {
    uint32_t r;
    asm("{.reg .b8 a, b, c, d; cvt.rn.satfinite.e2m1x2.f32 a, %2, %1; cvt.rn.satfinite.e2m1x2.f32 b, %4, %3; "
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5; cvt.rn.satfinite.e2m1x2.f32 d, %8, %7; mov.b32 %0, {a, b, c, d};}"
        : "=r"(r) : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y));
    return r;
}
// A scale byte as a half, in both halves of a word.
__device__ __forceinline__ uint32_t scale_half2(uint32_t byte) { return byte * 0x00800080u; }
__device__ __forceinline__ float scale_float(uint32_t byte) { return __half2float(__ushort_as_half(uint16_t(byte << 7))); }
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Eight elements of type DT at 16-byte aligned memory.
template <int DT> struct Piece {
    static constexpr int kWords = DT == ZC_FP32 ? 2 : 1, kBytes = 16 * kWords;
    uint4 v[kWords];
    __device__ __forceinline__ void load(const void *p) {
#pragma unroll
        for (int i = 0; i < kWords; i++) v[i] = __ldcs(static_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void store(void *p) const {
#pragma unroll
        for (int i = 0; i < kWords; i++) __stcs(static_cast<uint4 *>(p) + i, v[i]);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; i++) v[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float2 *x) const {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(v);
#pragma unroll
        for (int i = 0; i < 4; i++)
            x[i] = DT == ZC_FP32 ? make_float2(__uint_as_float(w[2 * i % (4 * kWords)]), __uint_as_float(w[(2 * i + 1) % (4 * kWords)])) : unpack2<DT>(w[i]);
    }
    __device__ __forceinline__ void put(const float2 *x) {  // rounded once
        uint32_t *w = reinterpret_cast<uint32_t *>(v);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (DT == ZC_FP32) w[2 * i % (4 * kWords)] = __float_as_uint(x[i].x), w[(2 * i + 1) % (4 * kWords)] = __float_as_uint(x[i].y);
            else w[i] = pack2<DT>(x[i].x, x[i].y);
        }
    }
    // Bits of the largest magnitude, as a float: an infinity's or above where there is one or a NaN.
    __device__ __forceinline__ uint32_t top() const {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(v);
        uint32_t t = 0;
        if constexpr (DT == ZC_FP32) {
#pragma unroll
            for (int i = 0; i < 8; i++) t = max(t, w[i] & 0x7FFFFFFFu);
            return t;
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) t = __vmaxu2(t, w[i] & 0x7FFF7FFFu);
            t = max(t >> 16, t & 0xFFFFu);
            return DT == ZC_BF16 ? t << 16 : __float_as_uint(unpack2<DT>(t).x);
        }
    }
};

// Positions (x) of the packed tokens [t0, t0 + n) and their sequences (y), by the whole CTA: each sequence's thread writes its
// own tokens, or, if they are many, its warp does. Tokens of no sequence (or of one whose counts are wrong) get position -1.
// Where counts fall, two sequences may claim a token: one store for both numbers, so that the position is its sequence's.
// block_tokens: a sequence must not be longer than its table; 0 for calls that do not use the table.
__device__ __forceinline__ void locate(const Batch &b, uint32_t block_tokens, uint32_t t0, uint32_t n, int2 *s_at, int32_t *d_status) {
    for (uint32_t i = threadIdx.x; i < n; i += blockDim.x) s_at[i] = make_int2(-1, 0);
    __syncthreads();
    // Of many sequences the first that matters is found by halving (9728 single tokens rotated: 43 us, with all of them looked at 60).
    uint32_t s0 = 0;
    if (b.n_seqs > 8 * blockDim.x)
        for (uint32_t above = b.n_seqs; above - s0 > 1;) {
            const uint32_t mid = (s0 + above) / 2;
            if (tokens_before(b, mid) <= t0) s0 = mid;
            else above = mid;
        }
    for (; s0 < b.n_seqs && (s0 == 0 || tokens_before(b, s0) < t0 + n); s0 += blockDim.x) {
        const uint32_t s = s0 + threadIdx.x;
        uint32_t lo = 0, hi = 0;
        int32_t from = 0;  // position of token lo
        if (s < b.n_seqs) {
            const Seq q = read_seq(b, s, d_status, block_tokens ? block_tokens : 0xFFFFFFFFu, false);
            if (q.ok && uint32_t(q.len) >= q.n) {
                lo = max(q.first, t0), hi = min(q.first + q.n, t0 + n);
                from = q.len - int32_t(q.n) + int32_t(lo - q.first);
            }
        }
        const bool many = int32_t(hi - lo) > 4;
        if (!many)
            for (uint32_t t = lo; t < hi; t++) s_at[t - t0] = make_int2(from + int32_t(t - lo), int32_t(s));
        uint32_t left = __ballot_sync(0xFFFFFFFFu, many);
        while (left) {
            const int of = __ffs(int(left)) - 1;
            left &= left - 1;
            const uint32_t l = __shfl_sync(0xFFFFFFFFu, lo, of), e = __shfl_sync(0xFFFFFFFFu, hi, of);
            const int32_t p = __shfl_sync(0xFFFFFFFFu, from, of);
            const uint32_t q = s - (threadIdx.x & 31) + of;
            for (uint32_t t = l + (threadIdx.x & 31); t < e; t += 32) s_at[t - t0] = make_int2(p + int32_t(t - l), int32_t(q));
        }
    }
    __syncthreads();
}

#endif  // __CUDACC__

} // namespace kv
} // namespace zc
