// kv_write.cu — new tokens quantised into the 8-bit cache.
//
// For each block that new tokens fall into, each head, and K and V apart:
// with a = the largest finite |x| of the new rows, `need` is the least power
// of two 2^e (e >= -126) with a <= 448 2^e. A block that held rows before
// keeps the larger of its scale (rounded up to a power of two) and `need`;
// when that grows, its old codes move to the new scale. New codes are
// x / scale to the nearest E4M3 value. Scales are powers of two, so that
// dividing by them is exact: the only rounding of a row is that to 4
// significant bits, and moving old codes rounds again only those that leave
// E4M3's normal range.
//
// One CTA does one block of one head, K or V, in one pass over its new rows:
// a thread keeps kHold pieces of 8 elements in registers while the CTA finds
// the largest magnitude, and then quantises them (256 threads hold 128 rows of
// 128 columns; rows beyond that are read again). The CTA is as small as that
// allows: what bounds it is the latency of its few dependent reads, which only
// more CTAs on an SM hide.
//
// Measured on a GB300: 104 MB of bfloat16 prompts (16978 tokens of 8 heads of
// 128, blocks of 64) in 19.7 us, 5.3 TB/s, 0.78 of the copy rate; the arithmetic
// units are at 49 % and 44 % of the warps are there: no unit's rate is the
// limit, a CTA's start is (its place in the batch, the sequence's length, then
// its rows: dependent reads, of which the first two need not be). Divisions
// by the row's pieces, four a piece at first, were 4 us of it; units of several
// heads in turn in one CTA, with the next rows on their way, were slower (27 us):
// they leave fewer CTAs. A decoding step of 32 tokens takes 5 us, a launch.
#include "kv_common.cuh"

namespace zc {
namespace kv {
namespace {

constexpr int kHold = 8;

// Eight elements from 16-byte aligned memory, as they are, and as floats.
template <int DT> struct Eight {
    uint4 v[DT == ZC_FP32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *p) {
        v[0] = __ldcs(static_cast<const uint4 *>(p));
        if (DT == ZC_FP32) v[DT == ZC_FP32 ? 1 : 0] = __ldcs(static_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ float2 pair(int i) const {  // elements 2i, 2i + 1
        const uint32_t *w = reinterpret_cast<const uint32_t *>(v);
        return DT == ZC_FP32 ? make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])) : unpack2<DT>(w[i]);
    }
    __device__ __forceinline__ uint32_t top() const {  // bits of the largest finite magnitude, as a float
        constexpr uint32_t kInf = DT == ZC_BF16 ? 0x7F80u : 0x7C00u;
        if (DT != ZC_FP32) {
            // two elements at a time, and one by one only where that finds an infinity or NaN
            const uint32_t *w = reinterpret_cast<const uint32_t *>(v);
            const uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
            const uint32_t t = max(m >> 16, m & 0xFFFFu);
            if (t < kInf) return __float_as_uint(DT == ZC_BF16 ? __uint_as_float(t << 16) : unpack2<DT>(t).x);
        }
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = pair(i);
            const uint32_t a = __float_as_uint(f.x) & 0x7FFFFFFFu, b = __float_as_uint(f.y) & 0x7FFFFFFFu;
            t = max(t, max(a < 0x7F800000u ? a : 0u, b < 0x7F800000u ? b : 0u));
        }
        return t;
    }
    __device__ __forceinline__ uint2 codes(float inv) const {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float2 f = pair(2 * i), g = pair(2 * i + 1);
            w[i] = float2_to_e4m3x2(f.x * inv, f.y * inv) | uint32_t(float2_to_e4m3x2(g.x * inv, g.y * inv)) << 16;
        }
        return make_uint2(w[0], w[1]);
    }
};

// Exponent field of the least power of two s >= 2^-126 with a <= 448 s, for
// the bits of a finite a >= 0: 448 = 1.75 2^8.
__device__ __forceinline__ uint32_t need_exponent(uint32_t a) {
    const int e = int(a >> 23) - 8 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return uint32_t(max(e, 1));
}
// Exponent field of a scale rounded up to a power of two.
__device__ __forceinline__ uint32_t ceil_exponent(float s) {
    const uint32_t u = __float_as_uint(s) & 0x7FFFFFFFu;
    return min(max((u >> 23) + ((u & 0x7FFFFFu) ? 1u : 0u), 1u), 254u);
}
__device__ __forceinline__ float two_to(int field) {  // 2^(field - 127), fields outside [1, 254] clamped
    return __uint_as_float(uint32_t(min(max(field, 1), 254)) << 23);
}

template <int DT, int kThreads> __device__ __forceinline__ void write_block(const MoveArgs &a, uint32_t &s_max) {
    uint32_t at;
    const uint32_t s = find_seq(a.b, blockIdx.x, 1, a.c.tokens, 2, at);
    const Seq q = read_seq(a.b, s, a.d_status, a.c.tokens, false);
    if (at == kNoSlot || !q.ok || q.n == 0 || uint32_t(q.len) < q.n) return;
    const uint32_t B = a.c.tokens, D = a.c.dim, h = blockIdx.y, kvi = blockIdx.z;
    Span span;
    if (!block_span(uint32_t(q.len), q.n, B, at, span)) return;
    const uint32_t start = uint32_t(q.len) - q.n, blk = span.blk, lo = span.lo, n0 = lo - blk * B, rows = span.hi - lo;
    const int elt = DT == ZC_FP32 ? 4 : 2;
    const uint8_t *x = static_cast<const uint8_t *>(a.x[kvi].p) +
                       ((int64_t(q.first) + (lo - start)) * a.x[kvi].token + int64_t(h) * a.x[kvi].head) * elt;
    const uint32_t per_row = D / 8, chunks = rows * per_row;

    const uint32_t inverse = 0xFFFFFFFFu / per_row + 1;  // i / per_row = i * inverse / 2^32 for the few thousand pieces of a block
    const int64_t stride = a.x[kvi].token * elt;
    auto piece_of = [&](uint32_t i) {
        const uint32_t row = __umulhi(i, inverse);
        return x + row * stride + (i - row * per_row) * (8 * elt);
    };
    Eight<DT> held[kHold];
    uint32_t top = 0;
#pragma unroll
    for (int n = 0; n < kHold; n++)
        if (threadIdx.x + n * kThreads < chunks) held[n].load(piece_of(threadIdx.x + n * kThreads));
    // (the block is looked up while the rows are on their way)
    const int64_t id = read_block(a.b, a.c, s, blk, a.d_status);
    if (id < 0) return;
    uint8_t *codes = a.c.code[kvi] + id * a.c.block_stride + int64_t(h) * B * D;
    float *scale = a.c.scale[kvi] + id * a.c.scale_stride + h;
    const float old = n0 ? *scale : 0.0f;
    if (threadIdx.x == 0) s_max = 0;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kHold; n++)
        if (threadIdx.x + n * kThreads < chunks) top = max(top, held[n].top());
    for (uint32_t i = threadIdx.x + kHold * kThreads; i < chunks; i += kThreads) {
        Eight<DT> e;
        e.load(piece_of(i));
        top = max(top, e.top());
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((threadIdx.x & 31) == 0) atomicMax(&s_max, top);
    __syncthreads();

    uint32_t field = need_exponent(s_max);
    if (n0) {
        field = max(field, ceil_exponent(old));
        const float now = two_to(int(field));
        if (now != old) {
            // 1 / now is exact: field <= 254 - 8 for a finite x, and a larger one only restates the old scale
            const float ratio = old / now;
            for (uint32_t i = threadIdx.x; i < n0 * per_row; i += kThreads) {
                uint2 *p = reinterpret_cast<uint2 *>(codes) + i;
                uint2 c = *p;
                uint16_t w[4] = {uint16_t(c.x), uint16_t(c.x >> 16), uint16_t(c.y), uint16_t(c.y >> 16)};
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const float2 f = e4m3x2_to_float2(w[k]);
                    w[k] = float2_to_e4m3x2(f.x * ratio, f.y * ratio);
                }
                *p = make_uint2(w[0] | uint32_t(w[1]) << 16, w[2] | uint32_t(w[3]) << 16);
            }
        }
    }
    const float inv = 1.0f / two_to(int(field));
    if (threadIdx.x == 0) *scale = two_to(int(field));
    uint2 *to = reinterpret_cast<uint2 *>(codes + int64_t(n0) * D);
#pragma unroll
    for (int n = 0; n < kHold; n++)
        if (threadIdx.x + n * kThreads < chunks) to[threadIdx.x + n * kThreads] = held[n].codes(inv);
    for (uint32_t i = threadIdx.x + kHold * kThreads; i < chunks; i += kThreads) {
        Eight<DT> e;
        e.load(piece_of(i));
        to[i] = e.codes(inv);
    }
}

template <int DT, int kThreads> __global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ MoveArgs a) {
    __shared__ uint32_t s_max;
    write_block<DT, kThreads>(a, s_max);
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) report_batch(a.b, a.c.tokens, a.d_status, threadIdx.x, kThreads, true);
}

// Threads by the pieces of a block that a call may write: as few as hold them. (Blocks of 160 pieces take 8 us with 64
// threads and 14 with 256, blocks of 1024 pieces 26 us with 128 and 33 with 256.)
template <int DT> void launch(const MoveArgs &a, cudaStream_t s) {
    const dim3 grid(slot_of(a.b.total, a.b.n_seqs, 1, a.c.tokens, 2), a.c.heads, 2);
    const uint32_t rows = a.b.most < a.c.tokens ? a.b.most : a.c.tokens, pieces = rows * (a.c.dim / 8);
    if (pieces <= 64 * kHold) write_kernel<DT, 64><<<grid, 64, 0, s>>>(a);
    else if (pieces <= 128 * kHold) write_kernel<DT, 128><<<grid, 128, 0, s>>>(a);
    else write_kernel<DT, 256><<<grid, 256, 0, s>>>(a);
}

} // namespace

int launch_write(int dtype, const MoveArgs &a, cudaStream_t s) {
    switch (dtype) {
    case ZC_BF16: launch<ZC_BF16>(a, s); break;
    case ZC_FP16: launch<ZC_FP16>(a, s); break;
    default: launch<ZC_FP32>(a, s); break;
    }
    return cudaGetLastError() == cudaSuccess ? ZC_OK : ZC_ECUDA;
}

} // namespace kv
} // namespace zc
