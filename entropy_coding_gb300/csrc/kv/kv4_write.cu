// kv4_write.cu — new tokens quantised into the 4-bit cache.
//
// For each 16 columns of a row, with a = the largest finite |x|:
//   scale = the scale byte's number nearest to a / 6 (ties to the even byte)
//   code  = the E2M1 number nearest to x / scale (ties to the even code)
// as if a / 6 and x / scale were exact: the scale is found by comparing a with
// 6 times the midpoint of two scales, which float32 holds, and a quotient is
// taken with the reciprocal in two floats, so that it is within 2^-46 before
// its rounding: that is enough for 16-bit x, whose quotients are either a
// midpoint of two codes, and then come out as it, or 2^-11 away from it; of
// float32's, those that round to a midpoint are moved off it by the sign of what
// remains. (With the reciprocal in one float x = 3.5 s, s = 1.75, misses its
// midpoint.)
//
// A thread has 16 columns of a packed token, K and V, head after head; a CTA as
// many tokens as that makes, so that it writes runs of rows. Its first reads do not wait
// for where the tokens belong: that is looked up meanwhile.
//
// Measured on a GB300: 16978 tokens of 8 heads of 128, bfloat16, 70 MB read and 20
// written, in about 14.5 us (6.1 TB/s); 32 tokens in 3. The arithmetic units are
// half busy: what counted was two numbers to an instruction, the type's own
// comparisons for the largest magnitude and a head's rows on their way while the
// one before them is worked on (27 us without); CTAs of 128 threads are faster
// than of 256 (by 4 us), which wait for one another's lookups.
#include "kv4_common.cuh"

namespace zc {
namespace kv {
namespace {

constexpr int kThreads = 128;

// Scale byte for 16 columns whose largest magnitude is a (finite).
__device__ __forceinline__ uint32_t scale_byte(float a) {
    // the byte below (or, by the rounding of the product, next to) a / 6, and then the nearer of it and the next
    const float x = fminf(a * (1.0f / 6.0f), 12288.0f);
    const uint32_t low = __half_as_ushort(__float2half_rz(x)) >> 7;
    const float middle = 6.0f * __half2float(__ushort_as_half(uint16_t(low << 7 | 0x40)));
    const uint32_t byte = low + (a > middle || (a == middle && (low & 1)) ? 1 : 0);
    return min(max(byte, 1u), kScaleMost);
}

// Codes of 16 columns, and their scale byte.
template <int DT> __device__ __forceinline__ uint2 quantise(const Piece<DT> (&in)[2], uint32_t &byte) {
    float2 x[8];
    in[0].get(x);
    in[1].get(x + 4);
    uint32_t top = max(in[0].top(), in[1].top());
    if (top > 0x7F800000u) {
        byte = kScaleNaN;
        return make_uint2(0, 0);
    }
    const bool infinite = top == 0x7F800000u;
    if (infinite) {
        top = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t u = __float_as_uint(x[i].x) & 0x7FFFFFFFu, v = __float_as_uint(x[i].y) & 0x7FFFFFFFu;
            top = max(top, max(u < 0x7F800000u ? u : 0u, v < 0x7F800000u ? v : 0u));
        }
    }
    byte = scale_byte(__uint_as_float(top));
    const float s = scale_float(byte);
    if (infinite) {
        const float most = 6.0f * s;
#pragma unroll
        for (int i = 0; i < 8; i++) x[i].x = fminf(fmaxf(x[i].x, -most), most), x[i].y = fminf(fmaxf(x[i].y, -most), most);
    }
    // 1 / s in two parts, neither negative: a zero keeps its sign
    const float inv = __frcp_rd(s), rest = fmaf(-s, inv, 1.0f) * inv;
    float2 q[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        q[i] = fma2(x[i], both(inv), mul2(x[i], both(rest)));
        if (DT == ZC_FP32) {
            const float2 left = fma2(q[i], both(-s), x[i]);
            auto off = [](float q, float left) {
                const uint32_t u = __float_as_uint(q);
                return left != 0.0f && (u & 0x1FFFFFu) == 0 && (u & 0x7FFFFFFFu) ? __uint_as_float((__float_as_int(left) ^ int(u)) < 0 ? u - 1 : u + 1) : q;
            };
            q[i] = make_float2(off(q[i].x, left.x), off(q[i].y, left.y));
        }
    }
    return make_uint2(floatx8_to_e2m1(q), floatx8_to_e2m1(q + 4));
}

template <int DT> __global__ void __launch_bounds__(kThreads) write4_kernel(const __grid_constant__ MoveArgs a, uint32_t heads) {
    __shared__ int2 s_at[kThreads];  // position, sequence
    __shared__ int32_t s_block[kThreads];
    const uint32_t B = a.c.tokens, per_row = a.c.dim / 16, tokens = kThreads / per_row, h0 = blockIdx.y * heads, h1 = min(h0 + heads, a.c.heads);
    const uint32_t t0 = blockIdx.x * tokens, n = min(tokens, a.b.total - t0);
    const uint32_t row = threadIdx.x / per_row, g = threadIdx.x - row * per_row;
    const bool mine = row < n;
    constexpr int elt = DT == ZC_FP32 ? 4 : 2;
    Piece<DT> next[2][2];
    auto ask = [&](uint32_t h) {
        if (!mine) return;
#pragma unroll
        for (int kv = 0; kv < 2; kv++) {
            const uint8_t *x = static_cast<const uint8_t *>(a.x[kv].p) + (int64_t(t0 + row) * a.x[kv].token + int64_t(h) * a.x[kv].head + g * 16) * elt;
            next[kv][0].load(x);
            next[kv][1].load(x + Piece<DT>::kBytes);
        }
    };
    after_the_last();
    ask(h0);
    locate(a.b, B, t0, n, s_at, a.d_status);
    if (threadIdx.x < n) {
        const int2 at = s_at[threadIdx.x];
        s_block[threadIdx.x] = at.x < 0 ? -1 : int32_t(read_block(a.b, a.c, uint32_t(at.y), block_of_16(a.c, uint32_t(at.x) / 16), a.d_status));
    }
    __syncthreads();
    const bool there = mine && s_block[mine ? row : 0] >= 0;
    int64_t code_at = 0, scale_at = 0;
    if (there) {
        const int64_t id = s_block[row];
        const uint32_t at = h0 * B + uint32_t(s_at[row].x) - block_of_16(a.c, uint32_t(s_at[row].x) / 16) * B;
        code_at = id * a.c.block_stride + int64_t(at) * a.c.row + g * 8;
        scale_at = id * a.c.scale_stride + int64_t(at) * per_row + g;
    }
    for (uint32_t h = h0; h < h1; h++) {
        Piece<DT> in[2][2] = {{next[0][0], next[0][1]}, {next[1][0], next[1][1]}};
        if (h + 1 < h1) ask(h + 1);  // the next head's are on their way while this one's are worked on
        if (!there) continue;
#pragma unroll
        for (int kv = 0; kv < 2; kv++) {
            uint32_t byte;
            const uint2 codes = quantise<DT>(in[kv], byte);
            *reinterpret_cast<uint2 *>(a.c.code[kv] + code_at) = codes;
            a.c.group[kv][scale_at] = uint8_t(byte);
        }
        code_at += int64_t(B) * a.c.row;
        scale_at += int64_t(B) * per_row;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) report_batch(a.b, B, a.d_status, threadIdx.x, kThreads, true);
}

template <int DT> int launch(const MoveArgs &a, cudaStream_t s) {
    const uint32_t tokens = kThreads / (a.c.dim / 16), runs = (a.b.total + tokens - 1) / tokens;
    const uint32_t heads = heads_of_a_cta(runs, a.c.heads);
    return launch_early(write4_kernel<DT>, dim3(runs, (a.c.heads + heads - 1) / heads), kThreads, 0, s, a, heads);
}

} // namespace

int launch_write4(int dtype, const MoveArgs &a, cudaStream_t s) {
    return dtype == ZC_BF16 ? launch<ZC_BF16>(a, s) : dtype == ZC_FP16 ? launch<ZC_FP16>(a, s) : launch<ZC_FP32>(a, s);
}

} // namespace kv
} // namespace zc
