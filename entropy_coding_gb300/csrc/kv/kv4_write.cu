// kv4_write.cu — new tokens quantised into the 4-bit cache.
//
// For each 16 columns of a row, with a = the largest finite |x|:
//   scale = the scale byte's number nearest to a / 6 (ties to the even byte)
//   code  = the E2M1 number nearest to x / scale (ties to the even code)
// as if a / 6 and x / scale were exact: the scale is found by comparing a with
// 6 times the midpoint of two scales, which float32 holds, and a quotient is
// rounded correctly (one division for 16 columns, two steps of refinement for
// each), which is enough for 16-bit x, whose quotients are either a midpoint of
// two codes or 2^-11 away from it; of float32's, those that round to a midpoint
// are moved off it by the sign of what remains.
//
// A thread has 16 columns; a CTA up to 64 packed tokens of one head, K and V,
// so that it writes runs of rows. Its reads do not wait for where the tokens
// belong: that is looked up meanwhile.
#include "kv4_common.cuh"

namespace zc {
namespace kv {
namespace {

constexpr int kThreads = 256, kTokens = 64;
constexpr int kPieces = kTokens * (kMaxHeadDim / 16) / kThreads;  // of K and of V, at most

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
    float x[16];
    in[0].get(x);
    in[1].get(x + 8);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    if (top >= 0x7F800000u) {
        bool nan = top > 0x7F800000u;
        if (nan) {
            byte = kScaleNaN;
            return make_uint2(0, 0);
        }
        top = 0;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const uint32_t u = __float_as_uint(x[i]) & 0x7FFFFFFFu;
            if (u < 0x7F800000u) top = max(top, u);
        }
    }
    byte = scale_byte(__uint_as_float(top));
    const float s = scale_float(byte), inv = 1.0f / s, most = 6.0f * s;
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float y = fminf(fmaxf(x[8 * h + i], -most), most), q0 = y * inv;
            q[i] = copysignf(fmaf(fmaf(-q0, s, y), inv, q0), y);  // (a zero keeps its sign)
            if (DT == ZC_FP32) {
                const float rest = fmaf(-q[i], s, y);
                const uint32_t u = __float_as_uint(q[i]);
                if (rest != 0.0f && (u & 0x1FFFFFu) == 0 && (u & 0x7FFFFFFFu)) q[i] = __uint_as_float((__float_as_int(rest) ^ int(u)) < 0 ? u - 1 : u + 1);
            }
        }
        w[h] = floatx8_to_e2m1(q);
    }
    return make_uint2(w[0], w[1]);
}

template <int DT> __global__ void __launch_bounds__(kThreads) write4_kernel(const __grid_constant__ MoveArgs a) {
    __shared__ int32_t s_pos[kTokens], s_block[kTokens];
    __shared__ uint32_t s_seq[kTokens];
    const uint32_t B = a.c.tokens, D = a.c.dim, h = blockIdx.y, per_row = D / 16;
    const uint32_t t0 = blockIdx.x * kTokens, n = min(uint32_t(kTokens), a.b.total - t0), units = n * per_row;
    const uint32_t inverse = 0xFFFFFFFFu / per_row + 1;  // i / per_row = i * inverse / 2^32 (1 piece a row: 0)
    auto row_of = [&](uint32_t i) { return inverse ? __umulhi(i, inverse) : i; };
    constexpr int elt = DT == ZC_FP32 ? 4 : 2;
    Piece<DT> in[2][kPieces][2];
#pragma unroll
    for (int p = 0; p < kPieces; p++) {
        const uint32_t i = threadIdx.x + p * kThreads, row = row_of(i);
        if (i >= units) continue;
#pragma unroll
        for (int kv = 0; kv < 2; kv++) {
            const uint8_t *x = static_cast<const uint8_t *>(a.x[kv].p) +
                               (int64_t(t0 + row) * a.x[kv].token + int64_t(h) * a.x[kv].head + (i - row * per_row) * 16) * elt;
            in[kv][p][0].load(x);
            in[kv][p][1].load(x + Piece<DT>::kBytes);
        }
    }
    locate(a.b, B, t0, n, s_pos, s_seq, a.d_status);
    for (uint32_t i = threadIdx.x; i < n; i += kThreads)
        s_block[i] = s_pos[i] < 0 ? -1 : int32_t(read_block(a.b, a.c, s_seq[i], block_of_16(a.c, uint32_t(s_pos[i]) / 16), a.d_status));
    __syncthreads();
#pragma unroll
    for (int p = 0; p < kPieces; p++) {
        const uint32_t i = threadIdx.x + p * kThreads, row = row_of(i);
        if (i >= units || s_block[row] < 0) continue;
        const int64_t id = s_block[row];
        const uint32_t g = i - row * per_row, at = h * B + uint32_t(s_pos[row]) - block_of_16(a.c, uint32_t(s_pos[row]) / 16) * B;
#pragma unroll
        for (int kv = 0; kv < 2; kv++) {
            uint32_t byte;
            const uint2 codes = quantise<DT>(in[kv][p], byte);
            *reinterpret_cast<uint2 *>(a.c.code[kv] + id * a.c.block_stride + int64_t(at) * a.c.row + g * 8) = codes;
            a.c.group[kv][id * a.c.scale_stride + int64_t(at) * per_row + g] = uint8_t(byte);
        }
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) report_batch(a.b, B, a.d_status, threadIdx.x, kThreads, true);
}

} // namespace

int launch_write4(int dtype, const MoveArgs &a, cudaStream_t s) {
    const dim3 grid((a.b.total + kTokens - 1) / kTokens, a.c.heads);
    switch (dtype) {
    case ZC_BF16: write4_kernel<ZC_BF16><<<grid, kThreads, 0, s>>>(a); break;
    case ZC_FP16: write4_kernel<ZC_FP16><<<grid, kThreads, 0, s>>>(a); break;
    default: write4_kernel<ZC_FP32><<<grid, kThreads, 0, s>>>(a); break;
    }
    return cudaGetLastError() == cudaSuccess ? ZC_OK : ZC_ECUDA;
}

} // namespace kv
} // namespace zc
