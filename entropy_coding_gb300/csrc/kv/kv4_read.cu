// kv4_read.cu — tokens of the 4-bit cache as numbers: code * scale, exact in
// every type.
//
// A thread has 8 columns: a word of codes, a scale byte, and one 16-byte store
// (two for float32, in pairs of threads), so that a warp's stores are whole runs of memory. A CTA
// has 64 packed tokens, K and V, head after head; all of a thread's reads of a
// head are in flight before the first is used.
//
// Measured on a GB300: 133678 tokens of 8 heads of 128 to bfloat16, 702 MB, four
// fifths of them written, in 111 us: 6.3 TB/s, 0.94 of the copy rate (one head a
// CTA, with its lookups before its reads, 148); 777 tokens of float16 in 3.3;
// 16978 tokens to float32, 159 MB, in 29.1 (5.5 TB/s).
#include "kv4_common.cuh"

namespace zc {
namespace kv {
namespace {

constexpr int kThreads = 256, kTokens = 64;
constexpr int kPieces = kTokens * (kMaxHeadDim / 8) / kThreads;  // of K and of V, at most

template <int DT> __device__ __forceinline__ void number(uint32_t codes, uint32_t byte, Piece<DT> &out) {
    uint32_t h[4];
    e2m1x8_to_half2x4(codes, h[0], h[1], h[2], h[3]);
    const uint32_t s = scale_half2(byte);
    float2 x[4];
#pragma unroll
    for (int k = 0; k < 4; k++) h[k] = mul_half2(h[k], s), x[k] = unpack2<ZC_FP16>(h[k]);
    if (DT == ZC_FP16) out.v[0] = make_uint4(h[0], h[1], h[2], h[3]);
    else out.put(x);
}

// The 32 bytes of each of two neighbours, each of whose stores of 16 bytes is then beside the other's: the first store is of
// the even thread's 32 bytes, the second of the odd one's, whole sectors. Both are here, in one row and as far: a row has an
// even number of pieces (head_dim is a multiple of 16). (16978 tokens: 40.4 us without, 29.1 with.)
__device__ __forceinline__ void store_paired(uint8_t *to, const Piece<ZC_FP32> &x) {
    const bool odd = threadIdx.x & 1;
    const uint32_t both = 3u << (threadIdx.x & 30);
    const uint4 give = odd ? x.v[0] : x.v[1];
    const uint4 got = make_uint4(__shfl_xor_sync(both, give.x, 1), __shfl_xor_sync(both, give.y, 1), __shfl_xor_sync(both, give.z, 1),
                                 __shfl_xor_sync(both, give.w, 1));
    uint4 *at = reinterpret_cast<uint4 *>(to - (odd ? 32 : 0)) + odd;
    __stcs(at, odd ? got : x.v[0]);
    __stcs(at + 2, odd ? x.v[1] : got);
}

template <int DT> __global__ void __launch_bounds__(kThreads) read4_kernel(const __grid_constant__ MoveArgs a, uint32_t heads) {
    __shared__ int2 s_at[kTokens];  // position, sequence
    __shared__ int32_t s_block[kTokens];
    const uint32_t B = a.c.tokens, D = a.c.dim, per_row = D / 8, h0 = blockIdx.y * heads, h1 = min(h0 + heads, a.c.heads);
    const uint32_t t0 = blockIdx.x * kTokens, n = min(uint32_t(kTokens), a.b.total - t0), units = n * per_row;
    const uint32_t inverse = 0xFFFFFFFFu / per_row + 1;  // i / per_row = i * inverse / 2^32
    after_the_last();
    locate(a.b, B, t0, n, s_at, a.d_status);
    for (uint32_t i = threadIdx.x; i < n; i += kThreads)
        s_block[i] = s_at[i].x < 0 ? -1 : int32_t(read_block(a.b, a.c, uint32_t(s_at[i].y), block_of_16(a.c, uint32_t(s_at[i].x) / 16), a.d_status));
    __syncthreads();
    int64_t code_at[kPieces], scale_at[kPieces];  // of the next head to be asked for
    bool there[kPieces];
#pragma unroll
    for (int p = 0; p < kPieces; p++) {
        const uint32_t i = threadIdx.x + p * kThreads, row = __umulhi(i, inverse);
        there[p] = i < units && s_block[row] >= 0;
        if (!there[p]) continue;
        const int64_t id = s_block[row];
        const uint32_t c = i - row * per_row, at = h0 * B + uint32_t(s_at[row].x) - block_of_16(a.c, uint32_t(s_at[row].x) / 16) * B;
        code_at[p] = id * a.c.block_stride + int64_t(at) * a.c.row + c * 4;
        scale_at[p] = id * a.c.scale_stride + int64_t(at) * (D / 16) + c / 2;
    }
    uint32_t codes[2][kPieces], byte[2][kPieces];
    auto ask = [&]() {
#pragma unroll
        for (int p = 0; p < kPieces; p++) {
            if (!there[p]) continue;
#pragma unroll
            for (int kv = 0; kv < 2; kv++) {
                codes[kv][p] = __ldcs(reinterpret_cast<const uint32_t *>(a.c.code[kv] + code_at[p]));
                byte[kv][p] = __ldg(a.c.group[kv] + scale_at[p]);
            }
            code_at[p] += int64_t(B) * a.c.row;
            scale_at[p] += int64_t(B) * (D / 16);
        }
    };
    constexpr int elt = DT == ZC_FP32 ? 4 : 2;
    ask();
    for (uint32_t h = h0; h < h1; h++) {
        uint32_t now[2][kPieces], by[2][kPieces];
#pragma unroll
        for (int p = 0; p < kPieces; p++) now[0][p] = codes[0][p], now[1][p] = codes[1][p], by[0][p] = byte[0][p], by[1][p] = byte[1][p];
        if (h + 1 < h1) ask();  // the next head's are on their way while this one's are written
#pragma unroll
        for (int p = 0; p < kPieces; p++) {
            if (!there[p]) continue;
            const uint32_t i = threadIdx.x + p * kThreads, row = __umulhi(i, inverse);
#pragma unroll
            for (int kv = 0; kv < 2; kv++) {
                Piece<DT> x;
                number<DT>(now[kv][p], by[kv][p], x);
                uint8_t *to = static_cast<uint8_t *>(a.x[kv].p) +
                              (int64_t(t0 + row) * a.x[kv].token + int64_t(h) * a.x[kv].head + (i - row * per_row) * 8) * elt;
                if constexpr (DT == ZC_FP32) store_paired(to, x);
                else x.store(to);
            }
        }
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) report_batch(a.b, B, a.d_status, threadIdx.x, kThreads, true);
}

template <int DT> int launch(const MoveArgs &a, cudaStream_t s) {
    const uint32_t runs = (a.b.total + kTokens - 1) / kTokens;
    const uint32_t heads = heads_of_a_cta(runs, a.c.heads);
    return launch_early(read4_kernel<DT>, dim3(runs, (a.c.heads + heads - 1) / heads), kThreads, 0, s, a, heads);
}

} // namespace

int launch_read4(int dtype, const MoveArgs &a, cudaStream_t s) {
    return dtype == ZC_BF16 ? launch<ZC_BF16>(a, s) : dtype == ZC_FP16 ? launch<ZC_FP16>(a, s) : launch<ZC_FP32>(a, s);
}

} // namespace kv
} // namespace zc
