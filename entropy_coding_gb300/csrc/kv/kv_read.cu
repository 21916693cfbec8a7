// kv_read.cu — tokens of the 8-bit cache as numbers: value(code) * scale,
// rounded once to the type asked for.
//
// One CTA does kTokens packed tokens of one head, K and V, 16 codes (16 bytes)
// a piece. A thread asks for all of its pieces before it converts the first:
// 8 reads in flight a thread for 128 columns.
//
// Measured on a GB300: 133678 tokens of 8 heads of 128 to bfloat16, 821 MB, in
// 142 us: 5.8 TB/s, 0.85 of the copy rate, with two thirds of the bytes written.
// 16 tokens a CTA and one read a thread took 155 us.
#include "kv_common.cuh"

namespace zc {
namespace kv {
namespace {

constexpr int kThreads = 128, kTokens = 64;
constexpr int kPieces = kTokens * (kMaxHeadDim / 16) / kThreads;  // of K and of V, at most

template <int DT> __device__ __forceinline__ void store16(void *p, const float (&x)[16]) {
    if (DT == ZC_FP32) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            static_cast<float4 *>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 2; i++)
            __stcs(static_cast<uint4 *>(p) + i, make_uint4(pack2<DT>(x[8 * i], x[8 * i + 1]), pack2<DT>(x[8 * i + 2], x[8 * i + 3]),
                                                    pack2<DT>(x[8 * i + 4], x[8 * i + 5]), pack2<DT>(x[8 * i + 6], x[8 * i + 7])));
    }
}

template <int DT> __device__ __forceinline__ void read_tokens(const MoveArgs &a) {
    uint32_t at;
    const uint32_t s = find_seq(a.b, blockIdx.x, 1, kTokens, 1, at);
    const Seq q = read_seq(a.b, s, a.d_status, a.c.tokens, false);
    if (at == kNoSlot || !q.ok || q.n == 0 || uint32_t(q.len) < q.n) return;
    const uint32_t B = a.c.tokens, D = a.c.dim, h = blockIdx.y;
    const uint32_t per_row = D / 16, t0 = at * kTokens, n = min(uint32_t(kTokens), q.n - min(q.n, t0)) * per_row;
    const uint32_t pos0 = uint32_t(q.len) - q.n + t0;
    const uint32_t inverse = 0xFFFFFFFFu / per_row + 1;  // i / per_row = i * inverse / 2^32 (1 piece a row: 0)
    auto row_of = [&](uint32_t i) { return inverse ? __umulhi(i, inverse) : i; };
    uint4 c[2][kPieces];
    float scale[2][kPieces];
    bool there[kPieces];
#pragma unroll
    for (int p = 0; p < kPieces; p++) {
        const uint32_t i = threadIdx.x + p * kThreads, row = row_of(i), pos = pos0 + row;
        there[p] = false;
        if (i >= n) continue;
        const uint32_t blk = block_of_16(a.c, pos / 16);
        const int64_t id = read_block(a.b, a.c, s, blk, a.d_status);
        if (id < 0) continue;
        there[p] = true;
        const int64_t off = id * a.c.block_stride + (int64_t(h) * B + (pos - blk * B)) * D + (i - row * per_row) * 16;
#pragma unroll
        for (int kv = 0; kv < 2; kv++) {
            c[kv][p] = __ldcs(reinterpret_cast<const uint4 *>(a.c.code[kv] + off));
            scale[kv][p] = __ldg(a.c.scale[kv] + id * a.c.scale_stride + h);
        }
    }
#pragma unroll
    for (int p = 0; p < kPieces; p++) {
        if (!there[p]) continue;
        const uint32_t i = threadIdx.x + p * kThreads, row = row_of(i);
#pragma unroll
        for (int kv = 0; kv < 2; kv++) {
            const uint32_t w[4] = {c[kv][p].x, c[kv][p].y, c[kv][p].z, c[kv][p].w};
            float x[16];
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const float2 f = e4m3x2_to_float2(uint16_t(w[k / 2] >> (16 * (k & 1))));
                x[2 * k] = f.x * scale[kv][p], x[2 * k + 1] = f.y * scale[kv][p];
            }
            const int elt = DT == ZC_FP32 ? 4 : 2;
            store16<DT>(static_cast<uint8_t *>(a.x[kv].p) +
                            (int64_t(q.first + t0 + row) * a.x[kv].token + int64_t(h) * a.x[kv].head + (i - row * per_row) * 16) * elt, x);
        }
    }
}

template <int DT> __global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ MoveArgs a) {
    read_tokens<DT>(a);
    if (blockIdx.x == 0 && blockIdx.y == 0) report_batch(a.b, a.c.tokens, a.d_status, threadIdx.x, kThreads, true);
}

} // namespace

int launch_read(int dtype, const MoveArgs &a, cudaStream_t s) {
    const dim3 grid(slot_of(a.b.total, a.b.n_seqs, 1, kTokens, 1), a.c.heads);
    switch (dtype) {
    case ZC_BF16: read_kernel<ZC_BF16><<<grid, kThreads, 0, s>>>(a); break;
    case ZC_FP16: read_kernel<ZC_FP16><<<grid, kThreads, 0, s>>>(a); break;
    default: read_kernel<ZC_FP32><<<grid, kThreads, 0, s>>>(a); break;
    }
    return cudaGetLastError() == cudaSuccess ? ZC_OK : ZC_ECUDA;
}

} // namespace kv
} // namespace zc
