// kv_rotate.cu — queries and keys before they meet the cache: a norm over each
// head's columns and the rotation of pairs of columns by the token's position,
// in one pass.
//
// Row x (a token's head), D columns, weights w, pair (a, b) with f turns a position:
//   y = x w / sqrt(sum x^2 / D + eps)
//   y_a' = y_a cos t - y_b sin t,  y_b' = y_b cos t + y_a sin t,  t = 2 pi f p
// f is a 64-bit fixed-point fraction of a turn: f p modulo 1 is the low 64 bits
// of an integer product, exact whatever the position; its quarter turn is split
// off, and what is left, within an eighth of a turn, is rounded once to float:
// a sine is right relative to itself, of a slow pair near the beginning too.
//
// A lane has 16 columns of a row, both of each of its 8 pairs, so that the
// rotation needs no other lane and the norm one sum over D / 16 lanes. A CTA has
// a few packed tokens with all their heads, a warp rows of one of them: the
// angles' sines and cosines are computed once, while the first rows are on
// their way, and stay in registers. Arithmetic is on two floats at a time.
//
// Measured on a GB300: 16978 tokens of 32 and 8 heads of 128, bfloat16, 348 MB
// read and written, in 62 us: 5.6 TB/s, 0.82 of the copy rate (neighbouring columns 63;
// float32, 695 MB, in 112: 0.92); 32 tokens in 3.5.
// Schedulers issue in 0.74 of the clocks, the arithmetic units are busy in 0.56:
// both the bytes and the instructions are near. Four CTAs an SM (64 registers) beat
// three (66 us); sines and cosines in registers and no addresses but sums beat
// neither (63.5, registers spilled).
#include "kv4_common.cuh"

namespace zc {
namespace kv {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kLanes = kMaxHeadDim / 16;   // of a row, at most

template <int kTokens> struct Shared {
    int2 at[kTokens];  // position, sequence
    // for lane c of a row, quarter j of its pairs (or columns): conflict-free as they are read
    float4 turn[kTokens][4][kLanes];  // cosines of two pairs, and sines
    float4 weight[2][4][kLanes];      // of q and k
};

// Where a lane's two runs of 8 columns begin: the halves of its pairs, or, behind the columns that turn, 16 in a row.
__device__ __forceinline__ uint32_t first_column(const RotateArgs &a, uint32_t c) { return 16 * c < a.rot ? 8 * c : 16 * c; }
__device__ __forceinline__ uint32_t second_column(const RotateArgs &a, uint32_t c) { return 16 * c < a.rot ? a.rot / 2 + 8 * c : 16 * c + 8; }

__device__ __forceinline__ float weight_at(const RotateArgs &a, int kv, uint32_t i) {
    switch (a.weight_dtype) {
    case ZC_FP32: return __ldg(static_cast<const float *>(a.weight[kv]) + i);
    case ZC_BF16: return __bfloat162float(static_cast<const __nv_bfloat16 *>(a.weight[kv])[i]);
    default: return __half2float(static_cast<const __half *>(a.weight[kv])[i]);
    }
}

// cos and sin of `position` times the pair's turns.
__device__ __forceinline__ float2 turned(const RotateArgs &a, uint32_t pair, int32_t position) {
    const uint64_t at = __ldg(reinterpret_cast<const unsigned long long *>(a.turns) + pair) * uint64_t(uint32_t(position));
    const uint32_t quarter = uint32_t((at + (uint64_t(1) << 61)) >> 62);
    float s, c;
    sincospif(__ll2float_rn(static_cast<long long>(at - (uint64_t(quarter) << 62))) * 0x1p-63f, &s, &c);
    if (quarter & 1) {
        const float t = s;
        s = c, c = -t;
    }
    return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

// The whole CTA: positions, sines and cosines, and weights.
template <bool kInterleaved, int kTokens> __device__ __forceinline__ void prepare(const RotateArgs &a, Shared<kTokens> &sm, uint32_t t0, uint32_t n) {
    locate(a.b, 0, t0, n, sm.at, a.d_status);
    const uint32_t pairs = a.rot / 2;
    for (uint32_t i = threadIdx.x; i < n * pairs; i += kThreads) {
        const uint32_t token = i / pairs, pair = i - token * pairs;
        if (sm.at[token].x < 0) continue;
        uint32_t c = pair / 8, m = pair % 8;
        if (kInterleaved) c = pair % (pairs / 2) / 4, m = pair % 4 + (pair < pairs / 2 ? 0 : 4);
        const float2 t = turned(a, pair, sm.at[token].x);
        float *to = reinterpret_cast<float *>(&sm.turn[token][m / 2][c]) + m % 2;
        to[0] = t.x, to[2] = t.y;
    }
    for (uint32_t i = threadIdx.x; i < 2 * a.dim; i += kThreads) {
        const int kv = i >= a.dim;
        const uint32_t k = i - kv * a.dim, c = k / 16, m = k % 16;
        if (a.weight[kv])
            reinterpret_cast<float *>(&sm.weight[kv][m / 4][c])[m % 4] = weight_at(a, kv, m < 8 ? first_column(a, c) + m : second_column(a, c) + m - 8);
    }
    __syncthreads();
}

// 1 / sqrt(sum x^2 / D + eps) of a row whose lanes are `lanes` neighbours; the whole warp calls it.
__device__ __forceinline__ float row_norm(const float2 (&x)[8], uint32_t lanes, float inverse_dim, float eps) {
    auto sum_of = [&](float by) {
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 y = by == 1.0f ? x[i] : mul2(x[i], both(by));
            s = fma2(y, y, s);
        }
        float t = s.x + s.y;
        for (uint32_t d = 1; d < lanes; d *= 2) t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
        return t;
    };
    const float sum = sum_of(1.0f);
    // Squares out of float's range: again with the larger of the row's largest magnitude and the root of eps brought to
    // about 1. (What is lost of a sum below 1e-25 matters only next to an eps that is as small.)
    const bool out = sum > 1e37f || (sum < 1e-25f && eps < 1e-20f);
    if (!__any_sync(0xFFFFFFFFu, out)) return rsqrtf(fmaf(sum, inverse_dim, eps));
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) top = fmaxf(top, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
    for (uint32_t d = 1; d < lanes; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const bool scale = out && top > 0.0f && top < INFINITY;
    const int e = scale ? min(int(__float_as_uint(fmaxf(top, sqrtf(eps))) >> 23) - 127, 120) : 0;
    const float by = __uint_as_float(uint32_t(127 - e) << 23);  // 2^-e
    const float again = sum_of(by);
    return rsqrtf(fmaf(again, inverse_dim, eps * by * by)) * by;
}

template <int DT, bool kInterleaved, int kTokens> __global__ void __launch_bounds__(kThreads, 4) rotate_kernel(const __grid_constant__ RotateArgs a) {
    __shared__ Shared<kTokens> sm;
    constexpr int elt = DT == ZC_FP32 ? 4 : 2, kShare = kWarps / kTokens;  // warps of a token
    const uint32_t t0 = blockIdx.x * kTokens, n = min(uint32_t(kTokens), a.b.total - t0);
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, token = warp / kShare;
    // lanes of a row, up to the next power of two, and rows that a warp does together
    const uint32_t used = a.dim / 16, lanes = used <= 1 ? 1 : used <= 2 ? 2 : used <= 4 ? 4 : 8, together = 32 / lanes;
    const uint32_t c = lane & (lanes - 1), all = a.heads[0] + a.heads[1];
    const bool mine = c < used && token < n, turns = 16 * c < a.rot;
    const uint32_t col0 = first_column(a, c), col1 = second_column(a, c);
    // a row's address in q or k, of the inputs or outputs
    auto at = [&](const Rows (&x)[2], uint32_t row) {
        const int kv = row >= a.heads[0];
        return static_cast<uint8_t *>(x[kv].p) + (int64_t(t0 + token) * x[kv].token + int64_t(row - (kv ? a.heads[0] : 0)) * x[kv].head) * elt;
    };
    const uint32_t r0 = warp % kShare * together;
    uint32_t row = r0 + lane / lanes;
    Piece<DT> next[2];
    auto ask = [&]() {
        if (mine && row < all) {
            const uint8_t *x = at(a.in, row);
            next[0].load(x + col0 * elt);
            next[1].load(x + col1 * elt);
        } else {
            next[0].clear();
            next[1].clear();
        }
    };
    after_the_last();
    ask();
    prepare<kInterleaved>(a, sm, t0, n);
    const bool held = token < n && sm.at[token < n ? token : 0].x >= 0;  // (the token belongs to a sequence)
    float2 cosine[4], sine[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float4 t = sm.turn[token][j][c];
        cosine[j] = make_float2(t.x, t.y), sine[j] = make_float2(t.z, t.w);
    }
    const float inverse_dim = 1.0f / float(a.dim);
    const bool norms = a.weight[0] || a.weight[1];
    // (the whole warp goes on as long as one of its rows is there: its sums are over all of it)
    for (uint32_t r = r0; held && r < all; r += kShare * together) {
        const uint32_t now = row;
        const int kv = now >= a.heads[0];
        float2 x[8];
        next[0].get(x);
        next[1].get(x + 4);
        row += kShare * together;
        ask();
        if (norms) {
            const float norm = row_norm(x, lanes, inverse_dim, a.eps);
            if (a.weight[kv]) {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float4 w = sm.weight[kv][j][c];
                    x[2 * j] = mul2(x[2 * j], mul2(make_float2(w.x, w.y), both(norm)));
                    x[2 * j + 1] = mul2(x[2 * j + 1], mul2(make_float2(w.z, w.w), both(norm)));
                }
            }
        }
        if (!mine || now >= all) continue;
        if (turns) {
            if (kInterleaved) {
#pragma unroll
                for (int m = 0; m < 8; m++) {
                    const float cs = m % 2 ? cosine[m / 2].y : cosine[m / 2].x, sn = m % 2 ? sine[m / 2].y : sine[m / 2].x;
                    x[m] = make_float2(fmaf(x[m].x, cs, -(x[m].y * sn)), fmaf(x[m].y, cs, x[m].x * sn));
                }
            } else {
#pragma unroll
                for (int m = 0; m < 4; m++) {
                    const float2 p = x[m], q = x[m + 4], minus = make_float2(-sine[m].x, -sine[m].y);
                    x[m] = fma2(p, cosine[m], mul2(q, minus)), x[m + 4] = fma2(q, cosine[m], mul2(p, sine[m]));
                }
            }
        }
        uint8_t *y = at(a.out, now);
        Piece<DT> out[2];
        out[0].put(x);
        out[1].put(x + 4);
        out[0].store(y + col0 * elt);
        out[1].store(y + col1 * elt);
    }
    if (blockIdx.x == 0) report_batch(a.b, 0xFFFFFFFFu, a.d_status, threadIdx.x, kThreads, true);
}

// Tokens of a CTA: one, which then has all of its warps, while that makes no more than 2 CTAs an SM; 4, and 8 of many. (32
// tokens of 40 heads of 128: 1 token 6.2 us, 4 tokens 8.2; 608 tokens: 4 tokens 9.5, 8 tokens 12.3; 2432 single tokens 16.4 and
// 18.3, 3648 26.1 and 22.1; 16978 tokens of prompts 65.5 and 63.6.)
template <int DT, bool kInterleaved> int launch(const RotateArgs &a, cudaStream_t s) {
    const uint32_t sms = uint32_t(sm_count());
    if (a.b.total <= 2 * sms) return launch_early(rotate_kernel<DT, kInterleaved, 1>, dim3(a.b.total), kThreads, 0, s, a);
    if (a.b.total <= 16 * sms) return launch_early(rotate_kernel<DT, kInterleaved, 4>, dim3((a.b.total + 3) / 4), kThreads, 0, s, a);
    return launch_early(rotate_kernel<DT, kInterleaved, 8>, dim3((a.b.total + 7) / 8), kThreads, 0, s, a);
}

template <int DT> int launch(bool interleaved, const RotateArgs &a, cudaStream_t s) { return interleaved ? launch<DT, true>(a, s) : launch<DT, false>(a, s); }

} // namespace

int launch_rotate(int dtype, bool interleaved, const RotateArgs &a, cudaStream_t s) {
    return dtype == ZC_BF16 ? launch<ZC_BF16>(interleaved, a, s) : dtype == ZC_FP16 ? launch<ZC_FP16>(interleaved, a, s) : launch<ZC_FP32>(interleaved, a, s);
}

} // namespace kv
} // namespace zc
