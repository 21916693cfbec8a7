// kv_rotate.cu — queries and keys before they meet the cache: a norm over each
// head's columns and the rotation of pairs of columns by the token's position,
// in one pass.
//
// Row x (a token's head), D columns, weights w, pair (a, b) with f turns a position:
//   y = x w / sqrt(sum x^2 / D + eps)
//   y_a' = y_a cos t - y_b sin t,  y_b' = y_b cos t + y_a sin t,  t = 2 pi f p
// f is a 64-bit fixed-point fraction of a turn: f p modulo 1 is the low 64 bits
// of an integer product, exact whatever the position; its quarter turn is split
// off, and what is left is within an eighth of a turn, where 32 bits are plenty.
//
// A lane has 16 columns of a row, both of each of its 8 pairs, so that the
// rotation needs no other lane and the norm one sum over D / 16 lanes. A CTA has
// kTokens packed tokens with all their heads: their angles' sines and cosines
// are computed once, for 16 columns of every head, while the first rows are on
// their way.
#include "kv4_common.cuh"

namespace zc {
namespace kv {
namespace {

constexpr int kThreads = 256, kTokens = 4;
constexpr int kUnroll = 2;                 // rows of a lane in flight
constexpr int kLanes = kMaxHeadDim / 16;   // of a row, at most

struct Shared {
    int32_t pos[kTokens];
    uint32_t seq[kTokens];
    // for lane c of a row, quarter j of its pairs (or columns): conflict-free as they are read
    float4 turn[kTokens][4][kLanes];  // cos, sin of two pairs
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
    const uint32_t at = uint32_t(__ldg(reinterpret_cast<const unsigned long long *>(a.turns) + pair) * uint64_t(uint32_t(position)) >> 32);
    const uint32_t quarter = (at + 0x20000000u) >> 30;
    float s, c;
    sincospif(float(int32_t(at - (quarter << 30))) * 0x1p-31f, &s, &c);
    if (quarter & 1) {
        const float t = s;
        s = c, c = -t;
    }
    return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

// The whole CTA: positions, sines and cosines, and weights.
template <bool kInterleaved> __device__ __forceinline__ void prepare(const RotateArgs &a, Shared &sm, uint32_t t0, uint32_t n) {
    locate(a.b, 0, t0, n, sm.pos, sm.seq, a.d_status);
    const uint32_t pairs = a.rot / 2;
    for (uint32_t i = threadIdx.x; i < n * pairs; i += kThreads) {
        const uint32_t token = i / pairs, pair = i - token * pairs;
        if (sm.pos[token] < 0) continue;
        uint32_t c = pair / 8, m = pair % 8;
        if (kInterleaved) c = pair % (pairs / 2) / 4, m = pair % 4 + (pair < pairs / 2 ? 0 : 4);
        reinterpret_cast<float2 *>(&sm.turn[token][m / 2][c])[m % 2] = turned(a, pair, sm.pos[token]);
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
__device__ __forceinline__ float row_norm(const float (&x)[16], uint32_t lanes, float inverse_dim, float eps) {
    auto sum_of = [&](float by) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i++) s = fmaf(x[i] * by, x[i] * by, s);
        for (uint32_t d = 1; d < lanes; d *= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        return s;
    };
    const float sum = sum_of(1.0f);
    // Squares out of float's range: again with the larger of the row's largest magnitude and the root of eps brought to
    // about 1. (What is lost of a sum below 1e-25 matters only next to an eps that is as small.)
    const bool out = sum > 1e37f || (sum < 1e-25f && eps < 1e-20f);
    if (!__any_sync(0xFFFFFFFFu, out)) return rsqrtf(fmaf(sum, inverse_dim, eps));
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i++) top = fmaxf(top, fabsf(x[i]));
    for (uint32_t d = 1; d < lanes; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const bool scale = out && top > 0.0f && top < INFINITY;
    const int e = scale ? min(int(__float_as_uint(fmaxf(top, sqrtf(eps))) >> 23) - 127, 120) : 0;
    const float by = __uint_as_float(uint32_t(127 - e) << 23);  // 2^-e
    const float again = sum_of(by);
    return rsqrtf(fmaf(again, inverse_dim, eps * by * by)) * by;
}

template <int DT, bool kInterleaved> __global__ void __launch_bounds__(kThreads) rotate_kernel(const __grid_constant__ RotateArgs a) {
    __shared__ Shared sm;
    constexpr int elt = DT == ZC_FP32 ? 4 : 2;
    const uint32_t t0 = blockIdx.x * kTokens, n = min(uint32_t(kTokens), a.b.total - t0);
    // lanes of a row, up to the next power of two, and the rows of the CTA that are done together
    const uint32_t used = a.dim / 16, lanes = used <= 1 ? 1 : used <= 2 ? 2 : used <= 4 ? 4 : 8;
    const uint32_t c = threadIdx.x & (lanes - 1), together = kThreads / lanes, all = a.heads[0] + a.heads[1];
    const bool mine = c < used, turns = 16 * c < a.rot;
    const uint32_t col0 = first_column(a, c), col1 = second_column(a, c);
    const float inverse_dim = 1.0f / float(a.dim);
    uint32_t token = 0, head = threadIdx.x / lanes;  // of the thread's next row
    for (bool first = true;; first = false) {
        Piece<DT> in[kUnroll][2];
        uint32_t at_token[kUnroll], at_head[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            while (head >= all && token < n) head -= all, token++;
            at_token[u] = token, at_head[u] = head;
            head += together;
            const bool there = mine && at_token[u] < n;
            const int kv = at_head[u] >= a.heads[0];
            if (there) {
                const Rows &r = a.in[kv];
                const uint8_t *x = static_cast<const uint8_t *>(r.p) + (int64_t(t0 + at_token[u]) * r.token + int64_t(at_head[u] - (kv ? a.heads[0] : 0)) * r.head) * elt;
                in[u][0].load(x + col0 * elt);
                in[u][1].load(x + col1 * elt);
            } else {
                in[u][0].clear();
                in[u][1].clear();
            }
        }
        if (first) prepare<kInterleaved>(a, sm, t0, n);
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const bool there = mine && at_token[u] < n;
            const int kv = at_head[u] >= a.heads[0];
            float x[16];
            in[u][0].get(x);
            in[u][1].get(x + 8);
            if (a.weight[0] || a.weight[1]) {
                const float norm = row_norm(x, lanes, inverse_dim, a.eps);
                if (there && a.weight[kv]) {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float4 w = sm.weight[kv][j][c];
                        x[4 * j] *= norm * w.x, x[4 * j + 1] *= norm * w.y, x[4 * j + 2] *= norm * w.z, x[4 * j + 3] *= norm * w.w;
                    }
                }
            }
            if (!there || sm.pos[at_token[u]] < 0) continue;
            if (turns) {
#pragma unroll
                for (int m = 0; m < 8; m++) {
                    const float2 t = reinterpret_cast<const float2 *>(&sm.turn[at_token[u]][m / 2][c])[m % 2];
                    const int i = kInterleaved ? 2 * m : m, j = kInterleaved ? 2 * m + 1 : m + 8;
                    const float p = x[i], q = x[j];
                    x[i] = fmaf(p, t.x, -(q * t.y)), x[j] = fmaf(q, t.x, p * t.y);
                }
            }
            const Rows &r = a.out[kv];
            uint8_t *y = static_cast<uint8_t *>(r.p) + (int64_t(t0 + at_token[u]) * r.token + int64_t(at_head[u] - (kv ? a.heads[0] : 0)) * r.head) * elt;
            Piece<DT> out[2];
            out[0].put(x);
            out[1].put(x + 8);
            out[0].store(y + col0 * elt);
            out[1].store(y + col1 * elt);
        }
        // (a warp goes on as long as one of its rows is there: its sums are over all of it)
        while (head >= all && token < n) head -= all, token++;
        if (!__any_sync(0xFFFFFFFFu, token < n)) break;
    }
    if (blockIdx.x == 0) report_batch(a.b, 0xFFFFFFFFu, a.d_status, threadIdx.x, kThreads, true);
}

template <int DT> void launch(bool interleaved, const RotateArgs &a, cudaStream_t s) {
    const uint32_t grid = (a.b.total + kTokens - 1) / kTokens;
    if (interleaved) rotate_kernel<DT, true><<<grid, kThreads, 0, s>>>(a);
    else rotate_kernel<DT, false><<<grid, kThreads, 0, s>>>(a);
}

} // namespace

int launch_rotate(int dtype, bool interleaved, const RotateArgs &a, cudaStream_t s) {
    switch (dtype) {
    case ZC_BF16: launch<ZC_BF16>(interleaved, a, s); break;
    case ZC_FP16: launch<ZC_FP16>(interleaved, a, s); break;
    default: launch<ZC_FP32>(interleaved, a, s); break;
    }
    return cudaGetLastError() == cudaSuccess ? ZC_OK : ZC_ECUDA;
}

} // namespace kv
} // namespace zc
