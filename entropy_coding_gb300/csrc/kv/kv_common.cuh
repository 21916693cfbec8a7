// kv_common.cuh — argument blocks and device helpers of the 8-bit key/value
// cache kernels (kv_write.cu, kv_read.cu, kv_rows.cu; the C ABI of the
// operators is in kv_api.cu and include/zc.h).
//
// The cache. For block b, head h, row r (a token of the block) and column d,
// the number is value(code) * scale[b][h], with E4M3 codes in
// [block][head][row][column] order and one float32 scale for each block and
// head, for K and for V apart.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kv_slots.h"
#include "zc.h"  // from include/ (on the -I path)

namespace zc {
namespace kv {

constexpr uint32_t kMaxHeadDim = 128, kMaxBlockTokens = 256;
constexpr float kCodeMax = 448.0f;  // the largest E4M3 value

// Clocks after which a wait is given up: about a second, or a short time under the test hook that makes it run out.
constexpr long long kWaitClocks = 1ll << 31, kWaitClocksTest = 1ll << 20;

// The cache and the batch as the kernels take them.
struct Cache {
    uint8_t *code[2];    // K, V
    float *scale[2];
    int64_t block_stride;  // bytes
    int64_t scale_stride;  // floats
    uint32_t n_blocks, heads, tokens, dim;
    uint32_t sixteenths;   // 2^32 / (tokens / 16), rounded up; 0 for 16 tokens
};

struct Batch {
    const int32_t *table;
    int64_t table_stride;
    const int32_t *cu;
    const int32_t *lens;
    uint32_t n_seqs, total, most, width;
};

// A [token][head][dim] tensor with its own strides (elements).
struct Rows {
    void *p;
    int64_t token, head;
};

struct MoveArgs {  // write and read
    Cache c;
    Batch b;
    Rows x[2];  // K, V
    int32_t *d_status;
};

struct AttendArgs {
    Cache c;
    Batch b;
    Rows q, out;
    float *lse;            // [total][heads] or null
    uint32_t heads, group;
    int dtype;             // of q and out
    float scale_log2;      // softmax scale * log2(e)
    uint32_t causal, window;
    uint32_t rows_most;    // a sequence of no more rows of a head goes to kv_rows.cu
    uint32_t *counters;    // workspace: an item's parts that are done, zero between calls
    uint32_t *group_counters;  // (kv_rows.cu) and those of a group of parts
    void *parts;           // workspace: partial results
    long long limit;       // clocks of a wait
    uint32_t stall;        // test hook: the copies are never asked for
    int32_t *d_status;
};

// The codes as tensor maps, K and V: columns, rows of all heads, blocks; a box
// is `rows` rows of `columns` bytes, swizzled over that width (64 or 128
// bytes). Columns past head_dim are read as zeros.
struct CodeMaps {
    CUtensorMap code[2];
};
int make_maps(const Cache &c, uint32_t columns, uint32_t rows, CodeMaps &m);

int launch_write(int dtype, const MoveArgs &a, cudaStream_t s);
int launch_read(int dtype, const MoveArgs &a, cudaStream_t s);
int sm_count();
// Attention of sequences with at most rows_most rows of a head (kv_rows.cu) and
// of those with more (kv_tiles.cu), and what their workspaces hold.
constexpr uint32_t kRowsMost = 16;
uint64_t rows_counters(const Batch &b, const Cache &c, uint32_t group);
uint64_t rows_group_counters();
uint64_t rows_part_bytes(const Cache &c);
int launch_rows(const AttendArgs &a, cudaStream_t s);
uint64_t tiles_counters(const Batch &b, const Cache &c, uint32_t group);
uint64_t tiles_part_bytes(const Cache &c);
int launch_tiles(const AttendArgs &a, cudaStream_t s);

#ifdef __CUDACC__

__device__ __forceinline__ void report(int32_t *d_status, int bits) { atomicOr(d_status, bits); }

// One sequence of the batch: n new tokens, packed from `first` on, the last
// of its `len` tokens.
struct Seq {
    uint32_t s, first, n;
    int32_t len;
    bool ok;
};

// Reads and checks sequence s; every thread that asks gets the same answer.
// `speak`: what is wrong is reported.
__device__ __forceinline__ Seq read_seq(const Batch &b, uint32_t s, int32_t *d_status, uint32_t block_tokens, bool speak) {
    const int32_t c0 = __ldg(b.cu + s), c1 = __ldg(b.cu + s + 1);
    Seq q;
    q.s = s;
    q.first = uint32_t(c0);
    q.n = uint32_t(c1 - c0);
    q.len = __ldg(b.lens + s);
    q.ok = counts_ok(c0, c1, q.len, b.total, b.most);
    if (!q.ok && speak) report(d_status, ZC_EFORMAT);
    if (q.ok && uint64_t(q.len) > uint64_t(b.width) * block_tokens) {
        if (speak) report(d_status, ZC_ECAPACITY);
        q.ok = false;
    }
    return q;
}

__device__ __forceinline__ uint32_t tokens_before(const Batch &b, uint32_t s) { return clamp_count(__ldg(b.cu + s), b.total); }

// Looks at every sequence of the batch, with threads first, first + step, ... of one CTA of a launch: the slots of a
// batch whose counts fall need not lead to the sequence that is to be reported. `held`: its new tokens have to be
// among the sequence's.
__device__ __forceinline__ void report_batch(const Batch &b, uint32_t block_tokens, int32_t *d_status, uint32_t first, uint32_t step, bool held) {
    for (uint32_t s = first; s < b.n_seqs; s += step) {
        const Seq q = read_seq(b, s, d_status, block_tokens, true);
        if (held && q.ok && uint32_t(q.len) < q.n) report(d_status, ZC_EFORMAT);
    }
}

// The sequence of slot u (the whole CTA calls this); `at`: the slot's index
// within the sequence, or kNoSlot. The CTA counts the f(s) at or below its
// slot: one round of loads for any batch up to the CTA's size, where a binary
// search would take one dependent load for each halving.
__device__ __forceinline__ uint32_t find_seq(const Batch &b, uint32_t u, uint32_t per, uint32_t unit, uint32_t extra, uint32_t &at) {
    uint32_t below = 0;
    for (uint32_t s0 = 0; s0 < b.n_seqs; s0 += blockDim.x) {
        const uint32_t s = s0 + threadIdx.x;
        bool in = false;
        if (s < b.n_seqs) in = slot_of(tokens_before(b, s), s, per, unit, extra) <= u;
        const uint32_t n = __syncthreads_count(in);
        below += n;
        if (n < blockDim.x) break;  // f grows with s
    }
    const uint32_t s = below ? below - 1 : 0;
    at = slot_within(u, slot_of(tokens_before(b, s), s, per, unit, extra), slot_of(tokens_before(b, s + 1), s + 1, per, unit, extra));
    return s;
}

// Block of a position's 16 (i = position / 16 < 2^27): i / (tokens / 16). With M = 2^32 / d + e, e < 1, and d <= 16,
// i M / 2^32 exceeds i / d by less than i / 2^32 < 1 / d: the floor is the same.
__device__ __forceinline__ uint32_t block_of_16(const Cache &c, uint32_t i) {
    return c.sixteenths ? __umulhi(i, c.sixteenths) : i;
}

// Block of the table, or -1 (reported) where the entry names none.
__device__ __forceinline__ int64_t read_block(const Batch &b, const Cache &c, uint32_t s, uint32_t i, int32_t *d_status) {
    const int32_t e = __ldg(b.table + int64_t(s) * b.table_stride + i);
    if (uint32_t(e) < c.n_blocks) return e;
    report(d_status, ZC_EFORMAT);
    return -1;
}

// ---------------------------------------------------------------------------
// Copies by the tensor memory accelerator, and the barriers that they complete.


__device__ __forceinline__ uint32_t smem_of(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void bar_init(uint64_t *bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_of(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_init_done() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
// Orders this thread's accesses to shared memory before later ones by copies.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void bar_expect(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_of(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_of(bar)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{.reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p;}"
                 : "=r"(ok) : "r"(smem_of(bar)), "r"(parity) : "memory");
    return ok;
}
// Waits for the phase of that parity; false after `limit` clocks.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, long long limit) {
    if (bar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!bar_try(bar, parity))
        if (clock64() - t0 > limit) return false;
    return true;
}
__device__ __forceinline__ void copy_box(void *dst, const CUtensorMap *map, int row, int block, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                     smem_of(dst)), "l"(map), "r"(0), "r"(row), "r"(block), "r"(smem_of(bar)) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---------------------------------------------------------------------------
// E4M3

// Two E4M3 codes (low byte first) to two halves; exact, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}
// Four codes to four halves, the low two and the high two.
__device__ __forceinline__ void e4m3x4_to_half2x2(uint32_t v, uint32_t &lo, uint32_t &hi) {
    asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}" : "=r"(lo), "=r"(hi) : "r"(v));
}
// Two floats to two codes, to nearest even, saturating at +-448, NaN stays NaN.
__device__ __forceinline__ uint16_t float2_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t v) {
    const uint32_t h = e4m3x2_to_half2(v);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Two 16-bit elements of type DT to floats, and back (rounded once).
template <int DT> __device__ __forceinline__ float2 unpack2(uint32_t v) {
    if (DT == ZC_FP16) return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <int DT> __device__ __forceinline__ uint32_t pack2(float a, float b) {
    if (DT == ZC_FP16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

#endif  // __CUDACC__

} // namespace kv
} // namespace zc
