// kv_slots.h — index arithmetic of a ragged batch, without a host copy of its
// counts: which sequence a slot of work belongs to, and which positions of it.
// Plain C++, for the kernels and for the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define ZC_KV_HD __host__ __device__ __forceinline__
#else
#define ZC_KV_HD inline
#endif

namespace zc {
namespace kv {

// Sequence s takes the slots from f(s) = floor(cu[s] * per / unit) + extra * s
// on; f(s + 1) - f(s) >= ceil(n * per / unit) + extra - 1, so extra = 1 gives
// every run of n tokens its ceil(n * per / unit) tiles, and extra = 2 the
// blocks of a run that may start inside one. A launch covers f(n_seqs) slots.
// (tokens * per < 2^31 and sequences < 2^24: the entry points see to it)
ZC_KV_HD uint32_t slot_of(uint32_t tokens, uint32_t s, uint32_t per, uint32_t unit, uint32_t extra) {
    return tokens * per / unit + extra * s;
}

// A count as the slots take it, whatever the device's memory holds.
ZC_KV_HD uint32_t clamp_count(int32_t c, uint32_t total) { return c < 0 ? 0 : uint32_t(c) < total ? uint32_t(c) : total; }

// Whether tokens [c0, c1) and a length can be those of a sequence.
ZC_KV_HD bool counts_ok(int32_t c0, int32_t c1, int32_t len, uint32_t total, uint32_t most) {
    return c0 >= 0 && c1 >= c0 && uint32_t(c1) <= total && uint32_t(c1 - c0) <= most && len >= 0 && len < (1 << 30);
}

// Index of slot u among the slots [f0, f1) of a sequence; kNoSlot where it is none of them: before the first
// sequence's, or, where the counts fall, found by f's that do not rise.
constexpr uint32_t kNoSlot = 0xFFFFFFFFu;
ZC_KV_HD uint32_t slot_within(uint32_t u, uint32_t f0, uint32_t f1) { return u >= f0 && u < f1 ? u - f0 : kNoSlot; }

// Of the last n of len tokens, those in the at-th block that they touch: positions [lo, hi) of block blk. False
// if they touch no more than `at` blocks. (n <= len < 2^30, at < 2^31 / block)
struct Span {
    uint32_t blk, lo, hi;
};
ZC_KV_HD bool block_span(uint32_t len, uint32_t n, uint32_t block, uint32_t at, Span &r) {
    const uint32_t start = len - n;
    r.blk = start / block + at;
    if (uint64_t(r.blk) * block >= len) return false;
    r.lo = start > r.blk * block ? start : r.blk * block;
    r.hi = len < (r.blk + 1) * block ? len : (r.blk + 1) * block;
    return true;
}

} // namespace kv
} // namespace zc
