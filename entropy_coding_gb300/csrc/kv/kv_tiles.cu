// kv_tiles.cu — attention of many query rows (prompts, chunks of prompts,
// longer drafts) over the 8-bit cache, on the fifth-generation tensor cores.
//
// An item is up to 256 rows of one sequence and key/value head, in two tiles
// of 128 (a row is one query token and query head, as in kv_rows.cu). Over
// tiles of 128 keys, with codes kc, vc and block scales ks, vs:
//   S = Q Kc^T            128 x 128 x dim, half operands, float32 in tensor memory
//   s_ij = S_ij ks_b c_i  (c_i: the row's power of two and the softmax scale, log2)
//   w_ij = 2^(s_ij - m_i + log2 vs_b - d_i + 9), rounded to half, back into tensor memory
//   O += W Vc             128 x dim x 128
//   l_i += sum_b (sum_{j in b} w_ij before rounding) 2^(d_i - 9 - log2 vs_b)
// m_i and m_i + d_i follow the row's maxima of s and of s + log2 vs (and may lag by
// 2^8 and 2^6), so O is in units of the largest contribution and l in units of
// the largest weight: block scales cost an exponent's bias for 16 columns, and no
// spread between them loses precision; half keeps its 11 bits down to 2^-23 of
// the largest w vs. A block whose scale is 2^69 below the unit adds less than
// 2^-60 of it and counts as 2^-69. out = O 2^(d - 9) / l.
//
// The work and the roles of a CTA's warps are in kv_tiles.cuh.
//
// Measured on a GB300: an 8192-token prompt (32 query heads, 8 key/value heads
// of 128, causal) in 462 to 464 us, 1.19 PFLOP/s, 0.60 of the measured bfloat16 rate;
// 912 tokens of two sequences over 28384 keys in 191 us (1.11 PFLOP/s). (454 and 186
// without the code for large scores, which these calls do not come to: the schedulers
// wait for instructions as it is, and a row's loop grows by it.) The
// tensor cores are busy half of the time. A key tile takes 1.7 us where its
// products take 1.05: a row tile's chain of scores, weights (about 1.1 us: two
// passes over the scores, 128 exponentials a thread on a unit shared by two
// warps, and the conversions' instructions beside them) and its own products is
// longer than the other tile's products cover. The weights stand where the
// scores were, so that the next scores wait for these sums: with 128 columns of
// output, columns for both do not fit; with 64 they would (2 x 128 of scores, 2 x
// 64 of weights, 2 x 64 of sums), which this layout does not use. An item of one
// row tile leaves half of the row threads without work. Shared memory is the next limit: by its rate the products take 1536
// clocks of it a key tile, the conversion 768, the copies 256. An item's
// beginning and end take about 7 us (queries 1.6, output 3, the first scores and
// the last sums with nothing beside them), joining a cut item 10: 32 columns and
// 2 parts at a time, read whether they are there or not (16 columns, 4 parts and
// predicated reads: 25 us).
#include "kv_tiles.cuh"

namespace zc {
namespace kv {

uint64_t tiles_counters(const Batch &b, const Cache &c, uint32_t group) {
    return uint64_t(slot_of(b.total, b.n_seqs, group, kRows, 1)) * c.heads;
}

uint64_t tiles_part_bytes(const Cache &c) {
    return uint64_t(sm_count()) * 2 * (c.dim <= 64 ? sizeof(Part<64>) : sizeof(Part<128>));
}

int launch_tiles(const AttendArgs &a, cudaStream_t s) { return a.c.dim <= 64 ? launch<8, 64>(a, s) : launch<8, 128>(a, s); }

} // namespace kv
} // namespace zc
