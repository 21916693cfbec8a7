// kv4_tiles.cu — attention of many query rows (prompts, chunks of prompts,
// longer drafts) over the 4-bit cache, on the fifth-generation tensor cores.
//
// As in kv_tiles.cu, over tiles of 128 keys:
//   S = Q K^T                 128 x 128 x dim, half operands, float32 in tensor memory
//   w_ij = 2^(S_ij c_i - m_i + 9), rounded to half, back into tensor memory
//   O += W V                  128 x dim x 128
//   l_i += sum_j w_ij before rounding
// with k and v = code * scale: their products are exact in half, so that the
// conversion's warps apply the scales, weights know no unit but that of the
// largest score, and out = O / l. Scores stay products until their exponentials:
// a row's scale goes into those.
//
// Measured on a GB300: an 8192-token prompt (32 query heads, 8 key/value heads of
// 128, causal) in 434 us, 1.27 PFLOP/s, 0.64 of the measured bfloat16 rate; 912
// tokens of two sequences over 28384 keys in 178 (1.19 PFLOP/s); 16 sequences of 2
// to 5 tokens, 8 query heads to a head, over up to 4096 keys in 22. A 4096-token
// prompt of heads of 64 in 121 us, 0.57 PFLOP/s: products are half as long there,
// the rows' work is not, and with this split of registers the kernel of 64 columns
// spills (132 bytes of stores, that of 128 columns 20).
// Of 3480 clocks a key tile the products' warp waits 850; their operations would
// take 2048, but scores' products read both operands from a shared memory that the
// conversion and the copies use too. A row tile's chain is 350 clocks for the
// maximum, 500 and 520 for the halves' weights, and its products. Exponentials beside the search for
// the maximum, done again where it has grown, leave the products waiting for
// longer (518 us for a whole tile, 484 for its first half, 443 with the maximum
// first); fewer registers for the rows and more for the conversion 443 to 437.
#include "kv_tiles.cuh"

namespace zc {
namespace kv {

int launch_tiles4(const AttendArgs &a, cudaStream_t s) { return a.c.dim <= 64 ? launch<4, 64>(a, s) : launch<4, 128>(a, s); }

} // namespace kv
} // namespace zc
