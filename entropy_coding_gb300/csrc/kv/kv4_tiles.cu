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
// largest score, and out = O / l.
#include "kv_tiles.cuh"

namespace zc {
namespace kv {

int launch_tiles4(const AttendArgs &a, cudaStream_t s) { return a.c.dim <= 64 ? launch<4, 64>(a, s) : launch<4, 128>(a, s); }

} // namespace kv
} // namespace zc
