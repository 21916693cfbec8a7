// kv_api.cu — the C ABI of the 8-bit key/value cache operators: argument
// checks and launches. As in zc_api.cu, no entry point allocates or
// synchronises; what only the device can see is reported through *d_status.
#include <atomic>
#include <cmath>

#include "kv_common.cuh"

namespace zc {
namespace kv {

// Streaming multiprocessors of the current device (asked for once).
int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return 1;
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

int make_maps(const Cache &c, uint32_t columns, uint32_t rows, CodeMaps &m) {
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<Encode> known{nullptr};
    Encode encode = known.load(std::memory_order_relaxed);
    if (!encode) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess || !f)
            return ZC_ECUDA;
        encode = reinterpret_cast<Encode>(f);
        known.store(encode, std::memory_order_relaxed);
    }
    const cuuint64_t size[3] = {c.dim, cuuint64_t(c.heads) * c.tokens, c.n_blocks};
    const cuuint64_t stride[2] = {c.dim, cuuint64_t(c.block_stride)};
    const cuuint32_t box[3] = {columns, rows, 1}, step[3] = {1, 1, 1};
    for (int i = 0; i < 2; i++)
        if (encode(&m.code[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c.code[i], size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   columns == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return ZC_EINVAL;
    return ZC_OK;
}

} // namespace kv
} // namespace zc

namespace {

using namespace zc::kv;

std::atomic<uint32_t> g_hooks{0};

uint64_t pad256(uint64_t x) { return (x + 255) & ~uint64_t(255); }

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int elt_bytes(int dtype) {
    switch (dtype) {
    case ZC_BF16: case ZC_FP16: return 2;
    case ZC_FP32: return 4;
    default: return 0;
    }
}

int make_cache(const zc_kv_cache *c, Cache &o) {
    if (!c || !c->d_k || !c->d_v || !c->d_k_scale || !c->d_v_scale) return ZC_EINVAL;
    if (c->head_dim == 0 || c->head_dim % 16 || c->head_dim > kMaxHeadDim) return ZC_EINVAL;
    if (c->block_tokens == 0 || c->block_tokens % 16 || c->block_tokens > kMaxBlockTokens) return ZC_EINVAL;
    if (c->kv_heads == 0 || c->kv_heads > 65535 || c->n_blocks == 0 || c->n_blocks > 0x7FFFFFFFu) return ZC_EINVAL;
    const int64_t need = int64_t(c->kv_heads) * c->block_tokens * c->head_dim;
    if (c->block_stride < need || c->block_stride % 16 || c->scale_stride < int64_t(c->kv_heads)) return ZC_EINVAL;
    if (c->block_stride >= int64_t(1) << 40) return ZC_EINVAL;  // of a tensor map
    if (c->block_stride > INT64_MAX / int64_t(c->n_blocks) || c->scale_stride > INT64_MAX / 4 / int64_t(c->n_blocks)) return ZC_EINVAL;
    if (!aligned(c->d_k, 16) || !aligned(c->d_v, 16) || !aligned(c->d_k_scale, 4) || !aligned(c->d_v_scale, 4)) return ZC_EINVAL;
    o.code[0] = static_cast<uint8_t *>(c->d_k);
    o.code[1] = static_cast<uint8_t *>(c->d_v);
    o.scale[0] = c->d_k_scale;
    o.scale[1] = c->d_v_scale;
    o.block_stride = c->block_stride;
    o.scale_stride = c->scale_stride;
    o.n_blocks = c->n_blocks;
    o.heads = c->kv_heads;
    o.tokens = c->block_tokens;
    o.dim = c->head_dim;
    const uint64_t d = o.tokens / 16;
    o.sixteenths = d == 1 ? 0 : uint32_t(((uint64_t(1) << 32) + d - 1) / d);
    return ZC_OK;
}

int make_batch(const zc_kv_batch *b, Batch &o) {
    if (!b) return ZC_EINVAL;
    if (b->n_seqs > 0x00FFFFFFu || b->total_tokens > 0x7FFFFFFFu || b->table_width > 0x7FFFFFFFu) return ZC_EINVAL;
    if (b->max_tokens > b->total_tokens || (b->total_tokens && (b->max_tokens == 0 || b->n_seqs == 0))) return ZC_EINVAL;
    if (uint64_t(b->max_tokens) * b->n_seqs < b->total_tokens) return ZC_EINVAL;
    if (b->n_seqs && (!b->d_table || !b->d_cu || !b->d_lens)) return ZC_EINVAL;
    if (b->n_seqs && (b->table_width == 0 || b->table_stride < int64_t(b->table_width))) return ZC_EINVAL;
    if (!aligned(b->d_table, 4) || !aligned(b->d_cu, 4) || !aligned(b->d_lens, 4)) return ZC_EINVAL;
    o.table = b->d_table;
    o.table_stride = b->table_stride;
    o.cu = b->d_cu;
    o.lens = b->d_lens;
    o.n_seqs = b->n_seqs;
    o.total = b->total_tokens;
    o.most = b->max_tokens;
    o.width = b->table_width;
    return ZC_OK;
}

// Rows of `heads` heads are read and written 16 bytes at a time.
int make_rows(const zc_kv_rows &r, int elt, Rows &o) {
    if (!r.d_data || !aligned(r.d_data, 16)) return ZC_EINVAL;
    if (r.token_stride % (16 / elt) || r.head_stride % (16 / elt)) return ZC_EINVAL;
    o.p = r.d_data;
    o.token = r.token_stride;
    o.head = r.head_stride;
    return ZC_OK;
}

int move(bool write, const zc_kv_cache *cache, const zc_kv_batch *batch, int dtype, const zc_kv_rows *k,
         const zc_kv_rows *v, int32_t *d_status, void *stream) {
    MoveArgs a{};
    const int elt = elt_bytes(dtype);
    if (!elt || !k || !v || !d_status || !aligned(d_status, 4)) return ZC_EINVAL;
    int st = make_cache(cache, a.c);
    if (st == ZC_OK) st = make_batch(batch, a.b);
    if (st != ZC_OK) return st;
    if (a.b.total == 0) return ZC_OK;
    if ((st = make_rows(*k, elt, a.x[0])) != ZC_OK || (st = make_rows(*v, elt, a.x[1])) != ZC_OK) return st;
    a.d_status = d_status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return write ? launch_write(dtype, a, s) : launch_read(dtype, a, s);
}

} // namespace

extern "C" void zc_kv_set_test_hooks(uint32_t hooks) { g_hooks.store(hooks & ZC_HOOK_KV_COPY_STALL, std::memory_order_relaxed); }

extern "C" int zc_kv_write(const zc_kv_cache *cache, const zc_kv_batch *batch, int dtype, const zc_kv_rows *k,
                           const zc_kv_rows *v, int32_t *d_status, void *stream) {
    return move(true, cache, batch, dtype, k, v, d_status, stream);
}

extern "C" int zc_kv_read(const zc_kv_cache *cache, const zc_kv_batch *batch, int dtype, const zc_kv_rows *k,
                          const zc_kv_rows *v, int32_t *d_status, void *stream) {
    return move(false, cache, batch, dtype, k, v, d_status, stream);
}

namespace {

// Which kernels a batch needs. A sequence's rows of a head are its new tokens times the group. Up to 16 of them the
// cache's bytes are what counts, and the kernel that streams them does the work; more rows fill the tensor cores'
// 128-row tiles. (16 sequences of up to 8000 keys: 16 rows 66 us there and 78 us on tiles; 20 or 32 rows, two passes
// over the bytes, 94 and 95 us there and 78 us on tiles.)
// A batch of prompts (more than a tile's rows) among single tokens runs both, each on its own sequences: a prompt of 400
// tokens among 47 single ones takes 134 us so and 185 us on tiles alone. The host does not know how many sequences are of
// which kind: where they have a tile's rows on average, or are no more than 8, the few single tokens are not worth a
// second launch (24 sequences, two of them single tokens: 63 us with both, 54 us on tiles), nor are drafts of uneven
// length (16 sequences of 2 to 5 tokens: 29 and 25 us). The average is moved by one long prompt: with 4 heads to a head
// 47 single tokens among a chunk of 2048 go to the tiles alone. Of a batch that runs both only sequences of up to 8 rows
// are streamed, where a single token has no more: room for 16 rows costs the streaming 1.35 times the time.
struct Plan {
    bool rows, tiles;
    uint32_t rows_most;
    uint64_t rows_counters, tiles_counters, part_bytes;
    Plan(const Batch &b, const Cache &c, uint32_t group) {
        tiles = uint64_t(b.most) * group > kRowsMost;
        rows = !tiles || (b.n_seqs > 8 && group <= kRowsMost && uint64_t(b.most) * group > 128 && uint64_t(b.total) * group < 128ull * b.n_seqs);
        rows_most = !rows ? 0 : tiles && group <= 8 ? 8 : kRowsMost;
        rows_counters = rows ? pad256(4 * zc::kv::rows_counters(b, c, group)) + pad256(4 * rows_group_counters()) : 0;
        tiles_counters = tiles ? pad256(4 * zc::kv::tiles_counters(b, c, group)) : 0;
        const uint64_t r = rows ? rows_part_bytes(c) : 0, t = tiles ? tiles_part_bytes(c) : 0;
        part_bytes = r > t ? r : t;
    }
    uint64_t counters() const { return rows_counters + tiles_counters; }
    uint64_t bytes() const { return counters() + part_bytes; }
};

// counters() or bytes() of a call's plan, 0 for invalid arguments
uint64_t planned(const zc_kv_cache *cache, const zc_kv_batch *batch, uint32_t heads, uint64_t (Plan::*bytes)() const) {
    Cache c{};
    Batch b{};
    if (make_cache(cache, c) != ZC_OK || make_batch(batch, b) != ZC_OK) return 0;
    if (heads == 0 || heads % c.heads || heads > 65535 || uint64_t(b.total) * heads > 0x7FFFFFFFu) return 0;
    return (Plan(b, c, heads / c.heads).*bytes)();
}

} // namespace

extern "C" uint64_t zc_kv_attend_workspace_size(const zc_kv_cache *cache, const zc_kv_batch *batch, uint32_t heads) {
    return planned(cache, batch, heads, &Plan::bytes);
}

extern "C" uint64_t zc_kv_attend_counter_bytes(const zc_kv_cache *cache, const zc_kv_batch *batch, uint32_t heads) {
    return planned(cache, batch, heads, &Plan::counters);
}

extern "C" int zc_kv_attend(const zc_kv_cache *cache, const zc_kv_batch *batch, int dtype, uint32_t heads,
                            const zc_kv_rows *q, const zc_kv_rows *out, float *d_lse, double scale, uint32_t flags,
                            uint32_t window, void *d_ws, uint64_t ws_bytes, int32_t *d_status, void *stream) {
    AttendArgs a{};
    if ((dtype != ZC_BF16 && dtype != ZC_FP16) || !q || !out || !d_status || !aligned(d_status, 4)) return ZC_EINVAL;
    if ((flags & ~ZC_KV_CAUSAL) || !std::isfinite(scale) || std::fabs(scale) > 1e18 || !aligned(d_lse, 4)) return ZC_EINVAL;
    int st = make_cache(cache, a.c);
    if (st == ZC_OK) st = make_batch(batch, a.b);
    if (st != ZC_OK) return st;
    if (heads == 0 || heads % a.c.heads || heads > 65535 || uint64_t(a.b.total) * heads > 0x7FFFFFFFu) return ZC_EINVAL;
    if (a.b.total == 0) return ZC_OK;
    if ((st = make_rows(*q, 2, a.q)) != ZC_OK || (st = make_rows(*out, 2, a.out)) != ZC_OK) return st;
    a.lse = d_lse;
    a.heads = heads;
    a.dtype = dtype;
    a.group = heads / a.c.heads;
    const Plan plan(a.b, a.c, a.group);
    if (!d_ws || !aligned(d_ws, 16)) return ZC_EINVAL;
    if (ws_bytes < plan.bytes()) return ZC_ECAPACITY;
    uint8_t *ws = static_cast<uint8_t *>(d_ws);
    a.parts = ws + plan.counters();
    a.rows_most = plan.rows_most;
    a.scale_log2 = float(scale * 1.4426950408889634);
    a.causal = flags & ZC_KV_CAUSAL;
    a.window = window < 1u << 30 ? window : 0;  // (lengths are below that: nothing is outside)
    a.d_status = d_status;
    a.stall = g_hooks.load(std::memory_order_relaxed) & ZC_HOOK_KV_COPY_STALL;
    a.limit = a.stall ? kWaitClocksTest : kWaitClocks;
    cudaStream_t str = static_cast<cudaStream_t>(stream);
    if (plan.tiles) {
        a.counters = reinterpret_cast<uint32_t *>(ws + plan.rows_counters);
        if ((st = launch_tiles(a, str)) != ZC_OK) return st;
    }
    if (plan.rows) {
        a.group_counters = reinterpret_cast<uint32_t *>(ws);
        a.counters = reinterpret_cast<uint32_t *>(ws + pad256(4 * rows_group_counters()));
        st = launch_rows(a, str);
    }
    return st;
}
