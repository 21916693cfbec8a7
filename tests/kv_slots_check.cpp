// The slots of ragged batches, as the kernels that write and read the 8-bit cache find them: with any counts and
// lengths every access is in range, and with counts that rise every token is met once.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "kv_slots.h"

using namespace zc::kv;

#define CHECK(x)                                                                                                      \
    if (!(x)) {                                                                                                       \
        std::printf("line %d: %s (n %u, slot %u, sequence %u)\n", __LINE__, #x, n, u, s);                             \
        std::exit(1);                                                                                                 \
    }

int main() {
    std::mt19937 rng(1);
    auto upto = [&](uint32_t n) { return uint32_t(rng() % n); };
    for (int round = 0; round < 60000; round++) {
        const uint32_t n = 1 + upto(round % 16 == 0 ? 150 : 9), block = 16 * (1 + upto(8)), threads = 64u << upto(3);
        const bool wild = round % 2;
        std::vector<int32_t> cu(n + 1), lens(n);
        uint32_t most = 1;
        for (uint32_t i = 1; i <= n; i++) cu[i] = cu[i - 1] + int32_t(upto(4) ? upto(40) : upto(400));
        const uint32_t total = uint32_t(cu[n]) + (wild ? upto(3) : 0);
        for (uint32_t i = 0; i < n; i++) {
            const uint32_t c = uint32_t(cu[i + 1] - cu[i]);
            most = c > most ? c : most;
            lens[i] = int32_t(c + (upto(2) ? upto(500) : 0));
        }
        if (wild) {
            for (int k = 0; k < 3; k++) cu[upto(n + 1)] = int32_t(upto(4) ? upto(total + 50) : rng());
            if (upto(4) == 0) lens[upto(n)] = int32_t(rng());
            if (upto(4) == 0) most = total;
        }
        if (total == 0) continue;
        for (int read = 0; read < 2; read++) {
            const uint32_t unit = read ? 64 : block, extra = read ? 1 : 2, slots = slot_of(total, n, 1, unit, extra);
            auto f = [&](uint32_t s) { return slot_of(clamp_count(cu[s], total), s, 1, unit, extra); };
            std::vector<int> met(total);
            for (uint32_t u = 0; u < slots; u++) {
                uint32_t below = 0;
                for (uint32_t s0 = 0; s0 < n; s0 += threads) {  // as the CTA counts them
                    uint32_t in = 0;
                    for (uint32_t s = s0; s < n && s < s0 + threads; s++) in += f(s) <= u;
                    below += in;
                    if (in < threads) break;
                }
                const uint32_t s = below ? below - 1 : 0, at = slot_within(u, f(s), f(s + 1));
                if (at == kNoSlot || !counts_ok(cu[s], cu[s + 1], lens[s], total, most)) continue;
                const uint32_t c = uint32_t(cu[s + 1] - cu[s]), len = uint32_t(lens[s]);
                if (c == 0 || len < c) continue;
                uint32_t first, rows;  // of the run
                if (read) {
                    const uint32_t t0 = at * unit;
                    CHECK(at < 1u << 24);
                    rows = c - (c < t0 ? c : t0) < unit ? c - (c < t0 ? c : t0) : unit;
                    first = t0;
                } else {
                    Span r;
                    if (!block_span(len, c, block, at, r)) continue;
                    CHECK(r.lo >= len - c && r.hi <= len && r.lo < r.hi && r.lo / block == r.blk && (r.hi - 1) / block == r.blk);
                    first = r.lo - (len - c), rows = r.hi - r.lo;
                }
                for (uint32_t t = first; t < first + rows; t++) {
                    CHECK(t < c && uint32_t(cu[s]) + t < total);
                    met[uint32_t(cu[s]) + t]++;
                }
            }
            if (!wild)
                for (uint32_t t = 0, u = 0, s = 0; t < total; t++) CHECK(met[t] == 1);
        }
    }
    std::printf("ok\n");
}
