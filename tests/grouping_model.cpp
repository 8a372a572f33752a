// The grouping of tokens by row on the CPU, behind the embedding runtime in place of the GPU's launches:
// the passes, digits, waves and places that the kernel has (where its waves look is group_part for both),
// one wave after the other.  What the sums would be given is kept for the test.
#include <vector>

#include "embedding_internal.h"

namespace adam_mi355x {

static std::vector<uint32_t> keys, order;

static void group_bucket(const GroupArgs &a, uint32_t bucket) {
    const uint32_t bins = 1u << a.bits, bucket0 = bucket << a.bucket_bits;
    const uint32_t limit = bucket0 < a.rows ? bucket0 : a.rows;
    const uint32_t width = a.rows - limit < (1u << a.bucket_bits) ? a.rows - limit : 1u << a.bucket_bits;
    uint32_t base = 0, len = a.tokens_n;
    for (uint32_t pass = 0; pass < a.passes; ++pass) {
        const uint32_t to = (a.passes - 1 - pass) & 1u;
        const bool first = pass == 0;
        auto key_at = [&](uint32_t i) -> uint64_t {
            if (!first) return a.keys[to ^ 1u][base + i];
            return a.wide ? static_cast<const uint64_t *>(a.tokens)[i] : static_cast<const uint32_t *>(a.tokens)[i];
        };
        auto digit_of = [&](uint32_t key) { return (key >> (pass * kDigitBits)) & (bins - 1); };
        struct One {
            uint32_t row, position;
        };
        std::vector<One> lists[kGroupWaves];
        uint32_t below = 0;
        for (uint32_t wave = 0; wave < kGroupWaves; ++wave) {
            const GroupPart part = group_part(first, wave, len);
            for (uint32_t p0 = part.first; p0 < part.end; p0 += part.look)
                for (uint32_t j = 0; j < kHeld; ++j)
                    for (uint32_t lane = 0; lane < 64; ++lane) {
                        const uint64_t i = p0 + (uint64_t)j * group_step(first) + lane;
                        if (i >= part.end) continue;
                        const uint64_t key = key_at((uint32_t)i);
                        if (key < limit) ++below;
                        if (key < bucket0 || key - bucket0 >= width) continue;
                        lists[wave].push_back({(uint32_t)key, (uint32_t)i});
                    }
        }
        if (first) {
            base = below;
            len = 0;
            for (const auto &list : lists) len += (uint32_t)list.size();
        }
        uint32_t place = base;
        std::vector<uint32_t> places[kGroupWaves];
        for (auto &p : places) p.assign(bins, 0);
        for (uint32_t wave = 0; wave < kGroupWaves; ++wave)
            for (const One &one : lists[wave]) ++places[wave][digit_of(one.row)];
        for (uint32_t digit = 0; digit < bins; ++digit)
            for (uint32_t wave = 0; wave < kGroupWaves; ++wave) {
                const uint32_t count = places[wave][digit];
                places[wave][digit] = place;
                place += count;
            }
        for (uint32_t wave = 0; wave < kGroupWaves; ++wave)
            for (const One &one : lists[wave]) {
                const uint32_t at = places[wave][digit_of(one.row)]++;
                a.keys[to][at] = one.row;
                a.order[to][at] = first ? one.position : a.order[to ^ 1u][base + one.position];
            }
    }
    if (bucket == kBuckets - 1)
        for (uint32_t i = base + len; i < a.tokens_n; ++i) a.keys[0][i] = kNoRow;
}

hipError_t launch_group(const GroupArgs &a, hipStream_t) {
    for (uint32_t bucket = 0; bucket < kBuckets; ++bucket) group_bucket(a, bucket);
    return hipSuccess;
}
hipError_t launch_sums(bool, bool, Goal, const SumArgs &a, hipStream_t) {
    keys.assign(a.keys, a.keys + a.tokens_n);
    order.assign(a.order, a.order + a.tokens_n);
    return hipSuccess;
}
hipError_t launch_lookup(bool, bool, const LookupArgs &, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_direct(bool, bool, Goal, const SumArgs &, const void *, bool, hipStream_t) { return hipErrorInvalidValue; }

}  // namespace adam_mi355x

extern "C" {
const uint32_t *model_keys() { return adam_mi355x::keys.data(); }
const uint32_t *model_order() { return adam_mi355x::order.data(); }
}
