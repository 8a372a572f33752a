// Internal interface between the host runtime and the gfx950 kernels of the
// embedding table's operations.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "adam_internal.h"

namespace adam_mi355x {

// ---------------------------------------------------------------- lookup
struct LookupArgs {
    const void *table;
    const void *tokens;
    void *out;
    uint64_t table_stride, out_stride;  // elements
    uint32_t tokens_n, rows, cols;
    uint32_t wide;  // 64-bit tokens
    float scale;
};
hipError_t launch_lookup(bool table_bf16, bool out_bf16, const LookupArgs &a, hipStream_t stream);

// ---------------------------------------------------------------- grouping
// The tokens' positions grouped by row, in the rows' order.  Row r is in bucket
// r >> bucket_bits, a workgroup a bucket; a bucket's rows are sorted by kDigitBits
// bits at a time, the lowest first.  (Rows in order, not spread over the buckets: what is
// read and written of the table then lies together, DRAM pages and translations
// serve more of it.)
constexpr uint32_t kBuckets = 256;
constexpr uint32_t kDigitBits = 10;
constexpr uint32_t kNoRow = 0xFFFFFFFFu;
constexpr uint32_t kGroupThreads = 1024, kGroupWaves = 16;
constexpr uint32_t kHeld = 8;  // positions that a lane has under way at a time (16: 0.4 to 1.5 us more, 4: 0.5 us less for 2304 and more for 65536)

// Where a wave looks in a pass over `len` positions: at first + k * step + lane for k < kHeld, then
// from first + look on, while that is below end.  A pass places by digit, then by wave, then in
// the order in which the wave looks, so
//   - the first pass, over all tokens, may look in any order: its waves look side by side, which the caches serve best;
//   - every later pass has to keep the order that the passes before it made (rows that are alike
//     in its digit are told apart by theirs), so its waves have one stretch each, in order.
struct GroupPart {
    uint32_t first, end, look;
};
constexpr uint32_t group_step(bool first_pass) { return first_pass ? kGroupThreads : 64; }
constexpr GroupPart group_part(bool first_pass, uint32_t wave, uint32_t len) {
    if (first_pass) return GroupPart{wave * 64, len, kGroupThreads * kHeld};
    const uint32_t part = (len / kGroupThreads + (len % kGroupThreads != 0)) * 64, first = wave * part;
    return GroupPart{first < len ? first : len, first + part < len ? first + part : len, 64 * kHeld};
}

struct GroupArgs {
    const void *tokens;
    uint32_t tokens_n, rows;
    uint32_t wide;
    uint32_t bucket_bits;   // at most kBuckets buckets
    uint32_t passes, bits;  // digits of a bucket's rows, and bits of each
    uint32_t *keys[2];      // the positions' rows: [0] the result (kNoRow behind the last), [1] between passes
    uint32_t *order[2];     // and the positions themselves
    uint32_t *arrivals;     // counters of the sums, set to zero
    uint64_t arrivals_n;
    uint8_t *named;         // of each row, whether a token names it (NULL: not wanted)
};
hipError_t launch_group(const GroupArgs &a, hipStream_t stream);

// ---------------------------------------------------------------- sums
// What becomes of a row's sum.
enum Goal : int { kWrite = 0, kAdd = 1, kAdam = 2, kAdamMax = 3 };

// Positions are taken in windows of 32 or 64: of a run of one row's positions
// that crosses a window's end, each window's piece is summed for itself first.

struct SumArgs {
    const uint32_t *keys, *order;
    uint32_t tokens_n, rows;
    const void *grad;
    uint64_t grad_stride;  // elements
    uint32_t cols;
    uint32_t window, windows;  // positions of a window, and how many windows
    uint32_t slices;   // of a row, 256 columns each
    float scale;
    uint32_t sum_groups;   // workgroups that sum; those behind them zero rows (kWrite)
    const uint8_t *named;
    float *partials;   // two rows a window: of the run that began before it, of the one that began in it
    uint64_t partial_stride;
    uint32_t *arrivals;  // of each slice: two counters a window, and one for the run that begins in it
    void *out;         // the table's gradient, or the table
    uint64_t out_stride;
    // the step
    float *m, *v, *w;
    float step, ibc2, decay, omb1, omb2, beta1, beta2, eps, wd;
    uint32_t l2, fast_ok;
};
hipError_t launch_sums(bool grad_bf16, bool out_bf16, Goal goal, const SumArgs &a, hipStream_t stream);

// Up to this many tokens need no grouping: each position looks through all of them, in
// time that grows with their square.  us for a bf16 gradient of 2048 columns and tokens as
// frequent as words are, this way / by groups: 1024 tokens 6.8 / 17, added to a
// table, 10 / 22 as a step; 2048 tokens 12.5 / 19 and 17 / 27; 4096 tokens 24 / 22 and 31 / 39.
// All of one row: 1024 tokens 16 / 17, 2048 tokens 33 / 19, 4096 tokens 67 / 25.
constexpr uint32_t kDirectTokens = 2048;
constexpr uint32_t kFewTokens = 1024;  // threads look at two tokens each, not at four (0.4 us)
hipError_t launch_direct(bool grad_bf16, bool out_bf16, Goal goal, const SumArgs &a, const void *tokens, bool wide,
                         hipStream_t stream);

}  // namespace adam_mi355x
