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
// The tokens' positions grouped by row.  Row r is in bucket r % kBuckets; a
// workgroup a bucket.  Within a bucket a position's key is r / kBuckets, taken
// kDigitBits bits at a time.
constexpr uint32_t kBuckets = 256;
constexpr uint32_t kDigitBits = 10;
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

struct GroupArgs {
    const void *tokens;
    uint32_t tokens_n, rows;
    uint32_t wide;
    uint32_t passes, bits;  // digits of a key, and bits of each
    uint32_t *keys[2];      // rows, grouped: [0] the result, [1] between passes (if there are several)
    uint32_t *order[2];     // and the positions they came from
    uint32_t *total;        // positions that name a row
    // rows that no token names, zeroed (NULL: not)
    void *zero;
    uint64_t zero_stride;  // bytes
    uint64_t zero_bytes;   // of a row
};
hipError_t launch_group(const GroupArgs &a, hipStream_t stream);

// ---------------------------------------------------------------- sums
// What becomes of a row's sum.
enum Goal : int { kWrite = 0, kAdd = 1, kAdam = 2, kAdamMax = 3 };

// Positions are taken in windows of kWindow: a run of one row's positions
// that crosses a window's end leaves a partial sum in each window.
constexpr uint32_t kWindow = 64;

struct SumArgs {
    const uint32_t *keys, *order, *total;
    const void *grad;
    uint64_t grad_stride;  // elements
    uint32_t cols;
    uint32_t portion;  // positions a wave starts runs in (a power of two up to kWindow)
    uint32_t slices;   // column slices of a row
    uint32_t windows;
    uint64_t units;    // waves' worth of work: portions * slices
    float scale;
    float *partials;   // two rows a window: of the run that began before it, of the one that began in it
    uint64_t partial_stride;
    void *out;         // the table's gradient, or the table
    uint64_t out_stride;
    // the step
    float *m, *v, *w;
    float step, ibc2, decay, omb1, omb2, beta1, beta2, eps, wd;
    uint32_t l2, fast_ok;
};
// Columns a wave takes of a row: 256 or 512.
constexpr uint32_t slice_cols(uint32_t cols) { return cols <= 256 ? 256 : 512; }
hipError_t launch_sums(bool grad_bf16, bool out_bf16, Goal goal, const SumArgs &a, hipStream_t stream);
// the runs that crossed windows, from their partial sums
hipError_t launch_joins(bool out_bf16, Goal goal, const SumArgs &a, hipStream_t stream);

}  // namespace adam_mi355x
