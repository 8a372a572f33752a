// Kernels of the embedding table's operations for gfx950 (MI355X): the lookup
// of rows by token, and its gradient or the rows' Adam step.
//
// The gradient of row r is the sum of the gradient's rows whose token is r.  Adding
// them with atomics would give other bits each time and pass every element
// through the cache's atomic units; here the positions are first grouped by
// row (4 bytes a token, against 512 and more of its gradient's row), then every
// wave sums whole runs in registers and writes a row once.  All of it is bound by
// memory: each row of the gradient and of the table is read and written once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "adam_element.h"
#include "embedding_internal.h"

namespace adam_mi355x {
namespace {

// Rows start at any element: 16- and 8-byte accesses aligned to the element, which
// global memory takes.
typedef float f32x4e __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4e __attribute__((ext_vector_type(4), aligned(2)));
typedef uint16_t u16x8e __attribute__((ext_vector_type(8), aligned(2)));

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ void narrow(float x, float &out) { out = x; }
__device__ __forceinline__ void narrow(float x, uint16_t &out) { out = (uint16_t)f32_to_bf16(x); }

template <class T> struct Vec4;
template <> struct Vec4<float> { typedef f32x4e type; };
template <> struct Vec4<uint16_t> { typedef u16x4e type; };

// Four columns of a row from p, the first n of which exist (n may be 0 or
// less, or more than 4): others are zero.
template <bool kStream, class T>
__device__ __forceinline__ f32x4 load4(const T *p, int32_t n) {
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
    if (n >= 4) {
        typename Vec4<T>::type x;
        if constexpr (kStream) x = __builtin_nontemporal_load(reinterpret_cast<const typename Vec4<T>::type *>(p));
        else x = *reinterpret_cast<const typename Vec4<T>::type *>(p);
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = widen((T)x[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k < n) r[k] = widen(p[k]);
    }
    return r;
}

template <class T>
__device__ __forceinline__ void store4(T *p, f32x4 r, int32_t n) {
    if (n >= 4) {
        typename Vec4<T>::type x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            T one;
            narrow(r[k], one);
            x[k] = one;
        }
        __builtin_nontemporal_store(x, reinterpret_cast<typename Vec4<T>::type *>(p));
    } else {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            T one;
            narrow(r[k], one);
            if (k < n) __builtin_nontemporal_store(one, p + k);
        }
    }
}

// The row a token names, or kNoRow.
template <bool kWide>
__device__ __forceinline__ uint32_t row_of(const void *tokens, uint32_t i, uint32_t rows) {
    if constexpr (kWide) {
        const uint64_t t = reinterpret_cast<const uint64_t *>(tokens)[i];
        return t < rows ? (uint32_t)t : kNoRow;
    } else {
        const uint32_t t = reinterpret_cast<const uint32_t *>(tokens)[i];  // negative ones are 2^31 and more
        return t < rows ? t : kNoRow;
    }
}

__device__ __forceinline__ uint32_t uniform_u32(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }
__device__ __forceinline__ uint32_t lane_u32(uint32_t x, uint32_t lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)x, (int)lane);
}

// ---------------------------------------------------------------- lookup
constexpr int kLookupThreads = 256;

template <class T, class O, bool kWide>
__global__ void __launch_bounds__(kLookupThreads) lookup_kernel(LookupArgs a, uint32_t slices, uint64_t units) {
    const uint32_t lane = threadIdx.x & 63u;
    for (uint64_t u = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < units; u += (uint64_t)gridDim.x * 4) {
        const uint32_t i = uniform_u32((uint32_t)(u / slices));
        const uint32_t c0 = uniform_u32((uint32_t)(u % slices)) * 512 + lane * 4;
        const uint32_t row = uniform_u32(row_of<kWide>(a.tokens, i, a.rows));
        const T *from = reinterpret_cast<const T *>(a.table) + (uint64_t)row * a.table_stride;
        O *to = reinterpret_cast<O *>(a.out) + (uint64_t)i * a.out_stride;
        f32x4 x[2] = {};
        if (row != kNoRow) {
#pragma unroll
            for (int g = 0; g < 2; ++g) x[g] = load4<false>(from + c0 + 256 * g, (int32_t)(a.cols - c0) - 256 * g);
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) store4(to + c0 + 256 * g, x[g] * a.scale, (int32_t)(a.cols - c0) - 256 * g);
    }
}

// ---------------------------------------------------------------- grouping
constexpr int kGroupThreads = 1024, kGroupWaves = 16;
constexpr uint32_t kGroupBlock = 256;  // positions a wave takes at a time, four a lane
constexpr uint32_t kMaxBins = 1u << kDigitBits;

// One workgroup a bucket: it reads every token and keeps those of its rows.
// Reading all tokens 256 times costs 8 bytes x 256 a token from the caches, and
// saves the passes over memory (with a launch each) of a sort by tiles.  The positions are
// placed by counting: each wave counts its own positions by digit, the counts
// become places by a sum over digits and waves, and each wave goes
// through the same positions again and places them.  Lanes with one digit are
// ranked by ballots, not by the order in which atomics arrive, so the result is
// always the same.
template <bool kWide>
__global__ void __launch_bounds__(kGroupThreads) group_kernel(GroupArgs a) {
    extern __shared__ uint32_t counts[];  // [kGroupWaves][bins]
    __shared__ uint32_t wave_sums[kGroupWaves];
    __shared__ uint32_t below_sum;
    __shared__ uint32_t named[kMaxBins / 32];  // bitmap of rows that a token names
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = uniform_u32(tid >> 6), bucket = blockIdx.x;
    const uint32_t bins = 1u << a.bits;
    uint32_t *mine = counts + wave * bins;
    uint32_t base = 0, len = a.tokens_n;
    if (tid == 0) below_sum = 0;
    for (uint32_t pass = 0; pass < a.passes; ++pass) {
        const uint32_t shift = 8 + pass * kDigitBits, to = (a.passes - 1 - pass) & 1u;
        const uint32_t *keys_in = a.keys[to ^ 1u], *order_in = a.order[to ^ 1u];
        for (uint32_t i = tid; i < kGroupWaves * bins; i += kGroupThreads) counts[i] = 0;
        __syncthreads();
        // the keys of this wave's positions from block `b` on; in the first pass kNoRow
        // for the other buckets' ones
        uint32_t below = 0;
        auto fetch = [&](uint32_t b, uint32_t (&key)[4], bool count) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t i = b * kGroupBlock + j * 64 + lane;
                key[j] = kNoRow;
                if (i < len) key[j] = pass == 0 ? row_of<kWide>(a.tokens, i, a.rows) : keys_in[base + i];
            }
            if (pass == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t in = key[j] & (kBuckets - 1);
                    if (count) below += key[j] != kNoRow && in < bucket ? 1u : 0u;
                    if (in != bucket) key[j] = kNoRow;
                }
            }
        };
        const uint32_t blocks = len / kGroupBlock + (len % kGroupBlock != 0);
        for (uint32_t b = wave; b < blocks; b += kGroupWaves) {
            uint32_t key[4];
            fetch(b, key, true);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (key[j] != kNoRow) atomicAdd(mine + ((key[j] >> shift) & (bins - 1)), 1u);
        }
        if (pass == 0) {
            for (int s = 32; s > 0; s >>= 1) below += __shfl_xor(below, s);
            if (lane == 0) atomicAdd(&below_sum, below);
        }
        __syncthreads();
        // counts to places
        uint32_t digit_total = 0;
        if (tid < bins) {
#pragma unroll
            for (int w = 0; w < kGroupWaves; ++w) {
                const uint32_t c = counts[w * bins + tid];
                counts[w * bins + tid] = digit_total;
                digit_total += c;
            }
        }
        uint32_t incl = digit_total;
        for (int s = 1; s < 64; s <<= 1) {
            const uint32_t x = __shfl_up(incl, s);
            if (lane >= (uint32_t)s) incl += x;
        }
        if (lane == 63) wave_sums[wave] = incl;
        const uint64_t any = __ballot(digit_total != 0);
        if (pass == 0 && lane < 2) named[2 * wave + lane] = (uint32_t)(any >> (32 * lane));
        __syncthreads();
        uint32_t before = 0, all = 0;
        for (int w = 0; w < kGroupWaves; ++w) {
            const uint32_t s = wave_sums[w];
            before += w < (int)wave ? s : 0u;
            all += s;
        }
        if (pass == 0) base = below_sum;
        const uint32_t first = base + before + incl - digit_total;
        if (tid < bins) {
#pragma unroll
            for (int w = 0; w < kGroupWaves; ++w) counts[w * bins + tid] += first;
        }
        __syncthreads();
        // places
        for (uint32_t b = wave; b < blocks; b += kGroupWaves) {
            uint32_t key[4];
            fetch(b, key, false);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint64_t same = __ballot(key[j] != kNoRow);
                if (same == 0) continue;
                const uint32_t digit = (key[j] >> shift) & (bins - 1);
                for (uint32_t k = 0; k < a.bits; ++k) {
                    const uint64_t set = __ballot((digit >> k) & 1u);
                    same &= (digit >> k) & 1u ? set : ~set;
                }
                if (key[j] != kNoRow) {
                    const uint32_t leader = (uint32_t)__builtin_ctzll(same);
                    const uint32_t rank = (uint32_t)__popcll(same & ((1ull << lane) - 1));
                    uint32_t place = 0;
                    if (lane == leader) place = atomicAdd(mine + digit, (uint32_t)__popcll(same));
                    place = __shfl(place, (int)leader) + rank;
                    const uint32_t i = b * kGroupBlock + j * 64 + lane;
                    if (place < a.tokens_n) {  // always, unless tokens change under the call
                        a.keys[to][place] = key[j];
                        a.order[to][place] = pass == 0 ? i : order_in[base + i];
                    }
                }
            }
        }
        if (pass == 0) len = all;
        __syncthreads();
    }
    if (bucket == kBuckets - 1 && tid == 0) *a.total = base + len;
    if (!a.zero) return;
    // the bucket's rows that no token names
    const uint32_t rows = a.rows > bucket ? (a.rows - bucket - 1) / kBuckets + 1 : 0;
    for (uint32_t r0 = 0; r0 < rows; r0 += kMaxBins) {
        if (a.passes > 1) {
            for (uint32_t i = tid; i < kMaxBins / 32; i += kGroupThreads) named[i] = 0;
            __syncthreads();
            for (uint32_t i = tid; i < len; i += kGroupThreads) {
                const uint32_t r = a.keys[0][base + i] / kBuckets;
                if (r >= r0 && r - r0 < kMaxBins) atomicOr(&named[(r - r0) / 32], 1u << (r % 32));
            }
            __syncthreads();
        }
        const uint32_t n = min(kMaxBins, rows - r0);
        for (uint32_t k = wave; k < n; k += kGroupWaves) {
            if ((uniform_u32(named[k / 32]) >> (k % 32)) & 1u) continue;
            char *row = reinterpret_cast<char *>(a.zero) + (uint64_t)((r0 + k) * (uint64_t)kBuckets + bucket) * a.zero_stride;
            const uint64_t fours = a.zero_bytes / 16;
            for (uint64_t c = lane; c < fours; c += 64)
                __builtin_nontemporal_store(u16x8e{}, reinterpret_cast<u16x8e *>(row) + c);
            const uint64_t rest = fours * 16 + lane * 2;
            if (rest < a.zero_bytes) __builtin_nontemporal_store((uint16_t)0, reinterpret_cast<uint16_t *>(row + rest));
        }
        if (a.passes > 1) __syncthreads();
    }
}

// ---------------------------------------------------------------- sums
constexpr int kSumThreads = 256;

// The update of four elements, adam_step's operations in its order (see there for
// the ranges of the short sequences).  n: how many of them exist.
template <bool kMax>
__device__ __forceinline__ void update4(const SumArgs &a, f32x4 &p, f32x4 g, f32x4 &m, f32x4 &v, f32x4 &w, int32_t n) {
    if (a.l2) {
#pragma unroll
        for (int k = 0; k < 4; ++k) g[k] = fmaf(a.wd, p[k], g[k]);
    }
    float m_lo = __builtin_inff(), m_hi = 0.0f, v_lo = __builtin_inff();
    f32x4 below;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        m[k] = fmaf(a.beta1, m[k], a.omb1 * g[k]);
        v[k] = fmaf(a.beta2, v[k], a.omb2 * (g[k] * g[k]));
        if constexpr (kMax) w[k] = fmaxf(w[k], v[k]);
        below[k] = kMax ? w[k] : v[k];
        m_lo = fminf(m_lo, fabsf(m[k]));
        m_hi = fmaxf(m_hi, fabsf(m[k]));
        v_lo = fminf(v_lo, below[k]);
    }
    if (__all(n <= 0 || (a.fast_ok && v_lo >= 0x1p-96f && m_lo >= 0x1p-40f && m_hi <= 0x1p40f))) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            p[k] = fmaf(-a.step, div_rn(m[k], fmaf(sqrt_rn(below[k]), a.ibc2, a.eps)), p[k] * a.decay);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            p[k] = fmaf(-a.step, m[k] / fmaf(sqrtf(below[k]), a.ibc2, a.eps), p[k] * a.decay);
    }
}

// A row's whole sum: written, added, or taken as the step's gradient.
template <class O, Goal kGoal, int kG>
__device__ __forceinline__ void finish(const SumArgs &a, uint32_t row, uint32_t c0, const f32x4 (&sum)[kG]) {
    O *to = reinterpret_cast<O *>(a.out) + (uint64_t)row * a.out_stride + c0;
    const int32_t left = (int32_t)(a.cols - c0);
    if constexpr (kGoal == kWrite) {
#pragma unroll
        for (int g = 0; g < kG; ++g) store4(to + 256 * g, sum[g] * a.scale, left - 256 * g);
    } else if constexpr (kGoal == kAdd) {
        f32x4 old[kG];
#pragma unroll
        for (int g = 0; g < kG; ++g) old[g] = load4<true>(to + 256 * g, left - 256 * g);
#pragma unroll
        for (int g = 0; g < kG; ++g) store4(to + 256 * g, old[g] + sum[g] * a.scale, left - 256 * g);
    } else {
        constexpr bool kMax = kGoal == kAdamMax;
        const uint64_t s = (uint64_t)row * a.cols + c0;
        f32x4 p[kG], m[kG], v[kG], w[kG];
#pragma unroll
        for (int g = 0; g < kG; ++g) {
            p[g] = load4<true>(to + 256 * g, left - 256 * g);
            m[g] = load4<true>(a.m + s + 256 * g, left - 256 * g);
            v[g] = load4<true>(a.v + s + 256 * g, left - 256 * g);
            if constexpr (kMax) w[g] = load4<true>(a.w + s + 256 * g, left - 256 * g);
        }
#pragma unroll
        for (int g = 0; g < kG; ++g) {
            update4<kMax>(a, p[g], sum[g] * a.scale, m[g], v[g], w[g], left - 256 * g);
            store4(to + 256 * g, p[g], left - 256 * g);
            store4(a.m + s + 256 * g, m[g], left - 256 * g);
            store4(a.v + s + 256 * g, v[g], left - 256 * g);
            if constexpr (kMax) store4(a.w + s + 256 * g, w[g], left - 256 * g);
        }
    }
}

// A wave takes the runs (of one row's positions) that begin in its portion of a
// window, in one slice of columns.  A run that crosses the window's end counts
// as beginning again in the next one, and leaves partial sums.
template <class T, class O, Goal kGoal, int kG>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(SumArgs a) {
    const uint32_t lane = threadIdx.x & 63u, total = *a.total;
    for (uint64_t u = (uint64_t)blockIdx.x * 4 + uniform_u32(threadIdx.x >> 6); u < a.units; u += (uint64_t)gridDim.x * 4) {
        const uint32_t first = uniform_u32((uint32_t)(u / a.slices)) * a.portion;
        const uint32_t c0 = uniform_u32((uint32_t)(u % a.slices)) * (256 * kG) + lane * 4;
        if (first >= total) break;
        const uint32_t w0 = first & ~(kWindow - 1), pos = w0 + lane;
        const uint32_t live = min(kWindow, total - w0);
        const bool in = lane < live;
        const uint32_t key = in ? a.keys[pos] : kNoRow, from = in ? a.order[pos] : 0u;
        const uint32_t last = w0 > 0 ? a.keys[w0 - 1] : kNoRow;
        const uint32_t next = total - w0 > kWindow ? a.keys[w0 + kWindow] : kNoRow;
        const uint32_t prev = __shfl_up(key, 1);
        const uint64_t heads = __ballot(in && (lane == 0 || key != prev));
        const bool continued = uniform_u32(key) == last;  // the window's first run began before it
        const uint32_t stop = min(first - w0 + a.portion, live);
        const int32_t left = (int32_t)(a.cols - c0);
        const uint64_t mine = heads >> (first - w0);
        uint32_t h = mine ? first - w0 + (uint32_t)__builtin_ctzll(mine) : kWindow;
        while (h < stop) {
            const uint64_t after = h + 1 < kWindow ? heads >> (h + 1) : 0;
            const uint32_t e = after ? h + 1 + (uint32_t)__builtin_ctzll(after) : live;
            const uint32_t row = lane_u32(key, h);
            f32x4 sum[kG] = {};
            auto fetch = [&](uint32_t k, f32x4 (&x)[kG]) {
                const T *p = reinterpret_cast<const T *>(a.grad) + (uint64_t)lane_u32(from, k) * a.grad_stride + c0;
#pragma unroll
                for (int g = 0; g < kG; ++g) x[g] = load4<true>(p + 256 * g, left - 256 * g);
            };
            uint32_t k = h;
            for (; k + 4 <= e; k += 4) {
                f32x4 x[4][kG];
#pragma unroll
                for (int j = 0; j < 4; ++j) fetch(k + j, x[j]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int g = 0; g < kG; ++g) sum[g] += x[j][g];
            }
            for (; k < e; ++k) {
                f32x4 x[kG];
                fetch(k, x);
#pragma unroll
                for (int g = 0; g < kG; ++g) sum[g] += x[g];
            }
            const bool began = !(h == 0 && continued), ends = !(e == kWindow && next == row);
            if (began && ends) {
                finish<O, kGoal, kG>(a, row, c0, sum);
            } else {
                float *to = a.partials + ((uint64_t)(w0 / kWindow) * 2 + (began ? 1 : 0)) * a.partial_stride + c0;
#pragma unroll
                for (int g = 0; g < kG; ++g) store4(to + 256 * g, sum[g], left - 256 * g);
            }
            h = after ? e : kWindow;
        }
    }
}

// The run that crosses the end of a window and began in it: its partial sums
// are the window's second, and the first of each window that it goes on into.
// A workgroup a window and slice; its waves take a quarter of the windows each.
template <class O, Goal kGoal, int kG>
__global__ void __launch_bounds__(kSumThreads) join_kernel(SumArgs a) {
    __shared__ f32x4 parts[3][kG][64];
    const uint32_t lane = threadIdx.x & 63u, wave = uniform_u32(threadIdx.x >> 6), total = *a.total;
    for (uint64_t u = blockIdx.x; u < (uint64_t)a.windows * a.slices; u += gridDim.x) {
        const uint32_t window = uniform_u32((uint32_t)(u / a.slices));
        const uint32_t end = (window + 1) * kWindow;
        if (end >= total) break;
        const uint32_t row = a.keys[end];
        if (a.keys[end - 1] != row) continue;
        if (window > 0 && a.keys[window * kWindow - 1] == row) continue;  // began before
        // windows that the run goes on into
        uint32_t more = 1;
        for (;;) {
            const uint64_t at = (uint64_t)end + (uint64_t)(more + lane) * kWindow;
            const uint64_t same = __ballot(at < total && a.keys[at < total ? at : 0] == row);
            const uint32_t got = ~same ? (uint32_t)__builtin_ctzll(~same) : 64u;
            more += got;
            if (got < 64) break;
        }
        const uint32_t c0 = uniform_u32((uint32_t)(u % a.slices)) * (256 * kG) + lane * 4;
        const int32_t left = (int32_t)(a.cols - c0);
        f32x4 sum[kG] = {};
        auto add = [&](uint64_t slot) {
            const float *p = a.partials + slot * a.partial_stride + c0;
#pragma unroll
            for (int g = 0; g < kG; ++g) sum[g] += load4<false>(p + 256 * g, left - 256 * g);
        };
        if (wave == 0) add((uint64_t)window * 2 + 1);
        const uint32_t quarter = (more + 3) / 4, k1 = min(more, (wave + 1) * quarter);
        for (uint32_t k = wave * quarter; k < k1; ++k) add((uint64_t)(window + 1 + k) * 2);
        if (wave > 0) {
#pragma unroll
            for (int g = 0; g < kG; ++g) parts[wave - 1][g][lane] = sum[g];
        }
        __syncthreads();
        if (wave == 0) {
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int g = 0; g < kG; ++g) sum[g] += parts[k][g][lane];
            finish<O, kGoal, kG>(a, row, c0, sum);
        }
        __syncthreads();
    }
}

constexpr uint64_t kMaxGrid = (1u << 24) - 1;  // grid.x * 256 work-items < 2^32
uint32_t grid_of(uint64_t workgroups) { return (uint32_t)std::min<uint64_t>(workgroups, kMaxGrid); }

template <class T, class O, Goal kGoal>
hipError_t launch_sums_of(const SumArgs &a, hipStream_t stream) {
    const dim3 grid(grid_of((a.units + 3) / 4));
    if (slice_cols(a.cols) == 256) hipLaunchKernelGGL((sum_kernel<T, O, kGoal, 1>), grid, dim3(kSumThreads), 0, stream, a);
    else hipLaunchKernelGGL((sum_kernel<T, O, kGoal, 2>), grid, dim3(kSumThreads), 0, stream, a);
    return hipGetLastError();
}

template <class O, Goal kGoal>
hipError_t launch_joins_of(const SumArgs &a, hipStream_t stream) {
    const dim3 grid(grid_of((uint64_t)a.windows * a.slices));
    if (slice_cols(a.cols) == 256) hipLaunchKernelGGL((join_kernel<O, kGoal, 1>), grid, dim3(kSumThreads), 0, stream, a);
    else hipLaunchKernelGGL((join_kernel<O, kGoal, 2>), grid, dim3(kSumThreads), 0, stream, a);
    return hipGetLastError();
}

template <class T, class O>
hipError_t launch_lookup_of(const LookupArgs &a, hipStream_t stream) {
    const uint32_t slices = (a.cols + 511) / 512;
    const uint64_t units = (uint64_t)a.tokens_n * slices;
    const dim3 grid(grid_of((units + 3) / 4));
    if (a.wide) hipLaunchKernelGGL((lookup_kernel<T, O, true>), grid, dim3(kLookupThreads), 0, stream, a, slices, units);
    else hipLaunchKernelGGL((lookup_kernel<T, O, false>), grid, dim3(kLookupThreads), 0, stream, a, slices, units);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lookup(bool table_bf16, bool out_bf16, const LookupArgs &a, hipStream_t stream) {
    if (table_bf16)
        return out_bf16 ? launch_lookup_of<uint16_t, uint16_t>(a, stream) : launch_lookup_of<uint16_t, float>(a, stream);
    return out_bf16 ? launch_lookup_of<float, uint16_t>(a, stream) : launch_lookup_of<float, float>(a, stream);
}

hipError_t launch_group(const GroupArgs &a, hipStream_t stream) {
    const size_t lds = (size_t)kGroupWaves * 4u << a.bits;
    if (a.wide) hipLaunchKernelGGL(group_kernel<true>, dim3(kBuckets), dim3(kGroupThreads), lds, stream, a);
    else hipLaunchKernelGGL(group_kernel<false>, dim3(kBuckets), dim3(kGroupThreads), lds, stream, a);
    return hipGetLastError();
}

hipError_t launch_sums(bool grad_bf16, bool out_bf16, Goal goal, const SumArgs &a, hipStream_t stream) {
    switch (goal) {
    case kWrite:
        if (grad_bf16)
            return out_bf16 ? launch_sums_of<uint16_t, uint16_t, kWrite>(a, stream)
                            : launch_sums_of<uint16_t, float, kWrite>(a, stream);
        return out_bf16 ? launch_sums_of<float, uint16_t, kWrite>(a, stream) : launch_sums_of<float, float, kWrite>(a, stream);
    case kAdd:
        if (grad_bf16)
            return out_bf16 ? launch_sums_of<uint16_t, uint16_t, kAdd>(a, stream)
                            : launch_sums_of<uint16_t, float, kAdd>(a, stream);
        return out_bf16 ? launch_sums_of<float, uint16_t, kAdd>(a, stream) : launch_sums_of<float, float, kAdd>(a, stream);
    case kAdam:
        return grad_bf16 ? launch_sums_of<uint16_t, float, kAdam>(a, stream) : launch_sums_of<float, float, kAdam>(a, stream);
    default:
        return grad_bf16 ? launch_sums_of<uint16_t, float, kAdamMax>(a, stream)
                         : launch_sums_of<float, float, kAdamMax>(a, stream);
    }
}

hipError_t launch_joins(bool out_bf16, Goal goal, const SumArgs &a, hipStream_t stream) {
    switch (goal) {
    case kWrite: return out_bf16 ? launch_joins_of<uint16_t, kWrite>(a, stream) : launch_joins_of<float, kWrite>(a, stream);
    case kAdd: return out_bf16 ? launch_joins_of<uint16_t, kAdd>(a, stream) : launch_joins_of<float, kAdd>(a, stream);
    case kAdam: return launch_joins_of<float, kAdam>(a, stream);
    default: return launch_joins_of<float, kAdamMax>(a, stream);
    }
}

}  // namespace adam_mi355x
