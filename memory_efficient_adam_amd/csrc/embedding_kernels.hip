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
#include <type_traits>

#include "adam_element.h"
#include "embedding_internal.h"

namespace adam_mi355x {
namespace {

// Rows start at any element: 16- and 8-byte accesses aligned to the element, which
// global memory takes.
typedef float f32x4e __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4e __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x8e __attribute__((ext_vector_type(8), aligned(2)));

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ void narrow(float x, float &out) { out = x; }
__device__ __forceinline__ void narrow(float x, uint16_t &out) { out = (uint16_t)f32_to_bf16(x); }

template <int kN> struct Int { static constexpr int value = kN; };

template <class T> struct Vec4;
template <> struct Vec4<float> { typedef f32x4e type; };
template <> struct Vec4<uint16_t> { typedef u16x4e type; };

// Four columns of a row as they are stored.  Loading and widening are apart:
// what follows a load in its branch waits for it there, and with it for every
// load before, so a widening in the branch would let one load be under way at a time.
template <class T>
struct Four {
    typename Vec4<T>::type x;

    // from p, the first n of which exist (n may be 0 or less, or more than 4): others are zero
    template <bool kStream>
    __device__ __forceinline__ void load(const T *p, int32_t n) {
        x = typename Vec4<T>::type{};
        if (n >= 4) {
            if constexpr (kStream) x = __builtin_nontemporal_load(reinterpret_cast<const typename Vec4<T>::type *>(p));
            else x = *reinterpret_cast<const typename Vec4<T>::type *>(p);
        } else if (n > 0) {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (k < n) x[k] = p[k];
        }
    }
    __device__ __forceinline__ f32x4 wide() const {
        return f32x4{widen((T)x[0]), widen((T)x[1]), widen((T)x[2]), widen((T)x[3])};
    }
};

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

// The row that a token names, or kNoRow.
__device__ __forceinline__ uint32_t row_of(uint64_t token, uint32_t rows) { return token < rows ? (uint32_t)token : kNoRow; }
// (negative ones are 2^31 and more)
__device__ __forceinline__ uint32_t row_of(uint32_t token, uint32_t rows) { return token < rows ? token : kNoRow; }

// A token in two words.
__device__ __forceinline__ uint32_t low_word(uint64_t token) { return (uint32_t)token; }
__device__ __forceinline__ uint32_t low_word(uint32_t token) { return token; }
__device__ __forceinline__ uint32_t high_word(uint64_t token) { return (uint32_t)(token >> 32); }
__device__ __forceinline__ uint32_t high_word(uint32_t) { return 0; }

__device__ __forceinline__ uint32_t uniform_u32(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }
__device__ __forceinline__ uint32_t lane_u32(uint32_t x, uint32_t lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)x, (int)lane);
}

// ---------------------------------------------------------------- lookup
constexpr int kLookupThreads = 256;

// out_i = scale table[x_i].  A wave a token and 512 columns: two loads of each lane are
// under way, and a workgroup's four waves are at four places of the table.  Bound by
// memory: 16384 tokens of 50304 x 2048, fp32 to bf16: 116 MB (rows named twice come
// from the caches) in 23 us, 5.0 TB/s, where a large copy reaches 4.9; by the launch
// for a few tokens (8 tokens: 3 us).

template <class T, class O, class Token>
__global__ void __launch_bounds__(kLookupThreads) lookup_kernel(LookupArgs a, uint32_t slices, uint64_t units) {
    const uint32_t lane = threadIdx.x & 63u;
    for (uint64_t u = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < units; u += (uint64_t)gridDim.x * 4) {
        const uint32_t i = uniform_u32((uint32_t)(u / slices));
        const uint32_t c0 = uniform_u32((uint32_t)(u % slices)) * 512 + lane * 4;
        const uint32_t row = uniform_u32(row_of(reinterpret_cast<const Token *>(a.tokens)[i], a.rows));
        const T *from = reinterpret_cast<const T *>(a.table) + (uint64_t)row * a.table_stride;
        O *to = reinterpret_cast<O *>(a.out) + (uint64_t)i * a.out_stride;
        const int32_t left = (int32_t)(a.cols - c0);
        Four<T> x[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) x[g].template load<false>(from + c0 + 256 * g, row != kNoRow ? left - 256 * g : 0);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            // 0 for padding, whatever the scale
            const f32x4 one = row != kNoRow ? x[g].wide() * a.scale : f32x4{0.f, 0.f, 0.f, 0.f};
            store4(to + c0 + 256 * g, one, left - 256 * g);
        }
    }
}

// Zeroes the rows [r0, r1) of a table that are not `named`, by a workgroup: rows one
// after the other, so that the workgroups in flight write one stretch of memory.
template <class O, class Named>
__device__ __forceinline__ void zero_rows(O *table, uint64_t stride, uint32_t cols, uint64_t r0, uint64_t r1, uint32_t threads,
                                          Named named) {
    constexpr uint32_t kPer = 16 / sizeof(O);
    for (uint64_t r = r0; r < r1; ++r) {
        if (named(r)) continue;
        O *const row = table + r * stride;
        const uint32_t whole = cols / kPer;
        for (uint32_t c = threadIdx.x; c < whole; c += threads) *reinterpret_cast<u16x8e *>(row + c * (uint64_t)kPer) = u16x8e{};
        const uint32_t rest = whole * kPer + threadIdx.x;
        if (rest < cols) row[rest] = O(0);
    }
}

// ---------------------------------------------------------------- grouping
constexpr uint32_t kListed = 64 * kHeld;  // positions of its bucket that a wave keeps: those of one look at most

// Orders a wave's LDS stores before its loads of what other lanes stored.
__device__ __forceinline__ void wave_lds_fence() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// One workgroup a bucket: it reads every token and keeps the positions of its
// rows.  Reading all tokens 256 times costs 8 bytes x 256 a token from the
// caches, and saves the passes over memory (with a launch each) of a sort by
// tiles.  The positions are placed by counting: each wave lists its own (in
// LDS; where they are too many it finds them again later) and counts them by digit,
// the counts become places by a sum over digits and waves, and each wave
// places its list, 64 positions at a time.  Lanes with one digit are ranked by
// ballots, not by the order in which atomics arrive, so positions of one
// digit keep the order of the waves and of each wave's looks, and the result is always
// the same.  In the passes after the first that has to be the order which the
// passes before left, or rows that only their digits tell apart get mixed again (group_part).
//
// What bounds it is the latency of the tokens' loads in each CU: 9 us for 16384 tokens
// of 64 bits, 21 for 65536, against 80 to 450 us of the sums behind it, where the buckets have
// much the same.  Where one has half of the tokens (ids in order of frequency) or all of them (one row),
// its workgroup places them and looks at every token again: 18 and 52 us for half of
// them, 60 us for 32768 tokens of one row.  256 buckets, one a CU:
// with 128 the whole call on narrow rows takes 1 to 4% more and with 64 3 to 13%, though the
// XCDs' caches then serve half and a quarter as much; and the largest table whose
// rows one digit tells apart, 262144 rows, becomes smaller (16384 tokens: 11 us there, 15 to 16 with
// a second digit, 42 in order of frequency).
template <class Token>
__global__ void __launch_bounds__(kGroupThreads) group_kernel(GroupArgs a) {
    extern __shared__ uint2 shared[];  // [kGroupWaves][kListed] {row, position}, then counts [kGroupWaves][bins]
    __shared__ uint32_t wave_sums[kGroupWaves];
    __shared__ uint32_t below_sum;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = uniform_u32(tid >> 6), bucket = blockIdx.x;
    const uint32_t bins = 1u << a.bits;
    uint32_t *const counts = reinterpret_cast<uint32_t *>(shared + kGroupWaves * kListed), *const mine = counts + wave * bins;
    uint2 *const list = shared + wave * kListed;
    uint32_t base = 0, len = a.tokens_n;
    // the bucket's rows are [bucket0, bucket0 + width); rows below `limit` are those of earlier buckets
    const uint32_t bucket0 = bucket << a.bucket_bits, limit = min(bucket0, a.rows), width = min(a.rows - limit, 1u << a.bucket_bits);
    if (tid == 0) below_sum = 0;
    for (uint64_t i = bucket * kGroupThreads + tid; i < a.arrivals_n; i += kBuckets * kGroupThreads) a.arrivals[i] = 0;
    for (uint32_t pass = 0; pass < a.passes; ++pass) {
        const uint32_t shift = pass * kDigitBits, to = (a.passes - 1 - pass) & 1u;
        const uint32_t *keys_in = a.keys[to ^ 1u], *order_in = a.order[to ^ 1u];
        const GroupPart part = group_part(pass == 0, wave, len);
        uint32_t below = 0, listed = 0;
        auto digit_of = [&](uint32_t key) { return (key >> shift) & (bins - 1); };
        // The bucket's positions among those of `in` at p0 + j * step + lane are listed behind the `listed`
        // ones and, the first time, counted.  A CU looks at every token, so instructions count: where no
        // position is behind the end they are loaded without clamping, and a token's words are compared apart (7% of
        // a call on 65536 tokens of 32 bits and narrow rows, 1% of one on 64 bits).
        auto look = [&](auto step, const auto *in, uint32_t p0, bool count) {
            typedef std::remove_cv_t<std::remove_pointer_t<decltype(in)>> Key;
            constexpr uint32_t kStep = decltype(step)::value;
            Key key[kHeld];
            if (p0 + (kHeld - 1) * kStep + 64 <= part.end) {
#pragma unroll
                for (uint32_t j = 0; j < kHeld; ++j) key[j] = (in + p0 + j * kStep)[lane];
            } else {
#pragma unroll
                for (uint32_t j = 0; j < kHeld; ++j) key[j] = in[min(p0 + j * kStep + lane, part.end - 1)];
#pragma unroll
                for (uint32_t j = 0; j < kHeld; ++j)
                    if (p0 + j * kStep + lane >= part.end) key[j] = ~Key(0);  // names no row
            }
#pragma unroll
            for (uint32_t j = 0; j < kHeld; ++j) {
                const uint32_t low = low_word(key[j]);
                uint32_t high = high_word(key[j]);
                if constexpr (sizeof(Key) == 8) asm("" : "+v"(high));  // compared as a word, not with the low one
                const bool fits = high == 0, have = fits && low - bucket0 < width;
                const uint64_t all = __builtin_amdgcn_ballot_w64(have);
                if (count) below += (uint32_t)__popcll(__builtin_amdgcn_ballot_w64(fits && low < limit));
                if (all == 0) continue;
                if (have) {
                    const uint32_t at = listed + (uint32_t)__popcll(all & ((1ull << lane) - 1));
                    if (at < kListed) list[at] = uint2{low, p0 + j * kStep + lane};
                    if (count) atomicAdd(mine + digit_of(low), 1u);
                }
                listed += (uint32_t)__popcll(all);
            }
        };
        auto look_at = [&](uint32_t p0, bool count) {
            if (pass == 0) look(Int<group_step(true)>(), reinterpret_cast<const Token *>(a.tokens), p0, count);
            else look(Int<group_step(false)>(), keys_in + base, p0, count);
        };
        for (uint32_t i = tid; i < kGroupWaves * bins; i += kGroupThreads) counts[i] = 0;
        __syncthreads();
        for (uint32_t p0 = part.first; p0 < part.end; p0 += part.look) look_at(p0, true);
        if (pass == 0 && lane == 0) atomicAdd(&below_sum, below);
        __syncthreads();
        // counts to places: thread d has digit d's of every wave
        uint32_t held[kGroupWaves], digit_total = 0;
        if (tid < bins) {
#pragma unroll
            for (uint32_t w = 0; w < kGroupWaves; ++w) held[w] = counts[w * bins + tid];
#pragma unroll
            for (uint32_t w = 0; w < kGroupWaves; ++w) {
                const uint32_t c = held[w];
                held[w] = digit_total;
                digit_total += c;
            }
        }
        uint32_t incl = digit_total;
        for (int s = 1; s < 64; s <<= 1) {
            const uint32_t x = __shfl_up(incl, s);
            if (lane >= (uint32_t)s) incl += x;
        }
        if (lane == 63) wave_sums[wave] = incl;
        __syncthreads();
        uint32_t before = 0, all = 0;
#pragma unroll
        for (uint32_t w = 0; w < kGroupWaves; ++w) {
            const uint32_t s = wave_sums[w];
            before += w < wave ? s : 0u;
            all += s;
        }
        if (pass == 0) base = uniform_u32(below_sum);
        const uint32_t first = base + before + incl - digit_total;
        if (tid < bins) {
#pragma unroll
            for (uint32_t w = 0; w < kGroupWaves; ++w) counts[w * bins + tid] = held[w] + first;
        }
        __syncthreads();
        // places
        auto place_list = [&]() {
            for (uint32_t k0 = 0; k0 < listed; k0 += 64) {
                const uint2 one = k0 + lane < listed ? list[k0 + lane] : uint2{kNoRow, 0};
                const uint32_t digit = digit_of(one.x);
                uint64_t same = __builtin_amdgcn_ballot_w64(one.x != kNoRow);
                for (uint32_t k = 0; k < a.bits; ++k) {
                    const uint64_t set = __builtin_amdgcn_ballot_w64((digit >> k) & 1u);
                    same &= (digit >> k) & 1u ? set : ~set;
                }
                if (one.x != kNoRow) {
                    const uint32_t leader = (uint32_t)__builtin_ctzll(same);
                    uint32_t place = 0;
                    if (lane == leader) place = atomicAdd(mine + digit, (uint32_t)__popcll(same));
                    place = __shfl(place, (int)leader) + (uint32_t)__popcll(same & ((1ull << lane) - 1));
                    if (place < a.tokens_n) {  // always, unless tokens change under the call
                        a.keys[to][place] = one.x;
                        a.order[to][place] = pass == 0 ? one.y : order_in[base + one.y];
                    }
                }
            }
        };
        if (listed <= kListed) {
            place_list();
        } else {
            for (uint32_t p0 = part.first; p0 < part.end; p0 += part.look) {
                listed = 0;
                look_at(p0, false);
                wave_lds_fence();
                place_list();
                wave_lds_fence();
            }
        }
        if (pass == 0) len = uniform_u32(all);
        __syncthreads();
    }
    // positions that name no row come last
    if (bucket == kBuckets - 1)
        for (uint32_t i = base + len + tid; i < a.tokens_n; i += kGroupThreads) a.keys[0][i] = kNoRow;
    if (!a.named) return;
    // which of the bucket's rows a token names
    for (uint32_t r = tid; r < width; r += kGroupThreads) a.named[(uint64_t)bucket0 + r] = 0;
    __syncthreads();
    for (uint32_t i = tid; i < len; i += kGroupThreads) {
        const uint32_t row = a.keys[0][base + i];
        if (row < a.rows) a.named[row] = 1;  // always, unless tokens change under the call
    }
}

// ---------------------------------------------------------------- sums
constexpr int kSumThreads = 256;
constexpr uint32_t kZeroRows = 8;  // rows that a workgroup zeroes
constexpr uint32_t kFan = 16;  // pieces of a run that are added up together

// The update of four elements, adam_step's operations in its order (see there for
// the ranges of the short sequences).  n: how many of them exist.
template <bool kMax>
__device__ __forceinline__ void update4(const SumArgs &a, f32x4 &p, f32x4 g, f32x4 &m, f32x4 &v, f32x4 &w, int32_t n) {
    if (a.l2) {
#pragma unroll
        for (int k = 0; k < 4; ++k) g[k] = fmaf(a.wd, p[k], g[k]);
    }
    float m_lo = __builtin_inff(), m_hi = 0.0f, v_lo = __builtin_inff(), v_hi = 0.0f;
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
        v_hi = fmaxf(v_hi, below[k]);
    }
    if (__all(n <= 0 || (a.fast_ok && v_lo >= 0x1p-96f && v_hi < __builtin_inff() && m_lo >= 0x1p-40f && m_hi <= 0x1p40f))) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            p[k] = fmaf(-a.step, div_rn(m[k], fmaf(sqrt_rn(below[k]), a.ibc2, a.eps)), p[k] * a.decay);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            p[k] = fmaf(-a.step, m[k] / fmaf(sqrtf(below[k]), a.ibc2, a.eps), p[k] * a.decay);
    }
}

// What a row's whole sum meets: nothing, the value it is added to, or the
// step's params and state, loaded before the sum so that both are under way
// together.
template <class O, Goal kGoal>
struct Target {
    Four<O> p;
    Four<float> m, v, w;

    __device__ __forceinline__ void load(const SumArgs &a, uint32_t row, uint32_t c0) {
        if constexpr (kGoal == kWrite) return;
        const int32_t left = (int32_t)(a.cols - c0);
        const uint64_t s = (uint64_t)row * a.cols + c0;
        p.template load<true>(reinterpret_cast<const O *>(a.out) + (uint64_t)row * a.out_stride + c0, left);
        if constexpr (kGoal >= kAdam) {
            m.template load<true>(a.m + s, left);
            v.template load<true>(a.v + s, left);
        }
        if constexpr (kGoal == kAdamMax) w.template load<true>(a.w + s, left);
    }

    __device__ __forceinline__ void finish(const SumArgs &a, uint32_t row, uint32_t c0, f32x4 sum) {
        const int32_t left = (int32_t)(a.cols - c0);
        O *to = reinterpret_cast<O *>(a.out) + (uint64_t)row * a.out_stride + c0;
        const uint64_t s = (uint64_t)row * a.cols + c0;
        const f32x4 one = sum * a.scale;
        if constexpr (kGoal == kWrite) {
            store4(to, one, left);
        } else if constexpr (kGoal == kAdd) {
            store4(to, p.wide() + one, left);
        } else {
            f32x4 ps = p.wide(), ms = m.wide(), vs = v.wide(), ws = {};
            if constexpr (kGoal == kAdamMax) ws = w.wide();
            update4<kGoal == kAdamMax>(a, ps, one, ms, vs, ws, left);
            store4(to, ps, left);
            store4(a.m + s, ms, left);
            store4(a.v + s, vs, left);
            if constexpr (kGoal == kAdamMax) store4(a.w + s, ws, left);
        }
    }
};

// sum += the rows at(k) + c0 for k in [from, to), the loads of up to kDeep rows
// under way together (as many batches of kDeep, then at most one each of 8, 4, 2 and 1).
template <int kDeep, class T, class At>
__device__ __forceinline__ void add_rows(f32x4 &sum, uint32_t from, uint32_t to, int32_t left, At at) {
    auto batch = [&](auto size) {
        constexpr int kN = decltype(size)::value;
        Four<T> x[kN];
#pragma unroll
        for (int j = 0; j < kN; ++j) x[j].template load<true>(at(from + j), left);
#pragma unroll
        for (int j = 0; j < kN; ++j) sum += x[j].wide();
        from += kN;
    };
    while (to - from >= (uint32_t)kDeep) batch(Int<kDeep>());
    if constexpr (kDeep > 8)
        if (to - from >= 8) batch(Int<8>());
    if constexpr (kDeep > 4)
        if (to - from >= 4) batch(Int<4>());
    if (to - from >= 2) batch(Int<2>());
    if (to - from >= 1) batch(Int<1>());
}

// Partial sums go to memory and come from it past the XCDs' own caches, by
// device-scope atomic accesses of 8 bytes (a lane's four columns, padding included).
__device__ __forceinline__ void put_partial(float *at, f32x4 x, int32_t n) {
    if (n <= 0) return;
    uint64_t *to = reinterpret_cast<uint64_t *>(at);
    __hip_atomic_store(to, __builtin_bit_cast(uint64_t, (f32x2{x[0], x[1]})), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(to + 1, __builtin_bit_cast(uint64_t, (f32x2{x[2], x[3]})), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x4 get_partial(const float *at, int32_t n) {
    if (n <= 0) return f32x4{0.f, 0.f, 0.f, 0.f};
    const uint64_t *from = reinterpret_cast<const uint64_t *>(at);
    const f32x2 x = __builtin_bit_cast(f32x2, __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    const f32x2 y = __builtin_bit_cast(f32x2, __hip_atomic_load(from + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    return f32x4{x[0], x[1], y[0], y[1]};
}

// Leaves a partial sum in slot `mine` and counts it in at *arrivals; true for
// the wave that comes last of n, which then has their sum, slot_at(0) first,
// slot_at(n - 1) last.
template <class Slot>
__device__ __forceinline__ bool meet(const SumArgs &a, f32x4 &sum, uint64_t mine, uint32_t n, Slot slot_at,
                                     uint32_t *arrivals, uint32_t c0) {
    const int32_t left = (int32_t)(a.cols - c0);
    float *const partials = a.partials + c0;
    put_partial(partials + mine * a.partial_stride, sum, left);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // in memory before it is counted
    uint32_t before = 0;
    if ((threadIdx.x & 63u) == 0)
        before = __hip_atomic_fetch_add(arrivals, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (uniform_u32(before) + 1 != n) return false;
    asm volatile("" ::: "memory");
    sum = f32x4{0.f, 0.f, 0.f, 0.f};
    for (uint32_t k = 0; k < n; k += 4) {
        f32x4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = get_partial(partials + slot_at(min(k + j, n - 1)) * a.partial_stride, left);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (k + j < n) sum += x[j];
    }
    return true;
}

// A workgroup takes a window of 4 kPer positions, each wave kPer of them, in one
// slice of 256 columns (512 columns a wave took 0 to 4% more).  Of the runs (of one row's positions) in the window
//   - those that lie in one wave's positions are summed by it, kBatch positions at a
//     time: their loads, and those of the rows that runs end on (params and state, which
//     come from memory in some 2 us under load), are all issued before the first is used;
//   - a run over several waves' positions is summed by the wave that it begins
//     in, from the others' sums of their first rows (in LDS);
//   - of a run over several windows each leaves a partial sum in memory, and the wave
//     that comes last adds them up in the order of the windows (kFan at a time,
//     then those sums).  No wave waits for another workgroup.
// Bound by memory: for 65536 tokens of 32000 x 4096 (bf16 gradient, words' frequencies, a
// tenth padding) 900 MB in 180 us when added to a table (5.0 TB/s), 2150 MB in 450 us as
// an AMSGrad step (4.8 TB/s; the params and three arrays of state lie in four
// places); for 16384 tokens of 50304 x 2048, 360 MB in 80 us as a step (4.5 TB/s, since the XCDs
// start some us apart and the last windows run alone).  Batches of four positions:
// two take 0 to 3% more.
template <class T, class O, Goal kGoal, int kPer>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(SumArgs a) {
    constexpr uint32_t kWin = 4 * kPer;
    constexpr int kBatch = 4, kDeep = 32 / (int)sizeof(T);
    __shared__ f32x4 leads[4][64];  // what each wave has of a run that began before its positions
    const uint32_t lane = threadIdx.x & 63u, wave = uniform_u32(threadIdx.x >> 6);
    if constexpr (kGoal == kWrite) {
        if (blockIdx.x >= a.sum_groups) {
            // the workgroups behind zero the rows that no token names, while the sums wait for memory
            for (uint64_t r0 = (uint64_t)(blockIdx.x - a.sum_groups) * kZeroRows; r0 < a.rows;
                 r0 += (uint64_t)(gridDim.x - a.sum_groups) * kZeroRows) {
                const uint64_t named = *reinterpret_cast<const uint64_t *>(a.named + r0);  // a byte a row
                zero_rows(reinterpret_cast<O *>(a.out), a.out_stride, a.cols, r0, min(r0 + kZeroRows, (uint64_t)a.rows), kSumThreads,
                          [&](uint64_t r) { return ((named >> (8 * (r - r0))) & 1u) != 0; });
            }
            return;
        }
    }
    // workgroups go to the 8 XCDs in turn: an XCD has all of a window's slices
    const uint64_t units = (a.windows + 7) / 8 * (uint64_t)a.slices * 8;
    for (uint64_t u = blockIdx.x; u < units; u += a.sum_groups) {
        const uint64_t window64 = u / 8 / a.slices * 8 + u % 8;
        if (window64 >= a.windows) continue;
        const uint32_t slice = (uint32_t)(u / 8 % a.slices);
        const uint32_t window = (uint32_t)window64, w0 = window * kWin, end = a.tokens_n - 1;
        // all of them loaded together, at clamped places
        // (order and keys in bounds even where tokens changed under the call)
        const uint32_t key_at = a.keys[min(w0 + lane, end)], from = min(a.order[min(w0 + lane, end)], end);
        const uint32_t last_at = a.keys[w0 > 0 ? w0 - 1 : 0], next_at = a.keys[min(w0 + kWin, end)];
        const uint32_t key = lane < kWin && lane <= end - w0 && key_at < a.rows ? key_at : kNoRow;
        const uint32_t live = (uint32_t)__popcll(__ballot(key != kNoRow));
        if (live == 0) continue;  // padding
        const uint32_t above = __shfl_up(key, 1), prev = lane > 0 ? above : (w0 > 0 ? last_at : kNoRow);
        const uint64_t heads = __ballot(key != kNoRow && key != prev);  // where runs begin
        const uint32_t next = end - w0 >= kWin ? uniform_u32(next_at) : kNoRow;
        // where the run at position h ends in the window
        auto end_of = [&](uint32_t h) {
            const uint64_t after = h + 1 < kWin ? heads >> (h + 1) : 0;
            return after ? h + 1 + (uint32_t)__builtin_ctzll(after) : live;
        };
        // this wave's positions [q0, qe): [q0, body) of a run that began before, then whole runs, and [tail, qe) of one that goes on
        const uint32_t q0 = min(wave * kPer, live), qe = min(q0 + kPer, live);
        const uint64_t in_mine = qe > q0 ? (heads >> q0) & (~0ull >> (64 - (qe - q0))) : 0;
        const uint32_t body = in_mine ? q0 + (uint32_t)__builtin_ctzll(in_mine) : qe;
        uint32_t tail = qe;
        if (in_mine) {
            const uint32_t h = q0 + 63u - (uint32_t)__builtin_clzll(in_mine), e = end_of(h);
            if (e > qe || (e == kWin && lane_u32(key, h) == next)) tail = h;
        }
        auto row_of_key = [&](uint32_t k) { return lane_u32(key, k); };
        const uint32_t c0 = slice * 256 + lane * 4;
        const int32_t left = (int32_t)(a.cols - c0);
        auto row_at = [&](uint32_t k) {
            return reinterpret_cast<const T *>(a.grad) + (uint64_t)lane_u32(from, k) * a.grad_stride + c0;
        };
        f32x4 sum = {};
        if (body > q0) {
            add_rows<kDeep, T>(sum, q0, body, left, row_at);
            leads[wave][lane] = sum;
        }
        for (uint32_t k = body; k < tail; k += kBatch) {
            Four<T> x[kBatch];
            Target<O, kGoal> target[kBatch];
            uint32_t closes = 0;  // positions that a run ends at
#pragma unroll
            for (uint32_t j = 0; j < kBatch; ++j) {
                if (k + j >= tail) continue;
                x[j].template load<true>(row_at(k + j), left);
                if (k + j + 1 == live || ((heads >> (k + j + 1)) & 1u)) {  // (k + j + 1 == 64 only where it is live)
                    closes |= 1u << j;
                    target[j].load(a, row_of_key(k + j), c0);
                }
            }
#pragma unroll
            for (uint32_t j = 0; j < kBatch; ++j) {
                if (k + j >= tail) continue;
                const f32x4 one = x[j].wide();
                sum = (heads >> (k + j)) & 1u ? one : sum + one;
                if ((closes >> j) & 1u) target[j].finish(a, row_of_key(k + j), c0, sum);
            }
        }
        // the run that goes on behind the wave's positions; in the first wave also the one that began before the window
        Target<O, kGoal> target;
        const bool goes_on = tail < qe, crosses = goes_on && end_of(tail) == kWin && next == row_of_key(tail);
        if (goes_on) {
            if (!crosses) target.load(a, row_of_key(tail), c0);
            sum = f32x4{0.f, 0.f, 0.f, 0.f};
            add_rows<kDeep, T>(sum, tail, qe, left, row_at);
        }
        __syncthreads();
        for (uint32_t k = 0; k < 2; ++k) {
            if (!(k == 0 ? goes_on : wave == 0 && body > 0)) continue;
            // k = 0: from this wave's sum; 1: from the first wave's lead
            const uint32_t h = k == 0 ? tail : 0, e = k == 0 ? end_of(h) : (body < qe ? body : end_of(qe - 1)), row = row_of_key(h);
            if (k == 1) sum = f32x4{0.f, 0.f, 0.f, 0.f};
            for (uint32_t w = k == 0 ? wave + 1 : 0; w * kPer < e; ++w) sum += leads[w][lane];
            bool all_in = true;
            if (k == 1 || crosses) {
                // the windows that the run has before this one and after it
                uint32_t earlier = 0, later = 0;
                while (k == 1 && window > earlier) {
                    const uint32_t w = window - earlier;
                    const uint64_t all = __ballot(w > lane && a.keys[(w > lane ? w - lane : 1) * kWin - 1] == row);
                    const uint32_t got = ~all ? (uint32_t)__builtin_ctzll(~all) : 64u;
                    earlier += got;
                    if (got < 64) break;
                }
                while (e == kWin && next == row) {
                    const uint64_t at = (uint64_t)w0 + (uint64_t)(later + 1 + lane) * kWin;
                    const uint64_t all = __ballot(at <= end && a.keys[at <= end ? at : end] == row);
                    const uint32_t got = ~all ? (uint32_t)__builtin_ctzll(~all) : 64u;
                    later += got;
                    if (got < 64) break;
                }
                const uint32_t start = window - earlier, pieces = earlier + 1 + later;
                const uint32_t fan = earlier / kFan, fans = (pieces + kFan - 1) / kFan;
                // the slot of a piece: its window's second where the run began there, else its first
                auto slot_of = [&](uint32_t piece) { return (uint64_t)(start + piece) * 2 + (piece == 0 ? 1 : 0); };
                uint32_t *const counters = a.arrivals + (uint64_t)slice * a.windows * 3;
                all_in = meet(a, sum, slot_of(earlier), min(kFan, pieces - fan * kFan),
                              [&](uint32_t i) { return slot_of(fan * kFan + i); }, counters + slot_of(fan * kFan), c0);
                if (all_in && fans > 1)
                    all_in = meet(a, sum, slot_of(fan * kFan), fans, [&](uint32_t i) { return slot_of(i * kFan); },
                                  counters + (uint64_t)a.windows * 2 + start, c0);
                if (all_in) target.load(a, row, c0);
            }
            if (all_in) target.finish(a, row, c0, sum);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- few tokens
constexpr int kDirectThreads = 512, kDirectWaves = kDirectThreads / 64;

// Up to kDirectTokens tokens in one launch and without a workspace: a workgroup a
// position (and, of few tokens, a share of the columns), which looks through all
// tokens for its row's.  The workgroups of a row's positions share the slices of its
// columns, each of them the positions of a slice among its waves, so that a row
// that many tokens name has many workgroups.  Where the whole gradient is written, the workgroups
// behind zero the rows that no token names, by the same look.
// kLooks: tokens that a thread looks at.
// Chains of dependent loads (tokens, the gradient's rows and the table's side) bound it,
// not bytes: 8 us for 333 tokens of 1000 x 771, written, and for 500 of 32000 x 770 as a step.
template <class Token, class T, class O, Goal kGoal, uint32_t kLooks>
__global__ void __launch_bounds__(kDirectThreads) direct_kernel(SumArgs a, const void *tokens, uint32_t splits, uint32_t zero_rows_each) {
    constexpr int kDeep = 32 / (int)sizeof(T);
    constexpr uint32_t kTokens = kLooks * kDirectThreads, kWords = kTokens / 64;
    __shared__ uint64_t masks[kWords];
    __shared__ uint32_t list[kTokens];
    __shared__ f32x4 parts[kDirectWaves][64];
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = uniform_u32(tid >> 6), n = a.tokens_n;
    const bool zeroes = blockIdx.x >= n * splits;
    const uint32_t i = zeroes ? 0 : blockIdx.x / splits, split = zeroes ? 0 : blockIdx.x % splits;
    const Token *const all = reinterpret_cast<const Token *>(tokens);
    Token token[kLooks], the_token = 0;
    if (n > 0) {  // (it is 0 only where there are rows to zero)
#pragma unroll
        for (uint32_t k = 0; k < kLooks; ++k) token[k] = all[min(k * kDirectThreads + tid, n - 1)];
        the_token = all[i];
    }
    auto row_at = [&](uint32_t k) { return k * kDirectThreads + tid < n ? row_of(token[k], a.rows) : kNoRow; };
    if constexpr (kGoal == kWrite) {
        if (zeroes) {
            uint32_t *const named = list;  // a bitmap
            const uint64_t r0 = (uint64_t)(blockIdx.x - n * splits) * zero_rows_each;
            if (tid < kTokens / 32) named[tid] = 0;
            __syncthreads();
#pragma unroll
            for (uint32_t k = 0; k < kLooks; ++k) {
                const uint32_t row = row_at(k);
                if (row != kNoRow && row >= r0 && row - r0 < zero_rows_each)
                    atomicOr(&named[(row - r0) / 32], 1u << ((row - r0) % 32));
            }
            __syncthreads();
            zero_rows(reinterpret_cast<O *>(a.out), a.out_stride, a.cols, r0, min(r0 + zero_rows_each, (uint64_t)a.rows), kDirectThreads,
                      [&](uint64_t r) { return (named[(r - r0) / 32] >> ((r - r0) % 32)) & 1u; });
            return;
        }
    }
    const uint32_t row = uniform_u32(row_of(the_token, a.rows));
    if (row == kNoRow) return;
    uint64_t same[kLooks];
#pragma unroll
    for (uint32_t k = 0; k < kLooks; ++k) {
        same[k] = __ballot(row_at(k) == row);
        if (lane == 0) masks[k * kDirectWaves + wave] = same[k];
    }
    __syncthreads();
    // the row's positions: how many, and how many before this workgroup's and before each of this wave's words
    const uint64_t word = lane < kWords ? masks[lane] : 0;
    uint32_t incl = (uint32_t)__popcll(word);
#pragma unroll
    for (uint32_t s = 1; s < kWords; s <<= 1) {
        const uint32_t x = __shfl_up(incl, s);
        if (lane >= s) incl += x;
    }
    const uint32_t excl = incl - (uint32_t)__popcll(word);
    const uint32_t count = lane_u32(incl, kWords - 1);
    const uint32_t rank = lane_u32(excl + (uint32_t)__popcll(word & ((1ull << (i % 64)) - 1)), i / 64);
    // this workgroup's slices: s0 + rank, s0 + rank + helpers, .. of the split's [s0, s1)
    const uint32_t per = (a.slices + splits - 1) / splits, s0 = min(a.slices, split * per), s1 = min(a.slices, s0 + per);
    const uint32_t helpers = min(count, s1 - s0);
    if (rank >= helpers) return;
#pragma unroll
    for (uint32_t k = 0; k < kLooks; ++k)
        if ((same[k] >> lane) & 1u)
            list[lane_u32(excl, k * kDirectWaves + wave) + (uint32_t)__popcll(same[k] & ((1ull << lane) - 1))] = k * kDirectThreads + tid;
    __syncthreads();
    const uint32_t have = (s1 - s0 - rank + helpers - 1) / helpers;  // slices, >= 1
    const uint32_t at_once = min(have, (uint32_t)kDirectWaves), shares = kDirectWaves / at_once;
    const uint32_t share = wave / at_once, each = (count + shares - 1) / shares;
    if (count == 1 && share > 0) return;
    for (uint32_t k = wave % at_once; k < have; k += at_once) {  // (once, unless shares is 1)
        const uint32_t c0 = (s0 + rank + k * helpers) * 256 + lane * 4;
        const int32_t left = (int32_t)(a.cols - c0);
        Target<O, kGoal> target;
        if (share == 0) target.load(a, row, c0);
        f32x4 sum = {};
        if (share < shares)
            add_rows<kDeep, T>(sum, min(count, share * each), min(count, (share + 1) * each), left, [&](uint32_t p) {
                return reinterpret_cast<const T *>(a.grad) + (uint64_t)uniform_u32(list[p]) * a.grad_stride + c0;
            });
        if (shares > 1 && count > 1) {
            parts[wave][lane] = sum;
            __syncthreads();
            if (share == 0)
                for (uint32_t p = 1; p < shares; ++p) sum += parts[wave + p * at_once][lane];
        }
        if (share == 0) target.finish(a, row, c0, sum);
    }
}

constexpr uint64_t kMaxGrid = (1u << 24) - 1;  // grid.x * 256 work-items < 2^32
uint32_t grid_of(uint64_t workgroups, uint64_t most = kMaxGrid) { return (uint32_t)std::min<uint64_t>(workgroups, most); }

template <class T, class O, Goal kGoal>
hipError_t launch_sums_of(const SumArgs &a, hipStream_t stream) {
    SumArgs b = a;
    b.sum_groups = grid_of((a.windows + 7) / 8 * (uint64_t)a.slices * 8, kMaxGrid / 2);
    const uint32_t zeros = kGoal == kWrite ? grid_of((a.rows + (uint64_t)kZeroRows - 1) / kZeroRows, kMaxGrid / 2) : 0u;
    const dim3 grid(b.sum_groups + zeros), block(kSumThreads);
    if (a.window == 32) hipLaunchKernelGGL((sum_kernel<T, O, kGoal, 8>), grid, block, 0, stream, b);
    else hipLaunchKernelGGL((sum_kernel<T, O, kGoal, 16>), grid, block, 0, stream, b);
    return hipGetLastError();
}

template <class T, class O, Goal kGoal>
hipError_t launch_direct_of(const SumArgs &a, const void *tokens, bool wide, hipStream_t stream) {
    // the rows to zero: 64 KB and more a workgroup, over some 1024 of them, but no more rows than its bitmap has
    const uint64_t each64 = std::max<uint64_t>(a.rows / 1024 + 1, 65536 / std::max<uint64_t>(a.cols * sizeof(O), 1));
    const uint32_t each = (uint32_t)std::min<uint64_t>(each64, kFewTokens);
    const uint32_t zeros = kGoal == kWrite ? (a.rows + each - 1) / each : 0u;
    const uint32_t splits = a.tokens_n == 0 ? 1u : std::min(a.slices, std::max(1u, 1024u / a.tokens_n));
    const dim3 grid(a.tokens_n * splits + zeros), block(kDirectThreads);
    constexpr uint32_t kFew = kFewTokens / kDirectThreads, kMore = kDirectTokens / kDirectThreads;
    const bool few = a.tokens_n <= kFewTokens;
    if (wide && few) hipLaunchKernelGGL((direct_kernel<uint64_t, T, O, kGoal, kFew>), grid, block, 0, stream, a, tokens, splits, each);
    else if (wide) hipLaunchKernelGGL((direct_kernel<uint64_t, T, O, kGoal, kMore>), grid, block, 0, stream, a, tokens, splits, each);
    else if (few) hipLaunchKernelGGL((direct_kernel<uint32_t, T, O, kGoal, kFew>), grid, block, 0, stream, a, tokens, splits, each);
    else hipLaunchKernelGGL((direct_kernel<uint32_t, T, O, kGoal, kMore>), grid, block, 0, stream, a, tokens, splits, each);
    return hipGetLastError();
}

template <class T> struct Type { typedef T type; };

// launch(gradient's type, result's type, goal) for the forms that there are.
template <class Launch>
hipError_t by_types(bool grad_bf16, bool out_bf16, Goal goal, Launch launch) {
    auto with = [&](auto o, auto g) { return grad_bf16 ? launch(Type<uint16_t>(), o, g) : launch(Type<float>(), o, g); };
    switch (goal) {
    case kWrite: return out_bf16 ? with(Type<uint16_t>(), Int<kWrite>()) : with(Type<float>(), Int<kWrite>());
    case kAdd: return out_bf16 ? with(Type<uint16_t>(), Int<kAdd>()) : with(Type<float>(), Int<kAdd>());
    case kAdam: return with(Type<float>(), Int<kAdam>());
    default: return with(Type<float>(), Int<kAdamMax>());
    }
}

template <class T, class O>
hipError_t launch_lookup_of(const LookupArgs &a, hipStream_t stream) {
    const uint32_t slices = (a.cols + 511) / 512;
    const uint64_t units = (uint64_t)a.tokens_n * slices;
    const dim3 grid(grid_of((units + 3) / 4));
    if (a.wide) hipLaunchKernelGGL((lookup_kernel<T, O, uint64_t>), grid, dim3(kLookupThreads), 0, stream, a, slices, units);
    else hipLaunchKernelGGL((lookup_kernel<T, O, uint32_t>), grid, dim3(kLookupThreads), 0, stream, a, slices, units);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lookup(bool table_bf16, bool out_bf16, const LookupArgs &a, hipStream_t stream) {
    if (table_bf16)
        return out_bf16 ? launch_lookup_of<uint16_t, uint16_t>(a, stream) : launch_lookup_of<uint16_t, float>(a, stream);
    return out_bf16 ? launch_lookup_of<float, uint16_t>(a, stream) : launch_lookup_of<float, float>(a, stream);
}

hipError_t launch_group(const GroupArgs &a, hipStream_t stream) {
    const size_t lds = (size_t)kGroupWaves * (kListed * sizeof(uint2) + (4u << a.bits));
    if (a.wide) hipLaunchKernelGGL(group_kernel<uint64_t>, dim3(kBuckets), dim3(kGroupThreads), lds, stream, a);
    else hipLaunchKernelGGL(group_kernel<uint32_t>, dim3(kBuckets), dim3(kGroupThreads), lds, stream, a);
    return hipGetLastError();
}

hipError_t launch_sums(bool grad_bf16, bool out_bf16, Goal goal, const SumArgs &a, hipStream_t stream) {
    return by_types(grad_bf16, out_bf16, goal, [&](auto t, auto o, auto g) {
        return launch_sums_of<typename decltype(t)::type, typename decltype(o)::type, (Goal)decltype(g)::value>(a, stream);
    });
}

hipError_t launch_direct(bool grad_bf16, bool out_bf16, Goal goal, const SumArgs &a, const void *tokens, bool wide,
                         hipStream_t stream) {
    return by_types(grad_bf16, out_bf16, goal, [&](auto t, auto o, auto g) {
        return launch_direct_of<typename decltype(t)::type, typename decltype(o)::type, (Goal)decltype(g)::value>(a, tokens, wide,
                                                                                                               stream);
    });
}

}  // namespace adam_mi355x
