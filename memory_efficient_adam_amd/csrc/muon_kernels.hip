// Muon on gfx950 (MI355X): the momentum update and the Newton-Schulz
// orthogonalisation of its result.
//
// The orthogonalisation is matrix products: per iteration A = X X^T,
// P = a I + b A + c A^2 and X <- P X, with X short x long (m x n).  They run
// on the fp16 matrix cores at fp32's accuracy: a factor is held as
// hi + 2^-11 lo, two fp16 values (22 bits), and hi hi + 2^-11 (hi lo + lo hi) is
// summed in fp32 (what is left out is below 2^-22 of the product).  Three fp16
// products cost a quarter of what the fp32 matrix instructions take for one.
// The factors are scaled by a power of two (X and A by 2^10, P by 2^8), and the
// remainder by 2^11 once more, so that no part of an entry that matters falls
// below fp16's range: an entry of X of 2^-24 still has all 22 bits, smaller ones
// an error of 2^-46.  One entry or column that holds nearly all of a matrix's
// norm leaves the others that small, and the iterations then grow them by the
// product of the a_k (485): with remainders in the scale of the high parts
// (errors of 2^-35 from 2^-13 down) such a matrix of 520 x 1600 was off by
// 1e-5, the small entries by up to 7e-3 of themselves.  The price is a sum of
// its own for the scaled products.  A and P are symmetric:
// only tiles on and below the diagonal are computed, and stored twice.  The
// term a X is a I in P, so that an update reads X once, as a factor.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "muon_internal.h"

namespace adam_mi355x {
namespace {

constexpr float kTiny = 0x1p-112f;  // smallest block maximum that is encoded (8-bit momentum)
constexpr float kScaleX = 1024.0f;  // X and A are held times 2^10
constexpr float kScaleP = 256.0f;   // P is held times 2^8
constexpr float kScaleLo = 2048.0f, kUnscaleLo = 1.0f / kScaleLo;  // remainders are held times 2^11 besides

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- small helpers
__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __uint_as_float(h << 16); }

// Round to nearest, ties to even, on the upper 16 bits; NaN -> 0x7FC0.
__device__ __forceinline__ uint32_t f32_to_bf16(float x) {
    if (x != x) return 0x7FC0u;
    const uint32_t u = __float_as_uint(x);
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

template <bool kBf16>
__device__ __forceinline__ float load_elem(const void *p, uint64_t i) {
    if constexpr (kBf16)
        return bf16_to_f32(static_cast<const uint16_t *>(p)[i]);
    else
        return static_cast<const float *>(p)[i];
}

// Two fp32 values as hi + 2^-11 lo each, packed: the sums hold 22 bits.  Pairs
// are converted in one instruction (to nearest even), and a remainder y - hi
// (exact, at most half of hi's last place: 2^11 times it stays in range) is one
// mixed-precision fma, which the compiler does not form by itself.
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void split2(float y0, float y1, uint32_t &hi, uint32_t &lo) {
    const half2v h = __builtin_convertvector((f32x2{y0, y1}), half2v);
    hi = __builtin_bit_cast(uint32_t, h);
    float r0, r1;
    asm("v_fma_mix_f32 %0, -%1, 1.0, %2 op_sel:[0,0,0] op_sel_hi:[1,0,0]" : "=v"(r0) : "v"(hi), "v"(y0));
    asm("v_fma_mix_f32 %0, -%1, 1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(r1) : "v"(hi), "v"(y1));
    const half2v l = __builtin_convertvector((f32x2{r0 * kScaleLo, r1 * kScaleLo}), half2v);
    lo = __builtin_bit_cast(uint32_t, l);
}
__device__ __forceinline__ void split4(float y0, float y1, float y2, float y3, u32x2 &hi, u32x2 &lo) {
    uint32_t h0, h1, l0, l1;
    split2(y0, y1, h0, l0);
    split2(y2, y3, h1, l1);
    hi = u32x2{h0, h1};
    lo = u32x2{l0, l1};
}
// Eight values as fragments.
__device__ __forceinline__ void split8(const float (&y)[8], half8 &hi, half8 &lo) {
    u32x4 h, l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a, b;
        split2(y[2 * i], y[2 * i + 1], a, b);
        h[i] = a;
        l[i] = b;
    }
    hi = __builtin_bit_cast(half8, h);
    lo = __builtin_bit_cast(half8, l);
}

// The value that an entry's high part and remainder stand for.
__device__ __forceinline__ float join(uint32_t hi, uint32_t lo) {
    return fmaf((float)__builtin_bit_cast(_Float16, (uint16_t)lo), kUnscaleLo, (float)__builtin_bit_cast(_Float16, (uint16_t)hi));
}

// Sum over the workgroup's kWaves waves in a fixed order (s: kWaves doubles).
template <int kWaves = 4>
__device__ __forceinline__ double block_sum(double x, double *s) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
    __syncthreads();
    double sum = s[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) sum += s[i];
    return sum;
}

// Consecutive tiles share factor rows, and workgroups are dealt to the 8 XCDs
// (each with an L2 of its own) in turn: workgroup id takes the tile that
// keeps each XCD on one run of consecutive tiles in each window of 2^window.
__device__ __forceinline__ uint32_t xcd_order(uint32_t id, uint32_t n, uint32_t window) {
    const uint32_t base = id >> window << window;
    const uint32_t in = id - base, count = ((n - base) >> window) ? 1u << window : n - base;
    const uint32_t xcd = in & 7u, per = count >> 3, rest = count & 7u;
    return base + xcd * per + min(xcd, rest) + (in >> 3);
}

typedef const __attribute__((address_space(4))) BlockDesc *ConstDescPtr;
typedef const __attribute__((address_space(4))) TensorRef *ConstTensorPtr;
typedef const __attribute__((address_space(4))) uint64_t *ConstU64Ptr;

// The matrix of a launch and, in t, the index of the tile within it (alike
// matrices) or its packed row and column blocks (table).
__device__ __forceinline__ MuonMat find_mat(const MuonWork &w, uint32_t id, uint32_t &t) {
    MuonMat m;
    if (w.tiles) {
        // (word by word through the constant address space: scalar loads)
        const uint64_t e = ((ConstU64Ptr)w.tiles)[id];
        const ConstU64Ptr p = (ConstU64Ptr)w.mats + (uint32_t)e * (uint32_t)(sizeof(MuonMat) / 8);
        t = (uint32_t)(e >> 32);
        uint64_t words[sizeof(MuonMat) / 8];
#pragma unroll
        for (uint32_t i = 0; i < sizeof(MuonMat) / 8; ++i) words[i] = p[i];
        __builtin_memcpy(&m, words, sizeof(m));
    } else {
        const uint32_t k = id / w.per_mat;
        t = id - k * w.per_mat;
        m = w.one;
        m.x_off += k * w.x_stride;
        m.a_off += k * w.a_stride;
        m.u_off += k * w.u_stride;
        m.o_off += k * w.o_stride;
        m.norm += k * w.norm_stride;
        m.index = k;
    }
    return m;
}

// Tile t of a lower triangle, row by row: ti >= tj.
__device__ __forceinline__ void triangle(uint32_t t, uint32_t &ti, uint32_t &tj) {
    uint32_t r = (uint32_t)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (r * (r + 1u) / 2u > t) --r;
    while ((r + 1u) * (r + 2u) / 2u <= t) ++r;
    ti = r;
    tj = t - r * (r + 1u) / 2u;
}

// Tile t of an mb x nb grid of tiles, in bands of 8 tile rows taken column by column:
// the workgroups of an XCD that run together then share both factors' rows.
__device__ __forceinline__ void banded(uint32_t t, uint32_t mb, uint32_t nb, uint32_t &ti, uint32_t &tj) {
    const uint32_t band = t / (8u * nb), first = band * 8u, high = min(8u, mb - first), in = t - band * 8u * nb;
    ti = first + in % high;
    tj = in / high;
}

// ---------------------------------------------------------------- images
// Byte position of element (row r, k) in an image whose rows hold `length`
// elements, for k a multiple of 4 (four elements lie side by side); remainders
// (split form) are 1 KB on.
template <int kForm>
constexpr uint32_t slab_length() { return kForm == kPlain ? 64u : 32u; }
template <int kForm>
__device__ __forceinline__ uint64_t image_pos(uint32_t r, uint32_t k, uint32_t length) {
    constexpr uint32_t kPer = slab_length<kForm>();
    const uint32_t fragment = ((k % kPer) >> 4) * (kForm == kPlain ? 1u : 2u);
    return ((uint64_t)(r >> 5) * (length / kPer) + k / kPer) * 4096u + fragment * 1024u +
           ((r & 31u) + (((k >> 3) & 1u) << 5)) * 16u + (k & 7u) * 2u;
}
constexpr uint32_t kRemainder = 1024u;

// ---------------------------------------------------------------- products
// How a product's result is cut: kRows x kCols tiles, each by a workgroup of
// kDown x kAcross waves, with kStages slabs of the factors in LDS.
template <int R, int C, int D, int A, int S, int W>
struct Tiling {
    static constexpr int kRows = R, kCols = C, kDown = D, kAcross = A, kStages = S;
    static constexpr int kWaves = D * A, kThreads = 64 * kWaves;
    static constexpr int kI = R / D / 32, kJ = C / A / 32;         // a wave's 32 x 32 blocks
    static constexpr int kStage = (R + C) * 128;                   // bytes of a slab of both factors
    // bytes of a slab of the right factor to 32 rows (mixed: half a plain slab,
    // as long as a split one), and the 1 KB pieces a wave fetches per slab
    static constexpr int right_bytes(int form) { return form == kMixed ? 2048 : 4096; }
    static constexpr int loads(int form) { return (R / 32 * 4096 + C / 32 * right_bytes(form)) / 1024 / kWaves; }
    static constexpr int kPerSimd = W;                             // waves per SIMD it is compiled for
    static_assert((R * 128 + C * 64) % (1024 * kWaves) == 0 && C * 64 % (1024 * kWaves) == 0, "every wave fetches as much");
};

// 16 bytes per lane from memory straight to LDS: lane i's go to base + 16 i.
__device__ __forceinline__ void dma16(const char *g, char *base) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)g,
                                     (__attribute__((address_space(3))) void *)base, 16, 0, 0);
}

// Waits until at most kLeft of the wave's fetches are under way and all of its
// LDS reads are done, then for the workgroup's other waves to get there.  (In
// assembly because __syncthreads() would wait for every fetch; the memory
// clobber keeps the compiler's own reads and fetches on their side of it.)
template <int kLeft>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(kLeft) : "memory");
}

template <class T, int kForm>
struct Sources {
    const char *at[T::loads(kForm)];  // this wave's pieces of the next slab
    uint32_t step[T::loads(kForm)];   // to those of the slab after it
};

template <class T, int kForm>
__device__ __forceinline__ void fetch(Sources<T, kForm> &src, char *stage, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < T::loads(kForm); ++i) {
        dma16(src.at[i] + lane * 16, stage + (wave * T::loads(kForm) + i) * 1024);
        src.at[i] += src.step[i];
    }
}

// rd and wr are different stages of LDS: without that promise the compiler
// would wait for the fetches before every read.
template <class T, int kForm>
__device__ __forceinline__ void slab(f32x16 (&acc)[T::kI][T::kJ], f32x16 (&cross)[T::kI][T::kJ], const char *__restrict rd, char *__restrict wr,
                                     Sources<T, kForm> &src, bool more, int wave, int lane) {
    constexpr int kSteps = kForm == kPlain ? 4 : 2;
    constexpr int kRight = T::right_bytes(kForm);
    if (more) fetch<T, kForm>(src, wr, wave, lane);
    const char *left = rd + (wave / T::kAcross) * (T::kI * 4096) + lane * 16;
    const char *right = rd + T::kRows * 128 + (wave % T::kAcross) * (T::kJ * kRight) + lane * 16;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        half8 l[T::kI], r[T::kJ], l2[T::kI], r2[T::kJ];
        const int at = k * (kForm == kPlain ? 1024 : 2048), at_r = k * (kForm == kSplit ? 2048 : 1024);
#pragma unroll
        for (int i = 0; i < T::kI; ++i) {
            l[i] = *reinterpret_cast<const half8 *>(left + i * 4096 + at);
            if constexpr (kForm != kPlain) l2[i] = *reinterpret_cast<const half8 *>(left + i * 4096 + at + kRemainder);
        }
#pragma unroll
        for (int j = 0; j < T::kJ; ++j) {
            r[j] = *reinterpret_cast<const half8 *>(right + j * kRight + at_r);
            if constexpr (kForm == kSplit) r2[j] = *reinterpret_cast<const half8 *>(right + j * kRight + at_r + kRemainder);
        }
#pragma unroll
        for (int i = 0; i < T::kI; ++i)
#pragma unroll
            for (int j = 0; j < T::kJ; ++j) {
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(l[i], r[j], acc[i][j], 0, 0, 0);
                if constexpr (kForm == kSplit)
                    cross[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(l[i], r2[j], cross[i][j], 0, 0, 0);
                if constexpr (kForm != kPlain)
                    cross[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(l2[i], r[j], cross[i][j], 0, 0, 0);
            }
    }
}

// sum = left right^T over `slabs` slabs (left, right: the tile's first slab;
// *_block: bytes from one 32-row block to the next), summed in runs of some
// kRun slabs: one sum that took every term of a long row in turn would
// lose more to fp32's rounding than the split factors do.  (The products with
// remainders, 2^-11 of the others, are one sum.)  kStages - 1 slabs
// are under way to LDS while the matrix cores work on one; at the barrier
// before slab s, its fetches are done and every wave has read slab s - 1,
// whose place the next fetch takes.
constexpr uint32_t kRun = 8;

template <class T, int kForm>
__device__ __forceinline__ void product(f32x16 (&sum)[T::kI][T::kJ], const char *left, uint64_t left_block,
                                        const char *right, uint64_t right_block, uint32_t slabs, char *lds) {
    constexpr int kS = T::kStages;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    Sources<T, kForm> src;
#pragma unroll
    for (int i = 0; i < T::loads(kForm); ++i) {
        // pieces: the left factor's, 4 to 32 rows, then the right one's, 4 or 2
        constexpr uint32_t kLeft = T::kRows / 8, kTo = T::right_bytes(kForm) / 1024;
        const uint32_t piece = wave * T::loads(kForm) + i, q = piece - kLeft;
        const bool is_left = piece < kLeft;
        src.at[i] = is_left ? left + (piece / 4u) * left_block + (piece % 4u) * 1024u
                            : right + (q / kTo) * right_block + (q % kTo) * 1024u;
        src.step[i] = is_left ? 4096u : (uint32_t)T::right_bytes(kForm);
    }
#pragma unroll
    for (int s = 0; s < kS - 1; ++s)
        if (s < (int)slabs) fetch<T, kForm>(src, lds + s * T::kStage, wave, lane);
    f32x16 acc[T::kI][T::kJ], cross[T::kI][T::kJ];
#pragma unroll
    for (int i = 0; i < T::kI; ++i)
#pragma unroll
        for (int j = 0; j < T::kJ; ++j) sum[i][j] = acc[i][j] = cross[i][j] = f32x16{};
    for (uint32_t s0 = 0; s0 < slabs; s0 += kS) {
#pragma unroll
        for (int u = 0; u < kS; ++u) {
            const uint32_t s = s0 + u;
            if (s >= slabs) break;
            if (s + (kS - 2) < slabs) wait_and_meet<(kS - 2) * T::loads(kForm)>();
            else wait_and_meet<0>();
            slab<T, kForm>(acc, cross, lds + u * T::kStage, lds + ((u + kS - 1) % kS) * T::kStage, src, s + (kS - 1) < slabs, wave,
                           lane);
        }
        if (s0 % kRun + kS >= kRun || s0 + kS >= slabs) {
#pragma unroll
            for (int i = 0; i < T::kI; ++i)
#pragma unroll
                for (int j = 0; j < T::kJ; ++j) {
                    sum[i][j] += acc[i][j];
                    acc[i][j] = f32x16{};
                }
        }
    }
    if constexpr (kForm != kPlain)
#pragma unroll
        for (int i = 0; i < T::kI; ++i)
#pragma unroll
            for (int j = 0; j < T::kJ; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[i][j][e] = fmaf(cross[i][j][e], kUnscaleLo, sum[i][j][e]);
}

// Four values down the rows of one column per lane -> four along a row: a
// 4 x 4 transpose of 16-bit values over each quad of lanes (two exchanges
// with the neighbouring lanes).  In: d = rows 0..3 of column lane % 4; out:
// columns 0..3 of row lane % 4.
__device__ __forceinline__ u32x2 quad_transpose(u32x2 d, uint32_t lane) {
    const uint32_t n0 = (uint32_t)__builtin_amdgcn_mov_dpp((int)d.x, 0xB1, 0xF, 0xF, true);
    const uint32_t n1 = (uint32_t)__builtin_amdgcn_mov_dpp((int)d.y, 0xB1, 0xF, 0xF, true);
    // even lane: {own low, neighbour's low}; odd: {neighbour's high, own high}
    // (v_perm_b32: selector bytes 0..3 take the second operand's bytes, 4..7 the first's)
    const uint32_t sel = (lane & 1u) ? 0x03020706u : 0x05040100u;
    const uint32_t e0 = __builtin_amdgcn_perm(n0, d.x, sel), e1 = __builtin_amdgcn_perm(n1, d.y, sel);
    const uint32_t m0 = (uint32_t)__builtin_amdgcn_mov_dpp((int)e0, 0x4E, 0xF, 0xF, true);
    const uint32_t m1 = (uint32_t)__builtin_amdgcn_mov_dpp((int)e1, 0x4E, 0xF, 0xF, true);
    return (lane & 2u) ? u32x2{m1, e1} : u32x2{e0, m0};
}

// A store that goes on to memory at once instead of staying in the XCD's L2,
// to be written back when the kernel ends: the factors are read next by
// other XCDs (eight matrices of 500 x 600: 215 -> 201 us).
__device__ __forceinline__ void store_through(char *at, u32x2 v) {
    __hip_atomic_store(reinterpret_cast<uint64_t *>(at), __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}

// Where in a block's piece of an image the four values 4 g .. 4 g + 3 of a
// lane go, from the place of g = 0: along the rows (values of a column are
// elements of the transposed image) or, after quad_transpose, down them.
constexpr uint32_t along(int g) { return (uint32_t)(g >> 1) * 2048u + (uint32_t)(g & 1) * 512u; }
constexpr uint32_t down(int g) { return (uint32_t)g * 128u; }

// A 32 x 32 block of values, at rows r0.. and columns c0.., into a split image whose
// rows hold `length` elements and, transposed, into one with `length_t` (either may be NULL).
__device__ __forceinline__ void store_block(const f32x16 &v, char *image, uint32_t length, char *transposed, uint32_t length_t,
                                            uint32_t r0, uint32_t c0, uint32_t lane) {
    const uint32_t r = r0 + 4u * (lane >> 5), c = c0 + (lane & 31u);
    char *const at = image + image_pos<kSplit>(r + (lane & 3u), c & ~3u, length);
    char *const at_t = transposed + image_pos<kSplit>(c, r, length_t);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        u32x2 h, l;
        split4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3], h, l);
        if (transposed) {
            store_through(at_t + along(g), h);
            store_through(at_t + along(g) + kRemainder, l);
        }
        if (image) {
            store_through(at + down(g), quad_transpose(h, lane));
            store_through(at + down(g) + kRemainder, quad_transpose(l, lane));
        }
    }
}

// The sums of a split tile's parts, in the order of the parts: true for the
// workgroup that comes last (it has them in acc), false for the others.  No
// workgroup waits for another: each leaves its own sums in memory, counts
// itself in once they are there, and the one that finds all others counted
// reads them.  Sums and counters go through device-scope atomic stores and
// loads, which the XCDs' L2 caches pass on and fetch anew; with fences for the
// whole device instead, each of which writes back and drops an XCD's L2, a
// 2048 x 2048 orthogonalisation took 2851 us instead of 769 unsplit.
template <class T>
__device__ __forceinline__ bool sum_parts(f32x16 (&acc)[T::kI][T::kJ], const MuonWork &w, uint32_t tile, uint32_t part,
                                          uint32_t wave, uint32_t lane, uint32_t *shared) {
    constexpr uint32_t kPairs = T::kRows * T::kCols / 2;
    uint64_t *all = reinterpret_cast<uint64_t *>(w.partial) + (uint64_t)tile * w.parts * kPairs +
                    wave * (T::kI * T::kJ * 8u * 64u) + lane;
#pragma unroll
    for (int i = 0; i < T::kI; ++i)
#pragma unroll
        for (int j = 0; j < T::kJ; ++j)
#pragma unroll
            for (int g = 0; g < 8; ++g)
                __hip_atomic_store(all + (uint64_t)part * kPairs + ((i * T::kJ + j) * 8 + g) * 64,
                                   __builtin_bit_cast(uint64_t, (f32x2{acc[i][j][2 * g], acc[i][j][2 * g + 1]})),
                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // every wave's stores are acknowledged before the workgroup is counted
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (threadIdx.x == 0) {
        const uint32_t before = __hip_atomic_fetch_add(&w.arrived[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (before + 1u == w.parts)  // for the next launch
            __hip_atomic_store(&w.arrived[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        shared[0] = before;
    }
    __syncthreads();
    if (shared[0] + 1u != w.parts) return false;
#pragma unroll
    for (int i = 0; i < T::kI; ++i)
#pragma unroll
        for (int j = 0; j < T::kJ; ++j) acc[i][j] = f32x16{};
    for (uint32_t p = 0; p < w.parts; ++p)
#pragma unroll
        for (int i = 0; i < T::kI; ++i)
#pragma unroll
            for (int j = 0; j < T::kJ; ++j)
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    const f32x2 v = __builtin_bit_cast(
                        f32x2, __hip_atomic_load(all + (uint64_t)p * kPairs + ((i * T::kJ + j) * 8 + g) * 64, __ATOMIC_RELAXED,
                                                 __HIP_MEMORY_SCOPE_AGENT));
                    acc[i][j][2 * g] += v.x;
                    acc[i][j][2 * g + 1] += v.y;
                }
    return true;
}

// The tiles of one product over all matrices of a launch.
//   kGram:       A = X X^T                        tiles ti >= tj, stored at both places
//   kPolynomial: P = a I + b A + c A A^T          the same
//   kCommuting:  a product of two polynomials in one A (symmetric too), or
//                two such products in one launch; one factor is a P
//   kUpdate:     X' = P X, stored as X' and X'^T
//   kLast..:     O = P X in the user's orientation (for a tall matrix the
//                factors change places), rounded to the output's type, or
//                applied to the params
template <class T, int kProduct, int kIn>
__global__ __launch_bounds__(T::kThreads) __attribute__((amdgpu_waves_per_eu(T::kPerSimd)))
void muon_product_kernel(MuonGemmArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[T::kStages * T::kStage];
    constexpr bool kLast = kProduct >= kLastBf16;
    constexpr bool kSquare = kProduct == kGram || kProduct == kPolynomial || kProduct == kCommuting;
    uint32_t t, ti, tj;
    // workgroups: the whole tiles of the first product and of the second, then
    // the parts of the others
    const uint32_t whole = a.work.n_whole, jobs = a.left2 ? 2u : 1u;
    uint32_t id = blockIdx.x, part = 0, parts = 1;
    bool second = false;
    if (id < whole * jobs) {
        second = id >= whole;
        id = xcd_order(second ? id - whole : id, whole, a.work.window);
    } else {
        parts = a.work.parts;
        const uint32_t rest = (a.work.n_tiles - whole) * parts;
        id -= whole * jobs;
        second = id >= rest;
        id = xcd_order(second ? id - rest : id, rest, a.work.window);
        part = id % parts;
        id = whole + id / parts;
    }
    const MuonMat m = find_mat(a.work, id, t);
    if (a.work.tiles) {
        ti = t & 0xFFFFu;
        tj = t >> 16;
    } else if constexpr (kSquare) {
        triangle(t, ti, tj);
    } else {
        const uint32_t across = (kLast && m.tall) ? T::kRows : T::kCols, down = (kLast && m.tall) ? T::kCols : T::kRows;
        banded(t, m.mp / down, m.np / across, ti, tj);
    }
    const uint32_t k = kProduct == kGram ? m.np : m.mp;  // length of the products
    // bytes of 32 rows of either factor
    const uint64_t block = (uint64_t)(k / slab_length<kIn>()) * 4096u;
    const uint64_t right_block = kIn == kMixed ? (uint64_t)(k / 64u) * 4096u : block;
    const char *left, *right;
    uint32_t row0, col0;  // of the result
    if constexpr (kSquare) {
        const char *f = a.left, *g = a.left;
        if constexpr (kProduct == kCommuting) {
            f = second ? a.left2 : a.left;
            g = second ? a.right2 : a.right;
        }
        const uint64_t off = kProduct == kGram ? m.x_off : m.a_off;
        row0 = ti * T::kRows;
        col0 = tj * T::kCols;
        left = f + off + (row0 >> 5) * block;
        right = g + off + (col0 >> 5) * block;
    } else {
        const bool swap = kLast && m.tall;
        row0 = (swap ? tj : ti) * T::kRows;
        col0 = (swap ? ti : tj) * T::kCols;
        const char *p = a.left + m.a_off, *x = a.right + m.x_off;
        static_assert(kIn != kMixed || kProduct == kUpdate, "no exchange of mixed factors");
        left = (swap ? x : p) + (row0 >> 5) * block;
        right = (swap ? p : x) + (col0 >> 5) * right_block;
    }
    const uint32_t slabs = k / slab_length<kIn>(), first = slabs * part / parts, last = slabs * (part + 1) / parts;
    f32x16 acc[T::kI][T::kJ];
    product<T, kIn>(acc, left + (uint64_t)first * 4096u, block,
                    right + (uint64_t)first * (uint32_t)T::right_bytes(kIn), right_block, last - first, lds);

    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (parts > 1) {
        const uint32_t tile = id - whole + (second ? a.work.n_tiles - whole : 0u);
        if (!sum_parts<T>(acc, a.work, tile, part, wave, lane, reinterpret_cast<uint32_t *>(lds))) return;
    }
    row0 += (wave / T::kAcross) * (T::kI * 32);
    col0 += (wave % T::kAcross) * (T::kJ * 32);
    // a raw X_0's factor is made up for here: once in an update, twice in X X^T
    const float phi = (kProduct == kGram || kProduct == kUpdate) && a.phi ? a.phi[m.index] : 1.0f;
    float *param = nullptr;
    float step = 0.0f;
    if constexpr (kProduct == kLastParams) {
        param = ((ConstTensorPtr)a.tensors + m.index)->p;
        step = (float)(a.lr * (a.scale == 1 ? m.scale_spectral : (a.scale == 2 ? m.scale_rms : 1.0)));
    }
#pragma unroll
    for (int i = 0; i < T::kI; ++i)
#pragma unroll
        for (int j = 0; j < T::kJ; ++j) {
            f32x16 v = acc[i][j];
            const uint32_t r0 = row0 + 32u * i, c0 = col0 + 32u * j;
            const uint32_t r = r0 + 4u * (lane >> 5), c = c0 + (lane & 31u);
            if constexpr (kSquare) {
                char *out = (second ? a.out2 : a.out) + m.a_off;
                if constexpr (kProduct == kGram) {
                    v *= phi * phi * (1.0f / kScaleX);
                } else if constexpr (kProduct == kCommuting) {
                    v *= 1.0f / kScaleP;
                } else {
                    // A's block, read from its mirror image: four values down a column lie side by side
                    const float cb = a.cb * (kScaleP / kScaleX), cc = a.cc * (kScaleP / (kScaleX * kScaleX));
                    const float ca = a.ca * kScaleP;
                    const char *const base = a.add + m.a_off + image_pos<kSplit>(c, r, m.mp);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const char *at = base + along(g);
                        const u32x2 h = *reinterpret_cast<const u32x2 *>(at);
                        const u32x2 l = *reinterpret_cast<const u32x2 *>(at + kRemainder);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t hw = q < 2 ? h.x : h.y, lw = q < 2 ? l.x : l.y;
                            const float av = join(hw >> (16 * (q & 1)), lw >> (16 * (q & 1)));
                            float x = fmaf(cb, av, cc * v[4 * g + q]);
                            if (r + 8u * g + q == c) x += ca;
                            v[4 * g + q] = x;
                        }
                    }
                }
                store_block(v, ti != tj ? out : nullptr, m.mp, out, m.mp, r0, c0, lane);
            } else if constexpr (kProduct == kUpdate) {
                v *= phi * (1.0f / kScaleP);
                store_block(v, a.out + m.x_off, m.np, a.out_t + m.x_off, m.mp, r0, c0, lane);
            } else {
                constexpr float kUnscale = 1.0f / (kScaleX * kScaleP);
                float old[16];
                if constexpr (kProduct == kLastParams) {  // all of the block's params at once, then the stores
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const uint32_t q = r + 8u * (e / 4) + (e & 3);
                        old[e] = param[q < m.rows && c < m.cols ? (uint64_t)q * m.cols + c : 0u];
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t q = r + 8u * (e / 4) + (e & 3);
                    if (q >= m.rows || c >= m.cols) continue;
                    const float o = v[e] * kUnscale;
                    if constexpr (kProduct == kLastParams) param[(uint64_t)q * m.cols + c] = fmaf(-step, o, old[e] * a.decay);
                    else if constexpr (kProduct == kLastBf16)
                        static_cast<uint16_t *>(a.o)[m.o_off + q * m.o_ld + c] = (uint16_t)f32_to_bf16(o);
                    else static_cast<float *>(a.o)[m.o_off + q * m.o_ld + c] = o;
                }
            }
        }
}

// ---------------------------------------------------------------- small matrices
// A whole orthogonalisation in one workgroup of 8 waves, X staying in
// registers, in one launch: 25 us for an fp32 matrix of 48 x 80 (one launch per
// product, 69), 85 us for 96 of 64 x 768 in bf16 (250).
//
// A wave holds blocks of 32 columns of X, block w + 8 b at wave w, as the
// matrix cores give them: lane l holds column l % 32, rows 8 g + 4 (l / 32) + q
// of each 32-row block in element 4 g + q.  Taken as a factor with k along the
// rows, eight such elements are one fragment whose k runs in the order
//   order(j, half) = j < 4 ? 4 half + j : 8 + 4 half + j - 4,
// which is as good as any as long as the other factor keeps to it.  So, with P
// stored in that order,
//   P X   = mfma(P, X)  gives the next X in the same arrangement, and
//   X^T P = mfma(X, P)  gives it transposed: lane = row of X, k along columns,
// which is what A = X X^T takes for both factors.  Nothing of X passes through
// LDS; the price is that P X is computed twice.  A is summed over the waves in LDS.
constexpr int kSmallWaves = 8;

__device__ __forceinline__ uint32_t k_order(uint32_t j, uint32_t half) { return (j & 3u) + 4u * half + ((j & 4u) << 1); }

// Square matrices in LDS: high parts and remainders, rows of 128 bytes whose
// 16-byte chunk 2 s + half holds elements 16 s + order(0..7, half).
struct SmallSquare {
    uint4 hi[64 * 8], lo[64 * 8];
};
__device__ __forceinline__ uint32_t small_pos(uint32_t row, uint32_t chunk) { return row * 128u + ((chunk ^ (row & 7u)) << 4); }
__device__ __forceinline__ half8 small_frag(const uint4 *image, uint32_t row, uint32_t chunk) {
    return *reinterpret_cast<const half8 *>(reinterpret_cast<const char *>(image) + small_pos(row, chunk));
}
// Four consecutive elements e..e+3 (e a multiple of 4) of a row.
__device__ __forceinline__ u32x2 *small_quad(uint4 *image, uint32_t row, uint32_t e) {
    const uint32_t s = e >> 4, k4 = (e >> 2) & 3u;
    return reinterpret_cast<u32x2 *>(reinterpret_cast<char *>(image) + small_pos(row, 2u * s + (k4 & 1u)) + (k4 >> 1) * 8u);
}

// Values read from LDS before are read again rather than kept: P's fragments are
// the same for every block of X, and holding them all would spill registers (96
// matrices of 64 x 768: 121 us without, 85 with).
__device__ __forceinline__ void forget_loads() { asm volatile("" ::: "memory"); }

__device__ __forceinline__ f32x16 mfma(half8 a, half8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
// The part of a product that has the remainders of one factor, times 2^11.
__device__ __forceinline__ f32x16 mfma_cross(half8 ah, half8 al, half8 bh, half8 bl, f32x16 c) {
    return mfma(al, bh, mfma(ah, bl, c));
}
__device__ __forceinline__ void add_cross(f32x16 &v, const f32x16 &cross) {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = fmaf(cross[e], kUnscaleLo, v[e]);
}
// a[s] b[s] summed over kSteps fragments.
template <int kSteps, class A, class B>
__device__ __forceinline__ f32x16 product_of_fragments(const A &a, const B &b) {
    f32x16 v = {}, cross = {};
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        half8 ah, al, bh, bl;
        a(s, ah, al);
        b(s, bh, bl);
        v = mfma(ah, bh, v);
        cross = mfma_cross(ah, al, bh, bl, cross);
    }
    add_cross(v, cross);
    return v;
}

template <int kRows, int kCols, bool kBf16>
__global__ __launch_bounds__(64 * kSmallWaves) void muon_small_kernel(MuonSmallArgs a) {
    constexpr int kSquare = kRows * (kRows + 1) / 2;  // 32 x 32 blocks of A on and below the diagonal
    constexpr int kSteps = 2 * kRows;                 // fragments along the rows of X
    __shared__ SmallSquare gram, poly;
    __shared__ float parts[kSmallWaves][kSquare * 16][64];
    __shared__ double s_sum[kSmallWaves];
    uint32_t t;
    const MuonMat m = find_mat(a.work, blockIdx.x, t);
    const uint32_t tid = threadIdx.x, lane = tid & 63u, ln = lane & 31u, half = lane >> 5;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(tid >> 6));
    const uint32_t n = m.tall ? m.rows : m.cols, n_short = m.tall ? m.cols : m.rows;
    const uint32_t active = min((uint32_t)kSmallWaves, (n + 31u) / 32u);

    // X_0 as it comes; every load is under way before the first is needed
    float raw[kCols][kSteps][8];
    const uint64_t row_step = m.tall ? 1 : m.u_ld, col_step = m.tall ? m.u_ld : 1;
#pragma unroll
    for (int b = 0; b < kCols; ++b) {
        const uint32_t col = 32u * (wave + kSmallWaves * b) + ln;
        const uint64_t at = m.u_off + 4u * half * row_step + col * col_step;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = 16u * s + k_order(j, half) < n_short && col < n;
                const float v = load_elem<kBf16>(a.u, in ? at + (16u * s + k_order(j, 0)) * row_step : m.u_off);
                raw[b][s][j] = in ? v : 0.0f;
            }
            __builtin_amdgcn_sched_barrier(0);  // a step at a time: fewer addresses are held
        }
    }
    // the first update multiplies by one: it only arranges X_0's columns for A
    for (uint32_t i = tid; i < 64u * 8u; i += 64u * kSmallWaves) {
        poly.hi[i] = uint4{0u, 0u, 0u, 0u};
        poly.lo[i] = uint4{0u, 0u, 0u, 0u};
    }
    double sum = 0.0;
#pragma unroll
    for (int b = 0; b < kCols; ++b)
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += (double)raw[b][s][j] * (double)raw[b][s][j];
    sum = block_sum<kSmallWaves>(sum, s_sum);
    if (tid < 32u * kRows) {
        char *quad = reinterpret_cast<char *>(small_quad(poly.hi, tid, tid & ~3u));
        reinterpret_cast<_Float16 *>(quad)[tid & 3u] = (_Float16)kScaleP;
    }
    const double inv = sum < __builtin_inf() ? (double)kScaleX / (sqrt(sum) + a.eps) : __builtin_nan("");

    half8 xh[kCols][kSteps], xl[kCols][kSteps];
#pragma unroll
    for (int b = 0; b < kCols; ++b)
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = (float)((double)raw[b][s][j] * inv);
            split8(y, xh[b][s], xl[b][s]);
        }
    __syncthreads();

    // rows of a square matrix, and the wave's block b of X, as factors
    auto square_rows = [&](const SmallSquare &m, uint32_t row) {
        return [&m, row, half](int s, half8 &h, half8 &l) {
            h = small_frag(m.hi, row, 2u * s + half);
            l = small_frag(m.lo, row, 2u * s + half);
        };
    };
    auto columns = [&](int b) {
        return [&, b](int s, half8 &h, half8 &l) {
            h = xh[b][s];
            l = xl[b][s];
        };
    };
    for (int it = 0; it < a.steps; ++it) {
        // X <- P X and, along the way, A = X X^T
        f32x16 acc[kSquare];
#pragma unroll
        for (int i = 0; i < kSquare; ++i) acc[i] = f32x16{};
#pragma unroll
        for (int b = 0; b < kCols; ++b) {
            const uint32_t col0 = 32u * (wave + kSmallWaves * b);
            if (col0 >= n) continue;
            forget_loads();
            half8 gh[kRows][2], gl[kRows][2];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                forget_loads();
                const f32x16 v = product_of_fragments<kSteps>(columns(b), square_rows(poly, 32u * i + ln));
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = v[8 * k + e] * (1.0f / kScaleP);
                    split8(y, gh[i][k], gl[i][k]);
                }
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i)
#pragma unroll
                for (int j = 0; j <= i; ++j) {
                    f32x16 cross = {};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        cross = mfma_cross(gh[i][k], gl[i][k], gh[j][k], gl[j][k], cross);
                        acc[i + j] = mfma(gh[i][k], gh[j][k], acc[i + j]);
                    }
                    add_cross(acc[i + j], cross);
                }
            if (it == 0) continue;  // P is still one
            forget_loads();
            f32x16 v[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) v[i] = product_of_fragments<kSteps>(square_rows(poly, 32u * i + ln), columns(b));
#pragma unroll
            for (int i = 0; i < kRows; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = v[i][8 * k + e] * (1.0f / kScaleP);
                    split8(y, xh[b][2 * i + k], xl[b][2 * i + k]);
                }
        }

        // A: the sums of the waves that hold columns together, stored with its mirror image
        if (wave < active)
#pragma unroll
            for (int i = 0; i < kSquare; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) parts[wave][i * 16 + e][lane] = acc[i][e];
        __syncthreads();
        for (uint32_t q = wave; q < kSquare * 4u; q += kSmallWaves) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = parts[0][q * 4 + e][lane];
#pragma unroll
            for (uint32_t w = 1; w < kSmallWaves; ++w)
                if (w < active)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] += parts[w][q * 4 + e][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= 1.0f / kScaleX;
            const uint32_t blk = q >> 2, g = q & 3u, bi = blk == 0 ? 0u : 1u, bj = blk == 2 ? 1u : 0u;
            const uint32_t r = 32u * bi + 8u * g + 4u * half, c = 32u * bj + ln;
            u32x2 h, l;
            split4(v[0], v[1], v[2], v[3], h, l);
            *small_quad(gram.hi, c, r) = h;
            *small_quad(gram.lo, c, r) = l;
            if (bi != bj) {
                *small_quad(gram.hi, r + (lane & 3u), c & ~3u) = quad_transpose(h, lane);
                *small_quad(gram.lo, r + (lane & 3u), c & ~3u) = quad_transpose(l, lane);
            }
        }
        __syncthreads();
        // P, one 32 x 32 block a wave, stored as its transpose (it is symmetric)
        if (wave < kRows * kRows) {
            const uint32_t bi = wave / kRows, bj = wave % kRows;
            const f32x16 p = product_of_fragments<kSteps>(square_rows(gram, 32u * bi + ln), square_rows(gram, 32u * bj + ln));
            const float ca = a.coefficients[3 * it] * kScaleP, cb = a.coefficients[3 * it + 1] * (kScaleP / kScaleX),
                        cc = a.coefficients[3 * it + 2] * (kScaleP / (kScaleX * kScaleX));
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t r = 32u * bi + 8u * g + 4u * half, c = 32u * bj + ln;
                const u32x2 h = *small_quad(gram.hi, c, r), l = *small_quad(gram.lo, c, r);
                float x[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t hw = q < 2 ? h.x : h.y, lw = q < 2 ? l.x : l.y;
                    const float av = join(hw >> (16 * (q & 1)), lw >> (16 * (q & 1)));
                    float v = fmaf(cb, av, cc * p[4 * g + q]);
                    if (r + q == c) v += ca;
                    x[q] = v;
                }
                u32x2 ph, pl;
                split4(x[0], x[1], x[2], x[3], ph, pl);
                *small_quad(poly.hi, c, r) = ph;
                *small_quad(poly.lo, c, r) = pl;
            }
        }
        __syncthreads();
    }

    // O = P X, lane = the user's column, so that a wave writes along rows
    float *param = nullptr;
    float step = 0.0f;
    if (a.product == kLastParams) {
        param = ((ConstTensorPtr)a.tensors + m.index)->p;
        step = (float)(a.lr * (a.scale == 1 ? m.scale_spectral : (a.scale == 2 ? m.scale_rms : 1.0)));
    }
#pragma unroll
    for (int b = 0; b < kCols; ++b) {
        const uint32_t col0 = 32u * (wave + kSmallWaves * b);
        if (col0 >= n) continue;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const auto p = square_rows(poly, 32u * i + ln);
            const f32x16 v = m.tall ? product_of_fragments<kSteps>(columns(b), p) : product_of_fragments<kSteps>(p, columns(b));
            const uint32_t r0 = (m.tall ? col0 : 32u * i) + 4u * half, c = m.tall ? 32u * i + ln : col0 + ln;
            float old[16];
            if (a.product == kLastParams) {  // all of the block's params at once, then the stores
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t r = r0 + 8u * (e / 4) + (e & 3);
                    old[e] = param[r < m.rows && c < m.cols ? (uint64_t)r * m.cols + c : 0u];
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t r = r0 + 8u * (e / 4) + (e & 3);
                if (r >= m.rows || c >= m.cols) continue;
                const float o = v[e] * (1.0f / (kScaleX * kScaleP));
                if (a.product == kLastParams) param[(uint64_t)r * m.cols + c] = fmaf(-step, o, old[e] * a.decay);
                else if (a.product == kLastBf16)
                    static_cast<uint16_t *>(a.o)[m.o_off + r * m.o_ld + c] = (uint16_t)f32_to_bf16(o);
                else static_cast<float *>(a.o)[m.o_off + r * m.o_ld + c] = o;
            }
            __builtin_amdgcn_sched_barrier(0);  // one block's addresses at a time
        }
    }
}

// ---------------------------------------------------------------- X_0
// Partial sums of squares of each matrix, in fp64 (a square of any finite
// fp32 value is exact there and never overflows): workgroup w of n_partials
// takes the 64 x 64 tiles w, w + n_partials, ..
template <bool kBf16>
__global__ __launch_bounds__(256) void muon_sums_kernel(MuonWork w, MuonSumArgs a) {
    __shared__ double s[4];
    uint32_t part;
    const MuonMat m = find_mat(w, blockIdx.x, part);
    const uint32_t across = (m.cols + 63u) / 64u, tiles = across * ((m.rows + 63u) / 64u);
    const uint32_t c_in = threadIdx.x & 63u, r_in = threadIdx.x >> 6;
    double sum = 0.0;
    for (uint32_t t = part; t < tiles; t += a.n_partials) {
        const uint32_t r0 = (t / across) * 64u + r_in, c = (t % across) * 64u + c_in;
        float x[16];  // all of the tile's loads before the first sum
#pragma unroll
        for (uint32_t i = 0; i < 16u; ++i) {
            const uint32_t r = r0 + 4u * i;
            x[i] = load_elem<kBf16>(a.u, m.u_off + (r < m.rows && c < m.cols ? r * m.u_ld + c : 0u));
        }
#pragma unroll
        for (uint32_t i = 0; i < 16u; ++i)
            if (r0 + 4u * i < m.rows && c < m.cols) sum += (double)x[i] * (double)x[i];
    }
    sum = block_sum(sum, s);
    if (threadIdx.x == 0) a.partials[m.norm + part] = sum;
}

// The images of X_0 and X_0^T, one 64 x 64 tile of the user's matrix a
// workgroup.  A norm that is not finite makes all of X_0 NaN.
template <bool kBf16, bool kRaw>
__global__ __launch_bounds__(256) void muon_prep_kernel(MuonWork w, MuonPrepArgs a) {
    constexpr int kForm = kRaw ? kPlain : kSplit;
    __shared__ double s[4];
    __shared__ float y[64][65];
    if (blockIdx.x == 0) a.arrived[threadIdx.x] = 0u;
    static_assert(kMaxSplit == 256, "one counter a thread");
    uint32_t t;
    const MuonMat m = find_mat(w, blockIdx.x, t);
    const uint32_t rp = m.tall ? m.np : m.mp, cp = m.tall ? m.mp : m.np;  // the user's matrix, padded
    uint32_t ti, tj;
    if (w.tiles) {
        ti = t & 0xFFFFu;
        tj = t >> 16;
    } else {
        ti = t / (cp / 64u);
        tj = t - ti * (cp / 64u);
    }
    const uint32_t c_in = threadIdx.x & 63u, r_in = threadIdx.x >> 6;
    const uint32_t c = tj * 64u + c_in;
    float v[16];
#pragma unroll
    for (uint32_t i = 0; i < 16u; ++i) {
        // always a load, so that the sixteen are under way together
        const uint32_t r = ti * 64u + r_in + 4u * i;
        v[i] = load_elem<kBf16>(a.u, m.u_off + (r < m.rows && c < m.cols ? r * m.u_ld + c : 0u));
    }
    double part = 0.0;
    for (uint32_t i = threadIdx.x; i < a.n_partials; i += 256u) part += a.partials[m.norm + i];
    const double sum = block_sum(part, s);
    double inv = sum < __builtin_inf() ? (double)kScaleX / (sqrt(sum) + a.eps) : __builtin_nan("");
    if constexpr (kRaw) {
        // the power of two that brings the norm (and so every entry) to below
        // 2^16, of which the largest bf16 value is in fp16's range: bf16's 8 bits
        // are exact down to 2^-33 of the norm, smaller entries have an error of
        // at most 2^-40 of it
        const double power = sum > 0.0 ? ldexp(1.0, 15 - ilogb(sqrt(sum))) : 1.0;
        if (t == 0 && threadIdx.x == 0) a.phi[m.index] = sum > 0.0 ? (float)(inv / power) : 0.0f;
        inv = sum < __builtin_inf() ? power : inv;
    }
#pragma unroll
    for (uint32_t i = 0; i < 16u; ++i) {
        const bool in = ti * 64u + r_in + 4u * i < m.rows && c < m.cols;
        y[r_in + 4u * i][c_in] = in ? (float)((double)v[i] * inv) : 0.0f;
    }
    __syncthreads();
    // by user rows (elements along the columns), then by user columns: 16 bytes
    // a thread, the 32 rows of a fragment side by side
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        char *dst = ((o == 0) == (m.tall == 0) ? a.x : a.xt) + m.x_off;
        const uint32_t length = o == 0 ? cp : rp;
        const uint32_t row0 = (o == 0 ? ti : tj) * 64u, k0 = (o == 0 ? tj : ti) * 64u;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t job = j * 256u + threadIdx.x, row = (job & 31u) + 32u * (job >> 8), k = ((job >> 5) & 7u) * 8u;
            u32x4 h, l;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t h0, l0;
                split2(o == 0 ? y[row][k + 2 * e] : y[k + 2 * e][row], o == 0 ? y[row][k + 2 * e + 1] : y[k + 2 * e + 1][row],
                       h0, l0);
                h[e] = h0;
                l[e] = l0;
            }
            char *at = dst + image_pos<kForm>(row0 + row, k0 + k, length);
            *reinterpret_cast<u32x4 *>(at) = h;
            if constexpr (kForm == kSplit) *reinterpret_cast<u32x4 *>(at + kRemainder) = l;
        }
    }
}

__global__ __launch_bounds__(256) void muon_norms_kernel(const double *partials, const uint2 *ranges, double *sums) {
    __shared__ double s[4];
    const uint2 range = ranges[blockIdx.x];
    double part = 0.0;
    for (uint32_t i = range.x + threadIdx.x; i < range.y; i += 256u) part += partials[i];
    const double sum = block_sum(part, s);
    if (threadIdx.x == 0) sums[blockIdx.x] = sum;
}

// ---------------------------------------------------------------- momentum
__device__ __forceinline__ void philox4x32_10(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t prod0 = (uint64_t)0xD2511F53u * c[0], prod1 = (uint64_t)0xCD9E8D57u * c[2];
        c[0] = (uint32_t)(prod1 >> 32) ^ c[1] ^ k0;
        c[1] = (uint32_t)prod1;
        c[2] = (uint32_t)(prod0 >> 32) ^ c[3] ^ k1;
        c[3] = (uint32_t)prod0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

__device__ __forceinline__ float block_max(float x, float *s) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor(x, d, 64));
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
    __syncthreads();
    return fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
}

// One 2048-element block of one matrix, as the Adam step takes its blocks:
// thread t holds elements 4t..4t+3 and 1024+4t..1024+4t+3.  Writes the new
// momentum, the update u (fp32) and the block's sum of u^2.
template <int kStorage, bool kGradBf16, bool kSR>
__global__ __launch_bounds__(256) void muon_momentum_kernel(MuonStepArgs a) {
    __shared__ double s_sum[4];
    __shared__ float s_max[4];
    const ConstDescPtr d = (ConstDescPtr)a.desc + blockIdx.x;
    const uint32_t lb_n = d->lb_n, n = (lb_n & (kBlock - 1)) + 1u, npad = (n + 15u) & ~15u, slot = d->slot;
    const uint64_t local = (uint64_t)(lb_n >> kBlockBits) * kBlock, gidx = (uint64_t)d->gidx16 * 16u;
    const void *g = ((ConstTensorPtr)a.tensors + d->tensor)->g;
    float mo[8], uo[8];
    const float old_scale = kStorage == kMuonQ8 ? a.m_scale[slot] : 0.0f;
    double sum = 0.0;
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t e0 = j * 1024u + 4u * threadIdx.x;
        float gv[4] = {0.0f, 0.0f, 0.0f, 0.0f}, mv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (e0 + 4u <= n) {
            if constexpr (kGradBf16) {
                const u32x2 q = *reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(g) + local + e0);
                gv[0] = __uint_as_float(q.x << 16);
                gv[1] = __uint_as_float(q.x & 0xFFFF0000u);
                gv[2] = __uint_as_float(q.y << 16);
                gv[3] = __uint_as_float(q.y & 0xFFFF0000u);
            } else {
                const f32x4 q = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(g) + local + e0);
#pragma unroll
                for (int i = 0; i < 4; ++i) gv[i] = q[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (e0 + i < n) gv[i] = load_elem<kGradBf16>(g, local + e0 + i);
        }
        if (e0 < npad) {
            if constexpr (kStorage == kMuonBf16) {
                const u32x2 q = *reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(a.m_state) + gidx + e0);
                mv[0] = __uint_as_float(q.x << 16);
                mv[1] = __uint_as_float(q.x & 0xFFFF0000u);
                mv[2] = __uint_as_float(q.y << 16);
                mv[3] = __uint_as_float(q.y & 0xFFFF0000u);
            } else if constexpr (kStorage == kMuonQ8) {
                const uint32_t q = *reinterpret_cast<const uint32_t *>(static_cast<const int8_t *>(a.m_state) + gidx + e0);
#pragma unroll
                for (int i = 0; i < 4; ++i) mv[i] = (float)(int8_t)(q >> (8 * i)) * (1.0f / 127.0f) * old_scale;
            } else {
                const f32x4 q = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(a.m_state) + gidx + e0);
#pragma unroll
                for (int i = 0; i < 4; ++i) mv[i] = q[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool live = e0 + i < n;  // padding takes no part, whatever it holds
            const float gp = gv[i] * a.omb, m = live ? fmaf(a.beta, mv[i], gp) : 0.0f;
            const float u = live ? (a.nesterov ? fmaf(a.beta, m, gp) : m) : 0.0f;
            mo[4 * j + i] = m;
            uo[4 * j + i] = u;
            sum += (double)u * (double)u;
            top = fmaxf(top, fabsf(m));
        }
        if (e0 < npad)  // u's segments are padded as the state's are
            *reinterpret_cast<f32x4 *>(a.u + (gidx - a.u_base) + e0) = f32x4{uo[4 * j], uo[4 * j + 1], uo[4 * j + 2], uo[4 * j + 3]};
    }
    sum = block_sum(sum, s_sum);
    if (threadIdx.x == 0) a.partials[slot - a.slot_base] = sum;

    float r = 0.0f;
    bool live = true;
    if constexpr (kStorage == kMuonQ8) {
        top = block_max(top, s_max);
        live = top >= kTiny;
        r = live ? 1.0f / top * 127.0f : 0.0f;
        if (threadIdx.x == 0) a.m_scale[slot] = live ? top : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t e0 = j * 1024u + 4u * threadIdx.x;
        if (e0 >= npad) continue;
        const float *m = mo + 4 * j;
        if constexpr (kStorage == kMuonBf16) {
            *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.m_state) + gidx + e0) =
                u32x2{f32_to_bf16(m[0]) | (f32_to_bf16(m[1]) << 16), f32_to_bf16(m[2]) | (f32_to_bf16(m[3]) << 16)};
        } else if constexpr (kStorage == kMuonF32) {
            *reinterpret_cast<f32x4 *>(static_cast<float *>(a.m_state) + gidx + e0) = f32x4{m[0], m[1], m[2], m[3]};
        } else {
            uint32_t ctr[4] = {0u, 0u, 0u, 0u}, codes = 0u;
            if constexpr (kSR) {
                const uint64_t grp = (((ConstU64Ptr)a.draw_first)[d->tensor] + local + e0) >> 2;
                ctr[0] = (uint32_t)grp;
                ctr[1] = (uint32_t)(grp >> 32);
                ctr[2] = a.t_lo;
                ctr[3] = a.t_hi;
                philox4x32_10(ctr, a.seed_lo, a.seed_hi);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float y = fminf(fabsf(m[i]) * r, 127.0f);
                float q;
                if constexpr (kSR) {
                    const float down = floorf(y), u = (float)(ctr[i] & 0xFFFFu) * 0x1p-16f;
                    q = down + (u < y - down ? 1.0f : 0.0f);
                } else {
                    q = rintf(y);
                }
                if (fabsf(m[i]) >= top) q = 127.0f;
                const int32_t k = live ? (int32_t)(m[i] < 0.0f ? -q : q) : 0;
                codes |= ((uint32_t)k & 0xFFu) << (8 * i);
            }
            *reinterpret_cast<uint32_t *>(static_cast<int8_t *>(a.m_state) + gidx + e0) = codes;
        }
    }
}

// The momentum's values, padding 0: fp32, or bf16 as it is.
template <int kStorage>
__global__ __launch_bounds__(256) void muon_decode_kernel(const BlockDesc *desc, const void *m_state, const float *m_scale,
                                                          void *dst) {
    const ConstDescPtr d = (ConstDescPtr)desc + blockIdx.x;
    const uint32_t n = (d->lb_n & (kBlock - 1)) + 1u, npad = (n + 15u) & ~15u;
    const uint64_t gidx = (uint64_t)d->gidx16 * 16u;
    const float scale = kStorage == kMuonQ8 ? m_scale[d->slot] : 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t e0 = j * 1024u + 4u * threadIdx.x;
        if (e0 >= npad) continue;
        if constexpr (kStorage == kMuonBf16) {
            u32x2 q = *reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(m_state) + gidx + e0);
            if (e0 + 4u > n) {
                q.x = (e0 < n ? q.x & 0xFFFFu : 0u) | (e0 + 1u < n ? q.x & 0xFFFF0000u : 0u);
                q.y = (e0 + 2u < n ? q.y & 0xFFFFu : 0u);
            }
            *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(dst) + gidx + e0) = q;
        } else {
            f32x4 v;
            if constexpr (kStorage == kMuonQ8) {
                const uint32_t q = *reinterpret_cast<const uint32_t *>(static_cast<const int8_t *>(m_state) + gidx + e0);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(q >> (8 * i)) * (1.0f / 127.0f) * scale;
            } else {
                v = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(m_state) + gidx + e0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (e0 + i >= n) v[i] = 0.0f;
            *reinterpret_cast<f32x4 *>(static_cast<float *>(dst) + gidx + e0) = v;
        }
    }
}

}  // namespace

// ---------------------------------------------------------------- launches
hipError_t launch_muon_momentum(int storage, bool grad_bf16, bool stochastic, const MuonStepArgs &a, hipStream_t s) {
    const dim3 grid(a.n_blocks), block(256);
#define MUON_MOMENTUM(st, sr)                                                                       \
    do {                                                                                            \
        if (grad_bf16) muon_momentum_kernel<st, true, sr><<<grid, block, 0, s>>>(a);                \
        else muon_momentum_kernel<st, false, sr><<<grid, block, 0, s>>>(a);                         \
    } while (0)
    if (storage == kMuonBf16) MUON_MOMENTUM(kMuonBf16, false);
    else if (storage == kMuonF32) MUON_MOMENTUM(kMuonF32, false);
    else if (stochastic) MUON_MOMENTUM(kMuonQ8, true);
    else MUON_MOMENTUM(kMuonQ8, false);
#undef MUON_MOMENTUM
    return hipGetLastError();
}

hipError_t launch_muon_norms(const double *partials, const uint2 *ranges, double *sums, uint32_t n_mats, hipStream_t s) {
    muon_norms_kernel<<<dim3(n_mats), dim3(256), 0, s>>>(partials, ranges, sums);
    return hipGetLastError();
}

hipError_t launch_muon_sums(bool bf16, const MuonWork &w, const MuonSumArgs &a, uint32_t n_mats, hipStream_t s) {
    const dim3 grid(n_mats * a.n_partials), block(256);
    if (bf16) muon_sums_kernel<true><<<grid, block, 0, s>>>(w, a);
    else muon_sums_kernel<false><<<grid, block, 0, s>>>(w, a);
    return hipGetLastError();
}

hipError_t launch_muon_prep(bool bf16, bool raw, int form, const MuonWork &w, const MuonPrepArgs &a, hipStream_t s) {
    const dim3 grid(w.n_tiles), block(256);
    if (form != (raw ? kPlain : kSplit) || (raw && !bf16)) return hipErrorInvalidValue;
    if (raw) muon_prep_kernel<true, true><<<grid, block, 0, s>>>(w, a);
    else if (bf16) muon_prep_kernel<true, false><<<grid, block, 0, s>>>(w, a);
    else muon_prep_kernel<false, false><<<grid, block, 0, s>>>(w, a);
    return hipGetLastError();
}

template <class T>
static hipError_t product_of(int product, int in, int jobs, const MuonGemmArgs &a, hipStream_t s) {
    const uint32_t per_job = a.work.n_whole + (a.work.n_tiles - a.work.n_whole) * a.work.parts;
    const dim3 grid(jobs * per_job), block(T::kThreads);
    if (jobs != (a.left2 ? 2 : 1)) return hipErrorInvalidValue;
#define MUON_CASE(p, i)                                                          \
    if (product == p && in == i) {                                               \
        muon_product_kernel<T, p, i><<<grid, block, 0, s>>>(a);                  \
        return hipGetLastError();                                                \
    }
    MUON_CASE(kGram, kSplit)
    MUON_CASE(kGram, kPlain)
    MUON_CASE(kPolynomial, kSplit)
    MUON_CASE(kCommuting, kSplit)
    MUON_CASE(kUpdate, kSplit)
    MUON_CASE(kUpdate, kMixed)
    MUON_CASE(kLastF32, kSplit)
    MUON_CASE(kLastBf16, kSplit)
    MUON_CASE(kLastParams, kSplit)
#undef MUON_CASE
    return hipErrorInvalidValue;
}

// 128 x 128 tiles: eight waves hide more of the latency while a CU has one
// tile; with more than one, two workgroups of four waves do, and their larger
// blocks read LDS less.  (us with four / eight waves: 252 tiles, P of 12
// matrices of 768^2 26.5 / 24.9 and X X^T 25.0 / 23.5; 432 tiles 38.6 / 39.6; 504 tiles, P of 24
// of them 43.0 / 43.8, X X^T of 24 of 768 x 2304 110 / 116; 2048 tiles, P X of four
// of 2048 x 4096 400 / 421; 4096 tiles, P X of four of 4096^2 1506 / 1538; but 2592
// tiles, P X of 24 of 768 x 2304, 240 / 232.  Three stages were slower in
// each but for 252 tiles, where they made no difference; four, and 128 x 256
// tiles, were slower when remainders had no sums of their own.)  64 x 64 tiles have three stages: three workgroups to a CU.
typedef Tiling<64, 64, 2, 2, 3, 3> Tiling64;
typedef Tiling<128, 128, 2, 4, 2, 4> Tiling128;
typedef Tiling<128, 128, 2, 2, 2, 2> Tiling128Many;
constexpr uint32_t kManyTiles = 384;

hipError_t launch_muon_product(int tiling, int product, int in, int jobs, const MuonGemmArgs &a, hipStream_t s) {
    if (tiling == kTile64) return product_of<Tiling64>(product, in, jobs, a, s);
    if (a.work.n_tiles >= kManyTiles) return product_of<Tiling128Many>(product, in, jobs, a, s);
    return product_of<Tiling128>(product, in, jobs, a, s);
}

hipError_t launch_muon_small(int64_t short_side, int64_t long_side, const MuonSmallArgs &a, hipStream_t s) {
    const dim3 grid(a.work.n_tiles), block(64 * kSmallWaves);
    const int cols = (int)((long_side + 255) / 256);
    if (short_side > kSmallShort || cols < 1 || cols > 3) return hipErrorInvalidValue;
#define MUON_SMALL(r, c)                                                    \
    if ((short_side <= 32) == (r == 1) && cols == c) {                      \
        if (a.u_bf16) muon_small_kernel<r, c, true><<<grid, block, 0, s>>>(a);            \
        else muon_small_kernel<r, c, false><<<grid, block, 0, s>>>(a);      \
        return hipGetLastError();                                           \
    }
    MUON_SMALL(1, 1)
    MUON_SMALL(1, 2)
    MUON_SMALL(1, 3)
    MUON_SMALL(2, 1)
    MUON_SMALL(2, 2)
    MUON_SMALL(2, 3)
#undef MUON_SMALL
    return hipErrorInvalidValue;
}

hipError_t launch_muon_decode(int storage, const BlockDesc *desc, uint32_t n_blocks, const void *m_state,
                              const float *m_scale, void *dst, hipStream_t s) {
    constexpr uint32_t kMost = 1u << 23;  // a launch has less than 2^32 threads
    hipError_t e = hipSuccess;
    for (uint32_t done = 0; done < n_blocks && e == hipSuccess; done += min(kMost, n_blocks - done)) {
        const dim3 grid(min(kMost, n_blocks - done)), block(256);
        const BlockDesc *d = desc + done;
        if (storage == kMuonBf16) muon_decode_kernel<kMuonBf16><<<grid, block, 0, s>>>(d, m_state, m_scale, dst);
        else if (storage == kMuonQ8) muon_decode_kernel<kMuonQ8><<<grid, block, 0, s>>>(d, m_state, m_scale, dst);
        else muon_decode_kernel<kMuonF32><<<grid, block, 0, s>>>(d, m_state, m_scale, dst);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace adam_mi355x
