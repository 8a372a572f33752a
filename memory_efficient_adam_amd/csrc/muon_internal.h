// Internal interface between the host runtime and the gfx950 kernels of the
// Muon step and the Newton-Schulz orthogonalisation.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "adam_internal.h"

namespace adam_mi355x {

// One matrix of a launch.  Its factor X is short x long (m x n, m <= n), the
// transpose of the user's matrix when that is tall.  A factor is kept as an
// "image" in the order in which the matrix instructions take it: blocks of 32
// rows; in each, slabs of 4 KB along the rows' elements; in each slab four
// fragments of 1 KB, whose 16 bytes at position l are what lane l holds: row
// l % 32, elements 8 (l / 32) .. + 7 of the fragment's 16.
//   split slabs (two fp16 values per element, the remainder times 2^11): 32
//     elements; fragments: high parts of the first 16, their remainders, the
//     same of the second 16;
//   plain slabs (one fp16 value per element; an X_0 taken as its bf16 source
//     has it): 64 elements, 16 per fragment.
// So a slab goes to LDS as it is, is read there without bank conflicts, and
// a wave's 32 x 32 block of a result is one contiguous piece of an image.
// Dimensions are padded to multiples of the tile with zeros, which every
// product keeps zero.
struct MuonMat {
    uint64_t x_off;   // byte offset in each of the X arrays
    uint64_t a_off;   // byte offset in the square arrays
    uint64_t u_off;   // element offset of the source matrix in its array
    uint64_t o_off;   // element offset of the output matrix in its array
    uint64_t u_ld, o_ld;  // row strides of source and output, in elements
    uint32_t mp, np;      // padded short and long side
    uint32_t rows, cols;
    uint32_t tall;        // rows > cols
    uint32_t index;       // tensor index (pointer table, scale factors)
    uint32_t norm;        // index of its first partial sum of squares
    uint32_t pad;
    double scale_spectral, scale_rms;
};
static_assert(sizeof(MuonMat) == 96, "matrix descriptor layout");

// One workgroup's tile: matrix, tile row, tile column.
struct MuonTile {
    uint32_t mat;
    uint16_t ti, tj;
};
static_assert(sizeof(MuonTile) == 8, "tile descriptor is one 8-byte load");

// Which matrices and tiles a launch covers: a table (tiles != NULL), or
// matrices alike, whose descriptors are `one` advanced by the strides, with
// per_mat of the n_tiles tiles each.
struct MuonWork {
    const MuonTile *tiles;
    const MuonMat *mats;
    uint32_t n_tiles;
    uint32_t per_mat;
    // Tiles from n_whole on are each taken by `parts` workgroups, a part of
    // the products' length each (parts > 1): their sums go to `partial`, and
    // the last of them to get there (by `arrived`) adds them up in order.
    uint32_t n_whole, parts;
    float *partial;
    uint32_t *arrived;
    MuonMat one;
    uint64_t x_stride, a_stride, u_stride, o_stride;
    uint32_t norm_stride;
    uint32_t window;  // log2 of the workgroups among which each XCD gets a run of tiles
};

// The factor arrays of one group of matrices.
constexpr int kSquares = 5;
struct MuonArrays {
    char *x[2], *xt[2];    // X and X^T, before and after an update
    char *square[kSquares];  // A = X X^T, the polynomials, their products
};

// How a product's factors are held: in split or plain slabs, or (kMixed, an
// update) the left one split and the right one plain.
enum MuonForm : int { kSplit = 0, kPlain = 1, kMixed = 2 };

// The 256 CUs take tiles in rounds; the tiles of a last round that would leave
// many of them idle are split.
constexpr uint32_t kCus = 256;
constexpr uint32_t kMaxSplit = kCus;        // tiles that are split
constexpr uint32_t kMaxParts = 8;
constexpr uint32_t kMaxPartials = 4 * kCus;  // workgroups for them

// Sum of squares: one fp64 partial per workgroup, per matrix n_partials.
struct MuonSumArgs {
    const void *u;
    double *partials;
    uint32_t n_partials;
};

struct MuonPrepArgs {
    uint32_t *arrived;  // cleared: kMaxSplit counters
    const void *u;
    const double *partials;
    uint32_t n_partials;
    double eps;
    char *x, *xt;
    float *phi;  // raw form: X_0 = phi (x as written)
};

struct MuonGemmArgs {
    MuonWork work;
    const char *left, *right;  // factor images, both with K along the rows
    const char *left2, *right2;  // a second product of the same launch (kCommuting; else NULL)
    char *out2;
    const char *add;           // A (polynomial only)
    char *out, *out_t;         // images written (out_t: X^T)
    const float *phi;          // what a raw X_0 is still to be multiplied by (else NULL)
    float ca, cb, cc;          // polynomial coefficients
    // last product: where O goes
    const TensorRef *tensors;  // params (step), by MuonMat::index
    void *o;                   // output array (orthogonalisation)
    double lr;
    float decay;
    int32_t scale;
};

// Whole orthogonalisations of matrices whose short side is at most kSmallShort
// and long side at most kSmallLong, one workgroup a matrix.
constexpr int64_t kSmallShort = 64, kSmallLong = 768;
constexpr int64_t kSmallBatch = int64_t(1) << 22;  // matrices of a launch: it has less than 2^32 threads
constexpr int kMaxIterations = 16;

struct MuonSmallArgs {
    MuonWork work;
    const void *u;
    void *o;                   // output array (orthogonalisation)
    const TensorRef *tensors;  // params (step)
    double eps;
    double lr;
    float decay;
    int32_t scale;
    int32_t product;           // kLastBf16, kLastF32, kLastParams
    int32_t u_bf16;
    int32_t steps;
    float coefficients[3 * kMaxIterations];
};

// ---------------------------------------------------------------- momentum
struct MuonStepArgs {
    const BlockDesc *desc;
    const TensorRef *tensors;
    const uint64_t *draw_first;
    void *m_state;       // bf16 / int8 codes / fp32
    float *m_scale;      // per block (Q8)
    float *u;            // the group's update matrices, flat as the state's segments
    double *partials;    // per block: sum of squares of u
    uint64_t u_base;     // flat state index of u[0]
    uint32_t slot_base;  // scale slot of partials[0]
    uint32_t n_blocks;
    float beta, omb;
    uint32_t nesterov;
    uint32_t seed_lo, seed_hi, t_lo, t_hi;
};

enum MuonStorage : int { kMuonBf16 = 1, kMuonQ8 = 2, kMuonF32 = 3 };

hipError_t launch_muon_momentum(int storage, bool grad_bf16, bool stochastic, const MuonStepArgs &a, hipStream_t s);
// sums[mats[i].norm] = the sum of matrix i's block partials
// [ranges[i].x, ranges[i].y), in a fixed order
hipError_t launch_muon_norms(const double *partials, const uint2 *ranges, double *sums, uint32_t n_mats,
                             hipStream_t s);
hipError_t launch_muon_sums(bool bf16, const MuonWork &w, const MuonSumArgs &a, uint32_t n_mats, hipStream_t s);
// raw: bf16 input times a power of two, exact in plain slabs (form kPlain), with
// the rest of the scale in phi; else form is kSplit
hipError_t launch_muon_prep(bool bf16, bool raw, int form, const MuonWork &w, const MuonPrepArgs &a, hipStream_t s);

enum MuonProduct : int { kGram, kPolynomial, kCommuting, kUpdate, kLastBf16, kLastF32, kLastParams };
// The tiles of the products (rows and columns of the result, waves): the
// dimensions of a matrix are padded to multiples of both of its products'
// tiles.
enum MuonTiling : int { kTile64, kTile128 };
// Bytes of a split workgroup's sums.
inline int64_t partial_bytes(int tiling) { return tiling == kTile128 ? 128 * 128 * 4 : 64 * 64 * 4; }
// in: the form of the factors read (those written are split); jobs: 2 with a
// second product (kCommuting), else 1
hipError_t launch_muon_product(int tiling, int product, int in, int jobs, const MuonGemmArgs &a, hipStream_t s);

// short_side, long_side: the largest of the launch's matrices
hipError_t launch_muon_small(int64_t short_side, int64_t long_side, const MuonSmallArgs &a, hipStream_t s);

hipError_t launch_muon_decode(int storage, const BlockDesc *desc, uint32_t n_blocks, const void *m_state,
                              const float *m_scale, void *dst, hipStream_t s);

}  // namespace adam_mi355x
