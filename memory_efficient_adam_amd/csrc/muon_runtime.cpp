// Host runtime behind the C ABI declared in include/muon_mi355x.h: argument
// validation, the momentum's layout (that of Adam's first moment), the
// descriptor and tile tables, workspace, and the launches of a step and of
// the orthogonalisation.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <string>
#include <vector>

#include "muon_internal.h"
#include "muon_mi355x.h"
#include "runtime_common.h"

using namespace adam_mi355x;

namespace {

constexpr int kTableSlots = 4;  // resident pointer tables per state
constexpr int kStageSlots = 8;  // pinned staging buffers per state

// Matrices go through the products together up to this many (padded)
// elements: 1 GB of X, and some 4000 tiles of 128 x 128.
constexpr int64_t kGroupElements = int64_t(1) << 26;
constexpr int64_t kMaxDim = int64_t(1) << 21;
constexpr int64_t kMaxSums = 1024;  // workgroups that share a matrix's sum of squares
// The growth of a rounding error up to which runs of three iterations are
// taken, and the shortest side for runs (see runs_of).
constexpr double kRunGrowth = 12.0;
constexpr int64_t kPairShort = 256, kTripleShort = 512;
constexpr float kDefaultCoefficients[3] = {3.4445f, -4.7750f, 2.0315f};

int fail(int code, const std::string &msg) { return set_last_error(code, msg); }

int hip_fail(hipError_t e, const char *what) {
    return fail(ADAM_EDEVICE, std::string(what) + ": " + hipGetErrorString(e));
}

// Runs an entry point's body: a host allocation failure inside it comes back
// as ADAM_ENOMEM instead of escaping through the C ABI.
template <class F>
auto guarded(F &&body) noexcept -> decltype(body()) {
    try {
        return body();
    } catch (const std::bad_alloc &) {
        try { return fail(ADAM_ENOMEM, "host allocation failed"); } catch (...) { return ADAM_ENOMEM; }
    } catch (...) {
        try { return fail(ADAM_EDEVICE, "unexpected host exception"); } catch (...) { return ADAM_EDEVICE; }
    }
}

int64_t pad_to(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
int64_t pad16(int64_t n) { return pad_to(n, 16); }
int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

struct TableSlot {
    TensorRef *dev = nullptr;
    std::vector<TensorRef> ptrs;
    uint64_t last_use = 0;
    bool valid = false;
};

struct Shape {
    int64_t rows, cols;
    int64_t numel() const { return rows * cols; }
    int64_t shorter() const { return std::min(rows, cols); }
    int64_t longer() const { return std::max(rows, cols); }
};

// ---------------------------------------------------------------- choice of tiles
// A launch's time in us by what was measured: a CU takes a slab of a 128 x 128
// tile in 0.70 us (split factors; several tiles on a CU take as much
// each) and of a 64 x 64 tile in 0.24; with 256 CUs the tiles go in rounds.
// The tiles beyond whole rounds may be cut into parts along the
// products' length, whose sums are written and read at 3500 bytes a ns.
// 5 us pass in a launch besides.
constexpr double kSlabTime[2] = {0.24, 0.70};  // by tiling
constexpr double kLaunchTime = 5.0;

struct Cut {
    uint32_t whole, parts;
    double time;
};
// slabs: the tiles' average; least: the fewest a tile has
Cut cut_tiles(int tiling, int64_t tiles, int64_t jobs, double slabs, int64_t least) {
    const double one = slabs * kSlabTime[tiling];
    const int64_t rest = tiles * jobs % kCus, rounds = tiles * jobs / kCus;
    Cut cut{(uint32_t)tiles, 1, (rest > 0 ? (double)(rounds + 1) : (double)rounds) * one + kLaunchTime};
    if (rest % jobs != 0) return cut;
    for (int64_t parts = 2; parts <= (int64_t)kMaxParts && parts * rest <= kMaxPartials && least / parts >= 4; ++parts) {
        const double time = (double)rounds * one + (double)((rest * parts + kCus - 1) / kCus) / (double)parts * one + 2.0 +
                            2.0 * (double)(rest * parts * partial_bytes(tiling)) / 3.5e6 + kLaunchTime;
        if (rest > 0 && time < cut.time) cut = Cut{(uint32_t)(tiles - rest / jobs), (uint32_t)parts, time};
    }
    return cut;
}

// The tiles of one kind of product over a set of matrices, for either tiling,
// and the length of the products in slabs.
struct Load {
    int64_t tiles[2] = {0, 0};
    double slabs[2] = {0.0, 0.0};  // summed over tiles
    int64_t least = kMaxDim, most = 0;  // in slabs, of a tile
    void add(double count, int64_t down, int64_t across, bool triangle, int64_t length) {
        for (int t = 0; t < 2; ++t) {
            const int64_t size = t == kTile128 ? 128 : 64, r = pad_to(down, size) / size, c = pad_to(across, size) / size;
            const int64_t n = (int64_t)count * (triangle ? r * (r + 1) / 2 : r * c);
            tiles[t] += n;
            slabs[t] += (double)n * (double)pad_to(length, size) / 32.0;
        }
        least = std::min(least, length / 32);
        most = std::max(most, length / 32);
    }
    // plain slabs hold twice the elements
    Cut cut(int tiling, int64_t n_tiles, int64_t jobs, int form) const {
        const double per = form == kPlain ? 2.0 : 1.0;
        return cut_tiles(tiling, n_tiles, jobs, slabs[tiling] / (double)std::max<int64_t>(1, tiles[tiling]) / per,
                         least / (int64_t)per);
    }
    // log2 of the workgroups among which each XCD gets a run of tiles.  Of long
    // and short tiles every XCD is to have its share (a step of 12 encoder
    // blocks' attention, X X^T over 768 and 2304: 1342 -> 1303 us).  Of very many
    // alike the XCDs are kept near each other, so that they find each other's
    // factors in the cache behind theirs (four matrices of 4096^2: 16425 -> 16237
    // us).  Of fewer each gets one run (1296 tiles, 12 of 2304 x 768: 579
    // us, 588 with windows of 1024).
    uint32_t window(int tiling) const { return most > least ? 8u : (tiles[tiling] >= 2048 ? 10u : 31u); }
    double time(int tiling, int64_t jobs = 1) const { return cut(tiling, tiles[tiling], jobs, kSplit).time; }
};

// What a set of matrices that go through the products together takes.
struct Work {
    Load gram, square, update;  // X X^T; products of square factors; P X
    int square_tiling = kTile64, update_tiling = kTile64;
    bool pairs = false, triples = false;  // whether runs of two or three iterations are to be taken
    int64_t shortest = kMaxDim;
    void add(const Shape &s, double count = 1.0) {
        shortest = std::min(shortest, s.shorter());
        gram.add(count, s.shorter(), s.shorter(), true, s.longer());
        square.add(count, s.shorter(), s.shorter(), true, s.shorter());
        update.add(count, s.shorter(), s.longer(), false, s.shorter());
    }
    void choose() {
        auto better = [](const Load &l, const Load &m) {
            return l.time(kTile128) + m.time(kTile128) <= l.time(kTile64) + m.time(kTile64) ? kTile128 : kTile64;
        };
        square_tiling = better(square, gram);
        update_tiling = better(update, update);
        const double g = gram.time(square_tiling), s = square.time(square_tiling), u = update.time(update_tiling);
        pairs = shortest >= kPairShort && g + u > 3.0 * s;
        triples = shortest >= kTripleShort && 2.0 * (g + u) > 4.0 * s + square.time(square_tiling, 2);
    }
    // Square arrays that its iterations use: A, P; in runs of two T, R too, of three U (run_products).
    int squares() const { return triples ? kSquares : (pairs ? 4 : 2); }
    int64_t pad() const { return square_tiling == kTile128 || update_tiling == kTile128 ? 128 : 64; }
    int64_t part_bytes() const {  // (small matrices have no tiles)
        return update.tiles[0] == 0 ? 0 : std::max(partial_bytes(square_tiling), partial_bytes(update_tiling));
    }
};

// A part of the list whose matrices go through the products together.
struct Group {
    int32_t first = 0, last = 0;  // tensors [first, last)
    int64_t x_bytes = 0, a_bytes = 0;  // of one X (or X^T) array and of one square array (small matrices have none)
    int64_t u_bytes = 0;               // of the update matrices
    int64_t block0 = 0, blocks = 0;    // 2048-element blocks
    int64_t flat0 = 0;                 // flat state index of its first element
    Work size;
    std::vector<MuonMat> mats;
    std::vector<MuonTile> prep, square, update, small;
    int64_t small_short = 0, small_long = 0;  // the largest sides of its small matrices
    std::vector<uint2> ranges;  // per matrix: its blocks within the group
    // where the tables stand in the state's device table array
    const MuonMat *d_mats = nullptr;
    const MuonTile *d_prep = nullptr, *d_square = nullptr, *d_update = nullptr, *d_small = nullptr;
    const uint2 *d_ranges = nullptr;
};

bool is_small(const Shape &s) { return s.shorter() <= kSmallShort && s.longer() <= kSmallLong; }
int size_of(int tiling) { return tiling == kTile128 ? 128 : 64; }
int64_t tiles_of(const Shape &s, int64_t tile) {
    return (pad_to(s.shorter(), tile) / tile) * (pad_to(s.longer(), tile) / tile);
}

// The groups of a list, without their tables.
std::vector<Group> plan(const std::vector<Shape> &shapes) {
    std::vector<Group> groups;
    const int32_t n = (int32_t)shapes.size();
    int64_t block = 0, flat = 0;
    for (int32_t k = 0; k < n;) {
        Group g;
        g.first = k;
        g.block0 = block;
        g.flat0 = flat;
        int64_t elements = 0;
        for (; k < n; ++k) {
            // (a small matrix takes its blocks of u alone)
            const bool small = is_small(shapes[k]);
            const int64_t more = small ? blocks_of(shapes[k].numel()) * kBlock : tiles_of(shapes[k], 128) * 16384;
            if (elements > 0 && elements + more > kGroupElements) break;
            elements += more;
            if (!small && more > 0) g.size.add(shapes[k]);
            block += blocks_of(shapes[k].numel());
            flat += pad16(shapes[k].numel());
        }
        g.last = k;
        g.blocks = block - g.block0;
        g.size.choose();
        for (int32_t i = g.first; i < g.last; ++i) {
            g.u_bytes += 4 * pad16(shapes[i].numel());
            if (shapes[i].numel() == 0 || is_small(shapes[i])) continue;
            const int64_t m = pad_to(shapes[i].shorter(), g.size.pad()), l = pad_to(shapes[i].longer(), g.size.pad());
            g.x_bytes += 4 * m * l;
            g.a_bytes += 4 * m * m;
        }
        if (g.blocks > 0) groups.push_back(std::move(g));
    }
    return groups;
}

// The workspace a group needs: four X arrays (u takes the place of the one that is
// written last), the square ones, the blocks' partial sums and the matrices' sums.
int64_t align256(int64_t n) { return pad_to(n, 256); }
int64_t workspace_bytes(const Work &w, int64_t x_bytes, int64_t u_bytes, int64_t a_bytes, int64_t n_partials) {
    return 3 * align256(x_bytes) + align256(std::max(x_bytes, u_bytes)) + w.squares() * align256(a_bytes) + 4 * kMaxSplit +
           kMaxPartials * w.part_bytes() + align256(8 * n_partials);
}
int64_t group_bytes(const Group &g) {
    return workspace_bytes(g.size, g.x_bytes, g.u_bytes, g.a_bytes, g.blocks) + align256(8 * (g.last - g.first));
}

struct Workspace {
    MuonArrays f;
    uint32_t *arrived;  // split tiles: counters and parts
    float *parts;
    double *partials, *sums;
    float *phi;
};

Workspace carve(char *base, const Work &size, int64_t x_bytes, int64_t u_bytes, int64_t a_bytes, int64_t n_partials) {
    Workspace w{};
    auto take = [&base](int64_t n) {
        char *p = base;
        base += align256(n);
        return p;
    };
    for (int i = 0; i < 2; ++i) {
        w.f.x[i] = take(i == 0 ? x_bytes : std::max(x_bytes, u_bytes));
        w.f.xt[i] = take(x_bytes);
    }
    for (int i = 0; i < size.squares(); ++i) w.f.square[i] = take(a_bytes);
    w.arrived = reinterpret_cast<uint32_t *>(take(4 * kMaxSplit));
    w.parts = reinterpret_cast<float *>(take(kMaxPartials * size.part_bytes()));
    w.partials = reinterpret_cast<double *>(take(8 * n_partials));
    w.sums = reinterpret_cast<double *>(base);  // step
    w.phi = reinterpret_cast<float *>(base);    // orthogonalisation
    return w;
}

int check_layout(const muon_layout *l) {
    if (!l) return fail(ADAM_EINVAL, "layout is NULL");
    if (l->storage != MUON_STORE_BF16 && l->storage != MUON_STORE_Q8 && l->storage != MUON_STORE_F32)
        return fail(ADAM_EINVAL, "unknown storage mode " + std::to_string(l->storage));
    if (l->grad_dtype != ADAM_GRAD_F32 && l->grad_dtype != ADAM_GRAD_BF16)
        return fail(ADAM_EINVAL, "unknown grad dtype " + std::to_string(l->grad_dtype));
    if (l->block_size != ADAM_BLOCK_SIZE)
        return fail(ADAM_EINVAL, "block_size must be " + std::to_string(ADAM_BLOCK_SIZE) + ", got " +
                                     std::to_string(l->block_size));
    if (l->options != 0) return fail(ADAM_EINVAL, "unknown layout option bits");
    return ADAM_OK;
}

int check_shape(int64_t rows, int64_t cols, const std::string &what) {
    if (rows < 0 || rows >= kMaxDim || cols < 0 || cols >= kMaxDim)
        return fail(ADAM_EINVAL, "dimension of " + what + " outside [0, 2^21)");
    if (rows * cols >= (int64_t(1) << 32)) return fail(ADAM_EINVAL, "rows * cols of " + what + " is 2^32 or more");
    return ADAM_OK;
}

int check_shapes(int32_t n, const int64_t *rows, const int64_t *cols, std::vector<Shape> &out) {
    if (n < 0) return fail(ADAM_EINVAL, "n_tensors < 0");
    if (n > 0 && (!rows || !cols)) return fail(ADAM_EINVAL, "rows or cols is NULL");
    out.clear();
    out.reserve(n);
    int64_t blocks = 0, padded = 0;
    for (int32_t k = 0; k < n; ++k) {
        if (int rc = check_shape(rows[k], cols[k], "tensor " + std::to_string(k))) return rc;
        out.push_back(Shape{rows[k], cols[k]});
        blocks += blocks_of(out[k].numel());
        padded += pad16(out[k].numel());
    }
    if (blocks >= (int64_t(1) << 31) || padded >= (int64_t(1) << 36))
        return fail(ADAM_EINVAL, "state too large: more than 2^31 - 1 blocks or 2^36 elements");
    return ADAM_OK;
}

int check_iteration(const muon_iteration &it) {
    if (it.steps < 1 || it.steps > MUON_MAX_STEPS)
        return fail(ADAM_EINVAL, "steps must be in [1, " + std::to_string(MUON_MAX_STEPS) + "]");
    if (!(it.eps > 0.0f) || !std::isfinite(it.eps)) return fail(ADAM_EINVAL, "eps must be finite and > 0");
    if (it.coefficients)
        for (int i = 0; i < 3 * it.steps; ++i)
            if (!(it.coefficients[i] >= -64.0f && it.coefficients[i] <= 64.0f))
                return fail(ADAM_EINVAL, "coefficient " + std::to_string(i) + " outside [-64, 64]");
    return ADAM_OK;
}

int check_hparams(const muon_hparams *hp, int32_t storage) {
    if (!hp) return fail(ADAM_EINVAL, "hparams is NULL");
    if (hp->t < 1) return fail(ADAM_EINVAL, "t must be >= 1");
    if (!(hp->lr >= 0.0f) || !std::isfinite(hp->lr)) return fail(ADAM_EINVAL, "lr must be finite and >= 0");
    if (!(hp->momentum >= 0.0f && hp->momentum < 1.0f)) return fail(ADAM_EINVAL, "momentum must be in [0, 1)");
    if (!(hp->weight_decay >= 0.0f) || !std::isfinite(hp->weight_decay))
        return fail(ADAM_EINVAL, "weight_decay must be finite and >= 0");
    if (hp->scale < MUON_SCALE_NONE || hp->scale > MUON_SCALE_RMS) return fail(ADAM_EINVAL, "unknown scale rule");
    if (hp->flags & ~(uint32_t)(MUON_F_NESTEROV | MUON_F_STOCHASTIC)) return fail(ADAM_EINVAL, "unknown flag bits");
    if (hp->reserved != 0) return fail(ADAM_EINVAL, "reserved must be 0");
    if ((hp->flags & MUON_F_STOCHASTIC) && storage != MUON_STORE_Q8)
        return fail(ADAM_EINVAL, "stochastic rounding applies to 8-bit storage only");
    return check_iteration(hp->iteration);
}

constexpr int64_t kDrawIndexLimit = int64_t(1) << 62;

int check_draw_first(const std::vector<Shape> &shapes, const int64_t *first) {
    if (!shapes.empty() && !first) return fail(ADAM_EINVAL, "draw index array is NULL");
    for (size_t k = 0; k < shapes.size(); ++k)
        if (first[k] < 0 || first[k] % 16 != 0 || first[k] > kDrawIndexLimit - pad16(shapes[k].numel()))
            return fail(ADAM_EINVAL, "draw index of tensor " + std::to_string(k) +
                                         " must be a multiple of 16 in [0, 2^62 - padded size]");
    return ADAM_OK;
}

int64_t element_bytes(int32_t storage) { return storage == MUON_STORE_F32 ? 4 : (storage == MUON_STORE_BF16 ? 2 : 1); }

// The coefficients of iteration k.
void coefficients_of(const muon_iteration &it, int k, float c[3]) {
    const float *p = it.coefficients ? it.coefficients + 3 * k : kDefaultCoefficients;
    for (int i = 0; i < 3; ++i) c[i] = p[i];
}

MuonSmallArgs small_args(const MuonWork &w, const void *u, bool u_bf16, const muon_iteration &it, int product) {
    MuonSmallArgs a{};
    a.work = w;
    a.u = u;
    a.u_bf16 = u_bf16;
    a.eps = (double)it.eps;
    a.product = product;
    a.steps = it.steps;
    for (int k = 0; k < it.steps; ++k) coefficients_of(it, k, a.coefficients + 3 * k);
    return a;
}

// Iterations go in runs.  Within one, X stays where it is: the iterates are
// polynomials in the run's first A = X X^T, so A' = P A P and X' = (P_2 P_1) X,
// and a run of L costs 3 m^2 n + (4 L - 3) m^3 multiply-adds (symmetric results
// counted by half) for the 3 L m^2 n + L m^3 of one iteration after the other.
// What it costs in accuracy is that A' carries A's rounding, grown by a^2, where
// one iteration after the other forms A anew.  The rounding errors of m^2 entries
// add up to a matrix of norm ~ m^(-1/2), so what counts is m: against plain fp32's
// own error (rank m/16 over a noise of 0.1, in fp64) the result was off by
// 1.1 to 1.25 times that with no runs; with runs by 4 times at 64 x 5000, 1.4 at
// 256 x 4096, 0.9 at 600 x 5000, and by 30 times with three iterations at 3 x 5000.
// So pairs are taken from kPairShort rows on, three iterations from kTripleShort
// on, once, first, and while |a_1 a_2| is at most kRunGrowth; four fail.
struct Run {
    int first, length;
};
std::vector<Run> runs_of(const muon_iteration &it, const Work &size) {
    auto a = [&](int k) {
        float c[3];
        coefficients_of(it, k, c);
        return std::fabs((double)c[0]);
    };
    std::vector<Run> runs;
    int k = 0;
    if (it.steps % 2 == 1) {  // pairs from the end, three iterations or one before them
        const bool three = size.triples && it.steps > 3 && a(0) * a(1) <= kRunGrowth && a(0) * a(1) * a(2) <= 64.0;
        runs.push_back(Run{0, three ? 3 : 1});
        k = runs[0].length;
    }
    while (size.pairs && k + 1 < it.steps) {
        if (a(k) * a(k + 1) <= 64.0) {  // an entry of P_2 P_1 has to stay below 256
            runs.push_back(Run{k, 2});
            k += 2;
        } else {
            runs.push_back(Run{k++, 1});
        }
    }
    while (k < it.steps) runs.push_back(Run{k++, 1});
    return runs;
}

// Whether a bf16 X_0 can be taken as it is: the first run ends before the last
// iteration.
bool raw_start(const muon_iteration &it, const Work &size) { return runs_of(it, size)[0].length < it.steps; }

// The products of all iterations, X_0 and X_0^T being in f.x[0], f.xt[0].
// raw: they are bf16 values times a power of two in plain slabs, and w.phi times
// them is X_0: their own products need one partial product for three, and P X
// two, in the first run, which is not the last (raw_start).
hipError_t run_products(const Workspace &w, const MuonWork &square, const MuonWork &update, const Work &size, bool raw,
                        const muon_iteration &it, int last, const MuonGemmArgs &into, hipStream_t s) {
    hipError_t e = hipSuccess;
    const MuonArrays &f = w.f;
    auto launch = [&](int product, MuonGemmArgs &g) {
        if (e != hipSuccess) return;
        const bool is_square = product == kGram || product == kPolynomial || product == kCommuting;
        const int tiling = is_square ? size.square_tiling : size.update_tiling;
        const Load &load = product == kGram ? size.gram : (is_square ? size.square : size.update);
        g.work = is_square ? square : update;
        const int in = g.phi ? (product == kGram ? kPlain : kMixed) : kSplit, jobs = g.left2 ? 2 : 1;
        const Cut cut = load.cut(tiling, g.work.n_tiles, jobs, in);
        g.work.window = load.window(tiling);
        g.work.n_whole = cut.whole;
        g.work.parts = cut.parts;
        g.work.partial = w.parts;
        g.work.arrived = w.arrived;
        e = launch_muon_product(tiling, product, in, jobs, g, s);
    };
    auto polynomial = [&](const char *a, char *p, int k) {
        float c[3];
        coefficients_of(it, k, c);
        MuonGemmArgs g{};
        g.left = g.add = a;
        g.out = p;
        g.ca = c[0];
        g.cb = c[1];
        g.cc = c[2];
        launch(kPolynomial, g);
    };
    auto commuting = [&](const char *left, const char *right, char *out, const char *left2 = nullptr,
                         const char *right2 = nullptr, char *out2 = nullptr) {
        MuonGemmArgs g{};
        g.left = left;
        g.right = right;
        g.out = out;
        g.left2 = left2;
        g.right2 = right2;
        g.out2 = out2;
        launch(kCommuting, g);
    };
    // (T, R and U only where the runs' lengths ask for them: Work::squares)
    char *const A = f.square[0], *const P = f.square[1], *const T = f.square[2], *const R = f.square[3],
               *const U = f.square[4];
    int cur = 0;
    for (const Run &run : runs_of(it, size)) {
        const float *phi = raw && run.first == 0 ? w.phi : nullptr;
        MuonGemmArgs g{};
        g.left = f.x[cur];
        g.out = A;
        g.phi = phi;
        launch(kGram, g);
        polynomial(A, P, run.first);
        const char *q = P;
        if (run.length >= 2) {
            commuting(P, A, T);  // A <- P A P
            commuting(P, T, A);
            polynomial(A, R, run.first + 1);
            if (run.length == 2) {
                commuting(R, P, T);
                q = T;
            } else {
                commuting(R, P, U, R, A, T);
                commuting(R, T, A);
                polynomial(A, P, run.first + 2);
                commuting(P, U, T);
                q = T;
            }
        }
        const int next = run.first + run.length;
        g = next < it.steps ? MuonGemmArgs{} : into;
        g.left = q;
        g.right = f.xt[cur];
        if (next < it.steps) {
            g.out = f.x[cur ^ 1];
            g.out_t = f.xt[cur ^ 1];
            g.phi = phi;
            launch(kUpdate, g);
            cur ^= 1;
        } else {
            launch(last, g);
        }
    }
    return e;
}

}  // namespace

struct muon_state {
    int device = -1;
    muon_layout layout{};
    std::vector<Shape> shapes;
    int64_t padded = 0, nblocks = 0;
    std::vector<Group> groups;
    void *m = nullptr;
    float *m_scale = nullptr;
    char *workspace = nullptr;
    char *d_tables = nullptr;  // block descriptors, draw indices, the groups' tables
    BlockDesc *d_desc = nullptr;
    std::vector<int64_t> draw_first;
    uint64_t *d_draw = nullptr;
    // device copies of the caller's pointer pairs: a few recent sets stay
    // resident, new ones go through a ring of pinned buffers
    TableSlot tables[kTableSlots];
    uint64_t table_clock = 0;
    TensorRef *stage[kStageSlots] = {};
    hipEvent_t stage_done[kStageSlots] = {};
    bool stage_pending[kStageSlots] = {};
    int next_stage = 0;
    int32_t n() const { return (int32_t)shapes.size(); }
};

namespace {

void release(muon_state *s) {
    if (!s) return;
    if (s->device >= 0) {
        int cur = -1;
        (void)hipGetDevice(&cur);
        if (cur != s->device) (void)hipSetDevice(s->device);
        (void)hipDeviceSynchronize();
        for (int i = 0; i < kStageSlots; ++i) {
            if (s->stage_done[i]) (void)hipEventDestroy(s->stage_done[i]);
            (void)hipHostFree(s->stage[i]);
        }
        for (int i = 0; i < kTableSlots; ++i) (void)hipFree(s->tables[i].dev);
        (void)hipFree(s->m);
        (void)hipFree(s->m_scale);
        (void)hipFree(s->workspace);
        (void)hipFree(s->d_tables);
        if (cur >= 0 && cur != s->device) (void)hipSetDevice(cur);
    }
    delete s;
}

int alloc(void **p, int64_t bytes) {
    if (bytes == 0) return ADAM_OK;
    if (hipMalloc(p, (size_t)bytes) != hipSuccess) {
        (void)hipGetLastError();
        *p = nullptr;
        return fail(ADAM_ENOMEM, "hipMalloc of " + std::to_string(bytes) + " bytes failed");
    }
    return ADAM_OK;
}

int alloc_zeroed(void **p, int64_t bytes, hipStream_t stream) {
    if (int rc = alloc(p, bytes)) return rc;
    if (bytes == 0) return ADAM_OK;
    hipError_t e = hipMemsetAsync(*p, 0, (size_t)bytes, stream);
    return e == hipSuccess ? ADAM_OK : hip_fail(e, "hipMemsetAsync");
}

// The descriptors and tiles of a group; long products first, so that the
// last workgroups of a launch are short ones.
void build_tables(Group &g, const std::vector<Shape> &shapes) {
    std::vector<int32_t> order;
    int64_t flat = 0, block = 0;
    std::vector<int64_t> flats, firsts;
    for (int32_t k = g.first; k < g.last; ++k) {
        flats.push_back(flat);
        firsts.push_back(block);
        flat += pad16(shapes[k].numel());
        block += blocks_of(shapes[k].numel());
        if (shapes[k].numel() > 0) order.push_back(k);
    }
    std::stable_sort(order.begin(), order.end(),
                     [&](int32_t a, int32_t b) { return shapes[a].longer() > shapes[b].longer(); });
    uint64_t x_off = 0, a_off = 0;
    const int64_t pad = g.size.pad();
    const uint32_t S = size_of(g.size.square_tiling), U = size_of(g.size.update_tiling);
    for (int32_t k : order) {
        const Shape &s = shapes[k];
        MuonMat m{};
        m.x_off = x_off;
        m.a_off = a_off;
        m.u_off = (uint64_t)flats[k - g.first];
        m.u_ld = (uint64_t)s.cols;
        m.mp = (uint32_t)pad_to(s.shorter(), pad);
        m.np = (uint32_t)pad_to(s.longer(), pad);
        m.rows = (uint32_t)s.rows;
        m.cols = (uint32_t)s.cols;
        m.tall = s.rows > s.cols;
        m.index = (uint32_t)k;
        const uint32_t i = (uint32_t)g.mats.size();
        m.norm = i;
        m.scale_spectral = std::sqrt(std::max(1.0, (double)s.rows / (double)s.cols));
        m.scale_rms = 0.2 * std::sqrt((double)s.longer());
        if (!is_small(s)) {
            x_off += 4ull * m.mp * m.np;
            a_off += 4ull * m.mp * m.mp;
        }
        g.mats.push_back(m);
        const int64_t b0 = firsts[k - g.first];
        g.ranges.push_back(uint2{(uint32_t)b0, (uint32_t)(b0 + blocks_of(s.numel()))});
        if (is_small(s)) {
            g.small.push_back(MuonTile{i, 0, 0});
            g.small_short = std::max(g.small_short, s.shorter());
            g.small_long = std::max(g.small_long, s.longer());
            continue;
        }
        const uint32_t sb = m.mp / S, mb = m.mp / U, nb = m.np / U;
        const uint32_t pr = (m.tall ? m.np : m.mp) / 64, pc = (m.tall ? m.mp : m.np) / 64;
        for (uint32_t a = 0; a < pr; ++a)
            for (uint32_t b = 0; b < pc; ++b) g.prep.push_back(MuonTile{i, (uint16_t)a, (uint16_t)b});
        for (uint32_t a = 0; a < sb; ++a)
            for (uint32_t b = 0; b <= a; ++b) g.square.push_back(MuonTile{i, (uint16_t)a, (uint16_t)b});
        for (uint32_t a0 = 0; a0 < mb; a0 += 8)  // bands of 8 tile rows, as the kernel takes them
            for (uint32_t b = 0; b < nb; ++b)
                for (uint32_t a = a0; a < std::min(mb, a0 + 8); ++a)
                    g.update.push_back(MuonTile{i, (uint16_t)a, (uint16_t)b});
    }
}

struct BufferView {
    void *ptr;
    int64_t bytes;
};

BufferView buffer_of(const muon_state *s, int32_t which) {
    const int32_t st = s->layout.storage;
    switch (which) {
    case ADAM_BUF_M_CODES: return st == MUON_STORE_Q8 ? BufferView{s->m, s->padded} : BufferView{nullptr, -1};
    case ADAM_BUF_M_SCALE: return st == MUON_STORE_Q8 ? BufferView{s->m_scale, 4 * s->nblocks} : BufferView{nullptr, -1};
    case ADAM_BUF_M_BF16: return st == MUON_STORE_BF16 ? BufferView{s->m, 2 * s->padded} : BufferView{nullptr, -1};
    case ADAM_BUF_M_F32: return st == MUON_STORE_F32 ? BufferView{s->m, 4 * s->padded} : BufferView{nullptr, -1};
    default: return BufferView{nullptr, -1};
    }
}

std::vector<int32_t> buffers_of(int32_t storage) {
    if (storage == MUON_STORE_Q8) return {ADAM_BUF_M_CODES, ADAM_BUF_M_SCALE};
    return {storage == MUON_STORE_BF16 ? ADAM_BUF_M_BF16 : ADAM_BUF_M_F32};
}

template <class T>
const T *place(std::vector<char> &bytes, const std::vector<T> &v) {  // as an offset, until the array is on the device
    bytes.resize((bytes.size() + 15) / 16 * 16);
    const size_t at = bytes.size();
    bytes.resize(at + v.size() * sizeof(T));
    if (!v.empty()) std::memcpy(bytes.data() + at, v.data(), v.size() * sizeof(T));
    return reinterpret_cast<const T *>(at);
}
template <class T>
const T *rebase(char *base, const T *offset) {
    return reinterpret_cast<const T *>(base + reinterpret_cast<size_t>(offset));
}

int create(muon_state **out, std::vector<Shape> shapes, const muon_layout *layout, const int64_t *draw_first,
           hipStream_t stream) {
    muon_state *s = new muon_state();
    struct Guard {
        muon_state *s;
        ~Guard() { release(s); }
    } guard{s};
    hipError_t e = hipGetDevice(&s->device);
    if (e != hipSuccess) {
        s->device = -1;
        return hip_fail(e, "hipGetDevice");
    }
    s->layout = *layout;
    s->shapes = std::move(shapes);
    const int32_t n = s->n();
    std::vector<BlockDesc> desc;
    s->draw_first.resize(n);
    for (int32_t k = 0; k < n; ++k) {
        const int64_t len = s->shapes[k].numel();
        for (int64_t b = 0; b * kBlock < len; ++b)
            desc.push_back(BlockDesc{(uint32_t)((s->padded + b * kBlock) / 16), (uint32_t)k,
                                     (uint32_t)((b << kBlockBits) | (std::min<int64_t>(kBlock, len - b * kBlock) - 1)),
                                     (uint32_t)desc.size()});
        s->draw_first[k] = draw_first ? draw_first[k] : s->padded;
        s->padded += pad16(len);
    }
    s->nblocks = (int64_t)desc.size();
    s->groups = plan(s->shapes);
    int64_t work_bytes = 0;
    std::vector<char> bytes;
    const BlockDesc *desc_at = place(bytes, desc);
    const int64_t *draw_at = place(bytes, s->draw_first);
    for (Group &g : s->groups) {
        build_tables(g, s->shapes);
        work_bytes = std::max(work_bytes, group_bytes(g));
        g.d_mats = place(bytes, g.mats);
        g.d_ranges = place(bytes, g.ranges);
        g.d_prep = place(bytes, g.prep);
        g.d_square = place(bytes, g.square);
        g.d_update = place(bytes, g.update);
        g.d_small = place(bytes, g.small);
    }
    int rc;
    if ((rc = alloc_zeroed(&s->m, element_bytes(layout->storage) * s->padded, stream)) ||
        (layout->storage == MUON_STORE_Q8 && (rc = alloc_zeroed((void **)&s->m_scale, 4 * s->nblocks, stream))) ||
        (rc = alloc((void **)&s->workspace, work_bytes)) || (rc = alloc((void **)&s->d_tables, (int64_t)bytes.size())))
        return rc;
    if (!bytes.empty()) {
        if ((e = hipMemcpyAsync(s->d_tables, bytes.data(), bytes.size(), hipMemcpyHostToDevice, stream)) != hipSuccess)
            return hip_fail(e, "table upload");
        s->d_desc = const_cast<BlockDesc *>(rebase(s->d_tables, desc_at));
        s->d_draw = reinterpret_cast<uint64_t *>(const_cast<int64_t *>(rebase(s->d_tables, draw_at)));
        for (Group &g : s->groups) {
            g.d_mats = rebase(s->d_tables, g.d_mats);
            g.d_ranges = rebase(s->d_tables, g.d_ranges);
            g.d_prep = rebase(s->d_tables, g.d_prep);
            g.d_square = rebase(s->d_tables, g.d_square);
            g.d_update = rebase(s->d_tables, g.d_update);
            g.d_small = rebase(s->d_tables, g.d_small);
        }
    }
    if (n > 0) {
        const size_t tbytes = (size_t)n * sizeof(TensorRef);
        for (int i = 0; i < kTableSlots; ++i)
            if ((rc = alloc((void **)&s->tables[i].dev, (int64_t)tbytes))) return rc;
        for (int i = 0; i < kStageSlots; ++i) {
            if (hipHostMalloc((void **)&s->stage[i], tbytes, hipHostMallocDefault) != hipSuccess) {
                (void)hipGetLastError();
                return fail(ADAM_ENOMEM, "pinned staging allocation failed");
            }
            if ((e = hipEventCreateWithFlags(&s->stage_done[i], hipEventDisableTiming)) != hipSuccess)
                return hip_fail(e, "hipEventCreate");
        }
    }
    if ((e = hipStreamSynchronize(stream)) != hipSuccess) return hip_fail(e, "hipStreamSynchronize");
    guard.s = nullptr;
    *out = s;
    return ADAM_OK;
}

// The device table that holds these pointers, uploading it if it is new.
int pointer_table(muon_state *s, float *const *params, const void *const *grads, hipStream_t stream, TensorRef **out) {
    const int32_t n = s->n();
    int slot = -1;
    for (int i = 0; i < kTableSlots && slot < 0; ++i) {
        const TableSlot &ts = s->tables[i];
        if (!ts.valid) continue;
        bool same = true;
        for (int32_t k = 0; k < n && same; ++k) same = ts.ptrs[k].p == params[k] && ts.ptrs[k].g == grads[k];
        if (same) slot = i;
    }
    if (slot < 0) {
        std::vector<const void *> seen;
        for (int32_t k = 0; k < n; ++k)
            if (s->shapes[k].numel() > 0) seen.push_back(params[k]);
        std::sort(seen.begin(), seen.end());
        if (std::adjacent_find(seen.begin(), seen.end()) != seen.end())
            return fail(ADAM_EINVAL, "two tensors have the same param pointer");
        slot = 0;  // least recently used (or never used) table
        for (int i = 1; i < kTableSlots; ++i)
            if (!s->tables[i].valid || (s->tables[slot].valid && s->tables[i].last_use < s->tables[slot].last_use)) slot = i;
        TableSlot &ts = s->tables[slot];
        const int st = s->next_stage;
        s->next_stage = (st + 1) % kStageSlots;
        hipError_t e;
        if (s->stage_pending[st]) {  // the ring wrapped onto a copy still queued
            if ((e = hipEventSynchronize(s->stage_done[st])) != hipSuccess) return hip_fail(e, "hipEventSynchronize");
            s->stage_pending[st] = false;
        }
        ts.valid = false;
        ts.ptrs.resize(n);
        for (int32_t k = 0; k < n; ++k) ts.ptrs[k] = TensorRef{params[k], grads[k]};
        std::memcpy(s->stage[st], ts.ptrs.data(), n * sizeof(TensorRef));
        e = hipMemcpyAsync(ts.dev, s->stage[st], n * sizeof(TensorRef), hipMemcpyHostToDevice, stream);
        if (e != hipSuccess) return hip_fail(e, "pointer table upload");
        if ((e = hipEventRecord(s->stage_done[st], stream)) != hipSuccess) return hip_fail(e, "hipEventRecord");
        s->stage_pending[st] = true;
        ts.valid = true;
    }
    s->tables[slot].last_use = ++s->table_clock;
    *out = s->tables[slot].dev;
    return ADAM_OK;
}

MuonWork table_work(const Group &g, const MuonTile *tiles, size_t count) {
    MuonWork w{};
    w.tiles = tiles;
    w.mats = g.d_mats;
    w.n_tiles = (uint32_t)count;
    w.per_mat = 1;
    return w;
}

}  // namespace

extern "C" {

int64_t muon_state_bytes(int32_t n_tensors, const int64_t *rows, const int64_t *cols, const muon_layout *layout) {
    return guarded([&]() -> int64_t {
        std::vector<Shape> shapes;
        if (int rc = check_shapes(n_tensors, rows, cols, shapes)) return rc;
        if (int rc = check_layout(layout)) return rc;
        int64_t total = 0;
        for (const Shape &s : shapes)
            total += pad16(s.numel()) * element_bytes(layout->storage) +
                     (layout->storage == MUON_STORE_Q8 ? 4 * blocks_of(s.numel()) : 0);
        return total;
    });
}

int64_t muon_state_workspace_bytes(int32_t n_tensors, const int64_t *rows, const int64_t *cols,
                                   const muon_layout *layout) {
    return guarded([&]() -> int64_t {
        std::vector<Shape> shapes;
        if (int rc = check_shapes(n_tensors, rows, cols, shapes)) return rc;
        if (int rc = check_layout(layout)) return rc;
        int64_t most = 0;
        for (const Group &g : plan(shapes)) most = std::max(most, group_bytes(g));
        return most;
    });
}

int muon_state_create(muon_state **out, int32_t n_tensors, const int64_t *rows, const int64_t *cols,
                      const muon_layout *layout, void *hip_stream) {
    return guarded([&]() -> int {
        if (!out) return fail(ADAM_EINVAL, "out is NULL");
        *out = nullptr;
        std::vector<Shape> shapes;
        if (int rc = check_shapes(n_tensors, rows, cols, shapes)) return rc;
        if (int rc = check_layout(layout)) return rc;
        return create(out, std::move(shapes), layout, nullptr, reinterpret_cast<hipStream_t>(hip_stream));
    });
}

void muon_state_destroy(muon_state *s) { release(s); }

int muon_step(muon_state *s, float *const *params, const void *const *grads, const muon_hparams *hp,
              const muon_layout *expect, void *hip_stream) {
    return guarded([&]() -> int {
        if (!s) return fail(ADAM_EINVAL, "state is NULL");
        if (!expect) return fail(ADAM_EINVAL, "expected layout is NULL");
        if (expect->storage != s->layout.storage || expect->grad_dtype != s->layout.grad_dtype ||
            expect->block_size != s->layout.block_size || expect->options != s->layout.options)
            return fail(ADAM_EMODE, "layout differs from the one the state was created with");
        int rc = check_hparams(hp, s->layout.storage);
        if (rc) return rc;
        const int32_t n = s->n();
        if (n > 0 && (!params || !grads)) return fail(ADAM_EINVAL, "params or grads is NULL");
        for (int32_t k = 0; k < n; ++k) {
            if (s->shapes[k].numel() == 0) continue;
            if (!params[k] || !grads[k]) return fail(ADAM_EINVAL, "NULL pointer for tensor " + std::to_string(k));
            if ((reinterpret_cast<uintptr_t>(params[k]) | reinterpret_cast<uintptr_t>(grads[k])) & 15u)
                return fail(ADAM_EALIGN, "tensor " + std::to_string(k) + " is not 16-byte aligned");
        }
        if (s->nblocks == 0) return ADAM_OK;
        int dev = -1;
        hipError_t e = hipGetDevice(&dev);
        if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
        if (dev != s->device)
            return fail(ADAM_EINVAL, "state lives on device " + std::to_string(s->device) + ", current is " +
                                         std::to_string(dev));
        hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
        // a graph would replay this call's t, hyperparameters and pointer table
        hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
        if ((e = hipStreamIsCapturing(stream, &capture)) != hipSuccess) return hip_fail(e, "hipStreamIsCapturing");
        if (capture != hipStreamCaptureStatusNone)
            return fail(ADAM_EINVAL, "muon_step cannot be recorded into a graph: the stream is capturing");
        TensorRef *tensors = nullptr;
        if ((rc = pointer_table(s, params, grads, stream, &tensors))) return rc;

        for (const Group &g : s->groups) {
            const Workspace w = carve(s->workspace, g.size, g.x_bytes, g.u_bytes, g.a_bytes, g.blocks);
            MuonStepArgs a{};
            a.desc = s->d_desc + g.block0;
            a.tensors = tensors;
            a.draw_first = s->d_draw;
            a.m_state = s->m;
            a.m_scale = s->m_scale;
            a.u = reinterpret_cast<float *>(w.f.x[1]);  // free until the first iteration writes there
            a.partials = w.partials;
            a.u_base = (uint64_t)g.flat0;
            a.slot_base = (uint32_t)g.block0;
            a.n_blocks = (uint32_t)g.blocks;
            a.beta = hp->momentum;
            a.omb = (float)(1.0 - (double)hp->momentum);
            a.nesterov = (hp->flags & MUON_F_NESTEROV) ? 1u : 0u;
            a.seed_lo = (uint32_t)hp->seed;
            a.seed_hi = (uint32_t)(hp->seed >> 32);
            a.t_lo = (uint32_t)(uint64_t)hp->t;
            a.t_hi = (uint32_t)((uint64_t)hp->t >> 32);
            if ((e = launch_muon_momentum(s->layout.storage, s->layout.grad_dtype == ADAM_GRAD_BF16,
                                          (hp->flags & MUON_F_STOCHASTIC) != 0, a, stream)) != hipSuccess)
                return hip_fail(e, "momentum launch");
            MuonGemmArgs into{};
            into.tensors = tensors;
            into.lr = (double)hp->lr;
            into.decay = (float)(1.0 - (double)hp->lr * (double)hp->weight_decay);
            into.scale = hp->scale;
            if (!g.small.empty()) {
                MuonSmallArgs small = small_args(table_work(g, g.d_small, g.small.size()), a.u, false, hp->iteration,
                                                 kLastParams);
                small.tensors = into.tensors;
                small.lr = into.lr;
                small.decay = into.decay;
                small.scale = into.scale;
                if ((e = launch_muon_small(g.small_short, g.small_long, small, stream)) != hipSuccess)
                    return hip_fail(e, "small matrices' launch");
            }
            if (g.update.empty()) continue;
            if ((e = launch_muon_norms(w.partials, g.d_ranges, w.sums, (uint32_t)g.mats.size(), stream)) != hipSuccess)
                return hip_fail(e, "norm launch");
            MuonPrepArgs p{};
            p.arrived = w.arrived;
            p.u = a.u;
            p.partials = w.sums;
            p.n_partials = 1;
            p.eps = (double)hp->iteration.eps;
            p.x = w.f.x[0];
            p.xt = w.f.xt[0];
            if ((e = launch_muon_prep(false, false, kSplit, table_work(g, g.d_prep, g.prep.size()), p, stream)) !=
                hipSuccess)
                return hip_fail(e, "preparation launch");
            if ((e = run_products(w, table_work(g, g.d_square, g.square.size()),
                                  table_work(g, g.d_update, g.update.size()), g.size, false, hp->iteration, kLastParams, into,
                                  stream)) != hipSuccess)
                return hip_fail(e, "product launch");
        }
        return ADAM_OK;
    });
}

int64_t muon_state_buffer_bytes(const muon_state *s, int32_t which) {
    return guarded([&]() -> int64_t {
        if (!s) return fail(ADAM_EINVAL, "state is NULL");
        const BufferView b = buffer_of(s, which);
        if (b.bytes < 0) return fail(ADAM_EINVAL, "buffer " + std::to_string(which) + " absent in this storage mode");
        return b.bytes;
    });
}

static int copy_buffer(muon_state *s, int32_t which, void *dst, const void *src, int64_t nbytes, void *hip_stream,
                       bool read) {
    return guarded([&]() -> int {
        const int64_t have = muon_state_buffer_bytes(s, which);
        if (have < 0) return (int)have;
        if (nbytes != have)
            return fail(ADAM_EINVAL, "nbytes " + std::to_string(nbytes) + " != buffer size " + std::to_string(have));
        if (nbytes == 0) return ADAM_OK;
        if (read ? !dst : !src) return fail(ADAM_EINVAL, "NULL buffer pointer");
        void *at = buffer_of(s, which).ptr;
        hipError_t e = hipMemcpyAsync(read ? dst : at, read ? at : src, (size_t)nbytes, hipMemcpyDefault,
                                      reinterpret_cast<hipStream_t>(hip_stream));
        return e == hipSuccess ? ADAM_OK : hip_fail(e, "hipMemcpyAsync");
    });
}

int muon_state_read(muon_state *s, int32_t which, void *dst, int64_t nbytes, void *hip_stream) {
    return copy_buffer(s, which, dst, nullptr, nbytes, hip_stream, true);
}

int muon_state_write(muon_state *s, int32_t which, const void *src, int64_t nbytes, void *hip_stream) {
    return copy_buffer(s, which, nullptr, src, nbytes, hip_stream, false);
}

int muon_state_momentum(muon_state *s, void *dst, int64_t nbytes, void *hip_stream) {
    return guarded([&]() -> int {
        if (!s) return fail(ADAM_EINVAL, "state is NULL");
        const int64_t need = s->padded * (s->layout.storage == MUON_STORE_BF16 ? 2 : 4);
        if (nbytes != need)
            return fail(ADAM_EINVAL, "nbytes " + std::to_string(nbytes) + " != momentum size " + std::to_string(need));
        if (nbytes == 0) return ADAM_OK;
        if (!dst) return fail(ADAM_EINVAL, "NULL destination");
        if (reinterpret_cast<uintptr_t>(dst) & 15u) return fail(ADAM_EALIGN, "destination is not 16-byte aligned");
        int dev = -1;
        hipError_t e = hipGetDevice(&dev);
        if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
        if (dev != s->device)
            return fail(ADAM_EINVAL, "state lives on device " + std::to_string(s->device) + ", current is " +
                                         std::to_string(dev));
        e = launch_muon_decode(s->layout.storage, s->d_desc, (uint32_t)s->nblocks, s->m, s->m_scale, dst,
                                          reinterpret_cast<hipStream_t>(hip_stream));
        return e == hipSuccess ? ADAM_OK : hip_fail(e, "decode launch");
    });
}

}  // extern "C"

// ---------------------------------------------------------------- checkpoint
namespace {
constexpr char kMagic[8] = {'M', 'E', 'A', 'M', 'M', 'U', 'O', 'N'};
constexpr uint32_t kFormatVersion = 1;
constexpr uint32_t kEndMarker = 0xFFFFFFFFu;

int64_t align8(int64_t n) { return pad_to(n, 8); }
int64_t header_bytes(int64_t n) { return 40 + 24 * n; }

// 64-bit multiply-xor hash over whole 8-byte words (little-endian).
uint64_t stream_hash(const uint8_t *p, int64_t n) {
    uint64_t h = 0x9E3779B97F4A7C15ull ^ (uint64_t)n;
    for (int64_t i = 0; i + 8 <= n; i += 8) {
        uint64_t w;
        std::memcpy(&w, p + i, 8);
        h = (h ^ w) * 0x100000001B3ull;
        h ^= h >> 29;
    }
    return h ^ (h >> 32);
}

template <class T>
void put(uint8_t *base, int64_t &off, T v) {
    std::memcpy(base + off, &v, sizeof(T));
    off += sizeof(T);
}
template <class T>
T get(const uint8_t *base, int64_t &off) {
    T v;
    std::memcpy(&v, base + off, sizeof(T));
    off += sizeof(T);
    return v;
}
}  // namespace

extern "C" {

int64_t muon_state_serialized_bytes(const muon_state *s) {
    return guarded([&]() -> int64_t {
        if (!s) return fail(ADAM_EINVAL, "state is NULL");
        int64_t n = header_bytes(s->n());
        for (int32_t b : buffers_of(s->layout.storage)) n += 16 + align8(buffer_of(s, b).bytes);
        return n + 16;
    });
}

int muon_state_save(muon_state *s, void *dst, int64_t nbytes, void *hip_stream) {
    return guarded([&]() -> int {
        if (!s || !dst) return fail(ADAM_EINVAL, "state or destination is NULL");
        const int64_t need = muon_state_serialized_bytes(s);
        if (nbytes != need)
            return fail(ADAM_EINVAL, "nbytes " + std::to_string(nbytes) + " != serialized size " + std::to_string(need));
        uint8_t *out = static_cast<uint8_t *>(dst);
        hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
        std::memcpy(out, kMagic, 8);
        int64_t off = 8;
        put<uint32_t>(out, off, kFormatVersion);
        put<uint32_t>(out, off, (uint32_t)header_bytes(s->n()));
        put<int32_t>(out, off, s->layout.storage);
        put<int32_t>(out, off, s->layout.grad_dtype);
        put<int32_t>(out, off, s->layout.block_size);
        put<uint32_t>(out, off, s->layout.options);
        put<int32_t>(out, off, s->n());
        put<uint32_t>(out, off, 0u);
        for (const Shape &z : s->shapes) put<int64_t>(out, off, z.rows);
        for (const Shape &z : s->shapes) put<int64_t>(out, off, z.cols);
        for (int64_t d : s->draw_first) put<int64_t>(out, off, d);
        const std::vector<int32_t> bufs = buffers_of(s->layout.storage);
        hipError_t e;
        for (int32_t b : bufs) {
            const BufferView v = buffer_of(s, b);
            put<uint32_t>(out, off, (uint32_t)b);
            put<uint32_t>(out, off, 0u);
            put<uint64_t>(out, off, (uint64_t)v.bytes);
            if (v.bytes > 0 &&
                (e = hipMemcpyAsync(out + off, v.ptr, (size_t)v.bytes, hipMemcpyDeviceToHost, stream)) != hipSuccess)
                return hip_fail(e, "state copy to host");
            std::memset(out + off + v.bytes, 0, (size_t)(align8(v.bytes) - v.bytes));
            off += align8(v.bytes);
        }
        if ((e = hipStreamSynchronize(stream)) != hipSuccess) return hip_fail(e, "hipStreamSynchronize");
        put<uint32_t>(out, off, kEndMarker);
        put<uint32_t>(out, off, (uint32_t)bufs.size());
        put<uint64_t>(out, off, stream_hash(out, off));
        return ADAM_OK;
    });
}

int muon_state_load(muon_state **out, const void *src, int64_t nbytes, void *hip_stream) {
    return guarded([&]() -> int {
        if (!out || !src) return fail(ADAM_EINVAL, "out or source is NULL");
        *out = nullptr;
        const uint8_t *in = static_cast<const uint8_t *>(src);
        if (nbytes < header_bytes(0) + 16 || nbytes % 8 != 0 || std::memcmp(in, kMagic, 8) != 0)
            return fail(ADAM_EINVAL, "not a serialized Muon state");
        int64_t off = 8;
        const uint32_t version = get<uint32_t>(in, off), hbytes = get<uint32_t>(in, off);
        if (version != kFormatVersion)
            return fail(ADAM_EINVAL, "unsupported state format version " + std::to_string(version));
        muon_layout lay{};
        lay.storage = get<int32_t>(in, off);
        lay.grad_dtype = get<int32_t>(in, off);
        lay.block_size = get<int32_t>(in, off);
        lay.options = get<uint32_t>(in, off);
        const int32_t n = get<int32_t>(in, off);
        const uint32_t zero = get<uint32_t>(in, off);
        if (n < 0 || zero != 0 || (int64_t)hbytes != header_bytes(n) || header_bytes(n) > nbytes - 16)
            return fail(ADAM_EINVAL, "corrupt state header");
        if (int rc = check_layout(&lay)) return rc;
        std::vector<int64_t> rows(n), cols(n), draw(n);
        for (int64_t &v : rows) v = get<int64_t>(in, off);
        for (int64_t &v : cols) v = get<int64_t>(in, off);
        for (int64_t &v : draw) v = get<int64_t>(in, off);
        std::vector<Shape> shapes;
        if (int rc = check_shapes(n, rows.data(), cols.data(), shapes)) return rc;
        if (int rc = check_draw_first(shapes, draw.data())) return rc;
        uint64_t want_hash = 0;
        std::memcpy(&want_hash, in + nbytes - 8, 8);
        if (stream_hash(in, nbytes - 8) != want_hash) return fail(ADAM_EINVAL, "serialized state checksum mismatch");
        int64_t padded = 0, nblocks = 0;
        for (const Shape &z : shapes) {
            padded += pad16(z.numel());
            nblocks += blocks_of(z.numel());
        }
        const std::vector<int32_t> bufs = buffers_of(lay.storage);
        std::vector<std::pair<int64_t, int64_t>> payload;
        for (int32_t b : bufs) {
            if (off + 16 > nbytes - 16) return fail(ADAM_EINVAL, "truncated serialized state");
            const uint32_t id = get<uint32_t>(in, off), pad = get<uint32_t>(in, off);
            const int64_t len = get<int64_t>(in, off);
            const int64_t expect = b == ADAM_BUF_M_SCALE ? 4 * nblocks : element_bytes(lay.storage) * padded;
            if ((int32_t)id != b || pad != 0 || len != expect)
                return fail(ADAM_EINVAL, "state record " + std::to_string(b) + " missing, out of order or of the wrong size");
            if (align8(len) > nbytes - 16 - off) return fail(ADAM_EINVAL, "truncated serialized state");
            payload.emplace_back(off, len);
            off += align8(len);
        }
        if (off != nbytes - 16) return fail(ADAM_EINVAL, "corrupt serialized state trailer");
        const uint32_t end = get<uint32_t>(in, off), count = get<uint32_t>(in, off);
        if (end != kEndMarker || count != bufs.size()) return fail(ADAM_EINVAL, "corrupt serialized state trailer");

        hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
        muon_state *s = nullptr;
        if (int rc = create(&s, std::move(shapes), &lay, draw.data(), stream)) return rc;
        hipError_t e = hipSuccess;
        for (size_t i = 0; i < bufs.size() && e == hipSuccess; ++i)
            if (payload[i].second > 0)
                e = hipMemcpyAsync(buffer_of(s, bufs[i]).ptr, in + payload[i].first, (size_t)payload[i].second,
                                   hipMemcpyHostToDevice, stream);
        if (e == hipSuccess) e = hipStreamSynchronize(stream);
        if (e != hipSuccess) {
            release(s);
            return hip_fail(e, "state copy to device");
        }
        *out = s;
        return ADAM_OK;
    });
}

int muon_state_set_draw_index(muon_state *s, const int64_t *first_index, void *hip_stream) {
    return guarded([&]() -> int {
        if (!s) return fail(ADAM_EINVAL, "state is NULL");
        if (int rc = check_draw_first(s->shapes, first_index)) return rc;
        if (s->n() == 0) return ADAM_OK;
        hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
        std::copy(first_index, first_index + s->n(), s->draw_first.begin());
        // stream order puts the copy after every earlier step that read the table
        hipError_t e = hipMemcpyAsync(s->d_draw, s->draw_first.data(), (size_t)s->n() * 8, hipMemcpyHostToDevice, stream);
        if (e != hipSuccess) return hip_fail(e, "draw-index upload");
        if ((e = hipStreamSynchronize(stream)) != hipSuccess) return hip_fail(e, "hipStreamSynchronize");
        return ADAM_OK;
    });
}

int32_t muon_state_get_draw_index(const muon_state *s, int64_t *first_index, int32_t max_tensors) {
    return guarded([&]() -> int32_t {
        if (!s) return fail(ADAM_EINVAL, "state is NULL");
        if (max_tensors > 0 && !first_index) return fail(ADAM_EINVAL, "first_index is NULL");
        for (int32_t k = 0; k < s->n() && k < max_tensors; ++k) first_index[k] = s->draw_first[k];
        return s->n();
    });
}

int32_t muon_state_describe(const muon_state *s, muon_layout *layout, int64_t *rows, int64_t *cols, int32_t max_tensors) {
    return guarded([&]() -> int32_t {
        if (!s || !layout) return fail(ADAM_EINVAL, "state or layout is NULL");
        if (max_tensors > 0 && (!rows || !cols)) return fail(ADAM_EINVAL, "rows or cols is NULL");
        *layout = s->layout;
        for (int32_t k = 0; k < s->n() && k < max_tensors; ++k) {
            rows[k] = s->shapes[k].rows;
            cols[k] = s->shapes[k].cols;
        }
        return s->n();
    });
}

}  // extern "C"

// ---------------------------------------------------------------- orthogonalisation
namespace {

// How a batch is cut: `chunk` matrices go through the products together.
struct BatchPlan {
    int64_t chunk = 1;
    Work size;                         // of a chunk
    int64_t mp = 0, np = 0;            // padded sides
    int64_t x_bytes = 0, a_bytes = 0;  // per matrix
    int64_t n_partials = 1;            // per matrix
    int64_t bytes = 0;
};

BatchPlan plan_batch(int64_t batch, const Shape &s) {
    BatchPlan p;
    p.chunk = std::max<int64_t>(1, std::min<int64_t>(batch, kGroupElements / (tiles_of(s, 128) * 16384)));
    p.size.add(s, (double)p.chunk);
    p.size.choose();
    p.mp = pad_to(s.shorter(), p.size.pad());
    p.np = pad_to(s.longer(), p.size.pad());
    p.x_bytes = 4 * p.mp * p.np;
    p.a_bytes = 4 * p.mp * p.mp;
    p.n_partials = std::min(kMaxSums, tiles_of(s, 64));
    p.bytes = workspace_bytes(p.size, p.x_bytes * p.chunk, 0, p.a_bytes * p.chunk, p.n_partials * p.chunk) + align256(4 * p.chunk);
    return p;
}

}  // namespace

extern "C" {

int64_t muon_orthogonalize_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
    return guarded([&]() -> int64_t {
        if (batch < 0 || batch >= (int64_t(1) << 31)) return fail(ADAM_EINVAL, "batch outside [0, 2^31)");
        if (int rc = check_shape(rows, cols, "the matrices")) return rc;
        if (batch == 0 || rows == 0 || cols == 0 || is_small(Shape{rows, cols})) return 0;
        return plan_batch(batch, Shape{rows, cols}).bytes;
    });
}

int muon_orthogonalize(const muon_matrices *mats, const void *x, void *out, const muon_iteration *iteration,
                       void *workspace, int64_t workspace_bytes, void *hip_stream) {
    return guarded([&]() -> int {
        if (!mats || !iteration) return fail(ADAM_EINVAL, "matrices or iteration is NULL");
        if (int rc = check_iteration(*iteration)) return rc;
        for (int32_t d : {mats->x_dtype, mats->out_dtype})
            if (d != ADAM_GRAD_F32 && d != ADAM_GRAD_BF16) return fail(ADAM_EINVAL, "unknown dtype " + std::to_string(d));
        const int64_t need = muon_orthogonalize_workspace_bytes(mats->batch, mats->rows, mats->cols);
        if (need < 0) return (int)need;
        const Shape shape{mats->rows, mats->cols};
        constexpr int64_t kMaxStride = int64_t(1) << 40, kMaxReach = int64_t(1) << 60;
        for (int64_t v : {mats->x_batch_stride, mats->x_row_stride, mats->out_batch_stride, mats->out_row_stride})
            if (v < 0 || v > kMaxStride) return fail(ADAM_EINVAL, "stride outside [0, 2^40]");
        if (mats->x_row_stride < shape.cols || mats->out_row_stride < shape.cols)
            return fail(ADAM_EINVAL, "row stride smaller than cols");
        if (mats->batch == 0 || shape.numel() == 0) return ADAM_OK;
        if (!x || !out || (need > 0 && !workspace)) return fail(ADAM_EINVAL, "NULL pointer");
        if (workspace_bytes < need)
            return fail(ADAM_EINVAL, "workspace of " + std::to_string(workspace_bytes) + " bytes, " + std::to_string(need) +
                                         " needed");
        const int64_t xe = mats->x_dtype == ADAM_GRAD_BF16 ? 2 : 4, oe = mats->out_dtype == ADAM_GRAD_BF16 ? 2 : 4;
        if (reinterpret_cast<uintptr_t>(x) % xe || reinterpret_cast<uintptr_t>(out) % oe)
            return fail(ADAM_EALIGN, "x or out is not aligned to its element");
        if (reinterpret_cast<uintptr_t>(workspace) % 256) return fail(ADAM_EALIGN, "workspace is not 256-byte aligned");
        // elements from the first of a matrix, and of all matrices, to the last
        const int64_t x_span = (shape.rows - 1) * mats->x_row_stride + shape.cols;
        const int64_t out_span = (shape.rows - 1) * mats->out_row_stride + shape.cols;
        int64_t x_all, out_all;
        if (__builtin_mul_overflow(mats->batch - 1, mats->x_batch_stride, &x_all) ||
            __builtin_mul_overflow(mats->batch - 1, mats->out_batch_stride, &out_all) || x_all >= kMaxReach - x_span ||
            out_all >= kMaxReach - out_span)
            return fail(ADAM_EINVAL, "strides reach beyond 2^60 elements");
        x_all += x_span;
        out_all += out_span;
        // one matrix after the other, or (heads of a fused weight) all their first rows
        // beside each other, then all their second ones
        const bool beside = mats->out_batch_stride >= shape.cols &&
                            (mats->batch - 1) * mats->out_batch_stride + shape.cols <= mats->out_row_stride;
        if (mats->batch > 1 && mats->out_batch_stride < out_span && !beside)
            return fail(ADAM_EINVAL, "out's matrices overlap: they are neither one after the other nor side by side");
        const bool in_place = x == out && xe == oe && mats->x_row_stride == mats->out_row_stride &&
                              (mats->batch == 1 || mats->x_batch_stride == mats->out_batch_stride);
        // interleaved views (one's rows between the other's) are refused too
        auto meet = [](const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
            const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
            return p < q + (uintptr_t)b_bytes && q < p + (uintptr_t)a_bytes;
        };
        if (!in_place && meet(x, x_all * xe, out, out_all * oe)) return fail(ADAM_EINVAL, "out overlaps x");
        if (need > 0 && (meet(workspace, need, x, x_all * xe) || meet(workspace, need, out, out_all * oe)))
            return fail(ADAM_EINVAL, "workspace overlaps x or out");

        hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
        MuonWork work{};
        work.one.rows = (uint32_t)shape.rows;
        work.one.cols = (uint32_t)shape.cols;
        work.one.u_ld = (uint64_t)mats->x_row_stride;
        work.one.o_ld = (uint64_t)mats->out_row_stride;
        work.one.tall = shape.rows > shape.cols;
        work.u_stride = (uint64_t)mats->x_batch_stride;
        work.o_stride = (uint64_t)mats->out_batch_stride;
        hipError_t e;
        if (is_small(shape)) {
            work.per_mat = 1;
            for (int64_t first = 0; first < mats->batch; first += kSmallBatch) {
                work.n_tiles = (uint32_t)std::min(kSmallBatch, mats->batch - first);
                work.one.u_off = (uint64_t)(first * mats->x_batch_stride);
                work.one.o_off = (uint64_t)(first * mats->out_batch_stride);
                MuonSmallArgs small = small_args(work, x, xe == 2, *iteration, oe == 2 ? kLastBf16 : kLastF32);
                small.o = out;
                if ((e = launch_muon_small(shape.shorter(), shape.longer(), small, stream)) != hipSuccess)
                    return hip_fail(e, "launch");
            }
            return ADAM_OK;
        }
        const BatchPlan p = plan_batch(mats->batch, shape);
        const Workspace w = carve(static_cast<char *>(workspace), p.size, p.x_bytes * p.chunk, 0, p.a_bytes * p.chunk,
                                  p.n_partials * p.chunk);
        work.one.mp = (uint32_t)p.mp;
        work.one.np = (uint32_t)p.np;
        work.x_stride = (uint64_t)p.x_bytes;
        work.a_stride = (uint64_t)p.a_bytes;
        work.norm_stride = (uint32_t)p.n_partials;
        for (int64_t first = 0; first < mats->batch; first += p.chunk) {
            const int64_t count = std::min(p.chunk, mats->batch - first);
            work.one.u_off = (uint64_t)(first * mats->x_batch_stride);
            work.one.o_off = (uint64_t)(first * mats->out_batch_stride);
            auto with = [&](int64_t per_mat) {
                MuonWork v = work;
                v.per_mat = (uint32_t)per_mat;
                v.n_tiles = (uint32_t)(per_mat * count);
                return v;
            };
            MuonSumArgs sums{x, w.partials, (uint32_t)p.n_partials};
            if ((e = launch_muon_sums(xe == 2, with(p.n_partials), sums, (uint32_t)count, stream)) != hipSuccess)
                return hip_fail(e, "sum launch");
            MuonPrepArgs prep{};
            prep.arrived = w.arrived;
            prep.u = x;
            prep.partials = w.partials;
            prep.n_partials = (uint32_t)p.n_partials;
            prep.eps = (double)iteration->eps;
            prep.x = w.f.x[0];
            prep.xt = w.f.xt[0];
            prep.phi = w.phi;
            const bool raw = xe == 2 && raw_start(*iteration, p.size);
            if ((e = launch_muon_prep(xe == 2, raw, raw ? kPlain : kSplit, with((p.mp / 64) * (p.np / 64)), prep, stream)) != hipSuccess)
                return hip_fail(e, "preparation launch");
            MuonGemmArgs into{};
            into.o = out;
            Work size = p.size;
            if (count != p.chunk) {  // the last chunk: its own counts, the tilings of the others
                Work rest;
                rest.add(shape, (double)count);
                size.gram = rest.gram;
                size.square = rest.square;
                size.update = rest.update;
            }
            const int64_t sb = p.mp / size_of(size.square_tiling), ub = p.mp / size_of(size.update_tiling),
                          lb = p.np / size_of(size.update_tiling);
            if ((e = run_products(w, with(sb * (sb + 1) / 2), with(ub * lb), size, raw, *iteration,
                                  oe == 2 ? kLastBf16 : kLastF32, into, stream)) != hipSuccess)
                return hip_fail(e, "product launch");
        }
        return ADAM_OK;
    });
}

}  // extern "C"
