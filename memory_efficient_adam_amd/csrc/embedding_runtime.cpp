// Host runtime behind the C ABI declared in include/embedding_mi355x.h:
// argument validation, the workspace's layout and the launches.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <new>
#include <string>

#include "embedding_internal.h"
#include "embedding_mi355x.h"
#include "runtime_common.h"

using namespace adam_mi355x;

namespace {

constexpr int64_t kMaxCount = int64_t(1) << 31;
constexpr int64_t kMaxStride = int64_t(1) << 40, kMaxReach = int64_t(1) << 60;

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

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t element_bytes(int32_t dtype) { return dtype == ADAM_GRAD_BF16 ? 2 : 4; }

int check_sizes(int64_t tokens, int64_t rows, int64_t cols) {
    if (rows < 0 || rows >= kMaxCount || cols < 0 || cols >= kMaxCount)
        return fail(ADAM_EINVAL, "rows or cols outside [0, 2^31)");
    if (tokens < 0 || tokens >= kMaxCount) return fail(ADAM_EINVAL, "tokens outside [0, 2^31)");
    return ADAM_OK;
}

int check_shape(const embedding_shape *s) {
    if (!s) return fail(ADAM_EINVAL, "shape is NULL");
    if (int rc = check_sizes(s->tokens, s->rows, s->cols)) return rc;
    for (int32_t d : {s->table_dtype, s->value_dtype})
        if (d != ADAM_GRAD_F32 && d != ADAM_GRAD_BF16) return fail(ADAM_EINVAL, "unknown dtype " + std::to_string(d));
    if (s->token_dtype != EMBEDDING_TOKENS_I32 && s->token_dtype != EMBEDDING_TOKENS_I64)
        return fail(ADAM_EINVAL, "unknown token dtype " + std::to_string(s->token_dtype));
    if (!std::isfinite(s->scale)) return fail(ADAM_EINVAL, "scale must be finite");
    for (int64_t v : {s->table_stride, s->value_stride})
        if (v < 0 || v > kMaxStride) return fail(ADAM_EINVAL, "stride outside [0, 2^40]");
    if (s->table_stride < s->cols) return fail(ADAM_EINVAL, "table stride smaller than cols");
    // counts below 2^31 times strides up to 2^40 do not overflow 2^71: by division
    for (auto [n, stride] : {std::pair<int64_t, int64_t>{s->rows, s->table_stride}, {s->tokens, s->value_stride}})
        if (n > 1 && stride > (kMaxReach - s->cols) / (n - 1))
            return fail(ADAM_EINVAL, "strides reach beyond 2^60 elements");
    return ADAM_OK;
}

struct Span {
    const void *at;
    int64_t bytes;
};
Span rows_span(const void *at, int64_t n, int64_t stride, int64_t cols, int32_t dtype) {
    return Span{at, n > 0 && cols > 0 ? ((n - 1) * stride + cols) * element_bytes(dtype) : 0};
}
bool meet(const Span &a, const Span &b) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.at), q = reinterpret_cast<uintptr_t>(b.at);
    return a.bytes > 0 && b.bytes > 0 && p < q + (uintptr_t)b.bytes && q < p + (uintptr_t)a.bytes;
}
bool unaligned(const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes != 0; }
int64_t token_bytes(const embedding_shape *s) { return s->token_dtype == EMBEDDING_TOKENS_I64 ? 8 : 4; }
Span token_span(const embedding_shape *s, const void *tokens) { return Span{tokens, s->tokens * token_bytes(s)}; }

// ---------------------------------------------------------------- gradient
// Windows of 32 positions up to this many tokens, which gives more waves something to
// do; of 64 beyond, which leaves fewer partial sums.  us for a bf16 gradient and 32000 x 4096,
// 32 / 64: 8192 tokens as frequent as words are, as a step 94 / 100, added to a table 49 / 48,
// every row as likely as the others 165 / 168 and 67 / 69; 32768 tokens 258 / 251 and 148 / 128,
// every row as likely 443 / 461 and 188 / 187.
constexpr int64_t kSmallTokens = 8192;

struct Plan {
    bool direct;  // in one launch, without a workspace
    uint32_t bucket_bits, passes, bits;
    int64_t window, windows, arrivals_n;
    int64_t arrivals, keys[2], order[2], named, partials, bytes;  // offsets in the workspace, and its size
};

Plan plan_gradient(int64_t tokens, int64_t rows, int64_t cols) {
    Plan p{};
    p.direct = tokens <= kDirectTokens;
    if (p.direct) return p;
    while ((int64_t(kBuckets) << p.bucket_bits) < rows) ++p.bucket_bits;
    p.passes = std::max<uint32_t>(1, (p.bucket_bits + kDigitBits - 1) / kDigitBits);
    p.bits = p.passes == 1 ? p.bucket_bits : kDigitBits;
    p.window = tokens <= kSmallTokens ? 32 : 64;
    p.windows = ceil_div(tokens, p.window);
    p.arrivals_n = 3 * p.windows * ceil_div(cols, 256);
    int64_t at = align256(4 * p.arrivals_n);
    for (uint32_t k = 0; k < (p.passes > 1 ? 2u : 1u); ++k) {
        p.keys[k] = at;
        p.order[k] = at + align256(4 * tokens);
        at = p.order[k] + align256(4 * tokens);
    }
    p.named = at;
    p.partials = at + align256(rows);
    p.bytes = p.partials + align256(2 * p.windows * ((cols + 3) / 4 * 16));
    return p;
}

// What both calls check of the gradient's side.
int check_gradient(const embedding_shape *s, const void *grad, const void *tokens, const void *table,
                   const void *workspace, int64_t workspace_bytes, int64_t need) {
    if (!table || (s->tokens > 0 && (!grad || !tokens)) || (need > 0 && !workspace))
        return fail(ADAM_EINVAL, "NULL pointer");
    if (workspace_bytes < need)
        return fail(ADAM_EINVAL, "workspace of " + std::to_string(workspace_bytes) + " bytes, " + std::to_string(need) +
                                     " needed");
    if (unaligned(grad, element_bytes(s->value_dtype)) || unaligned(table, element_bytes(s->table_dtype)) ||
        unaligned(tokens, token_bytes(s)))
        return fail(ADAM_EALIGN, "grad, tokens or the table is not aligned to its element");
    if (unaligned(workspace, 256)) return fail(ADAM_EALIGN, "workspace is not 256-byte aligned");
    const Span out = rows_span(table, s->rows, s->table_stride, s->cols, s->table_dtype);
    const Span in = rows_span(grad, s->tokens, s->value_stride, s->cols, s->value_dtype), ids = token_span(s, tokens);
    if (meet(out, in) || meet(out, ids)) return fail(ADAM_EINVAL, "the table's side overlaps grad or tokens");
    const Span ws{workspace, need};
    if (meet(ws, out) || meet(ws, in) || meet(ws, ids)) return fail(ADAM_EINVAL, "workspace overlaps another argument");
    return ADAM_OK;
}

SumArgs sum_args(const embedding_shape *s, const Plan &p, Goal goal, const void *grad, void *table, char *ws) {
    SumArgs a{};
    a.tokens_n = (uint32_t)s->tokens;
    a.rows = (uint32_t)s->rows;
    a.grad = grad;
    a.grad_stride = (uint64_t)s->value_stride;
    a.cols = (uint32_t)s->cols;
    a.slices = (uint32_t)ceil_div(s->cols, 256);
    a.scale = s->scale;
    a.out = table;
    a.out_stride = (uint64_t)s->table_stride;
    if (p.direct) return a;
    a.keys = reinterpret_cast<uint32_t *>(ws + p.keys[0]);
    a.order = reinterpret_cast<uint32_t *>(ws + p.order[0]);
    a.window = (uint32_t)p.window;
    a.windows = (uint32_t)p.windows;
    a.named = reinterpret_cast<uint8_t *>(ws + p.named);
    a.partials = reinterpret_cast<float *>(ws + p.partials);
    a.partial_stride = ((uint64_t)s->cols + 3) / 4 * 4;
    a.arrivals = reinterpret_cast<uint32_t *>(ws + p.arrivals);
    return a;
}

int run_gradient(const embedding_shape *s, const Plan &p, const void *tokens, char *ws, const SumArgs &a, Goal goal,
                 hipStream_t stream) {
    const bool grad_bf16 = s->value_dtype == ADAM_GRAD_BF16, out_bf16 = s->table_dtype == ADAM_GRAD_BF16;
    const bool wide = s->token_dtype == EMBEDDING_TOKENS_I64;
    hipError_t e;
    if (p.direct) {
        e = launch_direct(grad_bf16, out_bf16, goal, a, tokens, wide, stream);
        return e == hipSuccess ? ADAM_OK : hip_fail(e, "launch of the sums");
    }
    GroupArgs g{};
    g.tokens = tokens;
    g.tokens_n = a.tokens_n;
    g.rows = a.rows;
    g.wide = wide;
    g.bucket_bits = p.bucket_bits;
    g.passes = p.passes;
    g.bits = p.bits;
    for (int k = 0; k < 2; ++k) {
        g.keys[k] = reinterpret_cast<uint32_t *>(ws + p.keys[k]);
        g.order[k] = reinterpret_cast<uint32_t *>(ws + p.order[k]);
    }
    g.arrivals = a.arrivals;
    g.arrivals_n = (uint64_t)p.arrivals_n;
    g.named = goal == kWrite ? reinterpret_cast<uint8_t *>(ws + p.named) : nullptr;
    if ((e = launch_group(g, stream)) != hipSuccess) return hip_fail(e, "launch of the grouping");
    if ((e = launch_sums(grad_bf16, out_bf16, goal, a, stream)) != hipSuccess) return hip_fail(e, "launch of the sums");
    return ADAM_OK;
}

}  // namespace

extern "C" {

int embedding_lookup(const embedding_shape *shape, const void *table, const void *tokens, void *out, void *hip_stream) {
    return guarded([&]() -> int {
        if (int rc = check_shape(shape)) return rc;
        if (shape->value_stride < shape->cols) return fail(ADAM_EINVAL, "stride of out smaller than cols");
        if (shape->tokens == 0 || shape->cols == 0) return ADAM_OK;
        if ((shape->rows > 0 && !table) || !tokens || !out) return fail(ADAM_EINVAL, "NULL pointer");
        if (unaligned(table, element_bytes(shape->table_dtype)) || unaligned(out, element_bytes(shape->value_dtype)) ||
            unaligned(tokens, token_bytes(shape)))
            return fail(ADAM_EALIGN, "table, tokens or out is not aligned to its element");
        const Span to = rows_span(out, shape->tokens, shape->value_stride, shape->cols, shape->value_dtype);
        if (meet(to, rows_span(table, shape->rows, shape->table_stride, shape->cols, shape->table_dtype)) ||
            meet(to, token_span(shape, tokens)))
            return fail(ADAM_EINVAL, "out overlaps the table or tokens");
        LookupArgs a{};
        a.table = table;
        a.tokens = tokens;
        a.out = out;
        a.table_stride = (uint64_t)shape->table_stride;
        a.out_stride = (uint64_t)shape->value_stride;
        a.tokens_n = (uint32_t)shape->tokens;
        a.rows = (uint32_t)shape->rows;
        a.cols = (uint32_t)shape->cols;
        a.wide = shape->token_dtype == EMBEDDING_TOKENS_I64;
        a.scale = shape->scale;
        const hipError_t e = launch_lookup(shape->table_dtype == ADAM_GRAD_BF16, shape->value_dtype == ADAM_GRAD_BF16, a,
                                           reinterpret_cast<hipStream_t>(hip_stream));
        return e == hipSuccess ? ADAM_OK : hip_fail(e, "launch of the lookup");
    });
}

int64_t embedding_gradient_workspace_bytes(int64_t tokens, int64_t rows, int64_t cols) {
    return guarded([&]() -> int64_t {
        if (int rc = check_sizes(tokens, rows, cols)) return rc;
        if (rows == 0 || cols == 0) return 0;
        return plan_gradient(tokens, rows, cols).bytes;
    });
}

int embedding_gradient(const embedding_shape *shape, const void *grad, const void *tokens, void *table_grad,
                       int32_t accumulate, void *workspace, int64_t workspace_bytes, void *hip_stream) {
    return guarded([&]() -> int {
        if (int rc = check_shape(shape)) return rc;
        if (shape->rows == 0 || shape->cols == 0 || (accumulate && shape->tokens == 0)) return ADAM_OK;
        const Plan p = plan_gradient(shape->tokens, shape->rows, shape->cols);
        if (int rc = check_gradient(shape, grad, tokens, table_grad, workspace, workspace_bytes, p.bytes)) return rc;
        char *ws = static_cast<char *>(workspace);
        const Goal goal = accumulate ? kAdd : kWrite;
        return run_gradient(shape, p, tokens, ws, sum_args(shape, p, goal, grad, table_grad, ws), goal,
                            reinterpret_cast<hipStream_t>(hip_stream));
    });
}

int embedding_adam_step(const embedding_shape *shape, float *table, const void *grad, const void *tokens,
                        void *const *state, const adam_hparams *hp, const adam_layout *layout, void *workspace,
                        int64_t workspace_bytes, void *hip_stream) {
    return guarded([&]() -> int {
        if (int rc = check_shape(shape)) return rc;
        if (int rc = check_adam_layout(layout)) return rc;
        if (layout->storage != ADAM_STORE_F32) return fail(ADAM_EMODE, "the step of rows takes fp32 storage only");
        if (layout->grad_dtype != shape->value_dtype) return fail(ADAM_EMODE, "layout and shape differ in the gradient's type");
        if (int rc = check_adam_hparams(hp, layout->storage)) return rc;
        if (shape->table_dtype != ADAM_GRAD_F32 || shape->table_stride != shape->cols)
            return fail(ADAM_EINVAL, "the table must be fp32 and contiguous");
        if (shape->rows > 0 && shape->cols >= ((int64_t(1) << 32) + shape->rows - 1) / shape->rows)
            return fail(ADAM_EINVAL, "rows * cols outside [0, 2^32)");
        if (shape->rows == 0 || shape->cols == 0 || shape->tokens == 0) return ADAM_OK;
        const Plan p = plan_gradient(shape->tokens, shape->rows, shape->cols);
        if (int rc = check_gradient(shape, grad, tokens, table, workspace, workspace_bytes, p.bytes)) return rc;
        if (!state) return fail(ADAM_EINVAL, "state buffer array is NULL");
        if (unaligned(table, 16)) return fail(ADAM_EALIGN, "the table is not 16-byte aligned");
        const bool ams = (layout->options & ADAM_OPT_AMSGRAD) != 0;
        const int64_t bytes = 4 * ((shape->rows * shape->cols + 15) / 16 * 16);
        const Span whole[] = {rows_span(table, shape->rows, shape->cols, shape->cols, ADAM_GRAD_F32),
                              rows_span(grad, shape->tokens, shape->value_stride, shape->cols, shape->value_dtype),
                              token_span(shape, tokens), Span{workspace, p.bytes}};
        const int32_t buffers[] = {ADAM_BUF_M_F32, ADAM_BUF_V_F32, ADAM_BUF_VMAX_F32};
        for (int k = 0; k < (ams ? 3 : 2); ++k) {
            const Span one{state[buffers[k]], bytes};
            if (!one.at) return fail(ADAM_EINVAL, "state buffer " + std::to_string(buffers[k]) + " is NULL");
            if (unaligned(one.at, 16))
                return fail(ADAM_EALIGN, "state buffer " + std::to_string(buffers[k]) + " is not 16-byte aligned");
            for (const Span &s : whole)
                if (meet(one, s)) return fail(ADAM_EINVAL, "state buffer " + std::to_string(buffers[k]) + " overlaps another argument");
            for (int j = 0; j < k; ++j)
                if (meet(one, Span{state[buffers[j]], bytes})) return fail(ADAM_EINVAL, "state buffers overlap");
        }
        char *ws = static_cast<char *>(workspace);
        const Goal goal = ams ? kAdamMax : kAdam;
        SumArgs a = sum_args(shape, p, goal, grad, table, ws);
        StepArgs scalars{};
        adam_scalars(scalars, hp);
        a.m = static_cast<float *>(state[ADAM_BUF_M_F32]);
        a.v = static_cast<float *>(state[ADAM_BUF_V_F32]);
        a.w = ams ? static_cast<float *>(state[ADAM_BUF_VMAX_F32]) : nullptr;
        a.step = scalars.step;
        a.ibc2 = scalars.ibc2;
        a.decay = scalars.decay;
        a.omb1 = scalars.omb1;
        a.omb2 = scalars.omb2;
        a.beta1 = scalars.beta1;
        a.beta2 = scalars.beta2;
        a.eps = scalars.eps;
        a.wd = scalars.wd;
        a.l2 = scalars.l2;
        a.fast_ok = scalars.fast_ok;
        return run_gradient(shape, p, tokens, ws, a, goal, reinterpret_cast<hipStream_t>(hip_stream));
    });
}

}  // extern "C"
