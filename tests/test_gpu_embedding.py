"""The embedding operations on the GPU against their definitions in 64 bits:
sizes from nothing to several windows and digits, padding, types, strides, streams,
graphs, repeated bits, and the step of rows against the dense one."""
import math

import pytest
import torch

import embedding_ref as R
import memory_efficient_adam_amd as ma

pytestmark = pytest.mark.gpu

F32, BF16, I32, I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _tokens(gen, n, rows, kind="spread", ids=I64):
    """spread: as words are; same: one row; two: two rows by turns; ends: the
    first and last row and what lies just outside the table; none: padding alone."""
    if kind == "same":
        t = torch.full((n,), rows // 2, device="cuda")
    elif kind == "two":
        t = torch.arange(n, device="cuda") % 2 * (rows - 1)
    elif kind == "none":
        t = torch.where(torch.arange(n, device="cuda") % 2 == 0, -1, rows)
    elif kind == "ends":
        far = [2 ** 31 - 1, -2 ** 31] + ([2 ** 32, 2 ** 32 + 1, -2 ** 63, 2 ** 63 - 1] if ids == I64 else [])
        some = torch.tensor([0, rows - 1, -1, rows] + far, device="cuda")
        t = some[torch.randint(0, len(some), (n,), generator=gen, device="cuda")]
    elif kind == "flat":
        t = torch.randint(0, rows, (n,), generator=gen, device="cuda")
    else:
        u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
        t = (torch.exp(u * math.log(rows + 1.0)) - 1).long().clamp(0, rows - 1)
        t = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.1, -1, t)
    return t.to(ids)


def _values(gen, shape, dtype, size=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * size).to(dtype)


def _close(got, want, tolerance, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    over = (got - want).abs() - tolerance
    assert not (over > 0).any(), f"{what}: {int((over > 0).sum())} beyond tolerance, worst by {float(over.max()):.3g}"


def _padding_is_poison(grad, tokens, rows):
    """NaN and infinities in the rows of grad that no sum may read."""
    _, ok = R.inside(tokens, rows)
    bad = (~ok).nonzero().flatten().cuda()
    flat = grad.view(-1, grad.shape[-1])
    flat[bad[::2]] = float("nan")
    flat[bad[1::2]] = float("inf")


# (tokens, rows, cols, kind)
SIZES = [
    (1, 1, 1, "same"), (1, 300, 7, "flat"), (5, 3, 4, "ends"), (2, 2, 3, "two"), (64, 10, 256, "spread"),
    (65, 1, 257, "same"), (63, 1, 512, "same"), (64, 1, 8, "same"), (128, 1, 513, "same"), (129, 2, 5, "two"), (200, 7, 64, "none"),
    (300, 257, 100, "spread"), (1000, 70, 771, "spread"), (1023, 256, 770, "flat"), (1025, 1000, 33, "flat"),
    (5000, 300, 520, "spread"), (4500, 5, 130, "same"), (9000, 33, 64, "two"), (4097, 70001, 36, "flat"),
    (20000, 1000, 96, "spread"), (3000, 131073, 17, "flat"), (3000, 262144, 16, "flat"), (3000, 262145, 16, "flat"),
    (2000, 300007, 9, "ends"),
    # around the numbers of tokens from which another way is taken
    (1024, 60, 300, "spread"), (1025, 60, 300, "spread"), (2048, 60, 300, "spread"), (2049, 60, 300, "spread"),
    (512, 1, 2100, "same"), (2048, 1, 2100, "same"), (1024, 3, 4500, "two"), (2049, 1, 1030, "same"), (7, 2, 5000, "two"),
    (8192, 100, 257, "spread"), (8193, 100, 257, "spread"), (16384, 50, 4, "spread"), (16385, 50, 4, "flat"),
    # runs over more windows than are added up at once, and over more than 64 times 16 of them
    (20000, 1, 9, "same"), (70001, 2, 5, "two"), (140000, 2, 4, "two"),
]


# ---------------------------------------------------------------- lookup
@pytest.mark.parametrize("n,rows,cols,kind", SIZES)
def test_lookup(n, rows, cols, kind):
    gen = _gen(n + cols)
    for i, (table, out, ids) in enumerate([(F32, F32, I64), (F32, BF16, I32), (BF16, BF16, I64), (BF16, F32, I32)]):
        x, tokens = _values(gen, (rows, cols), table), _tokens(gen, n, rows, kind, ids)
        scale = (1.0, math.sqrt(cols), -0.37, 1.0)[i]
        got = ma.embedding_lookup(x, tokens, scale=scale, dtype=out)
        assert got.dtype == out
        want = R.lookup(x, tokens, scale)
        _close(got, want, R.lookup_tolerance(want, out), f"{table} {out}")
        _, ok = R.inside(tokens, rows)
        assert not got[~ok.cuda()].any()


def test_lookup_copies_bits_and_keeps_what_is_not_finite():
    for dtype in (F32, BF16):
        x = torch.tensor([[0.0, -0.0, float("inf"), -float("inf"), float("nan"), 1e-45, -3e38, 1.0]], device="cuda").to(dtype)
        got = ma.embedding_lookup(x, torch.tensor([0, -1, 0], device="cuda"))
        bits = torch.int32 if dtype == F32 else torch.int16
        assert torch.equal(torch.isnan(got[0]), torch.isnan(x[0]))
        keep = ~torch.isnan(x[0])
        assert torch.equal(got[0][keep].view(bits), x[0][keep].view(bits)) and torch.equal(got[0][keep], got[2][keep])
        assert not got[1].view(bits).any()


def test_lookup_of_nothing():
    x = torch.ones(5, 4, device="cuda")
    assert ma.embedding_lookup(x, torch.zeros(0, dtype=I64, device="cuda")).shape == (0, 4)
    assert ma.embedding_lookup(x, torch.zeros(3, 0, dtype=I32, device="cuda")).shape == (3, 0, 4)
    assert ma.embedding_lookup(torch.ones(5, 0, device="cuda"), torch.zeros(2, dtype=I64, device="cuda")).shape == (2, 0)
    got = ma.embedding_lookup(torch.ones(0, 4, device="cuda"), torch.zeros(2, dtype=I64, device="cuda"))
    assert got.shape == (2, 4) and not got.any()
    assert torch.equal(ma.embedding_lookup(x, torch.tensor(3, device="cuda")), x[3])


def test_lookup_strides_and_out():
    gen = _gen(3)
    whole = _values(gen, (40, 100), F32)
    tokens = _tokens(gen, 60, 40, "flat").view(6, 10)
    for x in (whole[:, 3:40], whole[::2, 1:8], whole[5:6, :77].expand(1, 77)):
        t = tokens % x.shape[0]
        assert torch.equal(ma.embedding_lookup(x, t), x[t])
        assert torch.equal(ma.embedding_lookup(x, t.t()), x[t.t()])
        assert torch.equal(ma.embedding_lookup(x, t[:, :-1]), x[t[:, :-1]])
    # into part of a larger buffer, whose other elements stay
    buffer = torch.full((6, 10, 50), 9.0, device="cuda")
    out = buffer[:, :, 5:42]
    assert ma.embedding_lookup(whole[:, 3:40], tokens, out=out) is out
    assert torch.equal(out, whole[:, 3:40][tokens]) and (buffer[:, :, :5] == 9).all() and (buffer[:, :, 42:] == 9).all()


# ---------------------------------------------------------------- gradient
@pytest.mark.parametrize("n,rows,cols,kind", SIZES)
def test_gradient(n, rows, cols, kind):
    gen = _gen(n * 3 + cols)
    cases = [(F32, F32, I64, False), (BF16, F32, I32, False), (BF16, BF16, I64, False), (F32, BF16, I32, True),
             (BF16, F32, I64, True), (BF16, BF16, I32, True)]
    for i, (dtype, out, ids, accumulate) in enumerate(cases):
        tokens, grad = _tokens(gen, n, rows, kind, ids), _values(gen, (n, cols), dtype)
        _padding_is_poison(grad, tokens, rows)
        scale = (1.0, math.sqrt(cols), -0.37)[i % 3]
        total, size, terms = R.gradient(torch.nan_to_num(grad, 0.0, 0.0, 0.0), tokens, rows, scale)
        if accumulate:
            into = _values(gen, (rows, cols), out)
            old = into.clone()
            got = ma.embedding_gradient(grad, tokens, rows, scale=scale, out=into, accumulate=True)
            assert got is into
            assert torch.equal(got[(terms == 0).cuda()], old[(terms == 0).cuda()])
            old = old.cpu().double()
            named = terms > 0
            _close(got[named.cuda()], (total + old)[named],
                   R.gradient_tolerance(total, size, terms, out, old)[named], f"{dtype} {out} added")
        else:
            got = ma.embedding_gradient(grad, tokens, rows, scale=scale, dtype=out)
            _close(got, total, R.gradient_tolerance(total, size, terms, out), f"{dtype} {out}")
            assert not got[(terms == 0).cuda()].any()


@pytest.mark.parametrize("rows,accumulate", [(2 ** 28 + 1003, True), (2 ** 28 + 1003, False)])
def test_gradient_of_three_digits(rows, accumulate):
    gen = _gen(11)
    tokens = torch.cat([_tokens(gen, 3000, rows, "flat"), torch.tensor([0, rows - 1, rows, 255, 256, rows - 1], device="cuda")])
    grad = torch.ones(tokens.numel(), 1, dtype=BF16, device="cuda")
    into = torch.zeros(rows, 1, dtype=BF16, device="cuda") if accumulate else None
    if not accumulate:  # what was in the memory has to go
        torch.full((rows, 1), 3.0, dtype=BF16, device="cuda")
    got = ma.embedding_gradient(grad, tokens, rows, dtype=BF16, out=into, accumulate=accumulate)
    valid, counts = torch.unique(tokens[tokens < rows], return_counts=True)
    assert torch.equal(got[valid, 0].long(), counts)
    assert int(got.float().sum(dtype=torch.float64)) == int(counts.sum())
    del got, into
    torch.cuda.empty_cache()


def test_gradient_of_nothing():
    none = torch.zeros(0, dtype=I64, device="cuda")
    out = torch.full((5, 9), 3.0, device="cuda")
    assert ma.embedding_gradient(torch.zeros(0, 9, device="cuda"), none, 5, out=out, accumulate=True) is out
    assert (out == 3).all()
    ma.embedding_gradient(torch.zeros(0, 9, device="cuda"), none, 5, out=out)
    assert not out.any()
    assert ma.embedding_gradient(torch.zeros(4, 0, device="cuda"), torch.zeros(4, dtype=I64, device="cuda"), 5).shape == (5, 0)
    assert ma.embedding_gradient(torch.zeros(4, 3, device="cuda"), torch.zeros(4, dtype=I64, device="cuda"), 0).shape == (0, 3)
    one = ma.embedding_gradient(torch.ones(3, device="cuda"), torch.tensor(1, device="cuda"), 2)
    assert one.tolist() == [[0, 0, 0], [1, 1, 1]]


def test_gradient_strides():
    gen = _gen(5)
    tokens = _tokens(gen, 300, 20, "spread")
    whole = _values(gen, (300, 90), BF16)
    for grad in (whole[:, 7:64], whole[:, 1:2], whole[:1, 3:50].expand(300, 47)):
        want = ma.embedding_gradient(grad.contiguous(), tokens, 20)
        assert torch.equal(ma.embedding_gradient(grad, tokens, 20), want)
        buffer = torch.full((20, 100), 5.0, device="cuda")
        out = buffer[:, 11:11 + grad.shape[1]]
        ma.embedding_gradient(grad, tokens, 20, out=out)
        assert torch.equal(out, want) and (buffer[:, :11] == 5).all() and (buffer[:, 11 + grad.shape[1]:] == 5).all()
    # tokens of a shifted batch, and a gradient of its shape
    batch = tokens.view(20, 15)
    grad = whole[:, :48].reshape(20, 15, 48)
    want = ma.embedding_gradient(grad[:, :-1].reshape(-1, 48), batch[:, :-1].reshape(-1), 20)
    assert torch.equal(ma.embedding_gradient(grad[:, :-1].contiguous(), batch[:, :-1], 20), want)


def test_values_that_are_not_finite_stay_in_their_rows():
    gen = _gen(6)
    tokens, grad = _tokens(gen, 2000, 50, "spread"), _values(gen, (2000, 300), F32)
    clean = ma.embedding_gradient(grad, tokens, 50)
    at = int((tokens == 3).nonzero()[0])
    grad[at, 7], grad[at, 8] = float("nan"), float("inf")
    dirty = ma.embedding_gradient(grad, tokens, 50)
    assert torch.isnan(dirty[3, 7]) and torch.isinf(dirty[3, 8])
    dirty[3, 7:9] = clean[3, 7:9]
    assert torch.equal(dirty, clean)


def test_a_call_repeated_gives_the_same_bits():
    gen = _gen(7)
    for n, rows, cols in ((700, 40, 300), (30000, 500, 260)):
        tokens, grad = _tokens(gen, n, rows, "spread"), _values(gen, (n, cols), F32)
        first = ma.embedding_gradient(grad, tokens, rows)
        for _ in range(5):
            assert torch.equal(ma.embedding_gradient(grad, tokens, rows), first)


# ---------------------------------------------------------------- step
def _buffers(gen, rows, cols, amsgrad):
    sizes = ma.state_buffer_sizes([rows * cols], "f32", amsgrad)
    out = {"m_f32": _values(gen, sizes["m_f32"] // 4, F32, 1e-3), "v_f32": _values(gen, sizes["v_f32"] // 4, F32, 1e-2).square()}
    if amsgrad:
        out["vmax_f32"] = out["v_f32"] * 1.5
    return out


@pytest.mark.parametrize("n,rows,cols,kind", [s for s in SIZES if s[1] * s[2] < 2 ** 24])
def test_step_is_the_dense_step_on_the_named_rows(n, rows, cols, kind):
    # bit for bit: the dense gradient's rows are the sums that the step takes
    gen = _gen(n + 5 * cols)
    for dtype, amsgrad, decoupled in ((F32, False, True), (BF16, True, True), (BF16, False, False), (F32, True, False)):
        tokens, grad = _tokens(gen, n, rows, kind, I64 if amsgrad else I32), _values(gen, (n, cols), dtype, 1e-2)
        _padding_is_poison(grad, tokens, rows)
        table, buffers = _values(gen, (rows, cols), F32, 0.1), _buffers(gen, rows, cols, amsgrad)
        dense_table, dense_buffers = table.clone(), {k: b.clone() for k, b in buffers.items()}
        old_table, old_buffers = table.clone(), {k: b.clone() for k, b in buffers.items()}
        kw = dict(t=7, amsgrad=amsgrad, decoupled=decoupled, **HP)
        g = ma.embedding_gradient(grad, tokens, rows, scale=1.7)
        ma.adam_step_noalloc([dense_table.view(-1)], [g.view(-1)], dense_buffers, storage="f32", grad_dtype="f32", **kw)
        ma.embedding_adam_step(table, grad, tokens, buffers, scale=1.7, **kw)
        t, ok = R.inside(tokens, rows)
        named = torch.zeros(rows, dtype=torch.bool)
        named[t[ok]] = True
        named = named.cuda()
        for k, got, dense, old in [("table", table, dense_table, old_table)] + \
                [(k, buffers[k], dense_buffers[k], old_buffers[k]) for k in buffers]:
            got, dense, old = (x.view(-1)[:rows * cols].view(rows, cols) for x in (got, dense, old))
            assert torch.equal(got[named], dense[named]), (k, dtype, amsgrad, decoupled)
            assert torch.equal(got[~named], old[~named]), (k, "rows that no token names")
        for k in buffers:
            assert torch.equal(buffers[k][rows * cols:], old_buffers[k][rows * cols:])


@pytest.mark.parametrize("amsgrad", [False, True])
def test_step_against_the_formula_in_64_bits(amsgrad):
    gen = _gen(21)
    n, rows, cols, steps = 3000, 90, 130, 3
    hp = {**HP, "eps": 1e-2}
    table = _values(gen, (rows, cols), F32, 0.1)
    buffers = {k: torch.zeros(b // 4, device="cuda") for k, b in ma.state_buffer_sizes([rows * cols], "f32", amsgrad).items()}
    p, m, v = table.cpu().double(), *(torch.zeros(rows, cols, dtype=torch.float64) for _ in range(2))
    w = torch.zeros_like(v) if amsgrad else None
    ep, em, ev, ew = (torch.zeros_like(v) for _ in range(4))
    start = p.clone()
    for t in range(1, steps + 1):
        tokens, grad = _tokens(gen, n, rows, "spread"), _values(gen, (n, cols), BF16, 1e-2)
        ma.embedding_adam_step(table, grad, tokens, buffers, amsgrad=amsgrad, t=t, **hp)
        total, size, terms = R.gradient(grad, tokens, rows, 1.0)
        eg = R.gradient_tolerance(total, size, terms, F32)
        hit = terms > 0
        old = [p[hit], total[hit], m[hit], v[hit], None if w is None else w[hit]]
        errors = R.adam_errors(*old, (ep[hit], eg[hit], em[hit], ev[hit], ew[hit]), t, **hp)
        for x, y in zip((p, m, v, w, ep, em, ev, ew), R.adam(*old, t, **hp) + errors):
            if x is not None:
                x[hit] = y
    for name, want, error in (("m_f32", m, em), ("v_f32", v, ev), ("vmax_f32", w, ew)):
        if want is not None:
            _close(buffers[name][:rows * cols].view(rows, cols), want, error, name)
    _close(table, p, ep, "table")
    moved = (p - start).abs() > 0.1 * hp["lr"]  # the tolerance tells a step from none
    assert moved.float().mean() > 0.5 and (ep[moved] < 0.05 * (p - start).abs()[moved]).float().mean() > 0.95


def test_rows_and_dense_steps_by_turns():
    gen = _gen(22)
    rows, cols = 64, 48  # every row is named, so that both kinds are the same step
    tokens, grad = torch.arange(rows, device="cuda").repeat(3), _values(gen, (3 * rows, cols), F32, 1e-2)
    first, second = (_values(_gen(1), (rows, cols), F32) for _ in range(2))
    a, b = ({k: torch.zeros(n // 4, device="cuda") for k, n in ma.state_buffer_sizes([rows * cols], "f32").items()}
            for _ in range(2))
    for t in range(1, 5):
        g = ma.embedding_gradient(grad, tokens, rows)
        ma.adam_step_noalloc([first.view(-1)], [g.view(-1)], a, storage="f32", t=t, **HP)
        if t % 2:
            ma.embedding_adam_step(second, grad, tokens, b, t=t, **HP)
        else:
            ma.adam_step_noalloc([second.view(-1)], [g.view(-1)], b, storage="f32", t=t, **HP)
        assert torch.equal(first, second) and all(torch.equal(a[k], b[k]) for k in a)


# ---------------------------------------------------------------- autograd
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward_is_the_gradient_and_the_difference_quotient(dtype):
    gen = _gen(31)
    table = _values(gen, (30, 20), dtype).requires_grad_()
    tokens = _tokens(gen, 200, 30, "spread").view(4, 50)
    weight = _values(gen, (4, 50, 20), F32)
    out = ma.embedding_lookup(table, tokens, scale=2.0, dtype=F32)
    (out * weight).sum().backward()
    assert table.grad.dtype == dtype
    assert torch.equal(table.grad, ma.embedding_gradient(weight, tokens, 30, scale=2.0, dtype=dtype))
    total, size, terms = R.gradient(weight, tokens, 30, 2.0)
    _close(table.grad, total, R.gradient_tolerance(total, size, terms, dtype))
    # a loss linear in the table: the quotient of any step is the derivative.  In 64 bits on the outputs, which a step
    # of a power of two changes exactly where table + step is exact
    with torch.no_grad():
        step = torch.zeros_like(table)
        step[:, 3] = 2.0 ** 4
        ones = torch.ones_like(table)
        high = ma.embedding_lookup(ones + step, tokens, scale=2.0, dtype=F32).double()
        low = ma.embedding_lookup(ones - step, tokens, scale=2.0, dtype=F32).double()
    quotient = ((high - low) * weight.double()).sum() / 2.0 ** 5
    assert abs(float(quotient) - float(total[:, 3].sum())) <= 1e-9 * float(size.sum())


def test_backward_of_other_arrangements():
    table = _values(_gen(32), (30, 20), F32).requires_grad_()
    tokens = torch.arange(60, device="cuda").view(4, 15) % 30
    ma.embedding_lookup(table, tokens).sum().backward()  # an expanded gradient
    assert (table.grad == 2).all()
    ma.embedding_lookup(table, tokens.t(), scale=0.5).transpose(0, 1).sum().backward()  # accumulates into .grad
    assert (table.grad == 3).all()
    with torch.no_grad():
        assert not ma.embedding_lookup(table, tokens).requires_grad
    out = ma.embedding_lookup(table, tokens)
    g, = torch.autograd.grad(out, table, torch.ones_like(out), create_graph=True)
    assert not g.requires_grad or pytest.raises(RuntimeError, g.sum().backward)


def test_refused_gradients():
    table = torch.ones(5, 4, device="cuda", requires_grad=True)
    tokens = torch.zeros(3, dtype=I64, device="cuda")
    with pytest.raises(ValueError, match="no gradient"):
        ma.embedding_lookup(table, tokens, out=torch.empty(3, 4, device="cuda"))
    with pytest.raises(ValueError, match="no gradient"):
        ma.embedding_gradient(torch.ones(3, 4, device="cuda", requires_grad=True), tokens, 5)
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level():
        dual = fwd.make_dual(torch.ones(5, 4, device="cuda"), torch.ones(5, 4, device="cuda"))
        with pytest.raises(ValueError, match="forward-mode"):
            ma.embedding_lookup(dual, tokens)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        x = torch.zeros(4, device="cuda")
        with torch.cuda.graph(graph):
            with pytest.raises(ValueError, match="captured"):
                ma.embedding_lookup(table, tokens)
            x.add_(1)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- streams, graphs, workspaces
def test_other_streams():
    gen = _gen(41)
    tokens, grad = _tokens(gen, 3000, 100, "spread"), _values(gen, (3000, 64), F32)
    table = _values(gen, (100, 64), F32)
    want = ma.embedding_gradient(grad, tokens, 100), ma.embedding_lookup(table, tokens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        # inputs that are written on the side stream just before
        with torch.cuda.stream(side):
            late = torch.zeros_like(grad)
            torch.cuda._sleep(20_000_000)
            late.copy_(grad)
        got = ma.embedding_gradient(late, tokens, 100, stream=stream), ma.embedding_lookup(table, tokens, stream=stream)
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_calls_at_once_in_their_own_workspaces():
    gen = _gen(42)
    sets = [(_tokens(gen, 5000, 200, "spread"), _values(gen, (5000, 300), F32)) for _ in range(2)]
    want = [ma.embedding_gradient(g, t, 200) for t, g in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [ma.embedding_gradient(g, t, 200, stream=s) for (t, g), s in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_of_all_three():
    gen = _gen(43)
    n, rows, cols = 2500, 120, 264
    tokens, grad = _tokens(gen, n, rows, "spread"), _values(gen, (n, cols), BF16, 1e-2)
    table, buffers = _values(gen, (rows, cols), F32), _buffers(gen, rows, cols, True)
    eager_table, eager_buffers = table.clone(), {k: b.clone() for k, b in buffers.items()}
    out, dense = torch.empty(n, cols, dtype=BF16, device="cuda"), torch.empty(rows, cols, device="cuda")
    need = ma.embedding_gradient_workspace_bytes(n, rows, cols)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")  # one for both calls: they are in order

    def work(x, state):
        ma.embedding_lookup(x, tokens, out=out)
        ma.embedding_gradient(grad, tokens, rows, out=dense, workspace=ws)
        ma.embedding_adam_step(x, grad, tokens, state, amsgrad=True, t=3, workspace=ws, **HP)
    with torch.no_grad():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            work(table, buffers)
        for i in range(4):
            tokens.copy_(_tokens(gen, n, rows, ("spread", "same", "flat", "ends")[i]))
            grad.copy_(_values(gen, (n, cols), BF16, 1e-2))
            graph.replay()
            got = out.clone(), dense.clone()
            work(eager_table, eager_buffers)
            torch.cuda.synchronize()
            assert torch.equal(got[0], out) and torch.equal(got[1], dense), i
            assert torch.equal(table, eager_table) and all(torch.equal(buffers[k], eager_buffers[k]) for k in buffers), i


def test_workspace_is_not_written_beyond_its_bytes():
    gen = _gen(44)
    for n, rows, cols in ((3, 5, 4), (700, 40, 100), (5000, 300, 100), (2000, 300000, 4)):
        tokens, grad = _tokens(gen, n, rows, "same"), _values(gen, (n, cols), F32)
        need = ma.embedding_gradient_workspace_bytes(n, rows, cols)
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        got = ma.embedding_gradient(grad, tokens, rows, workspace=ws)
        assert (ws[need:] == 0xA5).all()
        assert torch.equal(got, ma.embedding_gradient(grad, tokens, rows))


# ---------------------------------------------------------------- large offsets
def test_offsets_beyond_32_bits():
    rows, cols = 40000, 60000  # 2.4e9 elements, 4.8 GB in bf16
    table = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    at = [0, 17895, 35791, 35792, rows - 1]  # around 2^30, 2^31 elements
    for i, r in enumerate(at):
        table[r] = i + 1
    tokens = torch.tensor(at[::-1] + [-1], device="cuda")
    got = ma.embedding_lookup(table, tokens)
    assert got[:, 0].tolist() == [5, 4, 3, 2, 1, 0] and torch.equal(got[:, -1], got[:, 0])
    del table
    grad = got.float()
    out = torch.full((rows, cols), 7.0, dtype=BF16, device="cuda")
    ma.embedding_gradient(grad, tokens, rows, out=out)
    assert out[:, 0].nonzero().flatten().tolist() == at and out[:, -1].nonzero().flatten().tolist() == at
    assert [float(out[r, 123]) for r in at] == [1, 2, 3, 4, 5]
    del out
    # a gradient of more than 2^31 elements
    n = 36000
    grad = torch.ones(1, cols, dtype=BF16, device="cuda").repeat(n, 1)
    grad[n - 1] = 2
    tokens = torch.full((n,), 1, device="cuda")
    tokens[n - 1] = 0
    sums = ma.embedding_gradient(grad, tokens, 3)
    assert (sums[0] == 2).all() and (sums[1] == n - 1).all() and not sums[2].any()
    del grad
    # a table and state of 2^32 - 2^16 bytes and more
    rows, cols = 20000, 60000
    table = torch.zeros(rows, cols, device="cuda")
    buffers = {k: torch.zeros(b // 4, device="cuda") for k, b in ma.state_buffer_sizes([rows * cols], "f32").items()}
    tokens = torch.tensor([rows - 1, 0, 17896], device="cuda")
    ma.embedding_adam_step(table, torch.ones(3, cols, device="cuda"), tokens, buffers, t=1, **HP)
    for x in (table, buffers["m_f32"].view(rows, cols), buffers["v_f32"].view(rows, cols)):
        assert x[:, 0].nonzero().flatten().tolist() == [0, 17896, rows - 1]
        assert x[:, -1].nonzero().flatten().tolist() == [0, 17896, rows - 1]
    del table, buffers
    torch.cuda.empty_cache()
