"""The embedding calls and the steps together, as a training program uses them: a
table looked up by tokens (some of them padding), a weight behind it, a squared
error.  The table is stepped by its named rows, or by its dense gradient beside
the weight; every param and moment is compared with the same run in 64 bits, whose
possible distance from one in fp32 is carried along."""
import pytest
import torch

import embedding_ref as R
import memory_efficient_adam_amd as ma

pytestmark = pytest.mark.gpu

HP = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-2, weight_decay=0.1)
ROWS, COLS, OUT, SCALE, STEPS = 40, 24, 16, 3.0, 4
SHAPE = (5, 17)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


class Exact:
    """A param of the run in 64 bits, with its moments and what each may be off by."""

    def __init__(self, p):
        self.p = p.cpu().double()
        self.m, self.v = torch.zeros_like(self.p), torch.zeros_like(self.p)
        self.errors = [torch.zeros_like(self.p) for _ in range(3)]

    def step(self, g, eg, t, hit=slice(None)):
        old = [self.p[hit], g[hit], self.m[hit], self.v[hit], None]
        ep, em, ev = (e[hit] for e in self.errors)
        errors = R.adam_errors(*old, (ep, eg[hit], em, ev, None), t, **HP)[:3]
        for x, y in zip([self.p, self.m, self.v, *self.errors], [*R.adam(*old, t, **HP)[:3], *errors]):
            x[hit] = y


def _product(a, ea, b, eb):
    """a @ b and how far an fp32 product of it may be: the factors' errors, and a rounding for
    each of the sum's products and additions."""
    n = a.shape[1]
    big = (a.abs() + ea) @ (b.abs() + eb)
    return a @ b, ea @ (b.abs() + eb) + a.abs() @ eb + 1.01 * (n + 1) * R.U32 * big


def _exact_gradients(table, weight, tokens, target):
    """(table's, weight's) gradients with their errors, and which rows a token names."""
    t, ok = R.inside(tokens, ROWS)
    x, ex = torch.zeros(t.numel(), COLS, dtype=torch.float64), torch.zeros(t.numel(), COLS, dtype=torch.float64)
    x[ok] = table.p[t[ok]] * SCALE
    ex[ok] = table.errors[0][t[ok]] * SCALE
    ex = ex + R.U32 * (x.abs() + ex)
    w, ew = weight.p, weight.errors[0]
    h, eh = _product(x, ex, w, ew)
    d = (h - target) / t.numel()  # two roundings, and of 1 / n a third
    ed = eh / t.numel() + 3.03 * R.U32 * (d.abs() + eh / t.numel())
    gx, egx = _product(d, ed, w.t(), ew.t())
    gw, egw = _product(x.t(), ex.t(), d, ed)
    g, size, terms = R.gradient(gx, tokens, ROWS, SCALE)
    carried, _, _ = R.gradient(egx, tokens, ROWS, SCALE)
    return g, carried + R.gradient_tolerance(g, size + carried, terms, torch.float32), gw, egw, terms > 0


def _near(got, want, error, what):
    over = (got.cpu().double() - want).abs() - error
    assert not (over > 0).any(), (what, float(over.max()))
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("by_rows", [True, False])
def test_a_table_and_a_weight(by_rows):
    gen = torch.Generator(device="cuda").manual_seed(5)
    table = torch.randn(ROWS, COLS, generator=gen, device="cuda") * 0.3
    weight = torch.randn(COLS, OUT, generator=gen, device="cuda") * 0.3
    exact_table, exact_weight = Exact(table), Exact(weight)
    size = ROWS * COLS
    if by_rows:
        buffers = {k: torch.zeros(n // 4, device="cuda") for k, n in ma.state_buffer_sizes([size], "f32").items()}
        state = ma.adam_state_create([COLS * OUT], "f32")
    else:
        state = ma.adam_state_create([size, COLS * OUT], "f32")
    weight.requires_grad_()
    start = table.clone()
    for t in range(1, STEPS + 1):
        tokens = torch.randint(-3, ROWS - 8, SHAPE, generator=gen, device="cuda")  # the last rows are never named
        target = torch.randn(SHAPE + (OUT,), generator=gen, device="cuda")
        leaf = ma.embedding_lookup(table, tokens, scale=SCALE).requires_grad_() if by_rows else table.requires_grad_()
        x = leaf if by_rows else ma.embedding_lookup(table, tokens, scale=SCALE)
        loss = 0.5 * ((x @ weight - target) ** 2).sum() / tokens.numel()
        loss.backward()
        g, eg, gw, egw, named = _exact_gradients(exact_table, exact_weight, tokens, target.cpu().double().view(-1, OUT))
        if by_rows:
            ma.embedding_adam_step(table, leaf.grad, tokens, buffers, scale=SCALE, t=t, **HP)
            ma.adam_step(state, [weight], [weight.grad], t=t, **HP)
            exact_table.step(g, eg, t, named)
        else:
            _near(table.grad, g, eg, f"gradient of step {t}")
            ma.adam_step(state, [table, weight], [table.grad, weight.grad], t=t, **HP)
            exact_table.step(g, eg, t)
            table.grad = None
        exact_weight.step(gw, egw, t)
        weight.grad = None
        _near(table.detach(), exact_table.p, exact_table.errors[0], f"table after step {t}")
        _near(weight.detach(), exact_weight.p, exact_weight.errors[0], f"weight after step {t}")
    m = buffers["m_f32"] if by_rows else ma.adam_state_read(state, "m_f32")
    v = buffers["v_f32"] if by_rows else ma.adam_state_read(state, "v_f32")
    _near(m[:size].view(ROWS, COLS), exact_table.m, exact_table.errors[1], "m")
    _near(v[:size].view(ROWS, COLS), exact_table.v, exact_table.errors[2], "v")
    moved = (table.detach() - start).abs()
    assert moved[:ROWS - 8].max() > HP["lr"]
    if by_rows:  # rows that no token names stay, rows of a dense step decay
        assert not moved[ROWS - 8:].any()
    else:
        assert moved[ROWS - 8:].min() > 0
    # the bound tells the steps from each other
    assert exact_table.errors[0].max() < 1e-2 * HP["lr"]


def test_tables_of_a_model_beside_8_bit_states():
    """A table in fp32 states beside a weight in 8-bit ones: two states, each stepped by its own call,
    with the results that each has alone."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    table, weight = torch.randn(300, 64, generator=gen, device="cuda"), torch.randn(64, 128, generator=gen, device="cuda")
    alone = [table.clone(), weight.clone()]
    t32, t8 = ma.adam_state_create([300 * 64], "f32", "bf16"), ma.adam_state_create([64 * 128], "q8", "bf16")
    a32, a8 = ma.adam_state_create([300 * 64], "f32", "bf16"), ma.adam_state_create([64 * 128], "q8", "bf16")
    tokens = torch.randint(0, 300, (700,), generator=gen, device="cuda")
    for t in (1, 2, 3):
        grad = torch.randn(700, 64, generator=gen, device="cuda").bfloat16()
        g = ma.embedding_gradient(grad, tokens, 300, dtype=torch.bfloat16)
        gw = torch.randn(64, 128, generator=gen, device="cuda").bfloat16()
        ma.adam_step(t32, [table], [g], t=t, **HP)
        ma.adam_step(t8, [weight], [gw], t=t, stochastic=True, **HP)
        ma.adam_step(a8, [alone[1]], [gw], t=t, stochastic=True, **HP)
        ma.adam_step(a32, [alone[0]], [g.clone()], t=t, **HP)
    assert torch.equal(table, alone[0]) and torch.equal(weight, alone[1])
