"""GPU tests of how exact the orthogonalisation is: inputs and coefficients for
which a product's factors need all of their bits."""
import pytest
import torch

import memory_efficient_adam_amd as ma
import muon_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _with_singular_values(seed, shape, s):
    """A matrix of these singular values and random directions."""
    rows, cols = shape
    m = min(shape)
    u, _ = torch.linalg.qr(torch.randn(rows, m, generator=_gen(seed), device="cuda", dtype=torch.float64))
    v, _ = torch.linalg.qr(torch.randn(cols, m, generator=_gen(seed + 1), device="cuda", dtype=torch.float64))
    return (u * s) @ v.T.contiguous()


def _spectrum(kind, m):
    if kind == "decaying":
        return torch.logspace(0, -4, m, device="cuda", dtype=torch.float64)
    s = torch.full((m,), 1e-4 if kind == "one direction" else 0.1, device="cuda", dtype=torch.float64)
    s[:max(1, m // 16) if kind == "some directions" else 1] = 1.0
    return s


DEFAULT = muon_ref.DEFAULT
# the slope at singular value 0 is a; elsewhere a polynomial can be steep though its a is small, or 0
ITERATIONS = {"default": [DEFAULT] * 5, "last a is 0": [DEFAULT] * 4 + [(0.0, 2.5, -1.5)],
              "last a is small": [(3.0, -3.2, 1.2)] * 4 + [(0.1, 2.4, -1.5)],
              "a below 1 between": [DEFAULT] * 2 + [(0.5, 1.2, -0.7), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)]}


@pytest.mark.parametrize("iteration", ITERATIONS)
@pytest.mark.parametrize("kind", ["some directions", "decaying", "one direction"])
@pytest.mark.parametrize("shape", [(40, 60), (64, 768), (700, 50), (300, 500), (768, 2304), (1600, 520)], ids=str)
def test_a_bf16_result_is_off_by_its_own_rounding(shape, kind, iteration):
    """O' = bf16(O + E): an entry's distance from the nearest bf16 value changes by
    at most |E| when the entry does, so |O' - O| <= |bf16(O) - O| + 2 |E| in the
    Frobenius norm; E is what an fp32 result may be off by, 8 times plain fp32's
    own error and 2^-21."""
    cs = ITERATIONS[iteration]
    exact = _with_singular_values(7, shape, _spectrum(kind, min(shape)))
    for dtype in (torch.float32, torch.bfloat16):
        x = exact.to(dtype)
        out = ma.muon_orthogonalize(x, out=torch.empty(shape, dtype=torch.bfloat16, device="cuda"), coefficients=cs)
        ref = muon_ref.orthogonalize(x, coefficients=cs)
        norm = float(ref.norm())
        own = float((muon_ref.orthogonalize(x, dtype=torch.float32, coefficients=cs).double() - ref).norm()) / norm
        rounding = float((ref.bfloat16().double() - ref).norm()) / norm
        err = float((out.double() - ref).norm()) / norm
        assert err <= rounding + 2 * (8 * own + 2.0 ** -21), (str(dtype), err, rounding, own)


@pytest.mark.parametrize("where", ["entry", "row", "column"])
@pytest.mark.parametrize("shape", [(60, 90), (64, 700), (300, 30), (300, 500), (520, 1600), (1600, 520), (6, 300, 900)], ids=str)
def test_one_entry_row_or_column_that_holds_nearly_all_of_the_norm(shape, where):
    """The others are 1e-7 of it, and the iterations grow them by 485.

    As a whole (fp32 result): the large direction's singular value goes 1, 0.70,
    1.11, 0.72, 1.09; at slopes of 0.8 to 1.3 what an iteration adds is grown to
    at most 1.5 times, in all 6.5 times one iteration's share, some 4 roundings
    of 2^-23: 2^-18.1.  Apart from the large row and column: the rest grows
    linearly by a each time, an iteration rounds X and P to 2^-23 each, drops
    2^-24 in products with P and rounds sums, and |P| is up to 3 times a in
    absolute sums along the large direction: 5 * 5 * 2^-23 * 3 = 9e-6; entries of
    X_0 of 2.5e-9 have an error of at most 2^-46 besides, 5.7e-6 of them.  Both
    are below 2^-16.  From a bf16 matrix, entries below 2^-33 = 0.047 * 2.5e-9, 3.7 in
    a hundred, have an error of at most 2^-40 = 3.7e-4 * 2.5e-9: 7.1e-5 root mean square."""
    x = torch.randn(shape, generator=_gen(3), device="cuda")
    big = x.reshape(-1, *shape[-2:])
    i, j = shape[-2] // 3, shape[-1] // 5
    at = {"entry": (slice(None), i, j), "row": (slice(None), i), "column": (slice(None), slice(None), j)}[where]
    big[at] = 1e7 if where == "entry" else big[at] * 1e7
    for dtype in (torch.float32, torch.bfloat16):
        y = big.to(dtype)
        out = ma.muon_orthogonalize(y.reshape(shape), out=torch.empty(shape, device="cuda")).reshape(big.shape)
        for got, one in zip(out.double(), y):
            ref = muon_ref.orthogonalize(one)
            own = float((muon_ref.orthogonalize(one, dtype=torch.float32).double() - ref).norm() / ref.norm())
            err = float((got - ref).norm() / ref.norm())
            assert err <= 8 * own + 2.0 ** -18, (str(dtype), err, own)
            diff = got - ref
            for t in (diff, ref):
                if where != "column":
                    t[i] = 0.0
                if where != "row":
                    t[:, j] = 0.0
            rest = float(diff.norm() / ref.norm())
            assert rest <= 2.0 ** -16 + (7.1e-5 if dtype == torch.bfloat16 else 0.0), (str(dtype), rest)
