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
