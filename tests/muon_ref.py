"""Plain 64-bit statement of the Newton-Schulz orthogonalisation, and bounds on
how far a computation with rounded factors may be from it."""
import torch

DEFAULT = (3.4445, -4.7750, 2.0315)


def triples(steps, coefficients):
    # the library takes them as fp32 values
    rows = [coefficients or DEFAULT] * steps if coefficients is None or len(coefficients) == 3 and not isinstance(
        coefficients[0], (tuple, list)) else list(coefficients)
    return [tuple(float(torch.tensor(v, dtype=torch.float32)) for v in r) for r in rows]


def iterate(u, steps=5, coefficients=None, eps=1e-7, dtype=torch.float64):
    """[X_0, .., X_steps] of one matrix (short side first)."""
    x = u.double()
    if x.shape[0] > x.shape[1]:
        x = x.T.contiguous()
    # the norm in 64 bits also for an iteration in 32 (squares of 1e-30 vanish there)
    x = (x / (x.square().sum().sqrt() + float(torch.tensor(eps, dtype=torch.float32)))).to(dtype)
    xs = [x]
    for a, b, c in triples(steps, coefficients):
        g = x @ x.T.contiguous()
        x = a * x + (b * g + c * (g @ g)) @ x
        xs.append(x)
    return xs


def orthogonalize(u, **kw):
    o = iterate(u, **kw)[-1]
    return o.T.contiguous() if u.shape[0] > u.shape[1] else o


def slope(abc, top=1.25):
    """max |p'| over [0, top]: by how much an iteration can grow an error of X.
    (An odd matrix polynomial's derivative is bounded by its divided
    differences over +- the singular values, hence by max |p'|.)"""
    a, b, c = abc
    s = torch.linspace(0.0, top, 2001, dtype=torch.float64)
    return float((a + 3 * b * s ** 2 + 5 * c * s ** 4).abs().max())


def plain_from(steps, coefficients):
    """The first iteration whose factors may be single fp16 values (bf16 output)."""
    growth, first = 1.0, steps
    for k in range(steps - 1, -1, -1):
        growth *= abs(triples(steps, coefficients)[k][0])
        if growth > 12.0:
            break
        first = k
    return first


def bound(xs, steps=5, coefficients=None, bf16_out=False):
    """A bound on |O' - O|_F / |O|_F (xs: the exact iterates).

    Iteration k rounds X, A and P to 22 bits (2^-23 of each entry), leaves out
    lo*lo (2^-24 at most of a product term, in two products) and sums in fp32:
    at most 2^-20 |X_k|_F in all, counting |P| <= 4.  A growth by the later slopes
    then follows.  Single fp16 values: 2^-12 of each entry at most, 2^-12/sqrt(3)
    root mean square; the four roundings of an iteration (X, A as a factor and
    as a term, P) add as independent errors to 2 * 2^-12 / sqrt(3), doubled for |P| > 1.  A bf16 result is
    off by at most 2^-8 of each entry besides."""
    cs = triples(steps, coefficients)
    first = plain_from(steps, coefficients) if bf16_out else steps
    total, grow = 2.0 ** -20, 1.0
    norm = float(xs[-1].norm())
    for k in range(steps - 1, -1, -1):
        grow *= max(1.0, slope(cs[k]))
        eta = 2.0 ** -20 if k < first else 4 * 2.0 ** -12 / 3 ** 0.5
        total += grow * eta * float(xs[k].norm()) / max(norm, 1e-300)
    return total + (2.0 ** -8 if bf16_out else 0.0)
