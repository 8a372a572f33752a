"""The embedding operations from their definitions in 64 bits, on the CPU, and
how far a computation in fp32 may be from them (not a test module)."""
import numpy as np
import torch

U32 = 2.0 ** -24  # half a step of fp32, relative to the value
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f32(x):
    return float(np.float32(x))


def inside(tokens, rows):
    t = tokens.reshape(-1).cpu().long()
    return t, (t >= 0) & (t < rows)


def lookup(table, tokens, scale):
    t, ok = inside(tokens, table.shape[0])
    out = torch.zeros(t.numel(), table.shape[1], dtype=torch.float64)
    out[ok] = table.cpu().double()[t[ok]] * f32(scale)
    return out.reshape(tokens.shape + table.shape[1:])


def lookup_tolerance(want, dtype):
    # the product rounded to fp32, then to dtype
    return want.abs() * (U32 + HALF[dtype] * (1 + U32)) if dtype != torch.float32 else want.abs() * U32


def gradient(grad, tokens, rows, scale):
    """(sum, sum of sizes, terms) of each row: its gradient, what an error is relative to, and how many
    rows were summed."""
    t, ok = inside(tokens, rows)
    flat = grad.reshape(t.numel(), -1).cpu().double()[ok]
    total, size = (torch.zeros(rows, flat.shape[1], dtype=torch.float64) for _ in range(2))
    total.index_add_(0, t[ok], flat)
    size.index_add_(0, t[ok], flat.abs())
    terms = torch.bincount(t[ok], minlength=rows).double()
    return total * f32(scale), size * abs(f32(scale)), terms


def gradient_tolerance(total, size, terms, dtype, old=None):
    # fp32 sums of n terms in any order are off by (n - 1) U32 of the sum of sizes at most (first order; 1% covers
    # the others for n < 10^5), the scale's product by one more rounding, an addition to an old value by one; then dtype's
    slack = 1.01 * U32 * (terms[:, None].clamp(min=1) - 1) * size + U32 * total.abs() * 1.01
    value = total if old is None else total + old
    if old is not None:
        slack = slack + 1.01 * U32 * value.abs()
    if dtype != torch.float32:
        slack = slack + HALF[dtype] * (value.abs() + slack)
    return slack


def adam(p, g, m, v, w, t, lr, beta1, beta2, eps, weight_decay, decoupled=True):
    """One step in 64 bits with fp32's hyperparameters: (p, m, v, w)."""
    lr, beta1, beta2, eps, wd = (f32(x) for x in (lr, beta1, beta2, eps, weight_decay))
    if not decoupled:
        g = g + wd * p
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    w = None if w is None else torch.maximum(w, v)
    root = ((v if w is None else w) / (1 - beta2 ** t)).sqrt() + eps
    p = (p * (1 - lr * wd) if decoupled else p) - lr / (1 - beta1 ** t) * m / root
    return p, m, v, w


def adam_errors(p, g, m, v, w, errors, t, lr, beta1, beta2, eps, weight_decay, decoupled=True):
    """How far one step in fp32 may be from adam()'s: errors = (of p, g, m, v, w) before it,
    (of p, m, v, w) after it.  Each line: what the errors going in make of it, and a rounding
    (U32 of the value) for each operation and each scalar that the step holds in fp32."""
    ep, eg, em, ev, ew = errors
    new_p, new_m, new_v, new_w = adam(p, g, m, v, w, t, lr, beta1, beta2, eps, weight_decay, decoupled)
    if not decoupled:  # one fma
        eg = eg + f32(weight_decay) * ep + U32 * (g + f32(weight_decay) * p).abs() * 1.01
        g = g + f32(weight_decay) * p
    beta1, beta2 = f32(beta1), f32(beta2)
    g_most = g.abs() + eg
    # m: 1 - beta1, its product, the fma
    em = beta1 * em + (1 - beta1) * eg + U32 * (2.02 * (1 - beta1) * g_most + 1.01 * (new_m.abs() + em + eg))
    # v: g^2, 1 - beta2, their product, the fma
    ev = beta2 * ev + (1 - beta2) * eg * (2 * g.abs() + eg) + U32 * (3.03 * (1 - beta2) * g_most ** 2)
    ev = ev + 1.01 * U32 * (new_v + ev)
    if w is not None:
        ew = torch.maximum(ew, ev)
    x, ex = (new_v, ev) if w is None else (new_w, ew)
    # root: the square root, the scalar, the fma
    bc2 = 1 - beta2 ** t
    root = (x / bc2).sqrt() + f32(eps)
    high = ((x + ex) / bc2).sqrt() + f32(eps)
    low = ((x - ex).clamp(min=0) / bc2).sqrt() + f32(eps)
    er = torch.maximum(high - root, root - low) + 3.03 * U32 * high
    # the quotient (one rounding), the rate's rounding, p's product with its scalar and the fma
    rate = f32(lr) / (1 - beta1 ** t)
    q = new_m.abs() / root
    eq = (em + q * er) / (root - er).clamp(min=f32(eps) / 2)
    ep = ep + rate * eq + U32 * (2.02 * rate * (q + eq) + 2.02 * (p.abs() + ep) + 1.01 * (new_p.abs() + ep + rate * eq))
    return ep, em, ev, ew
