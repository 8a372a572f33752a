"""GPU tests of the Muon calls: the orthogonalisation against a 64-bit
statement of its formula, the momentum against the CPU oracle's first moment
(bit for bit), the step against both, runs of steps with checkpoints beside
Adam steps, streams, graph capture, and the refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

import memory_efficient_adam_amd as ma
import muon_ref
import oracle
import workloads

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


def _matrix(seed, shape, size=1e-3, noise=0.1):
    """A few directions that matter over noise."""
    g = _gen(seed)
    r = max(1, min(shape[-2:]) // 16)
    a = torch.randn(*shape[:-1], r, generator=g, device="cuda")
    b = torch.randn(*shape[:-2], r, shape[-1], generator=g, device="cuda")
    return size * (a @ b / math.sqrt(r) + noise * torch.randn(*shape, generator=g, device="cuda"))


def _check(out, x, **kw):
    """Every matrix of out against the 64-bit formula on x, within the derived
    bound; for fp32 outputs also within 8 times plain fp32's own error (each
    factor here has 2^-23 for its 2^-24, and 2^-22 is left out of a product)
    plus 2^-21 where fp32 happens to be exact."""
    bf16 = out.dtype == torch.bfloat16
    flat_x, flat_o = x.reshape(-1, *x.shape[-2:]), out.reshape(-1, *x.shape[-2:])
    for k in range(flat_x.shape[0]):
        xs = muon_ref.iterate(flat_x[k], **kw)
        ref = muon_ref.orthogonalize(flat_x[k], **kw)
        err = float((flat_o[k].double() - ref).norm() / ref.norm())
        steps, co = kw.get("steps", 5), kw.get("coefficients")
        tol = muon_ref.bound(xs, steps, co, bf16)
        assert err <= tol, (k, err, tol)
        if not bf16:
            f32 = muon_ref.orthogonalize(flat_x[k], dtype=torch.float32, **kw)
            own = float((f32.double() - ref).norm() / ref.norm())
            assert err <= 8 * own + 2.0 ** -21, (k, err, own)


SHAPES = [(1, 1), (1, 7), (5, 1), (2, 3), (16, 16), (33, 65), (63, 64), (64, 64), (65, 64), (65, 129), (200, 31),
          (128, 128), (129, 500), (300, 300), (1000, 768), (513, 1100), (1, 5000), (5000, 3),
          (64, 768), (767, 61), (20, 700), (300, 32), (64, 769), (50, 400), (65, 65)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_orthogonalize_against_the_formula(shape, dtype):
    x = _matrix(sum(shape), shape).to(dtype)
    _check(ma.muon_orthogonalize(x), x)


# enough tiles for the 128 x 128 kernels, with ragged edges; wide, tall, square
@pytest.mark.parametrize("shape", [(70, 48, 80), (5, 3, 64, 500), (17, 500, 1030), (17, 1030, 500), (9, 1024, 1024), (2900, 2950)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_orthogonalize_many_tiles(shape, dtype):
    x = _matrix(3, shape).to(dtype)
    _check(ma.muon_orthogonalize(x), x)


TRIPLES = [(3.0, -3.2, 1.2), (3.4445, -4.7750, 2.0315), (2.5, -2.5, 1.0), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0),
           (4.0, -6.0, 3.0), (2.0, -1.5, 0.5)]


# runs of iterations over one Gram matrix (wide enough), and one after the other
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6, 7])
@pytest.mark.parametrize("shape", [(6, 300, 900), (5, 1000, 333), (40, 60)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_orthogonalize_steps_and_coefficients(steps, shape, dtype):
    x = _matrix(steps, shape).to(dtype)
    for coefficients in (None, TRIPLES[4], TRIPLES[:steps]):
        kw = dict(steps=steps, coefficients=coefficients, eps=1e-6)
        _check(ma.muon_orthogonalize(x, **kw), x, **kw)


# large first coefficients: no run of three, no plain factors before the end
def test_orthogonalize_steep_coefficients():
    steep = [(8.28721, -23.5959, 17.3004), (4.1071, -2.9478, 0.5449), (3.9487, -2.9089, 0.5518),
             (3.3184, -2.4885, 0.5101), (2.3007, -1.6689, 0.4188)]
    for shape in ((6, 300, 900), (500, 520), (30, 700)):
        for dtype in (torch.float32, torch.bfloat16):
            x = _matrix(11, shape).to(dtype)
            _check(ma.muon_orthogonalize(x, coefficients=steep), x, coefficients=steep)


# the largest size a group of the step takes, and one matrix beyond it, are in
# the benchmark's range; these are the shapes where tables can go wrong
LIST = [(33, 65), (128, 64), (1, 77), (200, 31), (64, 64), (1, 1), (0, 5), (130, 257), (40, 2100), (2049, 3)]
STORAGES = [("f32", "q8_v_only"), ("bf16", "bf16"), ("q8", "q8")]
SCALES = {"none": lambda r, c: 1.0, "spectral": lambda r, c: math.sqrt(max(1.0, r / c)),
          "rms": lambda r, c: 0.2 * math.sqrt(max(r, c))}


def _f32(v):
    return float(np.float32(v))


def _encode(m, numels, stochastic, t, seed):
    """8-bit codes and block scales of flat padded fp32 momentum, as the header
    states them: |m| * fl(127 * fl(1/A)) to nearest even, or up iff the draw is
    below the fraction."""
    codes, scales, at = np.zeros(m.size, np.int8), [], 0
    for n in numels:
        for e in range(0, n, 2048):
            x = m[at + e:at + min(n, e + 2048)]
            top = np.abs(x).max()
            if top < np.float32(2.0 ** -112):
                scales.append(np.float32(0))
                continue
            y = np.abs(x) * (np.float32(1) / top * np.float32(127))
            if stochastic:
                u = oracle.sr_draws(seed, t, at + e, x.size, 0).astype(np.float32) * np.float32(2.0 ** -16)
                k = np.floor(y) + (u < y - np.floor(y))
            else:
                k = np.rint(y)
            k = np.where(np.abs(x) >= top, 127, np.minimum(k, 127))
            codes[at + e:at + e + x.size] = np.where(x < 0, -k, k).astype(np.int8)
            scales.append(top)
        at += (n + 15) // 16 * 16
    return codes, np.array(scales, np.float32)


class Reference:
    """The step on the host and in 64 bits.  Momentum in fp32 and bf16 is the
    Adam oracle's first moment on the same gradients; in 8 bits its fp32 update
    (fma with one rounding) and the encoder above.  The update is its formula
    in the library's rounding order, the orthogonalisation the 64-bit formula."""

    def __init__(self, shapes, storage, seed=7):
        self.shapes, self.storage = shapes, storage
        self.numels = [r * c for r, c in shapes]
        self.oracle = oracle.OracleState(self.numels, dict(STORAGES)[storage])
        padded = sum((n + 15) // 16 * 16 for n in self.numels)
        self.codes = np.zeros(padded, np.int8)
        self.scales = np.zeros(sum(-(-n // 2048) for n in self.numels), np.float32)
        self.params = [torch.randn(*s, generator=_gen(seed + k), device="cuda") * 0.02 for k, s in enumerate(shapes)]
        self.exact = [p.double() for p in self.params]

    def buffers(self):
        if self.storage == "q8":
            return {"m_codes": self.codes, "m_scale": self.scales}
        return {k: v for k, v in self.oracle.buffers().items() if k.startswith("m_")}

    def flat(self):
        bufs = self.buffers()
        if self.storage == "f32":
            return bufs["m_f32"].view(np.float32)
        if self.storage == "bf16":
            return (bufs["m_bf16"].astype(np.uint32) << 16).view(np.float32)
        flat, at, slot = np.zeros(self.codes.size, np.float32), 0, 0
        for n in self.numels:
            for e in range(0, n, 2048):
                q = self.codes[at + e:at + min(n, e + 2048)].astype(np.float32) * np.float32(1.0 / 127.0)
                flat[at + e:at + e + q.size] = q * self.scales[slot]
                slot += 1
            at += (n + 15) // 16 * 16
        return flat

    def momentum(self):
        flat, out, at = self.flat(), [], 0
        for n, s in zip(self.numels, self.shapes):
            out.append(torch.from_numpy(flat[at:at + n].reshape(s).copy()).cuda())
            at += (n + 15) // 16 * 16
        return out

    def step(self, grads, t, lr, momentum, weight_decay, nesterov, scale, stochastic=False, seed=42, **kw):
        """Returns, per matrix, how far params may be off: the update times the
        orthogonalisation's bound, and two roundings of the param (2^-24 each of
        what is rounded: p * decay, then the sum), doubled."""
        old = self.momentum()
        beta = _f32(momentum)
        if self.storage != "q8":
            self.oracle.step([np.zeros(n, np.float32) for n in self.numels],
                             [g.float().cpu().numpy().reshape(-1) for g in grads], t=t, lr=1e-3, beta1=momentum,
                             beta2=0.999, eps=1e-8, weight_decay=0.0)
        slack, new, at = [], np.zeros_like(self.flat()), 0
        for k, (g, m0) in enumerate(zip(grads, old)):
            if g.numel() == 0:
                slack.append(0.0)
                continue
            part = g.float() * _f32(1.0 - beta)
            m = (beta * m0.double() + part.double()).float()
            u = (beta * m.double() + part.double()).float() if nesterov else m
            new[at:at + m.numel()] = m.cpu().numpy().reshape(-1)
            at += (m.numel() + 15) // 16 * 16
            xs = muon_ref.iterate(u, **kw)
            rate = _f32(lr) * SCALES[scale](*self.shapes[k])
            o = muon_ref.orthogonalize(u, **kw)
            p = self.exact[k]
            self.exact[k] = p * (1.0 - _f32(lr) * _f32(weight_decay)) - rate * o
            update = rate * float(xs[-1].norm())
            tol = update * (muon_ref.bound(xs, kw.get("steps", 5), kw.get("coefficients")) + 2.0 ** -23)
            slack.append(tol + 2.0 ** -22 * float(p.norm()) + 2.0 ** -22 * update)
        if self.storage == "q8":
            self.codes, self.scales = _encode(new, self.numels, stochastic, t, seed)
        return slack


def _compare_state(state, ref):
    for name, want in ref.buffers().items():
        got = ma.muon_state_read(state, name).cpu().numpy().view(want.dtype)
        assert np.array_equal(got, want), name
    for got, want in zip(ma.muon_state_momentum(state), ref.momentum()):
        assert torch.equal(got.float(), want)


@pytest.mark.parametrize("storage,stochastic,gdt,nesterov,scale", [
    ("f32", False, "f32", True, "rms"), ("f32", False, "bf16", False, "none"), ("bf16", False, "f32", True, "spectral"),
    ("bf16", False, "bf16", True, "rms"), ("q8", False, "f32", False, "rms"), ("q8", False, "bf16", True, "spectral"),
    ("q8", True, "f32", True, "none"), ("q8", True, "bf16", False, "rms")])
def test_step_against_the_oracle_and_the_formula(storage, stochastic, gdt, nesterov, scale):
    ref = Reference(LIST, storage)
    params = [p.clone() for p in ref.params]
    state = ma.muon_state_create(LIST, storage, gdt)
    total = [0.0] * len(LIST)
    hp = dict(lr=3e-3, momentum=0.95, weight_decay=0.1, nesterov=nesterov, scale=scale, seed=99)
    for t in range(1, 5):
        grads = [_matrix(1000 * t + k, s) if s[0] * s[1] else torch.zeros(s, device="cuda") for k, s in enumerate(LIST)]
        if gdt == "bf16":
            grads = [g.bfloat16() for g in grads]
        ma.muon_step(state, params, grads, t=t, stochastic=stochastic, **hp)
        slack = ref.step(grads, t, stochastic=stochastic, **hp)
        _compare_state(state, ref)
        for k, p in enumerate(params):
            total[k] += slack[k]
            err = float((p.double() - ref.exact[k]).norm())
            assert err <= total[k], (t, k, err, total[k])
    state.destroy()
