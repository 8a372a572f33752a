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


# bf16 in and fp32 out, and the other way; runs, single fp16 values at the end, bf16 taken as it is
@pytest.mark.parametrize("steps", [1, 2, 3, 5])
@pytest.mark.parametrize("shape", [(40, 70), (129, 500), (6, 300, 900), (3, 1100, 520)], ids=str)
def test_orthogonalize_from_one_type_to_another(steps, shape):
    for dtype, out_dtype in ((torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)):
        x = _matrix(20 + steps, shape).to(dtype)
        out = torch.empty(shape, dtype=out_dtype, device="cuda")
        _check(ma.muon_orthogonalize(x, out=out, steps=steps), x, steps=steps)


# long and short products in one launch, several rounds of tiles, a rest that is split
def test_step_of_many_matrices_of_unequal_length():
    shapes = [(768, 2304)] * 13 + [(700, 768), (300, 2000), (64, 64)] * 7
    grads = [_matrix(30 + k, s) for k, s in enumerate(shapes)]
    params = [torch.zeros(s, device="cuda") for s in shapes]
    state = ma.muon_state_create(shapes, "f32")
    ma.muon_step(state, params, grads, t=1, lr=1.0, momentum=0.0, scale="none")
    for p, g in zip(params, grads):
        _check(-p, g)
    state.destroy()


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


# ---------------------------------------------------------------- layouts, streams, graphs
def test_orthogonalize_takes_strided_batches_and_writes_nothing_else():
    for shape in ((4, 60, 90), (3, 200, 310), (2, 700, 129)):
        b, r, c = shape
        big = _matrix(5, (b, r + 3, c + 7))
        x = big[:, 2:r + 2, 3:c + 3]  # not aligned to more than an element
        dest = torch.full((b, r + 4, c + 5), 7.0, device="cuda")
        out = dest[:, 1:r + 1, 4:c + 4]
        before = big.clone()
        assert ma.muon_orthogonalize(x, out=out) is out
        assert torch.equal(out, ma.muon_orthogonalize(x.contiguous()))
        assert torch.equal(big, before)
        dest[:, 1:r + 1, 4:c + 4] = 7.0
        assert bool((dest == 7.0).all())
        half = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        ma.muon_orthogonalize(x, out=half)  # fp32 in, bf16 out
        _check(half, x.contiguous())
        wide = ma.muon_orthogonalize(x.bfloat16(), out=torch.empty(shape, device="cuda"))  # bf16 in, fp32 out
        _check(wide, x.bfloat16())


def test_orthogonalize_in_place_broadcast_and_higher_batches():
    x = _matrix(6, (2, 3, 150, 140))
    want = ma.muon_orthogonalize(x)
    assert torch.equal(ma.muon_orthogonalize(x[:, 1]), want[:, 1])
    same = x[0, 0].expand(5, 150, 140)  # one matrix read five times
    assert all(torch.equal(o, want[0, 0]) for o in ma.muon_orthogonalize(same))
    assert ma.muon_orthogonalize(x, out=x) is x and torch.equal(x, want)
    with pytest.raises(ma.AdamError, match="overlaps"):
        flat = _matrix(6, (300, 140))
        ma.muon_orthogonalize(flat[:200], out=flat[100:])


def test_orthogonalize_batches_beyond_one_part():
    # 2^26 elements go through the products at a time: two parts and a rest
    x = _matrix(8, (1, 1024, 1100)).expand(130, 1024, 1100)
    out = ma.muon_orthogonalize(x)
    _check(out[:1], x[:1])
    assert all(torch.equal(out[0], o) or float((out[0] - o).norm()) < 1e-5 * float(o.norm()) for o in out[1:])


def test_orthogonalize_more_small_matrices_than_a_launch_has_workgroups():
    # 2^32 threads are one too many for a launch of 512 a matrix
    n = 2 ** 23 + 5
    x = torch.ones(n, 1, 1, device="cuda")
    x[1::2] = -2.0
    x[5::7] = 0.0
    out = ma.muon_orthogonalize(x)
    assert torch.equal(out, ma.muon_orthogonalize(x[:14]).repeat(n // 14 + 1, 1, 1)[:n])
    assert torch.equal(out[:, 0, 0].sign(), x[:, 0, 0].sign())


@pytest.mark.parametrize("shape", [(40, 70), (300, 300), (5, 600, 520), (2200, 2100)], ids=str)
def test_zero_and_nonfinite_matrices(shape):
    batch = 3
    x = _matrix(2, (batch,) + shape[-2:])
    good = ma.muon_orthogonalize(x)
    x[1] = 0.0
    out = ma.muon_orthogonalize(x)
    assert bool((out[1] == 0).all())
    for value in (float("nan"), float("inf"), float("-inf")):
        x[1] = 0.0
        x[1, -1, -1] = value
        out = ma.muon_orthogonalize(x)
        assert bool(out[1].isnan().all())
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])


@pytest.mark.parametrize("size", [1e-30, 1e-10, 1e30], ids=str)
def test_scales_of_the_gradient(size):
    # squares that leave fp32's range; eps is small beside the norm
    for shape in ((50, 60), (200, 333)):
        x = _matrix(4, shape, size=size)
        kw = dict(eps=1e-37)
        _check(ma.muon_orthogonalize(x, **kw), x, **kw)


@pytest.mark.parametrize("shape", [(33000, 34000), (34000, 33000), (70, 2 ** 21 - 1), (2 ** 21 - 1, 90)], ids=str)
def test_matrices_beyond_32_bit_offsets(shape):
    # one entry a row and column: each is its own singular value, the rest stays 0
    m = min(shape)
    if torch.cuda.mem_get_info()[0] < 60 * 2 ** 30:
        pytest.skip("needs 60 GB")
    g = _gen(12)
    at = torch.randperm(max(shape) - 1, generator=g, device="cuda")[:m]
    at[-1] = max(shape) - 1
    i = torch.arange(m, device="cuda")
    rows, cols = (i, at) if shape[0] < shape[1] else (at, i)
    values = 0.5 + torch.rand(m, generator=g, device="cuda")
    x = torch.zeros(shape, device="cuda")
    x[rows, cols] = values
    steps = [(3.4445, -4.7750, 2.0315)] * 2
    out = ma.muon_orthogonalize(x, steps=2)
    del x
    s = values.double() / values.double().norm()
    for a, b, c in muon_ref.triples(2, steps):
        s = a * s + b * s ** 3 + c * s ** 5
    got = out[rows, cols].double()
    # an entry of 2^-13 and more has 22 bits in each factor, a smaller one an error of 2^-35
    # in X_0, which the two iterations grow by 3.45 each
    tol = 8 * 2.0 ** -22 * s.abs() + 12 * 2.0 ** -35
    assert bool(((got - s).abs() <= tol).all()), float(((got - s).abs() / tol).max())
    out[rows, cols] = 0.0
    assert not bool(out.any())


def test_closed_forms():
    # one direction, and a diagonal: the polynomial of each singular value
    def poly(s, steps=5):
        for a, b, c in muon_ref.triples(steps, None):
            s = a * s + b * s ** 3 + c * s ** 5
        return s
    for shape in ((30, 50), (400, 260)):
        u = torch.randn(shape[0], 1, generator=_gen(1), device="cuda", dtype=torch.float64)
        v = torch.randn(1, shape[1], generator=_gen(2), device="cuda", dtype=torch.float64)
        o = ma.muon_orthogonalize((u @ v).float())
        want = poly(1.0) * (u / u.norm()) @ (v / v.norm())
        # rounding u v^T to fp32 leaves up to 2^-24 of its norm outside the one
        # direction, and X_0's two fp16 values 2^-23; singular values that small grow
        # by the product of the a_k (484.9), the direction's own goes to poly(1)
        growth = math.prod(abc[0] for abc in muon_ref.triples(5, None)) / abs(poly(1.0))
        assert float((o.double() - want).norm() / want.norm()) < growth * (2.0 ** -24 + 2.0 ** -23)
        n = min(shape)
        s = torch.linspace(1.0, 0.01, n, device="cuda", dtype=torch.float64)
        x = torch.zeros(shape, device="cuda", dtype=torch.float64)
        x[range(n), range(n)] = s
        o = ma.muon_orthogonalize(x.float())
        want = torch.zeros_like(x)
        want[range(n), range(n)] = poly(s / s.norm())
        assert float((o.double() - want).norm() / want.norm()) < 2.0 ** -16


def test_results_repeat_bit_for_bit_and_on_other_streams():
    for shape in ((64, 300), (1000, 768), (2, 2048, 2048), (24, 600, 700)):
        x = _matrix(9, shape)
        want = ma.muon_orthogonalize(x)
        for _ in range(3):
            assert torch.equal(ma.muon_orthogonalize(x), want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = ma.muon_orthogonalize(x, stream=side)
        two = ma.muon_orthogonalize(x)  # at the same time, its own workspace
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(two, want)
        raw = ma.muon_orthogonalize(x, stream=side.cuda_stream)
        side.synchronize()
        assert torch.equal(raw, want)


def test_calls_under_way_at_once_on_two_streams():
    # each with its own workspace and state; split tiles count arrivals in both
    xs = [_matrix(40, (768, 1000)), _matrix(41, (2, 1100, 1300))]
    want = [ma.muon_orthogonalize(x) for x in xs]
    shapes = [(768, 1000), (500, 500), (33, 65)]
    grads = [_matrix(42 + k, s) for k, s in enumerate(shapes)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    states = [ma.muon_state_create(shapes, "q8") for _ in streams]
    params = [[torch.zeros(s, device="cuda") for s in shapes] for _ in streams]
    torch.cuda.synchronize()
    got = [[], []]
    for t in range(1, 6):
        for i, stream in enumerate(streams):
            got[i].append(ma.muon_orthogonalize(xs[i], stream=stream))
            ma.muon_step(states[i], params[i], grads, t=t, lr=1e-2, stream=stream)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
    assert all(torch.equal(a, b) for a, b in zip(*params))
    assert all(torch.equal(a, b) for a, b in zip(*(ma.muon_state_momentum(s) for s in states)))


def test_orthogonalize_in_a_graph():
    for shape in ((48, 80), (3, 500, 700), (2048, 2048)):
        x = _matrix(1, shape)
        out, ws = torch.empty_like(x), torch.empty(
            max(1, ma.muon_orthogonalize_workspace_bytes(x.numel() // (shape[-1] * shape[-2]), *shape[-2:])),
            dtype=torch.uint8, device="cuda")
        ma.muon_orthogonalize(x, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ma.muon_orthogonalize(x, out=out, workspace=ws)
        for k in range(4):
            x.copy_(_matrix(20 + k, shape))
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ma.muon_orthogonalize(x)), k


# ---------------------------------------------------------------- states
def _grads(t, shapes, dtype=torch.float32):
    return [_matrix(100 * t + k, s).to(dtype) for k, s in enumerate(shapes)]


RUN = [(300, 520), (64, 64), (700, 300), (33, 7), (520, 300)]


@pytest.mark.parametrize("storage,stochastic", [("f32", False), ("bf16", False), ("q8", False), ("q8", True)])
def test_checkpoint_resumes_bit_for_bit(storage, stochastic):
    hp = dict(lr=1e-2, stochastic=stochastic, seed=5)
    state = ma.muon_state_create(RUN, storage)
    params = [torch.randn(*s, generator=_gen(k), device="cuda") * 0.02 for k, s in enumerate(RUN)]
    for t in (1, 2):
        ma.muon_step(state, params, _grads(t, RUN), t=t, **hp)
    ma.muon_state_set_draw_index(state, [16 * 10 ** 6 * (k + 1) for k in range(len(RUN))])
    blob = ma.muon_state_save(state)
    other = ma.muon_state_load(blob)
    assert other.shapes == RUN and other.storage == storage
    assert ma.muon_state_get_draw_index(other) == ma.muon_state_get_draw_index(state)
    copies = [p.clone() for p in params]
    for t in (3, 4):
        ma.muon_step(state, params, _grads(t, RUN), t=t, **hp)
        ma.muon_step(other, copies, _grads(t, RUN), t=t, **hp)
    assert all(torch.equal(a, b) for a, b in zip(params, copies))
    assert np.array_equal(ma.muon_state_save(state), ma.muon_state_save(other))
    bad = blob.copy()
    bad[-1] ^= 1
    with pytest.raises(ma.AdamError, match="checksum"):
        ma.muon_state_load(bad)


def test_shards_of_whole_matrices_draw_the_same_stream():
    params = [torch.zeros(s, device="cuda") for s in RUN]
    whole = ma.muon_state_create(RUN, "q8")
    parts = [ma.muon_state_create(RUN[:2], "q8"), ma.muon_state_create(RUN[2:], "q8")]
    first = ma.muon_state_get_draw_index(whole)
    ma.muon_state_set_draw_index(parts[1], first[2:])
    copies = [p.clone() for p in params]
    for t in (1, 2, 3):
        g = _grads(t, RUN)
        hp = dict(lr=1e-2, t=t, stochastic=True, seed=8)
        ma.muon_step(whole, params, g, **hp)
        ma.muon_step(parts[0], copies[:2], g[:2], **hp)
        ma.muon_step(parts[1], copies[2:], g[2:], **hp)
    got = ma.muon_state_momentum(parts[0]) + ma.muon_state_momentum(parts[1])
    assert all(torch.equal(a, b) for a, b in zip(ma.muon_state_momentum(whole), got))
    # tiles are chosen for the whole list: the params agree to the orthogonalisation's error
    for a, b in zip(params, copies):
        assert float((a - b).norm()) <= 2e-5 * float(a.norm())


def test_training_run_of_matrices_with_muon_and_the_rest_with_adam():
    # the two steps as a program uses them together: matrices and their biases,
    # states of both, a checkpoint of both in the middle
    biases = [s[0] for s in RUN]
    ref = Reference(RUN, "q8")
    W = [p.clone() for p in ref.params]
    b = [torch.zeros(n, device="cuda") for n in biases]
    b_ref = [np.zeros(n, np.float32) for n in biases]
    muon, adam = ma.muon_state_create(RUN, "q8", "bf16"), ma.adam_state_create(biases, "q8")
    adam_ref = oracle.OracleState(biases, "q8")
    total = [0.0] * len(RUN)
    adam_hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
    for t in range(1, 6):
        gW = _grads(t, RUN, torch.bfloat16)
        gb = workloads.host_grads(77, biases, t)
        ma.muon_step(muon, W, gW, t=t, lr=2e-3, weight_decay=0.05, stochastic=True, seed=3)
        ma.adam_step(adam, b, [torch.from_numpy(g).cuda() for g in gb], t=t, **adam_hp)
        slack = ref.step(gW, t, lr=2e-3, momentum=0.95, weight_decay=0.05, nesterov=True, scale="rms", stochastic=True, seed=3)
        adam_ref.step(b_ref, gb, t=t, **adam_hp)
        if t == 3:
            muon, adam = ma.muon_state_load(ma.muon_state_save(muon)), ma.adam_state_load(ma.adam_state_save(adam))
        _compare_state(muon, ref)
        for k in range(len(RUN)):
            total[k] += slack[k]
            assert float((W[k].double() - ref.exact[k]).norm()) <= total[k], (t, k)
            assert np.allclose(b[k].cpu().numpy(), b_ref[k], rtol=1e-5, atol=1e-9)


def test_groups_of_a_long_list():
    # more elements than go through the products at a time: every matrix as alone
    shapes = [(1024, 4096)] * 18 + [(40, 30), (4096, 1024)]
    state = ma.muon_state_create(shapes, "f32")
    one = _matrix(3, (1024, 4096))
    grads = [one] * 18 + [_matrix(4, (40, 30)), one.T.contiguous()]
    params = [torch.zeros(s, device="cuda") for s in shapes]
    ma.muon_step(state, params, grads, t=1, lr=1.0, momentum=0.0, nesterov=False, scale="none")
    want = -muon_ref.orthogonalize(one)
    for k, p in enumerate(params):
        if k == 18:
            continue
        got = p if k < 18 else p.T
        assert float((got.double() - want).norm() / want.norm()) < 1e-5, k
    _check(-params[18], grads[18])


def test_state_padding_and_parameters_beyond_a_matrix_stay():
    shapes = [(33, 65), (130, 257)]
    state = ma.muon_state_create(shapes, "f32")
    flat = torch.full((130 * 257 + 64,), 3.0, device="cuda")
    params = [torch.zeros(33, 65, device="cuda"), flat[:130 * 257].view(130, 257)]
    junk = ma.muon_state_read(state, "m_f32")
    junk.fill_(float("nan"))
    junk[:33 * 65] = 0.0
    at = (33 * 65 + 15) // 16 * 16
    junk[at:at + 130 * 257] = 0.0  # NaN in the padding alone
    ma.muon_state_write(state, "m_f32", junk)
    grads = _grads(1, shapes)
    ma.muon_step(state, params, grads, t=1, lr=1e-3)
    assert all(bool(p.isfinite().all()) for p in params) and bool((flat[130 * 257:] == 3.0).all())
    m = ma.muon_state_read(state, "m_f32")
    assert bool((m[33 * 65:at] == 0).all()) and bool((m[at + 130 * 257:] == 0).all())


def test_zero_gradients_and_a_nonfinite_one():
    shapes = [(100, 200), (50, 60), (300, 100)]
    state = ma.muon_state_create(shapes, "q8")
    params = [torch.randn(*s, generator=_gen(k), device="cuda") for k, s in enumerate(shapes)]
    before = [p.clone() for p in params]
    ma.muon_step(state, params, [torch.zeros(s, device="cuda") for s in shapes], t=1, lr=0.5, weight_decay=0.0)
    assert all(torch.equal(a, b) for a, b in zip(params, before))
    grads = _grads(2, shapes)
    grads[1][3, 4] = float("inf")
    ma.muon_step(state, params, grads, t=2, lr=1e-3)
    assert bool(params[1].isnan().all())
    assert bool(params[0].isfinite().all()) and bool(params[2].isfinite().all())


def test_a_step_on_a_side_stream_and_pointer_changes():
    shapes = [(96, 130), (400, 333)]
    a, b = (ma.muon_state_create(shapes, "bf16") for _ in range(2))
    pa = [torch.zeros(s, device="cuda") for s in shapes]
    pb = [p.clone() for p in pa]
    side = torch.cuda.Stream()
    for t in range(1, 12):  # more gradient sets than resident tables
        g = _grads(t, shapes)
        side.wait_stream(torch.cuda.current_stream())
        ma.muon_step(a, pa, g, t=t, lr=1e-3)
        ma.muon_step(b, pb, g, t=t, lr=1e-3, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(pa, pb))
    got = ma.muon_state_momentum(b, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, ma.muon_state_momentum(a)))


def test_step_refusals():
    shapes = [(16, 32), (40, 8)]
    state = ma.muon_state_create(shapes, "bf16")
    p, g = [torch.zeros(s, device="cuda") for s in shapes], _grads(1, shapes)
    ok = dict(lr=1e-3, t=1)
    for bad, what in ((dict(t=0), "t must"), (dict(lr=-1.0), "lr"), (dict(lr=float("nan")), "lr"), (dict(momentum=1.0), "momentum"),
                      (dict(weight_decay=-0.1), "weight_decay"), (dict(scale=7), "scale"), (dict(steps=0), "steps"),
                      (dict(steps=17), "steps"), (dict(eps=0.0), "eps"), (dict(coefficients=(1.0, 2.0, 100.0)), "coefficient"),
                      (dict(stochastic=True), "8-bit")):
        with pytest.raises(ma.AdamError, match=what) as e:
            ma.muon_step(state, p, g, **{**ok, **bad})
        assert e.value.code == -1
    with pytest.raises(ma.AdamError) as e:
        ma.muon_step(state, p, g, expect=("q8", "f32"), **ok)
    assert e.value.code == -2
    flat = torch.zeros(16 * 32 + 1, device="cuda")
    with pytest.raises(ma.AdamError) as e:
        ma.muon_step(state, [flat[1:].view(16, 32), p[1]], g, **ok)
    assert e.value.code == -3
    twice = ma.muon_state_create([(16, 32)] * 2, "bf16")
    with pytest.raises(ma.AdamError, match="same param"):
        ma.muon_step(twice, [p[0], p[0]], [g[0], g[0]], **ok)
    assert all(bool((x == 0).all()) for x in p)  # nothing ran
    with pytest.raises(ma.AdamError):
        ma.muon_state_read(state, "m_codes")
    with pytest.raises(ma.AdamError):
        ma.muon_state_read(state, "v_codes")
    with pytest.raises(ValueError, match="bytes"):
        ma.muon_state_write(state, "m_bf16", torch.zeros(3, device="cuda"))


def test_step_refuses_to_be_captured():
    shapes = [(64, 64)]
    state = ma.muon_state_create(shapes, "f32")
    p, g = [torch.zeros(64, 64, device="cuda")], _grads(1, shapes)
    x = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ma.AdamError, match="capturing"):
            ma.muon_step(state, p, g, t=1, lr=1e-3)
        x.add_(1.0)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert bool((x == k + 1).all()) and bool((p[0] == 0).all())


def test_workspace_of_the_caller():
    x = _matrix(1, (300, 400))
    need = ma.muon_orthogonalize_workspace_bytes(1, 300, 400)
    with pytest.raises(ma.AdamError, match="needed"):
        ma.muon_orthogonalize(x, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ma.AdamError, match="256"):
        ma.muon_orthogonalize(x, workspace=torch.empty(need + 8, dtype=torch.uint8, device="cuda")[8:])
    guard = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    out = ma.muon_orthogonalize(x, workspace=guard[:need])  # junk in the workspace, and nothing written behind it
    assert torch.equal(out, ma.muon_orthogonalize(x)) and bool((guard[need:] == 77).all())
