"""The step with fp32 moments on the GPU: bit for bit against the oracle's
fp32 mode, against the formula in 64 bits, over caller-owned buffers, in a
graph, through a checkpoint, and beyond 32-bit offsets."""
import numpy as np
import pytest
import torch

import memory_efficient_adam_amd as ma
import oracle
import workloads
from parity import to_device_grads

pytestmark = pytest.mark.gpu

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
RAGGED = list(workloads.RAGGED_SIZES) + [0, 40000, 7]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def _bits(x):
    return x.view(torch.int32).cpu().numpy()


def _same(state, params, ostate, host, where):
    for k, p in enumerate(params):
        assert np.array_equal(_bits(p), host[k].view(np.int32)), f"{where}: tensor {k}"
    for name, want in ostate.buffers().items():
        got = ma.adam_state_read(state, name).cpu().numpy()
        assert np.array_equal(got.view(np.int32), want.view(np.int32)), f"{where}: {name}"


@pytest.mark.parametrize("decoupled", [True, False])
@pytest.mark.parametrize("amsgrad", [False, True])
@pytest.mark.parametrize("gdt", ["f32", "bf16"])
def test_bit_for_bit_against_the_oracle(gdt, amsgrad, decoupled):
    host = workloads.host_params(81, RAGGED)
    params = [torch.from_numpy(p.copy()).cuda() for p in host]
    state = ma.adam_state_create(RAGGED, "f32", gdt, amsgrad=amsgrad)
    assert state.storage == "f32" and state.amsgrad == amsgrad
    ostate = oracle.OracleState(RAGGED, "f32", grad_bf16=gdt == "bf16", amsgrad=amsgrad)
    for t in range(1, 5):
        grads = workloads.host_grads(81, RAGGED, t, dist="normal_outliers", dtype=gdt)
        ma.adam_step(state, params, to_device_grads(grads, gdt), t=t, decoupled=decoupled, **HP)
        ostate.step(host, grads, t=t, decoupled=decoupled, **HP)
        _same(state, params, ostate, host, f"t={t}")
    state.destroy()


def test_extreme_gradients_stay_in_their_elements():
    # exact zeros, the least and largest numbers (whose squares under- and overflow), infinities and NaN
    values = np.array([0.0, -0.0, 1e-45, -1e-38, 1e-30, 1e-20, 3e38, -3e38, 1e19, 2e19, np.inf, -np.inf, np.nan],
                      np.float32)
    n = 5000
    host = workloads.host_params(82, [n])
    clean = [host[0].copy()]
    params, params2 = (torch.from_numpy(host[0].copy()).cuda() for _ in range(2))
    grad = workloads.host_grads(82, [n], 1)[0]
    at = np.arange(len(values)) * 381
    dirty = grad.copy()
    dirty[at] = values
    state, state2 = (ma.adam_state_create([n], "f32", "f32", amsgrad=True) for _ in range(2))
    ostate, ostate2 = (oracle.OracleState([n], "f32", amsgrad=True) for _ in range(2))
    for t in (1, 2):
        ma.adam_step(state, [params], [torch.from_numpy(dirty).cuda()], t=t, **HP)
        ma.adam_step(state2, [params2], [torch.from_numpy(grad).cuda()], t=t, **HP)
        ostate.step(host, [dirty], t=t, **HP)
        ostate2.step(clean, [grad], t=t, **HP)
    others = np.setdiff1d(np.arange(n), at)
    assert torch.equal(params[others], params2[others])
    got, want = params.cpu().numpy(), host[0]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    live = ~np.isnan(want)
    assert np.array_equal(got[live].view(np.int32), want[live].view(np.int32))
    _same(state2, [params2], ostate2, clean, "clean")


@pytest.mark.parametrize("amsgrad", [False, True])
def test_against_the_formula_in_64_bits(amsgrad):
    # Per step m and v take at most 2 and 3 roundings (of the product with 1 - beta; of g^2, the product and the fma)
    # and carry the error of the former value; p takes the two of its product and fma besides what the quotient has:
    # m's and half of v's, and six of sqrt, two fmas, division and the scalars.
    n, steps, half = 10007, 3, 2.0 ** -24
    gen = torch.Generator(device="cuda").manual_seed(7)
    p = torch.randn(n, generator=gen, device="cuda") * 0.02
    state = ma.adam_state_create([n], "f32", "f32", amsgrad=amsgrad)
    h = {k: float(np.float32(v)) for k, v in HP.items()}
    x, m, v, w = p.double(), *(torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(3))
    moved = torch.zeros_like(x)
    m_size, v_size = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(1, steps + 1):
        g = torch.randn(n, generator=gen, device="cuda") * 1e-3
        ma.adam_step(state, [p], [g], t=t, **HP)
        m = h["beta1"] * m + (1 - h["beta1"]) * g.double()
        m_size = h["beta1"] * m_size + (1 - h["beta1"]) * g.double().abs()
        v = h["beta2"] * v + (1 - h["beta2"]) * g.double() ** 2
        w = torch.maximum(w, v)
        root = ((w if amsgrad else v) / (1 - h["beta2"] ** t)).sqrt() + h["eps"]
        x = x * (1 - h["lr"] * h["weight_decay"]) - h["lr"] / (1 - h["beta1"] ** t) * m / root
        # |update| for the quotient's error: m's error is relative to the sum of sizes
        moved += h["lr"] / (1 - h["beta1"] ** t) * (m.abs() * 12 * t + m_size * 3 * t) / root
    got = {k: ma.adam_state_read(state, k)[:n].double() for k in ("m_f32", "v_f32") + (("vmax_f32",) if amsgrad else ())}
    # the scalars 1 - beta are rounded once too
    assert ((got["m_f32"] - m).abs() <= 4 * steps * half * m_size).all()
    assert ((got["v_f32"] - v).abs() <= 5 * steps * half * v).all()
    if amsgrad:
        assert ((got["vmax_f32"] - w).abs() <= 5 * steps * half * w).all()
    assert ((p.double() - x).abs() <= 1.01 * half * (3 * steps * x.abs().clamp(min=1e-3) + moved)).all()


@pytest.mark.parametrize("gdt,amsgrad", [("f32", False), ("bf16", True)])
def test_caller_owned_buffers_and_graphs(gdt, amsgrad):
    numels = [3000, 2048, 17, 12289, 0, 5000, 1]
    host = workloads.host_params(83, numels)
    params, params2 = ([torch.from_numpy(p.copy()).cuda() for p in host] for _ in range(2))
    state = ma.adam_state_create(numels, "f32", gdt, amsgrad=amsgrad)
    buffers = {k: torch.zeros(b // 4, dtype=torch.float32, device="cuda")
               for k, b in ma.state_buffer_sizes(numels, "f32", amsgrad).items()}
    grads = [torch.empty_like(g) for g in to_device_grads(workloads.host_grads(83, numels, 1, dtype=gdt), gdt)]

    def fill(t):
        for a, b in zip(grads, to_device_grads(workloads.host_grads(83, numels, t, dtype=gdt), gdt)):
            a.copy_(b)

    def same(where):
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(params, params2)):
            assert torch.equal(a.view(torch.int32), b.view(torch.int32)), (where, k)
        for k, b in buffers.items():
            assert torch.equal(ma.adam_state_read(state, k), b), (where, k)

    kw = dict(storage="f32", grad_dtype=gdt, amsgrad=amsgrad, t=3, **HP)
    for i in (1, 2):
        fill(i)
        ma.adam_step(state, params, grads, t=3, **HP)
        ma.adam_step_noalloc(params2, grads, buffers, **kw)
        same(f"call {i}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ma.adam_step_noalloc(params2, grads, buffers, **kw)
    for i in range(3, 7):
        fill(i)
        ma.adam_step(state, params, grads, t=3, **HP)
        graph.replay()
        same(f"replay {i}")
    state.destroy()


@pytest.mark.parametrize("amsgrad", [False, True])
def test_checkpoint_resumes_bit_for_bit(amsgrad):
    numels = [4099, 2048, 33]
    grads = [to_device_grads(workloads.host_grads(84, numels, t), "f32") for t in range(1, 5)]
    first = [torch.from_numpy(p).cuda() for p in workloads.host_params(84, numels)]
    state = ma.adam_state_create(numels, "f32", "f32", amsgrad=amsgrad)
    for t in (1, 2):
        ma.adam_step(state, first, grads[t - 1], t=t, **HP)
    second = [p.clone() for p in first]
    resumed = ma.adam_state_load(ma.adam_state_save(state))
    assert resumed.storage == "f32" and resumed.numels == numels and resumed.amsgrad == amsgrad
    for t in (3, 4):
        ma.adam_step(state, first, grads[t - 1], t=t, **HP)
        ma.adam_step(resumed, second, grads[t - 1], t=t, **HP)
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    names = ("m_f32", "v_f32") + (("vmax_f32",) if amsgrad else ())
    for name in names:
        assert torch.equal(ma.adam_state_read(state, name), ma.adam_state_read(resumed, name)), name
        ma.adam_state_write(resumed, name, torch.zeros_like(ma.adam_state_read(state, name)))
        assert not ma.adam_state_read(resumed, name).any()


def test_padding_of_a_written_state_takes_no_part():
    numels = [5, 2050]
    padded = 16 + 2064
    state = ma.adam_state_create(numels, "f32", "f32", amsgrad=True)
    for name in ("m_f32", "v_f32", "vmax_f32"):
        ma.adam_state_write(state, name, torch.full((padded,), float("nan"), device="cuda"))
        values = ma.adam_state_read(state, name)
        values[:5], values[16:16 + 2050] = 0.0, 0.0
        ma.adam_state_write(state, name, values)
    params = [torch.ones(n, device="cuda") for n in numels]
    ma.adam_step(state, params, [torch.ones_like(p) for p in params], t=1, **HP)
    for name in ("m_f32", "v_f32", "vmax_f32"):
        values = ma.adam_state_read(state, name)
        assert torch.isfinite(values).all() and not values[5:16].any() and not values[16 + 2050:].any(), name
    assert all(torch.isfinite(p).all() for p in params)


def test_refusals():
    state = ma.adam_state_create([100], "f32", "f32")
    p, g = torch.zeros(100, device="cuda"), torch.ones(100, device="cuda")
    for kw in (dict(stochastic=True), dict(percentile=99.9), dict(static_scales=True)):
        with pytest.raises(ma.AdamError, match="8-bit storage only"):
            ma.adam_step(state, [p], [g], t=1, **HP, **kw)
    with pytest.raises(ma.AdamError) as e:
        ma.adam_step(state, [p], [g], t=1, expect=("q8_v_only", "f32"), **HP)
    assert e.value.code == -2
    for name in ("v_codes", "v_scale", "m_codes", "vmax_f32"):
        with pytest.raises(ma.AdamError):
            ma.adam_state_read(state, name)
    assert not p.any()


def test_offsets_beyond_32_bits():
    # one tensor of more than 2^31 elements behind a small one: byte offsets pass 2^33
    numels = [33, 2 ** 31 + 4099]
    params = [torch.ones(n, device="cuda") for n in numels]
    state = ma.adam_state_create(numels, "f32", "bf16")
    grads = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in numels]
    at = [0, 1, 2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 4098]
    for i, k in enumerate(at):
        grads[1][k] = 0.5 + i
    ma.adam_step(state, params, grads, t=1, **{**HP, "weight_decay": 0.0})
    torch.cuda.synchronize()
    step = 2 ** 28  # nonzero counts in 32 bits
    moved = [first + k for first in range(0, numels[1], step)
             for k in (params[1][first:first + step] != 1.0).nonzero().flatten().tolist()]
    assert moved == at and not (params[0] != 1.0).any()
    m = torch.empty(16 * 3 + (2 ** 31 + 4099 + 15) // 16 * 16, device="cuda")
    ma.adam_state_read(state, "m_f32", out=m)
    assert [round(float(m[48 + k]) * 10, 4) for k in at] == [0.5 + i for i in range(len(at))]
    del m, params, grads
    state.destroy()
    torch.cuda.empty_cache()
