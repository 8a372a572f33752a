"""Second moments that are infinite (one finite gradient of 2e19 makes one, since its square is
beyond fp32) beside ordinary ones: the element's param moves by m / inf = 0 and stays finite, whatever
the others of its wave are, for moments that are stored as they are."""
import numpy as np
import pytest
import torch

import memory_efficient_adam_amd as ma
import oracle
import workloads
from parity import to_device_grads

pytestmark = pytest.mark.gpu

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
# where each is: one in a wave's 256 elements, several, in the ragged end
AT = [0, 3, 300, 517, 518, 2047, 2048, 2048 + 700, 4999]
INF, NEAR = np.float32(np.inf), np.float32(3.38e38)  # the largest bf16 below infinity is 3.39e38


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def _moments(n, amsgrad, seed):
    """m, v and the maximum of earlier steps (padded), some of v or of the maximum infinite or near it."""
    rng = np.random.default_rng(seed)
    m = (rng.standard_normal(n) * 1e-3).astype(np.float32)
    m = np.where(np.abs(m) < 1e-9, np.float32(1e-3), m)
    v = (rng.standard_normal(n).astype(np.float32) * 1e-3) ** 2 + np.float32(1e-9)
    w = v * np.float32(1.5)
    for i, k in enumerate(AT):
        if amsgrad and i % 3 == 1:
            w[k] = INF  # the maximum alone never falls again
        else:
            v[k] = w[k] = NEAR if i % 3 == 2 else INF
    out = {"m": m, "v": v}
    if amsgrad:
        out["vmax"] = w
    return {k: np.concatenate([x, np.zeros(-n % 16, np.float32)]).astype(np.float32) for k, x in out.items()}


@pytest.mark.parametrize("decoupled", [True, False])
@pytest.mark.parametrize("amsgrad", [False, True])
@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("storage", ["f32", "bf16"])
def test_the_dense_step(storage, gdt, amsgrad, decoupled):
    n = 5000
    host = workloads.host_params(91, [n])
    params = [torch.from_numpy(host[0].copy()).cuda()]
    state = ma.adam_state_create([n], storage, gdt, amsgrad=amsgrad)
    ostate = oracle.OracleState([n], storage, grad_bf16=gdt == "bf16", amsgrad=amsgrad)
    for k, x in _moments(n, amsgrad, 1).items():
        name = f"{k}_{storage}"
        bits = oracle.bf16_from_f32(x) if storage == "bf16" else x
        ostate.buffers()[name][:] = bits
        ma.adam_state_write(state, name, torch.from_numpy(bits.view(np.int16) if storage == "bf16" else bits).cuda())
    for t in range(5, 8):
        grads = workloads.host_grads(91, [n], t, dtype=gdt)
        ma.adam_step(state, params, to_device_grads(grads, gdt), t=t, decoupled=decoupled, **HP)
        ostate.step(host, grads, t=t, decoupled=decoupled, **HP)
        assert np.isfinite(host[0]).all()
        got = params[0].cpu().numpy()
        assert np.isfinite(got).all(), f"t={t}: not finite at {np.flatnonzero(~np.isfinite(got))}"
        assert np.array_equal(got.view(np.int32), host[0].view(np.int32)), f"t={t}"
        for name, want in ostate.buffers().items():
            have = ma.adam_state_read(state, name).cpu().numpy()
            assert np.array_equal(have.view(np.uint8), want.view(np.uint8)), (t, name)
    state.destroy()


@pytest.mark.parametrize("amsgrad", [False, True])
@pytest.mark.parametrize("count", [64, 3000])
def test_the_step_of_rows(count, amsgrad):
    rows, cols = 10, 500  # all rows are named, so that it is the dense step
    host = workloads.host_params(92, [rows * cols])
    table = torch.from_numpy(host[0].copy()).cuda().view(rows, cols)
    moments = _moments(rows * cols, amsgrad, 2)
    buffers = {f"{k}_f32": torch.from_numpy(x).cuda() for k, x in moments.items()}
    ostate = oracle.OracleState([rows * cols], "f32", amsgrad=amsgrad)
    for k, x in moments.items():
        ostate.buffers()[f"{k}_f32"][:] = x
    tokens = torch.arange(count, device="cuda") % rows
    for t in (5, 6):
        gen = torch.Generator(device="cuda").manual_seed(t)
        grad = torch.randn(count, cols, generator=gen, device="cuda") * 1e-3
        dense = ma.embedding_gradient(grad, tokens, rows)
        ma.embedding_adam_step(table, grad, tokens, buffers, amsgrad=amsgrad, t=t, **HP)
        ostate.step(host, [dense.cpu().numpy().ravel()], t=t, **HP)
        got = table.cpu().numpy().ravel()
        assert np.isfinite(host[0]).all() and np.isfinite(got).all(), f"t={t}: not finite at {np.flatnonzero(~np.isfinite(got))}"
        assert np.array_equal(got.view(np.int32), host[0].view(np.int32))
        for name, want in ostate.buffers().items():
            assert np.array_equal(buffers[name].cpu().numpy().view(np.int32), want.view(np.int32)), (t, name)


@pytest.mark.parametrize("storage", ["f32", "bf16"])
def test_one_large_gradient(storage):
    # beta1 = 0: the first moment is the next gradient at once, the second stays infinite
    n, hp = 4096, {**HP, "beta1": 0.0}
    params = [torch.ones(n, device="cuda")]
    state = ma.adam_state_create([n], storage, "f32")
    grad = torch.full((n,), 1e-3, device="cuda")
    grad[777] = 2e19
    ma.adam_step(state, params, [grad], t=1, **hp)
    grad[777] = 1e-3
    ma.adam_step(state, params, [grad], t=2, **hp)
    assert torch.isfinite(params[0]).all()
