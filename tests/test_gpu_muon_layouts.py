"""GPU tests of the layouts, streams and workspaces that the Muon calls take."""
import gc

import pytest
import torch

import memory_efficient_adam_amd as ma
import muon_ref
from memory_efficient_adam_amd import _binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def _randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


@pytest.mark.parametrize("rows,heads,d", [(96, 3, 64), (300, 5, 130), (65, 7, 33)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_heads_of_a_fused_weight_in_place_and_out_of_place(rows, heads, d, dtype):
    whole = _randn(rows, rows + 2, heads * d + 9).to(dtype)
    before = whole.clone()
    x = whole[1:rows + 1, 4:4 + heads * d].unflatten(1, (heads, d)).transpose(0, 1)
    want = ma.muon_orthogonalize(x.contiguous())
    dest = torch.full_like(whole, 5.0)
    out = dest[1:rows + 1, 4:4 + heads * d].unflatten(1, (heads, d)).transpose(0, 1)
    assert ma.muon_orthogonalize(x, out=out) is out
    assert torch.equal(out, want) and torch.equal(whole, before)
    assert ma.muon_orthogonalize(x, out=x) is x and torch.equal(x, want)
    for t, rest in ((dest, 5.0), (whole, before)):  # nothing else is written
        t[1:rows + 1, 4:4 + heads * d] = rest if isinstance(rest, float) else rest[1:rows + 1, 4:4 + heads * d]
        assert bool((t == rest).all())


@pytest.mark.parametrize("shape", [(0, 3, 40, 50), (3, 0, 40, 50), (2, 0, 3, 40, 50), (3, 2, 0, 50), (3, 2, 40, 0)], ids=str)
def test_empty_batches(shape):
    x = torch.empty(shape, device="cuda")
    assert ma.muon_orthogonalize(x).shape == x.shape
    assert ma.muon_orthogonalize(x, out=x) is x


@pytest.mark.parametrize("kind", ["muon", "adam"])
def test_a_buffer_read_on_a_side_stream_is_not_written_by_earlier_work(kind):
    # memory given back to the current stream's allocator while fills of it are
    # still queued there is no place for a copy that another stream makes now
    side = torch.cuda.Stream()
    if kind == "muon":
        state, read = ma.muon_state_create([(1024, 1024)], "f32"), ma.muon_state_read
        ma.muon_state_write(state, "m_f32", torch.full((1 << 20,), 3.0, device="cuda"))
    else:
        state, read = ma.adam_state_create([1 << 20], "q8_v_only"), ma.adam_state_read
        ma.adam_state_write(state, "m_f32", torch.full((1 << 20,), 3.0, device="cuda"))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    slow = torch.empty(1 << 28, device="cuda")
    reused = torch.empty(1 << 20, device="cuda")
    for _ in range(20):
        slow.fill_(1.0)
    reused.fill_(7.0)
    del reused
    got = read(state, "m_f32", stream=side)
    torch.cuda.synchronize()
    assert bool((got == 3.0).all())
    raw = read(state, "m_f32", stream=side.cuda_stream)
    side.synchronize()
    zero = read(state, "m_f32", stream=0)
    torch.cuda.synchronize()
    assert torch.equal(raw, got) and torch.equal(zero, got)
    state.destroy()


@pytest.mark.parametrize("large", [[(70, 90)], [(300, 900)] * 2, [(768, 2304), (128, 4000)], [(600, 600)]], ids=str)
def test_a_step_of_small_matrices_that_outweigh_the_large_ones(large):
    # the updates of all of them stand where the large ones' factors come to be
    shapes = [(64, 768)] * 20 + large + [(33, 65), (0, 5), (5, 0), (768, 64), (1, 1)] * 9 + [(700, 50)] * 30
    grads = [1e-3 * _randn(k, *s) for k, s in enumerate(shapes)]
    params = [torch.zeros(s, device="cuda") for s in shapes]
    state = ma.muon_state_create(shapes, "f32")
    for t in (1, 2):
        for p in params:
            p.zero_()
        ma.muon_step(state, params, grads, t=t, lr=1.0, momentum=0.0, scale="none")
        for k, (p, g) in enumerate(zip(params, grads)):
            if g.numel() == 0:
                continue
            ref = muon_ref.orthogonalize(g)
            own = float((muon_ref.orthogonalize(g, dtype=torch.float32).double() - ref).norm() / ref.norm())
            assert float((-p.double() - ref).norm() / ref.norm()) <= 8 * own + 2.0 ** -21, (t, k, shapes[k])
    state.destroy()


@pytest.mark.parametrize("kind", ["muon", "adam"])
@pytest.mark.parametrize("how", ["destroyed", "collected"])
def test_a_state_that_goes_during_a_capture_leaves_the_graph_whole(kind, how):
    make = {"muon": lambda: ma.muon_state_create([(70, 80)], "q8"), "adam": lambda: ma.adam_state_create([5000], "q8")}[kind]
    holder = [make()]
    if how == "collected":  # only the cycle collector ends it, as one that an exception's frames hold
        holder.append(holder)
    x = torch.zeros(1000, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.add_(1.0)
        if how == "destroyed":
            holder[0].destroy()
        del holder
        gc.collect()
        x.add_(1.0)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert bool((x == 2.0 * (k + 1)).all())
    assert len(_binding._waiting) == 1
    make()  # another state frees it
    assert not _binding._waiting


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(40, 70), (300, 300), (600, 520), (520, 1600)], ids=str)
def test_zero_and_nonfinite_bf16_matrices(shape, out_dtype):
    # (large ones are taken as they are, with the rest of the norm beside them)
    x = _randn(1, 4, *shape).bfloat16()
    x[3] = 0.0
    x[3, 0, 0] = 2.0 ** -133  # the least number
    run = lambda: ma.muon_orthogonalize(x, out=torch.empty(4, *shape, dtype=out_dtype, device="cuda"), eps=1e-43)  # noqa: E731
    good = run()
    s = 1.0  # one entry: its own singular value
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    assert abs(float(good[3, 0, 0]) - s) <= 2.0 ** -8 and int((good[3] != 0).sum()) == 1
    for value in (0.0, float("nan"), float("inf"), float("-inf")):
        x[1] = 0.0
        x[1, -1, -1] = value
        out = run()
        assert bool((out[1] == 0).all() if value == 0.0 else out[1].isnan().all())
        assert all(torch.equal(out[k], good[k]) for k in (0, 2, 3))
