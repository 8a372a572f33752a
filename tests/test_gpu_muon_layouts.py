"""GPU tests of the layouts, streams and workspaces that the Muon calls take."""
import pytest
import torch

import memory_efficient_adam_amd as ma

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
