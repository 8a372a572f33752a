"""The gradient and the step of rows on tokens that fill single buckets of the grouping, over tables whose
rows take one, two and three digits to tell apart: against 64 bits, the same bits each time, and the
step of rows equal to the dense one."""
import numpy as np
import pytest
import torch

import embedding_ref as R
import memory_efficient_adam_amd as ma
from grouping_tokens import KINDS, ROWS, tokens_of

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
COUNTS = [3000, 16384, 65536]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _inputs(kind, n, rows, dtype, wide):
    """(tokens, grad, its rows that are named, tokens by their number among those): columns by what a table may take."""
    cols = 1 if rows > 1 << 21 else 20
    tokens = tokens_of(kind, n, rows, seed=n)
    inside = (tokens >= 0) & (tokens < rows)
    named, back = np.unique(tokens[inside], return_inverse=True)
    compact = np.full(n, -1, np.int64)
    compact[inside] = back
    gen = torch.Generator(device="cuda").manual_seed(n + rows % 1000)
    grad = torch.randn(n, cols, generator=gen, device="cuda").to(dtype)
    grad[torch.from_numpy(~inside).cuda()] = float("nan")
    return (torch.from_numpy(tokens).cuda().to(torch.int64 if wide else torch.int32), grad,
            torch.from_numpy(named).cuda(), torch.from_numpy(compact), gen)


def _near(got, want, tolerance, what):
    over = (got.double().cpu() - want).abs() - tolerance
    assert not torch.isnan(over).any() and not (over > 0).any(), f"{what}: {int((over > 0).sum())}, worst by {float(over.max()):.3g}"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", ROWS)
def test_gradient(rows, kind):
    for i, n in enumerate(COUNTS):
        for dtype, out, accumulate in ((BF16, F32, False), (F32, F32, True), (BF16, BF16, True)):
            tokens, grad, named, compact, gen = _inputs(kind, n, rows, dtype, wide=(i + accumulate) % 2 == 0)
            total, size, terms = R.gradient(torch.nan_to_num(grad), compact, len(named), 0.7)
            cols = grad.shape[1]
            into = torch.full((rows, cols), 3.0, dtype=out, device="cuda")
            if accumulate:
                into[named] = torch.randn(len(named), cols, generator=gen, device="cuda").to(out)
            old = into[named].double().cpu() if accumulate else None
            first = into.clone()
            ma.embedding_gradient(grad, tokens, rows, scale=0.7, out=first, accumulate=accumulate)
            what = f"{n} {dtype} {out} {accumulate}"
            _near(first[named], total if old is None else total + old, R.gradient_tolerance(total, size, terms, out, old), what)
            for _ in range(2):
                again = into.clone()
                ma.embedding_gradient(grad, tokens, rows, scale=0.7, out=again, accumulate=accumulate)
                assert torch.equal(again, first), what
            first[named] = 3.0 if accumulate else 0.0
            assert (first == (3.0 if accumulate else 0.0)).all(), f"{what}: rows that no token names"


@pytest.mark.parametrize("amsgrad", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", ROWS)
def test_step(rows, kind, amsgrad):
    for i, n in enumerate(COUNTS):
        tokens, grad, named, _, gen = _inputs(kind, n, rows, F32 if amsgrad else BF16, wide=i % 2 == 0)
        cols = grad.shape[1]
        sizes = ma.state_buffer_sizes([rows * cols], "f32", amsgrad)
        old = {"table": torch.full((rows * cols,), 0.5, device="cuda"),
               **{k: torch.full((b // 4,), 0.25, device="cuda") for k, b in sizes.items()}}
        got, dense = ({k: x.clone() for k, x in old.items()} for _ in range(2))
        kw = dict(t=5, amsgrad=amsgrad, **HP)
        g = ma.embedding_gradient(grad, tokens, rows, scale=0.7)
        ma.adam_step_noalloc([dense["table"]], [g.view(-1)], {k: dense[k] for k in sizes}, storage="f32", **kw)
        ma.embedding_adam_step(got["table"].view(rows, cols), grad, tokens, {k: got[k] for k in sizes}, scale=0.7, **kw)
        for k in old:
            want = old[k].clone()
            want[:rows * cols].view(rows, cols)[named] = dense[k][:rows * cols].view(rows, cols)[named]
            assert torch.equal(got[k], want), (n, k)
        # the rows were stepped.  Not each has to move: where m / root is -(decay's 5e-6) / (the rate's 2.4e-3), to within half
        # a step of 0.5 (3e-8), the param stays, in the dense step too; of normal gradients that is one in 10^5
        moved = (got["table"].view(rows, cols)[named] != 0.5).any(dim=1)
        assert moved.double().mean() > 0.99
