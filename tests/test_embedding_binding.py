"""What the embedding calls' binding hands to the library and to torch, on host tensors and
with the library's calls recorded in place of made."""
import math

import pytest
import torch

import memory_efficient_adam_amd as ma
from memory_efficient_adam_amd import _embedding as E

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, t=1)


class Recorder:
    """The library, with the scales of the calls that it would make."""

    def __init__(self, real):
        self.scales = []
        self.embedding_gradient_workspace_bytes = real.embedding_gradient_workspace_bytes

        def call(shape, *arguments):
            self.scales.append(shape.scale)
            return 0
        self.embedding_lookup = self.embedding_gradient = self.embedding_adam_step = call


@pytest.fixture
def calls(monkeypatch):
    recorder = Recorder(E.library())
    monkeypatch.setattr(E, "library", lambda: recorder)
    monkeypatch.setattr(E, "_check_tensors", lambda *named: None)
    monkeypatch.setattr(E, "_current_stream", lambda device: 0)
    return recorder


def _state(n):
    return {k: torch.zeros(b // 4) for k, b in ma.state_buffer_sizes([n], "f32").items()}


def _each_call(**kw):
    table, tokens, grad = torch.ones(5, 4), torch.zeros(3, dtype=torch.int64), torch.ones(3, 4)
    ma.embedding_lookup(table, tokens, **kw)
    ma.embedding_lookup(table, tokens, out=torch.empty(3, 4), **kw)
    ma.embedding_gradient(grad, tokens, 5, **kw)
    ma.embedding_gradient(grad, tokens, 5, out=torch.empty(5, 4), **kw)
    ma.embedding_adam_step(table, grad, tokens, _state(20), **kw, **HP)


def test_a_scale_keeps_its_sign_whatever_was_called_before(calls):
    # 0.0 and -0.0 are equal, but the zeros that they make are not the same bits
    for scale in (0.0, -0.0, 0.0, 2.0, -2.0):
        calls.scales.clear()
        _each_call(scale=scale)
        assert [math.copysign(1.0, s) * abs(s) for s in calls.scales] == [scale] * 5
        assert [math.copysign(1.0, s) for s in calls.scales] == [math.copysign(1.0, scale)] * 5, scale


def test_what_a_call_writes_is_seen_by_autograd(calls):
    # a product that keeps x for its backward pass, x written over in between: torch's own calls make
    # that an error, not a gradient of the new values
    weight = torch.ones(3, 4, requires_grad=True)
    table, tokens, grad = torch.ones(5, 4), torch.zeros(3, dtype=torch.int64), torch.ones(3, 4)
    wide = torch.ones(5, 4, requires_grad=True)

    def after(x, by, write):
        loss = (x * by).sum()
        write()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    out, dense = torch.ones(3, 4), torch.ones(5, 4)
    after(out, weight, lambda: ma.embedding_lookup(table, tokens, out=out))
    after(dense, wide, lambda: ma.embedding_gradient(grad, tokens, 5, out=dense))
    after(dense, wide, lambda: ma.embedding_gradient(grad, tokens, 5, out=dense, accumulate=True))
    after(table, wide, lambda: ma.embedding_adam_step(table, grad, tokens, _state(20), **HP))
    # nothing that is only read, and tensors of inference mode have no count
    before = [x._version for x in (table, tokens, grad)]
    ma.embedding_lookup(table, tokens, out=out)
    ma.embedding_gradient(grad, tokens, 5, out=dense)
    assert [x._version for x in (table, tokens, grad)] == before
    with torch.inference_mode():
        ma.embedding_lookup(table, tokens, out=torch.empty(3, 4))
        ma.embedding_gradient(grad, tokens, 5, out=torch.empty(5, 4))
