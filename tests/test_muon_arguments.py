"""Arguments of the Muon calls, and what the binding makes of them, where no GPU
is needed: layouts of batches, workspaces, remembered tensors."""
import pytest
import torch

import memory_efficient_adam_amd as ma
from memory_efficient_adam_amd import _binding as B
from memory_efficient_adam_amd import _muon as M
from test_muon_host import OUT, X, _orth


# the heads of a (rows, heads * d) weight: matrices of rows x d, d apart, rows heads * d apart
HEADS = dict(batch=12, rows=100, cols=64, out_batch_stride=64, out_row_stride=12 * 64)


# (the pointers are no memory: calls that are not refused have to end at a missing device)
@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="would launch on pointers that are no memory")
def test_matrices_of_out_may_lie_side_by_side():
    x = dict(x_batch_stride=64, x_row_stride=12 * 64)
    assert _orth(**HEADS, **x) == -5
    assert _orth(out=X, **HEADS, **x) == -5  # in place
    assert _orth(**{**HEADS, "out_row_stride": 13 * 64}, **x) == -5
    for over in (dict(out_batch_stride=63), dict(out_row_stride=12 * 64 - 1), dict(batch=13), dict(out_batch_stride=0)):
        assert _orth(**{**HEADS, **over, **x}) == -1 and "overlap" in ma.adam_last_error(), over
    # all of them count where x may not lie
    last = X + 4 * (99 * 12 * 64 + 12 * 64)
    assert _orth(out=last - 4, **HEADS, **x) == -1 and "overlaps" in ma.adam_last_error()
    assert _orth(out=last, **HEADS, **x) == -5


def test_strides_whose_reach_does_not_fit_are_refused():
    # (batch - 1) * stride is 2^62, 2^64 (0 in 64 bits) or more
    for batch in (2 ** 20 + 1, 2 ** 22 + 1, 2 ** 24 + 1, 2 ** 31 - 1):
        for name in ("x_batch_stride", "out_batch_stride"):
            kw = {"batch": batch, "rows": 1, "cols": 8, "x_row_stride": 8, "out_row_stride": 8,
                  "x_batch_stride": 8, "out_batch_stride": 8, name: 2 ** 40}
            for out in (OUT, X + 2 ** 41):
                assert _orth(out=out, **kw) == -1 and "reach" in ma.adam_last_error(), kw
    kw = dict(batch=1, rows=2 ** 21 - 1, cols=8, out_row_stride=8)
    assert _orth(x_row_stride=2 ** 40, **kw) == -1 and "reach" in ma.adam_last_error()


def test_a_workspace_that_holds_x_or_out_is_refused():
    need = ma.muon_orthogonalize_workspace_bytes(2, 100, 80)
    size = 4 * 2 * 8000
    for ws in (X, X - need + 256, X + (size - 4) // 256 * 256, OUT, OUT - need + 256, OUT + (size - 4) // 256 * 256):
        assert _orth(ws=ws) == -1 and "workspace overlaps" in ma.adam_last_error(), hex(ws)
    assert _orth(x=OUT, ws=OUT) == -1 and "workspace overlaps" in ma.adam_last_error()  # in place


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="would launch on pointers that are no memory")
def test_a_workspace_beside_x_and_out_is_taken():
    need = ma.muon_orthogonalize_workspace_bytes(2, 100, 80)
    size = 4 * 2 * 8000
    assert need % 256 == 0 and size % 256 == 0
    for ws in (X - need, X + size, OUT - need, OUT + size):
        assert _orth(ws=ws) == -5, hex(ws)
    # a workspace larger than needed may hold them behind its used part
    assert _orth(ws=X - need, ws_bytes=1 << 40) == -5
    # matrices that need none
    assert _orth(rows=60, cols=80, ws=X, ws_bytes=1 << 30) == -5


# ---------------------------------------------------------------- the binding
@pytest.mark.parametrize("shape", [(0, 3, 40, 50), (3, 0, 40, 50), (2, 0, 3, 40, 50), (3, 2, 0, 50), (3, 2, 40, 0), (0, 0), (4, 0, 0)],
                         ids=str)
def test_empty_batches_of_any_arrangement_are_taken(shape):
    for t in (torch.zeros(shape), torch.zeros(shape).transpose(0, -3) if len(shape) > 3 else torch.zeros(shape),
              torch.zeros(shape).transpose(-1, -2)):
        batch, rows, cols, batch_stride, row_stride, code = M._matrices_of("x", tuple(t.shape), t.stride(), t.dtype)
        assert batch * rows * cols == 0 and (rows, cols) == tuple(t.shape[-2:]) and code == 0
        assert batch == 0 or batch == t.shape[:-2].numel()
        assert batch_stride >= 0 and row_stride >= cols  # as the library wants them


def _remembering_state(monkeypatch, params, grads):
    """A state that has checked these (host) tensors before, as one has on a device."""
    st = M.MuonState(None, [tuple(p.shape) for p in params], M.muon_layout(2, 0, 2048, 0), device=0)
    with monkeypatch.context() as m:
        m.setattr(M, "_check_matrices", lambda *a: None)
        with pytest.raises(ma.AdamError):  # reaches the library, which refuses the NULL state
            ma.muon_step(st, params, grads, lr=1e-3, t=1, stream=0)
    with pytest.raises(ma.AdamError):  # remembered
        ma.muon_step(st, params, grads, lr=1e-3, t=2, stream=0)
    return st


@pytest.mark.parametrize("what,change", [
    ("shape", lambda t: setattr(t, "data", t.data.view(6, 4))), ("contiguous", lambda t: t.t_()),
    ("numel", lambda t: setattr(t, "data", t.data[:3])), ("dtype", lambda t: setattr(t, "data", t.data.view(torch.int32)))])
@pytest.mark.parametrize("of", [0, 1], ids=["param", "grad"])
def test_a_remembered_tensor_that_changed_its_form_is_checked_again(monkeypatch, what, change, of):
    square = what == "contiguous"
    sets = [[torch.zeros(6, 6) if square else torch.zeros(4, 6), torch.zeros(3, 2)] for _ in range(2)]
    st = _remembering_state(monkeypatch, *sets)
    at = sets[of][0].data_ptr()
    change(sets[of][0])
    assert sets[of][0].data_ptr() == at
    with pytest.raises(ValueError, match=what):
        ma.muon_step(st, *sets, lr=1e-3, t=3, stream=0)


def test_no_forward_mode_gradient_is_dropped_unremarked():
    import torch.autograd.forward_ad as fwd
    x = torch.ones(4, 5)
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones(4, 5))
        for args in (dict(x=dual), dict(x=x, out=dual)):
            with pytest.raises(ValueError, match="forward-mode"):
                ma.muon_orthogonalize(**args)
            with torch.no_grad(), pytest.raises(ValueError, match="forward-mode"):
                ma.muon_orthogonalize(**args)
        for plain in (x, fwd.unpack_dual(dual).primal):
            with pytest.raises(ValueError, match="device"):  # the next check: a host tensor
                ma.muon_orthogonalize(plain)
    with pytest.raises(ValueError, match="forward-mode"):
        torch.func.jvp(lambda t: ma.muon_orthogonalize(t), (x,), (x,))


class _StreamOf:
    """What of a torch stream the binding looks at."""

    def __init__(self, index):
        self.device, self.cuda_stream = torch.device("cuda", index), 4096


@pytest.mark.parametrize("call", ["step", "orthogonalize"])
def test_a_stream_of_another_device_is_refused(monkeypatch, call):
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    empty = M.MuonState(None, [(0, 5)], M.muon_layout(3, 0, 2048, 0), device=0)
    none = [torch.zeros(0, 5)]
    if call == "step":
        with pytest.raises(ma.AdamError):  # the library refuses the NULL state
            ma.muon_step(empty, none, none, lr=1e-3, t=1, stream=_StreamOf(0))
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            ma.muon_step(empty, none, none, lr=1e-3, t=1, stream=_StreamOf(1))
    else:
        monkeypatch.setattr(torch.Tensor, "is_cuda", True)
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            ma.muon_orthogonalize(torch.zeros(70, 0, 5), stream=_StreamOf(1))


# ---------------------------------------------------------------- workspaces
def _workspace(shapes):
    return ma.muon_state_workspace_bytes(shapes, "q8")


@pytest.mark.parametrize("count,shape", [(4096, (64, 64)), (512, (16, 768)), (3000, (768, 3)), (20000, (1, 1))], ids=str)
def test_small_matrices_take_a_workspace_of_their_updates_alone(count, shape):
    n = shape[0] * shape[1]
    # u, a partial sum a block, a sum a matrix, the counters, and rounding to 256 bytes
    most = count * (4 * (n + 15 & ~15) + 8 * (-(-n // 2048)) + 8) + 1024 + 3 * 256
    assert 4 * n * count <= _workspace([shape] * count) <= most
    assert _workspace([shape] * count * 40) <= (1 << 28) + (1 << 26)  # 2^26 elements of u at a time


def test_small_matrices_add_their_updates_to_a_list_and_no_factors():
    large = [(1024, 1024)] * 4
    assert _workspace(large + [(64, 768)] * 3) <= _workspace(large) + 4 * 3 * 64 * 768 + 4096
    many = [(64, 768)] * 600
    assert _workspace(large + many) <= _workspace(large) + _workspace(many)


def test_square_factors_are_those_the_iterations_use():
    n = 4096 * 4096
    # no runs for square matrices: four arrays of X, A and P
    assert _workspace([(4096, 4096)] * 4) <= 4 * n * (16 + 8) + (1 << 26) + (1 << 20)
    # runs of three: five square arrays (long matrices, their Gram matrices are small)
    wide = _workspace([(768, 7680)])
    assert wide >= 16 * 768 * 7680 + 20 * 768 * 768


# ---------------------------------------------------------------- states that go
class _Cuda:
    """torch.cuda, as far as freeing a state asks it."""

    def __init__(self):
        self.cuda, self.capturing, self.initialized = self, False, True

    def is_initialized(self):
        return self.initialized

    def is_current_stream_capturing(self):
        if isinstance(self.capturing, Exception):
            raise self.capturing
        return self.capturing


def test_states_that_go_during_a_capture_are_freed_once_after_it():
    cuda, freed, waiting = _Cuda(), [], []
    release = lambda *a: B._release(*a, waiting=waiting, modules={"torch": cuda})  # noqa: E731
    for make in (lambda: M.MuonState(None, [(3, 4)], None), lambda: B.AdamState(None, [12], None)):
        states = [make() for _ in range(4)]
        for k, st in enumerate(states):
            st.handle, st._free, st._release = k + 1, freed.append, release
        states[0].destroy()
        assert freed == [1] and not waiting
        cuda.capturing = True
        states[1].destroy()
        release()
        assert freed == [1] and len(waiting) == 1
        cuda.capturing = RuntimeError("the query failed")  # nothing is known of a capture
        with pytest.raises(RuntimeError):
            states[2].destroy()
        cuda.capturing = False
        states[3].destroy()
        for st in states:
            st.destroy()
        assert sorted(freed) == [1, 2, 3, 4] and not waiting
        freed.clear()
    cuda.initialized, cuda.capturing = False, True  # no capture by torch without its runtime
    release(freed.append, 9)
    B._release(freed.append, 10, waiting=waiting, modules={})
    assert freed == [9, 10]
