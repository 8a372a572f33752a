"""The fp32 storage (ADAM_STORE_F32) where no GPU is needed: state sizes, the
checkpoint stream's records, and what a step refuses before any device call."""
import ctypes

import pytest

import memory_efficient_adam_amd as ma
from memory_efficient_adam_amd import _binding as B
from test_abi_host import _load_rc, _serialized

NUMELS = [5000, 17]
PADDED = 5008 + 32


def _records(amsgrad):
    return [(6, 4 * PADDED), (10, 4 * PADDED)] + ([(11, 4 * PADDED)] if amsgrad else [])


def test_state_bytes_and_buffers():
    numels = [1, 17, 2048, 2049, 6001, 0, 1048576]
    padded = sum((n + 15) // 16 * 16 for n in numels)
    assert ma.adam_state_bytes(numels, "f32", "f32") == 8 * padded
    assert ma.adam_state_bytes(numels, "f32", "bf16", amsgrad=True) == 12 * padded
    assert ma.state_buffer_sizes(numels, "f32") == {"m_f32": 4 * padded, "v_f32": 4 * padded}
    assert ma.state_buffer_sizes(numels, "f32", True) == {"m_f32": 4 * padded, "v_f32": 4 * padded,
                                                          "vmax_f32": 4 * padded}
    for name in ("v_f32", "vmax_f32"):
        assert name in B.BUFFERS and B._BUF_DTYPES[name] == "float32"


@pytest.mark.parametrize("amsgrad", [False, True])
def test_a_valid_stream_gets_past_validation(amsgrad):
    rc, h = _load_rc(_serialized(NUMELS, storage=4, options=int(amsgrad), records=_records(amsgrad)))
    if rc == 0:
        ma.library().adam_state_destroy(h)
    else:  # no GPU: the first device call is what fails
        assert rc in (-4, -5), ma.adam_last_error()


@pytest.mark.parametrize("records", [
    [(10, 4 * PADDED), (6, 4 * PADDED)],               # order
    [(6, 4 * PADDED), (10, 2 * PADDED)],               # size
    [(6, 4 * PADDED)],                                 # one missing
    [(6, 4 * PADDED), (5, 4 * PADDED)],                # another storage's buffer
    [(6, 4 * PADDED), (10, 4 * PADDED), (11, 4 * PADDED)],  # AMSGrad's without the option
])
def test_a_stream_of_other_records_is_refused(records):
    rc, h = _load_rc(_serialized(NUMELS, storage=4, records=records))
    assert rc == -1 and h is None


def test_a_claim_of_amsgrad_without_its_record_is_refused():
    rc, h = _load_rc(_serialized(NUMELS, storage=4, options=1, records=_records(False)))
    assert rc == -1 and h is None


@pytest.mark.parametrize("flag,name", [(2, "stochastic"), (4, "percentile"), (8, "static scales")])
def test_flags_of_8_bit_storage_are_refused(flag, name):
    lib = ma.library()
    hp = B.adam_hparams(1e-3, 0.9, 0.999, 1e-8, 0.0, 99.0, 1, 1 | flag, 0, 42)
    lay = B._layout("f32", "f32")
    n, numels = B._numels([5000])
    ptrs = ctypes.cast((ctypes.c_void_p * 1)(4096), ctypes.c_void_p)
    state = ctypes.cast((ctypes.c_void_p * 12)(*[4096] * 12), ctypes.c_void_p)
    assert lib.adam_step_noalloc(n, numels, ctypes.byref(lay), ptrs, ptrs, state, None, ctypes.byref(hp), None) == -1
    assert name in ma.adam_last_error()


def test_missing_and_unaligned_buffers_are_refused():
    lib = ma.library()
    hp = B.adam_hparams(1e-3, 0.9, 0.999, 1e-8, 0.0, 100.0, 1, 1, 0, 42)
    n, numels = B._numels([5000])
    ptrs = ctypes.cast((ctypes.c_void_p * 1)(4096), ctypes.c_void_p)

    def call(options=0, **buffers):
        lay = B._layout("f32", "bf16", options=options)
        state = (ctypes.c_void_p * 12)()
        for name, at in buffers.items():
            state[B.BUFFERS[name]] = at
        return lib.adam_step_noalloc(n, numels, ctypes.byref(lay), ptrs, ptrs, ctypes.cast(state, ctypes.c_void_p),
                                     None, ctypes.byref(hp), None)
    assert call(m_f32=4096) == -1 and "10" in ma.adam_last_error()
    assert call(v_f32=4096) == -1
    assert call(options=1, m_f32=4096, v_f32=8192) == -1 and "11" in ma.adam_last_error()
    assert call(m_f32=4096, v_f32=8200) == -3


def test_unknown_storages_stay_refused():
    for storage in (0, 5, -1):
        with pytest.raises(ma.AdamError):
            ma.adam_state_bytes([5], storage)
