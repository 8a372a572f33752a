"""The stream probe's storages are the step's without fp32 moments: those are refused by every call, not
answered with 0 bytes."""
import pytest

from memory_efficient_adam_amd import stream_probe as sp


@pytest.mark.parametrize("call", [sp.adam_stream_probe_bytes, sp.probe_buffers_shape, sp.probe_buffers])
def test_fp32_moments_are_refused(call):
    with pytest.raises(KeyError):
        call(4, "f32", "f32")


def test_the_others_have_bytes():
    for storage in ("bf16", "q8", "q8_v_only"):
        assert sp.adam_stream_probe_bytes(4, "f32", storage) > 0
