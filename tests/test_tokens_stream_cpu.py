"""The binding's check of streams (CPU): a stream of another GPU would run kernels there on this one's memory."""
import types

import pytest

import expert_offload_lru_amd as moe
from expert_offload_lru_amd import tokens


def test_a_stream_of_another_gpu_is_refused():
    def never(*args):
        raise AssertionError("called")

    with pytest.raises(moe.MoeError) as e:
        tokens._call(never, (), 0, types.SimpleNamespace(device_index=1, cuda_stream=1))
    assert e.value.code == moe.ERR_INVALID and "GPU 1" in str(e.value)
