"""CPU tests: further arguments that the sequence calls refuse before any CUDA call."""
import ctypes
import math

import pytest

import kv_cache_compression_two_b200 as ispa

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
L = ispa.lib()


@pytest.mark.parametrize("scale", [math.nan, math.inf])
def test_a_softmax_scale_that_is_no_number_is_refused(scale):
    a = ispa.attn_seq_desc(2, 8, 2, 128, ispa.ISPA_BF16, ispa.ISPA_BF16, True, scale)
    c = ispa.kvq_desc(2, 128, 16, 8, ispa.ISPA_KVQ_INT8)
    assert L.ispa_attn_prompt_workspace_bytes(ctypes.byref(a)) == 0
    assert L.ispa_attn_kvq_workspace_bytes(ctypes.byref(a), ctypes.byref(c)) == 0
    assert L.ispa_attn_prompt(ctypes.byref(a), 4, 4, FAKE, FAKE, FAKE, 1024, FAKE, 256, FAKE, 256, FAKE, FAKE, FAKE, 1 << 40,
                              None) == ispa.ISPA_ERR_INVALID_ARG
    assert L.ispa_attn_kvq(ctypes.byref(a), ctypes.byref(c), 4, FAKE, FAKE, 3, FAKE, FAKE, 1024, FAKE, FAKE, FAKE, FAKE,
                           1 << 40, None) == ispa.ISPA_ERR_INVALID_ARG
    assert "softmax_scale" in L.ispa_last_error().decode()
