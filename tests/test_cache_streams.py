"""The serving-cache calls refuse a stream of another device before anything is called."""
import types

import pytest
import torch

import exact_tiled_attention_21_gb300 as fa


def test_a_stream_of_another_device_is_refused():
    x = types.SimpleNamespace(device=torch.device("cuda", 0))
    there = types.SimpleNamespace(cuda_stream=5, device=torch.device("cuda", 1))
    for call in (lambda: fa.rope(x, None, stream=there),
                 lambda: fa.cache_append_fp8(x, x, None, None, None, None, None, None, stream=there),
                 lambda: fa.decode_paged_fp8(x, None, None, None, None, None, None, stream=there),
                 lambda: fa.cache_evict_fp8(x, None, None, None, None, None, None, None, 1, stream=there)):
        with pytest.raises(ValueError, match="another device"):
            call()
