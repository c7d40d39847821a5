"""CPU checks: every call of the binding refuses a pool that is not
(2, blocks, block size, kv heads, head size) by itself, before it looks for a
device or the library. A pool of K alone would have V read and written behind
its end."""
import pytest
import torch

from paged_kv_cache_120_gb300 import binding

H, I, F8 = torch.float16, torch.int32, torch.uint8
BAD = {"keys alone": (1, 4, 16, 2, 64), "three": (3, 4, 16, 2, 64), "no K and V": (4, 16, 2, 64), "flat": (2, 64, 2, 64),
       "layers": (2, 2, 4, 16, 2, 64)}


def calls(pool, codes):
    q, kv, i = torch.zeros(4, 8, 64, dtype=H), torch.zeros(4, 2, 64, dtype=H), torch.zeros(4, dtype=I)
    bt, cu, ws = torch.zeros(4, 2, dtype=I), torch.zeros(5, dtype=I), torch.zeros(256, dtype=F8)
    plan, b = torch.zeros(32, dtype=torch.int64), binding
    return {
        "reshape_and_cache": lambda: b.pa_reshape_and_cache(kv, kv, pool, i),
        "reshape_and_cache_fp8": lambda: b.pa_reshape_and_cache_fp8(kv, kv, codes, i, 1.0, 1.0),
        "decode_workspace": lambda: b.decode_workspace(q, pool),
        "decode_fp8_workspace": lambda: b.decode_fp8_workspace(q, codes),
        "decode": lambda: b.pa_decode(q, q, pool, bt, i, 0.1, ws),
        "decode_static_scratch": lambda: b.pa_decode_static_scratch(q, q, pool, bt, i, 0.1),
        "decode_fp8": lambda: b.pa_decode_fp8(q, q, codes, bt, i, 0.1, 1.0, 1.0, ws),
        "prefill_workspace": lambda: b.prefill_workspace(q, pool, 4, 1),
        "prefill": lambda: b.pa_prefill(q, q, pool, bt, cu, i, 0.1, 1),
        "prefill_fp8": lambda: b.pa_prefill_fp8(q, q, codes, bt, cu, i, 0.1, 1, 1.0, 1.0),
        "rope_and_cache": lambda: b.pa_rope_and_cache(q, q, kv, kv, pool, i, i, plan),
        "rope_and_cache_fp8": lambda: b.pa_rope_and_cache_fp8(q, q, kv, kv, codes, i, i, plan, 1.0, 1.0),
        "cross_attention_workspace": lambda: b.cross_attention_workspace(q, pool, 4, 1),
        "cross_attention": lambda: b.pa_cross_attention(q, q, pool, bt, cu, i, 0.1, 1),
        "cross_attention_fp8": lambda: b.pa_cross_attention_fp8(q, q, codes, bt, cu, i, 0.1, 1, 1.0, 1.0),
        "copy_blocks": lambda: b.pa_copy_blocks([pool, pool], torch.zeros(1, 2, dtype=I)),
    }


@pytest.mark.parametrize("call", list(calls(None, None)))
@pytest.mark.parametrize("shape", list(BAD.values()), ids=list(BAD))
def test_pools_of_another_shape_are_refused(call, shape):
    with pytest.raises(binding.PAError) as e:
        calls(torch.zeros(shape, dtype=H), torch.zeros(shape, dtype=F8))[call]()
    assert e.value.code == binding.PA_ERR_INVALID_ARG and "kv_cache" in str(e.value)


def test_copy_blocks_refuses_pools_that_differ():
    a = torch.zeros(2, 4, 16, 2, 64, dtype=H)
    for other in (torch.zeros(2, 3, 16, 2, 64, dtype=H), torch.zeros(2, 4, 16, 2, 64, dtype=torch.bfloat16), a[:1]):
        with pytest.raises(binding.PAError) as e:
            binding.pa_copy_blocks([a, other], torch.zeros(1, 2, dtype=I))
        assert e.value.code == binding.PA_ERR_INVALID_ARG
