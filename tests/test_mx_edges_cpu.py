"""Calls of the layer and the microscaled one at the ends of what they take, without a GPU (the
pointers passed here are never dereferenced)."""
import pytest

import adapter_apply_amd as aa
from tests import test_layer_cpu
from tests.test_layer_cpu import needs_no_gpu
from tests.test_mx_cpu import backward, forward


@needs_no_gpu
@pytest.mark.parametrize("kw", [dict(Ws=None), dict(W=None, Ws=None), dict(y=None, x=None, idx=None)], ids=str)
def test_no_tokens_need_no_pointers(kw):
    """As lora_linear: a call of no tokens does nothing, whatever its pointers; its sizes
    are checked all the same."""
    assert forward(T=0, **kw) == aa.LORA_OK
    assert forward(T=0, **dict(kw, ldw=2032)) == aa.LORA_E_SHAPE
    assert forward(T=0, **dict(kw, ldws=130)) == aa.LORA_E_ALIGN


@needs_no_gpu
@pytest.mark.parametrize("call", [test_layer_cpu.backward, backward], ids=["bf16", "mx"])
def test_dx_alone_of_no_tokens(call):
    """An empty dx has no address: nothing to do, but of one token it is missing."""
    assert call(T=0, dx=None, dA=None, dB=None) == aa.LORA_OK
    assert call(T=1, dx=None, dA=None, dB=None) == aa.LORA_E_NULL
