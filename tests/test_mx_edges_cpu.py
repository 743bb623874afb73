"""Calls of the microscaled layer at the ends of what they take, without a GPU (the
pointers passed here are never dereferenced)."""
import pytest

import adapter_apply_amd as aa
from tests.test_layer_cpu import needs_no_gpu
from tests.test_mx_cpu import forward


@needs_no_gpu
@pytest.mark.parametrize("kw", [dict(Ws=None), dict(W=None, Ws=None), dict(y=None, x=None, idx=None)], ids=str)
def test_no_tokens_need_no_pointers(kw):
    """As lora_linear: a call of no tokens does nothing, whatever its pointers; its sizes
    are checked all the same."""
    assert forward(T=0, **kw) == aa.LORA_OK
    assert forward(T=0, **dict(kw, ldw=2032)) == aa.LORA_E_SHAPE
    assert forward(T=0, **dict(kw, ldws=130)) == aa.LORA_E_ALIGN
