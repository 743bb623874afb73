"""Calls of the layer and the microscaled one at the ends of what they take, without a GPU (the
pointers passed here are never dereferenced)."""
import random

import pytest

import adapter_apply_amd as aa
from tests import test_layer_cpu
from tests.test_layer_cpu import i64, needs_no_gpu, ptrs
from tests.test_mx_cpu import FAKE, backward, forward


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


LONG = dict(T=8192, N=i64(14336, 14336), S=2, L=16, R=64, y=FAKE, ldy=28672, A=ptrs(2), B=ptrs(2),
            dA=ptrs(2, FAKE + (1 << 33)), dB=ptrs(2, FAKE + (1 << 34)), buf=FAKE)


@needs_no_gpu
def test_calls_need_the_workspace_that_they_use():
    """A bf16 copy of the projection is dx's of long batches alone: prompts forward, and
    gradients without dx or through bf16, do with less.  (Without a GPU, a call that passes
    its checks ends at its first launch.)"""
    args = (8192, 4096, (14336, 14336), 64, 16)
    small, full = aa.lora_linear_mx_forward_workspace_size(*args), aa.lora_linear_mx_workspace_size(*args)
    assert small == aa.lora_linear_workspace_size(*args) and full == small + 2 * 28672 * 4096
    for call, kw in ((forward, {}), (backward, dict(dx=None)), (backward, dict(dx=None, W=None, Ws=None)),
                     (backward, dict(Ws=None, ldw=4096)), (backward, dict(W=None, Ws=None))):
        a = dict(LONG, **kw)
        assert call(**a, wsb=small) == aa.LORA_E_LAUNCH, kw
        assert call(**a, wsb=small - 256) == aa.LORA_E_WORKSPACE, kw
    assert backward(**LONG, wsb=full) == aa.LORA_E_LAUNCH
    assert backward(**LONG, wsb=full - 256) == aa.LORA_E_WORKSPACE
    assert backward(**dict(LONG, dA=None, dB=None), wsb=full - 256) == aa.LORA_E_WORKSPACE
    # a wide gradient reads the codes
    one = dict(LONG, T=1, K=1 << 16, ldx=1 << 16, lddx=1 << 16, N=i64(64), S=1, ldy=64, ldw=1 << 15, ldws=1 << 11, R=8, L=4,
               A=ptrs(1), B=ptrs(1), dA=None, dB=None)
    assert backward(**one, wsb=aa.lora_linear_mx_forward_workspace_size(1, 1 << 16, [64], 8, 4)) == aa.LORA_E_LAUNCH


def test_workspace_sizes():
    """The bf16 copy is all that the two sizes differ by, and both grow with the tokens (a
    workspace for at most T tokens is one for fewer)."""
    rng = random.Random(23)
    pick = lambda lo, hi: int(2 ** rng.uniform(lo, hi))
    copies = 0
    for _ in range(3000):
        K, N = 8 * pick(0, 13), tuple(4 * pick(0, 12.8) for _ in range(rng.choice((1, 1, 2, 3, 8))))
        R, L = 8 * rng.choice((1, 2, 3, 4, 8, 16, 64)), pick(0, 10)
        before = (0, 0)
        for T in sorted({pick(0, 14) for _ in range(4)}):
            small = aa.lora_linear_mx_forward_workspace_size(T, K, N, R, L)
            full = aa.lora_linear_mx_workspace_size(T, K, N, R, L)
            copy = (2 * sum(N) * K + 255) // 256 * 256
            assert full - small in (0, copy) and small >= aa.lora_linear_workspace_size(T, K, N, R, L)
            assert small >= before[0] and full >= before[1], (T, K, N, R, L)
            before = small, full
            copies += full > small
    assert copies > 100
    with pytest.raises(aa.LoraError):
        aa.lora_linear_mx_forward_workspace_size(-1, 4096, [4096], 16, 8)
    assert aa.lib().lora_linear_mx_forward_workspace_size(1, 64, None, 1, 8, 1, None) == aa.LORA_E_NULL
