"""Microscaled storage at the ends of what it takes."""
import pytest
import torch

import adapter_apply_amd as aa
from tests import mx_util
from tests.test_gpu_mx import FILL, FMTS, bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
def test_store_of_the_longest_row(fmt):
    """A row of the most values a call takes: its end is stored and restored as its start."""
    K = 2 ** 31 - 8
    per = 16 if fmt == aa.LORA_MX_FP4 else 32              # code bytes of a block
    g = torch.Generator().manual_seed(9)
    parts = [(at, torch.randn((1, n), generator=g).to(bf16)) for at, n in ((0, 256), (2 ** 31 - 256, 248))]
    x = torch.zeros((1, K), dtype=bf16, device="cuda")
    for at, v in parts:
        x[:, at:at + v.shape[1]] = v
    codes, scales = aa.alloc_mx(1, K, fmt)
    codes.fill_(0xA5)
    scales.fill_(0xA5)
    aa.lora_mx_quantize(codes, scales, x, fmt)
    x.fill_(FILL)
    aa.lora_mx_dequantize(x, codes, scales, fmt)
    for at, v in parts:
        c, s = mx_util.quantize(v, fmt)
        assert torch.equal(scales[:, at // 32:at // 32 + s.shape[1]].cpu(), s), at
        assert torch.equal(codes[:, at // 32 * per:at // 32 * per + c.shape[1]].cpu(), c), at
        want = mx_util.restore(c, s, v.shape[1], fmt)
        assert torch.equal(x[:, at:at + v.shape[1]].cpu().double(), want), at
    end = parts[1][0]
    assert not bool(codes[:, 8 * per:end // 32 * per].any()) and not bool(scales[:, 8:end // 32].any())
    assert not bool(x[:, 256:end].any())
