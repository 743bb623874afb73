"""Microscaled storage and the layer on it at the ends of what they take."""
import pytest
import torch

import adapter_apply_amd as aa
from tests import mx_util
from tests.layer_util import within
from tests.test_gpu_mx import (FILL, FMTS, bf16, call_backward, check_backward, gradients, layer, run_forward,
                               workspace)

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


def test_gradient_through_a_projection_of_2_36_values():
    """One that is restored (128 GB of bf16): the tokens' dx are the sums of the rows that
    are not zero."""
    T, K, n, R = 8, 1 << 16, 1 << 20, 8
    if torch.cuda.mem_get_info()[1] < 200 << 30:                    # (the whole card's)
        pytest.skip("needs 180 GB")
    torch.cuda.empty_cache()
    g = torch.Generator().manual_seed(4)
    rows = torch.tensor([0, 1, 63, 64, 1 << 17, (1 << 18) - 1, 1 << 18, (1 << 19) + 5, n - 65, n - 1])
    code, scale = mx_util.quantize(torch.randn((len(rows), K), generator=g), aa.LORA_MX_FP4)
    w = mx_util.restore(code, scale, K, aa.LORA_MX_FP4)
    W = torch.zeros((n, K // 2), dtype=torch.uint8, device="cuda")
    Ws = torch.full((n, K // 32), 127, dtype=torch.uint8, device="cuda")
    W[rows.cuda()], Ws[rows.cuda()] = code.cuda(), scale.cuda()
    dy = torch.randn((T, n), generator=g).to(bf16)
    A, B = torch.zeros((1, R, K), dtype=bf16, device="cuda"), torch.zeros((1, n, R), dtype=bf16, device="cuda")
    x = torch.zeros((T, K), dtype=bf16, device="cuda")
    dA, dB = torch.full((1, R, K), FILL, device="cuda"), torch.full((1, n, R), FILL, device="cuda")
    dx = torch.full((T, K), FILL, dtype=bf16, device="cuda")
    ws = aa.alloc_linear_mx_workspace(T, K, [n], R, 1)
    aa.lora_linear_mx_backward(dx, [dA], [dB], dy.cuda(), x, W, [A], [B],
                               torch.full((T,), -1, dtype=torch.int32, device="cuda"), None,
                               torch.ones(1, device="cuda"), ws, W_scales=Ws)
    d = dy[:, rows].double()
    # 10 products (the others are zeros), each sum within 2^-23; one bf16 rounding
    tol = (d @ w).abs() * 2.0 ** -8 + 1.01 * 10 * 2.0 ** -23 * (d.abs() @ w.abs())
    assert bool(((dx.cpu().double() - d @ w).abs() <= tol).all())
    assert not bool(dA.any()) and not bool(dB.any())
    del ws, W
    torch.cuda.empty_cache()


def test_dx_alone_of_no_tokens():
    """With a bf16 and with a 4-bit projection."""
    c = layer((3, 72, (36,), 24, 3, 0), 1)
    e = lambda *s: torch.empty(s, dtype=bf16, device="cuda")
    args = (e(0, 72), None, None, e(0, 36), None)
    aa.lora_linear_backward(*args, c.W, c.A, c.B, c.idx[:0], c.rank, c.scale, workspace(c))
    aa.lora_linear_mx_backward(*args, c.Wq, c.A, c.B, c.idx[:0], c.rank, c.scale, workspace(c), W_scales=c.Ws)


@pytest.mark.parametrize("shape", [(2100, 5640, (100, 36), 72, 12, 4), (1, 4104, (8200,), 16, 2, 0),
                                   (20, 4104, (8200,), 8, 3, 0), (777, 1352, (1100, 36, 516), 24, 5, 0),
                                   (2100, 1032, (5000, 260), 16, 4, 0)], ids=str)
def test_workspaces_of_exactly_the_size(shape):
    """Calls on a workspace of the size that they need, the bytes around it left alone:
    forward and the weights' gradients without room for a bf16 projection, then all."""
    c = layer(shape, 47, x8=True)
    y_ref, y_tol, b_ref, b_tol = c.forward()
    args = (c.T, c.K, c.N, c.R, c.L)
    for size, with_dx in ((aa.lora_linear_mx_forward_workspace_size(*args), False),
                          (aa.lora_linear_mx_workspace_size(*args), True)):
        around = torch.full((size + 8192 + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        at = 4096 + (-around.data_ptr()) % 256
        ws = around[at:at + size]
        aa.lora_workspace_init(ws)
        for _ in range(2):
            _, y, buf = run_forward(c, ws=ws)
            within(y, y_ref, y_tol, "y")
            within(buf, b_ref, b_tol, "buf")
            dx = torch.empty((c.T, c.K), dtype=bf16, device="cuda") if with_dx else None
            dA, dB = gradients(c)
            call_backward(c, dx, dA, dB, buf=buf, W=with_dx, ws=ws)
            check_backward(c, buf, dx, dA, dB)
        assert bool((around[:at] == 0xA5).all()) and bool((around[at + size:] == 0xA5).all())
