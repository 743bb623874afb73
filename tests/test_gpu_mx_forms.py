"""Forms of the layer on a 4-bit projection that the shapes of tests/test_gpu_mx.py do not
reach (tests/test_mx_rules_cpu.py asks the library's rules that both together reach all),
against the 64-bit definitions."""
import pytest
import torch

import adapter_apply_amd as aa
from tests.layer_util import within
from tests.test_gpu_mx import FILL, bf16, call_backward, check_backward, gradients, layer, run_forward, workspace

pytestmark = pytest.mark.gpu

# T, K, N, R, L, extra columns
FORMS = [
    (1, 4248, (16, 3784, 9348), 16, 8, 4),
    (1, 9624, (4,), 24, 2, 0),
    (5, 11296, (4244, 32, 912), 8, 7, 4),
    (16, 8528, (4, 36), 8, 3, 0),
    (32, 5816, (244,), 8, 1, 4),
    (32, 15272, (200,), 8, 1, 0),
    (320, 8176, (12,), 8, 3, 4),
    (458, 4176, (1128,), 40, 2, 8),
    (463, 1584, (88, 4696), 16, 193, 8),
    (548, 384, (4648, 352, 4), 8, 254, 4),
    (794, 8, (4216,), 8, 2, 8),
    (874, 5056, (780, 336), 32, 22, 4),
    (905, 7904, (16, 268), 40, 2, 4),
    (2101, 352, (8,), 8, 1, 0),
    (2766, 1064, (4,), 128, 2, 4),
    (3146, 208, (44, 976, 380), 32, 3, 4),
    (3220, 1096, (556, 24, 16), 16, 1, 4),
    (3903, 1144, (76, 292, 120), 128, 2, 4),
]


@pytest.mark.parametrize("shape", FORMS, ids=str)
def test_forward_and_backward(shape):
    """y and u; dx, dA and dB of 8-bit activations; dx alone."""
    c = layer(shape, sum(shape[2]) + shape[0], x8=True, bias=shape[0] % 2 == 0, runs=shape[0] > 1000)
    y_ref, y_tol, b_ref, b_tol = c.forward()
    ws = workspace(c)
    full, y, buf = run_forward(c, ws=ws)
    within(y, y_ref, y_tol, "y")
    within(buf, b_ref, b_tol, "buf")
    assert bool((full[:, sum(c.N):] == FILL).all()), "columns past the slices were written"
    dx = torch.full((c.T, c.K), FILL, dtype=bf16, device="cuda")
    dA, dB = gradients(c)
    call_backward(c, dx, dA, dB, buf=buf, ws=ws)
    check_backward(c, buf, dx, dA, dB)
    dx.fill_(FILL)
    aa.lora_linear_mx_backward(dx, None, None, c.dy, None, c.Wq, c.A, c.B, c.idx, c.rank, c.scale, ws, W_scales=c.Ws)
    check_backward(c, buf, dx, None, None)
