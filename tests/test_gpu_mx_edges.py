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
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 180 << 30:
        pytest.skip("needs 175 GB")
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


# The forms of a few tokens and one, the tiles with and without a join, restored projections.
EDGE_SHAPES = [
    (1, 4104, (8200,), 16, 2, 0), (1, 72, (36, 20), 32, 3, 4), (1, 136, (16388,), 8, 2, 0),
    (7, 4104, (8200,), 16, 3, 4), (16, 1416, (260,), 16, 16, 0), (20, 4104, (8200,), 8, 3, 0),
    (32, 1032, (2600,), 8, 9, 4), (33, 8256, (1100, 36), 48, 5, 0), (256, 520, (260, 132), 16, 4, 4),
    (777, 1352, (1100, 36, 516), 24, 5, 0), (1200, 2048, (260,), 16, 3, 4), (2100, 1032, (5000, 260), 16, 4, 0),
    (2100, 5640, (100, 36), 72, 12, 4),
]


@pytest.mark.parametrize("shape", EDGE_SHAPES, ids=str)
def test_scale_255_stays_in_its_block(shape):
    """NaN blocks in the middle of a row and at the end of the last one, of W and of x:
    only their own outputs are NaN."""
    c = layer(shape, 41, x8=True, ragged=False)
    T, K, n, last = c.T, c.K, sum(c.N), mx_util.blocks(c.K) - 1
    c.idx[0] = c.idx[T // 2] = 0
    c.rank[:] = c.R
    buf = c.forward()[2].float()
    w_bad = [(n // 2, last // 2), (n - 1, last)]
    x_bad = [(0, last // 3), (T // 2, last)]
    for i, b in w_bad:
        c.Ws[i, b] = 255
    for t, b in x_bad:
        c.xs[t, b] = 255
    _, y, _ = run_forward(c, want_buf=False)
    want = torch.zeros((T, n), dtype=torch.bool, device="cuda")
    want[:, [i for i, _ in w_bad]] = True
    assert torch.equal(y.isnan(), want) and bool(torch.isfinite(y[~want]).all())
    dx = torch.full((T, K), FILL, dtype=bf16, device="cuda")
    dA, dB = gradients(c)
    call_backward(c, dx, dA, dB, buf=buf)
    want = torch.zeros((T, K), dtype=torch.bool, device="cuda")
    for _, b in w_bad:
        want[:, 32 * b:32 * b + 32] = True
    assert torch.equal(dx.isnan(), want) and bool(torch.isfinite(dx[~want]).all())
    want = torch.zeros((c.L, c.R, K), dtype=torch.bool, device="cuda")
    for _, b in x_bad:
        want[0, :, 32 * b:32 * b + 32] = True
    for t in dA:
        assert torch.equal(t.isnan(), want) and bool(torch.isfinite(t[~want]).all())
    assert all(bool(torch.isfinite(t).all()) for t in dB)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("shape", EDGE_SHAPES, ids=str)
def test_bad_adapter_stays_with_its_tokens(shape, bad):
    """A slot of infinities or NaN: tokens and gradients of all others keep their bits."""
    c = layer(shape, 43, x8=True, ragged=False)
    c.rank[:] = c.R
    c.idx[c.T // 2:] = torch.arange(c.T - c.T // 2, dtype=torch.int32, device="cuda") % (c.L + 1) - 1
    c.idx[0] = 0 if c.T > 1 else 1
    buf = c.forward()[2].float()
    ws = workspace(c)

    def step():
        _, y, u = run_forward(c, ws=ws)
        dx = torch.full((c.T, c.K), FILL, dtype=bf16, device="cuda")
        dA, dB = gradients(c)
        call_backward(c, dx, dA, dB, buf=buf, ws=ws)
        return y, u, dx, dA, dB

    y0, u0, dx0, dA0, dB0 = step()
    for t in (*c.A, *c.B):
        t[0] = bad
    y, u, dx, dA, dB = step()
    mine = c.idx != 0
    assert torch.equal(y[mine], y0[mine]) and torch.equal(u[:, mine], u0[:, mine]) and torch.equal(dx[mine], dx0[mine])
    for got, want in zip(dA + dB, dA0 + dB0):
        assert torch.equal(got[1:], want[1:])


@pytest.mark.parametrize("T,K,n", [(1, 1 << 21, 4200), (5, 1 << 21, 4200), (40, 1 << 21, 4200), (100, 40960, 212000)])
def test_codes_past_4_gb(T, K, n):
    """Rows and blocks at both ends of a projection of more bytes than 32 bits count, the
    rest of it zeros: y of one, a few and more tokens; dx of many rows alone, and with dA
    and dB."""
    R, g = 8, torch.Generator(device="cuda").manual_seed(6)
    rows = torch.tensor([0, 1, n // 2, n - 1], device="cuda")
    cols = torch.cat([torch.arange(32) + 32 * b for b in (0, K // 64, K // 32 - 1)]).cuda()
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").to(bf16)
    full = torch.zeros((len(rows), K), device="cuda")
    full[:, cols] = torch.randn((len(rows), len(cols)), generator=g, device="cuda")
    part = [aa.alloc_mx(len(rows), K, aa.LORA_MX_FP4), torch.empty_like(full)]
    aa.lora_mx_quantize(*part[0], full, aa.LORA_MX_FP4)
    aa.lora_mx_dequantize(part[1], *part[0], aa.LORA_MX_FP4)
    w = part[1][:, cols].double()
    W = torch.zeros((n, K // 2), dtype=torch.uint8, device="cuda")
    Ws = torch.full((n, K // 32), 127, dtype=torch.uint8, device="cuda")
    W[rows], Ws[rows] = part[0]
    x, dy = randn(T, K), randn(T, n)
    A, B = torch.zeros((1, R, K), dtype=bf16, device="cuda"), torch.zeros((1, n, R), dtype=bf16, device="cuda")
    A[:, :, cols], B[:, rows] = randn(1, R, len(cols)), randn(1, len(rows), R)
    a, b = A[0][:, cols].double(), B[0][rows].double()
    idx = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    idx[0] = 0
    one, ws = torch.ones(1, device="cuda"), aa.alloc_linear_mx_workspace(T, K, [n], R, 1)
    mine = (idx == 0).double()[:, None]

    def check(got, at, base, mags, u, v, other):
        # sums of the values that are not zero, at most 104 each and 16 splits of them; the
        # rank vector as two bf16 parts; one rounding of the result
        ref = base + mine * (u @ other)
        tol = ref.abs() * 2.0 ** -8 + 256 * 2.0 ** -23 * (mags + mine * (v @ other.abs())) + 2.0 ** -16 * mine * (v @ other.abs())
        assert bool(((got[:, at].double() - ref).abs() <= 1.01 * tol).all())
        assert int((got != 0).sum()) <= T * len(at)          # (every other one is a sum of zeros)

    xs, ds = x[:, cols].double(), dy[:, rows].double()
    y = torch.full((T, n), FILL, dtype=bf16, device="cuda")
    aa.lora_linear_mx(y, x, W, Ws, [A], [B], idx, None, one, ws)
    check(y, rows, xs @ w.T, xs.abs() @ w.abs().T, xs @ a.T, xs.abs() @ a.abs().T, b.T)
    if n < K:
        return
    for weights in (False, True):
        dx = torch.full((T, K), FILL, dtype=bf16, device="cuda")
        dA, dB = [torch.empty((1, R, K), device="cuda")], [torch.empty((1, n, R), device="cuda")]
        aa.lora_linear_mx_backward(dx, dA if weights else None, dB if weights else None, dy, x, W, [A], [B], idx, None,
                                   one, ws, W_scales=Ws)
        check(dx, cols, ds @ w, ds.abs() @ w.abs(), ds @ b, ds.abs() @ b.abs(), a)
