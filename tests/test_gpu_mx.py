"""Microscaled storage against its 64-bit definition, bit for bit, and the layer
and its gradient on a 4-bit projection and from 8-bit activations against the
64-bit definitions of the values that the codes stand for."""
import pytest
import torch

import adapter_apply_amd as aa
from tests import mx_util
from tests.layer_util import within
from tests.mx_util import MxLayer

pytestmark = pytest.mark.gpu

FILL = 7.0
FMTS = [aa.LORA_MX_FP4, aa.LORA_MX_INT8]
DTYPES = [torch.bfloat16, torch.float32]
bf16 = torch.bfloat16


# --------------------------------------------------------------------------
# storage
# --------------------------------------------------------------------------

def canvas(M, K, dtype, pad):
    """An [M, K] window of a wider, filled tensor, and the whole."""
    full = torch.full((M + 2, K + pad), FILL, dtype=dtype, device="cuda")
    return full[1:M + 1, :K], full


def mx_canvas(M, K, fmt, pad=32):
    cs, ss = aa._mx_shapes(M, K, fmt)
    c = torch.full((M + 2, cs[1] + pad), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((M + 2, ss[1] + pad), 0xA5, dtype=torch.uint8, device="cuda")
    return c[1:M + 1, :cs[1]], s[1:M + 1, :ss[1]], c, s


def untouched(full, M, cols, fill):
    return bool((full[0] == fill).all()) and bool((full[M + 1:] == fill).all()) and bool((full[:, cols:] == fill).all())


def check_store(x, fmt, pad=8):
    """Quantise and restore x (on the CPU); codes, scales and values bit for bit."""
    M, K = x.shape
    xin, _ = canvas(M, K, x.dtype, pad)
    xin.copy_(x)
    c, s, cf, sf = mx_canvas(M, K, fmt)
    aa.lora_mx_quantize(c, s, xin, fmt)
    want_c, want_s = mx_util.quantize(x, fmt)
    assert torch.equal(s.cpu(), want_s)
    assert torch.equal(c.cpu(), want_c)
    assert untouched(cf, M, c.shape[1], 0xA5) and untouched(sf, M, s.shape[1], 0xA5)
    for dt in DTYPES:
        out, full = canvas(M, K, dt, pad)
        aa.lora_mx_dequantize(out, c, s, fmt)
        want = mx_util.restore(want_c, want_s, K, fmt)
        got = out.cpu().double()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0)), dt
        assert untouched(full, M, K, FILL)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K", [(1, 8), (1, 32), (3, 40), (17, 128), (5, 136), (64, 1352), (130, 256), (33, 4096)])
def test_store(M, K, fmt, dtype):
    g = torch.Generator().manual_seed(M + K)
    x = torch.randn((M, K), generator=g) * torch.exp(4 * torch.randn((M, 1), generator=g))
    check_store(x.to(dtype), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_store_ties_and_powers(fmt):
    """Every multiple of a 256th up to a block's largest, at scales over all of
    bf16's and fp32's exponents, subnormals among them."""
    v = torch.arange(-2047, 2048, dtype=torch.float64)[:, None] / 1024        # |v| < 2
    for power in (0, -20, 40, 126, -125, -126, -130, -133, -140, -149):
        x = torch.zeros((v.shape[0], 32), dtype=torch.float64)
        x[:, 5:6] = v
        x[:, 6] = 1.9990234375
        x[::2, 6] = -1.0                                   # the element may be the block's largest
        check_store(torch.ldexp(x, torch.tensor(power)).to(torch.float32), fmt)
        check_store(torch.ldexp(x, torch.tensor(power)).to(bf16), fmt)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("fmt", FMTS)
def test_store_zeros_infinities_and_nan(fmt, dtype):
    g = torch.Generator().manual_seed(3)
    x = torch.randn((40, 200), generator=g)
    x[0] = 0
    x[1, 40], x[2, 199], x[3, 0], x[4, 33] = float("inf"), float("nan"), -float("inf"), -float("nan")
    x[5, 64:96] = 0
    x[6, 64:96] = -0.0
    x[7, 100] = torch.finfo(dtype).max
    x[8] = torch.finfo(dtype).min
    x[9, 32:64] = torch.finfo(dtype).tiny
    check_store(x.to(dtype), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_restore_every_code_and_scale(fmt):
    """All scale bytes against all code bytes; what passes a type's largest is
    infinite in fp32 and bf16 alike."""
    n = 16 if fmt == aa.LORA_MX_FP4 else 32
    codes = torch.arange(256, dtype=torch.uint8).reshape(256 // n, n).repeat(256, 1)
    scales = torch.zeros((codes.shape[0], 4), dtype=torch.uint8)
    scales[:, 0] = torch.arange(256).repeat_interleave(256 // n).to(torch.uint8)
    want = mx_util.restore(codes, scales, 32, fmt)
    for dt in DTYPES:
        out = torch.empty(want.shape, dtype=dt, device="cuda")
        aa.lora_mx_dequantize(out, codes.cuda(), scales.cuda(), fmt)
        assert torch.equal(out.cpu().isnan(), want.isnan())
        assert torch.equal(out.cpu().double().nan_to_num(nan=0.0, posinf=1e300, neginf=-1e300),
                           want.to(dt).double().nan_to_num(nan=0.0, posinf=1e300, neginf=-1e300))


@pytest.mark.parametrize("fmt", FMTS)
def test_store_rows_past_4_gb(fmt):
    """Byte offsets past 32 bits in the input, the codes and the output."""
    M, ld = 9, 1 << 29                                     # rows of 1 GB of bf16
    g = torch.Generator().manual_seed(5)
    x = torch.randn((M, 264), generator=g).to(bf16)
    xin = torch.empty((M * ld,), dtype=bf16, device="cuda").as_strided((M, 264), (ld, 1))
    xin.copy_(x)
    cs, ss = aa._mx_shapes(M, 264, fmt)
    codes = torch.empty((M * ld,), dtype=torch.uint8, device="cuda").as_strided(cs, (ld, 1))
    scales = torch.empty((M * ld,), dtype=torch.uint8, device="cuda").as_strided(ss, (ld, 1))
    aa.lora_mx_quantize(codes, scales, xin, fmt)
    want_c, want_s = mx_util.quantize(x, fmt)
    assert torch.equal(codes.cpu(), want_c) and torch.equal(scales.cpu(), want_s)
    xin.zero_()
    aa.lora_mx_dequantize(xin, codes, scales, fmt)
    assert torch.equal(xin.cpu().double(), mx_util.restore(want_c, want_s, 264, fmt))


def test_store_of_no_rows():
    c, s = aa.alloc_mx(0, 64, aa.LORA_MX_FP4)
    x = torch.empty((0, 64), dtype=bf16, device="cuda")
    aa.lora_mx_quantize(c, s, x, aa.LORA_MX_FP4)
    aa.lora_mx_dequantize(x, c, s, aa.LORA_MX_FP4)


# --------------------------------------------------------------------------
# the layer
# --------------------------------------------------------------------------

# T, K, N, R, L, extra columns
SHAPES = [
    (1, 8, (4,), 8, 1, 0),
    (1, 648, (72, 20), 16, 3, 0),
    (1, 4096, (512, 128, 128), 16, 8, 0),
    (1, 4104, (68, 4), 16, 2, 4),
    (1, 72, (36, 20), 32, 3, 4),
    (1, 64, (16400,), 16, 2, 0),
    (1, 640, (100,), 40, 2, 0),
    (2, 136, (40,), 8, 4, 0),
    (5, 2120, (100, 36), 16, 3, 4),
    (2, 24, (32800, 4), 8, 3, 0),
    (3, 72, (36,), 24, 3, 0),
    (16, 64, (64, 64), 16, 4, 8),
    (16, 1416, (260,), 16, 16, 0),
    (17, 136, (100, 36, 4), 40, 5, 4),
    (64, 256, (264,), 64, 130, 8),
    (12, 4096, (14336,), 32, 6, 4),
    (33, 8256, (1100, 36), 48, 5, 0),
    (65, 8200, (68,), 16, 5, 0),
    (70, 1032, (100, 360, 4), 40, 7, 4),
    (100, 512, (64, 100), 32, 7, 4),
    (128, 4096, (64, 1000), 64, 24, 8),
    (200, 520, (68, 132), 8, 9, 4),
    (256, 128, (128,), 128, 40, 0),
    (257, 128, (128, 8), 16, 3, 8),
    (300, 72, (260,), 512, 6, 4),
    (700, 64, (72,), 16, 64, 0),
    (777, 1352, (1100, 36, 516), 24, 5, 0),
    (1000, 136, (3200,), 32, 20, 8),
    (1000, 3208, (132, 60), 48, 20, 4),
    (1024, 392, (72,), 8, 40, 0),
    (1200, 2048, (260,), 16, 3, 4),
    (1500, 128, (72, 20), 24, 1024, 0),
    (2100, 136, (5000, 700), 64, 300, 0),
    (2100, 1032, (5000, 260), 16, 4, 0),
    (2100, 5640, (100, 36), 72, 12, 4),
    (4500, 64, (60,), 16, 2, 0),
    (9000, 72, (20, 12), 40, 1, 4),
]


# The forms of a few tokens: one and several rounds of K steps a split, more than 8
# splits, one and two blocks of tokens, ranks past one work-group's, rows short of the
# columns' blocks.
FEW_SHAPES = [
    (1, 4104, (8200,), 16, 2, 0),
    (1, 5000, (68, 36), 24, 3, 4),
    (1, 136, (16388,), 8, 2, 0),
    (2, 136, (40,), 80, 4, 0),
    (7, 4104, (8200,), 16, 3, 4),
    (3, 4104, (16004,), 8, 3, 0),
    (9, 5000, (260,), 16, 3, 4),
    (16, 520, (132, 4), 136, 20, 8),
    (17, 520, (4100,), 8, 2, 4),
    (20, 4104, (8200,), 8, 3, 0),
    (32, 5000, (2000, 132), 16, 3, 4),
    (32, 1032, (2600,), 8, 9, 4),
]


def layer(shape, seed, **kw):
    T, K, N, R, L, extra = shape
    return MxLayer(T, K, N, R, L, seed=seed, extra=extra, **kw)


def workspace(c):
    return aa.alloc_linear_mx_workspace(c.T, c.K, c.N, c.R, c.L)


def run_forward(c, want_buf=True, ws=None, stream=None):
    full = torch.full((c.T, c.ldn), FILL, dtype=bf16, device="cuda")
    y = full[:, :sum(c.N)]
    buf = torch.full((c.S, c.T, c.R), FILL, device="cuda") if want_buf else None
    aa.lora_linear_mx(y, c.x, c.Wq, c.Ws, c.A, c.B, c.idx, c.rank, c.scale, ws if ws is not None else workspace(c),
                      bias=c.bias, buf=buf, stream=stream)
    return full, y, buf


def gradients(c):
    return ([torch.full((c.L, c.R, c.K), FILL, device="cuda") for _ in c.N],
            [torch.full((c.L, n, c.R), FILL, device="cuda") for n in c.N])


def call_backward(c, dx, dA, dB, buf=None, W=True, ws=None, flags=0, stream=None):
    aa.lora_linear_mx_backward(dx, dA, dB, c.dy, c.x if c.xq is None else c.xq,
                               (c.W if c.Wq is None else c.Wq) if W else None, c.A, c.B, c.idx, c.rank, c.scale,
                               ws if ws is not None else workspace(c), buf=buf, x_scales=c.xs,
                               W_scales=c.Ws if W else None, flags=flags, stream=stream)


def check_backward(c, buf, dx, dA, dB, with_w=True):
    dx_ref, dx_tol, dA_ref, eA, dB_ref, eB = c.backward(with_w=with_w, buf=buf)
    if dx is not None:
        within(dx, dx_ref, dx_tol, "dx")
    for s in range(c.S):
        if dA is not None:
            within(dA[s], dA_ref[s], eA[s], f"dA[{s}]")
        if dB is not None:
            within(dB[s], dB_ref[s], eB[s], f"dB[{s}]")


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("shape", SHAPES + FEW_SHAPES, ids=str)
def test_forward(shape, bias):
    c = layer(shape, shape[0] + shape[1], bias=bias, runs=bias)
    y_ref, y_tol, b_ref, b_tol = c.forward()
    full, y, buf = run_forward(c, want_buf=not bias or shape[0] % 2 == 0)
    within(y, y_ref, y_tol, "y")
    if buf is not None:
        within(buf, b_ref, b_tol, "buf")
    assert bool((full[:, sum(c.N):] == FILL).all()), "columns past the slices were written"


@pytest.mark.parametrize("w4,x8", [(True, False), (True, True), (False, True)])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, w4, x8):
    T, K = shape[:2]
    c = layer(shape, T + K + 1, runs=x8, w4=w4, x8=x8)
    buf = c.forward()[2].float()
    full = torch.full((T, K + 8), FILL, dtype=bf16, device="cuda")
    dA, dB = gradients(c)
    call_backward(c, full[:, :K], dA, dB, buf=buf)
    check_backward(c, buf, full[:, :K], dA, dB)
    assert bool((full[:, K:] == FILL).all()), "columns past K were written"


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] < 1100], ids=str)
def test_backward_of_x_alone(shape):
    T, K = shape[:2]
    c = layer(shape, T + K + 2)
    full = torch.full((T, K + 8), FILL, dtype=bf16, device="cuda")
    ws = workspace(c)
    for _ in range(2):
        aa.lora_linear_mx_backward(full[:, :K], None, None, c.dy, None, c.Wq, c.A, c.B, c.idx, c.rank, c.scale, ws,
                                   W_scales=c.Ws)
        check_backward(c, None, full[:, :K], None, None)
        assert bool((full[:, K:] == FILL).all()), "columns past K were written"
        full[:, :K] = FILL


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] in (1, 17, 257, 777, 2100, 4500)], ids=str)
def test_weight_gradients_alone(shape):
    """From the checkpoint, without W, into sums of an earlier call; then dA alone."""
    c = layer(shape, 7, x8=True, w4=False)
    buf = c.forward()[2].float()
    ws = workspace(c)
    dA, dB = gradients(c)
    call_backward(c, None, dA, dB, buf=buf, W=False, ws=ws)
    check_backward(c, buf, None, dA, dB)
    call_backward(c, None, dA, dB, buf=buf, W=False, ws=ws, flags=aa.LORA_FLAG_ACCUMULATE)
    # Twice the gradient: each call's own error, and the additions, at most 16 splits
    # onto the old sum: 17 of 2^-24 of partial sums that are at most twice the sum of
    # magnitudes, 2^-18.9 of it, within the 40 * 2^-23 = 2^-17.7 that each bound
    # has beside its own sums' terms.
    _, _, dA_ref, eA, dB_ref, eB = c.backward(buf=buf)
    for s in range(c.S):
        within(dA[s], 2 * dA_ref[s], 2 * eA[s], f"twice dA[{s}]")
        within(dB[s], 2 * dB_ref[s], 2 * eB[s], f"twice dB[{s}]")
    only, _ = gradients(c)
    call_backward(c, None, only, None, W=False, ws=ws)
    check_backward(c, buf, None, only, None)


def test_whole_step():
    """As a training step runs them: the projection to 4 bits, the forward call,
    the activations to 8 bits, the backward call from both, the gradient's norm
    and clip; every product against its definition."""
    T, K, N, R, L = 300, 520, (260, 68), 16, 4
    c = MxLayer(T, K, N, R, L, seed=11, w4=True, x8=True)
    plain = MxLayer(T, K, N, R, L, seed=11, w4=False)         # the same values, not quantised
    Wq, Ws = aa.alloc_mx(sum(N), K, aa.LORA_MX_FP4)
    aa.lora_mx_quantize(Wq, Ws, plain.W, aa.LORA_MX_FP4)
    xq, xs = aa.alloc_mx(T, K, aa.LORA_MX_INT8)
    aa.lora_mx_quantize(xq, xs, plain.x, aa.LORA_MX_INT8)
    assert torch.equal(Wq, c.Wq) and torch.equal(xq, c.xq)
    ws = workspace(c)
    y = torch.empty((T, sum(N)), dtype=bf16, device="cuda")
    buf = torch.empty((2, T, R), device="cuda")
    aa.lora_linear_mx(y, plain.x, Wq, Ws, c.A, c.B, c.idx, c.rank, c.scale, ws, buf=buf)
    x8, c.x = c.x, plain.x
    y_ref, y_tol, b_ref, b_tol = c.forward()
    c.x = x8
    within(y, y_ref, y_tol, "y")
    within(buf, b_ref, b_tol, "buf")
    dx = torch.empty((T, K), dtype=bf16, device="cuda")
    dA, dB = gradients(c)
    aa.lora_linear_mx_backward(dx, dA, dB, c.dy, xq, Wq, c.A, c.B, c.idx, c.rank, c.scale, ws, buf=buf,
                               x_scales=xs, W_scales=Ws)
    check_backward(c, buf, dx, dA, dB)
    grads = dA + dB
    norm = torch.empty(L, device="cuda")
    aa.lora_grad_norm(norm, grads, aa.alloc_grad_workspace(grads))
    want = sum(g.double().reshape(L, -1).square().sum(1) for g in grads).sqrt()
    assert torch.allclose(norm.double(), want, rtol=2.0 ** -23)


def test_gradient_against_differences():
    """dx, dA and dB against central differences of the restored layer's own
    output in 64 bits: the loss is linear in each, so a difference is exact."""
    c = MxLayer(9, 40, (12, 8), 8, 2, seed=5, w4=True, x8=True, ragged=False)
    c.rank[:] = 8
    c.idx[:] = torch.tensor([0, 1, -1, 0, 1, 1, 0, 2, 0], dtype=torch.int32)
    buf = c.forward()[2].float()
    dx = torch.empty((9, 40), dtype=bf16, device="cuda")
    dA, dB = gradients(c)
    call_backward(c, dx, dA, dB, buf=buf)
    _, tol_x, _, tol_a, _, tol_b = c.backward(buf=buf)

    def loss(x, A, B):
        y = x @ c.W.double().T
        for t in range(9):
            i = int(c.idx[t])
            if 0 <= i < 2:
                for s, off, n in c.offsets():
                    y[t, off:off + n] += c.scale[i].double() * (x[t] @ A[s][i].T @ B[s][i].T)
        return (y * c.dy.double()).sum()

    base = [c.x.double(), [a.double() for a in c.A], [b.double() for b in c.B]]
    g = torch.Generator().manual_seed(1)
    for which, got, tol in ((0, dx, tol_x), (1, dA[0], tol_a[0]), (1, dA[1], tol_a[1]), (2, dB[0], tol_b[0]),
                            (2, dB[1], tol_b[1])):
        s = 1 if got is dA[1] or got is dB[1] else 0
        for _ in range(12):
            at = tuple(int(torch.randint(0, n, (1,), generator=g)) for n in got.shape)
            d = []
            for h in (1.0, -1.0):
                args = [base[0].clone(), [a.clone() for a in base[1]], [b.clone() for b in base[2]]]
                (args[0] if which == 0 else args[which][s])[at] += h
                d.append(loss(*args))
            want = (d[0] - d[1]) / 2
            # (u enters dB as fp32: one more rounding)
            slack = float(tol[at]) + 2.0 ** -20 * float(want.abs()) + 1e-9
            assert abs(float(got[at]) - float(want)) <= slack, (which, s, at)


def test_scale_255_stays_in_its_block():
    """NaN blocks of W reach their own outputs (y column, dx columns), those of x
    their own columns of dA, and nothing else."""
    c = MxLayer(40, 200, (68, 60), 16, 3, seed=2, w4=True, x8=True, ragged=False)
    c.Ws[7, 2] = 255
    c.xs[11, 1] = 255
    c.idx[11] = 0
    c.rank[:] = 16
    buf = c.forward()[2].float()
    _, y, _ = run_forward(c, want_buf=False)
    bad = y.isnan()
    assert bool(bad[:, 7].all()) and int(bad.sum()) == 40
    dx = torch.empty((40, 200), dtype=bf16, device="cuda")
    dA, dB = gradients(c)
    call_backward(c, dx, dA, dB, buf=buf)
    bad = dx.isnan()
    assert bool(bad[:, 64:96].all()) and int(bad.sum()) == 40 * 32
    for t in dA:
        bad = t.isnan()
        assert bool(bad[0, :, 32:64].all()) and int(bad.sum()) == 16 * 32
    assert not any(bool(t.isnan().any()) for t in dB)


def test_infinite_x_and_dy_stay_in_their_rows():
    for shape in [(3, 136, (40,), 8, 4, 0), (100, 512, (64, 100), 32, 7, 4), (1200, 2048, (260,), 16, 3, 4)]:
        c = layer(shape, 3)
        c.x[2, 5] = float("inf")
        c.dy[1, 3] = float("nan")
        _, y, _ = run_forward(c, want_buf=False)
        assert torch.isfinite(y[[i for i in range(c.T) if i != 2]].float()).all()
        dx = torch.empty((c.T, c.K), dtype=bf16, device="cuda")
        aa.lora_linear_mx_backward(dx, None, None, c.dy, None, c.Wq, c.A, c.B, c.idx, c.rank, c.scale, workspace(c),
                                   W_scales=c.Ws)
        assert bool(dx[1].isnan().all())
        assert torch.isfinite(dx[[i for i in range(c.T) if i != 1]].float()).all()


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] in (1, 5, 33, 256, 777, 2100)], ids=str)
def test_empty_slots_with_any_scale(shape):
    """A token of an empty slot (rank 0) gets the projection alone, whatever the
    slot's scale; and no ranks given: every slot has all of them."""
    c = layer(shape, 9, ragged=False)
    c.rank[:] = 0
    c.scale[:] = float("inf")
    y_ref, y_tol, _, _ = c.forward()
    _, y, buf = run_forward(c)
    within(y, y_ref, y_tol, "y")
    assert not bool(buf.any())
    c.rank[:] = c.R
    c.scale[:] = 0.5
    y_ref, y_tol, b_ref, b_tol = c.forward()
    rank, c.rank = c.rank, None
    _, y, buf = run_forward(c)
    c.rank = rank
    within(y, y_ref, y_tol, "y")
    within(buf, b_ref, b_tol, "buf")


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] in (1, 5, 16, 100, 1200, 2100)], ids=str)
def test_values_past_a_slots_rank(shape):
    """A and B hold other values past each slot's rank (a larger adapter before)."""
    c = layer(shape, 13, stale=True, x8=True)
    y_ref, y_tol, b_ref, b_tol = c.forward()
    _, y, buf = run_forward(c)
    within(y, y_ref, y_tol, "y")
    within(buf, b_ref, b_tol, "buf")
    dx = torch.empty((c.T, c.K), dtype=bf16, device="cuda")
    dA, dB = gradients(c)
    call_backward(c, dx, dA, dB, buf=buf)
    check_backward(c, buf, dx, dA, dB)


def test_segments_ready():
    """The backward call and a second layer reuse the segments in the workspace."""
    c = layer((1200, 2048, (260,), 16, 3, 4), 17, x8=True)
    ws = workspace(c)
    aa.lora_build_segments(c.idx, c.rank, c.L, c.R, ws)
    y_ref, y_tol, _, _ = c.forward()
    y = torch.empty((c.T, 260), dtype=bf16, device="cuda")
    buf = torch.empty((1, c.T, c.R), device="cuda")
    for _ in range(2):
        aa.lora_linear_mx(y, c.x, c.Wq, c.Ws, c.A, c.B, c.idx, c.rank, c.scale, ws, buf=buf,
                          flags=aa.LORA_FLAG_SEGMENTS_READY)
        within(y, y_ref, y_tol, "y")
    dx = torch.empty((c.T, c.K), dtype=bf16, device="cuda")
    dA, dB = gradients(c)
    call_backward(c, dx, dA, dB, buf=buf, ws=ws, flags=aa.LORA_FLAG_SEGMENTS_READY)
    check_backward(c, buf, dx, dA, dB)


def test_no_tokens():
    c = layer((3, 72, (36,), 24, 3, 0), 1, x8=True)
    ws = workspace(c)
    e = lambda *s, dt=bf16: torch.empty(s, dtype=dt, device="cuda")
    u8 = torch.uint8
    aa.lora_linear_mx(e(0, 36), e(0, 72), c.Wq, c.Ws, c.A, c.B, c.idx[:0], c.rank, c.scale, ws)
    dA, dB = gradients(c)
    aa.lora_linear_mx_backward(e(0, 72), dA, dB, e(0, 36), e(0, 96, dt=u8), c.Wq, c.A, c.B, c.idx[:0], c.rank, c.scale,
                               ws, buf=e(1, 0, 24, dt=torch.float32), x_scales=e(0, 4, dt=u8), W_scales=c.Ws)
    assert not any(bool(t.any()) for t in dA + dB)


def test_rows_and_slots_of_one_token_calls():
    """One token after another on one workspace, each with another slot or none: the
    counts that a call leaves are the next one's."""
    c = layer((40, 520, (260, 132), 16, 5, 0), 19)
    ws = aa.alloc_linear_mx_workspace(1, c.K, c.N, c.R, c.L)
    y_ref, y_tol, b_ref, b_tol = c.forward()
    for t in range(c.T):
        y = torch.full((1, 392), FILL, dtype=bf16, device="cuda")
        buf = torch.full((2, 1, 16), FILL, device="cuda")
        aa.lora_linear_mx(y, c.x[t:t + 1], c.Wq, c.Ws, c.A, c.B, c.idx[t:t + 1], c.rank, c.scale, ws, buf=buf)
        within(y, y_ref[t:t + 1], y_tol[t:t + 1], f"y of token {t}")
        within(buf, b_ref[:, t:t + 1], b_tol[:, t:t + 1], f"buf of token {t}")


def test_workspace_shared_by_layers_and_kinds():
    """Layers of several sizes, bf16 and 4-bit ones, in turn on one workspace as
    large as the largest needs."""
    shapes = [(257, 128, (128, 8), 16, 3, 0), (1, 4096, (512, 128, 128), 16, 8, 0), (2100, 136, (500, 72), 64, 30, 0),
              (64, 256, (264,), 64, 130, 8), (777, 1352, (1100, 36, 516), 24, 5, 0)]
    cs = [layer(s, 20 + i, x8=i % 2 == 0) for i, s in enumerate(shapes)]
    ws = max((workspace(c) for c in cs), key=lambda t: t.nbytes)
    for _ in range(2):
        for c in cs:
            y_ref, y_tol, b_ref, b_tol = c.forward()
            _, y, buf = run_forward(c, ws=ws)
            within(y, y_ref, y_tol, "y")
            within(buf, b_ref, b_tol, "buf")
            full = torch.empty((c.T, sum(c.N)), dtype=bf16, device="cuda")
            aa.lora_linear(full, c.x, c.W, c.A, c.B, c.idx, c.rank, c.scale, ws)
            within(full, y_ref, y_tol, "y of bf16 W")
            dx = torch.empty((c.T, c.K), dtype=bf16, device="cuda")
            dA, dB = gradients(c)
            call_backward(c, dx, dA, dB, buf=buf, ws=ws)
            check_backward(c, buf, dx, dA, dB)


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] in (1, 5, 33, 256, 777, 2100)] +
                         FEW_SHAPES[::3], ids=str)
def test_same_bits_on_another_stream_and_in_graphs(shape):
    """A call on a stream of its own, and two captured calls on one workspace,
    replayed between eager work: the bits of the eager call."""
    c = layer(shape, 31, x8=True)
    ws = workspace(c)
    _, y0, buf0 = run_forward(c, ws=ws)
    dx0 = torch.empty((c.T, c.K), dtype=bf16, device="cuda")
    dA0, dB0 = gradients(c)
    call_backward(c, dx0, dA0, dB0, buf=buf0, ws=ws)
    want = [t.clone() for t in (y0, buf0, dx0, *dA0, *dB0)]

    y, buf, dx = torch.empty_like(y0), torch.empty_like(buf0), torch.empty_like(dx0)
    dA, dB = gradients(c)
    xq, xs = aa.alloc_mx(c.T, c.K, aa.LORA_MX_INT8)
    x8 = torch.empty((c.T, c.K), dtype=bf16, device="cuda")

    def step():
        aa.lora_mx_quantize(xq, xs, c.x, aa.LORA_MX_INT8)
        aa.lora_mx_dequantize(x8, xq, xs, aa.LORA_MX_INT8)
        aa.lora_linear_mx(y, x8, c.Wq, c.Ws, c.A, c.B, c.idx, c.rank, c.scale, ws, bias=c.bias, buf=buf)
        aa.lora_linear_mx_backward(dx, dA, dB, c.dy, xq, c.Wq, c.A, c.B, c.idx, c.rank, c.scale, ws, buf=buf,
                                   x_scales=xs, W_scales=c.Ws)

    def check():
        torch.cuda.synchronize()
        for got, ref in zip((y, buf, dx, *dA, *dB), want):
            assert torch.equal(got, ref)
        for t in (y, buf, dx, *dA, *dB):
            t.fill_(FILL)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    check()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
            check()
        step()
        check()
