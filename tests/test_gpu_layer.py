"""lora_linear and lora_linear_backward against their 64-bit definitions."""
import pytest
import torch

import adapter_apply_amd as aa
from tests.layer_util import Layer, within

pytestmark = pytest.mark.gpu

FILL = 7.0

# T, K, N, R, L, extra columns: lengths around the tiles and the ways to the
# rank vectors and the delta, contraction lengths off the 64-step tile, slice
# widths off the column tiles and off 8, ranks off 16 and past 64, one slot and
# many.
SHAPES = [
    (1, 8, (4,), 8, 1, 0),                 # one launch
    (1, 648, (72, 20), 16, 3, 0),          # v as further columns of dx
    (70, 1032, (100, 360, 4), 40, 7, 4),
    (128, 4096, (64, 1000), 64, 24, 8),
    (1024, 392, (72,), 8, 40, 0),
    (1, 4096, (512, 128, 128), 16, 8, 0),
    (1, 72, (36, 20), 32, 3, 4),
    (1, 64, (16400,), 16, 2, 0),           # one token, many columns
    (1, 640, (100,), 40, 2, 0),            # up to 64 tokens
    (1, 4104, (68, 4), 16, 2, 4),
    (2, 136, (40,), 8, 4, 0),              # as many further columns as the layer's
    (5, 2120, (100, 36), 16, 3, 4),        # K splits that do not divide the K tiles
    (2, 24, (32800, 4), 8, 3, 0),          # few tokens, too many columns for one launch: tiles
    (3, 72, (36,), 24, 3, 0),
    (16, 64, (64, 64), 16, 4, 8),
    (17, 136, (100, 36, 4), 40, 5, 4),
    (64, 256, (264,), 64, 130, 8),
    (12, 4096, (14336,), 32, 6, 4),        # up to 64 tokens, a large projection: tiles
    (33, 8256, (1100, 36), 48, 5, 0),
    (65, 8200, (68,), 16, 5, 0),           # direct, K splits
    (100, 512, (64, 100), 32, 7, 4),       # direct, grouped rank vectors
    (200, 520, (68, 132), 8, 9, 4),
    (256, 128, (128,), 128, 40, 0),
    (257, 128, (128, 8), 16, 3, 8),
    (300, 72, (260,), 512, 6, 4),
    (700, 64, (72,), 16, 64, 0),
    (777, 1352, (1100, 36, 516), 24, 5, 0),
    (1000, 136, (3200,), 32, 20, 8),       # sorted, delta in the join; 128-wide tiles
    (1000, 3208, (132, 60), 48, 20, 4),    # 128-wide gradient tiles
    (1200, 2048, (260,), 16, 3, 4),        # sorted, delta in the tiles' K steps
    (1500, 128, (72, 20), 24, 1024, 0),
    (2100, 136, (5000, 700), 64, 300, 0),
    (2100, 1032, (5000, 260), 16, 4, 0),   # 256-wide forward tiles
    (2100, 5640, (100, 36), 72, 12, 4),    # 256-wide gradient tiles
    (4500, 64, (60,), 16, 2, 0),           # token splits of the weight gradients
    (9000, 72, (20, 12), 40, 1, 4),
]


def run_forward(c, bias=None, want_buf=True, ws=None):
    n = sum(c.N)
    full = torch.full((c.T, c.ldn), FILL, dtype=torch.bfloat16, device="cuda")
    y = full[:, :n]
    buf = torch.full((c.S, c.T, c.R), FILL, device="cuda") if want_buf else None
    ws = ws if ws is not None else aa.alloc_linear_workspace(c.T, c.K, c.N, c.R, c.L)
    aa.lora_linear(y, c.x, c.W, c.A, c.B, c.idx, c.rank, c.scale, ws, bias=c.bias, buf=buf)
    return full, y, buf


def run_backward(c, dx, buf=None, W=True, flags=0, ws=None, dA=None, dB=None):
    ws = ws if ws is not None else aa.alloc_linear_workspace(c.T, c.K, c.N, c.R, c.L)
    dA = dA or [torch.full((c.L, c.R, c.K), FILL, device="cuda") for _ in c.N]
    dB = dB or [torch.full((c.L, n, c.R), FILL, device="cuda") for n in c.N]
    aa.lora_linear_backward(dx, dA, dB, c.dy, c.x, c.W if W else None, c.A, c.B, c.idx, c.rank,
                            c.scale, ws, buf=buf, flags=flags)
    return dA, dB


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, bias):
    T, K, N, R, L, extra = shape
    c = Layer(T, K, N, R, L, seed=T + K, extra=extra, bias=bias, runs=bias)
    y_ref, y_tol, b_ref, b_tol = c.forward()
    full, y, buf = run_forward(c)
    within(y, y_ref, y_tol, "y")
    within(buf, b_ref, b_tol, "buf")
    assert bool((full[:, sum(N):] == FILL).all()), "columns past the slices were written"


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, given):
    T, K, N, R, L, extra = shape
    c = Layer(T, K, N, R, L, seed=T + K + 1, extra=extra, runs=given)
    buf = c.forward()[2].float() if given else None
    dx_ref, dx_tol, dA_ref, eA, dB_ref, eB = c.backward(buf=buf)
    full = torch.full((T, K + 8), FILL, dtype=torch.bfloat16, device="cuda")
    dA, dB = run_backward(c, full[:, :K], buf=buf)
    within(full[:, :K], dx_ref, dx_tol, "dx")
    for s in range(c.S):
        within(dA[s], dA_ref[s], eA[s], f"dA[{s}]")
        within(dB[s], dB_ref[s], eB[s], f"dB[{s}]")
    assert bool((full[:, K:] == FILL).all()), "columns past K were written"


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] < 1100], ids=str)
def test_backward_of_x_alone(shape):
    T, K, N, R, L, extra = shape
    c = Layer(T, K, N, R, L, seed=T + K + 2, extra=extra)
    dx_ref, dx_tol = c.backward()[:2]
    full = torch.full((T, K + 8), FILL, dtype=torch.bfloat16, device="cuda")
    ws = aa.alloc_linear_workspace(T, K, N, R, L)
    for _ in range(2):
        aa.lora_linear_backward(full[:, :K], None, None, c.dy, c.x, c.W, c.A, c.B, c.idx, c.rank, c.scale, ws)
        within(full[:, :K], dx_ref, dx_tol, "dx")
        assert bool((full[:, K:] == FILL).all()), "columns past K were written"
        full[:, :K] = FILL


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] in (17, 200, 1000, 2100)], ids=str)
def test_backward_in_place(shape):
    """W None: dx += the adapters' part; rows without an adapter keep their bits."""
    T, K, N, R, L, extra = shape
    c = Layer(T, K, N, R, L, seed=5, extra=extra)
    g = torch.Generator().manual_seed(3)
    base = torch.randn((T, K), generator=g).to(torch.bfloat16).cuda()
    dx = base.clone()
    run_backward(c, dx, W=False)
    ref, tol = c.backward(with_w=False)[:2]
    ref = ref + base.double()
    within(dx, ref, tol + ref.abs() * 2.0 ** -8, "dx")
    none = torch.ones(T, dtype=torch.bool, device="cuda")
    for _, _, m in c.members():
        none[m] = False
    assert torch.equal(dx[none], base[none])


@pytest.mark.parametrize("T,K", [(700, 136), (90, 1032)])
def test_accumulate_and_parts(T, K):
    """Two accumulated calls add up; a call that wants one output only gives
    the bits of the call that wants all."""
    N, R, L = (100, 36), 24, 5
    c = Layer(T, K, N, R, L, seed=9)
    dx = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    dA, dB = run_backward(c, dx)
    ws = aa.alloc_linear_workspace(T, K, N, R, L)
    for want in ("dx", "dA", "dB"):
        one_dx = torch.empty_like(dx) if want == "dx" else None
        one_A = [torch.empty_like(t) for t in dA] if want == "dA" else None
        one_B = [torch.empty_like(t) for t in dB] if want == "dB" else None
        aa.lora_linear_backward(one_dx, one_A, one_B, c.dy, c.x, c.W, c.A, c.B, c.idx, c.rank,
                                c.scale, ws)
        if one_dx is not None:
            assert torch.equal(one_dx, dx)
        for one, all_ in ((one_A, dA), (one_B, dB)):
            if one is not None:
                assert all(torch.equal(p, q) for p, q in zip(one, all_))
    sA, sB = [t.clone() for t in dA], [t.clone() for t in dB]
    run_backward(c, dx, flags=aa.LORA_FLAG_ACCUMULATE, dA=sA, dB=sB, ws=ws)
    # the split sums are added to what was there one after the other
    for p, q in zip(sA + sB, dA + dB):
        assert torch.allclose(p, 2 * q, rtol=0, atol=float(q.abs().max()) * 20 * 2.0 ** -23)


def test_more_than_a_million_tokens():
    """A narrow layer over more 16-token blocks than one dimension of a grid
    takes."""
    T, K, N, R, L = (1 << 20) + 40, 8, (4,), 8, 3
    c = Layer(T, K, N, R, L, seed=2)
    y_ref, y_tol, b_ref, b_tol = c.forward()
    full, y, buf = run_forward(c)
    within(y, y_ref, y_tol, "y")
    within(buf, b_ref, b_tol, "buf")
    dx_ref, dx_tol, dA_ref, eA, dB_ref, eB = c.backward()
    dx = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    dA, dB = run_backward(c, dx)
    within(dx, dx_ref, dx_tol, "dx")
    within(dA[0], dA_ref[0], eA[0], "dA")
    within(dB[0], dB_ref[0], eB[0], "dB")


def test_no_tokens():
    c = Layer(5, 64, (32,), 8, 3, seed=1)
    ws = aa.alloc_linear_workspace(5, 64, [32], 8, 3)
    e = lambda w: torch.empty((0, w), dtype=torch.bfloat16, device="cuda")
    idx = torch.empty((0,), dtype=torch.int32, device="cuda")
    aa.lora_linear(e(32), e(64), c.W, c.A, c.B, idx, c.rank, c.scale, ws)
    dA = [torch.full((3, 8, 64), FILL, device="cuda")]
    dB = [torch.full((3, 32, 8), FILL, device="cuda")]
    args = (e(32), e(64), c.W, c.A, c.B, idx, c.rank, c.scale, ws)
    aa.lora_linear_backward(e(64), dA, dB, *args, flags=aa.LORA_FLAG_ACCUMULATE)
    assert bool((dA[0] == FILL).all()) and bool((dB[0] == FILL).all())
    aa.lora_linear_backward(e(64), dA, dB, *args)
    assert bool((dA[0] == 0).all()) and bool((dB[0] == 0).all())


@pytest.mark.parametrize("T", [40, 600])
def test_no_adapter_anywhere(T):
    """Every token without an adapter: y is the projection, gradients are zero."""
    K, N, R, L = 72, (36, 8), 16, 4
    c = Layer(T, K, N, R, L, seed=2)
    c.idx.fill_(-1)
    c.idx[::2] = L + 3
    y_ref, y_tol, _, _ = c.forward()
    _, y, buf = run_forward(c)
    within(y, y_ref, y_tol, "y")
    assert bool((buf == 0).all())
    dx = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    dA, dB = run_backward(c, dx, buf=buf)
    assert all(bool((t == 0).all()) for t in dA + dB)
    ref, tol = c.backward()[:2]
    within(dx, ref, tol, "dx")


@pytest.mark.parametrize("T,K,N", [(1, 136, (100, 36)), (12, 136, (100, 36)), (100, 136, (100, 36)), (50, 1032, (100, 36)),
                                   (700, 136, (100, 36)), (1200, 2048, (260,)),
                                   (1100, 136, (3200,)), (2100, 1032, (5000, 260)),
                                   (2100, 5640, (100, 36))], ids=str)
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_bad_adapter_stays_alone(T, K, N, bad):
    """An infinity or NaN in one slot's A and B, and in one token's x and dy,
    reaches no other slot's tokens or gradients."""
    R, L = 16, 4
    c = Layer(T, K, N, R, L, seed=4, ragged=False)
    c.rank.fill_(R)
    c.idx.copy_((torch.arange(T, dtype=torch.int32) + (3 if T == 1 else 0)) % (L + 1) - 1)
    good = [run_forward(c)[1].clone()]
    dx = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    gA, gB = run_backward(c, dx)
    good.append(dx.clone())
    for t in (*c.A, *c.B):
        t[2, ..., 0] = bad
        t[2, 1] = bad
    row = min(3, T - 1)                         # a token of slot 2
    assert int(c.idx[row]) == 2
    c.x[row, 5] = bad
    c.dy[row, 7] = bad
    other = c.idx != 2
    y = run_forward(c)[1]
    assert torch.equal(y[other], good[0][other])
    bA, bB = run_backward(c, dx)
    assert torch.equal(dx[other], good[1][other])
    for p, q in zip(bA + bB, gA + gB):
        for i in (0, 1, 3):
            assert torch.equal(p[i], q[i]), i


@pytest.mark.parametrize("T", [40, 4500])
def test_bad_rows_keep_padded_ranks_zero(T):
    """An infinity in a token's x and dy leaves zeros at the ranks past its
    slot's own, and every other slot's gradient."""
    c = Layer(T, 136, (100, 36), 24, 3, seed=12)
    c.rank[:] = torch.tensor([24, 5, 13], device="cuda")
    clean = run_backward(c, None)
    hit = torch.nonzero(c.idx == 1).flatten()[0]
    c.x[hit, 3] = float("inf")
    c.dy[hit, 7] = float("nan")
    dA, dB = run_backward(c, None)
    for s in range(c.S):
        for i in (0, 2):
            assert torch.equal(dA[s][i], clean[0][s][i]) and torch.equal(dB[s][i], clean[1][s][i])
        assert bool(dA[s][1, :5].isnan().any())
        assert bool((dA[s][1, 5:] == 0).all()) and bool((dB[s][1, :, 5:] == 0).all())


@pytest.mark.parametrize("T", [33, 900])
def test_another_stream_and_repeats(T):
    """Calls on a stream of their own, and repeats, give the same bits."""
    c = Layer(T, 264, (132, 36), 32, 6, seed=6)
    _, y, buf = run_forward(c)
    dx = torch.empty((T, 264), dtype=torch.bfloat16, device="cuda")
    dA, dB = run_backward(c, dx, buf=buf)
    ws = aa.alloc_linear_workspace(T, 264, c.N, 32, 6)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(3):
            _, y2, buf2 = run_forward(c, ws=ws)
            dx2 = torch.empty_like(dx)
            dA2, dB2 = run_backward(c, dx2, buf=buf2, ws=ws)
    st.synchronize()
    assert torch.equal(y, y2) and torch.equal(buf, buf2) and torch.equal(dx, dx2)
    assert all(torch.equal(p, q) for p, q in zip(dA + dB, dA2 + dB2))


@pytest.mark.parametrize("T,K,N", [(20, 136, (100, 36)), (600, 136, (100, 36)), (5000, 136, (100, 36)),
                                   (90, 520, (264, 136))])
def test_graph_replays(T, K, N):
    """Two graphs on one workspace, replayed in turn with new inputs and eager
    calls between, equal the eager calls bit for bit."""
    R, L = 16, 5
    c = Layer(T, K, N, R, L, seed=7)
    ws = aa.alloc_linear_workspace(T, K, N, R, L)
    y = torch.empty((T, sum(N)), dtype=torch.bfloat16, device="cuda")
    buf = torch.empty((c.S, T, R), device="cuda")
    dx = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    dA = [torch.empty((L, R, K), device="cuda") for _ in N]
    dB = [torch.empty((L, n, R), device="cuda") for n in N]

    def fwd():
        aa.lora_linear(y, c.x, c.W, c.A, c.B, c.idx, c.rank, c.scale, ws, buf=buf)

    def bwd():
        aa.lora_linear_backward(dx, dA, dB, c.dy, c.x, c.W, c.A, c.B, c.idx, c.rank, c.scale, ws,
                                buf=buf)

    fwd(), bwd()
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        fwd()
    with torch.cuda.graph(g2):
        bwd()
    gen = torch.Generator().manual_seed(8)
    for rep in range(4):
        c.x.copy_(torch.randn((T, K), generator=gen).to(torch.bfloat16))
        c.idx.copy_(torch.randint(-1, L + 1, (T,), generator=gen).to(torch.int32))
        outs = (y, buf, dx, *dA, *dB)
        g1.replay(), g2.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        fwd(), bwd()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, outs)), rep


def test_segments_ready_shared_by_layers():
    """Segments built once on the layer workspace serve forward and gradient."""
    T, R, L = 700, 16, 5
    c = Layer(T, 136, (100, 36), R, L, seed=11)
    ws = aa.alloc_linear_workspace(T, 136, c.N, R, L)
    _, y, buf = run_forward(c)
    dx = torch.empty((T, 136), dtype=torch.bfloat16, device="cuda")
    dA, dB = run_backward(c, dx, buf=buf)
    aa.lora_build_segments(c.idx, c.rank, L, R, ws)
    y2, dx2 = torch.empty_like(y), torch.empty_like(dx)
    for _ in range(2):
        aa.lora_linear(y2, c.x, c.W, c.A, c.B, c.idx, c.rank, c.scale, ws,
                       flags=aa.LORA_FLAG_SEGMENTS_READY)
        dA2, dB2 = run_backward(c, dx2, buf=buf, ws=ws, flags=aa.LORA_FLAG_SEGMENTS_READY)
        assert torch.equal(y, y2) and torch.equal(dx, dx2)
        assert all(torch.equal(p, q) for p, q in zip(dA + dB, dA2 + dB2))


def test_no_ranks_given():
    """slot_rank None: every slot has rank R."""
    for T in (30, 400):
        c = Layer(T, 72, (36,), 24, 3, seed=12, ragged=False)
        c.rank.fill_(24)
        g = torch.Generator().manual_seed(1)
        for t in (*c.A, *c.B):
            t.copy_((torch.randn(t.shape, generator=g) * 0.1).to(torch.bfloat16))
        ws = aa.alloc_linear_workspace(T, 72, c.N, 24, 3)
        y = torch.empty((T, 36), dtype=torch.bfloat16, device="cuda")
        aa.lora_linear(y, c.x, c.W, c.A, c.B, c.idx, None, c.scale, ws)
        ref, tol, _, _ = c.forward()
        within(y, ref, tol, "y")


def test_gradient_against_differences():
    """dA and dB of loss = sum(dy * y) against differences of the 64-bit
    forward: the loss is linear in A for fixed B and the other way round, so a
    whole step of one element is exact."""
    c = Layer(50, 72, (36, 20), 8, 3, seed=13, ragged=False)
    c.rank.fill_(8)
    buf = c.forward()[2].float()
    dx = torch.empty((50, 72), dtype=torch.bfloat16, device="cuda")
    dA, dB = run_backward(c, dx, buf=buf)
    *_, eA, _, eB = c.backward(buf=buf)
    loss = lambda: float((c.forward()[0] * c.dy.double()).sum())
    base = loss()
    slots = {i for i, _, _ in c.members()}
    for tensors, grads, tols in ((c.A, dA, eA), (c.B, dB, eB)):
        for s, at in ((0, (0, 3, 5)), (1, (2, 1, 7)), (1, (0, 0, 0))):
            if at[0] not in slots:
                continue
            old = tensors[s][at].clone()
            tensors[s][at] = old + 1.0
            step = float(tensors[s][at].double() - old.double())
            diff = (loss() - base) / step
            tensors[s][at] = old
            # buf was rounded to fp32 once (2^-24), the rest is the bound of the call
            tol = float(tols[s][at]) * 1.01 + abs(base) * 2.0 ** -45
            assert abs(float(grads[s][at]) - diff) <= tol, (s, at)


def test_training_step_of_many_adapters():
    """Forward, gradient, per-adapter norm and clip in one run, two layers on
    one workspace: each stage against the 64-bit chain of the same inputs."""
    T, R, L = 300, 16, 4
    c1 = Layer(T, 136, (72, 64), R, L, seed=20, ragged=False)
    c2 = Layer(T, 136, (48,), R, L, seed=21, ragged=False)
    for c in (c1, c2):
        c.rank.fill_(R)
    c2.idx.copy_(c1.idx)
    ws = aa.alloc_linear_workspace(T, 136, (72, 64), R, L)
    grads = []
    for c in (c1, c2):
        _, y, buf = run_forward(c, ws=ws)
        within(y, *c.forward()[:2], "y")
        dx = torch.empty((T, 136), dtype=torch.bfloat16, device="cuda")
        dA, dB = run_backward(c, dx, buf=buf, ws=ws)
        dx_ref, dx_tol, dA_ref, eA, dB_ref, eB = c.backward(buf=buf)
        within(dx, dx_ref, dx_tol, "dx")
        for p, r, e in zip(dA + dB, dA_ref + dB_ref, eA + eB):
            within(p, r, e, "grad")
        grads += dA + dB
    gws = aa.alloc_grad_workspace(grads)
    norm = torch.empty((L,), device="cuda")
    aa.lora_grad_norm(norm, grads, gws)
    ref = sum(t.double().square().reshape(L, -1).sum(1) for t in grads).sqrt()
    assert bool(((norm.double() - ref).abs() <= ref * 2.0 ** -24 * 1.001).all())
    limit = (ref * torch.tensor([0.5, 2.0, 0.1, 1.5], device="cuda", dtype=torch.float64)).float()
    before = [t.clone() for t in grads]
    aa.lora_grad_clip(grads, grads, norm, limit)
    coef = (limit.double() / (norm.double() + 1e-6)).clamp(max=1.0)
    for p, q in zip(grads, before):
        # the sum, the quotient and the product are rounded once each
        want = q.double() * coef[:, None, None]
        assert bool(((p.double() - want).abs() <= want.abs() * 4 * 2.0 ** -24).all())
    assert torch.equal(grads[0][1], before[0][1])
