"""lora_linear and lora_linear_backward in every form that their rules choose,
against the 64-bit definitions; slots that hold other values past their rank."""
import pytest
import torch

import adapter_apply_amd as aa
from tests import layer_rules
from tests.layer_util import U32, Layer, within
from tests.test_gpu_layer import FILL, SHAPES, run_backward, run_forward

pytestmark = pytest.mark.gpu

# T, K, N, R, L, extra columns; forward | dx beside dA and dB | dx alone, as
# form, tile and K splits.
FORMS = [
    (256, 4096, (4096, 1024, 1024), 16, 8, 0),     # wide 128 5 | wide 128 7 | the same
    (500, 1608, (3100, 2404, 36), 16, 10, 4),      # wide 128 2, evened out | wide 128 6
    (520, 1672, (6004, 1100), 8, 12, 0),           # wide 128 3, evened out | tiles 128 7 | wide 128 6
    (467, 1704, (6272,), 24, 78, 8),               # join 128 2, evened out | tiles 128 8
    (464, 1648, (1332, 6876), 24, 29, 4),          # join 128 3, evened out | tiles 128 8 | wide 128 5
    (140, 6680, (3280, 76, 688), 24, 115, 0),      # join 128 7 | tiles 128 4
    (213, 1424, (32,), 128, 30, 0),                # join 64 2 | tiles 64 1
    (34, 80, (12056, 13424), 128, 2, 8),           # join 128 1 | tiles 64 8
    (1279, 1040, (1204, 1332), 16, 1, 0),          # tiles 128 1 | tiles 64 1, token splits
    (1070, 1224, (2688,), 64, 8, 8),               # tiles 128 2 | tiles 64 1
    (1499, 808, (576,), 32, 2, 0),                 # tiles 64 1 | tiles 64 1, token splits
    (500, 2056, (4004,), 8, 520, 4),               # direct 128 4 | tiles 128 7
    (640, 2056, (4992,), 8, 640, 0),               # direct 128 2, evened out | tiles 128 6
    (640, 72, (4996,), 8, 640, 0),                 # direct 128 1 | tiles 64 8
    (634, 5952, (1228,), 64, 45, 4),               # grouped 128 8 | tiles 128 1
    (153, 7752, (624, 1040), 40, 58, 8),           # join 64 6 | tiles 64 1 | wide 128 2, evened out
    (823, 2352, (1608,), 32, 72, 0),               # join 64 1 | tiles 64 1 | wide 128 3, evened out
    (422, 6768, (1588,), 24, 114, 4),              # join 128 8 | wide 128 3, evened out
    (165, 7776, (4124,), 40, 118, 0),              # join 128 7 | wide 128 2, evened out
    (398, 6232, (32,), 16, 3, 0),                  # direct 64 8 | wide 128 1
    (2823, 152, (6724, 1068, 372), 16, 1, 4),      # join 128 1 | tiles 128 8, token splits
]


def layer(shape, i, **more):
    T, K, N, R, L, extra = shape
    return Layer(T, K, N, R, L, seed=T + K + 40 + i, extra=extra, stale=True, **more)


@pytest.mark.parametrize("i,shape", list(enumerate(FORMS + SHAPES)), ids=str)
def test_forward(i, shape):
    c = layer(shape, i, bias=i % 2 == 0, runs=i % 3 == 0)
    y_ref, y_tol, b_ref, b_tol = c.forward()
    full, y, buf = run_forward(c, want_buf=i % 4 != 1)
    within(y, y_ref, y_tol, "y")
    if buf is not None:
        within(buf, b_ref, b_tol, "buf")
    assert bool((full[:, sum(c.N):] == FILL).all()), "columns past the slices were written"


@pytest.mark.parametrize("i,shape", list(enumerate(FORMS + SHAPES)), ids=str)
def test_backward(i, shape):
    T, K = shape[:2]
    c = layer(shape, i, runs=i % 3 == 1)
    buf = c.forward()[2].float() if i % 2 else None
    dx_ref, dx_tol, dA_ref, eA, dB_ref, eB = c.backward(buf=buf)
    full = torch.full((T, K + 8), FILL, dtype=torch.bfloat16, device="cuda")
    dA, dB = run_backward(c, full[:, :K], buf=buf)
    within(full[:, :K], dx_ref, dx_tol, "dx")
    for s in range(c.S):
        within(dA[s], dA_ref[s], eA[s], f"dA[{s}]")
        within(dB[s], dB_ref[s], eB[s], f"dB[{s}]")
    assert bool((full[:, K:] == FILL).all()), "columns past K were written"


@pytest.mark.parametrize("i,shape", [(i, s) for i, s in enumerate(FORMS) if s[0] < 1100], ids=str)
def test_backward_of_x_alone(i, shape):
    c = layer(shape, i)
    dx_ref, dx_tol = c.backward()[:2]
    full = torch.full((c.T, c.K + 8), FILL, dtype=torch.bfloat16, device="cuda")
    ws = aa.alloc_linear_workspace(c.T, c.K, c.N, c.R, c.L)
    aa.lora_linear_backward(full[:, :c.K], None, None, c.dy, c.x, c.W, c.A, c.B, c.idx, c.rank, c.scale, ws)
    within(full[:, :c.K], dx_ref, dx_tol, "dx")
    assert bool((full[:, c.K:] == FILL).all()), "columns past K were written"


@pytest.mark.parametrize("T,K,N,R,L", [s[:5] for s in FORMS if s[4] > 2 and s[4] < 128], ids=str)
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_bad_adapter_stays_alone(T, K, N, R, L, bad):
    """An infinity or NaN in one slot's A and B, and in one of its tokens' x and
    dy, reaches no other slot's tokens or gradients."""
    c = Layer(T, K, N, R, L, seed=4, ragged=False)
    c.rank.fill_(R)
    c.idx.copy_(torch.arange(T, dtype=torch.int32) % (L + 1) - 1)
    dx, alone = (torch.empty((T, K), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = aa.alloc_linear_workspace(T, K, N, R, L)

    def run():
        y = run_forward(c, ws=ws)[1].clone()
        dA, dB = run_backward(c, dx, ws=ws)
        aa.lora_linear_backward(alone, None, None, c.dy, c.x, c.W, c.A, c.B, c.idx, c.rank, c.scale, ws)
        return (y, dx.clone(), alone.clone()), dA + dB

    good, grads = run()
    for t in (*c.A, *c.B):
        t[2, ..., 0] = bad
        t[2, 1] = bad
    other = c.idx != 2
    assert 0 < int(other.sum()) < T
    c.x[3, 5] = bad                              # (a token of slot 2)
    c.dy[3, 7] = bad
    rows, bad_grads = run()
    for p, q in zip(rows, good):
        assert torch.equal(p[other], q[other])
        assert not bool(p[~other].isfinite().all())
    keep = [i for i in range(L) if i != 2]
    for p, q in zip(bad_grads, grads):
        assert torch.equal(p[keep], q[keep])


@pytest.mark.parametrize("K,N,R,L", [(136, (100, 36), 16, 4), (4096, (512, 128, 128), 16, 8), (4104, (68, 4), 16, 3),
                                     (136, (1000,), 40, 4), (72, (36,), 24, 9)], ids=str)
@pytest.mark.parametrize("slot", [0, -1])
def test_one_token_beside_a_bad_adapter(K, N, R, L, slot):
    """One token of another slot, or of none, while slot 2 holds infinities."""
    c = Layer(1, K, N, R, L, seed=5, ragged=False)
    c.rank.fill_(R)
    c.idx.fill_(slot)
    dx = torch.empty((1, K), dtype=torch.bfloat16, device="cuda")
    y = run_forward(c)[1].clone()
    dA, dB = run_backward(c, dx)
    want = [y, dx.clone(), *dA, *dB]
    for t in (*c.A, *c.B):
        t[2] = float("inf")
    y = run_forward(c)[1].clone()
    dA, dB = run_backward(c, dx)
    assert all(torch.equal(p, q) for p, q in zip([y, dx, *dA, *dB], want))


@pytest.mark.parametrize("T,K,N,R,L", [(4500, 64, (60,), 16, 2), (2823, 152, (6724, 1068, 372), 16, 1),
                                       (9000, 72, (20, 12), 40, 1), (1499, 808, (576,), 32, 2)], ids=str)
def test_accumulate_over_token_splits(T, K, N, R, L):
    """dA and dB added to what is there where a slot's tokens are split."""
    assert layer_rules.weight_splits(T, K, N, R, L) > 1
    c = Layer(T, K, N, R, L, seed=31, stale=True)
    _, _, dA_ref, eA, dB_ref, eB = c.backward()
    g = torch.Generator().manual_seed(6)
    start = lambda ref: [torch.randn(t.shape, generator=g).cuda() * t.abs().max().float() for t in ref]
    for dx in (None, torch.empty((T, K), dtype=torch.bfloat16, device="cuda")):
        oA, oB = start(dA_ref), start(dB_ref)
        dA, dB = [t.clone() for t in oA], [t.clone() for t in oB]
        run_backward(c, dx, flags=aa.LORA_FLAG_ACCUMULATE, dA=dA, dB=dB)
        for p, o, r, e in zip(dA + dB, oA + oB, dA_ref + dB_ref, eA + eB):
            # up to 16 split sums added one after the other to what was there: their
            # part in the old value, and in the sum as the bound e already counts
            # more additions than that
            within(p, r + o.double(), e + 17 * U32 * o.double().abs(), "sum")


@pytest.mark.parametrize("T,K,N", [(20, 136, (100, 36)), (96, 520, (264, 136)), (1200, 392, (100, 36))], ids=str)
def test_backward_without_x(T, K, N):
    """dx, and dB with a saved u, do not read x: the bits of the calls that get it."""
    c = Layer(T, K, N, 24, 5, seed=33, stale=True)
    ws = aa.alloc_linear_workspace(T, K, N, 24, 5)
    buf = run_forward(c)[2]
    for W in (c.W, None):
        for weights in (False, True):
            got = []
            for x in (c.x, None):
                dx = torch.full((T, K), 1.0, dtype=torch.bfloat16, device="cuda")
                dB = [torch.full((5, n, 24), FILL, device="cuda") for n in N] if weights else None
                aa.lora_linear_backward(dx, None, dB, c.dy, x, W, c.A, c.B, c.idx, c.rank, c.scale, ws,
                                        buf=buf if weights else None)
                got.append([dx, *(dB or [])])
            assert all(torch.equal(p, q) for p, q in zip(*got))


@pytest.mark.parametrize("T,L", [(4097, 1), (4700, 300), (8191, 7), (70000, 1024), (33000, 40)])
def test_tokens_without_a_slot_in_long_batches(T, L):
    """Their places behind the slots' rows, counted from the slots' runs: every
    row of y and dx is there once."""
    c = Layer(T, 16, (12,), 8, L, seed=T, stale=True, runs=L == 7)
    y_ref, y_tol, b_ref, b_tol = c.forward()
    assert 0 < sum(len(m) for _, _, m in c.members()) < T
    full, y, buf = run_forward(c)
    within(y, y_ref, y_tol, "y")
    within(buf, b_ref, b_tol, "buf")
    dx = torch.full((T, 16), FILL, dtype=torch.bfloat16, device="cuda")
    run_backward(c, dx)
    within(dx, *c.backward()[:2], "dx")


@pytest.mark.parametrize("p,q", [((4096, 64, (1020,), 8, 64), (7168, 64, (1024,), 8, 64)),
                                 ((5000, 72, (36,), 8, 3), (6000, 64, (64, 32), 16, 900)),
                                 ((1300, 136, (100, 36), 24, 5), (40, 4096, (4096,), 16, 8))], ids=str)
def test_layers_share_the_larger_workspace(p, q):
    """Forward and gradient of two layers in turn, the workspace as large as the
    larger one's: the bits of calls with workspaces of their own."""
    cs = [Layer(*s, seed=51 + i) for i, s in enumerate((p, q))]
    ws = max((aa.alloc_linear_workspace(*s) for s in (p, q)), key=lambda t: t.numel())

    def run(c, ws):
        y, buf = run_forward(c, ws=ws)[1:]
        dx = torch.empty((c.T, c.K), dtype=torch.bfloat16, device="cuda")
        return [y, buf, dx, *sum(run_backward(c, dx, ws=ws), [])]

    want = [run(c, None) for c in cs]
    for _ in range(2):
        for c, w in zip(cs, want):
            assert all(torch.equal(a, b) for a, b in zip(run(c, ws), w))
    aa.lora_workspace_check(ws)
