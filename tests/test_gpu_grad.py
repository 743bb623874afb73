"""lora_grad_norm and lora_grad_clip against their 64-bit definitions."""
import pytest
import torch

import adapter_apply_amd as aa

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
FILL = 7.0
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def definition(grads, L):
    total = torch.zeros((L,), dtype=torch.float64, device="cuda")
    for t in grads:
        total += t.double().square().reshape(L, -1).sum(1) if t.numel() else 0
    return total.sqrt()


def make(shapes, L, dtype, seed=0, std=1e-2):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn((L, *s), generator=g) * std).to(dtype).cuda() for s in shapes]


def check(grads, L, out=None):
    dt = grads[0].dtype
    ws = aa.alloc_grad_workspace(grads)
    norm = torch.full((L,), 7.0, device="cuda")
    aa.lora_grad_norm(norm, grads, ws)
    ref = definition(grads, L)
    # 64-bit sums, one rounding to fp32
    assert bool(((norm.double() - ref).abs() <= ref * 2.0 ** -24 * 1.001 + 1e-45).all()), (norm, ref)
    limit = (ref * torch.linspace(0.3, 1.4, L, device="cuda", dtype=torch.float64) + 1e-30).float()
    before = [t.clone() for t in grads]
    out = out or [torch.full_like(t, 7.0) for t in grads]
    aa.lora_grad_clip(out, grads, norm, limit)
    coef = (limit.double() / (norm.double() + 1e-6)).clamp(max=1.0)
    for o, t in zip(out, before):
        want = t.double() * coef.reshape(L, *[1] * (t.dim() - 1))
        # norm + 1e-6 and its constant, the quotient, the product, the storage rounding
        tol = want.abs() * (5 * 2.0 ** -24 + HALF[dt]) + 1e-44
        assert bool(((o.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,shapes", [
    (1, [(1,)]),
    (1, [(3,), (0,), (8191,), (8192,), (8193,), (16384 + 5,)]),
    (3, [(7,), (5, 11), (8, 1000), (1,)]),          # rows off 16 bytes
    (8, [(16, 512), (1024, 16)] * 3),
    (1024, [(8, 8)]),
    (2, [(3, i) for i in range(1, 230)]),           # several launches of tensors
    (1, [(1 << 22,), (12345, 77)]),
], ids=lambda v: str(v)[:30])
def test_norm_and_clip(L, shapes, dtype):
    check(make(shapes, L, DT[dtype], seed=len(shapes)), L)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_and_offset_pointers(dtype):
    L = 2
    base = make([(40001,)], 1, DT[dtype])[0].flatten()
    grads = [base[1:1 + L * 9000].view(L, 9000), base[20001:20001 + L * 777].view(L, 777)]
    keep = base.clone()
    check(grads, L, out=grads)
    assert torch.equal(base[:1], keep[:1]) and torch.equal(base[18001:20001], keep[18001:20001])
    assert torch.equal(base[20001 + L * 777:], keep[20001 + L * 777:])


def test_values_past_fp32_squares():
    """Squares that overflow or vanish in fp32 still give the norm."""
    grads = [torch.full((2, 1000), 1e30, device="cuda"), torch.zeros((2, 5), device="cuda")]
    grads[0][1] = 1e-30
    ws = aa.alloc_grad_workspace(grads)
    norm = torch.empty((2,), device="cuda")
    aa.lora_grad_norm(norm, grads, ws)
    ref = definition(grads, 2)
    assert bool(((norm.double() - ref).abs() <= ref * 2.0 ** -24 * 1.001).all())


def test_bad_slot_stays_alone():
    """An infinity or NaN in one slot's gradients changes no other slot."""
    grads = make([(50, 20), (333,)], 4, torch.float32)
    grads[0][1, 3, 4] = float("nan")
    grads[1][2, 5] = float("inf")
    norm, limit = torch.empty((4,), device="cuda"), torch.full((4,), 0.05, device="cuda")
    aa.lora_grad_norm(norm, grads, aa.alloc_grad_workspace(grads))
    assert bool(norm[1].isnan()) and bool(norm[2].isinf())
    out = [torch.empty_like(t) for t in grads]
    aa.lora_grad_clip(out, grads, norm, limit)
    for o, t in zip(out, grads):
        assert bool(o[1].isnan().all())
        finite = t[2].isfinite()
        assert bool((o[2][finite] == 0).all()) and bool(o[2][~finite].isnan().all())
        for i in (0, 3):
            want = t[i].double() * min(1.0, 0.05 / (float(norm[i]) + 1e-6))
            assert bool(((o[i].double() - want).abs() <= want.abs() * 6 * 2.0 ** -24).all())


def test_the_same_tensor_twice():
    """The norm counts it twice; the clip refuses it, also among empty tensors."""
    g = make([(50, 20), (333,), (0,)], 2, torch.float32)
    norm, once = torch.empty((2,), device="cuda"), torch.empty((2,), device="cuda")
    for n, t in ((once, g[:1]), (norm, [g[0], g[0]])):
        aa.lora_grad_norm(n, t, aa.alloc_grad_workspace(t))
    assert bool(((norm.double() - once.double() * 2 ** 0.5).abs() <= once.double() * 2.0 ** -23).all())
    keep = g[0].clone()
    with pytest.raises(Exception, match="shape|SHAPE|size"):
        aa.lora_grad_clip([g[0], g[1], g[0]], [g[0], g[1], g[0]], norm, norm * 0.1)
    assert torch.equal(g[0], keep)
    aa.lora_grad_clip([g[2], g[0], g[2]], [g[2], g[0], g[2]], once, once * 4)
    assert torch.equal(g[0], keep)


def test_graph_and_stream():
    grads = make([(50, 20), (9000,)], 3, torch.float32)
    ws = aa.alloc_grad_workspace(grads)
    norm, limit = torch.empty((3,), device="cuda"), torch.full((3,), 0.1, device="cuda")
    out = [torch.empty_like(t) for t in grads]

    def step():
        aa.lora_grad_norm(norm, grads, ws)
        aa.lora_grad_clip(out, grads, norm, limit)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    gen = torch.Generator().manual_seed(5)
    for rep in range(4):
        for t in grads:
            t.copy_(torch.randn(t.shape, generator=gen) * 1e-2)
        graph.replay()
        torch.cuda.synchronize()
        got = [norm.clone(), *[t.clone() for t in out]]
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step()
        st.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, [norm, *out])), rep


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,shapes", [
    (3, [(8192 * 700 + 5,)]),                       # 2103 chunks of one tensor
    (4, [(64, 128), (8200,)] * 200 + [(3,), (0,)]),   # a model: launches of 96 tensors, 2404 chunks
    (1024, [(3,), (8193,)]),                        # 3 chunks of each of 1024 slots
    (1, [(7,)] * 2100),
], ids=lambda v: str(v)[:30])
def test_more_chunks_than_are_counted(L, shapes, dtype):
    """Past 2048 chunks a launch of its own adds the partial sums; out of place,
    then in place."""
    grads = make(shapes, L, DT[dtype], seed=len(shapes))
    assert L * sum(-(-t[0].numel() // 8192) for t in grads) > 2048
    check(grads, L)
    check(grads, L, out=grads)


def test_norm_of_a_model_repeats_and_leaves_other_slots():
    """The same bits from call to call and from a graph; a NaN in one slot and
    the next call's small set (counted again on the same workspace) leave the
    others alone."""
    L = 4
    grads = make([(64, 128), (8200,)] * 200, L, torch.float32, seed=3)
    ws = aa.alloc_grad_workspace(grads)
    norm = torch.empty((L,), device="cuda")
    aa.lora_grad_norm(norm, grads, ws)
    want = norm.clone()
    small, ref = torch.empty((L,), device="cuda"), definition(grads[:3], L)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        aa.lora_grad_norm(norm, grads, ws)
    for _ in range(3):
        norm.fill_(FILL)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want)
        aa.lora_grad_norm(small, grads[:3], ws)
        assert bool(((small.double() - ref).abs() <= ref * 2.0 ** -24 * 1.001).all())
    grads[217][2, 5] = float("nan")
    aa.lora_grad_norm(norm, grads, ws)
    assert bool(norm[2].isnan()) and all(bool(norm[i] == want[i]) for i in (0, 1, 3))
