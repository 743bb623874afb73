"""Refusals of the layer, gradient, norm and clip entry points, without a GPU:
the C ABI returns the documented status before any launch (the pointers passed
here are never dereferenced), and the binding raises ValueError before the C
call."""
import ctypes as C

import pytest
import torch

import adapter_apply_amd as aa

FAKE = 0x7f0000001000
needs_no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                  reason="fake-pointer ABI checks run only without a GPU")


def ptrs(n, base=FAKE):
    return (C.c_void_p * n)(*[base + 0x100000 * i for i in range(n)])


def i64(*v):
    return (C.c_int64 * len(v))(*v)


BASE = dict(y=FAKE, ldy=6144, x=FAKE, ldx=4096, T=300, K=4096, W=FAKE, ldw=4096, bias=None,
            A=ptrs(3), B=ptrs(3), N=i64(4096, 1024, 1024), S=3, L=8, R=16, idx=FAKE, rank=FAKE,
            scale=FAKE, buf=None, dt=aa.LORA_DT_BF16, flags=0, ws=FAKE, wsb=1 << 40,
            dx=FAKE, lddx=4096, dA=ptrs(3), dB=ptrs(3))


def forward(**kw):
    a = dict(BASE, **kw)
    return aa.lib().lora_linear(a["y"], a["ldy"], a["x"], a["ldx"], a["T"], a["K"], a["W"], a["ldw"],
                                a["bias"], a["A"], a["B"], a["N"], a["S"], a["L"], a["R"], a["idx"],
                                a["rank"], a["scale"], a["buf"], a["dt"], a["flags"], a["ws"],
                                a["wsb"], None)


def backward(**kw):
    a = dict(BASE, **kw)
    return aa.lib().lora_linear_backward(
        a["dx"], a["lddx"], a["dA"], a["dB"], a["y"], a["ldy"], a["x"], a["ldx"], a["T"], a["K"],
        a["W"], a["ldw"], a["A"], a["B"], a["N"], a["S"], a["L"], a["R"], a["idx"], a["rank"],
        a["scale"], a["buf"], a["dt"], a["flags"], a["ws"], a["wsb"], None)


def hole(n, at):
    p = ptrs(n)
    p[at] = None
    return p


BOTH = [
    (dict(T=-1), aa.LORA_E_SHAPE),
    (dict(T=1 << 22), aa.LORA_E_SHAPE),
    (dict(L=0), aa.LORA_E_SHAPE),
    (dict(L=1025), aa.LORA_E_SHAPE),
    (dict(R=0), aa.LORA_E_RANK),
    (dict(R=520), aa.LORA_E_RANK),
    (dict(R=12), aa.LORA_E_ALIGN),
    (dict(S=0), aa.LORA_E_SLICES),
    (dict(S=9), aa.LORA_E_SLICES),
    (dict(dt=aa.LORA_DT_F32), aa.LORA_E_DTYPE),
    (dict(dt=7), aa.LORA_E_DTYPE),
    (dict(K=0), aa.LORA_E_SHAPE),
    (dict(K=4100), aa.LORA_E_SHAPE),
    (dict(K=4092), aa.LORA_E_ALIGN),
    (dict(ldx=4100), aa.LORA_E_ALIGN),
    (dict(ldx=4088), aa.LORA_E_SHAPE),
    (dict(ldw=4088), aa.LORA_E_SHAPE),
    (dict(ldw=4100), aa.LORA_E_ALIGN),
    (dict(N=None), aa.LORA_E_NULL),
    (dict(N=i64(4096, 0, 1024)), aa.LORA_E_SHAPE),
    (dict(N=i64(4096, 1022, 1024)), aa.LORA_E_ALIGN),
    (dict(N=i64(1 << 25, 4, 4), ldy=1 << 30), aa.LORA_E_SHAPE),
    (dict(ldy=6140), aa.LORA_E_SHAPE),
    (dict(ldy=6146), aa.LORA_E_ALIGN),
    (dict(y=None), aa.LORA_E_NULL),
    (dict(y=FAKE + 8), aa.LORA_E_ALIGN),
    (dict(x=None), aa.LORA_E_NULL),
    (dict(x=FAKE + 2), aa.LORA_E_ALIGN),
    (dict(W=FAKE + 8), aa.LORA_E_ALIGN),
    (dict(idx=None), aa.LORA_E_NULL),
    (dict(scale=None), aa.LORA_E_NULL),
    (dict(A=None), aa.LORA_E_NULL),
    (dict(A=hole(3, 1)), aa.LORA_E_NULL),
    (dict(B=hole(3, 2)), aa.LORA_E_NULL),
    (dict(A=ptrs(3, FAKE + 8)), aa.LORA_E_ALIGN),
    (dict(buf=FAKE + 8), aa.LORA_E_ALIGN),
    (dict(ws=None), aa.LORA_E_NULL),
    (dict(ws=FAKE + 16), aa.LORA_E_ALIGN),
    (dict(wsb=1024), aa.LORA_E_WORKSPACE),
]


@needs_no_gpu
@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(W=None), aa.LORA_E_NULL),
    (dict(bias=FAKE + 1), aa.LORA_E_ALIGN),
], ids=str)
def test_forward_refusals(kw, code):
    assert forward(**kw) == code


@needs_no_gpu
@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(ldy=6148), aa.LORA_E_ALIGN),               # whole 16-byte units when N % 8 == 0
    (dict(lddx=4088), aa.LORA_E_SHAPE),
    (dict(lddx=4100), aa.LORA_E_ALIGN),
    (dict(dx=FAKE + 8), aa.LORA_E_ALIGN),
    (dict(dx=None, dA=None, dB=None), aa.LORA_E_NULL),
    (dict(dA=hole(3, 0)), aa.LORA_E_NULL),
    (dict(dB=ptrs(3, FAKE + 4)), aa.LORA_E_ALIGN),
], ids=str)
def test_backward_refusals(kw, code):
    assert backward(**kw) == code


@needs_no_gpu
def test_no_tokens_needs_no_pointers():
    assert forward(T=0, y=None, x=None, W=None, ws=None, wsb=0) == aa.LORA_OK
    assert backward(T=0, y=None, x=None, ws=None, wsb=0,
                    flags=aa.LORA_FLAG_ACCUMULATE) == aa.LORA_OK


@pytest.mark.parametrize("grow", [dict(T=1000), dict(T=8192), dict(K=8192), dict(R=64), dict(L=64),
                                  dict(N=(4096, 1024, 1028)), dict(N=(4096, 1024, 1024, 8))])
def test_workspace_grows_with_every_size(grow):
    base = dict(T=300, K=4096, N=(4096, 1024, 1024), R=16, L=8)
    small = aa.lora_linear_workspace_size(**base)
    assert small % 256 == 0 and aa.lora_linear_workspace_size(**dict(base, **grow)) >= small


def test_workspace_size_refusals():
    n = C.c_size_t(0)
    size = aa.lib().lora_linear_workspace_size
    assert size(1, 64, i64(64), 1, 16, 4, None) == aa.LORA_E_NULL
    assert size(1, 64, None, 1, 16, 4, C.byref(n)) == aa.LORA_E_NULL
    assert size(1, 64, i64(62), 1, 16, 4, C.byref(n)) == aa.LORA_E_ALIGN
    assert size(1, 0, i64(64), 1, 16, 4, C.byref(n)) == aa.LORA_E_SHAPE
    assert size(0, 64, i64(64), 1, 16, 4, C.byref(n)) == aa.LORA_OK
    gsize = aa.lib().lora_grad_workspace_size
    assert gsize(i64(5, 0), 2, 3, C.byref(n)) == aa.LORA_OK and n.value % 256 == 0 and n.value > 0
    assert gsize(i64(-1), 1, 3, C.byref(n)) == aa.LORA_E_SHAPE
    assert gsize(i64(1), 1, 0, C.byref(n)) == aa.LORA_E_SHAPE
    assert gsize(None, 1, 1, C.byref(n)) == aa.LORA_E_NULL
    assert gsize(None, 0, 1, C.byref(n)) == aa.LORA_OK


@needs_no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(norm=None), aa.LORA_E_NULL),
    (dict(norm=FAKE + 2), aa.LORA_E_ALIGN),
    (dict(g=None), aa.LORA_E_NULL),
    (dict(g=hole(2, 1)), aa.LORA_E_NULL),
    (dict(g=ptrs(2, FAKE + 2)), aa.LORA_E_ALIGN),
    (dict(m=None), aa.LORA_E_NULL),
    (dict(m=i64(4, -4)), aa.LORA_E_SHAPE),
    (dict(n=-1), aa.LORA_E_SHAPE),
    (dict(L=0), aa.LORA_E_SHAPE),
    (dict(L=1025), aa.LORA_E_SHAPE),
    (dict(dt=5), aa.LORA_E_DTYPE),
], ids=str)
def test_norm_and_clip_refusals(kw, code):
    a = dict(norm=FAKE, g=ptrs(2), m=i64(64, 64), n=2, L=3, dt=aa.LORA_DT_F32, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    lib = aa.lib()
    assert lib.lora_grad_norm(a["norm"], a["g"], a["m"], a["n"], a["L"], a["dt"], a["ws"], a["wsb"],
                              None) == code
    assert lib.lora_grad_clip(a["g"], a["g"], a["m"], a["n"], a["L"], a["norm"], FAKE, a["dt"],
                              None) == code


@needs_no_gpu
def test_norm_and_clip_more_refusals():
    lib, m = aa.lib(), i64(64, 64)
    args = (FAKE, ptrs(2), m, 2, 3, aa.LORA_DT_F32)
    assert lib.lora_grad_norm(*args, None, 1 << 20, None) == aa.LORA_E_NULL
    assert lib.lora_grad_norm(*args, FAKE + 8, 1 << 20, None) == aa.LORA_E_ALIGN
    assert lib.lora_grad_norm(*args, FAKE, 8, None) == aa.LORA_E_WORKSPACE
    clip = lambda out, mx: lib.lora_grad_clip(out, ptrs(2), m, 2, 3, FAKE, mx, aa.LORA_DT_F32, None)
    assert clip(ptrs(2), None) == aa.LORA_E_NULL
    assert clip(None, FAKE) == aa.LORA_E_NULL
    assert clip(hole(2, 0), FAKE) == aa.LORA_E_NULL


@needs_no_gpu
def test_equal_outputs_are_refused():
    """Nothing is launched when two outputs are one: the same gradient twice, a
    tensor listed twice for the clip, an output that is another one's input."""
    other = dict(dx=FAKE + 0x4000000, dA=ptrs(3, FAKE + 0x1000000), dB=ptrs(3, FAKE + 0x2000000))
    for kw in (dict(dA=ptrs(3, FAKE + 0x2000000)), dict(dx=FAKE + 0x1100000),
               dict(dA=(C.c_void_p * 3)(FAKE, FAKE + 4096, FAKE))):
        assert backward(**dict(other, **kw)) == aa.LORA_E_SHAPE
    lib = aa.lib()

    def clip(out, g, m):
        arr = lambda v: (C.c_void_p * len(v))(*v)
        return lib.lora_grad_clip(arr(out), arr(g), i64(*m), len(m), 3, FAKE, FAKE, aa.LORA_DT_F32, None)

    at = [FAKE + 4096 * i for i in range(1, 400)]
    assert clip(at[:2] + at[:1], at[:2] + at[:1], (64, 64, 64)) == aa.LORA_E_SHAPE
    assert clip(at[:2], at[1:3], (64, 64)) == aa.LORA_E_SHAPE
    assert clip([at[5], at[5]], at[:2], (64, 64)) == aa.LORA_E_SHAPE
    assert clip(at[:200] + [at[77]], at[200:] + [at[0]] * 2, (8,) * 201) == aa.LORA_E_SHAPE


# --------------------------------------------------------------------------
# the binding
# --------------------------------------------------------------------------

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
T, K, L, R, N = 12, 64, 3, 16, (32, 16)


def tensors(**over):
    a = dict(y=torch.zeros(T, sum(N), dtype=BF), x=torch.zeros(T, K, dtype=BF),
             W=torch.zeros(sum(N), K, dtype=BF), bias=None, buf=None,
             A=[torch.zeros(L, R, K, dtype=BF) for _ in N],
             B=[torch.zeros(L, n, R, dtype=BF) for n in N], idx=torch.zeros(T, dtype=I32),
             rank=torch.full((L,), R, dtype=I32), scale=torch.ones(L),
             ws=torch.zeros(4096, dtype=torch.uint8), dx=torch.zeros(T, K, dtype=BF),
             dA=[torch.zeros(L, R, K) for _ in N], dB=[torch.zeros(L, n, R) for n in N])
    a.update(over)
    return a


def call_forward(a):
    aa.lora_linear(a["y"], a["x"], a["W"], a["A"], a["B"], a["idx"], a["rank"], a["scale"], a["ws"],
                   bias=a["bias"], buf=a["buf"])


def call_backward(a):
    aa.lora_linear_backward(a["dx"], a["dA"], a["dB"], a["y"], a["x"], a["W"], a["A"], a["B"],
                            a["idx"], a["rank"], a["scale"], a["ws"], buf=a["buf"])


BAD = {
    "fp32 x": dict(x=torch.zeros(T, K)),
    "fp32 y": dict(y=torch.zeros(T, sum(N))),
    "narrow y": dict(y=torch.zeros(T, sum(N) - 4, dtype=BF)),
    "short y": dict(y=torch.zeros(T - 1, sum(N), dtype=BF)),
    "W of other K": dict(W=torch.zeros(sum(N), K + 8, dtype=BF)),
    "W of other N": dict(W=torch.zeros(sum(N) + 4, K, dtype=BF)),
    "fp32 W": dict(W=torch.zeros(sum(N), K)),
    "transposed W": dict(W=torch.zeros(K, sum(N), dtype=BF).T),
    "int64 idx": dict(idx=torch.zeros(T, dtype=torch.int64)),
    "short rank": dict(rank=torch.zeros(L - 1, dtype=I32)),
    "bf16 buf": dict(buf=torch.zeros(2, T, R, dtype=BF)),
    "short buf": dict(buf=torch.zeros(1, T, R)),
    "B count": dict(B=[torch.zeros(L, 32, R, dtype=BF)]),
    "A of other L": dict(A=[torch.zeros(L + 1, R, K, dtype=BF)] * 2),
}


@pytest.mark.parametrize("name", sorted(BAD))
def test_binding_refuses(name):
    for call in (call_forward, call_backward):
        with pytest.raises(ValueError):
            call(tensors(**BAD[name]))


@pytest.mark.parametrize("over", [
    dict(bias=torch.zeros(sum(N))), dict(bias=torch.zeros(sum(N) + 1, dtype=BF))], ids=["dtype", "size"])
def test_forward_binding_refuses(over):
    with pytest.raises(ValueError, match="bias"):
        call_forward(tensors(**over))


same = torch.zeros(L, R, K)


@pytest.mark.parametrize("over", [
    dict(dx=torch.zeros(T, K)), dict(dx=torch.zeros(T, K + 8, dtype=BF)),
    dict(dA=[torch.zeros(L, R, K, dtype=BF)] * 2), dict(dA=[torch.zeros(L, R, K)]),
    dict(dB=[torch.zeros(L, 32, R)] * 2), dict(dA=[same, same])], ids=range(6))
def test_backward_binding_refuses(over):
    with pytest.raises(ValueError):
        call_backward(tensors(**over))


def test_binding_refuses_cpu_tensors():
    for call in (call_forward, call_backward):
        with pytest.raises(ValueError, match="GPU"):
            call(tensors())
    g = [torch.zeros(L, 8)]
    with pytest.raises(ValueError, match="GPU"):
        aa.lora_grad_norm(torch.zeros(L), g, torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="GPU"):
        aa.lora_grad_clip(g, g, torch.zeros(L), torch.zeros(L))


@pytest.mark.parametrize("grads", [
    [], [torch.zeros(L, 8, dtype=torch.float16)], [torch.zeros(L, 8), torch.zeros(L + 1, 8)],
    [torch.zeros(L, 8), torch.zeros(L, 8, dtype=BF)], [torch.zeros(8, L).T],
    [torch.zeros(())], [torch.zeros(L, 8), torch.zeros(())], [torch.zeros(0, 8)]], ids=range(8))
def test_grad_binding_refuses(grads):
    with pytest.raises(ValueError):
        aa.lora_grad_norm(torch.zeros(L), grads, torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError):
        aa.lora_grad_clip(grads, grads, torch.zeros(L), torch.zeros(L))


def test_clip_binding_refuses_other_outputs():
    g = [torch.zeros(L, 8), torch.zeros(L, 4)]
    for out in ([g[0]], [g[1], g[0]], [t.to(BF) for t in g]):
        with pytest.raises(ValueError):
            aa.lora_grad_clip(out, g, torch.zeros(L), torch.zeros(L))


@needs_no_gpu
@pytest.mark.parametrize("n", [2, 2047, 2048, 2049, 5000, 9001])
def test_equal_outputs_are_found_in_long_lists(n):
    """One pair of equal addresses among n tensors, at both ends and in the
    middle: two outputs, or an output and another tensor's gradient."""
    at = [FAKE + 4096 * i for i in range(1, 2 * n + 1)]
    m, lib = i64(*[8] * n), aa.lib()
    for i, j in {(0, n - 1), (n // 2, n - 1), (n - 2, n - 1), (0, n // 2 or 1)}:
        if i == j:
            continue
        out = (C.c_void_p * n)(*at[:n])
        grad = (C.c_void_p * n)(*at[n:])
        for arr, v in ((out, out[i]), (grad, out[i])):
            keep, arr[j] = arr[j], v
            assert lib.lora_grad_clip(out, grad, m, n, 3, FAKE, FAKE, aa.LORA_DT_F32,
                                      None) == aa.LORA_E_SHAPE, (n, i, j)
            arr[j] = keep


@needs_no_gpu
def test_clip_allocates_nothing():
    """The check of the outputs needs no host memory: with the address space
    held at its size it still finds the pair."""
    import os
    import subprocess
    import sys
    code = f"""
import ctypes as C, resource
import adapter_apply_amd as aa
n = 100000
out = (C.c_void_p * n)(*[{FAKE} + 4096 * i for i in range(n)])
out[n - 1] = out[1]
m = (C.c_int64 * n)(*[8] * n)
clip = aa.lib().lora_grad_clip
args = (out, out, m, n, 3, {FAKE}, {FAKE}, aa.LORA_DT_F32, None)
pages = int(open("/proc/self/statm").read().split()[0])
resource.setrlimit(resource.RLIMIT_AS, (pages * resource.getpagesize() + 65536,) * 2)
code = clip(*args)
raise SystemExit(0 if code == aa.LORA_E_SHAPE else 100 + code)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])


@pytest.mark.parametrize("alloc", [
    lambda d: aa.alloc_workspace(8, 64, 1, 16, 2, device=d),
    lambda d: aa.alloc_moe_workspace(8, 2, 1, 16, 2, 4, device=d),
    lambda d: aa.alloc_linear_workspace(8, 64, [32], 16, 2, device=d),
    lambda d: aa.alloc_grad_workspace([torch.zeros(2, 8)], device=d)], ids=range(4))
def test_workspace_is_cleared_on_its_own_device(alloc, monkeypatch):
    """The fill runs with the workspace's device current, whatever the caller's
    current device is, and the caller's comes back."""
    current, cleared = [0], []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *exc):
            current.pop()

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(aa, "lora_workspace_init", lambda ws, stream=None: cleared.append((current[-1], ws.device)))
    ws = alloc("cpu")                           # (stands for a GPU that is not the current one)
    assert cleared == [(ws.device, ws.device)] and current == [0]
    assert ws.data_ptr() % 256 == 0


@needs_no_gpu
def test_backward_needs_x_only_where_it_is_read():
    """dA, and dB without a saved u: else a call without x gets as far as its
    first launch (which fails without a GPU)."""
    for kw in (dict(), dict(dB=None), dict(dA=None), dict(dx=None, dB=None), dict(dA=None, dx=None),
               dict(dB=None, buf=FAKE)):
        assert backward(x=None, ldx=0, **kw) == aa.LORA_E_NULL
    for kw in (dict(dA=None, dB=None), dict(dA=None, buf=FAKE), dict(dA=None, dx=None, buf=FAKE),
               dict(dA=None, dB=None, W=None)):
        assert backward(x=None, ldx=0, **dict(dict(dx=FAKE + 0x4000000), **kw)) == aa.LORA_E_LAUNCH
    assert backward(x=None, ldx=0, K=4092, dA=None, dB=None) == aa.LORA_E_ALIGN


def test_backward_binding_needs_x_only_where_it_is_read():
    for over in (dict(), dict(dB=None), dict(dA=None)):
        with pytest.raises(ValueError, match="x is needed"):
            call_backward(tensors(x=None, **over))
    for over in (dict(dA=None, dB=None), dict(dA=None, buf=torch.zeros(2, T, R))):
        with pytest.raises(ValueError, match="GPU"):      # (the next check)
            call_backward(tensors(x=None, **over))
    for over in (dict(dx=torch.zeros(T + 1, K, dtype=BF)), dict(W=torch.zeros(sum(N), K + 8, dtype=BF))):
        with pytest.raises(ValueError, match="shape"):
            call_backward(tensors(x=None, dA=None, dB=None, **over))
    for name in ("x", "W"):
        with pytest.raises(ValueError, match="x and W are needed"):
            call_forward(tensors(**{name: None}))


@pytest.mark.parametrize("dy", [torch.zeros((), dtype=BF), torch.zeros(T, dtype=BF), torch.zeros(T, sum(N))],
                         ids=["no dims", "one dim", "fp32"])
def test_backward_binding_refuses_dy_without_x(dy):
    with pytest.raises(ValueError, match="dy"):
        call_backward(tensors(x=None, dA=None, dB=None, y=dy))
