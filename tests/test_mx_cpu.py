"""Refusals of the microscaled entry points without a GPU (the pointers passed
here are never dereferenced), and the tests' own 64-bit formats against values
written out by hand."""
import ctypes as C

import pytest
import torch

import adapter_apply_amd as aa
from tests import mx_util
from tests.test_layer_cpu import FAKE, hole, i64, needs_no_gpu, ptrs

bf16 = torch.bfloat16


# --------------------------------------------------------------------------
# the formats
# --------------------------------------------------------------------------

def test_fp4_by_hand():
    x = torch.zeros((1, 32))
    x[0, :12] = torch.tensor([6.0, 7.0, 5.0, 2.5, 3.5, 0.25, 0.75, 1.25, 1.75, -0.3, -6.5, 0.2])
    c, s = mx_util.quantize(x, aa.LORA_MX_FP4)
    assert s.tolist() == [[127, 0, 0, 0]]
    v = mx_util.restore(c, s, 32, aa.LORA_MX_FP4)[0, :12].tolist()
    assert v == [6.0, 6.0, 4.0, 2.0, 4.0, 0.0, 1.0, 1.0, 2.0, -0.5, -6.0, 0.0]
    assert c[0, :2].tolist() == [7 | 7 << 4, 6 | 4 << 4]


def test_int8_by_hand():
    x = torch.zeros((1, 40))
    x[0, :4] = torch.tensor([1.5, -1.999, 0.5 / 64, 1.5 / 64])
    x[0, 32] = -3.0e-39
    c, s = mx_util.quantize(x, aa.LORA_MX_INT8)
    assert s.tolist() == [[127, 0, 0, 0]]
    assert c.view(torch.int8)[0, :4].tolist() == [96, -127, 0, 2]
    assert mx_util.restore(c, s, 40, aa.LORA_MX_INT8)[0, 0] == 1.5


def test_non_finite_blocks():
    x = torch.ones((1, 96))
    x[0, 3], x[0, 70] = float("inf"), float("nan")
    for fmt in (aa.LORA_MX_FP4, aa.LORA_MX_INT8):
        c, s = mx_util.quantize(x, fmt)
        v = mx_util.restore(c, s, 96, fmt)
        assert s[0, :3].tolist()[0] == 255 and s[0, 2] == 255
        assert v[0, :32].isnan().all() and (v[0, 32:64] == 1).all() and v[0, 64:].isnan().all()


# --------------------------------------------------------------------------
# the C ABI
# --------------------------------------------------------------------------

STORE = dict(codes=FAKE, ldc=2048, scales=FAKE, lds=128, x=FAKE, ldx=4096, M=100, K=4096,
             fmt=aa.LORA_MX_FP4, dt=aa.LORA_DT_BF16)


def store(quantize, **kw):
    a = dict(STORE, **kw)
    mx, x = (a["codes"], a["ldc"], a["scales"], a["lds"]), (a["x"], a["ldx"])
    f = aa.lib().lora_mx_quantize if quantize else aa.lib().lora_mx_dequantize
    return f(*(mx + x if quantize else x + mx), a["M"], a["K"], a["fmt"], a["dt"], None)


STORE_BAD = [
    (dict(M=-1), aa.LORA_E_SHAPE),
    (dict(M=1 << 26), aa.LORA_E_SHAPE),
    (dict(M=1 << 22), aa.LORA_E_SHAPE),
    (dict(M=1 << 27, K=8, ldx=8, ldc=16, lds=4), aa.LORA_E_SHAPE),
    (dict(M=1 << 62), aa.LORA_E_SHAPE),
    (dict(K=0), aa.LORA_E_SHAPE),
    (dict(K=4100, ldx=4104, lds=132, ldc=2080), aa.LORA_E_ALIGN),
    (dict(ldx=4088), aa.LORA_E_SHAPE),
    (dict(ldx=4100), aa.LORA_E_ALIGN),
    (dict(ldx=4098, dt=aa.LORA_DT_F32), aa.LORA_E_ALIGN),
    (dict(ldc=2032), aa.LORA_E_SHAPE),
    (dict(fmt=aa.LORA_MX_INT8), aa.LORA_E_SHAPE),
    (dict(ldc=2056), aa.LORA_E_ALIGN),
    (dict(lds=124), aa.LORA_E_SHAPE),
    (dict(lds=130), aa.LORA_E_ALIGN),
    (dict(K=4104, ldx=4104, ldc=2064, lds=129), aa.LORA_E_SHAPE),
    (dict(fmt=2), aa.LORA_E_DTYPE),
    (dict(fmt=-1), aa.LORA_E_DTYPE),
    (dict(dt=2), aa.LORA_E_DTYPE),
    (dict(codes=None), aa.LORA_E_NULL),
    (dict(scales=None), aa.LORA_E_NULL),
    (dict(x=None), aa.LORA_E_NULL),
    (dict(codes=FAKE + 8), aa.LORA_E_ALIGN),
    (dict(scales=FAKE + 2), aa.LORA_E_ALIGN),
    (dict(x=FAKE + 8), aa.LORA_E_ALIGN),
]


@needs_no_gpu
@pytest.mark.parametrize("quantize", [True, False])
@pytest.mark.parametrize("kw,code", STORE_BAD, ids=str)
def test_store_refuses(kw, code, quantize):
    assert store(quantize, **kw) == code


@needs_no_gpu
def test_store_of_no_rows_launches_nothing():
    for q in (True, False):
        assert store(q, M=0, codes=None, scales=None, x=None) == aa.LORA_OK


BASE = dict(y=FAKE, ldy=6144, x=FAKE, ldx=4096, xs=None, ldxs=0, T=300, K=4096, W=FAKE, ldw=2048,
            Ws=FAKE, ldws=128, bias=None, A=ptrs(3), B=ptrs(3), N=i64(4096, 1024, 1024), S=3, L=8, R=16,
            idx=FAKE, rank=FAKE, scale=FAKE, buf=None, dt=aa.LORA_DT_BF16, flags=0, ws=FAKE,
            wsb=1 << 40, dx=FAKE, lddx=4096, dA=ptrs(3), dB=ptrs(3, FAKE + (1 << 32)))


def forward(**kw):
    a = dict(BASE, **kw)
    return aa.lib().lora_linear_mx(
        a["y"], a["ldy"], a["x"], a["ldx"], a["T"], a["K"], a["W"], a["ldw"], a["Ws"], a["ldws"], a["bias"],
        a["A"], a["B"], a["N"], a["S"], a["L"], a["R"], a["idx"], a["rank"], a["scale"], a["buf"], a["dt"],
        a["flags"], a["ws"], a["wsb"], None)


def backward(**kw):
    a = dict(BASE, **kw)
    return aa.lib().lora_linear_mx_backward(
        a["dx"], a["lddx"], a["dA"], a["dB"], a["y"], a["ldy"], a["x"], a["ldx"], a["xs"], a["ldxs"],
        a["T"], a["K"], a["W"], a["ldw"], a["Ws"], a["ldws"], a["A"], a["B"], a["N"], a["S"], a["L"],
        a["R"], a["idx"], a["rank"], a["scale"], a["buf"], a["dt"], a["flags"], a["ws"], a["wsb"], None)


BOTH = [
    (dict(T=-1), aa.LORA_E_SHAPE),
    (dict(R=12), aa.LORA_E_ALIGN),
    (dict(S=9), aa.LORA_E_SLICES),
    (dict(dt=aa.LORA_DT_F32), aa.LORA_E_DTYPE),
    (dict(K=4092), aa.LORA_E_ALIGN),
    (dict(ldx=4088), aa.LORA_E_SHAPE),
    (dict(ldw=2032), aa.LORA_E_SHAPE),
    (dict(ldw=2056), aa.LORA_E_ALIGN),
    (dict(ldws=124), aa.LORA_E_SHAPE),
    (dict(ldws=130), aa.LORA_E_ALIGN),
    (dict(W=FAKE + 8), aa.LORA_E_ALIGN),
    (dict(Ws=FAKE + 2), aa.LORA_E_ALIGN),
    (dict(y=None), aa.LORA_E_NULL),
    (dict(idx=None), aa.LORA_E_NULL),
    (dict(scale=None), aa.LORA_E_NULL),
    (dict(A=hole(3, 1)), aa.LORA_E_NULL),
    (dict(B=hole(3, 2)), aa.LORA_E_NULL),
    (dict(ws=None), aa.LORA_E_NULL),
    (dict(wsb=4096), aa.LORA_E_WORKSPACE),
]


@needs_no_gpu
@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("kw,code", BOTH, ids=str)
def test_layer_refuses(kw, code, call):
    assert call(**kw) == code


@needs_no_gpu
@pytest.mark.parametrize("kw,code", [(dict(Ws=None), aa.LORA_E_NULL), (dict(W=None), aa.LORA_E_NULL),
                                     (dict(x=None), aa.LORA_E_NULL)], ids=str)
def test_forward_refuses(kw, code):
    assert forward(**kw) == code


X8 = dict(xs=FAKE, ldxs=128, ldx=4096, buf=FAKE)


@needs_no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(X8, buf=None), aa.LORA_E_NULL),
    (dict(X8, x=None), aa.LORA_E_NULL),
    (dict(X8, ldx=4080), aa.LORA_E_SHAPE),
    (dict(X8, ldx=4104), aa.LORA_E_ALIGN),
    (dict(X8, ldxs=124), aa.LORA_E_SHAPE),
    (dict(X8, ldxs=129), aa.LORA_E_ALIGN),
    (dict(X8, x=FAKE + 8), aa.LORA_E_ALIGN),
    (dict(X8, xs=FAKE + 1), aa.LORA_E_ALIGN),
    (dict(Ws=None), aa.LORA_E_SHAPE),                 # bf16 W: ldw in elements
    (dict(dx=None, dA=None, dB=None), aa.LORA_E_NULL),
    (dict(dA=ptrs(3), dB=ptrs(3)), aa.LORA_E_SHAPE),
], ids=str)
def test_backward_refuses(kw, code):
    assert backward(**kw) == code


@needs_no_gpu
def test_no_tokens():
    assert forward(T=0) == aa.LORA_OK
    assert backward(T=0, dA=None, dB=None) == aa.LORA_OK


def test_workspace_size():
    f = aa.lora_linear_mx_workspace_size
    assert f(256, 4096, [4096, 1024, 1024], 16, 8) >= aa.lora_linear_workspace_size(
        256, 4096, [4096, 1024, 1024], 16, 8)
    with pytest.raises(aa.LoraError):
        f(-1, 4096, [4096], 16, 8)
    with pytest.raises(aa.LoraError):
        f(1, 4096, [4094], 16, 8)
    n = C.c_size_t(0)
    assert aa.lib().lora_linear_mx_workspace_size(1, 64, None, 1, 8, 1, C.byref(n)) == aa.LORA_E_NULL
    assert aa.lib().lora_linear_mx_workspace_size(1, 64, i64(64), 1, 8, 1, None) == aa.LORA_E_NULL


# T, N, R, L, whether the few-token kernels take it
@pytest.mark.parametrize("T,N,R,L,few", [
    (1, (4, ), 8, 1, True), (16, (4096, 1024, 1024), 16, 8, True), (16, (64,), 512, 1024, True),
    (17, (4096,), 16, 8, True), (32, (4096, 1024, 1024), 16, 8, False), (32, (2600,), 8, 9, True),
    (33, (65536,), 8, 1, False), (1, (65540,), 8, 1, False), (1, (64,) * 8, 136, 4, False)])
def test_few_tokens_rule(T, N, R, L, few):
    f = aa.lib()._ZN2aa6mx_fewEiPKliii
    f.restype, f.argtypes = C.c_bool, [C.c_int32, C.POINTER(C.c_int64), C.c_int32, C.c_int32, C.c_int32]
    assert f(T, i64(*N), len(N), R, L) is few


# --------------------------------------------------------------------------
# the binding
# --------------------------------------------------------------------------

def test_alloc_shapes():
    c, s = aa.alloc_mx(5, 1352, aa.LORA_MX_FP4, device="cpu")
    assert c.shape == (5, 688) and s.shape == (5, 44) and c.dtype is s.dtype is torch.uint8
    c, s = aa.alloc_mx(0, 64, aa.LORA_MX_INT8, device="cpu")
    assert c.shape == (0, 64) and s.shape == (0, 4)
    with pytest.raises(ValueError):
        aa.alloc_mx(1, 64, 2, device="cpu")


def test_binding_store():
    x = torch.zeros((4, 64), dtype=bf16)
    c, s = aa.alloc_mx(4, 64, aa.LORA_MX_FP4, device="cpu")
    bad = [
        dict(x=x.half()), dict(x=x[0]), dict(x=x[:, ::2]), dict(x=x[:3]), dict(x=torch.zeros((4, 72), dtype=bf16)),
        dict(codes=c.view(torch.int8)), dict(codes=c[:, :16]), dict(codes=c[:2]), dict(scales=s[:, :2]),
        dict(scales=s.view(torch.int8)), dict(fmt=aa.LORA_MX_INT8), dict(fmt=7),
        dict(codes=torch.zeros((4, 64), dtype=torch.uint8)[:, ::2]),
        dict(),                                           # on the CPU
    ]
    for kw in bad:
        a = dict(dict(x=x, codes=c, scales=s, fmt=aa.LORA_MX_FP4), **kw)
        with pytest.raises(ValueError):
            aa.lora_mx_quantize(a["codes"], a["scales"], a["x"], a["fmt"])
        with pytest.raises(ValueError):
            aa.lora_mx_dequantize(a["x"], a["codes"], a["scales"], a["fmt"])


def binding_layer():
    z = lambda *s, dt=bf16: torch.zeros(s, dtype=dt)
    u8 = torch.uint8
    return dict(y=z(6, 40), x=z(6, 64), W=z(40, 32, dt=u8), W_scales=z(40, 4, dt=u8), A=[z(2, 8, 64)],
                B=[z(2, 40, 8)], idx=z(6, dt=torch.int32), rank=z(2, dt=torch.int32), scale=z(2, dt=torch.float32),
                ws=z(256, dt=u8), bias=None, buf=z(1, 6, 8, dt=torch.float32))


def test_binding_forward():
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)
    for kw in [dict(W=z(40, 64, dt=bf16)), dict(W=z(40, 48)), dict(W=z(36, 32)), dict(W_scales=z(40, 2)),
               dict(W_scales=None), dict(W=None), dict(x=None), dict(x=z(6, 64)), dict(bias=z(36, dt=bf16)),
               dict(buf=z(1, 6, 16, dt=torch.float32)), dict()]:
        a = dict(binding_layer(), **kw)
        with pytest.raises(ValueError):
            aa.lora_linear_mx(a["y"], a["x"], a["W"], a["W_scales"], a["A"], a["B"], a["idx"], a["rank"],
                              a["scale"], a["ws"], bias=a["bias"], buf=a["buf"])


def test_binding_backward():
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)
    f32 = torch.float32
    x8 = dict(x=z(6, 64), x_scales=z(6, 4))
    for kw in [dict(W=None), dict(W_scales=None), dict(x8, x=None), dict(x8, buf=None), dict(x8, x=z(5, 64)),
               dict(x8, x=z(6, 32)), dict(x8, x_scales=z(6, 8)), dict(x8, x=z(6, 64, dt=bf16)),
               dict(x=z(6, 64)), dict(x8, W=z(40, 48)), dict(W=z(40, 64, dt=bf16)), dict(dx=z(6, 72, dt=bf16)),
               dict(dA=[z(2, 8, 64)]), dict(dB=[z(2, 40, 16, dt=f32)]), dict(x=None), dict(x8)]:
        a = dict(binding_layer(), dx=z(6, 64, dt=bf16), dA=[z(2, 8, 64, dt=f32)], dB=[z(2, 40, 8, dt=f32)],
                 x_scales=None)
        a.update(kw)
        with pytest.raises(ValueError):
            aa.lora_linear_mx_backward(a["dx"], a["dA"], a["dB"], a["y"], a["x"], a["W"], a["A"], a["B"],
                                       a["idx"], a["rank"], a["scale"], a["ws"], buf=a["buf"],
                                       x_scales=a["x_scales"], W_scales=a["W_scales"])


def test_benchmark_counters_are_those_of_its_kernels():
    """No workload of the benchmark runs the layer's sources, so its counters outlive them."""
    import importlib
    import json
    import pathlib
    bench = importlib.import_module("bench")
    root = pathlib.Path(bench.ROOT)
    for f in root.glob("profiles/pmc_*.json"):
        assert json.loads(f.read_text())["kernel_hash"] == bench.kernel_hash(), f.name
