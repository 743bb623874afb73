"""The microscaled formats in 64 bits, written from their definition, and layers
whose projection or activations are held in them."""
import torch

import adapter_apply_amd as aa
from tests.layer_util import Layer

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def blocks(K):
    return (K + 31) // 32


def quantize(x, fmt):
    """Codes and scales of a matrix on the CPU, by search over the elements."""
    M, K = x.shape
    n = blocks(K)
    v = torch.zeros((M, 32 * n), dtype=torch.float64)
    v[:, :K] = x.to(torch.float64)
    v = v.reshape(M, n, 32)
    finite = torch.isfinite(v).all(2)
    v = torch.where(finite[:, :, None], v, torch.zeros_like(v))
    top = v.abs().amax(2)
    e = torch.frexp(top).exponent - 1 - (2 if fmt == aa.LORA_MX_FP4 else 0)
    e = torch.where(top > 0, e, -127).clamp(min=-127)
    r = torch.ldexp(v, -e[:, :, None])
    if fmt == aa.LORA_MX_FP4:
        d = (r.abs()[..., None] - GRID).abs()
        best = d.amin(-1, keepdim=True)
        # the nearest, of two the even code
        rank = torch.where(d == best, torch.arange(8) % 2, 2)
        code = rank.argmin(-1).to(torch.uint8) | (torch.signbit(r).to(torch.uint8) << 3)
        code = code.reshape(M, 16 * n, 2)
        code = code[..., 0] | code[..., 1] << 4
    else:
        code = torch.round(r * 64).clamp(-127, 127).to(torch.int8).view(torch.uint8).reshape(M, 32 * n)
    scales = torch.zeros((M, (n + 3) // 4 * 4), dtype=torch.uint8)
    scales[:, :n] = torch.where(finite, e + 127, 255).to(torch.uint8)
    return code, scales


def restore(code, scales, K, fmt):
    """The values that codes and scales stand for, 64 bits."""
    M, n = code.shape[0], blocks(K)
    if fmt == aa.LORA_MX_FP4:
        c = torch.stack((code & 15, code >> 4), 2).reshape(M, n, 32).long()
        v = GRID.to(code.device)[c & 7] * (1 - 2 * (c >> 3))
    else:
        v = code.view(torch.int8).reshape(M, n, 32).to(torch.float64) / 64
    b = scales[:, :n].to(torch.int32)[:, :, None]
    v = torch.where(b == 255, torch.full_like(v, float("nan")), torch.ldexp(v, b - 127))
    return v.reshape(M, 32 * n)[:, :K]


def window(t, extra):
    """t as a window of rows `extra` bytes wider."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), 0xA5, dtype=torch.uint8, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


class MxLayer(Layer):
    """A Layer whose W (w4) and x (x8) are replaced by what their codes stand
    for, so that its 64-bit definitions and bounds are those of the codes."""

    def __init__(self, *args, w4=True, x8=False, device="cuda", **kw):
        super().__init__(*args, device="cpu", **kw)
        extra = kw.get("extra", 0)
        put = lambda t, pad: window(t.to(device), pad * (extra > 0))
        self.Wq = self.Ws = self.xq = self.xs = None
        if w4:
            c, s = quantize(self.W, aa.LORA_MX_FP4)
            self.W = restore(c, s, self.K, aa.LORA_MX_FP4).to(torch.bfloat16)
            self.Wq, self.Ws = put(c, 48), put(s, 8)
        if x8:
            c, s = quantize(self.x, aa.LORA_MX_INT8)
            self.x = restore(c, s, self.K, aa.LORA_MX_INT8).to(torch.bfloat16)
            self.xq, self.xs = put(c, 16), put(s, 12)
        for name in ("x", "W", "dy", "bias", "idx", "rank", "scale"):
            t = getattr(self, name)
            if t is not None:
                base = t._base if t.dim() == 2 and t._base is not None else t
                moved = base.to(device)
                setattr(self, name, moved[:, :t.shape[1]] if t.dim() == 2 else moved)
        self.A, self.B = [t.to(device) for t in self.A], [t.to(device) for t in self.B]
