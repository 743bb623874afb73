"""The adapter layer beside a frozen projection: cases, plain forms and calls.

Operators:
  lora_linear           y = x W^T + bias + scale[i] (x A_i^T) B_i^T, i = idx[t], rounded once
  lora_linear_backward  dx, dA, dB of it (W and the bias are frozen)
  lora_grad_norm/_clip  each adapter's global gradient norm over all its tensors, and the clip

Every case is a dict of plain values; "N" lists the packed slices' widths.
The plain forms put every token's rank-r vector at its slot's place of a wide
[T, L * R] matrix, so that all adapters go through one product.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _layer(name, op, T, K, N, R, L, mix, **more):
    c = {"name": name, "op": op, "T": T, "K": K, "N": ",".join(str(n) for n in N), "R": R, "L": L,
         "mix": mix, "bias": False, "ragged_rank": False, "dx": True}
    c.update(more)
    return c


def _grads(name, layers, K, N, R, L, dtype):
    return {"name": name, "op": "clip", "layers": layers, "K": K, "N": ",".join(str(n) for n in N),
            "R": R, "L": L, "dtype": dtype}


def listed():
    return [
        # one request decoding: one token through the merged QKV projection
        _layer("linear_token", "linear", 1, 4096, (4096, 1024, 1024), 16, 8, "random"),
        # a decode batch of many requests, each with its own adapter or none
        _layer("linear_decode", "linear", 256, 4096, (4096, 1024, 1024), 16, 8, "random"),
        # a decode batch over many adapters of unequal ranks
        _layer("linear_many", "linear", 1024, 8192, (8192,), 128, 128, "random", ragged_rank=True),
        # odd sizes: a small model's layer with a bias, widths and lengths off every tile
        _layer("linear_ragged", "linear", 777, 1352, (1100, 36, 516), 24, 5, "runs", bias=True,
               ragged_rank=True),
        # prompts of 32 requests through the gate_up projection
        _layer("linear_prefill", "linear", 8192, 4096, (14336, 14336), 64, 16, "runs"),
        # a fine-tuning step on a few short examples
        _layer("backward_short", "backward", 96, 4096, (4096, 1024, 1024), 16, 4, "runs"),
        # odd sizes, unequal ranks
        _layer("backward_ragged", "backward", 1501, 1352, (1100, 36, 516), 40, 7, "runs",
               ragged_rank=True),
        # the down projection's adapters only (nothing below them is trained)
        _layer("backward_weights", "backward", 4096, 14336, (4096,), 32, 8, "runs", dx=False),
        # a fine-tuning step of 16 adapters at once through gate_up
        _layer("backward_prefill", "backward", 8192, 4096, (14336, 14336), 64, 16, "runs"),
        # one layer's adapters
        _grads("clip_layer", 1, 4096, (4096, 1024, 1024), 16, 8, "f32"),
        # odd sizes in the storage type
        _grads("clip_odd", 5, 1352, (1100, 36, 516), 24, 3, "bf16"),
        # all adapter gradients of a 32-layer model
        _grads("clip_model", 32, 4096, (4096, 1024, 1024, 14336, 14336), 16, 4, "f32"),
    ]


def _logint(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("linear", "linear", "backward", "backward", "clip"))
    S = rng.choice((1, 1, 2, 3))
    K = _logint(rng, 256, 8192, 8)
    N = [_logint(rng, 32, 14336 if S < 3 else 4096, 4) for _ in range(S)]
    R = rng.choice((8, 16, 16, 24, 32, 64, 128))
    L = _logint(rng, 1, 64)
    if op == "clip":
        layers = _logint(rng, 1, 32)
        while layers * L * R * (S * K + sum(N)) > 110_000_000:
            L = max(1, L // 2)
            layers = max(1, layers * 3 // 4)
        c = _grads("", layers, K, N, R, L, rng.choice(("f32", "bf16")))
    else:
        T = _logint(rng, 1, 8192)
        while T * K * sum(N) > 8192 * 4096 * 20000:
            T = max(1, T * 2 // 3)
        c = _layer("", op, T, K, N, R, L, rng.choice(("random", "runs")),
                   bias=op == "linear" and rng.random() < 0.3, ragged_rank=rng.random() < 0.5,
                   dx=op == "linear" or rng.random() < 0.8)
    del c["name"]
    return c


def _widths(case):
    return [int(n) for n in case["N"].split(",")]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(g, shape, std, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _tokens(case, g):
    """Adapter slot of each token: drawn per token (a decode batch) or per run
    of tokens (the prompts of a prefill batch); a tenth without an adapter."""
    T, L = case["T"], case["L"]
    if case["mix"] == "random":
        idx = torch.randint(0, L, (T,), generator=g, device="cuda", dtype=torch.int32)
        none = torch.rand((T,), generator=g, device="cuda") < 0.1
    else:
        n = max(1, T // 256)
        cuts = torch.rand((T,), generator=g, device="cuda") < n / T
        run = torch.cumsum(cuts.to(torch.int32), 0)
        slots = torch.randint(0, L, (T + 1,), generator=g, device="cuda", dtype=torch.int32)
        idx = slots[run]
        none = (torch.rand((T + 1,), generator=g, device="cuda") < 0.1)[run]
    return torch.where(none, -1, idx).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    N, K, R, L = _widths(case), case["K"], case["R"], case["L"]
    st = {"case": dict(case)}
    if case["op"] == "clip":
        dt = _DT[case["dtype"]]
        # one buffer for each projection's gradients, all layers; a tensor per layer
        flat = []
        for n in N:
            flat.append(_normal(g, (case["layers"], L, R, K), 1e-3, dt))
            flat.append(_normal(g, (case["layers"], L, n, R), 2e-3, dt))
        grads = [t[i] for i in range(case["layers"]) for t in flat]
        # limits on both sides of the norms, as a step meets them
        est = math.sqrt(sum(t[0].numel() * (1e-6 if i % 2 == 0 else 4e-6) for i, t in enumerate(grads)))
        st["grads"] = grads
        st["max_norm"] = est * (0.4 + torch.rand((L,), generator=g, device="cuda"))
        st["flat"] = [torch.empty_like(t) for t in flat]
        st["out"] = [t[i] for i in range(case["layers"]) for t in st["flat"]]
        st["norm"] = torch.empty((L,), device="cuda", dtype=torch.float32)
        if own:
            import adapter_apply_amd as aa
            st["ws"] = aa.alloc_grad_workspace(grads)
        return st
    T, dt, S = case["T"], torch.bfloat16, len(N)
    st["x"] = _normal(g, (T, K), 1.0, dt)
    st["W"] = _normal(g, (sum(N), K), 0.02, dt)
    st["A"] = [_normal(g, (L, R, K), 0.02, dt) for _ in N]
    st["B"] = [_normal(g, (L, n, R), 0.02, dt) for n in N]
    st["bias"] = _normal(g, (sum(N),), 0.5, dt) if case["bias"] else None
    st["idx"] = _tokens(case, g)
    if case["ragged_rank"]:
        rank = torch.randint(0, R // 8 + 1, (L,), generator=g, device="cuda", dtype=torch.int32) * 8
        for t in st["A"]:
            t.mul_((torch.arange(R, device="cuda") < rank[:, None])[:, :, None])
        for t in st["B"]:
            t.mul_((torch.arange(R, device="cuda") < rank[:, None])[:, None, :])
    else:
        rank = torch.full((L,), R, device="cuda", dtype=torch.int32)
    st["rank"] = rank
    st["scale"] = torch.rand((L,), generator=g, device="cuda") + 0.5
    # x A^T, fp32 [S, T, R]: the forward call's by-product, which its backward reads
    st["buf"] = torch.empty((S, T, R), device="cuda", dtype=torch.float32)
    if case["op"] == "linear":
        st["y"] = torch.empty((T, sum(N)), device="cuda", dtype=dt)
    else:
        where = _place(st)
        for s in range(S):
            st["buf"][s] = _shrink(st, s, where)
        st["dy"] = _normal(g, (T, sum(N)), 1.0, dt)
        st["dx"] = torch.empty((T, K), device="cuda", dtype=dt) if case["dx"] else None
        st["dA"] = [torch.empty((L, R, K), device="cuda", dtype=torch.float32) for _ in N]
        st["dB"] = [torch.empty((L, n, R), device="cuda", dtype=torch.float32) for n in N]
    if own:
        import adapter_apply_amd as aa
        st["ws"] = aa.alloc_linear_workspace(T, K, N, R, L)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _place(st):
    """[T, L * R] truth values: the columns of each token's slot and true ranks."""
    L, R = st["case"]["L"], st["case"]["R"]
    slot = torch.arange(L, device="cuda")
    mine = (st["idx"][:, None] == slot) & (st["rank"] > 0)
    ranks = torch.arange(R, device="cuda") < st["rank"][:, None]
    return (mine[:, :, None] & ranks).reshape(-1, L * R)


def _fold(wide, where, L, R):
    """Each token's own R columns of a [T, L * R] matrix."""
    return torch.where(where, wide, 0.0).reshape(-1, L, R).sum(1)


def _unfold(u, where, L):
    """A [T, R] matrix put at each token's slot of [T, L * R], zero elsewhere."""
    return torch.where(where, u.repeat(1, L), 0.0)


def _shrink(st, s, where):
    c = st["case"]
    A = st["A"][s].float().reshape(c["L"] * c["R"], c["K"])
    return _fold(st["x"].float() @ A.T, where, c["L"], c["R"])


def _token_scale(st):
    L = st["case"]["L"]
    return st["scale"][st["idx"].clamp(0, L - 1).long()][:, None]


def _plain_linear(st):
    c = st["case"]
    L, R = c["L"], c["R"]
    y = st["x"].float() @ st["W"].float().T
    if st["bias"] is not None:
        y += st["bias"].float()
    where, sc = _place(st), _token_scale(st)
    buf, off = torch.empty_like(st["buf"]), 0
    for s, n in enumerate(_widths(c)):
        buf[s] = _shrink(st, s, where)
        B = st["B"][s].float().permute(0, 2, 1).reshape(L * R, n)
        y[:, off:off + n] += _unfold(sc * buf[s], where, L) @ B
        off += n
    return {"y": y.to(torch.bfloat16), "buf": buf}


def _plain_backward(st):
    c = st["case"]
    L, R, K = c["L"], c["R"], c["K"]
    where, sc = _place(st), _token_scale(st)
    x, dy = st["x"].float(), st["dy"].float()
    dx = dy @ st["W"].float() if c["dx"] else None
    dA, dB, off = [], [], 0
    for s, n in enumerate(_widths(c)):
        d = dy[:, off:off + n]
        B = st["B"][s].float().permute(0, 2, 1).reshape(L * R, n)
        v = torch.where(where, sc * (d @ B.T), 0.0)
        u = _unfold(sc * st["buf"][s], where, L)
        dA.append((v.T @ x).reshape(L, R, K))
        dB.append((d.T @ u).reshape(n, L, R).permute(1, 0, 2).contiguous())
        if dx is not None:
            dx += v @ st["A"][s].float().reshape(L * R, K)
        off += n
    return {"dx": None if dx is None else dx.to(torch.bfloat16), "dA": dA, "dB": dB}


def _plain_clip(st):
    total = 0
    for t in st["grads"]:
        total = total + t.double().square().reshape(t.shape[0], -1).sum(1)
    norm = total.sqrt().float()
    coef = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0)
    for o, t in zip(st["out"], st["grads"]):
        o.copy_(t.float() * coef[:, None, None])
    return {"norm": norm, "out": st["flat"]}


def run(state):
    st, c = state, state["case"]
    if not own:
        return {"linear": _plain_linear, "backward": _plain_backward, "clip": _plain_clip}[c["op"]](st)
    import adapter_apply_amd as aa
    if c["op"] == "linear":
        aa.lora_linear(st["y"], st["x"], st["W"], st["A"], st["B"], st["idx"], st["rank"],
                       st["scale"], st["ws"], bias=st["bias"], buf=st["buf"])
        return {"y": st["y"], "buf": st["buf"]}
    if c["op"] == "backward":
        aa.lora_linear_backward(st["dx"], st["dA"], st["dB"], st["dy"], st["x"],
                                st["W"] if c["dx"] else None, st["A"], st["B"], st["idx"],
                                st["rank"], st["scale"], st["ws"], buf=st["buf"])
        return {"dx": st["dx"], "dA": st["dA"], "dB": st["dB"]}
    aa.lora_grad_norm(st["norm"], st["grads"], st["ws"])
    aa.lora_grad_clip(st["out"], st["grads"], st["norm"], st["max_norm"])
    return {"norm": st["norm"], "out": st["flat"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    N, K, R, L = _widths(case), case["K"], case["R"], case["L"]
    S, n = len(N), sum(N)
    if case["op"] == "clip":
        m = case["layers"] * L * R * (S * K + n)
        e = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * m * e + 8 * L, "flops": 3 * m}
    T = case["T"]
    runs = T if case["mix"] == "random" else max(1, T // 256)
    slots = L * (1.0 - (1.0 - 1.0 / L) ** runs)          # slots that draw a token
    rank = R / 2 if case["ragged_rank"] else R
    adapters = 2 * slots * rank * (S * K + n)
    delta = 2 * 0.9 * T * rank * (S * K + n)
    if case["op"] == "linear":
        return {"bytes": 2 * (T * K + n * K + T * n) + adapters + 4 * S * T * R,
                "flops": 2 * T * K * n + delta}
    b = 2 * (T * K + T * n) + 4 * S * T * R + 4 * L * R * (S * K + n) + 2 * slots * rank * n
    f = 2 * 0.9 * T * rank * (n + S * K + n)
    if case["dx"]:
        b += 2 * (n * K + T * K) + 2 * slots * rank * S * K
        f += 2 * T * K * n + 2 * 0.9 * T * rank * S * K
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------
# the definition, in 64 bits, slot by slot
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "clip":
        L = case["L"]
        norm = torch.stack([sum(torch.dot(t[i].to(f64).flatten(), t[i].to(f64).flatten())
                                for t in st["grads"]).sqrt() for i in range(L)])
        ratio = st["max_norm"].to(f64) / (norm + 1e-6)
        kinds = len(st["flat"])
        out = []
        for k in range(kinds):
            o = torch.stack([t.to(f64) for t in st["grads"][k::kinds]])
            for i in range(L):
                o[:, i] *= torch.minimum(ratio[i], torch.ones_like(ratio[i]))
            out.append(o)
        return {"norm": norm, "out": out}
    N = _widths(case)
    members = {}
    ranks = st["rank"].tolist()
    for t, i in enumerate(st["idx"].tolist()):
        if 0 <= i < case["L"] and ranks[i] > 0:
            members.setdefault(i, []).append(t)
    members = {i: torch.tensor(m, device="cuda") for i, m in members.items()}
    x, W = st["x"].to(f64), st["W"].to(f64)
    if case["op"] == "linear":
        y = torch.matmul(x, W.t())
        if st["bias"] is not None:
            y = y + st["bias"].to(f64)
        buf = torch.zeros(st["buf"].shape, dtype=f64, device="cuda")
        for i, m in members.items():
            r, lo = ranks[i], 0
            for s, n in enumerate(N):
                u = x[m] @ st["A"][s][i, :r].to(f64).t()
                buf[s, m, :r] = u
                y[m, lo:lo + n] += st["scale"][i].to(f64) * (u @ st["B"][s][i, :, :r].to(f64).t())
                lo += n
        return {"y": y, "buf": buf}
    dy = st["dy"].to(f64)
    dx = torch.matmul(dy, W) if case["dx"] else None
    dA = [torch.zeros(t.shape, dtype=f64, device="cuda") for t in st["dA"]]
    dB = [torch.zeros(t.shape, dtype=f64, device="cuda") for t in st["dB"]]
    for i, m in members.items():
        r, lo, sc = ranks[i], 0, st["scale"][i].to(f64)
        for s, n in enumerate(N):
            d = dy[m, lo:lo + n]
            v = sc * (d @ st["B"][s][i, :, :r].to(f64))
            dA[s][i, :r] = v.t() @ x[m]
            dB[s][i, :, :r] = sc * (d.t() @ st["buf"][s, m, :r].to(f64))
            if dx is not None:
                dx[m] += v @ st["A"][s][i, :r].to(f64)
            lo += n
    return {"dx": dx, "dA": dA, "dB": dB}
