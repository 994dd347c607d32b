"""Cases that time the operators around an int8 layer that is being adapted.

The int8 projection itself is frozen: what a user serves or trains beside it
are low-rank adapters and layer norms. Three families are measured, each in
the sizes of the layers that this repository works with (4096 -> 16384,
12288 -> 36864 and their neighbours) and in odd ones:

  norm / norm_backward   layer norm and its gradients
  lora / lora_backward   adapters of many requests beside a projection
  clip                   global gradient norm over many tensors, and clipping

`own` false: the plain form in elementary torch operations in 32 bits; true:
the library's kernels. Both take what prepare() gives.
"""

import math
import random

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"f16": 2, "bf16": 2, "f32": 4}
_EPS = 1e-5


def listed():
    return [
        # the norm in front of a projection while 8 requests are decoded: a call of microseconds, latency only
        dict(name="norm decode", op="norm", s=8, h=12288, x="f16", w="f16"),
        # the same norm over a prompt of the headline projection
        dict(name="norm prompt", op="norm", s=4096, h=12288, x="f16", w="f16"),
        # a residual stream kept in 32 bits, a ragged number of rows and a width that no vector divides
        dict(name="norm odd f32", op="norm", s=1531, h=5141, x="f32", w="f32"),
        # the norm's gradients in a fine-tuning step of the wide layer
        dict(name="norm backward wide", op="norm_backward", s=4096, h=12288, x="f16", w="f16"),
        # the narrower layer, one row short of a full batch, bf16 with the norm's parameters in 32 bits
        dict(name="norm backward bf16", op="norm_backward", s=2047, h=4096, x="bf16", w="f32"),
        # one token of one request through the narrower layer: the smallest serving call
        dict(name="lora one token", op="lora", s=1, h=4096, o=16384, r=8, G=4, requests=1, bare=0, x="bf16"),
        # a decode batch: 64 requests, one token each, 24 adapters resident, 4 requests on the base model
        dict(name="lora decode batch", op="lora", s=64, h=12288, o=36864, r=16, G=24, requests=64, bare=4, x="f16"),
        # five prompts of different lengths in one prefill of the headline projection
        dict(name="lora prompts", op="lora", s=4096, h=12288, o=36864, r=16, G=8, requests=5, bare=1, x="f16"),
        # a small training batch of three sequences, an adapter each
        dict(name="lora backward small", op="lora_backward", s=301, h=4096, o=16384, r=8, G=3, requests=3, bare=0, x="bf16"),
        # a training step of the headline projection, rank 64, two adapters trained at once
        dict(name="lora backward wide", op="lora_backward", s=4096, h=12288, o=36864, r=64, G=2, requests=2, bare=0, x="f16"),
        # the gradients of an adapter run: many small 32-bit tensors, odd norm widths among them
        dict(name="clip adapters", op="clip", layers=32, h=4099, f=16384, r=16, full=False, ratio=4.0, x="f32"),
        # the gradients of two whole layers in 16 bits with their norms in 32: the largest case
        dict(name="clip full layers", op="clip", layers=2, h=4096, f=16384, r=1, full=True, ratio=3.0, x="f16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "lora", "lora_backward", "clip"])
    if op in ("norm", "norm_backward"):
        x, w = rng.choice([("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        h = _log_int(rng, 256, 16384)
        return dict(op=op, s=_log_int(rng, 1, 4096), h=h - h % rng.choice([1, 2, 8, 64]), x=x, w=w)
    if op == "clip":
        full = rng.random() < 0.3
        h = _log_int(rng, 256, 4096 if full else 12288)
        layers = _log_int(rng, 1, 2 if full else 48)
        return dict(op=op, layers=layers, h=h, f=h * 4 - rng.choice([0, 0, 3]), r=_log_int(rng, 4, 64), full=full,
                    ratio=rng.choice([0.5, 2.0, 8.0]), x=rng.choice(["f16", "bf16", "f32"] if not full else ["f16", "bf16"]))
    s = _log_int(rng, 1, 4096)
    requests = min(s, rng.choice([1, 2, 3, 5, 8, 17, 33, 64]))
    return dict(op=op, s=s, h=64 * _log_int(rng, 4, 192), o=64 * _log_int(rng, 4, 576), r=_log_int(rng, 4, 64),
                G=_log_int(rng, 1, 32), requests=requests, bare=rng.choice([0, 0, 1]) if requests > 1 else 0,
                x=rng.choice(["f16", "bf16"]))


def _shapes(case):
    """(shape, type) of each gradient of a clip case."""
    h, f, r, x = case["h"], case["f"], case["r"], case["x"]
    if case["full"]:  # a whole layer: QKV, output, both halves of the feed-forward, two norms
        layer = [((h, 3 * h), x), ((h, h), x), ((h, f), x), ((f, h), x)] + [((h,), "f32")] * 4
    else:             # two adapted projections and a norm
        layer = [((r, h), x), ((r, f), x), ((r, f), x), ((r, h), x), ((h,), "f32"), ((h,), "f32")]
    return layer * case["layers"]


def work(case):
    op = case["op"]
    if op == "clip":
        sizes = [(math.prod(shape), _BYTES[t]) for shape, t in _shapes(case)]
        return {"bytes": 2 * sum(n * b for n, b in sizes), "flops": 3 * sum(n for n, _ in sizes)}
    s, h, e = case["s"], case["h"], _BYTES[case["x"]]
    if op == "norm":
        return {"bytes": 2 * s * h * e + 2 * h * _BYTES[case["w"]] + 8 * s, "flops": 8 * s * h}
    if op == "norm_backward":
        return {"bytes": 3 * s * h * e + h * _BYTES[case["w"]] + 8 * s + 8 * h, "flops": 16 * s * h}
    o, r, G = case["o"], case["r"], case["G"]
    used = min(case["requests"] - case["bare"], G)
    weights, ids = used * r * (h + o) * e, 4 * s + 4 * G
    if op == "lora":
        return {"bytes": s * h * e + 2 * s * o * e + 4 * s * r + weights + ids, "flops": 2 * s * r * (h + o)}
    return {"bytes": s * o * e + 3 * s * h * e + 4 * s * r + weights + 4 * G * r * (h + o) + ids,
            "flops": 4 * s * r * (h + o)}


# ------------------------------------------------------------------ inputs

def _stream(g, s, h, dtype):
    """A residual stream: values near N(0, 1) about a small offset of each row, and a few columns that are large."""
    x = torch.randn((s, h), generator=g, device="cuda")
    x += 0.1 * torch.randn((s, 1), generator=g, device="cuda")
    cols = torch.randint(0, h, (6,), generator=g, device="cuda")
    x[:, cols] *= 12.0
    return x.to(dtype)


def _grad(g, s, h, dtype):
    """A gradient: small values whose size differs from row to row, as tokens' losses do."""
    rows = torch.exp(torch.randn((s, 1), generator=g, device="cuda"))
    return (2e-3 * rows * torch.randn((s, h), generator=g, device="cuda")).to(dtype)


def _ids(case, seed):
    """The adapter of each token: the requests' tokens follow one another, each request has at least one."""
    rng = random.Random(seed)
    s, n, G = case["s"], case["requests"], case["G"]
    cuts = [0] + sorted(rng.sample(range(1, s), n - 1)) + [s]
    which = [-1] * case["bare"] + [k % G for k in range(n - case["bare"])]
    names = rng.sample(range(G), G)
    which = [names[k] if k >= 0 else -1 for k in which]
    rng.shuffle(which)
    return [w for w, a, b in zip(which, cuts, cuts[1:]) for _ in range(b - a)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, st = case["op"], {"case": case}
    if op == "clip":
        shapes = _shapes(case)
        st["grads"] = [(1e-3 * torch.randn(shape, generator=g, device="cuda")).to(_TYPES[t]) for shape, t in shapes]
        # the scaled gradients go where an optimiser reads them: one flat buffer for each type, tensor after tensor
        kinds = sorted({t for _, t in shapes})
        st["flat"] = {t: torch.empty(sum(math.prod(sh) for sh, k in shapes if k == t), dtype=_TYPES[t], device="cuda")
                      for t in kinds}
        views = {t: iter(st["flat"][t].split([math.prod(sh) for sh, k in shapes if k == t])) for t in kinds}
        st["out"] = [next(views[t]).view(shape) for shape, t in shapes]
        st["max_norm"] = 1e-3 * math.sqrt(sum(math.prod(sh) for sh, _ in shapes)) / case["ratio"]
        return st
    s, h, dtype = case["s"], case["h"], _TYPES[case["x"]]
    st["X"] = _stream(g, s, h, dtype)
    if op in ("norm", "norm_backward"):
        wt = _TYPES[case["w"]]
        st["weight"] = (1.0 + 0.2 * torch.randn(h, generator=g, device="cuda")).to(wt)
        if op == "norm":
            st["bias"] = (0.1 * torch.randn(h, generator=g, device="cuda")).to(wt)
        else:
            st["dY"] = _grad(g, s, h, dtype)
            wide = st["X"].double()
            mean = wide.mean(1)
            st["mean"] = mean.float()
            st["rstd"] = (1.0 / torch.sqrt((wide - mean[:, None]).square().mean(1) + _EPS)).float()
        return st
    o, r, G = case["o"], case["r"], case["G"]
    st["A"] = (torch.randn((G, r, h), generator=g, device="cuda") / math.sqrt(h)).to(dtype)
    st["B"] = (0.02 * torch.randn((G, r, o), generator=g, device="cuda")).to(dtype)
    st["scale"] = 0.5 + 2.0 * torch.rand(G, generator=g, device="cuda")
    st["ids"] = torch.tensor(_ids(case, seed), dtype=torch.int32, device="cuda")
    if op == "lora":
        st["base"] = torch.randn((s, o), generator=g, device="cuda").to(dtype)
    else:
        st["base"] = _grad(g, s, h, dtype)
        st["dY"] = _grad(g, s, o, dtype)
        st["T"] = _own_rows(st["X"].float() @ st["A"].float().reshape(G * r, h).t(), st["ids"], G)
    return st


# ------------------------------------------------------------------ plain forms

def _own_rows(wide, ids, G):
    """[s, G r] -> [s, r]: each token's own adapter's part, 0 where it has none."""
    wide = wide.reshape(ids.numel(), G, -1)
    rows = wide[torch.arange(ids.numel(), device=ids.device), ids.long().clamp(min=0)]
    return torch.where(ids[:, None] >= 0, rows, torch.zeros_like(rows))


def _spread(rows, ids, scale):
    """[s, r] -> [s, G r]: scaled, in the columns of the token's own adapter, 0 elsewhere."""
    G = scale.numel()
    mine = ids[:, None] == torch.arange(G, device=ids.device, dtype=ids.dtype)
    rows = rows[:, None, :] * scale[None, :, None]
    return torch.where(mine[:, :, None], rows, torch.zeros_like(rows)).reshape(ids.numel(), -1)


def _plain_norm(st):
    x = st["X"].float()
    mean = x.sum(1) / x.shape[1]
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / x.shape[1] + _EPS)
    y = d * rstd[:, None] * st["weight"].float() + st["bias"].float()
    return {"Y": y.to(st["X"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_backward(st):
    dy, rstd = st["dY"].float(), st["rstd"][:, None]
    n = (st["X"].float() - st["mean"][:, None]) * rstd
    g = dy * st["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    return {"dX": dx.to(st["X"].dtype), "d_weight": (dy * n).sum(0), "d_bias": dy.sum(0)}


def _plain_lora(st):
    A, B, ids = st["A"].float(), st["B"].float(), st["ids"]
    G, r, h = A.shape
    T = _own_rows(st["X"].float() @ A.reshape(G * r, h).t(), ids, G)
    Y = st["base"].float() + _spread(T, ids, st["scale"]) @ B.reshape(G * r, -1)
    return {"Y": Y.to(st["X"].dtype), "T": T}


def _plain_lora_backward(st):
    A, B, ids, scale = st["A"].float(), st["B"].float(), st["ids"], st["scale"]
    G, r, h = A.shape
    dy = st["dY"].float()
    dT = _spread(_own_rows(dy @ B.reshape(G * r, -1).t(), ids, G), ids, scale)
    dX = st["base"].float() + dT @ A.reshape(G * r, h)
    dA = dT.t() @ st["X"].float()
    dB = _spread(st["T"], ids, scale).t() @ dy
    return {"dX": dX.to(st["X"].dtype), "dA": dA.reshape(A.shape), "dB": dB.reshape(B.shape)}


def _plain_clip(st):
    total = torch.sqrt(torch.stack([g.float().square().sum() for g in st["grads"]]).sum())
    c = torch.clamp(st["max_norm"] / (total + 1e-6), max=1.0)
    [o.copy_(g.float() * c) for o, g in zip(st["out"], st["grads"])]
    return {"norm": total.reshape(1), **st["flat"]}


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "lora": _plain_lora,
                "lora_backward": _plain_lora_backward, "clip": _plain_clip}[op](st)
    import int8_quantized_matmul_amd as i8
    if op == "norm":
        Y, mean, rstd = i8.layer_norm(st["X"], st["weight"], st["bias"], _EPS)
        return {"Y": Y, "mean": mean, "rstd": rstd}
    if op == "norm_backward":
        dX, d_weight, d_bias = i8.layer_norm_backward(st["dY"], st["X"], st["weight"], st["mean"], st["rstd"])
        return {"dX": dX, "d_weight": d_weight, "d_bias": d_bias}
    if op == "lora":
        Y, T = i8.lora_forward(st["X"], st["A"], st["B"], st["ids"], st["scale"], base=st["base"])
        return {"Y": Y, "T": T}
    if op == "lora_backward":
        dX, dA, dB = i8.lora_backward(st["dY"], st["X"], st["T"], st["A"], st["B"], st["ids"], st["scale"],
                                      base=st["base"])
        return {"dX": dX, "dA": dA, "dB": dB}
    return {"norm": i8.clip_grad_norm(st["grads"], st["max_norm"], out=st["out"]), **st["flat"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def _normed(x, w, b):
    """Layer norm from its definition; var as the mean square less the squared mean, exact enough in 64 bits."""
    m = x.mean(dim=1, keepdim=True)
    v = x.pow(2).mean(dim=1, keepdim=True) - m.pow(2)
    r = (v + _EPS).rsqrt()
    return (x - m) * r * w + b, m, r


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        gs = [g.double().reshape(-1) for g in st["grads"]]
        total = math.sqrt(sum(float(torch.dot(g, g)) for g in gs))
        c = min(1.0, st["max_norm"] / (total + 1e-6))
        flat = {t: torch.cat([c * g for g, (_, k) in zip(gs, _shapes(case)) if k == t]) for t in st["flat"]}
        return {"norm": torch.tensor([total], dtype=torch.float64), **flat}
    if op == "norm":
        y, m, r = _normed(st["X"].double(), st["weight"].double(), st["bias"].double())
        return {"Y": y, "mean": m[:, 0], "rstd": r[:, 0]}
    if op == "norm_backward":  # the gradients of the definition itself
        x = st["X"].double().requires_grad_()
        w = st["weight"].double().requires_grad_()
        b = torch.zeros_like(w).requires_grad_()
        y, _, _ = _normed(x, w, b)
        dx, dw, db = torch.autograd.grad(y, (x, w, b), st["dY"].double())
        return {"dX": dx, "d_weight": dw, "d_bias": db}
    ids = _ids(case, seed)
    rows = {k: torch.tensor([i for i, v in enumerate(ids) if v == k], device="cuda") for k in set(ids) if k >= 0}
    x, base, scale = st["X"].double(), st["base"].double(), st["scale"].double()
    if op == "lora":
        T = torch.zeros((case["s"], case["r"]), dtype=torch.float64, device="cuda")
        for k, i in rows.items():
            T[i] = x[i] @ st["A"][k].double().t()
            base[i] += scale[k] * (T[i] @ st["B"][k].double())
        return {"Y": base, "T": T}
    dA = torch.zeros(st["A"].shape, dtype=torch.float64, device="cuda")
    dB = torch.zeros(st["B"].shape, dtype=torch.float64, device="cuda")
    for k, i in rows.items():
        dy, a, b = st["dY"][i].double(), st["A"][k].double(), st["B"][k].double()
        dt = scale[k] * (dy @ b.t())
        base[i] += dt @ a
        dA[k] = dt.t() @ x[i]
        dB[k] = scale[k] * (st["T"][i].double().t() @ dy)
    return {"dX": base, "dA": dA, "dB": dB}
