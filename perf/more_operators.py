"""Timed cases of the dense block that stands beside the routed experts: its
training in 16 bits, the clipping of its gradients, and its products in 8-bit
integers for serving.

* ``ffn`` / ``ffn_grad``: the gated feed-forward block, (silu(x Wg^T) * x Wu^T) Wd^T,
  and its gradients by the rows and the weights;
* ``clip``: the norm of many gradients together, and the gradients scaled to it;
* ``int8``: products in 8-bit integers with a scale per token and per channel, plain
  or with the gate's activation in the same call.

Where ``own`` is true ``run`` calls the framework; otherwise it computes the
same operators with elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
TINY = 2.0 ** -100  # floor of a row's absolute maximum in the 8-bit quantisation


def listed():
    return [
        # a decode step of one sequence through a dense layer: its weights are read once
        dict(name="ffn_token", kind="ffn", T=1, H=2048, I=8192, keep=False, dtype="bf16"),
        # a ragged prefill chunk, no size a multiple of a tile
        dict(name="ffn_ragged", kind="ffn", T=333, H=2056, I=1032, keep=False, dtype="fp16"),
        # a training step's micro-batch, with what the backward pass needs kept
        dict(name="ffn_train", kind="ffn", T=8192, H=2048, I=8192, keep=True, dtype="bf16"),
        # the gradients of a small step, odd sizes
        dict(name="ffn_grad_small", kind="ffn_grad", T=133, H=1032, I=520, dtype="fp16"),
        # the gradients of the training step
        dict(name="ffn_grad_train", kind="ffn_grad", T=8192, H=2048, I=8192, dtype="bf16"),
        # the gradients of one norm, one router and their like: a few small tensors, not clipped
        dict(name="clip_small", kind="clip", tensors=6, total=40000, over=0.5, dtype="fp32"),
        # a layer's gradients
        dict(name="clip_layer", kind="clip", tensors=12, total=60000000, over=20.0, dtype="bf16"),
        # a whole model's, in full precision, many of them
        dict(name="clip_model", kind="clip", tensors=300, total=600000000, over=5.0, dtype="fp32"),
        # one token through one projection
        dict(name="int8_token", kind="int8", T=1, N=4096, K=4096, gated=False, dtype="bf16"),
        # a ragged chunk: no size a multiple of a tile
        dict(name="int8_ragged", kind="int8", T=333, N=4168, K=2064, gated=False, dtype="fp16"),
        # a full prefill through the gate and up projections with the activation
        dict(name="int8_gated", kind="int8", T=8192, N=16384, K=2048, gated=True, dtype="bf16"),
        # and back through the down projection
        dict(name="int8_long", kind="int8", T=8192, N=2048, K=8192, gated=False, dtype="bf16"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    kind = rng.choice(["ffn", "ffn_grad", "clip", "int8"])
    if kind in ("ffn", "ffn_grad"):
        H, I = _log_int(rng, 64, 8192, 8), _log_int(rng, 64, 8192, 8)
        most = 8192 * 2048 * 8192 // (H * I)
        c = dict(kind=kind, T=_log_int(rng, 1, max(1, min(16384, most))), H=H, I=I,
                 dtype=rng.choice(["bf16", "fp16"]))
        if kind == "ffn":
            c["keep"] = rng.random() < 0.5
        return c
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if kind == "clip":
        n = _log_int(rng, 1, 400)
        return dict(kind=kind, tensors=n, total=_log_int(rng, max(n, 100), 600000000),
                    over=rng.choice([0.5, 1.5, 20.0]), dtype=dtype)
    gated = rng.random() < 0.4
    N, K = _log_int(rng, 64, 16384, 16 if gated else 8), _log_int(rng, 64, 8192, 16)
    most = 8192 * 16384 * 2048 // (N * K)
    return dict(kind=kind, T=_log_int(rng, 1, max(1, min(16384, most))), N=N, K=K, gated=gated, dtype=dtype)


# ---------------------------------------------------------------- inputs

def _sizes(n, total):
    """Sizes of n tensors, about `total` elements together: most of them small (norms,
    biases, single numbers), a few hold nearly everything."""
    rng = random.Random(n * 1000003 + total)
    share = [math.exp(rng.uniform(0.0, 9.0)) for _ in range(n)]
    scale = total / sum(share)
    return [max(1, int(s * scale)) for s in share]


def _places(sizes):
    """Where tensors of these sizes begin in one buffer, at multiples of 64, and its length."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // 64) * 64)
    return at


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dt)

    s = {"case": c}
    if c["kind"] in ("ffn", "ffn_grad"):
        T, H, I = c["T"], c["H"], c["I"]
        s["w_gu"], s["w_dn"] = normal(2 * I, H, scale=H ** -0.5), normal(H, I, scale=I ** -0.5)
        s["x"] = normal(T, H)
        if c["kind"] == "ffn_grad":
            s["gu"] = (s["x"].float() @ s["w_gu"].float().t()).to(dt)
            s["dy"] = normal(T, H, scale=0.5)
    elif c["kind"] == "clip":
        sizes = _sizes(c["tensors"], c["total"])
        s["grads"] = [normal(n, scale=0.02) for n in sizes]
        # the border, `over` times below the norm that such gradients have
        s["max_norm"] = 0.02 * math.sqrt(c["total"]) / c["over"]
        # the clipped ones stand in one buffer, as what an optimizer reads does, with zeros between them
        s["flat"] = torch.zeros(_places(sizes)[-1], dtype=dt, device="cuda")
        s["clipped"] = [s["flat"][a:a + n] for a, n in zip(_places(sizes), sizes)]
    else:
        N, K = c["N"], c["K"]
        s["x"] = normal(c["T"], K)
        s["codes"] = torch.randint(-127, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
        s["scales"] = (torch.rand(N, generator=gen, device="cuda") + 0.5) * (K ** -0.5 / 64)
    return s


# ---------------------------------------------------------------- plain forms (32 bits)

def _plain_ffn(s):
    c = s["case"]
    dt = s["x"].dtype
    gu = s["x"].float() @ s["w_gu"].float().t()
    g, u = gu[:, :c["I"]], gu[:, c["I"]:]
    y = ((g / (1 + torch.exp(-g)) * u) @ s["w_dn"].float().t()).to(dt)
    return {"y": y, "gu": gu.to(dt)} if c["keep"] else {"y": y}


def _plain_ffn_grad(s):
    I, dt = s["case"]["I"], s["x"].dtype
    g, u = s["gu"][:, :I].float(), s["gu"][:, I:].float()
    dy = s["dy"].float()
    sg = 1 / (1 + torch.exp(-g))
    h = g * sg * u
    dh = dy @ s["w_dn"].float()
    dgu = torch.cat([dh * u * (sg * (1 + g * (1 / (1 + torch.exp(g))))), dh * (g * sg)], 1)
    return {"dx": (dgu @ s["w_gu"].float()).to(dt), "dw_gu": (dgu.t() @ s["x"].float()).to(dt),
            "dw_dn": (dy.t() @ h).to(dt)}


def _plain_clip(s):
    squares = torch.stack([g.float().square().sum() for g in s["grads"]])
    norm = squares.sum().sqrt()
    c = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    for out, g in zip(s["clipped"], s["grads"]):
        out.copy_(g.float() * c)
    return {"norm": norm.reshape(1), "grads": s["flat"]}


def _plain_int8(s):
    c = s["case"]
    x = s["x"].float()
    a = x.abs().amax(1, keepdim=True).clamp_min(TINY)
    top = torch.full_like(a, 127.0)  # a tensor: torch multiplies by a rounded reciprocal for a number
    q = torch.round(x * (top / a))
    z = (q @ s["codes"].float().t()) * (a / top) * s["scales"]
    if c["gated"]:
        g, u = z[:, :c["N"] // 2], z[:, c["N"] // 2:]
        z = g / (1 + torch.exp(-g)) * u
    return {"out": z.to(s["x"].dtype)}


def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(kind, state)
    return {"ffn": _plain_ffn, "ffn_grad": _plain_ffn_grad, "clip": _plain_clip, "int8": _plain_int8}[kind](state)


# ---------------------------------------------------------------- the framework's calls

def _own(kind, s):
    import bit_block_quantized_nvfp4_amd as moe

    c = s["case"]
    if kind == "ffn":
        W = moe.DenseWeights(s["w_gu"], s["w_dn"])
        if c["keep"]:
            y, gu = moe.moe_dense_ffn(W, s["x"], keep=True)
            return {"y": y, "gu": gu}
        return {"y": moe.moe_dense_ffn(W, s["x"])}
    if kind == "ffn_grad":
        W = moe.DenseWeights(s["w_gu"], s["w_dn"])
        dx, dw_gu, dw_dn = moe.moe_dense_ffn_grad(W, s["dy"], s["x"], s["gu"])
        return {"dx": dx, "dw_gu": dw_gu, "dw_dn": dw_dn}
    if kind == "clip":
        norm = moe.moe_grad_norm(s["grads"])
        moe.moe_grad_clip(s["grads"], norm, s["max_norm"], out=s["clipped"])
        return {"norm": norm, "grads": s["flat"]}
    return {"out": moe.moe_int8_linear(moe.Int8Matrix(s["codes"], s["scales"]), s["x"], gated=c["gated"])}


# ---------------------------------------------------------------- floors

def work(case):
    c = case
    size = SIZES[c["dtype"]]
    if c["kind"] == "ffn":  # x and the weights in, y (and the kept projections) back
        T, H, I = c["T"], c["H"], c["I"]
        return {"bytes": (3 * H * I + 2 * T * H + (2 * T * I if c["keep"] else 0)) * size, "flops": 6 * T * H * I}
    if c["kind"] == "ffn_grad":  # dy, x, the projections and the weights in; dx and the weights' gradients back
        T, H, I = c["T"], c["H"], c["I"]
        return {"bytes": (6 * H * I + 3 * T * H + 2 * T * I) * size, "flops": 12 * T * H * I}
    if c["kind"] == "clip":
        n = sum(_sizes(c["tensors"], c["total"]))
        return {"bytes": 2 * n * size, "flops": 3 * n}
    T, N, K = c["T"], c["N"], c["K"]
    out = N // 2 if c["gated"] else N
    return {"bytes": N * K + 4 * N + T * (K + out) * size, "flops": 2 * T * N * K}


# ---------------------------------------------------------------- the definition in 64 bits

def _silu_64(z):
    return z * torch.sigmoid(z)


def _exact_ffn(s):
    I = s["case"]["I"]
    x, W = s["x"].double(), s["w_gu"].double()
    gate, up = torch.mm(W[:I], x.t().contiguous()), torch.mm(W[I:], x.t().contiguous())
    out = {"y": torch.mm(s["w_dn"].double(), _silu_64(gate) * up).t()}
    if s["case"]["keep"]:
        out["gu"] = torch.cat([gate, up]).t()
    return out


def _exact_ffn_grad(s):
    I = s["case"]["I"]
    gate, up = s["gu"].double().split(I, dim=1)
    sg = torch.sigmoid(gate)
    dy, x, W = s["dy"].double(), s["x"].double(), s["w_gu"].double()
    dh = torch.mm(dy, s["w_dn"].double())
    dg = dh * up * sg + dh * up * gate * sg * torch.sigmoid(-gate)
    du = dh * _silu_64(gate)
    return {"dx": torch.addmm(torch.mm(dg, W[:I]), du, W[I:]),
            "dw_gu": torch.cat([torch.mm(dg.t().contiguous(), x), torch.mm(du.t().contiguous(), x)]),
            "dw_dn": torch.mm(dy.t().contiguous(), _silu_64(gate) * up)}


def _exact_clip(s):
    total = 0.0
    for g in s["grads"]:
        total += float(torch.dot(g.double(), g.double()))
    norm = math.sqrt(total)
    c = min(1.0, s["max_norm"] / (norm + 1e-6))
    pieces = []
    for g in s["grads"]:
        pieces += [c * g.double(), torch.zeros(-g.numel() % 64, dtype=torch.float64, device="cuda")]
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"), "grads": torch.cat(pieces)}


def _exact_int8(s):
    """The multiplier 127 / a, its product with a value and the scale a / 127 are
    fp32 numbers by definition: they say to which side a value on the border of
    two codes goes."""
    x = s["x"].double()
    a = x.abs().max(1).values.clamp_min(TINY).float()[:, None]
    top = torch.full_like(a, 127.0)
    q = torch.round((x * (top / a).double()).float().double())
    z = torch.mm(s["codes"].double(), q.t().contiguous()) * s["scales"].double()[:, None]
    z = z.t() * (a / top).double()
    if s["case"]["gated"]:
        gate, up = z.split(s["case"]["N"] // 2, dim=1)
        z = _silu_64(gate) * up
    return {"out": z}


def exact(case, seed):
    return {"ffn": _exact_ffn, "ffn_grad": _exact_ffn_grad, "clip": _exact_clip,
            "int8": _exact_int8}[case["kind"]](prepare(case, seed))
