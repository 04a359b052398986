"""Timed cases of the operators around the routed MoE layer.

Three families, each forward and (for training) backward:

* ``sort`` / ``sort_grad``: tokens copied into expert order and combined back
  with their routing weights; the gradients of both and of the routing weights;
* ``norm`` / ``norm_grad``: the norm after a block with its gate and residual
  scale, fused with the norm before the next block; its gradients;
* ``linear`` / ``experts``: products in e4m3 with one scale per block of 128,
  dense and for the experts' FFN.

Where ``own`` is true ``run`` calls the framework; otherwise it computes the
same operators with elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FP8 = torch.float8_e4m3fn
BLOCK = 128
TINY = 2.0 ** -100  # floor of a block's absolute maximum in the e4m3 quantisation
EPS = 1e-6


def listed():
    return [
        # one decode step of eight sequences: latency of two small launches
        dict(name="sort_decode", kind="sort", T=8, H=2048, E=512, K=10, shared=True, gate=True, dtype="bf16"),
        # a prefill chunk
        dict(name="sort_prefill", kind="sort", T=4096, H=2048, E=512, K=10, shared=True, gate=True, dtype="fp16"),
        # a small training step in full precision, odd sizes, no shared expert
        dict(name="sort_grad_small", kind="sort_grad", T=133, H=1032, E=8, K=2, shared=False, gate=False, dtype="fp32"),
        # a training step's micro-batch
        dict(name="sort_grad_train", kind="sort_grad", T=8192, H=2048, E=512, K=10, shared=True, gate=True, dtype="bf16"),
        # one decode step: the block's output into the residual stream, then the next norm
        dict(name="norm_decode", kind="norm", T=5, H=2048, gate="token", post=True, pre=True, dtype="bf16"),
        # a long prefill
        dict(name="norm_long", kind="norm", T=32768, H=2048, gate="element", post=True, pre=True, dtype="bf16"),
        # the same in training, an odd number of rows
        dict(name="norm_grad_train", kind="norm_grad", T=8191, H=2048, gate="token", post=True, pre=True, dtype="bf16"),
        # a single token through one projection
        dict(name="linear_token", kind="linear", T=1, N=2048, K=2048, dtype="bf16"),
        # a ragged chunk: no size a multiple of a tile
        dict(name="linear_ragged", kind="linear", T=333, N=4168, K=2064, dtype="bf16"),
        # a full prefill through a square projection
        dict(name="linear_long", kind="linear", T=8192, N=4096, K=4096, dtype="bf16"),
        # the experts of one decode step
        dict(name="experts_decode", kind="experts", T=8, H=2048, E=512, K=10, I=512, shared=True),
        # the experts of a prefill chunk
        dict(name="experts_prefill", kind="experts", T=4096, H=2048, E=512, K=10, I=512, shared=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    kind = rng.choice(["sort", "sort_grad", "norm", "norm_grad", "linear", "experts"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    size = 4 if dtype == "fp32" else 2
    if kind in ("sort", "sort_grad"):
        H, E = _log_int(rng, 64, 4096, 8), _log_int(rng, 4, 512)
        K = rng.randint(1, min(E, 10))
        shared = rng.random() < 0.6
        most = (4096 if kind == "sort" else 8192) * 11 * 2048 * 2 // ((K + 1) * H * size)
        return dict(kind=kind, T=_log_int(rng, 1, max(1, min(8192, most))), H=H, E=E, K=K, shared=shared,
                    gate=shared and rng.random() < 0.5, dtype=dtype)
    if kind in ("norm", "norm_grad"):
        H = _log_int(rng, 64, 8192, 8)
        most = (32768 if kind == "norm" else 8191) * 2048 * 2 // (H * size)
        gates = ["none", "token", "element"] if kind == "norm" else ["none", "token"]
        return dict(kind=kind, T=_log_int(rng, 1, max(1, min(32768, most))), H=H, gate=rng.choice(gates),
                    post=rng.random() < 0.8, pre=rng.random() < 0.8, dtype=dtype)
    if kind == "linear":
        N, K = _log_int(rng, 64, 8192, 8), _log_int(rng, 64, 8192, 16)
        most = 8192 * 4096 * 4096 // (N * K)
        return dict(kind=kind, T=_log_int(rng, 1, max(1, min(8192, most))), N=N, K=K, dtype=dtype)
    H, I = 128 * rng.randint(2, 16), 128 * rng.randint(1, 4)
    E = _log_int(rng, 4, 512)
    return dict(kind=kind, T=_log_int(rng, 1, 4096), H=H, E=E, K=rng.randint(1, min(E, 10)), I=I,
                shared=rng.random() < 0.6)


# ---------------------------------------------------------------- inputs

def _route(T, E, K, shared, gen):
    """Routing and permutation of a batch whose experts differ in popularity."""
    dev = "cuda"
    z = torch.randn(T, E, generator=gen, device=dev) + 0.5 * torch.randn(E, generator=gen, device=dev)
    top, ids = torch.topk(z, K, dim=1)
    w = torch.softmax(top, dim=1)
    flat = ids.reshape(-1)
    if shared:
        flat = torch.cat([flat, torch.full((T,), E, device=dev, dtype=flat.dtype)])
    G = E + int(shared)
    order = torch.argsort(flat, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=dev)
    counts = torch.bincount(flat, minlength=G)
    offsets = torch.zeros(G + 1, dtype=torch.int64, device=dev)
    offsets[1:] = torch.cumsum(counts, 0)
    active = torch.nonzero(counts).reshape(-1)
    groups = torch.full((G + 1,), -1, dtype=torch.int32, device=dev)
    groups[0] = active.numel()
    groups[1:1 + active.numel()] = active.int()
    return dict(logits=z, ids=ids.int(), w=w, counts=counts.int(), offsets=offsets.int(), sorted_slot=order.int(),
                slot_pos=pos.int(), groups=groups, routed=int((active < E).sum()), cap=int(counts[:E].max()))


def _codes(shape, gen):
    """e4m3 codes of weights with a spread of about one, and no NaN code."""
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) * 100).clamp_(-448, 448).to(FP8)


def _block_scales(shape, spread, gen):
    return (torch.rand(shape, generator=gen, device="cuda") + 0.5) * (spread / 100)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=None, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype or DTYPES[c["dtype"]])

    s = {"case": c}
    if c["kind"] in ("sort", "sort_grad"):
        T, H, K = c["T"], c["H"], c["K"]
        S = T * K + (T if c["shared"] else 0)
        s.update(_route(T, c["E"], K, c["shared"], gen))
        s["y"] = normal(S, H)
        s["gate"] = normal(T, dtype=torch.float32) if c["gate"] else None
        if c["kind"] == "sort":
            s["x"] = normal(T, H)
        else:
            s["dxs"], s["dout"] = normal(S, H), normal(T, H)
    elif c["kind"] in ("norm", "norm_grad"):
        T, H = c["T"], c["H"]
        s["a"], s["b"] = 0.875, 0.5
        s["r"], s["y"] = normal(T, H, scale=4.0), normal(T, H, scale=0.7)
        s["w_post"] = 1 + 0.2 * normal(H, dtype=torch.float32) if c["post"] else None
        s["w_pre"] = 1 + 0.2 * normal(H, dtype=torch.float32) if c["pre"] else None
        s["gate"] = (normal(T, dtype=torch.float32) if c["gate"] == "token" else
                     normal(T, H) if c["gate"] == "element" else None)
        if c["kind"] == "norm_grad":
            r2, _, s["rstd_post"], s["rstd_pre"] = _plain_norm(s)
            s["r_out"] = r2
            s["dr"] = normal(T, H)
            s["dn"] = normal(T, H) if c["pre"] else None
    elif c["kind"] == "linear":
        N, K = c["N"], c["K"]
        s["x"] = normal(c["T"], K)
        s["codes"] = _codes((N, K), gen)
        s["scales"] = _block_scales((-(-N // BLOCK), -(-K // BLOCK)), K ** -0.5, gen)
    else:
        T, H, I = c["T"], c["H"], c["I"]
        G = c["E"] + int(c["shared"])
        s.update(_route(T, c["E"], c["K"], c["shared"], gen))
        s["x"] = normal(T, H, dtype=torch.bfloat16)
        s["gu"], s["dn"] = _codes((G, 2 * I, H), gen), _codes((G, H, I), gen)
        s["gu_scales"] = _block_scales((G, 2 * I // BLOCK, H // BLOCK), H ** -0.5, gen)
        s["dn_scales"] = _block_scales((G, H // BLOCK, I // BLOCK), I ** -0.5, gen)
    return s


# ---------------------------------------------------------------- plain forms (32 bits)

def _tokens(s):
    """Token of each sorted position."""
    c = s["case"]
    slot = s["sorted_slot"].long()
    TK = c["T"] * c["K"]
    return torch.where(slot < TK, slot // c["K"], slot - TK)


def _shared_weight(s):
    c = s["case"]
    if s["gate"] is not None:
        return torch.sigmoid(s["gate"])
    return torch.ones(c["T"], device="cuda")


def _slot_weights(s):
    """Weight of every slot's row, in slot order (routed, then shared)."""
    w = s["w"].reshape(-1)
    return torch.cat([w, _shared_weight(s)]) if s["case"]["shared"] else w


def _sum_slots(rows, s):
    """Sum over each token's slots of rows given in slot order."""
    c = s["case"]
    TK, H = c["T"] * c["K"], rows.shape[1]
    total = rows[:TK].reshape(c["T"], c["K"], H).sum(1)
    return total + rows[TK:] if c["shared"] else total


def _plain_sort(s):
    y = s["y"]
    xs = s["x"][_tokens(s)]
    rows = y[s["slot_pos"].long()].float() * _slot_weights(s)[:, None]
    return {"xs": xs, "out": _sum_slots(rows, s).to(y.dtype)}


def _plain_sort_grad(s):
    c = s["case"]
    T, K, E, dt = c["T"], c["K"], c["E"], s["y"].dtype
    pos = s["slot_pos"].long()
    dx = _sum_slots(s["dxs"][pos].float(), s).to(dt)
    dout = s["dout"].float()
    w = _slot_weights(s)
    dy = (dout[_tokens(s)] * w[s["sorted_slot"].long()][:, None]).to(dt)
    token = torch.arange(T, device="cuda").repeat_interleave(K)
    if c["shared"]:
        token = torch.cat([token, torch.arange(T, device="cuda")])
    dots = (dout[token] * s["y"][pos].float()).sum(1)
    dw = dots[:T * K].reshape(T, K)
    dz = s["w"] * (dw - (s["w"] * dw).sum(1, keepdim=True))
    dlogits = torch.zeros(T, E, device="cuda").scatter_(1, s["ids"].long(), dz)
    out = {"dx": dx, "dy": dy, "dw": dw, "dlogits": dlogits}
    if c["gate"]:
        sg = _shared_weight(s)
        out["dgate"] = sg * (1 - sg) * dots[T * K:]
    return out


def _plain_norm(s):
    r, y = s["r"].float(), s["y"].float()
    rstd_post = rstd_pre = n = None
    u = y
    if s["w_post"] is not None:
        rstd_post = torch.rsqrt(y.square().mean(1) + EPS)
        u = y * rstd_post[:, None] * s["w_post"]
    if s["gate"] is not None:
        sg = torch.sigmoid(s["gate"].float())
        u = u * (sg if sg.dim() == 2 else sg[:, None])
    r2 = (s["a"] * r + s["b"] * u).to(s["r"].dtype)
    if s["w_pre"] is not None:
        v = r2.float()
        rstd_pre = torch.rsqrt(v.square().mean(1) + EPS)
        n = (v * rstd_pre[:, None] * s["w_pre"]).to(s["r"].dtype)
    return r2, n, rstd_post, rstd_pre


def _plain_norm_grad(s):
    dt = s["r"].dtype
    D, y = s["dr"].float(), s["y"].float()
    out = {}
    if s["w_pre"] is not None:
        xh = s["r_out"].float() * s["rstd_pre"][:, None]
        dn = s["dn"].float()
        g = dn * s["w_pre"]
        D = D + s["rstd_pre"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
        out["dw_pre"] = (dn * xh).sum(0)
    out["dr"] = (s["a"] * D).to(dt)
    yh = y * s["rstd_post"][:, None] if s["w_post"] is not None else y
    u = yh * s["w_post"] if s["w_post"] is not None else y
    du = s["b"] * D
    if s["gate"] is not None:
        sg = torch.sigmoid(s["gate"])[:, None]
        out["dgate"] = (du * u * sg * (1 - sg)).sum(1)
        du = du * sg
    if s["w_post"] is not None:
        out["dw_post"] = (du * yh).sum(0)
        g = du * s["w_post"]
        du = s["rstd_post"][:, None] * (g - yh * (g * yh).mean(1, keepdim=True))
    out["dy"] = du.to(dt)
    return out


def _quantised(x):
    """The values (in 32 bits) that the rows of x have in e4m3 with a scale per 128."""
    T, K = x.shape
    nb = -(-K // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - K)).reshape(T, nb, BLOCK)
    a = v.abs().amax(2, keepdim=True).clamp_min(TINY)
    top = torch.full_like(a, 448.0)  # a tensor: torch multiplies by a rounded reciprocal for a number
    q = (v * (top / a)).to(FP8).float()
    return (q * (a / top)).reshape(T, nb * BLOCK)[:, :K]


def _dequantised(codes, scales):
    """Weights [..., N, K] in 32 bits from their codes and 128x128 block scales."""
    N, K = codes.shape[-2:]
    s = scales.repeat_interleave(BLOCK, dim=-1)[..., :K].repeat_interleave(BLOCK, dim=-2)[..., :N, :]
    return codes.float() * s


def _plain_linear(s):
    W = _dequantised(s["codes"], s["scales"])
    return {"out": (_quantised(s["x"]) @ W.t().contiguous()).to(s["x"].dtype)}


def _silu_mul(z, I):
    g, u = z[..., :I], z[..., I:]
    return g / (1 + torch.exp(-g)) * u


def _plain_experts(s):
    c = s["case"]
    T, K, E, H, I = c["T"], c["K"], c["E"], c["H"], c["I"]
    n, cap = s["routed"], s["cap"]
    x = _quantised(s["x"])
    # the routed rows, group by group, each group padded to the largest
    group = s["groups"][1:1 + n].long()
    first = s["offsets"].long()[group]
    row = first[:, None] + torch.arange(cap, device="cuda")
    real = row < (first + s["counts"].long()[group])[:, None]
    row = torch.where(real, row, 0)
    xp = x[(s["sorted_slot"].long()[row] // K).clamp(max=T - 1)] * real[..., None]
    z = torch.bmm(_dequantised(s["gu"][group], s["gu_scales"][group]), xp.transpose(1, 2).contiguous())
    h = _quantised(_silu_mul(z.transpose(1, 2), I).reshape(n * cap, I)).reshape(n, cap, I)
    y = torch.bmm(_dequantised(s["dn"][group], s["dn_scales"][group]), h.transpose(1, 2).contiguous())
    out = torch.empty(s["sorted_slot"].numel(), H, dtype=torch.bfloat16, device="cuda")
    out[row[real]] = y.transpose(1, 2)[real].to(torch.bfloat16)
    if c["shared"]:
        z = x @ _dequantised(s["gu"][E], s["gu_scales"][E]).t().contiguous()
        h = _quantised(_silu_mul(z, I))
        out[T * K:] = (h @ _dequantised(s["dn"][E], s["dn_scales"][E]).t().contiguous()).to(torch.bfloat16)
    return {"y": out}


def _some(d):
    return {k: v for k, v in d.items() if v is not None}


def run(state):
    s = state
    c = s["case"]
    kind = c["kind"]
    if own:
        return _own(kind, s)
    if kind == "norm":
        r2, n, rstd_post, rstd_pre = _plain_norm(s)
        return _some({"r": r2, "n": n, "rstd_post": rstd_post, "rstd_pre": rstd_pre})
    return {"sort": _plain_sort, "sort_grad": _plain_sort_grad, "norm_grad": _plain_norm_grad,
            "linear": _plain_linear, "experts": _plain_experts}[kind](s)


# ---------------------------------------------------------------- the framework's calls

def _own(kind, s):
    import bit_block_quantized_nvfp4_amd as moe

    c = s["case"]
    if kind == "sort":
        xs = moe.moe_dispatch(s["x"], s["slot_pos"], c["K"], c["shared"])
        if s["gate"] is not None:
            out = moe.moe_combine_gated(s["y"], s["w"], s["slot_pos"], s["gate"], c["K"])
        else:
            out = moe.moe_combine(s["y"], s["w"], s["slot_pos"], c["K"], c["shared"])
        return {"xs": xs, "out": out}
    if kind == "sort_grad":
        dx = moe.moe_dispatch_grad(s["dxs"], s["slot_pos"], c["K"], c["shared"])
        dy, dw, dgate = moe.moe_combine_grad(s["dout"], s["y"], s["w"], s["slot_pos"], c["K"], c["shared"],
                                             gate=s["gate"])
        dlogits = moe.moe_route_topk_grad(s["ids"], s["w"], dw, c["E"])
        return _some({"dx": dx, "dy": dy, "dw": dw, "dlogits": dlogits, "dgate": dgate})
    if kind == "norm":
        r2, n, rstd_post, rstd_pre = moe.moe_block_norm(s["r"], s["y"], gate=s["gate"], w_post=s["w_post"],
                                                        w_pre=s["w_pre"], res_scale=s["a"], out_scale=s["b"], eps=EPS)
        return _some({"r": r2, "n": n, "rstd_post": rstd_post, "rstd_pre": rstd_pre})
    if kind == "norm_grad":
        dr, dy, dgate, dw_post, dw_pre = moe.moe_block_norm_grad(
            s["dr"], s["dn"], s["r_out"], s["y"], gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"],
            rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"], res_scale=s["a"], out_scale=s["b"])
        return _some({"dr": dr, "dy": dy, "dgate": dgate, "dw_post": dw_post, "dw_pre": dw_pre})
    if kind == "linear":
        return {"out": moe.moe_fp8_linear(moe.FP8Matrix(s["codes"], s["scales"]), s["x"])}
    W = moe.FP8Weights(s["gu"], s["gu_scales"], s["dn"], s["dn_scales"], c["E"], c["H"], c["I"], c["shared"])
    return {"y": moe.moe_fp8_expert_ffn(W, s["x"], c["K"], s["offsets"], s["sorted_slot"], s["groups"])}


# ---------------------------------------------------------------- floors

def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[c.get("dtype", "bf16")]
    if c["kind"] in ("sort", "sort_grad"):
        T, H, K = c["T"], c["H"], c["K"]
        S = T * K + (T if c["shared"] else 0)
        index = 4 * (T * K + S + (T if c["gate"] else 0))
        if c["kind"] == "sort":  # x, y in; xs, out back
            return {"bytes": 2 * (T + S) * H * size + index, "flops": 2 * S * H}
        back = 4 * (T * K + T * c["E"] + T * K + (T if c["gate"] else 0))
        return {"bytes": (2 * T + 3 * S) * H * size + index + back, "flops": 4 * S * H}
    if c["kind"] in ("norm", "norm_grad"):
        T, H = c["T"], c["H"]
        gate = {"none": 0, "token": 4 * T, "element": T * H * size}[c["gate"]]
        norms = c["post"] + c["pre"]
        if c["kind"] == "norm":  # r, y, gate in; r, n, statistics back
            return {"bytes": (3 + c["pre"]) * T * H * size + gate + norms * (4 * H + 4 * T), "flops": 12 * T * H}
        # dr, y (dn, r) in; dr, dy back; gate in and its gradient back
        return {"bytes": (4 + 2 * c["pre"]) * T * H * size + 2 * gate + norms * (8 * H + 4 * T), "flops": 24 * T * H}
    if c["kind"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": N * K + 4 * (-(-N // BLOCK)) * (-(-K // BLOCK)) + T * (N + K) * size, "flops": 2 * T * N * K}
    T, H, K, I = c["T"], c["H"], c["K"], c["I"]
    S = T * K + (T if c["shared"] else 0)
    # experts that a batch of this size is expected to reach, with equal chances
    active = c["E"] * (1 - (1 - K / c["E"]) ** T) + (1 if c["shared"] else 0)
    return {"bytes": active * 3 * H * I + T * H * 2 + S * H * 2, "flops": 6 * S * H * I}


# ---------------------------------------------------------------- the definition in 64 bits

def _e4m3_64(v):
    """Nearest e4m3 value (ties to even) of each value of v, |v| <= 448."""
    _, e = torch.frexp(v)
    step = torch.exp2((e.double() - 1).clamp_min(-6.0) - 3)
    return torch.round(v / step) * step


def _rows_64(x):
    """The rows of x as e4m3 times its scales, in 64 bits.  The multiplier 448 / a,
    its product with a value and the scale a / 448 are fp32 numbers by
    definition: rows of 16-bit values have many quotients right on the borders
    of e4m3, and this says to which side those go."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for b in range(0, x.shape[1], BLOCK):
        v = x[:, b:b + BLOCK].double()
        a = v.abs().max(1, keepdim=True).values.clamp_min(TINY).float()
        top = torch.full_like(a, 448.0)
        out[:, b:b + BLOCK] = _e4m3_64((v * (top / a).double()).float().double()) * (a / top).double()
    return out


def _matrix_64(codes, scales):
    W = codes.to(torch.float64)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            W[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= scales[i, j].double()
    return W


def _exact_sort(s):
    c = s["case"]
    T, K, H = c["T"], c["K"], c["H"]
    pos = s["slot_pos"].long()
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    xs = torch.empty(pos.numel(), H, dtype=torch.float64, device="cuda")
    for k in range(K):
        p = pos[k:T * K:K]
        out += s["w"][:, k, None].double() * s["y"][p].double()
        xs[p] = s["x"].double()
    if c["shared"]:
        p = pos[T * K:]
        xs[p] = s["x"].double()
        out += s["y"][p].double() / (1 + torch.exp(-s["gate"].double()))[:, None] if c["gate"] else s["y"][p].double()
    return {"xs": xs, "out": out}


def _exact_sort_grad(s):
    c = s["case"]
    T, K, H, E = c["T"], c["K"], c["H"], c["E"]
    pos = s["slot_pos"].long()
    dout = s["dout"].double()
    dx = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    dy = torch.empty(pos.numel(), H, dtype=torch.float64, device="cuda")
    dw = torch.empty(T, K, dtype=torch.float64, device="cuda")
    for k in range(K):
        p = pos[k:T * K:K]
        dx += s["dxs"][p].double()
        dy[p] = s["w"][:, k, None].double() * dout
        dw[:, k] = (dout * s["y"][p].double()).sum(1)
    out = {"dx": dx, "dy": dy, "dw": dw}
    if c["shared"]:
        p = pos[T * K:]
        dx += s["dxs"][p].double()
        dy[p] = dout
        if c["gate"]:
            sg = 1 / (1 + torch.exp(-s["gate"].double()))
            dy[p] = sg[:, None] * dout
            out["dgate"] = sg * (1 - sg) * (dout * s["y"][p].double()).sum(1)
    w = s["w"].double()
    mean = (w * dw).sum(1)
    dlogits = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    token = torch.arange(T, device="cuda")
    for k in range(K):
        dlogits[token, s["ids"][:, k].long()] = w[:, k] * (dw[:, k] - mean)
    out["dlogits"] = dlogits
    return out


def _exact_norm(s):
    y, H = s["y"].double(), s["y"].shape[1]
    out = {}
    if s["w_post"] is not None:
        out["rstd_post"] = (y.pow(2).sum(1) / H + EPS).pow(-0.5)
        y = torch.einsum("th,t,h->th", y, out["rstd_post"], s["w_post"].double())
    if s["gate"] is not None:
        g = s["gate"].double()
        y = y / (1 + torch.exp(-(g if g.dim() == 2 else g[:, None])))
    out["r"] = s["a"] * s["r"].double() + s["b"] * y
    if s["w_pre"] is not None:
        v = out["r"].to(s["r"].dtype).double()
        out["rstd_pre"] = (v.pow(2).sum(1) / H + EPS).pow(-0.5)
        out["n"] = torch.einsum("th,t,h->th", v, out["rstd_pre"], s["w_pre"].double())
    return out


def _exact_norm_grad(s):
    def back(g, w, v, rstd):
        """Gradient by v of v * rstd * w: rstd * (g w) - rstd^3 v <g w, v> / H."""
        g = g * w.double()
        return rstd[:, None] * g - (rstd.pow(3) * (g * v).sum(1) / v.shape[1])[:, None] * v

    y, D, out = s["y"].double(), s["dr"].double(), {}
    if s["w_pre"] is not None:
        v, rstd, dn = s["r_out"].double(), s["rstd_pre"].double(), s["dn"].double()
        D = D + back(dn, s["w_pre"], v, rstd)
        out["dw_pre"] = torch.einsum("th,th,t->h", dn, v, rstd)
    out["dr"] = D * s["a"]
    u = y if s["w_post"] is None else torch.einsum("th,t,h->th", y, s["rstd_post"].double(), s["w_post"].double())
    du = D * s["b"]
    if s["gate"] is not None:
        sg = 1 / (1 + torch.exp(-s["gate"].double()))
        out["dgate"] = (sg - sg * sg) * (du * u).sum(1)
        du = du * sg[:, None]
    if s["w_post"] is not None:
        out["dw_post"] = torch.einsum("th,th,t->h", du, y, s["rstd_post"].double())
        du = back(du, s["w_post"], y, s["rstd_post"].double())
    out["dy"] = du
    return out


def _exact_experts(s):
    c = s["case"]
    T, K, I = c["T"], c["K"], c["I"]
    x = _rows_64(s["x"])
    offsets = s["offsets"].tolist()
    slots = s["sorted_slot"].long()
    y = torch.empty(slots.numel(), c["H"], dtype=torch.float64, device="cuda")
    for g in range(len(offsets) - 1):
        a, b = offsets[g], offsets[g + 1]
        if a == b:
            continue
        rows = slots[a:b] // K if g < c["E"] else slots[a:b] - T * K
        z = torch.mm(_block_64(s["gu"][g], s["gu_scales"][g]), x[rows].t().contiguous()).t()
        gate, up = z[:, :I], z[:, I:]
        h = _rows_64(gate * up / (1 + torch.exp(-gate)))
        y[a:b] = torch.mm(_block_64(s["dn"][g], s["dn_scales"][g]), h.t().contiguous()).t()
    return {"y": y}


def _block_64(codes, scales):
    """codes [N, K] times their block scales, N and K whole blocks."""
    N, K = codes.shape
    W = codes.to(torch.float64).view(N // BLOCK, BLOCK, K // BLOCK, BLOCK)
    return (W * scales.double()[:, None, :, None]).view(N, K)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "linear":
        W = _matrix_64(s["codes"], s["scales"])
        return {"out": torch.mm(W, _rows_64(s["x"]).t().contiguous()).t()}
    return {"sort": _exact_sort, "sort_grad": _exact_sort_grad, "norm": _exact_norm,
            "norm_grad": _exact_norm_grad, "experts": _exact_experts}[kind](s)
