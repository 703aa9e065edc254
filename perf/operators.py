"""Cases of the operators around a ternary linear layer: the root-mean-square norm that
quantizes to int8 as it normalises (and its gradient), the layer itself on activations that
are int8 already (both directions), and a whole mixture-of-experts layer with ternary experts
for a few tokens. `run` computes a case in plain torch operations, or, where `own` is true,
through the library's entry points; `exact` computes it from the definition in 64 bits.

Sizes: hidden and feed-forward widths of the 700M (1536, 4096), 3B (3200, 8640) and 70B (8192,
28672) workloads, and generic ones for the experts, for which there is no workload."""

import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
_DTYPES = {"bf16": BF16, "f32": F32}


def listed():
    return [
        # one decoded token of the 70B width: nothing but latency
        dict(name="norm_1x8192", op="norm", M=1, K=8192, dtype="bf16", residual=True),
        # a prompt of 4096 tokens: the largest norm, bound by memory
        dict(name="norm_4096x8192", op="norm", M=4096, K=8192, dtype="bf16", residual=True),
        # the first norm of a stack (nothing to add yet) in fp32, an odd batch
        dict(name="norm_1021x3200_f32", op="norm", M=1021, K=3200, dtype="f32", residual=False),
        # training: gradient through the norm of a 4096-token batch, residual stream in bf16
        dict(name="normgrad_4096x8192", op="normgrad", M=4096, K=8192, dtype="bf16", residual=True),
        # the same in fp32 on a ragged batch of the 700M width, first norm of a stack
        dict(name="normgrad_777x1536_f32", op="normgrad", M=777, K=1536, dtype="f32", residual=False),
        # one decoded token through the 70B up projection
        dict(name="proj_1_up", op="proj", M=1, N=28672, K=8192, dtype="bf16"),
        # sixteen sequences decoded together through the 70B down projection
        dict(name="proj_16_down", op="proj", M=16, N=8192, K=28672, dtype="bf16"),
        # training step of the 700M up projection: both gradients of 4096 tokens
        dict(name="projgrad_4096_up", op="projgrad", M=4096, N=4096, K=1536),
        # a ragged small batch through the 3B down projection
        dict(name="projgrad_130_down", op="projgrad", M=130, N=3200, K=8640),
        # one decoded token, many narrow experts
        dict(name="moe_1_of_64", op="moe", M=1, D=4096, F=1536, E=64, top_k=8, act="silu", renorm=True),
        # sixteen sequences decoded together: nearly every expert has a token or two
        dict(name="moe_16_of_64", op="moe", M=16, D=4096, F=1536, E=64, top_k=8, act="silu", renorm=True),
        # the largest batch on few wide experts of the 3B widths, squared ReLU, weights as the
        # softmax gives them
        dict(name="moe_64_of_8", op="moe", M=64, D=3200, F=8640, E=8, top_k=2, act="relu2", renorm=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "normgrad", "proj", "proj", "projgrad", "moe", "moe"])
    if op in ("norm", "normgrad"):
        K = 64 * _log_int(rng, 1, 448)
        M = _log_int(rng, 1, min(4096, 4096 * 8192 // K))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if dtype == "f32":
            M = max(1, M // 2)
        return dict(op=op, M=M, K=K, dtype=dtype, residual=rng.random() < 0.7)
    if op == "proj":
        K = 64 * _log_int(rng, 4, 448)
        N = _log_int(rng, 100, min(28672, 28672 * 8192 // K))
        M = _log_int(rng, 1, 512)
        M = max(1, min(M, int(5e10 / (2.0 * N * K))))
        return dict(op=op, M=M, N=N, K=K, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "projgrad":
        K = 64 * _log_int(rng, 2, 135)
        N = 64 * _log_int(rng, 2, 135)
        M = max(1, min(_log_int(rng, 1, 4096), int(1e11 / (4.0 * N * K))))
        return dict(op=op, M=M, N=N, K=K)
    D = 64 * _log_int(rng, 8, 64)
    F = 64 * _log_int(rng, 4, 135)
    E = max(2, min(_log_int(rng, 4, 128), 64 * 4096 * 1536 // (D * F)))
    return dict(op=op, M=_log_int(rng, 1, 64), D=D, F=F, E=E, top_k=rng.randint(1, min(8, E)),
                act=rng.choice(["silu", "relu2"]), renorm=rng.random() < 0.5)


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _pack(codes):
    """Trits {-1, 0, 1} [..., K] as 2-bit codes [..., K/4]: trit 16g + 4j + i is in bits 2j of byte
    i of the 4-byte word g."""
    u = (codes + 1).to(torch.uint8).unflatten(-1, (-1, 4, 4))
    return (u[..., 0, :] | u[..., 1, :] << 2 | u[..., 2, :] << 4 | u[..., 3, :] << 6).flatten(-2)


def _ternary(g, *shape):
    """Codes and absmean of Gaussian weights, as the weight quantization leaves them."""
    w = torch.randn(shape, generator=g, device="cuda") * 0.02
    gamma = w.abs().mean((-1, -2))
    return (w / (gamma + 1e-5)[..., None, None]).round_().clamp_(-1, 1).to(torch.int8), gamma


def _experts(g, E, N, K):
    packed = torch.empty((E, N, K // 4), dtype=torch.uint8, device="cuda")
    gamma = torch.empty(E, device="cuda")
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        codes, gm = _ternary(g, min(step, E - e), N, K)
        packed[e:e + step], gamma[e:e + step] = _pack(codes), gm
    return packed, gamma


def _stream(g, M, K, dtype):
    """A residual stream: Gaussian, with one channel in a hundred twenty times as large."""
    x = torch.randn((M, K), generator=g, device="cuda")
    x[:, torch.randperm(K, generator=g, device="cuda")[: -(-K // 100)]] *= 20
    return x.to(dtype)


def _codes(g, M, K):
    """Int8 activations and scales, as the activation quantization leaves them."""
    x = torch.randn((M, K), generator=g, device="cuda")
    a = x.abs().amax(-1)
    return (x * (127.0 / a)[:, None]).round_().clamp_(-127, 127).to(torch.int8), a / 127.0


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if s["op"] in ("norm", "normgrad"):
        M, K, dt = s["M"], s["K"], _DTYPES[s["dtype"]]
        s["eps"] = 1e-5
        s["weight"] = 1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")
        if s["op"] == "norm":
            s["x"] = _stream(g, M, K, dt)
            s["r"] = _stream(g, M, K, dt) if s["residual"] else None
            if own:
                s["h"] = torch.empty_like(s["x"]) if s["residual"] else None
                s["xq"] = torch.empty((M, K), dtype=torch.int8, device="cuda")
                s["scale"], s["rstd"] = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        else:
            s["h"] = _stream(g, M, K, dt)
            s["rstd"] = (s["h"].float().square().mean(-1) + s["eps"]).rsqrt()
            s["grad_n"] = torch.randn((M, K), generator=g, device="cuda") * 0.01
            s["grad_h"] = (torch.randn((M, K), generator=g, device="cuda") * 0.01).to(dt) if s["residual"] else None
            if own:
                import ternary_weight_linear_03_b200 as bl
                s["ws"] = bl.rmsnorm_backward_workspace(M, K)
    elif s["op"] == "proj":
        codes, s["gamma"] = _ternary(g, s["N"], s["K"])
        s["packed"] = _pack(codes)
        s["gamma"] = s["gamma"].reshape(1)
        s["xq"], s["scale"] = _codes(g, s["M"], s["K"])
        if own:
            import ternary_weight_linear_03_b200 as bl
            s["ws"] = bl.workspace(s["M"], s["N"], s["K"])
    elif s["op"] == "projgrad":
        codes, s["gamma"] = _ternary(g, s["N"], s["K"])
        s["packedT"] = _pack(codes.T.contiguous())
        s["gamma"] = s["gamma"].reshape(1)
        s["xq"], s["scale"] = _codes(g, s["M"], s["K"])
        s["grad_y"] = (torch.randn((s["M"], s["N"]), generator=g, device="cuda") * 0.01).to(BF16)
        if own:
            import ternary_weight_linear_03_b200 as bl
            s["ws"] = bl.backward_workspace(s["M"], s["N"], s["K"])
    else:
        D, F, E = s["D"], s["F"], s["E"]
        # normalised hidden states, and a router whose logits spread by a few units
        s["x"] = torch.randn((s["M"], D), generator=g, device="cuda").to(BF16)
        s["router"] = (torch.randn((E, D), generator=g, device="cuda") * (2.0 / math.sqrt(D))).to(BF16)
        s["gate"], s["gate_gamma"] = _experts(g, E, F, D)
        s["up"], s["up_gamma"] = _experts(g, E, F, D)
        s["down"], s["down_gamma"] = _experts(g, E, D, F)
        if own:
            import ternary_weight_linear_03_b200 as bl
            s["layer"] = bl.MoeLayer(s["router"], s["gate"], s["gate_gamma"], s["up"], s["up_gamma"],
                                     s["down"], s["down_gamma"], top_k=s["top_k"],
                                     activation=s["act"], renormalize=s["renorm"])
            s["ws"] = bl.moe_workspace(s["M"], s["layer"])
    return s


# --------------------------------------------------------------------------- plain forms
def _unpack(packed, dtype=F32):
    """2-bit codes [..., K/4] -> trits [..., K]."""
    shift = torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=packed.device)[:, None]
    u = (packed.unflatten(-1, (-1, 1, 4)) >> shift) & 3
    return u.flatten(-3).to(dtype).sub_(1)


def _quantize(p):
    """Rows of p as whole numbers of [-127, 127], and their absolute maxima."""
    a = p.abs().amax(-1, keepdim=True)
    r = torch.full_like(a, 127) / a  # one division: 127 / a as a number and a tensor takes two steps
    q = torch.where(a > 0, (p * r).round().clamp(-127, 127), torch.zeros_like(p))
    return q, a


def _norm(s):
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
    hf = h.float()
    rstd = 1.0 / (hf.square().mean(-1, keepdim=True) + s["eps"]).sqrt()
    q, a = _quantize(hf * s["weight"])
    scale = a * rstd / 127.0
    return {"h": h, "values": (q * scale).to(BF16), "scale": scale[:, 0], "rstd": rstd[:, 0]}


def _normgrad(s):
    hat = s["h"].float() * s["rstd"][:, None]
    d = s["grad_n"] * s["weight"]
    gx = s["rstd"][:, None] * (d - hat * (d * hat).mean(-1, keepdim=True))
    if s["grad_h"] is not None:
        gx = gx + s["grad_h"].float()
    return {"grad_x": gx.to(s["h"].dtype), "grad_weight": (s["grad_n"] * hat).sum(0)}


def _proj(s):
    acc = s["xq"].float() @ _unpack(s["packed"]).T  # whole numbers below 2^24: exact
    return (acc * (s["scale"] * s["gamma"])[:, None]).to(_DTYPES[s["dtype"]])


def _projgrad(s):
    G = s["grad_y"].float()
    xt = (s["xq"].float() * s["scale"][:, None]).to(BF16).float()
    return {"grad_x": (G @ _unpack(s["packedT"]).T) * s["gamma"], "grad_w": G.T @ xt}


def _act(g, act):
    return g / (1 + (-g).exp()) if act == "silu" else g.clamp(min=0).square()


def _moe(s):
    M, k = s["M"], s["top_k"]
    x = s["x"].float()
    logits = x @ s["router"].float().T
    ids = logits.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = logits.softmax(-1).gather(-1, ids)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    q, a = _quantize(x)
    flat = ids.reshape(-1)
    if M * k < s["E"]:  # few pairs: each with its own copy of the expert
        gather = lambda t: _unpack(t[flat])  # noqa: E731
        lin = lambda v, t: (gather(t) @ v[..., None])[..., 0]  # noqa: E731
    else:  # every expert on every pair, of which its own are kept
        lin = lambda v, t: (v @ _unpack(t).transpose(-1, -2))[flat, torch.arange(M * k, device=v.device)]  # noqa: E731
    qk = q.repeat_interleave(k, 0)
    sk = (a / 127.0).repeat_interleave(k, 0)
    gate = lin(qk, s["gate"]) * (sk * s["gate_gamma"][flat][:, None])
    up = lin(qk, s["up"]) * (sk * s["up_gamma"][flat][:, None])
    hq, ha = _quantize(_act(gate, s["act"]) * up)
    out = lin(hq, s["down"]) * (ha / 127.0 * s["down_gamma"][flat][:, None])
    return (out.view(M, k, -1) * w[..., None]).sum(1).to(BF16)


def run(s):
    op = s["op"]
    if not own:
        return {"norm": _norm, "normgrad": _normgrad, "proj": _proj, "projgrad": _projgrad, "moe": _moe}[op](s)
    import ternary_weight_linear_03_b200 as bl
    if op == "norm":
        xq, scale, h, rstd = bl.rmsnorm_quantize(s["x"], s["weight"], s["r"], eps=s["eps"], h=s["h"],
                                                 xq=s["xq"], scale=s["scale"], rstd=s["rstd"])
        # the int8 codes as the values they stand for
        values = torch.empty(xq.shape, dtype=BF16, device=xq.device)
        return {"h": h, "values": torch.mul(xq, scale[:, None], out=values), "scale": scale, "rstd": rstd}
    if op == "normgrad":
        gx, gw = bl.rmsnorm_backward(s["grad_n"], s["h"], s["weight"], s["rstd"], grad_h=s["grad_h"],
                                     out_dtype=s["h"].dtype, ws=s["ws"])
        return {"grad_x": gx, "grad_weight": gw}
    if op == "proj":
        return bl.forward_quantized(s["xq"], s["scale"], s["packed"], s["gamma"],
                                    out_dtype=_DTYPES[s["dtype"]], ws=s["ws"])
    if op == "projgrad":
        gx, gw = bl.backward_quantized(s["xq"], s["scale"], s["grad_y"], s["packedT"], s["gamma"], ws=s["ws"])
        return {"grad_x": gx, "grad_w": gw}
    return bl.moe_forward(s["x"], s["layer"], out_dtype=BF16, ws=s["ws"])


# -------------------------------------------------------------------------- definitions
def _trits64(packed):
    """2-bit codes [..., K/4] -> trits in 64 bits: byte i of word g, bits 2j -> 16g + 4j + i."""
    b = packed.to(torch.int16).unflatten(-1, (-1, 4))
    planes = [torch.remainder(torch.div(b, 4 ** j, rounding_mode="floor"), 4) for j in range(4)]
    return torch.stack(planes, -2).flatten(-3).double() - 1


def _absmax_codes64(v):
    # The layer's definition rounds 127 / a and its product with a value to fp32 before the
    # code: values of a / 2, common among bf16 activations, would otherwise all be ties.
    top = v.abs().max(-1).values
    safe = torch.where(top > 0, top, torch.ones_like(top))
    r = (torch.full_like(safe, 127) / safe).float().double()
    return torch.round((v * r[..., None]).float().double()), top / 127.0


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "norm":
        h = s["x"].double() if s["r"] is None else (s["x"].double() + s["r"].double()).to(s["x"].dtype).double()
        rstd = (h.pow(2).sum(-1) / s["K"] + s["eps"]).pow(-0.5)
        q, sc = _absmax_codes64(h * rstd[:, None] * s["weight"].double())
        return {"h": h, "values": q * sc[:, None], "scale": sc, "rstd": rstd}
    if op == "normgrad":
        h, gn, w = s["h"].double(), s["grad_n"].double(), s["weight"].double()
        rs = s["rstd"].double()[:, None]
        gx = gn * w * rs - h * rs.pow(3) * ((gn * w * h).sum(-1, keepdim=True) / s["K"])
        if s["grad_h"] is not None:
            gx += s["grad_h"].double()
        return {"grad_x": gx, "grad_weight": torch.einsum("tk,tk,t->k", gn, h, rs[:, 0])}
    if op == "proj":
        if s["M"] * s["N"] * s["K"] > 3e11:
            return None
        acc = torch.cat([s["xq"].double() @ _trits64(part).T for part in s["packed"].split(4096)], 1)
        return acc * s["scale"].double()[:, None] * s["gamma"].double()
    if op == "projgrad":
        G = s["grad_y"].double()
        # the layer's definition holds the dequantized activations in bf16
        xt = (s["xq"].float() * s["scale"][:, None]).to(BF16).double()
        return {"grad_x": s["gamma"].double() * (G @ _trits64(s["packedT"]).T), "grad_w": G.T @ xt}
    x = s["x"].double()
    z = x @ s["router"].double().T
    e = torch.exp(z - z.amax(-1, keepdim=True))
    prob = e / e.sum(-1, keepdim=True)
    chosen = torch.argsort(z, dim=-1, descending=True, stable=True)[:, : s["top_k"]]
    mask = torch.zeros_like(prob).scatter_(1, chosen, 1.0)
    wt = prob * mask
    if s["renorm"]:
        wt = wt / wt.sum(-1, keepdim=True)
    q, sc = _absmax_codes64(x)
    y = torch.zeros_like(x)
    for j in range(s["E"]):
        t = mask[:, j].nonzero()[:, 0]
        if not len(t):
            continue
        gate = (q[t] * sc[t, None]) @ _trits64(s["gate"][j]).T * s["gate_gamma"][j].double()
        up = (q[t] * sc[t, None]) @ _trits64(s["up"][j]).T * s["up_gamma"][j].double()
        inner = (gate * torch.sigmoid(gate) if s["act"] == "silu" else torch.relu(gate).pow(2)) * up
        hq, hs = _absmax_codes64(inner)
        y[t] += wt[t, j, None] * ((hq * hs[:, None]) @ _trits64(s["down"][j]).T) * s["down_gamma"][j].double()
    return y


# ------------------------------------------------------------------------------- floors
def work(case):
    op = case["op"]
    if op in ("norm", "normgrad"):
        M, K, e = case["M"], case["K"], 2 if case["dtype"] == "bf16" else 4
        if op == "norm":  # x (and the residual, and their sum) once, the codes once
            return {"bytes": M * K * (e * (3 if case["residual"] else 1) + 1) + 8 * M + 4 * K, "flops": 6 * M * K}
        # h, both gradients in, one out
        return {"bytes": M * K * (e * (3 if case["residual"] else 2) + 4) + 4 * M + 8 * K, "flops": 10 * M * K}
    if op == "proj":
        M, N, K, e = case["M"], case["N"], case["K"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": N * K // 4 + M * K + 4 * M + e * M * N, "flops": 2 * M * N * K}
    if op == "projgrad":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": N * K // 4 + M * K + 2 * M * N + 4 * M * K + 4 * N * K, "flops": 4 * M * N * K}
    M, D, F, E, k = (case[n] for n in ("M", "D", "F", "E", "top_k"))
    # each expert that has a token is read once: as many as M independent choices of k meet
    active = E * (1 - (1 - k / E) ** M)
    return {"bytes": active * 3 * D * F / 4 + 2 * E * D + 4 * M * D, "flops": 2 * M * k * 3 * D * F + 2 * M * E * D}
