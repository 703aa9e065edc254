"""The mixture-of-experts layer with ternary experts (bitlinear_moe_forward) against its
definition in 64 bits.

The definition rounds twice to int8, so the bound follows the codes (u = 2^-24 a rounding):
  * the codes of x are the definition's, bit for bit (fp32 steps of one division and one product);
  * G and U carry 3 u, act(G) U then (16 + 4 |G|) u; with the same for the row's maximum and two
    roundings of the quantizer a code of the inner row can differ, by one, only where the scaled
    value lies within that of a half; each such place adds one scale step times its trit;
  * the logits are fp32 dot products: (D / 32 + 16) u sum|x r|; the weights' error is twice the
    largest of a token, and E + 16 roundings of the softmax."""

import ctypes

import numpy as np
import pytest
import torch

import ternary_weight_linear_03_b200 as bl
from oracle import oracle as orc
from ternary_weight_linear_03_b200 import synthetic as syn

FAKE = 0x10000
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def _fake(**kw):
    f = dict(router=FAKE, gate=FAKE, up=FAKE, down=FAKE, gate_gamma=FAKE, up_gamma=FAKE, down_gamma=FAKE,
             router_dtype=1, E=8, D=128, F=192, top_k=2, act=0, renormalize=1)
    return bl.Moe(**{**f, **kw})


def test_argument_checks():
    lib = bl.load_library()
    size = lib.bitlinear_moe_workspace_size
    assert size(4, _fake()) > 0 and size(64, _fake()) > size(4, _fake())

    def call(x=FAKE, xt=1, M=4, y=FAKE, yt=1, ws=FAKE, n=1 << 30, **kw):
        m = _fake(**kw)
        return lib.bitlinear_moe_forward(x, xt, M, ctypes.byref(m), y, yt, ws, n, None)

    for bad in (dict(x=None), dict(y=None), dict(xt=2), dict(yt=2), dict(router=None), dict(gate=None),
                dict(up=None), dict(down=None), dict(gate_gamma=None), dict(up_gamma=None),
                dict(down_gamma=None), dict(router_dtype=2), dict(act=2), dict(act=-1)):
        assert call(**bad) == 1, bad
    for bad in (dict(M=0), dict(M=65), dict(E=0), dict(E=513), dict(top_k=0), dict(top_k=9), dict(D=100),
                dict(D=0), dict(F=0), dict(F=96), dict(E=64, top_k=17), dict(D=65536, F=65536), dict(D=16448), dict(F=16448)):
        assert call(**bad) == 2, bad
    for bad in (dict(x=FAKE + 8), dict(y=FAKE + 8), dict(ws=FAKE + 8), dict(router=FAKE + 2),
                dict(gate=FAKE + 4), dict(up=FAKE + 4), dict(down=FAKE + 4), dict(gate_gamma=FAKE + 4),
                dict(up_gamma=FAKE + 4), dict(down_gamma=FAKE + 4)):
        assert call(**bad) == 3, bad
    assert call(ws=None) == 7
    assert call(n=size(4, _fake()) - 256) == 7
    assert lib.bitlinear_moe_forward(FAKE, 1, 4, None, FAKE, 1, FAKE, 1 << 30, None) == 1
    assert size(4, None) == 0 and size(65, _fake()) == 0


def _layer(E, D, F, seed, rtype=BF16, spread=2.0, **kw):
    router = (torch.randn((E, D), generator=syn.gen(seed)) * (spread / D ** 0.5)).to(rtype)
    parts = {}
    for i, (name, shape) in enumerate((("gate", (E, F, D)), ("up", (E, F, D)), ("down", (E, D, F)))):
        W = torch.randn(shape, generator=syn.gen(seed + 1 + i)) * 0.02
        parts[name], parts[name + "_gamma"] = bl.quantize_expert_weights(W.cuda())
    return bl.MoeLayer(router.cuda(), parts["gate"], parts["gate_gamma"], parts["up"], parts["up_gamma"],
                       parts["down"], parts["down_gamma"], **kw)


def _quantize(v):
    """Codes and scales of the rows of v with the definition's fp32 steps (v in 64 bits)."""
    a = np.abs(v).max(-1)
    f = np.where(a > 0, np.float32(127.0) / np.where(a > 0, a, 1).astype(np.float32), 0).astype(np.float64)
    t = v * f[:, None]
    return np.clip(np.rint(t.astype(np.float32)), -127, 127).astype(np.float64), a / 127, t


def _reference(x, layer, act, renorm):
    """(y, bound on the error before y's own rounding) of the definition in 64 bits."""
    router, gate, up, down, gg, ug, dg = [t.cpu() for t in layer.tensors]
    M, E, k = x.shape[0], layer.E, layer.top_k
    xd, rd = x.double().numpy(), router.double().numpy()
    logits = xd @ rd.T
    dl = (layer.D / 32 + 16) * U * (np.abs(xd) @ np.abs(rd).T)
    order = np.argsort(-logits, axis=1, kind="stable")
    e = np.exp(logits - logits.max(1, keepdims=True))
    if k < E:  # a wide enough gap behind the chosen ones, or an exact tie
        rows = np.arange(M)
        gap = logits[rows, order[:, k - 1]] - logits[rows, order[:, k]]
        assert ((gap == 0) | (gap > 2 * dl.max(1))).all(), "the choice itself is within rounding"
    q, s, _ = _quantize(xd)
    y = np.zeros((M, layer.D))
    tol = np.zeros_like(y)
    for t in range(M):
        chosen = order[t, :k]
        w = e[t, chosen] / (e[t, chosen].sum() if renorm else e[t].sum())
        wrel = 2 * dl[t].max() + (E + 16) * U
        for j, wt in zip(chosen, w):
            cg, cu, cd = (orc.unpack(p[j].numpy(), K).astype(np.float64)
                          for p, K in ((gate, layer.D), (up, layer.D), (down, layer.F)))
            G = (cg @ q[t]) * s[t] * float(gg[j])
            Uv = (cu @ q[t]) * s[t] * float(ug[j])
            inner = (G / (1 + np.exp(-G)) if act == "silu" else np.maximum(G, 0) ** 2) * Uv
            rel = (16 + 4 * np.abs(G)) * U
            hq, hs, scaled = _quantize(inner[None])
            worst = rel[np.argmax(np.abs(inner))] + 4 * U
            near = np.abs(np.abs(scaled[0] - np.floor(scaled[0])) - 0.5) <= np.abs(scaled[0]) * (rel + worst) + 1e-12
            o = (cd @ hq[0]) * hs[0] * float(dg[j])
            y[t] += wt * o
            flips = (np.abs(cd) @ near) * hs[0] * float(dg[j])
            tol[t] += wt * (flips + np.abs(o) * (worst + wrel + 4 * U)) + k * U * np.abs(wt * o)
    return y, tol


def _check(x, layer, act, renorm, otype=F32):
    y = bl.moe_forward(x.cuda(), layer, out_dtype=otype)
    assert bl.get_device_status() == 0
    ref, tol = _reference(x, layer, act, renorm)
    tol = tol * (1 + 2.0 ** -7) + np.abs(ref) * (2.0 ** -8 if otype == BF16 else U) + 1e-30
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= tol).all(), float((err / tol).max())
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("M,E,D,F,top_k,act,renorm,xtype,rtype,otype", [
    (1, 1, 64, 64, 1, "silu", True, BF16, BF16, F32),
    (1, 16, 512, 320, 4, "silu", True, BF16, BF16, BF16),
    (2, 8, 320, 448, 2, "relu2", False, F32, F32, F32),
    (5, 64, 256, 192, 8, "silu", False, BF16, F32, F32),
    (9, 4, 576, 1088, 4, "silu", True, BF16, BF16, F32),      # every expert, nine tokens each
    (17, 3, 1024, 64, 2, "relu2", True, F32, BF16, BF16),
    (33, 2, 64, 832, 1, "silu", True, BF16, BF16, F32),
    (64, 8, 384, 256, 2, "silu", True, BF16, BF16, F32),
    (64, 1, 192, 128, 1, "silu", False, BF16, BF16, F32),     # one expert takes every token
    (3, 512, 128, 64, 16, "silu", True, BF16, BF16, F32),
    (1, 20, 4096, 1536, 8, "silu", True, BF16, BF16, F32),
    (12, 33, 1600, 704, 3, "relu2", False, BF16, BF16, BF16),
])
def test_moe_matches_definition(M, E, D, F, top_k, act, renorm, xtype, rtype, otype):
    layer = _layer(E, D, F, seed=M + E + D, rtype=rtype, top_k=top_k, activation=act, renormalize=renorm)
    x = torch.randn((M, D), generator=syn.gen(D + F)).to(xtype)
    _check(x, layer, act, renorm, otype)


@pytest.mark.gpu
def test_ties_go_to_the_lowest_expert_and_zero_rows_give_zero():
    layer = _layer(40, 128, 64, seed=1, top_k=3, activation="silu", renormalize=True)
    router = layer.tensors[0]
    router.zero_()
    router[5::9] = 1.0  # equal logits for the experts 5, 14, 23, 32
    x = torch.randn((4, 128), generator=syn.gen(3)).bfloat16()
    x[:, 0] = 20.0   # their sum is positive
    x[2] = 0.0       # every logit 0: the experts 0, 1, 2; codes all zero
    y = _check(x, layer, "silu", True)
    assert (y[2] == 0).all()


@pytest.mark.gpu
def test_nonfinite_rows_are_reported_and_the_others_stay():
    layer = _layer(16, 256, 128, seed=2, top_k=4)
    x = torch.randn((6, 256), generator=syn.gen(3)).bfloat16().cuda()
    want = bl.moe_forward(x, layer)
    assert bl.get_device_status() == 0
    for bad in (float("nan"), float("inf"), -float("inf")):
        z = x.clone()
        z[1, 7] = bad
        z[4] = bad
        got = bl.moe_forward(z, layer)
        assert bl.get_device_status() == 6
        for t in (0, 2, 3, 5):
            assert torch.equal(got[t], want[t])


@pytest.mark.gpu
def test_experts_beyond_4_gb():
    """Expert 299's matrices begin past 2^32 bytes of each stack (16.8 MB an expert); all others are
    zero. The same tokens through a layer of that expert alone give the same bits."""
    E, D, F = 300, 16384, 4096
    g = torch.Generator(device="cuda").manual_seed(3)

    def stack(N, K):
        t = torch.full((E, N, K // 4), 0x55, dtype=torch.uint8, device="cuda")  # every trit 0
        u = torch.randint(0, 3, (4, N, K // 4), generator=g, device="cuda", dtype=torch.uint8)
        t[E - 1] = u[0] | u[1] << 2 | u[2] << 4 | u[3] << 6
        return t, torch.full((E,), 0.02, device="cuda")

    gate, up, down = stack(F, D), stack(F, D), stack(D, F)
    router = torch.zeros((E, D), device="cuda")
    router[E - 1, 0] = 1.0
    x = torch.randn((3, D), generator=g, device="cuda").bfloat16()
    x[:, 0] = 2.0
    layer = bl.MoeLayer(router, *gate, *up, *down, top_k=1)
    only = bl.MoeLayer(router[-1:].contiguous(), *[t[-1:].clone() for p in (gate, up, down) for t in p], top_k=1)
    y = bl.moe_forward(x, layer)
    assert torch.equal(y, bl.moe_forward(x, only)) and (y != 0).any() and bl.get_device_status() == 0


@pytest.mark.gpu
def test_same_bits_in_any_batch_and_again():
    """A token's output does not depend on the tokens beside it, nor on what the workspace held."""
    layer = _layer(8, 512, 704, seed=4, top_k=3)
    x = torch.randn((23, 512), generator=syn.gen(5)).bfloat16().cuda()
    ws = bl.moe_workspace(64, layer)
    ws.fill_(0xFF)
    y = bl.moe_forward(x, layer, ws=ws)
    assert torch.equal(y, bl.moe_forward(x, layer, ws=ws))
    for t in (0, 11, 22):
        ws.fill_(0xAB)
        assert torch.equal(y[t:t + 1], bl.moe_forward(x[t:t + 1].contiguous(), layer, ws=ws))
    assert torch.equal(y[3:20], bl.moe_forward(x[3:20].contiguous(), layer))


@pytest.mark.gpu
def test_norm_then_experts_captured_and_replayed():
    """A block's second half as it decodes: norm of the residual stream, experts, and the next
    block's norm adds them; captured twice into graphs that share a workspace, replayed in turn."""
    M, D = 3, 512
    layer = _layer(16, D, 320, seed=6, top_k=4)
    gain = (1.0 + 0.1 * torch.randn(D, generator=syn.gen(7))).cuda()
    ws = bl.moe_workspace(M, layer)

    def step(x, r):
        normed = torch.empty_like(x)
        _, _, h, _ = bl.rmsnorm_quantize(x, gain, r, normed=normed)
        y = bl.moe_forward(normed, layer, ws=ws)
        xq, scale, h2, _ = bl.rmsnorm_quantize(y, gain, h)
        return y, xq, scale, h2

    ins = [(syn.activations(M, D, 10 + i).cuda(), syn.activations(M, D, 20 + i).cuda()) for i in range(3)]
    want = [step(*p) for p in ins]
    y, normed = want[0][0], torch.empty_like(ins[0][0])
    bl.rmsnorm_quantize(ins[0][0], gain, ins[0][1], normed=normed)
    ref, tol = _reference(normed.cpu(), layer, "silu", True)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= tol * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(ref) + 1e-30).all()
    graphs = []
    for i in range(2):
        a, b = ins[i][0].clone(), ins[i][1].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(a, b)
        graphs.append((g, a, b, out))
    for j in (2, 0, 1):
        for g, a, b, out in graphs:
            a.copy_(ins[j][0])
            b.copy_(ins[j][1])
            g.replay()
            for u, v in zip(out, want[j]):
                assert torch.equal(u, v)
    assert bl.get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("E,D,xtype,rtype", [(8, 3200, BF16, BF16), (64, 4096, BF16, BF16), (3, 16384, BF16, BF16),
                                             (24, 4096, F32, BF16), (150, 1600, BF16, F32), (512, 4160, BF16, BF16)])
def test_routing_does_not_depend_on_the_batch(E, D, xtype, rtype):
    """Rows long enough that a dot product has several terms per lane, on both sides of every change of
    blocks per token (18 and 19 tokens on 148 SMs): the same logits, so the same fp32 weights and sums."""
    layer = _layer(E, D, 64, seed=E, rtype=rtype, top_k=min(E, 8), renormalize=False)
    x = torch.randn((64, D), generator=syn.gen(D)).to(xtype).cuda()
    y = bl.moe_forward(x, layer, out_dtype=F32)
    for M in (1, 2, 9, 18, 19, 37):
        assert torch.equal(bl.moe_forward(x[:M].contiguous(), layer, out_dtype=F32), y[:M]), M
    assert bl.get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "relu2"])
@pytest.mark.parametrize("which,bad", [("gate", float("nan")), ("up", float("nan")), ("gate", 1e38), ("up", 1e38)])
def test_nonfinite_inner_rows_are_reported(act, which, bad):
    """An activation times the other factor that is NaN or passes fp32 in one chosen expert, in either place."""
    layer = _layer(4, 128, 64, seed=1, top_k=4, activation=act)
    x = 100 * torch.randn((3, 128), generator=syn.gen(3)).cuda()
    bl.moe_forward(x, layer)
    assert bl.get_device_status() == 0
    layer.tensors[4 if which == "gate" else 5][2] = bad
    bl.moe_forward(x, layer)
    assert bl.get_device_status() == 6


def _random_layer(E, D, F, seed, **kw):
    """Random trits and, for each token, a random order of the experts with gaps between the logits: the
    router picks x[t, :E] out, which holds a permutation of whole 32nds."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def stack(N, K):
        u = torch.randint(0, 3, (4, E, N, K // 4), generator=g, device="cuda", dtype=torch.uint8)
        return u[0] | u[1] << 2 | u[2] << 4 | u[3] << 6, 0.01 + 0.02 * torch.rand(E, generator=g, device="cuda")

    router = torch.zeros((E, D), device="cuda")
    router[torch.arange(E), torch.arange(E)] = 0.5
    return bl.MoeLayer(router.bfloat16(), *stack(F, D), *stack(F, D), *stack(D, F), **kw)


def _random_tokens(M, E, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((M, D), generator=g, device="cuda")
    x[:, :E] = torch.rand((M, E), generator=g, device="cuda").argsort(-1) / 32.0
    return x.bfloat16() if E <= 256 else x  # more 32nds than bf16 holds


def _trits64(packed):
    """2-bit codes [N, K/4] -> trits [N, K] in 64 bits."""
    b = packed.to(torch.int32).unflatten(-1, (-1, 4))
    return torch.stack([(b >> 2 * j) & 3 for j in range(4)], -2).flatten(-3).double() - 1


def _codes64(v):
    """_quantize on the GPU."""
    a = v.abs().amax(-1)
    f = torch.where(a > 0, torch.full_like(a, 127).float() / a.float(), torch.zeros_like(a).float()).double()
    t = v * f[:, None]
    return t.float().double().round().clamp(-127, 127), a / 127, t


def _reference_by_expert(x, layer, act, renorm):
    """_reference, expert by expert on the GPU: (y, bound on the error before y's own rounding)."""
    router, gate, up, down, gg, ug, dg = layer.tensors
    E, k = layer.E, layer.top_k
    xd = x.double()
    logits = xd @ router.double().T
    dl = ((layer.D / 32 + 16) * U * (xd.abs() @ router.double().abs().T)).amax(1)
    order = logits.argsort(dim=-1, descending=True, stable=True)
    if k < E:
        ranked = logits.gather(1, order)
        assert (ranked[:, k - 1] - ranked[:, k] > 2 * dl).all()
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    chosen = torch.zeros_like(e, dtype=torch.bool).scatter_(1, order[:, :k], True)
    w = e / ((e * chosen).sum(1, keepdim=True) if renorm else e.sum(1, keepdim=True))
    q, s, _ = _codes64(xd)
    y, tol = torch.zeros_like(xd), torch.zeros_like(xd)
    for j in range(E):
        t = chosen[:, j].nonzero()[:, 0]
        if not len(t):
            continue
        cd = _trits64(down[j])
        G = (q[t] @ _trits64(gate[j]).T) * s[t, None] * gg[j].double()
        Uv = (q[t] @ _trits64(up[j]).T) * s[t, None] * ug[j].double()
        inner = (G / (1 + torch.exp(-G)) if act == "silu" else G.clamp(min=0).square()) * Uv
        rel = (16 + 4 * G.abs()) * U
        hq, hs, scaled = _codes64(inner)
        worst = rel.gather(1, inner.abs().argmax(1, keepdim=True)) + 4 * U
        near = ((scaled - scaled.floor()).abs() - 0.5).abs() <= scaled.abs() * (rel + worst) + 1e-12
        o = (hq @ cd.T) * (hs * dg[j].double())[:, None]
        flips = (near.double() @ cd.abs().T) * (hs * dg[j].double())[:, None]
        wrel = 2 * dl[t, None] + (E + 16) * U
        wt = w[t, j, None]
        y[t] += wt * o
        tol[t] += wt * (flips + o.abs() * (worst + wrel + 4 * U)) + k * U * (wt * o).abs()
    return y, tol


@pytest.mark.gpu
@pytest.mark.parametrize("M,E,D,F,top_k,act", [
    # 16 columns: several turns of all warps over both widths, several groups of an expert's tokens
    (24, 2, 4224, 8320, 1, "silu"), (40, 3, 4224, 4544, 2, "relu2"),
    # up to 4 and up to 8 tokens, rows wider than a turn
    (3, 2, 8320, 9024, 1, "silu"), (7, 2, 8320, 8960, 2, "relu2"),
    # stretches of a block that end a run at its limit and go on in the same expert: 8 columns, gate and
    # up / down; 16 columns, gate and up / down
    (64, 128, 512, 1536, 8, "silu"), (64, 128, 4096, 64, 8, "silu"),
    (64, 8, 192, 8640, 2, "silu"), (64, 8, 16384, 64, 2, "relu2"),
    # every limit: pairs, experts and choices; both widths
    (64, 512, 512, 64, 16, "silu"), (64, 1, 16384, 16384, 1, "silu"),
])
def test_moe_of_wide_rows_and_long_stretches(M, E, D, F, top_k, act):
    layer = _random_layer(E, D, F, seed=D + F, top_k=top_k, activation=act)
    x = _random_tokens(M, E, D, seed=M)
    y = bl.moe_forward(x, layer, out_dtype=F32)
    assert bl.get_device_status() == 0
    ref, tol = _reference_by_expert(x, layer, act, True)
    err = (y.double() - ref).abs()
    tol = tol * (1 + 2.0 ** -7) + U * ref.abs() + 1e-30
    assert (err <= tol).all(), float((err / tol).max())
    y16 = bl.moe_forward(x, layer)
    assert torch.equal(y16, y.bfloat16())


@pytest.mark.gpu
def test_the_two_references_agree():
    """The reference by expert against the one by token, on a layer that both can take."""
    layer = _random_layer(6, 128, 192, seed=1, top_k=2)
    x = _random_tokens(5, 6, 128, seed=2)
    a, ta = _reference(x.cpu(), layer, "silu", True)
    b, tb = _reference_by_expert(x, layer, "silu", True)
    np.testing.assert_allclose(b.cpu().numpy(), a, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(tb.cpu().numpy(), ta, rtol=1e-9, atol=1e-13)
