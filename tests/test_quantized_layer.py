"""The BitLinear layer on activations that are int8 already (bitlinear_forward_quantized,
bitlinear_backward_quantized): the forward bit for bit the oracle's integer sums and rescale, the
gradients within the accumulation's bound (n 2^-22 sum|terms| + 2^-23 |ref|, as for
bitlinear_backward)."""

import numpy as np
import pytest
import torch

import ternary_weight_linear_03_b200 as bl
from oracle import oracle as orc
from ternary_weight_linear_03_b200 import synthetic as syn

FAKE = 0x10000


def test_argument_checks():
    lib = bl.load_library()

    def call(q=FAKE, s=FAKE, p=FAKE, g=FAKE, y=FAKE, yt=1, M=4, N=100, K=128, ws=FAKE, n=1 << 30):
        return lib.bitlinear_forward_quantized(q, s, p, g, y, yt, M, N, K, ws, n, None)

    for bad in (dict(q=None), dict(s=None), dict(p=None), dict(g=None), dict(y=None), dict(yt=2)):
        assert call(**bad) == 1, bad
    for bad in (dict(M=0), dict(N=0), dict(K=100), dict(K=0), dict(N=1 << 25)):
        assert call(**bad) == 2, bad
    for bad in (dict(q=FAKE + 8), dict(s=FAKE + 4), dict(p=FAKE + 4), dict(g=FAKE + 4), dict(y=FAKE + 2)):
        assert call(**bad) == 3, bad
    assert call(M=300, ws=None) == 7 and call(M=300, n=16) == 7 and call(M=300, ws=FAKE + 8) == 3

    # rows too wide for the few-token kernel: the workspace covers the tensor-core path's staging
    # (8 bytes a token beside the split sums) although bitlinear_forward would need none
    need = lib.bitlinear_workspace_size(2, 1 << 13, 65536 + 64)
    assert need >= 2 * (65536 + 64) + 2 * 8
    assert call(M=2, N=1 << 13, K=65536 + 64, ws=None) == 7
    assert call(M=2, N=1 << 13, K=65536 + 64, n=2 * (65536 + 64)) == 7

    def back(q=FAKE, s=FAKE, gy=FAKE, p=FAKE, g=FAKE, gx=FAKE, gw=FAKE, M=4, N=128, K=64, ws=FAKE, n=1 << 30):
        return lib.bitlinear_backward_quantized(q, s, gy, p, g, gx, gw, M, N, K, ws, n, None)

    for bad in (dict(gy=None), dict(gx=None, gw=None), dict(p=None), dict(g=None), dict(q=None), dict(s=None)):
        assert back(**bad) == 1, bad
    assert back(N=100) == 2 and back(M=0) == 2 and back(gx=FAKE + 4) == 3
    need = lib.bitlinear_backward_quantized_workspace_size(4, 128, 64)
    assert back(n=need - 1) == 7 and back(ws=None) == 7 and back(ws=None, gw=None) == 7
    assert lib.bitlinear_backward_quantized_workspace_size(4, 100, 64) == 0


def _codes(M, K, seed):
    q = torch.randint(-127, 128, (M, K), generator=syn.gen(seed), dtype=torch.int32).to(torch.int8)
    s = torch.rand(M, generator=syn.gen(seed + 1)) * 0.05
    s[0] = 0.0
    return q, s


SHAPES = [(M, N, K) for M in (1, 2, 7, 8, 9, 16, 17, 40) for N, K in ((37, 64), (300, 192), (640, 1536))] + [
    (1, 1, 64), (3, 129, 320), (5, 8640, 3200), (16, 3200, 8640), (12, 1000, 28672), (15, 64, 28672),
    (257, 200, 448), (4, 70, 65536), (16, 70, 65536),
    (1, 70, 65600), (2, 300, 98304)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward_matches_oracle(M, N, K):
    q, s = _codes(M, K, M + 3 * N + 5 * K)
    packed, gamma = bl.quantize_weights(syn.weights(N, K, 0.02, seed=N + K).cuda())
    acc = orc.contract_i32(q.numpy(), orc.unpack(packed.cpu().numpy(), K))
    ref = orc.rescale(acc, s.numpy(), np.float32(gamma.item()))
    out = torch.full((M + 1, N), 7.0, device="cuda")  # the row behind the last token stays
    y = bl.forward_quantized(q.cuda(), s.cuda(), packed, gamma, y=out[:M])
    np.testing.assert_array_equal(y.cpu().numpy(), ref)
    assert (out[M] == 7.0).all()
    y16 = bl.forward_quantized(q.cuda(), s.cuda(), packed, gamma)
    assert torch.equal(y16.cpu(), torch.from_numpy(ref).bfloat16())
    assert bl.get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 6, 16, 64, 300])
def test_forward_equals_forward_of_the_unquantized(M):
    """forward(x) and quantize_acts + forward_quantized: the same bits."""
    x = syn.activations(M, 1536, seed=M, outlier_frac=0.01).cuda()
    packed, gamma = bl.quantize_weights(syn.weights(640, 1536, 0.02, seed=1).cuda())
    assert torch.equal(bl.forward(x, packed, gamma), bl.forward_quantized(*bl.quantize_acts(x), packed, gamma))


@pytest.mark.gpu
def test_forward_of_very_many_rows():
    """More rows than the GPU's blocks join at once (several rounds of 32 tiles of 16 per block),
    the last tile ragged; the reference is the exact fp32 product of the codes (below 2^24)."""
    M, N, K = 3, 160001, 8192
    q, s = _codes(M, K, 4)
    q, s = q.cuda(), s.cuda()
    g = torch.Generator(device="cuda").manual_seed(5)
    u = torch.randint(0, 3, (4, N, K // 16, 4), generator=g, device="cuda", dtype=torch.uint8)
    packed = (u[0] | u[1] << 2 | u[2] << 4 | u[3] << 6).view(N, K // 4)
    gamma = torch.full((1,), 0.5, device="cuda")
    y = bl.forward_quantized(q, s, packed, gamma, out_dtype=torch.float32)
    for a in range(0, N, 20000):
        c = u[:, a:a + 20000].permute(1, 2, 0, 3).reshape(-1, K).float() - 1
        assert torch.equal(y[:, a:a + 20000], (q.float() @ c.T) * (s * gamma)[:, None])


@pytest.mark.gpu
def test_forward_extremes():
    """All codes and trits at their largest: sums of 127 K in magnitude."""
    M, N, K = 16, 64, 28672
    q = torch.full((M, K), 127, dtype=torch.int8)
    q[1::2] = -127
    W = torch.ones((N, K))
    W[1::3] = -1.0
    packed, gamma = bl.quantize_weights(W.cuda())
    y = bl.forward_quantized(q.cuda(), torch.ones(M).cuda(), packed, gamma, out_dtype=torch.float32)
    want = (127.0 * K) * torch.where(torch.arange(M) % 2 == 0, 1.0, -1.0)[:, None] * W[:, 0]
    assert torch.equal(y.cpu(), want * gamma.item())


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (130, 640, 1536), (300, 128, 320), (1025, 128, 192),
                                   (2600, 192, 64), (33, 2112, 64)])
def test_backward_matches_oracle(M, N, K):
    q, s = _codes(M, K, M + N + K)
    G = (torch.randn((M, N), generator=syn.gen(M)) * 0.01).bfloat16()
    packed, gamma = bl.quantize_weights(syn.weights(N, K, 0.02, seed=2).cuda())
    packedT = bl.pack_transpose(packed)
    gx, gw = bl.backward_quantized(q.cuda(), s.cuda(), G.cuda(), packedT, gamma)
    codes = orc.unpack(packed.cpu().numpy(), K).astype(np.float64)
    Gf = G.double().numpy()
    g = float(gamma.item())
    xt = (q.float() * s[:, None]).bfloat16().double().numpy()
    for got, ref, mag, n in ((gx, g * (Gf @ codes), g * (np.abs(Gf) @ np.abs(codes)), N),
                             (gw, Gf.T @ xt, np.abs(Gf).T @ np.abs(xt), M)):
        err = np.abs(got.cpu().numpy().astype(np.float64) - ref)
        assert (err <= n * 2.0 ** -22 * mag + 2.0 ** -23 * np.abs(ref)).all()
    only_x, none = bl.backward_quantized(q.cuda(), s.cuda(), G.cuda(), packedT, gamma, need_w=False)
    assert none is None and torch.equal(only_x, gx)


@pytest.mark.gpu
def test_training_step_through_norm_and_layer():
    """norm -> layer -> both backward passes, as a training step runs them: each stage's inputs
    are the one before's outputs, and the gradients of x and the gain are the formula's."""
    M, N, K = 200, 640, 1536
    x = syn.activations(M, K, 1, outlier_frac=0.01)
    r = syn.activations(M, K, 2)
    w = 1.0 + 0.2 * torch.randn(K, generator=syn.gen(3))
    G = (torch.randn((M, N), generator=syn.gen(4)) * 0.01).bfloat16()
    gh = (torch.randn((M, K), generator=syn.gen(5)) * 0.01)
    packed, gamma = bl.quantize_weights(syn.weights(N, K, 0.02, seed=6).cuda())
    xq, scale, h, rstd = bl.rmsnorm_quantize(x.cuda(), w.cuda(), r.cuda())
    y = bl.forward_quantized(xq, scale, packed, gamma, out_dtype=torch.float32)
    acc = bl.contract_i32(xq, packed)
    assert torch.equal(y, bl.rescale(acc, scale, gamma, out_dtype=torch.float32))
    gn, gW = bl.backward_quantized(xq, scale, G.cuda(), bl.pack_transpose(packed), gamma)
    gx, gw = bl.rmsnorm_backward(gn, h, w.cuda(), rstd, grad_h=gh.cuda())
    g64, h64, rs = gn.cpu().double(), h.cpu().double(), rstd.cpu().double()[:, None]
    hat, d = h64 * rs, g64 * w.double()
    mean, u = (d * hat).mean(-1, keepdim=True), 2.0 ** -24
    want = gh.double() + rs * (d - hat * mean)
    tol = 8 * u * (gh.double().abs() + rs * (d.abs() + (hat * mean).abs()))  # as in test_rmsnorm.py
    tol += rs * hat.abs() * 52 * u * (d * hat).abs().mean(-1, keepdim=True)
    assert ((gx.cpu().double() - want).abs() <= tol).all()
    want = (g64 * hat).sum(0)
    assert ((gw.cpu().double() - want).abs() <= (M + 4) * u * (g64 * hat).abs().sum(0)).all()
    assert gW.shape == (N, K) and bl.get_device_status() == 0


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    """A decode step captured into a graph and replayed on new inputs; the same on a side stream."""
    M, N, K = 4, 640, 1536
    packed, gamma = bl.quantize_weights(syn.weights(N, K, 0.02, seed=6).cuda())
    w = torch.ones(K).cuda()
    xs = [syn.activations(M, K, i).cuda() for i in range(3)]
    r = syn.activations(M, K, 9).cuda()

    def step(x):
        xq, scale, h, _ = bl.rmsnorm_quantize(x, w, r)
        return bl.forward_quantized(xq, scale, packed, gamma), h

    want = [step(x) for x in xs]
    static = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [step(x) for x in xs]
    torch.cuda.synchronize()
    for (a, b), (c, d) in zip(want, got):
        assert torch.equal(a, c) and torch.equal(b, d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = step(static)
    for x, (a, b) in zip(xs, want):
        static.copy_(x)
        graph.replay()
        assert torch.equal(y, a) and torch.equal(h, b)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (77, 640, 320), (700, 128, 192)])
def test_each_gradient_alone(M, N, K):
    """One gradient without the other: the same bits, and the other's operands are not needed."""
    q, s = _codes(M, K, M)
    G = (torch.randn((M, N), generator=syn.gen(M)) * 0.01).bfloat16().cuda()
    packed, gamma = bl.quantize_weights(syn.weights(N, K, 0.02, seed=2).cuda())
    args = q.cuda(), s.cuda(), G, bl.pack_transpose(packed), gamma
    gx, gw = bl.backward_quantized(*args)
    none, only_w = bl.backward_quantized(*args, need_x=False)
    assert none is None and torch.equal(only_w, gw)
    only_x, none = bl.backward_quantized(*args, need_w=False)
    assert none is None and torch.equal(only_x, gx)
    ws, stream = bl.backward_workspace(M, N, K), torch.cuda.current_stream().cuda_stream
    again = torch.full_like(gw, float("nan"))
    assert bl.load_library().bitlinear_backward_quantized(
        args[0].data_ptr(), args[1].data_ptr(), G.data_ptr(), None, None, None, again.data_ptr(), M, N, K,
        ws.data_ptr(), ws.numel(), stream) == 0
    assert torch.equal(again, gw)
    again = torch.full_like(gx, float("nan"))
    assert bl.load_library().bitlinear_backward_quantized(
        None, None, G.data_ptr(), args[3].data_ptr(), gamma.data_ptr(), again.data_ptr(), None, M, N, K,
        ws.data_ptr(), ws.numel(), stream) == 0
    assert torch.equal(again, gx)


# A contraction of n terms runs in parts of 512: 32 matrix instructions of 16 terms each, and one fp32
# addition per part. The tensor core truncates: at each instruction the accumulator and the 16 products
# are cut at the place of the largest, two places (2^-23 of the sum so far) at most in all; over the
# 2063 instructions of one accumulator below that is 2.4e-4, of which 1.8e-4 is measured.
def _split_bound(n, mag):
    return (2 * min(-(-n // 16), 32) * 2.0 ** -23 + -(-n // 512) * 2.0 ** -24) * mag


@pytest.mark.gpu
@pytest.mark.parametrize("n", [500, 4096, 33000])
@pytest.mark.parametrize("side", ["tokens", "outputs"])
def test_long_sums_of_one_sign_are_taken_in_parts(n, side):
    """Terms of one sign, where truncation errors add up: one accumulator for all of 33000 terms is
    off by 1.8e-4 (bitlinear_backward's, measured), parts of 512 by the bound's 1.2e-5 at most."""
    n = -(-n // 64) * 64 if side == "outputs" else n
    M, N, K = (n, 64, 64) if side == "tokens" else (40, n, 64)
    q = torch.randint(64, 128, (M, K), generator=syn.gen(1)).to(torch.int8)
    s = 0.5 + torch.rand(M, generator=syn.gen(2))
    G = (0.5 + torch.rand((M, N), generator=syn.gen(3))).bfloat16()
    packed, gamma = bl.quantize_weights(torch.ones((N, K)).cuda())
    gx, gw = bl.backward_quantized(q.cuda(), s.cuda(), G.cuda(), bl.pack_transpose(packed), gamma)
    if side == "tokens":
        got, ref = gw, G.double().T @ (q.float() * s[:, None]).bfloat16().double()
    else:
        got, ref = gx, (float(gamma.item()) * G.double().sum(1, keepdim=True)).expand(M, K)
    err = (got.cpu().double() - ref).abs()
    bound = _split_bound(n, ref) + 2.0 ** -23 * ref
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (130, 640, 1536), (1025, 128, 192), (2600, 192, 64), (33, 2112, 64)])
def test_gradients_within_the_bound_of_their_parts(M, N, K):
    """As test_backward_matches_oracle, with a bound that does not grow with the length: a token
    left out or counted twice among 2600 exceeds it."""
    q, s = _codes(M, K, M + N + K)
    G = (torch.randn((M, N), generator=syn.gen(M)) * 0.01).bfloat16()
    packed, gamma = bl.quantize_weights(syn.weights(N, K, 0.02, seed=2).cuda())
    gx, gw = bl.backward_quantized(q.cuda(), s.cuda(), G.cuda(), bl.pack_transpose(packed), gamma)
    codes = torch.from_numpy(orc.unpack(packed.cpu().numpy(), K)).double()
    g, xt = float(gamma.item()), (q.float() * s[:, None]).bfloat16().double()
    for got, ref, mag, n in ((gx, g * (G.double() @ codes), g * (G.double().abs() @ codes.abs()), N),
                             (gw, G.double().T @ xt, G.double().abs().T @ xt.abs(), M)):
        err = (got.cpu().double() - ref).abs()
        assert (err <= _split_bound(n, mag) + 2.0 ** -23 * ref.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 40])
def test_two_projections_of_one_row_on_two_streams_captured(M):
    """Kernels that may start before the one ahead of them has ended, behind a fork and before a join:
    the next norm adds what both streams left. As called, and from a graph."""
    N, K = 512, 512
    gain = torch.ones(K).cuda()
    x, r = syn.activations(M, K, 1).cuda(), syn.activations(M, K, 2).cuda()
    weights = [bl.quantize_weights(syn.weights(N, K, 0.02, seed=s).cuda()) for s in (3, 4)]
    side = torch.cuda.Stream()

    def step(other):
        xq, scale, h, _ = bl.rmsnorm_quantize(x, gain, r)
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        a = bl.forward_quantized(xq, scale, *weights[0])
        b = bl.forward_quantized(xq, scale, *weights[1], stream=side if other else None)
        here.wait_stream(side)
        return (a, b, *bl.rmsnorm_quantize(a, gain, b))

    want = [t.clone() for t in step(False)]
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(step(True), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(True)
    for _ in range(10):
        for t in out:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert bl.get_device_status() == 0
