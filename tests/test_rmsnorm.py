"""RMS norm with an int8 output (bitlinear_rmsnorm_quantize) and its gradient.

h and the codes are compared bit for bit with the definition's fp32 steps; the row statistics and
the gradients with 64-bit sums, within what their roundings allow (u = 2^-24 a rounding):
  * a row's sum of squares is at most 32 terms in a row in one thread and 10 tree additions, all
    positive: 48 u, halved by the root; with the division by K, eps, the root and 1/root 28 u. The
    scale adds two roundings, a normalised value two and its storage half a step.
  * the gradient's dot product has the same shape: 52 u sum|d hat| with the roundings of d and hat."""

import numpy as np
import pytest
import torch

import ternary_weight_linear_03_b200 as bl
from ternary_weight_linear_03_b200 import synthetic as syn

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below fails its checks first
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def test_argument_checks():
    f = bl.load_library().bitlinear_rmsnorm_quantize

    def call(x=FAKE, r=FAKE, xt=1, w=FAKE, wt=0, eps=1e-5, M=4, K=128, h=FAKE, n=None, q=FAKE, s=FAKE, rs=FAKE):
        return f(x, r, xt, w, wt, eps, M, K, h, n, q, s, rs, None)

    for bad in (dict(x=None), dict(w=None), dict(q=None), dict(s=None), dict(xt=2), dict(wt=3),
                dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**bad) == 1, bad
    for bad in (dict(M=0), dict(K=0), dict(K=96), dict(K=32768 + 64), dict(M=1 << 26)):
        assert call(**bad) == 2, bad
    for bad in (dict(x=FAKE + 8), dict(r=FAKE + 2), dict(w=FAKE + 4), dict(h=FAKE + 8), dict(n=FAKE + 8),
                dict(q=FAKE + 1), dict(s=FAKE + 4), dict(rs=FAKE + 4)):
        assert call(**bad) == 3, bad


def test_backward_argument_checks():
    lib = bl.load_library()
    assert lib.bitlinear_rmsnorm_backward_workspace_size(0, 128) == 0
    assert lib.bitlinear_rmsnorm_backward_workspace_size(4, 100) == 0
    assert lib.bitlinear_rmsnorm_backward_workspace_size(4, 32768 + 64) == 0
    need = lib.bitlinear_rmsnorm_backward_workspace_size(4, 128)
    assert need >= 4 * 128 * 4

    def call(g=FAKE, gt=0, h=FAKE, ht=1, w=FAKE, wt=0, rs=FAKE, gh=None, gx=FAKE, xt=1, gw=FAKE, M=4, K=128,
             ws=FAKE, n=need):
        return lib.bitlinear_rmsnorm_backward(g, gt, h, ht, w, wt, rs, gh, gx, xt, gw, M, K, ws, n, None)

    for bad in (dict(g=None), dict(h=None), dict(w=None), dict(rs=None), dict(gx=None), dict(gw=None),
                dict(gt=2), dict(ht=2), dict(wt=-1), dict(xt=2)):
        assert call(**bad) == 1, bad
    for bad in (dict(M=0), dict(K=100), dict(K=32768 + 64)):
        assert call(**bad) == 2, bad
    for bad in (dict(g=FAKE + 8), dict(gh=FAKE + 8), dict(gx=FAKE + 8), dict(gw=FAKE + 4), dict(ws=FAKE + 8)):
        assert call(**bad) == 3, bad
    assert call(ws=None) == 7 and call(n=need - 1) == 7


def test_binding_refuses_what_the_library_cannot_see():
    x = torch.zeros((4, 128))
    with pytest.raises(ValueError):
        bl.rmsnorm_quantize(x, torch.ones(128))  # not on the GPU


def _rows(M, K, dtype, seed, residual):
    x = syn.activations(M, K, seed, dtype, outlier_frac=0.01)
    r = syn.activations(M, K, seed + 1, dtype) if residual else None
    w = 1.0 + 0.2 * torch.randn(K, generator=syn.gen(seed + 2))
    return x, r, w


def _codes_of(p):
    """The definition's fp32 steps on the CPU: codes and absolute maxima of the rows of p."""
    p = p.numpy()
    a = np.abs(p).max(-1).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        f = (np.float32(127.0) / a).astype(np.float32)
        t = (p * f[:, None]).astype(np.float32)
    q = np.where(p == 0, 0, np.clip(np.rint(np.where(p == 0, 0, t)), -127, 127)).astype(np.int8)
    return q, a


def _cuda(t):
    return None if t is None else t.cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,dtype,wtype,residual", [
    (1, 64, BF16, F32, True), (1, 8192, BF16, F32, True), (3, 1536, F32, BF16, True),
    (5, 4096, BF16, F32, False), (2, 4160, BF16, BF16, True), (3, 8256, F32, F32, True),
    (7, 28672, BF16, F32, True), (2, 32768, F32, F32, False), (33, 3200, BF16, BF16, False),
    (1021, 320, BF16, F32, True), (700, 1536, BF16, F32, True),
])
def test_norm_matches_definition(M, K, dtype, wtype, residual):
    x, r, w = _rows(M, K, dtype, 3 * M + K, residual)
    w = w.to(wtype)
    normed = torch.full((M, K), float("nan"), dtype=dtype, device="cuda")
    xq, scale, h, rstd = bl.rmsnorm_quantize(x.cuda(), w.cuda(), _cuda(r), normed=normed)
    assert bl.get_device_status() == 0
    href = x if r is None else (x.float() + r.float()).to(dtype)
    assert torch.equal(h.cpu(), href)
    q, a = _codes_of(href.float() * w.float())
    np.testing.assert_array_equal(xq.cpu().numpy(), q)
    h64, w64 = href.double(), w.double()
    rs = 1.0 / (h64.square().mean(-1) + 1e-5).sqrt()
    assert ((rstd.cpu().double() - rs).abs() <= 28 * U * rs).all()
    sc = torch.from_numpy(a).double() * rs / 127
    assert ((scale.cpu().double() - sc).abs() <= 30 * U * sc).all()
    n = h64 * rs[:, None] * w64
    tol = (30 * U + (2.0 ** -8 if dtype == BF16 else 0)) * n.abs()
    assert ((normed.cpu().double() - n).abs() <= tol).all()


@pytest.mark.gpu
def test_norm_edge_rows():
    """Zero rows, one value, ties of the code, huge and tiny rows; in place; without rstd."""
    K = 256
    x = torch.zeros((7, K))
    x[1, 5] = -3.0
    x[2, :] = 2.0
    x[2, 0] = 127.0
    x[2, 1:9] = torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5, -126.5])
    x[3, :] = torch.randn(K, generator=syn.gen(1)) * 1e16
    x[4, :] = torch.randn(K, generator=syn.gen(2)) * 1e-18
    x[5, 3] = 2.0 ** -149
    x[6, :] = -1.0
    w = torch.ones(K)
    w[200:] = 0.0
    buf = x.cuda()
    xq, scale, h, rstd = bl.rmsnorm_quantize(buf, w.cuda(), torch.zeros_like(buf), h=buf)
    assert h.data_ptr() == buf.data_ptr() and bl.get_device_status() == 0
    q, a = _codes_of(x * w)
    np.testing.assert_array_equal(xq.cpu().numpy(), q)
    rs = 1.0 / (x.double().square().mean(-1) + 1e-5).sqrt()
    assert ((rstd.cpu().double() - rs).abs() <= 28 * U * rs).all()
    assert scale[0] == 0 and (xq[0] == 0).all()
    sc = torch.from_numpy(a).double() * rs / 127
    assert ((scale.cpu().double() - sc).abs() <= 30 * U * sc + 2.0 ** -149).all()
    lib = bl.load_library()
    again = torch.empty_like(xq)
    assert lib.bitlinear_rmsnorm_quantize(
        buf.data_ptr(), None, 0, w.cuda().data_ptr(), 0, 1e-5, 7, K, None, None, again.data_ptr(),
        scale.data_ptr(), None, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(again, xq)


@pytest.mark.gpu
def test_norm_writes_its_own_rows_only():
    """Outputs that are the first rows of larger buffers: what lies behind stays."""
    M, K = 5, 1536
    x, r, w = _rows(M, K, BF16, 11, True)
    bufs = [torch.full((M + 1, K), 3, dtype=t, device="cuda") for t in (torch.int8, BF16, BF16)]
    vecs = [torch.full((M + 4,), 3.0, device="cuda") for _ in range(2)]
    bl.rmsnorm_quantize(x.cuda(), w.cuda(), r.cuda(), xq=bufs[0][:M], h=bufs[1][:M], normed=bufs[2][:M],
                        scale=vecs[0][:M], rstd=vecs[1][:M])
    for t in bufs:
        assert (t[M] == 3).all() and not (t[:M] == 3).all()
    for t in vecs:
        assert (t[M:] == 3).all() and not (t[:M] == 3).any()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38])
def test_norm_reports_nonfinite_rows(bad):
    x = torch.ones((3, 128))
    x[1, 77] = bad
    bl.rmsnorm_quantize(x.cuda(), torch.ones(128).cuda())
    assert bl.get_device_status() == 6
    bl.rmsnorm_quantize(torch.ones((3, 128)).cuda(), torch.ones(128).cuda())
    assert bl.get_device_status() == 0


def _backward_reference(g, h, w, rstd, gh):
    g, h, w, rs = g.double(), h.double(), w.double(), rstd.double()[:, None]
    hat, d = h * rs, g * w
    mean = (d * hat).mean(-1, keepdim=True)
    gx = rs * (d - hat * mean)
    mag = rs * (d.abs() + hat.abs() * mean.abs())
    slack = rs * hat.abs() * 52 * U * (d * hat).abs().mean(-1, keepdim=True)
    if gh is not None:
        gx, mag = gx + gh.double(), mag + gh.double().abs()
    return gx, 8 * U * mag + slack, (g * hat).sum(0), (g * hat).abs().sum(0)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,htype,gtype,otype,past", [
    (1, 64, BF16, F32, BF16, True), (1, 8192, F32, F32, F32, False), (5, 1536, BF16, BF16, F32, True),
    (777, 1536, F32, F32, F32, True), (300, 4160, BF16, F32, BF16, True), (40, 8256, BF16, BF16, BF16, False),
    (9, 28672, BF16, F32, F32, True), (3, 32768, F32, BF16, F32, False), (1500, 320, BF16, F32, BF16, True),
    (2, 16384, F32, F32, BF16, True),
])
def test_backward_matches_formula(M, K, htype, gtype, otype, past):
    h, _, w = _rows(M, K, htype, M + 7 * K, False)
    g = (torch.randn((M, K), generator=syn.gen(K)) * 0.01).to(gtype)
    gh = (torch.randn((M, K), generator=syn.gen(K + 1)) * 0.01).to(otype) if past else None
    rstd = (1.0 / (h.double().square().mean(-1) + 1e-5).sqrt()).float()
    gx, gw = bl.rmsnorm_backward(g.cuda(), h.cuda(), w.cuda(), rstd.cuda(), grad_h=_cuda(gh), out_dtype=otype)
    rx, tol, rw, aw = _backward_reference(g, h, w, rstd, gh)
    assert ((gx.cpu().double() - rx).abs() <= tol + (2.0 ** -8 if otype == BF16 else 0) * rx.abs()).all()
    assert ((gw.cpu().double() - rw).abs() <= (M + 4) * U * aw).all()
    # the same bits again, and with grad_x in grad_h's memory
    into = gh.cuda() if past else torch.empty_like(gx)
    gx2, gw2 = bl.rmsnorm_backward(g.cuda(), h.cuda(), w.cuda(), rstd.cuda(),
                                   grad_h=into if past else None, grad_x=into)
    assert torch.equal(gx, gx2) and torch.equal(gw, gw2)


@pytest.mark.gpu
def test_backward_matches_differences():
    """Central differences, in 64 bits, of L = sum g n + sum gh h with n = h rstd w."""
    M, K, eps = 3, 128, 1e-5
    x, r, w = _rows(M, K, F32, 5, True)
    g = torch.randn((M, K), generator=syn.gen(8))
    gh = torch.randn((M, K), generator=syn.gen(9))
    _, _, h, rstd = bl.rmsnorm_quantize(x.cuda(), w.cuda(), r.cuda(), eps=eps)
    gx, gw = bl.rmsnorm_backward(g.cuda(), h, w.cuda(), rstd, grad_h=gh.cuda())
    h64 = h.cpu().double()

    def loss(h, w):
        n = h / (h.square().mean(-1, keepdim=True) + eps).sqrt() * w
        return (g.double() * n + gh.double() * h).sum()

    step = 1e-5
    for t, k in ((0, 0), (1, 77), (2, 127), (2, 5)):
        e = torch.zeros_like(h64)
        e[t, k] = step
        want = (loss(h64 + e, w.double()) - loss(h64 - e, w.double())) / (2 * step)
        # the difference quotient's own error: step^2 times third derivatives, cancellation 1e-16 / step
        assert abs(gx[t, k].item() - want.item()) <= 1e-4 * (1 + abs(want.item()))
        e = torch.zeros(K, dtype=torch.float64)
        e[k] = step
        want = (loss(h64, w.double() + e) - loss(h64, w.double() - e)) / (2 * step)
        assert abs(gw[k].item() - want.item()) <= 1e-4 * (1 + abs(want.item()))


@pytest.mark.gpu
@pytest.mark.parametrize("wtype", [F32, BF16])
@pytest.mark.parametrize("K", [128, 1536, 28672])
@pytest.mark.parametrize("bad,under", [(float("nan"), 1.0), (float("nan"), 0.0), (float("inf"), 1.0),
                                       (float("inf"), 0.0), (-float("inf"), 0.0)])
def test_norm_reports_nonfinite_gains(bad, under, K, wtype):
    """A NaN in the gain, or an infinite gain over a zero, makes p NaN and leaves the sum of squares finite."""
    for dtype in (F32, BF16):
        x = torch.ones((3, K), dtype=dtype)
        x[:, K - 3] = under
        w = torch.ones(K)
        w[K - 3] = bad
        bl.rmsnorm_quantize(x.cuda(), w.to(wtype).cuda())
        assert bl.get_device_status() == 6
        bl.rmsnorm_quantize(x.cuda(), torch.ones(K, dtype=wtype).cuda())
        assert bl.get_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("K,dtype", [(28672, BF16), (20480, BF16), (32768, F32), (3200, F32), (1536, BF16)])
@pytest.mark.parametrize("every", [8, 16, 64])
def test_norm_statistics_of_squares_lost_one_by_one(K, dtype, every):
    """A large square followed by many of just under half its last place: a running sum drops each of them
    whole, which for 64 in a row is 31 u of rstd, beyond the 28 u stated above."""
    x = torch.full((200, K), 2.0 ** -12 * (1 - 2.0 ** -8), dtype=dtype)
    nv = K // 8
    ones = nv // (every // 8)
    x[:, : 8 * ones : 8] = 1.0
    _, scale, _, rstd = bl.rmsnorm_quantize(x.cuda(), torch.ones(K).cuda(), eps=1e-10)
    assert bl.get_device_status() == 0
    rs = 1.0 / (x.double().square().mean(-1) + 1e-10).sqrt()
    assert ((rstd.cpu().double() - rs).abs() <= 28 * U * rs).all()
    assert ((scale.cpu().double() - rs / 127).abs() <= 30 * U * rs / 127).all()


@pytest.mark.gpu
def test_norm_reports_rows_whose_normalised_values_pass_fp32():
    """One value in a row of 64 is 8 after the norm; a gain of 3e38 is finite, and so is p."""
    x = torch.zeros((2, 64))
    x[1, 3] = 1.0
    w = torch.full((64,), 4e37)
    bl.rmsnorm_quantize(x.cuda(), w.cuda(), eps=1e-12)
    assert bl.get_device_status() == 0
    w[3] = 3e38
    bl.rmsnorm_quantize(x.cuda(), w.cuda(), eps=1e-12)
    assert bl.get_device_status() == 6


@pytest.mark.gpu
def test_rows_beyond_4_gb():
    """fp32 rows that begin past 2^32 bytes, forward and backward, against the same rows alone."""
    K = 16384
    M = (1 << 31) // K - 1  # the largest batch of these rows
    last = torch.randn((3, K), generator=syn.gen(1)).cuda()
    w = (1.0 + 0.2 * torch.randn(K, generator=syn.gen(2))).cuda()
    x = torch.zeros((M, K), device="cuda")
    x[-3:] = last
    xq, scale, h, rstd = bl.rmsnorm_quantize(x, w, x, h=x)  # x + x, in place
    xq1, scale1, h1, rstd1 = bl.rmsnorm_quantize(last, w, last)
    assert torch.equal(xq[-3:], xq1) and torch.equal(h[-3:], h1) and (xq[:-3] == 0).all()
    assert ((rstd[-3:] - rstd1).abs() <= 2 * 28 * U * rstd1).all()
    assert ((scale[-3:] - scale1).abs() <= 2 * 30 * U * scale1).all()
    del xq
    g = torch.zeros((M, K), device="cuda")
    g[-3:] = last.flip(1)
    g1, rs = g[-3:].clone(), rstd.clone()
    rs[-3:] = rstd1
    gx, gw = bl.rmsnorm_backward(g, h, w, rs)
    gx1, gw1 = bl.rmsnorm_backward(g1, h1, w, rstd1)
    assert torch.equal(gx[-3:], gx1) and (gx[:-3] == 0).all()
    mag = (g1.double() * h1.double() * rstd1.double()[:, None]).abs().sum(0)
    assert ((gw - gw1).abs() <= 2 * 7 * U * mag).all()
    assert bl.get_device_status() == 0
