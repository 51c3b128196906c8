"""GPU tests of lfa_rotary and lfa_group_norm / lfa_group_norm_backward against 64-bit forms
(tests/token_ref.py), and of the layer that decay attention, rotary and norm make up.

Tolerances.
  * rotary: y = mscale (a c - b s): three fp32 roundings, the cosine's and sine's own error (the reduced angle
    is rounded to fp32, 2^-24 of at most pi, sincospif adds 2 units: 2^-22 absolute), so 8 * 2^-24 *
    mscale (|a| + |b|); bf16 adds half a step, 2^-8 |y|.
  * group norm: the mean of n values is within c 2^-24 of mean|x| with c = 64 (sums run over short chains that
    are joined in trees), the variance about it likewise, so xhat is within c 2^-24 (|x| + mean|x|) rstd plus c
    2^-24 |xhat|; gamma and the activation (slope at most 1.13, expf / erff within 4 units) carry that on; bf16
    adds 2^-8 |y|.
  * its gradients: sums of n terms in such chains (c 2^-24 of the sum of absolute values), dx adds the same
    for each of its three terms; bf16 adds 2^-8 |dx|.
"""
import pytest
import torch

from laplacian_nystr_attention_avg_b200 import decay
from tests import token_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _tok(B, H, N, d, dtype, g, order):
    t = torch.randn((B, H, N, d) if order == "bhnd" else (B, N, H, d), generator=g, device="cuda").to(dtype)
    return t if order == "bhnd" else t.transpose(1, 2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(8, 2), (64, 64), (128, 96), (128, 128), (72, 20), (40, 6), (256, 128)])
@pytest.mark.parametrize("B,N,H,H2,order", [(1, 1, 1, 0, "bhnd"), (3, 37, 5, 2, "bnhd")])
def test_rotary(B, N, H, H2, order, d, rot, layout, dtype):
    g = torch.Generator("cuda").manual_seed(d + rot)
    x, x2 = _tok(B, H, N, d, dtype, g, order), (_tok(B, H2, N, d, dtype, g, order) if H2 else None)
    pos = torch.randint(0, 2 ** 31 - 1, (B, N), generator=g, device="cuda").to(torch.int32)
    pos[0, 0] = 0
    if N > 2:
        pos[:, 1], pos[:, 2] = 2 ** 31 - 1, -5
    freqs, _ = decay.rotary_frequencies(rot)
    for inverse in (False, True):
        y, y2 = decay.rotary(x, pos, freqs, x2=x2, layout=layout, mscale=1.25, inverse=inverse)
        for src, out in ((x, y), (x2, y2)):
            if src is None:
                assert out is None
                continue
            ref = R.rotate(src.double(), pos, freqs, layout == "interleaved", 1.25, inverse)
            T = 1.25 * (src.double().abs() + R.rotate(src.double().abs(), torch.zeros_like(pos), freqs, False, 1.0, False).amax(-1, keepdim=True))
            bound = 8 * U * T + (2.0 ** -8 * ref.abs() if dtype == BF else 0)
            assert ((out.double() - ref).abs() <= bound).all()
            assert torch.equal(out[..., rot:], src[..., rot:])
        z, z2 = x.clone(), None if x2 is None else x2.clone()
        decay.rotary(z, pos, freqs, x2=z2, layout=layout, mscale=1.25, inverse=inverse, out=z, out2=z2)   # in place
        assert torch.equal(z, y) and (z2 is None or torch.equal(z2, y2))


def test_rotary_inverse_is_the_transpose():
    """<rotary(x), u> = <x, rotary(u, inverse)> for every x and u; the rotation is linear, so this is its gradient."""
    g = torch.Generator("cuda").manual_seed(3)
    x, u = _tok(2, 3, 50, 64, F32, g, "bnhd"), _tok(2, 3, 50, 64, F32, g, "bhnd")
    pos = torch.randint(0, 10 ** 6, (2, 50), generator=g, device="cuda").to(torch.int32)
    freqs, ms = decay.rotary_frequencies(48, scaling="ramp", factor=8.0, context=4096)
    for layout in ("half", "interleaved"):
        y, _ = decay.rotary(x, pos, freqs, layout=layout, mscale=ms)
        w, _ = decay.rotary(u, pos, freqs, layout=layout, mscale=ms, inverse=True)
        a, b = float((y.double() * u).sum()), float((x.double() * w).sum())
        assert abs(a - b) <= 32 * U * float((y.double() * u).abs().sum())
        assert abs(a) > 1.0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotary_many_tokens_and_heads(dtype):
    g = torch.Generator("cuda").manual_seed(4)
    x = _tok(2, 33, 1001, 64, dtype, g, "bnhd")
    pos = torch.arange(2002, device="cuda", dtype=torch.int32).view(2, 1001)
    freqs, _ = decay.rotary_frequencies(64)
    y, _ = decay.rotary(x, pos, freqs)
    ref = R.rotate(x.double(), pos, freqs, False, 1.0, False)
    bound = 8 * U * 2 * x.double().abs().amax(-1, keepdim=True) + (2.0 ** -8 * ref.abs() if dtype == BF else 0)
    assert ((y.double() - ref).abs() <= bound).all()


# ---- group norm ---------------------------------------------------------------------------------------

C_SUM = 64
SHAPES = [(1, 1, 8, 1), (1, 1, 8, 8), (5, 1, 64, 4), (777, 1, 1024, 16), (3, 49, 40, 4), (2, 3136, 64, 32), (2, 784, 320, 32),
          (3, 130, 10, 1), (2, 257, 72, 9), (1, 6000, 24, 3), (4, 2, 2304, 32), (2, 1000, 512, 1), (1, 12544, 256, 8)]


def _norm_inputs(B, N, C, dtype, affine, offset, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    x = (torch.randn((B, N, C), generator=g, device="cuda") + offset).to(dtype)
    gamma = 1 + 0.3 * torch.randn((C,), generator=g, device="cuda") if affine else None
    beta = 0.3 * torch.randn((C,), generator=g, device="cuda") if affine else None
    return x, gamma, beta, g


def _d(t):
    return None if t is None else t.double()


def _xhat_error(x, groups, eps):
    """Bound on the error of xhat, and xhat, elementwise in 64 bits."""
    g = x.reshape(x.shape[0], x.shape[1], groups, -1)
    mean = g.mean((1, 3), keepdim=True)
    rstd = (((g - mean) ** 2).mean((1, 3), keepdim=True) + eps) ** -0.5
    xh = (g - mean) * rstd
    err = C_SUM * U * ((g.abs() + g.abs().mean((1, 3), keepdim=True)) * rstd + xh.abs())
    # an error e of the mean moves the variance by e^2 only; the rounding of x - mean moves it like xhat
    err = err + xh.abs() * C_SUM * U * (g.abs().mean((1, 3), keepdim=True) * rstd)
    return err.reshape(x.shape), xh.reshape(x.shape), mean, rstd


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("B,N,C,G", SHAPES)
def test_group_norm(B, N, C, G, act, dtype):
    affine = (B + N) % 2 == 1 or act != "none"
    x, gamma, beta, _ = _norm_inputs(B, N, C, dtype, affine, 0.5, C + N)
    y, mean, rstd = decay.group_norm(x, G, gamma, beta, eps=1e-5, act=act)
    ref, rm, rr = R.group_norm(x.double(), G, _d(gamma), _d(beta), 1e-5, act)
    err, xh, _, _ = _xhat_error(x.double(), G, 1e-5)
    scale = 1.0 if gamma is None else gamma.double().abs()
    z = xh * scale + (0 if beta is None else beta.double().abs())
    bound = 1.13 * (err * scale + 4 * U * z.abs()) + 16 * U * (z.abs() + ref.abs()) + (2.0 ** -8 * ref.abs() if dtype == BF else 0) + 1e-30
    bad = (y.double() - ref).abs() > bound
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {float(((y.double() - ref).abs() / bound).max()):.3g}"
    ma = x.double().abs().reshape(B, N, G, -1).mean((1, 3))
    assert ((mean.double() - rm).abs() <= C_SUM * U * ma).all()
    assert ((rstd.double() - rr).abs() <= C_SUM * U * rr * (1 + ma * rr)).all()
    z = x.clone()
    decay.group_norm(z, G, gamma, beta, act=act, out=z)     # in place
    assert torch.equal(z, y)


def test_group_norm_of_values_far_from_zero():
    """mean 1000, deviation 1, in fp32: a difference of sums of squares would lose everything."""
    x, gamma, beta, _ = _norm_inputs(2, 500, 64, F32, True, 1000.0, 1)
    y, mean, rstd = decay.group_norm(x, 8, gamma, beta)
    ref, rm, rr = R.group_norm(x.double(), 8, _d(gamma), _d(beta), 1e-5, "none")
    err, _, _, _ = _xhat_error(x.double(), 8, 1e-5)
    assert ((y.double() - ref).abs() <= err * gamma.double().abs() + 16 * U * (ref.abs() + 1)).all()


def test_group_norm_of_constant_groups():
    x = torch.full((2, 30, 16), 3.0, device="cuda")
    y, mean, rstd = decay.group_norm(x, 4, act="none", eps=1e-5)
    assert (y == 0).all() and (mean == 3).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)


def _norm_grads(x, dy, G, gamma, beta, eps, act):
    leaves = [t.double().requires_grad_() for t in (x, gamma, beta) if t is not None]
    ga, be = (leaves[1], leaves[2]) if gamma is not None else (None, None)
    y, _, _ = R.group_norm(leaves[0], G, ga, be, eps, act)
    return torch.autograd.grad((y * dy.double()).sum(), leaves)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("B,N,C,G", SHAPES)
def test_group_norm_backward(B, N, C, G, act, dtype):
    affine = (B + N) % 2 == 1 or act != "none"
    if N * (C // G) < 8:
        affine = False
    x, gamma, beta, g = _norm_inputs(B, N, C, dtype, affine, 0.5, C + N)
    dy = torch.randn((B, N, C), generator=g, device="cuda").to(dtype)
    _, mean, rstd = decay.group_norm(x, G, gamma, beta, act=act)
    dx, dgamma, dbeta = decay.group_norm_backward(x, dy, mean, rstd, G, gamma, beta, act=act)
    grads = _norm_grads(x, dy, G, gamma, beta, 1e-5, act)
    err, xh, _, rs = _xhat_error(x.double(), G, 1e-5)
    sc = torch.ones(C, dtype=torch.float64, device="cuda") if gamma is None else gamma.double().abs()
    # dz = dy act'(z) with |act''| <= 0.8 on an error of z, and |act'| <= 1.13
    edz = dy.double().abs() * (0.8 * (err * sc + 4 * U * (xh.abs() * sc + 1)) + 8 * U * 1.13)
    adz = 1.13 * dy.double().abs()

    def grouped(t):
        return t.reshape(B, N, G, -1)

    gz, egz = grouped(adz * sc), grouped(edz * sc + 2 * U * adz * sc)
    m1, em1 = gz.mean((1, 3), keepdim=True), egz.mean((1, 3), keepdim=True)
    gx, egx = gz * grouped(xh).abs(), egz * grouped(xh).abs() + gz * grouped(err)
    m2, em2 = gx.mean((1, 3), keepdim=True), egx.mean((1, 3), keepdim=True)
    size = gz + m1 + grouped(xh).abs() * m2
    bound = rs * (egz + em1 + grouped(xh).abs() * em2 + grouped(err) * m2 + C_SUM * U * size)
    bound = bound + C_SUM * U * (1 + grouped(x.double().abs()).mean((1, 3), keepdim=True) * rs) * rs * size
    bound = bound.reshape(x.shape) + (2.0 ** -8 * grads[0].abs() if dtype == BF else 0) + 1e-30
    bad = (dx.double() - grads[0]).abs() > bound
    assert not bad.any(), f"dx: {int(bad.sum())}, worst {float(((dx.double() - grads[0]).abs() / bound).max()):.3g}"
    if gamma is None:
        assert dgamma is None and dbeta is None
    else:
        eb = edz.sum((0, 1)) + C_SUM * U * adz.sum((0, 1))
        eg = (edz * xh.abs() + adz * err).sum((0, 1)) + C_SUM * U * (adz * xh.abs()).sum((0, 1))
        assert ((dbeta.double() - grads[2]).abs() <= eb).all()
        assert ((dgamma.double() - grads[1]).abs() <= eg).all()
    d2 = dy.clone()
    _, dg2, db2 = decay.group_norm_backward(x, d2, mean, rstd, G, gamma, beta, act=act, dx=d2)   # in place of dy
    assert torch.equal(d2, dx)
    if gamma is not None:
        assert torch.equal(dg2, dgamma) and torch.equal(db2, dbeta)


def test_group_norm_gradient_against_differences():
    x, gamma, beta, g = _norm_inputs(2, 40, 24, F32, True, 0.5, 5)
    dy = torch.randn(x.shape, generator=g, device="cuda")
    _, mean, rstd = decay.group_norm(x, 3, gamma, beta, act="silu")
    grads = decay.group_norm_backward(x, dy, mean, rstd, 3, gamma, beta, act="silu")
    at, h = [x, gamma, beta], 2.0 ** -6
    for i in range(3):
        u = torch.randn(at[i].shape, generator=g, device="cuda")

        def loss(sign):
            a = [t + sign * h * u if j == i else t for j, t in enumerate(at)]
            return float((decay.group_norm(a[0], 3, a[1], a[2], act="silu")[0].double() * dy).sum())

        diff = (loss(1) - loss(-1)) / (2 * h)
        want = float((grads[i].double() * u).sum())
        n = float(u.norm())
        # the step's third-order term: h^2 / 6 times a third derivative of the size of the gradient's own
        # terms (|u|^3 summed), and the loss's rounding 2^-24 sqrt(terms) / h
        assert abs(diff - want) <= h * h * n * float(dy.norm()) + 2.0 ** -20 / h * float(dy.norm()), i


@pytest.mark.parametrize("dtype", [BF, F32])
def test_repeated_calls_graph_and_stream(dtype):
    x, gamma, beta, g = _norm_inputs(3, 700, 96, dtype, True, 0.5, 6)
    dy = torch.randn(x.shape, generator=g, device="cuda").to(dtype)

    def both(stream=None):
        y, m, r = decay.group_norm(x, 8, gamma, beta, act="gelu", stream=stream)
        return (y, m, r) + decay.group_norm_backward(x, dy, m, r, 8, gamma, beta, act="gelu", stream=stream)

    want = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = both(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = both()
    for _ in range(3):
        gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_more_than_32_bits_of_elements():
    """2.3e9 elements: rows from both ends against the same rows alone."""
    B, C, G = 70000, 32768, 64
    x = torch.empty((B, 1, C), dtype=BF, device="cuda")
    x.copy_(torch.arange(C, device="cuda").remainder(97).to(BF) * 0.1)
    x[0] += 1
    x[-1] *= -2
    y, mean, rstd = decay.group_norm(x, G, act="silu")
    rows = torch.tensor([0, 1, B // 2, B - 1], device="cuda")
    want, m, r = decay.group_norm(x[rows].contiguous(), G, act="silu")
    assert torch.equal(y[rows], want) and torch.equal(mean[rows], m) and torch.equal(rstd[rows], r)
    freqs, _ = decay.rotary_frequencies(128)
    pos = torch.arange(B, device="cuda", dtype=torch.int32).view(1, B)
    v = x.view(1, B, C // 128, 128).transpose(1, 2)
    z, _ = decay.rotary(v, pos, freqs, out=y.view(1, B, C // 128, 128).transpose(1, 2))
    w, _ = decay.rotary(v[:, :, rows].contiguous(), pos[:, rows].contiguous(), freqs)
    assert torch.equal(z[:, :, rows], w)


MANY = [(8191, 1, 1024, 16), (8191, 1, 768, 12), (5003, 1, 1280, 20), (120011, 1, 40, 5), (40009, 1, 24, 3), (700, 1, 2392, 299),
        (3, 1, 4099, 4099)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("B,N,C,G", MANY)
def test_group_norm_of_many_tokens(B, N, C, G, act, dtype):
    """Several rounds of samples a thread with a ragged tail, and group counts that are no power of two: the
    tolerances of the shapes above."""
    test_group_norm(B, N, C, G, act, dtype)
    test_group_norm_backward(B, N, C, G, act, dtype)


def test_tokens_past_32_bits_of_elements():
    """2.3e9 elements in groups of one vector a thread: rows from both ends against the same rows alone (a sample's
    arithmetic does not depend on its place), and dgamma, dbeta of the three rows whose dy is not zero."""
    B, C, G = 2200000, 1024, 16
    g = torch.Generator("cuda").manual_seed(12)
    rows = torch.tensor([0, 1, B // 2, B - 1], device="cuda")
    few = torch.randn((4, 1, C), generator=g, device="cuda").to(BF)
    dfew = torch.randn((4, 1, C), generator=g, device="cuda").to(BF)
    ga, be = 1 + 0.3 * torch.randn(C, generator=g, device="cuda"), 0.3 * torch.randn(C, generator=g, device="cuda")
    x, dy = (torch.zeros((B, 1, C), dtype=BF, device="cuda") for _ in range(2))
    x[rows], dy[rows] = few, dfew
    y, mean, rstd = decay.group_norm(x, G, ga, be, act="silu")
    want, m, r = decay.group_norm(few, G, ga, be, act="silu")
    assert torch.equal(y[rows], want) and torch.equal(mean[rows], m) and torch.equal(rstd[rows], r)
    dx, dg, db = decay.group_norm_backward(x, dy, mean, rstd, G, ga, be, act="silu", dx=y)
    w, wg, wb = decay.group_norm_backward(few, dfew, m, r, G, ga, be, act="silu")
    assert torch.equal(dx[rows], w)
    # four terms each, joined in another order: three roundings of a partial sum, at most the sum of absolute terms
    xh = ((few.double().view(4, G, -1) - m.double()[..., None]) * r.double()[..., None]).view(4, 1, C)
    adz = 1.13 * dfew.double().abs()
    assert ((dg - wg).double().abs() <= 8 * U * (adz * xh.abs()).sum((0, 1))).all()
    assert ((db - wb).double().abs() <= 8 * U * adz.sum((0, 1))).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("B,N,C,G", [(1, 1, 4096, 512), (2, 49, 4096, 64), (2, 1024, 4096, 8)])
def test_activations_from_end_to_end(B, N, C, G, act, dtype):
    """gamma = 0 leaves z = beta, so y = act(beta), and with dy = 1 in one row dbeta = act'(beta), in all three ways
    through the data. Relative to themselves (U = 2^-24; subnormal results to fp32's smallest step, some of them in
    the factors): silu in fp32: expf 2 units of 2U, 1 + e and the reciprocal 3U, three products 3U: 16 U; its slope is
    p + z p q of factors like that: 32 U of the two terms. gelu: the tail's smooth factor 2^-21, expf 2 units of 2U, its
    argument z^2 / 2 rounded twice, z^2 U, products 4U: (24 + 2 z^2) U in value and slope. In bf16, half a step, and
    ex2 of a rounded argument: |z| U more for silu, z^2 U for gelu, whose smooth factor is within 2^-16; silu below
    z = -87, where the exponential leaves fp32, is within 1e-35 of its value."""
    beta = torch.cat([torch.linspace(-14, 14, C // 2), torch.linspace(-101, 100, C - C // 2)]).cuda()
    g = torch.Generator("cuda").manual_seed(7)
    x = torch.randn((B, N, C), generator=g, device="cuda").to(dtype)
    gamma = torch.zeros(C, device="cuda")
    y, mean, rstd = decay.group_norm(x, G, gamma, beta, act=act)
    z = beta.double()
    if act == "silu":
        p, q = torch.sigmoid(z), torch.sigmoid(-z)
        value, terms, each = z * p, (p, z * p * q), 32 * U + 0 * z
        if dtype == BF:
            each = each + 4 * z.abs() * U
    else:
        cdf = 0.5 * torch.special.erfc(-z * 0.5 ** 0.5)
        value, terms = z * cdf, (cdf, z * torch.exp(-0.5 * z * z) * 0.3989422804014327)
        each = (24 + 2 * z * z) * U
        if dtype == BF:
            each = each + 2 * z * z * U + 2.0 ** -16
    tiny = 2.0 ** -140 if dtype == F32 else 1e-35
    ref = value.expand(B, N, C)
    bound = each * value.abs() + (2.0 ** -8 * value.abs() if dtype == BF else 0) + tiny
    bad = (y.double() - ref).abs() > bound
    assert not bad.any(), f"{int(bad.sum())}, z from {float(z.expand(B, N, C)[bad].min())} to {float(z.expand(B, N, C)[bad].max())}"
    dy = torch.zeros((B, N, C), dtype=dtype, device="cuda")
    dy[-1, -1] = 1
    _, _, dbeta = decay.group_norm_backward(x, dy, mean, rstd, G, gamma, beta, act=act)
    slope = terms[0] + terms[1]
    size = terms[0].abs() + terms[1].abs()
    if act == "silu" and dtype == BF:   # p (1 - p) from the rounded p: 2 U |z| p
        size = size + z.abs() * terms[0] * U / each
    bad = (dbeta.double() - slope).abs() > each * size + tiny
    assert not bad.any(), f"{int(bad.sum())}, z from {float(z[bad].min())} to {float(z[bad].max())}"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,N,C,G", [(5, 1, 64, 4), (3, 49, 40, 4), (2, 257, 72, 9), (3, 130, 10, 1), (2, 3136, 64, 32), (1, 6000, 24, 3)])
def test_values_that_are_not_finite_stay_in_their_group(B, N, C, G, dtype):
    """NaN and infinities in one group of one sample, of x or dy: every other group as without them, bit by bit, and
    dgamma, dbeta of the other groups' channels."""
    x, gamma, beta, g = _norm_inputs(B, N, C, dtype, True, 0.5, 3)
    dy = torch.randn((B, N, C), generator=g, device="cuda").to(dtype)
    at, n = G // 2, C // G
    mine = torch.zeros((B, N, C), dtype=torch.bool, device="cuda")
    mine[-1, :, at * n:(at + 1) * n] = True
    y, m, r = decay.group_norm(x, G, gamma, beta, act="silu")
    grads = decay.group_norm_backward(x, dy, m, r, G, gamma, beta, act="silu")
    for odd in (float("nan"), float("inf"), -float("inf")):
        bad = x.clone()
        bad[-1, N // 2, at * n] = odd
        y1, m1, r1 = decay.group_norm(bad, G, gamma, beta, act="silu")
        assert torch.equal(y1[~mine], y[~mine]) and not torch.isfinite(y1[mine]).any()
        assert torch.equal(torch.isfinite(m1), torch.isfinite(r1)) and int((~torch.isfinite(m1)).sum()) == 1
        bad_dy = dy.clone()
        bad_dy[-1, N // 2, at * n] = odd
        for args in ((bad, dy, m1, r1), (x, bad_dy, m, r)):
            dx, dg, db = decay.group_norm_backward(*args, G, gamma, beta, act="silu")
            assert torch.equal(dx[~mine], grads[0][~mine]) and not torch.isfinite(dx[mine]).any()
            assert torch.equal(dg[~mine[-1, 0]], grads[1][~mine[-1, 0]]) and torch.equal(db[~mine[-1, 0]], grads[2][~mine[-1, 0]])


# ---- the layer -----------------------------------------------------------------------------------------

def _layer(B, N, H, dk, dv, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    ld = -0.02 * torch.arange(1, H + 1, device="cuda", dtype=F32)
    gamma, beta = 1 + 0.1 * torch.randn(H * dv, generator=g, device="cuda"), 0.1 * torch.randn(H * dv, generator=g, device="cuda")
    freqs, ms = decay.rotary_frequencies(dk // 2, scaling="ntk", factor=4.0)
    mod = decay.DecayAttention(ld, gamma, beta, freqs, mscale=ms, layout="interleaved")
    q, k, v = (torch.randn((B, N, H, d), generator=g, device="cuda") for d in (dk, dk, dv))
    pos = (torch.arange(N, device="cuda") + 100000).to(torch.int32).expand(B, N).contiguous()
    return mod, q, k, v, pos, g


def _layer_ref(mod, q, k, v, pos, S0, gamma, beta):
    B, N, H, dv = v.shape
    qr, kr = (R.rotate(t.transpose(1, 2), pos, mod.freqs, True, mod.mscale, False) for t in (q, k))
    o, S = R.decay_forward(qr, kr, v.transpose(1, 2), mod.log_decay, q.shape[3] ** -0.5, S0, None)
    y, _, _ = R.group_norm(o.transpose(1, 2).reshape(B * N, 1, H * dv), H, gamma, beta, mod.eps, mod.act)
    return y.reshape(B, N, H * dv), S


def test_layer_prompt_steps_and_gradients_fp32():
    """Prompt, then single tokens from its state, then the gradients of the prompt: against the 64-bit layer.
    Everything is fp32; the norm divides by the deviation of a token's head, so the tolerance is 2^-24 times a
    few hundred roundings times the largest ratio of that division: 1e-3 of the output's own size."""
    B, N, H, dk, dv = 2, 150, 4, 32, 64
    mod, q, k, v, pos, g = _layer(B, N + 3, H, dk, dv)
    S0 = torch.randn((B, H, dk, dv), generator=g, device="cuda")
    cut = [t[:, :N].contiguous() for t in (q, k, v)]
    y, S, saved = mod.forward(*cut, pos[:, :N].contiguous(), S0=S0)
    leaves = [t.double().requires_grad_() for t in (*cut, S0, mod.gamma, mod.beta)]
    ry, rS = _layer_ref(mod, *leaves[:3], pos[:, :N], leaves[3], leaves[4], leaves[5])
    assert ((y.double() - ry).abs().max() <= 1e-3 * ry.abs().max())
    assert float((y.double() - ry.detach()).norm() / ry.detach().norm()) <= 1e-5
    dy, dS = torch.randn(y.shape, generator=g, device="cuda"), torch.randn(S.shape, generator=g, device="cuda")
    want = torch.autograd.grad((ry * dy).sum() + (rS * dS).sum(), leaves)
    got = mod.backward(saved, dy, dS)
    for a, b in zip(got, want):
        assert float((a.double() - b).norm() / b.norm()) <= 1e-4
    fy, _ = _layer_ref(mod, q.double(), k.double(), v.double(), pos, S0.double(), mod.gamma.double(), mod.beta.double())
    for t in range(N, N + 3):
        yt = mod.step(q[:, t], k[:, t], v[:, t], S, pos[:, t].contiguous())
        assert float((yt.double() - fy[:, t]).norm() / fy[:, t].norm()) <= 1e-5


def test_layer_bf16_ragged_runs_and_trains():
    B, N, H, dk, dv = 3, 200, 4, 64, 64
    mod, q, k, v, pos, g = _layer(B, N, H, dk, dv, 1)
    q, k, v = (t.to(BF) for t in (q, k, v))
    lengths = torch.tensor([200, 0, 131], dtype=torch.int32, device="cuda")
    for stream in (None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        y, S, saved = mod.forward(q, k, v, pos, lengths=lengths, stream=stream)
        grads = mod.backward(saved, torch.ones_like(y), stream=stream)
        torch.cuda.synchronize()
        assert all(torch.isfinite(t).all() for t in (y, S, *grads))
        assert (grads[0][1] == 0).all() and (grads[0][2, 131:] == 0).all()


def test_norm_graphs_replayed_at_once():
    """Large groups, forward and backward, in two graphs on two streams."""
    g = torch.Generator("cuda").manual_seed(8)
    sets = [[torch.randn((4, 1500, 64), generator=g, device="cuda").to(BF) for _ in range(2)] for _ in range(2)]
    ga, be = (torch.randn(64, generator=g, device="cuda") for _ in range(2))

    def call(x, dy):
        y, m, r = decay.group_norm(x, 4, ga, be, act="silu")
        return (y, m, r) + decay.group_norm_backward(x, dy, m, r, 4, ga, be, act="silu")

    want = [call(*s) for s in sets]
    graphs, got, streams = [], [], [torch.cuda.Stream() for _ in sets]
    for s in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got.append(call(*s))
        graphs.append(gr)
    torch.cuda.synchronize()
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, o))


def test_layer_bf16_ragged_values():
    """Every stage of a ragged bf16 batch against the 64-bit form of the same stage on its valid rows: rotation, the
    norm of o (the tolerances above), o (2^-8 of the sum of absolute terms twice over: weights and state, output), then
    the gradients of the whole backward from the saved tensors. Its roundings to bf16, each at most 2^-8 of what it
    rounds: dO, the weights or state, dq / dk / dv, the rotation. Independent of each other, so normwise within
    sqrt(4) 2^-8 (the rounding errors' own average, 2^-8 / sqrt 3, is the margin)."""
    B, N, H, dk, dv = 3, 300, 4, 64, 48
    mod, q, k, v, pos, g = _layer(B, N, H, dk, dv, 2)
    q, k, v = (t.to(BF) for t in (q, k, v))
    lens = [300, 0, 131]
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    S0 = torch.randn((B, H, dk, dv), generator=g, device="cuda")
    y, S, saved = mod.forward(q, k, v, pos, S0=S0, lengths=lengths)
    qr, kr, _, o = saved[:4]
    valid = torch.arange(N, device="cuda")[None, :] < lengths[:, None]
    for src, out in ((q, qr), (k, kr)):
        ref = R.rotate(src.transpose(1, 2).double(), pos, mod.freqs, True, mod.mscale, False)
        T = mod.mscale * 2 * src.double().abs().transpose(1, 2).amax(-1, keepdim=True)
        assert ((out.double() - ref).abs() <= 8 * U * T + 2.0 ** -8 * ref.abs()).all()
    a = [t.double() for t in (qr, kr, v.transpose(1, 2))]
    ro, rS = R.decay_forward(*a, mod.log_decay, dk ** -0.5, S0.double(), lengths)
    To, TS = R.decay_forward(*(t.abs() for t in a), mod.log_decay, dk ** -0.5, S0.double().abs(), lengths)
    assert ((o.transpose(1, 2).double() - ro).abs() <= 2.0 ** -8 * (ro.abs() + To * (1 + 2.0 ** -6))).all()
    assert ((S.double() - rS).abs() <= 2.0 ** -15 * TS).all()
    ry, _, _ = R.group_norm(o.double().view(B * N, 1, H * dv), H, mod.gamma.double(), mod.beta.double(), mod.eps, mod.act)
    err, xh, _, _ = _xhat_error(o.double().view(B * N, 1, H * dv), H, mod.eps)
    bound = 2 * (err * mod.gamma.double().abs() + 16 * U * (xh.abs() + 1)) + 16 * U * ry.abs() + 2.0 ** -8 * ry.abs()
    assert ((y.view(B * N, 1, -1).double() - ry).abs() <= bound).all()

    dy = torch.randn((B, N, H * dv), generator=g, device="cuda").to(BF) * valid[..., None]
    dS = torch.randn(S.shape, generator=g, device="cuda")
    got = mod.backward(saved, dy, dS)
    leaf_o, ga, be = o.double().view(B * N, 1, -1).requires_grad_(), mod.gamma.double().requires_grad_(), mod.beta.double().requires_grad_()
    z, _, _ = R.group_norm(leaf_o, H, ga, be, mod.eps, mod.act)
    do, dga, dbe = torch.autograd.grad((z * dy.double().view(B * N, 1, -1)).sum(), (leaf_o, ga, be))
    do = do.view(B, N, H, dv).transpose(1, 2)
    dq, dk_, dv_, dS0 = R.decay_grads(*a, mod.log_decay, dk ** -0.5, S0.double(), lengths, do, dS.double())
    dq, dk_ = (R.rotate(t, pos, mod.freqs, True, mod.mscale, True) for t in (dq, dk_))
    want = [dq.transpose(1, 2), dk_.transpose(1, 2), dv_.transpose(1, 2), dS0, dga, dbe]
    for name, x, w, tol in zip(("dq", "dk", "dv", "dS0", "dgamma", "dbeta"), got, want, [2 * 2.0 ** -8] * 4 + [2.0 ** -16] * 2):
        assert x.shape == w.shape
        rel = float((x.double() - w).norm() / w.norm())
        assert rel <= tol, f"{name}: {rel:.2e}"
        if name in ("dq", "dk", "dv"):
            assert (x[~valid] == 0).all(), name


def test_layer_takes_gradients_of_any_layout():
    """dy of a sum is one broadcast number, and a slice of a wider tensor has gaps: as their contiguous copies."""
    B, N, H, dk, dv = 2, 70, 4, 32, 64
    mod, q, k, v, pos, g = _layer(B, N, H, dk, dv, 3)
    y, S, saved = mod.forward(q, k, v, pos)
    wide = torch.randn((B, N, 2 * H * dv), generator=g, device="cuda")
    for dy in (torch.ones((), device="cuda").expand(B, N, H * dv), wide[..., H * dv:], wide.view(B, 2 * H * dv, N)[:, :H * dv].transpose(1, 2)):
        got, want = mod.backward(saved, dy), mod.backward(saved, dy.contiguous())
        assert all(torch.equal(a, b) for a, b in zip(got, want))
