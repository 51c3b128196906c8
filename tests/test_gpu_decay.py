"""GPU tests of the decay attention calls (lfa_decay_forward, lfa_decay_backward, lfa_decay_step) against the
dense causal form in 64 bits (tests/token_ref.py).

Tolerances. T denotes the same form on absolute values (|q|, |k|, |v|, |S0|): the sum that every rounding
is relative to.
  * fp32: every output is a sum of products whose worst-case rounding is (terms) 2^-24 T: at most 128 products
    of channels, 128 tokens within a chunk and one addition per chunk, plus 16 for the factors (expf and
    expm1f within 2 units, their argument's rounding 2^-24 |n log_decay|, at most 88 of which leave a
    number above fp32's range of underflow), so bound (128 + 128 + N/32 + 16 + 88) 2^-24 T.
  * bf16: the output's own rounding 2^-8 |o| (half a step of bf16), one bf16 rounding (2^-8) of each weight
    decay^(i-j) q_i.k_j or of the state that q meets: 2^-8 T in the worst case, plus the fp32 bound. Normwise,
    for independent random terms the errors add as their squares do and the terms' squares sum to the
    output's, so |err| <= sqrt(2) 2^-8 |o| (taken with 10 % for the finite sample).
  * states of bf16 tensors: fp32 sums of exact products of v with k's decayed rows split in two bf16 parts
    (2^-16 at most), so 2^-16 T plus the fp32 bound; normwise 2^-16 likewise.
"""
import math

import pytest
import torch

from laplacian_nystr_attention_avg_b200 import decay, lfa
from tests import token_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _mk(shape, dtype, g, order="bhnd"):
    B, H, N, d = shape
    if order == "bhnd":
        return torch.randn(shape, generator=g, device="cuda").to(dtype)
    if order == "bnhd":
        return torch.randn((B, N, H, d), generator=g, device="cuda").to(dtype).transpose(1, 2)
    # "packed": a slice of a wider tensor, as one projection for q, k, v leaves it
    return torch.randn((B, N, H, 3 * d), generator=g, device="cuda").to(dtype)[..., d:2 * d].transpose(1, 2)


def _log_decay(H, kind="mixed"):
    vals = {"mixed": [-0.03, -2.0 ** -12, -0.7, 0.0, -8.0, -float("inf")], "slow": [-2.0 ** -10],
            "one": [0.0]}[kind]
    return torch.tensor([vals[i % len(vals)] for i in range(H)], dtype=F32, device="cuda")


def _poison(t, lengths):
    """NaN and infinities on the rows behind each sequence's end."""
    if lengths is not None:
        for b, L in enumerate(lengths.tolist()):
            t[b, :, max(0, L):] = float("nan")
            t[b, :, max(0, L) + 1::2] = float("inf")


def _inputs(B, H, N, dk, dv, dtype, order="bhnd", state=True, lengths=None, kind="mixed", seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    q, k, v = _mk((B, H, N, dk), dtype, g, order), _mk((B, H, N, dk), dtype, g, order), _mk((B, H, N, dv), dtype, g, order)
    S0 = torch.randn((B, H, dk, dv), generator=g, device="cuda") if state else None
    L = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    for t in (q, k, v):
        _poison(t, L)
    return q, k, v, _log_decay(H, kind), S0, L, g


def _clean(t, L):
    t = t.double()
    if L is not None:
        for b, n in enumerate(L.tolist()):
            t[b, :, max(0, n):] = 0
    return t


def _f32_bound(N, T):
    return (128 + 128 + N / 32 + 16 + 88) * 2.0 ** -24 * T + 1e-37


def _check_rows(got, ref, T, N, dtype, what):
    err = (got.double() - ref).abs()
    bound = _f32_bound(N, T)
    if dtype == BF:
        bound = bound + 2.0 ** -8 * ref.abs() + 2.0 ** -8 * T * (1 + 2.0 ** -8)
    assert torch.isfinite(got).all(), what
    bad = err > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} over the bound, worst {float((err / bound).max()):.3g}"
    if dtype == BF and ref.numel() >= 4096:
        rel = float(err.norm() / ref.norm())
        assert rel <= 1.1 * math.sqrt(2) * 2.0 ** -8, f"{what}: normwise {rel:.2e}"


def _check_state(got, ref, T, N, dtype, what):
    err = (got.double() - ref).abs()
    bound = _f32_bound(N, T) + (2.0 ** -16 * T if dtype == BF else 0.0)
    assert torch.isfinite(got).all(), what
    assert not (err > bound).any(), f"{what}: worst {float((err / bound).max()):.3g} of the bound"
    assert float(err.norm() / ref.norm().clamp(min=1e-30)) <= (2.0 ** -16 if dtype == BF else 2e-6), what


def _run_forward(B, H, N, dk, dv, dtype, order="bhnd", state=True, lengths=None, kind="mixed", seed=0):
    q, k, v, ld, S0, L, _ = _inputs(B, H, N, dk, dv, dtype, order, state, lengths, kind, seed)
    scale = dk ** -0.5
    O = torch.full_like(v, 7.0)
    o, S = decay.decay_forward(q, k, v, ld, S0=S0, lengths=L, O=O, return_state=True)
    assert decay.decay_status() == 0
    q, k, v = (_clean(t, L) for t in (q, k, v))
    ro, rS = R.decay_forward(q, k, v, ld, scale, None if S0 is None else S0.double(), L)
    To, TS = R.decay_forward(q.abs(), k.abs(), v.abs(), ld, scale, None if S0 is None else S0.double().abs(), L)
    for b in range(B):
        n = N if L is None else max(0, min(N, int(L[b])))
        assert (o[b, :, n:] == 7.0).all(), "rows behind the end were written"
        _check_rows(o[b, :, :n], ro[b, :, :n], To[b, :, :n], N, dtype, f"o[{b}]")
    _check_state(S, rS, TS, N, dtype, "S")


SIZES = [(8, 8), (16, 64), (64, 64), (40, 128), (128, 128), (72, 24)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1, 2, 31, 33, 127, 128, 129, 257, 640])
def test_forward_lengths(N, dtype):
    _run_forward(2, 6, N, 64, 64, dtype, seed=N)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("order,state", [("bhnd", False), ("bnhd", True), ("packed", True)])
def test_forward_sizes(dk, dv, order, state, dtype):
    _run_forward(2, 3, 300, dk, dv, dtype, order, state, seed=dk + dv)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [32, 128])
def test_forward_ragged_padding_holds_anything(d, dtype):
    _run_forward(7, 6, 400, d, d, dtype, "bnhd", True, [0, 1, 400, 128, 129, 255, 77], seed=d)
    _run_forward(2, 2, 200, d, d, dtype, "bhnd", False, [-3, 1000], seed=d + 1)   # clamped to [0, N]


def test_fp32_channels_of_four():
    _run_forward(1, 2, 70, 12, 20, F32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,N,d", [(1, 1, 9000, 64), (1, 2, 5000, 128), (3, 2, 2500, 32)])
def test_forward_long(B, H, N, d, dtype):
    """Few units over long sequences: the work is split along the sequence."""
    lengths = None if B == 1 else [N, 1300, 1]
    _run_forward(B, H, N, d, d, dtype, "bhnd", True, lengths, "slow", seed=N)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pieces_equal_the_whole(dtype):
    """A sequence in pieces, the state handed on in place, against the sequence at once: same bounds."""
    q, k, v, ld, S0, _, _ = _inputs(1, 4, 700, 64, 48, dtype, "bnhd")
    S = S0.clone()
    parts = []
    for a, b in ((0, 1), (1, 130), (130, 131), (131, 700)):
        o, S = decay.decay_forward(q[:, :, a:b], k[:, :, a:b], v[:, :, a:b], ld, S0=S, S_out=S)
        parts.append(o)
    o = torch.cat(parts, 2)
    ro, rS = R.decay_forward(q.double(), k.double(), v.double(), ld, 64 ** -0.5, S0.double(), None)
    To, TS = R.decay_forward(q.double().abs(), k.double().abs(), v.double().abs(), ld, 64 ** -0.5, S0.double().abs(), None)
    _check_rows(o, ro, To, 700, dtype, "o")
    _check_state(S, rS, TS, 700, dtype, "S")


def _run_backward(B, H, N, dk, dv, dtype, order="bhnd", state=True, lengths=None, kind="mixed", seed=0):
    q, k, v, ld, S0, L, g = _inputs(B, H, N, dk, dv, dtype, order, state, lengths, kind, seed)
    dO = _mk((B, H, N, dv), dtype, g, "bnhd")
    _poison(dO, L)
    dS = torch.randn((B, H, dk, dv), generator=g, device="cuda") if state else None
    scale = dk ** -0.5
    outs = [torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").fill_(7.0) for t in (q, k, v)]
    dq, dk_, dv_, dS0 = decay.decay_backward(q, k, v, ld, dO, S0=S0, lengths=L, dS_out=dS, dQ=outs[0], dK=outs[1],
                                             dV=outs[2], return_state=True)
    assert decay.decay_status() == 0
    q, k, v, dO = (_clean(t, L) for t in (q, k, v, dO))
    S0d = None if S0 is None else S0.double()
    dSd = None if dS is None else dS.double()
    ref = R.decay_grads(q, k, v, ld, scale, S0d, L, dO, dSd)
    T = R.decay_grads(q.abs(), k.abs(), v.abs(), ld, scale, None if S0 is None else S0d.abs(), L, dO.abs(),
                      None if dS is None else dSd.abs())
    for name, got, r, t in (("dq", dq, ref[0], T[0]), ("dk", dk_, ref[1], T[1]), ("dv", dv_, ref[2], T[2])):
        for b in range(B):
            n = N if L is None else max(0, min(N, int(L[b])))
            assert (got[b, :, n:] == 7.0).all(), f"{name}: rows behind the end were written"
            _check_rows(got[b, :, :n], r[b, :, :n], t[b, :, :n], N, dtype, f"{name}[{b}]")
    _check_state(dS0, ref[3], T[3], N, dtype, "dS0")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1, 2, 33, 128, 129, 257, 640])
def test_backward_lengths(N, dtype):
    _run_backward(2, 6, N, 64, 64, dtype, seed=N)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("order,state", [("bhnd", False), ("packed", True)])
def test_backward_sizes(dk, dv, order, state, dtype):
    _run_backward(2, 3, 300, dk, dv, dtype, order, state, seed=dk + dv)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [32, 128])
def test_backward_ragged_padding_holds_anything(d, dtype):
    _run_backward(7, 6, 400, d, d, dtype, "bnhd", True, [0, 1, 400, 128, 129, 255, 77], seed=d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,N,d", [(1, 1, 6000, 64), (1, 2, 3500, 128), (3, 1, 2500, 32)])
def test_backward_long(B, H, N, d, dtype):
    lengths = None if B == 1 else [N, 1300, 1]
    _run_backward(B, H, N, d, d, dtype, "bhnd", True, lengths, "slow", seed=N)


def test_gradients_against_differences():
    """O and S are linear in each of q, k, v, S0, so a difference of step 1 is the derivative itself: it must
    agree with <gradient, direction> up to the fp32 rounding of both sides."""
    q, k, v, ld, S0, _, g = _inputs(2, 3, 200, 32, 48, F32)
    dO = _mk(v.shape, F32, g)
    dS = torch.randn(S0.shape, generator=g, device="cuda")

    def loss(q, k, v, S0):
        o, S = decay.decay_forward(q, k, v, ld, S0=S0, return_state=True)
        return float((o.double() * dO).sum() + (S.double() * dS).sum())

    at = [q, k, v, S0]
    grads = decay.decay_backward(q, k, v, ld, dO, S0=S0, dS_out=dS, return_state=True)
    base = loss(*at)
    To, TS = R.decay_forward(*(2 * t.double().abs() for t in (q, k, v)), ld, 32 ** -0.5, 2 * S0.double().abs(), None)
    # The roundings of different outputs are independent, each at most 64 2^-24 (the longest chain of a
    # T-sized output is far shorter on average) of T |dO|: their sum over the outputs has a standard deviation
    # below the root of the sum of squares. Six of those, for the two forwards and the gradient's own sum.
    each = torch.cat([(To * dO.abs()).flatten(), (TS * dS.abs()).flatten()])
    tol = 6 * 64 * 2.0 ** -24 * float(each.norm())
    for i in range(4):
        u = torch.randn(at[i].shape, generator=g, device="cuda")
        moved = [t + u if j == i else t for j, t in enumerate(at)]
        diff = loss(*moved) - base
        want = float((grads[i].double() * (moved[i].double() - at[i].double())).sum())
        assert abs(diff - want) <= tol, (i, diff, want)
        assert abs(want) > 2 * tol, "the direction shows nothing"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 8, 8), (1, 8, 64, 64), (33, 3, 128, 128), (5, 2, 40, 72), (300, 1, 24, 16)])
def test_step(B, H, dk, dv, dtype):
    g = torch.Generator("cuda").manual_seed(B)
    q, k, v = (torch.randn((B, H, d), generator=g, device="cuda").to(dtype) for d in (dk, dk, dv))
    n = B + 4
    S = torch.randn((n, H, dk, dv), generator=g, device="cuda")
    slots = torch.randperm(n, generator=g, device="cuda")[:B].to(torch.int32)
    ld = _log_decay(H)
    S1 = S.clone()
    o = decay.decay_step(q, k, v, ld, S1, slots=slots)
    at = slots.long()
    lam = R.decays(ld, torch.tensor(1, device="cuda"))[:, None, None]
    ref = S.double().clone()
    ref[at] = lam * S.double()[at] + k.double()[..., None] * v.double()[..., None, :]
    T = lam * S.double()[at].abs() + k.double().abs()[..., None] * v.double().abs()[..., None, :]
    assert ((S1.double()[at] - ref[at]).abs() <= 4 * 2.0 ** -24 * T + 1e-37).all()
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(S1[rest], S[rest])
    ro = dk ** -0.5 * (q.double()[..., None, :] @ ref[at]).squeeze(-2)
    To = dk ** -0.5 * (q.double().abs()[..., None, :] @ T).squeeze(-2)
    bound = (dk + 8) * 2.0 ** -24 * To + (2.0 ** -8 * ro.abs() if dtype == BF else 0) + 1e-37
    assert ((o.double() - ro).abs() <= bound).all()


def test_step_slots_that_are_padding_or_named_twice():
    B, H, d = 6, 2, 16
    g = torch.Generator("cuda").manual_seed(1)
    q, k, v = (torch.randn((B, H, d), generator=g, device="cuda") for _ in range(3))
    S = torch.randn((4, H, d, d), generator=g, device="cuda")
    ld = _log_decay(H)
    slots = torch.tensor([2, -1, 0, 2, 4, 0], dtype=torch.int32, device="cuda")
    S1 = S.clone()
    o = decay.decay_step(q, k, v, ld, S1, slots=slots)
    S2 = S.clone()
    o2 = decay.decay_step(q[[0, 2]].contiguous(), k[[0, 2]].contiguous(), v[[0, 2]].contiguous(), ld, S2,
                          slots=torch.tensor([2, 0], dtype=torch.int32, device="cuda"))
    assert torch.equal(S1, S2) and torch.equal(o[[0, 2]], o2)
    assert (o[[1, 3, 4, 5]] == 0).all()


def test_steps_equal_the_prompt_form():
    q, k, v, ld, S0, _, _ = _inputs(2, 4, 20, 32, 64, F32)
    S = S0.clone()
    rows = [decay.decay_step(q[:, :, t], k[:, :, t], v[:, :, t], ld, S) for t in range(20)]
    ro, rS = R.decay_forward(q.double(), k.double(), v.double(), ld, 32 ** -0.5, S0.double(), None)
    To, TS = R.decay_forward(q.double().abs(), k.double().abs(), v.double().abs(), ld, 32 ** -0.5, S0.double().abs(), None)
    _check_rows(torch.stack(rows, 2), ro, To, 20, F32, "o")
    _check_state(S, rS, TS, 20, F32, "S")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_repeated_calls_are_bit_identical(dtype):
    q, k, v, ld, S0, _, g = _inputs(2, 3, 1500, 64, 64, dtype)
    dO = _mk(v.shape, dtype, g)
    a = decay.decay_forward(q, k, v, ld, S0=S0, return_state=True) + decay.decay_backward(
        q, k, v, ld, dO, S0=S0, return_state=True)
    for _ in range(5):
        b = decay.decay_forward(q, k, v, ld, S0=S0, return_state=True) + decay.decay_backward(
            q, k, v, ld, dO, S0=S0, return_state=True)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_other_stream_and_graph(dtype):
    q, k, v, ld, S0, _, g = _inputs(1, 4, 2000, 64, 64, dtype)
    dO = _mk(v.shape, dtype, g)
    want = decay.decay_forward(q, k, v, ld, S0=S0, return_state=True) + decay.decay_backward(q, k, v, ld, dO, S0=S0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = decay.decay_forward(q, k, v, ld, S0=S0, return_state=True, stream=s) + decay.decay_backward(
        q, k, v, ld, dO, S0=S0, stream=s.cuda_stream)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got) if a is not None)
    # two graphs, replayed in turn
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(decay.decay_forward(q, k, v, ld, S0=S0, return_state=True) +
                        decay.decay_backward(q, k, v, ld, dO, S0=S0))
        graphs.append(gr)
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, o) if a is not None)


def test_two_streams_at_once():
    """Calls that overlap on the GPU have workspaces of their own."""
    sets = [_inputs(1, 4, 3000, 64, 64, BF, seed=i) for i in range(2)]
    want = [decay.decay_forward(q, k, v, ld, S0=S0, return_state=True) + decay.decay_backward(q, k, v, ld, v, S0=S0)
            for q, k, v, ld, S0, _, _ in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(4):
        for i, (q, k, v, ld, S0, _, _) in enumerate(sets):
            got[i] = decay.decay_forward(q, k, v, ld, S0=S0, return_state=True, stream=streams[i]) + \
                decay.decay_backward(q, k, v, ld, v, S0=S0, stream=streams[i])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g) if a is not None)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_offsets_beyond_32_bits(dtype):
    """Batches more than 2^31 elements apart in one buffer, inputs and output."""
    d, H, N, far = 64, 2, 150, (1 << 31) + 64
    g = torch.Generator("cuda").manual_seed(9)
    buf = torch.empty(far + 4 * H * N * d, dtype=dtype, device="cuda")

    def place(i):
        t = buf.as_strided((2, H, N, d), (far, N * d, d, 1), i * H * N * d)
        t.copy_(torch.randn((2, H, N, d), generator=g, device="cuda"))
        return t

    q, k, v, O = (place(i) for i in range(4))
    ld = _log_decay(H)
    decay.decay_forward(q, k, v, ld, O=O)
    want, _ = decay.decay_forward(q.contiguous(), k.contiguous(), v.contiguous(), ld)
    assert torch.equal(O, want)
    grads = decay.decay_backward(q, k, v, ld, v.contiguous(), dQ=O, dK=None, dV=None)[0] if dtype == F32 else None
    if grads is not None:
        want = decay.decay_backward(q.contiguous(), k.contiguous(), v.contiguous(), ld, v.contiguous())[0]
        assert torch.equal(grads, want)


def test_step_in_a_pool_beyond_32_bits():
    H, d, n = 16, 128, 8300     # 8300 x 262144 floats: the last slots lie behind element 2^31
    S = torch.empty((n, H, d, d), device="cuda")
    g = torch.Generator("cuda").manual_seed(2)
    slots = torch.tensor([0, 8299, 8192], dtype=torch.int32, device="cuda")
    S[slots.long()] = torch.randn((3, H, d, d), generator=g, device="cuda")
    small = S[slots.long()].clone()
    q, k, v = (torch.randn((3, H, d), generator=g, device="cuda") for _ in range(3))
    ld = _log_decay(H)
    o = decay.decay_step(q, k, v, ld, S, slots=slots)
    assert torch.equal(o, decay.decay_step(q, k, v, ld, small))
    assert torch.equal(S[slots.long()], small)


def test_refused_on_the_device():
    q, k, v, ld, _, _, _ = _inputs(2, 2, 40, 16, 16, F32)
    with pytest.raises(ValueError):
        decay.decay_forward(q[:1].expand(2, -1, -1, -1), k, v, ld)
    with pytest.raises(ValueError):
        decay.decay_forward(q, k, v, ld, O=torch.zeros_like(v[:1]).expand(2, -1, -1, -1))
    with pytest.raises(ValueError):
        decay.decay_forward(q, k, v, ld, O=torch.zeros(2, 2, 16, 40, device="cuda").transpose(2, 3))
    with pytest.raises(lfa.LfaError):
        decay.decay_forward(q, k, v, ld, O=v)
    with pytest.raises(ValueError):
        decay.decay_forward(q, k.cpu(), v, ld)
    with pytest.raises(TypeError):
        decay.decay_forward(q, k.double(), v, ld)
    with pytest.raises(ValueError):
        decay.decay_backward(q, k, v, ld, v, dQ=torch.empty_like(q).transpose(1, 2).contiguous().transpose(1, 2))
    assert torch.isfinite(decay.decay_forward(q, k, v, ld)[0]).all()


def test_scale_held_in_a_tensor():
    """A changed value counts, though the object stays."""
    q, k, v, ld, _, _, _ = _inputs(1, 2, 40, 16, 16, F32)
    scale = torch.tensor(0.5)
    first = decay.decay_forward(q, k, v, ld, scale=scale)[0]
    scale.mul_(2)
    assert torch.equal(decay.decay_forward(q, k, v, ld, scale=scale)[0], 2 * first)


def test_two_graphs_replayed_at_once():
    """Each captured graph has a workspace of its own (sequences long enough to be cut in segments)."""
    sets = [_inputs(1, 4, 2500, 64, 64, BF, seed=20 + i) for i in range(2)]
    calls = [lambda s=s: decay.decay_forward(s[0], s[1], s[2], s[3], S0=s[4], return_state=True) +
             decay.decay_backward(s[0], s[1], s[2], s[3], s[2], S0=s[4]) for s in sets]
    want = [f() for f in calls]
    graphs, got, streams = [], [], [torch.cuda.Stream() for _ in sets]
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(f())
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, o) if a is not None)


ONE_SIDED = [F32, BF]
ODD = [float("nan"), float("inf"), -float("inf")]


def _clean_rows(got, ref, T, rows, N, dtype, what, columns=None):
    got, ref, T = (t[..., rows, :] if columns is None else t[..., rows, :][..., columns] for t in (got, ref, T))
    if got.numel():
        _check_rows(got, ref, T, N, dtype, what)


@pytest.mark.parametrize("dtype", ONE_SIDED)
@pytest.mark.parametrize("B,H,N,dk,dv", [(1, 2, 300, 64, 48), (1, 2, 290, 128, 128), (2, 3, 140, 24, 16), (1, 1, 1400, 40, 72)])
@pytest.mark.parametrize("at", [0, 1, 40, 127, 130, 139])
def test_forward_does_not_see_later_tokens(B, H, N, dk, dv, at, dtype):
    """NaN and infinities at one token leave what the formula forms without it: the outputs before it and, for a
    single channel of v, the other channels; for q, every other token."""
    q, k, v, ld, S0, _, _ = _inputs(B, H, N, dk, dv, dtype, "bnhd", seed=at)
    scale = dk ** -0.5
    ro, rS = R.decay_forward(q.double(), k.double(), v.double(), ld, scale, S0.double(), None)
    To, TS = R.decay_forward(q.double().abs(), k.double().abs(), v.double().abs(), ld, scale, S0.double().abs(), None)
    n = torch.arange(N, device="cuda")
    for i, odd in enumerate(ODD):
        for name in "qkv":
            t = {"q": q, "k": k, "v": v}[name].clone(memory_format=torch.preserve_format)
            c = (5 * i + at) % t.shape[3]
            others = torch.arange(t.shape[3], device="cuda") != c
            t[:, :, at, c] = odd
            if name != "v":
                t[:, :, at] = odd
            o, S = decay.decay_forward(*(t if name == m else x for m, x in (("q", q), ("k", k), ("v", v))), ld, S0=S0,
                                       return_state=True)
            _clean_rows(o, ro, To, n != at if name == "q" else n < at, N, dtype, f"{name} {odd}")
            assert not torch.isfinite(o[:, :, at]).all()
            if name == "v":
                _clean_rows(o, ro, To, n >= 0, N, dtype, f"other channels, {odd}", others)
                _check_state(S[..., others], rS[..., others], TS[..., others], N, dtype, "S, other channels")
            if name == "q":
                _check_state(S, rS, TS, N, dtype, "S")
    assert decay.decay_status() == 0


@pytest.mark.parametrize("dtype", ONE_SIDED)
@pytest.mark.parametrize("B,H,N,dk,dv", [(1, 2, 300, 64, 48), (1, 2, 290, 128, 128), (2, 3, 140, 24, 16), (1, 1, 1400, 40, 72)])
@pytest.mark.parametrize("at", [0, 1, 40, 127, 130, 139])
def test_backward_does_not_see_the_other_side(B, H, N, dk, dv, at, dtype):
    """One token's NaN or infinities: dq before it, dk and dv behind it, and what does not meet it at all."""
    q, k, v, ld, S0, _, g = _inputs(B, H, N, dk, dv, dtype, "bnhd", seed=at)
    dO = _mk((B, H, N, dv), dtype, g, "bnhd")
    dS = torch.randn(S0.shape, generator=g, device="cuda")
    at_once = [q, k, v, dO]
    q64, k64, v64, dO64 = (t.double() for t in at_once)
    ref = R.decay_grads(q64, k64, v64, ld, dk ** -0.5, S0.double(), None, dO64, dS.double())
    T = R.decay_grads(q64.abs(), k64.abs(), v64.abs(), ld, dk ** -0.5, S0.double().abs(), None, dO64.abs(), dS.double().abs())
    n = torch.arange(N, device="cuda")
    before, behind, rest = n < at, n > at, n != at
    good = {"q": (n >= 0, behind, behind), "k": (before, n >= 0, rest), "v": (before, rest, n >= 0),
            "dO": (rest, behind, behind)}
    for i, odd in enumerate(ODD):
        for j, name in enumerate(("q", "k", "v", "dO")):
            t = [x.clone(memory_format=torch.preserve_format) if m == j else x for m, x in enumerate(at_once)]
            if i == 0:
                t[j][:, :, at] = odd
            else:
                t[j][:, :, at, (5 * i + at) % t[j].shape[3]] = odd
            got = decay.decay_backward(t[0], t[1], t[2], ld, t[3], S0=S0, dS_out=dS, return_state=True)
            for what, x, r, a, rows in zip(("dq", "dk", "dv"), got, ref, T, good[name]):
                _clean_rows(x, r, a, rows, N, dtype, f"{what}, {name} {odd}")
            if name in "kv":
                _check_state(got[3], ref[3], T[3], N, dtype, "dS0")
    assert decay.decay_status() == 0


LONG = [(40, 64, "bnhd"), (72, 128, "packed"), (128, 24, "bhnd"), (64, 16, "packed")]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv,order", LONG)
def test_segments_of_unequal_widths(dk, dv, order, dtype):
    """Long and ragged sequences of few units, cut in segments, with dk and dv apart: forward and backward."""
    lengths = [2300, 1281, 0, 1]
    _run_forward(4, 2, 2300, dk, dv, dtype, order, True, lengths, "slow", seed=dk)
    _run_backward(4, 2, 2300, dk, dv, dtype, order, True, lengths, "slow", seed=dv)


def test_bf16_gradients_beyond_32_bits():
    """All tensors in one buffer, batches more than 2^31 elements apart, gradients among them."""
    d, H, N, far = 64, 2, 150, (1 << 31) + 64
    g = torch.Generator("cuda").manual_seed(10)
    buf = torch.empty(far + 8 * H * N * d, dtype=BF, device="cuda")
    t = [buf.as_strided((2, H, N, d), (far, N * d, d, 1), i * H * N * d) for i in range(7)]
    for x in t[:4]:
        x.copy_(torch.randn((2, H, N, d), generator=g, device="cuda"))
    q, k, v, dO, dQ, dK, dV = t
    ld = _log_decay(H)
    got = decay.decay_backward(q, k, v, ld, dO, dQ=dQ, dK=dK, dV=dV)
    want = decay.decay_backward(q.contiguous(), k.contiguous(), v.contiguous(), ld, dO.contiguous())
    for a, b, into in zip(got, want, (dQ, dK, dV)):
        assert a is into and torch.equal(a, b)


@pytest.mark.parametrize("B,H,N,dk,dv,lengths", [
    (1, 2, 8, 64, 64, None), (1, 2, 128, 128, 128, None), (1, 2, 4096, 64, 64, None), (2, 3, 1000, 40, 72, [1000, 333]),
    (1, 2, 500, 128, 24, None), (1, 1, 9000, 64, 64, None), (3, 2, 5000, 72, 128, [5000, 0, 700]), (160, 1, 300, 64, 48, None)])
def test_returned_states_of_bf16_tensors_are_fp32(B, H, N, dk, dv, lengths):
    """k's decayed rows keep the 24 bits of their fp32 products (2^-24), so what is left is the tensor cores' sums: three
    parts of 128 tokens in products of 16 make 24 accumulations a chunk, each cutting off 2^-24 on average of a partial
    sum, whose norm is at most the sum's for independent terms. 24 2^-24 of the norm, whether the chunks' states add up
    in one run or in segments."""
    q, k, v, ld, S0, L, g = _inputs(B, H, N, dk, dv, BF, "bnhd", True, lengths, "slow", seed=N)
    dO = _mk((B, H, N, dv), BF, g, "bnhd")
    _poison(dO, L)
    dS = torch.randn(S0.shape, generator=g, device="cuda")
    _, S = decay.decay_forward(q, k, v, ld, S0=S0, lengths=L, return_state=True)
    dS0 = decay.decay_backward(q, k, v, ld, dO, S0=S0, lengths=L, dS_out=dS, return_state=True)[3]
    q, k, v, dO = (_clean(t, L) for t in (q, k, v, dO))
    want = R.decay_forward(q, k, v, ld, dk ** -0.5, S0.double(), L)[1]
    grads = R.decay_grads(q, k, v, ld, dk ** -0.5, S0.double(), L, dO, dS.double())
    for name, got, ref in (("S", S, want), ("dS0", dS0, grads[3])):
        for b in range(B):
            rel = float((got[b].double() - ref[b]).norm() / ref[b].norm())
            assert rel <= 24 * 2.0 ** -24, f"{name}[{b}]: {rel:.2e}"
