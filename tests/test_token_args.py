"""Host-side refusals of the token operators (no device work: every call must fail its checks first), the
frequency table, and the 64-bit forms that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

from laplacian_nystr_attention_avg_b200 import build as lfa_build
from laplacian_nystr_attention_avg_b200 import decay, lfa
from tests import token_ref as R

BAD, UNSUP = lfa.LFA_ERR_INVALID_ARG, lfa.LFA_ERR_UNSUPPORTED
A = 1 << 20   # an aligned non-null address, never used


@pytest.fixture(scope="module")
def lib():
    lfa_build.build()
    return decay.load()


def _dc(**kw):
    strides = {k: kw.pop(k) for k in list(kw) if k.endswith("stride")}
    base = dict(B=2, heads=3, N=5, dk=16, dv=24, dtype=lfa.LFA_BF16, scale=0.25)
    base.update(kw)
    c = decay.DecayConfig(*base.values())
    for k, v in strides.items():
        getattr(c, k)[:] = v
    return c


CONFIGS = [
    (dict(B=0), BAD), (dict(heads=0), BAD), (dict(N=0), BAD), (dict(scale=float("nan")), BAD), (dict(scale=math.inf), BAD),
    (dict(dtype=2), UNSUP), (dict(dk=4), UNSUP), (dict(dk=12), UNSUP), (dict(dk=136), UNSUP), (dict(dv=0), UNSUP),
    (dict(dv=20), UNSUP), (dict(dtype=lfa.LFA_F32, dk=10), UNSUP), (dict(B=1 << 20, heads=1 << 10), UNSUP),
    (dict(N=(1 << 28) + 1), UNSUP),
]
STRIDES = [
    dict(q_stride=(240, 80, 17)), dict(k_stride=(240, 80, -16)), dict(v_stride=(0, 0, 24)), dict(q_stride=(240, 0, 16)),
    dict(o_stride=(360, 120, 16)),        # rows of o overlap
    dict(o_stride=(120, 120, 24)),        # batches share memory with heads
]


def _forward(lib, c, **kw):
    a = dict(Q=A, K=2 * A, V=3 * A, ld=A, S0=None, L=None, O=4 * A, S=None, ws=A, n=1 << 30)
    a.update(kw)
    return lib.lfa_decay_forward(c, a["Q"], a["K"], a["V"], a["ld"], a["S0"], a["L"], a["O"], a["S"], a["ws"], a["n"], None)


def _backward(lib, c, **kw):
    a = dict(Q=A, K=2 * A, V=3 * A, ld=A, S0=None, L=None, dO=4 * A, dS=None, dQ=5 * A, dK=6 * A, dV=7 * A, dS0=None,
             ws=A, n=1 << 30)
    a.update(kw)
    return lib.lfa_decay_backward(c, *(a[k] for k in ("Q", "K", "V", "ld", "S0", "L", "dO", "dS", "dQ", "dK", "dV", "dS0",
                                                      "ws", "n")), None)


@pytest.mark.parametrize("kw,want", CONFIGS)
def test_decay_refuses_configs(lib, kw, want):
    c = _dc(**kw)
    assert lib.lfa_decay_workspace_size(c, 0) == 0 and lib.lfa_decay_workspace_size(c, 1) == 0
    assert _forward(lib, c) == want and _backward(lib, c) == want
    assert lib.lfa_decay_step(c, A, A, A, A, A, None, 8, 4 * A, None) == want


@pytest.mark.parametrize("kw", STRIDES)
def test_decay_refuses_strides(lib, kw):
    c = _dc(**kw)
    assert _forward(lib, c) == BAD
    if "o_stride" not in kw:
        assert _backward(lib, c) == BAD


def test_decay_gradients_may_not_overlap_themselves(lib):
    assert _backward(lib, _dc(k_stride=(240, 80, 8))) == BAD


@pytest.mark.parametrize("kw", [dict(Q=None), dict(K=None), dict(V=None), dict(O=None), dict(ld=None), dict(Q=A + 8),
                                dict(O=A + 2), dict(S0=A + 4), dict(S=A + 8), dict(O=A), dict(O=3 * A)])
def test_decay_forward_refuses_pointers(lib, kw):
    assert _forward(lib, _dc(), **kw) == BAD


@pytest.mark.parametrize("kw", [dict(Q=None), dict(dO=None), dict(dQ=None), dict(dK=A + 2), dict(dV=None), dict(dS=A + 4),
                                dict(dS0=A + 4), dict(dQ=A), dict(dK=4 * A), dict(dQ=6 * A), dict(dV=5 * A),
                                dict(S0=8 * A, dS0=8 * A), dict(dS=8 * A, dS0=8 * A)])
def test_decay_backward_refuses_pointers(lib, kw):
    assert _backward(lib, _dc(), **kw) == BAD


def test_decay_step_refuses(lib):
    step = lib.lfa_decay_step
    ok = _dc(N=1)
    assert step(_dc(N=2), A, A, A, A, A, None, 8, 4 * A, None) == BAD
    assert step(ok, A, A, A, A, A, None, 1, 4 * A, None) == BAD       # two rows, one state
    assert step(ok, A, A, A, A, A, A, 0, 4 * A, None) == BAD
    for i in (0, 1, 2, 3, 4):
        p = [A] * 5
        p[i] = None
        assert step(ok, *p, None, 8, 4 * A, None) == BAD
    assert step(ok, A, A, A, A, A + 8, None, 8, 4 * A, None) == BAD
    assert step(ok, A, A, A, A, A, None, 8, None, None) == BAD


def test_decay_workspace_sizes(lib):
    for N in (1, 128, 129, 65536):
        for bwd in (0, 1):
            n = lib.lfa_decay_workspace_size(_dc(B=1, heads=1, N=N), bwd)
            assert n >= 256 and n % 256 == 0
    c = _dc(B=1, heads=1, N=65536)          # split along the sequence: the states need room
    for call, bwd in ((_forward, 0), (_backward, 1)):
        n = lib.lfa_decay_workspace_size(c, bwd)
        assert n > 256
        assert call(lib, c, ws=None) == BAD and call(lib, c, ws=A + 16, n=n) == BAD and call(lib, c, n=n - 1) == BAD


def _rc(**kw):
    base = dict(B=2, N=5, d=64, rot=32, heads=3, heads2=0, dtype=lfa.LFA_BF16, interleaved=0, inverse=0, mscale=1.0)
    base.update(kw)
    strides = {k: base.pop(k) for k in list(base) if k.endswith("stride")}
    c = decay.RotaryConfig(*base.values())
    for k, v in strides.items():
        getattr(c, k)[:] = v
    return c


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), BAD), (dict(N=0), BAD), (dict(heads=0), BAD), (dict(heads2=-1), BAD), (dict(mscale=math.nan), BAD),
    (dict(rot=0), BAD), (dict(rot=31), BAD), (dict(rot=66), BAD), (dict(d=4), UNSUP), (dict(d=60), UNSUP), (dict(d=264), UNSUP),
    (dict(d=256, rot=130), UNSUP), (dict(dtype=5), UNSUP), (dict(y_stride=(960, 320, 32)), BAD), (dict(x_stride=(960, 320, 65)), BAD),
    (dict(B=1 << 11, N=1 << 20), UNSUP),
])
def test_rotary_refuses_configs(lib, kw, want):
    assert lib.lfa_rotary(_rc(**kw), A, None, A, A, 2 * A, None, None) == want


def test_rotary_refuses_pointers(lib):
    r, c = lib.lfa_rotary, _rc()
    assert r(c, None, None, A, A, 2 * A, None, None) == BAD
    assert r(c, A, None, None, A, 2 * A, None, None) == BAD
    assert r(c, A, None, A, None, 2 * A, None, None) == BAD
    assert r(c, A, None, A, A, None, None, None) == BAD
    assert r(c, A + 2, None, A, A, 2 * A, None, None) == BAD
    assert r(c, A, A, A, A, 2 * A, 3 * A, None) == BAD                # a second tensor without heads2
    assert r(_rc(heads2=2), A, None, A, A, 2 * A, None, None) == BAD  # heads2 without a second tensor
    assert r(_rc(x_stride=(960, 64, 192)), A, None, A, A, A, None, None) == BAD   # in place, other strides
    two = _rc(heads2=3)
    assert r(two, A, 2 * A, A, A, 3 * A, 3 * A, None) == BAD           # one output for both
    assert r(two, A, 2 * A, A, A, 2 * A, A, None) == BAD               # crossed over


def _nc(**kw):
    base = dict(B=2, N=5, C=64, groups=4, dtype=lfa.LFA_BF16, act=1, eps=1e-5)
    base.update(kw)
    return decay.NormConfig(*base.values())


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), BAD), (dict(N=0), BAD), (dict(C=0), BAD), (dict(groups=0), BAD), (dict(groups=3), BAD), (dict(eps=0.0), BAD),
    (dict(eps=math.nan), BAD), (dict(act=3), BAD), (dict(act=-1), BAD), (dict(dtype=2), UNSUP), (dict(B=1 << 16, N=1 << 16), UNSUP),
    (dict(N=1 << 20, C=1 << 12), UNSUP),
])
def test_norm_refuses_configs(lib, kw, want):
    c = _nc(**kw)
    assert lib.lfa_group_norm_workspace_size(c, 0) == 0
    assert lib.lfa_group_norm(c, A, A, A, 2 * A, A, A, A, 1 << 30, None) == want
    assert lib.lfa_group_norm_backward(c, A, A, A, A, A, A, 2 * A, A, A, A, 1 << 30, None) == want


def test_norm_refuses_pointers(lib):
    f, b, c = lib.lfa_group_norm, lib.lfa_group_norm_backward, _nc()
    n = 1 << 30
    for p in ([None, A, A, 2 * A, A, A, A, n], [A, A, None, 2 * A, A, A, A, n], [A, None, A, 2 * A, A, A, A, n],
              [A, A, A, None, A, A, A, n], [A, A, A, 2 * A, None, A, A, n], [A + 2, A, A, 2 * A, A, A, A, n]):
        assert f(c, *p, None) == BAD
    big = _nc(N=1 << 16)                     # in row chunks: needs a workspace
    assert lib.lfa_group_norm_workspace_size(big, 0) > 256
    for p in ([A, A, A, 2 * A, A, A, None, n], [A, A, A, 2 * A, A, A, A, 256], [A, A, A, 2 * A, A, A, A + 16, n]):
        assert f(big, *p, None) == BAD
    for p in ([None, A, A, A, A, A, 2 * A, A, A, A, n], [A, None, A, A, A, A, 2 * A, A, A, A, n],
              [A, A, None, A, A, A, 2 * A, A, A, A, n], [A, A, A, A, A, A, 2 * A, None, A, A, n],
              [A, A, A, A, None, None, 2 * A, A, A, A, n], [A, A, A, A, A, A, None, A, A, A, n],
              [A, A, A, A, A, A, 2 * A, A, A, A, 0]):
        assert b(c, *p, None) == BAD


def test_binding_refuses_host_tensors_and_wrong_kinds():
    q = torch.zeros(1, 2, 4, 16)
    ld = torch.zeros(2)
    with pytest.raises(ValueError):
        decay.decay_forward(q, q, q, ld)
    with pytest.raises(ValueError):
        decay.decay_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], ld, torch.zeros(1, 2, 16, 16))
    with pytest.raises(TypeError):
        decay.decay_forward(q.half(), q, q, ld)
    with pytest.raises(ValueError):
        decay.decay_forward(q[:, :, :0], q, q, ld)
    with pytest.raises(TypeError):
        decay.group_norm([1.0], 1)
    with pytest.raises(ValueError):
        decay.group_norm(torch.zeros(2, 3, 8), 2)
    with pytest.raises(ValueError):
        decay.rotary(q, torch.zeros(1, 4, dtype=torch.int32), torch.ones(4, dtype=torch.float64), layout="other")


def test_rotary_frequencies():
    f, ms = decay.rotary_frequencies(64, device="cpu")
    assert f.dtype == torch.float64 and ms == 1.0 and f[0] == 1.0 and abs(float(f[31]) - 10000.0 ** (-62 / 64)) < 1e-15
    lin, _ = decay.rotary_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin, f / 4, rtol=1e-15)
    ntk, _ = decay.rotary_frequencies(64, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == 1.0 and abs(float(ntk[31] / f[31]) - 0.25) < 1e-12
    ramp, ms = decay.rotary_frequencies(64, scaling="ramp", factor=4.0, context=2048, device="cpu")
    turns = f * 2048 / (2 * math.pi)
    assert torch.equal(ramp[turns > 40], f[turns > 40]) and torch.allclose(ramp[turns < 0.7], f[turns < 0.7] / 4, rtol=1e-12)
    assert ((ramp <= f) & (ramp >= f / 4 * (1 - 1e-12))).all() and abs(ms - (0.1 * math.log(4) + 1)) < 1e-15
    for kw in (dict(rot=3), dict(rot=0), dict(rot=8, base=1.0), dict(rot=8, factor=0.5), dict(rot=8, scaling="x"),
               dict(rot=8, scaling="ramp"), dict(rot=8, scaling="ramp", context=10, fast=1.0, slow=2.0)):
        with pytest.raises(ValueError):
            decay.rotary_frequencies(device="cpu", **kw)


def test_dense_form_is_the_recurrence():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(2, 3, 17, d, generator=g, dtype=torch.float64) for d in (4, 4, 6))
    S0 = torch.randn(2, 3, 4, 6, generator=g, dtype=torch.float64)
    ld = torch.tensor([-0.1, 0.0, -float("inf")])
    lengths = torch.tensor([17, 5])
    o, S = R.decay_forward(q, k, v, ld, 0.5, S0, lengths)
    for b in range(2):
        st = S0[b].clone()
        for t in range(int(lengths[b])):
            st = torch.exp(ld.double())[:, None, None] * st + k[b, :, t, :, None] * v[b, :, t, None, :]
            assert torch.allclose(o[b, :, t], 0.5 * (q[b, :, t, None] @ st)[:, 0], atol=1e-12)
        assert torch.allclose(S[b], st, atol=1e-12)


def test_a_small_workspace_is_not_taken_for_none(lib):
    # the backward's channel sums of 8 channels are 64 bytes: the size must still differ from "none is used"
    for C, groups in ((8, 1), (8, 8), (4, 2)):
        c = _nc(B=1, N=1, C=C, groups=groups, dtype=lfa.LFA_F32)
        n = lib.lfa_group_norm_workspace_size(c, 1)
        assert n > 256
        assert lib.lfa_group_norm_backward(c, A, A, A, A, A, A, 2 * A, A, A, None, 0, None) == BAD


@pytest.mark.parametrize("shape,strides", [((2, 2, 4, 8), (0, 0, 0, 1)), ((2, 2, 4, 8), (0, 32, 8, 1)),
                                           ((2, 1, 1, 8), (0, 0, 0, 1)), ((2, 3, 8), (0, 0, 1)), ((1, 3, 8), (8, 0, 1))])
def test_broadcast_tensors_are_refused(shape, strides):
    """All strides zero would read as contiguous to the library, beyond the tensor's memory."""
    t = torch.zeros(1024).as_strided(shape, strides)
    with pytest.raises(ValueError, match="broadcast"):
        decay._tokens(t, "q", shape, torch.float32, t.device)
    one = torch.zeros(8).as_strided((1, 1, 1, 8), (0, 0, 0, 1))   # a single row is not broadcast
    assert decay._tokens(one, "q", (1, 1, 1, 8), torch.float32, one.device) == (0, 0, 0, 1)


def test_sizes_past_32_bits_are_refused():
    """The library's fields are 32-bit ints: 2^32 + 1 must not come in as 1. (Meta tensors hold no memory.)"""
    def of(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="meta")

    many, ld = (1 << 32) + 1, of(1, dtype=torch.float32)
    calls = [lambda: decay.group_norm(of(many, 1, 8), 1), lambda: decay.group_norm(of(2, 3, 8), (1 << 32) + 4),
             lambda: decay.group_norm(of(2, 3, 8), -(1 << 32) + 4),
             lambda: decay.group_norm_backward(of(1, many, 8), of(1, many, 8), ld, ld, 1),
             lambda: decay.rotary(of(1, 1, many, 8), None, None),
             lambda: decay.decay_forward(of(many, 1, 1, 8), of(many, 1, 1, 8), of(many, 1, 1, 8), ld),
             lambda: decay.decay_backward(of(1, many, 1, 8), None, None, ld, None),
             lambda: decay.decay_step(of(1, many, 8), None, None, ld, None)]
    for call in calls:
        with pytest.raises(ValueError, match="32 bits"):
            call()
    assert decay._size((1 << 31) - 1, "n") == (1 << 31) - 1 and decay._size(-(1 << 31), "n") == -(1 << 31)
    with pytest.raises(ValueError, match="empty"):
        decay.group_norm(of(0, 1, 8), 1)


@pytest.mark.parametrize("G", [3, 5, 6, 12, 20, 40, 96])
@pytest.mark.parametrize("dtype,es", [(lfa.LFA_BF16, 2), (lfa.LFA_F32, 4)])
def test_per_token_norm_backward_takes_one_wave(lib, G, dtype, es):
    """The backward's workspace holds 2 C sums per record, and a block (256 threads in teams of T, a team per group of
    one token) fills 256 / T / G records. At most 2 blocks an SM run at once: more would leave a few to run alone."""
    n = 64
    T = n * es // 16   # one 16-byte vector a thread
    c = _nc(B=20000, N=1, C=n * G, groups=G, dtype=dtype)
    records = (lib.lfa_group_norm_workspace_size(c, 1) - 256) // (2 * n * G * 4)
    assert 0.9 * 296 <= records * G / (256 // T) <= 296


@pytest.mark.parametrize("B,C,G,dtype,es", [(1, 131064, 16383, lfa.LFA_BF16, 2), (1, (1 << 20) - 1, (1 << 20) - 1, lfa.LFA_F32, 4),
                                            (3, 8 * 299, 299, lfa.LFA_BF16, 2), (1, 24, 3, lfa.LFA_BF16, 2), (2, 4099, 4099, lfa.LFA_BF16, 2)])
def test_norm_backward_workspace_follows_the_data(lib, B, C, G, dtype, es):
    """Channel sums are two floats per channel and record; there are never more than twice as many records as rows."""
    n = lib.lfa_group_norm_workspace_size(_nc(B=B, N=1, C=C, groups=G, dtype=dtype), 1)
    assert 256 < n <= 512 + 2 * B * 2 * C * 4


@pytest.mark.parametrize("units,N,dk,dv,bwd,segs", [
    (147, 1024, 128, 128, 0, 1), (64, 1024, 128, 128, 0, 1), (37, 1024, 128, 128, 0, 8), (8, 8000, 128, 128, 0, 63),
    (24, 2048, 128, 128, 1, 1), (36, 2048, 128, 128, 1, 4), (147, 784, 32, 64, 0, 1), (64, 784, 64, 64, 0, 7),
    (64, 784, 32, 64, 0, 7), (12, 2048, 64, 128, 1, 16), (30, 2048, 128, 64, 1, 6), (30, 2048, 64, 128, 1, 6)])
def test_fp32_segments_count_blocks(lib, units, N, dk, dv, bwd, segs):
    """A block takes 64 columns of a unit's run, and at more than 64 rows of the state one fills an SM: units whose
    blocks fill most of the SMs by themselves are not cut. The workspace holds one state (backward: two) per segment of a cut call."""
    n = lib.lfa_decay_workspace_size(_dc(B=units, heads=1, N=N, dk=dk, dv=dv, dtype=lfa.LFA_F32), bwd)
    states = units * segs * dk * dv * 4 * (2 if bwd else 1)
    assert n == 256 + (states if segs > 1 else 0)


@pytest.mark.parametrize("units,N,d,bwd,segs", [
    (8, 1024, 128, 0, 8), (8, 512, 128, 0, 1), (24, 1024, 128, 0, 4), (24, 1024, 128, 1, 1), (40, 1024, 64, 0, 1),
    (40, 2048, 128, 0, 3), (70, 1024, 64, 0, 1), (70, 2048, 64, 0, 1), (74, 4096, 128, 0, 2), (8, 2048, 64, 0, 16), (8, 65536, 64, 0, 18),
    (147, 65536, 64, 0, 1), (148, 65536, 64, 0, 1), (1, 128, 64, 0, 1)])
def test_bf16_segments_win_their_cost(lib, units, N, d, bwd, segs):
    """Segments cost two launches, a join and a second reading: no call is cut for less."""
    n = lib.lfa_decay_workspace_size(_dc(B=units, heads=1, N=N, dk=d, dv=d), bwd)
    assert n == 256 + (units * segs * d * d * 4 * (2 if bwd else 1) if segs > 1 else 0)
