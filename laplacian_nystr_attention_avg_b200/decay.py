"""Token operators of liblfa.so (include/lfa.h): linear attention with a decay per head (prompt form,
backward, single token), rotary positions, group norm with an activation, and the layer they make up.

Argument checks and marshalling only: every step runs in the library's CUDA kernels. Attention tensors are
[B, heads, N, d] with any strides for batch, head and token (a transposed [B, N, heads, d] needs no copy;
broadcast ones are refused), bfloat16 or float32, channels contiguous. Work is enqueued on `stream` (default: the current stream of the
tensors' device); buffers that a call makes itself belong to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional, Tuple

import torch

from . import lfa
from .lfa import LFA_BF16, LFA_F32, _check, _ptr, _require

ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
_DTYPES = {torch.bfloat16: LFA_BF16, torch.float32: LFA_F32}
_L3 = ctypes.c_longlong * 3


class DecayConfig(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("heads", ctypes.c_int), ("N", ctypes.c_int), ("dk", ctypes.c_int),
                ("dv", ctypes.c_int), ("dtype", ctypes.c_int), ("scale", ctypes.c_float), ("q_stride", _L3),
                ("k_stride", _L3), ("v_stride", _L3), ("o_stride", _L3)]


class RotaryConfig(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("d", ctypes.c_int), ("rot", ctypes.c_int),
                ("heads", ctypes.c_int), ("heads2", ctypes.c_int), ("dtype", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("inverse", ctypes.c_int), ("mscale", ctypes.c_float),
                ("x_stride", _L3), ("x2_stride", _L3), ("y_stride", _L3), ("y2_stride", _L3)]


class NormConfig(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("C", ctypes.c_int), ("groups", ctypes.c_int),
                ("dtype", ctypes.c_int), ("act", ctypes.c_int), ("eps", ctypes.c_float)]


_lib: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """The library with the token operators' signatures declared (raises if it has not been built)."""
    global _lib
    if _lib is None:
        lib = lfa.load()
        vp, sz, ci = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        dc, rc, nc = (ctypes.POINTER(c) for c in (DecayConfig, RotaryConfig, NormConfig))
        for name, res, args in (
                ("lfa_decay_workspace_size", sz, [dc, ci]),
                ("lfa_decay_forward", ci, [dc] + [vp] * 9 + [sz, vp]),
                ("lfa_decay_backward", ci, [dc] + [vp] * 13 + [sz, vp]),
                ("lfa_decay_step", ci, [dc] + [vp] * 6 + [ci, vp, vp]),
                ("lfa_decay_status", ci, [vp]),
                ("lfa_rotary", ci, [rc] + [vp] * 7),
                ("lfa_group_norm_workspace_size", sz, [nc, ci]),
                ("lfa_group_norm", ci, [nc] + [vp] * 7 + [sz, vp]),
                ("lfa_group_norm_backward", ci, [nc] + [vp] * 10 + [sz, vp])):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


# ---- checks -------------------------------------------------------------------------------------

def _tokens(t: torch.Tensor, name: str, shape, dtype, device) -> Tuple[int, ...]:
    """Reject a token tensor the library cannot address; returns its batch, head and token strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    st = t.stride()
    if st[-1] != 1:
        raise ValueError(f"{name}: channels must be contiguous (strides {st})")
    if 0 in st and any(n > 1 and a == 0 for n, a in zip(shape, st)):   # three zeros mean contiguous to the library
        raise ValueError(f"{name}: a broadcast tensor (strides {st}); give a contiguous copy")
    return st


def _size(n, name: str) -> int:
    """A size that the library's 32-bit fields hold (ctypes would keep the low 32 bits of any other)."""
    n = int(n)
    if not -1 << 31 <= n < 1 << 31:
        raise ValueError(f"{name}: {n} does not fit 32 bits")
    return n


def _first(t: torch.Tensor, name: str, dims: int) -> torch.device:
    """The tensor that sets a call's sizes, dtype and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name}: expected {dims} dimensions, got shape {tuple(t.shape)}")
    if t.numel() == 0:
        raise ValueError(f"{name}: empty (shape {tuple(t.shape)})")
    for n in t.shape:
        _size(n, f"{name}: a size")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name}: dtype {t.dtype}, expected bfloat16 or float32")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: on {t.device}, expected a CUDA device")
    return t.device


def _state(t: Optional[torch.Tensor], name: str, shape, device) -> None:
    if t is not None:
        _require(t, name, shape, torch.float32, device)


@contextlib.contextmanager
def _switched(device: int, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device)
            with torch.cuda.stream(s):
                yield


# the plain query: CUDA is up wherever there is a CUDA tensor
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _in(device: int, stream):
    """Context in which a run of calls and allocations goes to `stream` of the device."""
    if stream is None and device == torch.cuda.current_device():
        return contextlib.nullcontext()
    return _switched(device, stream)


def _elsewhere(t, stream) -> bool:
    """Whether a call on tensor t has to leave the current device or stream (see _switched)."""
    return isinstance(t, torch.Tensor) and t.is_cuda and (stream is not None or t.get_device() != _current_device())


def _cur(device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device)


# Checked configurations by the shapes, strides, dtypes and devices of a call's arguments: a repeated shape is
# checked once.
_plans = {}


def _plan(kind, extra, tensors, check):
    """check()'s answer for arguments of these shapes (errors are raised anew each time)."""
    try:
        key = (kind, extra, *[None if t is None else (t.shape, t.stride(), t.dtype, t.get_device()) for t in tensors])
        plan = _plans.get(key)
    except (AttributeError, TypeError, RuntimeError):
        key = plan = None
    if plan is None:
        plan = check()
        if key is not None:
            if len(_plans) >= 4096:
                _plans.clear()
            _plans[key] = plan
    return plan


def _number(x):
    """A scale as the value it has now: one held in a tensor may change under the same object."""
    return None if x is None else float(x)


def _workspace(nbytes: int, device: torch.device) -> Optional[torch.Tensor]:
    """A call's workspace (torch allocations are 512-byte aligned). None where it uses none, or refuses its
    configuration: the call itself then says why."""
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes > 256 else None


# ---- decay attention -------------------------------------------------------------------------------

def _decay_config(q, k, v, log_decay, lengths, scale):
    device = _first(q, "q", 4)
    B, heads, N, dk = q.shape
    if not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("v: expected a 4-dimensional tensor")
    dv = _size(v.shape[3], "v: channels")
    cfg = DecayConfig(B, heads, N, dk, dv, _DTYPES[q.dtype], dk ** -0.5 if scale is None else float(scale))
    cfg.q_stride[:] = _tokens(q, "q", (B, heads, N, dk), q.dtype, device)[:3]
    cfg.k_stride[:] = _tokens(k, "k", (B, heads, N, dk), q.dtype, device)[:3]
    cfg.v_stride[:] = _tokens(v, "v", (B, heads, N, dv), q.dtype, device)[:3]
    _require(log_decay, "log_decay", (heads,), torch.float32, device)
    if lengths is not None:
        _require(lengths, "lengths", (B,), torch.int32, device)
    return cfg, device


def _new(like: torch.Tensor, lengths) -> torch.Tensor:
    return torch.empty_like(like) if lengths is None else torch.zeros_like(like)


def _strided_like(like: torch.Tensor, lengths) -> torch.Tensor:
    t = torch.empty_strided(like.shape, like.stride(), dtype=like.dtype, device=like.device)
    return t if lengths is None else t.zero_()


def decay_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, *, scale=None,
                  S0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                  O: Optional[torch.Tensor] = None, S_out: Optional[torch.Tensor] = None,
                  return_state: bool = False, stream=None):
    """Causal linear attention with a decay per head (lfa_decay_forward): o_t = scale sum_{j<=t}
    exp(log_decay (t-j)) (q_t . k_j) v_j plus the part of S0. Returns (O, S_out).

    q, k [B, heads, N, dk], v [B, heads, N, dv]; log_decay float32 [heads]; scale defaults to dk ** -0.5;
    S0, S_out float32 [B, heads, dk, dv] (S_out may be S0; made if return_state, else None if not given);
    lengths int32 [B]: rows of O behind a sequence's end stay as they were (zeros in an O made here).
    """
    if _elsewhere(q, stream):
        with _switched(q.get_device(), stream):
            return decay_forward(q, k, v, log_decay, scale=scale, S0=S0, lengths=lengths, O=O, S_out=S_out,
                                 return_state=return_state)
    lib = load()

    def check():
        cfg, device = _decay_config(q, k, v, log_decay, lengths, scale)
        state = (cfg.B, cfg.heads, cfg.dk, cfg.dv)
        _state(S0, "S0", state, device)
        _state(S_out, "S_out", state, device)
        cfg.o_stride[:] = _tokens(_new(v, lengths) if O is None else O, "O", v.shape, q.dtype, device)[:3]
        return cfg, device, state, lib.lfa_decay_workspace_size(cfg, 0)

    cfg, device, state, nbytes = _plan("forward", _number(scale), (q, k, v, log_decay, S0, lengths, O, S_out), check)
    if O is None:
        O = _new(v, lengths)
    if S_out is None and return_state:
        S_out = torch.empty(state, dtype=torch.float32, device=device)
    ws = _workspace(nbytes, device)
    _check(lib.lfa_decay_forward(cfg, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(S0),
                                 _ptr(lengths), O.data_ptr(), _ptr(S_out), _ptr(ws), nbytes,
                                 _cur(device.index)), "lfa_decay_forward")
    return O, S_out


def decay_backward(q, k, v, log_decay, dO, *, scale=None, S0=None, lengths=None, dS_out=None, dQ=None, dK=None,
                   dV=None, dS0=None, return_state: bool = False, stream=None):
    """Gradients of <dO, O> + <dS_out, S_out> (lfa_decay_backward). Returns (dQ, dK, dV, dS0).

    dO [B, heads, N, dv]; dQ, dK, dV need the strides of q, k, v (made so if not given); dS0 is made if
    return_state. Rows behind a sequence's end stay as they were (zeros in tensors made here). log_decay gets no
    gradient.
    """
    if _elsewhere(q, stream):
        with _switched(q.get_device(), stream):
            return decay_backward(q, k, v, log_decay, dO, scale=scale, S0=S0, lengths=lengths, dS_out=dS_out, dQ=dQ,
                                  dK=dK, dV=dV, dS0=dS0, return_state=return_state)
    lib = load()

    def check():
        cfg, device = _decay_config(q, k, v, log_decay, lengths, scale)
        state = (cfg.B, cfg.heads, cfg.dk, cfg.dv)
        for name, t in (("S0", S0), ("dS_out", dS_out), ("dS0", dS0)):
            _state(t, name, state, device)
        cfg.o_stride[:] = _tokens(dO, "dO", v.shape, q.dtype, device)[:3]
        for name, t, like in (("dQ", dQ, q), ("dK", dK, k), ("dV", dV, v)):
            if t is not None:
                st = _tokens(t, name, like.shape, q.dtype, device)
                if any(n > 1 and a != b for n, a, b in zip(like.shape, st, like.stride())):
                    raise ValueError(f"{name}: strides {st}, expected {like.stride()}")
        return cfg, device, state, lib.lfa_decay_workspace_size(cfg, 1)

    cfg, device, state, nbytes = _plan("backward", _number(scale),
                                       (q, k, v, log_decay, dO, S0, lengths, dS_out, dQ, dK, dV, dS0), check)
    dQ, dK, dV = (_strided_like(like, lengths) if t is None else t for t, like in ((dQ, q), (dK, k), (dV, v)))
    if dS0 is None and return_state:
        dS0 = torch.empty(state, dtype=torch.float32, device=device)
    ws = _workspace(nbytes, device)
    _check(lib.lfa_decay_backward(cfg, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(S0),
                                  _ptr(lengths), dO.data_ptr(), _ptr(dS_out), dQ.data_ptr(), dK.data_ptr(),
                                  dV.data_ptr(), _ptr(dS0), _ptr(ws), nbytes, _cur(device.index)),
           "lfa_decay_backward")
    return dQ, dK, dV, dS0


def decay_step(q, k, v, log_decay, S, *, scale=None, slots=None, O=None, stream=None) -> torch.Tensor:
    """One token of every row (lfa_decay_step): S is updated in place, returns o [B, heads, dv].

    q, k [B, heads, dk], v [B, heads, dv]; S float32 [n_slots, heads, dk, dv]; row b uses S[slots[b]]
    (slots int32 [B]), or S[b]. Rows with a slot outside the pool, or one that an earlier row has too, change
    nothing and get zeros.
    """
    if _elsewhere(q, stream):
        with _switched(q.get_device(), stream):
            return decay_step(q, k, v, log_decay, S, scale=scale, slots=slots, O=O)

    def check():
        device = _first(q, "q", 3)
        B, heads, dk = q.shape
        if not isinstance(v, torch.Tensor) or v.dim() != 3:
            raise ValueError("v: expected a 3-dimensional tensor")
        dv = _size(v.shape[2], "v: channels")
        if not isinstance(S, torch.Tensor) or S.dim() != 4 or S.shape[0] < 1:
            raise ValueError("S: expected a [n_slots, heads, dk, dv] tensor")
        cfg = DecayConfig(B, heads, 1, dk, dv, _DTYPES[q.dtype], dk ** -0.5 if scale is None else float(scale))
        cfg.q_stride[:2] = _tokens(q, "q", (B, heads, dk), q.dtype, device)[:2]
        cfg.k_stride[:2] = _tokens(k, "k", (B, heads, dk), q.dtype, device)[:2]
        cfg.v_stride[:2] = _tokens(v, "v", (B, heads, dv), q.dtype, device)[:2]
        cfg.o_stride[:2] = _tokens(torch.empty_like(v) if O is None else O, "O", v.shape, q.dtype, device)[:2]
        _require(log_decay, "log_decay", (heads,), torch.float32, device)
        _require(S, "S", (S.shape[0], heads, dk, dv), torch.float32, device)
        if slots is not None:
            _require(slots, "slots", (B,), torch.int32, device)
        return cfg, device.index, _size(S.shape[0], "S: slots")

    cfg, device, n_slots = _plan("step", _number(scale), (q, k, v, log_decay, S, slots, O), check)
    if O is None:
        O = torch.empty_like(v)
    _check(load().lfa_decay_step(cfg, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), S.data_ptr(),
                                 _ptr(slots), n_slots, O.data_ptr(), _cur(device)), "lfa_decay_step")
    return O


def decay_status(stream=None, device=None) -> int:
    """LFA_OK, or LFA_ERR_TIMEOUT once after a decay call on the device gave up a wait (lfa_decay_status)."""
    device = torch.device("cuda" if device is None else device)
    with _switched(torch.cuda.current_device() if device.index is None else device.index, stream):
        return int(load().lfa_decay_status(_cur(torch.cuda.current_device())))


# ---- rotary positions --------------------------------------------------------------------------------

def rotary_frequencies(rot: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                       context: int = 0, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """Frequencies base ** (-2 i / rot) of the rot / 2 channel pairs, stretched for contexts `factor` times as
    long as the trained one, as float64 on `device`, and the magnitude factor to pass as `mscale`.

    scaling "linear": all frequencies / factor. "ntk": the base grows so that the slowest pair is stretched by
    `factor` and the fastest is kept. "ramp": pairs that turn more than `fast` times within the trained
    `context` are kept, those below `slow` turns are divided by factor, in between linear in the pair's index;
    the magnitude is 0.1 ln(factor) + 1.
    """
    if rot < 2 or rot % 2 or not base > 1.0 or not factor >= 1.0:
        raise ValueError(f"rot {rot} (even, >= 2), base {base} (> 1), factor {factor} (>= 1)")
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot)
    mscale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "ntk":
        if rot > 2:
            f = (base * factor ** (rot / (rot - 2))) ** (-2.0 * i / rot)
    elif scaling == "ramp":
        if context < 1 or not fast > slow > 0:
            raise ValueError(f"ramp: context {context} (>= 1), fast {fast} > slow {slow} > 0")

        def index(turns):   # the pair that turns so often within the context
            return rot * math.log(context / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rot - 1)
        w = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - w) + f / factor * w
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling != "none":
        raise ValueError(f"scaling: {scaling!r}")
    return f.to(device), mscale


def rotary(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, *, x2: Optional[torch.Tensor] = None,
           layout: str = "half", mscale: float = 1.0, inverse: bool = False, out: Optional[torch.Tensor] = None,
           out2: Optional[torch.Tensor] = None, stream=None):
    """Rotary positions (lfa_rotary) on x [B, heads, N, d] and, in the same launch, x2 [B, heads2, N, d].
    Returns (y, y2).

    positions int32 [B, N]; freqs float64 [rot / 2]: the first rot channels turn, the others are copied.
    layout "half" pairs channels (i, i + rot/2), "interleaved" (2i, 2i+1). inverse: the transpose, which
    takes gradients of the outputs to gradients of the inputs. out may be x (and out2 x2).
    """
    if _elsewhere(x, stream):
        with _switched(x.get_device(), stream):
            return rotary(x, positions, freqs, x2=x2, layout=layout, mscale=mscale, inverse=inverse, out=out, out2=out2)

    def check():
        device = _first(x, "x", 4)
        B, heads, N, d = x.shape
        if layout not in ("half", "interleaved"):
            raise ValueError(f"layout: {layout!r}")
        if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
            raise ValueError("freqs: expected a 1-dimensional tensor")
        _require(positions, "positions", (B, N), torch.int32, device)
        _require(freqs, "freqs", (freqs.shape[0],), torch.float64, device)
        if x2 is not None and (not isinstance(x2, torch.Tensor) or x2.dim() != 4 or x2.shape[1] < 1):
            raise ValueError("x2: expected a [B, heads2, N, d] tensor")
        if x2 is None and out2 is not None:
            raise ValueError("out2 without x2")
        heads2 = 0 if x2 is None else _size(x2.shape[1], "x2: heads")
        cfg = RotaryConfig(B, N, d, _size(2 * freqs.shape[0], "freqs: channels"), heads, heads2, _DTYPES[x.dtype], layout == "interleaved",
                           bool(inverse), float(mscale))
        cfg.x_stride[:] = _tokens(x, "x", (B, heads, N, d), x.dtype, device)[:3]
        cfg.y_stride[:] = _tokens(torch.empty_like(x) if out is None else out, "out", x.shape, x.dtype, device)[:3]
        if x2 is not None:
            cfg.x2_stride[:] = _tokens(x2, "x2", (B, heads2, N, d), x.dtype, device)[:3]
            y2 = torch.empty_like(x2) if out2 is None else out2
            cfg.y2_stride[:] = _tokens(y2, "out2", x2.shape, x.dtype, device)[:3]
        return cfg, device.index

    cfg, device = _plan("rotary", (layout, float(mscale), bool(inverse)), (x, positions, freqs, x2, out, out2), check)
    if out is None:
        out = torch.empty_like(x)
    if out2 is None and x2 is not None:
        out2 = torch.empty_like(x2)
    _check(load().lfa_rotary(cfg, x.data_ptr(), _ptr(x2), positions.data_ptr(), freqs.data_ptr(), out.data_ptr(),
                             _ptr(out2), _cur(device)), "lfa_rotary")
    return out, out2


# ---- group norm ----------------------------------------------------------------------------------------

def _norm_config(x, groups, gamma, beta, eps, act):
    groups = _size(groups, "groups")
    device = _first(x, "x", 3)
    if act not in ACTIVATIONS:
        raise ValueError(f"act: {act!r}")
    if (gamma is None) != (beta is None):
        raise ValueError("gamma and beta: both or neither")
    B, N, C = x.shape
    _require(x, "x", (B, N, C), x.dtype, device)
    for name, t in (("gamma", gamma), ("beta", beta)):
        if t is not None:
            _require(t, name, (C,), torch.float32, device)
    return NormConfig(B, N, C, groups, _DTYPES[x.dtype], ACTIVATIONS[act], float(eps)), device


def group_norm(x: torch.Tensor, groups: int, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
               *, eps: float = 1e-5, act: str = "none", out: Optional[torch.Tensor] = None, stream=None):
    """act(group norm(x)) for x [B, N, C], channels last (lfa_group_norm): statistics over the N tokens and
    C / groups channels of a sample's group. Returns (y, mean, rstd), the statistics float32 [B, groups].

    gamma, beta float32 [C] or None; act "none", "silu" or "gelu" (exact); out may be x.
    """
    if _elsewhere(x, stream):
        with _switched(x.get_device(), stream):
            return group_norm(x, groups, gamma, beta, eps=eps, act=act, out=out)
    lib = load()

    def check():
        cfg, device = _norm_config(x, groups, gamma, beta, eps, act)
        if out is not None:
            _require(out, "out", x.shape, x.dtype, device)
        return cfg, device, lib.lfa_group_norm_workspace_size(cfg, 0)

    cfg, device, nbytes = _plan("norm", (int(groups), float(eps), act), (x, gamma, beta, out), check)
    if out is None:
        out = torch.empty_like(x)
    ws = _workspace(nbytes, device)
    mean = torch.empty((cfg.B, cfg.groups), dtype=torch.float32, device=device)
    rstd = torch.empty((cfg.B, cfg.groups), dtype=torch.float32, device=device)
    _check(lib.lfa_group_norm(cfg, x.data_ptr(), _ptr(gamma), _ptr(beta), out.data_ptr(), mean.data_ptr(),
                              rstd.data_ptr(), _ptr(ws), nbytes, _cur(device.index)), "lfa_group_norm")
    return out, mean, rstd


def group_norm_backward(x, dy, mean, rstd, groups: int, gamma=None, beta=None, *, eps: float = 1e-5, act: str = "none",
                        dx=None, stream=None):
    """Gradients of group_norm from its inputs and saved statistics (lfa_group_norm_backward). Returns
    (dx, dgamma, dbeta), the last two float32 [C], or None without gamma. dx may be dy."""
    if _elsewhere(x, stream):
        with _switched(x.get_device(), stream):
            return group_norm_backward(x, dy, mean, rstd, groups, gamma, beta, eps=eps, act=act, dx=dx)
    lib = load()

    def check():
        cfg, device = _norm_config(x, groups, gamma, beta, eps, act)
        _require(dy, "dy", x.shape, x.dtype, device)
        for name, t in (("mean", mean), ("rstd", rstd)):
            _require(t, name, (cfg.B, cfg.groups), torch.float32, device)
        if dx is not None:
            _require(dx, "dx", x.shape, x.dtype, device)
        return cfg, device, lib.lfa_group_norm_workspace_size(cfg, 1)

    cfg, device, nbytes = _plan("norm_backward", (int(groups), float(eps), act), (x, dy, mean, rstd, gamma, beta, dx), check)
    if dx is None:
        dx = torch.empty_like(x)
    ws = _workspace(nbytes, device)
    dgamma = dbeta = None
    if gamma is not None:
        dgamma = torch.empty(cfg.C, dtype=torch.float32, device=device)
        dbeta = torch.empty(cfg.C, dtype=torch.float32, device=device)
    _check(lib.lfa_group_norm_backward(cfg, x.data_ptr(), dy.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                       _ptr(gamma), _ptr(beta), dx.data_ptr(), _ptr(dgamma), _ptr(dbeta),
                                       _ptr(ws), nbytes, _cur(device.index)), "lfa_group_norm_backward")
    return dx, dgamma, dbeta


# ---- the layer -------------------------------------------------------------------------------------------

class DecayAttention:
    """The attention part of a decay-attention layer, between its projections: rotary positions on q and k,
    decay attention, and a group norm (one group per head) with an activation on every token's output.

    Tensors are as the projections leave them: q, k [B, N, heads, dk], v [B, N, heads, dv], y
    [B, N, heads * dv]. gamma, beta: float32 [heads * dv] or None. freqs: float64 [rot / 2] or None (no
    positions), with mscale as rotary_frequencies returns them.
    """

    def __init__(self, log_decay: torch.Tensor, gamma=None, beta=None, freqs=None, *, mscale: float = 1.0,
                 layout: str = "half", scale=None, eps: float = 1e-5, act: str = "silu"):
        load()
        self.log_decay, self.gamma, self.beta, self.freqs = log_decay, gamma, beta, freqs
        self.mscale, self.layout, self.scale, self.eps, self.act = mscale, layout, scale, eps, act
        self.heads = int(log_decay.shape[0])

    def _rotate(self, q, k, positions, inverse):
        if self.freqs is None:
            return q, k
        if positions is None:
            raise ValueError("positions: needed with freqs")
        return rotary(q, positions, self.freqs, x2=k, layout=self.layout, mscale=self.mscale, inverse=inverse)

    def forward(self, q, k, v, positions=None, *, S0=None, lengths=None, stream=None):
        """Returns (y, S_out, saved): saved is what backward needs. With lengths, rows of y behind a
        sequence's end are the norm of zeros."""
        with _in(_first(v, "v", 4).index, stream):
            qr, kr = self._rotate(q.transpose(1, 2), k.transpose(1, 2), positions, False)
            o = (torch.empty if lengths is None else torch.zeros)(v.shape, dtype=v.dtype, device=v.device)
            _, S = decay_forward(qr, kr, v.transpose(1, 2), self.log_decay, scale=self.scale, S0=S0, lengths=lengths,
                                 O=o.transpose(1, 2), return_state=True)
            B, N, heads, dv = v.shape
            y, mean, rstd = group_norm(o.view(B * N, 1, heads * dv), heads, self.gamma, self.beta, eps=self.eps,
                                       act=self.act)
        return y.view(B, N, heads * dv), S, (qr, kr, v, o, mean, rstd, positions, S0, lengths)

    def backward(self, saved, dy, dS_out=None, *, stream=None):
        """Gradients (dq, dk, dv, dS0, dgamma, dbeta) of <dy, y> + <dS_out, S_out>. With lengths, dy counts in
        dgamma and dbeta on the rows behind a sequence's end too: give zeros there."""
        qr, kr, v, o, mean, rstd, positions, S0, lengths = saved
        B, N, heads, dv = v.shape
        flat = (B * N, 1, heads * dv)
        with _in(v.get_device(), stream):
            do, dgamma, dbeta = group_norm_backward(o.view(flat), dy.reshape(flat).contiguous(), mean, rstd, heads, self.gamma,
                                                    self.beta, eps=self.eps, act=self.act)
            dq, dk, dvt, dS0 = decay_backward(qr, kr, v.transpose(1, 2), self.log_decay,
                                              do.view(v.shape).transpose(1, 2), scale=self.scale, S0=S0,
                                              lengths=lengths, dS_out=dS_out, return_state=True)
            dq, dk = self._rotate(dq, dk, positions, True)
        return dq.transpose(1, 2), dk.transpose(1, 2), dvt.transpose(1, 2), dS0, dgamma, dbeta

    def step(self, q, k, v, S, positions=None, *, slots=None, stream=None):
        """One token of every row: q, k [B, heads, dk], v [B, heads, dv], positions [B]; S is updated in place.
        Returns y [B, heads * dv]."""
        B, heads, dv = v.shape
        with _in(_first(v, "v", 3).index, stream):
            if self.freqs is not None:
                pos = None if positions is None else positions.unsqueeze(-1)
                qr, kr = self._rotate(q.unsqueeze(2), k.unsqueeze(2), pos, False)
                q, k = qr.squeeze(2), kr.squeeze(2)
            o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
            decay_step(q, k, v, self.log_decay, S, scale=self.scale, slots=slots, O=o)
            y, _, _ = group_norm(o.view(B, 1, heads * dv), heads, self.gamma, self.beta, eps=self.eps, act=self.act)
        return y.view(B, heads * dv)
