"""Plain 64-bit forms of the token operators (decay attention, rotary positions, group norm), used by the
GPU tests only. Everything is computed on float64 tensors; nothing is shared with the library."""
import torch


def decays(log_decay, n):
    """exp(log_decay * n) per head with decay^0 = 1 (also for -inf); [heads, *n.shape]."""
    ld = log_decay.double().reshape(-1, *([1] * n.dim()))
    return torch.where(n == 0, torch.ones((), dtype=torch.float64, device=n.device), torch.exp(ld * n.clamp(min=1)))


def decay_forward(q, k, v, log_decay, scale, S0, lengths):
    """Dense causal form, sequence by sequence: (O, S); rows behind a sequence's end are zero."""
    B, H, N, dk = q.shape
    S0 = torch.zeros(B, H, dk, v.shape[3], dtype=torch.float64, device=q.device) if S0 is None else S0
    outs, states = [], []
    for b in range(B):
        L = N if lengths is None else max(0, min(N, int(lengths[b])))
        i = torch.arange(L, device=q.device)
        n = i[:, None] - i[None, :]
        D = decays(log_decay, n.clamp(min=0)) * (n >= 0)
        qb, kb, vb = q[b, :, :L], k[b, :, :L], v[b, :, :L]
        o = scale * (((qb @ kb.transpose(-1, -2)) * D) @ vb + decays(log_decay, i + 1)[..., None] * (qb @ S0[b]))
        outs.append(torch.nn.functional.pad(o, (0, 0, 0, N - L)))
        kw = kb * decays(log_decay, L - 1 - i)[..., None]
        states.append(kw.transpose(-1, -2) @ vb + decays(log_decay, torch.tensor(L, device=q.device))[:, None, None] * S0[b])
    return torch.stack(outs), torch.stack(states)


def decay_grads(q, k, v, log_decay, scale, S0, lengths, dO, dS):
    """Gradients of <dO, O> + <dS, S> from the dense form: (dq, dk, dv, dS0)."""
    S0 = torch.zeros(*q.shape[:2], q.shape[3], v.shape[3], dtype=torch.float64, device=q.device) if S0 is None else S0
    leaves = [t.clone().requires_grad_() for t in (q, k, v, S0)]
    o, S = decay_forward(*leaves[:3], log_decay, scale, leaves[3], lengths)
    loss = 0.0
    for b in range(q.shape[0]):
        L = q.shape[2] if lengths is None else max(0, min(q.shape[2], int(lengths[b])))
        loss = loss + (o[b, :, :L] * dO[b, :, :L]).sum()
    if dS is not None:
        loss = loss + (S * dS).sum()
    g = torch.autograd.grad(loss, leaves, allow_unused=True)
    return [torch.zeros_like(t) if x is None else x for x, t in zip(g, leaves)]


def rotate(x, positions, freqs, interleaved, mscale, inverse):
    y = x.clone()
    rot = 2 * freqs.numel()
    th = positions.double()[:, None, :, None] * freqs
    c, s = mscale * torch.cos(th), mscale * torch.sin(th) * (-1 if inverse else 1)
    ia = torch.arange(rot // 2, device=x.device)
    ia, ib = (2 * ia, 2 * ia + 1) if interleaved else (ia, ia + rot // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def activation(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / 2 ** 0.5))
    return z


def group_norm(x, groups, gamma, beta, eps, act):
    g = x.reshape(x.shape[0], x.shape[1], groups, -1)
    mean = g.mean((1, 3), keepdim=True)
    var = ((g - mean) ** 2).mean((1, 3), keepdim=True)
    rstd = (var + eps) ** -0.5
    z = ((g - mean) * rstd).reshape(x.shape)
    if gamma is not None:
        z = z * gamma + beta
    return activation(z, act), mean[:, 0, :, 0], rstd[:, 0, :, 0]
