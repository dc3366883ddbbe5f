"""fp64 references of the operators around the recurrence, on the CPU, from
their definitions (token by token, sequence by sequence); differentiable, so
that torch's gradients of them are the gradients of the formulas.  Shares no
code with the package.
"""
import math

import torch

F64 = torch.float64


def seq_bounds(B, T, cu):
    """[(first row, last row + 1)] of each sequence on the flat token axis."""
    if cu is None:
        return [(b * T, b * T + T) for b in range(B)]
    return list(zip(cu[:-1], cu[1:]))


def conv(x, weight, bias, init, bounds, silu):
    """x [rows, D]; init [N, W-1, D] or None -> out [rows, D], final [N, W-1, D]."""
    W = weight.shape[1]
    out, final = [], []
    for n, (a, b) in enumerate(bounds):
        s0 = init[n] if init is not None else x.new_zeros(W - 1, x.shape[1])
        ext = torch.cat([s0, x[a:b]])
        for t in range(b - a):
            p = (ext[t:t + W] * weight.t()).sum(0)
            if bias is not None:
                p = p + bias
            out.append(p * torch.sigmoid(p) if silu else p)
        final.append(ext[len(ext) - (W - 1):])
    return torch.stack(out) if out else x.new_zeros(0, x.shape[1]), torch.stack(final)


def scan(x, delta, A, Bm, Cm, D, z, bias, softplus, init, bounds):
    """x, delta, z [rows, D]; Bm, Cm [rows, G, S] -> out [rows, D], final [N, D, S]."""
    ch, S = A.shape
    G = Bm.shape[1]
    dt = delta if bias is None else delta + bias
    if softplus:
        dt = torch.clamp(dt, min=0) + torch.log1p(torch.exp(-dt.abs()))
    out, final = [], []
    for n, (a, b) in enumerate(bounds):
        h = init[n] if init is not None else x.new_zeros(ch, S)
        for t in range(a, b):
            Bt = Bm[t].repeat_interleave(ch // G, 0)
            Ct = Cm[t].repeat_interleave(ch // G, 0)
            h = torch.exp(dt[t][:, None] * A) * h + (dt[t] * x[t])[:, None] * Bt
            y = (Ct * h).sum(1)
            if D is not None:
                y = y + D * x[t]
            if z is not None:
                y = y * z[t] * torch.sigmoid(z[t])
            out.append(y)
        final.append(h)
    return torch.stack(out) if out else x.new_zeros(0, ch), torch.stack(final)


def norm(x, weight, positions, inv_freq, l2, pairs, eps):
    """x [tokens, H, d] -> [tokens, H, d]."""
    d = x.shape[-1]
    ss = (x * x).sum(-1, keepdim=True)
    u = x / torch.sqrt((ss if l2 else ss / d) + eps)
    if weight is not None:
        u = u * weight
    if inv_freq is None:
        return u
    half = inv_freq.numel()
    first = torch.arange(half) * 2 if pairs else torch.arange(half)
    second = first + 1 if pairs else first + half
    ang = positions.to(F64)[:, None] * inv_freq.to(F64)
    # whole turns taken off exactly as fp64 allows, as the angle of a rotation
    cos, sin = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    a, b = u[..., first], u[..., second]
    y = u.clone()
    y[..., first] = a * cos - b * sin
    y[..., second] = a * sin + b * cos
    return y


def rel_l2(got, ref):
    got, ref = got.detach().to("cpu", F64), ref.detach().to("cpu", F64)
    den = float(ref.norm())
    num = float((got - ref).norm())
    return num / den if den else num


def bar(dtype):
    """Relative L2: what is held in fp32 has the library's fp32 bar (1e-5, some
    hundred fp32 roundings); one rounding to bf16 adds at most half a step,
    eps / 2 = 2^-8 of each value."""
    return 1e-5 + (torch.finfo(torch.bfloat16).eps / 2 if dtype == torch.bfloat16 else 0.0)


def log_uniform(gen, n, lo, hi):
    u = torch.rand(n, generator=gen, dtype=F64)
    return torch.exp(math.log(lo) + u * (math.log(hi) - math.log(lo)))
