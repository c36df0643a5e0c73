"""Plain 64-bit forms of rotary positions and differential attention, with the error bounds that the
tests use.  Everything is computed from the definitions on whole score matrices.

A rounding to bf16 is off by at most HALF = 2^-8 of the value (half a step).
"""
import math

import torch

HALF = 2.0 ** -8


def rope(x, positions, inv_freq, axis=None, interleaved=False, inverse=False):
    """x [..., heads, rows, d] with positions [axes, ..., rows]; returns float64."""
    x = x.double()
    half = inv_freq.numel()
    axis = torch.zeros(half, dtype=torch.long) if axis is None else axis.long()
    angle = positions.double()[axis] * inv_freq.double().view(-1, *([1] * (positions.dim() - 1)))
    angle = torch.where(positions[0] < 0, 0.0, angle).movedim(0, -1).unsqueeze(-3)
    if inverse:
        angle = -angle
    y = x.clone()
    a, b = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
            else (slice(0, half), slice(half, 2 * half)))
    y[..., a] = x[..., a] * angle.cos() - x[..., b] * angle.sin()
    y[..., b] = x[..., a] * angle.sin() + x[..., b] * angle.cos()
    return y


def rope_bound(x, want, half, interleaved=False):
    """One rounding of the result, and 2^-20 of the pair for the angle, the sine and the cosine (both
    in fp32: the angle 2^-24 of half a turn, the functions two steps) and three fp32 roundings."""
    pair = torch.zeros_like(want)
    a, b = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
            else (slice(0, half), slice(half, 2 * half)))
    size = x[..., a].double().abs() + x[..., b].double().abs()
    pair[..., a] = size
    pair[..., b] = size
    return HALF * want.abs() + 2.0 ** -20 * pair


def allowed(n, causal, window):
    i, j = torch.arange(n)[:, None], torch.arange(n)[None]
    ok = torch.ones(n, n, dtype=torch.bool)
    if causal:
        ok &= j <= i
    if window > 0:
        ok &= j >= i - window
        if not causal:
            ok &= j <= i + window
    return ok


def forward(q, k, v, lam, scale, ok):
    """One sequence: q [2H, n, d], k [2Hkv, m, d], v [Hkv, m, 2d], ok [n, m].  Returns a dict: o, o2
    [H, n, 2d], lse [2H, n], p [2H, n, m], the bounds of o, o2 and lse."""
    q, k, v, lam = (t.double() for t in (q, k, v, lam))
    H, G = q.shape[0] // 2, q.shape[0] // k.shape[0]
    kk = k.view(-1, 2, *k.shape[1:]).repeat_interleave(G, 0).flatten(0, 1)
    vv = v.repeat_interleave(G, 0)
    s = (q @ kk.transpose(1, 2) * scale).masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(s, 2)
    p = torch.exp(s - lse.masked_fill(lse == -math.inf, 0.0)[..., None])
    p1, p2 = p[0::2], p[1::2]
    o2 = p2 @ vv
    o = p1 @ vv - lam[:, None, None] * o2
    # scores are fp32 sums of d products: off by at most d 2^-24 of the sum of their magnitudes
    ds = (q.abs() @ kk.abs().transpose(1, 2) * scale).masked_fill(~ok, 0.0).amax((1, 2)) * q.shape[-1] * 2.0 ** -24
    ds = ds.view(H, 2).amax(1)[:, None, None]
    # a weight is rounded once to bf16, and off by its score's error (in the sum, too) and by the
    # fp32 exponential, sums and products (2^-12 covers sums of up to 2^12 terms)
    weight = HALF + 2.0 ** -12 + 2.5 * ds
    a1, a2 = p1 @ vv.abs(), p2 @ vv.abs()
    bound2 = weight * a2 + HALF * o2.abs()
    bound = weight * (a1 + lam.abs()[:, None, None] * a2) + HALF * o.abs()
    bound_lse = (ds[:, 0].repeat_interleave(2, 0) * 2 + 2.0 ** -17) * torch.ones_like(lse) + lse.abs().nan_to_num(0, 0, 0) * 2.0 ** -22
    return dict(o=o, o2=o2, lse=lse, p=p, o_bound=bound, o2_bound=bound2, lse_bound=bound_lse)


def backward(q, k, v, lam, o, o2, dout, lse, scale, ok, rounded=0.0):
    """One sequence's gradients by the formulas on what the forward pass saved (any precision), and their
    bounds.  `rounded`: how far o and o2 are from the definition's, relative (HALF where the kernels'
    own are compared with gradients of the definition)."""
    q, k, v, lam, o, o2, dout, lse = (t.double() for t in (q, k, v, lam, o, o2, dout, lse))
    H, Hkv, n, d = q.shape[0] // 2, k.shape[0] // 2, q.shape[1], q.shape[2]
    G = H // Hkv
    kk = k.view(Hkv, 2, -1, d).repeat_interleave(G, 0)              # [H, 2, m, d]
    qq, vv = q.view(H, 2, n, d), v.repeat_interleave(G, 0)
    w = lam[:, None, None]
    s = (qq @ kk.transpose(2, 3) * scale).masked_fill(~ok, -math.inf)
    p = torch.exp(s - lse.view(H, 2, n, 1)) * torch.stack((torch.ones_like(w), -w), 1)
    dot2 = (dout * o2).sum(2, keepdim=True)
    dot = torch.stack(((dout * o).sum(2, keepdim=True) + w * dot2, dot2), 1)    # [H, 2, n, 1]
    dp = (dout @ vv.transpose(1, 2))[:, None]
    ds = p * (dp - dot)
    heads = lambda t: t.view(Hkv, G, *t.shape[1:]).sum(1)
    dq = (ds @ kk * scale).flatten(0, 1)
    dk = heads(ds.transpose(2, 3) @ qq * scale).flatten(0, 1)
    dv = heads((p.sum(1)).transpose(1, 2) @ dout)
    dlam = -dot2.sum((1, 2))
    # A weight is off by its score's error (fp32 sums of d products) and 2^-20 for the fp32 LSE, the
    # exponential and its argument; dP - D by fp32 sums of 2d products and what o and o2 are off;
    # what enters the products is rounded once to bf16; their sums are fp32 (2^-12: 2^12 terms).
    err = ((qq.abs() @ kk.abs().transpose(2, 3) * scale).masked_fill(~ok, 0.0).amax((1, 2, 3)) * d * 2.0 ** -23
           + 2.0 ** -20 + lse.view(H, -1).abs().amax(1) * 2.0 ** -23)[:, None, None, None]
    size2 = (dout.abs() * o2.abs()).sum(2, keepdim=True)
    size1 = (dout.abs() * o.abs()).sum(2, keepdim=True) + w.abs() * size2
    size = torch.stack((size1, size2), 1)
    off = 2 * d * 2.0 ** -24 * ((dout.abs() @ vv.abs().transpose(1, 2))[:, None] + size) + rounded * size
    rel = HALF + 2.0 ** -12 + err
    eds = rel * ds.abs() + p.abs() * (1 + HALF) * off
    ep = rel * p.abs()
    bq = (eds @ kk.abs() * scale).flatten(0, 1) + HALF * dq.abs()
    bk = heads(eds.transpose(2, 3) @ qq.abs() * scale).flatten(0, 1) + HALF * dk.abs()
    bv = heads(ep.sum(1).transpose(1, 2) @ dout.abs()) + HALF * dv.abs()
    blam = (rounded + 2.0 ** -16) * size2.sum((1, 2))
    return (dq, dk, dv, dlam), (bq, bk, bv, blam)


def check(got, want, bound, name):
    """|got - want| <= bound everywhere; infinities equal."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.isfinite(got).logical_or(got == want).all(), f"{name}: not finite"
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin], want[~fin]), f"{name}: infinities differ"
    over = ((got - want).abs() - bound)[fin]
    if over.numel():
        assert over.max() <= 0, f"{name}: {(over > 0).sum()} of {over.numel()} beyond the bound, worst by {over.max():.3e}"
