"""Differential attention's backward pass against the formulas in 64 bits, and against 64-bit
differentiation of the definition."""
import math

import pytest
import torch

from tests import diff_reference as ref
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu
NAMES = ("dq", "dk", "dv", "dlam")


def fa():
    require_gpu()
    import exact_attention_55_gb300 as module
    return module


def make(shape, seed, size=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * size).bfloat16()


def weights(H, seed=5):
    return torch.rand(H, generator=torch.Generator().manual_seed(seed)) * 0.8 + 0.1


def saved(q, k, v, lam, scale, ok):
    """What a forward pass in 64 bits saves, rounded to its outputs' types."""
    w = ref.forward(q, k, v, lam, scale, ok)
    return w["o"].bfloat16(), w["o2"].bfloat16(), w["lse"].float()


def compare(m, q, k, v, lam, dout, causal, window, scale=None):
    B, N, d = q.shape[0], q.shape[2], q.shape[3]
    scale = scale or 1 / math.sqrt(d)
    ok = ref.allowed(N, causal, window)
    o, o2, lse = (torch.stack(t) for t in zip(*(saved(q[b], k[b], v[b], lam, scale, ok) for b in range(B))))
    got = m.attn_diff_bwd_bf16(*(t.cuda() for t in (q, k, v, lam, o, o2, dout, lse)), scale=scale, causal=causal,
                               window=window)
    assert m.attn_get_device_status() == m.ATTN_OK
    wants = [ref.backward(q[b], k[b], v[b], lam, o[b], o2[b], dout[b], lse[b], scale, ok) for b in range(B)]
    for i, name in enumerate(NAMES[:3]):
        ref.check(got[i], torch.stack([w[0][i] for w in wants]), torch.stack([w[1][i] for w in wants]), name)
    ref.check(got[3], sum(w[0][3] for w in wants), sum(w[1][3] for w in wants), "dlam")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 63, 64, 65, 128, 130, 256, 333])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 70), (False, 40)])
def test_batched(d, N, causal, window):
    m = fa()
    q, k, v, g = make((2, 4, N, d), 1), make((2, 4, N, d), 2), make((2, 2, N, 2 * d), 3), make((2, 2, N, 2 * d), 4)
    compare(m, q, k, v, weights(2), g, causal, window)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (4, 2), (6, 3)])
def test_shared_heads(d, H, Hkv):
    m = fa()
    q, k, v = make((2, 2 * H, 200, d), 5), make((2, 2 * Hkv, 200, d), 6), make((2, Hkv, 200, 2 * d), 7)
    compare(m, q, k, v, weights(H), make((2, H, 200, 2 * d), 8), True, 0, 0.2)


@pytest.mark.parametrize("d", [64, 128])
def test_many_tiles(d):
    """More steps than the ring has slots, more units than the card has SMs, weights above 1, 0 and negative."""
    m = fa()
    N = 900
    lam = torch.tensor([1.7, 0.0, -0.6])
    q, k, v = make((7, 6, N, d), 9, 1.5), make((7, 6, N, d), 10, 1.5), make((7, 3, N, 2 * d), 11)
    compare(m, q, k, v, lam, make((7, 3, N, 2 * d), 12), True, 0)


@pytest.mark.parametrize("d", [64, 128])
def test_of_the_definition(d):
    """Forward and backward of the kernels against 64-bit automatic differentiation of the definition."""
    m = fa()
    N, H, Hkv = 260, 4, 2
    q, k, v, g = make((1, 2 * H, N, d), 13), make((1, 2 * Hkv, N, d), 14), make((1, Hkv, N, 2 * d), 15), make((1, H, N, 2 * d), 16)
    lam, scale, ok = weights(H), 1 / math.sqrt(d), ref.allowed(N, True, 0)
    dev = [t.cuda() for t in (q, k, v, lam)]
    o, lse, o2 = m.attn_diff_fwd_bf16(*dev, causal=True, save_o2=True)
    got = m.attn_diff_bwd_bf16(*dev, o, o2, g.cuda(), lse, causal=True)
    leaves = [t.double().requires_grad_() for t in (q, k, v, lam)]
    w = ref.forward(*(t[0] for t in leaves[:3]), leaves[3], scale, ok)
    want = torch.autograd.grad((w["o"] * g[0].double()).sum(), leaves)
    # the kernels' o and o2 are within their bounds of the definition's: as a share of sum P |V|
    _, bounds = ref.backward(q[0], k[0], v[0], lam, w["o"].detach(), w["o2"].detach(), g[0], w["lse"].detach(), scale, ok)
    p = w["p"].detach().view(H, 2, N, N)
    vv = v[0].double().abs().repeat_interleave(H // Hkv, 0)
    share = (p @ vv[:, None])                                        # sum P_m |V|
    go = g[0].double().abs()
    lamw = lam.double()[:, None, None]
    off2 = (go * (w["o2_bound"].detach())).sum(2, keepdim=True)
    off1 = (go * w["o_bound"].detach()).sum(2, keepdim=True) + lamw * off2
    extra = p * torch.stack((off1, off2), 1) * torch.stack((torch.ones_like(lamw), lamw), 1)
    kk = k[0].double().abs().view(Hkv, 2, N, d).repeat_interleave(H // Hkv, 0)
    eq = (extra @ kk * scale).flatten(0, 1)
    ek = (extra.transpose(2, 3) @ q[0].double().abs().view(H, 2, N, d) * scale).view(Hkv, H // Hkv, 2, N, d).sum(1).flatten(0, 1)
    lse_off = 2 * w["lse_bound"].detach().max()                      # the kernel's LSE moves every weight
    more = (eq, ek, 0.0, off2.sum((1, 2)))
    for name, a, b, c, e in zip(NAMES, got, want, bounds, more):
        a = a if name == "dlam" else a[0]
        b = b.detach() if name == "dlam" else b[0].detach()
        ref.check(a, b, (c + e) * (1 + 2.0 ** -7) + lse_off * c / ref.HALF, name)
    assert share.isfinite().all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [128, 129], [5, 0, 300, 64, 1], [0, 0, 7], [200] * 3])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50)])
def test_packed(d, lens, causal, window):
    """Every sequence by itself; tokens outside all of them hold NaN, and their gradients stay."""
    m = fa()
    H, Hkv, pad = 4, 2, 40
    n = sum(lens)
    T = n + pad
    q, k, v, g = make((T, 2 * H, d), 17), make((T, 2 * Hkv, d), 18), make((T, Hkv, 2 * d), 19), make((T, H, 2 * d), 20)
    for t in (q, k, v, g):
        t[n:] = float("nan")
    o, o2, lse = torch.full_like(g, float("nan")), torch.full_like(g, float("nan")), torch.full((2 * H, T), float("nan"))
    lam, scale = weights(H), 1 / math.sqrt(d)
    cu = [0]
    wants = []
    for length in lens:
        s = slice(cu[-1], cu[-1] + length)
        cu.append(s.stop)
        if length == 0:
            continue
        ok = ref.allowed(length, causal, window)
        rows = [t[s].transpose(0, 1) for t in (q, k, v, g)]
        a, b, c = saved(*rows[:3], lam, scale, ok)
        o[s], o2[s], lse[:, s] = a.transpose(0, 1), b.transpose(0, 1), c
        wants.append((s, ref.backward(*rows[:3], lam, a, b, rows[3], c, scale, ok)))
    outs = [torch.full(t.shape, 7.0, dtype=torch.bfloat16, device="cuda") for t in (q, k, v)]
    dlam = m.attn_diff_bwd_bf16_varlen(*(t.cuda() for t in (q, k, v, lam, o, o2, g, lse)),
                                       torch.tensor(cu, dtype=torch.int32).cuda(), max(lens), causal=causal,
                                       window=window, dq=outs[0], dk=outs[1], dv=outs[2])[3]
    assert m.attn_get_device_status() == m.ATTN_OK
    for s, (want, bound) in wants:
        for i in range(3):
            ref.check(outs[i][s].transpose(0, 1), want[i], bound[i], NAMES[i])
    assert all((t[n:] == 7).all() for t in outs)
    ref.check(dlam, sum(w[0][3] for _, w in wants), sum(w[1][3] for _, w in wants), "dlam")


def test_more_sequences_than_the_table():
    m = fa()
    lens = torch.randint(0, 150, (260,), generator=torch.Generator().manual_seed(21)).tolist()
    T, d = sum(lens), 64
    q, k, v, g = make((T, 2, d), 22), make((T, 2, d), 23), make((T, 1, 2 * d), 24), make((T, 1, 2 * d), 25)
    cu = torch.tensor([0] + [sum(lens[:i + 1]) for i in range(260)], dtype=torch.int32)
    lam = weights(1)
    dev = [t.cuda() for t in (q, k, v, lam)]
    o, lse, o2 = m.attn_diff_fwd_bf16_varlen(*dev, cu.cuda(), 150, causal=True, save_o2=True)
    got = m.attn_diff_bwd_bf16_varlen(*dev, o, o2, g.cuda(), lse, cu.cuda(), 150, causal=True)
    total, most = 0.0, 0.0
    for i, (a, length) in enumerate(zip(cu.tolist(), lens)):
        if length == 0:
            continue
        s = slice(a, a + length)
        rows = [t[s].transpose(0, 1) for t in (q, k, v, o.cpu(), o2.cpu(), g)]
        want, bound = ref.backward(*rows[:3], lam, *rows[3:], lse[:, s].cpu(), 0.125, ref.allowed(length, True, 0))
        total, most = total + want[3], most + bound[3]
        if i % 13 == 0:
            for j in range(3):
                ref.check(got[j][s].transpose(0, 1), want[j], bound[j], NAMES[j])
    ref.check(got[3], total, most, "dlam")


def test_no_tokens():
    m = fa()
    q, k, v, g = (torch.empty(0, h, w, dtype=torch.bfloat16, device="cuda") for h, w in ((4, 64), (2, 64), (1, 128), (2, 128)))
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    dlam = torch.full((2,), 3.0, device="cuda")
    m.attn_diff_bwd_bf16_varlen(q, k, v, weights(2).cuda(), g, g, g, torch.empty(4, 0, device="cuda"), cu, 0, dlam=dlam)
    assert (dlam == 0).all()


def test_same_bits_every_time_and_graph():
    """Sums have a fixed order: two runs, another stream and a replayed graph give the same bits."""
    m = fa()
    d, H = 64, 6
    q, k, v, g = make((3, 2 * H, 700, d), 26).cuda(), make((3, 4, 700, d), 27).cuda(), make((3, 2, 700, 2 * d), 28).cuda(), make((3, H, 700, 2 * d), 29).cuda()
    lam = weights(H).cuda()
    o, lse, o2 = m.attn_diff_fwd_bf16(q, k, v, lam, causal=True, save_o2=True)
    args = (q, k, v, lam, o, o2, g, lse)
    want = m.attn_diff_bwd_bf16(*args, causal=True)
    again = m.attn_diff_bwd_bf16(*args, causal=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = m.attn_diff_bwd_bf16(*args, causal=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, again, other))
    outs = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.attn_diff_bwd_bf16(*args, causal=True, dq=outs[0], dk=outs[1], dv=outs[2], dlam=outs[3])
    for _ in range(2):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals():
    m = fa()
    q, k, v, g = (make(s, i).cuda() for i, s in enumerate([(1, 4, 8, 64), (1, 2, 8, 64), (1, 1, 8, 128), (1, 2, 8, 128)]))
    lam, lse = weights(2).cuda(), torch.zeros(1, 4, 8, device="cuda")
    good = dict(q=q, k=k, v=v, lam=lam, o=g, o2=g, dout=g, lse=lse)
    m.attn_diff_bwd_bf16(**good)
    for bad in (dict(o2=None), dict(dout=g.float()), dict(lse=lse[:, :2].contiguous()), dict(dq=torch.empty_like(k)),
                dict(dlam=torch.empty(1, device="cuda"))):
        with pytest.raises(TypeError):
            m.attn_diff_bwd_bf16(**{**good, **bad})
    with pytest.raises(m.AttnError):
        m.attn_diff_bwd_bf16(**good, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(m.AttnError):
        m.attn_diff_bwd_bf16(**good, scale=-1.0)
