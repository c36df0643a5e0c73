"""Differential attention's forward pass against a plain 64-bit form."""
import math

import pytest
import torch

from tests import diff_reference as ref
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu


def fa():
    require_gpu()
    import exact_attention_55_gb300 as module
    return module


def make(shape, seed, size=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * size).bfloat16()


def weights(H, seed=5):
    return torch.rand(H, generator=torch.Generator().manual_seed(seed)) * 0.8 + 0.1


def compare(m, q, k, v, lam, causal, window, scale, save=True):
    B, N, d = q.shape[0], q.shape[2], q.shape[3]
    o, lse, o2 = m.attn_diff_fwd_bf16(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), scale=scale, causal=causal,
                                      window=window, save_o2=save)
    assert m.attn_get_device_status() == m.ATTN_OK
    assert (o2 is not None) == save
    ok = ref.allowed(N, causal, window)
    for b in range(B):
        want = ref.forward(q[b], k[b], v[b], lam, scale or 1 / math.sqrt(d), ok)
        ref.check(o[b], want["o"], want["o_bound"], f"o {b}")
        ref.check(lse[b], want["lse"], want["lse_bound"], f"lse {b}")
        if save:
            ref.check(o2[b], want["o2"], want["o2_bound"], f"o2 {b}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 2, 63, 127, 128, 129, 256, 300])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 70), (False, 40)])
def test_batched(d, N, causal, window):
    m = fa()
    q, k, v = make((2, 4, N, d), 1), make((2, 4, N, d), 2), make((2, 2, N, 2 * d), 3)
    compare(m, q, k, v, weights(2), causal, window, None, save=N % 2 == 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (4, 2), (6, 3)])
def test_shared_heads(d, H, Hkv):
    m = fa()
    q, k, v = make((2, 2 * H, 200, d), 4), make((2, 2 * Hkv, 200, d), 5), make((2, Hkv, 200, 2 * d), 6)
    compare(m, q, k, v, weights(H), True, 0, 0.2)


@pytest.mark.parametrize("d", [64, 128])
def test_many_tiles_and_large_scores(d):
    """Longer than a CTA's ring, running maxima that move, weights above 1 and negative."""
    m = fa()
    N = 1100
    q, k, v = make((1, 2, N, d), 7, 3.0), make((1, 2, N, d), 8, 3.0), make((1, 1, N, 2 * d), 9)
    for lam in (1.7, -0.5, 0.0):
        compare(m, q, k, v, torch.tensor([lam]), True, 0, None)
        compare(m, q, k, v, torch.tensor([lam]), False, 333, None)


def test_equal_maps_cancel():
    """lam = 1 and equal maps: both accumulators are the same sums, so O is exactly 0."""
    m = fa()
    q, k, v = make((1, 1, 300, 64), 10), make((1, 1, 300, 64), 11), make((1, 1, 300, 128), 12)
    o, lse, _ = m.attn_diff_fwd_bf16(q.repeat(1, 2, 1, 1).cuda(), k.repeat(1, 2, 1, 1).cuda(), v.cuda(),
                                     torch.ones(1).cuda(), causal=True)
    assert torch.equal(lse[:, 0], lse[:, 1])
    assert o.abs().max().item() <= 2.0 ** -20 * v.abs().max().item()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [128, 129], [5, 0, 300, 64, 1], [0, 0, 7], [200] * 3])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50)])
def test_packed(d, lens, causal, window):
    """Every sequence by itself; tokens outside all of them hold NaN and stay as they are."""
    m = fa()
    H, Hkv, pad = 4, 2, 40
    n = sum(lens)
    T = n + pad
    q, k, v = make((T, 2 * H, d), 13), make((T, 2 * Hkv, d), 14), make((T, Hkv, 2 * d), 15)
    for t in (q, k, v):
        t[n:] = float("nan")
    cu = torch.tensor([0] + [sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)
    lam = weights(H)
    o = torch.full((T, H, 2 * d), 7.0, dtype=torch.bfloat16, device="cuda")
    o2, lse = torch.full_like(o, 7.0), torch.full((2 * H, T), 7.0, device="cuda")
    m.attn_diff_fwd_bf16_varlen(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), cu.cuda(), max(lens), causal=causal,
                                window=window, o=o, o2=o2, lse=lse)
    assert m.attn_get_device_status() == m.ATTN_OK
    for a, length in zip(cu.tolist(), lens):
        if length == 0:
            continue
        s = slice(a, a + length)
        want = ref.forward(q[s].transpose(0, 1), k[s].transpose(0, 1), v[s].transpose(0, 1), lam, 1 / math.sqrt(d),
                           ref.allowed(length, causal, window))
        ref.check(o[s].transpose(0, 1), want["o"], want["o_bound"], "o")
        ref.check(o2[s].transpose(0, 1), want["o2"], want["o2_bound"], "o2")
        ref.check(lse[:, s], want["lse"], want["lse_bound"], "lse")
    assert (o[n:] == 7).all() and (o2[n:] == 7).all() and (lse[:, n:] == 7).all()


def test_sequences_beside_nan():
    """What the sequences around one hold does not reach it."""
    m = fa()
    lens, d = [100, 60, 90], 64
    T = sum(lens)
    q, k, v = make((T, 2, d), 16), make((T, 2, d), 17), make((T, 1, 2 * d), 18)
    cu = torch.tensor([0, 100, 160, 250], dtype=torch.int32).cuda()
    lam = weights(1).cuda()
    clean = m.attn_diff_fwd_bf16_varlen(q.cuda(), k.cuda(), v.cuda(), lam, cu, 100)[0]
    for t in (q, k, v):
        t[160:] = float("nan")
    dirty = m.attn_diff_fwd_bf16_varlen(q.cuda(), k.cuda(), v.cuda(), lam, cu, 100)[0]
    assert torch.equal(clean[:160], dirty[:160]) and dirty[160:].isnan().all()


def test_more_sequences_than_the_table():
    m = fa()
    gen = torch.Generator().manual_seed(19)
    lens = torch.randint(0, 150, (260,), generator=gen).tolist()
    T, d = sum(lens), 64
    q, k, v = make((T, 2, d), 20), make((T, 2, d), 21), make((T, 1, 2 * d), 22)
    cu = torch.tensor([0] + [sum(lens[:i + 1]) for i in range(260)], dtype=torch.int32)
    lam = weights(1)
    o = m.attn_diff_fwd_bf16_varlen(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), cu.cuda(), 150, causal=True)[0]
    for a, length in list(zip(cu.tolist(), lens))[::17]:
        if length:
            s = slice(a, a + length)
            want = ref.forward(q[s].transpose(0, 1), k[s].transpose(0, 1), v[s].transpose(0, 1), lam, 0.125,
                               ref.allowed(length, True, 0))
            ref.check(o[s].transpose(0, 1), want["o"], want["o_bound"], "o")


@pytest.mark.parametrize("d", [64, 128])
def test_many_units_of_one_step(d):
    """Several units a CTA with a single step each, where the two maps' warps are furthest apart: the same bits
    however the units fall on the CTAs."""
    m = fa()
    B, H, N = 96, 8, 100
    q, k, v = make((B, 2 * H, N, d), 20).cuda(), make((B, 2 * H, N, d), 21).cuda(), make((B, H, N, 2 * d), 22).cuda()
    lam = weights(H).cuda()
    o, lse, _ = m.attn_diff_fwd_bf16(q, k, v, lam, causal=True)
    for b in range(0, B, 19):
        one = slice(b, b + 1)
        o1, lse1, _ = m.attn_diff_fwd_bf16(q[one], k[one], v[one], lam, causal=True)
        assert torch.equal(o[one], o1) and torch.equal(lse[one], lse1)
    compare(m, q[:1].cpu(), k[:1].cpu(), v[:1].cpu(), lam.cpu(), True, 0, None)


def test_window_wider_than_the_sequence():
    m = fa()
    q, k, v = (make(s, i).cuda() for i, s in enumerate([(1, 2, 200, 64), (1, 2, 200, 64), (1, 1, 200, 128)]))
    lam = weights(1).cuda()
    for causal in (False, True):
        want = m.attn_diff_fwd_bf16(q, k, v, lam, causal=causal)
        for window in (199, 200, 2 ** 31 - 1):
            got = m.attn_diff_fwd_bf16(q, k, v, lam, causal=causal, window=window)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_streams_and_graph():
    m = fa()
    q, k, v = make((2, 8, 600, 128), 23).cuda(), make((2, 4, 600, 128), 24).cuda(), make((2, 2, 600, 256), 25).cuda()
    lam = weights(4).cuda()
    want = m.attn_diff_fwd_bf16(q, k, v, lam, causal=True, save_o2=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = m.attn_diff_fwd_bf16(q, k, v, lam, causal=True, save_o2=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.attn_diff_fwd_bf16(q, k, v, lam, causal=True, o=outs[0], lse=outs[1], o2=outs[2])
    lam *= 0.5
    graph.replay()
    torch.cuda.synchronize()
    want = m.attn_diff_fwd_bf16(q, k, v, lam, causal=True, save_o2=True)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals():
    m = fa()
    q, k, v = (make(s, i).cuda() for i, s in enumerate([(1, 4, 8, 64), (1, 2, 8, 64), (1, 1, 8, 128)]))
    lam = weights(2).cuda()
    m.attn_diff_fwd_bf16(q, k, v, lam)
    with pytest.raises(ValueError):
        m.attn_diff_fwd_bf16(q[:, :3].contiguous(), k, v, lam)
    with pytest.raises(ValueError):
        m.attn_diff_fwd_bf16(q, k.repeat(1, 3, 1, 1), v.repeat(1, 3, 1, 1), lam)
    for bad in (dict(lam=lam[:1].clone()), dict(lam=lam.bfloat16()), dict(v=v[..., :64].contiguous()), dict(q=q.half()),
                dict(k=k.transpose(2, 3).contiguous().transpose(2, 3)), dict(o=torch.empty_like(q))):
        with pytest.raises(TypeError):
            m.attn_diff_fwd_bf16(**{**dict(q=q, k=k, v=v, lam=lam), **bad})
    for bad in (dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(m.AttnError):
            m.attn_diff_fwd_bf16(q, k, v, lam, **bad)
    with pytest.raises(m.AttnError):
        m.attn_diff_fwd_bf16(*(torch.zeros(1, h, 8, w, dtype=torch.bfloat16, device="cuda") for h, w in ((4, 96), (2, 96), (1, 192))), lam)
