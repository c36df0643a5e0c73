"""Rotary positions against a plain 64-bit form."""
import pytest
import torch

from tests import diff_reference as ref
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu


def fa():
    require_gpu()
    import exact_attention_55_gb300 as module
    return module


def make(shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


def frequencies(half, base=10000.0):
    return torch.pow(torch.tensor(base), -torch.arange(half, dtype=torch.float32) / half)


def compare(got, x, pos, freq, name, axis=None, interleaved=False, inverse=False, packed=True):
    """x and got packed [T, H, d] or [B, H, N, d]; pos [axes, ...]."""
    rows = x.transpose(0, 1) if packed else x
    want = ref.rope(rows, pos, freq, axis, interleaved, inverse)
    bound = ref.rope_bound(rows, want, freq.numel(), interleaved)
    ref.check(got.transpose(0, 1) if packed else got, want, bound, name)


@pytest.mark.parametrize("T,hq,hk,d,rot", [(1, 1, 1, 64, 64), (5, 4, 1, 128, 128), (33, 6, 2, 64, 32), (257, 2, 2, 256, 256),
                                           (19, 3, 1, 96, 80), (2, 40, 8, 16, 16), (1000, 32, 8, 128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [1, 3])
def test_packed(T, hq, hk, d, rot, interleaved, axes):
    m = fa()
    q, k = make((T, hq, d), 1), make((T, hk, d), 2)
    freq = frequencies(rot // 2)
    gen = torch.Generator().manual_seed(3)
    pos = torch.randint(0, 200000, (axes, T), generator=gen, dtype=torch.int32)
    axis = torch.randint(0, axes, (rot // 2,), generator=gen, dtype=torch.int32) if axes > 1 else None
    args = (pos.cuda() if axes > 1 else pos[0].cuda(), freq.cuda())
    more = dict(axis=None if axis is None else axis.cuda(), interleaved=interleaved)
    for inverse in (False, True):
        qo, ko = m.attn_rope_bf16(q.cuda(), k.cuda(), *args, inverse=inverse, **more)
        compare(qo, q, pos, freq, "q", axis, interleaved, inverse)
        compare(ko, k, pos, freq, "k", axis, interleaved, inverse)


@pytest.mark.parametrize("B,H,N,d", [(1, 1, 1, 64), (3, 4, 130, 128), (2, 8, 77, 64)])
def test_batched(B, H, N, d):
    m = fa()
    q, k = make((B, H, N, d), 4), make((B, 2 * H, N, d), 5)
    pos = torch.randint(0, 5000, (2, B, N), generator=torch.Generator().manual_seed(6), dtype=torch.int32)
    freq, axis = frequencies(d // 4), (torch.arange(d // 4) % 2).to(torch.int32)
    qo, ko = m.attn_rope_bf16(q.cuda(), k.cuda(), pos.cuda(), freq.cuda(), axis=axis.cuda())
    compare(qo, q, pos, freq, "q", axis, packed=False)
    compare(ko, k, pos, freq, "k", axis, packed=False)
    qo, none = m.attn_rope_bf16(q.cuda(), None, pos[0].contiguous().cuda(), freq.cuda())
    assert none is None
    compare(qo, q, pos[:1], freq, "q alone", packed=False)


def test_columns_of_a_projection_in_place():
    m = fa()
    T, hq, hk, d = 70, 8, 2, 128
    both = make((T, hq + 2 * hk, d), 7).cuda()
    kept = both.clone()
    pos, freq = torch.arange(T, dtype=torch.int32) + 9000, frequencies(d // 2)
    q, k = both[:, :hq], both[:, hq:hq + hk]
    qo, ko = m.attn_rope_bf16(q, k, pos.cuda(), freq.cuda(), q_out=q, k_out=k)
    assert qo.data_ptr() == q.data_ptr() and ko.data_ptr() == k.data_ptr()
    compare(both[:, :hq], kept[:, :hq].cpu(), pos[None], freq, "q")
    compare(both[:, hq:hq + hk], kept[:, hq:hq + hk].cpu(), pos[None], freq, "k")
    assert torch.equal(both[:, hq + hk:], kept[:, hq + hk:])


def test_views_of_batches():
    """[B, N, H, d] memory seen as [B, H, N, d]; keys broadcast over the batch."""
    m = fa()
    B, H, N, d = 2, 3, 50, 64
    q = make((B, N, H, d), 8).cuda().transpose(1, 2)
    k = make((1, 2, N, d), 9).cuda().expand(B, -1, -1, -1)
    pos = torch.arange(N, dtype=torch.int32).repeat(B, 1)
    pos[1] += 100
    freq = frequencies(d // 2)
    qo, ko = m.attn_rope_bf16(q, k, pos.cuda(), freq.cuda())
    compare(qo, q.cpu(), pos[None], freq, "q", packed=False)
    compare(ko, k.cpu(), pos[None], freq, "k", packed=False)
    with pytest.raises(ValueError):
        m.attn_rope_bf16(q, k, pos.cuda(), freq.cuda(), k_out=k)


def test_padding_keeps_its_rows():
    """A negative position on axis 0 copies the row bit for bit, NaN and infinities too."""
    m = fa()
    x = make((6, 2, 64), 10)
    x[1, 0, :8] = torch.tensor([float("nan"), float("inf"), -0.0, 0.0, 1.0, -float("inf"), 3.0, float("nan")])
    pos = torch.tensor([[5, -1, 7, -1, 0, -2], [3, 4, -4, 5, 0, 1]], dtype=torch.int32)
    freq, axis = frequencies(32), (torch.arange(32) % 2).to(torch.int32)
    for interleaved in (False, True):
        out, _ = m.attn_rope_bf16(x.cuda(), None, pos.cuda(), freq.cuda(), axis=axis.cuda(), interleaved=interleaved)
        pad = pos[0] < 0
        assert torch.equal(out.cpu()[pad].view(torch.int16), x[pad].view(torch.int16))
        compare(out[~pad.cuda()], x[~pad], pos[:, ~pad], freq, "rest", axis, interleaved)


@pytest.mark.parametrize("far", [(1 << 20) - 3, (1 << 30) + 12345, (1 << 31) - 1])
def test_far_positions(far):
    """The angle keeps its digits: 2^-32 of a turn and |position| 2^-63, here 2^-30 turns at most."""
    m = fa()
    x = make((4, 1, 128), 11)
    pos = torch.tensor([[far, far - 1, far - 7, far // 3]], dtype=torch.int32)
    freq = frequencies(64)
    freq[1], freq[2], freq[3], freq[4] = -0.7, 0.0, 1e-30, 1.9
    out, _ = m.attn_rope_bf16(x.cuda(), None, pos[0].cuda(), freq.cuda())
    # 64-bit floats hold position * frequency (31 + 24 bits) to 2^-52 of 2^32 radians: 2^-21 in the
    # worst; whole turns are taken off exactly instead
    from fractions import Fraction
    turn = Fraction(0)
    for i in range(60):                      # pi = 16 arctan(1/5) - 4 arctan(1/239)
        turn += 2 * Fraction((-1) ** i, 2 * i + 1) * (Fraction(16, 5 ** (2 * i + 1)) - Fraction(4, 239 ** (2 * i + 1)))
    want = x.transpose(0, 1).double().clone()
    for t in range(4):
        for i in range(64):
            a = Fraction(int(pos[0, t])) * Fraction(float(freq[i]))
            a = torch.tensor(float(a - turn * round(a / turn)), dtype=torch.float64)
            u, w = x[t, 0, i].double(), x[t, 0, 64 + i].double()
            want[0, t, i] = u * a.cos() - w * a.sin()
            want[0, t, 64 + i] = u * a.sin() + w * a.cos()
    ref.check(out.transpose(0, 1), want, ref.rope_bound(x.transpose(0, 1), want, 64), f"position {far}")


def test_inverse_is_the_gradient():
    """<R x, g> = <x, R' g>, and R' R x = x up to the two roundings."""
    m = fa()
    x, g = make((40, 4, 128), 12), make((40, 4, 128), 13)
    pos, freq = torch.arange(40, dtype=torch.int32).cuda() * 1000, frequencies(64).cuda()
    y, _ = m.attn_rope_bf16(x.cuda(), None, pos, freq)
    back, _ = m.attn_rope_bf16(y, None, pos, freq, inverse=True)
    pair = x.double().abs()
    pair = (pair[..., :64] + pair[..., 64:]).repeat(1, 1, 2)
    # y's rounding turns into at most HALF (|x| + |y|) of the pair, the second adds HALF |x|
    assert ((back.cpu().double() - x.double()).abs() <= ref.HALF * (2 * pair + x.double().abs()) + 2.0 ** -18 * pair).all()
    gx, _ = m.attn_rope_bf16(g.cuda(), None, pos, freq, inverse=True)
    lhs = (y.cpu().double() * g.double()).sum()
    rhs = (x.double() * gx.cpu().double()).sum()
    size = (y.cpu().double().abs() * g.double().abs()).sum() + (x.double().abs() * gx.cpu().double().abs()).sum()
    assert abs(lhs - rhs) <= (ref.HALF + 2.0 ** -17) * size


def test_nothing_to_turn():
    m = fa()
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, _ = m.attn_rope_bf16(q, None, torch.empty(0, dtype=torch.int32, device="cuda"), frequencies(32).cuda())
    assert out.shape == q.shape


def test_streams_and_graph():
    m = fa()
    q, k = make((300, 8, 128), 14).cuda(), make((300, 2, 128), 15).cuda()
    pos, freq = torch.arange(300, dtype=torch.int32).cuda(), frequencies(64).cuda()
    want = m.attn_rope_bf16(q, k, pos, freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = m.attn_rope_bf16(q, k, pos, freq, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.zeros_like(q), torch.zeros_like(k)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.attn_rope_bf16(q, k, pos, freq, q_out=outs[0], k_out=outs[1])
    pos += 17
    graph.replay()
    torch.cuda.synchronize()
    want = m.attn_rope_bf16(q, k, pos, freq)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals():
    m = fa()
    q, pos, freq = make((8, 2, 64), 16).cuda(), torch.arange(8, dtype=torch.int32).cuda(), frequencies(32).cuda()
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(positions=pos.long()), dict(inv_freq=freq.double()),
                dict(axis=torch.zeros(31, dtype=torch.int32, device="cuda")), dict(positions=pos[:7].contiguous())):
        with pytest.raises(TypeError):
            m.attn_rope_bf16(**{**dict(q=q, k=None, positions=pos, inv_freq=freq), **bad})
    with pytest.raises(ValueError):
        m.attn_rope_bf16(q, q[:7], pos, freq)
    with pytest.raises(ValueError):
        m.attn_rope_bf16(q.transpose(1, 2).contiguous().transpose(1, 2), None, pos, freq)
    for f in (frequencies(33), frequencies(40), frequencies(0)):
        with pytest.raises(m.AttnError):
            m.attn_rope_bf16(q, None, pos, f.cuda())
    flat = torch.zeros(8 * 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(m.AttnError):
        m.attn_rope_bf16(flat[4:].view(8, 2, 64), None, pos, freq)
    with pytest.raises(m.AttnError):
        m.attn_rope_bf16(torch.zeros(8, 2, 68, dtype=torch.bfloat16, device="cuda")[..., :64], None, pos, freq)
