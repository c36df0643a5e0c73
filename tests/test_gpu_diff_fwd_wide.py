"""Differential attention's forward pass at d = 128 without O_2 in its two-launch form (at least 25 steps of
128 x 128 scores an SM: hundreds of heads here, of which some are checked) against the plain 64-bit form, with the bounds of the one-launch form: the weights' difference is
rounded once, which is off by no more than its two terms rounded by themselves."""
import math

import pytest
import torch

from tests import diff_reference as ref
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu
D = 128


def fa():
    require_gpu()
    import exact_attention_55_gb300 as module
    return module


def make(shape, seed, size=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * size).bfloat16()


def weights(H):
    return torch.rand(H, generator=torch.Generator().manual_seed(5)) * 0.8 + 0.1


def batched(B, H, G, N, seed=1, size=1.0):
    return make((B, 2 * H, N, D), seed, size), make((B, 2 * G, N, D), seed + 1, size), make((B, G, N, 2 * D), seed + 2)


def compare(m, q, k, v, lam, causal, window, scale=None, batches=None):
    o, lse, _ = m.attn_diff_fwd_bf16(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), scale=scale, causal=causal, window=window)
    assert m.attn_get_device_status() == m.ATTN_OK
    N = q.shape[2]
    for b in batches or range(q.shape[0]):
        want = ref.forward(q[b], k[b], v[b], lam, scale or 1 / math.sqrt(D), ref.allowed(N, causal, window))
        ref.check(o[b], want["o"], want["o_bound"], f"o {b}")
        ref.check(lse[b], want["lse"], want["lse_bound"], f"lse {b}")


@pytest.mark.parametrize("N", [257, 300, 383, 384, 385, 512, 640, 769])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 256), (False, 300)])
def test_batched(N, causal, window):
    compare(fa(), *batched(40, 8, 8, N), weights(8), causal, window, batches=(0, 19, 39))


@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (4, 2), (12, 3)])
def test_shared_heads(H, G):
    B = 204 // H
    compare(fa(), *batched(B, H, G, 400), weights(H), True, 0, 0.2, batches=(0, B // 2, B - 1))


def test_many_tiles_and_large_scores():
    """The running maximum moves often: scores up to some hundred, and a last key that outweighs all."""
    q, k, v = batched(3, 16, 16, 1500, seed=11, size=3.0)
    k[:, :, 1400] *= 4
    compare(fa(), q, k, v, weights(16), True, 0, 0.3, batches=(1,))


def test_weights_of_zero_and_of_equal_maps():
    m = fa()
    q, k, v = batched(40, 8, 8, 300, seed=21)
    compare(m, q, k, v, torch.zeros(8), True, 0, batches=(3,))
    q[:, 1::2], k[:, 1::2] = q[:, ::2], k[:, ::2]
    o, _, _ = m.attn_diff_fwd_bf16(q.cuda(), k.cuda(), v.cuda(), torch.ones(8).cuda(), causal=True)
    assert not o.any()


@pytest.mark.parametrize("lens", [[700, 1, 513, 0, 257, 300], [257] * 12, [2000, 5], [128, 600, 256, 640, 129]])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 256)])
def test_packed(lens, causal, window):
    """Rows before the first sequence and behind the last are NaN on the way in, and left as they were."""
    m = fa()
    H, G, lead, trail = 64, 16, 3, 70
    T = lead + sum(lens) + trail
    q, k, v = make((T, 2 * H, D), 31), make((T, 2 * G, D), 32), make((T, G, 2 * D), 33)
    for t in (q, k, v):
        t[:lead] = t[T - trail:] = float("nan")
    cu = torch.tensor([lead] + lens).cumsum(0).to(torch.int32)
    lam = weights(H)
    o = torch.full((T, H, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2 * H, T), 7.0, device="cuda")
    m.attn_diff_fwd_bf16_varlen(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), cu.cuda(), max(lens), causal=causal, window=window,
                                o=o, lse=lse)
    assert m.attn_get_device_status() == m.ATTN_OK
    assert (o[:lead] == 7).all() and (o[T - trail:] == 7).all() and (lse[:, :lead] == 7).all() and (lse[:, T - trail:] == 7).all()
    some = [0, 1, 2, 7, 62, 63]                     # value groups of four heads
    for s, n in enumerate(lens):
        if n == 0:
            continue
        rows = slice(int(cu[s]), int(cu[s + 1]))
        for h in some:
            g = h // (H // G)
            one = ref.forward(q[rows, 2 * h:2 * h + 2].transpose(0, 1), k[rows, 2 * g:2 * g + 2].transpose(0, 1),
                              v[rows, g:g + 1].transpose(0, 1), lam[h:h + 1], 1 / math.sqrt(D), ref.allowed(n, causal, window))
            ref.check(o[rows, h:h + 1].transpose(0, 1), one["o"], one["o_bound"], f"o {s} {h}")
            ref.check(lse[2 * h:2 * h + 2, rows], one["lse"], one["lse_bound"], f"lse {s} {h}")


def test_sequences_between_nan():
    """A sequence's neighbours in memory do not reach it."""
    m = fa()
    H, lens = 80, [300, 333, 400]
    T = sum(lens)
    q, k, v = make((T, 2 * H, D), 41).cuda(), make((T, 2 * H, D), 42).cuda(), make((T, H, 2 * D), 43).cuda()
    cu, lam = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda(), weights(H).cuda()
    want = m.attn_diff_fwd_bf16_varlen(q, k, v, lam, cu, 400, causal=False)
    for t in (q, k, v):
        t[:300] = float("nan")
        t[633:] = float("inf")
    got = m.attn_diff_fwd_bf16_varlen(q, k, v, lam, cu, 400, causal=False)
    assert torch.equal(got[0][300:633], want[0][300:633]) and torch.equal(got[1][:, 300:633], want[1][:, 300:633])
    assert got[0][:300].isnan().all() and got[0][633:].isnan().all()
    assert got[1][:, :300].isnan().all() and got[1][:, 633:].isnan().all()


def test_more_sequences_than_the_table():
    m = fa()
    lens = [257 + 7 * (i % 5) for i in range(230)]
    T = sum(lens)
    q, k, v = make((T, 4, D), 51), make((T, 2, D), 52), make((T, 1, 2 * D), 53)
    cu, lam = torch.tensor([0] + lens).cumsum(0).to(torch.int32), weights(2)
    o, lse, _ = m.attn_diff_fwd_bf16_varlen(q.cuda(), k.cuda(), v.cuda(), lam.cuda(), cu.cuda(), max(lens), causal=True)
    assert m.attn_get_device_status() == m.ATTN_OK
    for s in (0, 1, 100, 228, 229):
        rows = slice(int(cu[s]), int(cu[s + 1]))
        want = ref.forward(q[rows].transpose(0, 1), k[rows].transpose(0, 1), v[rows].transpose(0, 1), lam, 1 / math.sqrt(D),
                           ref.allowed(lens[s], True, 0))
        ref.check(o[rows].transpose(0, 1), want["o"], want["o_bound"], f"o {s}")
        ref.check(lse[:, rows], want["lse"], want["lse_bound"], f"lse {s}")


def test_infinite_keys():
    """A key whose scores are -inf for every query has no weight; rows that see no other have an LSE of -inf and
    an output of 0; a NaN score makes its row's output and LSE NaN."""
    m = fa()
    q, k, v = batched(40, 8, 8, 300, seed=61)
    q = q.abs() + 0.1
    k[:, :, 0] = -float("inf")
    k[2, 0, 250] = float("nan")
    o, lse, _ = m.attn_diff_fwd_bf16(q.cuda(), k.cuda(), v.cuda(), weights(8).cuda(), causal=True)
    assert not o[:, :, 0].any() and (lse[:, :, 0] == -float("inf")).all()
    keep = torch.ones(40, 8, 300, dtype=torch.bool)
    keep[2, 0, 250:] = False
    assert torch.equal(o.cpu().isnan().any(-1), ~keep)
    assert lse[2, 0, 250:].isnan().all() and not lse[2, 1].isnan().any()


def test_same_bits_every_time_streams_and_graph():
    m = fa()
    q, k, v = (t.cuda() for t in batched(10, 8, 4, 700, seed=71))
    lam = weights(8).cuda()
    first = m.attn_diff_fwd_bf16(q, k, v, lam, causal=True)[:2]
    # the one-launch form, which gives O_2 too, rounds the maps' weights one by one
    one = m.attn_diff_fwd_bf16(q, k, v, lam, causal=True, save_o2=True)[0]
    assert not torch.equal(one, first[0]) and (one - first[0]).abs().max() < 0.1
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(3):                              # two calls at once
        for s in side:
            with torch.cuda.stream(s):
                outs.append(m.attn_diff_fwd_bf16(q, k, v, lam, causal=True)[:2])
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse, _ = m.attn_diff_fwd_bf16(q, k, v, lam, causal=True)
    q.copy_(q.flip(2))
    want = m.attn_diff_fwd_bf16(q, k, v, lam, causal=True)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert m.attn_get_device_status() == m.ATTN_OK


@pytest.mark.parametrize("withheld", [0, 1, 2, 5])
def test_withheld_load(withheld):
    m = fa()
    q, k, v = (t.cuda() for t in batched(2, 65, 65, 600, seed=81))
    lam = weights(65).cuda()
    want = m.attn_diff_fwd_bf16(q, k, v, lam, causal=True)
    assert m.attn_get_device_status() == m.ATTN_OK
    m.attn_selftest_diff_fwd_withheld_load(q, k, v, lam, torch.empty_like(want[0]), torch.empty_like(want[1]), causal=True,
                                           withheld=withheld)
    assert m.attn_get_device_status() == m.ATTN_ERR_TIMEOUT
    got = m.attn_diff_fwd_bf16(q, k, v, lam, causal=True)
    assert m.attn_get_device_status() == m.ATTN_OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
