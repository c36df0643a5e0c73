"""Differential attention's forward pass at d = 128 in one launch (which O_2 asks for) and in two, on the same inputs:
batches are sized by the card's SMs so that a call without O_2 takes two launches by a factor of two, and that it did
is read from the bits, since the forms round at different places."""
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


def sequences(H, N, causal):
    """Sequences of N tokens that make twice 25 steps of 128 x 128 scores for every SM."""
    rows, keys = (N + 127) // 128, ((N // 2 + 64 if causal else N) + 127) // 128
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return math.ceil(2 * 25 * sms / (2 * H * rows * keys))


def both(m, q, k, v, lam, **mask):
    """(o, lse) of the one-launch form and of the two-launch form."""
    dev = [t.cuda() for t in (q, k, v, lam)]
    one = m.attn_diff_fwd_bf16(*dev, save_o2=True, **mask)[:2]
    two = m.attn_diff_fwd_bf16(*dev, **mask)[:2]
    assert m.attn_get_device_status() == m.ATTN_OK
    assert not torch.equal(one[0], two[0]), "the call without O_2 took one launch"
    return one, two


def exact_scores(B, H, G, N, level):
    """Queries and keys whose scores (scale 1) are exact in fp32 in every order of their sums: +-level for all keys of
    a map, and multiples of 1/4 of at most 8 beside it."""
    gen = torch.Generator().manual_seed(91)
    q, k = torch.zeros(B, 2 * H, N, D), torch.zeros(B, 2 * G, N, D)
    q[..., 1:9] = torch.randint(-1, 2, (B, 2 * H, N, 8), generator=gen).float()
    k[..., 1:9] = torch.randint(-4, 5, (B, 2 * G, N, 8), generator=gen).float() / 4
    q[..., 0] = level / 512
    k[:, 0::2, :, 0], k[:, 1::2, :, 0] = 512, -512
    return q.bfloat16(), k.bfloat16()


def plain(q, k, v, lam, scale, ok):
    """One sequence's o, lse and bounds where scores are exact: what is off are the weights, each rounded once to bf16
    (or their difference, which is off by no more), the fp32 exponentials, sums and products (2^-12), and O's rounding;
    the LSE by four fp32 roundings."""
    want = ref.forward(q, k, v, lam, scale, ok)
    H, G = q.shape[0] // 2, q.shape[0] // k.shape[0]
    vv = v.double().abs().repeat_interleave(G, 0)
    size = want["p"][0::2] @ vv + lam.double().abs()[:, None, None] * (want["p"][1::2] @ vv)
    return want["o"], (ref.HALF + 2.0 ** -12) * size + ref.HALF * want["o"].abs(), want["lse"], want["lse"].abs() * 2.0 ** -22 + 2.0 ** -17


@pytest.mark.parametrize("level", [0, 2 ** 14, 2 ** 18])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 200)])
def test_large_log_sum_exps(level, causal, window):
    """Scores of some 2^18 that differ by little: a log-sum-exp in fp32 is off by several 2^-7 of a unit there, which
    must not be an error of the weights."""
    m = fa()
    H, G, N = 4, 2, 400
    B = sequences(H, N, causal) if not window else 2 * sequences(H, N, causal)
    q, k = exact_scores(B, H, G, N, level)
    v, lam, ok = make((B, G, N, 2 * D), 92), weights(H), ref.allowed(N, causal, window)
    for name, (o, lse) in zip(("one", "two"), both(m, q, k, v, lam, scale=1.0, causal=causal, window=window)):
        for b in (0, B // 2, B - 1):
            want, bound, ls, ls_bound = plain(q[b], k[b], v[b], lam, 1.0, ok)
            ref.check(o[b], want, bound, f"o {name} {b}")
            ref.check(lse[b], ls, ls_bound, f"lse {name} {b}")


def test_rows_without_a_weight_in_one_map():
    """A row whose every score in one map is -inf has the other map alone, in both forms."""
    m = fa()
    H, N = 4, 300
    B = sequences(H, N, True)
    q, k, v = make((B, 2 * H, N, D), 93).abs() + 0.1, make((B, 2 * H, N, D), 94), make((B, H, N, 2 * D), 95)
    lam = weights(H)
    assert (q[0].double() @ k[0].double().abs().transpose(1, 2)).max() / math.sqrt(D) < 16
    k[0, 0, :140] = k[0, 3, :140] = -float("inf")        # map 1 of head 0, map 2 of head 1
    for name, (o, lse) in zip(("one", "two"), both(m, q, k, v, lam, causal=True)):
        want = ref.forward(q[0], k[0], v[0], lam, 1 / math.sqrt(D), ref.allowed(N, True, 0).expand(2 * H, N, N)
                           & (k[0, :, :, :1].transpose(1, 2) > -float("inf")))
        ref.check(lse[0], want["lse"], torch.full_like(want["lse"], 1e-3), f"lse {name}")
        a = want["p"][0::2] @ v[0].double().abs()
        b = lam[:, None, None] * (want["p"][1::2] @ v[0].double().abs())
        # beside the roundings above: scores are fp32 sums of 128 products whose magnitudes add up to less than 2^4, so
        # off by 2^-13, and a weight by that much twice (in itself and in the sum)
        ref.check(o[0], want["o"], (ref.HALF + 2.0 ** -11) * (a + b) + ref.HALF * want["o"].abs(), f"o {name}")


@pytest.mark.parametrize("causal", [False, True])
def test_uneven_lengths(causal):
    """One long document beside many short ones, in both forms."""
    m = fa()
    lens, H, G = [50, 7, 2500] + [50] * 5, 64, 16
    T, cu = sum(lens), torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    q, k, v = make((T, 2 * H, D), 96), make((T, 2 * G, D), 97), make((T, G, 2 * D), 98)
    lam = weights(H)
    dev = [t.cuda() for t in (q, k, v, lam, cu)]
    one = m.attn_diff_fwd_bf16_varlen(*dev, max(lens), causal=causal, save_o2=True)
    two = m.attn_diff_fwd_bf16_varlen(*dev, max(lens), causal=causal)
    assert m.attn_get_device_status() == m.ATTN_OK
    assert not torch.equal(one[0], two[0]), "the call without O_2 took one launch"
    for s, n in enumerate(lens):
        rows = slice(int(cu[s]), int(cu[s + 1]))
        for h in (0, 63):
            g = h // (H // G)
            want = ref.forward(*(t[rows, a:b].transpose(0, 1) for t, a, b in ((q, 2 * h, 2 * h + 2), (k, 2 * g, 2 * g + 2), (v, g, g + 1))),
                               lam[h:h + 1], 1 / math.sqrt(D), ref.allowed(n, causal, 0))
            for name, (o, lse, _) in (("one", one), ("two", two)):
                ref.check(o[rows, h:h + 1].transpose(0, 1), want["o"], want["o_bound"], f"o {name} {s} {h}")
                ref.check(lse[2 * h:2 * h + 2, rows], want["lse"], want["lse_bound"], f"lse {name} {s} {h}")
