"""The weights of differential attention's decoding step are off by at most 2^-17 of themselves: they enter as two
bf16 numbers.  Values far from zero and maps whose difference nearly cancels leave outputs of the size of the weights'
errors, so a weight rounded once to bf16 (off by 2^-8) does not pass, which is shown on the plain form."""
import math

import pytest
import torch

from tests import diff_reference as ref
from tests.conftest import require_gpu

PAGE = 64


def inputs(H, kv, d, nq, L, seed):
    """Scores (scale 1) are exact in fp32: multiples of 1/4 of at most 8."""
    gen = torch.Generator().manual_seed(seed)
    q, k = torch.zeros(2 * H, nq, d), torch.zeros(L, 2 * kv, d)
    q[..., :8] = torch.randint(-1, 2, (2 * H, nq, 8), generator=gen).float()
    k[..., :8] = torch.randint(-4, 5, (L, 2 * kv, 8), generator=gen).float() / 4
    v = torch.randn(L, 2 * kv, d, generator=gen) + 4
    return q.bfloat16(), k.bfloat16(), v.bfloat16(), torch.full((H,), 1.0)


def seen_by(nq, L, window):
    at, j = torch.arange(L - nq, L)[:, None], torch.arange(L)[None]
    ok = j <= at
    return ok & (j >= at - window) if window else ok


def expected(q, k, v, lam, ok):
    """O and its bound.  A weight is off by 2^-17 for what two bf16 numbers leave of it; by 2^-18 for the exponential
    and its fp32 argument of at most 16, and its sum by as much; the fp32 sums of the tensor cores by a step of the
    running sum for every 16 keys, and for 64 more of the joining.  O is rounded once to bf16."""
    L, kv, d = k.shape[0], k.shape[1] // 2, k.shape[2]
    G = q.shape[0] // (2 * kv)
    want = ref.forward(q, k.transpose(0, 1), v.reshape(L, kv, 2 * d).transpose(0, 1), lam, 1.0, ok)
    vv = v.double().reshape(L, kv, 2 * d).transpose(0, 1).abs().repeat_interleave(G, 0)
    size = want["p"][0::2] @ vv + lam[:, None, None] * (want["p"][1::2] @ vv)
    return want, (2.0 ** -17 + 2.0 ** -17 + (L / 16 + 64) * 2.0 ** -23) * size + ref.HALF * want["o"].abs()


def test_the_bound_tells_one_rounding_from_two():
    q, k, v, lam = inputs(2, 2, 64, 1, 100, 1)
    ok = seen_by(1, 100, 0)
    want, bound = expected(q, k, v, lam, ok)
    vv = v.double().reshape(100, 2, 128).transpose(0, 1)
    top = want["p"].amax(-1, keepdim=True)
    w = want["p"] / top                                           # relative to the running maximum, as stored
    once = w.bfloat16().double()
    twice = once + (w - once).bfloat16().double()
    out = lambda x: (x[0::2] * top[0::2]) @ vv - lam[:, None, None] * ((x[1::2] * top[1::2]) @ vv)
    assert ((out(twice) - want["o"]).abs() <= bound).all()
    assert ((out(once) - want["o"]).abs() > 2 * bound).any()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,kv,nq", [(2, 2, 1), (8, 2, 1), (2, 2, 3), (8, 1, 1), (16, 2, 2)])
@pytest.mark.parametrize("L,window", [(20, 0), (100, 0), (300, 50), (6000, 0)])
def test_weights(d, H, kv, nq, L, window):
    require_gpu()
    import exact_attention_55_gb300 as m
    q, k, v, lam = inputs(H, kv, d, nq, L, 7)
    pages = (L + PAGE - 1) // PAGE
    caches = []
    for rows in (k, v):
        c = torch.zeros(pages, PAGE, 2 * kv, d, dtype=torch.bfloat16)
        c.view(-1, 2 * kv, d)[:L] = rows
        caches.append(c.transpose(1, 2).contiguous().cuda())
    o, _ = m.attn_diff_decode_bf16_paged(q[None].cuda(), *caches, lam.cuda(),
                                         torch.arange(pages, dtype=torch.int32).view(1, -1).cuda(),
                                         torch.tensor([L], dtype=torch.int32).cuda(), scale=1.0, window=window)
    assert m.attn_get_device_status() == m.ATTN_OK
    want, bound = expected(q, k, v, lam, seen_by(nq, L, window))
    ref.check(o[0], want["o"], bound, "o")
