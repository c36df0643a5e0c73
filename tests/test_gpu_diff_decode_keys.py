"""Keys of differential attention's decoding step whose scores are not finite: they reach the log-sum-exp of their own
map alone, and a key whose score is -inf has no weight there."""
import math

import pytest
import torch

from tests import diff_reference as ref
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu
PAGE = 64


def fa():
    require_gpu()
    import exact_attention_55_gb300 as module
    return module


def make(shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


def paged(rows):
    """[L, heads, d] as pages in order."""
    L, heads, d = rows.shape
    pages = (L + PAGE - 1) // PAGE
    out = torch.zeros(pages, PAGE, heads, d, dtype=torch.bfloat16)
    out.view(-1, heads, d)[:L] = rows
    return out.transpose(1, 2).contiguous()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,kv,nq", [(1, 1, 1), (4, 1, 1), (2, 2, 3), (8, 1, 1), (8, 2, 3)])
@pytest.mark.parametrize("L,at", [(100, 17), (100, 99), (6000, 3333)])
@pytest.mark.parametrize("bad", [float("nan"), -float("inf")])
@pytest.mark.parametrize("mp", [0, 1])
def test_one_maps_key(d, H, kv, nq, L, at, bad, mp):
    m = fa()
    q, k, v = make((1, 2 * H, nq, d), 1).abs() + 0.1, make((L, 2 * kv, d), 2), make((L, 2 * kv, d), 3)
    lam = torch.rand(H, generator=torch.Generator().manual_seed(4)) * 0.8 + 0.1
    k[at, mp] = bad                                    # key pair 0's map mp
    pages = (L + PAGE - 1) // PAGE
    table = torch.arange(pages, dtype=torch.int32).view(1, -1)
    o, lse = m.attn_diff_decode_bf16_paged(q.cuda(), paged(k).cuda(), paged(v).cuda(), lam.cuda(), table.cuda(),
                                           torch.tensor([L], dtype=torch.int32).cuda())
    assert m.attn_get_device_status() == m.ATTN_OK
    # the definition, a key with a score of -inf masked in its map
    pos, j = torch.arange(L - nq, L)[:, None], torch.arange(L)[None]
    seen = (j <= pos).expand(2 * H, nq, L).clone()
    hit = torch.zeros(2 * H, nq, dtype=torch.bool)     # rows of q whose scores have a NaN
    mine = [2 * h + mp for h in range(H // kv)]
    if math.isnan(bad):
        hit[mine] = seen[0, :, at]
    seen[mine, :, at] = False
    kk, vv = k.clone(), v.reshape(L, kv, 2 * d).transpose(0, 1)
    kk[at, mp] = 0
    want = ref.forward(q[0], kk.transpose(0, 1), vv, lam, 1 / math.sqrt(d), seen)
    nan_o = hit.view(H, 2, nq).any(1)
    lse, o = lse[0].cpu(), o[0].cpu()
    assert torch.equal(lse.isnan(), hit)
    assert torch.equal(o.isnan().all(-1), nan_o) and torch.equal(o.isnan().any(-1), nan_o)
    keep, rows = ~nan_o, ~hit
    ref.check(lse[rows], want["lse"][rows], want["lse_bound"][rows], "lse")
    ref.check(o[keep], want["o"][keep], want["o_bound"][keep], "o")
