"""GPU: what many light keys add to O beside a few heavy ones (attn_decode_fp8_paged).

A row whose softmax has a few heavy keys that hold no value, and tens of thousands of light
ones far below them, has its O from the light keys alone, so a weight that is rounded
to 0, or to the next step of a short format, shows in full."""
import numpy as np
import pytest
import torch

from tests import paged_reference as ref
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu

PAGE, LIGHT_PAGES, LIGHT = 64, 5, 1023    # pages of light keys, and how many of them a sequence has
BELOW = (20.6, 22.3, 24.4, 25.05, 26.0, 27.7)   # log2 of a heavy key's weight over a light one's


@pytest.fixture(scope="module")
def fa():
    require_gpu()
    import exact_attention_55_gb300 as fa
    fa.load_library()
    return fa


def heavy_and_light(rng, d, rows, fmt):
    """One key head's keys and values: heavy keys every 16 of the first two pages, whose K is one
    along d = 0 and whose V is 0; all others have K = 0 and positive values.  Query row r is
    a_r along d = 0, so that its scores are a_r at the heavy keys and 0 at the others."""
    pages = 2 + LIGHT_PAGES
    K = np.zeros((pages, PAGE, d), np.float32)
    V = (1.0 + rng.random((pages, PAGE, d))).astype(np.float32)
    K[:2, ::16, 0] = 1.0
    V[:2, ::16] = 0.0
    q = np.zeros((rows, d), np.float32)
    q[:, 0] = np.log(2.0) * np.array([BELOW[r % len(BELOW)] for r in range(rows)])
    q = torch.from_numpy(q).bfloat16()
    table = np.concatenate([[0, 1], 2 + np.arange(LIGHT) % LIGHT_PAGES]).astype(np.int32)
    return ref.encode(K, fmt), ref.encode(V, fmt), q, table


@pytest.mark.parametrize("d,rows,units", [(64, 1, 1024), (64, 16, 640), (128, 8, 1024), (128, 16, 640), (256, 8, 640),
                                          (64, 32, 320), (64, 128, 320), (128, 32, 320), (128, 64, 320), (128, 128, 320),
                                          (256, 64, 320), (256, 128, 320)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_light_keys_beside_heavy_ones(fa, fmt, d, rows, units):
    """More units than ranges, so that units stay whole and a row's maximum holds for all its
    keys.  The bound, with l the sum of weights relative to a heavy key's and n the light keys:
    scores as in paged_reference.decode_fp8 (ds each); a weight is rounded to fp16, half a step
    of 2^-11, and never more than 2^-31 of the largest (a step below fp16's normal numbers at
    2^6 times the weight); fp32 sums 2^-22 n / 16; O in bf16 2^-8."""
    rng = np.random.default_rng(rows)
    kc, vc, q, one = heavy_and_light(rng, d, rows, fmt)
    B = units // 4                                       # 4 key heads with the same content
    k8, v8 = (torch.from_numpy(c[:, None].repeat(4, 1)).cuda() for c in (kc, vc))
    ones = torch.ones(k8.shape[0], 4, 1, device="cuda")
    table = torch.from_numpy(one).cuda().expand(B, len(one)).contiguous()
    L = len(one) * PAGE - 5
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    query = q[None, None, :, None].expand(B, 4, rows, 1, d).reshape(B, 4 * rows, 1, d).cuda()
    o, lse = fa.attn_decode_fp8_paged(query, k8, v8, ones, ones, table, lens, fmt=fmt, scale=1.0)
    assert fa.attn_get_device_status() == fa.ATTN_OK

    t = np.arange(L)
    K, V = (ref.decode(c[one[t // PAGE], t % PAGE], fmt).astype(np.float64) for c in (kc, vc))
    s = q.double().numpy() @ K.T
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    want, want_lse = p @ V / l, (m + np.log(l))[:, 0]
    ds = d * 2.0 ** -23 * m + 2.0 ** -21 * (1 + m)
    tol = want * (2.0 ** -8 + 2.0 ** -11 + 2 * ds + 2.0 ** -22 * L / 16) + 2.0 ** -31 / l * V.sum(0)
    lse_tol = ds[:, 0] + 2.0 ** -22 * (L / 16 + np.abs(want_lse))
    # the bound itself is tight: a light key's whole weight lost would be several times it
    assert (tol < 0.3 * want).all()
    o, lse = (x.double().cpu().numpy() for x in (o, lse))
    off = np.abs(o.reshape(B * 4, rows, d) - want)
    assert (off <= tol).all(), (off / want).max((0, 2)).tolist()
    assert (np.abs(lse.reshape(B * 4, rows) - want_lse) <= lse_tol).all()
