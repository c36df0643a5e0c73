"""A training step over packed documents: rotary positions that start over in each, differential attention, its
gradients with those of the maps' weights, and the rotation back."""
import math

import pytest
import torch

from tests import diff_reference as ref
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu


def make(shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["batched", "packed"])
def test_step_with_the_weights_gradient(d, layout):
    require_gpu()
    import exact_attention_55_gb300 as m
    H, Hkv = 4, 2
    lens = [150, 150] if layout == "batched" else [140, 1, 0, 259]
    T, cu = sum(lens), torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    q, k, v, g = make((T, 2 * H, d), 1), make((T, 2 * Hkv, d), 2), make((T, Hkv, 2 * d), 3), make((T, H, 2 * d), 4)
    lam, half = torch.tensor([0.2, 0.4, 0.6, 0.8]), d // 2
    freq = torch.pow(torch.tensor(10000.0), -torch.arange(half, dtype=torch.float32) / half)
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens])
    if layout == "batched":
        B, N = len(lens), lens[0]
        put = lambda t: t.view(B, N, *t.shape[1:]).transpose(1, 2).contiguous().cuda()
        rows = lambda t, b: t[b].cpu()
        logs = lambda t, b: t[b].cpu()
        args, fwd, bwd = (pos.view(B, N).cuda(), freq.cuda()), m.attn_diff_fwd_bf16, m.attn_diff_bwd_bf16
    else:
        put = lambda t: t.cuda()
        rows = lambda t, b: t[int(cu[b]):int(cu[b + 1])].transpose(0, 1).cpu()
        logs = lambda t, b: t[:, int(cu[b]):int(cu[b + 1])].cpu()
        args, seqs = (pos.cuda(), freq.cuda()), (cu.cuda(), max(lens))
        fwd = lambda *a, **o: m.attn_diff_fwd_bf16_varlen(*a, *seqs, **o)
        bwd = lambda *a, **o: m.attn_diff_bwd_bf16_varlen(*a, *seqs, **o)
    q, k, v, g = put(q), put(k), put(v), put(g)
    qr, kr = m.attn_rope_bf16(q, k, *args)
    o, lse, o2 = fwd(qr, kr, v, lam.cuda(), causal=True, save_o2=True)
    dqr, dkr, dv, dlam = bwd(qr, kr, v, lam.cuda(), o, o2, g, lse, causal=True)
    dq, dk = m.attn_rope_bf16(dqr, dkr, *args, inverse=True)
    assert m.attn_get_device_status() == m.ATTN_OK
    total, most = 0.0, 0.0
    for b, n in enumerate(lens):
        if n == 0:
            continue
        want, bound = ref.backward(*(rows(t, b) for t in (qr, kr, v)), lam, *(rows(t, b) for t in (o, o2, g)),
                                   logs(lse, b), 1 / math.sqrt(d), ref.allowed(n, True, 0))
        for got, w, e, name in zip((dqr, dkr, dv), want, bound, ("dq", "dk", "dv")):
            ref.check(rows(got, b), w, e, f"{name} {b}")
        total, most = total + want[3], most + bound[3]
        at = torch.arange(n, dtype=torch.int32)[None]
        for got, x, inverse, name in ((qr, q, False, "q"), (kr, k, False, "k"), (dq, dqr, True, "dq"), (dk, dkr, True, "dk")):
            turned = ref.rope(rows(x, b), at, freq, inverse=inverse)
            ref.check(rows(got, b), turned, ref.rope_bound(rows(x, b), turned, half), f"turned {name} {b}")
    ref.check(dlam, total, most, "dlam")
