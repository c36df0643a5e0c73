"""Differential attention and rotary positions on tensors of more than 2^31 elements: the last rows of the last
heads, with a window of one key so that they depend on few rows."""
import math

import pytest
import torch

from tests import diff_reference as ref
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu
N, H, D, LAST = 66000, 128, 128, 150


def fa():
    require_gpu()
    import exact_attention_55_gb300 as module
    return module


def make(shape, seed):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("packed", [False, True])
def test_forward_and_backward(packed):
    m = fa()
    shape = (lambda heads, width: (N, heads, width)) if packed else (lambda heads, width: (1, heads, N, width))
    q, k, v, g = (make(shape(*s), i) for i, s in enumerate(((2 * H, D), (2, D), (1, 2 * D), (H, 2 * D))))
    assert q.numel() > 2 ** 31 and g.numel() > 2 ** 31
    lam = torch.rand(H, device="cuda")
    mask = dict(causal=True, window=1)
    cu = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    if packed:
        one = m.attn_diff_fwd_bf16_varlen(q, k, v, lam, cu, N, **mask)
        o, lse, o2 = m.attn_diff_fwd_bf16_varlen(q, k, v, lam, cu, N, save_o2=True, **mask)
        grads = m.attn_diff_bwd_bf16_varlen(q, k, v, lam, o, o2, g, lse, cu, N, **mask)
    else:
        one = m.attn_diff_fwd_bf16(q, k, v, lam, **mask)
        o, lse, o2 = m.attn_diff_fwd_bf16(q, k, v, lam, save_o2=True, **mask)
        grads = m.attn_diff_bwd_bf16(q, k, v, lam, o, o2, g, lse, **mask)
    assert m.attn_get_device_status() == m.ATTN_OK
    rows = lambda t: (t[-LAST:].transpose(0, 1) if packed else t[0, :, -LAST:]).cpu()
    ls = (lse if packed else lse[0])[:, -LAST:].cpu()
    ok = ref.allowed(LAST, True, 1)
    want = ref.forward(rows(q)[-2:], rows(k), rows(v), lam[-1:].cpu(), 1 / math.sqrt(D), ok)
    seen = slice(1, None)                            # the first of these rows sees a key before them
    for out, logs in ((o, ls), (one[0], (one[1] if packed else one[1][0])[:, -LAST:].cpu())):
        ref.check(rows(out)[-1:, seen], want["o"][:, seen], want["o_bound"][:, seen], "o")
        ref.check(logs[-2:, seen], want["lse"][:, seen], want["lse_bound"][:, seen], "lse")
    ref.check(rows(o2)[-1:, seen], want["o2"][:, seen], want["o2_bound"][:, seen], "o2")
    back, bound = ref.backward(rows(q)[-2:], rows(k), rows(v), lam[-1:].cpu(), rows(o)[-1:], rows(o2)[-1:], rows(g)[-1:],
                               ls[-2:], 1 / math.sqrt(D), ok)
    ref.check(rows(grads[0])[-2:, seen], back[0][:, seen], bound[0][:, seen], "dq")
    # the last key's gradients, over all heads
    all_heads = [ref.backward(rows(q)[2 * h:2 * h + 2], rows(k), rows(v), lam[h:h + 1].cpu(), rows(o)[h:h + 1], rows(o2)[h:h + 1],
                              rows(g)[h:h + 1], ls[2 * h:2 * h + 2], 1 / math.sqrt(D), ok) for h in range(H)]
    for i, name in ((1, "dk"), (2, "dv")):
        total = sum(x[0][i][:, -1] for x in all_heads)
        allowed = sum(x[1][i][:, -1] for x in all_heads)
        ref.check(rows(grads[i])[:, -1], total, allowed, name)
    # d lam of the last head: minus the sum of dO . O_2
    second, up = (o2[:, -1], g[:, -1]) if packed else (o2[0, -1], g[0, -1])
    terms = second.double() * up.double()
    assert abs(grads[3][-1].item() + terms.sum().item()) <= 2.0 ** -16 * terms.abs().sum().item()


def test_rope():
    m = fa()
    x = make((N, 2 * H, D), 9)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    freq = torch.pow(torch.tensor(1e4), -torch.arange(D // 2) / (D // 2))
    y, _ = m.attn_rope_bf16(x, None, pos, freq.cuda())
    assert m.attn_get_device_status() == m.ATTN_OK
    part, last = x[-LAST:].transpose(0, 1).cpu(), pos[-LAST:].cpu()
    want = ref.rope(part, last[None], freq)
    ref.check(y[-LAST:].transpose(0, 1), want, ref.rope_bound(part, want, D // 2), "rope")
