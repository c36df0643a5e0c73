"""Failure detection of differential attention's kernels: a load that never comes runs their bounded waits
out, the status says so, and the next normal call gives what it gave before."""
import pytest
import torch

from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu


def fa():
    require_gpu()
    import exact_attention_55_gb300 as module
    return module


def make(shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("withheld", [0, 3])
def test_forward_and_backward(d, withheld):
    m = fa()
    N = 1000
    q, k, v, g = make((1, 4, N, d), 1), make((1, 2, N, d), 2), make((1, 1, N, 2 * d), 3), make((1, 2, N, 2 * d), 4)
    lam = torch.tensor([0.3, 0.7], device="cuda")
    o, lse, o2 = m.attn_diff_fwd_bf16(q, k, v, lam, causal=True, save_o2=True)
    grads = m.attn_diff_bwd_bf16(q, k, v, lam, o, o2, g, lse, causal=True)
    assert m.attn_get_device_status() == m.ATTN_OK
    m.attn_selftest_diff_fwd_withheld_load(q, k, v, lam, torch.empty_like(o), torch.empty_like(lse), causal=True,
                                           withheld=withheld)
    assert m.attn_get_device_status() == m.ATTN_ERR_TIMEOUT
    ws = torch.empty(m.attn_diff_bwd_workspace_bytes(1, 2, N), dtype=torch.uint8, device="cuda")
    m.attn_selftest_diff_bwd_withheld_load(q, k, v, lam, o, o2, g, lse, *(torch.empty_like(t) for t in grads), ws,
                                           causal=True, withheld=withheld)
    assert m.attn_get_device_status() == m.ATTN_ERR_TIMEOUT
    again = m.attn_diff_fwd_bf16(q, k, v, lam, causal=True, save_o2=True)
    assert all(torch.equal(a, b) for a, b in zip(again, (o, lse, o2)))
    again = m.attn_diff_bwd_bf16(q, k, v, lam, o, o2, g, lse, causal=True, workspace=ws)
    assert m.attn_get_device_status() == m.ATTN_OK
    assert all(torch.equal(a, b) for a, b in zip(again, grads))


@pytest.mark.parametrize("d,nq", [(64, 1), (64, 3), (128, 1), (128, 2)])
def test_decoding(d, nq):
    m = fa()
    H, kv, page, L = 8, 2, 64, 60000
    width = (L + page - 1) // page
    kc, vc = make((width, 2 * kv, page, d), 5), make((width, 2 * kv, page, d), 6)
    table = torch.randperm(width).to(torch.int32).view(1, -1).cuda()
    lens = torch.tensor([L], dtype=torch.int32).cuda()
    q, lam = make((1, 2 * H, nq, d), 7), torch.rand(H, device="cuda")
    ws = torch.empty(m.attn_diff_decode_workspace_bytes(H, kv, nq, d), dtype=torch.uint8, device="cuda")
    want = m.attn_diff_decode_bf16_paged(q, kc, vc, lam, table, lens, workspace=ws)
    assert m.attn_get_device_status() == m.ATTN_OK
    bad = [torch.empty_like(t) for t in want]
    m.attn_selftest_diff_decode_withheld_load(q, kc, vc, lam, table, lens, *bad, ws)
    assert m.attn_get_device_status() == m.ATTN_ERR_TIMEOUT
    got = m.attn_diff_decode_bf16_paged(q, kc, vc, lam, table, lens, workspace=ws)
    assert m.attn_get_device_status() == m.ATTN_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_limits_are_checked():
    m = fa()
    q, k, v = make((1, 2, 8, 64), 8), make((1, 2, 8, 64), 9), make((1, 1, 8, 128), 10)
    for bad in (dict(withheld=-1), dict(timeout_ns=0), dict(timeout_ns=10 ** 10)):
        with pytest.raises(m.AttnError):
            m.attn_selftest_diff_fwd_withheld_load(q, k, v, torch.ones(1).cuda(), torch.empty_like(v),
                                                   torch.empty(1, 2, 8, device="cuda"), **bad)
