"""Differential attention's decoding step over a paged cache against a plain 64-bit form."""
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


def cache(lens, kv, d, page, width, seed, fill=float("nan")):
    """Keys and values in pages of random order; everything that no sequence owns holds `fill`."""
    gen = torch.Generator().manual_seed(seed)
    pages = sum((n + page - 1) // page for n in lens) + 2
    order = torch.randperm(pages, generator=gen).tolist()
    kc, vc = (torch.full((pages, 2 * kv, page, d), fill, dtype=torch.bfloat16) for _ in range(2))
    table = torch.randint(-5, pages + 5, (len(lens), width), generator=gen, dtype=torch.int32)
    rows = []
    for b, n in enumerate(lens):
        k, v = make((n, 2 * kv, d), seed + 10 + 2 * b), make((n, 2 * kv, d), seed + 11 + 2 * b)
        rows.append((k, v))
        for j in range((n + page - 1) // page):
            pg = order.pop()
            table[b, j] = pg
            part = slice(j * page, min(n, (j + 1) * page))
            kc[pg, :, :part.stop - part.start] = k[part].transpose(0, 1)
            vc[pg, :, :part.stop - part.start] = v[part].transpose(0, 1)
    return kc, vc, table, rows


def expected(q, rows, lam, scale, window):
    """Of one sequence: q [2H, nq, d], rows (k, v) [L, 2Hkv, d]."""
    k, v = rows
    L, nq = k.shape[0], q.shape[1]
    at, j = torch.arange(L - nq, L)[:, None], torch.arange(L)[None]
    ok = j <= at
    if window > 0:
        ok &= j >= at - window
    kv = k.shape[1] // 2
    return ref.forward(q, k.transpose(0, 1), v.reshape(L, kv, 2 * k.shape[2]).transpose(0, 1), lam, scale, ok)


def compare(m, lens, H, kv, d, nq, page, window=0, seed=100, width=None, size=1.0):
    width = width or max(1, (max(lens) + page - 1) // page)
    kc, vc, table, rows = cache(lens, kv, d, page, width, seed)
    q, lam = make((len(lens), 2 * H, nq, d), seed + 1, size), weights(H)
    o, lse = m.attn_diff_decode_bf16_paged(q.cuda(), kc.cuda(), vc.cuda(), lam.cuda(), table.cuda(),
                                           torch.tensor(lens, dtype=torch.int32).cuda(), window=window)
    assert m.attn_get_device_status() == m.ATTN_OK
    for b, n in enumerate(lens):
        if n == 0:
            assert (o[b] == 0).all() and (lse[b] == -math.inf).all()
            continue
        want = expected(q[b], rows[b], lam, 1 / math.sqrt(d), window)
        ref.check(o[b], want["o"], want["o_bound"], f"o {b}")
        ref.check(lse[b], want["lse"], want["lse_bound"], f"lse {b}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,kv,nq", [(1, 1, 1), (2, 2, 3), (4, 1, 1), (4, 1, 2), (8, 2, 4), (3, 1, 5), (8, 1, 8), (5, 5, 8)])
@pytest.mark.parametrize("window", [0, 37])
def test_rows_and_heads(d, H, kv, nq, window):
    """One product for both maps, several, and several passes; lengths from none to a few tiles."""
    compare(fa(), [0, 1, 2, 15, 16, 17, 64, 65, 200], H, kv, d, nq, 16, window)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 1024])
def test_pages(d, page):
    compare(fa(), [5, 63, 129, 700, 1500], 4, 2, d, 2, page)
    compare(fa(), [5, 63, 129, 700, 1500], 4, 2, d, 1, page, window=300)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[20000], [9000, 1, 0, 4000], [2500] * 9 + [31]])
@pytest.mark.parametrize("H,kv,nq", [(2, 2, 1), (8, 2, 2), (8, 1, 3)])
def test_split_and_joined(d, lens, H, kv, nq):
    compare(fa(), lens, H, kv, d, nq, 64)


@pytest.mark.parametrize("d", [64, 128])
def test_large_scores(d):
    """Running maxima that move by much, within a CTA and between parts."""
    compare(fa(), [3000, 100], 2, 1, d, 1, 32, size=6.0)


def test_short_tables_are_whole():
    compare(fa(), [384, 1, 200, 0, 33], 8, 2, 128, 2, 64, width=6)
    compare(fa(), [300] * 200, 2, 2, 64, 1, 16, width=20)


def test_many_sequences():
    gen = torch.Generator().manual_seed(3)
    compare(fa(), torch.randint(0, 500, (300,), generator=gen).tolist(), 2, 1, 64, 1, 16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_only_the_newest_see(d, bad):
    """A NaN or infinite value at the newest token makes its own query's columns NaN and no other's; a NaN
    key makes its own query's row NaN."""
    m = fa()
    H = kv = 2
    nq, L = 3, 150
    kc, vc, table, rows = cache([L], kv, d, 64, 3, 7)
    q, lam = make((1, 2 * H, nq, d), 8), weights(H)
    args = lambda k, v: (q.cuda(), k.cuda(), v.cuda(), lam.cuda(), table.cuda(), torch.tensor([L], dtype=torch.int32).cuda())
    clean, clean_lse = m.attn_diff_decode_bf16_paged(*args(kc, vc))
    pg, at = int(table[0, (L - 1) // 64]), (L - 1) % 64
    v2 = vc.clone()
    v2[pg, 1, at, 5] = bad                           # head 0's second half, column d + 5
    o, lse = m.attn_diff_decode_bf16_paged(*args(kc, v2))
    hit = torch.zeros_like(clean, dtype=torch.bool)
    hit[0, 0, nq - 1, d + 5] = True
    assert o[hit].isnan().all() or (bad == float("inf") and not o[hit].isfinite().any())
    assert torch.equal(o[~hit], clean[~hit]) and torch.equal(lse, clean_lse)
    k2 = kc.clone()
    k2[pg, 2, at] = float("nan")                     # head 1, map 1
    o, lse = m.attn_diff_decode_bf16_paged(*args(k2, vc))
    assert o[0, 1, nq - 1].isnan().all() and lse[0, 2, nq - 1].isnan()
    assert torch.equal(o[0, 0], clean[0, 0]) and torch.equal(o[0, 1, :nq - 1], clean[0, 1, :nq - 1])


def test_against_the_forward_pass():
    """The newest rows of the causal forward pass are the decoding step's, within both bounds."""
    m = fa()
    H, kv, d, L, nq = 4, 2, 128, 777, 4
    kc, vc, table, rows = cache([L], kv, d, 32, 25, 9, fill=0.0)
    k, v = rows[0]
    q = make((2 * H, L, d), 10)
    lam = weights(H)
    o, lse, _ = m.attn_diff_fwd_bf16(q[None].cuda(), k.transpose(0, 1)[None].contiguous().cuda(),
                                     v.reshape(L, kv, 2 * d).transpose(0, 1)[None].contiguous().cuda(), lam.cuda(), causal=True)
    newest = q[None, :, L - nq:].contiguous()
    od, lsed = m.attn_diff_decode_bf16_paged(newest.cuda(), kc.cuda(), vc.cuda(), lam.cuda(), table.cuda(),
                                             torch.tensor([L], dtype=torch.int32).cuda())
    want = expected(newest[0], rows[0], lam, 1 / math.sqrt(d), 0)
    ref.check(od[0], o[0, :, L - nq:].cpu().double(), 2 * want["o_bound"], "o")
    ref.check(lsed[0], lse[0, :, L - nq:].cpu().double(), 2 * want["lse_bound"], "lse")


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 elements: the pages at its end are the ones that are read."""
    m = fa()
    pages, kv, page, d = 66000, 4, 64, 128
    need = 2 * pages * 2 * kv * page * d * 2
    if torch.cuda.mem_get_info()[0] < need + (4 << 30):
        pytest.skip("not enough memory")
    kc = torch.zeros(pages, 2 * kv, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    L = 150
    table = torch.tensor([[pages - 1, pages - 3, 1]], dtype=torch.int32)
    k, v = make((L, 2 * kv, d), 11), make((L, 2 * kv, d), 12)
    for j in range(3):
        n = min(64, L - 64 * j)
        kc[table[0, j].item(), :, :n] = k[64 * j:64 * j + n].transpose(0, 1).cuda()
        vc[table[0, j].item(), :, :n] = v[64 * j:64 * j + n].transpose(0, 1).cuda()
    q, lam = make((1, 2 * kv, 1, d), 13), weights(kv)
    o, lse = m.attn_diff_decode_bf16_paged(q.cuda(), kc, vc, lam.cuda(), table.cuda(), torch.tensor([L], dtype=torch.int32).cuda())
    want = expected(q[0], (k, v), lam, 1 / math.sqrt(d), 0)
    ref.check(o[0], want["o"], want["o_bound"], "o")


def test_streams_graphs_and_workspaces():
    """Two streams at once with a workspace each; a captured step follows lengths and lam; the workspace's
    contents do not matter."""
    m = fa()
    H, kv, d, nq = 8, 2, 64, 2
    lens = [3000, 77, 1200]
    kc, vc, table, _ = cache(lens, kv, d, 16, 188, 14)
    kc, vc, table = kc.cuda(), vc.cuda(), table.cuda()
    q, lam, n = make((3, 2 * H, nq, d), 15).cuda(), weights(H).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    size = m.attn_diff_decode_workspace_bytes(H, kv, nq, d)
    want = m.attn_diff_decode_bf16_paged(q, kc, vc, lam, table, n)
    other = m.attn_diff_decode_bf16_paged(q.flip(0), kc, vc, lam, table.flip(0).contiguous(), n.flip(0))
    ws = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        a = m.attn_diff_decode_bf16_paged(q, kc, vc, lam, table, n, workspace=ws[0], stream=streams[0])
        b = m.attn_diff_decode_bf16_paged(q.flip(0), kc, vc, lam, table.flip(0).contiguous(), n.flip(0), workspace=ws[1], stream=streams[1])
        got.append((a, b))
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(x, y) for x, y in zip(a, want))
        assert all(torch.equal(x, y) for x, y in zip(b, other))
    outs = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.attn_diff_decode_bf16_paged(q, kc, vc, lam, table, n, workspace=ws[0], o=outs[0], lse=outs[1])
    n -= 40
    lam *= 0.3
    graph.replay()
    torch.cuda.synchronize()
    want = m.attn_diff_decode_bf16_paged(q, kc, vc, lam, table, n)
    assert all(torch.equal(x, y) for x, y in zip(outs, want))


def test_refusals():
    m = fa()
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    q, lam = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda"), weights(2).cuda()
    table, n = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    good = dict(q=q, k_cache=kc, v_cache=kc, lam=lam, page_table=table, seq_lens=n)
    m.attn_diff_decode_bf16_paged(**good)
    for bad in (dict(q=q.half()), dict(lam=lam[:1].clone()), dict(seq_lens=n.long()), dict(page_table=table.long()),
                dict(k_cache=kc.float()), dict(o=torch.empty_like(q))):
        with pytest.raises(TypeError):
            m.attn_diff_decode_bf16_paged(**{**good, **bad})
    for bad in (dict(q=q[:, :3].contiguous()), dict(v_cache=kc[:, :1].contiguous())):
        with pytest.raises(ValueError):
            m.attn_diff_decode_bf16_paged(**{**good, **bad})
    small = torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    odd = torch.zeros(4, 6, 16, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(k_cache=small, v_cache=small), dict(k_cache=odd, v_cache=odd), dict(scale=0.0),
                dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")),
                dict(q=torch.zeros(1, 4, 9, 64, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(m.AttnError):
            m.attn_diff_decode_bf16_paged(**{**good, **bad})
