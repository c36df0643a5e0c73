"""The operators together: a training step of rotary positions and differential attention, and a serving
loop over a paged cache."""
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


def make(shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


def frequencies(half):
    return torch.pow(torch.tensor(10000.0), -torch.arange(half, dtype=torch.float32) / half)


def test_training_step():
    """Gradients of q and k through the rotation and the attention, against 64-bit differentiation.  The
    rotated rows are rounded once, forward and backward; each bound follows from that."""
    m = fa()
    B, H, Hkv, N, d = 2, 4, 2, 150, 64
    q, k, v, g = make((B, 2 * H, N, d), 1), make((B, 2 * Hkv, N, d), 2), make((B, Hkv, N, 2 * d), 3), make((B, H, N, 2 * d), 4)
    lam, freq = torch.tensor([0.2, 0.4, 0.6, 0.8]), frequencies(d // 2)
    pos = torch.arange(N, dtype=torch.int32).repeat(B, 1)
    args = (pos.cuda(), freq.cuda())
    qr, kr = m.attn_rope_bf16(q.cuda(), k.cuda(), *args)
    o, lse, o2 = m.attn_diff_fwd_bf16(qr, kr, v.cuda(), lam.cuda(), causal=True, save_o2=True)
    dqr, dkr, dv, dlam = m.attn_diff_bwd_bf16(qr, kr, v.cuda(), lam.cuda(), o, o2, g.cuda(), lse, causal=True)
    dq, dk = m.attn_rope_bf16(dqr, dkr, *args, inverse=True)
    assert m.attn_get_device_status() == m.ATTN_OK
    # the attention's gradients are the formula's on the rotated rows that the kernels saw; the last
    # rotation is then checked on its own inputs
    scale, ok = 1 / math.sqrt(d), ref.allowed(N, True, 0)
    for b in range(B):
        want, bound = ref.backward(qr[b].cpu(), kr[b].cpu(), v[b], lam, o[b].cpu(), o2[b].cpu(), g[b], lse[b].cpu(), scale, ok)
        for got, w, e, name in zip((dqr, dkr, dv), want, bound, ("dq", "dk", "dv")):
            ref.check(got[b], w, e, name)
    for got, x, name in ((dq, dqr, "dq"), (dk, dkr, "dk")):
        want = ref.rope(x.cpu(), pos[None], freq, inverse=True)
        ref.check(got, want, ref.rope_bound(x.cpu(), want, d // 2), name)
    for got, x, name in ((qr, q, "q"), (kr, k, "k")):
        want = ref.rope(x, pos[None], freq)
        ref.check(got, want, ref.rope_bound(x, want, d // 2), name)


def test_serving_loop_in_a_graph():
    """Prompts and then single tokens of three requests: plan, rotary positions, append and decoding, each step
    replayed from one captured graph, against attention over the rotated rows of each request."""
    m = fa()
    H, kv, d, page, pages, B, T = 4, 2, 64, 16, 40, 3, 24
    freq = frequencies(d // 2)
    kc, vc = (torch.full((pages, 2 * kv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((B, 10), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()
    left = torch.tensor([pages], dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    fused = torch.zeros(T, 2 * H + 4 * kv, d, dtype=torch.bfloat16, device="cuda")       # one projection's output
    lam, dfreq = torch.tensor([0.3, 0.1, 0.9, 0.5]).cuda(), freq.cuda()
    last = torch.zeros(B, dtype=torch.long, device="cuda")                              # row of each request's newest token
    state = {}

    def step():
        plan = m.attn_paged_plan(new, lens, table, free, left, page, T, seq_lens_out=lens, free_count_out=left)
        cu, slots, positions = plan[2], plan[3], plan[4]
        q, k = m.attn_rope_bf16(fused[:, :2 * H], fused[:, 2 * H:2 * H + 2 * kv], positions, dfreq)
        m.attn_cache_append_bf16(k, fused[:, 2 * H + 2 * kv:], kc, vc, slots)
        torch.sub(cu[1:], 1, out=last)
        newest = q[last].view(B, 2 * H, 1, d).contiguous()
        o, lse = m.attn_diff_decode_bf16_paged(newest, kc, vc, lam, table, lens)
        state.update(o=o, lse=lse, q=newest, slots=slots)

    counts = [[7, 24 - 7 - 5, 5]] + [[1, 1, 1]] * 20
    rows = [[] for _ in range(B)]
    graph = None
    for s, count in enumerate(counts):
        data = make((T, 2 * H + 4 * kv, d), 100 + s)
        fused.copy_(data)
        new.copy_(torch.tensor(count, dtype=torch.int32))
        if s == 1:                                    # the first step ran by itself; the rest replay
            keep = [t.clone() for t in (table, left, lens, kc, vc)]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for t, old in zip((table, left, lens, kc, vc), keep):
                t.copy_(old)
        if graph is None:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        at = 0
        for b, n in enumerate(count):
            rows[b].append(data[at:at + n])
            at += n
        if s % 7 and s != len(counts) - 1:
            continue
        for b in range(B):
            mine = torch.cat(rows[b])
            L = mine.shape[0]
            assert lens[b].item() == L
            pos = torch.arange(L, dtype=torch.int32)[None]
            # the kernels round the rotated rows once: what the cache and the step hold is that rounding
            qk = ref.rope(mine[:, :2 * H + 2 * kv].transpose(0, 1), pos, freq).bfloat16()
            k, v = qk[2 * H:], mine[:, 2 * H + 2 * kv:].reshape(L, kv, 2 * d).transpose(0, 1)
            got_q = state["q"][b, :, 0].cpu()
            assert ((got_q.double() - qk[:2 * H, -1].double()).abs() <= 2 * ref.HALF * qk[:2 * H, -1].double().abs() + 2.0 ** -17).all()
            # where the fp32 rotation lands on the other side of a rounding, one element of a key row differs by
            # a step: 2^-7 of |q k| < 16 over sqrt(64), so that key's weight by 2^-6 at most, times a share of the
            # spread of v that one key among many can have
            want = ref.forward(got_q[:, None], k, v, lam.cpu(), 1 / math.sqrt(d), torch.ones(1, L, dtype=torch.bool))
            ref.check(state["o"][b], want["o"], want["o_bound"] + 2.0 ** -6, f"step {s}, request {b}")
    assert m.attn_get_device_status() == m.ATTN_OK
