"""Cases and plain forms of rotary positions and of differential attention.

Four operators, each reached through functions of the package:

  rope         attn_rope_bf16: rotary positions on one or several axes, of queries and keys
               together; inverse=True is its backward pass
  diff_fwd     attn_diff_fwd_bf16, attn_diff_fwd_bf16_varlen: O = (P1 - lam P2) V, the
               difference of two softmax maps under a learned weight for each head
  diff_bwd     attn_diff_bwd_bf16, attn_diff_bwd_bf16_varlen: its gradients
  diff_decode  attn_diff_decode_bf16_paged: the newest tokens' attention over a paged cache

Head h of a differential attention owns the query heads 2h and 2h + 1 of width d and one value
head of width 2d; several heads may share a pair of key heads and its value head.

``run`` computes them in plain torch, or calls the package where ``own`` is true.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decoding step of 16 requests, far into long contexts: latency counts
        dict(name="rope_step_b16", op="rope", layout="packed", batch=1, rows=16, hq=32, hk=8, d=128, rot=128,
             axes=1, interleaved=False, inverse=False, far=131072, pad=0),
        # a prefill chunk of video tokens: three axes, columns of one projection's output, rows of padding
        dict(name="rope_video_prefill", op="rope", layout="packed", batch=1, rows=8191, hq=32, hk=8, d=128,
             rot=128, axes=3, interleaved=False, inverse=False, far=32768, pad=37),
        # gradients of a training batch's queries and keys: the inverse rotation, half of each row
        dict(name="rope_train_backward", op="rope", layout="batched", batch=4, rows=4096, hq=16, hk=16, d=64,
             rot=32, axes=1, interleaved=True, inverse=True, far=4096, pad=0),
        # a short evaluation batch without a mask
        dict(name="diff_fwd_short", op="diff_fwd", layout="batched", batch=2, heads=4, kv=4, d=64, n=257,
             lo=257, seqs=1, causal=False, window=0, save=False),
        # documents packed into one training batch, key heads shared
        dict(name="diff_fwd_packed", op="diff_fwd", layout="packed", batch=1, heads=8, kv=4, d=64, n=16384,
             lo=200, seqs=9, causal=True, window=0, save=True),
        # one long context at the wide head size
        dict(name="diff_fwd_long", op="diff_fwd", layout="batched", batch=1, heads=16, kv=4, d=128, n=16384,
             lo=16384, seqs=1, causal=True, window=0, save=False),
        # gradients of a short batch
        dict(name="diff_bwd_short", op="diff_bwd", layout="batched", batch=2, heads=4, kv=4, d=64, n=300,
             lo=300, seqs=1, causal=True, window=0),
        # gradients of a training batch
        dict(name="diff_bwd_train", op="diff_bwd", layout="batched", batch=4, heads=8, kv=8, d=64, n=4096,
             lo=4096, seqs=1, causal=True, window=0),
        # gradients over packed documents with a sliding window, shared key heads, the wide head size
        dict(name="diff_bwd_packed", op="diff_bwd", layout="packed", batch=1, heads=8, kv=2, d=128, n=8192,
             lo=333, seqs=5, causal=True, window=2047),
        # decoding 16 full contexts, every head its own keys
        dict(name="diff_decode_b16", op="diff_decode", batch=16, heads=8, kv=8, d=128, nq=1, page=64,
             len_lo=8192, len_hi=8192, window=0),
        # a ragged batch with shared key heads and two drafted tokens each
        dict(name="diff_decode_ragged", op="diff_decode", batch=48, heads=16, kv=4, d=64, nq=2, page=16,
             len_lo=37, len_hi=9000, window=0),
        # one long sequence: the split over keys and the joining
        dict(name="diff_decode_long", op="diff_decode", batch=1, heads=8, kv=2, d=128, nq=1, page=64,
             len_lo=131001, len_hi=131001, window=0),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over lo .. hi."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "diff_fwd", "diff_bwd", "diff_decode"])
    if op == "rope":
        d = rng.choice([64, 128, 256])
        hk = rng.choice([1, 2, 4, 8, 16])
        hq = hk * rng.choice([1, 2, 4]) if hk <= 8 else hk
        layout = rng.choice(["packed", "batched"])
        batch = 1 if layout == "packed" else _log(rng, 1, 8)
        most = min(16384, 8191 * 40 * 128 // (batch * (hq + hk) * d))
        rows = _log(rng, 1, most)
        rot = rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)])
        return dict(op=op, layout=layout, batch=batch, rows=rows, hq=hq, hk=hk, d=d, rot=rot,
                    axes=rng.choice([1, 1, 2, 3, 4]), interleaved=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, far=_log(rng, 64, 1 << 20),
                    pad=rng.randint(0, min(64, rows - 1)))
    d = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4]) if kv <= 4 else kv
    if op == "diff_decode":
        nq = rng.choice([1, 1, 2, 3, 4])
        batch = _log(rng, 1, 64)
        most = min(131072, 16 * 8192 * 8 * 128 // (batch * kv * d))
        hi = _log(rng, 1, most)
        return dict(op=op, batch=batch, heads=heads, kv=kv, d=d, nq=nq, page=rng.choice([16, 32, 64, 128]),
                    len_lo=rng.choice([0, 1, min(hi, 100), hi]), len_hi=hi,
                    window=rng.choice([0, 0, _log(rng, 16, 4096)]))
    causal = rng.random() < 0.7
    n = _log(rng, 1, 8192 if op == "diff_fwd" else 5000)
    layout = rng.choice(["packed", "batched"])
    window = rng.choice([0, 0, _log(rng, 1, 3000)])
    most = (64 << 20) if op == "diff_fwd" else (25 << 20)           # (query, key) pairs of all heads, d 64
    batch = max(1, min(_log(rng, 1, 4), 8 * most // (n * n * heads) * 64 // d))
    heads, kv = (heads, kv) if batch * n * n * heads * d // 64 <= 16 * most else (kv, kv)
    case = dict(op=op, layout=layout, batch=batch if layout == "batched" else 1, heads=heads, kv=kv, d=d, n=n,
                lo=n if layout == "batched" else rng.choice([0, 1, 1 + n // 50]),
                seqs=1 if layout == "batched" else rng.randint(1, 12), causal=causal, window=window)
    if op == "diff_fwd":
        case["save"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _spans(case, seed):
    """First tokens of the sequences of a packed case, and its end."""
    rng = random.Random(seed * 7919 + 13)
    cuts = sorted(rng.randint(0, case["n"]) for _ in range(case["seqs"] - 1))
    cu = [0] + cuts + [case["n"]]
    for i in range(1, len(cu) - 1):                     # at least `lo` tokens where there is room
        cu[i] = min(max(cu[i], cu[i - 1] + case["lo"]), case["n"])
    return cu


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    state = dict(case=case)
    d = case["d"]
    if case["op"] == "rope":
        axes, half, batch, rows = case["axes"], case["rot"] // 2, case["batch"], case["rows"]
        exponent = torch.arange(half, device="cuda", dtype=torch.float32) / half
        state["inv_freq"] = torch.pow(torch.tensor(10000.0, device="cuda"), -exponent)
        # a run of pairs for each axis, the first the shortest, as for time, height and width
        state["axis"] = None
        if axes > 1:
            bounds = [half * i // (axes + 1) for i in range(1, axes)]
            bounds = [max(1, b) if half >= axes else b for b in bounds]
            ax = torch.zeros(half, dtype=torch.int32, device="cuda")
            for b in bounds:
                ax[b:] += 1
            state["axis"] = ax
        shape = (batch, rows) if case["layout"] == "batched" else (rows,)
        start = int(torch.randint(0, max(1, case["far"] - rows), (1,), generator=gen, device="cuda"))
        pos = [torch.arange(start, start + rows, device="cuda").expand(shape)]
        for i in range(1, axes):                        # places within a frame
            pos.append(torch.randint(0, 64 * i, shape, generator=gen, device="cuda"))
        pos = torch.stack(pos).to(torch.int32)
        if case["pad"]:
            pos[..., rows - case["pad"]:] = -1
        state["positions"] = pos if axes > 1 else pos[0].contiguous()
        if case["layout"] == "batched":
            state["q"] = _randn(gen, batch, case["hq"], rows, d).bfloat16()
            state["k"] = _randn(gen, batch, case["hk"], rows, d).bfloat16()
        else:                                           # columns of one projection
            both = _randn(gen, rows, case["hq"] + 2 * case["hk"], d).bfloat16()
            state["q"], state["k"] = both[:, :case["hq"]], both[:, case["hq"]:case["hq"] + case["hk"]]
        return state

    H, Hkv = case["heads"], case["kv"]
    state["lam"] = 0.2 + 0.6 * torch.rand(H, generator=gen, device="cuda")
    if case["op"] == "diff_decode":
        B, page, nq = case["batch"], case["page"], case["nq"]
        lens = torch.randint(case["len_lo"], case["len_hi"] + 1, (B,), generator=gen, device="cuda")
        lens[0] = case["len_hi"]
        width = (case["len_hi"] + page - 1) // page
        pages = B * width + 3
        order = torch.randperm(pages, generator=gen, device="cuda")[: B * width]
        state["table"] = order.view(B, width).to(torch.int32).contiguous()
        state["lens"] = lens.to(torch.int32)
        state["kc"] = torch.empty(pages, 2 * Hkv, page, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        state["vc"] = torch.empty(pages, 2 * Hkv, page, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        state["q"] = _randn(gen, B, 2 * H, nq, d).bfloat16()
        return state

    if case["layout"] == "batched":
        lead = lambda heads: (case["batch"], heads, case["n"])
    else:
        lead = lambda heads: (case["n"], heads)
        state["spans"] = _spans(case, seed)
        state["cu"] = torch.tensor(state["spans"], dtype=torch.int32, device="cuda")
        state["longest"] = max(b - a for a, b in zip(state["spans"], state["spans"][1:]))
    state["q"] = _randn(gen, *lead(2 * H), d).bfloat16()
    state["k"] = _randn(gen, *lead(2 * Hkv), d).bfloat16()
    state["v"] = _randn(gen, *lead(Hkv), 2 * d).bfloat16()
    if case["op"] == "diff_bwd":                        # what the forward pass left, and the gradient from above
        state["dout"] = _randn(gen, *lead(H), 2 * d).bfloat16()
        state["o"], state["lse"], state["o2"] = _plain_fwd(state, True)
    return state


# ------------------------------------------------------------------ plain forms
def _plain_rope(state):
    case = state["case"]
    pos, half = state["positions"], case["rot"] // 2
    if case["axes"] == 1:
        pos = pos[None]
    axis = state["axis"].long() if state["axis"] is not None else torch.zeros(half, dtype=torch.long, device="cuda")
    angle = pos[axis].double() * state["inv_freq"].double().view(half, *([1] * (pos.dim() - 1)))
    angle = torch.where(pos[0] < 0, 0.0, angle).movedim(0, -1)
    if case["inverse"]:
        angle = -angle
    head = 1 if case["layout"] == "batched" else -2
    cos, sin = angle.cos().float().unsqueeze(head), angle.sin().float().unsqueeze(head)

    def turn(x):
        x = x.float()
        y = x.clone()
        if case["interleaved"]:
            a, b = slice(0, case["rot"], 2), slice(1, case["rot"], 2)
        else:
            a, b = slice(0, half), slice(half, case["rot"])
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., a] * sin + x[..., b] * cos
        return y.bfloat16()

    return turn(state["q"]), turn(state["k"])


def _problems(state):
    """(heads of q, k, v and further tensors as [heads, rows, width]; where results go) of each sequence."""
    case = state["case"]
    if case["layout"] == "batched":
        return [lambda t, b=b: t[b] for b in range(case["batch"])]
    return [lambda t, a=a, b=b: t[a:b].transpose(0, 1) for a, b in zip(state["spans"], state["spans"][1:]) if b > a]


def _lse_view(state, lse):
    case = state["case"]
    if case["layout"] == "batched":
        return [lse[b] for b in range(case["batch"])]
    return [lse[:, a:b] for a, b in zip(state["spans"], state["spans"][1:]) if b > a]


def _allowed(case, r0, r1, n):
    i = torch.arange(r0, r1, device="cuda")[:, None]
    j = torch.arange(n, device="cuda")[None]
    ok = torch.ones(r1 - r0, n, dtype=torch.bool, device="cuda")
    if case["causal"]:
        ok &= j <= i
    if case["window"] > 0:
        ok &= j >= i - case["window"]
        if not case["causal"]:
            ok &= j <= i + case["window"]
    return ok


def _plain_fwd(state, save):
    case = state["case"]
    d, H, G = case["d"], case["heads"], case["heads"] // case["kv"]
    q, k, v, lam = state["q"], state["k"], state["v"], state["lam"]
    shape = (case["batch"], H, case["n"], 2 * d) if case["layout"] == "batched" else (case["n"], H, 2 * d)
    o = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    o2 = torch.zeros_like(o) if save else None
    lse = torch.zeros((case["batch"], 2 * H, case["n"]) if case["layout"] == "batched" else (2 * H, case["n"]),
                      device="cuda")
    scale = 1.0 / math.sqrt(d)
    for part, ls in zip(_problems(state), _lse_view(state, lse)):
        pq, pk, pv, po = part(q), part(k), part(v), part(o)
        po2 = part(o2) if save else None
        n = pq.shape[1]
        step = max(1, min(n, (1 << 26) // n))
        for r0 in range(0, n, step):
            r1 = min(n, r0 + step)
            ok = _allowed(case, r0, r1, n)
            for h in range(H):
                outs = []
                for m in range(2):
                    s = pq[2 * h + m, r0:r1].float() @ pk[2 * (h // G) + m].float().t() * scale
                    s = s.masked_fill(~ok, -math.inf)
                    top = s.amax(1, keepdim=True)
                    p = torch.exp(s - top)
                    total = p.sum(1, keepdim=True)
                    ls[2 * h + m, r0:r1] = (top + torch.log(total))[:, 0]
                    outs.append((p @ pv[h // G].float()) / total)
                po[h, r0:r1] = (outs[0] - lam[h] * outs[1]).bfloat16()
                if save:
                    po2[h, r0:r1] = outs[1].bfloat16()
    return o, lse, o2


def _plain_bwd(state):
    case = state["case"]
    d, H, G = case["d"], case["heads"], case["heads"] // case["kv"]
    lam = state["lam"]
    names = ("q", "k", "v", "o", "o2", "dout")
    dq, dk, dv = (torch.zeros(state[x].shape, device="cuda") for x in ("q", "k", "v"))
    dlam = torch.zeros(H, dtype=torch.float64, device="cuda")
    scale = 1.0 / math.sqrt(d)
    for part, ls in zip(_problems(state), _lse_view(state, state["lse"])):
        pq, pk, pv, po, po2, pg = (part(state[x]) for x in names)
        gq, gk, gv = part(dq), part(dk), part(dv)
        n = pq.shape[1]
        step = max(1, min(n, (1 << 26) // n))
        for r0 in range(0, n, step):
            r1 = min(n, r0 + step)
            ok = _allowed(case, r0, r1, n)
            for h in range(H):
                g, out2 = pg[h, r0:r1].float(), po2[h, r0:r1].float()
                out1 = po[h, r0:r1].float() + lam[h] * out2
                below = g @ pv[h // G].float().t()
                dots = ((g * out1).sum(1, keepdim=True), (g * out2).sum(1, keepdim=True))
                dlam[h] -= dots[1].double().sum()
                mix = 0.0
                for m in range(2):
                    qm, km = pq[2 * h + m, r0:r1].float(), pk[2 * (h // G) + m].float()
                    p = torch.exp(qm @ km.t() * scale - ls[2 * h + m, r0:r1, None]).masked_fill(~ok, 0.0)
                    if m == 1:
                        p = -lam[h] * p
                    mix = mix + p
                    ds = p * (below - dots[m])
                    gq[2 * h + m, r0:r1] = ds @ km * scale
                    gk[2 * (h // G) + m] += ds.t() @ qm * scale
                gv[h // G] += mix.t() @ g
    return dq.bfloat16(), dk.bfloat16(), dv.bfloat16(), dlam.float()


def _cached(state, b, L):
    """Keys [2 Hkv, L, d] and values [Hkv, L, 2d] of sequence b."""
    case = state["case"]
    pages = state["table"][b, : (L + case["page"] - 1) // case["page"]].long()
    k = state["kc"][pages].transpose(0, 1).reshape(2 * case["kv"], -1, case["d"])[:, :L]
    v = state["vc"][pages].transpose(0, 1).reshape(2 * case["kv"], -1, case["d"])[:, :L]
    v = v.reshape(case["kv"], 2, L, case["d"]).transpose(1, 2).reshape(case["kv"], L, 2 * case["d"])
    return k, v


def _plain_decode(state):
    case = state["case"]
    B, H, Hkv, d, nq = case["batch"], case["heads"], case["kv"], case["d"], case["nq"]
    G = H // Hkv
    o = torch.zeros(B, H, nq, 2 * d, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, 2 * H, nq), -math.inf, device="cuda")
    scale = 1.0 / math.sqrt(d)
    for b, L in enumerate(state["lens"].tolist()):
        if L == 0:
            continue
        k, v = _cached(state, b, L)
        at = torch.arange(L - nq, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None]
        ok = j <= at
        if case["window"] > 0:
            ok &= j >= at - case["window"]
        q = state["q"][b].view(Hkv, G, 2, nq, d).transpose(1, 2).reshape(2 * Hkv, G * nq, d).float()
        s = (q @ k.float().transpose(1, 2) * scale).masked_fill(~ok.repeat(G, 1), -math.inf)
        top = s.amax(2, keepdim=True)
        p = torch.exp(s - top.masked_fill(top == -math.inf, 0.0))
        total = p.sum(2, keepdim=True)
        p = (p / total.masked_fill(total == 0.0, 1.0)).view(Hkv, 2, G * nq, L)
        out = p @ v.float()[:, None]
        out = out.view(Hkv, 2, G, nq, 2 * d).transpose(1, 2).reshape(H, 2, nq, 2 * d)
        o[b] = (out[:, 0] - state["lam"][:, None, None] * out[:, 1]).bfloat16()
        ls = (top + torch.log(total)).view(Hkv, 2, G, nq).transpose(1, 2).reshape(2 * H, nq)
        lse[b] = ls
    return o, lse


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "rope":
            return _plain_rope(state)
        if op == "diff_fwd":
            out = _plain_fwd(state, case["save"])
            return out if case["save"] else out[:2]
        return _plain_bwd(state) if op == "diff_bwd" else _plain_decode(state)

    import exact_attention_55_gb300 as fa
    if op == "rope":
        return fa.attn_rope_bf16(state["q"], state["k"], state["positions"], state["inv_freq"], axis=state["axis"],
                                 interleaved=case["interleaved"], inverse=case["inverse"])
    if op == "diff_decode":
        return fa.attn_diff_decode_bf16_paged(state["q"], state["kc"], state["vc"], state["lam"], state["table"],
                                              state["lens"], window=case["window"])
    mask = dict(causal=case["causal"], window=case["window"])
    if op == "diff_fwd":
        if case["layout"] == "batched":
            out = fa.attn_diff_fwd_bf16(state["q"], state["k"], state["v"], state["lam"], save_o2=case["save"], **mask)
        else:
            out = fa.attn_diff_fwd_bf16_varlen(state["q"], state["k"], state["v"], state["lam"], state["cu"],
                                               state["longest"], save_o2=case["save"], **mask)
        return out if case["save"] else out[:2]
    saved = [state[x] for x in ("q", "k", "v", "lam", "o", "o2", "dout", "lse")]
    if case["layout"] == "batched":
        return fa.attn_diff_bwd_bf16(*saved, **mask)
    return fa.attn_diff_bwd_bf16_varlen(*saved, state["cu"], state["longest"], **mask)


# ------------------------------------------------------------------ work
def _pairs(n, causal, window):
    """Allowed (query, key) pairs of a sequence of n tokens."""
    w = window if window > 0 else n
    left = sum(min(i, w) + 1 for i in range(n)) if w < n else n * (n + 1) // 2
    return left if causal else 2 * left - n


def work(case):
    d = case["d"]
    if case["op"] == "rope":
        rows = case["batch"] * case["rows"]
        elements = rows * (case["hq"] + case["hk"]) * d
        return {"bytes": 4 * elements + 4 * rows * case["axes"] + 4 * case["rot"],
                "flops": 3 * rows * (case["hq"] + case["hk"]) * case["rot"]}
    H, Hkv = case["heads"], case["kv"]
    if case["op"] == "diff_decode":
        B, nq = case["batch"], case["nq"]
        keys = B * (case["len_lo"] + case["len_hi"]) / 2                # the lengths' mean
        seen = min(keys, B * (case["window"] + nq)) if case["window"] else keys
        return {"bytes": int(seen * Hkv * 8 * d + B * nq * H * (8 * d + 8) + B * 4),
                "flops": int(seen * nq * H * 8 * d)}
    if case["layout"] == "batched":
        tokens = case["batch"] * case["n"]
        pairs = case["batch"] * _pairs(case["n"], case["causal"], case["window"])
    else:                                                              # equal documents
        tokens = case["n"]
        pairs = case["seqs"] * _pairs(max(1, case["n"] // case["seqs"]), case["causal"], case["window"])
    qb, kb, ob = tokens * 2 * H * d * 2, tokens * 2 * Hkv * d * 2, tokens * H * 2 * d * 2
    lse = tokens * 2 * H * 4
    if case["op"] == "diff_fwd":
        return {"bytes": qb + 2 * kb + ob * (2 if case["save"] else 1) + lse, "flops": pairs * H * 8 * d}
    return {"bytes": 2 * (qb + 2 * kb) + 3 * ob + lse + 4 * H, "flops": pairs * H * 20 * d}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """Results from the definitions in 64 bits."""
    state = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(state)
    d, H = case["d"], case["heads"]
    G = H // case["kv"]
    lam = state["lam"].double()
    if case["op"] == "diff_decode":
        o = torch.zeros(case["batch"], H, case["nq"], 2 * d, dtype=torch.float64, device="cuda")
        lse = torch.full((case["batch"], 2 * H, case["nq"]), -math.inf, dtype=torch.float64, device="cuda")
        for b, L in enumerate(state["lens"].tolist()):
            if L == 0:
                continue
            k, v = _cached(state, b, L)
            for i in range(case["nq"]):
                last = L - case["nq"] + i
                first = max(0, last - case["window"]) if case["window"] else 0
                if last < 0:
                    continue
                kk, vv = k[:, first:last + 1].double(), v[:, first:last + 1].double()
                q = state["q"][b, :, i].double().view(H, 2, d)
                kh = kk.view(case["kv"], 2, -1, d).repeat_interleave(G, 0)
                s = torch.einsum("hmd,hmnd->hmn", q, kh) / math.sqrt(d)
                lse[b, :, i] = torch.logsumexp(s, 2).view(2 * H)
                p = torch.softmax(s, 2)
                o[b, :, i] = torch.einsum("hn,hnd->hd", p[:, 0] - lam[:, None] * p[:, 1],
                                          vv.repeat_interleave(G, 0))
        return o, lse
    if case["op"] == "diff_fwd":
        return _exact_fwd(state, lam, G)
    return _exact_bwd(state, lam, G)


def _exact_rope(state):
    case = state["case"]
    half = case["rot"] // 2
    pos = state["positions"].double().view(case["axes"], -1)
    freq = state["inv_freq"].double()
    angle = torch.zeros(pos.shape[1], half, dtype=torch.float64, device="cuda")
    for i in range(case["axes"]):
        mine = state["axis"] == i if state["axis"] is not None else torch.ones(half, dtype=torch.bool, device="cuda")
        angle += torch.outer(pos[i], torch.where(mine, freq, 0.0))
    angle[pos[0] < 0] = 0.0
    turn = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)
    if case["layout"] == "batched":
        turn = turn.view(case["batch"], 1, case["rows"], half)
    else:
        turn = turn.view(case["rows"], 1, half)
    out = []
    for x in (state["q"].double(), state["k"].double()):
        r, rest = x[..., :case["rot"]], x[..., case["rot"]:]
        if case["interleaved"]:
            z = torch.complex(r[..., 0::2].contiguous(), r[..., 1::2].contiguous()) * turn
            y = torch.stack((z.real, z.imag), -1).flatten(-2)
        else:
            z = torch.complex(r[..., :half].contiguous(), r[..., half:].contiguous()) * turn
            y = torch.cat((z.real, z.imag), -1)
        out.append(torch.cat((y, rest), -1))
    return tuple(out)


def _blocks(case, n):
    """(first row, last row, first key, last key) of blocks of queries with the keys that they may see."""
    step = max(64, min(n, 2048, (1 << 24) // n))
    for r0 in range(0, n, step):
        r1 = min(n, r0 + step)
        k0 = max(0, r0 - case["window"]) if case["window"] > 0 else 0
        k1 = r1 if case["causal"] else min(n, r1 + case["window"]) if case["window"] > 0 else n
        yield r0, r1, k0, k1


def _exact_fwd(state, lam, G):
    case = state["case"]
    d, H = case["d"], case["heads"]
    batched = case["layout"] == "batched"
    o = torch.zeros((case["batch"], H, case["n"], 2 * d) if batched else (case["n"], H, 2 * d),
                    dtype=torch.float64, device="cuda")
    o2 = torch.zeros_like(o)
    lse = torch.zeros((case["batch"], 2 * H, case["n"]) if batched else (2 * H, case["n"]),
                      dtype=torch.float64, device="cuda")
    for part, ls in zip(_problems(state), _lse_view(state, lse)):
        q, k, v, po, po2 = (part(t) for t in (state["q"], state["k"], state["v"], o, o2))
        for h in range(H):
            g = h // G
            vv, kk = v[g].double(), [k[2 * g + m].double() for m in range(2)]
            for r0, r1, k0, k1 in _blocks(case, q.shape[1]):
                hide = ~_allowed(case, r0, r1, k1)[:, k0:]
                maps = []
                for m in range(2):
                    s = (q[2 * h + m, r0:r1].double() @ kk[m][k0:k1].t()).div_(math.sqrt(d))
                    s.masked_fill_(hide, -math.inf)
                    ls[2 * h + m, r0:r1] = torch.logsumexp(s, 1)
                    maps.append(torch.softmax(s, 1))
                po2[h, r0:r1] = maps[1] @ vv[k0:k1]
                po[h, r0:r1] = (maps[0] - lam[h] * maps[1]) @ vv[k0:k1]
    return (o, lse, o2) if case["save"] else (o, lse)


def _exact_bwd(state, lam, G):
    """The gradients' formulas on what the forward pass saved."""
    case = state["case"]
    d, H = case["d"], case["heads"]
    c = 1.0 / math.sqrt(d)
    dq, dk, dv = (torch.zeros(state[x].shape, dtype=torch.float64, device="cuda") for x in ("q", "k", "v"))
    dlam = torch.zeros(H, dtype=torch.float64, device="cuda")
    for part, ls in zip(_problems(state), _lse_view(state, state["lse"])):
        q, k, v, o, o2, do = (part(state[x]) for x in ("q", "k", "v", "o", "o2", "dout"))
        gq, gk, gv = part(dq), part(dk), part(dv)
        for h in range(H):
            g = h // G
            vv, kk = v[g].double(), [k[2 * g + m].double() for m in range(2)]
            second = (do[h].double() * o2[h].double()).sum(1)
            first = (do[h].double() * o[h].double()).sum(1) + lam[h] * second
            dlam[h] -= second.sum()
            for r0, r1, k0, k1 in _blocks(case, q.shape[1]):
                see = _allowed(case, r0, r1, k1)[:, k0:]
                up = do[h, r0:r1].double()
                dp = up @ vv[k0:k1].t()
                w = []
                for m in range(2):
                    x = (q[2 * h + m, r0:r1].double() @ kk[m][k0:k1].t()).mul_(c) - ls[2 * h + m, r0:r1, None].double()
                    w.append(torch.where(see, x.exp_(), 0.0))
                w[1] *= -lam[h]
                gv[g, k0:k1] += (w[0] + w[1]).t() @ up
                for m, dot in enumerate((first, second)):
                    ds = w[m].mul_(dp - dot[r0:r1, None])
                    gq[2 * h + m, r0:r1] = c * (ds @ kk[m][k0:k1])
                    gk[2 * g + m, k0:k1] += c * (ds.t() @ q[2 * h + m, r0:r1].double())
    return dq, dk, dv, dlam
