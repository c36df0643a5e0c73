"""Cases and plain forms of the operators that serve from a paged key/value cache.

Four operators, each reached through one function of the package:

  plan         attn_paged_plan: pages, slots, positions and lengths of one serving step, from
               the lengths of the requests
  append_bf16  attn_cache_append_bf16: new keys and values into a bf16 cache
  append_fp8   attn_cache_append_fp8: the same into an 8-bit cache with one scale for each
               block of tokens and head, which grows with the block
  decode_fp8   attn_decode_fp8_paged: attention of the newest tokens over the 8-bit cache

``run`` computes them in plain torch, or calls the package where ``own`` is true.
"""
import json
import math
import random

import torch

own = False

FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0),
       "e4m3_pow2": (torch.float8_e4m3fn, 448.0)}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of a small batch: every request gets one token, a few get a page
        dict(name="plan_step_b16", op="plan", batch=16, page=64, len_lo=1, len_hi=8000, max_len=8192,
             chunked=0.0, new_hi=1, pad=0, short=False),
        # a step that mixes decoding with chunked prefill, padded to a captured token count
        dict(name="plan_mixed_b1024", op="plan", batch=1024, page=16, len_lo=0, len_hi=8192, max_len=16384,
             chunked=0.05, new_hi=1024, pad=333, short=True),
        # the same step's keys and values into a bf16 cache: 16 rows of 16 heads
        dict(name="append_bf16_step_b16", op="append_bf16", batch=16, heads=16, d=128, page=64, len_lo=100,
             len_hi=8000, new_lo=1, new_hi=1, pad=0, fused=False),
        # a prefill chunk whose keys and values are columns of one projection's output
        dict(name="append_bf16_prefill", op="append_bf16", batch=5, heads=16, d=128, page=64, len_lo=0,
             len_hi=3001, new_lo=1500, new_hi=4500, pad=17, fused=True),
        # one decoding step into the 8-bit cache, padded to a captured batch of 64
        dict(name="append_fp8_step_b61", op="append_fp8", batch=61, heads=8, d=128, page=64, block=64, fmt="e4m3",
             len_lo=30, len_hi=2000, new_lo=1, new_hi=1, pad=3, fused=True),
        # short prompts that start and end inside blocks, small pages, power-of-two scales
        dict(name="append_fp8_ragged_d64", op="append_fp8", batch=37, heads=6, d=64, page=16, block=16,
             fmt="e4m3_pow2", len_lo=0, len_hi=50, new_lo=1, new_hi=70, pad=0, fused=False),
        # a large prefill into 128-token blocks
        dict(name="append_fp8_prefill", op="append_fp8", batch=8, heads=16, d=128, page=128, block=128, fmt="e4m3",
             len_lo=0, len_hi=1000, new_lo=3500, new_hi=4500, pad=0, fused=True),
        # one short conversation: latency
        dict(name="decode_b1_short", op="decode_fp8", batch=1, heads=8, kv_heads=8, nq=1, d=64, page=16, block=16,
             fmt="e4m3", len_lo=300, len_hi=300, window=0),
        # the repository's decoding workload with the cache in 8 bits
        dict(name="decode_b16_h16_l8192", op="decode_fp8", batch=16, heads=16, kv_heads=16, nq=1, d=128, page=64,
             block=64, fmt="e4m3", len_lo=8192, len_hi=8192, window=0),
        # a serving batch of uneven lengths whose query heads share key heads four to one
        dict(name="decode_gqa_ragged_b48", op="decode_fp8", batch=48, heads=32, kv_heads=8, nq=1, d=128, page=64,
             block=64, fmt="e4m3_pow2", len_lo=37, len_hi=9000, window=0),
        # several new tokens a request (speculative decoding) under a sliding window
        dict(name="decode_spec_window", op="decode_fp8", batch=8, heads=32, kv_heads=4, nq=4, d=128, page=32,
             block=32, fmt="e5m2", len_lo=3000, len_hi=12000, window=4095),
        # one very long document with wide heads
        dict(name="decode_long_d256", op="decode_fp8", batch=1, heads=16, kv_heads=2, nq=1, d=256, page=128,
             block=128, fmt="e4m3", len_lo=131001, len_hi=131001, window=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "append_bf16", "append_fp8", "append_fp8", "decode_fp8", "decode_fp8", "decode_fp8"])
    page = rng.choice([16, 32, 64, 128, 256])
    d = rng.choice([64, 128, 128, 256])
    if op == "plan":
        hi = _log_int(rng, 1, 8192)
        return dict(op=op, batch=_log_int(rng, 1, 1024), page=page, len_lo=rng.randint(0, hi), len_hi=hi,
                    max_len=16384, chunked=rng.choice([0.0, 0.03, 0.05]), new_hi=rng.choice([1, 7, 300, 1000]),
                    pad=rng.choice([0, 1, 50, 301]), short=rng.random() < 0.3)
    fmt = rng.choice(list(FP8))
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= page])
    if op != "decode_fp8":
        heads, batch = rng.choice([1, 2, 3, 4, 8, 16]), _log_int(rng, 1, 64)
        most = max(1, min(4500, 24000 // batch, 24000 * 2048 // (batch * heads * d)))
        new_hi = rng.choice([1, 1, 5, _log_int(rng, 1, most)])
        c = dict(op=op, batch=batch, heads=heads, d=d, page=page, len_lo=0, len_hi=_log_int(rng, 1, 1500),
                 new_lo=rng.randint(1, new_hi), new_hi=new_hi, pad=rng.choice([0, 0, 3, 40]), fused=rng.random() < 0.5)
        if op == "append_fp8":
            c.update(block=block, fmt=fmt)
        return c
    kv = rng.choice([1, 2, 3, 4, 8, 16])
    group, nq = rng.choice([1, 1, 2, 4, 5, 8, 16]), rng.choice([1, 1, 1, 2, 3, 4, 8])
    batch = _log_int(rng, 1, 64)
    hi = _log_int(rng, 1, max(1, min(131072, 100_000_000 // (batch * kv * d))))
    return dict(op=op, batch=batch, heads=kv * group, kv_heads=kv, nq=nq, d=d, page=page, block=block, fmt=fmt,
                len_lo=max(1, hi // rng.choice([1, 2, 50])), len_hi=hi,
                window=0 if rng.random() < 0.7 else _log_int(rng, 1, 4096))


# ------------------------------------------------------------------ lengths: of the case, not of the seed
def _rng(case):
    return random.Random(json.dumps({k: v for k, v in case.items() if k != "name"}, sort_keys=True))


def _decode_lens(case):
    r = _rng(case)
    return [_log_int(r, case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]


def _append_lens(case):
    r = _rng(case)
    return [(r.randint(case["len_lo"], case["len_hi"]), r.randint(case["new_lo"], case["new_hi"]))
            for _ in range(case["batch"])]


def _plan_lens(case):
    r, out = _rng(case), []
    for b in range(case["batch"]):
        new = 1 if r.random() >= case["chunked"] else r.randint(0, case["new_hi"])
        out.append((r.randint(case["len_lo"], case["len_hi"]), new))
    return out


def _pages(n, page):
    return -(-n // page)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"op": case["op"], "page": case["page"]}
    page = case["page"]

    def ints(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device="cuda")

    def codes(shape, fmt):
        # codes of a block whose largest value took the format's largest code, as for normal data
        dtype, top = FP8[fmt]
        x = torch.empty(shape, dtype=torch.uint8, device="cuda")
        flat = x.reshape(-1)
        for i in range(0, flat.numel(), 1 << 28):
            n = min(1 << 28, flat.numel() - i)
            r = torch.randn(n, generator=g, device="cuda").mul_(top / 3.6).clamp_(-top, top)
            flat[i:i + n] = r.to(dtype).view(torch.uint8)
        return x

    def scales(pages, heads, nblk, fmt):
        top = FP8[fmt][1]
        x = (2.7 + 1.5 * torch.rand((pages, heads, nblk), generator=g, device="cuda")) / top
        return torch.exp2(torch.ceil(torch.log2(x))) if fmt == "e4m3_pow2" else x

    def table_of(counts, width, total):
        perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        # an unused entry names no page
        table = torch.full((len(counts), width), -1, dtype=torch.int32, device="cuda")
        start = torch.cumsum(ints([0] + counts[:-1], torch.int64), 0)
        col = torch.arange(width, device="cuda")
        used = col[None] < ints(counts, torch.int64)[:, None]
        table[used] = perm[(start[:, None] + col[None])[used]]
        return table, perm

    if case["op"] == "plan":
        lens = _plan_lens(case)
        old = [_pages(n, page) for n, _ in lens]
        want = [_pages(n + m, page) for n, m in lens]
        need, width = sum(want) - sum(old), case["max_len"] // page
        free = max(1, need // 2 if case["short"] else need + 7)   # short: the pool runs out on the way
        s["page_table"], perm = table_of(old, width, sum(old) + free)
        s.update(num_tokens=sum(m for _, m in lens) + case["pad"], new_lens=ints([m for _, m in lens]),
                 seq_lens=ints([n for n, _ in lens]), free_pages=perm[sum(old):].contiguous(), free_count=ints([free]))
        return s
    d = case["d"]
    if case["op"] == "decode_fp8":
        lens, heads, fmt = _decode_lens(case), case["kv_heads"], case["fmt"]
        counts = [_pages(n, page) for n in lens]
        total = sum(counts) + 3
        s["page_table"], _ = table_of(counts, max(counts), total)
        s["q"] = torch.randn((case["batch"], case["heads"], case["nq"], d), generator=g, device="cuda").to(torch.bfloat16)
        for n in ("k", "v"):
            s[n + "_cache"] = codes((total, heads, page, d), fmt)
            s[n + "_scales"] = scales(total, heads, page // case["block"], fmt)
        s.update(seq_lens=ints(lens), window=case["window"], fmt=fmt, scale=1.0 / math.sqrt(d))
        return s
    lens, heads = _append_lens(case), case["heads"]
    counts = [_pages(n + m, page) for n, m in lens]
    total = sum(counts) + 3
    table, _ = table_of(counts, max(counts), total)
    new = ints([m for _, m in lens], torch.int64)
    row = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), new)
    first = torch.cumsum(new, 0) - new
    pos = torch.arange(int(row.numel()), device="cuda") - first[row] + ints([n for n, _ in lens], torch.int64)[row]
    slot = table[row, pos // page].long() * page + pos % page
    # padded rows carry no slot
    s["slot_map"] = torch.cat([slot, torch.full((case["pad"],), -1, dtype=torch.int64, device="cuda")])
    T = s["slot_map"].numel()
    # keys and values after a projection: normal, a few large entries; `fused`: columns of [q, k, v]
    x = torch.randn((T, 2 * heads * d), generator=g, device="cuda")
    x *= torch.where(torch.rand((T, 2 * heads * d), generator=g, device="cuda") < 1e-3, 8.0, 1.0)
    x = x.to(torch.bfloat16)
    if case["fused"]:
        x = torch.cat([torch.zeros((T, 2 * heads * d), dtype=torch.bfloat16, device="cuda"), x], 1)[:, 2 * heads * d:]
        s["k"], s["v"] = (x[:, i * heads * d:(i + 1) * heads * d].unflatten(1, (heads, d)) for i in (0, 1))
    else:
        s["k"], s["v"] = (x[:, i * heads * d:(i + 1) * heads * d].reshape(T, heads, d).contiguous() for i in (0, 1))
    for n in ("k", "v"):
        if case["op"] == "append_fp8":
            s["fmt"] = case["fmt"]
            s[n + "_cache"] = codes((total, heads, page, d), case["fmt"])
            s[n + "_scales"] = scales(total, heads, page // case["block"], case["fmt"])
        else:
            s[n + "_cache"] = torch.randn((total, heads, page, d), generator=g, device="cuda").to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        import exact_attention_55_gb300 as fa
        if s["op"] == "plan":
            out = fa.attn_paged_plan(s["new_lens"], s["seq_lens"], s["page_table"], s["free_pages"], s["free_count"],
                                     s["page"], s["num_tokens"])
            return dict(zip(("seq_lens", "free_count", "cu_new", "slot_map", "positions", "served"), out),
                        page_table=s["page_table"])
        if s["op"] == "append_bf16":
            k, v = fa.attn_cache_append_bf16(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slot_map"])
            return {"k": k, "v": v}
        if s["op"] == "append_fp8":
            fa.attn_cache_append_fp8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                     s["slot_map"], fmt=s["fmt"])
            return _as_values(s)
        o, lse = fa.attn_decode_fp8_paged(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                          s["page_table"], s["seq_lens"], fmt=s["fmt"], scale=s["scale"],
                                          window=s["window"])
        return {"o": o, "lse": lse}
    return {"plan": _plan, "append_bf16": _append_bf16, "append_fp8": _append_fp8, "decode_fp8": _decode}[s["op"]](s)


def _as_values(s):
    dtype = FP8[s["fmt"]][0]
    return {"k": s["k_cache"].view(dtype), "v": s["v_cache"].view(dtype), "k_scales": s["k_scales"],
            "v_scales": s["v_scales"]}


def _plan(s):
    page, T, table = s["page"], s["num_tokens"], s["page_table"]
    B, width = table.shape
    n = s["new_lens"].long().clamp(min=0)
    L = s["seq_lens"].long().clamp(0, width * page)
    ends = torch.cumsum(n, 0)
    fits = (L + n <= width * page) & (ends <= T)
    old = (L + page - 1) // page
    need = torch.where(fits, (L + n + page - 1) // page - old, 0)
    base = torch.cumsum(need, 0) - need
    free = s["free_count"].long().clamp(0, s["free_pages"].numel())
    served = fits & ((need == 0) | (base + need <= free))
    col = torch.arange(width, device=table.device)
    k = base[:, None] + col[None] - old[:, None]
    fresh = served[:, None] & (col[None] >= old[:, None]) & (col[None] < (old + need)[:, None])
    table = torch.where(fresh, s["free_pages"][(free - 1 - k).clamp(0, s["free_pages"].numel() - 1)], table)
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(ends, t, right=True)
    real = b < B
    b = b.clamp(max=B - 1)
    real &= served[b]
    pos = L[b] + t - (ends - n)[b]
    page_of = table[b, (pos // page).clamp(0, width - 1)].long()
    zero = torch.zeros(1, dtype=torch.int64, device=table.device)
    return {"seq_lens": torch.where(served, L + n, L).int(), "free_count": (free - (need * served).sum()).int(),
            "cu_new": torch.cat([zero, ends]).clamp(max=T).int(),
            "slot_map": torch.where(real, page_of * page + pos % page, -1),
            "positions": torch.where(real, pos, -1).int(), "served": served.int(), "page_table": table}


def _append_bf16(s):
    page, real = s["page"], s["slot_map"] >= 0
    slot = s["slot_map"][real]
    for n in ("k", "v"):
        s[n + "_cache"][slot // page, :, slot % page] = s[n][real]
    return {"k": s["k_cache"], "v": s["v_cache"]}


def _append_fp8(s):
    page, real = s["page"], s["slot_map"] >= 0
    dtype, top = FP8[s["fmt"]]
    slot = s["slot_map"][real]
    for n in ("k", "v"):
        x = s[n][real].float()
        pages, heads, nblk = s[n + "_scales"].shape
        block = page // nblk
        blk, off = slot // block, slot % block             # block number over the whole cache
        hit, where_ = torch.unique(blk, return_inverse=True)
        first = torch.full((hit.numel(),), block, dtype=torch.int64, device=x.device).scatter_reduce(0, where_, off, "amin")
        big = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
        big = torch.zeros((hit.numel(), heads), device=x.device).scatter_reduce(
            0, where_[:, None].expand(-1, heads), big, "amax")
        want = big / top
        if s["fmt"] == "e4m3_pow2":
            m, e = torch.frexp(want)                        # want = m * 2^e, m in [0.5, 1): the next power of two
            want = torch.where(want > 0, torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e)), 0.0)
        at = (hit // nblk, slice(None), hit % nblk)
        old = torch.where(first[:, None] > 0, s[n + "_scales"][at], 0.0)
        new = torch.maximum(old, want)
        s[n + "_scales"][at] = new
        by = torch.where(new > 0, new, 1.0)
        cache = s[n + "_cache"].view(pages, heads, nblk, block, x.shape[-1])
        was = cache[at]
        y = (was.view(dtype).float() * old[..., None, None]) / by[..., None, None]
        y = y.clamp(-top, top).to(dtype).view(torch.uint8)
        row = torch.arange(block, device=x.device)
        keep = (row[None, None] < first[:, None, None]) & (new > old)[..., None]
        cache[at] = torch.where(keep[..., None], y, was)
        y = (x / by[where_][..., None]).clamp(-top, top).to(dtype).view(torch.uint8)
        s[n + "_cache"][slot // page, :, slot % page] = y
    return _as_values(s)


def _decode(s):
    q, table = s["q"].float(), s["page_table"].long().clamp(0, s["k_cache"].shape[0] - 1)
    B, H, nq, d = q.shape
    pages, heads, page, _ = s["k_cache"].shape
    nblk, N = s["k_scales"].shape[2], table.shape[1] * page

    def values(n):
        x = s[n + "_cache"][table].view(FP8[s["fmt"]][0]).float()
        x = x.view(B, table.shape[1], heads, nblk, page // nblk, d) * s[n + "_scales"][table][..., None, None]
        return x.view(B, table.shape[1], heads, page, d).transpose(1, 2).reshape(B, heads, N, d)

    pos = s["seq_lens"].long()[:, None] - nq + torch.arange(nq, device=q.device)[None]    # [B, nq]
    j = torch.arange(N, device=q.device)
    seen = j <= pos[..., None]
    if s["window"] > 0:
        seen &= j >= pos[..., None] - s["window"]
    seen = seen[:, None, None]                                                             # [B, 1, 1, nq, N]
    x = (q.view(B, heads, -1, d) * s["scale"]) @ values("k").transpose(-1, -2)
    x = x.view(B, heads, H // heads, nq, N).masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, heads, -1, N) @ values("v")).view(B, heads, H // heads, nq, d)
    o = o / torch.where(l > 0, l, 1.0)
    return {"o": o.view(B, H, nq, d).to(torch.bfloat16), "lse": (m + torch.log(l)).view(B, H, nq)}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "plan":
        lens = _plan_lens(case)
        tokens = sum(m for _, m in lens) + case["pad"]
        taken = sum(_pages(n + m, case["page"]) - _pages(n, case["page"]) for n, m in lens)
        return {"bytes": tokens * 12 + case["batch"] * (8 + 4 + 12) + taken * 8, "flops": 0}
    if case["op"] == "decode_fp8":
        d, keys, pairs = case["d"], 0, 0
        for L in _decode_lens(case):
            lo = max(0, L - case["nq"] - case["window"]) if case["window"] > 0 else 0
            keys += L - lo
            for i in range(case["nq"]):
                last = L - case["nq"] + i
                pairs += max(0, last + 1 - (max(0, last - case["window"]) if case["window"] > 0 else 0))
        cache = 2 * keys * case["kv_heads"] * (d + 4 / case["block"])
        rows = case["batch"] * case["heads"] * case["nq"]
        return {"bytes": cache + rows * (4 * d + 4), "flops": 4 * pairs * case["heads"] * d}
    tokens = sum(m for _, m in _append_lens(case))
    out = 1 if case["op"] == "append_fp8" else 2
    values = 2 * tokens * case["heads"] * case["d"]
    return {"bytes": values * (2 + out) + 8 * (tokens + case["pad"]), "flops": 2 * values if out == 1 else 0}


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "append_bf16":
        return {n: _exact_rows(s, n) for n in ("k", "v")}
    if case["op"] == "append_fp8":
        out = {}
        for n in ("k", "v"):
            out[n], out[n + "_scales"] = _exact_blocks(s, n)
        return out
    return _exact_decode(s)


def _exact_rows(s, n):
    cache = s[n + "_cache"].double()
    slots = s["slot_map"].tolist()
    for t, slot in enumerate(slots):
        if slot >= 0:
            cache[slot // s["page"], :, slot % s["page"]] = s[n][t].double()
    return cache


def _nearest(x, fmt):
    """x on the format's grid, ties to even, largest value where it is beyond."""
    mantissa, least, top = {"e5m2": (2, -14, 57344.0)}.get(fmt, (3, -6, 448.0))
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** (least - 20)))).clamp(min=least)
    step = torch.exp2(e - mantissa)
    return (torch.round(x / step) * step).clamp(-top, top)


def _exact_blocks(s, n):
    fmt, page = s["fmt"], s["page"]
    dtype, top = FP8[fmt]
    cache, scales = s[n + "_cache"].view(dtype).double(), s[n + "_scales"].double()
    block = page // scales.shape[2]
    slots, t = s["slot_map"].tolist(), 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        end = t + 1
        while end < len(slots) and slots[end] == slots[end - 1] + 1 and slots[end] // block == slots[t] // block:
            end += 1
        p, r, c = slots[t] // page, slots[t] % page, slots[t] % page // block
        x = s[n][t:end].double().transpose(0, 1)                       # [heads, run, d]
        want = x.abs().amax((1, 2)) / top
        if fmt == "e4m3_pow2":
            want = torch.exp2(torch.ceil(torch.log2(want)))
        old = scales[p, :, c] if r % block else torch.zeros_like(want)
        new = torch.maximum(old, want)
        if r % block:
            rows = slice(c * block, r)
            again = _nearest(cache[p, :, rows] * (old / new)[:, None, None], fmt)
            cache[p, :, rows] = torch.where((new > old)[:, None, None], again, cache[p, :, rows])
        cache[p, :, r:r + end - t] = _nearest(x / new[:, None, None], fmt)
        scales[p, :, c] = new
        t = end
    return cache, scales


def _exact_decode(s):
    q, window = s["q"].double(), s["window"]
    B, H, nq, d = q.shape
    pages, heads, page, _ = s["k_cache"].shape
    o = torch.zeros((B, H, nq, d), dtype=torch.float64, device=q.device)
    lse = torch.full((B, H, nq), -math.inf, dtype=torch.float64, device=q.device)
    for b, L in enumerate(s["seq_lens"].tolist()):
        used = s["page_table"][b, :_pages(L, page)].long()
        full = {}
        for n in ("k", "v"):
            x = s[n + "_cache"][used].view(FP8[s["fmt"]][0]).double()
            x = x * torch.repeat_interleave(s[n + "_scales"][used].double(), page // s[n + "_scales"].shape[2], 2)[..., None]
            full[n] = x.permute(1, 0, 2, 3).reshape(heads, -1, d)[:, :L]
        for i in range(nq):
            last = L - nq + i
            first = max(0, last - window) if window > 0 else 0
            if last < 0:
                continue
            rows = q[b, :, i].view(heads, H // heads, d)
            x = torch.einsum("hgd,hnd->hgn", rows, full["k"][:, first:last + 1]) * s["scale"]
            z = torch.logsumexp(x, -1, keepdim=True)
            o[b, :, i] = torch.einsum("hgn,hnd->hgd", torch.exp(x - z), full["v"][:, first:last + 1]).reshape(H, d)
            lse[b, :, i] = z.reshape(H)
    return {"o": o, "lse": lse}
