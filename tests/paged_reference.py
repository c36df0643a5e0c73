"""Plain implementations of the paged-cache operators for the tests: Python loops and
numpy, 64 bits where the operator computes, IEEE fp32 where its definition says so."""
from __future__ import annotations

import math

import numpy as np

import oracle

TOP = {"e4m3": 448.0, "e4m3_pow2": 448.0, "e5m2": 57344.0}


def encode(x, fmt):
    return (oracle.e5m2_encode if fmt == "e5m2" else oracle.e4m3_encode)(np.ascontiguousarray(x, np.float32))


def decode(codes, fmt):
    return (oracle.e5m2_decode if fmt == "e5m2" else oracle.e4m3_decode)(codes)


# ------------------------------------------------------------------ plan
def plan(new_lens, seq_lens, page_table, free_pages, free_count, ps, num_tokens):
    """Request after request; returns a dict of numpy arrays, page_table among them."""
    table = np.array(page_table)
    B, max_pages = table.shape
    cap, free = max_pages * ps, min(max(int(np.ravel(free_count)[0]), 0), len(free_pages))
    out = dict(seq_lens=[], served=[], cu_new=[0], slot_map=[-1] * num_tokens, positions=[-1] * num_tokens)
    row, wanted, taken = 0, 0, 0
    for b in range(B):
        n, L = max(int(new_lens[b]), 0), min(max(int(seq_lens[b]), 0), cap)
        old = -(-L // ps)
        ok = L + n <= cap and row + n <= num_tokens
        if ok:
            need = -(-(L + n) // ps) - old
            ok = need == 0 or wanted + need <= free
            for k in range(need if ok else 0):
                table[b, old + k] = free_pages[free - 1 - wanted - k]
            taken += need if ok else 0
            wanted += need
        for j in range(n if ok else 0):
            pos = L + j
            page = int(table[b, pos // ps])
            out["slot_map"][row + j] = page * ps + pos % ps if page >= 0 else -1
            out["positions"][row + j] = pos
        row += n
        out["cu_new"].append(min(row, num_tokens))
        out["served"].append(int(ok))
        out["seq_lens"].append(L + n if ok else L)
    out = {k: np.array(v, np.int64 if k == "slot_map" else np.int32) for k, v in out.items()}
    out["free_count"] = np.array([free - taken], np.int32)
    out["page_table"] = table
    return out


# ------------------------------------------------------------------ 8-bit append
def append_fp8(x, cache, scales, slot_map, fmt):
    """x fp32 [T, H, d] (bf16 values); cache uint8 [pages, H, ps, d] and scales fp32
    [pages, H, nblk] are updated in place, run after run."""
    pages, H, ps, d = cache.shape
    block = ps // scales.shape[2]
    slots = [int(s) if 0 <= s < pages * ps else -1 for s in slot_map]
    top = np.float32(TOP[fmt])
    t = 0
    with np.errstate(all="ignore"):
        while t < len(slots):
            if slots[t] < 0:
                t += 1
                continue
            end = t + 1
            while end < len(slots) and slots[end] == slots[end - 1] + 1 and slots[end] % block != 0:
                end += 1
            page, row = divmod(slots[t], ps)
            blk, o = divmod(row, block)
            for h in range(H):
                v = x[t:end, h].astype(np.float32)
                a = np.abs(v)
                a = np.float32(a[np.isfinite(a)].max(initial=0.0))
                need = np.float32(a / top)
                if fmt == "e4m3_pow2" and need > 0:
                    m, e = math.frexp(float(need))
                    need = np.float32(math.ldexp(1.0, e - 1 if m == 0.5 else e))
                old = scales[page, h, blk] if o > 0 else np.float32(0)
                s = max(old, need)
                if o > 0 and s > old:
                    rows = slice(blk * block, blk * block + o)
                    y = (decode(cache[page, h, rows], fmt).astype(np.float32) * old).astype(np.float32) / s
                    cache[page, h, rows] = encode(y, fmt)
                by = s if s > 0 else np.float32(1)
                cache[page, h, row:row + end - t] = encode((v / by).astype(np.float32), fmt)
                scales[page, h, blk] = s
            t = end


# ------------------------------------------------------------------ decoding over the 8-bit cache
def decode_fp8(q, kc, vc, ks, vs, table, lens, fmt, scale, window=0):
    """O, LSE in float64 and, element by element, how far a kernel may be off.

    The bound adds what the kernel rounds, with p the softmax weights, w_j = p_j vs_j:
      scores: q and k8 are exact factors, summed in fp32 (d products, a tensor core may
        truncate: 2^-23 of the sum of magnitudes each), then scaled, shifted and
        exponentiated (2^-21 of the largest magnitude):
        ds = d 2^-23 max_j scale ks_j sum|q k8| + 2^-21 (1 + max|s|)
        moves a weight by ds and the normalised result by 2 ds;
      weights in fp16: half a step, 2^-11 of each, and below fp16's normal numbers
        2^-25 of the largest weight (times 2, as a scale's mantissa is split off).  The
        kernels take weights relative to max_j p_j 2^e_j, where e_j is the exponent of vs_j
        but at least 60 below that of the largest scale (and of 1), so that a block with the
        scale 0 still counts in the sum; the largest weight is therefore
        max_j p_j max(vs_j, 2^-60 max(1, largest vs)), not max_j p_j vs_j: a row whose softmax
        sits on blocks of scale 0 has its fp16 step there;
      sums of n weights in fp32 by 16s: 2^-22 n / 16;
      O in bf16: 2^-8 of the value.
    """
    q = np.asarray(q, np.float64)
    B, H, nq, d = q.shape
    pages, Hkv, ps, _ = kc.shape
    block = ps // ks.shape[2]
    o, lse = np.zeros((B, H, nq, d)), np.full((B, H, nq), -np.inf)
    o_tol, lse_tol = np.zeros((B, H, nq, d)), np.zeros((B, H, nq))
    for b in range(B):
        L = min(max(int(lens[b]), 0), table.shape[1] * ps)
        t = np.arange(L)
        page = np.clip(table[b, t // ps], 0, pages - 1)
        for h in range(H):
            hk = h // (H // Hkv)
            K8 = decode(kc[page, hk, t % ps], fmt).astype(np.float64)
            V8 = decode(vc[page, hk, t % ps], fmt).astype(np.float64)
            ksc = ks[page, hk, t % ps // block].astype(np.float64)
            vsc = vs[page, hk, t % ps // block].astype(np.float64)
            for i in range(nq):
                last = L - nq + i
                first = max(0, last - window) if window > 0 else 0
                if last < 0:
                    continue
                j = slice(first, last + 1)
                s = scale * ksc[j] * (K8[j] @ q[b, h, i])
                m = s.max()
                e = np.exp(s - m)
                p = e / e.sum()
                o[b, h, i] = (p * vsc[j]) @ V8[j]
                lse[b, h, i] = m + np.log(e.sum())
                ds = (d * 2.0 ** -23 * (scale * ksc[j] * (np.abs(K8[j]) @ np.abs(q[b, h, i]))).max()
                      + 2.0 ** -21 * (1 + np.abs(s).max()))
                n = last + 1 - first
                w = p * vsc[j]
                avg = w @ np.abs(V8[j])
                w_max = (p * np.maximum(vsc[j], 2.0 ** -60 * max(1.0, vsc[j].max()))).max()
                o_tol[b, h, i] = (2.0 ** -8 * np.abs(o[b, h, i]) + avg * (2.0 ** -11 + 2 * ds + 2.0 ** -22 * n / 16)
                                  + 2.0 ** -24 * w_max * np.abs(V8[j]).sum(0) + 1e-30)
                lse_tol[b, h, i] = ds + 2.0 ** -22 * (n / 16 + abs(lse[b, h, i]))
    return o, lse, o_tol, lse_tol


def make_cache(rng, lens, Hkv, d, ps, block, fmt, spare=3, stale=True):
    """A filled 8-bit cache: codes and scales of normal data, pages in a shuffled order, unused
    table entries -1.  `stale`: what lies behind the sequences is NaN codes and NaN scales."""
    need = [-(-int(n) // ps) for n in lens]
    pages, width = sum(need) + spare, max(1, max(need))
    perm, used = rng.permutation(pages), 0
    table = np.full((len(lens), width), -1, np.int32)
    out = []
    for _ in range(2):
        x = rng.standard_normal((pages, Hkv, ps, d)).astype(np.float32)
        nblk = ps // block
        xb = x.reshape(pages, Hkv, nblk, block, d)
        xb *= np.exp2(rng.integers(-4, 5, (pages, Hkv, nblk))).astype(np.float32)[..., None, None]
        s = (np.abs(xb).max((3, 4)) / np.float32(TOP[fmt])).astype(np.float32)
        if fmt == "e4m3_pow2":
            s = np.exp2(np.ceil(np.log2(s))).astype(np.float32)
        out.append([encode(xb / s[..., None, None], fmt).reshape(x.shape), s])
    live = np.zeros((pages, ps), bool)
    for b, n in enumerate(need):
        table[b, :n] = perm[used:used + n]
        used += n
        t = np.arange(int(lens[b]))
        live[table[b, t // ps], t % ps] = True
    if stale:
        for codes, s in out:
            codes.transpose(0, 2, 1, 3)[~live] = 0x7F
            s.transpose(0, 2, 1)[~live.reshape(pages, -1, block).any(2)] = np.nan
    (kc, ks), (vc, vs) = out
    return kc, vc, ks, vs, table
