"""GPU parity of the paged-cache operators (attn_paged_plan, attn_cache_append_bf16,
attn_cache_append_fp8, attn_decode_fp8_paged) against plain implementations, at the sizes,
masks and contents where they can go wrong."""
import math

import numpy as np
import pytest
import torch

from tests import paged_reference as ref
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu
FORMATS = ["e4m3", "e5m2", "e4m3_pow2"]


@pytest.fixture(scope="module")
def fa():
    require_gpu()
    import exact_attention_55_gb300 as fa
    fa.load_library()
    return fa


def cuda(a, dtype=None):
    t = torch.from_numpy(np.array(a))
    return (t if dtype is None else t.to(dtype)).cuda()


# ------------------------------------------------------------------ plan
def plan_case(rng, B, ps, max_pages, hi_len, hi_new, free, pad):
    seq = rng.integers(0, hi_len + 1, B).astype(np.int32)
    new = rng.integers(0, hi_new + 1, B).astype(np.int32)
    owned = B * max_pages
    table = rng.permutation(owned).astype(np.int32).reshape(B, max_pages)
    stack = (owned + rng.permutation(max(free, 1))).astype(np.int32)
    return new, seq, table, stack, np.array([free], np.int32), ps, int(new.sum()) + pad


def run_plan(fa, new, seq, table, stack, count, ps, T, **kw):
    t = [cuda(a) for a in (new, seq, table, stack, count)]
    outs = fa.attn_paged_plan(*t, ps, T, **kw)
    got = dict(zip(("seq_lens", "free_count", "cu_new", "slot_map", "positions", "served"), outs), page_table=t[2])
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in got.items()}


def check_plan(fa, case):
    want, got = ref.plan(*case), run_plan(fa, *case)
    for k in want:
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)


@pytest.mark.parametrize("B", [1, 2, 31, 129, 700, 5000, 16384])
@pytest.mark.parametrize("ps", [1, 16, 64])
def test_plan(fa, B, ps):
    rng = np.random.default_rng(B + ps)
    width = -(-70 // ps)
    check_plan(fa, plan_case(rng, B, ps, width, 40, 30, B * width, pad=B % 3))


@pytest.mark.parametrize("free", [0, 1, 7, 40, 41])
def test_plan_with_too_few_pages(fa, free):
    """The pool runs out on the way: later requests that need no page are still served."""
    rng = np.random.default_rng(free)
    check_plan(fa, plan_case(rng, 60, 16, 8, 90, 30, free, pad=5))


def test_plan_of_long_requests(fa):
    """Many tokens of few requests (several CTAs), a request that overruns its table, one
    that adds nothing, negative lengths and counts, a page table entry below zero."""
    rng = np.random.default_rng(3)
    new = np.array([9000, 0, 20000, -5, 12345, 1, 6], np.int32)
    seq = np.array([17, 30, 64, 12, -9, 2 ** 31 - 1, 20], np.int32)
    table = rng.permutation(7 * 400).astype(np.int32).reshape(7, 400)
    table[6, 1] = -1
    stack = (5000 + rng.permutation(4000)).astype(np.int32)
    for T in (int(new.clip(0).sum()), int(new.clip(0).sum()) + 1000, 29001, 0):
        check_plan(fa, (new, seq, table, stack, np.array([3900], np.int32), 64, T))
    check_plan(fa, (new, seq, table, stack, np.array([99999], np.int32), 64, 41352))
    check_plan(fa, (new, seq, table, stack, np.array([-4], np.int32), 64, 41352))


def test_plan_of_very_many_rows(fa):
    """2^28 and more packed rows: the outputs' one allocation is sized in 64 bits."""
    T, i32 = (1 << 28) + 7, dict(dtype=torch.int32, device="cuda")
    new, lens = torch.tensor([3, 0, 2], **i32), torch.tensor([5, 1, 16], **i32)
    table = torch.tensor([[4, -1], [2, -1], [1, -1]], **i32)
    out = fa.attn_paged_plan(new, lens, table, torch.tensor([7, 9], **i32), torch.tensor([2], **i32), 16, T)
    seq, left, cu, slots, pos, served = out
    assert seq.tolist() == [8, 1, 18] and left.tolist() == [1] and cu.tolist() == [0, 3, 3, 5]
    assert served.tolist() == [1, 1, 1] and table[2].tolist() == [1, 9]
    assert slots[:5].tolist() == [4 * 16 + 5, 4 * 16 + 6, 4 * 16 + 7, 9 * 16, 9 * 16 + 1]
    assert pos[:5].tolist() == [5, 6, 7, 16, 17]
    assert slots.numel() == pos.numel() == T and (slots[5:] == -1).all() and (pos[5:] == -1).all()


def test_plan_in_place_and_again(fa):
    """seq_lens and free_count may be their own outputs; steps follow one another."""
    rng = np.random.default_rng(4)
    new, seq, table, stack, count, ps, _ = plan_case(rng, 300, 16, 30, 40, 20, 3000, 0)
    t = [cuda(a) for a in (new, seq, table, stack, count)]
    for step in range(4):
        T = int(new.sum())
        want = ref.plan(new, seq, table, stack, count, ps, T)
        outs = fa.attn_paged_plan(*t, ps, T, seq_lens_out=t[1], free_count_out=t[4])
        torch.cuda.synchronize()
        seq, table, count = want["seq_lens"], want["page_table"], want["free_count"]
        np.testing.assert_array_equal(t[1].cpu().numpy(), seq)
        np.testing.assert_array_equal(t[2].cpu().numpy(), table)
        np.testing.assert_array_equal(t[4].cpu().numpy(), count)
        np.testing.assert_array_equal(outs[3].cpu().numpy(), want["slot_map"])


# ------------------------------------------------------------------ appends
def slots_of(rng, lens, news, ps, pad=0, spare=3):
    need = [-(-(L + n) // ps) for L, n in zip(lens, news)]
    pages, used, slots = sum(need) + spare, 0, []
    perm = rng.permutation(pages)
    for L, n, c in zip(lens, news, need):
        own = perm[used:used + c]
        used += c
        pos = np.arange(L, L + n)
        slots.append(own[pos // ps] * ps + pos % ps)
    return pages, np.concatenate(slots + [np.full(pad, -1)]).astype(np.int64)


def rows_of(rng, T, H, d, outliers=True):
    x = rng.standard_normal((T, H, d)).astype(np.float32)
    if outliers:
        x[rng.random(x.shape) < 2e-3] *= 30
    return torch.from_numpy(x).bfloat16()


def strided(k, v, how):
    """K and V as separate tensors, or as columns of one wider matrix."""
    if how == "whole":
        return k.cuda(), v.cuda()
    T, H, d = k.shape
    wide = torch.full((T, 2 * H * d + 8), float("nan"), dtype=torch.bfloat16)
    wide[:, :H * d], wide[:, H * d + 8:] = k.reshape(T, -1), v.reshape(T, -1)
    wide = wide.cuda()
    return wide[:, :H * d].unflatten(1, (H, d)), wide[:, H * d + 8:].unflatten(1, (H, d))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ps", [1, 16, 128])
@pytest.mark.parametrize("how", ["whole", "columns"])
def test_append_bf16(fa, d, ps, how):
    rng = np.random.default_rng(d + ps)
    pages, slots = slots_of(rng, [0, 5, 130, 17], [1, 40, 3, 200], ps, pad=2)
    slots[3] = pages * ps            # outside the cache: skipped
    k, v = rows_of(rng, len(slots), 3, d), rows_of(rng, len(slots), 3, d)
    kc, vc = (torch.randn(pages, 3, ps, d).bfloat16() for _ in range(2))
    want = [kc.clone(), vc.clone()]
    for t, s in enumerate(slots):
        if 0 <= s < pages * ps:
            want[0][s // ps, :, s % ps], want[1][s // ps, :, s % ps] = k[t], v[t]
    kd, vd = strided(k, v, how)
    got = fa.attn_cache_append_bf16(kd, vd, kc.cuda(), vc.cuda(), cuda(slots))
    torch.cuda.synchronize()
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])


def check_append_fp8(fa, rng, slots, pages, H, d, ps, block, fmt, how="whole", k=None, v=None, prior=None):
    T = len(slots)
    k = rows_of(rng, T, H, d) if k is None else k
    v = rows_of(rng, T, H, d) if v is None else v
    if prior is None:
        codes = [rng.integers(0, 256, (pages, H, ps, d)).astype(np.uint8) for _ in range(2)]
        scales = [np.exp2(rng.uniform(-12, -4, (pages, H, ps // block))).astype(np.float32) for _ in range(2)]
        for c in codes:       # old rows hold finite codes
            c[(c & 0x7F) >= (0x7C if fmt == "e5m2" else 0x7F)] = 0x11
        if fmt == "e4m3_pow2":
            scales = [np.exp2(np.round(np.log2(s))).astype(np.float32) for s in scales]
    else:
        codes, scales = prior
    dev = [cuda(c) for c in codes + scales]
    kd, vd = strided(k, v, how)
    fa.attn_cache_append_fp8(kd, vd, dev[0], dev[1], dev[2], dev[3], cuda(slots), fmt=fmt)
    torch.cuda.synchronize()
    for x, c, s in ((k, codes[0], scales[0]), (v, codes[1], scales[1])):
        ref.append_fp8(x.float().numpy(), c, s, slots, fmt)
    for n, got, want in zip(("k_scales", "v_scales", "k", "v"), (dev[2], dev[3], dev[0], dev[1]),
                            (scales[0], scales[1], codes[0], codes[1])):
        np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=n)
    return codes, scales


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d,ps,block", [(64, 16, 16), (64, 64, 32), (128, 64, 64), (128, 256, 128), (256, 128, 128),
                                        (256, 32, 16)])
def test_append_fp8(fa, fmt, d, ps, block):
    rng = np.random.default_rng(d + ps + block)
    lens = [0, 1, 15, 16, 17, 63, 100, 127, 128, 200, 31]
    news = [1, 1, 1, 1, 30, 2, 1, 1, 128, 77, 300]
    pages, slots = slots_of(rng, lens, news, ps, pad=3)
    check_append_fp8(fa, rng, slots, pages, 3, d, ps, block, fmt, how="columns" if d == 128 else "whole")


@pytest.mark.parametrize("block", [16, 64, 128])
def test_append_fp8_one_token_each(fa, block):
    """A decoding step: every token is a run of its own, some slots are padding in between."""
    rng = np.random.default_rng(block)
    lens = list(rng.integers(0, 300, 150))
    pages, slots = slots_of(rng, lens, [1] * 150, 128)
    slots[::7] = -1
    slots[3] = pages * 128
    slots[4] = 2 ** 40
    check_append_fp8(fa, rng, slots, pages, 2, 128, 128, block, "e4m3")


def test_append_fp8_step_by_step_is_deterministic(fa):
    """A block that fills token by token, growing its scale on the way."""
    rng = np.random.default_rng(9)
    ps, H, d = 64, 2, 64
    codes = [np.full((3, H, ps, d), 0x7F, np.uint8) for _ in range(2)]
    scales = [np.full((3, H, 1), np.nan, np.float32) for _ in range(2)]
    for t in range(70):
        x = (rows_of(rng, 1, H, d).float() * 1.07 ** t).bfloat16()
        slot = np.array([t if t < 64 else 2 * 64 + t - 64])
        codes, scales = check_append_fp8(fa, rng, slot, 3, H, d, ps, ps, "e4m3", k=x, v=x * 3, prior=(codes, scales))


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_fp8_unusual_values(fa, fmt):
    """Zeros, infinities, NaN, the largest and the smallest bf16 values, and a block that is
    all zero before its first other value."""
    rng = np.random.default_rng(10)
    T, H, d, ps = 96, 2, 64, 32
    k = rows_of(rng, T, H, d)
    k[0:32] = 0
    k[33, 0, 5], k[34, 1, 6], k[35, 0, 7] = float("inf"), float("-inf"), float("nan")
    k[64:80] *= 1e-38
    k[80:96] = k[80:96].sign() * 3.3e38
    v = k.flip(0).contiguous()
    check_append_fp8(fa, rng, np.arange(T), 4, H, d, ps, 16, fmt, k=k, v=v)
    zero = torch.zeros(4, H, d, dtype=torch.bfloat16)
    prior = check_append_fp8(fa, rng, np.arange(4), 4, H, d, ps, 32, fmt, k=zero, v=zero)
    check_append_fp8(fa, rng, np.arange(4, 12), 4, H, d, ps, 32, fmt, prior=prior)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_append_fp8_requantises_every_code(fa, fmt):
    """Every code under pairs of an old and a larger new scale: any mantissas, neighbours, large
    ratios, scales near fp32's limits.  The new codes are those of IEEE fp32 (code * old) / s."""
    rng = np.random.default_rng(70)
    T, d, ps = 6000, 256, 16
    amax = np.exp2(rng.uniform(-126, 126, T)).astype(np.float32)
    amax[:3000] = np.exp2(rng.uniform(-8, 8, 3000)).astype(np.float32)
    k = torch.zeros(T, 1, d, dtype=torch.bfloat16)
    k[:, 0, 0] = torch.from_numpy(amax).bfloat16()
    s = (k[:, 0, 0].float().numpy() / np.float32(ref.TOP[fmt])).astype(np.float32)
    ratio = np.exp2(-rng.uniform(0, 6, T)).astype(np.float32)
    ratio[::4] = 1 - rng.integers(1, 5, ratio[::4].shape).astype(np.float32) * np.float32(2.0 ** -24)
    ratio[1::4] = np.exp2(-rng.integers(0, 12, ratio[1::4].shape)).astype(np.float32)
    ratio[2::40] = np.float32(1e-30)
    old = (s * ratio).astype(np.float32)
    codes = np.tile(np.arange(256, dtype=np.uint8), (T, 1))
    kc = np.zeros((T, 1, ps, d), np.uint8)
    kc[:, 0, 0] = codes
    got = [cuda(kc), cuda(kc), cuda(old.reshape(T, 1, 1)), cuda(old.reshape(T, 1, 1))]
    fa.attn_cache_append_fp8(k.cuda(), k.cuda(), *got, cuda(np.arange(T, dtype=np.int64) * ps + 1), fmt=fmt)
    with np.errstate(all="ignore"):
        want = ref.encode((ref.decode(codes, fmt).astype(np.float32) * old[:, None]).astype(np.float32) / s[:, None], fmt)
    want[old >= s] = codes[old >= s]
    for cache, scale in ((got[0], got[2]), (got[1], got[3])):
        assert (scale.cpu().numpy()[:, 0, 0] == np.maximum(s, old)).all()
        bad = np.argwhere(cache.cpu().numpy()[:, 0, 0] != want)
        assert len(bad) == 0, (len(bad), bad[:3], [(old[t], s[t], c) for t, c in bad[:3]])


@pytest.mark.parametrize("d,block", [(64, 16), (128, 128), (256, 64)])
def test_append_fp8_large_call_equals_small_ones(fa, d, block):
    """How many tokens and heads a CTA takes depends on the call's size; the bytes do not: a long
    call against the same tokens in calls that end at blocks, both behind filled rows."""
    g = torch.Generator(device="cuda").manual_seed(block)
    T, H, ps = 24000, 3, 128
    k, v = (torch.randn(T, H, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    pages = T // ps + 2
    slots = torch.randperm(pages, device="cuda", generator=g)[:, None] * ps + torch.arange(ps, device="cuda")
    slots = slots.flatten()[5:5 + T].contiguous()
    caches = [torch.randint(0, 100, (pages, H, ps, d), dtype=torch.uint8, device="cuda", generator=g) for _ in range(2)]
    scales = [torch.full((pages, H, ps // block), 1e-3, device="cuda") for _ in range(2)]
    big = [t.clone() for t in caches + scales]
    fa.attn_cache_append_fp8(k, v, *big, slots)
    cuts = [0] + list(range(block - 5, T, 16 * block)) + [T]
    for a, b in zip(cuts, cuts[1:]):
        fa.attn_cache_append_fp8(k[a:b], v[a:b], *caches, *scales, slots[a:b])
    for x, y in zip(big, caches + scales):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ decoding
# Many query rows under one key head go to a kernel of their own (tcgen05) once the step is
# large; how large it is follows from the table's width, so a table of this many keys, most of
# its entries unused, brings short sequences there too.
WIDE_TABLE = 1 << 18


def widen(table, ps, keys=WIDE_TABLE):
    return np.concatenate([table, np.full((len(table), keys // ps), -1, np.int32)], 1)


def check_decode(fa, lens, H, Hkv, nq, d, ps, block, fmt, window=0, seed=0, qmul=1.0, stale=True, scale=None, wide=False):
    rng = np.random.default_rng(seed)
    kc, vc, ks, vs, table = ref.make_cache(rng, lens, Hkv, d, ps, block, fmt, stale=stale)
    if wide:
        table = widen(table, ps)
    q = (torch.from_numpy(rng.standard_normal((len(lens), H, nq, d)).astype(np.float32)) * qmul).bfloat16()
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o, lse = fa.attn_decode_fp8_paged(q.cuda(), cuda(kc), cuda(vc), cuda(ks), cuda(vs), cuda(table),
                                      cuda(np.array(lens, np.int32)), fmt=fmt, scale=scale, window=window)
    assert fa.attn_get_device_status() == fa.ATTN_OK
    compare_decode(o, lse, ref.decode_fp8(q.double().numpy(), kc, vc, ks, vs, table, lens, fmt, scale, window))


def compare_decode(o, lse, want):
    o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
    ro, rl, o_tol, l_tol = want
    empty = np.isneginf(rl)
    assert (np.isneginf(lse) == empty).all() and (o[empty] == 0).all()
    assert np.isfinite(o).all()
    off = np.abs(o - ro)
    assert (off <= o_tol).all(), f"O: {(off / np.maximum(o_tol, 1e-300)).max()} of the bound"
    off = np.abs(lse[~empty] - rl[~empty])
    assert (off <= l_tol[~empty]).all(), f"LSE: {(off / l_tol[~empty]).max()} of the bound"


LENS = [1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 130, 500]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("nq,group", [(1, 1), (1, 4), (3, 2), (8, 1), (2, 8), (8, 5)])
def test_decode_fp8(fa, d, fmt, nq, group):
    check_decode(fa, LENS, 2 * group, 2, nq, d, 32, 16, fmt, seed=d + nq)


@pytest.mark.parametrize("ps,block", [(16, 16), (64, 16), (64, 64), (128, 128), (256, 64), (1024, 128)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_fp8_page_sizes(fa, ps, block, d):
    check_decode(fa, [700, 33, 1025, 0, 1], 6, 3, 2, d, ps, block, "e4m3", seed=ps + block)


@pytest.mark.parametrize("window", [1, 5, 16, 100, 127, 128, 400, 100000])
@pytest.mark.parametrize("nq", [1, 4])
def test_decode_fp8_window(fa, window, nq):
    """Sliding windows; the pages before a window hold NaN codes and scales, as freed ones may."""
    lens, d, ps, block = [1, 3, 100, 129, 600, 1111], 64, 32, 16
    rng = np.random.default_rng(window)
    kc, vc, ks, vs, table = ref.make_cache(rng, lens, 2, d, ps, block, "e4m3")
    for b, L in enumerate(lens):
        lo = max(0, L - nq - window)
        for t in range(lo):
            kc[table[b, t // ps], :, t % ps], vc[table[b, t // ps], :, t % ps] = 0x7F, 0xFF
        for blk in range(lo // block):
            ks[table[b, blk * block // ps], :, blk % (ps // block)] = np.nan
            vs[table[b, blk * block // ps], :, blk % (ps // block)] = np.inf
        table[b, :lo // ps] = -1
    q = torch.from_numpy(rng.standard_normal((len(lens), 6, nq, d)).astype(np.float32)).bfloat16()
    o, lse = fa.attn_decode_fp8_paged(q.cuda(), cuda(kc), cuda(vc), cuda(ks), cuda(vs), cuda(table),
                                      cuda(np.array(lens, np.int32)), scale=0.125, window=window)
    assert fa.attn_get_device_status() == fa.ATTN_OK
    compare_decode(o, lse, ref.decode_fp8(q.double().numpy(), kc, vc, ks, vs, table, lens, "e4m3", 0.125, window))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 32, 33, 48, 100])
def test_decode_fp8_many_query_heads(fa, rows, d):
    """One key head under any number of query heads."""
    check_decode(fa, [300, 64, 5], rows, 1, 1, d, 64, 64, "e4m3", seed=rows)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [17, 31, 32, 33, 64, 65, 100, 128, 129, 300])
def test_decode_fp8_wide_rows(fa, rows, d):
    """The kernel for many rows: 32, 64 and 128 rows a CTA, more in groups, some not full."""
    check_decode(fa, [300, 0, 64, 5, 1], rows, 1, 1, d, 64, 64, "e4m3", seed=rows, wide=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq,group", [(1, 20), (2, 16), (3, 16), (4, 8), (8, 5), (8, 16)])
def test_decode_fp8_wide(fa, d, fmt, nq, group):
    check_decode(fa, LENS + [1000], 2 * group, 2, nq, d, 32, 16, fmt, seed=d + nq, wide=True)


@pytest.mark.parametrize("ps,block", [(16, 16), (64, 16), (128, 128), (256, 64), (1024, 128)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_fp8_wide_page_sizes(fa, ps, block, d):
    check_decode(fa, [700, 33, 1025, 0, 1], 3 * 12, 3, 2, d, ps, block, "e4m3", seed=ps + block, wide=True)


@pytest.mark.parametrize("window", [1, 16, 100, 127, 500])
@pytest.mark.parametrize("nq,group", [(1, 32), (4, 16), (8, 16)])
def test_decode_fp8_wide_window(fa, window, nq, group):
    """Windows in the kernel for many rows (enough sequences for it), freed pages before them."""
    B, d, ps, block = 60, 64, 32, 16
    rng = np.random.default_rng(window + nq)
    lens = [int(n) for n in rng.integers(0, 900, B)]
    heads = -(-2432 // (B * -(-(window + nq) // 64) * (nq * group // 16 - 1)))
    kc, vc, ks, vs, table = ref.make_cache(rng, lens, heads, d, ps, block, "e4m3")
    for b, L in enumerate(lens):
        lo = max(0, L - nq - window)
        for t in range(lo):
            kc[table[b, t // ps], :, t % ps], vc[table[b, t // ps], :, t % ps] = 0x7F, 0xFF
        for blk in range(lo // block):
            ks[table[b, blk * block // ps], :, blk % (ps // block)] = np.nan
            vs[table[b, blk * block // ps], :, blk % (ps // block)] = np.inf
        table[b, :lo // ps] = -1
    q = torch.from_numpy(rng.standard_normal((B, heads * group, nq, d)).astype(np.float32)).bfloat16()
    o, lse = fa.attn_decode_fp8_paged(q.cuda(), cuda(kc), cuda(vc), cuda(ks), cuda(vs), cuda(table),
                                      cuda(np.array(lens, np.int32)), scale=0.125, window=window)
    assert fa.attn_get_device_status() == fa.ATTN_OK
    some = sorted(set(rng.integers(0, B, 12).tolist()) | {int(np.argmin(lens))})   # the reference is slow
    hs = [0, heads * group - 1, group // 2]
    kv = [0, heads - 1]
    want = [ref.decode_fp8(q[some][:, [h]].double().numpy(), kc[:, [h // group]], vc[:, [h // group]],
                           ks[:, [h // group]], vs[:, [h // group]], table[some], [lens[b] for b in some],
                           "e4m3", 0.125, window) for h in hs]
    assert kv[0] == hs[0] // group and kv[1] == hs[1] // group
    for h, w in zip(hs, want):
        compare_decode(o[some][:, [h]], lse[some][:, [h]], w)


def test_decode_fp8_wide_short_tables(fa):
    """Many short sequences under many rows: no head is split, nothing is joined."""
    rng = np.random.default_rng(30)
    lens = [int(n) for n in rng.integers(0, 385, 40)]
    check_decode(fa, lens, 64, 4, 8, 64, 64, 64, "e4m3", seed=31)


@pytest.mark.parametrize("d,H", [(256, 64), (128, 48), (64, 128)])
def test_decode_fp8_wide_many_parts(fa, d, H):
    """A few sequences over one key head: each unit's many rows come in many parts."""
    check_decode(fa, [2600, 3100, 1, 2900, 3000, 700, 2750, 3090], H, 1, 1, d, 64, 64, "e4m3", seed=d, wide=True)


def test_decode_fp8_wide_long(fa):
    """Parts of long and short sequences, several CTAs on each, joined."""
    check_decode(fa, [20001, 3, 7000, 1, 129], 32, 1, 1, 128, 64, 64, "e4m3_pow2", seed=32, wide=True)
    check_decode(fa, [9000], 20, 1, 4, 256, 128, 128, "e5m2", seed=33, wide=True)
    check_decode(fa, [5000] * 3, 64, 2, 1, 64, 16, 16, "e4m3", seed=34, wide=True)


def test_decode_fp8_long_and_ragged(fa):
    """Sequences of very different lengths, many CTAs on one of them."""
    check_decode(fa, [40001, 3, 7000, 1, 129, 12345], 4, 2, 1, 128, 64, 64, "e4m3_pow2", seed=11)
    check_decode(fa, [20000], 8, 1, 2, 256, 128, 128, "e4m3", seed=12)
    check_decode(fa, [9001] * 3, 3, 3, 1, 64, 16, 16, "e5m2", seed=13)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq,group", [(1, 3), (2, 4), (4, 4), (3, 8), (8, 7)])
def test_decode_fp8_split_heads(fa, d, nq, group):
    """Heads of more keys than one CTA keeps whole, under any number of query rows."""
    check_decode(fa, [1500, 2, 700, 385], 2 * group, 2, nq, d, 64, 32, "e4m3", seed=d + group)
    check_decode(fa, [2100], group, 1, nq, d, 64, 32, "e5m2", window=999, seed=d + nq)


@pytest.mark.parametrize("seed", range(24))
def test_decode_fp8_random_cases(fa, seed):
    rng = np.random.default_rng(1000 + seed)
    ps = int(rng.choice([16, 32, 64, 128]))
    block = int(rng.choice([b for b in (16, 32, 64, 128) if b <= ps]))
    B, Hkv, group = int(rng.integers(1, 9)), int(rng.integers(1, 5)), int(rng.choice([1, 1, 2, 4, 6, 16]))
    hi = int(np.exp(rng.uniform(0, np.log(1800))))
    check_decode(fa, list(rng.integers(0, hi + 1, B)), Hkv * group, Hkv, int(rng.integers(1, 9)),
                 int(rng.choice([64, 128, 256])), ps, block, FORMATS[seed % 3],
                 window=int(rng.choice([0, 0, rng.integers(1, hi + 2), 2 ** 31 - 1])), seed=seed)


def test_caches_beyond_32_bit_offsets(fa):
    """Pages whose bytes start past 2^32 in caches of 5 GB: rows appended there, then read."""
    pages, Hkv, ps, d = 41000, 8, 128, 128
    rng = np.random.default_rng(24)
    kc, vc = (torch.empty((pages, Hkv, ps, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((pages, Hkv, 1), device="cuda") for _ in range(2))
    own = np.array([pages - 1, 33000, 3, pages - 2], np.int32)
    L = 4 * ps - 5
    slots = own[np.arange(L) // ps].astype(np.int64) * ps + np.arange(L) % ps
    k, v = rows_of(rng, L, Hkv, d), rows_of(rng, L, Hkv, d)
    fa.attn_cache_append_fp8(k.cuda(), v.cuda(), kc, vc, ks, vs, cuda(slots))
    small = [np.zeros((4, Hkv, ps, d), np.uint8), np.zeros((4, Hkv, ps, d), np.uint8),
             np.zeros((4, Hkv, 1), np.float32), np.zeros((4, Hkv, 1), np.float32)]
    ref.append_fp8(k.float().numpy(), small[0], small[2], np.arange(L), "e4m3")
    ref.append_fp8(v.float().numpy(), small[1], small[3], np.arange(L), "e4m3")
    at = torch.from_numpy(own).long().cuda()
    for got, want in zip((ks, vs), small[2:]):
        np.testing.assert_array_equal(got[at].cpu().numpy(), want)
    for got, want in zip((kc, vc), small):
        got = got[at].transpose(1, 2).reshape(4 * ps, Hkv, d)[:L].cpu().numpy()
        np.testing.assert_array_equal(got, want.transpose(0, 2, 1, 3).reshape(4 * ps, Hkv, d)[:L])
    q = torch.from_numpy(rng.standard_normal((1, 16, 1, d)).astype(np.float32)).bfloat16()
    o, lse = fa.attn_decode_fp8_paged(q.cuda(), kc, vc, ks, vs, cuda(own[None]), cuda(np.array([L], np.int32)), scale=0.1)
    table = np.arange(4, dtype=np.int32)[None]
    compare_decode(o, lse, ref.decode_fp8(q.double().numpy(), small[0], small[1], small[2], small[3], table, [L], "e4m3", 0.1))
    del kc, vc
    kb, vb = (torch.empty((pages, Hkv, ps, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.attn_cache_append_bf16(k.cuda(), v.cuda(), kb, vb, cuda(slots))
    for got, want in ((kb, k), (vb, v)):
        assert torch.equal(got[at].transpose(1, 2).reshape(4 * ps, Hkv, d)[:L].cpu(), want)


def test_a_slot_named_twice_stays_in_its_block(fa):
    """Tokens that name one block out of order leave that block unspecified and no other."""
    rng = np.random.default_rng(25)
    slots = np.array([5, 5, 5, 40, 41, 2, 7, 70, -1, 71], np.int64)
    H, d, ps = 2, 64, 32
    k, v = rows_of(rng, len(slots), H, d), rows_of(rng, len(slots), H, d)
    codes = [rng.integers(0, 100, (4, H, ps, d)).astype(np.uint8) for _ in range(2)]
    scales = [np.full((4, H, 1), 0.01, np.float32) for _ in range(2)]
    dev = [cuda(a) for a in codes + scales]
    fa.attn_cache_append_fp8(k.cuda(), v.cuda(), *dev, cuda(slots))
    torch.cuda.synchronize()
    for x, c, s in ((k, codes[0], scales[0]), (v, codes[1], scales[1])):
        ref.append_fp8(x.float().numpy(), c, s, slots, "e4m3")
    # block 0 is named out of order and block 2 (70, -1, 71) with a gap: neither's tokens are
    # consecutive, so both are unspecified
    for got, want in zip(dev, codes + scales):
        np.testing.assert_array_equal(got.cpu().numpy()[1::2], want[1::2])
    kb = torch.zeros(4, H, ps, d, dtype=torch.bfloat16, device="cuda")
    vb = torch.zeros_like(kb)
    fa.attn_cache_append_bf16(k.cuda(), v.cuda(), kb, vb, cuda(slots))
    row = kb[0, :, 5].cpu()
    assert any(torch.equal(row[0], k[i, 0]) for i in range(3)) and torch.equal(kb[1, :, 8].cpu(), k[3])


def test_decode_fp8_workspace_and_outputs(fa):
    """A workspace of exactly the bytes asked for, whatever it holds; a smaller one is refused;
    given outputs are the ones returned."""
    rng = np.random.default_rng(26)
    lens, Hkv, d = [3000, 0, 700], 2, 128
    kc, vc, ks, vs, table = ref.make_cache(rng, lens, Hkv, d, 64, 64, "e4m3")
    args = [torch.randn(3, 8, 2, d).bfloat16().cuda()] + [cuda(a) for a in (kc, vc, ks, vs, table, np.array(lens, np.int32))]
    want = fa.attn_decode_fp8_paged(*args)
    need = fa.attn_decode_fp8_workspace_bytes(8, Hkv, 2, d)
    for fill in (float("nan"), 0.0, 1e30):
        ws = torch.full((need // 4,), fill, device="cuda")
        o, lse = torch.full_like(want[0], 7), torch.full_like(want[1], 7)
        got = fa.attn_decode_fp8_paged(*args, workspace=ws, o=o, lse=lse)
        assert got[0] is o and got[1] is lse
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(fa.AttnError):
        fa.attn_decode_fp8_paged(*args, workspace=torch.empty(need // 4 - 4, device="cuda"))
    assert fa.attn_get_device_status() == fa.ATTN_OK


def test_append_of_nothing(fa):
    x = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    c, s = torch.full((2, 2, 16, 64), 9, dtype=torch.uint8, device="cuda"), torch.ones(2, 2, 1, device="cuda")
    fa.attn_cache_append_fp8(x, x, c, c, s, s, none)
    fa.attn_cache_append_bf16(x, x, c.bfloat16(), c.bfloat16(), none)
    gone = torch.full((3,), -1, dtype=torch.int64, device="cuda")
    fa.attn_cache_append_fp8(torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda"),
                             torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda"), c, c, s, s, gone)
    torch.cuda.synchronize()
    assert (c == 9).all() and (s == 1).all()


@pytest.mark.parametrize("qmul", [0.0, 1e-30, 1e-4, 300.0, 1e30])
@pytest.mark.parametrize("wide", [False, True])
def test_decode_fp8_query_magnitudes(fa, qmul, wide):
    """Queries far outside fp16's range keep their scores (softmax scale chosen to match)."""
    check_decode(fa, [100, 17], 48 if wide else 4, 2, 2, 128, 32, 32, "e4m3", qmul=qmul, seed=14,
                 scale=0.1 / max(qmul, 1e-30) if qmul else 0.1, wide=wide)


@pytest.mark.parametrize("H", [4, 40])
def test_decode_fp8_query_rows_of_mixed_magnitude(fa, H):
    """Within a row: values down to 2^-20 of the row's largest still count."""
    rng = np.random.default_rng(15)
    d, lens = 128, [200]
    kc, vc, ks, vs, table = ref.make_cache(rng, lens, 1, d, 32, 32, "e4m3")
    if H > 16:
        table = widen(table, 32)
    q = rng.standard_normal((1, H, 1, d)).astype(np.float32)
    q[..., 1:] *= np.exp2(-rng.integers(0, 21, d - 1)).astype(np.float32)
    q = torch.from_numpy(q).bfloat16()
    o, lse = fa.attn_decode_fp8_paged(q.cuda(), cuda(kc), cuda(vc), cuda(ks), cuda(vs), cuda(table),
                                      cuda(np.array(lens, np.int32)), scale=0.3)
    compare_decode(o, lse, ref.decode_fp8(q.double().numpy(), kc, vc, ks, vs, table, lens, "e4m3", 0.3))


@pytest.mark.parametrize("H", [4, 40, 200])
def test_decode_fp8_scales_far_apart(fa, H):
    """Blocks whose scales lie 2^40 apart, zero scales among them, in K and in V."""
    rng = np.random.default_rng(16)
    d, lens, fmt = 64, [300, 70], "e4m3"
    kc, vc, ks, vs, table = ref.make_cache(rng, lens, 2, d, 32, 16, fmt)
    if H > 16:
        table = widen(table, 32)
    ks[:], vs[:] = np.nan_to_num(ks, nan=0.01), np.nan_to_num(vs, nan=0.01)
    vs *= np.exp2(rng.integers(-20, 21, vs.shape)).astype(np.float32)
    vs[rng.random(vs.shape) < 0.2] = 0
    ks[rng.random(ks.shape) < 0.2] = 0
    q = torch.from_numpy(rng.standard_normal((2, H, 1, d)).astype(np.float32)).bfloat16()
    o, lse = fa.attn_decode_fp8_paged(q.cuda(), cuda(kc), cuda(vc), cuda(ks), cuda(vs), cuda(table),
                                      cuda(np.array(lens, np.int32)), scale=0.125)
    compare_decode(o, lse, ref.decode_fp8(q.double().numpy(), kc, vc, ks, vs, table, lens, fmt, 0.125))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [2, 10, 20, 40])
def test_decode_fp8_nan_at_a_key_only_later_queries_see(fa, fmt, d, H):
    """A NaN value at the newest token reaches the last query alone (and there only its own
    coordinate); a NaN key reaches every query that sees it."""
    rng = np.random.default_rng(17)
    lens, nq, ps = [70, 64], 3, 32
    kc, vc, ks, vs, table = ref.make_cache(rng, lens, 1, d, ps, 32, fmt)
    if H > 2:
        table = widen(table, ps)
    clean = (vc.copy(), kc.copy())
    for b, L in enumerate(lens):
        vc[table[b, (L - 1) // ps], 0, (L - 1) % ps, 7] = 0x7F
    kc[table[1, (lens[1] - 2) // ps], 0, (lens[1] - 2) % ps, 3] = 0xFF
    q = torch.from_numpy(rng.standard_normal((2, H, nq, d)).astype(np.float32)).bfloat16()
    o, lse = fa.attn_decode_fp8_paged(q.cuda(), cuda(kc), cuda(vc), cuda(ks), cuda(vs), cuda(table),
                                      cuda(np.array(lens, np.int32)), fmt=fmt, scale=0.1)
    want = ref.decode_fp8(q.double().numpy(), clean[1], clean[0], ks, vs, table, lens, fmt, 0.1)
    o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
    nan = np.zeros(o.shape, bool)
    nan[0, :, 2, 7] = True
    nan[1, :, 1:] = True
    assert (np.isnan(o) == nan).all()
    assert (np.abs(o - want[0]) <= want[2])[~nan].all()
    seen = np.zeros(lse.shape, bool)
    seen[1, :, 1:] = True
    assert (np.isnan(lse) == seen).all() and (np.abs(lse - want[1]) <= want[3])[~seen].all()


def test_decode_fp8_bad_page_numbers_stay_inside(fa):
    """Page numbers far outside the cache and lengths beyond the table are clamped: values
    are then unspecified, the call finishes, and later calls are right."""
    rng = np.random.default_rng(18)
    kc, vc, ks, vs, table = ref.make_cache(rng, [100, 40], 2, 64, 32, 32, "e4m3")
    bad = table.copy()
    bad[0, 1], bad[1, 0] = 2 ** 31 - 1, -2 ** 31
    q = torch.randn(2, 2, 1, 64).bfloat16().cuda()
    dev = [cuda(a) for a in (kc, vc, ks, vs)]
    fa.attn_decode_fp8_paged(q, *dev, cuda(bad), cuda(np.array([2 ** 31 - 1, -7], np.int32)))
    assert fa.attn_get_device_status() == fa.ATTN_OK
    check_decode(fa, [100, 40], 2, 2, 1, 64, 32, 32, "e4m3", seed=19)


@pytest.mark.parametrize("withheld", [0, 3])
@pytest.mark.parametrize("d,group,nq", [(64, 1, 1), (128, 8, 1), (128, 16, 1), (256, 1, 2),     # narrow
                                        (64, 8, 4), (128, 8, 4), (128, 8, 8), (256, 16, 8)])    # wide
@pytest.mark.parametrize("B,L", [(5, 8000), (70, 1000)])       # fewer units than CTAs, and more
def test_decode_fp8_kernels_abort_on_a_withheld_load(fa, B, L, d, group, nq, withheld):
    """One load of every CTA is never issued: the bounded waits on it run out, the status says
    so, the joining kernel stays inside whatever the workspace held, and the next call is
    right."""
    g = torch.Generator(device="cuda").manual_seed(withheld + d)
    Hkv, ps = 8, 64
    width = -(-L // ps)
    kc, vc = (torch.randint(0, 0x78, (B * width, Hkv, ps, d), dtype=torch.uint8, device="cuda", generator=g) for _ in range(2))
    ks, vs = (torch.rand(B * width, Hkv, 1, device="cuda", generator=g) * 0.01 for _ in range(2))
    table = torch.randperm(B * width, device="cuda", generator=g).to(torch.int32).view(B, width)
    if group * nq > 16:
        table = cuda(widen(table.cpu().numpy(), ps))
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    lens[B // 2] = 0
    q = torch.randn(B, group * Hkv, nq, d, device="cuda", generator=g).bfloat16()
    o1, lse1 = fa.attn_decode_fp8_paged(q, kc, vc, ks, vs, table, lens)
    assert fa.attn_get_device_status() == fa.ATTN_OK
    need = fa.attn_decode_fp8_workspace_bytes(group * Hkv, Hkv, nq, d)
    ws = torch.randint(0, 6, (need // 4,), dtype=torch.int32, device="cuda", generator=g)
    ws[::5] = torch.randint(-2 ** 31, 2 ** 31 - 1, ws[::5].shape, dtype=torch.int32, device="cuda", generator=g)
    fa.attn_selftest_decode_fp8_withheld_load(q, kc, vc, ks, vs, table, lens, torch.empty_like(o1),
                                              torch.empty_like(lse1), ws, withheld=withheld)
    assert fa.attn_get_device_status() == fa.ATTN_ERR_TIMEOUT
    o2, lse2 = fa.attn_decode_fp8_paged(q, kc, vc, ks, vs, table, lens)
    assert fa.attn_get_device_status() == fa.ATTN_OK
    assert torch.equal(o1, o2) and torch.equal(lse1, lse2)


# ------------------------------------------------------------------ together
def serve(fa, fmt, steps, seed=0, graph=False):
    """A small serving loop: a prefill step, then decoding steps; returns the outputs of every
    step, the cache, and the keys and values that went in."""
    rng = np.random.default_rng(seed)
    B, H, Hkv, d, ps, block, pages, width = 5, 8, 2, 128, 32, 16, 64, 8
    st = dict(seq=cuda(np.zeros(B, np.int32)), table=cuda(np.full((B, width), -1, np.int32)),
              stack=cuda(rng.permutation(pages).astype(np.int32)), count=cuda(np.array([pages], np.int32)))
    kc, vc = (torch.full((pages, Hkv, ps, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, Hkv, ps // block), float("nan"), device="cuda") for _ in range(2))
    history, outs = [[] for _ in range(B)], []
    for step in range(steps):
        new = np.array([70, 1, 33, 0, 128] if step == 0 else [1, 1, 1, 1, 1], np.int32)
        T = int(new.sum()) + 2
        k, v = rows_of(rng, T, Hkv, d), rows_of(rng, T, Hkv, d)
        q = torch.from_numpy(rng.standard_normal((B, H, 1, d)).astype(np.float32)).bfloat16()
        seq, count, cu, slots, pos, served = fa.attn_paged_plan(
            cuda(new), st["seq"], st["table"], st["stack"], st["count"], ps, T,
            seq_lens_out=st["seq"], free_count_out=st["count"])
        fa.attn_cache_append_fp8(k.cuda(), v.cuda(), kc, vc, ks, vs, slots, fmt=fmt)
        outs.append((q, *fa.attn_decode_fp8_paged(q.cuda(), kc, vc, ks, vs, st["table"], seq, fmt=fmt), seq.cpu()))
        row = 0
        for b in range(B):
            history[b] += [(k[row + j], v[row + j]) for j in range(new[b])]
            row += new[b]
        assert served.all()
    torch.cuda.synchronize()
    return st, (kc, vc, ks, vs), outs, history


@pytest.mark.parametrize("fmt", FORMATS)
def test_serving_loop(fa, fmt):
    """Plan, append and decode as they are used together: the last step against attention over
    the cache's own values, and those values against the keys and values that went in, off by
    at most half a step of the format per rewriting of a block."""
    steps = 20
    st, cache, outs, history = serve(fa, fmt, steps)
    kc, vc, ks, vs = (t.cpu().numpy() for t in cache)
    table = st["table"].cpu().numpy()
    q, o, lse, seq = outs[-1]
    lens = seq.numpy()
    assert lens.tolist() == [70 + 19, 1 + 19, 33 + 19, 19, 128 + 19]
    compare_decode(o, lse, ref.decode_fp8(q.double().numpy(), kc, vc, ks, vs, table, lens, fmt, 1 / math.sqrt(128)))
    half = 2.0 ** -3 if fmt == "e5m2" else 2.0 ** -4       # half a step relative to the value
    least = 2.0 ** -17 if fmt == "e5m2" else 2.0 ** -10    # and below the normal numbers
    for b, L in enumerate(lens):
        t = np.arange(L)
        page, row = table[b, t // 32], t % 32
        for codes, s, which in ((kc, ks, 0), (vc, vs, 1)):
            got = ref.decode(codes[page, :, row], fmt) * s[page, :, row // 16][..., None]
            x = np.stack([h[which].float().numpy() for h in history[b]])
            sc = s[page, :, row // 16][..., None]
            assert (np.abs(got - x) <= 16 * (half * np.abs(x) + least * sc)).all()


def test_serving_step_in_a_graph(fa):
    """One captured step (plan, append, decode, all in place) replayed token after token gives
    what the same steps give eagerly, and a second graph may share its buffers when they are
    replayed in turn."""
    B, H, Hkv, d, ps, pages, width = 6, 4, 2, 64, 16, 80, 12

    def fresh():
        rng = np.random.default_rng(21)
        return dict(new=cuda(np.array([1, 1, 0, 1, 1, 1], np.int32)), seq=cuda(rng.integers(0, 40, B).astype(np.int32)),
                    table=cuda(np.arange(B * width, dtype=np.int32).reshape(B, width) % 40),
                    stack=cuda((40 + rng.permutation(40)).astype(np.int32)), count=cuda(np.array([40], np.int32)),
                    kc=torch.full((pages, Hkv, ps, d), 0x20, dtype=torch.uint8, device="cuda"),
                    vc=torch.full((pages, Hkv, ps, d), 0x21, dtype=torch.uint8, device="cuda"),
                    ks=torch.full((pages, Hkv, 1), 0.01, device="cuda"), vs=torch.full((pages, Hkv, 1), 0.02, device="cuda"),
                    k=torch.zeros(B, Hkv, d, dtype=torch.bfloat16, device="cuda"),
                    v=torch.zeros(B, Hkv, d, dtype=torch.bfloat16, device="cuda"),
                    q=torch.zeros(B, H, 1, d, dtype=torch.bfloat16, device="cuda"),
                    o=torch.zeros(B, H, 1, d, dtype=torch.bfloat16, device="cuda"),
                    lse=torch.zeros(B, H, 1, device="cuda"),
                    ws=torch.empty(max(4, fa.attn_decode_fp8_workspace_bytes(H, Hkv, 1, d) // 4), device="cuda"))

    def step(s):
        out = fa.attn_paged_plan(s["new"], s["seq"], s["table"], s["stack"], s["count"], ps, B,
                                 seq_lens_out=s["seq"], free_count_out=s["count"])
        fa.attn_cache_append_fp8(s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], out[3])
        fa.attn_decode_fp8_paged(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["seq"], workspace=s["ws"],
                                 o=s["o"], lse=s["lse"])

    gen = torch.Generator().manual_seed(5)
    inputs = [[torch.randn(t, generator=gen).bfloat16().cuda() for t in ((B, Hkv, d), (B, Hkv, d), (B, H, 1, d))]
              for _ in range(12)]
    eager, want = fresh(), []
    for kvq in inputs:
        for n, t in zip(("k", "v", "q"), kvq):
            eager[n].copy_(t)
        step(eager)
        want.append((eager["o"].clone(), eager["lse"].clone()))
    s = fresh()
    warm = fresh()
    step(warm)                                   # first calls outside capture
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s)
        graphs.append(g)
    for i, kvq in enumerate(inputs):
        for n, t in zip(("k", "v", "q"), kvq):
            s[n].copy_(t)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(s["o"], want[i][0]) and torch.equal(s["lse"], want[i][1]), i
    for n in ("kc", "vc", "ks", "vs", "seq", "table", "count"):
        assert torch.equal(s[n], eager[n]), n
    assert fa.attn_get_device_status() == fa.ATTN_OK


def test_calls_on_other_streams(fa):
    """Concurrent streams, each with its own workspace, give the sequential results; a call
    takes the stream it is given."""
    rng = np.random.default_rng(22)
    cases = []
    for seed, (H, Hkv, d) in enumerate([(4, 2, 64), (8, 1, 128), (3, 3, 256), (40, 1, 128)]):
        lens = [3000, 17, 900]
        kc, vc, ks, vs, table = ref.make_cache(rng, lens, Hkv, d, 32, 32, "e4m3")
        if H > 16:
            table = widen(table, 32)
        q = torch.randn(3, H, 1, d, generator=torch.Generator().manual_seed(seed)).bfloat16()
        cases.append([t.cuda() if isinstance(t, torch.Tensor) else cuda(t)
                      for t in (q, kc, vc, ks, vs, table, np.array(lens, np.int32))])
    want = [fa.attn_decode_fp8_paged(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [torch.empty(max(4, fa.attn_decode_fp8_workspace_bytes(c[0].shape[1], c[1].shape[1], 1, c[0].shape[3]) // 4),
                      device="cuda") for c in cases]
    for _ in range(3):
        got = [fa.attn_decode_fp8_paged(*c, workspace=w, stream=s) for c, w, s in zip(cases, ws, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_fp8_kernels_side_by_side(fa):
    """Narrow and wide kernels of several head sizes on streams of their own, in flight together,
    give what each gives alone; so do two calls of one kind."""
    rng = np.random.default_rng(90)
    calls = []
    for d, H, nq, wide in ((64, 32, 4, True), (128, 16, 4, True), (128, 16, 4, True), (256, 32, 8, True),
                           (128, 8, 1, False), (64, 2, 8, False), (256, 8, 1, False), (128, 8, 1, False)):
        lens = [int(n) for n in rng.integers(1, 6000, 12)]
        kc, vc, ks, vs, table = ref.make_cache(rng, lens, 2, d, 64, 64, "e4m3", stale=False)
        if wide:
            table = widen(table, 64)
        q = torch.from_numpy(rng.standard_normal((len(lens), H, nq, d)).astype(np.float32)).bfloat16().cuda()
        calls.append((q, *(cuda(a) for a in (kc, vc, ks, vs, table, np.array(lens, np.int32)))))
    alone = [fa.attn_decode_fp8_paged(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        got = [fa.attn_decode_fp8_paged(*c, stream=st) for c, st in zip(calls, streams) for _ in range(2)]
        torch.cuda.synchronize()
        for i, (o, lse) in enumerate(got):
            assert torch.equal(o, alone[i // 2][0]) and torch.equal(lse, alone[i // 2][1])
    assert fa.attn_get_device_status() == fa.ATTN_OK


def test_workspace_belongs_to_the_calls_stream(fa):
    """Calls on a given stream without a workspace, while the current stream allocates and
    overwrites blocks of the same sizes: nobody else gets a workspace that is in use."""
    rng = np.random.default_rng(23)
    lens, Hkv, d = [30000, 5], 2, 128
    kc, vc, ks, vs, table = ref.make_cache(rng, lens, Hkv, d, 64, 64, "e4m3")
    q = torch.randn(2, 8, 1, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    args = [q.cuda()] + [cuda(a) for a in (kc, vc, ks, vs, table, np.array(lens, np.int32))]
    want = fa.attn_decode_fp8_paged(*args)
    torch.cuda.synchronize()
    nbytes = fa.attn_decode_fp8_workspace_bytes(8, Hkv, 1, d)
    s = torch.cuda.Stream()
    outs = []
    for _ in range(30):
        outs.append(fa.attn_decode_fp8_paged(*args, stream=s))
        for _ in range(3):
            torch.empty(nbytes // 4, device="cuda").fill_(float("nan"))
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_refusals(fa):
    """What the binding refuses on the device: types, shapes, a cache of the other format."""
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(5, 2, 32, 64, dtype=torch.uint8, device="cuda")
    s = torch.zeros(5, 2, 2, device="cuda")
    table, lens = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    ok = [q, c, c, s, s, table, lens]
    fa.attn_decode_fp8_paged(*ok)
    for i, t in ((0, q.float()), (0, q.transpose(1, 2)), (1, c[:, :1]), (1, c.view(torch.float8_e5m2)), (3, s[:, :, :1]),
                 (4, s.double()), (5, table.long()), (5, table[:1]), (6, lens[:1]), (6, lens.cpu())):
        bad = list(ok)
        bad[i] = t
        with pytest.raises((TypeError, ValueError, fa.AttnError)):   # AttnError: [2, 1, 4, 64] has 1 head over 2
            fa.attn_decode_fp8_paged(*bad)
    with pytest.raises(ValueError):
        fa.attn_decode_fp8_paged(*ok, fmt="int8")
    with pytest.raises(fa.AttnError):
        fa.attn_decode_fp8_paged(q[:, :3].contiguous(), *ok[1:])             # 3 heads over 2
    x, slots = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        fa.attn_cache_append_fp8(x.transpose(0, 1), x.transpose(0, 1), c, c, s, s, slots[:2])
    with pytest.raises(TypeError):
        fa.attn_cache_append_fp8(x, x, c, c, s, s, slots.int())
    with pytest.raises(fa.AttnError):
        fa.attn_cache_append_fp8(x[:1].expand(3, 2, 64), x, c, c, s, s, slots)  # tokens that overlap
    with pytest.raises(TypeError):
        fa.attn_cache_append_bf16(x, x, c, c, slots)
    with pytest.raises(TypeError):
        fa.attn_paged_plan(lens.long(), lens, table, lens, lens[:1], 16, 4)
    assert fa.attn_get_device_status() == fa.ATTN_OK
