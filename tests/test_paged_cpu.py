"""CPU checks of the paged-cache operators: arguments the C entry points and the binding
refuse before any launch, and the plain implementations the GPU tests compare with."""
import numpy as np
import pytest
import torch

import oracle
from tests import paged_reference as ref

P = 0x10000  # an aligned fake device address; no call below reaches the GPU


@pytest.fixture(scope="module")
def lib():
    from exact_attention_55_gb300 import build
    path = build.build()
    import exact_attention_55_gb300 as fa
    return fa.load_library(path)


@pytest.mark.parametrize("change,expected", [
    ({0: 0}, 1), ({1: 0}, 1), ({2: 0}, 1), ({3: 0}, 1), ({4: 0}, 1), ({5: 0}, 1), ({6: 0}, 1),
    ({7: 0}, 1), ({8: 0}, 1), ({9: 0}, 1), ({10: 0}, 1),      # null pointers
    ({11: 0}, 1), ({13: 0}, 1), ({14: -1}, 1), ({15: -1}, 1),  # B, max_pages, capacity, tokens
    ({11: 16385}, 2),                                          # too many requests
    ({12: 48}, 2), ({12: 0}, 2), ({12: 131072}, 2),            # page size
    ({12: 65536, 13: 32768}, 2),                               # 2^31 positions
    ({8: P + 4}, 3), ({0: P + 2}, 3),                          # alignment
])
def test_plan_argument_errors(lib, change, expected):
    args = [P] * 11 + [4, 64, 8, 100, 32]
    for i, v in change.items():
        args[i] = v
    assert lib.attn_paged_plan(*args, None) == expected


@pytest.mark.parametrize("change,expected", [
    ({0: 0}, 1), ({2: 0}, 1), ({4: 0}, 1),           # null pointers
    ({5: -1}, 1), ({6: 0}, 1), ({11: 0}, 1),         # T, Hkv, num_pages
    ({5: 0}, 0),                                     # no tokens: nothing to do
    ({7: 96}, 2), ({10: 24}, 2), ({6: 65536}, 2),    # d, page size, heads
    ({8: 1000}, 1),                                  # a token stride shorter than a token
    ({8: 1028}, 3), ({0: P + 8}, 3), ({4: P + 4}, 3),
    ({11: 1 << 29}, 2),                              # pages * heads beyond 31 bits
])
def test_append_argument_errors(lib, change, expected):
    # k, v, k_cache, v_cache, slot_map, T, Hkv, d, k_stride, v_stride, page_size, num_pages
    args = [P] * 5 + [7, 8, 128, 1024, 1024, 64, 100]
    for i, v in change.items():
        args[i] = v
    assert lib.attn_cache_append_bf16(*args, None) == expected
    args[5:5] = [P, P]                               # the 8-bit form: scales before slot_map
    args[4], args[6] = args[6], args[4]
    assert lib.attn_cache_append_fp8(*args, 64, 0, None) == expected


@pytest.mark.parametrize("page,block,fmt,scales,expected", [
    (64, 128, 0, P, 2), (64, 48, 0, P, 2), (64, 8, 0, P, 2), (8, 8, 0, P, 2),
    (64, 64, 3, P, 1), (64, 64, -1, P, 1), (64, 64, 0, 0, 1), (64, 64, 0, P + 2, 3),
])
def test_append_fp8_argument_errors(lib, page, block, fmt, scales, expected):
    args = [P, P, P, P, scales, P, P, 7, 8, 128, 1024, 1024, page, 100, block, fmt]
    assert lib.attn_cache_append_fp8(*args, None) == expected


DECODE = [P] * 9 + [2, 8, 4, 1, 128, 64, 100, 16, 64, 0, 0.1, 0, P, 1 << 30]


@pytest.mark.parametrize("change,expected", [
    ({i: 0}, 1) for i in range(9)] + [
    ({9: 0}, 1), ({10: 6}, 1), ({11: 0}, 1), ({12: 0}, 1),     # B; H % Hkv; Hkv; nq
    ({12: 9}, 2), ({13: 96}, 2), ({14: 8}, 2), ({14: 48}, 2),  # nq, d, page size
    ({17: 128}, 2), ({17: 8}, 2), ({18: 3}, 1),                # block, format
    ({19: 0.0}, 1), ({19: float("nan")}, 1), ({19: float("inf")}, 1),
    ({16: 1 << 26}, 2), ({15: 1 << 30}, 2),                    # positions, pages * heads
    ({0: P + 8}, 3), ({8: P + 2}, 3), ({3: P + 1}, 3), ({21: P + 8}, 3),
])
def test_decode_fp8_argument_errors(lib, change, expected):
    args = list(DECODE)
    for i, v in change.items():
        args[i] = v
    assert lib.attn_decode_fp8_paged(*args, None) == expected


@pytest.mark.parametrize("withheld,limit,expected", [(-1, 10 ** 6, 1), (0, 0, 1), (0, 3 * 10 ** 9, 1)])
def test_decode_fp8_selftest_argument_errors(lib, withheld, limit, expected):
    args = DECODE[:19] + DECODE[21:] + [withheld, limit]
    assert lib.attn_selftest_decode_fp8_withheld_load(*args, None) == expected


def test_binding_refuses_cpu_tensors():
    import exact_attention_55_gb300 as fa
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    s = torch.zeros(4, 2, 1)
    with pytest.raises(TypeError):
        fa.attn_paged_plan(i, i, i[None], i, i[:1], 16, 4)
    with pytest.raises(TypeError):
        fa.attn_cache_append_bf16(x, x, c.bfloat16(), c.bfloat16(), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        fa.attn_cache_append_fp8(x, x, c, c, s, s, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        fa.attn_decode_fp8_paged(x[None], c, c, s, s, i[None], i[:1])


def test_reference_decode_is_the_oracles():
    """Unit scales, no window, one query head per key head: the oracle's decoding step."""
    rng = np.random.default_rng(0)
    lens, H, nq, d, ps = [5, 33, 16], 2, 3, 64, 16
    kc, vc, ks, vs, table = ref.make_cache(rng, lens, H, d, ps, 16, "e4m3", stale=False)
    ks[:], vs[:] = 1.0, 1.0
    q = rng.standard_normal((3, H, nq, d))
    o, lse, _, _ = ref.decode_fp8(q, kc, vc, ks, vs, table, lens, "e4m3", 0.01)
    ro, rl = oracle.attn_decode_paged_f64(q, ref.decode(kc, "e4m3"), ref.decode(vc, "e4m3"), table, lens, 0.01)
    np.testing.assert_allclose(o, ro, rtol=0, atol=1e-10)
    np.testing.assert_allclose(lse, rl, rtol=0, atol=1e-10)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e4m3_pow2"])
def test_reference_append_of_whole_blocks_is_the_oracles_quantiser(fmt):
    """Whole 128-token blocks written at once give the block quantiser's codes and scales."""
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((256, 2, 64)).astype(np.float32)).bfloat16().float().numpy()
    cache, scales = np.zeros((2, 2, 128, 64), np.uint8), np.full((2, 2, 1), np.nan, np.float32)
    ref.append_fp8(x, cache, scales, np.arange(256), fmt)
    x8, sc = oracle.quantize_fp8_blockwise(torch.from_numpy(x).bfloat16().permute(1, 0, 2)[None].contiguous(), 128, fmt=fmt)
    np.testing.assert_array_equal(cache.transpose(1, 0, 2, 3).reshape(1, 2, 256, 64), x8)
    np.testing.assert_array_equal(scales.transpose(1, 0, 2).reshape(1, 2, 2), sc)


def test_reference_plan_keeps_pages_apart():
    rng = np.random.default_rng(2)
    seq, new = rng.integers(0, 100, 20), rng.integers(0, 40, 20)
    table = np.arange(20 * 10, dtype=np.int32).reshape(20, 10) + 1000
    out = ref.plan(new, seq, table, np.arange(500, dtype=np.int32), 500, 16, int(new.sum()) + 3)
    slots = out["slot_map"][out["slot_map"] >= 0]
    assert len(set(slots.tolist())) == len(slots) == int(new.sum())
    assert out["served"].all() and (out["seq_lens"] == seq + new).all()
