"""GPU: a serving loop over the 8-bit paged cache against the plain operators, step by step."""
import numpy as np
import pytest
import torch

from tests import paged_reference as ref
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    require_gpu()
    import exact_attention_55_gb300 as fa
    fa.load_library()
    return fa


def cuda(a):
    return torch.from_numpy(np.array(a)).cuda()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e4m3_pow2"])
def test_a_serving_loop_holds_exactly_what_its_appends_define(fa, fmt):
    """Plan, append and decode step after step: the cache's codes and scales are those of the
    plain append over the same steps, bit for bit, and each step's O and LSE are those of
    attention over them."""
    rng = np.random.default_rng(31)
    B, H, Hkv, d, ps, block, pages, width = 5, 8, 2, 128, 32, 16, 64, 8
    seq = cuda(np.zeros(B, np.int32))
    table = cuda(np.full((B, width), -1, np.int32))
    stack, count = cuda(rng.permutation(pages).astype(np.int32)), cuda(np.array([pages], np.int32))
    caches = [torch.full((pages, Hkv, ps, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((pages, Hkv, ps // block), float("nan"), device="cuda") for _ in range(2)]
    plain = [(c.cpu().numpy().copy(), s.cpu().numpy().copy()) for c, s in zip(caches, scales)]
    grown = 0
    for step in range(20):
        new = np.array([70, 1, 33, 0, 128] if step == 0 else [1, 1, 1, 1, 1], np.int32)
        T = int(new.sum()) + 2
        rows = [torch.from_numpy((rng.standard_normal((T, Hkv, d)) * np.exp2(rng.integers(-3, 4, (T, 1, 1))))
                                 .astype(np.float32)).bfloat16() for _ in range(2)]
        q = torch.from_numpy(rng.standard_normal((B, H, 1, d)).astype(np.float32)).bfloat16()
        out = fa.attn_paged_plan(cuda(new), seq, table, stack, count, ps, T, seq_lens_out=seq, free_count_out=count)
        fa.attn_cache_append_fp8(rows[0].cuda(), rows[1].cuda(), *caches, *scales, out[3], fmt=fmt)
        o, lse = fa.attn_decode_fp8_paged(q.cuda(), *caches, *scales, table, seq, fmt=fmt)
        assert out[5].all()
        slots = out[3].cpu().numpy()
        for (codes, sc), x, got, got_s in zip(plain, rows, caches, scales):
            was = sc.copy()
            ref.append_fp8(x.float().numpy(), codes, sc, slots, fmt)
            grown += int((np.isfinite(was) & (sc > was)).sum())
            np.testing.assert_array_equal(got.cpu().numpy(), codes, err_msg=f"step {step}")
            np.testing.assert_array_equal(got_s.cpu().numpy(), sc, err_msg=f"step {step}")
        want = ref.decode_fp8(q.double().numpy(), plain[0][0], plain[1][0], plain[0][1], plain[1][1],
                              table.cpu().numpy(), seq.cpu().numpy(), fmt, 1 / np.sqrt(d))
        seen = np.isfinite(want[1])
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        assert (np.abs(o - want[0]) <= want[2]).all()
        assert (np.abs(lse[seen] - want[1][seen]) <= want[3][seen]).all() and (lse[~seen] == -np.inf).all()
    assert grown > 20                                     # steps that rewrote earlier rows are among them
