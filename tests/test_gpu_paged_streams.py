"""GPU: outputs of paged-cache calls on a given stream, read and dropped on the current one."""
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


def test_a_dropped_output_is_not_written_while_the_current_stream_reads_it(fa):
    """Each call's O is read on the current stream, which is busy for a while, and dropped at once;
    the next call on the side stream, which waits for nobody, must not be given its memory."""
    rng = np.random.default_rng(41)
    lens = [200, 37, 90, 1]
    kc, vc, ks, vs, table = ref.make_cache(rng, lens, 2, 128, 64, 64, "e4m3")
    cache = [cuda(a) for a in (kc, vc, ks, vs, table, np.array(lens, np.int32))]
    qs = [torch.randn(4, 8, 1, 128, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(8)]
    want = [fa.attn_decode_fp8_paged(q, *cache) for q in qs]
    torch.cuda.synchronize()
    side, current, kept, places = torch.cuda.Stream(), torch.cuda.current_stream(), [], []
    for q in qs:
        o, lse = fa.attn_decode_fp8_paged(q, *cache, stream=side)
        places.append((o.data_ptr(), lse.data_ptr()))
        current.wait_stream(side)
        torch.cuda._sleep(20_000_000)                    # about 10 ms
        kept.append((o.clone(), lse.clone()))
        del o, lse
    torch.cuda.synchronize()
    assert len({p for pair in places for p in pair}) == 2 * len(qs)
    for a, b in zip(kept, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    del kept
    assert fa.attn_get_device_status() == fa.ATTN_OK


def test_a_dropped_plan_is_not_written_while_the_current_stream_reads_it(fa):
    i32 = dict(dtype=torch.int32, device="cuda")
    new = [torch.full((3,), n, **i32) for n in range(1, 7)]
    lens, stack, count = torch.zeros(3, **i32), torch.arange(30, **i32), torch.tensor([30], **i32)
    table = torch.full((3, 4), -1, **i32)
    want = [fa.attn_paged_plan(n, lens, table, stack, count, 16, 20) for n in new]
    torch.cuda.synchronize()
    side, current, kept, places = torch.cuda.Stream(), torch.cuda.current_stream(), [], []
    for n in new:
        out = fa.attn_paged_plan(n, lens, table, stack, count, 16, 20, stream=side)
        places.append(out[0].data_ptr())
        current.wait_stream(side)
        torch.cuda._sleep(20_000_000)
        kept.append([t.clone() for t in out])
        del out
    torch.cuda.synchronize()
    assert len(set(places)) == len(new)
    for a, b in zip(kept, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_outputs_on_the_current_stream_are_used_again(fa):
    """Without a given stream, or with the current one given, a dropped output's memory is the
    next call's, as for any tensor of that stream."""
    rng = np.random.default_rng(42)
    kc, vc, ks, vs, table = ref.make_cache(rng, [300], 1, 64, 64, 64, "e4m3")
    args = [torch.randn(1, 4, 1, 64).bfloat16().cuda()] + [cuda(a) for a in (kc, vc, ks, vs, table, np.array([300], np.int32))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for kw in ({}, {"stream": side}):
            places = set()
            for _ in range(10):
                o, lse = fa.attn_decode_fp8_paged(*args, **kw)
                places.add((o.data_ptr(), lse.data_ptr()))
                del o, lse
            assert len(places) <= 2
    torch.cuda.synchronize()
