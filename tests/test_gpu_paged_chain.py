"""GPU: paged-cache calls one right behind the other, each reading what the one ahead has
just written, give what they give with the device idle in between."""
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


@pytest.mark.parametrize("d,H,nq,L", [(64, 8, 1, 200), (128, 8, 1, 200), (256, 8, 1, 200), (128, 4, 4, 3000),
                                      (128, 64, 1, 9000), (256, 32, 2, 9000)])
def test_queries_that_the_step_ahead_wrote(fa, d, H, nq, L):
    """A step's O is the next step's q, in the same two buffers by turns.  Tables of up to 384
    keys have no joining grid, so there a step's own kernel follows the step's ahead."""
    rng = np.random.default_rng(d + L)
    lens = [int(n) for n in rng.integers(1, L, 24)]
    kc, vc, ks, vs, table = ref.make_cache(rng, lens, 2, d, 64, 64, "e4m3", stale=False)
    args = [cuda(a) for a in (kc, vc, ks, vs, table, np.array(lens, np.int32))]
    first = torch.randn(len(lens), H, nq, d, generator=torch.Generator().manual_seed(d)).bfloat16().cuda()
    ws = torch.empty(fa.attn_decode_fp8_workspace_bytes(H, 2, nq, d) // 4 + 4, device="cuda")

    def chain(wait):
        a, b, lse, out = first.clone(), torch.empty_like(first), torch.empty(len(lens), H, nq, device="cuda"), []
        for step in range(12):
            fa.attn_decode_fp8_paged(a, *args, scale=0.3, workspace=ws, o=b, lse=lse)
            if wait:
                torch.cuda.synchronize()
                out.append(b.clone())
                torch.cuda.synchronize()
            a, b = b, a
        return out if wait else [a]

    want = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False)[0], want[-1])
    assert fa.attn_get_device_status() == fa.ATTN_OK
