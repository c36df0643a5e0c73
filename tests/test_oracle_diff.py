"""The 64-bit reference of differential attention and rotary positions against automatic differentiation and
against differences."""
import math

import pytest
import torch

from tests import diff_reference as ref


def problem(H, Hkv, n, d, seed):
    gen = torch.Generator().manual_seed(seed)
    shapes = [(2 * H, n, d), (2 * Hkv, n, d), (Hkv, n, 2 * d), (H,), (H, n, 2 * d)]
    return [torch.randn(*s, generator=gen, dtype=torch.float64) for s in shapes]


@pytest.mark.parametrize("H,Hkv,causal,window", [(1, 1, True, 0), (4, 2, True, 3), (3, 1, False, 0), (2, 2, False, 2)])
def test_gradients(H, Hkv, causal, window):
    q, k, v, lam, g = problem(H, Hkv, 9, 4, H)
    scale, ok = 0.5, ref.allowed(9, causal, window)
    leaves = [t.clone().requires_grad_() for t in (q, k, v, lam)]
    w = ref.forward(*leaves, scale, ok)
    auto = torch.autograd.grad((w["o"] * g).sum(), leaves)
    formula, _ = ref.backward(q, k, v, lam, w["o"].detach(), w["o2"].detach(), g, w["lse"].detach(), scale, ok)
    for a, b in zip(auto, formula):
        assert torch.allclose(a, b, rtol=1e-10, atol=1e-12)
    # and by central differences along random directions
    gen = torch.Generator().manual_seed(7)
    for i, t in enumerate((q, k, v, lam)):
        step = torch.randn(t.shape, generator=gen, dtype=torch.float64)
        at = [x.clone() for x in (q, k, v, lam)]
        value = []
        for sign in (1, -1):
            at[i] = t + sign * 1e-6 * step
            value.append((ref.forward(*at, scale, ok)["o"] * g).sum())
        assert math.isclose((value[0] - value[1]).item() / 2e-6, (formula[i] * step).sum().item(), rel_tol=1e-6, abs_tol=1e-7)


def test_difference_of_two_softmaxes():
    q, k, v, lam, _ = problem(2, 1, 6, 4, 11)
    w = ref.forward(q, k, v, lam, 0.3, ref.allowed(6, True, 0))
    for h in range(2):
        maps = [torch.softmax((q[2 * h + m] @ k[m].t() * 0.3).masked_fill(~ref.allowed(6, True, 0), -math.inf), 1)
                for m in range(2)]
        assert torch.allclose(w["o"][h], (maps[0] - lam[h] * maps[1]) @ v[0], atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(interleaved):
    """A rotation: lengths of pairs are kept, the inverse undoes it, and positions add up."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(2, 5, 16, generator=gen, dtype=torch.float64)
    freq, axis = torch.rand(6, generator=gen), torch.tensor([0, 1, 0, 1, 1, 0])
    pos = torch.tensor([[0, 3, 10, 2, 7], [4, -2, 0, 9, 1]])
    y = ref.rope(x, pos, freq, axis, interleaved)
    assert torch.allclose(ref.rope(y, pos, freq, axis, interleaved, True), x, atol=1e-12)
    assert torch.equal(y[..., 12:], x[..., 12:])
    assert torch.allclose(y.pow(2).sum(-1), x.pow(2).sum(-1))
    twice = ref.rope(y, pos, freq, axis, interleaved)
    assert torch.allclose(twice, ref.rope(x, 2 * pos, freq, axis, interleaved), atol=1e-12)
    pos[0, 2] = -1
    assert torch.equal(ref.rope(x, pos, freq, axis, interleaved)[:, 2], x[:, 2])
