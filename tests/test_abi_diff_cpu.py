"""CPU checks of the C ABI of rotary positions and differential attention: bad arguments are refused
before a GPU is touched, and the binding refuses tensors that are not on one."""
import ctypes

import pytest
import torch

P = 0x1000        # an aligned non-null pointer; every call below is refused before it is followed


@pytest.fixture(scope="module")
def lib():
    from exact_attention_55_gb300 import build
    path = build.build()
    import exact_attention_55_gb300 as fa
    return fa.load_library(path)


def changed(args, change):
    args = list(args)
    for i, v in change.items():
        args[i] = v
    return args


@pytest.mark.parametrize("change,expected", [
    ({8: 0}, 0),                   # no batch: nothing to do
    ({9: 0}, 0),
    ({0: 0}, 1), ({2: 0}, 1), ({4: 0}, 1), ({5: 0}, 1), ({1: 0}, 1), ({3: 0}, 1),
    ({10: 0}, 1), ({11: -1}, 1), ({14: 0}, 1), ({8: -1}, 1),
    ({12: 72}, 2), ({12: 272}, 2), ({13: 24}, 2), ({13: 80}, 2), ({13: 0}, 2), ({14: 256}, 2),
    ({8: 70000, 9: 70000}, 2), ({9: 1 << 28, 10: 1, 11: 0, 12: 256}, 2),
    ({0: P + 8}, 3), ({3: P + 2}, 3), ({4: P + 2}, 3), ({5: P + 1}, 3), ({6: P + 2}, 3),
])
def test_rope_arguments(lib, change, expected):
    strides = (ctypes.c_longlong * 12)(*([4096, 512, 64] * 4))
    # q, k, q_out, k_out, positions, inv_freq, axis, strides, B, N, Hq, Hk, d, rot, axes, interleaved, inverse
    args = [P, P, P, P, P, P, 0, ctypes.addressof(strides), 1, 8, 8, 8, 64, 64, 1, 0, 0]
    assert lib.attn_rope_bf16(*changed(args, change), None) == expected


@pytest.mark.parametrize("place", range(12))
def test_rope_strides(lib, place):
    strides = (ctypes.c_longlong * 12)(*([4096, 512, 64] * 4))
    strides[place] += 4
    assert lib.attn_rope_bf16(P, P, P, P, P, P, 0, ctypes.addressof(strides), 1, 8, 8, 8, 64, 64, 1, 0, 0, None) == 3
    assert lib.attn_rope_bf16(P, P, P, P, P, P, 0, None, 1, 8, 8, 8, 64, 64, 1, 0, 0, None) == 1


@pytest.mark.parametrize("change,expected", [
    ({0: 0}, 1), ({1: 0}, 1), ({2: 0}, 1), ({3: 0}, 1), ({4: 0}, 1), ({5: 0}, 1),
    ({7: 0}, 1), ({8: 0}, 1), ({9: 0}, 1), ({9: 3}, 1), ({10: 0}, 1), ({12: 0.0}, 1), ({12: float("inf")}, 1),
    ({11: 96}, 2), ({11: 256}, 2), ({10: 0x7fffffff}, 2), ({8: 70000, 9: 70000}, 2),
    ({0: P + 8}, 3), ({2: P + 2}, 3), ({3: P + 2}, 3), ({5: P + 1}, 3), ({6: P + 4}, 3),
])
def test_forward_arguments(lib, change, expected):
    # q, k, v, lam, o, lse, o2, B, H, Hkv, N, d, scale, causal, window
    args = [P, P, P, P, P, P, P, 2, 4, 2, 100, 64, 0.1, 1, 0]
    assert lib.attn_diff_fwd_bf16(*changed(args, change), None) == expected


@pytest.mark.parametrize("change,expected", [
    ({10: 0, 9: 0}, 0), ({9: 0}, 0),
    ({8: 0}, 1), ({9: 300}, 1), ({10: -1}, 1), ({7: 0}, 1), ({0: 0}, 1), ({12: 3}, 1), ({14: -1.0}, 1),
    ({13: 32}, 2), ({7: P + 2}, 3), ({1: P + 2}, 3),
])
def test_packed_forward_arguments(lib, change, expected):
    # q, k, v, lam, o, lse, o2, cu, S, max_seqlen, T, H, Hkv, d, scale, causal, window
    args = [P, P, P, P, P, P, 0, P, 3, 100, 250, 4, 2, 64, 0.1, 1, 0]
    assert lib.attn_diff_fwd_bf16_varlen(*changed(args, change), None) == expected


def test_backward_workspace(lib):
    assert lib.attn_diff_bwd_workspace_bytes(2, 3, 100) == 2048 + 2 * 2 * 3 * 100 * 4
    assert lib.attn_diff_bwd_workspace_bytes(0, 3, 100) == 0


@pytest.mark.parametrize("change,expected", [
    *[({i: 0}, 1) for i in range(13)], ({13: 4096}, 1), ({14: 0}, 1), ({16: 3}, 1), ({19: 0.0}, 1),
    ({18: 256}, 2), ({17: 0x7fffffff, 13: 1 << 60}, 2),
    *[({i: P + 8}, 3) for i in (0, 1, 2, 4, 5, 6, 8, 9, 10, 12)], ({3: P + 2}, 3), ({7: P + 2}, 3), ({11: P + 1}, 3),
])
def test_backward_arguments(lib, change, expected):
    # q, k, v, lam, o, o2, dout, lse, dq, dk, dv, dlam, ws, ws_bytes, B, H, Hkv, N, d, scale, causal, window
    args = [P] * 13 + [1 << 20, 2, 4, 2, 100, 64, 0.1, 1, 0]
    assert lib.attn_diff_bwd_bf16(*changed(args, change), None) == expected


@pytest.mark.parametrize("change,expected", [
    ({11: 0}, 1), ({14: 0}, 1), ({15: 0}, 1), ({16: 300}, 1), ({17: -1}, 1), ({13: 100}, 1), ({0: 0}, 1),
    ({19: 3}, 1), ({20: 96}, 2), ({14: P + 2}, 3), ({12: P + 8}, 3),
])
def test_packed_backward_arguments(lib, change, expected):
    # ... ws, ws_bytes, cu, S, max_seqlen, T, H, Hkv, d, scale, causal, window
    args = [P] * 13 + [1 << 20, P, 3, 100, 250, 4, 2, 64, 0.1, 1, 0]
    assert lib.attn_diff_bwd_bf16_varlen(*changed(args, change), None) == expected


@pytest.mark.parametrize("change,expected", [
    *[({i: 0}, 1) for i in range(8)], ({8: 0}, 1), ({10: 3}, 1), ({11: 0}, 1), ({14: 0}, 1), ({15: 0}, 1), ({16: -0.1}, 1),
    ({12: 256}, 2), ({11: 9}, 2), ({13: 8}, 2), ({13: 48}, 2), ({13: 1 << 17}, 2), ({8: 1 << 19}, 2), ({15: 1 << 30}, 2),
    ({0: P + 8}, 3), ({1: P + 2}, 3), ({3: P + 2}, 3), ({4: P + 2}, 3), ({18: P + 8}, 3),
])
def test_decoding_arguments(lib, change, expected):
    # q, kc, vc, lam, table, lens, o, lse, B, H, Hkv, nq, d, page_size, num_pages, max_pages, scale, window, ws, ws_bytes
    args = [P] * 8 + [2, 4, 2, 1, 64, 64, 10, 4, 0.1, 0, P, 1 << 40]
    assert lib.attn_diff_decode_bf16_paged(*changed(args, change), None) == expected


def test_decoding_workspace_refusals(lib):
    for bad in ((0, 1, 1, 64), (4, 3, 1, 64), (4, 2, 0, 64), (4, 2, 9, 64), (4, 2, 1, 256)):
        assert lib.attn_diff_decode_workspace_bytes(*bad) == 0


def test_binding_refuses_cpu_tensors():
    import exact_attention_55_gb300 as fa
    q, v, lam = torch.zeros(1, 2, 8, 64).bfloat16(), torch.zeros(1, 1, 8, 128).bfloat16(), torch.ones(1)
    cu = torch.tensor([0, 8], dtype=torch.int32)
    with pytest.raises(TypeError):
        fa.attn_rope_bf16(q, None, torch.zeros(1, 8, dtype=torch.int32), torch.ones(32))
    with pytest.raises(TypeError):
        fa.attn_diff_fwd_bf16(q, q, v, lam)
    with pytest.raises(TypeError):
        fa.attn_diff_fwd_bf16_varlen(q[0], q[0], v[0], lam, cu, 8)
    with pytest.raises(TypeError):
        fa.attn_diff_fwd_bf16_varlen(q[0], q[0], v[0], lam, None, 8)
    with pytest.raises(TypeError):
        fa.attn_diff_bwd_bf16(q, q, v, lam, v, v, v, torch.zeros(1, 2, 8))
    with pytest.raises(TypeError):
        fa.attn_diff_decode_bf16_paged(q, q, q, lam, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
