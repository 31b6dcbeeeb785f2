"""Backward passes of no value heads (no query heads) over keys that there are: the sums
over none of them are zeros, in every token that a sequence holds."""
import ctypes

import pytest
import torch

import selective_state_space_44_amd as ssm
from test_gpu_delta import BF16, DEV, F32, cu_of, say

pytestmark = pytest.mark.gpu


def dirty(shape, dtype):
    """Memory that an allocation of as many bytes takes next is not zero."""
    t = torch.full(shape, 7.0, dtype=dtype, device=DEV)
    torch.cuda.synchronize()
    del t


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("packed", [False, True])
def test_delta(packed, io):
    say("delta, no heads", packed, io)
    lead = (70,) if packed else (2, 35)
    q = torch.randn((*lead, 3, 16), device=DEV).to(io)
    v, b = (torch.zeros((*lead, 0) + s, dtype=io, device=DEV) for s in ((8,), ()))
    cu = cu_of([30, 0, 40]) if packed else None
    for _ in range(3):
        for _ in range(4):
            dirty(q.shape, io)
        g = ssm.gated_delta_bwd(q, q, v, b.float(), b, dy=v, cu_seqlens=cu)
        assert torch.all(g["dq"] == 0) and torch.all(g["dk"] == 0)
        assert g["dv"].shape == v.shape and g["dlog_decay"].shape == b.shape
    leaf = q.clone().requires_grad_()
    o, _ = ssm.GatedDelta.apply(leaf, q, v, b.float(), b, None, 0.3, cu)
    dirty(q.shape, io)
    assert torch.all(torch.autograd.grad(o.sum(), leaf)[0] == 0)


@pytest.mark.parametrize("io", [BF16, F32])
def test_delta_leaves_tokens_of_no_sequence(io):
    say("delta, no heads, uncovered", io)
    T, G, K = 50, 3, 24
    code = 1 if io is BF16 else 0
    lib = ssm.load_library()
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    x = torch.randn(T, G, K, device=DEV).to(io)
    none = torch.zeros(16, device=DEV)
    for cuts, rows in (([5, 9, 9, 40], slice(5, 40)), ([-3, 60], slice(0, 50)), ([20, 20], slice(0, 0))):
        cu = torch.tensor(cuts, dtype=torch.int32, device=DEV)
        dq, dk = (torch.full((T, G, K), 7.0, dtype=io, device=DEV) for _ in "12")
        st = lib.ssm_delta_bwd(len(cuts) - 1, T, p(cu), 0, G, K, 8, code, p(x), G * K, p(x), G * K, None, 0,
                               None, None, 1.0, None, None, 0, None, p(dq), p(dk), None, None, None, None,
                               None, 0, None)
        torch.cuda.synchronize()
        assert st == ssm.SSM_OK
        for d in (dq, dk):
            assert torch.all(d[rows] == 0)
            d[rows] = 7.0
            assert torch.all(d == 7.0)


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("packed", [False, True])
def test_linear_attention(packed, io):
    say("linear attention, no heads", packed, io)
    lead = (70,) if packed else (2, 35)
    k = torch.randn((*lead, 3, 16), device=DEV).to(io)
    v = torch.randn((*lead, 3, 24), device=DEV).to(io)
    q, y = (torch.zeros((*lead, 0, n), dtype=io, device=DEV) for n in (16, 24))
    ld = torch.zeros(0, device=DEV)
    cu = cu_of([30, 0, 40]) if packed else None
    for _ in range(3):
        for _ in range(4):
            dirty(k.shape, io)
            dirty(v.shape, io)
        g = ssm.linear_attn_bwd(q, k, v, ld, dy=y, cu_seqlens=cu, need_dlog_decay=True)
        assert torch.all(g["dk"] == 0) and torch.all(g["dv"] == 0)
        assert g["dq"].shape == q.shape and g["dlog_decay"].shape == (0,)


@pytest.mark.parametrize("io", [BF16, F32])
def test_linear_attention_leaves_tokens_of_no_sequence(io):
    say("linear attention, no heads, uncovered", io)
    T, G, K, V = 50, 3, 24, 40
    code = 1 if io is BF16 else 0
    lib = ssm.load_library()
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    k, v = (torch.randn(T, G, n, device=DEV).to(io) for n in (K, V))
    for cuts, rows in (([5, 9, 9, 40], slice(5, 40)), ([-3, 60], slice(0, 50)), ([20, 20], slice(0, 0))):
        cu = torch.tensor(cuts, dtype=torch.int32, device=DEV)
        dk, dv = (torch.full((T, G, n), 7.0, dtype=io, device=DEV) for n in (K, V))
        st = lib.ssm_linattn_bwd(len(cuts) - 1, T, p(cu), 0, G, K, V, code, None, 0, p(k), G * K, p(v), G * V,
                                 None, 1.0, None, None, 0, None, None, p(dk), p(dv), None, None, 0, None, 0,
                                 None)
        torch.cuda.synchronize()
        assert st == ssm.SSM_OK
        for d in (dk, dv):
            assert torch.all(d[rows] == 0)
            d[rows] = 7.0
            assert torch.all(d == 7.0)
