"""Workspaces that are missing, short or misaligned, in the shapes of the
objectives that need one, and scales past what fp32 holds (no GPU): refused
before any pointer is touched."""

import ctypes

import pytest

from quantized_rank_fine_amd import qlora as q

P = 0x10000          # aligned for every element


@pytest.fixture(scope="module")
def L():
    return q.lib()


@pytest.mark.parametrize("pairs,tokens", [(1, 16385), (2, 300000), (9, 100), (64, 131072),
                                          (1000, 20000), (1 << 20, 1 << 20)])
def test_pref_workspace(L, pairs, tokens):
    """Slices, a workgroup to a pair, and the pairs' losses by the workspace."""
    n = q.qlora_pref_workspace_bytes(pairs, tokens)
    assert n > 0
    pref = ctypes.byref(q.pref_struct(q.PREF_SIGMOID, 0.1))

    def call(ws, size):
        return L.qlora_pref_loss(P, None, None, P, pairs, tokens, pref, P, P, P, ws, size, None)

    assert call(P, n - 1) == 5 and call(P, 0) == 5
    assert call(None, n) == 1
    assert call(P + 4, n) == 3


@pytest.mark.parametrize("T,V,dt", [(4, 200000, q.F32), (1, 131073, q.BF16), (64, 65537, q.F32),
                                    (64, 1 << 24, q.BF16)])
def test_token_logp_workspace(L, T, V, dt):
    n = q.qlora_token_logp_workspace_bytes(T, V, dt)
    assert n > 0

    def call(ws, size):
        return L.qlora_token_logp_fwd(P, V, T, V, dt, P, 1.0, P, P, None, ws, size, None)

    assert call(P, n - 1) == 5 and call(P, 0) == 5
    assert call(None, n) == 1
    assert call(P + 2, n) == 3


@pytest.mark.parametrize("T,V", [(1, 5), (9000, 1000), (64, 65537), (1, 200000)])
def test_policy_logits_workspace(L, T, V):
    n = q.qlora_policy_logits_workspace_bytes(T, V, q.BF16)
    assert n > 0
    pol = ctypes.byref(q.policy_struct(q.OBJ_CLIP))

    def call(ws, size):
        return L.qlora_policy_logits(P, V, T, V, q.BF16, P, 1.0, None, None, None, None, pol, P,
                                     None, P, V, ws, size, None)

    assert call(P, n - 1) == 5 and call(P, 0) == 5
    assert call(None, n) == 1
    assert call(P + 8, n) == 3


@pytest.mark.parametrize("T", [8193, 100000, 1 << 30])
def test_policy_workspace(L, T):
    n = q.qlora_policy_workspace_bytes(T)
    assert n > 0
    pol = ctypes.byref(q.policy_struct(q.OBJ_NLL))

    def call(ws, size):
        return L.qlora_policy_loss(P, None, T, None, None, None, None, pol, P, P, None, ws, size,
                                   None)

    assert call(P, n - 1) == 5 and call(P, 0) == 5
    assert call(None, n) == 1
    assert call(P + 4, n) == 3


@pytest.mark.parametrize("s", [2.4e38, 3.4e38])
def test_scales_past_fp32(L, s):
    """s log2 e has to be a number in fp32, or every row would be NaN."""
    pol = ctypes.byref(q.policy_struct(q.OBJ_CLIP))
    big = 1 << 20
    for scale, status in ((s, 7), (2.3e38, 1)):          # (1: on to the missing pointers)
        assert L.qlora_token_logp_fwd(None, 8, 1, 8, q.F32, P, scale, P, P, None, None, 0,
                                      None) == status
        assert L.qlora_token_logp_bwd(None, 8, 1, 8, q.F32, P, scale, P, None, P, None, P, 8,
                                      None) == status
        assert L.qlora_policy_logits(None, 8, 1, 8, q.F32, P, scale, None, None, None, None, pol,
                                     P, None, P, 8, P, big, None) == status
