"""Full-attention entry points at the edges of their contracts, without a GPU."""
import ctypes
import os

import pytest
import torch

import sparse_attention_long_nsa_b200 as nsa

H = nsa.Heads(64, 4, 192, 128)
INV, WS = nsa.NSA_ERR_INVALID_ARG, nsa.NSA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nsa.LIB_PATH):
        from sparse_attention_long_nsa_b200 import build
        build.build()
    return nsa.lib()


def ref(x):
    return ctypes.byref(x)


# ---------------------------------------------------------------- nothing to do

def norm_call(L, N, q=None, v=None, v_out=None, w=16, n_rows=0, rows=None, d_rot=64, stride=64 * 192, k_out=None):
    rp = nsa.RopeParams(d_rot, 0, 1e-6)
    return L.nsa_qk_norm_rope(q, stride, q, 4 * 192, v, 4 * 128, w, w, 16, q, rows, n_rows, N, ref(H), ref(rp), q, k_out, v_out,
                              None)


def test_norm_of_no_tokens_takes_null_arrays(L):
    """An empty array has no address: N = 0 is nothing to do, whatever the per-token
    pointers are; geometry, weights and parameters are still checked."""
    assert norm_call(L, 0) == nsa.NSA_OK
    assert norm_call(L, 0, v_out=16, k_out=16, n_rows=5) == nsa.NSA_OK    # no values, a real cache
    for kw in (dict(w=None), dict(w=8), dict(d_rot=-16), dict(n_rows=-1, rows=16), dict(stride=64 * 192 - 8)):
        assert norm_call(L, 0, **kw) == INV, kw
    assert norm_call(L, 1) == INV


@pytest.mark.parametrize("back", [False, True])
def test_attention_over_empty_prompts_takes_null_arrays(L, back):
    def call(cu, scale=0.0, h=H):
        arr = (ctypes.c_int32 * len(cu))(*cu)
        if back:
            return L.nsa_full_prefill_backward(None, None, None, None, None, None, arr, len(cu) - 1, ref(h), scale, None, None, None,
                                               None, 0, None)
        return L.nsa_full_prefill(None, None, None, arr, len(cu) - 1, ref(h), scale, None, None, None, 0, None)
    assert call((0, 0)) == nsa.NSA_OK and call((0,) * 129) == nsa.NSA_OK
    for cu in ((0, 5, 0), (1, 1), (0, -1), (0, -4, 0), (0, 0, 3)):
        assert call(cu) == INV, cu
    assert call((0, 0), scale=-1.0) == INV and call((0, 0), h=nsa.Heads(64, 3, 192, 128)) == INV


def test_binding_names_a_missing_first_tensor(L):
    cu = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(TypeError, match="^q: expected a tensor, got NoneType"):
        nsa.nsa_full_prefill(None, None, None, cu, H, None)
    with pytest.raises(TypeError, match="^cu_seqlens: expected a tensor, got list"):
        nsa.nsa_full_prefill(None, None, None, [0, 3], H, None)
    with pytest.raises(TypeError, match="^q: "):
        nsa.nsa_qk_norm_rope(None, None, None, None, None, None, H, nsa.RopeParams(0, 0, 1e-6), None, None)
    with pytest.raises(TypeError, match="^q: "):
        nsa.nsa_full_tree_decode(None, None, None, None, None, None, 3, H, None)


# ---------------------------------------------------------------- in place

def test_norm_in_place_needs_packed_rows(L):
    """Outputs are packed: over inputs of a wider stride one token's result would lie
    over another's input. One token, or packed rows, is allowed (and launches: not here)."""
    h, rp = nsa.Heads(4, 1, 64, 64), nsa.RopeParams(64, 0, 1e-6)
    A, B, C = 1 << 12, 1 << 13, 1 << 14      # addresses that no refused call follows

    def forward(q_out=B, k_out=C, qs=256, ks=64, rows=None):
        return L.nsa_qk_norm_rope(A, qs, A + 512, ks, None, 0, A, A, A, A, rows, 10, 10, ref(h), ref(rp), q_out, k_out, None, None)

    def backward(dq=B, dk=C, dqs=256, dks=64):
        return L.nsa_qk_norm_rope_backward(A, 256, A, 64, A, A, A, A, 10, B, C, ref(h), ref(rp), dq, dqs, dk, dks, A, A, A, 1 << 30,
                                           None)
    assert forward(q_out=A, qs=384) == INV and forward(k_out=A + 512, ks=384) == INV
    assert backward(dqs=384) == INV and backward(dks=384) == INV
