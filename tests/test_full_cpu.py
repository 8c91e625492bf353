"""Full-attention operators without a GPU: refusals of the C ABI and of the binding,
workspace sizes, the tree masks, and the plain forms the GPU tests compare with
(against brute force, differences and autograd)."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import sparse_attention_long_nsa_b200 as nsa
from tests import full_ref as R


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nsa.LIB_PATH):
        from sparse_attention_long_nsa_b200 import build
        build.build()
    return nsa.lib()


H = nsa.Heads(64, 4, 192, 128)
P16 = ctypes.c_void_p(16)
BIG = 1 << 40
INV, UNS, WS = nsa.NSA_ERR_INVALID_ARG, nsa.NSA_ERR_UNSUPPORTED, nsa.NSA_ERR_WORKSPACE


def ref(x):
    return ctypes.byref(x)


def test_ops_and_limits(L):
    assert (nsa.NSA_OP_FULL_PREFILL, nsa.NSA_OP_FULL_BACKWARD, nsa.NSA_OP_TREE_DECODE, nsa.NSA_OP_ROPE_BACKWARD) == (6, 7, 8, 9)
    assert nsa.NSA_MAX_NODES == 64


def test_workspace_sizes(L):
    size = nsa.nsa_full_workspace_size
    assert size(nsa.NSA_OP_FULL_PREFILL, H, 1, 8192, 8192, 0) >= 256
    assert size(nsa.NSA_OP_FULL_BACKWARD, H, 1, 8192, 8192, 0) >= 256 + 8192 * 64 * 8 + 2 * 148 * 128 * 320 * 4
    one, wide = (size(nsa.NSA_OP_TREE_DECODE, H, 4, 0, 1000, m) for m in (8, 9))
    assert wide > one >= 2 * 148 * 128 * 132 * 4          # 128 rows, then 256
    assert size(nsa.NSA_OP_ROPE_BACKWARD, H, 1, 8192, 0, 0) >= 148 * 2 * 192 * 4
    # the backward's workspace serves the forward
    assert size(nsa.NSA_OP_FULL_BACKWARD, H, 1, 0, 0, 0) >= size(nsa.NSA_OP_FULL_PREFILL, H, 1, 0, 0, 0)
    for bad in ((5, H, 1, 10, 10, 1), (nsa.NSA_OP_FULL_PREFILL, nsa.Heads(64, 5, 192, 128), 1, 10, 10, 0),
                (nsa.NSA_OP_FULL_PREFILL, nsa.Heads(64, 4, 96, 128), 1, 10, 10, 0),
                (nsa.NSA_OP_FULL_PREFILL, H, 0, 10, 10, 0), (nsa.NSA_OP_FULL_PREFILL, H, 129, 10, 10, 0),
                (nsa.NSA_OP_FULL_BACKWARD, H, 1, -1, 10, 0), (nsa.NSA_OP_TREE_DECODE, H, 1, 0, 0, 1),
                (nsa.NSA_OP_TREE_DECODE, H, 1, 0, 10, 0), (nsa.NSA_OP_TREE_DECODE, H, 1, 0, 10, 65)):
        assert size(*bad) == 0, bad


def rope_call(L, h=H, d_rot=64, inter=0, eps=1e-6, q=16, qs=None, k=16, ks=None, v=16, vs=None, w=16, f=16, pos=16, rows=None,
              n_rows=10, N=10, qo=16, ko=16, vo=16):
    p = nsa.RopeParams(d_rot, inter, eps)
    qs = h.H_q * h.d_k if qs is None else qs
    ks = h.H_kv * h.d_k if ks is None else ks
    vs = h.H_kv * h.d_v if vs is None else vs
    return L.nsa_qk_norm_rope(q, qs, k, ks, v, vs, w, w, f, pos, rows, n_rows, N, ref(h), ref(p), qo, ko, vo, None)


def test_rope_refusals(L):
    assert rope_call(L, N=0, n_rows=0) == nsa.NSA_OK                       # nothing to do: nothing is launched
    for kw in (dict(q=None), dict(q=8), dict(k=None), dict(k=24), dict(w=None), dict(w=8), dict(f=None), dict(pos=None),
               dict(f=18), dict(pos=17), dict(rows=20), dict(qo=None), dict(qo=8), dict(ko=None), dict(ko=20), dict(v=None), dict(vo=None), dict(v=8), dict(vo=8),
               dict(N=-1), dict(n_rows=9), dict(n_rows=-1, rows=16), dict(qs=64 * 192 - 8), dict(ks=4 * 192 + 4),
               dict(vs=4 * 128 - 8), dict(d_rot=-16), dict(d_rot=208), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(h=nsa.Heads(64, 3, 192, 128))):
        assert rope_call(L, **kw) == INV, kw
    for kw in (dict(d_rot=24), dict(h=nsa.Heads(60, 4, 192, 128)), dict(h=nsa.Heads(64, 4, 100, 128), d_rot=0),
               dict(N=1 << 31, n_rows=1 << 31)):
        assert rope_call(L, **kw) == UNS, kw


def test_rope_backward_refusals(L):
    def call(h=H, d_rot=64, ptr=16, dqs=64 * 192, dks=4 * 192, N=10, ws=BIG, grad=16, dw=16):
        p = nsa.RopeParams(d_rot, 1, 1e-6)
        return L.nsa_qk_norm_rope_backward(ptr, h.H_q * h.d_k, ptr, h.H_kv * h.d_k, ptr, ptr, ptr, ptr, N, grad, grad, ref(h),
                                           ref(p), 16, dqs, 16, dks, dw, dw, 16, ws, None)
    for kw in (dict(ptr=None), dict(ptr=8), dict(N=-1), dict(dqs=64 * 192 - 8), dict(dks=4 * 192 + 2), dict(grad=None),
               dict(grad=8), dict(dw=None), dict(d_rot=300)):
        assert call(**kw) == INV, kw
    assert call(d_rot=8) == UNS
    assert call(ws=1000) == WS


def prefill_call(L, h=H, cu=(0, 100), ptr=16, scale=0.0, ws=BIG, batch=None, back=False):
    arr = (ctypes.c_int32 * len(cu))(*cu)
    B = len(cu) - 1 if batch is None else batch
    if back:
        return L.nsa_full_prefill_backward(ptr, ptr, ptr, ptr, ptr, ptr, arr, B, ref(h), scale, ptr, ptr, ptr, ptr, ws, None)
    return L.nsa_full_prefill(ptr, ptr, ptr, arr, B, ref(h), scale, ptr, None, ptr, ws, None)


@pytest.mark.parametrize("back", [False, True])
def test_prefill_refusals(L, back):
    assert prefill_call(L, cu=(0, 0, 0), back=back) == nsa.NSA_OK
    for kw in (dict(ptr=None), dict(ptr=8), dict(cu=(1, 100)), dict(cu=(0, 100, 50)), dict(batch=0), dict(batch=-1),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(h=nsa.Heads(64, 3, 192, 128)),
               dict(h=nsa.Heads(0, 0, 192, 128))):
        assert prefill_call(L, back=back, **kw) == INV, kw
    for kw in (dict(h=nsa.Heads(60, 4, 192, 128)), dict(h=nsa.Heads(64, 4, 192, 192)), dict(h=nsa.Heads(64, 2, 64, 64)),
               dict(cu=(0,) * 130)):
        assert prefill_call(L, back=back, **kw) == UNS, kw
    assert prefill_call(L, ws=200, back=back) == WS


def tree_call(L, h=H, ptr=16, B=2, M=4, Lmax=100, max_len=100, scale=0.0, ws=BIG, paged=None, table=16):
    if paged is not None:
        pages, size, cols = paged
        return L.nsa_full_tree_decode_paged(ptr, ptr, ptr, pages, size, table, cols, ptr, None, None, B, M, max_len, ref(h),
                                            scale, ptr, None, ptr, ws, None)
    return L.nsa_full_tree_decode(ptr, ptr, ptr, ptr, None, None, B, M, Lmax, max_len, ref(h), scale, ptr, None, ptr, ws, None)


def test_tree_refusals(L):
    for kw in (dict(ptr=None), dict(ptr=8), dict(B=0), dict(M=0), dict(max_len=0), dict(max_len=101), dict(scale=-0.5),
               dict(scale=float("nan")), dict(h=nsa.Heads(64, 3, 192, 128)), dict(paged=(4, 32, 4)), dict(paged=(4, 96, 4)),
               dict(paged=(0, 64, 4)), dict(paged=(4, 64, 0)), dict(paged=(4, 64, 1)), dict(paged=(4, 64, 4), table=None)):
        assert tree_call(L, **kw) == INV, kw
    for kw in (dict(B=129), dict(M=65), dict(h=nsa.Heads(60, 4, 192, 128)), dict(paged=(1 << 25, 64, 4)),
               dict(paged=(4, 64, 1 << 26)), dict(B=128, Lmax=1 << 25, max_len=1 << 25)):
        assert tree_call(L, **kw) == UNS, kw
    assert tree_call(L, ws=300) == WS


def test_profile_slots_named(L):
    names = [nsa.lib().nsa_profile_slot_name(i).decode() for i in range(nsa.NSA_PROFILE_SLOTS)]
    assert names[-5:] == ["rope", "rope_bwd", "full_attn", "full_bwd", "tree_attn"] and len(set(names)) == len(names)


def test_binding_refuses_host_tensors(L):
    h = nsa.Heads(4, 1, 64, 64)
    t = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    kv = torch.zeros((3, 1, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        nsa.nsa_full_prefill(t, kv, kv, cu, h, t, None, torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        nsa.nsa_qk_norm_rope(t, kv, kv, kv, kv, cu, h, nsa.RopeParams(0, 0, 1e-6), t, kv)
    with pytest.raises(ValueError, match="CUDA"):
        nsa.nsa_full_tree_decode(t.unsqueeze(0), kv, kv, cu, None, None, 3, h, t)
    for bad in (cu.long(), torch.tensor([0], dtype=torch.int32), cu.unsqueeze(0), torch.arange(6, dtype=torch.int32)[::3]):
        with pytest.raises(ValueError, match="cu_seqlens"):
            nsa.nsa_full_prefill(t, kv, kv, bad, h, t)


# ---------------------------------------------------------------- masks

def test_tree_mask_from_parents():
    p = torch.tensor([[-1, 0, 0, 1, 2, -1], [-1, 0, 1, 2, 3, 4]])
    m = nsa.tree_mask_from_parents(p)
    assert m.tolist() == [[1, 0b11, 0b101, 0b1011, 0b10101, 0b100000], [1, 3, 7, 15, 31, 63]]
    chain = torch.arange(-1, 63).unsqueeze(0)
    assert nsa.tree_mask_from_parents(chain)[0].tolist() == R.as_int64([(2 << i) - 1 for i in range(64)])
    g = torch.Generator().manual_seed(3)
    for M in (1, 7, 64):
        par = torch.tensor([[-1] + [int(torch.randint(-1, i, (1,), generator=g)) for i in range(1, M)]])
        words = []
        for i in range(M):
            words.append((1 << i) | (words[int(par[0, i])] if par[0, i] >= 0 else 0))
        assert nsa.tree_mask_from_parents(par)[0].tolist() == R.as_int64(words)
    for bad in ([[0]], [[-1, 1]], [[-2]], [[-1, 2, 0]]):
        with pytest.raises(ValueError):
            nsa.tree_mask_from_parents(torch.tensor(bad))
    with pytest.raises(ValueError):
        nsa.tree_mask_from_parents(torch.full((1, 65), -1))


# ---------------------------------------------------------------- the plain forms

def brute_attention(q, k, v, see, scale):
    out, lse = np.zeros((len(q), v.shape[1])), np.full(len(q), -math.inf)
    for i in range(len(q)):
        js = [j for j in range(len(k)) if see[i, j]]
        if not js:
            continue
        s = [scale * sum(float(a) * float(b) for a, b in zip(q[i], k[j])) for j in js]
        m = max(s)
        z = sum(math.exp(x - m) for x in s)
        lse[i] = m + math.log(z)
        for x, j in zip(s, js):
            out[i] += math.exp(x - m) / z * v[j].numpy()
    return torch.tensor(out), torch.tensor(lse)


def test_plain_attention_against_brute_force():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((n, d), generator=g, dtype=torch.float64) for n, d in ((5, 6), (9, 6), (9, 4)))
    see = torch.rand((5, 9), generator=g) < 0.5
    see[2] = False                          # a row that sees nothing
    see[:, 3] = False                       # a key that no row sees
    k[3], v[3] = float("nan"), float("inf")
    x = R.attention(q, k, v, see, 0.3)
    o, lse = brute_attention(q, torch.nan_to_num(k), torch.nan_to_num(v, posinf=0), see, 0.3)
    assert torch.allclose(x["out"], o, atol=1e-12) and torch.allclose(x["lse"], lse, atol=1e-12)
    assert (x["out"][2] == 0).all() and x["lse"][2] == -math.inf


def test_plain_gradients_against_autograd_and_differences():
    g = torch.Generator().manual_seed(2)
    q, k, v, do = (torch.randn((7, d), generator=g, dtype=torch.float64) for d in (6, 6, 4, 4))
    see = R.causal(7, "cpu")
    f = lambda q, k, v: (R.attention(q, k, v, see, 0.4)["out"] * do).sum()   # noqa: E731
    leaves = [t.clone().requires_grad_(True) for t in (q, k, v)]
    want = torch.autograd.grad(f(*leaves), leaves)
    got, _ = R.attention_backward(q, k, v, see, 0.4, do)
    for n, w in zip(("dq", "dk", "dv"), want):
        assert torch.allclose(got[n], w, atol=1e-12), n
    for n, i in (("dq", 0), ("dk", 1), ("dv", 2)):
        for at in ((0, 0), (3, 2), (6, 3)):
            d = [torch.zeros_like(t) for t in (q, k, v)]
            d[i][at] = 1e-6
            up, dn = f(q + d[0], k + d[1], v + d[2]), f(q - d[0], k - d[1], v - d[2])
            assert abs(float((up - dn) / 2e-6 - got[n][at])) < 1e-7, (n, at)


@pytest.mark.parametrize("inter", [False, True])
def test_plain_rope_and_its_gradients(inter):
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn((3, 2, 16), generator=g, dtype=torch.float64) for _ in range(2))
    w = 1 + 0.1 * torch.randn((16,), generator=g, dtype=torch.float64)
    f, pos = torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float32), torch.tensor([0, 7, 100000], dtype=torch.int32)
    y = R.rope(x, w, f, pos, 8, inter, 1e-6)
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    for t in range(3):
        for i in range(4):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + 4)
            th = int(pos[t]) * float(f[i])
            z = complex(n[t, 0, a], n[t, 0, b]) * complex(math.cos(th), math.sin(th))
            assert abs(z.real - y[t, 0, a]) < 1e-9 and abs(z.imag - y[t, 0, b]) < 1e-9
    assert torch.equal(y[..., 8:], n[..., 8:])
    lx, lw = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    want = torch.autograd.grad((R.rope(lx, lw, f, pos, 8, inter, 1e-6) * dy).sum(), (lx, lw))
    dx, dw, _ = R.rope_backward(x, w, f, pos, 8, inter, 1e-6, dy)
    assert torch.allclose(dx, want[0], atol=1e-12) and torch.allclose(dw, want[1], atol=1e-12)


def test_plain_tree_equals_prompt_rows_on_each_path():
    """A node's result is that of the last row of the prompt its path makes."""
    g = torch.Generator().manual_seed(4)
    P, M, Hq, Hk, d, dv = 6, 5, 4, 2, 8, 6
    words = R.random_tree(M, g)
    q = torch.randn((1, M, Hq, d), generator=g, dtype=torch.float64)
    k, v = torch.randn((P + M, Hk, d), generator=g, dtype=torch.float64), torch.randn((P + M, Hk, dv), generator=g, dtype=torch.float64)
    got = R.tree(q, lambda b, L: k[:L], lambda b, L: v[:L], [P + M], [M], [words], Hk, 0.5)[0]
    for i in range(M):
        path = list(range(P)) + [P + j for j in range(M) if (words[i] >> j) & 1]
        n = len(path)
        qq = torch.zeros((n, Hq, d), dtype=torch.float64)
        qq[-1] = q[0, i]
        r = R.prefill(qq, k[path], v[path], [n], Hk, 0.5)
        assert torch.allclose(r["out"][-1], got["out"][i], atol=1e-12) and torch.allclose(r["lse"][-1], got["lse"][i], atol=1e-12)
