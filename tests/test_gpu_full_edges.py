"""Full-attention operators on the GPU at the edges of their contracts, against the
plain fp64 forms and bounds of tests/full_ref.py."""
import pytest
import torch

import sparse_attention_long_nsa_b200 as nsa
from tests import full_ref as R
from tests.test_gpu_full import caches, check_tree, gen, randn, rope_tol, run_tree, ws_for

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


# ---------------------------------------------------------------- nodes that no mask names

def pages_of(k, v, page, seed):
    """The rows of contiguous caches in shuffled pages: pools and block table."""
    B, Lmax, per = k.shape[0], k.shape[1], k.shape[1] // page
    perm = torch.randperm(B * per, generator=gen(seed), device="cuda")
    pools = [torch.empty((B * per, page, *t.shape[2:]), dtype=BF, device="cuda") for t in (k, v)]
    for p, t in zip(pools, (k, v)):
        p[perm] = t.view(B * per, page, *t.shape[2:])
    return (*pools, perm.to(torch.int32).view(B, per).contiguous())


def tree_around(M, hidden, g):
    """Words of a random tree over the nodes outside `hidden`; the others name nothing
    and are named by nobody."""
    words = [0] * M
    live = [i for i in range(M) if i not in hidden]
    for n, i in enumerate(live):
        words[i] = 1 << i
        if n:
            words[i] |= words[live[int(torch.randint(0, n, (1,), generator=g))]]
    return words


@pytest.mark.parametrize("dims,Hq,Hk,M,lens,page", [
    ((64, 64), 4, 1, 5, [5, 64, 130, 700], 0),          # 128 rows, V of 64 channels
    ((192, 128), 16, 2, 8, [8, 150, 129, 1000], 64),    # 128 rows, V of 128 channels
    ((128, 64), 16, 1, 16, [16, 70, 135, 2000], 64),    # 256 rows in one block
    ((64, 128), 64, 4, 13, [13, 140, 6000], 0),         # 256 rows, the second half not full; cut units
    ((128, 128), 32, 2, 64, [64, 150, 300, 1023], 128)])    # several blocks; nodes in two key tiles
def test_tree_cache_rows_of_nodes_that_no_mask_names(dims, Hq, Hk, M, lens, page):
    """Padded node slots without n_nodes: the slots' cache rows were never written and
    hold NaN and infinities, no mask names them; every other node's result is as if they
    were finite."""
    h = nsa.Heads(Hq, Hk, *dims)
    B, Lmax = len(lens), -(-max(lens) // 128) * 128
    k, v = caches(lens, Lmax, h, 7 + M)[:2]
    q = randn((B, M, Hq, dims[0]), gen(M))
    cpu = torch.Generator().manual_seed(M)
    masks = []
    for b, L in enumerate(lens):
        # padding at the end, nodes in the middle, the first node, all but the last
        hidden = [set(range(M - M // 3 - 1, M)), {1, M // 2, M - 2}, {0, 2, M - 1}, set(range(M - 1))][b]
        masks.append(tree_around(M, hidden, cpu))
    good = run_tree(q, (k, v, None, None, None), lens, None, masks, max(lens), h)
    for b, L in enumerate(lens):
        for i in range(M):
            if not any((w >> i) & 1 for w in masks[b]):
                k[b, L - M + i] = float("nan") if i & 1 else float("-inf")
                v[b, L - M + i] = float("inf") if i & 1 else float("nan")
    kv = (k, v, *(pages_of(k, v, page, 5) if page else (None,) * 3))
    out, lse = run_tree(q, kv, lens, None, masks, max(lens), h)
    assert torch.equal(out, good[0]) and torch.equal(lse, good[1])
    check_tree(out, lse, q, kv, lens, [M] * B, masks, h, dims[0] ** -0.5)
    if page:
        po, pl = run_tree(q, kv, lens, None, masks, max(lens), h, paged=True)
        assert torch.equal(po, out) and torch.equal(pl, lse)


@pytest.mark.parametrize("dims", [(192, 128), (64, 64)])
def test_tree_chain_longer_than_a_block_keeps_later_nodes_out(dims):
    """33 drafts of 16 heads a group are three blocks of rows; the last draft's values
    are NaN and reach its own rows only."""
    h = nsa.Heads(16, 1, *dims)
    lens, M = [500, 33], 33
    k, v = caches(lens, 512, h, 8)[:2]
    q = randn((2, M, 16, dims[0]), gen(9))
    kv = (k, v, None, None, None)
    good = run_tree(q, kv, lens, [M, M], None, 500, h)
    for b, L in enumerate(lens):
        v[b, L - 1] = float("nan")
    out, lse = run_tree(q, kv, lens, [M, M], None, 500, h)
    assert torch.equal(out[:, :M - 1], good[0][:, :M - 1]) and torch.equal(lse, good[1])
    assert torch.isnan(out[:, M - 1].float()).all()


# ---------------------------------------------------------------- norm and rotary position

@pytest.mark.parametrize("d_k", [64, 192])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d_rot", [0, 32])
def test_rope_channels_that_do_not_rotate_stay_apart(d_k, inter, d_rot):
    """A value or weight that is not finite, of a channel that does not rotate, is that
    channel's alone (a value's norm apart)."""
    h = nsa.Heads(4, 2, d_k, 64)
    g = gen(3)
    q, k = randn((9, 4, d_k), g), randn((9, 2, d_k), g)
    w_q, w_k = (1 + 0.2 * randn((d_k,), g, torch.float32) for _ in range(2))
    f = torch.linspace(1, 0.01, d_rot // 2, device="cuda")
    pos = torch.arange(9, device="cuda", dtype=torch.int32) * 1000
    for i, c in enumerate(range(d_rot, d_k, 5)):
        q[i % 9, i % 4, c] = float("inf") if i & 1 else float("-inf")
    w_q[d_rot + 1::7], w_k[d_rot + 2::9], w_k[d_k - 1] = float("inf"), float("-inf"), float("nan")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    nsa.nsa_qk_norm_rope(q, k, w_q, w_k, f, pos, h, nsa.RopeParams(d_rot, int(inter), 1e-6), qo, ko)
    for got, x, w in ((qo, q, w_q), (ko, k, w_k)):
        want = R.rope(x, w, f, pos, d_rot, inter, 1e-6)
        fin_w = torch.nan_to_num(w.double(), 0, 0, 0).abs()
        big = (torch.nan_to_num(x.double(), 0, 0, 0).abs() * fin_w).amax(-1, keepdim=True) / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6)
        R.assert_within(got, want, rope_tol(want, 2 * big), "rope")


# ---------------------------------------------------------------- refusals of the binding

def empty(*s):
    return torch.empty(s, dtype=BF, device="cuda")


@pytest.mark.parametrize("cu", [[0, 5, 0], [0, -4, 0], [1, 0], [0, -1]])
def test_binding_leaves_bad_cu_seqlens_to_the_library(cu):
    """A last entry of 0 does not make the others right."""
    h = nsa.Heads(8, 2, 64, 64)
    q, kv, lse = empty(0, 8, 64), empty(0, 2, 64), torch.empty((0, 8), device="cuda")
    cu = torch.tensor(cu, dtype=torch.int32)
    ws = ws_for(nsa.NSA_OP_FULL_BACKWARD, h, 2, 0, 0)
    for call in (lambda: nsa.nsa_full_prefill(q, kv, kv, cu, h, q, lse, ws),
                 lambda: nsa.nsa_full_prefill(q, kv, kv, cu, h, q),
                 lambda: nsa.nsa_full_prefill_backward(q, kv, kv, q, lse, q, cu, h, q, kv, kv, ws)):
        with pytest.raises(nsa.NSAError) as e:
            call()
        assert e.value.status == nsa.NSA_ERR_INVALID_ARG


def test_empty_calls_need_no_workspace():
    h, rp = nsa.Heads(8, 2, 64, 64), nsa.RopeParams(0, 0, 1e-6)
    q, kv, lse = empty(0, 8, 64), empty(0, 2, 64), torch.empty((0, 8), device="cuda")
    cu, w = torch.zeros(3, dtype=torch.int32), torch.ones(64, device="cuda")
    nsa.nsa_full_prefill(q, kv, kv, cu, h, q)
    nsa.nsa_full_prefill_backward(q, kv, kv, q, lse, q, cu, h, q, kv, kv, None)
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    nsa.nsa_qk_norm_rope(q, kv, w, w, None, pos, h, rp, q, empty(3, 2, 64), kv, empty(3, 2, 64))
    st = torch.cuda.Stream()
    dw = [torch.full((64,), 5.0, device="cuda") for _ in range(2)]
    st.wait_stream(torch.cuda.current_stream())
    nsa.nsa_qk_norm_rope_backward(q, kv, w, w, None, pos, q, kv, h, rp, q, kv, *dw, None, stream=st)
    st.synchronize()
    assert (dw[0] == 0).all() and (dw[1] == 0).all()


def test_binding_names_a_missing_tensor():
    """None for a tensor that a call needs is a TypeError with the argument's name."""
    h, rp = nsa.Heads(8, 2, 64, 64), nsa.RopeParams(32, 0, 1e-6)
    q, kv, lse, w = empty(4, 8, 64), empty(4, 2, 64), torch.empty((4, 8), device="cuda"), torch.ones(64, device="cuda")
    f, i32 = torch.ones(16, device="cuda"), torch.ones(4, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 4], dtype=torch.int32)
    ws = ws_for(nsa.NSA_OP_FULL_BACKWARD, h, 1, 4, 4)
    q4, pool = q.unsqueeze(1), empty(4, 64, 2, 64)
    calls = (
        (nsa.nsa_qk_norm_rope, dict(q=q, k=kv, w_q=w, w_k=w, inv_freq=f, positions=i32, heads=h, rope=rp, q_out=q, k_out=kv), ()),
        (nsa.nsa_qk_norm_rope_backward, dict(q=q, k=kv, w_q=w, w_k=w, inv_freq=f, positions=i32, dq_out=q, dk_out=kv, heads=h,
                                             rope=rp, dq=q, dk=kv, dw_q=w, dw_k=w, ws=ws), ("ws",)),
        (nsa.nsa_full_prefill, dict(q=q, k=kv, v=kv, cu_seqlens=cu, heads=h, out=q, ws=ws), ("ws",)),
        (nsa.nsa_full_prefill_backward, dict(q=q, k=kv, v=kv, out=q, lse=lse, dout=q, cu_seqlens=cu, heads=h, dq=q, dk=kv, dv=kv,
                                             ws=ws), ("ws",)),
        (nsa.nsa_full_tree_decode, dict(q=q4, k_cache=pool, v_cache=pool, cache_lens=i32, n_nodes=None, tree_mask=None, max_len=64,
                                        heads=h, out=q4, ws=ws), ("ws",)),
        (nsa.nsa_full_tree_decode_paged, dict(q=q4, k_pool=pool, v_pool=pool, block_table=i32.view(4, 1), cache_lens=i32,
                                              n_nodes=None, tree_mask=None, max_len=64, heads=h, out=q4, ws=ws), ("ws",)))
    for fn, args, by_value in calls:
        for name, t in args.items():
            if isinstance(t, torch.Tensor):
                with pytest.raises(ValueError if name in by_value else TypeError, match=rf"^{name}\b"):
                    fn(**{**args, name: None})
    with pytest.raises(TypeError, match="v_out"):
        nsa.nsa_qk_norm_rope(q, kv, w, w, f, i32, h, rp, q, kv, kv, [1])
