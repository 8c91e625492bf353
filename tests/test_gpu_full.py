"""Full-attention operators on the GPU against their plain fp64 forms, elementwise
within the bounds derived in tests/full_ref.py."""
import math

import pytest
import torch

import sparse_attention_long_nsa_b200 as nsa
from tests import full_ref as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
DIMS = [(64, 64), (64, 128), (128, 64), (128, 128), (192, 64), (192, 128)]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, g, dtype=BF, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def ws_for(op, h, batch=1, total=0, max_len=0, nodes=0):
    n = nsa.nsa_full_workspace_size(op, h, batch, total, max_len, nodes)
    assert n > 0
    return nsa.alloc_workspace(n, "cuda")


# ---------------------------------------------------------------- norm and rotary position

def rope_inputs(N, h, d_rot, seed, fused, far=False):
    g = gen(seed)
    wq, wk, wv = h.H_q * h.d_k, h.H_kv * h.d_k, h.H_kv * h.d_v
    x = randn((N, wq + wk + wv), g, scale=1.5)
    q, k, v = x[:, :wq], x[:, wq:wq + wk], x[:, wq + wk:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q, k, v = (t.unflatten(1, (n, d)) for t, n, d in ((q, h.H_q, h.d_k), (k, h.H_kv, h.d_k), (v, h.H_kv, h.d_v)))
    w_q, w_k = 1 + 0.3 * randn((h.d_k,), g, torch.float32), 1 + 0.3 * randn((h.d_k,), g, torch.float32)
    i = torch.arange(d_rot // 2, device="cuda", dtype=torch.float64)
    f = (10000.0 ** (-2 * i / max(d_rot, 1))).float()
    pos = torch.randint(0, 1 << (30 if far else 13), (N,), generator=g, device="cuda", dtype=torch.int32)
    if far:
        pos[0] = -5
    return q, k, v, w_q, w_k, f, pos


# fp32 chain of a few roundings on each value, then half a bf16 step; the angle is
# exact to 2^-24 pi radians + the sine's own 2^-22
def rope_tol(want, y_abs):
    return R.U * want.abs() * 1.01 + 64 * R.E * y_abs


@pytest.mark.parametrize("N,Hq,Hk,dims,d_rot,inter,fused", [
    (1, 4, 1, (64, 64), 64, False, False), (1, 64, 4, (192, 128), 64, True, True), (7, 16, 2, (128, 128), 128, False, True),
    (333, 4, 4, (64, 128), 16, True, False), (1000, 24, 12, (192, 64), 192, False, True),
    (297, 8, 1, (128, 64), 0, True, False), (2500, 8, 2, (192, 128), 176, True, False), (64, 64, 4, (192, 128), 48, False, True)])
def test_rope_forward(N, Hq, Hk, dims, d_rot, inter, fused):
    h = nsa.Heads(Hq, Hk, *dims)
    q, k, v, w_q, w_k, f, pos = rope_inputs(N, h, d_rot, 11 + N, fused, far=True)
    qo, ko, vo = (torch.full((N, n, d), 7.0, dtype=BF, device="cuda") for n, d in ((Hq, dims[0]), (Hk, dims[0]), (Hk, dims[1])))
    rp = nsa.RopeParams(d_rot, int(inter), 1e-6)
    nsa.nsa_qk_norm_rope(q, k, w_q, w_k, f, pos, h, rp, qo, ko, v, vo)
    for got, x, w in ((qo, q, w_q), (ko, k, w_k)):
        want = R.rope(x, w, f, pos, d_rot, inter, 1e-6)
        big = (x.double().abs() * w.double().abs()).amax(-1, keepdim=True) / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6)
        R.assert_within(got, want, rope_tol(want, 2 * big), "rope")
    assert torch.equal(vo, v)
    if not fused:   # in place gives the same bits; without values too
        q2, k2 = q.clone(), k.clone()
        nsa.nsa_qk_norm_rope(q2, k2, w_q, w_k, f, pos, h, rp, q2, k2)
        assert torch.equal(q2, qo) and torch.equal(k2, ko)


def test_rope_cache_rows_and_padding():
    h = nsa.Heads(16, 2, 128, 64)
    N, R_ = 37, 100
    q, k, v, w_q, w_k, f, pos = rope_inputs(N, h, 64, 5, True)
    rp = nsa.RopeParams(64, 0, 1e-5)
    plain_q, plain_k, plain_v = torch.empty((N, 16, 128), dtype=BF, device="cuda"), torch.empty((N, 2, 128), dtype=BF, device="cuda"), torch.empty((N, 2, 64), dtype=BF, device="cuda")
    nsa.nsa_qk_norm_rope(q, k, w_q, w_k, f, pos, h, rp, plain_q, plain_k, v, plain_v)
    rows = torch.randperm(R_, generator=gen(1), device="cuda")[:N].contiguous()
    rows[3], rows[9], rows[20] = -1, R_, 1 << 40   # padding and rows outside the cache
    qo = torch.empty_like(plain_q)
    ko, vo = torch.full((R_, 2, 128), 3.0, dtype=BF, device="cuda"), torch.full((R_, 2, 64), 4.0, dtype=BF, device="cuda")
    nsa.nsa_qk_norm_rope(q, k, w_q, w_k, f, pos, h, rp, qo, ko.view(4, 25, 2, 128), v, vo.view(4, 25, 2, 64), rows)
    want_k, want_v = torch.full_like(ko, 3.0), torch.full_like(vo, 4.0)
    in_ = (rows >= 0) & (rows < R_)
    want_k[rows[in_]], want_v[rows[in_]] = plain_k[in_], plain_v[in_]
    assert torch.equal(qo, plain_q) and torch.equal(ko, want_k) and torch.equal(vo, want_v)


def test_rope_values_of_one_head_do_not_reach_another():
    h = nsa.Heads(4, 2, 64, 64)
    q, k, v, w_q, w_k, f, pos = rope_inputs(20, h, 32, 6, False)
    rp = nsa.RopeParams(32, 1, 1e-6)
    a, b = (torch.empty((20, 4, 64), dtype=BF, device="cuda"), torch.empty((20, 2, 64), dtype=BF, device="cuda"))
    nsa.nsa_qk_norm_rope(q, k, w_q, w_k, f, pos, h, rp, a, b)
    q2 = q.clone()
    q2[5, 2] = float("nan")
    q2[6, 0, 3] = float("inf")
    q2[7, 1] = 0
    c, d = torch.empty_like(a), torch.empty_like(b)
    nsa.nsa_qk_norm_rope(q2, k, w_q, w_k, f, pos, h, rp, c, d)
    keep = torch.ones((20, 4), dtype=torch.bool, device="cuda")
    keep[5, 2] = keep[6, 0] = keep[7, 1] = False
    assert torch.equal(c[keep], a[keep]) and torch.equal(d, b)
    assert torch.isnan(c[5, 2]).all() and (c[7, 1] == 0).all()


@pytest.mark.parametrize("N,Hq,Hk,dims,d_rot,inter,fused", [
    (1, 4, 1, (64, 64), 64, False, False), (333, 4, 1, (64, 64), 32, True, False), (1025, 64, 4, (192, 128), 192, False, True),
    (77, 16, 16, (128, 128), 0, False, True), (700, 8, 2, (128, 64), 112, True, True)])
def test_rope_backward(N, Hq, Hk, dims, d_rot, inter, fused):
    h = nsa.Heads(Hq, Hk, *dims)
    q, k, v, w_q, w_k, f, pos = rope_inputs(N, h, d_rot, 21 + N, fused)
    g = gen(N)
    gq, gk = randn((N, Hq, dims[0]), g), randn((N, Hk, dims[0]), g)
    fused_grad = torch.zeros((N, (Hq + 2 * Hk) * dims[0]), dtype=BF, device="cuda")
    dq = fused_grad[:, :Hq * dims[0]].unflatten(1, (Hq, dims[0]))
    dk = fused_grad[:, Hq * dims[0]:(Hq + Hk) * dims[0]].unflatten(1, (Hk, dims[0]))
    dwq, dwk = torch.empty_like(w_q), torch.empty_like(w_k)
    rp = nsa.RopeParams(d_rot, int(inter), 1e-6)
    ws = ws_for(nsa.NSA_OP_ROPE_BACKWARD, h, 1, N)
    nsa.nsa_qk_norm_rope_backward(q, k, w_q, w_k, f, pos, gq, gk, h, rp, dq, dk, dwq, dwk, ws)
    for dx, dw, x, w, dy in ((dq, dwq, q, w_q, gq), (dk, dwk, k, w_k, gk)):
        want, wdw, mag = R.rope_backward(x, w, f, pos, d_rot, inter, 1e-6, dy)
        # a row's terms: r u and h mean(u h), each at most r max|dn| max|w| times a small factor
        r = 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6)
        row = r * (dy.double().abs().amax(-1, keepdim=True) * 2 * w.double().abs().max()) * (1 + x.double().abs().amax(-1, keepdim=True) * r)
        R.assert_within(dx, want, R.U * want.abs() * 1.01 + (64 + dims[0]) * R.E * row, "dx")
        n = N * x.shape[1]
        R.assert_within(dw, wdw, (64 + 8 * math.sqrt(n)) * R.E * mag * 2, "dw")   # partial sums of a thread, a block, the blocks
    assert (fused_grad[:, (Hq + Hk) * dims[0]:] == 0).all()
    again = [torch.empty_like(t) for t in (w_q, w_k)]
    nsa.nsa_qk_norm_rope_backward(q, k, w_q, w_k, f, pos, gq, gk, h, rp, gq, gk, *again, ws)   # over its inputs
    assert torch.equal(again[0], dwq) and torch.equal(again[1], dwk) and torch.equal(gq, dq) and torch.equal(gk, dk)


# ---------------------------------------------------------------- prompts

def prompt(lens, h, seed, extra=0):
    g = gen(seed)
    N = sum(lens)
    q, k, v = randn((N + extra, h.H_q, h.d_k), g), randn((N + extra, h.H_kv, h.d_k), g), randn((N + extra, h.H_kv, h.d_v), g)
    cu = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32)
    return q, k, v, cu


def run_prefill(q, k, v, cu, h, scale=0.0, stream=None):
    N = int(cu[-1])
    out = torch.full((q.shape[0], h.H_q, h.d_v), 9.0, dtype=BF, device="cuda")
    lse = torch.full((q.shape[0], h.H_q), 9.0, device="cuda")
    ws = ws_for(nsa.NSA_OP_FULL_PREFILL, h, cu.numel() - 1, N, N)
    nsa.nsa_full_prefill(q, k, v, cu, h, out, lse, ws, scale=scale, stream=stream)
    nsa.nsa_check_device_status(ws, stream)
    return out, lse


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("Hq,Hk,lens", [
    (4, 1, [1]), (16, 1, [129]), (2, 2, [300, 1, 0, 128, 127]), (8, 4, [64, 65, 511]), (16, 2, [513, 40]), (32, 4, [1500, 7, 700])])
def test_prefill(dims, Hq, Hk, lens):
    h = nsa.Heads(Hq, Hk, *dims)
    q, k, v, cu = prompt(lens, h, 3, extra=5)
    out, lse = run_prefill(q, k, v, cu, h)
    N = sum(lens)
    want = R.prefill(q[:N], k[:N], v[:N], lens, Hk, dims[0] ** -0.5)
    R.assert_within(out[:N], want["out"], want["out_tol"], "out")
    R.assert_within(lse[:N], want["lse"], want["lse_tol"], "lse")
    assert (out[N:] == 9).all() and (lse[N:] == 9).all()   # rows behind the last sequence


@pytest.mark.parametrize("dims,Hq,Hk,lens", [((64, 64), 16, 16, [2600, 130, 1]), ((192, 128), 16, 16, [2433, 255]),
                                             ((64, 128), 24, 12, [1700, 129]), ((128, 64), 40, 40, [1000])])
def test_prefill_blocks_of_256_rows_whose_halves_end_in_different_tiles(dims, Hq, Hk, lens):
    """One or two query heads a key head and enough blocks for all SMs: the second half
    of a block sees a key tile that the first does not, or does not exist."""
    h = nsa.Heads(Hq, Hk, *dims)
    q, k, v, cu = prompt(lens, h, 5)
    out, lse = run_prefill(q, k, v, cu, h)
    want = R.prefill(q, k, v, lens, Hk, dims[0] ** -0.5)
    R.assert_within(out, want["out"], want["out_tol"], "out")
    R.assert_within(lse, want["lse"], want["lse_tol"], "lse")


def test_prefill_largest_batch_and_many_empty_sequences():
    h = nsa.Heads(8, 4, 64, 64)
    lens = [(37 * i) % 90 if i % 3 else 0 for i in range(128)]
    q, k, v, cu = prompt(lens, h, 6)
    out, lse = run_prefill(q, k, v, cu, h)
    do = randn(tuple(out.shape), gen(6))
    want = R.prefill(q, k, v, lens, 4, 0.125, do)
    R.assert_within(out, want["out"], want["out_tol"], "out")
    R.assert_within(lse, want["lse"], want["lse_tol"], "lse")
    for n, t in zip(("dq", "dk", "dv"), run_backward(q, k, v, cu, h, do)):
        R.assert_within(t, want[n], want[n + "_tol"], n)


def test_prefill_long_heads_of_the_8k_prompt():
    h = nsa.Heads(16, 1, 192, 128)
    q, k, v, cu = prompt([6000], h, 4)
    out, lse = run_prefill(q, k, v, cu, h, scale=0.11)
    want = R.prefill(q, k, v, [6000], 1, 0.11)
    R.assert_within(out, want["out"], want["out_tol"], "out")
    R.assert_within(lse, want["lse"], want["lse_tol"], "lse")


@pytest.mark.parametrize("dims,lens,Hq,Hk", [((192, 128), [700, 300], 16, 1), ((64, 64), [129, 64], 2, 1)])
def test_prefill_large_scores_and_growing_maxima(dims, lens, Hq, Hk):
    """Scores of some hundreds and row maxima that grow along the keys (every tile rescales)."""
    h = nsa.Heads(Hq, Hk, *dims)
    q, k, v, cu = prompt(lens, h, 8)
    ramp = torch.linspace(0.2, 6, q.shape[0], device="cuda").view(-1, 1, 1)
    k = (k.float().abs() * ramp).to(BF)
    q = q.float().abs().to(BF)
    out, lse = run_prefill(q, k, v, cu, h)
    want = R.prefill(q, k, v, lens, Hk, dims[0] ** -0.5)
    R.assert_within(out, want["out"], want["out_tol"], "out")
    R.assert_within(lse, want["lse"], want["lse_tol"], "lse")


def test_prefill_nan_of_one_sequence_stays_there():
    h = nsa.Heads(8, 2, 128, 128)
    lens = [200, 77, 300]
    q, k, v, cu = prompt(lens, h, 9, extra=64)
    ref, rlse = run_prefill(q, k, v, cu, h)
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    for t in (q2, k2, v2):
        t[200:277] = float("nan")
        t[577:] = float("inf")
    out, lse = run_prefill(q2, k2, v2, cu, h)
    keep = torch.cat([torch.arange(0, 200), torch.arange(277, 577)]).cuda()
    assert torch.equal(out[keep], ref[keep]) and torch.equal(lse[keep], rlse[keep])
    assert torch.isnan(out[200:277].float()).all()


def test_prefill_same_bits_again_on_another_stream_and_replayed():
    h = nsa.Heads(32, 4, 192, 128)
    lens = [900, 333]
    q, k, v, cu = prompt(lens, h, 10)
    out, lse = run_prefill(q, k, v, cu, h)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o2, l2 = run_prefill(q, k, v, cu, h, stream=st)
    st.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    ws = ws_for(nsa.NSA_OP_FULL_PREFILL, h, 2, sum(lens), 900)
    o3, l3 = torch.empty_like(out), torch.empty_like(lse)
    qs = q.clone()
    nsa.nsa_full_prefill(qs, k, v, cu, h, o3, l3, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nsa.nsa_full_prefill(qs, k, v, cu, h, o3, l3, ws)
    q_new = randn(q.shape, gen(77))
    want, wl = run_prefill(q_new, k, v, cu, h)
    qs.copy_(q_new)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o3, want) and torch.equal(l3, wl)


# ---------------------------------------------------------------- backward of the prompts

def run_backward(q, k, v, cu, h, do, scale=0.0, ws=None):
    N = int(cu[-1])
    out, lse = run_prefill(q, k, v, cu, h, scale)
    g = [torch.full_like(t, 9.0) for t in (q, k, v)]
    ws = ws_for(nsa.NSA_OP_FULL_BACKWARD, h, cu.numel() - 1, N, N) if ws is None else ws
    nsa.nsa_full_prefill_backward(q, k, v, out, lse, do, cu, h, *g, ws, scale=scale)
    nsa.nsa_check_device_status(ws)
    return g


def check_backward(q, k, v, lens, h, do, got, scale):
    N = sum(lens)
    want = R.prefill(q[:N], k[:N], v[:N], lens, h.H_kv, scale, do[:N])
    for t, n in zip(got, ("dq", "dk", "dv")):
        R.assert_within(t[:N], want[n], want[n + "_tol"], n)
        assert (t[N:] == 9).all()   # rows behind the last sequence


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("Hq,Hk,lens", [
    (4, 1, [1]), (16, 1, [129]), (2, 2, [300, 1, 0, 128, 127]), (8, 4, [64, 65, 511]), (16, 2, [513, 40]), (32, 4, [1100, 7, 600])])
def test_backward(dims, Hq, Hk, lens):
    h = nsa.Heads(Hq, Hk, *dims)
    q, k, v, cu = prompt(lens, h, 13, extra=3)
    do = randn((q.shape[0], Hq, dims[1]), gen(14))
    check_backward(q, k, v, lens, h, do, run_backward(q, k, v, cu, h, do), dims[0] ** -0.5)


def test_backward_long_and_scale():
    h = nsa.Heads(16, 1, 192, 128)
    q, k, v, cu = prompt([3000], h, 15)
    do = randn((3000, 16, 128), gen(16), scale=30)
    check_backward(q, k, v, [3000], h, do, run_backward(q, k, v, cu, h, do, 0.05), 0.05)


def test_backward_nan_of_one_sequence_stays_there():
    h = nsa.Heads(8, 2, 192, 128)
    lens = [200, 77, 300]
    q, k, v, cu = prompt(lens, h, 17, extra=130)
    do = randn((q.shape[0], 8, 128), gen(18))
    ref = run_backward(q, k, v, cu, h, do)
    bad = [t.clone() for t in (q, k, v, do)]
    for t in bad:
        t[200:277] = float("nan")
        t[577:] = float("inf")
    got = run_backward(bad[0], bad[1], bad[2], cu, h, bad[3])
    keep = torch.cat([torch.arange(0, 200), torch.arange(277, 577)]).cuda()
    for a, b in zip(got, ref):
        assert torch.equal(a[keep], b[keep])


def test_backward_same_bits_again_and_replayed():
    h = nsa.Heads(32, 4, 128, 128)
    lens = [900, 333]
    q, k, v, cu = prompt(lens, h, 19)
    do = randn((1233, 32, 128), gen(20))
    ref = run_backward(q, k, v, cu, h, do)
    assert all(torch.equal(a, b) for a, b in zip(ref, run_backward(q, k, v, cu, h, do)))
    ws = ws_for(nsa.NSA_OP_FULL_BACKWARD, h, 2, 1233, 900)
    out, lse = torch.empty_like(do), torch.empty((1233, 32), device="cuda")
    g = [torch.empty_like(t) for t in (q, k, v)]

    def step():
        nsa.nsa_full_prefill(q, k, v, cu, h, out, lse, ws)   # one workspace for both
        nsa.nsa_full_prefill_backward(q, k, v, out, lse, do, cu, h, *g, ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in g:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, g))


def test_prompts_past_32_bit_offsets():
    """128 sequences, 3.4e9 query elements: norm and rotation, attention and gradients of
    the last sequence, which lies beyond 2^31 in every tensor but the keys'."""
    h, L, B = nsa.Heads(64, 4, 192, 128), 2190, 128
    lens = [L + 9 * (b == 5) for b in range(B)]
    q, k, v, cu = prompt(lens, h, 23)
    N = sum(lens)
    assert N * 64 * 128 > 1 << 31
    g = gen(24)
    last = slice(N - L, N)
    w = 1 + 0.1 * randn((192,), g, torch.float32)
    f = torch.linspace(1, 1e-4, 48, device="cuda")
    pos = torch.arange(N, device="cuda", dtype=torch.int32)
    k_out = torch.empty_like(k)
    nsa.nsa_qk_norm_rope(q, k, w, w, f, pos, h, nsa.RopeParams(96, 0, 1e-6), q, k_out)   # queries in place
    x = prompt(lens, h, 23)[0][last]
    want = R.rope(x, w, f, pos[last], 96, False, 1e-6)
    big = (x.double().abs() * w.double()).amax(-1, keepdim=True) / torch.sqrt(x.double().square().mean(-1, keepdim=True))
    R.assert_within(q[last], want, rope_tol(want, 2 * big), "rope")
    del x, want, big
    out, lse = run_prefill(q, k_out, v, cu, h)
    do = randn((N, 64, 128), g)
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
    ws = ws_for(nsa.NSA_OP_FULL_BACKWARD, h, B, N, L + 9)
    nsa.nsa_full_prefill_backward(q, k_out, v, out, lse, do, cu, h, dq, dk, dv, ws)
    nsa.nsa_check_device_status(ws)
    r = R.prefill(q[last], k_out[last], v[last], [L], 4, 192 ** -0.5, do[last])
    for name, t in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        R.assert_within(t[last], r[name], r[name + "_tol"], name)


# ---------------------------------------------------------------- drafted tokens over a cache

def caches(lens, Lmax, h, seed, page=0, poison=True):
    """Contiguous caches and, with `page`, the same contents in shuffled pages. Rows
    past a length hold NaN and infinities."""
    g = gen(seed)
    B = len(lens)
    k, v = randn((B, Lmax, h.H_kv, h.d_k), g), randn((B, Lmax, h.H_kv, h.d_v), g)
    if poison:
        for b, L in enumerate(lens):
            k[b, L:], v[b, L:] = float("nan"), float("inf")
    if not page:
        return k, v, None, None, None
    per = Lmax // page
    perm = torch.randperm(B * per + 2, generator=g, device="cuda")[:B * per]
    kp = torch.full((B * per + 2, page, h.H_kv, h.d_k), float("nan"), dtype=BF, device="cuda")
    vp = torch.full((B * per + 2, page, h.H_kv, h.d_v), float("nan"), dtype=BF, device="cuda")
    kp[perm], vp[perm] = k.view(B * per, page, h.H_kv, h.d_k), v.view(B * per, page, h.H_kv, h.d_v)
    table = perm.to(torch.int32).view(B, per).contiguous()
    for b, L in enumerate(lens):   # entries that no length reaches
        table[b, -(-L // page):] = -7
    return k, v, kp, vp, table


def run_tree(q, kv, lens, nodes, masks, max_len, h, scale=0.0, paged=False, ws=None, lse=True):
    B, M = q.shape[:2]
    k, v, kp, vp, table = kv
    out = torch.full((B, M, h.H_q, h.d_v), 9.0, dtype=BF, device="cuda")
    ls = torch.full((B, M, h.H_q), 9.0, device="cuda") if lse else None
    ws = ws_for(nsa.NSA_OP_TREE_DECODE, h, B, 0, max_len, M) if ws is None else ws
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    nd = None if nodes is None else torch.tensor(nodes, dtype=torch.int32, device="cuda")
    md = None if masks is None else torch.tensor([R.as_int64(w) + [0] * (M - len(w)) for w in masks], device="cuda")
    if paged:
        nsa.nsa_full_tree_decode_paged(q, kp, vp, table, ld, nd, md, max_len, h, out, ls, ws, scale)
    else:
        nsa.nsa_full_tree_decode(q, k, v, ld, nd, md, max_len, h, out, ls, ws, scale)
    nsa.nsa_check_device_status(ws)
    return out, ls


def check_tree(out, lse, q, kv, lens, nodes, masks, h, scale):
    k, v = kv[0], kv[1]
    want = R.tree(q, lambda b, L: k[b, :L], lambda b, L: v[b, :L], lens, nodes, masks, h.H_kv, scale)
    for b, n in enumerate(nodes):
        if n:
            R.assert_within(out[b, :n], want[b]["out"], want[b]["tol"], f"out of sequence {b}")
            R.assert_within(lse[b, :n], want[b]["lse"], want[b]["lse_tol"], f"lse of sequence {b}")
        assert (out[b, n:] == 9).all() and (lse[b, n:] == 9).all()   # rows past the last node


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("Hq,Hk,M,lens,nodes,page", [
    (4, 1, 1, [1, 64, 65, 128, 129], [1] * 5, 0),
    (16, 1, 1, [3000, 1, 777], [1] * 3, 64),
    (16, 2, 8, [8, 500, 1000, 0], [8, 5, 1, 0], 0),
    (32, 2, 64, [64, 700, 130], [64, 63, 17], 128),
    (8, 8, 64, [200, 64, 65, 1023], [64, 64, 2, 33], 256),
    (16, 4, 33, [2100], [33], 0)])
def test_tree(dims, Hq, Hk, M, lens, nodes, page):
    h = nsa.Heads(Hq, Hk, *dims)
    Lmax = -(-max(lens) // 256) * 256
    kv = caches(lens, Lmax, h, 31 + M, page)
    q = randn((len(lens), M, Hq, dims[0]), gen(M))
    cpu = torch.Generator().manual_seed(M)
    masks = [R.random_tree(n, cpu) for n in nodes]
    out, lse = run_tree(q, kv, lens, nodes, masks, max(lens), h)
    check_tree(out, lse, q, kv, lens, nodes, masks, h, dims[0] ** -0.5)
    if page:
        po, pl = run_tree(q, kv, lens, nodes, masks, max(lens), h, paged=True)
        assert torch.equal(po, out) and torch.equal(pl, lse)


def test_tree_chain_equals_mask_and_matches_prompt():
    """The chain (no mask) equals its mask, and the last rows of a prompt."""
    h = nsa.Heads(16, 4, 128, 64)
    L, M = 400, 20
    q, k, v, cu = prompt([L], h, 12)
    want, wl = run_prefill(q, k, v, cu, h)
    Lmax = 512
    kc, vc = torch.full((1, Lmax, 4, 128), float("nan"), dtype=BF, device="cuda"), torch.full((1, Lmax, 4, 64), float("nan"), dtype=BF, device="cuda")
    kc[0, :L], vc[0, :L] = k, v
    qt = q[L - M:].unsqueeze(0).contiguous()
    a = run_tree(qt, (kc, vc, None, None, None), [L], [M], None, Lmax, h)
    b = run_tree(qt, (kc, vc, None, None, None), [L], None, [[(2 << i) - 1 for i in range(M)]], L, h)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    r = R.prefill(q, k, v, [L], 4, 128 ** -0.5)
    R.assert_within(a[0][0], r["out"][L - M:], r["out_tol"][L - M:], "chain")
    R.assert_within(a[1][0], r["lse"][L - M:], r["lse_tol"][L - M:], "chain lse")


@pytest.mark.parametrize("Lmax", [77, 129, 200])
def test_tree_caches_of_odd_length(Lmax):
    """Tiles reach into the next sequence's rows, which hold NaN, and past the cache."""
    h = nsa.Heads(16, 4, 192, 64)
    lens, nodes = [Lmax, 70, Lmax - 1, 1], [3, 2, 3, 1]
    kv = caches(lens, Lmax, h, 44)
    q = randn((4, 3, 16, 192), gen(3))
    out, lse = run_tree(q, kv, lens, nodes, None, Lmax, h)
    check_tree(out, lse, q, kv, lens, nodes, None, h, 192 ** -0.5)


def test_tree_128_sequences():
    h = nsa.Heads(4, 2, 64, 64)
    lens = [1 + (53 * i) % 700 for i in range(128)]
    nodes = [min(L, i % 5) for i, L in enumerate(lens)]
    kv = caches(lens, 704, h, 45, page=64)
    q = randn((128, 4, 4, 64), gen(4))
    a = run_tree(q, kv, lens, nodes, None, 700, h)
    check_tree(*a, q, kv, lens, nodes, None, h, 0.125)
    b = run_tree(q, kv, lens, nodes, None, 700, h, paged=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tree_rows_that_see_nothing():
    """No prefix and masks without bits: zeros and -infinity."""
    h = nsa.Heads(8, 2, 64, 64)
    lens, nodes = [6, 300], [6, 6]
    kv = caches(lens, 512, h, 41)
    q = randn((2, 6, 8, 64), gen(2))
    masks = [[0, 1 << 1, 0, 1 << 40, 1 << 63, (1 << 6) - 1], [0, 0, 1, 2, 4, 0]]
    out, lse = run_tree(q, kv, lens, nodes, masks, 300, h)
    check_tree(out, lse, q, kv, lens, nodes, masks, h, 64 ** -0.5)
    assert (out[0, 0] == 0).all() and (lse[0, 0] == -math.inf).all() and (out[0, 3] == 0).all()


def test_tree_long_caches_split_over_all_blocks():
    """One long sequence cut into 148 runs, and many short ones of a few tiles."""
    h = nsa.Heads(16, 1, 192, 128)
    for lens, M in (([50001], 3), ([130 + 17 * i for i in range(100)], 1)):
        kv = caches(lens, -(-max(lens) // 64) * 64, h, 51)
        q = randn((len(lens), M, 16, 192), gen(5))
        out, lse = run_tree(q, kv, lens, [M] * len(lens), None, max(lens), h)
        check_tree(out, lse, q, kv, lens, [M] * len(lens), None, h, 192 ** -0.5)


def test_tree_offsets_past_32_bits():
    """A cache of more than 2^32 elements: the last sequence lies beyond."""
    h = nsa.Heads(16, 8, 192, 128)
    Lmax, B = 1 << 17, 22   # 22 * 2^17 * 8 * 192 = 4.4e9 elements
    k = torch.zeros((B, Lmax, 8, 192), dtype=BF, device="cuda")
    v = torch.zeros((B, Lmax, 8, 128), dtype=BF, device="cuda")
    g = gen(3)
    L = 300
    k[-1, :L], v[-1, :L] = randn((L, 8, 192), g), randn((L, 8, 128), g)
    lens, nodes = [0] * (B - 1) + [L], [0] * (B - 1) + [2]
    q = randn((B, 2, 16, 192), g)
    out, lse = run_tree(q, (k, v, None, None, None), lens, nodes, None, Lmax, h)
    check_tree(out, lse, q, (k, v), lens, nodes, None, h, 192 ** -0.5)


def test_tree_lengths_out_of_range_are_recorded():
    h = nsa.Heads(8, 2, 64, 64)
    kv = caches([100, 100, 100, 100], 128, h, 61, poison=False)
    q = randn((4, 4, 8, 64), gen(8))
    for lens, nodes in (([100, 101, 50, 60], [4, 4, 4, 4]), ([100, 3, 50, 60], [4, 4, 4, 4]),
                        ([100, 70, 50, 60], [4, 5, 4, 4]), ([100, 70, 50, 60], [4, -1, 4, 4]), ([100, -3, 50, 60], [4, 0, 4, 4])):
        ws = ws_for(nsa.NSA_OP_TREE_DECODE, h, 4, 0, 100, 4)
        with pytest.raises(nsa.NSAError) as e:
            run_tree(q, kv, lens, nodes, None, 100, h, ws=ws)
        assert e.value.status == nsa.NSA_ERR_DEVICE_CHECK
        ok = [100, 70, 50, 60]
        good, gl = run_tree(q, kv, ok, [4, 0, 4, 4], None, 100, h, ws=ws)
        check_tree(good, gl, q, kv, ok, [4, 0, 4, 4], None, h, 0.125)


def test_tree_bad_page_is_recorded():
    h = nsa.Heads(8, 2, 64, 64)
    kv = list(caches([100, 200], 256, h, 62, page=64))
    kv[2] = torch.nan_to_num(kv[2], 0, 0, 0)
    kv[3] = torch.nan_to_num(kv[3], 0, 0, 0)
    kv[4][1, 1] = 1000
    q = randn((2, 1, 8, 64), gen(8))
    with pytest.raises(nsa.NSAError) as e:
        run_tree(q, kv, [100, 200], [1, 1], None, 200, h, paged=True)
    assert e.value.status == nsa.NSA_ERR_DEVICE_CHECK


def test_tree_captured_graphs_share_a_workspace():
    """Two captured calls on one workspace, replayed in turn with changed lengths."""
    h = nsa.Heads(16, 2, 128, 128)
    B, M, Lmax = 3, 5, 1024
    kv = caches([Lmax] * B, Lmax, h, 71, poison=False)
    ws = ws_for(nsa.NSA_OP_TREE_DECODE, h, B, 0, Lmax, M)
    q = [randn((B, M, 16, 128), gen(80 + i)) for i in range(2)]
    ld = torch.tensor([900, 10, 500], dtype=torch.int32, device="cuda")
    nd = torch.tensor([5, 3, 1], dtype=torch.int32, device="cuda")
    outs = [torch.full((B, M, 16, 128), 9.0, dtype=BF, device="cuda") for _ in range(2)]
    graphs = []
    for i in range(2):
        nsa.nsa_full_tree_decode(q[i], kv[0], kv[1], ld, nd, None, Lmax, h, outs[i], None, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            nsa.nsa_full_tree_decode(q[i], kv[0], kv[1], ld, nd, None, Lmax, h, outs[i], None, ws)
        graphs.append(g)
    for lens, nodes in (([5, 1000, 77], [5, 5, 2]), ([1024, 1, 300], [4, 1, 5])):
        ld.copy_(torch.tensor(lens, dtype=torch.int32))
        nd.copy_(torch.tensor(nodes, dtype=torch.int32))
        for i in (0, 1, 0):
            outs[i].fill_(9.0)
            graphs[i].replay()
        for i in range(2):
            want, _ = run_tree(q[i], kv, lens, nodes, None, Lmax, h)
            assert torch.equal(outs[i], want)
