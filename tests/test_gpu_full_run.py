"""Runs of the full-attention operators together, as a training layer and a serving
step use them, beside the sparse operators, on several streams and captured."""
import threading

import pytest
import torch

import sparse_attention_long_nsa_b200 as nsa
from tests import full_ref as R
from tests.test_gpu_full import gen, prompt, randn, rope_tol, run_backward, run_prefill, run_tree, ws_for

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def freqs(d_rot):
    i = torch.arange(d_rot // 2, device="cuda", dtype=torch.float64)
    return (500000.0 ** (-2 * i / d_rot)).float()


def test_training_layer():
    """Projections -> norm and rotation -> attention -> gradients of everything, each
    stage against its fp64 form on the inputs it was given."""
    h, lens, d_rot = nsa.Heads(16, 2, 128, 128), [333, 1, 200], 96
    N = sum(lens)
    g = gen(1)
    x = randn((N, (16 + 2 * 2) * 128), g)
    q, k, v = (x[:, a:b].unflatten(1, (-1, 128)) for a, b in ((0, 2048), (2048, 2304), (2304, 2560)))
    w_q, w_k = 1 + 0.2 * randn((128,), g, torch.float32), 1 + 0.2 * randn((128,), g, torch.float32)
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    f, rp = freqs(d_rot), nsa.RopeParams(d_rot, 0, 1e-6)
    cu = torch.tensor([0, 333, 334, 534], dtype=torch.int32)
    qr, kr, vr = (torch.empty((N, n, 128), dtype=BF, device="cuda") for n in (16, 2, 2))
    nsa.nsa_qk_norm_rope(q, k, w_q, w_k, f, pos, h, rp, qr, kr, v, vr)
    out, lse = run_prefill(qr, kr, vr, cu, h)
    do = randn((N, 16, 128), g)
    gq, gk, gv = run_backward(qr, kr, vr, cu, h, do)
    dx = torch.zeros_like(x)
    dq, dk = dx[:, :2048].unflatten(1, (-1, 128)), dx[:, 2048:2304].unflatten(1, (-1, 128))
    dwq, dwk = torch.empty_like(w_q), torch.empty_like(w_k)
    nsa.nsa_qk_norm_rope_backward(q, k, w_q, w_k, f, pos, gq, gk, h, rp, dq, dk, dwq, dwk,
                                  ws_for(nsa.NSA_OP_ROPE_BACKWARD, h, 1, N))
    r = R.prefill(qr, kr, vr, lens, 2, 128 ** -0.5, do)
    for name, got in (("out", out), ("lse", lse), ("dq", gq), ("dk", gk), ("dv", gv)):
        R.assert_within(got, r[name], r[name + "_tol"], name)
    for t, dt, w, dw, gr in ((q, dq, w_q, dwq, gq), (k, dk, w_k, dwk, gk)):
        want, wdw, mag = R.rope_backward(t, w, f, pos, d_rot, False, 1e-6, gr)
        rms = 1 / torch.sqrt(t.double().square().mean(-1, keepdim=True) + 1e-6)
        row = rms * gr.double().abs().amax(-1, keepdim=True) * 2 * w.double().abs().max() * (1 + t.double().abs().amax(-1, keepdim=True) * rms)
        R.assert_within(dt, want, R.U * want.abs() * 1.01 + 192 * R.E * row, "projection gradient")
        R.assert_within(dw, wdw, (64 + 8 * (N * t.shape[1]) ** 0.5) * R.E * mag * 2, "weight gradient")


def test_serving_prompt_then_drafts_on_a_paged_cache():
    """Prompts written to pages through cache_rows, then a tree of drafts written behind
    them and verified; a sequence without drafts stays out (padding rows)."""
    h, d_rot, page, B, M = nsa.Heads(16, 2, 192, 128), 64, 64, 3, 7
    lens, nodes = [200, 63, 130], [7, 0, 4]
    g, cpu = gen(2), torch.Generator().manual_seed(2)
    per = 6
    kp, vp = (torch.full((B * per, page, 2, d), float("nan"), dtype=BF, device="cuda") for d in (192, 128))
    table = torch.randperm(B * per, generator=g, device="cuda").int().view(B, per).contiguous()
    w_q, w_k = 1 + 0.2 * randn((192,), g, torch.float32), 1 + 0.2 * randn((192,), g, torch.float32)
    f, rp = freqs(d_rot), nsa.RopeParams(d_rot, 1, 1e-6)

    def rows_of(b, t):
        return (table[b].long()[t // page] * page + t % page)

    # the prompts
    N = sum(lens)
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)]).cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).cuda()
    rows = torch.cat([rows_of(b, torch.arange(n, device="cuda")) for b, n in enumerate(lens)])
    q, k, v = randn((N, 16, 192), g), randn((N, 2, 192), g), randn((N, 2, 128), g)
    qr = torch.empty_like(q)
    nsa.nsa_qk_norm_rope(q, k, w_q, w_k, f, pos.int(), h, rp, qr, kp, v, vp, rows)
    want_k = R.rope(k, w_k, f, pos, d_rot, True, 1e-6)
    got_k = kp.view(-1, 2, 192)[rows]
    big = k.double().abs().amax(-1, keepdim=True) * w_k.abs().max() / torch.sqrt(k.double().square().mean(-1, keepdim=True))
    R.assert_within(got_k, want_k, rope_tol(want_k, 2 * big), "cached keys")
    assert torch.equal(vp.view(-1, 2, 128)[rows], v)
    assert int(torch.isfinite(kp.view(-1, 2, 192)[:, 0, 0]).sum()) == N      # no other row was written
    cu = torch.tensor([0, 200, 263, 393], dtype=torch.int32)
    out, lse = run_prefill(qr, got_k.contiguous(), v, cu, h)
    # drafts: positions by depth, padded slots with row -1
    words = [R.random_tree(n, cpu) for n in nodes]
    depth = [[bin(w).count("1") - 1 for w in ws] + [0] * (M - len(ws)) for ws in words]
    dpos = torch.tensor([[lens[b] + depth[b][i] for i in range(M)] for b in range(B)], device="cuda")
    drows = torch.stack([torch.cat([rows_of(b, lens[b] + torch.arange(nodes[b], device="cuda")),
                                    torch.full((M - nodes[b],), -1, device="cuda")]) for b in range(B)])
    dq, dk, dv = randn((B * M, 16, 192), g), randn((B * M, 2, 192), g), randn((B * M, 2, 128), g)
    dqr = torch.empty_like(dq)
    nsa.nsa_qk_norm_rope(dq, dk, w_q, w_k, f, dpos.int().flatten(), h, rp, dqr, kp, dv, vp, drows.flatten().contiguous())
    assert int(torch.isfinite(kp.view(-1, 2, 192)[:, 0, 0]).sum()) == N + sum(nodes)
    full = [a + b for a, b in zip(lens, nodes)]
    o, l = run_tree(dqr.view(B, M, 16, 192), (None, None, kp, vp, table), full, nodes, words, max(full), h, paged=True)
    kof = lambda b, L: kp.view(-1, 2, 192)[rows_of(b, torch.arange(L, device="cuda"))]   # noqa: E731
    vof = lambda b, L: vp.view(-1, 2, 128)[rows_of(b, torch.arange(L, device="cuda"))]   # noqa: E731
    r = R.tree(dqr.view(B, M, 16, 192), kof, vof, full, nodes, words, 2, 192 ** -0.5)
    for b in r:
        R.assert_within(o[b, :nodes[b]], r[b]["out"], r[b]["tol"], f"drafts of {b}")
        R.assert_within(l[b, :nodes[b]], r[b]["lse"], r[b]["lse_tol"], f"lse of {b}")
    # the path to a node, as a prompt, ends in the node's result
    b, i = 0, 6
    path = [j for j in range(7) if (words[0][i] >> j) & 1]
    kk = torch.cat([kof(0, 200), kof(0, 207)[[200 + j for j in path]]])
    vv = torch.cat([vof(0, 200), vof(0, 207)[[200 + j for j in path]]])
    qq = torch.cat([qr[:200], dqr.view(B, M, 16, 192)[0, path]])
    po, _ = run_prefill(qq, kk, vv, torch.tensor([0, len(kk)], dtype=torch.int32), h)
    tol = r[0]["tol"][i]
    R.assert_within(po[-1], o[0, i].double(), 2 * tol, "path as a prompt")


@pytest.mark.parametrize("dims,Hq,Hk,T", [((64, 64), 4, 1, 500), ((192, 128), 16, 1, 700)])
def test_sparse_prefill_with_a_full_window_is_full_attention(dims, Hq, Hk, T):
    """The sparse prefill with its gate on a window over the whole prompt: the same
    attention, both within the bound of the fp64 result."""
    h = nsa.Heads(Hq, Hk, *dims)
    q, k, v, cu = prompt([T], h, 7)
    p = nsa.make_params(top_n=4, window=T)
    g = gen(8)
    dk, dv = dims
    kc, vc = nsa.compress(k, v, randn((32 * dk, dk), g, torch.float32, 0.02), randn((32, dk), g, torch.float32, 0.02),
                          randn((32 * dv, dv), g, torch.float32, 0.02), randn((32, dv), g, torch.float32, 0.02), [T], h, p)
    gates = torch.zeros((T, Hq, 3), device="cuda")
    gates[..., 2] = 1
    sparse = nsa.prefill(q, k, v, kc, vc, gates, cu, h, p)
    out, lse = run_prefill(q, k, v, cu, h)
    r = R.prefill(q, k, v, [T], Hk, dk ** -0.5)
    R.assert_within(out, r["out"], r["out_tol"], "full")
    R.assert_within(sparse, r["out"], r["out_tol"], "sparse with a full window")


def test_calls_of_two_threads_on_two_streams():
    h = nsa.Heads(16, 2, 128, 64)
    jobs = []
    for i in range(2):
        lens = [700 + 100 * i, 33]
        q, k, v, cu = prompt(lens, h, 30 + i)
        do = randn((sum(lens), 16, 64), gen(40 + i))
        jobs.append((q, k, v, cu, do, run_backward(q, k, v, cu, h, do)))
    torch.cuda.synchronize()
    got, errs = [None, None], []

    def work(i):
        try:
            q, k, v, cu, do, _ = jobs[i]
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(20):
                    got[i] = run_backward(q, k, v, cu, h, do)
            st.synchronize()
        except Exception as e:   # noqa: BLE001
            errs.append(e)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not errs, errs
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], jobs[i][5]))


def test_captured_norm_rope_and_gradient():
    h, rp = nsa.Heads(8, 2, 64, 64), nsa.RopeParams(64, 0, 1e-6)
    g = gen(50)
    N = 40
    q, k = randn((N, 8, 64), g), randn((N, 2, 64), g)
    w = 1 + 0.1 * randn((64,), g, torch.float32)
    pos, f = torch.arange(N, device="cuda", dtype=torch.int32), freqs(64)
    bufs = [torch.empty_like(t) for t in (q, k, q, k)] + [torch.empty_like(w) for _ in range(2)]
    ws = ws_for(nsa.NSA_OP_ROPE_BACKWARD, h, 1, N)

    def step():
        nsa.nsa_qk_norm_rope(q, k, w, w, f, pos, h, rp, bufs[0], bufs[1])
        nsa.nsa_qk_norm_rope_backward(q, k, w, w, f, pos, bufs[0], bufs[1], h, rp, bufs[2], bufs[3], bufs[4], bufs[5], ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    q.copy_(randn((N, 8, 64), gen(51)))
    pos.add_(1000)
    step()
    want = [t.clone() for t in bufs]
    for t in bufs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bufs, want))


def test_empty_inputs():
    h, rp = nsa.Heads(8, 2, 64, 64), nsa.RopeParams(32, 0, 1e-6)
    e = lambda *s: torch.empty(s, dtype=BF, device="cuda")   # noqa: E731
    w, f = torch.ones(64, device="cuda"), freqs(32)
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    nsa.nsa_qk_norm_rope(e(0, 8, 64), e(0, 2, 64), w, w, f, pos, h, rp, e(0, 8, 64), e(5, 2, 64))
    dw = [torch.full((64,), 5.0, device="cuda") for _ in range(2)]
    nsa.nsa_qk_norm_rope_backward(e(0, 8, 64), e(0, 2, 64), w, w, f, pos, e(0, 8, 64), e(0, 2, 64), h, rp, e(0, 8, 64),
                                  e(0, 2, 64), *dw, ws_for(nsa.NSA_OP_ROPE_BACKWARD, h))
    assert (dw[0] == 0).all() and (dw[1] == 0).all()
    cu = torch.zeros(3, dtype=torch.int32)
    out, lse = run_prefill(e(4, 8, 64), e(4, 2, 64), e(4, 2, 64), cu, h)
    assert (out == 9).all() and (lse == 9).all()
    run_prefill(e(0, 8, 64), e(0, 2, 64), e(0, 2, 64), cu, h)


def test_binding_refusals():
    h = nsa.Heads(8, 2, 64, 64)
    q, k, v, cu = prompt([20], h, 60)
    out, ws = torch.empty_like(q), ws_for(nsa.NSA_OP_FULL_PREFILL, h, 1, 20, 20)
    for bad, err in (((q.float(), k, v), TypeError), ((q, k.transpose(1, 2).contiguous(), v), ValueError),
                     ((q.transpose(0, 1).contiguous().transpose(0, 1), k, v), ValueError), ((q[:10].contiguous(), k, v), ValueError),
                     ((q, k, v.cpu()), ValueError)):
        with pytest.raises(err):
            nsa.nsa_full_prefill(*bad, cu, h, out, None, ws)
    with pytest.raises(ValueError, match="ws"):
        nsa.nsa_full_prefill(q, k, v, cu, h, out)
    with pytest.raises(nsa.NSAError) as e:
        nsa.nsa_full_prefill(q, k, v, cu, h, out, None, ws[:128])
    assert e.value.status == nsa.NSA_ERR_WORKSPACE
    rp, w, f = nsa.RopeParams(32, 0, 1e-6), torch.ones(64, device="cuda"), freqs(32)
    pos = torch.arange(20, device="cuda", dtype=torch.int32)
    ko = torch.empty((15, 2, 64), dtype=BF, device="cuda")
    with pytest.raises(nsa.NSAError) as e:      # fewer rows than tokens and no cache_rows
        nsa.nsa_qk_norm_rope(q, k, w, w, f, pos, h, rp, out, ko)
    assert e.value.status == nsa.NSA_ERR_INVALID_ARG
    for kw in (dict(positions=pos.long()), dict(positions=pos[:10]), dict(inv_freq=f[:8]), dict(cache_rows=pos),
               dict(v=v), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        a = dict(q=q, k=k, w_q=w, w_k=w, inv_freq=f, positions=pos, heads=h, rope=rp, q_out=out, k_out=torch.empty_like(k)) | kw
        with pytest.raises((ValueError, TypeError)):
            nsa.nsa_qk_norm_rope(**a)


def test_checking_build_agrees():
    """The checking build (20 ms wait limit) gives the same bits and records nothing."""
    h = nsa.Heads(16, 2, 192, 128)
    q, k, v, cu = prompt([600, 77], h, 70)
    do = randn((677, 16, 128), gen(71))
    kc, vc = k[:640].unsqueeze(0).contiguous(), v[:640].unsqueeze(0).contiguous()
    qt = q[:12].unsqueeze(0).contiguous()
    run = lambda: [*run_prefill(q, k, v, cu, h), *run_backward(q, k, v, cu, h, do),   # noqa: E731
                   *run_tree(qt, (kc, vc, None, None, None), [640], [12], None, 640, h)]
    want = run()
    with nsa.checking_library():
        got = run()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("what", ["prompt", "short prompt", "drafts", "gradient"])
def test_withheld_tile_is_recorded_and_the_next_call_is_right(what):
    """Checking build: a loader withholds a tile, the waits on it run out (20 ms), the
    status word says so; the next call on the same workspace is right again."""
    h = nsa.Heads(16, 2, 128, 128)
    T = 70 if what == "short prompt" else 1500
    q, k, v, cu = prompt([T], h, 80)
    do = randn((T, 16, 128), gen(81))
    out, lse = run_prefill(q, k, v, cu, h)
    ws = nsa.alloc_workspace(max(nsa.nsa_full_workspace_size(nsa.NSA_OP_FULL_BACKWARD, h, 1, T, T, 0),
                                 nsa.nsa_full_workspace_size(nsa.NSA_OP_TREE_DECODE, h, 1, 0, T, 4)), "cuda")
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")

    def call():
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        g = [torch.zeros_like(t) for t in (q, k, v)]
        if what == "gradient":
            nsa.nsa_full_prefill_backward(q, k, v, out, lse, do, cu, h, *g, ws)
        elif what == "drafts":
            o = torch.zeros((1, 4, 16, 128), dtype=BF, device="cuda")
            nsa.nsa_full_tree_decode(q[T - 4:].unsqueeze(0).contiguous(), k.unsqueeze(0), v.unsqueeze(0), lens, None, None, T, h, o,
                                     None, ws)
        else:
            nsa.nsa_full_prefill(q, k, v, cu, h, o, l, ws)
        nsa.nsa_check_device_status(ws)
        return [o, l, *g]
    want = call()
    with nsa.checking_library():
        nsa.nsa_test_set_fault(nsa.FAULT_FULL_BWD_TILE if what == "gradient" else nsa.FAULT_FULL_TILE)
        try:
            with pytest.raises(nsa.NSAError) as e:
                call()
            assert e.value.status == nsa.NSA_ERR_DEVICE_CHECK
        finally:
            nsa.nsa_test_set_fault(nsa.FAULT_NONE)
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
