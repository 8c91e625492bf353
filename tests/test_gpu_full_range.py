"""Full-attention operators on the GPU over more of their range: large scores in the
gradients, scales of the drafted tokens, long sequences, masks made on the device.

Bounds are those of tests/full_ref.py. One term is added where scores are large: delta
takes the forward's out, whose P was rounded to bf16 as well, so it is off by
  sum_j p_j (u + 2 max|ds| + L e) |dO . v_j|
(u, e as there), which reaches dS as scale p_j times that. With unit-normal scores the
roundings of many p average out; with one or two keys that carry a row they need not."""
import pytest
import torch

import sparse_attention_long_nsa_b200 as nsa
from tests import full_ref as R
from tests.test_gpu_full import BF, caches, check_tree, gen, prompt, randn, run_backward, run_prefill, run_tree

pytestmark = pytest.mark.gpu


def gradients(q, k, v, see, scale, do):
    """R.attention_backward with the added term."""
    g, e = R.attention_backward(q, k, v, see, scale, do)
    p = R.attention(q, k, v, see, scale)["p"]
    ds = scale * q.shape[1] * R.E * (q.double().abs() @ k.double().abs().T).amax(1, keepdim=True)
    d = scale * p * ((R.U + 2 * ds + k.shape[0] * R.E) * (p * (do.double() @ v.double().T).abs()).sum(1, keepdim=True))
    e["dq"] = e["dq"] + d @ k.double().abs()
    e["dk"] = e["dk"] + d.T @ q.double().abs()
    return g, e


def final(g, e):
    return 1.05 * (e + R.U * (g.abs() + e)) + 1e-30


def check_all(q, k, v, do, lens, h, scale, got, rows=4096):
    """out, lse and gradients of every sequence and head, `rows` query rows at a time."""
    out, lse, dq, dk, dv = got
    G, at = h.H_q // h.H_kv, 0
    for L in lens:
        sl = slice(at, at + L)
        for c in range(h.H_kv):
            f = dict(dtype=torch.float64, device="cuda")
            sums = {n: [torch.zeros((L, d), **f), torch.zeros((L, d), **f)] for n, d in (("dk", h.d_k), ("dv", h.d_v))}
            for hq in range(c * G, (c + 1) * G):
                for r0 in range(0, L, rows):
                    r1 = min(L, r0 + rows)
                    rs = slice(at + r0, at + r1)
                    see = torch.arange(r1, device="cuda")[None] <= torch.arange(r0, r1, device="cuda")[:, None]
                    ks, vs = k[at:at + r1, c], v[at:at + r1, c]       # later keys are seen by none of the rows
                    x = R.attention(q[rs, hq], ks, vs, see, scale)
                    R.assert_within(out[rs, hq], x["out"], x["tol"], "out")
                    R.assert_within(lse[rs, hq], x["lse"], x["lse_tol"], "lse")
                    del x
                    g, e = gradients(q[rs, hq], ks, vs, see, scale, do[rs, hq])
                    R.assert_within(dq[rs, hq], g["dq"], final(g["dq"], e["dq"]), "dq")
                    for n, (s, t) in sums.items():
                        s[:r1] += g[n]
                        t[:r1] += e[n]
            for (n, (s, t)), got_n in zip(sums.items(), (dk, dv)):
                R.assert_within(got_n[sl, c], s, final(s, t + L * G * R.E * s.abs()), n)
        at += L


def run_all(q, k, v, cu, h, do, scale=0.0):
    return *run_prefill(q, k, v, cu, h, scale), *run_backward(q, k, v, cu, h, do, scale)


@pytest.mark.parametrize("dims,lens,Hq,Hk", [((192, 128), [700, 300], 16, 1), ((64, 64), [129, 64, 1], 2, 1),
                                             ((128, 64), [513], 8, 2)])
@pytest.mark.parametrize("what", ["growing maxima", "all scores near 300"])
def test_backward_large_scores(dims, lens, Hq, Hk, what):
    """exp(s - lse) where both are some hundreds: rows that one or two keys carry, and
    rows whose keys all share a large common score."""
    h = nsa.Heads(Hq, Hk, *dims)
    q, k, v, cu = prompt(lens, h, 41)
    if what == "growing maxima":
        ramp = torch.linspace(0.2, 40, q.shape[0], device="cuda").view(-1, 1, 1)
        q, k = q.float().abs().to(BF), (k.float().abs() * ramp).to(BF)
    else:   # a common part of 300 in every score, and a part of about one
        common = (300 * dims[0] ** 0.5 / dims[0]) ** 0.5
        q, k = (q.float() + common).to(BF), (k.float() * 0.3 + common).to(BF)
    do = randn((q.shape[0], Hq, dims[1]), gen(42))
    got = run_all(q, k, v, cu, h, do)
    assert float(got[1].abs().max()) > 150
    check_all(q, k, v, do, lens, h, dims[0] ** -0.5, got)


@pytest.mark.parametrize("dims,Hq,Hk,lens", [((64, 64), 4, 1, [65536]), ((192, 128), 16, 1, [20011, 1, 4100]),
                                             ((128, 128), 2, 2, [130, 40001])])
def test_long_sequences(dims, Hq, Hk, lens):
    h = nsa.Heads(Hq, Hk, *dims)
    q, k, v, cu = prompt(lens, h, 43)
    do = randn((q.shape[0], Hq, dims[1]), gen(44))
    check_all(q, k, v, do, lens, h, dims[0] ** -0.5, run_all(q, k, v, cu, h, do))


@pytest.mark.parametrize("scale", [0.31, 0.004])
@pytest.mark.parametrize("dims,Hq,Hk,M,lens,page", [
    ((192, 128), 16, 1, 3, [40000], 64),           # cut into runs, 128 rows
    ((128, 64), 16, 1, 20, [9000, 33, 500], 128),  # cut into runs, 256 rows, two blocks
    ((64, 64), 4, 2, 7, [100, 7], 0)])             # not cut
def test_tree_scale(dims, Hq, Hk, M, lens, page, scale):
    h = nsa.Heads(Hq, Hk, *dims)
    kv = caches(lens, -(-max(lens) // 128) * 128, h, 45, page)
    q = randn((len(lens), M, Hq, dims[0]), gen(46))
    cpu = torch.Generator().manual_seed(47)
    masks = [R.random_tree(M, cpu) for _ in lens]
    nodes = [M] * len(lens)
    out, lse = run_tree(q, kv, lens, nodes, masks, max(lens), h, scale)
    check_tree(out, lse, q, kv, lens, nodes, masks, h, scale)
    if page:
        po, pl = run_tree(q, kv, lens, nodes, masks, max(lens), h, scale, paged=True)
        assert torch.equal(po, out) and torch.equal(pl, lse)


def test_tree_mask_from_parents_on_the_device():
    g = torch.Generator().manual_seed(5)
    p = torch.tensor([[-1] + [int(torch.randint(-1, i, (1,), generator=g)) for i in range(1, 64)] for _ in range(5)])
    want = nsa.tree_mask_from_parents(p)
    for t in (p, p.to(torch.int32)):
        got = nsa.tree_mask_from_parents(t.cuda())
        assert got.device.type == "cuda" and got.dtype == torch.int64 and torch.equal(got.cpu(), want)
    with pytest.raises(ValueError):
        nsa.tree_mask_from_parents(torch.tensor([[-1, 1]], device="cuda"))
