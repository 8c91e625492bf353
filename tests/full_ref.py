"""Plain fp64 forms of the full-attention operators (any torch device), with the
error bounds their bf16 results are held to. They share no code with the kernels.

Bounds, u = 2^-8 (half a bf16 step, relative), e = 2^-24 (half an fp32 step):
  scores    |ds| <= scale * d_k * e * sum_i |q_i k_i|  (fp32 accumulation)
  out       P is rounded to bf16 for the product with V and the result once more:
            u sum_j p_j |v_j| + u |o|, and the scores' error moves every p_j by
            at most 2 max|ds| relative
  lse       max|ds| + L e (the sum) + 2^-21 (exp2 and log2 of the hardware)
  gradients P and dS are rounded to bf16 for their products and the results once
            more; delta = sum dO o takes the rounded o: |d delta| <= u sum |dO| |o|
A factor of 1.05 covers second-order terms, and fp32 sums of up to n terms add n e.
"""
import math

import torch

U, E = 2.0 ** -8, 2.0 ** -24


def rope(x, w, inv_freq, pos, d_rot, interleaved, eps):
    """x [N, H, d] -> fp64 result of norm and rotation."""
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    return turn(y, inv_freq, pos, d_rot, interleaved, 1)


def turn(y, inv_freq, pos, d_rot, interleaved, sign):
    if d_rot == 0:
        return y
    a = pos.double()[:, None] * inv_freq.double()[None]
    c, s = torch.cos(a)[:, None], sign * torch.sin(a)[:, None]
    i = torch.arange(d_rot // 2, device=y.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + d_rot // 2)
    out = y.clone()
    out[..., ia] = y[..., ia] * c - y[..., ib] * s
    out[..., ib] = y[..., ia] * s + y[..., ib] * c
    return out


def rope_backward(x, w, inv_freq, pos, d_rot, interleaved, eps, dy):
    x, w = x.double(), w.double()
    d = x.shape[-1]
    dn = turn(dy.double(), inv_freq, pos, d_rot, interleaved, -1)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    u = dn * w
    dx = r * u - x * r ** 3 * (u * x).sum(-1, keepdim=True) / d
    return dx, (dn * x * r).sum((0, 1)), (dn * x * r).abs().sum((0, 1))


def attention(q, k, v, see, scale):
    """q [R, d], k [L, d], v [L, dv], see bool [R, L] -> out, lse and their bounds.
    Keys that no row sees are not read."""
    q, k, v = q.double(), k.double(), v.double()
    live = see.any(0)
    k = torch.where(live[:, None], k, 0.0)
    v = torch.where(live[:, None], v, 0.0)
    s = torch.where(see, scale * (q @ k.T), -math.inf)
    ds = scale * q.shape[1] * E * (q.abs() @ k.abs().T).amax(1)
    lse = torch.logsumexp(s, 1)
    p = torch.where(torch.isinf(lse)[:, None], 0.0, torch.exp(s - lse[:, None]))
    o, a = p @ v, p @ v.abs()
    L = k.shape[0]
    tol = 1.05 * (U * (a + o.abs()) + (2 * ds[:, None] + L * E + 2.0 ** -20) * a) + 1e-30
    return dict(out=o, lse=lse, p=p, tol=tol, lse_tol=1.05 * (ds + L * E + 2.0 ** -21 * (1 + lse.abs().nan_to_num(0, 0, 0))))


def attention_backward(q, k, v, see, scale, do):
    """Gradients of one query head (rows of q) and their bounds."""
    f = attention(q, k, v, see, scale)
    q, k, v, do, p, o = q.double(), k.double(), v.double(), do.double(), f["p"], f["out"]
    n = max(q.shape[0], k.shape[0])
    ds_s = scale * q.shape[1] * E * (q.abs() @ k.abs().T).amax(1)[:, None] + n * E + 2.0 ** -19   # relative error of p
    dp = do @ v.T
    dp_e = v.shape[1] * E * (do.abs() @ v.abs().T)
    delta = (do * o).sum(1, keepdim=True)
    delta_e = (U + v.shape[1] * E) * (do.abs() * o.abs()).sum(1, keepdim=True) * 1.05
    s = scale * p * (dp - delta)
    # error of dS before and after its rounding to bf16
    s_e = scale * p * (dp_e + delta_e) + 2 * ds_s * scale * p * (dp - delta).abs()
    s_e = s_e + U * (s.abs() + s_e)
    p_e = p * (U + 2 * ds_s)
    r = dict(dq=s @ k, dk=s.T @ q, dv=p.T @ do)
    e = dict(dq=s_e @ k.abs() + n * E * (s.abs() @ k.abs()), dk=s_e.T @ q.abs() + n * E * (s.abs().T @ q.abs()),
             dv=p_e.T @ do.abs() + n * E * (p.T @ do.abs()))
    return r, e


def causal(L, device):
    i = torch.arange(L, device=device)
    return i[None] <= i[:, None]


def prefill(q, k, v, lens, H_kv, scale, do=None, heads=None):
    """Packed prompts [N, H, d]: dict of out, lse (and dq, dk, dv) with *_tol."""
    N, Hq, dk = q.shape
    G, dv, dev = Hq // H_kv, v.shape[-1], q.device
    f = dict(dtype=torch.float64, device=dev)
    r = dict(out=torch.zeros((N, Hq, dv), **f), out_tol=torch.zeros((N, Hq, dv), **f), lse=torch.zeros((N, Hq), **f),
             lse_tol=torch.zeros((N, Hq), **f))
    if do is not None:
        for n, h, d in (("dq", Hq, dk), ("dk", H_kv, dk), ("dv", H_kv, dv)):
            r[n], r[n + "_tol"] = torch.zeros((N, h, d), **f), torch.zeros((N, h, d), **f)
    at = 0
    for L in lens:
        sl = slice(at, at + L)
        at += L
        if L == 0:
            continue
        see = causal(L, dev)
        for h in range(Hq):
            a = (q[sl, h], k[sl, h // G], v[sl, h // G], see, scale)
            x = attention(*a)
            r["out"][sl, h], r["out_tol"][sl, h] = x["out"], x["tol"]
            r["lse"][sl, h], r["lse_tol"][sl, h] = x["lse"], x["lse_tol"]
            if do is not None:
                g, e = attention_backward(*a, do[sl, h])
                r["dq"][sl, h], r["dq_tol"][sl, h] = g["dq"], e["dq"]
                for n in ("dk", "dv"):
                    r[n][sl, h // G] += g[n]
                    r[n + "_tol"][sl, h // G] += e[n]
    if do is not None:
        for n in ("dq", "dk", "dv"):   # the final rounding
            r[n + "_tol"] = 1.05 * (r[n + "_tol"] + U * (r[n].abs() + r[n + "_tol"])) + 1e-30
    return r


def tree_see(n, L, mask_row_words, device):
    """[n, L] visibility: everything before the nodes, and the nodes the words name."""
    see = torch.ones((n, L), dtype=torch.bool, device=device)
    for i in range(n):
        for j in range(n):
            see[i, L - n + j] = bool((mask_row_words[i] >> j) & 1)
    return see


def tree(q, k_of, v_of, lens, nodes, masks, H_kv, scale):
    """q [B, M, H_q, d]; k_of(b, L), v_of(b, L) give a sequence's first L rows
    [L, H_kv, d]; masks[b]: words (None: a chain). Returns {(b): dict of [n, H_q, ...]}."""
    res = {}
    G = q.shape[2] // H_kv
    for b, (L, n) in enumerate(zip(lens, nodes)):
        if n == 0:
            continue
        words = masks[b] if masks is not None else [(2 << i) - 1 for i in range(n)]
        see = tree_see(n, L, words, q.device)
        k, v = k_of(b, L), v_of(b, L)
        xs = [attention(q[b, :n, h], k[:, h // G], v[:, h // G], see, scale) for h in range(q.shape[2])]
        res[b] = {m: torch.stack([x[m] for x in xs], 1) for m in ("out", "tol", "lse", "lse_tol")}
    return res


def random_tree(M, gen):
    """Words of a random tree of M nodes: node i hangs below an earlier one."""
    words = []
    for i in range(M):
        w = 1 << i
        if i:
            w |= words[int(torch.randint(0, i, (1,), generator=gen))]
        words.append(w)
    return words


def as_int64(words):
    return [w - (1 << 64) if w >= (1 << 63) else w for w in words]


def assert_within(got, want, tol, what):
    """|got - want| <= tol elementwise, infinities and NaN in the same places."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    fin = torch.isfinite(want)
    over = ((got - want).abs() - tol)[fin]
    if over.numel():
        i = int(over.argmax())
        assert float(over.max()) <= 0, (f"{what}: off by {float((got - want).abs()[fin][i]):.3e}, "
                                        f"allowed {float(tol.expand_as(want)[fin][i]):.3e}")
