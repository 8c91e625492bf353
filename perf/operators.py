"""Cases of the operators around full (dense) attention, with their plain forms.

Five calls are measured:

  rope       nsa_qk_norm_rope: RMS norm of every query and key head and the rotary
             position in one pass, keys and values written to their cache rows
  rope_bwd   nsa_qk_norm_rope_backward: gradients of the projections and of the norm weights
  prefill    nsa_full_prefill: causal attention over packed prompts, grouped heads
  train      nsa_full_prefill and nsa_full_prefill_backward, as a training step runs them
  tree       nsa_full_tree_decode[_paged]: attention of drafted tokens (a tree, or one
             token) over a cache

With `own` false `run` computes them with elementary torch operations in fp32 (angles
in fp64), rounded once at the end; with `own` true it calls this package.
"""
from __future__ import annotations

import math

import torch

own = False

BF16 = torch.bfloat16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 32 sequences: queries in place, keys and values to their cache rows
        dict(name="rope_decode", op="rope", N=32, H_q=64, H_kv=4, d_k=192, d_v=128, d_rot=64, interleaved=True,
             cache=True, fused=True, max_pos=65536),
        # the 8K prompt's projections, a slice of one fused projection
        dict(name="rope_prefill_8k", op="rope", N=8192, H_q=64, H_kv=4, d_k=192, d_v=128, d_rot=192,
             interleaved=False, cache=False, fused=True, max_pos=8192),
        # gradients of the same, and of a small odd batch of short heads
        dict(name="rope_bwd_8k", op="rope_bwd", N=8192, H_q=64, H_kv=4, d_k=192, d_v=128, d_rot=192,
             interleaved=False, fused=True, max_pos=8192),
        dict(name="rope_bwd_small", op="rope_bwd", N=333, H_q=4, H_kv=1, d_k=64, d_v=64, d_rot=32, interleaved=True,
             fused=False, max_pos=131072),
        # the 1024-token prompt with 4 query heads on one key head
        dict(name="prefill_tiny", op="prefill", lens="1024", H_q=4, H_kv=1, d_k=64, d_v=64),
        # prompts of different lengths packed into one call
        dict(name="prefill_ragged", op="prefill", lens="4096,1,777,2500,63", H_q=32, H_kv=4, d_k=128, d_v=128),
        # the 8K prompt
        dict(name="prefill_8k", op="prefill", lens="8192", H_q=64, H_kv=4, d_k=192, d_v=128),
        # training steps: a packed batch of short sequences, and one long sequence
        dict(name="train_ragged", op="train", lens="300,1,1025,130", H_q=8, H_kv=2, d_k=128, d_v=64),
        dict(name="train_4k", op="train", lens="4096", H_q=64, H_kv=4, d_k=192, d_v=128),
        # single tokens over ragged paged caches
        dict(name="tree_single_paged", op="tree", B=16, M=1, lo=8192, hi=131072, H_q=64, H_kv=4, d_k=192, d_v=128,
             page=64),
        # 16 drafted tokens per sequence over 16K caches
        dict(name="tree_draft16", op="tree", B=32, M=16, lo=16384, hi=16384, H_q=64, H_kv=4, d_k=192, d_v=128,
             page=0),
        # a small batch of wide trees over short caches
        dict(name="tree_wide_short", op="tree", B=3, M=61, lo=70, hi=2000, H_q=16, H_kv=2, d_k=128, d_v=128, page=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    H_q, H_kv = rng.choice([(4, 1), (8, 8), (16, 2), (32, 4), (64, 4), (24, 12)])
    d_k, d_v = rng.choice([(64, 64), (128, 128), (192, 128), (128, 64), (64, 128), (192, 64)])
    heads = dict(H_q=H_q, H_kv=H_kv, d_k=d_k, d_v=d_v)
    op = rng.choice(["rope", "rope_bwd", "prefill", "train", "tree"])
    if op in ("rope", "rope_bwd"):
        c = dict(op=op, N=_log(rng, 1, 8192), d_rot=16 * rng.randint(0, d_k // 16), interleaved=rng.random() < 0.5,
                 fused=rng.random() < 0.5, max_pos=_log(rng, 8192, 1 << 20), **heads)
        if op == "rope":
            c["cache"] = rng.random() < 0.5
        return c
    if op in ("prefill", "train"):
        n = rng.randint(1, 5)
        # the padded score matrices of the plain form stay below the largest listed case's
        cap = int(math.sqrt((64 * 8192 * 8192 if op == "prefill" else 64 * 4096 * 4096) / (n * H_q)))
        top = min(8192 if op == "prefill" else 4096, cap)
        lens = [_log(rng, 1, top) for _ in range(n)]
        return dict(op=op, lens=",".join(str(x) for x in lens), **heads)
    M = _log(rng, 1, 64)
    B = _log(rng, 1, 32)
    budget = 32 * 16384 * 4 * 320 * 1024   # keys x widths x rows of the widest listed tree
    hi = min(131072, budget // (B * H_kv * (d_k + d_v) * max(M * H_q // H_kv, 128)), (1 << 31) // (B * H_kv * (d_k + d_v)))
    hi = max(M, _log(rng, 64, max(65, hi)))
    lo = max(M, _log(rng, 1, hi))
    return dict(op="tree", B=B, M=M, lo=lo, hi=hi, page=rng.choice([0, 64, 128, 256]), **heads)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(shape, g, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _projections(c, g, N):
    """q, k, v of N tokens: three tensors, or views of one fused projection."""
    wq, wk, wv = c["H_q"] * c["d_k"], c["H_kv"] * c["d_k"], c["H_kv"] * c["d_v"]
    if c.get("fused"):
        x = _randn((N, wq + wk + wv), g)
        q, k, v = x[:, :wq], x[:, wq:wq + wk], x[:, wq + wk:]
    else:
        q, k, v = _randn((N, wq), g), _randn((N, wk), g), _randn((N, wv), g)
    return (q.unflatten(1, (c["H_q"], c["d_k"])), k.unflatten(1, (c["H_kv"], c["d_k"])),
            v.unflatten(1, (c["H_kv"], c["d_v"])))


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    s = dict(case=c)
    dev = "cuda"
    if c["op"] in ("rope", "rope_bwd"):
        N, dk, dv, dr = c["N"], c["d_k"], c["d_v"], c["d_rot"]
        s["q"], s["k"], s["v"] = _projections(c, g, N)
        s["w_q"] = 1.0 + 0.2 * _randn((dk,), g, torch.float32)
        s["w_k"] = 1.0 + 0.2 * _randn((dk,), g, torch.float32)
        i = torch.arange(dr // 2, dtype=torch.float64, device=dev)
        s["inv_freq"] = (10000.0 ** (-2.0 * i / max(dr, 1))).float()
        s["eps"] = 1e-6
        if c["op"] == "rope" and c["cache"]:   # a token each of N sequences, at the end of its cache
            s["pos"] = torch.randint(0, c["max_pos"], (N,), generator=g, device=dev, dtype=torch.int32)
            rows = 2 * N + 3
            s["rows"] = torch.randperm(rows, generator=g, device=dev)[:N].contiguous()
            s["k_out"] = torch.zeros((rows, c["H_kv"], dk), dtype=BF16, device=dev)
            s["v_out"] = torch.zeros((rows, c["H_kv"], dv), dtype=BF16, device=dev)
        else:                                   # consecutive tokens that end at max_pos
            s["pos"] = torch.arange(c["max_pos"] - N, c["max_pos"], device=dev, dtype=torch.int32)
            s["rows"] = None
            s["k_out"] = torch.zeros((N, c["H_kv"], dk), dtype=BF16, device=dev)
            s["v_out"] = None
        s["q_out"] = torch.empty((N, c["H_q"], dk), dtype=BF16, device=dev)
        if c["op"] == "rope_bwd":
            s["dq_out"] = _randn((N, c["H_q"], dk), g)
            s["dk_out"] = _randn((N, c["H_kv"], dk), g)
            s["dq"], s["dk"] = torch.empty_like(s["dq_out"]), torch.empty_like(s["dk_out"])
            s["dw_q"], s["dw_k"] = torch.empty_like(s["w_q"]), torch.empty_like(s["w_k"])
    elif c["op"] in ("prefill", "train"):
        lens = [int(x) for x in c["lens"].split(",")]
        N = sum(lens)
        s["lens"] = lens
        s["cu"] = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32)
        s["q"], s["k"], s["v"] = _projections(c, g, N)
        s["out"] = torch.empty((N, c["H_q"], c["d_v"]), dtype=BF16, device=dev)
        s["lse"] = torch.empty((N, c["H_q"]), dtype=torch.float32, device=dev)
        # where each token stands in a padded batch, and each padded place's token
        seq = torch.cat([torch.full((L,), b, dtype=torch.int64) for b, L in enumerate(lens)])
        pos = torch.cat([torch.arange(L, dtype=torch.int64) for L in lens])
        s["seq"], s["pos"] = seq.to(dev), pos.to(dev)
        first = torch.tensor([sum(lens[:b]) for b in range(len(lens))], dtype=torch.int64).unsqueeze(1)
        s["place"] = (first + torch.arange(max(lens)).unsqueeze(0)).clamp(max=N - 1).to(dev)
        s["len_dev"] = torch.tensor(lens, device=dev)
        if c["op"] == "train":
            s["dout"] = _randn((N, c["H_q"], c["d_v"]), g)
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[n]) for n in ("q", "k", "v"))
    else:
        B, M, page = c["B"], c["M"], c["page"]
        cpu = torch.Generator()
        cpu.manual_seed(int(seed))
        nodes = torch.randint(1, M + 1, (B,), generator=cpu)
        nodes[0] = M
        lens = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=cpu)
        lens[-1] = c["hi"]
        # node 0 is the last accepted token; every other node hangs below an earlier one
        mask = torch.zeros((B, M, M), dtype=torch.bool)
        for i in range(M):
            if i:
                parent = (torch.rand((B,), generator=cpu) * i).long()
                mask[:, i] = mask[torch.arange(B), parent]
            mask[:, i, i] = True
        bits = torch.zeros((B, M), dtype=torch.int64)
        for j in range(M):
            bits |= mask[:, :, j].long() << j
        s["mask"] = bits.to(dev)
        s["nodes"], s["lens"] = nodes.to(dev, torch.int32), lens.to(dev, torch.int32)
        s["max_len"] = int(c["hi"])
        Lmax = -(-c["hi"] // 256) * 256
        s["q"] = _randn((B, M, c["H_q"], c["d_k"]), g)
        if page:
            per = Lmax // page
            s["table"] = torch.randperm(B * per, generator=g, device=dev).to(torch.int32).view(B, per)
            s["k"] = torch.empty((B * per, page, c["H_kv"], c["d_k"]), dtype=BF16, device=dev).normal_(generator=g)
            s["v"] = torch.empty((B * per, page, c["H_kv"], c["d_v"]), dtype=BF16, device=dev).normal_(generator=g)
        else:
            s["table"] = None
            s["k"] = torch.empty((B, Lmax, c["H_kv"], c["d_k"]), dtype=BF16, device=dev).normal_(generator=g)
            s["v"] = torch.empty((B, Lmax, c["H_kv"], c["d_v"]), dtype=BF16, device=dev).normal_(generator=g)
        s["out"] = torch.zeros((B, M, c["H_q"], c["d_v"]), dtype=BF16, device=dev)
        s["lse"] = torch.zeros((B, M, c["H_q"]), dtype=torch.float32, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _cos_sin(pos, inv_freq):
    a = pos.double().unsqueeze(1) * inv_freq.double().unsqueeze(0)
    return a.cos().float().unsqueeze(1), a.sin().float().unsqueeze(1)


def _rotate(y, cos, sin, dr, interleaved):
    """Each pair (a, b) becomes (a cos - b sin, a sin + b cos)."""
    r, rest = y[..., :dr], y[..., dr:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = r[..., :dr // 2], r[..., dr // 2:]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((r, rest), dim=-1)


def _plain_rope(s):
    c = s["case"]
    cos, sin = _cos_sin(s["pos"], s["inv_freq"])

    def one(x, w):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w
        return _rotate(y, cos, sin, c["d_rot"], c["interleaved"]).to(BF16)
    q, k = one(s["q"], s["w_q"]), one(s["k"], s["w_k"])
    if s["rows"] is None:
        return dict(q=q, k=k)
    s["k_out"][s["rows"]] = k
    s["v_out"][s["rows"]] = s["v"]
    return dict(q=q, k=s["k_out"], v=s["v_out"])


def _plain_rope_bwd(s):
    c = s["case"]
    cos, sin = _cos_sin(s["pos"], s["inv_freq"])

    def one(x, w, dy):
        x = x.float()
        dn = _rotate(dy.float(), cos, -sin, c["d_rot"], c["interleaved"])
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
        h = x * r
        dx = r * (dn * w - h * (dn * w * h).mean(-1, keepdim=True))
        return dx.to(BF16), (dn * h).double().sum((0, 1)).float()
    dq, dw_q = one(s["q"], s["w_q"], s["dq_out"])
    dk, dw_k = one(s["k"], s["w_k"], s["dk_out"])
    return dict(dq=dq, dk=dk, dw_q=dw_q, dw_k=dw_k)


def _plain_attention(s, backward):
    c = s["case"]
    Hk, G, dk, dv = c["H_kv"], c["H_q"] // c["H_kv"], c["d_k"], c["d_v"]
    sc = dk ** -0.5
    B, L = s["place"].shape
    at = torch.arange(L, device="cuda")
    # padded [B, H_kv, (L, G) or L, d]
    q = s["q"].float()[s["place"]].view(B, L, Hk, G, dk).permute(0, 2, 3, 1, 4)
    k = s["k"].float()[s["place"]].transpose(1, 2)
    v = s["v"].float()[s["place"]].transpose(1, 2)
    real = at.view(1, L) < s["len_dev"].view(B, 1)
    k, v = (x * real.view(B, 1, L, 1) for x in (k, v))
    p = (q.reshape(B, Hk, G * L, dk) @ k.transpose(2, 3)).view(B, Hk, G, L, L)
    p.mul_(sc).masked_fill_(at.view(1, L) > at.view(L, 1), -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    p.div_(z)
    lse = (m + z.log()).squeeze(-1)
    o = (p.view(B, Hk, G * L, L) @ v).view(B, Hk, G, L, dv)

    def packed(x):   # [B, H_kv, G, L, ...] -> [N, H_q, ...]
        x = x.movedim(3, 1).flatten(2, 3)
        return x[s["seq"], s["pos"]]
    res = dict(out=packed(o).to(BF16), lse=packed(lse))
    if not backward:
        return res
    do = s["dout"].float()[s["place"]].view(B, L, Hk, G, dv).permute(0, 2, 3, 1, 4) * real.view(B, 1, 1, L, 1)
    flat = lambda x: x.reshape(B, Hk, G * L, x.shape[-1])   # noqa: E731
    gv = flat(p).transpose(2, 3) @ flat(do)
    ds = (flat(do) @ v.transpose(2, 3)).view_as(p)
    ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(sc)
    del p
    gq = (flat(ds) @ k).view(B, Hk, G, L, dk)
    gk = flat(ds).transpose(2, 3) @ flat(q)
    res["dq"] = packed(gq).to(BF16)
    res["dk"] = gk.transpose(1, 2)[s["seq"], s["pos"]].to(BF16)
    res["dv"] = gv.transpose(1, 2)[s["seq"], s["pos"]].to(BF16)
    return res


def _plain_tree(s):
    c = s["case"]
    B, M, Hk, G, dk, dv = c["B"], c["M"], c["H_kv"], c["H_q"] // c["H_kv"], c["d_k"], c["d_v"]
    L = s["max_len"]
    if s["table"] is None:
        k, v = s["k"][:, :L], s["v"][:, :L]
    else:
        pages = s["table"][:, : -(-L // c["page"])].long()
        k, v = (x[pages].flatten(1, 2)[:, :L] for x in (s["k"], s["v"]))
    lens, nodes = s["lens"].long().view(B, 1, 1), s["nodes"].long().view(B, 1, 1)
    j = torch.arange(L, device="cuda").view(1, 1, L) - (lens - nodes)   # node of each key; below 0: the prefix
    bit = (s["mask"].view(B, M, 1) >> j.clamp(0, 63)) & 1
    see = (j < 0) | ((j < nodes) & (bit == 1))                          # [B, M, L]
    q = s["q"].float().view(B, M, Hk, G, dk).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * M, dk)
    p = (q @ k.float().permute(0, 2, 3, 1)).view(B, Hk, G, M, L)
    p.mul_(dk ** -0.5).masked_fill_(~see.view(B, 1, 1, M, L), -math.inf)
    m = p.amax(-1, keepdim=True)
    p.sub_(m.clamp(min=-1e30)).exp_()
    z = p.sum(-1, keepdim=True)
    live = (torch.arange(L, device="cuda").view(1, L) < lens.view(B, 1)).view(B, 1, L, 1)
    o = p.view(B, Hk, G * M, L) @ v.transpose(1, 2).float().masked_fill_(~live, 0.0)
    o = o.view(B, Hk, G, M, dv) / z
    real = (torch.arange(M, device="cuda").view(1, M) < nodes.view(B, 1)).view(B, M, 1)
    lse = (m + z.log()).squeeze(-1).permute(0, 3, 1, 2).flatten(2)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)
    return dict(out=torch.where(real.unsqueeze(-1), o, 0.0).to(BF16), lse=torch.where(real, lse, 0.0))


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    import sparse_attention_long_nsa_b200 as nsa
    c = s["case"]
    op = c["op"]
    if "heads" not in s:   # what a user's program keeps: the geometry and the workspace
        s["heads"] = h = nsa.Heads(c["H_q"], c["H_kv"], c["d_k"], c["d_v"])
        if op in ("rope", "rope_bwd"):
            s["rope"] = nsa.RopeParams(c["d_rot"], int(c["interleaved"]), s["eps"])
        size = nsa.nsa_full_workspace_size
        if op == "rope_bwd":
            s["ws"] = nsa.alloc_workspace(size(nsa.NSA_OP_ROPE_BACKWARD, h, 1, c["N"], 0, 0), "cuda")
        elif op in ("prefill", "train"):
            what = nsa.NSA_OP_FULL_PREFILL if op == "prefill" else nsa.NSA_OP_FULL_BACKWARD
            s["ws"] = nsa.alloc_workspace(size(what, h, len(s["lens"]), sum(s["lens"]), max(s["lens"]), 0), "cuda")
        elif op == "tree":
            s["ws"] = nsa.alloc_workspace(size(nsa.NSA_OP_TREE_DECODE, h, c["B"], 0, s["max_len"], c["M"]), "cuda")
    h = s["heads"]
    if op == "rope":
        nsa.nsa_qk_norm_rope(s["q"], s["k"], s["w_q"], s["w_k"], s["inv_freq"], s["pos"], h, s["rope"], s["q_out"],
                             s["k_out"], s["v"] if s["v_out"] is not None else None, s["v_out"], s["rows"])
        if s["rows"] is None:
            return dict(q=s["q_out"], k=s["k_out"])
        return dict(q=s["q_out"], k=s["k_out"], v=s["v_out"])
    if op == "rope_bwd":
        nsa.nsa_qk_norm_rope_backward(s["q"], s["k"], s["w_q"], s["w_k"], s["inv_freq"], s["pos"], s["dq_out"],
                                      s["dk_out"], h, s["rope"], s["dq"], s["dk"], s["dw_q"], s["dw_k"], s["ws"])
        return {n: s[n] for n in ("dq", "dk", "dw_q", "dw_k")}
    if op in ("prefill", "train"):
        nsa.nsa_full_prefill(s["q"], s["k"], s["v"], s["cu"], h, s["out"], s["lse"], s["ws"])
        if op == "prefill":
            return dict(out=s["out"], lse=s["lse"])
        nsa.nsa_full_prefill_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["cu"], h, s["dq"],
                                      s["dk"], s["dv"], s["ws"])
        return {n: s[n] for n in ("out", "lse", "dq", "dk", "dv")}
    if s["table"] is None:
        nsa.nsa_full_tree_decode(s["q"], s["k"], s["v"], s["lens"], s["nodes"], s["mask"], s["max_len"], h, s["out"],
                                 s["lse"], s["ws"])
    else:
        nsa.nsa_full_tree_decode_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], s["nodes"], s["mask"],
                                       s["max_len"], h, s["out"], s["lse"], s["ws"])
    return dict(out=s["out"], lse=s["lse"])


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "rope":
        return _plain_rope(state)
    if op == "rope_bwd":
        return _plain_rope_bwd(state)
    if op in ("prefill", "train"):
        return _plain_attention(state, op == "train")
    return _plain_tree(state)


# ---------------------------------------------------------------------------
# work: every input read once, every output written once; the products of the visible pairs
# ---------------------------------------------------------------------------

def work(case):
    c = case
    Hq, Hk, dk, dv = c["H_q"], c["H_kv"], c["d_k"], c["d_v"]
    if c["op"] == "rope":
        n = c["N"]
        width = (Hq + Hk) * dk + (Hk * dv if c["cache"] else 0)
        return dict(bytes=4 * n * width + 8 * dk + 2 * c["d_rot"] + n * (12 if c["cache"] else 4),
                    flops=n * (Hq + Hk) * (4 * dk + 3 * c["d_rot"]))
    if c["op"] == "rope_bwd":
        n = c["N"]
        return dict(bytes=6 * n * (Hq + Hk) * dk + 16 * dk + 2 * c["d_rot"] + 4 * n,
                    flops=n * (Hq + Hk) * (10 * dk + 3 * c["d_rot"]))
    if c["op"] in ("prefill", "train"):
        lens = [int(x) for x in c["lens"].split(",")]
        n, pairs = sum(lens), sum(x * (x + 1) // 2 for x in lens)
        fwd = dict(bytes=2 * n * (Hq + Hk) * (dk + dv) + 4 * n * Hq, flops=2 * pairs * Hq * (dk + dv))
        if c["op"] == "prefill":
            return fwd
        # backward: q, k, v, out, dout and lse in, dq, dk, dv out; five products
        return dict(bytes=fwd["bytes"] + 2 * n * (Hq * (2 * dk + 2 * dv) + 2 * Hk * (dk + dv)) + 4 * n * Hq,
                    flops=fwd["flops"] + 2 * pairs * Hq * (3 * dk + 2 * dv))
    B, M = c["B"], c["M"]
    keys = (B - 1) * (c["lo"] + c["hi"]) / 2 + c["hi"]        # expected, as the lengths are drawn
    rows = M + (B - 1) * (M + 1) / 2
    return dict(bytes=2 * keys * Hk * (dk + dv) + 2 * rows * Hq * (dk + dv) + 4 * rows * Hq + 8 * B * M,
                flops=2 * keys * rows / B * Hq * (dk + dv))


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one head group of one sequence at a time
# ---------------------------------------------------------------------------

def _exact_rope(s, backward):
    c = s["case"]
    dr = c["d_rot"]
    theta = s["pos"].double()[:, None] * s["inv_freq"].double()[None]
    turn = torch.polar(torch.ones_like(theta), theta)[:, None, :]        # e^{i theta}

    def as_pairs(x):
        r = x[..., :dr]
        return torch.complex(r[..., 0::2].contiguous(), r[..., 1::2].contiguous()) if c["interleaved"] else \
            torch.complex(r[..., :dr // 2].contiguous(), r[..., dr // 2:].contiguous())

    def from_pairs(z, x):
        y = x.clone()
        if c["interleaved"]:
            y[..., 0:dr:2], y[..., 1:dr:2] = z.real, z.imag
        else:
            y[..., :dr // 2], y[..., dr // 2:dr] = z.real, z.imag
        return y

    def forward(x, w):
        x = x.double()
        y = w.double() * x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["d_k"] + s["eps"])
        return from_pairs(as_pairs(y) * turn, y)

    def grads(x, w, dy):
        x, w, dy = x.double(), w.double(), dy.double()
        dn = from_pairs(as_pairs(dy) * turn.conj(), dy)
        rms = torch.sqrt(x.square().sum(-1, keepdim=True) / c["d_k"] + s["eps"])
        u = dn * w
        return u / rms - x * (u * x).sum(-1, keepdim=True) / (c["d_k"] * rms ** 3), (dn * x / rms).sum((0, 1))
    if backward:
        dq, dwq = grads(s["q"], s["w_q"], s["dq_out"])
        dk, dwk = grads(s["k"], s["w_k"], s["dk_out"])
        return dict(dq=dq, dk=dk, dw_q=dwq, dw_k=dwk)
    q, k = forward(s["q"], s["w_q"]), forward(s["k"], s["w_k"])
    if s["rows"] is None:
        return dict(q=q, k=k)
    ko, vo = s["k_out"].double(), s["v_out"].double()
    ko.index_copy_(0, s["rows"], k)
    vo.index_copy_(0, s["rows"], s["v"].double())
    return dict(q=q, k=ko, v=vo)


def _exact_attention(s, backward):
    c = s["case"]
    Hq, Hk, dk, dv = c["H_q"], c["H_kv"], c["d_k"], c["d_v"]
    G, N = Hq // Hk, s["q"].shape[0]
    sc = 1.0 / math.sqrt(dk)
    f = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.empty((N, Hq, dv), **f), torch.empty((N, Hq), **f)
    gq, gk, gv = torch.zeros((N, Hq, dk), **f), torch.zeros((N, Hk, dk), **f), torch.zeros((N, Hk, dv), **f)
    at = 0
    for L in s["lens"]:
        sl = slice(at, at + L)
        at += L
        hidden = torch.ones((L, L), dtype=torch.bool, device="cuda").triu(1)
        for h in range(Hq):
            q, k, v = s["q"][sl, h].double(), s["k"][sl, h // G].double(), s["v"][sl, h // G].double()
            x = torch.where(hidden, -math.inf, sc * (q @ k.T))
            lse[sl, h] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[sl, h, None])
            out[sl, h] = p @ v
            if backward:
                do = s["dout"][sl, h].double()
                gv[sl, h // G] += p.T @ do
                dp = do @ v.T
                ds = sc * p * (dp - (p * dp).sum(1, keepdim=True))
                gq[sl, h] = ds @ k
                gk[sl, h // G] += ds.T @ q
    res = dict(out=out, lse=lse)
    return dict(res, dq=gq, dk=gk, dv=gv) if backward else res


def _exact_tree(s):
    c = s["case"]
    Hk, G, dk, dv = c["H_kv"], c["H_q"] // c["H_kv"], c["d_k"], c["d_v"]
    out, lse = s["out"].double().zero_(), s["lse"].double().zero_()
    for b, (L, n) in enumerate(zip(s["lens"].tolist(), s["nodes"].tolist())):
        if s["table"] is None:
            k, v = s["k"][b, :L], s["v"][b, :L]
        else:
            t = torch.arange(L, device="cuda")
            page = s["table"][b].long()[t // c["page"]]
            k, v = s["k"][page, t % c["page"]], s["v"][page, t % c["page"]]
        see = torch.ones((n, L), dtype=torch.bool, device="cuda")
        see[:, L - n:] = torch.tensor([[(m >> j) & 1 == 1 for j in range(n)] for m in s["mask"][b, :n].tolist()],
                                      device="cuda")
        for g in range(Hk):
            kg, vg = k[:, g].double(), v[:, g].double()
            q = s["q"][b, :n, g * G:(g + 1) * G].double()
            x = torch.where(see[:, None], torch.einsum("ihd,ld->ihl", q, kg) / math.sqrt(dk), -math.inf)
            z = torch.logsumexp(x, -1)
            lse[b, :n, g * G:(g + 1) * G] = z
            out[b, :n, g * G:(g + 1) * G] = torch.exp(x - z[..., None]) @ vg
    return dict(out=out, lse=lse)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rope", "rope_bwd"):
        return _exact_rope(s, op == "rope_bwd")
    if op in ("prefill", "train"):
        return _exact_attention(s, op == "train")
    return _exact_tree(s)
