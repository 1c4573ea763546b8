"""The decoder operators of drafted tokens, as cases to measure: attention of a token tree over
a paged cache, verification of drafted tokens, the append of the accepted path to the cache, the
RMS norm with residual and 8-bit output, and the 8-bit matrix product.

``run`` computes a case in plain torch (``own = False``) or through the library (``own = True``).
"""
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


def listed():
    return [
        # one token of one sequence over a short cache: the plain decode step, latency counts
        dict(name="attn step", op="attn", B=1, N=1, H=32, HK=32, D=128, ctx=512, page=16, dtype="f16"),
        # trees of 26 drafted tokens of 4 sequences of unlike lengths, grouped heads, paged cache
        dict(name="attn trees", op="attn", B=4, N=26, H=64, HK=8, D=128, ctx=8191, page=64, dtype="bf16"),
        # the widest tree over a long contiguous cache
        dict(name="attn long", op="attn", B=1, N=64, H=64, HK=8, D=128, ctx=65536, page=0, dtype="f16"),
        # a draft model's chain of 4 tokens for one user
        dict(name="verify chain", op="verify", B=1, N=5, V=32000, dtype="f16", tree=0, q=True, temp=0.8),
        # a batch of sampled trees, up to 3 siblings, large vocabulary
        dict(name="verify trees", op="verify", B=16, N=32, V=131072, dtype="f16", tree=3, q=True, temp=1.0),
        # the FFN's fp32 output of a tree of 8 tokens joins an fp16 residual; both outputs
        dict(name="norm step", op="norm", T=8, d=4096, x="f32", res="f16", y=True),
        # a prompt's rows
        dict(name="norm prompt", op="norm", T=4096, d=8192, x="f16", res="f16", y=False),
        # one token through a fused query/key/value projection
        dict(name="product step", op="linear", M=1, N=12288, K=4096, dtype="f16", bias=False),
        # a tree of 48 tokens through a grouped-head projection
        dict(name="product tree", op="linear", M=48, N=10240, K=8192, dtype="f16", bias=True),
        # a prompt through a square projection
        dict(name="product prompt", op="linear", M=4096, N=8192, K=8192, dtype="bf16", bias=False),
        # the accepted path of one tree enters the cache
        dict(name="append path", op="append", B=1, N=16, HK=32, D=128, ctx=1000, page=16, dtype="f16", all=False),
        # every token of a batch's prompt pieces enters the cache
        dict(name="append prompts", op="append", B=64, N=64, HK=32, D=128, ctx=700, page=64, dtype="bf16", all=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def _odd(rng, lo, hi):
    """The same, odd (listed sizes are mostly even): hi is left out where it is even."""
    return min(_log(rng, lo, hi) | 1, hi - 1 + hi % 2)


def draw(rng):
    op = rng.choice(["attn", "attn", "verify", "norm", "linear", "append"])
    if op == "attn":
        H, HK = rng.choice([(32, 32), (64, 8), (16, 16), (40, 8), (8, 1), (12, 4), (96, 96)])
        D = rng.choice([64, 64, 128, 128, 128, 80, 256])
        B, N = _log(rng, 1, 32), _log(rng, 1, 64)
        ctx = _odd(rng, 1, 65536)
        # no more than the longest listed case's cache bytes and products
        ctx = max(1, min(ctx, 65536 * 8 * 128 // (B * HK * D), 65536 * 64 * 64 * 128 // (B * N * H * D)))
        return dict(op=op, B=B, N=N, H=H, HK=HK, D=D, ctx=ctx, page=rng.choice([0, 16, 16, 64, 48, 256]),
                    dtype=rng.choice(["f16", "bf16"]))
    if op == "verify":
        V, B, N = _odd(rng, 500, 131072), _log(rng, 1, 32), _log(rng, 1, 64)
        B = max(1, min(B, 16 * 32 * 131072 // (N * V)))
        return dict(op=op, B=B, N=N, V=V, dtype=rng.choice(["f16", "bf16", "f32"]), tree=rng.choice([0, 0, 2, 4]),
                    q=rng.random() < 0.7, temp=rng.choice([0.0, 0.6, 1.0, 1.3]))
    if op == "norm":
        d, T = 8 * _odd(rng, 64, 2048), _odd(rng, 1, 4096)
        return dict(op=op, T=max(1, min(T, 4096 * 8192 // d)), d=d, x=rng.choice(["f16", "bf16", "f32"]),
                    res=rng.choice(["f16", "bf16", "f32"]), y=rng.random() < 0.5)
    if op == "linear":
        K, N, M = 16 * _odd(rng, 32, 1024), _odd(rng, 100, 16384), _odd(rng, 1, 4096)
        M = max(1, min(M, 4096 * 8192 * 8192 // (K * N)))
        return dict(op=op, M=M, N=N, K=K, dtype=rng.choice(["f16", "bf16", "f32"]), bias=rng.random() < 0.5)
    return dict(op=op, B=_log(rng, 1, 64), N=_log(rng, 1, 64), HK=rng.choice([1, 4, 8, 32]), D=rng.choice([64, 80, 128]),
                ctx=_odd(rng, 1, 2000), page=rng.choice([0, 16, 48, 64]), dtype=rng.choice(["f16", "bf16"]),
                all=rng.random() < 0.3)


def _trees(r, B, N, width):
    """Parents [B][N] of random trees (a chain for width 0), and the widest family's size."""
    rows, most = [], 1
    for _ in range(B):
        par, kids = [-1], [0] * N
        for i in range(1, N):
            if width == 0:
                p = i - 1
            else:
                p = r.choice([j for j in range(max(0, i - 2 * width), i) if kids[j] < width])
            kids[p] += 1
            par.append(p)
        most = max([most] + kids)
        rows.append(par)
    return rows, most


def _ancestors(rows):
    """[B][N][N] truth values: node i sees node j where j is i or above it."""
    out = []
    for par in rows:
        m = []
        for i, p in enumerate(par):
            row = list(m[p]) if p >= 0 else [False] * len(par)
            row[i] = True
            m.append(row)
        out.append(m)
    return torch.tensor(out, device=DEV)


def _words(anc):
    """Truth values [B][N][N] as 64-bit mask words [B][N], bit j for node j."""
    bit = torch.bitwise_left_shift(torch.ones((), dtype=torch.int64, device=DEV),
                                   torch.arange(anc.shape[2], device=DEV))
    return (anc.to(torch.int64) * bit).sum(2)


def _cache(c, g, r):
    """A paged cache (page > 0, shuffled pages) or a contiguous one, with room for N more tokens."""
    B, N, HK, D, dt = c["B"], c["N"], c["HK"], c["D"], DT[c["dtype"]]
    # sequences of unlike lengths, the first at the full one
    lens = [c["ctx"]] + [max(1, int(c["ctx"] * (0.4 + 0.6 * r.random()))) for _ in range(B - 1)]
    room = c["ctx"] + N
    if c["page"] == 0:
        page, width, pages, table = room, 1, B, None
    else:
        page, width = c["page"], -(-room // c["page"])
        pages = B * width
        table = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).view(B, width).contiguous()
    k = torch.randn(pages, page, HK, D, generator=g, device=DEV).to(dt)
    v = torch.randn(pages, page, HK, D, generator=g, device=DEV).to(dt)
    return dict(k=k, v=v, table=table, ctx_len=torch.tensor(lens, dtype=torch.int32, device=DEV),
                slots=torch.arange(B, device=DEV)[:, None] if table is None else table.long(), page=page)


def prepare(case, seed):
    c, g, r = case, torch.Generator(DEV).manual_seed(seed), random.Random(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    s = dict(case=c)
    if c["op"] in ("attn", "append"):
        B, N, HK, D, dt = c["B"], c["N"], c["HK"], c["D"], DT[c["dtype"]]
        s.update(_cache(c, g, r))
        s.update(k_new=randn(B, N, HK, D).to(dt), v_new=randn(B, N, HK, D).to(dt))
        if c["op"] == "attn":
            s["q"] = (2 * randn(B, N, c["H"], D)).to(dt)  # sharper than uniform attention
            s["anc"] = _ancestors(_trees(r, B, N, 3)[0])
            s["words"] = _words(s["anc"])
            s["scale"] = D ** -0.5
            if own:
                s["out"] = torch.empty(B, N, c["H"], D, dtype=dt, device=DEV)
        else:
            n = [N if c["all"] else r.randint(1, N) for _ in range(B)]
            nodes = [sorted(r.sample(range(N), k)) + [-1] * (N - k) for k in n]
            s.update(n=torch.tensor(n, dtype=torch.int32, device=DEV),
                     nodes=torch.tensor(nodes, dtype=torch.int32, device=DEV))
            if own:
                s["len_out"] = torch.empty(B, dtype=torch.int32, device=DEV)
    elif c["op"] == "verify":
        B, N, V = c["B"], c["N"], c["V"]
        rows, width = _trees(r, B, N, c["tree"])
        par = torch.tensor(rows, device=DEV)
        # a language model's logits: a broad floor, a few likely tokens; the draft model is near it
        base = 2.0 * randn(B, N, V)
        base += 7.0 * (torch.rand(B, N, V, generator=g, device=DEV) < 8.0 / V)
        s["logits"] = base.to(DT[c["dtype"]])
        near = torch.softmax((base + 0.7 * randn(B, N, V)) / (c["temp"] or 1.0), dim=2)
        above = par.clamp(min=0)
        if c["q"]:
            cdf = near.cumsum(2)  # each node's token from its parent's draft distribution
            u = torch.rand(B, N, 1, generator=g, device=DEV) * torch.take_along_dim(cdf[:, :, -1:], above[:, :, None], 1)
            tok = torch.searchsorted(torch.take_along_dim(cdf, above[:, :, None], 1), u).squeeze(2).clamp(max=V - 1)
            del cdf
        else:  # the draft's most likely tokens, by rank among the siblings
            top = near.topk(min(V, width), dim=2).indices
            rank = torch.tensor([[sum(p == q for q in row[:i]) for i, p in enumerate(row)] for row in rows], device=DEV)
            tok = torch.take_along_dim(torch.take_along_dim(top, above[:, :, None], 1), rank[:, :, None], 2).squeeze(2)
        s.update(q=near if c["q"] else None, tokens=tok.to(torch.int32), parents=par.to(torch.int32), width=width,
                 anc=_ancestors(rows), temp=torch.full((B,), c["temp"], device=DEV),
                 u=torch.rand(B, N, generator=g, device=DEV), u_next=torch.rand(B, generator=g, device=DEV))
        if own:
            s.update(nodes=torch.empty(B, N, dtype=torch.int32, device=DEV),
                     out=torch.empty(B, N, dtype=torch.int32, device=DEV), n=torch.empty(B, dtype=torch.int32, device=DEV))
    elif c["op"] == "norm":
        T, d = c["T"], c["d"]
        s.update(x=randn(T, d).to(DT[c["x"]]), res=(3 * randn(T, d)).to(DT[c["res"]]), w=1 + 0.2 * randn(d), eps=1e-5)
        if own:
            s.update(res_out=torch.empty_like(s["res"]), q8=torch.empty(T, d, dtype=torch.int8, device=DEV),
                     scale=torch.empty(T, device=DEV),
                     y=torch.empty(T, d, dtype=torch.float16, device=DEV) if c["y"] else None)
    else:
        M, N, K = c["M"], c["N"], c["K"]
        # rows as a per-token quantiser leaves them: normal values whose largest is near 127
        s.update(xq=(32 * randn(M, K)).round().clamp(-127, 127).to(torch.int8),
                 wq=(32 * randn(N, K)).round().clamp(-127, 127).to(torch.int8),
                 xs=0.02 + 0.02 * torch.rand(M, generator=g, device=DEV),
                 ws=(1 + torch.rand(N, generator=g, device=DEV)) / (32 * K ** 0.5),
                 bias=randn(N) if c["bias"] else None)
        if own:
            s["y"] = torch.empty(M, N, dtype=DT[c["dtype"]], device=DEV)
    if own:
        _handles(c, s)
    return s


def _handles(c, s):
    """What a program keeps between steps: the context and the operator's handle."""
    import activation_sparse_ffn_layer_amd as pi

    s["pi"], s["ctx"] = pi, pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)
    if c["op"] in ("attn", "append"):
        s["cache"] = pi.KvCache(s["ctx"], s["k"], s["v"])
    if c["op"] == "attn":
        s["attn"] = pi.Attn(s["ctx"], s["cache"], c["H"], max_batch=c["B"], max_nodes=c["N"], scale=s["scale"])
    elif c["op"] == "verify":
        s["ver"] = pi.Verifier(s["ctx"], c["V"], max_batch=c["B"], max_nodes=c["N"])
    elif c["op"] == "linear":
        s["lin"] = pi.Linear(s["ctx"], s["wq"], s["ws"], s["bias"], max_tokens=c["M"])


def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


# ---------------------------------------------------------------- through the library

def _own_attn(s):
    s["pi"].tree_attention(s["ctx"], s["attn"], s["q"], s["k_new"], s["v_new"], s["words"], s["table"], s["ctx_len"],
                           s["out"])
    return s["out"]


def _own_append(s):
    s["pi"].kv_append(s["ctx"], s["cache"], s["k_new"], s["v_new"], s["table"], s["ctx_len"], s["len_out"], s["nodes"],
                      s["n"])
    return s["k"], s["v"], s["len_out"]


def _own_verify(s):
    s["pi"].verify(s["ctx"], s["ver"], s["logits"], s["tokens"], s["parents"], s["u"], s["u_next"], s["nodes"], s["out"],
                   s["n"], q=s["q"], temperature=s["temp"])
    return s["nodes"], s["out"], s["n"]


def _own_norm(s):
    s["pi"].add_rmsnorm(s["ctx"], s["x"], s["res"], s["w"], s["eps"], s["res_out"], q=s["q8"], scale=s["scale"], y=s["y"])
    return s["res_out"], _values(s["q8"], s["scale"]), s["scale"], s["y"]


def _own_linear(s):
    s["pi"].linear_q8(s["ctx"], s["lin"], s["xq"], s["xs"], s["y"])
    return s["y"]


_run_own = dict(attn=_own_attn, append=_own_append, verify=_own_verify, norm=_own_norm, linear=_own_linear)


# ---------------------------------------------------------------- in plain torch

def _values(q8, scale):
    """The values that 8-bit integers stand for, as fp16."""
    return torch.mul(q8, scale[:, None], out=torch.empty(q8.shape, dtype=torch.float16, device=DEV))


def _plain_attn(s):
    c = s["case"]
    B, N, H, HK, D, G = c["B"], c["N"], c["H"], c["HK"], c["D"], c["H"] // c["HK"]
    L = s["slots"].shape[1] * s["page"]
    held = (torch.arange(L, device=DEV) < s["ctx_len"][:, None])[:, :, None, None]
    whole = lambda old, new: torch.cat(  # noqa: E731  [B][HK][L + N][D], zeros where nothing is held
        [torch.where(held, old[s["slots"]].reshape(B, L, HK, D).float(), 0.0), new.float()], 1).transpose(1, 2).contiguous()
    k, v = whole(s["k"], s["k_new"]), whole(s["v"], s["v_new"])
    q = s["q"].float().view(B, N, HK, G, D).permute(0, 2, 1, 3, 4).reshape(B, HK, N * G, D)
    sees = torch.cat([held[:, None, :, 0, 0].expand(B, N, L), s["anc"]], 2)
    w = (q @ k.transpose(2, 3) * s["scale"]).view(B, HK, N, G, L + N)
    w = torch.where(sees[:, None, :, None], w, -torch.inf)
    w = torch.exp(w - w.amax(4, keepdim=True))
    w = w / w.sum(4, keepdim=True)
    o = w.view(B, HK, N * G, L + N) @ v
    return o.view(B, HK, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, H, D).to(s["q"].dtype)


def _plain_append(s):
    c, B, N = s["case"], s["case"]["B"], s["case"]["N"]
    j = torch.arange(N, device=DEV)
    at = s["ctx_len"].long()[:, None] + j
    page = torch.take_along_dim(s["slots"], at // s["page"], 1)
    off = at % s["page"]
    new = (j < s["n"][:, None])[:, :, None, None]
    src = s["nodes"].long().clamp(min=0)[:, :, None, None]
    s["k"][page, off] = torch.where(new, torch.take_along_dim(s["k_new"], src, 1), s["k"][page, off])
    s["v"][page, off] = torch.where(new, torch.take_along_dim(s["v_new"], src, 1), s["v"][page, off])
    return s["k"], s["v"], s["ctx_len"] + s["n"]


def _plain_verify(s):
    # in 64 bits: tokens are picked where a sum over the vocabulary passes a given number
    c, q = s["case"], s["q"]
    B, N, V = c["B"], c["N"], c["V"]
    par, tok = s["parents"].long(), s["tokens"].long()
    if c["temp"] == 0.0:  # all weight at the most likely token, the lowest index of equals
        l = s["logits"].float()
        first = torch.where(l == l.amax(2, keepdim=True), torch.arange(V, device=DEV), V).amin(2, keepdim=True)
        p = (torch.arange(V, device=DEV) == first).double()
    else:
        z = s["logits"].double() / s["temp"].double()[:, None, None]
        p = torch.exp(z - z.amax(2, keepdim=True))
        p = p / p.sum(2, keepdim=True)
    i = torch.arange(N, device=DEV)
    before = (par[:, :, None] == par[:, None, :]) & (i[None, :] < i[:, None])  # earlier siblings
    up = par.clamp(min=0)
    pt = p[torch.arange(B, device=DEV)[:, None], up, tok]  # the target's probability of each node's token
    if q is not None:
        coef, left = [torch.zeros(B, N, dtype=torch.float64, device=DEV)], [torch.ones(B, N, dtype=torch.float64, device=DEV)]
        qd = q.double()
        for _ in range(s["width"]):  # one rejection more each, for every family at once
            coef.append(coef[-1] + left[-1])
            left.append((p - coef[-1][:, :, None] * qd).clamp(min=0).sum(2))
        coef, left = torch.stack(coef, 2), torch.stack(left, 2)
        rank = before.sum(2)
        bi = torch.arange(B, device=DEV)[:, None]
        qt, cj, sj = qd[bi, up, tok], coef[bi, up, rank], left[bi, up, rank]
        ok = s["u"].double() * sj * qt < (pt - cj * qt).clamp(min=0)
    else:
        again = (before & (tok[:, :, None] == tok[:, None, :])).any(2)
        sj = 1 - (before * torch.where(again, 0.0, pt)[:, None, :]).sum(2)
        ok = (s["u"].double() * sj < pt) & ~again
    took = ok & ~(before & ok[:, None, :]).any(2)
    took[:, 0] = True
    on = (took[:, None, :] | ~s["anc"]).all(2)
    n = on.sum(1)
    nodes = torch.where(on, i, N).sort(1).values
    last = torch.take_along_dim(nodes, n[:, None] - 1, 1)
    kids = (par == last) & (i > 0)
    pl = torch.take_along_dim(p, last[:, :, None], 1).squeeze(1)
    if q is not None:
        k = kids.sum(1, keepdim=True)[:, :, None]
        cl = torch.take_along_dim(torch.take_along_dim(coef, last[:, :, None], 1), k, 2).squeeze(1)
        rest = (pl - cl * torch.take_along_dim(qd, last[:, :, None], 1).squeeze(1)).clamp(min=0)
    else:
        gone = torch.zeros(B, V + 1, dtype=torch.bool, device=DEV).scatter(1, torch.where(kids, tok, V), True)[:, :V]
        rest = torch.where(gone, 0.0, pl)
    rest = torch.where(rest.amax(1, keepdim=True) > 0, rest, pl)
    cum = rest.cumsum(1)
    held = torch.where(rest > 0, torch.arange(V, device=DEV), -1).amax(1)
    nxt = torch.minimum((cum <= s["u_next"].double()[:, None] * cum[:, -1:]).sum(1), held)
    down = torch.take_along_dim(tok, torch.cat([nodes[:, 1:], torch.full_like(last, N)], 1).clamp(max=N - 1), 1)
    out = torch.where(i < n[:, None] - 1, down, torch.where(i == n[:, None] - 1, nxt[:, None], -1))
    return torch.where(nodes < N, nodes, -1).to(torch.int32), out.to(torch.int32), n.to(torch.int32)


def _plain_norm(s):
    r = (s["x"].float() + s["res"].float()).to(s["res"].dtype)
    h = r.float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + s["eps"]) * s["w"]
    scale = y.abs().amax(1) / 127
    q8 = torch.round(y / scale[:, None])
    return r, _values(q8, scale), scale, y.half() if s["case"]["y"] else None


def _plain_linear(s):
    y = s["xq"].float() @ s["wq"].float().t() * s["xs"][:, None] * s["ws"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(DT[s["case"]["dtype"]])


_run_plain = dict(attn=_plain_attn, append=_plain_append, verify=_plain_verify, norm=_plain_norm, linear=_plain_linear)


def work(case):
    c, e = case, {"f16": 2, "bf16": 2, "f32": 4}
    if c["op"] == "attn":
        # the first sequence is at the full length, the others at 0.7 of it on average
        tokens = c["ctx"] * (1 + 0.7 * (c["B"] - 1))
        rows = 2 * c["HK"] * (tokens + c["B"] * c["N"]) + 2 * c["H"] * c["B"] * c["N"]
        return {"bytes": 2 * c["D"] * rows, "flops": 4 * c["H"] * c["D"] * c["N"] * (tokens + c["B"] * c["N"] / 2)}
    if c["op"] == "append":
        n = c["B"] * (c["N"] if c["all"] else (c["N"] + 1) / 2)
        return {"bytes": 2 * 2 * 2 * c["HK"] * c["D"] * n, "flops": 0}
    if c["op"] == "verify":
        # every node's logits, and one row of the draft's probabilities for each sequence
        return {"bytes": c["B"] * c["V"] * (c["N"] * e[c["dtype"]] + (4 if c["q"] else 0)), "flops": 20 * c["B"] * c["N"] * c["V"]}
    if c["op"] == "norm":
        return {"bytes": c["T"] * c["d"] * (e[c["x"]] + 2 * e[c["res"]] + 1 + (2 if c["y"] else 0)) + 4 * c["d"] + 4 * c["T"],
                "flops": 8 * c["T"] * c["d"]}
    return {"bytes": c["N"] * c["K"] + c["M"] * c["K"] + e[c["dtype"]] * c["M"] * c["N"] + 4 * (c["M"] + c["N"]),
            "flops": 2 * c["M"] * c["N"] * c["K"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return dict(attn=_exact_attn, append=_exact_append, verify=_exact_verify, norm=_exact_norm, linear=_exact_linear)[case["op"]](s)


def _positions(s, b, n):
    """Page and offset of sequence b's first n positions."""
    j = torch.arange(n, device=DEV)
    return s["slots"][b][torch.div(j, s["page"], rounding_mode="floor")], torch.remainder(j, s["page"])


def _exact_attn(s):
    c = s["case"]
    out = torch.zeros(c["B"], c["N"], c["H"], c["D"], dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        at = _positions(s, b, int(s["ctx_len"][b]))
        for h in range(c["H"]):
            g = h * c["HK"] // c["H"]
            old = s["q"][b, :, h].double() @ s["k"][at[0], at[1], g].double().t() * s["scale"]
            new = s["q"][b, :, h].double() @ s["k_new"][b, :, g].double().t() * s["scale"]
            new[~s["anc"][b]] = -torch.inf
            w = torch.softmax(torch.cat([old, new], 1), 1)
            out[b, :, h] = w[:, :old.shape[1]] @ s["v"][at[0], at[1], g].double() + w[:, old.shape[1]:] @ s["v_new"][b, :, g].double()
    return out


def _exact_append(s):
    k, v = s["k"].double(), s["v"].double()
    for b in range(s["case"]["B"]):
        n, L = int(s["n"][b]), int(s["ctx_len"][b])
        page, off = _positions(s, b, L + n)
        src = s["nodes"][b, :n].long()
        k[page[L:], off[L:]] = s["k_new"][b, src].double()
        v[page[L:], off[L:]] = s["v_new"][b, src].double()
    return k, v, s["ctx_len"] + s["n"]


def _exact_verify(s):
    c = s["case"]
    nodes = torch.full((c["B"], c["N"]), -1, dtype=torch.int32)
    out, count = nodes.clone(), torch.zeros(c["B"], dtype=torch.int32)
    par, tok, u = s["parents"].tolist(), s["tokens"].tolist(), s["u"].tolist()
    for b in range(c["B"]):
        cur, path = 0, [0]
        while True:
            l = s["logits"][b, cur].double().cpu()
            if c["temp"] > 0:
                p = torch.softmax(l / float(s["temp"][b]), 0)
            else:
                p = torch.zeros_like(l)
                p[(l == l.max()).nonzero()[0, 0]] = 1
            r, found = p.clone(), None
            for i in range(cur + 1, c["N"]):  # r: what is left of the target, normalised
                if par[b][i] != cur:
                    continue
                t = tok[b][i]
                qd = s["q"][b, cur].double().cpu() if s["q"] is not None else None
                if u[b][i] * (1.0 if qd is None else float(qd[t])) < float(r[t]):
                    found = i
                    break
                if qd is None:
                    r[t] = 0
                else:
                    r = (r - qd).clamp(min=0)
                r = r / r.sum() if float(r.sum()) > 0 else r
            if found is None:
                break
            path.append(found)
            cur = found
        if float(r.sum()) == 0:
            r = p
        cum = r.cumsum(0)
        nxt = min(int((cum <= float(s["u_next"][b]) * float(cum[-1])).sum()), int(r.nonzero()[-1, 0]))
        nodes[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
        out[b, :len(path)] = torch.tensor([tok[b][i] for i in path[1:]] + [nxt], dtype=torch.int32)
        count[b] = len(path)
    return nodes, out, count


def _exact_norm(s):
    total = s["x"].double() + s["res"].double()
    h = total.to(s["res"].dtype).double()  # the norm is of the residual as it is stored
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + s["eps"]) * s["w"].double()
    scale = y.abs().amax(1) / 127
    return total, torch.round(y / scale[:, None]) * scale[:, None], scale, y if s["case"]["y"] else None


def _exact_linear(s):
    y = (s["xq"].double() @ s["wq"].double().t()) * s["xs"].double()[:, None] * s["ws"].double()[None, :]
    return y if s["bias"] is None else y + s["bias"].double()
