"""The decoder's operators around prompts and the 4-bit cache, as cases to measure: norm and rotary
positions of query and key heads, attention over whole prompts of packed sequences, the key/value
cache held in 4 bits (written, read back), and attention of a token tree over that cache.

``run`` computes a case in plain torch (``own = False``) or through the library (``own = True``).
"""
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"
BLOCK = 32  # elements of a head that share a scale in the 4-bit cache


def listed():
    return [
        # the heads of 8 drafted tokens of one step, positions only: latency counts
        dict(name="rope step", op="rope", T=8, H=32, HK=32, D=128, rot=128, dtype="f16", norm=False, pairs=False),
        # a prompt's grouped heads, each normalised first, out of the fused projection
        dict(name="rope prompt", op="rope", T=8192, H=64, HK=8, D=128, rot=128, dtype="bf16", norm=True, pairs=False),
        # accepted paths of up to 8 tokens of 16 users enter the 4-bit cache and are read back from it
        dict(name="write paths", op="write", B=16, N=8, HK=8, D=128, ctx=1000, page=16, dtype="f16", all=False, by_head=True),
        # prompts of a batch enter it
        dict(name="write prompts", op="write", B=16, N=1024, HK=8, D=128, ctx=0, page=64, dtype="bf16", all=True, by_head=True),
        # one user's held prompt, read for its continuation
        dict(name="read prompt", op="read", B=1, HK=8, D=128, ctx=4001, page=16, dtype="f16", by_head=True),
        # the long prompts of a batch
        dict(name="read prompts", op="read", B=8, HK=8, D=128, ctx=16384, page=64, dtype="bf16", by_head=True),
        # one token of one sequence over a short 4-bit cache
        dict(name="attn4 step", op="attn4", B=1, N=1, H=32, HK=32, D=128, ctx=512, page=16, dtype="f16", by_head=True),
        # one token each of many users
        dict(name="attn4 batch", op="attn4", B=64, N=1, H=64, HK=8, D=128, ctx=8191, page=64, dtype="bf16", by_head=True),
        # trees of 26 drafted tokens over long caches
        dict(name="attn4 trees", op="attn4", B=4, N=26, H=64, HK=8, D=128, ctx=32768, page=64, dtype="f16", by_head=True),
        # a short prompt of one user
        dict(name="prompt short", op="prompt", B=1, L=500, held=0, H=32, HK=32, D=128, dtype="f16"),
        # packed prompts of unlike lengths, some continued after a held part
        dict(name="prompt packed", op="prompt", B=16, L=2047, held=1500, H=64, HK=8, D=128, dtype="bf16"),
        # one long prompt
        dict(name="prompt long", op="prompt", B=1, L=16384, held=0, H=32, HK=8, D=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def _odd(rng, lo, hi):
    """The same, odd (listed sizes are mostly even): hi is left out where it is even."""
    return min(_log(rng, lo, hi) | 1, hi - 1 + hi % 2)


HEADS = [(32, 32), (64, 8), (16, 16), (40, 8), (8, 1), (12, 4), (32, 8), (96, 96)]


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn4", "attn4", "prompt", "prompt"])
    H, HK = rng.choice(HEADS)
    dtype = rng.choice(["f16", "bf16"])
    if op == "rope":
        D = rng.choice([64, 128, 128, 80, 256])
        T = max(1, min(_odd(rng, 1, 16384), 8192 * 72 * 128 // ((H + HK) * D)))
        return dict(op=op, T=T, H=H, HK=HK, D=D, rot=rng.choice([D, D, D // 2]), dtype=rng.choice(["f16", "bf16", "f32"]),
                    norm=rng.random() < 0.5, pairs=rng.random() < 0.4)
    if op == "prompt":
        D = rng.choice([64, 64, 128, 128, 128, 96, 80, 256])
        B, L, held = _log(rng, 1, 32), _odd(rng, 1, 8192), rng.choice([0, 0, _odd(rng, 1, 8192)])
        c = dict(op=op, B=B, L=L, held=held, H=H, HK=HK, D=D, dtype=dtype)
        top = 4 * 32 * 128 * 16384 * 8192
        while work(c)["flops"] > top // 4 or B * H * (L + held) * L > 1 << 33:
            c["L"], c["held"] = L, held = max(1, L // 2), held // 2
        return c
    D, page, by_head = rng.choice([64, 128, 128, 128, 96, 256]), rng.choice([0, 16, 16, 64, 48, 256]), rng.random() < 0.7
    if op == "write":
        B, N, ctx = _log(rng, 1, 64), _log(rng, 1, 1024), rng.choice([0, _odd(rng, 1, 2000)])
        N = max(1, min(N, 16 * 1024 * 8 * 128 // (B * HK * D)))
        return dict(op=op, B=B, N=N, HK=HK, D=D, ctx=ctx, page=page, dtype=dtype, all=rng.random() < 0.5, by_head=by_head)
    if op == "read":
        B, ctx = _log(rng, 1, 32), _odd(rng, 1, 16384)
        ctx = max(1, min(ctx, 8 * 16384 * 8 * 128 // (B * HK * D)))
        return dict(op=op, B=B, HK=HK, D=D, ctx=ctx, page=page, dtype=dtype, by_head=by_head)
    B, N, ctx = _log(rng, 1, 64), rng.choice([1, _log(rng, 1, 64)]), _odd(rng, 1, 32768)
    # no more than the listed cases' cache bytes and products
    ctx = max(1, min(ctx, 64 * 8 * 8192 * 128 // (B * HK * D), 4 * 26 * 64 * 32768 * 128 // (B * N * H * D)))
    return dict(op=op, B=B, N=N, H=H, HK=HK, D=D, ctx=ctx, page=page, dtype=dtype, by_head=by_head)


def _share(b, top):
    """Length of the b-th of several sequences of unlike lengths: the first is at the full one, the
    others between 0.4 and 1 of it."""
    return top if b == 0 else int(top * (0.4 + 0.6 * ((0.618034 * b) % 1.0)))


def _prompt_lens(c):
    """(new tokens, tokens held before) of every sequence; where some are held, every third holds none."""
    return [(max(1, _share(b, c["L"])), 0 if b % 3 == 2 else _share(b, c["held"])) for b in range(c["B"])]


def _cache_lens(c):
    return [_share(b, c["ctx"]) for b in range(c["B"])]


def _path_lens(c):
    return [c["N"] if c["all"] else max(1, _share(b, c["N"])) for b in range(c["B"])]


# ---------------------------------------------------------------- the 4-bit format

def _quantize(x):
    """Codes [..][D/32][16] and scales [..][D/32] of fp32 values [..][D]: byte j of a block holds element j
    in its low half and element j + 16 in its high half; a value is (code - 8) * scale."""
    b = x.unflatten(-1, (-1, BLOCK))
    hi, lo = b.amax(-1), b.amin(-1)
    m = torch.where(hi >= -lo, hi, lo)
    s = (m / -8).to(torch.bfloat16).float().clamp(-8160, 8160).to(torch.float16)
    f = s.float().unsqueeze(-1)
    q = torch.where(f == 0, 8.0, torch.round(b / f) + 8).clamp(0, 15).to(torch.uint8)
    return (q[..., :16] | (q[..., 16:] << 4)).flatten(-2), s


def _values(codes, scales):
    """fp32 values [..][D] of codes [..][D/2] and scales [..][D/32]."""
    c = codes.unflatten(-1, (-1, 16))
    q = torch.cat([c & 15, c >> 4], -1).float() - 8
    return (q * scales.float().unsqueeze(-1)).flatten(-2)


def _pages(c, more):
    """Pages of every sequence and their table, with room for ``more`` tokens after ctx."""
    room = c["ctx"] + more
    return (room, 1, c["B"]) if c["page"] == 0 else (c["page"], -(-room // c["page"]), c["B"] * -(-room // c["page"]))


def _cache(c, g, more):
    B, HK, D = c["B"], c["HK"], c["D"]
    page, width, pages = _pages(c, more)
    table = None
    if c["page"]:
        table = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).view(B, width).contiguous()
    s = dict(table=table, page=page, slots=torch.arange(B, device=DEV)[:, None] if table is None else table.long(),
             ctx_len=torch.tensor(_cache_lens(c), dtype=torch.int32, device=DEV))
    for n in "kv":
        # a head's tokens of a page next to each other, or a token's heads
        shape = (pages, HK, page, D) if c["by_head"] else (pages, page, HK, D)
        codes, scales = _quantize(torch.randn(shape, generator=g, device=DEV).to(DT[c["dtype"]]).float())
        s[n], s[n + "_scale"] = [t.transpose(1, 2) if c["by_head"] else t for t in (codes, scales)]
    return s


def _ancestors(r, B, N):
    """[B][N][N] truth values of random trees: node i sees node j where j is i or above it."""
    out = torch.zeros(B, N, N, dtype=torch.bool)
    for b in range(B):
        for i in range(N):
            if i:
                out[b, i] = out[b, r.randrange(max(0, i - 6), i)]
            out[b, i, i] = True
    return out.to(DEV)


def _words(anc):
    """Truth values [B][N][N] as 64-bit mask words [B][N], bit j for node j."""
    bit = torch.bitwise_left_shift(torch.ones((), dtype=torch.int64, device=DEV), torch.arange(anc.shape[2], device=DEV))
    return (anc.to(torch.int64) * bit).sum(2)


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, g, r = case, torch.Generator(DEV).manual_seed(seed), random.Random(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    s, op, dt, D = dict(case=c), c["op"], DT[c["dtype"]], c["D"]
    empty = lambda *n, dtype=dt: torch.empty(*n, dtype=dtype, device=DEV)  # noqa: E731
    if op == "rope":
        T, H, HK = c["T"], c["H"], c["HK"]
        qkv = (1.5 * randn(T, H + 2 * HK, D)).to(dt)
        s.update(q=qkv[:, :H], k=qkv[:, H:H + HK], eps=1e-6)
        # tokens of a few sequences: runs of positions from somewhere in a long context on
        first = torch.randint(0, 131072, (max(1, T // 64),), generator=g, device=DEV)
        at = torch.arange(T, device=DEV)
        s["pos"] = (first[(at // 64).clamp(max=len(first) - 1)] + at % 64).to(torch.int32)
        s["freq"] = (10000.0 ** (-2 * torch.arange(c["rot"] // 2, device=DEV).double() / c["rot"])).float()
        s["wq"], s["wk"] = [1 + 0.2 * randn(D) if c["norm"] else None for _ in range(2)]
        s["q_out"], s["k_out"] = empty(T, H, D), empty(T, HK, D)
    elif op == "prompt":
        lens = _prompt_lens(c)
        cu_q, cu_k = _offsets([n for n, _ in lens]), _offsets([n + h for n, h in lens])
        Tq, Tk = sum(n for n, _ in lens), sum(n + h for n, h in lens)
        s.update(lens=lens, cu_q=cu_q, cu_k=cu_k, q=(2 * randn(Tq, c["H"], D)).to(dt), k=randn(Tk, c["HK"], D).to(dt),
                 v=randn(Tk, c["HK"], D).to(dt), out=empty(Tq, c["H"], D), scale=D ** -0.5)
    else:
        B, HK = c["B"], c["HK"]
        N = c.get("N", 0)
        s.update(_cache(c, g, N))
        if op != "read":
            s.update(k_new=randn(B, N, HK, D).to(dt), v_new=randn(B, N, HK, D).to(dt))
        if op == "attn4":
            s.update(q=(2 * randn(B, N, c["H"], D)).to(dt), anc=_ancestors(r, B, N), scale=D ** -0.5, out=empty(B, N, c["H"], D))
            s["words"] = _words(s["anc"])
        elif op == "write":
            n = _path_lens(c)
            nodes = [sorted(r.sample(range(N), m)) + [-1] * (N - m) for m in n]
            s.update(n=torch.tensor(n, dtype=torch.int32, device=DEV), nodes=torch.tensor(nodes, dtype=torch.int32, device=DEV),
                     len_out=empty(B, dtype=torch.int32), cu=_offsets(n), rows=sum(n))
        else:
            s.update(cu=_offsets(_cache_lens(c)), rows=sum(_cache_lens(c)))
        if op != "attn4":
            s.update(k_out=empty(s["rows"], HK, D), v_out=empty(s["rows"], HK, D))
    if own:
        _handles(c, s)
    return s


def _handles(c, s):
    """What a program keeps between steps: the context and the operators' handles."""
    import activation_sparse_ffn_layer_amd as pi

    s["pi"], s["ctx"] = pi, pi.Context(max_batch=1, max_d=64, max_ffn=64, max_rank=0)
    if c["op"] in ("attn4", "write", "read"):
        s["cache"] = pi.KvCache4(s["ctx"], s["k"], s["v"], s["k_scale"], s["v_scale"], DT[c["dtype"]])
    if c["op"] == "attn4":
        s["attn"] = pi.Attn(s["ctx"], s["cache"], c["H"], max_batch=c["B"], max_nodes=c["N"], scale=s["scale"])
    elif c["op"] == "prompt":
        s["attn"] = pi.PromptAttn(s["ctx"], c["H"], c["HK"], c["D"], DT[c["dtype"]], max_tokens=s["q"].shape[0],
                                  max_batch=c["B"], scale=s["scale"])


def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


# ---------------------------------------------------------------- through the library

def _own_rope(s):
    s["pi"].qk_norm_rope(s["ctx"], s["q"], s["k"], s["pos"], s["freq"], s["q_out"], s["k_out"], q_norm=s["wq"],
                         k_norm=s["wk"], eps=s["eps"], interleaved=s["case"]["pairs"])
    return s["q_out"], s["k_out"]


def _own_write(s):
    s["pi"].kv_append(s["ctx"], s["cache"], s["k_new"], s["v_new"], s["table"], s["ctx_len"], s["len_out"], s["nodes"], s["n"])
    s["pi"].kv_read(s["ctx"], s["cache"], s["table"], s["len_out"], s["cu"], s["k_out"], s["v_out"], start=s["ctx_len"])
    return s["k_out"], s["v_out"], s["len_out"]


def _own_read(s):
    s["pi"].kv_read(s["ctx"], s["cache"], s["table"], s["ctx_len"], s["cu"], s["k_out"], s["v_out"])
    return s["k_out"], s["v_out"]


def _own_attn4(s):
    s["pi"].tree_attention(s["ctx"], s["attn"], s["q"], s["k_new"], s["v_new"], s["words"], s["table"], s["ctx_len"], s["out"])
    return s["out"]


def _own_prompt(s):
    s["pi"].prompt_attention(s["ctx"], s["attn"], s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"])
    return s["out"]


_run_own = dict(rope=_own_rope, write=_own_write, read=_own_read, attn4=_own_attn4, prompt=_own_prompt)


# ---------------------------------------------------------------- in plain torch

def _plain_rope(s):
    c = s["case"]
    h = c["rot"] // 2
    angle = s["pos"].double()[:, None] * s["freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(2, keepdim=True) + s["eps"]) * w
        if c["pairs"]:
            a, b = y[..., 0:2 * h:2], y[..., 1:2 * h:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
        else:
            a, b = y[..., :h], y[..., h:2 * h]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
        out.append(torch.cat([turned, y[..., 2 * h:]], 2).to(x.dtype))
    return tuple(out)


def _rows(s, start):
    """Page and offset of every row that is read: sequence b's positions from start[b] on."""
    cu = s["cu"].long()
    row = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(cu, row, right=True) - 1
    at = row - cu[b] + (0 if start is None else start.long()[b])
    return s["slots"][b, at // s["page"]], at % s["page"]


def _read_back(s, start=None):
    page, off = _rows(s, start)
    return tuple(_values(s[n][page, off], s[n + "_scale"][page, off]).to(DT[s["case"]["dtype"]]) for n in "kv")


def _plain_write(s):
    c = s["case"]
    j = torch.arange(c["N"], device=DEV)
    new = j < s["n"][:, None]
    at = (s["ctx_len"].long()[:, None] + j)[new]
    b = torch.arange(c["B"], device=DEV)[:, None].expand_as(new)[new]
    page, off = s["slots"][b, at // s["page"]], at % s["page"]
    src = s["nodes"].long()[new]
    for n in "kv":
        s[n][page, off], s[n + "_scale"][page, off] = _quantize(s[n + "_new"][b, src].float())
    return _read_back(s, s["ctx_len"]) + (s["ctx_len"] + s["n"],)


def _plain_read(s):
    return _read_back(s)


def _plain_attn4(s):
    c = s["case"]
    B, N, H, HK, D, G = c["B"], c["N"], c["H"], c["HK"], c["D"], c["H"] // c["HK"]
    L = s["slots"].shape[1] * s["page"]
    held = (torch.arange(L, device=DEV) < s["ctx_len"][:, None])[:, :, None, None]

    def whole(n):  # [B][HK][L + N][D], zeros where nothing is held
        old = _values(s[n][s["slots"]], s[n + "_scale"][s["slots"]]).reshape(B, L, HK, D)
        return torch.cat([torch.where(held, old, 0.0), s[n + "_new"].float()], 1).transpose(1, 2).contiguous()

    q = s["q"].float().view(B, N, HK, G, D).permute(0, 2, 1, 3, 4).reshape(B, HK, N * G, D)
    sees = torch.cat([held[:, None, :, 0, 0].expand(B, N, L), s["anc"]], 2)
    w = (q @ whole("k").transpose(2, 3).contiguous() * s["scale"]).view(B, HK, N, G, L + N)
    w = torch.where(sees[:, None, :, None], w, -torch.inf)
    w = torch.exp(w - w.amax(4, keepdim=True))
    w = w / w.sum(4, keepdim=True)
    o = w.view(B, HK, N * G, L + N) @ whole("v")
    return o.view(B, HK, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, H, D).to(s["q"].dtype)


def _plain_prompt(s):
    c = s["case"]
    G, out = c["H"] // c["HK"], s["out"]
    q0 = k0 = 0
    for n, held in s["lens"]:
        m = n + held
        seen = torch.arange(m, device=DEV) <= torch.arange(held, m, device=DEV)[:, None]
        for g in range(c["HK"]):
            k, v = s["k"][k0:k0 + m, g].float(), s["v"][k0:k0 + m, g].float()
            step = max(1, min(G, (1 << 30) // (n * m)))  # heads of the group at once
            for h in range(g * G, (g + 1) * G, step):
                e = min(h + step, (g + 1) * G)
                q = s["q"][q0:q0 + n, h:e].float().transpose(0, 1).reshape(-1, c["D"])
                w = (q @ k.t() * s["scale"]).view(-1, n, m)
                w = torch.where(seen, w, -torch.inf)
                w = torch.exp(w - w.amax(2, keepdim=True))
                w = w / w.sum(2, keepdim=True)
                out[q0:q0 + n, h:e] = (w.view(-1, m) @ v).view(-1, n, c["D"]).transpose(0, 1).to(out.dtype)
        q0, k0 = q0 + n, k0 + m
    return out


_run_plain = dict(rope=_plain_rope, write=_plain_write, read=_plain_read, attn4=_plain_attn4, prompt=_plain_prompt)


def work(case):
    c, D = case, case["D"]
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rope":
        n = c["T"] * (c["H"] + c["HK"]) * D
        return {"bytes": 2 * e * n + 4 * c["T"], "flops": (6 if c["norm"] else 3) * n}
    if c["op"] == "prompt":
        lens = _prompt_lens(c)
        rows = sum(2 * c["H"] * n + 2 * c["HK"] * (n + h) for n, h in lens)
        return {"bytes": e * D * rows, "flops": 4 * c["H"] * D * sum(n * h + n * (n + 1) // 2 for n, h in lens)}
    packed = 2 * c["HK"] * (D // 2 + D // 16)  # a position's keys and values in the cache
    plain = 2 * c["HK"] * D * e
    if c["op"] == "write":
        return {"bytes": sum(_path_lens(c)) * (2 * plain + 2 * packed), "flops": 0}
    if c["op"] == "read":
        return {"bytes": sum(_cache_lens(c)) * (packed + plain), "flops": 0}
    held, new = sum(_cache_lens(c)), c["B"] * c["N"]
    return {"bytes": held * packed + new * plain + 2 * e * D * c["H"] * new,
            "flops": 4 * c["H"] * D * c["N"] * (held + c["B"] * c["N"] / 2)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return dict(rope=_exact_rope, write=_exact_write, read=_exact_read, attn4=_exact_attn4, prompt=_exact_prompt)[case["op"]](s)


def _exact_rope(s):
    c = s["case"]
    half = c["rot"] // 2
    z = torch.exp(1j * torch.outer(s["pos"].double(), s["freq"].double()))  # a pair turns as a complex number
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(y.square().mean(2, keepdim=True) + s["eps"]) * w.double()
        i = torch.arange(half, device=DEV)
        first, second = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + half)
        t = torch.complex(y[..., first], y[..., second]) * z[:, None]
        o = y.clone()
        o[..., first], o[..., second] = t.real, t.imag
        out.append(o)
    return tuple(out)


def _unpack(codes, scales):
    """float64 values of codes [..][D/2], element by element of a block."""
    parts = []
    for b in range(scales.shape[-1]):
        byte = codes[..., 16 * b:16 * b + 16].long()
        parts += [(byte % 16 - 8) * scales[..., b:b + 1].double(), (byte // 16 - 8) * scales[..., b:b + 1].double()]
    return torch.cat(parts, -1)


def _held(s, name, b, first, last):
    """Positions first..last of sequence b as float64 [..][HK][D]."""
    at = torch.arange(first, last, device=DEV)
    page = s["slots"][b][torch.div(at, s["page"], rounding_mode="floor")]
    off = torch.remainder(at, s["page"])
    return _unpack(s[name][page, off], s[name + "_scale"][page, off])


def _exact_write(s):
    out = []
    for name in "kv":
        rows = torch.cat([s[name + "_new"][b, s["nodes"][b, :int(s["n"][b])].long()] for b in range(s["case"]["B"])]).double()
        for e in range(0, s["case"]["D"], BLOCK):
            x = rows[..., e:e + BLOCK]
            big = torch.take_along_dim(x, x.abs().argmax(-1, keepdim=True), -1)
            big = torch.where(x.amax(-1, keepdim=True) == big.abs(), big.abs(), big)  # of two alike the positive one
            scale = (big / -8).to(torch.bfloat16).double().clamp(-8160, 8160).half().double()
            code = torch.where(scale == 0, 0.0, torch.round(x / torch.where(scale == 0, 1.0, scale))).clamp(-8, 7)
            rows[..., e:e + BLOCK] = code * scale
        out.append(rows)
    return tuple(out) + (s["ctx_len"] + s["n"],)


def _exact_read(s):
    lens = s["ctx_len"].tolist()
    return tuple(torch.cat([_held(s, n, b, 0, m) for b, m in enumerate(lens)]) for n in "kv")


def _exact_attn4(s):
    c = s["case"]
    out = torch.zeros(c["B"], c["N"], c["H"], c["D"], dtype=torch.float64, device=DEV)
    G = c["H"] // c["HK"]
    for b in range(c["B"]):
        n = int(s["ctx_len"][b])
        k = torch.cat([_held(s, "k", b, 0, n), s["k_new"][b].double()])
        v = torch.cat([_held(s, "v", b, 0, n), s["v_new"][b].double()])
        for g in range(c["HK"]):
            for h in range(g * G, g * G + G):
                x = s["q"][b, :, h].double() @ k[:, g].t() * s["scale"]
                x[:, n:][~s["anc"][b]] = -torch.inf
                out[b, :, h] = torch.softmax(x, 1) @ v[:, g]
    return out


def _exact_prompt(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    G = c["H"] // c["HK"]
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(c["B"]):
        n, m = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        for h in range(c["H"]):
            k, v = (s[x][ck[b]:ck[b + 1], h // G].double() for x in "kv")
            for i in range(0, n, 4096):  # rows at once
                e = min(n, i + 4096)
                x = s["q"][cq[b] + i:cq[b] + e, h].double() @ k.t() * s["scale"]
                x += torch.full_like(x, -torch.inf).triu(m - n + i + 1)
                out[cq[b] + i:cq[b] + e, h] = torch.softmax(x, 1) @ v
    return out
