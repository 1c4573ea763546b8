"""Plain statements of the decoder operators in 64 bits on the CPU, for the tests."""
import torch


def cache_rows(pages, table, b, n):
    """The first n positions of sequence b of a cache tensor [pages][tokens][heads][dim] (on the
    CPU) as float64; positions of pages outside the cache are zeros."""
    size = pages.shape[1]
    out = torch.zeros(n, *pages.shape[2:], dtype=torch.float64)
    for p in range(n):
        page = b if table is None else int(table[b, p // size])
        if 0 <= page < pages.shape[0]:
            out[p] = pages[page, p % size].double()
    return out


def tree_attention(q, k_pages, v_pages, k_new, v_new, sees, table, ctx_len, scale):
    """(out, spread, score): the attention in float64, sum w |v| beside it (what an error relative
    to the weights scales with), and the largest sum |q||k| * scale of a row. ``sees`` [B][N][N]."""
    B, N, H, D = q.shape
    HK = k_pages.shape[2]
    out = torch.zeros(B, N, H, D, dtype=torch.float64)
    spread, score = torch.zeros_like(out), torch.zeros(B, N, H, 1, dtype=torch.float64)
    for b in range(B):
        n = int(ctx_len[b])
        kc, vc = cache_rows(k_pages, table, b, n), cache_rows(v_pages, table, b, n)
        for h in range(H):
            g = h * HK // H
            k = torch.cat([kc[:, g], k_new[b, :, g].double()])
            v = torch.cat([vc[:, g], v_new[b, :, g].double()])
            for i in range(N):
                seen = torch.cat([torch.ones(n, dtype=torch.bool), sees[b, i]])
                if not seen.any():
                    continue
                ks, vs, x = k[seen], v[seen], q[b, i, h].double()
                w = torch.softmax(ks @ x * scale, 0)
                out[b, i, h] = w @ vs
                spread[b, i, h] = w @ vs.abs()
                score[b, i, h] = (ks.abs() @ x.abs()).max() * scale
    return out, spread, score


def verify(logits, tokens, parents, u, u_next, q, temperature):
    """Rejection sampling of one tree: (nodes, tokens) of the path."""
    N, V = logits.shape
    cur, path = 0, [0]
    while True:
        z = logits[cur].double()
        z = torch.where(z.isnan(), -torch.inf, z).clamp(max=torch.finfo(torch.float32).max)
        if z.max() == -torch.inf:
            return path, [int(tokens[i]) for i in path[1:]] + [-1]
        if temperature > 0:
            p = torch.softmax((z - z.max()) / temperature, 0)
        else:
            p = torch.zeros(V, dtype=torch.float64)
            p[int((z == z.max()).nonzero()[0, 0])] = 1
        r, found = p.clone(), None
        for i in range(cur + 1, N):
            if int(parents[i]) != cur:
                continue
            t = int(tokens[i])
            inside = 0 <= t < V
            if inside and float(u[i]) * (1.0 if q is None else float(q[cur, t])) < float(r[t]):
                found = i
                break
            if q is not None:
                r = (r - q[cur].double()).clamp(min=0)
            elif inside:
                r[t] = 0
            r = r / r.sum() if float(r.sum()) > 0 else r
        if found is None:
            break
        path.append(found)
        cur = found
    if float(r.sum()) == 0:
        r = p
    cum = r.cumsum(0)
    nxt = min(int((cum <= float(u_next) * float(cum[-1])).sum()), int(r.nonzero()[-1, 0]))
    return path, [int(tokens[i]) for i in path[1:]] + [nxt]
