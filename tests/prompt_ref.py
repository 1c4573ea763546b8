"""Plain statements of the prompt and 4-bit cache operators in 64 bits on the CPU, for the tests."""
import torch


def quantize(x):
    """(codes uint8 [..][D/2], scales fp16 [..][D/32]) of values [..][D]: a block of 32 has the scale -m/8, m its
    largest element by magnitude (the positive one of two alike), rounded to 8 significant bits, at most 8160."""
    b = x.double().unflatten(-1, (-1, 32))
    odd = ~b.isfinite().all(-1)
    b = torch.where(odd[..., None], 0.0, b)
    hi, lo = b.amax(-1), b.amin(-1)
    m = torch.where(hi >= -lo, hi, lo)
    s = (m / -8).to(torch.bfloat16).double().clamp(-8160, 8160).to(torch.float16)
    d = s.double()[..., None]
    q = torch.where(d == 0, 8.0, torch.round(b / torch.where(d == 0, 1.0, d)) + 8).clamp(0, 15).to(torch.uint8)
    q = torch.where(odd[..., None], torch.full_like(q, 8), q)
    s = torch.where(odd, torch.full_like(s, float("nan")), s)
    return (q[..., :16] + 16 * q[..., 16:]).flatten(-2), s


def values(codes, scales):
    """float64 values [..][D] of codes and scales."""
    c = codes.unflatten(-1, (-1, 16)).to(torch.int64)
    q = torch.cat([c % 16, c // 16], -1).double() - 8
    return (q * scales.double()[..., None]).flatten(-2)


def rope(x, w, pos, freq, eps, pairs):
    """(out, size): heads [T][H][D] normalised and turned, and beside each element the magnitudes that its sum has."""
    y = x.double()
    if w is not None:
        mean = y.square().mean(-1, keepdim=True) + eps
        y = torch.where(mean > 0, y / mean.sqrt(), 0.0) * w.double()
    h = 0 if freq is None else freq.numel()
    out, size = y.clone(), y.abs()
    if h:
        angle = pos.double()[:, None] * freq.double()
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        i = torch.arange(h)
        f, g = (2 * i, 2 * i + 1) if pairs else (i, i + h)
        a, b = y[..., f], y[..., g]
        out[..., f], out[..., g] = a * c - b * s, b * c + a * s
        size[..., f] = size[..., g] = a.abs() + b.abs()
    return out, size


def prompt(q, k, v, cu_q, cu_k, scale):
    """(out, spread, score): causal attention of packed sequences, sum w |v| and the largest sum |q||k| * scale of a
    row beside it. Rows of no sequence are NaN."""
    T, H, D = q.shape
    G = H // k.shape[1]
    out = torch.full((T, H, D), float("nan"), dtype=torch.float64)
    spread, score = torch.zeros_like(out), torch.zeros(T, H, 1, dtype=torch.float64)
    for b in range(len(cu_q) - 1):
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for h in range(H):
            K, V = (x[cu_k[b]:cu_k[b + 1], h // G].double() for x in (k, v))
            for i in range(n):
                t, seen = cu_q[b] + i, max(0, i + 1 + m - n)
                x, ks, vs = q[t, h].double(), K[:seen], V[:seen]
                if seen == 0:
                    out[t, h] = 0
                    continue
                w = torch.softmax(ks @ x * scale, 0)
                out[t, h], spread[t, h] = w @ vs, w @ vs.abs()
                score[t, h] = (ks.abs() @ x.abs()).max() * scale
    return out, spread, score
