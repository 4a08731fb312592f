"""Plain 64-bit forms of the operators of a batch's decode step on a paged cache, with the error bounds of their results."""
import math
from fractions import Fraction

import torch

from spec_ref import TWO_PI, U_BF16, U_FP32, row_of


def normed(x, weight, eps):
    """x [N][heads][dim] -> float64 x w / sqrt(mean(x^2) + eps), weight [dim] or [heads][dim]."""
    x = x.double()
    return x * weight.double() / torch.sqrt(x.square().mean(dim=-1, keepdim=True) + eps)


def turned(x, pos, axis, inv_freq, off, interleaved, dims):
    """x float64 [N][heads][dim] with dims [off, off + 2 len(inv_freq)) turned, pair j by pos[t][axis[j]]; and the bound of a
    32-bit computation from bf16 values, rounded once to bf16.

    A normed value is x r w: the sum of `dims` squares is off by at most dims 2^-24 relative (its root by half of that), the
    mean, eps and root by 2^-22, the two products by 2^-24 each; turning adds the sine's and cosine's 1e-6 < 2^-19 and
    three roundings.  All of it applies to |x| + |y| of a pair (a value that is not turned: to itself)."""
    half = len(inv_freq)
    off32 = (dims + 8) * U_FP32 + 2.0**-22 + 2.0**-19
    y, mag = x.clone(), x.abs()
    if half:
        turns = [Fraction(f) / TWO_PI for f in inv_freq]
        ang = torch.tensor([[2 * math.pi * float(p[axis[j]] * turns[j] % 1) for j in range(half)] for p in pos],
                           dtype=torch.float64, device=x.device).view(len(pos), half)
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        part = slice(off, off + 2 * half)
        if interleaved:
            u, w = x[..., part][..., 0::2], x[..., part][..., 1::2]
            y[..., part] = torch.stack([u * c - w * s, w * c + u * s], dim=-1).flatten(-2)
            mag[..., part] = (u.abs() + w.abs()).repeat_interleave(2, -1)
        else:
            u, w = x[..., part][..., :half], x[..., part][..., half:]
            y[..., part] = torch.cat([u * c - w * s, w * c + u * s], dim=-1)
            mag[..., part] = torch.cat([u.abs() + w.abs()] * 2, dim=-1)
    return y, U_BF16 * y.abs() + off32 * mag * (1 + U_BF16) + 2.0**-133  # the last: a subnormal's half step


def chosen(weights, n, keep, first, recent):
    """The entries that stay of n, ascending: weights a list of floats."""
    if n <= keep:
        return list(range(n))
    sure = set(range(first)) | set(range(n - recent, n))
    key = lambda p: (0 if math.isnan(weights[p]) else 1, -weights[p] if not math.isnan(weights[p]) else 0.0, p)  # noqa: E731
    rest = sorted((p for p in range(n) if p not in sure), key=key)
    return sorted(sure | set(rest[: keep - len(sure)]))


def evict(pages, table, max_pages, weights, out, lens, keep, first, recent):
    """pages [P][page][record], weights and out [R][lists][C] on the CPU -> the same after an eviction, exactly."""
    pages, new = pages.clone(), out.clone()
    R, lists, _ = weights.shape
    page, rec = pages.shape[1], pages.shape[2]
    was, now, width = pages.view(-1, rec).clone(), pages.view(-1, rec), rec // lists
    for r in range(R):
        for x in range(lists):
            kept = chosen(weights[r, x].tolist(), lens[r], keep, first[r], recent)
            new[r, x, : lens[r]] = 0.0
            new[r, x, : len(kept)] = weights[r, x, kept]
            cols = slice(x * width, (x + 1) * width)
            if kept:
                to = [row_of(table, r, i, page, max_pages) for i in range(len(kept))]
                at = [row_of(table, r, p, page, max_pages) for p in kept]
                now[to, cols] = was[at, cols]
    return pages, new, [min(n, keep) for n in lens]


def same(a, b):
    """Equal bit for bit, NaN included."""
    kind = {2: torch.int16, 4: torch.int32, 8: torch.int64}[a.element_size()]
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


def attention(cfg, rows, q, scale, own, only=None):
    """rows[r]: [n][record] of what request r sees, the last own[r] of them its own; q [R][Hq][Dqk]; only: the
    (request, head) pairs to compute, the others get no bound.

    Returns (out, bound) [R][Hq][Dv], as spec_ref.tree's in every term, and for each request the softmax weights of its own rows
    [Hq][own] with their bounds: a score is off by (Dqk + 2) 2^-24 |scale| sum |q K|, 2^x by 2^-21 relative, the normaliser
    by as much and n 2^-24 for its sum."""
    R, Hq, Dqk = q.shape
    Hkv, Dv = cfg.num_kv_heads, cfg.head_dim_v
    out = torch.zeros((R, Hq, Dv), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    weights = [torch.zeros((2, Hq, n), dtype=torch.float64, device=q.device) for n in own]
    for r in range(R):
        x = rows[r].double()
        if x.shape[0] == 0:
            continue
        for h in range(Hq):
            if only is not None and (r, h) not in only:
                bound[r, h] = math.inf
                weights[r][1, h] = math.inf
                continue
            if cfg.layout == 0:
                k, v = x[:, :Dqk], x[:, :Dv]
            else:
                g = h // (Hq // Hkv) * (Dqk + Dv)
                k, v = x[:, g:g + Dqk], x[:, g + Dqk:g + Dqk + Dv]
            qq = q[r, h].double()
            p = torch.softmax(k @ qq * scale, dim=0)
            out[r, h] = p @ v
            off = (Dqk + 2) * U_FP32 * abs(scale) * float((k.abs() @ qq.abs()).max())
            w = U_BF16 + off + 2.0**-21 + k.shape[0] * U_FP32
            bound[r, h] = U_BF16 * out[r, h].abs() + 2 * w * (1 + w) * (p @ v.abs()) * (1 + U_BF16)
            e = 2 * (off + 2.0**-21) + k.shape[0] * U_FP32
            if own[r]:
                weights[r][0, h] = p[-own[r]:]
                weights[r][1, h] = p[-own[r]:] * e * (1 + e) + 2.0**-126  # the last: exponents below the normal numbers'
    return out, bound, weights
