"""Plain 64-bit forms of the speculative-decoding operators, with the error bounds of their results."""
import math
from fractions import Fraction

import torch

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")

# largest relative error of one rounding (half a step)
U_BF16, U_FP32 = 2.0**-8, 2.0**-24


def row_of(table, r, p, page_tokens, max_pages):
    page = int(table[r][p // page_tokens]) if table is not None else r * max_pages + p // page_tokens
    return page * page_tokens + p % page_tokens


def sees(mask, r, i, j):
    return (int(mask[r][i][j // 64]) >> (j % 64)) & 1 == 1


def tree(cfg, context_rows, node_rows, q, mask, nodes, scale, only=None):
    """context_rows[r], node_rows[r]: [n][record] tensors; q [R][T][Hq][Dqk]; mask, nodes host lists;
    only: the (request, node, head) triples to compute, the others get no bound.

    Returns (out, bound) in float64, [R][T][Hq][Dv].  The bound, per value:
      - the output's rounding: 2^-8 |o|;
      - each weight rounded to bf16, the normaliser summing the rounded weights: the weighted mean moves by
        at most 2^-8 in its numerator and its denominator, 2 * 2^-8 * A with A = sum p |V|;
      - a score is a 32-bit dot product of exact bf16 products: it is off by at most
        (Dqk + 2) 2^-24 |scale| sum |q K|, and 2^x by 2^-21 relative (argument reduction and function): 2 A times both;
      - sums of n weights and products in 32 bits: n 2^-24, likewise 2 A."""
    R, T, Hq, Dqk = q.shape
    Hkv, Dv = cfg.num_kv_heads, cfg.head_dim_v
    out = torch.zeros((R, T, Hq, Dv), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for r in range(R):
        nn = nodes[r]
        if nn == 0:
            continue
        rows = torch.cat([context_rows[r], node_rows[r][:nn]]).double()
        n = rows.shape[0]
        ok = torch.ones((nn, n), dtype=torch.bool)
        for i in range(nn):
            for j in range(nn):
                ok[i, n - nn + j] = sees(mask, r, i, j)
        ok = ok.to(q.device)
        for h in range(Hq):
            if cfg.layout == 0:
                k, v = rows[:, :Dqk], rows[:, :Dv]
            else:
                g = h // (Hq // Hkv) * (Dqk + Dv)
                k, v = rows[:, g:g + Dqk], rows[:, g + Dqk:g + Dqk + Dv]
            qq = q[r, :nn, h].double()
            # values that a node does not see (NaN among them) have no part in anything
            for i in range(nn):
                if only is not None and (r, i, h) not in only:
                    bound[r, i, h] = math.inf
                    continue
                if not bool(ok[i].any()):
                    continue
                kk, vv = k[ok[i]], v[ok[i]]
                s = kk @ qq[i] * scale
                p = torch.softmax(s, dim=0)
                out[r, i, h] = p @ vv
                a = p @ vv.abs()
                # |scale|: an error bound is a magnitude (a negative scale would lower it below the roundings')
                off = (Dqk + 2) * U_FP32 * abs(scale) * float((kk.abs() @ qq[i].abs()).max())
                w = U_BF16 + off + 2.0**-21 + vv.shape[0] * U_FP32
                bound[r, i, h] = U_BF16 * out[r, i, h].abs() + 2 * w * (1 + w) * a * (1 + U_BF16)
    return out, bound


def assert_tree(got, want, bound, nodes, before=None):
    for r, nn in enumerate(nodes):
        g = got[r, :nn].double()
        err = (g - want[r, :nn]).abs()
        assert bool(torch.isfinite(g).all()), (r, "not finite")
        assert bool((err <= bound[r, :nn]).all()), (r, float((err - bound[r, :nn]).max()), float(err.max()))
        if before is not None:
            assert torch.equal(got[r, nn:], before[r, nn:]), (r, "rows behind the nodes in use")


def rotated(x, pos, inv_freq, off, interleaved):
    """x [N][heads][dim] -> float64 with dims [off, off + 2 len(inv_freq)) rotated, and the bound of a
    32-bit computation rounded once to bf16: the rounding, and 2^-20 of |x| + |y| for the angle's sine and
    cosine (1e-6 at most, stated with the operator) and three 32-bit roundings."""
    half = len(inv_freq)
    turns = [Fraction(f) / TWO_PI for f in inv_freq]
    ang = torch.tensor([[2 * math.pi * float(p * t % 1) for t in turns] for p in pos], dtype=torch.float64,
                       device=x.device).view(len(pos), half)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    y = x.double().clone()
    b = torch.zeros_like(y)
    part = slice(off, off + 2 * half)
    if interleaved:
        u, w = x[..., part][..., 0::2].double(), x[..., part][..., 1::2].double()
        z, e = torch.stack([u * c - w * s, w * c + u * s], dim=-1).flatten(-2), (u.abs() + w.abs()).repeat_interleave(2, -1)
    else:
        u, w = x[..., part][..., :half].double(), x[..., part][..., half:].double()
        z, e = torch.cat([u * c - w * s, w * c + u * s], dim=-1), torch.cat([u.abs() + w.abs()] * 2, dim=-1)
    y[..., part] = z
    b[..., part] = U_BF16 * z.abs() + 2.0**-20 * e
    return y, b
