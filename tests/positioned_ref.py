"""Plain 64-bit forms (CPU) of the norm + rotation, the paged append and the tree
attention, and the error bounds their fp32 kernels are held to.

u = 2^-24, one rounding of fp32 to nearest.  `half(t)` is the rounding of a result
to type t, relative: half a step, torch.finfo(t).eps / 2."""
import decimal
import math

import torch

U = 2.0 ** -24
PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")


def half(dtype):
    return torch.finfo(dtype).eps / 2


def angles(pos, inv_freq):
    """pos * inv_freq modulo a turn, the product and the reduction in 100 digits
    (a float64 is an exact decimal), as float64 [T, 1, pairs]."""
    with decimal.localcontext() as ctx:
        ctx.prec = 100
        f = [decimal.Decimal(float(x)) for x in inv_freq]
        two_pi = 2 * PI
        rows = [[float((int(p) * x) % two_pi) for x in f] for p in pos]
    return torch.tensor(rows, dtype=torch.float64).reshape(len(pos), 1, len(f))


def rotate(x, ang, start, style):
    """x [T, heads, d] float64, ang [T, 1, rot/2]; style 0: pairs (p, p + rot/2), 1: (2p, 2p + 1)."""
    n = ang.shape[-1]
    if n == 0:
        return x
    p = torch.arange(n)
    a, b = (start + p, start + p + n) if style == 0 else (start + 2 * p, start + 2 * p + 1)
    c, s = ang.cos(), ang.sin()
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm(x, w, eps):
    x = x.double()
    return x if w is None else x * w.double() / (x.square().mean(-1, keepdim=True) + eps).sqrt()


def norm_rope(x, w, eps, ang, start, style):
    return rotate(norm(x, w, eps), ang, start, style)


def norm_rope_bound(x, w, eps, ang, start, style, out_dtype):
    """Largest error of one fp32 evaluation y = r (x A + x' B), rounded once:
      r  : 4 fma + 1 add + <= 4 shuffle adds + eps: 10u on r^2, 5u on r; rsqrtf 2 ulp = 4u  ->  9u
      A,B: cos/sin of a reduced angle |a| <= pi/4: conversion, constant and product 3u|a|, series
           remainder < 0.04u, evaluation < 1.6u  ->  4u absolute; times the weight  ->  5u |w|
      y  : product, fma, product by r  ->  3u
    17u of r (|x w| + |x' w'|); 20u taken."""
    n = norm(x, w, eps).abs()
    both = n.clone()
    k = ang.shape[-1]
    if k:
        p = torch.arange(k)
        a, b = (start + p, start + p + k) if style == 0 else (start + 2 * p, start + 2 * p + 1)
        both[..., a] = both[..., b] = n[..., a] + n[..., b]
    y = norm_rope(x, w, eps, ang, start, style)
    # (1 + half) on the fp32 error: it is rounded along with the value
    return half(out_dtype) * y.abs() + 1.01 * 20 * U * both + 1e-30


def paged_rows(pages, table, b, S):
    """Rows 0 .. S-1 of sequence b: [S, Hk, d]."""
    page = pages.shape[2]
    s = torch.arange(S)
    return pages[table[b].long()[s // page], :, s % page]


def tree_attention(q, Kp, Vp, table, lens, q_start, mask, scale, W=-1, pos=None):
    """[R, H, d] float64 outputs and [R, H] log-sum-exps; rows outside every sequence are NaN."""
    R, H, d = q.shape
    Hk = Kp.shape[1]
    O = torch.full((R, H, d), math.nan, dtype=torch.float64)
    lse = torch.full((R, H), math.nan, dtype=torch.float64)
    A = torch.full((R, H, d), math.nan, dtype=torch.float64)  # sum of p |v|: the scale of the error
    for b in range(len(lens)):
        L, n = int(lens[b]), int(q_start[b + 1] - q_start[b])
        for i in range(n):
            r = int(q_start[b]) + i
            lo = 0 if W < 0 else min(L, max(0, int(pos[r]) - W + 1))
            m = int(mask[r]) & (1 << 64) - 1
            at = list(range(lo, L)) + [L + j for j in range(n) if m >> j & 1]
            if not at:
                O[r], lse[r], A[r] = 0, -math.inf, 0
                continue
            at = torch.tensor(at)
            page = Kp.shape[2]
            pg = table[b].long()[at // page]
            K, V = Kp[pg, :, at % page].double(), Vp[pg, :, at % page].double()
            x = q[r].double().view(Hk, H // Hk, d)
            z = torch.einsum("hgd,khd->hgk", x, K) * scale
            l = torch.logsumexp(z, -1)
            p = (z - l[..., None]).exp()
            O[r] = torch.einsum("hgk,khd->hgd", p, V).reshape(H, d)
            A[r] = torch.einsum("hgk,khd->hgd", p, V.abs()).reshape(H, d)
            lse[r] = l.reshape(H)
    return O, lse, A
