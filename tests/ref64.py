"""Plain 64-bit forms of the norm-and-rotation pair and of the shared-prefix
attention (torch float64, any device), for the tests."""
import math

import torch


def angles(pos, inv_freq):
    """cos, sin [b, S, 1, R/2] at integer positions [b, S]."""
    a = pos.double()[:, :, None, None] * inv_freq.double()
    return a.cos(), a.sin()


def _turn(y, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    z = y.clone()
    if interleaved:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        z[..., 0:R:2], z[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., : R // 2], y[..., R // 2: R]
        z[..., : R // 2], z[..., R // 2: R] = a * cos - b * sin, b * cos + a * sin
    return z


def _pos(x, pos):
    b, S = x.shape[:2]
    return pos if pos is not None else torch.arange(S, device=x.device).expand(b, S)


def norm_rope(x, w, eps, inv_freq, pos=None, interleaved=False):
    """(z, y): rotated and not yet rotated normed heads of x [b, S, heads, D]."""
    x = x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if w is None else w.double()
    y = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt() * w
    if inv_freq is None:
        return y, y
    return _turn(y, *angles(_pos(x, pos), inv_freq), interleaved), y


def norm_rope_bwd(x, g, w, eps, inv_freq, pos=None, interleaved=False):
    """(dx, dw, scale of dx's terms [.., 1], bound on the fp32 error of dw [D]): 512 * 2^-24
    of the sum of its terms' magnitudes for the additions, and for the terms themselves, which
    turn g back and may cancel there, 2^-20 of the row's largest |g| (angles within 2^-22 and
    three roundings of 2^-24, each relative to |g_a| + |g_b|)."""
    x, g = x.double(), g.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if w is None else w.double()
    r = ((x * x).mean(-1, keepdim=True) + eps) ** -0.5
    xh = x * r
    turned = (g.abs().amax(-1, keepdim=True) * xh.abs()).sum((0, 1, 2))
    if inv_freq is not None:
        cos, sin = angles(_pos(x, pos), inv_freq)
        g = _turn(g, cos, -sin, interleaved)
    e = g * w
    dx = r * (e - xh * (e * xh).mean(-1, keepdim=True))
    size = r * (e.abs().amax(-1, keepdim=True) + xh.abs().amax(-1, keepdim=True) * (e * xh).abs().mean(-1, keepdim=True))
    bound = 512 * 2.0 ** -24 * (g * xh).abs().sum((0, 1, 2)) + 2.0 ** -20 * turned
    return dx, (g * xh).sum((0, 1, 2)), size, bound


def prefix_attn(q, k, v, cu, lens, scale=None, join=None):
    """(O, lse, weighted |v| per output, bound on the scores' fp32 error) for lists cu, lens;
    rows outside the groups are NaN."""
    n, Hq, D = q.shape
    H = k.shape[2]
    G = Hq // H
    scale = scale or 1 / math.sqrt(D)
    O = torch.full((n, Hq, D), float("nan"), dtype=torch.float64, device=q.device)
    lse = torch.full((n, Hq), float("nan"), dtype=torch.float64, device=q.device)
    mass = torch.zeros_like(O)
    ds = 0.0
    for j in range(len(cu) - 1):
        lo, hi, ln = cu[j], cu[j + 1], lens[j]
        for h in range(H):
            hs = slice(h * G, (h + 1) * G)
            qq, kk, vv = q[lo:hi, hs].double(), k[j, :ln, h].double(), v[j, :ln, h].double()
            if hi == lo:
                continue
            s = torch.einsum("igd,td->igt", qq, kk) * scale
            z = torch.logsumexp(s, -1) if ln else torch.full(s.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
            p = torch.exp(s - z[..., None]) if ln else s
            O[lo:hi, hs] = torch.einsum("igt,td->igd", p, vv)
            mass[lo:hi, hs] = torch.einsum("igt,td->igd", p, vv.abs())
            lse[lo:hi, hs] = z
            if ln:
                ds = max(ds, float(torch.einsum("igd,td->igt", qq.abs(), kk.abs()).max()) * scale * D * 2.0 ** -24)
    if join is not None:
        O2, lse2 = join[0].double(), join[1].double()
        L = torch.logaddexp(lse, lse2)
        w1 = torch.where(lse == -math.inf, torch.zeros_like(L), torch.exp(lse - L))
        w2 = torch.where(lse2 == -math.inf, torch.zeros_like(L), torch.exp(lse2 - L))
        O2 = torch.where(w2[..., None] > 0, O2, torch.zeros_like(O2))
        O = O * w1[..., None] + O2 * w2[..., None]
        mass = mass * w1[..., None] + O2.abs() * w2[..., None]
        lse = L
    return O, lse, mass, ds
