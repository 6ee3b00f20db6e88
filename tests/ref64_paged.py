"""Plain 64-bit forms of the operators on a paged cache (torch, any device), for the
tests: one sequence and head at a time, from lists cu and lens."""
import math

import torch


def slots(x, table, i, h, length):
    """The slots of sequence i and head h of a cache [pages, H, page, ...] in a row."""
    page = x.shape[2]
    return x[table[i, :-(-length // page)].long(), h].flatten(0, 1)[:length]


def put(x, table, i, h, t, values):
    page = x.shape[2]
    t = torch.as_tensor(t, device=x.device)
    x[table[i].long()[t // page], h, t % page] = values


def attn(q, kp, vp, table, lens, cu, scale=None):
    """(O, lse, weighted |v| per output, bound on the scores' fp32 error); rows of no
    sequence are NaN, rows that see nothing 0 and -inf."""
    T, Hq, D = q.shape
    H = kp.shape[1]
    G = Hq // H
    scale = scale or 1 / math.sqrt(D)
    O = torch.full((T, Hq, D), float("nan"), dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), float("nan"), dtype=torch.float64, device=q.device)
    mass = torch.zeros_like(O)
    ds = 0.0
    for i, length in enumerate(lens):
        lo, hi = cu[i], cu[i + 1]
        if hi == lo:
            continue
        sees = length - (hi - lo) + 1 + torch.arange(hi - lo, device=q.device)
        for h in range(H):
            hs = slice(h * G, (h + 1) * G)
            x, kk, vv = q[lo:hi, hs].double(), slots(kp, table, i, h, length).double(), slots(vp, table, i, h, length).double()
            s = torch.einsum("rgd,td->rgt", x, kk) * scale
            hidden = torch.arange(length, device=q.device) >= sees[:, None, None]
            s = s.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(s, -1) if length else torch.full(s.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
            p = torch.exp(s - z[..., None]).masked_fill(hidden, 0.0)
            O[lo:hi, hs] = torch.einsum("rgt,td->rgd", p, vv)
            mass[lo:hi, hs] = torch.einsum("rgt,td->rgd", p, vv.abs())
            lse[lo:hi, hs] = z
            if length:
                ds = max(ds, float(torch.einsum("rgd,td->rgt", x.abs(), kk.abs()).max()) * scale * D * 2.0 ** -24)
    return O, lse, mass, ds


def mass(q, lse, kp, scores, table, lens, cu, decay, scale=None):
    """(scores after, bound on the fp32 error of each).  A term exp(s - lse) is off by its
    scores' error ds (D roundings of 2^-24 of sum |q k|), by four roundings of 2^-24 of the
    exponent's parts in units of log 2, and by 2^-21 for the exponential; the sum of N terms
    and the old score by N + 2 roundings; each term may be flushed below 1e-37."""
    T, Hq, D = q.shape
    H = kp.shape[1]
    G = Hq // H
    scale = scale or 1 / math.sqrt(D)
    out, bound = scores.double(), torch.zeros_like(scores, dtype=torch.float64)
    for i, length in enumerate(lens):
        lo, hi = cu[i], cu[i + 1]
        if length == 0:
            continue
        last = length - (hi - lo) + torch.arange(hi - lo, device=q.device)
        for h in range(H):
            hs = slice(h * G, (h + 1) * G)
            x, kk, z = q[lo:hi, hs].double(), slots(kp, table, i, h, length).double(), lse[lo:hi, hs].double()[..., None]
            old = slots(out, table, i, h, length)
            s = torch.einsum("rgd,td->rgt", x, kk) * scale
            hidden = (torch.arange(length, device=q.device) > last[:, None, None]) | (z == -math.inf)
            w = torch.exp(s - z).masked_fill(hidden, 0.0)
            ds = torch.einsum("rgd,td->rgt", x.abs(), kk.abs()) * scale * D * 2.0 ** -24
            off = ds + 4 * 1.45 * 2.0 ** -24 * (s.abs() + z.abs()) + 2.0 ** -21
            n = (hi - lo) * G
            total = w.sum((0, 1)) + (decay * old if decay else 0.0)
            put(out, table, i, h, torch.arange(length), total)
            put(bound, table, i, h, torch.arange(length),
                (w * off.masked_fill(hidden, 0.0)).sum((0, 1)) + (n + 2) * 2.0 ** -24 * total.abs() + n * 1e-37)
    return out, bound


def evict(kp, vp, scores, table, lens, s, w, k):
    """(kp, vp, scores, kept, new_lens) after, new tensors."""
    kp, vp, scores = kp.clone(), vp.clone(), scores.clone()
    B, H = s + w + k, kp.shape[1]
    kept = torch.full((len(lens), H, B), -1, dtype=torch.int32)
    for i, length in enumerate(lens):
        for h in range(H):
            stay = list(range(length))
            if length > B:
                sc = [-math.inf if x != x else x for x in slots(scores, table, i, h, length).tolist()]
                best = sorted(range(s, length - w), key=lambda t: (-sc[t], t))[:k]
                stay = stay[:s] + sorted(best) + stay[length - w:]
            kept[i, h, :len(stay)] = torch.tensor(stay, dtype=torch.int32)
            src = torch.tensor(stay, dtype=torch.long, device=kp.device)
            for x in (kp, vp, scores):
                put(x, table, i, h, torch.arange(len(stay)), slots(x, table, i, h, length)[src])
    return kp, vp, scores, kept.to(kp.device), torch.tensor([min(x, B) for x in lens], dtype=torch.int32, device=kp.device)
