"""Cases of the operators around the attention: the per-head norm of queries and
keys with the position rotation in the same pass (forward and backward), and the
decode attention over prefixes that groups of sequences share.

A case is a dict of plain values; "op" names the operator:
  "qk"      kvpop.qk_norm_rope
  "qk_bwd"  kvpop.qk_norm_rope_bwd
  "prefix"  kvpop.prefix_attn
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 1.0e6


def qk_case(name, op, b, S, H, G, D, R, interleaved, packed, far):
    c = {"name": name, "op": op, "b": b, "S": S, "H": H, "G": G, "D": D, "R": R, "interleaved": interleaved,
         "packed": packed, "far": far}
    if not name:
        del c["name"]
    return c


def prefix_case(name, groups, lens, H, G, D, join):
    c = {"name": name, "op": "prefix", "groups": ",".join(map(str, groups)), "lens": ",".join(map(str, lens)), "H": H,
         "G": G, "D": D, "join": join}
    if not name:
        del c["name"]
    return c


def ints(text):
    return [int(x) for x in text.split(",")]


def listed():
    return [
        # one decode step of a small batch: two sequences far into their context, latency only
        qk_case("qk_decode_2", "qk", 2, 1, 8, 4, 128, 128, False, True, 131072),
        # one decode step of the 64-sequence decode workload
        qk_case("qk_decode_64", "qk", 64, 1, 8, 4, 128, 128, False, True, 131072),
        # odd everything: three short prompts, D = 64, half of the dims rotated in adjacent pairs, a chunk at an offset
        qk_case("qk_odd", "qk", 3, 1021, 2, 3, 64, 32, True, False, 50000),
        # the Qwen3-4B-like layer's prompt, q and k as views of the packed projection
        qk_case("qk_prefill_16k", "qk", 1, 16384, 8, 4, 128, 128, False, True, 0),
        # the long-context workload's prompt
        qk_case("qk_prefill_131k", "qk", 1, 131072, 8, 4, 128, 128, False, True, 0),
        # training on short odd sequences, D = 64, adjacent pairs
        qk_case("qk_bwd_odd", "qk_bwd", 3, 1021, 2, 3, 64, 32, True, False, 50000),
        # training on the Qwen3-4B-like layer: gradients into the packed projection's gradient
        qk_case("qk_bwd_16k", "qk_bwd", 1, 16384, 8, 4, 128, 128, False, True, 0),
        # two samples of one short prompt on a tiny model
        prefix_case("prefix_tiny", [2], [257], 1, 2, 64, False),
        # eight prompts of different lengths with ragged numbers of samples, joined with each sequence's own cache
        prefix_case("prefix_ragged_8", [8, 16, 1, 5, 12, 3, 8, 11], [8192, 1531, 4096, 63, 7000, 2049, 512, 5001], 8, 4, 128,
                    True),
        # 64 samples of one 16k prompt
        prefix_case("prefix_64x16k", [64], [16384], 8, 4, 128, True),
        # 16 samples of one document of the longest supported length
        prefix_case("prefix_16x131k", [16], [131072], 8, 4, 128, True),
        # two prompts with 256 samples each: as much arithmetic as memory traffic and more
        prefix_case("prefix_256x8k", [256, 256], [8192, 8000], 8, 4, 128, True),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["qk", "qk", "qk_bwd", "prefix", "prefix", "prefix"])
    D = rng.choice([64, 128])
    H = rng.randint(1, 8)
    if kind != "prefix":
        G = rng.randint(1, 8)
        R = rng.choice([D, D, D // 2, 16, 0])
        row = (G + 1) * H * D
        most = (131072 if kind == "qk" else 16384) * 40 * 128 // row  # no more values than the largest listed case
        T = log_int(rng, 1, min(most, 131072))
        b = rng.choice([1, 1, 2, 3, 5])
        if rng.random() < 0.25:
            b, S = min(T, 512), 1
        else:
            S = max(1, T // b)
        return qk_case("", kind, b, S, H, G, D, R, rng.random() < 0.4, rng.random() < 0.5, rng.choice([0, 1000, 131072, 1000000]))
    G = rng.choice([1, 2, 4, 8])
    m = rng.choice([1, 1, 2, 3, 6, 11])
    lens = [log_int(rng, 1, 131072 // m) for _ in range(m)]
    most = 64e9 / (4 * H * G * D * sum(lens))  # flop of the largest listed case
    groups = [log_int(rng, 1, max(1, min(256, int(most)))) for _ in range(m)]
    return prefix_case("", groups, lens, H, G, D, rng.random() < 0.7)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    H, G, D = case["H"], case["G"], case["D"]
    Hq = H * G
    if case["op"] == "prefix":
        groups, lens = ints(case["groups"]), ints(case["lens"])
        n, m, P = sum(groups), len(groups), max(lens)
        cu = [0]
        for g in groups:
            cu.append(cu[-1] + g)
        s = {"op": "prefix", "H": H, "G": G, "gmax": max(groups),
             "q": randn(n, Hq, D), "k": randn(m, P, H, D), "v": randn(m, P, H, D),
             "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"),
             "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "join": None}
        if case["join"]:
            # what a sequence's own cache of a few thousand keys gives: an average of values, and its log-sum-exp
            s["join"] = (randn(n, Hq, D, scale=0.05), randn(n, Hq, dtype=torch.float32, scale=0.3) + 8.0)
        return s
    b, S, R = case["b"], case["S"], case["R"]
    s = {"op": case["op"], "interleaved": case["interleaved"]}
    # a projection's output: heads of different sizes
    if case["packed"]:
        qkv = randn(b, S, (Hq + 2 * H) * D, scale=1.7)
        s["q"] = qkv[..., : Hq * D].view(b, S, Hq, D)
        s["k"] = qkv[..., Hq * D:(Hq + H) * D].view(b, S, H, D)
    else:
        s["q"] = randn(b, S, Hq, D, scale=1.7)
        s["k"] = randn(b, S, H, D, scale=0.6)
    s["wq"] = 1.0 + randn(D, dtype=torch.float32, scale=0.2)
    s["wk"] = 1.0 + randn(D, dtype=torch.float32, scale=0.2)
    s["inv_freq"] = None
    if R:
        s["inv_freq"] = (THETA ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)).float()
    s["pos"] = None
    if case["far"]:
        # single tokens: each sequence at a position of its own; prompts: chunks that begin anywhere
        start = torch.randint(0, case["far"], (b, 1), generator=gen, device="cuda", dtype=torch.int32)
        s["pos"] = start + torch.arange(S, device="cuda", dtype=torch.int32)
    if case["op"] == "qk_bwd":
        s["dq"] = randn(b, S, Hq, D, dtype=torch.float32, scale=0.02)
        s["dk"] = randn(b, S, H, D, dtype=torch.float32, scale=0.05)
        if case["packed"]:
            dqkv = torch.zeros(b, S, (Hq + 2 * H) * D, dtype=torch.bfloat16, device="cuda")
            s["dq_in"] = dqkv[..., : Hq * D].view(b, S, Hq, D)
            s["dk_in"] = dqkv[..., Hq * D:(Hq + H) * D].view(b, S, H, D)
        else:
            s["dq_in"] = torch.zeros(b, S, Hq, D, dtype=torch.bfloat16, device="cuda")
            s["dk_in"] = torch.zeros(b, S, H, D, dtype=torch.bfloat16, device="cuda")
        s["dwq"] = torch.zeros(D, dtype=torch.float32, device="cuda")
        s["dwk"] = torch.zeros(D, dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def angles(s):
    """cos and sin [b or 1, S, 1, R/2] in 32 bits, from angles in 64."""
    b, S = s["q"].shape[:2]
    pos = s["pos"] if s["pos"] is not None else torch.arange(S, device="cuda")[None]
    a = pos.double()[:, :, None, None] * s["inv_freq"].double()
    return a.cos().float(), a.sin().float()


def pairs(y, R, interleaved):
    """The two members of each rotated pair, each [..., R/2]."""
    if interleaved:
        return y[..., 0:R:2], y[..., 1:R:2]
    return y[..., : R // 2], y[..., R // 2: R]


def rotated(y, s, back):
    if s["inv_freq"] is None:
        return y
    R = 2 * s["inv_freq"].numel()
    cos, sin = angles(s)
    if back:
        sin = -sin
    a, c = pairs(y, R, s["interleaved"])
    z = torch.empty_like(y)
    za, zc = pairs(z, R, s["interleaved"])
    za.copy_(a * cos - c * sin)
    zc.copy_(c * cos + a * sin)
    z[..., R:] = y[..., R:]
    return z


def norm_rope(x, w, s):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return rotated(x * r * w, s, False).to(torch.bfloat16)


def norm_rope_grad(x, g, w, s):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    dy = rotated(g, s, True)
    dw = (dy * xh).sum((0, 1, 2))
    e = dy * w
    dx = r * (e - xh * (e * xh).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), dw


def prefix_plain(s):
    q, cu, lens, H, G, gmax = s["q"], s["cu"].long(), s["lens"].long(), s["H"], s["G"], s["gmax"]
    n, Hq, D = q.shape
    m, P = s["k"].shape[:2]
    # the groups' rows side by side, padded to the largest group: [m, H, gmax * G, D]
    idx = (cu[:-1, None] + torch.arange(gmax, device="cuda")).clamp(max=n - 1)
    qg = q[idx].float().view(m, gmax, H, G, D).permute(0, 2, 1, 3, 4).reshape(m, H, gmax * G, D)
    keep = (torch.arange(P, device="cuda") < lens[:, None])[:, None]  # [m, 1, P]
    sc = torch.matmul(qg, s["k"].float().permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    sc = sc.masked_fill(~keep[:, :, None], -math.inf)
    mx = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - mx)
    l = p.sum(-1, keepdim=True)
    v = s["v"].float().permute(0, 2, 1, 3).masked_fill(~keep[..., None], 0.0)
    o = torch.matmul(p, v) / l
    lse = (mx + torch.log(l))[..., 0]
    # back to one row a sequence
    i = torch.arange(n, device="cuda")
    gid = torch.searchsorted(cu, i, right=True) - 1
    off = i - cu[gid]
    o = o.view(m, H, gmax, G, D)[gid, :, off].reshape(n, Hq, D)
    lse = lse.view(m, H, gmax, G)[gid, :, off].reshape(n, Hq)
    if s["join"] is not None:
        o2, lse2 = s["join"]
        top = torch.maximum(lse, lse2)
        a, c = torch.exp(lse - top), torch.exp(lse2 - top)
        o = (o * a[..., None] + o2.float() * c[..., None]) / (a + c)[..., None]
        lse = top + torch.log(a + c)
    return o.to(torch.bfloat16), lse


def run(s):
    if own:
        from fixed_budget_kv_gb300 import kvpop
        if s["op"] == "qk":
            return kvpop.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], EPS, s["inv_freq"], pos=s["pos"],
                                      interleaved=s["interleaved"])
        if s["op"] == "qk_bwd":
            return kvpop.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["wq"], s["wk"], EPS, s["inv_freq"],
                                          pos=s["pos"], interleaved=s["interleaved"],
                                          out=(s["dq_in"], s["dk_in"], s["dwq"], s["dwk"]))
        return kvpop.prefix_attn(s["q"], s["k"], s["v"], cu=s["cu"], lens=s["lens"], join=s["join"])
    if s["op"] == "qk":
        return norm_rope(s["q"], s["wq"], s), norm_rope(s["k"], s["wk"], s)
    if s["op"] == "qk_bwd":
        dq, dwq = norm_rope_grad(s["q"], s["dq"], s["wq"], s)
        dk, dwk = norm_rope_grad(s["k"], s["dk"], s["wk"], s)
        s["dq_in"].copy_(dq)
        s["dk_in"].copy_(dk)
        s["dwq"].copy_(dwq)
        s["dwk"].copy_(dwk)
        return s["dq_in"], s["dk_in"], s["dwq"], s["dwk"]
    return prefix_plain(s)


def work(case):
    H, G, D = case["H"], case["G"], case["D"]
    Hq = H * G
    if case["op"] == "prefix":
        groups, lens = ints(case["groups"]), ints(case["lens"])
        n = sum(groups)
        rows = n * Hq * (2 * D * 2 + 4)  # q, O, lse
        if case["join"]:
            rows += n * Hq * (D * 2 + 4)
        return {"bytes": sum(lens) * H * D * 4 + rows + 4 * (2 * len(lens) + 1),
                "flops": 4 * Hq * D * sum(a * b for a, b in zip(groups, lens))}
    T = case["b"] * case["S"]
    values = T * (Hq + H) * D
    small = 4 * (2 * D + case["R"] // 2) + (4 * T if case["far"] else 0)
    if case["op"] == "qk":
        return {"bytes": 4 * values + small, "flops": 10 * values}
    return {"bytes": 8 * values + small + 8 * D, "flops": 20 * values}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def turns(s):
    """e^(i t f) for every position and frequency, complex, [b or 1, S, 1, R/2]."""
    S = s["q"].shape[1]
    t = torch.arange(S, device="cuda", dtype=torch.float64)[None] if s["pos"] is None else s["pos"].to(torch.float64)
    phase = torch.einsum("bs,f->bsf", t, s["inv_freq"].to(torch.float64))[:, :, None]
    return torch.polar(torch.ones_like(phase), phase)


def spin(y, s, conj):
    if s["inv_freq"] is None:
        return y
    R = 2 * s["inv_freq"].numel()
    u = turns(s)
    u = u.conj() if conj else u
    head, rest = y[..., :R], y[..., R:]
    if s["interleaved"]:
        z = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (R // 2, 2)).contiguous()) * u).flatten(-2)
    else:
        c = torch.complex(head[..., : R // 2].contiguous(), head[..., R // 2:].contiguous()) * u
        z = torch.cat([c.real, c.imag], -1)
    return torch.cat([z, rest], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prefix":
        H, G, D = case["H"], case["G"], case["D"]
        q, k, v = s["q"], s["k"], s["v"]
        o = torch.empty(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        at = 0
        for j, (g, length) in enumerate(zip(ints(case["groups"]), ints(case["lens"]))):
            for h in range(H):
                x = q[at:at + g, h * G:(h + 1) * G].double()
                logits = torch.einsum("igd,td->igt", x, k[j, :length, h].double()) / math.sqrt(D)
                z = torch.logsumexp(logits, -1)
                lse[at:at + g, h * G:(h + 1) * G] = z
                o[at:at + g, h * G:(h + 1) * G] = torch.einsum("igt,td->igd", (logits - z[..., None]).exp(),
                                                               v[j, :length, h].double())
            at += g
        if s["join"] is not None:
            o2, lse2 = s["join"][0].double(), s["join"][1].double()
            both = torch.logaddexp(lse, lse2)
            o = o * (lse - both).exp()[..., None] + o2 * (lse2 - both).exp()[..., None]
            lse = both
        return o, lse
    out = []
    for name in ("q", "k"):
        x, w = s[name].double(), s["w" + name].double()
        size = ((x ** 2).sum(-1, keepdim=True) / case["D"] + EPS).sqrt()
        if case["op"] == "qk":
            out.append(spin(w * (x / size), s, False))
            continue
        unit = x / size
        dy = spin(s["d" + name].double(), s, True)
        e = dy * w
        out.append((e - unit * ((e * unit).sum(-1, keepdim=True) / case["D"])) / size)
        out.append(torch.einsum("bshd,bshd->d", dy, unit))
    return tuple(out) if case["op"] == "qk" else (out[0], out[2], out[1], out[3])
