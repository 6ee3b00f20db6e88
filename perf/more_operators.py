"""Cases of the operators on a paged key/value cache: appending new tokens, the attention
of chunks of new tokens over the pages, the attention weight that each held key
receives, and eviction from the pages by that weight.

A case is a dict of plain values; "op" names the operator:
  "append"  kvpop.paged_append
  "attn"    kvpop.paged_attn
  "mass"    kvpop.paged_mass
  "evict"   kvpop.paged_evict
"chunks" and "lens" give each sequence's new tokens and the slots it holds with them.
"""
import math

import torch

own = False

SIGMA = 1.5  # spread of the attention logits


def paged_case(name, op, chunks, lens, H, G, D, page, decay=1.0, packed=False, budget=""):
    c = {"name": name, "op": op, "chunks": ",".join(map(str, chunks)), "lens": ",".join(map(str, lens)), "H": H, "G": G,
         "D": D, "page": page}
    if op == "append":
        c["packed"] = packed
    if op == "mass":
        c["decay"] = decay
    if op == "evict":
        c["budget"] = budget
    if not name:
        del c["name"]
    return c


def ints(text):
    return [int(x) for x in text.split(",")]


def spread(n, lo, hi):
    """n lengths from lo to hi, evenly over their logarithm, in no order."""
    return [int(lo * (hi / lo) ** ((i * 37 % n) / max(n - 1, 1))) for i in range(n)]


def listed():
    return [
        # one decode step of 64 sequences: each sequence's new key and value into its last page
        paged_case("append_decode_64", "append", [1] * 64, spread(64, 500, 9001), 8, 4, 128, 64),
        # a whole prompt into the pages; keys come from the norm, values are a part of the packed projection
        paged_case("append_prompt_16k", "append", [16384], [16384], 8, 4, 128, 64, packed=True),
        # one decode step of two short sequences of a tiny model: latency only
        paged_case("attn_decode_tiny", "attn", [1, 1], [257, 90], 1, 2, 64, 16),
        # one decode step of 64 sequences at very different lengths
        paged_case("attn_decode_64", "attn", [1] * 64, spread(64, 500, 16001), 8, 4, 128, 64),
        # a mixed step of continuous batching: odd chunks of prompts and decode rows together
        paged_case("attn_mixed_12", "attn", [1, 517, 1, 1, 1300, 33, 1, 1, 255, 1, 4, 1],
                   [8000, 517, 1531, 4099, 9001, 2080, 63, 7001, 3001, 512, 700, 12001], 8, 4, 128, 32),
        # a chunk of a long prompt, late in it: as much arithmetic as a step can have
        paged_case("attn_chunk_4k_of_32k", "attn", [4096], [32768], 8, 4, 128, 128),
        # weights of one decode step, faded a little at each
        paged_case("mass_decode_64", "mass", [1] * 64, spread(64, 500, 16001), 8, 4, 128, 64, decay=0.98),
        # the last 32 tokens of a document of the longest supported length look back over it
        paged_case("mass_window_32_of_131k", "mass", [32], [131072], 8, 4, 128, 64, decay=0.0),
        # weights of a whole chunk of a long prompt
        paged_case("mass_chunk_4k_of_32k", "mass", [4096], [32768], 8, 4, 128, 128),
        # two short sequences of a tiny model, D = 64
        paged_case("evict_tiny", "evict", [1, 1], [300, 97], 1, 2, 64, 16, budget="4,32,64"),
        # 64 sequences, some over the decode workload's budget by a page or a few, some not yet
        paged_case("evict_64", "evict", [1] * 64, spread(64, 1700, 4099), 8, 4, 128, 64, budget="16,512,1520"),
        # a document of the longest supported length cut down to the long-context budget
        paged_case("evict_131k", "evict", [1], [131072], 8, 4, 128, 64, budget="16,1024,3056"),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "mass", "mass", "mass", "evict", "evict"])
    D = rng.choice([64, 128])
    H = rng.randint(1, 8)
    G = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    n = rng.choice([1, 1, 2, 3, 7, 16, 48])
    lens = [log_int(rng, 1, 131072 // n) for _ in range(n)]
    budget = ""
    if op == "evict":
        B = log_int(rng, 8, 4096)
        s, w = rng.randint(0, min(16, B // 4)), rng.randint(0, B // 2)
        budget = "%d,%d,%d" % (s, w, B - s - w)
    if rng.random() < 0.4 or op == "evict":
        chunks = [1] * n
    else:
        # no more (row, slot) pairs than the largest listed case, padded rows and slots counted too
        most = 4096 * 32768 * 4 * 8 * 128 // (n * max(lens) * G * H * D)
        chunks = [log_int(rng, 1, max(1, min(x, most, 16384 // n))) if rng.random() < 0.7 else 1 for x in lens]
    return paged_case("", op, chunks, lens, H, G, D, page, decay=rng.choice([0.0, 1.0, 0.9]), packed=rng.random() < 0.5,
                      budget=budget)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    H, G, D, page = case["H"], case["G"], case["D"], case["page"]
    chunks, lens = ints(case["chunks"]), ints(case["lens"])
    n, T = len(lens), sum(chunks)
    held = [-(-x // page) for x in lens]
    pages = sum(held) + 3  # a few pages are free
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    # a sequence's pages lie anywhere; places behind its last page hold nothing of use
    at = torch.tensor([0] + held[:-1], device="cuda").cumsum(0)
    place = torch.arange(max(held), device="cuda")
    used = place < torch.tensor(held, device="cuda")[:, None]
    table = torch.where(used, order[(at[:, None] + place).clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    cu = torch.tensor([0] + chunks, dtype=torch.int32, device="cuda").cumsum(0).to(torch.int32)
    s = {"op": case["op"], "H": H, "G": G, "page": page, "cmax": max(chunks), "L": max(lens),
         "k": randn(pages, H, page, D), "v": randn(pages, H, page, D),
         "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "cu": None if max(chunks) == 1 else cu, "rows": cu}
    if case["op"] == "attn":
        s["scores"] = None
        s["q"] = randn(T, H * G, D, scale=SIGMA)
    elif case["op"] == "append":
        s["scores"] = randn(pages, H, page, dtype=torch.float32).exp()
        s["k_new"] = randn(T, H, D)
        s["v_new"] = randn(T, (G + 2) * H * D)[:, (G + 1) * H * D:].view(T, H, D) if case["packed"] else randn(T, H, D)
    elif case["op"] == "mass":
        # what the keys have received lately: as much as this call adds
        s["scores"] = randn(pages, H, page, dtype=torch.float32).exp() * (T * G / sum(lens))
        s["q"] = randn(T, H * G, D, scale=SIGMA)
        # the log-sum-exp of such logits over the slots that each row sees
        gid, off = rows_of(s, T)
        sees = (s["lens"][gid] - (cu[1:] - cu[:-1])[gid] + off + 1).float()
        s["lse"] = sees.log()[:, None] + SIGMA ** 2 / 2 + randn(T, H * G, dtype=torch.float32, scale=0.05)
        s["decay"] = case["decay"]
    else:
        # weights received so far: a few keys have most of it; slots that nothing has looked at yet have none, and tie
        s["scores"] = randn(pages, H, page, dtype=torch.float32, scale=2.0).exp()
        s["scores"] *= torch.rand(s["scores"].shape, generator=gen, device="cuda") > 0.05
        s["budget"] = ints(case["budget"])
        s["out"] = (torch.empty(n, H, sum(s["budget"]), dtype=torch.int32, device="cuda"),
                    torch.empty(n, dtype=torch.int32, device="cuda"))
    return s


def rows_of(s, T):
    """The sequence of each row and the row's place in it."""
    i = torch.arange(T, device="cuda")
    gid = torch.searchsorted(s["rows"].long(), i, right=True) - 1
    return gid, i - s["rows"].long()[gid]


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def slots_of(s):
    """Page and place of every slot up to the longest length: [n, L] and [L]."""
    t = torch.arange(s["L"], device="cuda")
    return s["table"].long()[:, t // s["page"]].clamp(min=0), t % s["page"]


def logits(s):
    """Rows padded to the longest chunk against slots padded to the longest length:
    [n, H, cmax * G, L] in 32 bits, -inf where a row does not see a slot."""
    q, cu, H, G, cmax = s["q"], s["rows"].long(), s["H"], s["G"], s["cmax"]
    T, Hq, D = q.shape
    n = cu.numel() - 1
    pg, at = slots_of(s)
    k = s["k"][pg, :, at].float()  # [n, L, H, D]
    r = torch.arange(cmax, device="cuda")
    idx = (cu[:-1, None] + r).clamp(max=T - 1)
    x = q[idx].float().view(n, cmax, H, G, D).permute(0, 2, 1, 3, 4).reshape(n, H, cmax * G, D)
    sc = torch.matmul(x, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    c = cu[1:] - cu[:-1]
    sees = (s["lens"].long() - c)[:, None] + r + 1  # [n, cmax]
    keep = torch.arange(s["L"], device="cuda") < sees[:, :, None]
    keep = (keep & (r < c[:, None])[:, :, None])[:, :, None].expand(n, cmax, G, s["L"]).reshape(n, 1, cmax * G, s["L"])
    return sc.masked_fill_(~keep, -math.inf), pg, at


def attn_plain(s):
    T, Hq, D = s["q"].shape
    n, H, G, cmax = s["lens"].numel(), s["H"], s["G"], s["cmax"]
    sc, pg, at = logits(s)
    mx = sc.amax(-1, keepdim=True)
    sc = sc.sub_(mx.clamp(min=-1e30)).exp_()
    l = sc.sum(-1, keepdim=True)
    held = (torch.arange(s["L"], device="cuda") < s["lens"][:, None])[:, :, None, None]
    v = s["v"][pg, :, at].float().masked_fill_(~held, 0.0)
    o = torch.matmul(sc, v.permute(0, 2, 1, 3)) / l
    lse = (mx + torch.log(l))[..., 0]
    gid, off = rows_of(s, T)
    o = o.view(n, H, cmax, G, D)[gid, :, off].reshape(T, Hq, D)
    return o.to(torch.bfloat16), lse.view(n, H, cmax, G)[gid, :, off].reshape(T, Hq)


def mass_plain(s):
    n, H, G, cmax, cu = s["lens"].numel(), s["H"], s["G"], s["cmax"], s["rows"].long()
    sc, pg, at = logits(s)
    idx = (cu[:-1, None] + torch.arange(cmax, device="cuda")).clamp(max=s["q"].shape[0] - 1)
    lse = s["lse"][idx].view(n, cmax, H, G).permute(0, 2, 1, 3).reshape(n, H, cmax * G, 1)
    got = sc.sub_(lse).exp_().sum(2)  # [n, H, L]
    # slots behind a length repeat the last one's update
    t = torch.minimum(torch.arange(s["L"], device="cuda"), s["lens"].long()[:, None] - 1)
    got = got.gather(2, t[:, None].expand(n, H, s["L"])).permute(0, 2, 1)
    pg, at = pg.gather(1, t), at[t]
    scores = s["scores"]
    scores[pg, :, at] = got + scores[pg, :, at] * s["decay"] if s["decay"] else got
    return scores


def append_plain(s):
    T = s["k_new"].shape[0]
    gid, off = rows_of(s, T)
    cu = s["rows"].long()
    t = s["lens"].long()[gid] - (cu[1:] - cu[:-1])[gid] + off
    pg, at = s["table"].long()[gid, t // s["page"]], t % s["page"]
    s["k"][pg, :, at] = s["k_new"]
    s["v"][pg, :, at] = s["v_new"]
    s["scores"][pg, :, at] = 0.0
    return s["k"], s["v"], s["scores"]


def evict_plain(s):
    sinks, w, k = s["budget"]
    B = sinks + w + k
    lens, L = s["lens"].long(), s["L"]
    pg, at = slots_of(s)
    sc = s["scores"][pg, :, at].permute(0, 2, 1)  # [n, H, L]
    n, H, _ = sc.shape
    t = torch.arange(L, device="cuda")
    free = (t >= sinks) & (t < lens[:, None] - w)  # may go
    over = lens > B
    # places in the order (score falling, slot rising) of the slots that may go
    order = torch.where(free[:, None], sc, -math.inf).sort(dim=-1, descending=True, stable=True).indices
    place = torch.empty_like(order).scatter_(2, order, t.expand(n, H, L))
    stays = ((t < lens[:, None]) & ~free)[:, None] | (free[:, None] & (place < k))
    stays = torch.where(over[:, None, None], stays, (t < lens[:, None])[:, None])
    # the kept slots first, in their order
    kept = torch.where(stays, t, L + 1).sort(-1).values[:, :, :B]
    if kept.shape[2] < B:
        kept = torch.cat([kept, kept.new_full((n, H, B - kept.shape[2]), L + 1)], 2)
    new = torch.minimum(lens, torch.full_like(lens, B))
    # places behind the new length repeat the last one's move
    j = torch.minimum(torch.arange(B, device="cuda"), new[:, None] - 1)  # [n, B]
    src = kept.gather(2, j[:, None].expand(n, H, B))
    seq, head = torch.arange(n, device="cuda")[:, None, None], torch.arange(H, device="cuda")[None, :, None]
    table, page = s["table"].long(), s["page"]
    p0, a0 = table[seq, src // page], src % page
    p1, a1 = table[seq, j[:, None] // page], j[:, None] % page
    for x in (s["k"], s["v"], s["scores"]):
        x[p1, head, a1] = x[p0, head, a0]
    s["out"][0].copy_(torch.where(torch.arange(B, device="cuda") < new[:, None, None], kept, -1))
    s["out"][1].copy_(new)
    return (s["k"], s["v"], s["scores"]) + s["out"]


def run(s):
    if own:
        from fixed_budget_kv_gb300 import kvpop
        if s["op"] == "attn":
            return kvpop.paged_attn(s["q"], s["k"], s["v"], s["table"], s["lens"], cu=s["cu"])
        if s["op"] == "mass":
            return kvpop.paged_mass(s["q"], s["lse"], s["k"], s["scores"], s["table"], s["lens"], cu=s["cu"],
                                    decay=s["decay"])
        if s["op"] == "append":
            kvpop.paged_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], cu=s["cu"],
                               scores=s["scores"])
            return s["k"], s["v"], s["scores"]
        kept, new = kvpop.paged_evict(s["k"], s["v"], s["scores"], s["table"], s["lens"], *s["budget"], out=s["out"])
        return s["k"], s["v"], s["scores"], kept, new
    return {"attn": attn_plain, "mass": mass_plain, "append": append_plain, "evict": evict_plain}[s["op"]](s)


def work(case):
    H, G, D, page = case["H"], case["G"], case["D"], case["page"]
    chunks, lens = ints(case["chunks"]), ints(case["lens"])
    T, Hq, slots = sum(chunks), H * G, sum(lens)
    pairs = sum(c * x - c * (c - 1) // 2 for c, x in zip(chunks, lens))
    small = 4 * (2 * len(lens) + 1) + 4 * sum(-(-x // page) for x in lens)
    if case["op"] == "append":
        return {"bytes": T * H * (8 * D + 4) + 4 * 3 * len(lens), "flops": 0}
    if case["op"] == "attn":
        return {"bytes": slots * H * D * 4 + T * Hq * (4 * D + 4) + small, "flops": 4 * Hq * D * pairs}
    if case["op"] == "mass":
        return {"bytes": slots * H * (2 * D + (8 if case["decay"] else 4)) + T * Hq * (2 * D + 4) + small,
                "flops": 2 * Hq * D * pairs}
    sinks, w, k = ints(case["budget"])
    B, total = sinks + w + k, small
    for x in lens:
        total += 4 * H * B  # the list of kept slots
        if x > B:
            # slots before the first that goes stay where they are
            first = sinks + (x - sinks - w + 1) / (x - B + 1) - 1
            total += H * ((B - first) * (8 * D + 8) + 4 * (x - sinks - w))
    return {"bytes": int(total), "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one sequence and head at a time
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    H, G, D, page, op = case["H"], case["G"], case["D"], case["page"], case["op"]
    chunks, lens = ints(case["chunks"]), ints(case["lens"])
    k, v, scores = s["k"], s["v"], s["scores"]

    def flat(x, i, h, length):
        """The slots of one sequence and head in a row."""
        return x[s["table"][i, :-(-length // page)].long(), h].flatten(0, 1)[:length]

    def put(x, i, h, at, values):
        t = torch.as_tensor(at, device="cuda")
        x[s["table"][i].long()[t // page], h, t % page] = values

    if op in ("attn", "mass"):
        q = s["q"]
        o = torch.empty(q.shape, dtype=torch.float64, device="cuda")
        z = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        acc = scores.double() if op == "mass" else None
        row = 0
        for i, (c, length) in enumerate(zip(chunks, lens)):
            last = length - c + torch.arange(c, device="cuda")  # the last slot that each row sees
            for h in range(H):
                key = flat(k, i, h, length).double()
                got = torch.zeros(length, dtype=torch.float64, device="cuda")
                for a in range(0, c, 1024):
                    b = min(c, a + 1024)
                    hidden = torch.arange(length, device="cuda")[None] > last[a:b, None]
                    x = q[row + a:row + b, h * G:(h + 1) * G].double()
                    lg = (torch.einsum("rgd,td->rgt", x, key) / math.sqrt(D)).masked_fill(hidden[:, None], -math.inf)
                    if op == "mass":
                        got += (lg - s["lse"][row + a:row + b, h * G:(h + 1) * G, None].double()).exp().sum((0, 1))
                        continue
                    lz = torch.logsumexp(lg, -1)
                    z[row + a:row + b, h * G:(h + 1) * G] = lz
                    o[row + a:row + b, h * G:(h + 1) * G] = torch.einsum("rgt,td->rgd", (lg - lz[..., None]).exp(),
                                                                         flat(v, i, h, length).double())
                if op == "mass":
                    old = flat(acc, i, h, length)
                    put(acc, i, h, torch.arange(length), got + case["decay"] * old)
            row += c
        return acc if op == "mass" else (o, z)
    if op == "append":
        row = 0
        for i, (c, length) in enumerate(zip(chunks, lens)):
            for h in range(H):
                for x, new in ((k, s["k_new"][row:row + c, h]), (v, s["v_new"][row:row + c, h]),
                               (scores, torch.zeros(c, device="cuda"))):
                    put(x, i, h, torch.arange(length - c, length), new)
            row += c
        return k, v, scores
    sinks, w, keep = ints(case["budget"])
    B = sinks + w + keep
    kept = torch.full((len(lens), H, B), -1, dtype=torch.int32)
    for i, length in enumerate(lens):
        for h in range(H):
            slots = list(range(length))
            if length > B:
                sc = flat(scores, i, h, length).tolist()
                best = sorted(range(sinks, length - w), key=lambda t: (-sc[t], t))[:keep]
                slots = slots[:sinks] + sorted(best) + slots[length - w:]
            kept[i, h, :len(slots)] = torch.tensor(slots, dtype=torch.int32)
            src = torch.tensor(slots, device="cuda")
            for x in (k, v, scores):
                put(x, i, h, torch.arange(len(slots)), flat(x, i, h, length)[src])
    return k, v, scores, kept.cuda(), torch.tensor([min(x, B) for x in lens], dtype=torch.int32, device="cuda")
