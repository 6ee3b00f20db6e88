"""The calls on a paged cache on the GPU against the 64-bit forms, alone and together
as a server would use them.

Tolerances.  O: half a bf16 step of the result (2^-8) plus the softmax weights'
rounding to bf16 (2^-8 of the weighted mean of |v|) plus the scores' fp32 error ds
(at most D roundings of 2^-24 of sum |q k|, which moves a weight by 2 ds relative)
and 2^-16 for the fp32 sums and exponentials.  LSE: ds plus 2^-20 relative.  Received
weight: ref64_paged.mass.  Appended and moved values, kept slots and lengths: equal."""
import math

import pytest
import torch

import ref64_paged as ref
from fixed_budget_kv_gb300 import kvpop

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    kvpop.device_status(reset=True)
    yield
    st, words = kvpop.device_status(reset=True)
    assert st == 0, f"device status {words}"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Held:
    """A cache with the pages of sequences of these lengths anywhere, and places of the table
    behind a sequence's last page that hold nothing of use."""

    def __init__(self, lens, H, page, D, seed, spare=2, dtype=torch.bfloat16):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        held = [-(-x // page) for x in lens]
        pages = sum(held) + spare
        order = torch.randperm(pages, generator=self.gen, device="cuda").to(torch.int32)
        self.table = torch.full((len(lens), max(max(held), 1) + 1), -77, dtype=torch.int32, device="cuda")
        a = 0
        for i, c in enumerate(held):
            self.table[i, :c] = order[a:a + c]
            a += c
        self.kp, self.vp = self.randn(pages, H, page, D), self.randn(pages, H, page, D)
        self.scores = self.randn(pages, H, page).float().exp()
        self.n, self.lens, self.lens_list = len(lens), i32(lens), list(lens)

    def randn(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda").bfloat16()

    def used(self):
        """Whether a place of the cache is a slot of a sequence: [pages, H, page]."""
        on = torch.zeros(self.kp.shape[:3], dtype=torch.bool, device="cuda")
        for i, length in enumerate(self.lens_list):
            for h in range(on.shape[1] if length else 0):
                ref.put(on, self.table, i, h, torch.arange(length).cuda(), True)
        return on


def sums(chunks):
    cu = [0]
    for c in chunks:
        cu.append(cu[-1] + c)
    return cu


def check_attn(O, lse, q, c, cu, scale=None):
    rO, rl, mass, ds = ref.attn(q, c.kp, c.vp, c.table, c.lens_list, cu, scale)
    on = slice(cu[0], cu[-1])
    O, lse, rO, rl, mass = O[on].double(), lse[on].double(), rO[on], rl[on], mass[on]
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty) and (O[empty] == 0).all()
    assert ((lse - rl).abs()[~empty] <= ds + 2.0 ** -20 * (1 + rl.abs()[~empty])).all(), float((lse - rl).abs()[~empty].max())
    bad = ~((O - rO).abs() <= 2.0 ** -8 * rO.abs() + (2.0 ** -8 + 2 * ds + 2.0 ** -16) * mass)
    assert not bad.any(), f"O: {int(bad.sum())} off, worst {float((O - rO).abs().max())}"


def check_mass(got, before, q, lse, c, cu, decay, scale=None):
    want, bound = ref.mass(q, lse, c.kp, before, c.table, c.lens_list, cu, decay, scale)
    assert torch.equal(got[~c.used()], before[~c.used()])
    off = (got.double() - want).abs() - bound
    assert (off <= 0).all(), f"{int((off > 0).sum())} off, worst by {float(off.max())}"


CASES = [
    # chunks, lens, H, G, D, page
    ([1], [1], 1, 1, 64, 16),                                   # one row, one slot
    ([1], [130], 1, 1, 128, 16),
    ([1, 1], [257, 90], 1, 2, 64, 16),
    ([2], [2], 1, 2, 64, 32),                                   # a prompt of two
    ([7], [128], 2, 4, 128, 64),
    ([128], [128], 2, 4, 128, 128),                             # a whole prompt of whole tiles
    ([127, 1, 64], [127, 500, 300], 2, 4, 128, 32),             # prompts and a decode row
    ([5, 0, 2, 9], [40, 0, 0, 3], 2, 4, 128, 16),               # no rows; no slots; more rows than slots
    ([33], [700], 2, 4, 128, 256),                              # one row more than 128 rows of a head
    ([64], [1000], 2, 4, 128, 64),
    ([65, 1], [513, 2], 1, 4, 64, 16),                          # one row more than 256
    ([300], [900], 1, 8, 64, 64),
    ([90], [400], 1, 16, 128, 32),
    ([5], [333], 1, 64, 64, 128),
    ([3, 2], [200, 131], 2, 128, 128, 64),                      # one token a row tile
    ([260], [2600], 1, 1, 128, 512),                            # pages longer than a tile
    ([513], [513], 3, 2, 64, 65536),                            # a contiguous cache
    ([1] * 70, [(37 * i) % 400 for i in range(70)], 2, 4, 128, 16),   # more sequences than a warp has lanes
    ([(13 * i) % 7 for i in range(40)], [(91 * i) % 300 for i in range(40)], 2, 2, 64, 32),
    ([1], [20000], 8, 4, 128, 64),                              # one row over all SMs
    ([1] * 9, [1 + 900 * i for i in range(9)], 8, 8, 128, 64),
    ([700], [5000], 8, 4, 128, 64),
    ([600, 3, 0, 200], [900, 700, 40, 200], 2, 4, 128, 32),     # a long chunk beside others, for 512 rows a sequence
    ([530], [777], 2, 1, 128, 16),
    ([521], [2000], 1, 16, 64, 256),                            # sixteen tokens a row tile
    ([1030, 1100], [1030, 3001], 2, 1, 64, 64),
]


def name(c):
    return "T{}n{}L{}H{}G{}D{}p{}".format(sum(c[0]), len(c[0]), max(c[1]), *c[2:])


@pytest.mark.parametrize("case", CASES, ids=name)
def test_attention(case):
    chunks, lens, H, G, D, page = case
    c = Held(lens, H, page, D, seed=sum(lens))
    q, cu = c.randn(sum(chunks), H * G, D), sums(chunks)
    O, lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, None if max(chunks) == min(chunks) == 1 else i32(cu))
    check_attn(O, lse, q, c, cu)


@pytest.mark.parametrize("decay", [0.0, 0.75, 1.0])
@pytest.mark.parametrize("case", CASES, ids=name)
def test_received_weight(case, decay):
    chunks, lens, H, G, D, page = case
    c = Held(lens, H, page, D, seed=sum(lens) + 1)
    q, cu = c.randn(sum(chunks), H * G, D), sums(chunks)
    lse = ref.attn(q, c.kp, c.vp, c.table, c.lens_list, cu)[1].float()
    before = c.scores.clone()
    if decay == 0.0:
        c.scores.fill_(float("nan"))  # not read
        before = torch.where(c.used(), before, c.scores)
        got = kvpop.paged_mass(q, lse, c.kp, c.scores, c.table, c.lens, i32(cu), decay=decay)
        assert torch.equal(torch.isnan(got), torch.isnan(before))
        check_mass(got.nan_to_num(1.0), before.nan_to_num(1.0), q, lse, c, cu, decay)
        return
    got = kvpop.paged_mass(q, lse, c.kp, c.scores, c.table, c.lens, i32(cu), decay=decay)
    assert got.data_ptr() == c.scores.data_ptr()
    check_mass(got, before, q, lse, c, cu, decay)


@pytest.mark.parametrize("case", CASES, ids=name)
@pytest.mark.parametrize("packed", [False, True])
def test_append(case, packed):
    chunks, lens, H, G, D, page = case
    c = Held(lens, H, page, D, seed=sum(lens) + 2)
    T, cu = sum(chunks), sums(chunks)
    if packed:
        qkv = c.randn(T, (G + 2) * H * D)
        k, v = qkv[:, G * H * D:(G + 1) * H * D].view(T, H, D), qkv[:, (G + 1) * H * D:].view(T, H, D)
    else:
        k, v = c.randn(T, H, D), c.randn(T, H, D)
    want = [x.clone() for x in (c.kp, c.vp, c.scores)]
    for i, n in enumerate(lens):
        r0, r1 = cu[i], cu[i + 1]
        first = max(0, (r1 - r0) - n)  # rows that have no slot
        if r1 - r0 > first:
            t = torch.arange(n - (r1 - r0) + first, n)
            for h in range(H):
                ref.put(want[0], c.table, i, h, t.cuda(), k[r0 + first:r1, h])
                ref.put(want[1], c.table, i, h, t.cuda(), v[r0 + first:r1, h])
                ref.put(want[2], c.table, i, h, t.cuda(), 0.0)
    kvpop.paged_append(k, v, c.kp, c.vp, c.table, c.lens, i32(cu), scores=None if packed else c.scores)
    assert torch.equal(c.kp, want[0]) and torch.equal(c.vp, want[1])
    if not packed:
        assert torch.equal(c.scores, want[2])


@pytest.mark.parametrize("H,D", [(9, 128), (16, 128), (21, 128), (17, 64), (32, 64), (39, 64)])
def test_append_of_many_heads(H, D):
    """More heads than a warp takes at a time, and what is left over."""
    lens, cu = [100, 7, 260], [0, 30, 31, 171]
    c = Held(lens, H, 32, D, seed=H)
    qkv = c.randn(171, 3 * H * D)
    k, v = qkv[:, H * D:2 * H * D].view(171, H, D), qkv[:, 2 * H * D:].view(171, H, D)
    want = [x.clone() for x in (c.kp, c.vp, c.scores)]
    for i, n in enumerate(lens):
        t = torch.arange(n - (cu[i + 1] - cu[i]), n).cuda()
        for h in range(H):
            for x, y in zip(want, (k[cu[i]:cu[i + 1], h], v[cu[i]:cu[i + 1], h], 0.0)):
                ref.put(x, c.table, i, h, t, y)
    kvpop.paged_append(k, v, c.kp, c.vp, c.table, c.lens, i32(cu), scores=c.scores)
    assert all(torch.equal(a, b) for a, b in zip((c.kp, c.vp, c.scores), want))


EVICT = [
    # lens, H, page, D, (s, w, k)
    ([6], 1, 16, 64, (1, 1, 3)),
    ([300, 97, 0, 1, 100, 101], 2, 16, 64, (4, 32, 64)),
    ([1000, 999, 64], 3, 64, 128, (0, 0, 65)),                   # no sinks, no window
    ([1000, 40], 2, 32, 128, (5, 35, 0)),                        # sinks and window alone
    ([500], 2, 32, 128, (0, 0, 1)),
    ([500, 498], 2, 128, 64, (3, 490, 5)),                       # almost everything stays
    ([2049] * 3, 8, 64, 128, (16, 512, 1520)),
    ([4099, 1700, 2048, 2049, 3333] * 8, 8, 64, 128, (16, 512, 1520)),
    ([30000], 1, 64, 64, (7, 100, 9001)),
    ([131072], 2, 256, 64, (16, 1024, 3056)),
    ([300001], 1, 16, 64, (1, 2, 5000)),                         # a CTA's part that is not held in shared memory
]


@pytest.mark.parametrize("ties", ["", "many", "all"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: "n{}L{}H{}p{}D{}b{}".format(len(c[0]), max(c[0]), *c[1:]))
def test_eviction(case, ties):
    lens, H, page, D, budget = case
    c = Held(lens, H, page, D, seed=sum(lens))
    if ties == "many":
        c.scores = (c.scores * 4).round() / 4 * (torch.rand(c.scores.shape, generator=c.gen, device="cuda") > 0.5)
    elif ties == "all":
        c.scores.fill_(0.25)
    want = ref.evict(c.kp, c.vp, c.scores, c.table, lens, *budget)
    kept, new = kvpop.paged_evict(c.kp, c.vp, c.scores, c.table, c.lens, *budget)
    assert torch.equal(kept, want[3]) and torch.equal(new, want[4])
    for got, x in zip((c.kp, c.vp, c.scores), want):
        assert torch.equal(got, x)


def test_eviction_of_unusual_scores():
    """NaN, infinities, both zeros, negative values and denormals keep their order; the new
    lengths may replace the old ones."""
    lens, budget = [700, 650], (2, 9, 300)
    c = Held(lens, 2, 32, 64, seed=5)
    pick = torch.tensor([float("nan"), math.inf, -math.inf, 0.0, -0.0, -1.5, 1e-42, -1e-42, 3.4e38, -3.4e38, 1.0], device="cuda")
    c.scores = pick[torch.randint(0, 11, c.scores.shape, generator=c.gen, device="cuda")]
    want = ref.evict(c.kp, c.vp, c.scores, c.table, lens, *budget)
    kept, new = kvpop.paged_evict(c.kp, c.vp, c.scores, c.table, c.lens, *budget,
                                  out=(torch.empty(2, 2, 311, dtype=torch.int32, device="cuda"), c.lens))
    assert new.data_ptr() == c.lens.data_ptr()
    assert torch.equal(kept, want[3]) and torch.equal(c.lens, want[4])
    assert torch.equal(c.kp, want[0]) and torch.equal(c.vp, want[1])
    assert torch.equal(c.scores.nan_to_num(7.0), want[2].nan_to_num(7.0))


@pytest.mark.parametrize("D", [64, 128])
def test_scale_and_peaked_rows(D):
    c = Held([900, 400], 2, 64, D, seed=D)
    q = c.randn(70, 8, D) * 3
    cu = [0, 60, 70]
    for scale in (0.0, 0.5, 0.01):
        O, lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32(cu), scale=scale)
        check_attn(O, lse, q, c, cu, scale)
        before = c.scores.clone()
        check_mass(kvpop.paged_mass(q, lse, c.kp, c.scores, c.table, c.lens, i32(cu), scale=scale), before, q, lse, c, cu, 1.0,
                   scale)


def test_growing_scores():
    """Scores that grow along the slots move the running maximum at every tile."""
    c = Held([1500], 1, 64, 128, seed=1)
    q = c.randn(3, 4, 128)
    k = (q[0, 0].float() * torch.linspace(-1, 1, 1500, device="cuda")[:, None] * 0.8).bfloat16()
    ref.put(c.kp, c.table, 0, 0, torch.arange(1500).cuda(), k)
    O, lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32([0, 3]))
    check_attn(O, lse, q, c, [0, 3])


@pytest.mark.parametrize("chunk", [3, 40, 70, 150])
@pytest.mark.parametrize("D", [64, 128])
def test_weights_taken_again(D, chunk):
    """Scores that grow by about three at every tile in some rows of each warp and fall in others: the
    weights against the old reference are stored, then taken again and stored over, at every tile.  The same
    bits each time."""
    n = 1700
    c = Held([n], 2, 32, D, seed=chunk)
    u = c.randn(D).float()
    q = (u * torch.linspace(-1, 1, chunk * 8, device="cuda")[torch.randperm(chunk * 8, generator=c.gen, device="cuda")][:, None])
    q = q.bfloat16().view(chunk, 8, D)
    k = u * (torch.linspace(-1, 1, n, device="cuda")[:, None] * 20 * math.sqrt(D) / float(u @ u))
    for h in range(2):
        ref.put(c.kp, c.table, 0, h, torch.arange(n).cuda(), (k + 0.1 * c.randn(n, D).float()).bfloat16())
    O, lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32([0, chunk]))
    check_attn(O, lse, q, c, [0, chunk])
    for _ in range(20):
        again = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32([0, chunk]))
        assert torch.equal(again[0], O) and torch.equal(again[1], lse)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.0e38])
@pytest.mark.parametrize("chunks", [[1, 1], [40, 1], [70, 3]], ids=str)
def test_places_behind_a_length_are_never_used(bad, chunks):
    """Places behind the last slot, free pages and rows of other sequences may hold anything."""
    lens, cu = [131, 260], sums(chunks)
    c = Held(lens, 2, 64, 128, seed=2)
    q = c.randn(sum(chunks) + 3, 8, 128)
    used = c.used()
    want = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32(cu))
    s0 = c.scores.clone()
    m0 = kvpop.paged_mass(q, want[1], c.kp, s0.clone(), c.table, c.lens, i32(cu))
    for x in (c.kp, c.vp):
        x[~used] = bad
    q[cu[-1]:] = bad
    out = (torch.full_like(q, 5.0), torch.full((q.shape[0], 8), 5.0, device="cuda"))
    kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32(cu), out=out)
    assert torch.equal(out[0][:cu[-1]], want[0][:cu[-1]]) and torch.equal(out[1][:cu[-1]], want[1][:cu[-1]])
    assert (out[0][cu[-1]:] == 5).all() and (out[1][cu[-1]:] == 5).all()
    assert torch.equal(kvpop.paged_mass(q, want[1], c.kp, s0, c.table, c.lens, i32(cu)), m0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.0e38])
@pytest.mark.parametrize("scale", [0.0, 3.0])
@pytest.mark.parametrize("chunks", [[3, 1], [40, 29], [133, 150]], ids=str)
def test_rows_of_others_add_nothing(bad, scale, chunks):
    """Rows behind the sequences, which share tiles with theirs, and rows that saw nothing hold
    anything, at scales that would take a large product to infinity."""
    c = Held([300, 280], 2, 32, 64, seed=9)
    T, cu = sum(chunks), sums(chunks)
    q = 0.1 * c.randn(T + 40, 8, 64)
    lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32(cu), scale=scale)[1]
    lse[T:] = 0.0
    lse[1, 2] = -math.inf
    before = c.scores.clone()
    want = kvpop.paged_mass(q, lse, c.kp, c.scores.clone(), c.table, c.lens, i32(cu), scale=scale)
    check_mass(want, before, q, lse, c, cu, 1.0, scale)
    q[T:], lse[T:] = bad, bad
    q[1, 2] = bad
    assert torch.equal(kvpop.paged_mass(q, lse, c.kp, c.scores, c.table, c.lens, i32(cu), scale=scale), want)


def test_rows_outside_the_sequences():
    c = Held([300, 200], 2, 32, 64, seed=3)
    q, cu = c.randn(20, 4, 64), [3, 9, 15]
    O, lse = torch.full_like(q, 5.0), torch.full((20, 4), 5.0, device="cuda")
    kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32(cu), out=(O, lse))
    check_attn(O, lse, q, c, cu)
    for t in (O, lse):
        assert (t[:3] == 5).all() and (t[15:] == 5).all()
    before = c.scores.clone()
    check_mass(kvpop.paged_mass(q, lse, c.kp, c.scores, c.table, c.lens, i32(cu)), before, q, lse, c, cu, 1.0)
    k, v = c.randn(20, 2, 64), c.randn(20, 2, 64)
    kp, vp = c.kp.clone(), c.vp.clone()
    kvpop.paged_append(k, v, kp, vp, c.table, c.lens, i32(cu))
    want = c.kp.clone()
    for i in range(2):
        for h in range(2):
            ref.put(want, c.table, i, h, torch.arange(c.lens_list[i] - 6, c.lens_list[i]).cuda(), k[cu[i]:cu[i + 1], h])
    assert torch.equal(kp, want)


def test_nan_in_a_query_stays_in_its_row():
    c = Held([2000], 2, 64, 128, seed=11)
    for T in (1, 6, 90):
        q = c.randn(T, 8, 128)
        clean = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32([0, T]))
        q[T // 2, 3, 7] = float("nan")
        O, lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32([0, T]))
        assert torch.isnan(O[T // 2, 3]).all() and torch.isnan(lse[T // 2, 3])
        keep = torch.ones(T, 8, dtype=torch.bool, device="cuda")
        keep[T // 2, 3] = False
        assert torch.equal(O[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


def test_rows_that_saw_nothing_add_nothing():
    """lse = -inf: the row adds no weight, whatever it holds; a NaN row makes what it sees NaN."""
    c = Held([100], 1, 16, 64, seed=12)
    q = c.randn(4, 2, 64)
    lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32([0, 4]))[1]
    lse[1] = -math.inf
    q[1] = float("nan")
    before = c.scores.clone()
    q2 = q.clone()
    q2[1] = 0
    got = kvpop.paged_mass(q, lse, c.kp, c.scores, c.table, c.lens, i32([0, 4]))
    check_mass(got, before, q2, lse, c, [0, 4], 1.0)
    lse[3, 0] = float("nan")
    got = kvpop.paged_mass(q, lse, c.kp, c.scores, c.table, c.lens, i32([0, 4]))
    assert torch.isnan(ref.slots(got, c.table, 0, 0, 100)).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,chunk,rows", [(4, 40, [13]), (4, 40, [35]), (2, 150, [0, 77]), (1, 600, [100, 431]),
                                          (2, 300, [1, 140, 298]), (8, 400, [65])], ids=str)
def test_nan_of_a_row_stays_in_the_slots_it_sees(D, G, chunk, rows):
    """A NaN lse anywhere in a chunk, in both forms: the slots that its row sees are NaN, and those
    behind it and of other heads have the bits that they have without it."""
    H, lens = 2, [700, 1030]
    c = Held(lens, H, 32, D, seed=chunk + D)
    q, cu = c.randn(2 * chunk, H * G, D), i32([0, chunk, 2 * chunk])
    lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, cu)[1]
    want = kvpop.paged_mass(q, lse, c.kp, c.scores.clone(), c.table, c.lens, cu)
    nan_q = q.clone()
    for r in rows:  # of the second sequence and the first head's last query head
        nan_q[chunk + r, G - 1, 5] = float("nan")
    bad = kvpop.paged_attn(nan_q, c.kp, c.vp, c.table, c.lens, cu)[1]
    assert int(torch.isnan(bad).sum()) == len(rows)
    got = kvpop.paged_mass(nan_q, bad, c.kp, c.scores.clone(), c.table, c.lens, cu)
    same = kvpop.paged_mass(q, bad, c.kp, c.scores.clone(), c.table, c.lens, cu)
    assert torch.equal(torch.isnan(got), torch.isnan(same)) and torch.equal(got.nan_to_num(-1), same.nan_to_num(-1))
    last = lens[1] - chunk + max(rows)  # the last slot that one of them sees
    mine, clean = ref.slots(got, c.table, 1, 0, lens[1]), ref.slots(want, c.table, 1, 0, lens[1])
    assert torch.isnan(mine[:last + 1]).all()
    assert torch.equal(mine[last + 1:], clean[last + 1:])
    assert torch.equal(ref.slots(got, c.table, 1, 1, lens[1]), ref.slots(want, c.table, 1, 1, lens[1]))
    for h in range(H):
        assert torch.equal(ref.slots(got, c.table, 0, h, lens[0]), ref.slots(want, c.table, 0, h, lens[0]))


def test_lengths_and_rows_out_of_range_are_clamped():
    c = Held([150, 96], 1, 32, 64, seed=5)
    c.table[:, 3:] = -1
    table = c.table[:, :3].contiguous()
    q = c.randn(10, 2, 64)
    want = kvpop.paged_attn(q, c.kp, c.vp, table, i32([96, 0]), i32([0, 5, 10]))
    got = kvpop.paged_attn(q, c.kp, c.vp, table, i32([99999, -4]), i32([-7, 5, 4000]))
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert (want[0][5:] == 0).all() and (want[1][5:] == -math.inf).all()
    kept, new = kvpop.paged_evict(c.kp, c.vp, c.scores, table, i32([99999, -4]), 1, 2, 100)
    assert new.tolist() == [96, 0] and (kept[1] == -1).all()


def test_overlapping_sequences_are_reported():
    """Sequences that have more than T rows in all: the status says so and nothing is written."""
    c = Held([150, 150, 150], 1, 16, 64, seed=13)
    q, cu = c.randn(10, 2, 64), i32([0, 8, 2, 10])
    O, lse = torch.full_like(q, 3.0), torch.full((10, 2), 3.0, device="cuda")
    kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, cu, out=(O, lse))
    assert kvpop.device_status(reset=True)[0] == 1
    assert (O == 3.0).all() and (lse == 3.0).all()
    before = c.scores.clone()
    kvpop.paged_mass(q, lse, c.kp, c.scores, c.table, c.lens, cu)
    assert kvpop.device_status(reset=True)[0] == 1
    assert torch.equal(c.scores, before)


@pytest.mark.parametrize("bad", [-1, 1 << 30, 9])
def test_pages_that_do_not_exist_are_reported(bad):
    """Their slots read as zeros, and nothing is written to them."""
    c = Held([100, 60], 2, 32, 64, seed=14, spare=3)
    assert c.kp.shape[0] == 9
    q, cu = c.randn(12, 4, 64), [0, 8, 12]
    table = c.table.clone()
    table[0, 1] = bad
    z = Held([100, 60], 2, 32, 64, seed=14, spare=3)
    z.kp[z.table[0, 1].long()] = 0
    z.vp[z.table[0, 1].long()] = 0
    O, lse = kvpop.paged_attn(q, c.kp, c.vp, table, c.lens, i32(cu))
    assert kvpop.device_status(reset=True)[0] == 1
    check_attn(O, lse, q, z, cu)
    before = c.scores.clone()
    kvpop.paged_mass(q, lse, c.kp, c.scores, table, c.lens, i32(cu))
    assert kvpop.device_status(reset=True)[0] == 1
    gone = c.table[0, 1].long()
    assert torch.equal(c.scores[gone], before[gone])
    z.scores = before.clone()
    want, bound = ref.mass(q, lse, z.kp, before, z.table, z.lens_list, cu, 1.0)
    others = torch.arange(9, device="cuda") != gone
    assert ((c.scores.double() - want).abs() <= bound)[others].all()
    kp, vp, sc = c.kp.clone(), c.vp.clone(), c.scores.clone()
    table[0, 3], table[0, 1] = bad, c.table[0, 1]
    kvpop.paged_append(c.randn(12, 2, 64), c.randn(12, 2, 64), c.kp, c.vp, table, c.lens, i32(cu), scores=c.scores)
    assert kvpop.device_status(reset=True)[0] == 1
    for x, y in ((c.kp, kp), (c.vp, vp), (c.scores, sc)):
        there = c.table[0, :3].long()  # slots 92 .. 95 are new there, 96 .. 99 have no page
        assert torch.equal(x[there[:2]], y[there[:2]]) and torch.equal(x[there[2], :, :28], y[there[2], :, :28])
        assert not torch.equal(x[there[2], :, 28:], y[there[2], :, 28:])
    kept, new = kvpop.paged_evict(c.kp, c.vp, c.scores, table, c.lens, 2, 2, 30)
    assert kvpop.device_status(reset=True)[0] == 1
    assert new.tolist() == [34, 34] and (kept >= 0).all()


@pytest.mark.parametrize("lens,gone", [([300, 97], [(0, 0), (0, 5), (1, 1)]), ([300, 97], [(0, 18), (1, 0), (1, 2)]),
                                       ([9000, 8500], [(0, 0), (0, 100), (0, 101), (0, 300), (1, 531)])], ids=str)
@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_eviction_where_pages_do_not_exist(lens, gone, bad):
    """Slots of a page that does not exist rank last, behind any score and by their place; nothing moves
    from or to them.  Sinks, slots between and the window; one CTA a head and a cluster of them."""
    H, page, s, w, k = 2, 16, 3, 20, 41
    c = Held(lens, H, page, 64, seed=len(gone) + lens[0])
    B = s + w + k
    few = 0.004 if lens[0] > 1000 else 0.1  # fewer slots with a finite score than stay: the ties of the others count
    c.scores = torch.where(torch.rand(c.scores.shape, generator=c.gen, device="cuda") < few, c.scores.log(), -math.inf)
    table = c.table.clone()
    for i, p in gone:
        table[i, p] = bad
    want = [x.clone() for x in (c.kp, c.vp, c.scores)]
    lists = torch.full((2, H, B), -1, dtype=torch.int32)
    for i, length in enumerate(lens):
        exists = [(i, t // page) not in gone for t in range(length)]
        for h in range(H):
            sc = [x if e else -math.inf for x, e in zip(ref.slots(c.scores, c.table, i, h, length).tolist(), exists)]
            best = sorted(range(s, length - w), key=lambda t: (-sc[t], t))[:k]
            stay = list(range(s)) + sorted(best) + list(range(length - w, length))
            lists[i, h] = torch.tensor(stay, dtype=torch.int32)
            moves = [(j, t) for j, t in enumerate(stay) if exists[j] and exists[t]]
            src = torch.tensor([t for _, t in moves], device="cuda")
            for x, old in zip(want, (c.kp, c.vp, c.scores)):
                ref.put(x, c.table, i, h, torch.tensor([j for j, _ in moves]).cuda(), ref.slots(old, c.table, i, h, length)[src])
    kept, new = kvpop.paged_evict(c.kp, c.vp, c.scores, table, c.lens, s, w, k)
    assert kvpop.device_status(reset=True)[0] == 1
    assert torch.equal(kept.cpu(), lists) and new.tolist() == [B, B]
    assert all(torch.equal(a, b) for a, b in zip((c.kp, c.vp, c.scores), want))


@pytest.mark.parametrize("width", [1, 40, 600, 8192])
def test_a_table_wider_than_the_sequences(width):
    """The same bits from every call whatever the table's width."""
    lens, cu = [900, 33, 2100, 512] * 9, i32(sums([3, 1, 40, 2] * 9))
    c = Held(lens, 8, 64, 64, seed=41)
    tables = [c.table, torch.cat([c.table, torch.full((36, width), 1 << 20, dtype=torch.int32, device="cuda")], 1)]
    q, k, v = c.randn(46 * 9, 16, 64), c.randn(46 * 9, 8, 64), c.randn(46 * 9, 8, 64)
    results = []
    for table in tables:
        kp, vp, scores = c.kp.clone(), c.vp.clone(), c.scores.clone()
        kvpop.paged_append(k, v, kp, vp, table, c.lens, cu, scores=scores)
        O, lse = kvpop.paged_attn(q, kp, vp, table, c.lens, cu)
        kvpop.paged_mass(q, lse, kp, scores, table, c.lens, cu)
        results.append([O, lse, kp, vp, scores.clone(), *kvpop.paged_evict(kp, vp, scores, table, c.lens, 4, 60, 200), scores])
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_few_heads_in_a_wide_table():
    """A cluster for a head that has a few slots."""
    c = Held([300, 97, 5], 1, 16, 64, seed=43)
    want = ref.evict(c.kp, c.vp, c.scores, c.table, c.lens_list, 4, 32, 64)
    table = torch.cat([c.table, torch.full((3, 8192), -5, dtype=torch.int32, device="cuda")], 1)
    kept, new = kvpop.paged_evict(c.kp, c.vp, c.scores, table, c.lens, 4, 32, 64)
    assert torch.equal(kept, want[3]) and torch.equal(new, want[4])
    assert all(torch.equal(a, b) for a, b in zip((c.kp, c.vp, c.scores), want))


def test_strided_pools():
    """K and V of several layers in one pool: pages that are apart."""
    lens, chunks = [200, 70, 129], [20, 1, 129]
    c = Held(lens, 2, 32, 128, seed=6)
    pages = c.kp.shape[0]
    pool = c.randn(pages, 3, 2, 2, 32, 128)
    kp, vp = pool[:, 1, 0], pool[:, 1, 1]
    kp.copy_(c.kp)
    vp.copy_(c.vp)
    q, cu = c.randn(150, 8, 128), sums(chunks)
    k, v = c.randn(150, 2, 128), c.randn(150, 2, 128)
    rest = pool.clone()
    for x, y in ((c.kp, c.vp), (kp, vp)):
        kvpop.paged_append(k, v, x, y, c.table, c.lens, i32(cu))
    want, got = (kvpop.paged_attn(q, x, y, c.table, c.lens, i32(cu)) for x, y in ((c.kp, c.vp), (kp, vp)))
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    s = c.scores.clone()
    kvpop.paged_mass(q, want[1], c.kp, c.scores, c.table, c.lens, i32(cu))
    kvpop.paged_mass(q, want[1], kp, s, c.table, c.lens, i32(cu))
    assert torch.equal(s, c.scores)
    a = kvpop.paged_evict(c.kp, c.vp, c.scores, c.table, c.lens, 2, 10, 60)
    b = kvpop.paged_evict(kp, vp, s, c.table, c.lens, 2, 10, 60)
    assert torch.equal(a[0], b[0]) and torch.equal(kp, c.kp) and torch.equal(vp, c.vp) and torch.equal(s, c.scores)
    keep = torch.ones(3, dtype=torch.bool)
    keep[1] = False
    assert torch.equal(pool[:, keep], rest[:, keep])


def test_one_page_of_any_stride():
    """A cache of one page, as a view whose stride over pages is a head's."""
    c = Held([50], 4, 64, 128, seed=15, spare=0)
    assert c.kp.shape[0] == 1
    q, k, v, cu = c.randn(7, 8, 128), c.randn(7, 4, 128), c.randn(7, 4, 128), i32([0, 7])
    odd = [x[0][:, None].clone().transpose(0, 1) for x in (c.kp, c.vp)]
    assert odd[0].is_contiguous() and odd[0].stride(0) == 64 * 128
    results = []
    for kp, vp, scores in ((c.kp, c.vp, c.scores.clone()), (*odd, c.scores.clone())):
        kvpop.paged_append(k, v, kp, vp, c.table, c.lens, cu, scores=scores)
        O, lse = kvpop.paged_attn(q, kp, vp, c.table, c.lens, cu)
        kvpop.paged_mass(q, lse, kp, scores, c.table, c.lens, cu)
        results.append([O, lse, *kvpop.paged_evict(kp, vp, scores, c.table, c.lens, 2, 9, 20), kp, vp, scores])
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_sequences_may_share_pages_they_read():
    lens = [300, 300, 300]
    c = Held([300], 2, 64, 128, seed=7)
    table = c.table.expand(3, -1).contiguous()
    q = c.randn(3, 8, 128)
    O, lse = kvpop.paged_attn(q, c.kp, c.vp, table, i32(lens))
    for i in range(3):
        one = kvpop.paged_attn(q[i:i + 1], c.kp, c.vp, c.table, c.lens)
        c1 = Held([300], 2, 64, 128, seed=7)
        check_attn(*one, q[i:i + 1], c1, [0, 1])
        assert torch.allclose(one[1], lse[i:i + 1], atol=1e-5)


def test_streams_graphs_and_repeats():
    """A side stream, and all calls captured in one graph, replayed with other lengths, rows and
    data: each replay equals the eager calls, bit for bit."""
    lens, cu0 = [600, 77, 300], [0, 20, 21, 66]
    c = Held([640] * 3, 2, 32, 128, seed=8)
    q, k, v = c.randn(66, 8, 128), c.randn(66, 2, 128), c.randn(66, 2, 128)
    ln, cu = i32(lens), i32(cu0)
    first = [x.clone() for x in (c.kp, c.vp, c.scores)]

    def step(kp, vp, scores, stream=None):
        kvpop.paged_append(k, v, kp, vp, c.table, ln, cu, scores=scores, stream=stream)
        O, lse = kvpop.paged_attn(q, kp, vp, c.table, ln, cu, stream=stream)
        kvpop.paged_mass(q, lse, kp, scores, c.table, ln, cu, decay=0.5, stream=stream)
        kept, new = kvpop.paged_evict(kp, vp, scores, c.table, ln, 3, 20, 100, stream=stream)
        return O, lse, kept, new

    def eager(stream=None):
        state = [x.clone() for x in first]
        return list(step(*state, stream=stream)) + state
    want = eager()
    side = torch.cuda.Stream()
    state = [x.clone() for x in first]
    side.wait_stream(torch.cuda.current_stream())
    got = list(step(*state, stream=side)) + state
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    state = [x.clone() for x in first]
    with torch.cuda.graph(g):
        out = list(step(*state))
    for lv, cv in ((lens, cu0), ([1, 600, 0], [0, 1, 66, 66]), ([128, 129, 640], [0, 0, 2, 60])):
        ln.copy_(i32(lv))
        cu.copy_(i32(cv))
        q.normal_()
        k.normal_()
        for x, y in zip(state, first):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        want = eager()
        rows = slice(cv[0], cv[-1])
        assert torch.equal(out[0][rows], want[0][rows]) and torch.equal(out[1][rows], want[1][rows])
        assert all(torch.equal(a, b) for a, b in zip(out[2:] + state, want[2:])), lv


def test_two_streams_at_once():
    c = Held([3000, 100], 4, 64, 128, seed=9)
    q, cu = c.randn(41, 16, 128), i32([0, 40, 41])
    want = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, cu)
    sc = kvpop.paged_mass(q, want[1], c.kp, c.scores.clone(), c.table, c.lens, cu)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs, weights = [], []
    for _ in range(8):
        for s in streams:
            outs.append(kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, cu, stream=s))
            with torch.cuda.stream(s):
                mine = c.scores.clone()
                weights.append(kvpop.paged_mass(q, outs[-1][1], c.kp, mine, c.table, c.lens, cu))
    torch.cuda.synchronize()
    assert all(torch.equal(O, want[0]) and torch.equal(lse, want[1]) for O, lse in outs)
    assert all(torch.equal(w, sc) for w in weights)


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements: its last pages are as good as the first."""
    pages, H, page, D = 2200, 8, 1024, 128
    kp, vp = (torch.zeros(pages, H, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c = Held([3000], H, page, D, seed=10, spare=0)
    last = torch.tensor([pages - 1, pages - 3, pages - 2], device="cuda")
    kp[last], vp[last] = c.kp[c.table[0, :3].long()], c.vp[c.table[0, :3].long()]
    c.kp, c.vp, c.table = kp, vp, last.to(torch.int32)[None].contiguous()
    c.scores = torch.rand(pages, H, page, device="cuda")
    q, cu = c.randn(5, 32, D), [0, 5]
    k, v = c.randn(5, H, D), c.randn(5, H, D)
    kvpop.paged_append(k, v, kp, vp, c.table, c.lens, i32(cu))
    for h in range(H):
        assert torch.equal(ref.slots(kp, c.table, 0, h, 3000)[-5:], k[:, h])
    O, lse = kvpop.paged_attn(q, kp, vp, c.table, c.lens, i32(cu))
    check_attn(O, lse, q, c, cu)
    before = c.scores.clone()
    check_mass(kvpop.paged_mass(q, lse, kp, c.scores, c.table, c.lens, i32(cu)), before, q, lse, c, cu, 1.0)
    rows = [ref.slots(kp, c.table, 0, h, 3000).clone() for h in range(H)]
    kept, _ = kvpop.paged_evict(kp, vp, c.scores, c.table, c.lens, 4, 100, 1000)
    for h in range(H):
        assert torch.equal(ref.slots(kp, c.table, 0, h, 1104), rows[h][kept[0, h].long()])


def test_long_context():
    """One row and an observation window over 131 072 slots; more than 2^15 keys in one sum."""
    for T, H, G, D in ((1, 1, 1, 64), (32, 2, 4, 128)):
        c = Held([131072], H, 64, D, seed=T)
        c.vp += 1  # a sum that does not cancel
        q, cu = c.randn(T, H * G, D), [0, T]
        O, lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32(cu))
        check_attn(O, lse, q, c, cu)
        before = c.scores.clone()
        check_mass(kvpop.paged_mass(q, lse, c.kp, c.scores, c.table, c.lens, i32(cu), decay=0.0), before, q, lse, c, cu, 0.0)


def test_binding_refusals():
    c = Held([100, 50], 2, 32, 64, seed=9)
    q, k = c.randn(2, 4, 64), c.randn(2, 2, 64)
    with pytest.raises(ValueError, match="bfloat16"):
        kvpop.paged_attn(q.float(), c.kp, c.vp, c.table, c.lens)
    with pytest.raises(ValueError, match="vp"):
        kvpop.paged_attn(q, c.kp, c.vp[1:], c.table, c.lens)
    with pytest.raises(ValueError, match="page must be contiguous"):
        kvpop.paged_attn(q, c.kp.transpose(1, 2), c.vp.transpose(1, 2), c.table, c.lens)
    with pytest.raises(ValueError, match="cu"):
        kvpop.paged_attn(c.randn(3, 4, 64), c.kp, c.vp, c.table, c.lens)
    with pytest.raises(ValueError, match="lens"):
        kvpop.paged_append(k, k, c.kp, c.vp, c.table, c.lens.long())
    with pytest.raises(ValueError, match="table"):
        kvpop.paged_append(k, k, c.kp, c.vp, c.table[:, :2], c.lens)
    with pytest.raises(ValueError, match="lse"):
        kvpop.paged_mass(q, torch.zeros(2, 3, device="cuda"), c.kp, c.scores, c.table, c.lens)
    with pytest.raises(ValueError, match="scores"):
        kvpop.paged_evict(c.kp, c.vp, c.scores[1:], c.table, c.lens, 1, 1, 1)
    with pytest.raises(ValueError, match="heads of a token"):
        kvpop.paged_append(c.randn(2, 64, 2).transpose(1, 2), k, c.kp, c.vp, c.table, c.lens)
    with pytest.raises(kvpop.KvpopError):
        kvpop.paged_attn(c.randn(2, 6, 64), c.kp, c.vp, c.table, c.lens)        # G = 3
    with pytest.raises(kvpop.KvpopError):
        kvpop.paged_evict(c.kp, c.vp, c.scores, c.table, c.lens, 0, 0, 0)


def test_serving_loop():
    """A prompt arrives in chunks beside sequences that decode: norm and rotation, append,
    attention joined with a shared prefix, received weight, eviction when a sequence has grown
    past its budget by a page.  Beside it a plain account of what each head holds."""
    H, G, D, page, s, w, kk = 2, 4, 128, 16, 2, 8, 22
    Hq, n, B = H * G, 3, 32
    gen = torch.Generator(device="cuda").manual_seed(20)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    f = (1.0e6 ** (-torch.arange(0, D, 2).double() / D)).float().cuda()
    wq, wk = 1 + 0.1 * randn(D), 1 + 0.1 * randn(D)
    prefix_k, prefix_v = randn(1, 70, H, D).bfloat16(), randn(1, 70, H, D).bfloat16()
    kp, vp = (torch.full((30, H, page, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    scores = torch.full((30, H, page), float("nan"), device="cuda")
    table = torch.full((n, 8), -1, dtype=torch.int32)
    free = list(range(30))
    lens, pos = [0] * n, [70] * n
    own = [[[] for _ in range(H)] for _ in range(n)]  # per head: (key, value, weight) of each slot
    for step in range(14):
        chunks = [1, 1, [17, 20, 1, 9, 30][step % 5]]
        cu = sums(chunks)
        T = cu[-1]
        for i in range(n):
            lens[i] += chunks[i]
            while sum(int(x) >= 0 for x in table[i]) * page < lens[i]:
                table[i, sum(int(x) >= 0 for x in table[i])] = free.pop()
        qkv = randn(T, 1, (Hq + 2 * H) * D).bfloat16()
        x, y = qkv[..., : Hq * D].view(T, 1, Hq, D), qkv[..., Hq * D:(Hq + H) * D].view(T, 1, H, D)
        v = qkv[:, 0, (Hq + H) * D:].view(T, H, D)
        p = i32([[pos[i] + r] for i in range(n) for r in range(chunks[i])])
        q, k = kvpop.qk_norm_rope(x, y, wq, wk, 1e-6, f, p)
        q, k = q[:, 0], k[:, 0]
        tb, ln, cud = table.cuda(), i32(lens), i32(cu)
        kvpop.paged_append(k, v, kp, vp, tb, ln, cud, scores=scores)
        mine = kvpop.paged_attn(q, kp, vp, tb, ln, cud)
        O, lse = kvpop.prefix_attn(q, prefix_k, prefix_v, join=mine)
        kvpop.paged_mass(q, lse, kp, scores, tb, ln, cud)
        for i in range(n):
            for h in range(H):
                held = own[i][h]
                held += [[k[r, h].double(), v[r, h].double(), 0.0] for r in range(cu[i], cu[i + 1])]
                pk, pv = prefix_k[0, :, h].double(), prefix_v[0, :, h].double()
                ka, va = torch.stack([e[0] for e in held]), torch.stack([e[1] for e in held])
                got = torch.zeros(len(held), dtype=torch.float64, device="cuda")
                for r in range(cu[i], cu[i + 1]):
                    m = len(held) - (cu[i + 1] - r) + 1
                    sc = (torch.cat([pk, ka[:m]]) @ q[r, h * G:(h + 1) * G].double().T) / math.sqrt(D)
                    z = torch.logsumexp(sc, 0)
                    assert float((lse[r, h * G:(h + 1) * G] - z).abs().max()) <= 2e-3
                    pr = torch.exp(sc - z)
                    o = pr.T @ torch.cat([pv, va[:m]])
                    assert float((O[r, h * G:(h + 1) * G].double() - o).abs().max()) <= 2e-2
                    got[:m] += pr[70:].sum(1)
                for e, gsum in zip(held, got.tolist()):
                    e[2] += gsum
                have = ref.slots(scores, tb, i, h, lens[i]).double()
                want = torch.tensor([e[2] for e in held], device="cuda", dtype=torch.float64)
                assert float((have - want).abs().max()) <= 1e-4 * (1 + float(want.max()))
        for i in range(n):
            pos[i] += chunks[i]
        if max(lens) > B + page:
            kept, new = kvpop.paged_evict(kp, vp, scores, tb, ln, s, w, kk)
            for i in range(n):
                for h in range(H):
                    stay = kept[i, h].tolist()[:min(lens[i], B)]
                    if lens[i] > B:
                        weights = [e[2] for e in own[i][h]]
                        mid = stay[s:s + kk]
                        assert stay[:s] == list(range(s)) and stay[s + kk:] == list(range(lens[i] - w, lens[i]))
                        gone = set(range(s, lens[i] - w)) - set(mid)
                        # the weights differ from the account's by rounding only
                        assert min(weights[t] for t in mid) >= max(weights[t] for t in gone) - 1e-4 * (1 + max(weights))
                    own[i][h] = [own[i][h][t] for t in stay]
                    ks = torch.stack([e[0] for e in own[i][h]])
                    assert torch.equal(ref.slots(kp, tb, i, h, len(stay)).double(), ks)
                lens[i] = min(lens[i], B)
                assert int(new[i]) == lens[i]
                used = -(-lens[i] // page)
                free += [int(t) for t in table[i, used:] if t >= 0]
                table[i, used:] = -1


def test_many_sequences():
    """More sequences than a warp takes at a time, whole windows of them without rows or without
    slots, and shares that begin in a later window."""
    chunks = [[0, 1, 2, 40][i % 4] if not 64 <= i < 140 else 0 for i in range(300)]
    lens = [(i * 37) % 400 if not 160 <= i < 230 else 0 for i in range(300)]
    c = Held(lens, 1, 16, 64, seed=12)
    cu = sums(chunks)
    q = c.randn(cu[-1], 4, 64)
    O, lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32(cu))
    check_attn(O, lse, q, c, cu)
    before = c.scores.clone()
    check_mass(kvpop.paged_mass(q, lse, c.kp, c.scores, c.table, c.lens, i32(cu), decay=0.5), before, q, lse, c, cu, 0.5)


def test_sums_of_more_than_one_run():
    """A CTA's tiles of one item beyond the 256 that it sums in one run: decode rows over so many
    slots, blocks of 256 rows, and received weight of so many query tiles."""
    c = Held([5_600_000], 1, 1024, 64, seed=21)
    c.vp += 1  # a sum that does not cancel
    q = c.randn(1, 1, 64)
    O, lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens)
    check_attn(O, lse, q, c, [0, 1])
    c = Held([33000], 152, 128, 64, seed=22)
    q = c.randn(64, 152 * 4, 64)
    O, lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32([0, 64]))
    check_attn(O, lse, q, c, [0, 64])
    c = Held([530], 152, 64, 64, seed=23)
    q = c.randn(530, 152 * 128, 64)
    lse = torch.full((530, 152 * 128), 6.5, device="cuda") + torch.randn(530, 152 * 128, generator=c.gen, device="cuda") * 0.1
    before = c.scores.clone()
    check_mass(kvpop.paged_mass(q, lse, c.kp, c.scores, c.table, c.lens, i32([0, 530])), before, q, lse, c, [0, 530], 1.0)


@pytest.mark.parametrize("D,G,S,page", [(128, 4, 900, 64), (64, 2, 515, 16)])
def test_against_the_contiguous_calls(D, G, S, page):
    """A whole prompt: the attention over the pages is the library's dense attention (its tolerances,
    2e-2 and 2e-3), and the weight that its keys receive is the future target with an empty window
    (the log of the same sum, 2e-2)."""
    H = 2
    c = Held([S], H, page, D, seed=D)
    q, k, v = c.randn(S, H * G, D), c.randn(S, H, D), c.randn(S, H, D)
    kvpop.paged_append(k, v, c.kp, c.vp, c.table, c.lens, i32([0, S]), scores=c.scores)
    O, lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32([0, S]))
    dO, dl = kvpop.attn_fwd(q[None], k[None], v[None])
    assert float((O.float() - dO[0].float()).abs().max()) <= 2e-2
    assert float((lse - dl[0].T).abs().max()) <= 2e-3
    kvpop.paged_mass(q, lse, c.kp, c.scores, c.table, c.lens, i32([0, S]))
    target = kvpop.future_target(q[None], k[None], dl, 0)
    for h in range(H):
        got = ref.slots(c.scores, c.table, 0, h, S).log()
        assert float((got - target[0, h]).abs().max()) <= 2e-2


@pytest.mark.parametrize("chunk,last", [(100, 10), (300, 32), (40, 1), (513, 300)])
def test_observation_window(chunk, last):
    """The attention of whole chunks, and the weight that only their last rows give."""
    lens = [chunk + 333, chunk, 700 + chunk]
    c = Held(lens, 2, 32, 128, seed=chunk)
    cu = sums([chunk] * 3)
    q = c.randn(3 * chunk, 8, 128)
    O, lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32(cu))
    check_attn(O, lse, q, c, cu)
    rows = torch.cat([torch.arange(x - last, x) for x in cu[1:]]).cuda()
    before = c.scores.clone()
    got = kvpop.paged_mass(q[rows], lse[rows], c.kp, c.scores, c.table, c.lens, i32(sums([last] * 3)), decay=0.5)
    check_mass(got, before, q[rows], lse[rows], c, sums([last] * 3), 0.5)


@pytest.mark.parametrize("chunk,length", [(64, 90), (64, 300), (70, 130), (128, 140), (129, 280), (129, 700)])
def test_short_items_in_turn(chunk, length):
    """Many items of one or a few tiles of rows for every SM, with tiles of keys that no row sees."""
    n = 150
    c = Held([length + i % 3 for i in range(n)], 4, 32, 64, seed=length)
    q, cu = c.randn(n * chunk, 16, 64), sums([chunk] * n)
    O, lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32(cu))
    check_attn(O, lse, q, c, cu)
    before = c.scores.clone()
    got = kvpop.paged_mass(q, lse, c.kp, c.scores, c.table, c.lens, i32(cu))
    check_mass(got, before, q, lse, c, cu, 1.0)
    for _ in range(20):
        assert torch.equal(kvpop.paged_mass(q, lse, c.kp, before.clone(), c.table, c.lens, i32(cu)), got)


def test_two_graphs_in_turn():
    """Two captured steps on the same cache, replayed in turn on two streams' order: each has its
    own workspace, and each replay equals the eager calls."""
    lens, cu = [700, 130], [0, 40, 41]
    c = Held(lens, 2, 32, 128, seed=31)
    q1, q2 = c.randn(41, 8, 128), c.randn(41, 8, 128)

    def step(q, scores):
        O, lse = kvpop.paged_attn(q, c.kp, c.vp, c.table, c.lens, i32_cu)
        return O, lse, kvpop.paged_mass(q, lse, c.kp, scores, c.table, c.lens, i32_cu, decay=0.0)
    i32_cu = i32(cu)
    want = [step(q, c.scores.clone()) for q in (q1, q2)]
    graphs, outs = [], []
    for q in (q1, q2):
        mine = c.scores.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(q, mine))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
        assert torch.equal(got[2][c.used()], w[2][c.used()])
