"""kvpop_prefix_attn on the GPU against the 64-bit form, and a decode loop and a
training step that use it and the norm-and-rotation pair with the library's own
attention.

Tolerances.  O: half a bf16 step of the result (2^-8) plus the softmax weights'
rounding to bf16 (2^-8 of the weighted mean of |v|) plus the scores' fp32 error ds
(at most D roundings of 2^-24 of sum |q k|, which moves a weight by 2 ds relative)
and 2^-16 for the fp32 sums and exponentials.  LSE: ds plus 2^-20 relative."""
import math

import numpy as np
import pytest
import torch

import oracle
import ref64
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


def make(groups, P, H, G, D, seed, join=False, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, m = sum(groups), len(groups)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    q, k, v = (randn(n, H * G, D) * scale).bfloat16(), randn(m, P, H, D).bfloat16(), randn(m, P, H, D).bfloat16()
    j = ((randn(n, H * G, D) * 0.1).bfloat16(), randn(n, H * G) + 5) if join else None
    return q, k, v, j


def check(O, lse, q, k, v, cu, lens, join=None, scale=None, rows=None):
    rO, rl, mass, ds = ref64.prefix_attn(q, k, v, cu, lens, scale, join)
    sel = slice(None) if rows is None else rows
    O, lse, rO, rl, mass = O[sel].double(), lse[sel].double(), rO[sel], rl[sel], mass[sel]
    ninf = rl == -math.inf
    assert torch.equal(lse == -math.inf, ninf)
    assert ((lse - rl).abs()[~ninf] <= ds + 2.0 ** -20 * (1 + rl.abs()[~ninf])).all(), float((lse - rl).abs()[~ninf].max())
    tol = 2.0 ** -8 * rO.abs() + (2.0 ** -8 + 2 * ds + 2.0 ** -16) * mass
    bad = ~((O - rO).abs() <= tol)
    assert not bad.any(), f"O: {int(bad.sum())} off, worst {float((O - rO).abs().max())}"


CASES = [
    # groups, lens, P, H, G, D, join
    ([1], [1], 1, 1, 1, 64, False),                              # one row, one key
    ([1], [130], 130, 1, 1, 128, True),
    ([2], [257], 257, 1, 2, 64, False),
    ([3], [128], 128, 2, 4, 128, False),                         # whole tiles
    ([5], [127], 300, 2, 4, 128, True),                          # a length that ends inside a tile
    ([5, 0, 2, 9], [0, 50, 129, 384], 400, 2, 4, 128, True),     # no keys, no sequences
    ([32], [700], 700, 2, 4, 128, False),                        # 128 rows
    ([33], [700], 701, 1, 4, 128, True),                         # 129 rows
    ([64], [1000], 1000, 2, 4, 128, False),                      # 256 rows
    ([65, 1], [513, 2], 513, 1, 4, 64, True),                    # 257 rows
    ([150], [900], 900, 1, 4, 128, True),                        # 600 rows: three blocks
    ([200], [300], 300, 3, 8, 64, False),
    ([9], [400], 400, 1, 16, 128, True),
    ([5], [333], 333, 1, 64, 64, False),
    ([3], [200], 200, 2, 128, 128, True),                        # one sequence a row tile
    ([4] * 37, list(range(0, 37 * 11, 11)), 400, 2, 4, 128, True),   # more groups than a warp has lanes
    ([1] * 90, [129] * 90, 140, 4, 2, 64, False),                # more work items than SMs
    ([16], [20000], 20000, 8, 4, 128, True),                     # a long prefix split over all SMs
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "n{}m{}P{}H{}G{}D{}j{}".format(sum(c[0]), len(c[0]), *c[2:6], int(c[6])))
def test_prefix_attention(case):
    groups, lens, P, H, G, D, join = case
    q, k, v, j = make(groups, P, H, G, D, seed=P + sum(groups), join=join)
    cu = [0] + np.cumsum(groups).tolist()
    O, lse = kvpop.prefix_attn(q, k, v, i32(cu), i32(lens), j)
    check(O, lse, q, k, v, cu, lens, j)


def test_many_groups():
    """More groups than a warp takes at a time, whole windows of them without work, and
    a share that begins in a later window."""
    groups, lens = [], []
    for j in range(300):
        groups.append([0, 1, 2, 5][j % 4] if not 64 <= j < 140 else (3 if j % 2 else 0))
        lens.append((j * 37) % 400 if not 64 <= j < 140 else (0 if j % 2 else 200))
    q, k, v, j2 = make(groups, 400, 1, 4, 64, seed=12, join=True)
    cu = [0] + np.cumsum(groups).tolist()
    O, lse = kvpop.prefix_attn(q, k, v, i32(cu), i32(lens), j2)
    check(O, lse, q, k, v, cu, lens, j2)


def test_overlapping_groups_are_reported():
    """Groups that cover more than n sequences: the status says so and nothing is written."""
    q, k, v, _ = make([5, 5], 150, 1, 2, 64, seed=13)
    k3, v3 = torch.cat([k, k[:1]]), torch.cat([v, v[:1]])
    O, lse = torch.full_like(q, 3.0), torch.full((10, 2), 3.0, device="cuda")
    kvpop.prefix_attn(q, k3, v3, i32([0, 8, 2, 10]), i32([150, 150, 150]), out=(O, lse))
    st, words = kvpop.device_status(reset=True)
    assert st == 1, words
    assert (O == 3.0).all() and (lse == 3.0).all()


@pytest.mark.parametrize("D", [64, 128])
def test_defaults_and_scale(D):
    """One prefix without cu and lens; a scale of the caller's; peaked and flat rows."""
    q, k, v, _ = make([10], 500, 2, 4, D, seed=D, scale=3.0)
    O, lse = kvpop.prefix_attn(q, k, v)
    check(O, lse, q, k, v, [0, 10], [500])
    O, lse = kvpop.prefix_attn(q, k, v, scale=0.5)
    check(O, lse, q, k, v, [0, 10], [500], scale=0.5)
    k.zero_()
    O, lse = kvpop.prefix_attn(q, k, v)
    check(O, lse, q, k, v, [0, 10], [500])


def test_growing_scores():
    """Scores that grow along the keys move the running maximum at every tile."""
    q, k, v, _ = make([3], 1500, 1, 4, 128, seed=1)
    k = (q[:1, :1].float() * torch.linspace(-1, 1, 1500, device="cuda")[None, :, None, None] * 0.8).bfloat16()
    k = k.reshape(1, 1500, 1, 128).contiguous()
    O, lse = kvpop.prefix_attn(q, k, v)
    check(O, lse, q, k, v, [0, 3], [1500])


@pytest.mark.parametrize("groups", [[6, 40], [70, 3]], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.0e38])
def test_keys_past_the_length_are_never_used(bad, groups):
    lens, P = [131, 260], 400
    q, k, v, j = make(groups, P, 2, 4, 128, seed=2, join=True)
    cu = [0, groups[0], sum(groups)]
    ref = kvpop.prefix_attn(q, k, v, i32(cu), i32(lens), j)
    for b, ln in enumerate(lens):
        k[b, ln:] = bad
        v[b, ln:] = bad
    got = kvpop.prefix_attn(q, k, v, i32(cu), i32(lens), j)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_join_edges():
    """lse2 = -inf: nothing joins, whatever O2 holds; no keys: the joined result alone;
    neither: zeros and -inf; a dominant side gives that side."""
    q, k, v, j = make([4, 4], 200, 1, 2, 64, seed=3, join=True)
    O2, l2 = j
    l2[0] = -math.inf
    O2[0] = float("nan")
    l2[4] = -math.inf
    O2[4] = float("inf")
    l2[1] = 500.0
    l2[2] = -500.0
    cu, lens = [0, 4, 8], [200, 0]
    O, lse = kvpop.prefix_attn(q, k, v, i32(cu), i32(lens), (O2, l2))
    check(O, lse, q, k, v, cu, lens, (O2, l2))
    assert torch.equal(O[5:], O2[5:]) and torch.equal(O[1], O2[1])
    assert (O[4] == 0).all() and (lse[4] == -math.inf).all()
    empty, el = kvpop.prefix_attn(q, k, v, i32(cu), i32([0, 0]), (O2, l2))
    check(empty, el, q, k, v, cu, [0, 0], (O2, l2))
    alone, al = kvpop.prefix_attn(q, k, v, i32(cu), i32(lens))
    assert torch.equal(alone[0], O[0]) and torch.equal(alone[2], O[2])
    assert (alone[4:] == 0).all() and (al[4:] == -math.inf).all()


def test_in_place_join_and_rows_outside():
    """The result may replace what it joins; rows outside the groups stay as they were."""
    q, k, v, j = make([12], 300, 2, 4, 128, seed=4, join=True)
    cu, lens = [3, 9], [300]
    ref = kvpop.prefix_attn(q, k, v, i32(cu), i32(lens), j)
    O, lse = j[0].clone(), j[1].clone()
    kvpop.prefix_attn(q, k, v, i32(cu), i32(lens), (O, lse), out=(O, lse))
    assert torch.equal(O[3:9], ref[0][3:9]) and torch.equal(lse[3:9], ref[1][3:9])
    for a, b in ((O, j[0]), (lse, j[1])):
        assert torch.equal(a[:3], b[:3]) and torch.equal(a[9:], b[9:])
    full = [torch.full((12, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((12, 8), 5.0, device="cuda")]
    kvpop.prefix_attn(q, k, v, i32(cu), i32(lens), None, out=tuple(full))
    assert all((t[:3] == 5).all() and (t[9:] == 5).all() for t in full)
    assert torch.isfinite(full[0].float()).all()


def test_moving_reference():
    """Scores whose maximum rises steeply between the tiles of a row, in both streams and for
    one row among many, with values near the end of their range."""
    q, k, v, _ = make([40], 1100, 1, 4, 128, seed=14)
    k *= 0.02
    for t, f in ((140, 3.0), (300, 6.0), (650, 9.0), (900, 12.0)):
        k[0, t, 0] = (q[7, 1].float() * f / 12.0).bfloat16()
    v *= 1e30
    O, lse = kvpop.prefix_attn(q, k, v, scale=0.5)
    check(O, lse, q, k, v, [0, 40], [1100], scale=0.5)


@pytest.mark.parametrize("G", [1, 64, 128])
def test_in_place_join_of_split_rows(G):
    """The same where several CTAs share a row and a row's outputs take several rounds."""
    q, k, v, j = make([4], 5000, 1, G, 128, seed=G, join=True)
    ref = kvpop.prefix_attn(q, k, v, None, None, j)
    check(*ref, q, k, v, [0, 4], [5000], j)
    O, lse = j[0].clone(), j[1].clone()
    kvpop.prefix_attn(q, k, v, None, None, (O, lse), out=(O, lse))
    assert torch.equal(O, ref[0]) and torch.equal(lse, ref[1])


def test_nan_in_a_query_stays_in_its_row():
    q, k, v, j = make([6], 2000, 2, 4, 128, seed=11, join=True)
    clean = kvpop.prefix_attn(q, k, v, None, None, j)
    q[2, 3, 7] = float("nan")
    for lens in ([2000], [100]):
        O, lse = kvpop.prefix_attn(q, k, v, None, i32(lens), j)
        assert torch.isnan(O[2, 3]).all() and torch.isnan(lse[2, 3])
        assert int(torch.isnan(O.float()).any(-1).sum()) == 1
    O, lse = kvpop.prefix_attn(q, k, v, None, None, j)
    keep = torch.ones(6, 8, dtype=torch.bool, device="cuda")
    keep[2, 3] = False
    assert torch.equal(O[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


def test_out_of_range_groups_and_lengths_are_clamped():
    q, k, v, _ = make([5, 5], 150, 1, 2, 64, seed=5)
    want = kvpop.prefix_attn(q, k, v, i32([0, 5, 10]), i32([150, 0]))
    got = kvpop.prefix_attn(q, k, v, i32([-7, 5, 4000]), i32([99999, -4]))
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_stream_graph_and_repeat():
    """Side stream, and a captured call replayed with other lengths and data: each replay
    equals the eager call, bit for bit."""
    groups, P = [20, 1, 45], 600
    q, k, v, j = make(groups, P, 2, 4, 128, seed=6, join=True)
    cu = i32([0, 20, 21, 66])
    lens = i32([600, 77, 300])
    ref = kvpop.prefix_attn(q, k, v, cu, lens, j)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kvpop.prefix_attn(q, k, v, cu, lens, j, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = kvpop.prefix_attn(q, k, v, cu, lens, j)
    for lv in ([600, 77, 300], [1, 600, 0], [128, 129, 590]):
        lens.copy_(i32(lv))
        q.normal_()
        g.replay()
        torch.cuda.synchronize()
        ref = kvpop.prefix_attn(q, k, v, cu, lens, j)
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1]), lv


def test_two_streams_at_once():
    q, k, v, j = make([40], 3000, 4, 4, 128, seed=7, join=True)
    ref = kvpop.prefix_attn(q, k, v, None, None, j)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        outs += [kvpop.prefix_attn(q, k, v, None, None, j, stream=s) for s in streams]
    torch.cuda.synchronize()
    for O, lse in outs:
        assert torch.equal(O, ref[0]) and torch.equal(lse, ref[1])


def test_offsets_past_32_bits():
    """Prefixes of more than 2^31 elements: the last one is right."""
    m, P, H, G, D = 5, 131072, 32, 2, 128
    k = torch.empty(m, P, H, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(m, P, H, D, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(8)
    for t in (k, v):
        t[-1, -1000:] = torch.randn(1000, H, D, generator=gen, device="cuda").bfloat16()
        t[-1, :-1000] = 0
    q = torch.randn(2, H * G, D, generator=gen, device="cuda").bfloat16()
    cu, lens = [0, 0, 0, 0, 0, 2], [P] * m
    O, lse = kvpop.prefix_attn(q, k, v, i32(cu), i32(lens))
    check(O, lse, q, k, v, cu, lens)


def test_binding_refusals():
    q, k, v, j = make([4], 100, 2, 2, 64, seed=9, join=True)
    with pytest.raises(ValueError, match="bfloat16"):
        kvpop.prefix_attn(q.float(), k, v)
    with pytest.raises(ValueError, match="pv"):
        kvpop.prefix_attn(q, k, v[:, :50].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        kvpop.prefix_attn(q, k[:, ::2], v[:, ::2])
    with pytest.raises(ValueError, match="cu"):
        kvpop.prefix_attn(q, k, v, cu=i32([0, 2, 4]))
    with pytest.raises(ValueError, match="lens"):
        kvpop.prefix_attn(q, k, v, lens=torch.tensor([100], device="cuda"))
    with pytest.raises(ValueError, match="lse2"):
        kvpop.prefix_attn(q, k, v, join=(j[0], j[1][:2].contiguous()))
    with pytest.raises(kvpop.KvpopError):
        kvpop.prefix_attn(q, torch.cat([k, k]), torch.cat([v, v]))           # two prefixes, no groups
    with pytest.raises(kvpop.KvpopError):
        kvpop.prefix_attn(q, k, v, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


def test_decode_over_a_shared_prompt():
    """Samples of two prompts decode together: norm and rotation, the step on each
    sequence's own cache (which holds all of its own tokens here), and the prompt joined.
    Against one 64-bit softmax over the rotated keys of prompt and own tokens, with the
    library's tolerances for O (2e-2) and LSE (2e-3)."""
    groups, lens, P = [3, 2], [150, 97], 150
    H, G, D, s, w, kk, steps = 2, 4, 128, 2, 8, 8, 12
    Hq, n, m = H * G, sum(groups), len(groups)
    gen = torch.Generator(device="cuda").manual_seed(10)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    wq, wk = 1 + 0.1 * randn(D), 1 + 0.1 * randn(D)
    f = (1.0e6 ** (-torch.arange(0, D, 2).double() / D)).float().cuda()
    prompt = randn(m, P, (Hq + 2 * H) * D).bfloat16()
    pq, pk = prompt[..., : Hq * D].view(m, P, Hq, D), prompt[..., Hq * D:(Hq + H) * D].view(m, P, H, D)
    pv = prompt[..., (Hq + H) * D:].reshape(m, P, H, D).contiguous()
    _, pk2 = kvpop.qk_norm_rope(pq, pk, wq, wk, 1e-6, f)
    cu, ln = i32([0, 3, 5]), i32(lens)
    gid = [0, 0, 0, 1, 1]
    start = i32([lens[j] for j in gid])[:, None]
    cache = kvpop.Cache(n, H, G, D, s, w, kk)
    own_k, own_v = [], []
    for i in range(steps):
        qkv = randn(n, 1, (Hq + 2 * H) * D).bfloat16()
        q, k = qkv[..., : Hq * D].view(n, 1, Hq, D), qkv[..., Hq * D:(Hq + H) * D].view(n, 1, H, D)
        v = qkv[..., (Hq + H) * D:].reshape(n, H, D).contiguous()
        pos = (start + i).contiguous()
        q2, k2 = kvpop.qk_norm_rope(q, k, wq, wk, 1e-6, f, pos)
        O2, l2, _ = cache.step(q2[:, 0], k2[:, 0], v, randn(n, H))
        O, lse = kvpop.prefix_attn(q2[:, 0], pk2, pv, cu, ln, (O2, l2))
        q64, kp = q2[:, 0].double(), pk2.double()
        for got, x, ww in ((q2, q, wq), (k2, k, wk)):
            z, y = ref64.norm_rope(x, ww, 1e-6, f, pos)
            assert ((got.double() - z).abs() <= 2.0 ** -8 * z.abs() + 2.0 ** -17 * y.abs().amax(-1, keepdim=True)).all()
        own_k.append(k2[:, 0].double())
        own_v.append(v.double())
        for r in range(n):
            j = gid[r]
            ka = torch.cat([kp[j, : lens[j]], torch.stack([t[r] for t in own_k])])
            va = torch.cat([pv[j, : lens[j]].double(), torch.stack([t[r] for t in own_v])])
            for hq in range(Hq):
                sc = (ka[:, hq // G] @ q64[r, hq]) / math.sqrt(D)
                assert abs(float(lse[r, hq]) - float(torch.logsumexp(sc, 0))) <= 2e-3
                o = torch.softmax(sc, 0) @ va[:, hq // G]
                assert float((O[r, hq].double() - o).abs().max()) <= 2e-2
    cache.close()


def test_training_step_through_norm_and_sparse_attention():
    """Projections -> norm and rotation -> mask, sparse attention -> its gradient -> the
    projections' and weights' gradient: the attention's part against the oracle (1e-2 of
    the largest entry, as its own tests have it), the norm's part against the 64-bit form
    on the gradients that the attention gave."""
    b, S, H, G, D, s, w, kk = 1, 200, 2, 4, 128, 4, 32, 40
    Hq = H * G
    gen = torch.Generator(device="cuda").manual_seed(12)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    qkv = randn(b, S, (Hq + 2 * H) * D).bfloat16()
    q, k = qkv[..., : Hq * D].view(b, S, Hq, D), qkv[..., Hq * D:(Hq + H) * D].view(b, S, H, D)
    v = qkv[..., (Hq + H) * D:].reshape(b, S, H, D).contiguous()
    wq, wk = 0.5 + 0.1 * randn(D), 0.5 + 0.1 * randn(D)
    f = (1.0e4 ** (-torch.arange(0, D, 2).double() / D)).float().cuda()
    prio, dO = randn(b, H, S), randn(b, S, Hq, D).bfloat16()
    q2, k2 = kvpop.qk_norm_rope(q, k, wq, wk, 1e-6, f)
    _, _, ev, lists = kvpop.mask(prio, s, w, kk)
    O, lse = kvpop.attn_fwd(q2, k2, v, 0.0, ev, lists, (s, w, kk))
    gq, gk, gv = kvpop.attn_bwd(q2, k2, v, O, dO, lse, ev, lists, (s, w, kk))
    got = kvpop.qk_norm_rope_bwd(q, k, gq, gk, wq, wk, 1e-6, f)
    r, tau, _ = oracle.mask(prio.cpu().numpy(), s, w, kk)
    rq, rk, _ = oracle.attn_bwd(q2.float().cpu().numpy(), k2.float().cpu().numpy(), v.float().cpu().numpy(),
                                dO.float().cpu().numpy(), 1 / math.sqrt(D), r, tau, s, w)
    for g, ref in ((gq, rq), (gk, rk)):
        assert np.abs(g.cpu().numpy() - ref).max() <= 1e-2 * np.abs(ref).max()
    for dx, dw, x, g, ww in ((got[0], got[2], q, gq, wq), (got[1], got[3], k, gk, wk)):
        rx, rw, size, bound = ref64.norm_rope_bwd(x, g, ww, 1e-6, f)
        assert ((dx.double() - rx).abs() <= 2.0 ** -8 * rx.abs() + 2.0 ** -17 * size).all()
        assert ((dw.double() - rw).abs() <= bound).all()


@pytest.mark.parametrize("byte", [0x01, 0x7f, 0xff])
def test_a_call_without_work_uses_nothing_of_the_workspace(byte):
    """A refused call gives its CTAs no work by the same path as the kernel's check of its shared
    memory, which no call can make fail.  Each CTA still says that it shares no item: the merge
    takes no rows from what the workspace held before."""
    groups, P, H, G, D = [6, 6], 900, 2, 4, 128
    q, k, v, j = make(groups, P, H, G, D, seed=15, join=True)
    k3, v3 = torch.cat([k, k[:1]]), torch.cat([v, v[:1]])
    ws = torch.full((kvpop.prefix_attn_workspace_size(12, 3, P, H * G, H, D),), byte, dtype=torch.uint8, device="cuda")
    O, lse = torch.full_like(q, 3.0), torch.full((12, H * G), 3.0, device="cuda")
    kvpop.prefix_attn(q, k3, v3, i32([0, 11, 1, 12]), i32([P] * 3), j, workspace=ws, out=(O, lse))
    assert kvpop.device_status(reset=True)[0] == 1
    assert (O == 3.0).all() and (lse == 3.0).all()
    got = kvpop.prefix_attn(q, k3, v3, i32([0, 5, 5, 12]), i32([P, 7, 100]), j, workspace=ws)
    check(*got, q, k3, v3, [0, 5, 5, 12], [P, 7, 100], j)


def test_overlapping_groups_leave_rows_without_keys_alone():
    """The refusal of overlapping groups covers the groups of length 0 among them, with and
    without a join, in place too; the next call is as good as ever."""
    q, k, v, j = make([5, 5, 4], 150, 1, 2, 64, seed=16, join=True)
    cu, lens = i32([0, 9, 2, 14]), i32([150, 0, 0])
    for join in (None, j):
        O, lse = torch.full_like(q, 3.0), torch.full((14, 2), 3.0, device="cuda")
        kvpop.prefix_attn(q, k, v, cu, lens, join, out=(O, lse))
        assert kvpop.device_status(reset=True)[0] == 1
        assert (O == 3.0).all() and (lse == 3.0).all()
    O, lse = j[0].clone(), j[1].clone()
    kvpop.prefix_attn(q, k, v, cu, lens, (O, lse), out=(O, lse))
    assert kvpop.device_status(reset=True)[0] == 1
    assert torch.equal(O, j[0]) and torch.equal(lse, j[1])
    check(*kvpop.prefix_attn(q, k, v, i32([0, 9, 9, 14]), lens, j), q, k, v, [0, 9, 9, 14], [150, 0, 0], j)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("D,G,groups,P", [(64, 1, [3], 100), (128, 4, [6], 1), (128, 4, [40], 120), (64, 2, [2] * 90, 300),
                                          (128, 128, [3] * 60, 400)], ids=str)
def test_nan_rows_without_a_join(D, G, groups, P, bad):
    """A row that becomes NaN reads nothing where there is nothing to join, whether a CTA has its
    item alone or shares it: a NaN or an infinity in a query, then in a key.  A single softmax of
    the same scores says which rows those are."""
    H, n, m = 2, sum(groups), len(groups)
    q, k, v, _ = make(groups, P, H, G, D, seed=21 + P)
    cu = [0] + np.cumsum(groups).tolist()
    clean = kvpop.prefix_attn(q, k, v, i32(cu))
    q2, k2 = q.clone(), k.clone()
    q2[n // 2, G, 5] = bad
    k2[m // 2, P - 1, 0, 3] = bad
    rows = torch.zeros(2, n, H * G, dtype=torch.bool, device="cuda")
    rows[0, n // 2, G] = True
    rows[1, cu[m // 2]:cu[m // 2 + 1], :G] = True
    for qq, kk, row in ((q2, k, rows[0]), (q, k2, rows[1])):
        O, lse = kvpop.prefix_attn(qq, kk, v, i32(cu))
        assert torch.equal(O[~row], clean[0][~row]) and torch.equal(lse[~row], clean[1][~row])
        if bad != bad:
            assert torch.isnan(O[row]).all() and torch.isnan(lse[row]).all()


def long_segments(P):
    """As many row blocks as SMs over a prefix of P keys, then a group of short ones: every CTA
    has about P keys of an item or two, and the last CTA many items after them.  All keys but the
    last of the long prefix score 0 and have values of 1, so the result is known: LSE within 2^-20
    of the terms' size as elsewhere and 2^-16 for the sum over the runs of keys, O within half a
    bf16 step and 2^-9 (see test_long_sums) of 1."""
    blocks, short, G, D = torch.cuda.get_device_properties(0).multi_processor_count, 40, 128, 64
    n, at = 2 * (blocks + short), 2 * blocks
    gen = torch.Generator(device="cuda").manual_seed(17)
    q = torch.randn(n, G, D, generator=gen, device="cuda").bfloat16()
    kl, vl = (torch.randn(2, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.empty(2, P, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[0], v[0] = 0, 1
    k[0, -1, 0], v[0, -1, 0], k[1, 0, 0], v[1, 0, 0] = kl[0], vl[0], kl[1], vl[1]
    O, lse = kvpop.prefix_attn(q, k, v, i32([0, at, n]), i32([P, 1]))
    assert kvpop.device_status(reset=False)[0] == 0
    s = torch.einsum("igd,jd->jig", q.double(), kl.double()) / math.sqrt(D)
    z = torch.logaddexp(s[0, :at], torch.tensor(math.log(P - 1), dtype=torch.float64, device="cuda"))
    last = torch.exp(s[0, :at] - z)[..., None]
    o = 1 - last + last * vl[0].double()
    mass = 1 - last + last * vl[0].double().abs()
    assert ((lse[:at].double() - z).abs() <= 2.0 ** -16 + 2.0 ** -20 * z.abs()).all()
    assert ((O[:at].double() - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -9 + 2.0 ** -8 * last) * mass).all()
    assert ((lse[at:].double() - s[1, at:]).abs() <= 2.0 ** -16 + 2.0 ** -20 * s[1, at:].abs()).all()
    assert torch.equal(O[at:], vl[1].expand(n - at, G, D))


def test_a_prefix_that_takes_longer_than_the_wait_limit():
    """A wait gives up after 2 s, and two of the waits last a segment: at 1.6 us a key tile of 256
    rows at D = 64 this prefix takes a CTA 2.5 s, in many segments (103 GB of keys and values)."""
    torch.cuda.empty_cache()
    long_segments(200_000_001)
    torch.cuda.empty_cache()


def test_short_groups_after_a_long_one():
    long_segments(100_001)


@pytest.mark.parametrize("D", [64, 128])
def test_long_sums(D):
    """Millions of equal weights in one CTA: the softmax weights are exactly 1, so O is the mean
    of the values, within half a bf16 step (2^-8) and what a sum of 2^15 products may lose where
    every one is cut off to the accumulator's 24 bits: 2^15 x 2^-23 of the sum so far, 2^-9 of
    the whole one.  (A single run of all keys came out 2.4% too small.)"""
    P, G, blocks = (1 << 22) + 37, 128, torch.cuda.get_device_properties(0).multi_processor_count + 1
    gen = torch.Generator(device="cuda").manual_seed(18)
    q = torch.randn(2 * blocks, G, D, generator=gen, device="cuda").bfloat16()
    k, v = (torch.empty(1, P, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k.zero_()
    mean = torch.zeros(D, dtype=torch.float64, device="cuda")
    for i in range(0, P, 1 << 18):
        part = v[0, i:i + (1 << 18), 0]
        part.copy_((0.5 + torch.rand(part.shape, generator=gen, device="cuda")) * (1 + torch.arange(D, device="cuda") / D))
        mean += part.double().sum(0) / P
    O, lse = kvpop.prefix_attn(q, k, v)
    assert ((O.double() - mean).abs() <= (2.0 ** -8 + 2.0 ** -9) * mean).all(), float(((O.double() - mean) / mean).abs().max())
    assert ((lse.double() - math.log(P)).abs() <= 2.0 ** -16).all()


@pytest.mark.parametrize("G,H,n,join", [(128, 1, 306, True), (128, 1, 306, False), (4, 160, 9, True), (32, 160, 3, False)],
                         ids=str)
def test_items_of_several_runs(G, H, n, join):
    """More items than SMs and a prefix of several runs of key tiles, with one row tile and with
    two: scores that fall, rise and fall again along the keys, so that the first, a middle or the
    last run of an item carries most of the weight; joined in place; the same bits again."""
    P, D = 70001, 64
    gen = torch.Generator(device="cuda").manual_seed(19 + G)
    q = torch.randn(n, H * G, D, generator=gen, device="cuda").bfloat16()
    k, v = (torch.randn(1, P, H, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    for i, (a, b) in enumerate(((100, 1100), (40000, 41000), (69000, 70001))):
        k[0, a:b] += 0.6 * q[2 * i % n, ::G][None, :, :]
    j = ((torch.randn(n, H * G, D, generator=gen, device="cuda") * 0.1).bfloat16(),
         torch.randn(n, H * G, generator=gen, device="cuda") + 10) if join else None
    ref = kvpop.prefix_attn(q, k, v, join=j)
    for lo in (0, n - 3):
        rows = slice(lo, lo + 3)
        jj = (j[0][rows], j[1][rows]) if join else None
        check(ref[0][rows], ref[1][rows], q[rows], k, v, [0, 3], [P], jj)
    out = (j[0].clone(), j[1].clone()) if join else (torch.empty_like(ref[0]), torch.empty_like(ref[1]))
    kvpop.prefix_attn(q, k, v, join=out if join else None, out=out)
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])


def test_nan_in_one_run_of_keys():
    """A NaN among the keys of one run makes the rows of its head NaN, as in a single softmax."""
    H, n, P, D = 160, 3, 70000, 64
    gen = torch.Generator(device="cuda").manual_seed(20)
    q = torch.randn(n, H, D, generator=gen, device="cuda").bfloat16()
    k, v = (torch.randn(1, P, H, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    clean = kvpop.prefix_attn(q, k, v)
    for h, t in ((3, 5), (77, 40000), (159, P - 1)):
        k[0, t, h, 1] = float("nan")
    O, lse = kvpop.prefix_attn(q, k, v)
    bad = torch.zeros(H, dtype=torch.bool, device="cuda")
    bad[[3, 77, 159]] = True
    assert torch.isnan(O[:, bad]).all() and torch.isnan(lse[:, bad]).all()
    assert torch.equal(O[:, ~bad], clean[0][:, ~bad]) and torch.equal(lse[:, ~bad], clean[1][:, ~bad])


@pytest.mark.parametrize("D,H,G,m,top", [(128, 8, 4, 3, 300), (64, 3, 1, 40, 9), (128, 1, 2, 256, 3), (64, 1, 4, 700, 2),
                                         (128, 5, 1, 257, 1), (64, 1, 128, 5, 7)], ids=str)
def test_rows_without_keys(D, H, G, m, top):
    """Groups of length 0 of all sizes, by themselves and between groups with keys, over several
    windows of groups, joined in place and not; rows outside the groups stay as they were."""
    rng = np.random.default_rng(m)
    for keys in (0.0, 0.3):
        groups = rng.integers(0, top + 1, m)
        groups[m // 2] = top
        lens = np.where(rng.random(m) < keys, 33, 0)
        n = int(groups.sum()) + 5
        cu = (2 + np.concatenate([[0], np.cumsum(groups)])).tolist()
        q, k, v, j = make([n] + [0] * (m - 1), 40, H, G, D, seed=m, join=True)
        j[1][::7] = -math.inf
        j[0][::14] = float("nan")
        for join in (j, None):
            O, lse = torch.full_like(q, 3.0), torch.full((n, H * G), 3.0, device="cuda")
            kvpop.prefix_attn(q, k, v, i32(cu), i32(lens), join, out=(O, lse))
            check(O, lse, q, k, v, cu, lens.tolist(), join, rows=slice(2, n - 3))
            for t in (O, lse):
                assert (t[:2] == 3.0).all() and (t[n - 3:] == 3.0).all()
            if join:
                O2, l2 = j[0].clone(), j[1].clone()
                kvpop.prefix_attn(q, k, v, i32(cu), i32(lens), (O2, l2), out=(O2, l2))
                assert torch.equal(O2[2:n - 3], O[2:n - 3]) and torch.equal(l2[2:n - 3], lse[2:n - 3])


def test_many_rows_without_keys_take_no_longer_than_with_keys():
    """512 sequences without a prefix beside some with one, joined: at most four times the time
    of the same rows with 128 keys (as long as it; one CTA for all of a group took 39 times)."""
    q, k, v, j = make([512, 8], 200, 8, 4, 128, seed=23, join=True)
    cu = i32([0, 512, 520])

    def best(lens):
        out = (torch.empty_like(q), torch.empty(520, 32, device="cuda"))
        times = []
        for _ in range(10):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(5):
                kvpop.prefix_attn(q, k, v, cu, lens, j, out=out)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    assert best(i32([0, 200])) <= 4 * best(i32([128, 200]))
