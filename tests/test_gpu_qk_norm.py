"""kvpop_qk_norm_rope and its gradient on the GPU against the 64-bit form.

Tolerances.  Outputs are rounded to bf16 once: half a step, 2^-8 of the value.
Before that, fp32: the sum of squares and the products carry a few dozen
roundings of 2^-24, the angles at most 2^-22 rad (an fp32 fraction of a turn and
sincospif), each relative to the row's largest terms -- 2^-17 of them covers both.
Weight gradients are fp32 sums in a tree whose longest path is below 512
additions, so 512 * 2^-24 of the sum of the terms' magnitudes, and 2^-20 of what
the terms turn back (ref64.norm_rope_bwd says why)."""
import pytest
import torch

import ref64
from fixed_budget_kv_gb300 import kvpop

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    kvpop.device_status(reset=True)
    yield
    st, words = kvpop.device_status(reset=True)
    assert st == 0, f"device status {words}"


def freqs(R, theta=1.0e6):
    if not R:
        return None
    return (theta ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().cuda()


def make(b, S, Hq, H, D, seed, packed=False, scale=1.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    if packed:
        qkv = (randn(b, S, (Hq + 2 * H) * D) * scale).bfloat16()
        q, k = qkv[..., : Hq * D].view(b, S, Hq, D), qkv[..., Hq * D:(Hq + H) * D].view(b, S, H, D)
    else:
        q, k = (randn(b, S, Hq, D) * scale).bfloat16(), (randn(b, S, H, D) * scale).bfloat16()
    return q, k, 1 + 0.2 * randn(D), 1 + 0.2 * randn(D), randn(b, S, Hq, D), randn(b, S, H, D)


def check_fwd(got, x, w, f, pos, inter, what):
    z, y = ref64.norm_rope(x, w, EPS, f, pos, inter)
    tol = 2.0 ** -8 * z.abs() + 2.0 ** -17 * y.abs().amax(-1, keepdim=True)
    bad = (got.double() - z).abs() > tol
    assert not bad.any() and torch.isfinite(got.float()).all(), f"{what}: {int(bad.sum())} off"


def check_bwd(dx, dw, x, g, w, f, pos, inter, what):
    rx, rw, size, bound = ref64.norm_rope_bwd(x, g, w, EPS, f, pos, inter)
    bad = (dx.double() - rx).abs() > 2.0 ** -8 * rx.abs() + 2.0 ** -17 * size
    assert not bad.any() and torch.isfinite(dx.float()).all(), f"{what}: dx {int(bad.sum())} off"
    if dw is not None:
        assert ((dw.double() - rw).abs() <= bound).all(), f"{what}: dw"


CASES = [
    # b, S, Hq, H, D, R, interleaved, packed, positions
    (1, 1, 8, 2, 128, 128, False, False, None),        # one token
    (64, 1, 32, 8, 128, 128, False, True, 131072),     # a decode step
    (7, 1, 5, 1, 64, 64, True, True, 1000),            # heads that do not fill a pass
    (1, 300, 32, 8, 128, 128, False, True, None),
    (3, 101, 6, 2, 64, 32, True, False, 50000),        # half of the dims, adjacent pairs
    (2, 77, 3, 3, 128, 64, False, True, 2000000000),   # half of the dims, halves; positions near 2^31
    (1, 130, 1, 1, 128, 16, False, False, None),
    (1, 50, 2, 1, 64, 16, True, False, 9),
    (2, 33, 4, 4, 64, 0, False, True, None),           # norm only
    (1, 5000, 4, 1, 128, 128, True, False, None),      # more tokens than warps
    (1, 3, 130, 65, 64, 64, False, False, None),       # many heads
]


def ids(c):
    return "b{}S{}Hq{}H{}D{}R{}i{}p{}@{}".format(*(int(x) if isinstance(x, bool) else x for x in c))


def positions(b, S, start):
    if start is None:
        return None
    base = torch.arange(b, device="cuda", dtype=torch.int32)[:, None] * 7 + start
    return (base + torch.arange(S, device="cuda", dtype=torch.int32)).contiguous()


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward_and_backward(case):
    b, S, Hq, H, D, R, inter, packed, start = case
    q, k, wq, wk, gq, gk = make(b, S, Hq, H, D, seed=sum(case[:6]), packed=packed)
    f, pos = freqs(R), positions(b, S, start)
    qo, ko = kvpop.qk_norm_rope(q, k, wq, wk, EPS, f, pos, inter)
    check_fwd(qo, q, wq, f, pos, inter, "q")
    check_fwd(ko, k, wk, f, pos, inter, "k")
    dq, dk, dwq, dwk = kvpop.qk_norm_rope_bwd(q, k, gq, gk, wq, wk, EPS, f, pos, inter)
    check_bwd(dq, dwq, q, gq, wq, f, pos, inter, "q")
    check_bwd(dk, dwk, k, gk, wk, f, pos, inter, "k")


def test_no_weights_and_no_weight_gradients():
    q, k, _, _, gq, gk = make(2, 40, 4, 2, 128, seed=5)
    f = freqs(128)
    qo, ko = kvpop.qk_norm_rope(q, k, None, None, EPS, f)
    check_fwd(qo, q, None, f, None, False, "q")
    check_fwd(ko, k, None, f, None, False, "k")
    out = (torch.empty_like(q), torch.empty_like(k), None, None)
    dq, dk, a, b = kvpop.qk_norm_rope_bwd(q, k, gq, gk, None, None, EPS, f, out=out)
    assert a is None and b is None
    check_bwd(dq, None, q, gq, None, f, None, False, "q")
    check_bwd(dk, None, k, gk, None, f, None, False, "k")


def test_zero_rows_and_large_values():
    """A row of zeros stays zeros (eps > 0) with a finite gradient; rows near the bf16
    range's ends are normed like any other as long as their squares fit 32 bits."""
    q, k, wq, wk, gq, gk = make(1, 8, 4, 2, 64, seed=6)
    q[0, 0] = 0
    q[0, 1] *= 1e15
    q[0, 2] *= 1e-12
    f = freqs(64)
    qo, ko = kvpop.qk_norm_rope(q, k, wq, wk, EPS, f)
    assert (qo[0, 0] == 0).all()
    check_fwd(qo, q, wq, f, None, False, "q")
    dq, dk, dwq, dwk = kvpop.qk_norm_rope_bwd(q, k, gq, gk, wq, wk, EPS, f)
    check_bwd(dq, dwq, q, gq, wq, f, None, False, "q")


def test_bad_row_stays_in_its_row():
    q, k, wq, wk, gq, gk = make(1, 9, 4, 2, 128, seed=7)
    f = freqs(128)
    clean, _ = kvpop.qk_norm_rope(q, k, wq, wk, EPS, f)
    q2 = q.clone()
    q2[0, 4, 1, 77] = float("nan")
    q2[0, 4, 2, 3] = float("inf")
    got, _ = kvpop.qk_norm_rope(q2, k, wq, wk, EPS, f)
    assert torch.isnan(got[0, 4, 1]).all()
    keep = torch.ones(1, 9, 4, dtype=torch.bool, device="cuda")
    keep[0, 4, 1:3] = False
    assert torch.equal(got[keep], clean[keep])


def test_negative_and_extreme_positions():
    q, k, wq, wk, _, _ = make(1, 6, 2, 1, 128, seed=8)
    f = freqs(128)
    pos = torch.tensor([[-1, -100000, 2147483647, -2147483648, 0, 1048576]], dtype=torch.int32, device="cuda")
    qo, ko = kvpop.qk_norm_rope(q, k, wq, wk, EPS, f, pos)
    check_fwd(qo, q, wq, f, pos, False, "q")


def test_in_place_and_strided_gradients():
    """In place for contiguous inputs; gradients written into a packed projection's
    gradient leave its value part alone."""
    b, S, Hq, H, D = 2, 65, 8, 2, 128
    q, k, wq, wk, gq, gk = make(b, S, Hq, H, D, seed=9)
    f = freqs(D)
    ref = kvpop.qk_norm_rope(q, k, wq, wk, EPS, f)
    grads = kvpop.qk_norm_rope_bwd(q, k, gq, gk, wq, wk, EPS, f)
    dqkv = torch.full((b, S, (Hq + 2 * H) * D), 7.0, dtype=torch.bfloat16, device="cuda")
    views = (dqkv[..., : Hq * D].view(b, S, Hq, D), dqkv[..., Hq * D:(Hq + H) * D].view(b, S, H, D))
    out = kvpop.qk_norm_rope_bwd(q, k, gq, gk, wq, wk, EPS, f,
                                 out=(*views, torch.empty_like(wq), torch.empty_like(wk)))
    for a, r in zip(out, grads):
        assert torch.equal(a, r)  # the same bits: the sums' order is fixed
    assert (dqkv[..., (Hq + H) * D:] == 7.0).all()
    q2, k2 = q.clone(), k.clone()
    kvpop.qk_norm_rope(q2, k2, wq, wk, EPS, f, out=(q2, k2))
    assert torch.equal(q2, ref[0]) and torch.equal(k2, ref[1])


def test_stream_graph_and_repeat():
    """On a side stream, and captured and replayed on new data, the same bits."""
    q, k, wq, wk, gq, gk = make(2, 200, 8, 2, 128, seed=10, packed=True)
    f = freqs(128)
    ref = kvpop.qk_norm_rope(q, k, wq, wk, EPS, f) + kvpop.qk_norm_rope_bwd(q, k, gq, gk, wq, wk, EPS, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (kvpop.qk_norm_rope(q, k, wq, wk, EPS, f, stream=side)
           + kvpop.qk_norm_rope_bwd(q, k, gq, gk, wq, wk, EPS, f, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    for a, r in zip(got, ref):
        assert torch.equal(a, r)
    q0, k0 = torch.zeros_like(q), torch.zeros_like(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = kvpop.qk_norm_rope(q0, k0, wq, wk, EPS, f) + kvpop.qk_norm_rope_bwd(q0, k0, gq, gk, wq, wk, EPS, f)
    q0.copy_(q)
    k0.copy_(k)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, r in zip(out, ref):
        assert torch.equal(a, r)


def test_offsets_past_32_bits():
    """A packed projection of more than 2^31 elements: the last tokens are right."""
    b, S, Hq, H, D = 1, 90000, 1, 1, 128
    width = 24576
    buf = torch.empty(b, S, width, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(11)
    buf[:, -200:] = torch.randn(b, 200, width, generator=gen, device="cuda").bfloat16()
    buf[:, :-200, -256:] = 1
    q, k = buf[..., -256:-128].view(b, S, 1, D), buf[..., -128:].view(b, S, 1, D)
    f = freqs(D)
    qo, ko = kvpop.qk_norm_rope(q, k, None, None, EPS, f)
    tail = torch.arange(S - 200, S, device="cuda", dtype=torch.int32)[None]
    check_fwd(qo[:, -200:], q[:, -200:], None, f, tail, False, "q")
    check_fwd(ko[:, -200:], k[:, -200:], None, f, tail, False, "k")


def test_binding_refusals():
    q, k, wq, wk, gq, gk = make(2, 8, 4, 2, 64, seed=12)
    f = freqs(64)
    ok = (q, k, wq, wk, EPS, f)
    with pytest.raises(ValueError, match="bfloat16"):
        kvpop.qk_norm_rope(q.float(), *ok[1:])
    with pytest.raises(ValueError, match="contiguous"):
        kvpop.qk_norm_rope(q.transpose(1, 2), *ok[1:])
    with pytest.raises(ValueError, match="evenly"):
        kvpop.qk_norm_rope(torch.empty(2, 9, 4, 64, dtype=torch.bfloat16, device="cuda")[:, :8], *ok[1:])
    with pytest.raises(ValueError, match="pos"):
        kvpop.qk_norm_rope(*ok, pos=torch.zeros(8, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="wq"):
        kvpop.qk_norm_rope(q, k, wq[:32].contiguous(), wk, EPS, f)
    with pytest.raises(ValueError, match="k must be"):
        kvpop.qk_norm_rope(q, k[:1], wq, wk, EPS, f)
    with pytest.raises(kvpop.KvpopError):
        kvpop.qk_norm_rope(q, k, wq, wk, EPS, freqs(64)[:5].contiguous())   # R = 10
    with pytest.raises(ValueError, match="dq"):
        kvpop.qk_norm_rope_bwd(q, k, gq[:1].contiguous(), gk, wq, wk, EPS, f)
    with pytest.raises(ValueError, match="dwk"):
        kvpop.qk_norm_rope_bwd(q, k, gq, gk, wq, wk, EPS, f,
                               out=(torch.empty_like(q), torch.empty_like(k), wq, wq.double()))


@pytest.mark.parametrize("packed", [False, True])
def test_gradients_in_place(packed):
    """The gradients may replace q and k, contiguous or as parts of the packed projection."""
    q, k, wq, wk, gq, gk = make(3, 90, 6, 2, 64, seed=13, packed=packed)
    f = freqs(32)
    ref = kvpop.qk_norm_rope_bwd(q, k, gq, gk, wq, wk, EPS, f, interleaved=True)
    got = kvpop.qk_norm_rope_bwd(q, k, gq, gk, wq, wk, EPS, f, interleaved=True,
                                 out=(q, k, torch.empty_like(wq), torch.empty_like(wk)))
    for a, r in zip(got, ref):
        assert torch.equal(a, r)


def exact_angles(pos, inv_freq):
    """cos, sin [b, S, 1, R/2] of position times frequency, the product and its whole turns in
    integers: the frequency is a 24-bit integer times a power of two, 1 / 2 pi has 480 bits."""
    N = 480

    def arctan_inv(x):  # of 1/x, times 2^600
        s = t = (1 << 600) // x
        k, sign = 1, -1
        while t:
            t //= x * x
            k += 2
            s += sign * (t // k)
            sign = -sign
        return s
    inv_turn = (1 << (N + 600)) // (8 * (4 * arctan_inv(5) - arctan_inv(239)))  # Machin's formula for pi / 4
    turns = []
    for t in pos.flatten().tolist():
        for f in inv_freq.tolist():
            num, den = f.as_integer_ratio()
            x = t * num * inv_turn // den & ((1 << N) - 1)
            turns.append(x / (1 << N) if x >> (N - 1) == 0 else -((1 << N) - x) / (1 << N))
    a = 2 * torch.pi * torch.tensor(turns, dtype=torch.float64, device="cuda").view(*pos.shape, 1, -1)
    return a.cos(), a.sin()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("inter", [False, True])
def test_any_finite_frequency(D, inter):
    """Frequencies over the whole range of fp32, at positions to the ends of int32."""
    f = torch.tensor([1.0, -0.7, 6.25, 1000.5, 2.0 ** 20, 3.1e9, 2.0 ** 40 + 2.0 ** 20, 2.0 ** 63, 1e20, 1.7e28, 3.3e38,
                      -3.4028234663852886e38, 1e-20, 1e-44, 0.0, 2.0 ** 24 + 2], dtype=torch.float32, device="cuda")
    pos = torch.tensor([[0, 1, -1, 2, 2147483647, -2147483648, 123456789, 40000, 1 << 30]], dtype=torch.int32, device="cuda")
    q, k, wq, wk, gq, gk = make(1, 9, 6, 3, D, seed=30)
    cos, sin = exact_angles(pos, f)
    qo, ko = kvpop.qk_norm_rope(q, k, wq, wk, EPS, f, pos, inter)
    dq, dk, dwq, dwk = kvpop.qk_norm_rope_bwd(q, k, gq, gk, wq, wk, EPS, f, pos, inter)
    for x, w, z, g, dx, dw in ((q, wq, qo, gq, dq, dwq), (k, wk, ko, gk, dk, dwk)):
        y = ref64.norm_rope(x, w, EPS, None)[1]
        want = ref64._turn(y, cos, sin, inter)
        assert ((z.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -17 * y.abs().amax(-1, keepdim=True)).all()
        back = ref64._turn(g.double(), cos, -sin, inter)
        rx, rw, size, bound = ref64.norm_rope_bwd(x, back, w, EPS, None)
        turned = (g.double().abs().amax(-1, keepdim=True) * x.double().abs() /
                  ((x.double() ** 2).mean(-1, keepdim=True) + EPS).sqrt()).sum((0, 1, 2))
        assert ((dx.double() - rx).abs() <= 2.0 ** -8 * rx.abs() + 2.0 ** -17 * size).all()
        assert ((dw.double() - rw).abs() <= bound + 2.0 ** -20 * turned).all()


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("D,inter", [(64, False), (64, True), (128, False), (128, True)])
def test_frequencies_that_are_not_finite(D, inter, weights):
    """Their pairs come out NaN and the others as ever; backward every dx of a token is NaN, as
    the mean over the row is, and the weight gradients of the pairs alone."""
    q, k, wq, wk, gq, gk = make(2, 30, 5, 2, D, seed=31)
    if not weights:
        wq = wk = None
    f = freqs(48)
    clean = kvpop.qk_norm_rope(q, k, wq, wk, EPS, f, None, inter)
    cdw = kvpop.qk_norm_rope_bwd(q, k, gq, gk, wq, wk, EPS, f, None, inter)[2:]
    g = f.clone()
    pair = torch.tensor([0, 7, 8, 23], device="cuda")
    g[pair] = torch.tensor([float("nan"), float("inf"), -float("inf"), float("nan")], device="cuda")
    off = torch.cat([2 * pair, 2 * pair + 1] if inter else [pair, pair + 24])
    keep = torch.ones(D, dtype=torch.bool, device="cuda")
    keep[off] = False
    got = kvpop.qk_norm_rope(q, k, wq, wk, EPS, g, None, inter)
    out = kvpop.qk_norm_rope_bwd(q, k, gq, gk, wq, wk, EPS, g, None, inter)
    for z, c in zip(got, clean):
        assert torch.isnan(z[..., off]).all() and torch.equal(z[..., keep], c[..., keep])
    assert all(torch.isnan(dx).all() for dx in out[:2])
    for dw, c in zip(out[2:], cdw):
        assert torch.isnan(dw[off]).all() and torch.equal(dw[keep], c[keep])


def test_calls_go_to_the_current_stream():
    """Without a stream a call goes to torch's current one, read through calls of torch's binding
    that are not public: they have to say what the public one says, and work queued before a call
    on that stream has to come before it."""
    q, k, wq, wk, _, _ = make(1, 400, 8, 2, 128, seed=32)
    f = freqs(128)
    want = kvpop.qk_norm_rope(q, k, wq, wk, EPS, f)
    side = torch.cuda.Stream()
    assert kvpop._stream() == torch.cuda.current_stream().cuda_stream
    src, late = q.clone(), torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        assert kvpop._stream() == side.cuda_stream == torch.cuda.current_stream().cuda_stream
        torch.cuda._sleep(20_000_000)
        late.copy_(src)
        got = kvpop.qk_norm_rope(late, k, wq, wk, EPS, f)
    assert kvpop._stream() == torch.cuda.current_stream().cuda_stream != side.cuda_stream
    assert kvpop._stream(side) == side.cuda_stream
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
