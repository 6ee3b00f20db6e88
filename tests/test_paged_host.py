"""Refusals of the calls on a paged cache (host checks: nothing is launched), and the
64-bit forms that the GPU tests compare with, checked against one softmax and against
a step-by-step account."""
import ctypes
import math

import pytest
import torch

import ref64_paged as ref
from fixed_budget_kv_gb300 import kvpop

P = ctypes.c_void_p(256)
BIG = 1 << 40


def at(x):
    return ctypes.c_void_p(x)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return kvpop.load()


def append(lib, k=P, ks=128, v=P, vs=128, T=4, n=2, H=2, D=64, cu=P, lens=P, table=P, most=3, kp=P, kps=2048, vp=P, vps=2048,
           pages=9, page=16, scores=P):
    return lib.kvpop_paged_append(k, ks, v, vs, T, n, H, D, cu, lens, table, most, kp, kps, vp, vps, pages, page, scores, None)


def attn(lib, q=P, T=4, n=2, Hq=4, H=2, D=64, cu=P, lens=P, table=P, most=3, kp=P, kps=2048, vp=P, vps=2048, pages=9, page=16,
         O=P, lse=P, ws=P, nb=BIG):
    return lib.kvpop_paged_attn(q, T, n, Hq, H, D, 0.0, cu, lens, table, most, kp, kps, vp, vps, pages, page, O, lse, ws, nb, None)


def mass(lib, q=P, lse=P, T=4, n=2, Hq=4, H=2, D=64, decay=1.0, cu=P, lens=P, table=P, most=3, kp=P, kps=2048, pages=9, page=16,
         scores=P, ws=P, nb=BIG):
    return lib.kvpop_paged_mass(q, lse, T, n, Hq, H, D, 0.0, decay, cu, lens, table, most, kp, kps, pages, page, scores, ws, nb,
                                None)


def evict(lib, kp=P, kps=2048, vp=P, vps=2048, scores=P, n=2, H=2, D=64, s=1, w=2, k=3, lens=P, table=P, most=3, pages=9, page=16,
          kept=P, new=P):
    return lib.kvpop_paged_evict(kp, kps, vp, vps, scores, n, H, D, kvpop.Budget(s, w, k), lens, table, most, pages, page, kept,
                                 new, None)


# what every call refuses
SHARED = [
    (dict(lens=None), 1), (dict(table=None), 1), (dict(kp=None), 1), (dict(n=0), 1), (dict(H=0), 1), (dict(most=0), 1),
    (dict(pages=0), 1), (dict(page=0), 1), (dict(page=-16), 1), (dict(kps=2040), 1),
    (dict(D=96, kps=1 << 20, vps=1 << 20), 2), (dict(page=8), 2), (dict(page=48, kps=1 << 20, vps=1 << 20), 2),
    (dict(page=1 << 17, kps=1 << 30, vps=1 << 30), 2), (dict(kps=2052), 2), (dict(kp=at(264)), 2), (dict(lens=at(258)), 2),
    (dict(table=at(257)), 2), (dict(most=1 << 27), 2), (dict(kps=1 << 38), 2),
]
ROWS = [(dict(T=0), 1), (dict(cu=None), 1), (dict(T=(1 << 24) + 1), 2), (dict(n=65536), 2), (dict(cu=at(258)), 2)]
QUERY = [
    (dict(q=None), 1), (dict(lse=None), 1), (dict(ws=None), 1), (dict(nb=1), 1), (dict(Hq=0), 1), (dict(Hq=5), 1),
    (dict(Hq=6), 2), (dict(q=at(264)), 2), (dict(ws=at(272)), 2), (dict(lse=at(258)), 2),
    (dict(T=1 << 24, H=64, Hq=64 * 64, kps=1 << 20, vps=1 << 20), 2),                    # T * Hq
    (dict(T=1 << 20, Hq=128, H=1, most=1 << 26, kps=1 << 20, vps=1 << 20), 2),           # tiles of rows and keys
]


def only(calls, call):
    """Refusals without arguments that `call` lacks."""
    names = call.__code__.co_varnames[:call.__code__.co_argcount]
    return [({a: b for a, b in kw.items() if a in names}, code) for kw, code in calls if next(iter(kw)) in names]


def refused(call, calls):
    return [pytest.param(call, kw, code, id=f"{call.__name__}-{kw}") for kw, code in only(calls, call)]


@pytest.mark.parametrize("call,kw,code", [
    *refused(append, SHARED + ROWS), *refused(attn, SHARED + ROWS + QUERY), *refused(mass, SHARED + ROWS + QUERY),
    *refused(evict, SHARED),
    *refused(append, [(dict(k=None), 1), (dict(v=None), 1), (dict(vp=None), 1), (dict(ks=120), 1), (dict(vs=64), 1),
                      (dict(ks=132), 2), (dict(v=at(264)), 2), (dict(vps=2047), 1), (dict(scores=at(258)), 2)]),
    *refused(attn, [(dict(O=None), 1), (dict(vp=None), 1), (dict(vp=at(264)), 2), (dict(O=at(264)), 2)]),
    *refused(mass, [(dict(scores=None), 1), (dict(decay=-0.1), 1), (dict(decay=1.5), 1), (dict(decay=float("nan")), 1),
                    (dict(scores=at(258)), 2)]),
    *refused(evict, [(dict(scores=None), 1), (dict(kept=None), 1), (dict(new=None), 1), (dict(vp=None), 1), (dict(s=-1), 1),
                     (dict(k=-1), 1), (dict(s=0, w=0, k=0), 1), (dict(s=1 << 30), 1), (dict(n=40000), 2),
                     (dict(scores=at(260)), 2), (dict(kept=at(258)), 2), (dict(new=at(257)), 2)]),
])
def test_refusals(lib, call, kw, code):
    assert call(lib, **kw) == code
    assert lib.kvpop_last_error()


@pytest.mark.parametrize("what", ["attn", "mass"])
def test_workspace_sizes(lib, what):
    size = getattr(kvpop, f"paged_{what}_workspace_size")
    assert 0 < size(2, 2, 2, 1, 64, 2, 16) <= size(16384, 64, 32, 8, 128, 2048, 64) < 1 << 28
    fn = getattr(lib, f"kvpop_paged_{what}_workspace_size")
    nb = ctypes.c_size_t(7)
    assert fn(2, 2, 2, 1, 64, 2, 16, None) == 1
    for args, code in [((0, 2, 2, 1, 64, 2, 16), 1), ((2, 2, 3, 2, 64, 2, 16), 1), ((2, 2, 2, 1, 48, 2, 16), 2),
                       ((2, 2, 3, 1, 64, 2, 16), 2), ((2, 2, 2, 1, 64, 2, 24), 2), ((2, 70000, 2, 1, 64, 2, 16), 2),
                       ((1 << 24, 2, 128, 1, 64, 1 << 26, 16), 2), (((1 << 31) - 1, (1 << 31) - 1, 1 << 30, 1 << 30, 64, 1, 16), 2),
                       ((1, 1, 1, 1, 64, (1 << 31) - 1, 65536), 2)]:
        assert fn(*args, ctypes.byref(nb)) == code, args
        assert nb.value == 7 and lib.kvpop_last_error()


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    kp = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kvpop.paged_append(x, x, kp, kp, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        kvpop.paged_attn(x, kp, kp, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        kvpop.paged_mass(x, x[..., 0].float(), kp, kp[..., 0].float(), table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        kvpop.paged_evict(kp, kp, kp[..., 0].float(), table, lens, 1, 1, 1)


def test_stride_of_one_page():
    """The stride of a dimension of one means nothing, whatever a view makes of it."""
    x = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16)
    dev = x.get_device()
    for view in (x.transpose(0, 1), x[:, 0][None], x.as_strided((1, 4, 16, 64), (7, 1024, 64, 1))):
        assert view.is_contiguous() and kvpop._page_stride(view, dev, "kp") == 4096
    x = torch.zeros(3, 4, 16, 64, dtype=torch.bfloat16)
    assert kvpop._page_stride(x, dev, "kp") == 4096


def cache(gen, n, H, page, D, lens):
    held = [-(-x // page) for x in lens]
    order = torch.randperm(sum(held) + 1, generator=gen)
    table = torch.full((n, max(held) + 1), -1, dtype=torch.int32)
    a = 0
    for i, c in enumerate(held):
        table[i, :c] = order[a:a + c]
        a += c
    kp, vp = (torch.randn(sum(held) + 1, H, page, D, generator=gen, dtype=torch.float64) for _ in range(2))
    return kp, vp, table


def test_forms_against_one_softmax():
    """Row r of a chunk of c is row len - c + r of the whole causal attention, and the mass of
    all rows of a prompt sums to the number of its rows and heads."""
    gen = torch.Generator().manual_seed(1)
    lens, cu, H, G, D = [37, 5], [0, 9, 14], 2, 2, 16
    kp, vp, table = cache(gen, 2, H, 16, D, lens)
    q = torch.randn(14, H * G, D, generator=gen, dtype=torch.float64)
    O, lse, _, _ = ref.attn(q, kp, vp, table, lens, cu)
    got, bound = ref.mass(q, lse, kp, torch.zeros(kp.shape[:3], dtype=torch.float64), table, lens, cu, 1.0)
    for i, length in enumerate(lens):
        c = cu[i + 1] - cu[i]
        for h in range(H):
            k, v = (torch.cat([x[table[i, t // 16], h, t % 16][None] for t in range(length)]) for x in (kp, vp))
            total = torch.zeros(length, dtype=torch.float64)
            for r in range(c):
                for g in range(G):
                    m = length - c + r + 1
                    sc = k[:m] @ q[cu[i] + r, h * G + g] / 4.0
                    p = torch.softmax(sc, 0)
                    assert torch.allclose(O[cu[i] + r, h * G + g], p @ v[:m], atol=1e-12)
                    assert math.isclose(float(lse[cu[i] + r, h * G + g]), float(torch.logsumexp(sc, 0)), abs_tol=1e-12)
                    total[:m] += p
            assert torch.allclose(ref.slots(got, table, i, h, length), total, atol=1e-12)
    assert math.isclose(float(got.sum()), 14 * H * G, rel_tol=1e-12) and (bound >= 0).all()


def test_eviction_form_by_hand():
    table = torch.tensor([[2, 0], [1, -1]], dtype=torch.int32)
    scores = torch.zeros(3, 1, 16)
    # sequence 0: 18 slots, s = 1, w = 2, k = 3; ties go to the lower slot, NaN is the worst
    line = [9.0, 1.0, 5.0, float("nan"), 5.0, 2.0, 5.0, 0.0, -0.0, 1.0, 5.0, 0.5, 0.25, 0.0, 1.0, 2.0, 7.0, 8.0]
    for t, x in enumerate(line):
        scores[table[0, t // 16], 0, t % 16] = x
    kp = torch.arange(3 * 16, dtype=torch.float64).reshape(3, 1, 16, 1)
    k2, _, s2, kept, new = ref.evict(kp, kp, scores, table, [18, 4], 1, 2, 3)
    assert kept[0, 0].tolist() == [0, 2, 4, 6, 16, 17] and kept[1, 0].tolist() == [0, 1, 2, 3, -1, -1]
    assert new.tolist() == [6, 4]
    assert ref.slots(k2, table, 0, 0, 6)[:, 0].tolist() == [32, 34, 36, 38, 0, 1]
    assert ref.slots(s2, table, 0, 0, 6).tolist() == [9, 5, 5, 5, 7, 8]
    assert torch.equal(ref.slots(k2, table, 0, 0, 18)[6:], ref.slots(kp, table, 0, 0, 18)[6:])
