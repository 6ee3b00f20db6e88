"""Refusals of the norm-and-rotation pair and of the shared-prefix attention
(host checks: nothing is launched), and the 64-bit forms that the GPU tests
compare with, checked against differences and against a single softmax."""
import ctypes
import math

import pytest
import torch

import ref64
from fixed_budget_kv_gb300 import kvpop

P = ctypes.c_void_p(256)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return kvpop.load()


def fwd(lib, q=P, qs=512, k=P, ks=128, b=1, S=4, Hq=8, H=2, D=64, wq=P, wk=P, eps=1e-6, f=P, R=64, pos=None, qo=P, ko=P):
    return lib.kvpop_qk_norm_rope(q, qs, k, ks, b, S, Hq, H, D, wq, wk, eps, f, R, 0, pos, qo, ko, None)


FWD_REFUSALS = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1),
    (dict(b=0), 1), (dict(S=0), 1), (dict(Hq=0), 1), (dict(H=-1), 1),
    (dict(D=96), 2), (dict(D=32), 2),
    (dict(R=-16), 1), (dict(R=80), 1), (dict(R=64, f=None), 1), (dict(R=24), 2),
    (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(qs=504), 1), (dict(ks=64), 1),                      # tokens overlap
    (dict(qs=516), 2), (dict(ks=130), 2),                     # rows off the 16-byte grid
    (dict(q=ctypes.c_void_p(264)), 2), (dict(ko=ctypes.c_void_p(258)), 2),
    (dict(b=65536, S=65536), 2), (dict(H=70000, ks=70000 * 64), 2),
]


@pytest.mark.parametrize("kw,code", FWD_REFUSALS, ids=lambda x: str(x))
def test_norm_rope_refusals(lib, kw, code):
    assert fwd(lib, **kw) == code
    assert lib.kvpop_last_error()


def bwd(lib, q=P, qs=512, ks=128, dq=P, dk=P, dqs=512, dks=128, D=64, R=64, f=P, dqi=P, ws=P, n=None):
    n = kvpop.qk_norm_rope_bwd_workspace_size(64) if n is None else n
    return lib.kvpop_qk_norm_rope_bwd(q, qs, P, ks, dq, dk, 1, 4, 8, 2, D, P, P, 1e-6, f, R, 0, None, dqi, dqs, P, dks, P,
                                      P, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(dq=None), 1), (dict(dk=None), 1), (dict(dqi=None), 1), (dict(ws=None), 1),
    (dict(n=16), 1), (dict(D=80), 2), (dict(R=40), 2), (dict(f=None), 1), (dict(dqs=256), 1), (dict(dks=132), 2),
    (dict(dq=ctypes.c_void_p(260)), 2), (dict(ws=ctypes.c_void_p(272)), 2),
], ids=lambda x: str(x))
def test_norm_rope_bwd_refusals(lib, kw, code):
    assert bwd(lib, **kw) == code
    assert lib.kvpop_last_error()


def test_norm_rope_bwd_workspace(lib):
    assert kvpop.qk_norm_rope_bwd_workspace_size(128) >= kvpop.qk_norm_rope_bwd_workspace_size(64) > 0
    n = ctypes.c_size_t()
    assert lib.kvpop_qk_norm_rope_bwd_workspace_size(96, ctypes.byref(n)) == 2
    assert lib.kvpop_qk_norm_rope_bwd_workspace_size(64, None) == 1


def prefix(lib, q=P, k=P, n=4, m=1, L=100, Hq=8, H=2, D=64, cu=P, lens=P, O2=None, lse2=None, O=P, lse=P, ws=P, nb=1 << 40):
    return lib.kvpop_prefix_attn(q, k, P, n, m, L, Hq, H, D, 0.0, cu, lens, O2, lse2, O, lse, ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(O=None), 1), (dict(lse=None), 1), (dict(ws=None), 1),
    (dict(n=0), 1), (dict(m=0), 1), (dict(L=0), 1), (dict(Hq=7), 1), (dict(H=0), 1),
    (dict(D=96), 2), (dict(Hq=6), 2),                         # G = 3 does not divide 128
    (dict(m=2, cu=None), 1),                                  # several prefixes need groups
    (dict(O2=P), 1), (dict(lse2=P), 1),                       # one half of a join
    (dict(nb=16), 1),
    (dict(q=ctypes.c_void_p(264)), 2), (dict(O=ctypes.c_void_p(258)), 2), (dict(O2=ctypes.c_void_p(264), lse2=P), 2),
    (dict(ws=ctypes.c_void_p(272)), 2), (dict(m=70000), 2), (dict(n=(1 << 24) + 1), 2), (dict(H=70000, Hq=70000), 2),
    (dict(L=(1 << 30) + 1), 2), (dict(n=1 << 24, H=64, Hq=4096, L=1 << 20), 2),   # more tiles than 2^31
], ids=lambda x: str(x))
def test_prefix_refusals(lib, kw, code):
    assert prefix(lib, **kw) == code
    assert lib.kvpop_last_error()


def test_prefix_workspace(lib):
    small = kvpop.prefix_attn_workspace_size(2, 1, 64, 4, 1, 64)
    large = kvpop.prefix_attn_workspace_size(512, 4, 131072, 32, 8, 128)
    assert 0 < small <= large < 1 << 28
    nb = ctypes.c_size_t()
    assert lib.kvpop_prefix_attn_workspace_size(2, 1, 64, 4, 1, 64, None) == 1
    assert lib.kvpop_prefix_attn_workspace_size(2, 1, 64, 4, 0, 64, ctypes.byref(nb)) == 1
    assert lib.kvpop_prefix_attn_workspace_size(2, 1, 64, 4, 1, 48, ctypes.byref(nb)) == 2


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kvpop.qk_norm_rope(x, x, None, None, 1e-6, None)
    with pytest.raises(ValueError, match="CUDA"):
        kvpop.qk_norm_rope_bwd(x, x, x.float(), x.float(), None, None, 1e-6, None)
    with pytest.raises(ValueError, match="CUDA"):
        kvpop.prefix_attn(x[0], x, x)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 16), (64, 0)])
def test_norm_rope_gradient_against_differences(D, R, interleaved):
    """d/dh of sum(g * z) along random directions of x and w, by central differences in
    64 bits: h = 1e-5 leaves h^2 (1e-10) of the third derivative and 1e-16 / h (1e-11)
    of rounding, so 1e-7 of the terms' size is generous."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(2, 3, 2, D, generator=gen, dtype=torch.float64)
    g = torch.randn(2, 3, 2, D, generator=gen, dtype=torch.float64)
    w = 1 + 0.2 * torch.randn(D, generator=gen, dtype=torch.float64)
    f = (10000.0 ** (-torch.arange(0, R, 2).double() / R)).float() if R else None
    pos = torch.tensor([[5, 6, 7], [100000, 100001, -3]], dtype=torch.int32)
    dx, dw, _, _ = ref64.norm_rope_bwd(x, g, w, 1e-6, f, pos, interleaved)

    def val(xx, ww):
        return float((g * ref64.norm_rope(xx, ww, 1e-6, f, pos, interleaved)[0]).sum())
    for _ in range(5):
        d = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        e = torch.randn(w.shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        assert abs((val(x + h * d, w) - val(x - h * d, w)) / (2 * h) - float((dx * d).sum())) < 1e-6
        assert abs((val(x, w + h * e) - val(x, w - h * e)) / (2 * h) - float((dw * e).sum())) < 1e-6


def test_prefix_form_against_one_softmax():
    """Joining the attention over keys [0, a) with that over [a, P) is one softmax over [0, P)."""
    gen = torch.Generator().manual_seed(4)
    q = torch.randn(3, 4, 64, generator=gen, dtype=torch.float64)
    k = torch.randn(1, 30, 2, 64, generator=gen, dtype=torch.float64)
    v = torch.randn(1, 30, 2, 64, generator=gen, dtype=torch.float64)
    O2, l2, _, _ = ref64.prefix_attn(q, k[:, 11:], v[:, 11:], [0, 3], [19])
    O, lse, mass, _ = ref64.prefix_attn(q, k, v, [0, 3], [11], join=(O2, l2))
    for i in range(3):
        for hq in range(4):
            s = (k[0, :, hq // 2] @ q[i, hq]) / 8.0
            p = torch.softmax(s, 0)
            assert torch.allclose(O[i, hq], p @ v[0, :, hq // 2], atol=1e-12)
            assert math.isclose(float(lse[i, hq]), float(torch.logsumexp(s, 0)), abs_tol=1e-12)
    assert (mass >= O.abs() - 1e-12).all()


@pytest.mark.parametrize("n,m,L,H,G", [((1 << 31) - 1, 1, 1 << 30, 1 << 23, 128), (1914826685, 1950157578, 469102189, 19575053, 64),
                                       (4, (1 << 31) - 1, 1 << 30, (1 << 31) - 1, 1), ((1 << 24) + 1, 1, 1, 1, 1),
                                       (1, 65536, 1, 1, 1), (1, 1, 1, 65536, 1), (1, 1, 1, 1024, 64), (1 << 24, 1, 1, 2, 64)],
                         ids=str)
def test_prefix_workspace_of_refused_sizes(lib, n, m, L, H, G):
    """What the attention refuses has no workspace either, however large the sizes' products."""
    nb = ctypes.c_size_t(7)
    assert lib.kvpop_prefix_attn_workspace_size(n, m, L, H * G, H, 64, ctypes.byref(nb)) == 2
    assert nb.value == 7 and lib.kvpop_last_error()
