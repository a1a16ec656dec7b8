"""Refusals of the rotary, per-head-norm and tree-attention entry points: on the host,
before any CUDA call, through the C ABI and through the binding."""
import ctypes

import pytest
import torch

import block_sparse_long_10_b200 as qsa
from block_sparse_long_10_b200 import build as qbuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
SIZE_MAX = ctypes.c_size_t(-1).value
F = ctypes.c_void_p(0x10000)       # aligned, never dereferenced by host validation
ODD = ctypes.c_void_p(0x10004)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qsa.load()


def _caller(fn, names, good):
    def call(**kw):
        assert set(kw) <= set(names), kw
        return fn(*[kw.get(n, good[n]) for n in names])
    return call


def test_rope(lib):
    names = "x xs y ys dt B T H D f rot lay m tr pos pos0 s".split()
    good = dict(x=F, xs=512, y=F, ys=512, dt=0, B=2, T=3, H=4, D=128, f=F, rot=64, lay=0, m=1.0,
                tr=0, pos=None, pos0=None, s=None)
    call = _caller(lib.qsa_rope, names, good)
    assert call(T=0) == OK and call(T=0, x=None, y=None) == OK
    for kw in (dict(x=None), dict(y=None), dict(f=None), dict(B=0), dict(T=-1), dict(H=0),
               dict(D=0), dict(rot=-8), dict(rot=136), dict(dt=2), dict(lay=2), dict(m=NAN),
               dict(m=INF), dict(x=ODD), dict(y=ODD), dict(f=ODD), dict(pos=ODD), dict(pos0=ODD),
               dict(xs=511), dict(xs=513), dict(ys=516), dict(ys=-512), dict(ys=520)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=96), dict(D=512, xs=2048, ys=2048), dict(rot=12), dict(D=16, rot=16)):
        assert call(**kw) == UNSUPPORTED, kw


def test_norm_rope(lib):
    names = ("q qs k ks v vs B T Hq Hkv D qw kw eps f rot lay m pos pos0 qo ko vo slot L ws "
             "s").split()
    good = dict(q=F, qs=2560, k=F, ks=2560, v=F, vs=2560, B=2, T=3, Hq=16, Hkv=2, D=128, qw=F,
                kw=F, eps=1e-6, f=F, rot=128, lay=0, m=1.0, pos=None, pos0=None, qo=F, ko=F,
                vo=F, slot=F, L=64, ws=None, s=None)
    call = _caller(lib.qsa_qk_norm_rope, names, good)
    assert call(T=0) == OK
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(vo=None), dict(qo=None),
               dict(ko=None), dict(f=None), dict(B=0), dict(T=-1), dict(Hq=0), dict(Hkv=0),
               dict(eps=-1.0), dict(eps=NAN), dict(m=NAN), dict(lay=-1), dict(rot=136),
               dict(slot=None), dict(L=-1), dict(qs=2047), dict(ks=255), dict(vs=257),
               dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(qo=ODD), dict(ko=ODD), dict(vo=ODD),
               dict(qw=ODD), dict(kw=ODD), dict(slot=ODD), dict(ws=ODD)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=96, rot=96), dict(rot=4)):
        assert call(**kw) == UNSUPPORTED, kw


def test_norm_rope_backward(lib):
    n = lib.qsa_qk_norm_rope_backward_workspace_size(2, 3, 16, 2, 128)
    assert 256 < n < SIZE_MAX
    for bad in ((0, 3, 16, 2, 128), (2, -1, 16, 2, 128), (2, 3, 0, 2, 128), (2, 3, 16, 0, 128),
                (2, 3, 16, 2, 96)):
        assert lib.qsa_qk_norm_rope_backward_workspace_size(*bad) == SIZE_MAX
    names = ("dq dk dt q qs k ks B T Hq Hkv D qw kw eps f rot lay m pos pos0 oq ok ot dqw dkw ws "
             "wsb s").split()
    good = dict(dq=F, dk=F, dt=1, q=F, qs=2048, k=F, ks=256, B=2, T=3, Hq=16, Hkv=2, D=128, qw=F,
                kw=F, eps=1e-6, f=F, rot=128, lay=1, m=1.0, pos=None, pos0=None, oq=F, ok=F, ot=1,
                dqw=F, dkw=F, ws=F, wsb=n, s=None)
    call = _caller(lib.qsa_qk_norm_rope_backward, names, good)
    assert call(T=0, dqw=None, dkw=None) == OK
    assert call(T=0, f=None) == INVALID  # the weight gradients are written: a launch
    for kw in (dict(dq=None), dict(dk=None), dict(q=None), dict(k=None), dict(oq=None),
               dict(ok=None), dict(f=None), dict(dt=2), dict(ot=-1), dict(qw=None), dict(kw=None),
               dict(eps=NAN), dict(lay=3), dict(rot=160), dict(qs=2040), dict(ks=260),
               dict(dq=ODD), dict(oq=ODD), dict(qw=ODD), dict(ot=0)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(ws=None), dict(wsb=n - 1), dict(ws=ODD)):
        assert call(**kw) == WORKSPACE, kw
    assert call(D=80, rot=80) == UNSUPPORTED and call(rot=20) == UNSUPPORTED


def test_tree_decode(lib):
    n = lib.qsa_dense_tree_decode_workspace_size(2, 8, 16, 2, 128)
    m = lib.qsa_sparse_tree_decode_workspace_size(2, 8, 16, 128, 4, 2048)
    assert 256 < n < SIZE_MAX and 256 < m < SIZE_MAX
    for bad in ((0, 8, 16, 2, 128), (2, 0, 16, 2, 128), (2, 8, 16, 3, 128), (2, 8, 16, 0, 128),
                (2, 8, 16, 2, 0), (2, 257, 16, 2, 128), (2 ** 24, 8, 16, 2, 128),
                (1, 65536, 65536, 1, 128), (2, 8, 16, 2, 96)):
        assert lib.qsa_dense_tree_decode_workspace_size(*bad) == SIZE_MAX, bad
    for bad in ((0, 8, 16, 128, 4, 2048), (2, 8, 16, 128, 0, 2048), (2, 8, 16, 128, 4, 2),
                (2, 8, 16, 128, 4, 2047), (2, 257, 16, 128, 4, 2048),
                (2 ** 24, 8, 16, 128, 4, 2048), (2, 8, 2 ** 30, 128, 4, 2048),
                (2, 8, 16, 96, 4, 2048)):
        assert lib.qsa_sparse_tree_decode_workspace_size(*bad) == SIZE_MAX, bad
    dense = "q k v sl L par nd B N Hq Hkv D sc o lse ws wsb s".split()
    sparse = "q k v sl L sel sb sn par nd B N Hq Hkv D r bud sc o lse ws wsb s".split()
    good = dict(q=F, k=F, v=F, sl=F, L=1000, sel=F, sb=4096, sn=512, par=F, nd=None, B=2, N=8,
                Hq=16, Hkv=2, D=128, r=4, bud=2048, sc=0.1, o=F, lse=None, ws=F, wsb=max(n, m),
                s=None)
    for fn, names in ((lib.qsa_dense_tree_decode, dense), (lib.qsa_sparse_tree_decode, sparse)):
        call = _caller(fn, names, good)
        for kw in (dict(q=None), dict(k=None), dict(v=None), dict(sl=None), dict(par=None),
                   dict(o=None), dict(B=0), dict(N=0), dict(L=0), dict(Hkv=0), dict(Hkv=3),
                   dict(sc=NAN), dict(sc=INF), dict(q=ODD), dict(k=ODD), dict(v=ODD),
                   dict(o=ODD)):
            assert call(**kw) == INVALID, kw
        for kw in (dict(N=257), dict(D=96), dict(Hq=64), dict(Hkv=8), dict(L=2 ** 31),
                   dict(B=2 ** 24)):
            assert call(**kw) == UNSUPPORTED, kw
        for kw in (dict(ws=None), dict(wsb=256), dict(ws=ODD)):
            assert call(**kw) == WORKSPACE, kw
    call = _caller(lib.qsa_sparse_tree_decode, sparse, good)
    for kw in (dict(sel=None), dict(r=0), dict(bud=3), dict(bud=2046), dict(sb=-1), dict(sn=-1)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(r=8), dict(bud=4100)):
        assert call(**kw) == UNSUPPORTED, kw


def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    f = torch.ones(8, dtype=torch.float64)
    with pytest.raises(ValueError):
        qsa.qsa_rope(x, x, f)                      # not on a GPU
    with pytest.raises(TypeError):
        qsa.qsa_rope(x.half(), x.half(), f)
    with pytest.raises(TypeError):
        qsa.qsa_qk_norm_rope(x.float(), x, x, x, f)
    with pytest.raises(TypeError):
        qsa.qsa_qk_norm_rope_backward(x.half(), x, x, x, x, x, f)
    z = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: qsa.qsa_dense_tree_decode(x, x, x, z, z[None], x, None),
                 lambda: qsa.qsa_sparse_tree_decode(x, x, x, z, z[None, None], z[None], x, None)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("Hq,Hkv,D,most", [(4, 4, 64, 30393), (1, 1, 64, 116508),
                                           (16, 2, 128, 59918)])
def test_sparse_tree_stages_fit_32_bits(lib, Hq, Hkv, D, most):
    """256 drafts, a budget of 4096: a row has ceil((1024 + 1 + 64) Hkv / 16) + 3 stages (276,
    72, 140), and all of B * 256 rows at most 2^31 - 1.  (The calls that fit lack a workspace.)"""
    names = "q k v sl L sel sb sn par nd B N Hq Hkv D r bud sc o lse ws wsb s".split()
    good = dict(q=F, k=F, v=F, sl=F, L=1000, sel=F, sb=0, sn=0, par=F, nd=None, B=most, N=256,
                Hq=Hq, Hkv=Hkv, D=D, r=4, bud=4096, sc=0.1, o=F, lse=None, ws=None, wsb=0, s=None)
    call = _caller(lib.qsa_sparse_tree_decode, names, good)
    size = lib.qsa_sparse_tree_decode_workspace_size
    assert call() == WORKSPACE and size(most, 256, Hq, D, 4, 4096) < SIZE_MAX
    assert call(B=most + 1) == UNSUPPORTED
    assert call(B=most + 1, bud=2048) == WORKSPACE  # fewer stages a row
    # the size function, which is not told Hkv, has none where no Hkv fits
    assert size(230000, 256, Hq, D, 4, 4096) == SIZE_MAX


def test_norm_rope_in_place_where_the_layouts_agree_only(lib):
    """Rows written elsewhere than where they were read would be read again: a strided input,
    or slots, in place."""
    at = lambda i: ctypes.c_void_p(0x10000 * (i + 1))
    names = ("q qs k ks v vs B T Hq Hkv D qw kw eps f rot lay m pos pos0 qo ko vo slot L ws "
             "s").split()
    good = dict(q=at(0), qs=2048, k=at(1), ks=256, v=at(2), vs=256, B=2, T=3, Hq=16, Hkv=2, D=128,
                qw=F, kw=F, eps=1e-6, f=F, rot=128, lay=0, m=1.0, pos=None, pos0=None, qo=at(3),
                ko=at(4), vo=at(5), slot=None, L=3, ws=None, s=None)
    call = _caller(lib.qsa_qk_norm_rope, names, good)
    for kw in (dict(qo=at(0), qs=2560), dict(ko=at(1), ks=2560), dict(vo=at(2), vs=2560),
               dict(ko=at(1), slot=F), dict(vo=at(2), slot=F), dict(ko=at(1), slot=F, L=9),
               dict(ko=at(1), slot=F, B=1, T=1)):
        assert call(**kw) == INVALID, kw
