"""GPU parity of qsa_rope, qsa_qk_norm_rope and its backward against the fp64 oracle
(oracle/rope.py), through the C ABI.

Bounds, derived from the arithmetic (u = half a step of the output type, relative;
eps32 = 2^-24):
  * a reduced angle is rounded once to fp32 (at most pi * eps32 off) and its sine and
    cosine are within 2 ulp (2^-23): with the product by mscale each is within 2^-21.
    A rotated value is two products and a sum of them: it is off by at most
    2^-20 (|a| + |b|) mscale, plus u |y|.
  * a head's sum of squares adds at most 2 VEC + 5 = 21 terms in any chain and rsqrt is
    within 2 ulp: z is within 2^-19 relative, which joins the bound above.
  * dx = r (g - xh mean(g xh)): each factor within 2^-19 of its size, so dx is within
    2^-17 r (|g| + |xh| mean |g xh|), g = weight dz, with |dz| taken as |a| + |b|.
  * dweight sums rows in fp32, at most a few hundred in any chain here (512 * 2^-24 =
    2^-15), each term within 2^-17 of |dz| |xh|: off by at most 2^-14 sum |dz xh|.
"""
import numpy as np
import pytest
import torch

import block_sparse_long_10_b200 as qsa
from oracle import rope

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=BF):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def _size(x, rot, layout):
    """|a| + |b| of each value's pair, |x| where it is not turned."""
    x = np.abs(x)
    out = x.copy()
    a, b = rope.pairs(rot, layout)
    out[..., a] = out[..., b] = x[..., a] + x[..., b]
    return out


def _check(got, ref, bound, dtype, what):
    got = _f64(got)
    assert np.isfinite(got).all(), what
    off = np.abs(got - ref) - HALF_STEP[dtype] * np.abs(ref) - bound
    assert (off <= 0).all(), (what, float(off.max()), int((off > 0).sum()))


def _freq(rot, scaling="none"):
    return qsa.qsa_rope_frequencies(1e6, rot, scaling, 8.0, 32768.0, device=DEV)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,T,H,D,rot", [
    (1, 1, 1, 32, 8), (3, 1, 4, 64, 32), (2, 5, 3, 64, 64), (1, 333, 16, 128, 128),
    (2, 67, 5, 128, 24), (1, 9, 2, 256, 256), (1, 70, 1, 32, 16), (2, 3, 7, 128, 0),
    (1, 5000, 2, 128, 64)])
def test_rope(B, T, H, D, rot, layout, dtype):
    g = _gen(B * T + D)
    x = _randn(g, B, T, H, D, dtype=dtype)
    f, m = _freq(rot, "by-parts") if rot else (None, 1.0)
    pos = torch.randint(-1000, 1 << 21, (B, T), generator=g, device=DEV)
    freq = [] if f is None else _f64(f)
    for transpose in (False, True):
        y = torch.full_like(x, float("nan"))
        qsa.qsa_rope(x, y, f, pos=pos, layout=layout, mscale=m, transpose=transpose)
        ref = rope.rope(_f64(x), pos.cpu().numpy(), freq, layout, m, transpose)
        _check(y, ref, 2.0 ** -20 * m * _size(_f64(x), rot, layout), dtype, "rope")
        if rot < D:
            assert torch.equal(y[..., rot:], x[..., rot:])  # copied, not computed
        z = x.clone()
        qsa.qsa_rope(z, z, f, pos=pos, layout=layout, mscale=m, transpose=transpose)
        assert torch.equal(z, y)  # in place


def test_rope_far_positions():
    """Positions up to 2^40: the fp64 turn p f / 2 pi is off by 2^-52 of itself (two
    products), so the angle by 2 pi * 2^-52 * 2^40 * f / 2 pi = f 2^-12."""
    g = _gen(5)
    x = _randn(g, 1, 64, 2, 64, dtype=F32)
    f, _ = _freq(64)
    pos = torch.randint(1 << 39, 1 << 40, (1, 64), generator=g, device=DEV)
    y = torch.empty_like(x)
    qsa.qsa_rope(x, y, f, pos=pos)
    xl, fl, pl = _f64(x).astype(np.longdouble), _f64(f).astype(np.longdouble), pos.cpu().numpy()
    angle = pl[..., None, None].astype(np.longdouble) * fl
    a, b = rope.pairs(64, "half")
    ref = np.empty_like(xl)
    ref[..., a] = xl[..., a] * np.cos(angle) - xl[..., b] * np.sin(angle)
    ref[..., b] = xl[..., b] * np.cos(angle) + xl[..., a] * np.sin(angle)
    size = _size(_f64(x), 64, "half")
    slack = 2.0 ** -20 + 2 * np.concatenate([_f64(f)] * 2) * 2.0 ** -12
    _check(y, ref.astype(np.float64), size * slack, F32, "far")


def test_positions_from_rows_and_parts_of_a_projection():
    g = _gen(7)
    packed = _randn(g, 3, 40, 4 * 64 + 2 * 64)
    x = packed[..., 256:].unflatten(-1, (2, 64))
    f, _ = _freq(64)
    pos0 = torch.tensor([0, 17, 1 << 20], device=DEV)
    rows = torch.arange(40, device=DEV)
    y, z = torch.empty(3, 40, 2, 64, dtype=BF, device=DEV), packed.clone()
    qsa.qsa_rope(x, y, f, pos0=pos0)
    zk = z[..., 256:].unflatten(-1, (2, 64))
    qsa.qsa_rope(zk, zk, f, pos=pos0[:, None] + rows)
    assert torch.equal(y, zk) and torch.equal(z[..., :256], packed[..., :256])
    qsa.qsa_rope(x, y, f)
    w = torch.empty_like(y)
    qsa.qsa_rope(x, w, f, pos=rows.expand(3, 40).contiguous())
    assert torch.equal(y, w)


def test_rope_is_its_gradient():
    """<dy, R x> = <R^T dy, x>, and the map is linear: the transposed call is the
    gradient.  Each side sums n products within 2^-19 of their size."""
    g = _gen(8)
    x, dy = _randn(g, 2, 50, 4, 128, dtype=F32), _randn(g, 2, 50, 4, 128, dtype=F32)
    f, m = _freq(96, "by-parts")
    for layout in ("half", "interleaved"):
        y, dx = torch.empty_like(x), torch.empty_like(x)
        qsa.qsa_rope(x, y, f, layout=layout, mscale=m)
        qsa.qsa_rope(dy, dx, f, layout=layout, mscale=m, transpose=True)
        a, b = (_f64(dy) * _f64(y)).sum(), (_f64(dx) * _f64(x)).sum()
        assert abs(a - b) <= 2.0 ** -18 * m * (_size(_f64(x), 96, layout) * np.abs(_f64(dy))).sum()


CASES = [(1, 1, 1, 1, 32, 8), (64, 1, 16, 2, 128, 128), (2, 77, 4, 1, 64, 32),
         (1, 1030, 8, 4, 128, 48), (3, 5, 2, 2, 256, 256), (1, 33, 5, 3, 64, 24),
         (2, 9, 4, 2, 128, 0), (1, 300, 1, 1, 32, 32)]


def _weights(g, D, which):
    w = lambda: 1 + 0.3 * torch.randn(D, generator=g, device=DEV)
    return w() if which[0] else None, w() if which[1] else None


@pytest.mark.parametrize("which", [(True, True), (True, False), (False, False)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot", CASES)
def test_norm_rope(B, T, Hq, Hkv, D, rot, layout, which):
    g = _gen(B * T + D + rot)
    packed = _randn(g, B, T, (Hq + 2 * Hkv) * D)
    q = packed[..., :Hq * D].unflatten(-1, (Hq, D))
    k = packed[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    v = packed[..., (Hq + Hkv) * D:].unflatten(-1, (Hkv, D))
    qw, kw = _weights(g, D, which)
    f, m = _freq(rot, "linear") if rot else (None, 1.0)
    freq = [] if f is None else _f64(f)
    L = T + 9
    slot = torch.stack([torch.randperm(L, generator=g, device=DEV)[:T] for _ in range(B)])
    slot[0, T // 2] = -1
    pos = torch.randint(0, 1 << 18, (B, T), generator=g, device=DEV)
    kc, vc = _randn(g, B, L, Hkv, D), _randn(g, B, L, Hkv, D)
    k0, v0 = kc.clone(), vc.clone()
    qo = torch.full((B, T, Hq, D), float("nan"), dtype=BF, device=DEV)
    kwargs = dict(q_weight=qw, k_weight=kw, eps=1e-5, pos=pos, layout=layout, mscale=m)
    qsa.qsa_qk_norm_rope(q, k, qo, kc, f, v=v, v_out=vc, slot=slot, **kwargs)
    p = pos.cpu().numpy()
    out = {}
    for n, x, w in (("q", q, qw), ("k", k, kw)):
        w = None if w is None else _f64(w)
        z = rope.norm(_f64(x), w, 1e-5)
        out[n] = rope.rope(z, p, freq, layout, m), (2.0 ** -20 + 2.0 ** -19) * m * _size(z, rot, layout)
    _check(qo, *out["q"], BF, "q")
    ko, vo = (torch.full((B, T, Hkv, D), float("nan"), dtype=BF, device=DEV) for _ in range(2))
    qsa.qsa_qk_norm_rope(q, k, qo, ko, f, v=v, v_out=vo, **kwargs)  # rows, no caches
    _check(ko, *out["k"], BF, "k")
    assert torch.equal(vo, v)
    for b in range(B):  # the caches hold the same rows, and nothing else changed
        on = slot[b] >= 0
        k0[b, slot[b][on]], v0[b, slot[b][on]] = ko[b][on], v[b][on]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    kk = torch.empty_like(ko)
    qsa.qsa_qk_norm_rope(q, k, qo, kk, f, **kwargs)  # without values
    assert torch.equal(kk, ko)


def test_norm_rope_slot_out_of_range_is_recorded_and_not_written():
    g = _gen(3)
    q, k = _randn(g, 2, 3, 4, 64), _randn(g, 2, 3, 1, 64)
    f, _ = _freq(64)
    kc = torch.zeros(2, 8, 1, 64, dtype=BF, device=DEV)
    qo, ws = torch.empty_like(q), qsa.workspace(256, DEV)
    slot = torch.tensor([[0, 8, 1], [-5, 1 << 40, 7]], device=DEV)
    qsa.qsa_qk_norm_rope(q, k, qo, kc, f, slot=slot, ws=ws)
    assert qsa.qsa_check_device_status(ws) == 7
    assert kc.abs().sum((2, 3)).gt(0).tolist() == [[True, True] + [False] * 6,
                                                   [False] * 7 + [True]]
    qsa.qsa_qk_norm_rope(q, k, qo, kc, f, slot=slot.clamp(0, 7), ws=ws)
    assert qsa.qsa_check_device_status(ws) == 0


@pytest.mark.parametrize("Hq,Hkv,D,rot", [(16, 2, 128, 128), (5, 3, 64, 24), (4, 1, 256, 256)])
def test_rows_do_not_depend_on_their_batch(Hq, Hkv, D, rot):
    """A token's rows have the same bits in a batch of thousands (many rounds of the GPU, several
    rows at a time) and in one of dozens."""
    g = _gen(D + rot)
    B, T, cut = 2, 9001, 60
    packed = _randn(g, B, T, (Hq + 2 * Hkv) * D)
    part = lambda x: (x[..., :Hq * D].unflatten(-1, (Hq, D)),
                      x[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D)),
                      x[..., (Hq + Hkv) * D:].unflatten(-1, (Hkv, D)))
    f, m = _freq(rot, "by-parts")
    qw, kw = _weights(g, D, (True, True))
    pos = torch.randint(0, 1 << 20, (B, T), generator=g, device=DEV)
    d = {t: (_randn(g, B, T, Hq, D, dtype=t), _randn(g, B, T, Hkv, D, dtype=t)) for t in (BF, F32)}

    def run(lo, hi):
        p = pos[:, lo:hi].contiguous()
        q, k, v = part(packed[:, lo:hi].contiguous())
        kwargs = dict(q_weight=qw, k_weight=kw, pos=p, mscale=m)
        out = [torch.empty(B, hi - lo, h, D, dtype=BF, device=DEV) for h in (Hq, Hkv, Hkv)]
        qsa.qsa_qk_norm_rope(q, k, out[0], out[1], f, v=v, v_out=out[2], **kwargs)
        for t, (dq, dk) in d.items():
            a, b = dq[:, lo:hi].contiguous(), dk[:, lo:hi].contiguous()
            out += [torch.empty_like(a), torch.empty_like(b), torch.empty_like(a)]
            qsa.qsa_qk_norm_rope_backward(a, b, q, k, out[-3], out[-2], f, **kwargs)
            qsa.qsa_rope(a, out[-1], f, pos=p, mscale=m, transpose=True)
        return out

    whole = run(0, T)
    for lo in (0, 4000, T - cut):
        for a, b in zip(whole, run(lo, lo + cut)):
            assert torch.equal(a[:, lo:lo + cut], b)


def test_refusals():
    g = _gen(2)
    q, k = _randn(g, 2, 3, 4, 64), _randn(g, 2, 3, 2, 64)
    f, _ = _freq(64)
    w, pos = torch.ones(64, device=DEV), torch.zeros(2, 3, dtype=torch.int64, device=DEV)
    e = torch.empty_like
    for error, call in (
            (TypeError, lambda: qsa.qsa_rope(q, e(q).float(), f)),
            (ValueError, lambda: qsa.qsa_rope(q, e(q)[:, :2], f)),
            (TypeError, lambda: qsa.qsa_rope(q, e(q), f.float())),
            (ValueError, lambda: qsa.qsa_rope(q, e(q), f.cpu())),
            (ValueError, lambda: qsa.qsa_rope(q, e(q), f, layout="pairs")),
            (ValueError, lambda: qsa.qsa_rope(q.transpose(1, 2), e(q).transpose(1, 2), f)),
            (ValueError, lambda: qsa.qsa_rope(q, e(q), f, pos=pos[:1])),
            (qsa.QSAError, lambda: qsa.qsa_rope(q, e(q), f, mscale=float("inf"))),
            (qsa.QSAError, lambda: qsa.qsa_rope(q, e(q), f[:3])),
            (ValueError, lambda: qsa.qsa_qk_norm_rope(q, k, e(q), e(k), f, v=k)),
            (ValueError, lambda: qsa.qsa_qk_norm_rope(q, k, e(q), e(k)[:, :2], f)),
            (TypeError, lambda: qsa.qsa_qk_norm_rope(q, k, e(q), e(k), f, q_weight=w.double())),
            (ValueError, lambda: qsa.qsa_qk_norm_rope(q, k, e(q), e(k), f, q_weight=w[:32])),
            (ValueError, lambda: qsa.qsa_qk_norm_rope(q, k, e(q), e(k), f, ws=qsa.workspace(128))),
            (TypeError, lambda: qsa.qsa_qk_norm_rope(q, k, e(q), e(k), f, slot=pos.int())),
            (qsa.QSAError, lambda: qsa.qsa_qk_norm_rope(q, k, e(q), e(k), f, eps=-1.0)),
            (TypeError, lambda: qsa.qsa_qk_norm_rope_backward(q, k.float(), q, k, e(q), e(k), f)),
            (qsa.QSAError, lambda: qsa.qsa_qk_norm_rope_backward(
                q, k, q, k, e(q), e(k), f, q_weight=w, dq_weight=e(w)))):  # no workspace
        with pytest.raises(error):
            call()


def test_norm_of_zero_and_huge_rows():
    """A row of zeros stays zero (eps > 0); rows of 2^60 keep their norm: their squares
    (2^120) and sums stay below fp32's range."""
    f, _ = _freq(32)
    x = torch.zeros(1, 3, 2, 64, dtype=BF, device=DEV)
    x[0, 1] = 2.0 ** 60
    x[0, 2] = 2.0 ** -70  # squares vanish: x / sqrt(eps)
    w = torch.ones(64, device=DEV)
    qo, ko = torch.empty_like(x), torch.empty_like(x)
    qsa.qsa_qk_norm_rope(x, x, qo, ko, f, q_weight=w, k_weight=w, eps=1e-6)
    assert bool((qo[0, 0] == 0).all())
    for x_, y, t in ((x[:, 1:], qo[:, 1:], "q"), (x[:, 1:], ko[:, 1:], "k")):
        z = rope.norm(_f64(x_), _f64(w), 1e-6)
        ref = rope.rope(z, [[1, 2]], _f64(f))
        _check(y, ref, 2.0 ** -18 * _size(z, 32, "half"), BF, t)


@pytest.mark.parametrize("types", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot", CASES)
def test_norm_rope_backward(B, T, Hq, Hkv, D, rot, layout, types):
    g = _gen(B * T + D + rot + 1)
    td, tx = types
    q, k = _randn(g, B, T, Hq, D), _randn(g, B, T, Hkv, D)
    d_q, d_k = _randn(g, B, T, Hq, D, dtype=td), _randn(g, B, T, Hkv, D, dtype=td)
    f, m = _freq(rot, "by-parts") if rot else (None, 1.0)
    freq = [] if f is None else _f64(f)
    pos = torch.randint(0, 1 << 18, (B, T), generator=g, device=DEV)
    ws = qsa.workspace(qsa.qsa_qk_norm_rope_backward_workspace_size(B, T, Hq, Hkv, D), DEV)
    for which in ((True, True), (False, True)):
        qw, kw = _weights(g, D, which)
        dq = torch.full((B, T, Hq, D), float("nan"), dtype=tx, device=DEV)
        dk = torch.full((B, T, Hkv, D), float("nan"), dtype=tx, device=DEV)
        dqw = None if qw is None else torch.full((D,), float("nan"), device=DEV)
        dkw = torch.full((D,), float("nan"), device=DEV)
        call = lambda dq, dk, dqw, dkw: qsa.qsa_qk_norm_rope_backward(
            d_q, d_k, q, k, dq, dk, f, ws, q_weight=qw, k_weight=kw, dq_weight=dqw, dk_weight=dkw,
            eps=1e-5, pos=pos, layout=layout, mscale=m)
        call(dq, dk, dqw, dkw)
        for n, d, x, w, dx, dw in (("q", d_q, q, qw, dq, dqw), ("k", d_k, k, kw, dk, dkw)):
            w = None if w is None else _f64(w)
            ref, refw = rope.norm_rope_grad(_f64(d), _f64(x), w, 1e-5, pos.cpu().numpy(), freq,
                                            layout, m)
            size = m * _size(_f64(d), rot, layout)  # of dz
            if w is None:
                _check(dx, ref, 2.0 ** -20 * size, tx, n)
                continue
            r = 1 / np.sqrt((_f64(x) ** 2).mean(-1, keepdims=True) + 1e-5)
            xh, u = np.abs(_f64(x) * r), np.abs(w) * size
            _check(dx, ref, 2.0 ** -17 * r * (u + xh * (u * xh).mean(-1, keepdims=True)), tx, n)
            _check(dw, refw, 2.0 ** -14 * (size * xh).sum((0, 1, 2)), F32, n + " weight")
        a, b = torch.empty_like(dq), torch.empty_like(dk)
        call(a, b, None, torch.empty_like(dkw))  # one weight gradient, the same bits
        assert torch.equal(a, dq) and torch.equal(b, dk)
        again = torch.empty_like(dkw)
        call(a, b, dqw, again)
        assert torch.equal(again, dkw)


def test_norm_rope_backward_against_differences():
    """A directional difference of the fp64 forward along a random direction."""
    g = _gen(11)
    q, k = _randn(g, 2, 11, 4, 64), _randn(g, 2, 11, 2, 64)
    d_q, d_k = _randn(g, 2, 11, 4, 64, dtype=F32), _randn(g, 2, 11, 2, 64, dtype=F32)
    qw, kw = _weights(g, 64, (True, True))
    f, m = _freq(32, "by-parts")
    dq, dk = torch.empty_like(d_q), torch.empty_like(d_k)
    dqw, dkw = torch.empty_like(qw), torch.empty_like(kw)
    ws = qsa.workspace(qsa.qsa_qk_norm_rope_backward_workspace_size(2, 11, 4, 2, 64), DEV)
    qsa.qsa_qk_norm_rope_backward(d_q, d_k, q, k, dq, dk, f, ws, q_weight=qw, k_weight=kw,
                                  dq_weight=dqw, dk_weight=dkw, layout="interleaved", mscale=m)
    pos = np.tile(np.arange(11), (2, 1))
    rng = np.random.default_rng(0)
    for x, w, d, dx, dw in ((q, qw, d_q, dq, dqw), (k, kw, d_k, dk, dkw)):
        x, w, d = _f64(x), _f64(w), _f64(d)
        ex, ew = rng.normal(size=x.shape), rng.normal(size=w.shape)
        loss = lambda h: (rope.norm_rope(x + h * ex, w + h * ew, 1e-6, pos, _f64(f), "interleaved",
                                         m) * d).sum()
        h = 1e-5
        want = (loss(h) - loss(-h)) / (2 * h)  # off by about h^2 of its third derivative
        got = (_f64(dx) * ex).sum() + (_f64(dw) * ew).sum()
        scale = np.abs(_f64(dx) * ex).sum() + np.abs(_f64(dw) * ew).sum()
        assert abs(got - want) <= 2.0 ** -17 * scale


def test_empty_calls():
    f, _ = _freq(64)
    e = torch.empty(2, 0, 4, 64, dtype=BF, device=DEV)
    qsa.qsa_rope(e, e, f)
    k = torch.empty(2, 0, 1, 64, dtype=BF, device=DEV)
    cache = torch.ones(2, 5, 1, 64, dtype=BF, device=DEV)
    qsa.qsa_qk_norm_rope(e, k, e, cache, f, slot=torch.empty(2, 0, dtype=torch.int64, device=DEV))
    assert bool((cache == 1).all())
    w = torch.ones(64, device=DEV)
    dqw, dkw = torch.full((64,), 3.0, device=DEV), torch.full((64,), 3.0, device=DEV)
    ws = qsa.workspace(qsa.qsa_qk_norm_rope_backward_workspace_size(2, 0, 4, 1, 64), DEV)
    qsa.qsa_qk_norm_rope_backward(e, k, e, k, e, k, f, ws, q_weight=w, k_weight=w, dq_weight=dqw,
                                  dk_weight=dkw)
    assert bool((dqw == 0).all()) and bool((dkw == 0).all())


def test_captured_and_replayed_with_new_inputs():
    g = _gen(13)
    q, k = _randn(g, 4, 6, 8, 128), _randn(g, 4, 6, 2, 128)
    f, _ = _freq(128)
    w = torch.ones(128, device=DEV)
    d_q, d_k = _randn(g, 4, 6, 8, 128, dtype=F32), _randn(g, 4, 6, 2, 128, dtype=F32)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    dq, dk, dqw, dkw = (torch.empty_like(t) for t in (d_q, d_k, w, w))
    ws = qsa.workspace(qsa.qsa_qk_norm_rope_backward_workspace_size(4, 6, 8, 2, 128), DEV)

    def step():
        qsa.qsa_qk_norm_rope(q, k, qo, ko, f, q_weight=w, k_weight=w)
        qsa.qsa_qk_norm_rope_backward(d_q, d_k, q, k, dq, dk, f, ws, q_weight=w, k_weight=w,
                                      dq_weight=dqw, dk_weight=dkw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    q.copy_(_randn(g, 4, 6, 8, 128))
    d_q.copy_(_randn(g, 4, 6, 8, 128, dtype=F32))
    graph.replay()
    got = [t.clone() for t in (qo, ko, dq, dk, dqw, dkw)]
    step()
    for a, b in zip(got, (qo, ko, dq, dk, dqw, dkw)):
        assert torch.equal(a, b)
