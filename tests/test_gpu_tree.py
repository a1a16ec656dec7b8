"""GPU parity of qsa_dense_tree_decode and qsa_sparse_tree_decode against the fp64
oracle (oracle/tree.py), through the C ABI.

Bounds, derived (eps32 = 2^-24, bf16 half a step 2^-8):
  * a logit is D exact products summed in fp32, in any order, scaled: off by at most
    dx = 2 D eps32 scale sum |q k| (a factor 2 for sums that truncate) plus 2^-20, the
    base-2 exponent's rounding at logits up to 16.
  * lse moves by at most the largest dx, and by the sum's own rounding and log2's
    (2^-20 + 2^-22 |lse|).
  * the probabilities are rounded to bf16 for the product with v (2^-8) and are off by
    2 dx: o moves by at most (2^-8 + 2 dx + 2^-18) sum p |v|, and is rounded: 2^-8 |o|.
"""
import numpy as np
import pytest
import torch

import block_sparse_long_10_b200 as qsa
from oracle import rope as rope_oracle
from oracle import tree

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _f64(t):
    return t.detach().double().cpu().numpy()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _parents(kind, B, N, seed):
    r = np.random.default_rng(seed)
    i = np.arange(N)
    if kind == "chain":
        p = np.tile(i - 1, (B, 1))
    elif kind == "star":
        p = np.full((B, N), -1)
    else:
        p = np.stack([[r.integers(-1, j) for j in range(N)] for _ in range(B)])
    return torch.tensor(p, dtype=torch.int32, device=DEV)


def _make(B, N, Hq, Hkv, D, prefix, drafts, seed, kind="random", L=None, q_scale=1.5):
    g = _gen(seed)
    L = max(max(prefix) + N, 1) + 3 if L is None else L
    x = dict(q=(q_scale * torch.randn(B, N, Hq, D, generator=g, device=DEV)).to(BF),
             k=torch.full((B, L, Hkv, D), float("nan"), dtype=BF, device=DEV),
             v=torch.full((B, L, Hkv, D), float("nan"), dtype=BF, device=DEV))
    for b, (P, n) in enumerate(zip(prefix, drafts)):  # rows past the sequence hold NaN
        x["k"][b, :P + n] = torch.randn(P + n, Hkv, D, generator=g, device=DEV).to(BF)
        x["v"][b, :P + n] = torch.randn(P + n, Hkv, D, generator=g, device=DEV).to(BF)
    x["seqlens"] = torch.tensor([p + n for p, n in zip(prefix, drafts)], dtype=torch.int32,
                                device=DEV)
    x["n_draft"] = torch.tensor(drafts, dtype=torch.int32, device=DEV)
    x["parent"] = _parents(kind, B, N, seed)
    return x


def _sel(prefix, N, kb, seed):
    """Random selections in random order, entries out of range among them."""
    r = np.random.default_rng(seed)
    out = np.full((len(prefix), N, kb), -1, np.int32)
    for b, P in enumerate(prefix):
        for i in range(N):
            n = int(r.integers(0, min(kb, P // 4) + 1))
            row = list(r.permutation(P // 4)[:n])
            row += [int(r.choice([-1, -7, P // 4, P // 4 + 5, 2 ** 30])) for _ in range(kb - n)]
            out[b, i] = r.permutation(row)
    return torch.tensor(out, device=DEV)


def _run(x, sel=None, budget=None, scale=None, n_draft=True, ws=None):
    B, N, Hq, D = x["q"].shape
    Hkv = x["k"].shape[2]
    o = torch.full_like(x["q"], 7.0)
    lse = torch.full((B, N, Hq), 7.0, device=DEV)
    kw = dict(n_draft=x["n_draft"] if n_draft else None, scale=scale, lse=lse)
    if sel is None:
        ws = ws if ws is not None else qsa.workspace(
            qsa.qsa_dense_tree_decode_workspace_size(B, N, Hq, Hkv, D), DEV)
        qsa.qsa_dense_tree_decode(x["q"], x["k"], x["v"], x["seqlens"], x["parent"], o, ws, **kw)
    else:
        ws = ws if ws is not None else qsa.workspace(
            qsa.qsa_sparse_tree_decode_workspace_size(B, N, Hq, D, 4, budget), DEV)
        qsa.qsa_sparse_tree_decode(x["q"], x["k"], x["v"], x["seqlens"], sel, x["parent"], o, ws,
                                   budget=budget, **kw)
    return o, lse, ws


def _check(x, o, lse, prefix, drafts, sel=None, scale=None, rows=None):
    B, N, Hq, D = x["q"].shape
    scale = D ** -0.5 if scale is None else scale
    q, parent, o_, lse_ = _f64(x["q"]), x["parent"].cpu().numpy(), _f64(o), _f64(lse)
    sel = None if sel is None else sel.cpu().numpy()
    for b, (P, n) in enumerate(zip(prefix, drafts)):
        k, v = _f64(x["k"][b, :P + n]), _f64(x["v"][b, :P + n])
        for i in range(N):
            if i >= n:  # left as they were
                assert (o_[b, i] == 7).all() and (lse_[b, i] == 7).all(), (b, i)
                continue
            if rows is not None and i not in rows:
                continue
            at = tree.tokens(P, i, parent[b], None if sel is None else sel[b, i])
            ro, rl, mass, size = tree.attend(q[b, i], k, v, at, scale)
            dx = 2 * D * 2.0 ** -24 * size + 2.0 ** -20
            off = np.abs(lse_[b, i] - rl) - dx - 2.0 ** -20 - 2.0 ** -22 * np.abs(rl)
            assert (off <= 0).all(), (b, i, "lse", float(off.max()))
            bound = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * dx[:, None] + 2.0 ** -18) * mass
            off = np.abs(o_[b, i] - ro) - bound
            assert np.isfinite(o_[b, i]).all() and (off <= 0).all(), (b, i, "o", float(off.max()))


SHAPES = [
    # B, N, Hq, Hkv, D, prefix lengths, drafts
    (1, 1, 1, 1, 64, [0], [1]),
    (1, 1, 16, 2, 128, [1], [1]),
    (3, 5, 4, 1, 64, [127, 128, 129], [5, 3, 1]),
    (4, 7, 16, 2, 128, [0, 3, 400, 1001], [7, 0, 5, 7]),
    (2, 16, 8, 1, 128, [255, 513], [16, 9]),
    (2, 17, 8, 1, 128, [640, 131], [17, 16]),
    (1, 33, 32, 4, 64, [700], [33]),
    (2, 64, 16, 2, 128, [300, 77], [64, 33]),
    (1, 100, 4, 4, 128, [515], [100]),
    (1, 256, 8, 1, 64, [260], [256]),
    (1, 256, 2, 2, 128, [5], [255]),
    (5, 3, 2, 1, 128, [2000, 0, 64, 1, 1500], [3, 3, 0, 1, 2]),
]


@pytest.mark.parametrize("kind", ["random", "chain", "star"])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,prefix,drafts", SHAPES)
def test_dense_tree(B, N, Hq, Hkv, D, prefix, drafts, kind):
    x = _make(B, N, Hq, Hkv, D, prefix, drafts, seed=N + D, kind=kind)
    o, lse, ws = _run(x)
    assert qsa.qsa_check_device_status(ws) == 0
    _check(x, o, lse, prefix, drafts, rows=set(range(0, N, max(1, N // 9))) | {N - 1})


@pytest.mark.parametrize("kind", ["random", "chain"])
@pytest.mark.parametrize("budget", [4, 64, 512])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,prefix,drafts", SHAPES)
def test_sparse_tree(B, N, Hq, Hkv, D, prefix, drafts, budget, kind):
    x = _make(B, N, Hq, Hkv, D, prefix, drafts, seed=N + D + 1, kind=kind)
    sel = _sel(prefix, N, budget // 4, seed=N)
    o, lse, ws = _run(x, sel, budget)
    assert qsa.qsa_check_device_status(ws) == 0
    _check(x, o, lse, prefix, drafts, sel, rows=set(range(0, N, max(1, N // 9))) | {N - 1})


def test_sparse_tree_full_budget_and_shared_selection():
    prefix, drafts = [9001, 4096], [6, 6]
    x = _make(2, 6, 16, 2, 128, prefix, drafts, seed=5)
    sel = _sel(prefix, 6, 1024, seed=6)
    o, lse, _ = _run(x, sel, 4096)
    _check(x, o, lse, prefix, drafts, sel)
    one = sel[:, :1].expand(2, 6, 1024)  # a row stride of 0
    o, lse, _ = _run(x, one, 4096)
    _check(x, o, lse, prefix, drafts, one)
    turned = sel.transpose(0, 1).contiguous().transpose(0, 1)  # [N,B,kb] in memory
    a, b = _run(x, sel, 4096), _run(x, turned, 4096)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_sparse_tree_of_every_block_is_dense():
    prefix, drafts = [777, 130], [9, 4]
    x = _make(2, 9, 8, 2, 64, prefix, drafts, seed=9)
    sel = torch.arange(256, dtype=torch.int32, device=DEV).expand(2, 9, 256)
    o, lse, _ = _run(x, sel, 1024)
    _check(x, o, lse, prefix, drafts)  # against the dense definition


def test_single_draft_is_dense_decode():
    prefix = [0, 5, 1023, 300]
    x = _make(4, 1, 16, 2, 128, prefix, [1] * 4, seed=2, L=1024)
    o, lse, _ = _run(x, n_draft=False)
    x["k"].nan_to_num_(0.0)
    x["v"].nan_to_num_(0.0)
    o2, lse2 = torch.empty_like(x["q"][:, 0]), torch.empty(4, 16, device=DEV)
    ws = qsa.workspace(qsa.qsa_dense_gqa_decode_workspace_size(4, 1024, 16, 128), DEV)
    qsa.qsa_dense_gqa_decode(x["q"][:, 0].contiguous(), x["k"], x["v"], x["seqlens"], o2, ws,
                             lse=lse2)
    # both are within the module's bounds of one value; logits here are under 16, p |v| under 4
    assert float((o[:, 0].float() - o2.float()).abs().max()) <= 2 * (2 ** -8 * 4 + 2 ** -8 * 4)
    assert float((lse[:, 0] - lse2).abs().max()) <= 2 * (2 * 128 * 2 ** -24 * 32 + 2 ** -18)


@pytest.mark.parametrize("sparse", [False, True])
def test_other_branches_may_hold_anything(sparse):
    """Infinities and NaN in a draft's rows reach that draft's descendants only."""
    prefix, drafts, N = [203], [12], 12
    x = _make(1, N, 16, 2, 128, prefix, drafts, seed=4)
    # two branches: even drafts hang on even ones, odd on odd
    x["parent"] = torch.tensor([[j - 2 if j >= 2 else -1 for j in range(N)]], dtype=torch.int32,
                               device=DEV)
    sel = _sel(prefix, N, 16, 3) if sparse else None
    good = _run(x, sel, 64)
    for bad in (float("nan"), float("inf"), float("-inf")):
        y = {n: t.clone() for n, t in x.items()}
        y["k"][0, 203 + 3] = bad
        y["v"][0, 203 + 3] = bad
        o, lse, _ = _run(y, sel, 64)
        clean = [j for j in range(N) if j % 2 == 0 or j < 3]
        assert torch.equal(o[0, clean], good[0][0, clean])
        assert torch.equal(lse[0, clean], good[1][0, clean])
        assert not bool(torch.isfinite(o[0, 3].float()).all())


@pytest.mark.parametrize("B,N,Hq,Hkv,D,top", [(1, 9, 8, 2, 64, 250), (2, 40, 16, 2, 128, 380),
                                              (9, 64, 16, 2, 128, 120), (1, 256, 8, 1, 64, 77)])
def test_infinite_values_reach_their_descendants_only(B, N, Hq, Hkv, D, top):
    """One infinite value of a draft: that dim of its descendants' heads becomes infinite (their
    weight on the draft is not zero), every other bit stays."""
    prefix, drafts = [top - 5 * b for b in range(B)], [N - b % 3 for b in range(B)]
    x = _make(B, N, Hq, Hkv, D, prefix, drafts, seed=41)
    good = _run(x)
    for j, g, d, bad in ((N // 3, Hkv - 1, D - 1, float("inf")), (0, 0, 3, float("-inf"))):
        y = dict(x, v=x["v"].clone())
        for b in range(B):
            y["v"][b, prefix[b] + j, g, d] = bad
        o, lse, ws = _run(y)
        assert qsa.qsa_check_device_status(ws) == 0
        want = good[0].clone()
        G = Hq // Hkv
        for b in range(B):
            for i in range(drafts[b]):
                if prefix[b] + j in tree.tokens(prefix[b], i, x["parent"][b].tolist()):
                    want[b, i, g * G:(g + 1) * G, d] = bad
        assert torch.equal(o, want) and torch.equal(lse, good[1])


def test_nan_in_a_row_of_the_prefix_reaches_every_row():
    """A key that is not a number is in every row's sum."""
    x = _make(1, 6, 8, 1, 128, [700], [6], seed=43)
    for at in (0, 130, 699):
        y = dict(x, k=x["k"].clone())
        y["k"][0, at, 0, 5] = float("nan")
        o, lse, _ = _run(y)
        assert bool(o.isnan().all()) and bool(lse.isnan().all())
    y = dict(x, k=x["k"].clone())  # an infinite score: inf - inf
    y["k"][0, 200, 0] = float("inf")
    y["q"] = x["q"].abs()
    o, lse, _ = _run(y)
    assert bool(o.isnan().all())


def test_refusals():
    x = _make(2, 4, 8, 2, 64, [30, 40], [4, 4], seed=44)
    sel = _sel([30, 40], 4, 16, 1)
    ws = qsa.workspace(qsa.qsa_sparse_tree_decode_workspace_size(2, 4, 8, 64, 4, 64), DEV)
    ws = qsa.workspace(max(ws.numel(), qsa.qsa_dense_tree_decode_workspace_size(2, 4, 8, 2, 64)),
                       DEV)
    base = dict(q=x["q"], k_cache=x["k"], v_cache=x["v"], seqlens=x["seqlens"],
                parent=x["parent"], o=torch.empty_like(x["q"]), ws=ws)
    bad = [(TypeError, dict(q=x["q"].float())), (TypeError, dict(seqlens=x["seqlens"].long())),
           (TypeError, dict(k_cache=None)), (ValueError, dict(v_cache=x["v"][:, :-1])),
           (ValueError, dict(parent=x["parent"][:, :3])), (ValueError, dict(o=base["o"][:1])),
           (ValueError, dict(parent=x["parent"].T.contiguous().T)), (ValueError, dict(q=x["q"][0])),
           (ValueError, dict(seqlens=x["seqlens"].cpu())), (qsa.QSAError, dict(ws=None)),
           (qsa.QSAError, dict(ws=ws[:256])), (qsa.QSAError, dict(scale=float("nan"))),
           (ValueError, dict(n_draft=x["n_draft"][:1])), (TypeError, dict(lse=base["o"]))]
    for call, more, extra in (
            (qsa.qsa_dense_tree_decode, {}, []),
            (qsa.qsa_sparse_tree_decode, dict(sel=sel, budget=64),
             [(ValueError, dict(sel=sel[:, :, :15])), (TypeError, dict(sel=sel.long())),
              (ValueError, dict(sel=sel.transpose(1, 2).contiguous().transpose(1, 2))),
              (ValueError, dict(budget=60)), (qsa.QSAError, dict(budget=64, r=8, sel=sel[:, :, :8]))])):
        call(**{**base, **more})
        for error, kw in bad + extra:
            with pytest.raises(error):
                call(**{**base, **more, **kw})


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0])
def test_scales(scale):
    """Any finite scale; at 1.0 logits reach beyond 100 and the softmax is nearly one-hot
    (the base-2 exponent's rounding, 2^-24 of it, is within dx's first term there)."""
    prefix, drafts = [300, 11], [5, 5]
    x = _make(2, 5, 8, 1, 128, prefix, drafts, seed=8)
    for sel in (None, _sel(prefix, 5, 128, 4)):
        o, lse, _ = _run(x, sel, 512, scale=scale)
        _check(x, o, lse, prefix, drafts, sel, scale=scale)


@pytest.mark.parametrize("B,N,Hq,Hkv,D,top", [(40, 5, 8, 4, 128, 2600), (24, 40, 32, 4, 128, 2500),
                                              (60, 3, 2, 2, 64, 5000), (16, 200, 8, 1, 64, 3000)])
def test_long_runs(B, N, Hq, Hkv, D, top):
    """More tiles (and stages of selections) than SMs by far: each SM's ring of copies wraps
    several times, goes over from sequence to sequence, and meets drafts on the way."""
    prefix = [top - (37 * b) % 1111 for b in range(B)]
    drafts = [N - (b % 3) * (N // 4) for b in range(B)]
    x = _make(B, N, Hq, Hkv, D, prefix, drafts, seed=31)
    sel = _sel(prefix, N, 512, 32)
    for s in (None, sel):
        first = _run(x, s, 2048)
        assert qsa.qsa_check_device_status(first[2]) == 0
        some = sorted({0, 1, B // 2, B - 1})
        part = {n: t[some] for n, t in x.items()}
        _check(part, first[0][some], first[1][some], [prefix[b] for b in some],
               [drafts[b] for b in some], None if s is None else s[some], rows={0, N // 2, N - 1})
        for _ in range(5):  # all rows, whatever the timing
            again = _run(x, s, 2048, ws=first[2])
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("B,N,Hq,Hkv,D,prefix", [
    (2, 14, 16, 2, 128, [9001, 4]), (4, 12, 16, 2, 64, [3000, 1, 2999, 130]),
    (1, 128, 8, 1, 128, [20000]), (3, 64, 16, 2, 128, [7000, 6000, 5]), (1, 256, 32, 4, 64, [4100])])
def test_many_parts_of_a_row(B, N, Hq, Hkv, D, prefix):
    """Long prefixes, few units: each row's parts come from many SMs, for one to a few
    thousand (row, head) pairs."""
    drafts = [N - b for b in range(B)]
    x = _make(B, N, Hq, Hkv, D, prefix, drafts, seed=71)
    o, lse, ws = _run(x)
    assert qsa.qsa_check_device_status(ws) == 0
    rows = {0, N // 2, N - B, N - 1}
    _check(x, o, lse, prefix, drafts, rows=rows)
    sel = _sel(prefix, N, 512, 72)
    o, lse, ws = _run(x, sel, 2048)
    assert qsa.qsa_check_device_status(ws) == 0
    _check(x, o, lse, prefix, drafts, sel, rows=rows)


def test_growing_logits_move_the_running_maximum():
    """Keys that grow along the cache: the maximum moves in every tile."""
    prefix, drafts = [1500], [4]
    x = _make(1, 4, 8, 1, 128, prefix, drafts, seed=10)
    ramp = torch.linspace(0.05, 3.0, 1504, device=DEV)[None, :, None, None]
    for order in (ramp, ramp.flip(1)):
        y = dict(x, k=x["k"].clone())
        y["k"][:, :1504] = (x["q"].mean((1, 2))[:, None, None] * 4 * order).to(BF) \
            + 0.1 * x["k"][:, :1504]
        o, lse, _ = _run(y)
        _check(y, o, lse, prefix, drafts)


@pytest.mark.parametrize("sparse", [False, True])
def test_bad_lengths_and_parents_are_recorded(sparse):
    prefix, drafts = [40, 40, 40, 40], [3, 3, 3, 3]
    x = _make(4, 3, 4, 1, 64, prefix, drafts, seed=1, L=43)
    sel = _sel(prefix, 3, 16, 1) if sparse else None
    good = _run(x, sel, 64)
    for name, value in (("seqlens", 2), ("seqlens", 44), ("seqlens", -1), ("n_draft", 4),
                        ("n_draft", -1), ("seqlens", 2 ** 31 - 1), ("n_draft", -2 ** 31)):
        y = dict(x, **{name: x[name].clone()})
        y[name][1] = value
        o, lse, ws = _run(y, sel, 64)
        assert qsa.qsa_check_device_status(ws) == 7, (name, value)
        assert bool((o[1] == 0).all()) and bool((lse[1] == float("-inf")).all())
        for b in (0, 2, 3):
            assert torch.equal(o[b], good[0][b]) and torch.equal(lse[b], good[1][b])
    for value in (-2, 1, 2, 2 ** 30):
        y = dict(x, parent=x["parent"].clone())
        y["parent"][2, 1] = value
        o, lse, ws = _run(y, sel, 64)
        assert qsa.qsa_check_device_status(ws) == 7, value
        y["parent"][2, 1] = -1  # such a chain ends there
        ref = _run(y, sel, 64)
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_nothing_to_attend_to_is_left_alone():
    x = _make(2, 4, 4, 1, 64, [9, 0], [0, 0], seed=3)
    o, lse, ws = _run(x)
    assert bool((o == 7).all()) and bool((lse == 7).all())
    assert qsa.qsa_check_device_status(ws) == 0


def test_offsets_past_32_bits():
    """The last sequence's rows lie more than 2^32 bytes and 2^31 elements in."""
    L, prefix, drafts = 1500000, [17, 0, 0, 2049], [3, 0, 0, 5]
    g = _gen(12)
    B, N, Hq, Hkv, D = 4, 5, 8, 4, 128
    x = dict(q=torch.randn(B, N, Hq, D, generator=g, device=DEV).to(BF),
             k=torch.empty(B, L, Hkv, D, dtype=BF, device=DEV),
             v=torch.empty(B, L, Hkv, D, dtype=BF, device=DEV))
    for b, (P, n) in enumerate(zip(prefix, drafts)):
        for t in (x["k"], x["v"]):
            t[b, :P + n] = torch.randn(P + n, Hkv, D, generator=g, device=DEV).to(BF)
    assert 3 * L * Hkv * D > 2 ** 31
    x["seqlens"] = torch.tensor([p + n for p, n in zip(prefix, drafts)], dtype=torch.int32,
                                device=DEV)
    x["n_draft"] = torch.tensor(drafts, dtype=torch.int32, device=DEV)
    x["parent"] = _parents("random", B, N, 3)
    for sel in (None, _sel(prefix, N, 128, 4)):
        o, lse, _ = _run(x, sel, 512)
        _check(x, o, lse, prefix, drafts, sel)
    f, _ = qsa.qsa_rope_frequencies(1e4, 128, device=DEV)
    slot = torch.full((B, 1), L - 1, dtype=torch.int64, device=DEV)
    q, k = x["q"][:, :1].contiguous(), torch.randn(B, 1, Hkv, D, generator=g, device=DEV).to(BF)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    qsa.qsa_qk_norm_rope(q, k, qo, x["k"], f, v=k, v_out=x["v"], slot=slot, pos=slot)
    qsa.qsa_qk_norm_rope(q, k, qo, ko, f, pos=slot)
    assert torch.equal(x["k"][:, -1:], ko) and torch.equal(x["v"][:, -1:], k)


@pytest.mark.parametrize("sparse", [False, True])
def test_repeats_and_replays_to_the_same_bits(sparse):
    prefix, drafts = [900, 333], [8, 6]
    x = _make(2, 8, 16, 2, 128, prefix, drafts, seed=6)
    sel = _sel(prefix, 8, 64, 2) if sparse else None
    first = _run(x, sel, 256)
    for _ in range(3):
        o, lse, _ = _run(x, sel, 256, ws=first[2])  # a used workspace
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    B, N, Hq, D = x["q"].shape
    o, lse = torch.full_like(x["q"], 7.0), torch.full((B, N, Hq), 7.0, device=DEV)

    def step():
        if sparse:
            qsa.qsa_sparse_tree_decode(x["q"], x["k"], x["v"], x["seqlens"], sel, x["parent"], o,
                                       first[2], n_draft=x["n_draft"], budget=256, lse=lse)
        else:
            qsa.qsa_dense_tree_decode(x["q"], x["k"], x["v"], x["seqlens"], x["parent"], o,
                                      first[2], n_draft=x["n_draft"], lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # other lengths at replay: they live on the device
    x["seqlens"].copy_(torch.tensor([640, 12], dtype=torch.int32))
    x["n_draft"].copy_(torch.tensor([2, 8], dtype=torch.int32))
    o.fill_(7.0)
    lse.fill_(7.0)
    graph.replay()
    if sparse:
        sel = sel.clone()
    _check(x, o, lse, [638, 4], [2, 8], sel)


def test_on_a_given_stream_and_on_the_current_one():
    prefix, drafts = [900, 20], [5, 3]
    x = _make(2, 5, 8, 2, 64, prefix, drafts, seed=51)
    sel = _sel(prefix, 5, 64, 52)
    f, _ = qsa.qsa_rope_frequencies(1e4, 64, device=DEV)
    good = _run(x), _run(x, sel, 256)
    turned = torch.empty_like(x["q"])
    qsa.qsa_rope(x["q"], turned, f)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for given in (True, False):
        o, l = [torch.empty_like(x["q"]) for _ in range(3)], torch.empty(2, 5, 8, device=DEV)
        for t in o:
            t.fill_(7.0)
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(20000000)  # the current stream is busy
        kw = dict(stream=side) if given else {}
        with torch.cuda.stream(torch.cuda.current_stream() if given else side):
            qsa.qsa_dense_tree_decode(x["q"], x["k"], x["v"], x["seqlens"], x["parent"], o[0],
                                      good[0][2], n_draft=x["n_draft"], lse=l, **kw)
            qsa.qsa_sparse_tree_decode(x["q"], x["k"], x["v"], x["seqlens"], sel, x["parent"],
                                       o[1], good[1][2], n_draft=x["n_draft"], budget=256, **kw)
            qsa.qsa_rope(x["q"], o[2], f, **kw)
        side.synchronize()
        assert not torch.cuda.current_stream().query()  # nothing waited for it
        assert torch.equal(o[0], good[0][0]) and torch.equal(o[1], good[1][0])
        assert torch.equal(o[2], turned)
        torch.cuda.synchronize()


def test_two_calls_at_once():
    """Calls of two streams, each with its own workspace, share the GPU and no result."""
    cases = []
    for seed, prefix, drafts in ((81, [3000, 70], [9, 12]), (82, [40, 5000], [12, 2])):
        x = _make(2, 12, 16, 2, 128, prefix, drafts, seed=seed)
        sel = _sel(prefix, 12, 128, seed)
        cases.append((x, sel, _run(x), _run(x, sel, 512)))
    torch.cuda.synchronize()
    streams, results = [torch.cuda.Stream() for _ in cases], []
    for _ in range(10):
        for stream, (x, sel, dense, sparse) in zip(streams, cases):
            with torch.cuda.stream(stream):
                results.append((_run(x, ws=dense[2]), dense))
                results.append((_run(x, sel, 512, ws=sparse[2]), sparse))
    torch.cuda.synchronize()
    for got, good in results:
        assert torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])


def test_norm_rotate_select_attend_together():
    """A verification step as it is used: drafted tokens' projections are normed, rotated at
    prefix + depth and put into the caches at their rows; the indexer's queries are rotated,
    each draft selects its blocks; the tree attends over them."""
    g = _gen(21)
    B, N, Hq, Hkv, D, Hi, Di, budget = 2, 6, 16, 2, 128, 4, 64, 256
    kb, P, L = budget // 4, [1022, 513], 1056
    x = _make(B, N, Hq, Hkv, D, P, [N] * B, seed=22, L=L)
    for b in range(B):  # the drafts' rows are not there yet
        x["k"][b, P[b]:] = float("nan")
        x["v"][b, P[b]:] = float("nan")
    packed = torch.randn(B, N, (Hq + 2 * Hkv) * D, generator=g, device=DEV).to(BF)
    q = packed[..., :Hq * D].unflatten(-1, (Hq, D))
    k = packed[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    v = packed[..., (Hq + Hkv) * D:].unflatten(-1, (Hkv, D))
    w = 1 + 0.1 * torch.randn(D, generator=g, device=DEV)
    f, m = qsa.qsa_rope_frequencies(1e6, D, "by-parts", 4.0, 512.0, device=DEV)
    depth = torch.zeros(B, N, dtype=torch.int64)
    for b in range(B):
        for i, p in enumerate(x["parent"][b].tolist()):
            depth[b, i] = 0 if p < 0 else depth[b, p] + 1
    start = torch.tensor(P)[:, None]
    pos, slot = (start + depth).to(DEV), (start + torch.arange(N)).to(DEV)
    ws = qsa.workspace(qsa.qsa_sparse_tree_decode_workspace_size(B, N, Hq, D, 4, budget), DEV)
    q_new = torch.empty(B, N, Hq, D, dtype=BF, device=DEV)
    qsa.qsa_qk_norm_rope(q, k, q_new, x["k"], f, v=v, v_out=x["v"], q_weight=w, k_weight=w,
                         pos=pos, mscale=m, slot=slot, ws=ws)
    # the selection of every draft, over the committed blocks
    q_idx = torch.randn(N, B, Hi, Di, generator=g, device=DEV).to(BF)
    fi, _ = qsa.qsa_rope_frequencies(1e6, 32, device=DEV)
    qsa.qsa_rope(q_idx, q_idx, fi, pos=pos.T.contiguous())
    k_idx = torch.randn(B, L, Di, generator=g, device=DEV).to(BF)
    pooled = torch.empty(B, L // 4, Di, dtype=BF, device=DEV)
    qsa.qsa_pool(k_idx, pooled)
    sel = torch.empty(N, B, kb, dtype=torch.int32, device=DEV)
    wsi = qsa.workspace(qsa.qsa_index_topk_decode_workspace_size(B, L // 4, 4, budget), DEV)
    at = torch.tensor([p + 1 for p in P], dtype=torch.int32, device=DEV)
    weights = torch.rand(B, Hi, generator=g, device=DEV)
    for i in range(N):
        qsa.qsa_index_topk_decode(q_idx[i], weights, pooled, at, sel[i], wsi, 4, budget)
    o = torch.full((B, N, Hq, D), 7.0, dtype=BF, device=DEV)
    lse = torch.full((B, N, Hq), 7.0, device=DEV)
    qsa.qsa_sparse_tree_decode(q_new, x["k"], x["v"], x["seqlens"], sel.transpose(0, 1),
                               x["parent"], o, ws, budget=budget, lse=lse)
    assert qsa.qsa_check_device_status(ws) == 0 and qsa.qsa_check_device_status(wsi) == 0
    y = dict(x, q=q_new)
    _check(y, o, lse, P, [N] * B, sel.transpose(0, 1))
    ref = rope_oracle.norm_rope(_f64(k), _f64(w), 1e-6, pos.cpu().numpy(), _f64(f), "half", m)
    for b in range(B):
        got = _f64(x["k"][b, P[b]:P[b] + N])
        assert np.abs(got - ref[b]).max() <= 2.0 ** -8 * np.abs(ref[b]).max() * 1.01
        assert torch.equal(x["v"][b, P[b]:P[b] + N], v[b])
    dense = qsa.workspace(qsa.qsa_dense_tree_decode_workspace_size(B, N, Hq, Hkv, D), DEV)
    o.fill_(7.0)
    qsa.qsa_dense_tree_decode(q_new, x["k"], x["v"], x["seqlens"], x["parent"], o, dense, lse=lse)
    _check(y, o, lse, P, [N] * B)
