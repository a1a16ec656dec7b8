"""GPU tests of the layer's front and of trees of drafted tokens where the calls allow more
than the parity tests use: workspaces at any 16-byte boundary, outputs in place of inputs,
steps that follow one another without a pause."""
import pytest
import torch

import block_sparse_long_10_b200 as qsa
from tests.test_gpu_tree import _make, _run, _sel

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,prefix", [
    (2, 5, 16, 2, 128, [700, 3]), (1, 40, 8, 1, 128, [3000]), (3, 3, 4, 1, 64, [128, 0, 50]),
    (1, 33, 32, 4, 64, [900])])
def test_tree_workspaces_at_any_16_byte_boundary(B, N, Hq, Hkv, D, prefix, sparse):
    """The header asks for 16-byte alignment: the same bits at every such offset, and nothing
    behind the size that the library asks for is written."""
    x = _make(B, N, Hq, Hkv, D, prefix, [N] * B, seed=7)
    sel = _sel(prefix, N, 64, 3) if sparse else None
    good = _run(x, sel, 256)
    n = good[2].numel()
    for offset in (0, 16, 32, 48):
        buf = torch.zeros(n + 128, dtype=torch.uint8, device=DEV)
        buf[offset + n:] = 0xA5
        ws = buf[offset:offset + n]
        assert ws.data_ptr() % 64 == offset
        o, lse, _ = _run(x, sel, 256, ws=ws)
        assert qsa.qsa_check_device_status(ws) == 0
        assert torch.equal(o, good[0]) and torch.equal(lse, good[1])
        assert bool((buf[offset + n:] == 0xA5).all()) and bool((buf[:offset] == 0).all())


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("N,Hq,Hkv", [(1, 1, 1), (2, 8, 2), (4, 16, 2)])
def test_lengths_change_right_behind_steps_without_drafts(N, Hq, Hkv, sparse):
    """Steps of which no sequence has a draft write nothing; the lengths change in the stream
    right behind each call, and the next one has its own."""
    B, D = 300, 64
    prefix = [17 + (b * 37) % 400 for b in range(B)]
    x = _make(B, N, Hq, Hkv, D, prefix, [N] * B, seed=13)
    sel = _sel(prefix, N, 16, 5) if sparse else None
    good = _run(x, sel, 64)
    lens = x["seqlens"].clone(), x["n_draft"].clone()
    none = lens[0] - N, torch.zeros_like(lens[1])
    ws, results = good[2], []
    for step in range(12):
        for name, value in zip(("seqlens", "n_draft"), lens if step % 3 == 2 else none):
            x[name].copy_(value)
        results.append(_run(x, sel, 64, ws=ws))
    assert qsa.qsa_check_device_status(ws) == 0
    for step, (o, lse, _) in enumerate(results):
        if step % 3 == 2:
            assert torch.equal(o, good[0]) and torch.equal(lse, good[1])
        else:
            assert bool((o == 7).all()) and bool((lse == 7).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("Hq,Hkv,D,rot", [(16, 2, 128, 128), (5, 3, 64, 24)])
def test_norm_rotation_and_gradients_in_place(Hq, Hkv, D, rot, layout):
    """Rows are fetched batches ahead of those being written, over many rounds of the GPU: in
    place the bits are the same."""
    g = torch.Generator(device=DEV).manual_seed(D + rot)
    B, T = 2, 9001
    rand = lambda *s, dtype=BF: torch.randn(*s, generator=g, device=DEV).to(dtype)
    q, k, v = rand(B, T, Hq, D), rand(B, T, Hkv, D), rand(B, T, Hkv, D)
    f, m = qsa.qsa_rope_frequencies(1e6, rot, "by-parts", 8.0, 32768.0, device=DEV)
    qw, kw = (1 + 0.3 * rand(D, dtype=F32) for _ in range(2))
    pos = torch.randint(0, 1 << 20, (B, T), generator=g, device=DEV)
    how = dict(pos=pos, layout=layout, mscale=m)
    norm = dict(q_weight=qw, k_weight=kw, **how)
    out = [torch.empty_like(t) for t in (q, k, v)]
    qsa.qsa_qk_norm_rope(q, k, out[0], out[1], f, v=v, v_out=out[2], **norm)
    a, b, c = q.clone(), k.clone(), v.clone()
    qsa.qsa_qk_norm_rope(a, b, a, b, f, v=c, v_out=c, **norm)
    for got, want in zip((a, b, c), out):
        assert torch.equal(got, want)
    ws = qsa.workspace(qsa.qsa_qk_norm_rope_backward_workspace_size(B, T, Hq, Hkv, D), DEV)
    for dtype in (BF, F32):
        d_q, d_k = rand(B, T, Hq, D, dtype=dtype), rand(B, T, Hkv, D, dtype=dtype)
        want = [torch.empty_like(t) for t in (d_q, d_k, qw, kw)]
        qsa.qsa_qk_norm_rope_backward(d_q, d_k, q, k, want[0], want[1], f, ws, dq_weight=want[2],
                                      dk_weight=want[3], **norm)
        turned = torch.empty_like(d_q)
        qsa.qsa_rope(d_q, turned, f, transpose=True, **how)
        a, b, c = d_q.clone(), d_k.clone(), d_q.clone()
        w = [torch.empty_like(t) for t in (qw, kw)]
        qsa.qsa_qk_norm_rope_backward(a, b, q, k, a, b, f, ws, dq_weight=w[0], dk_weight=w[1],
                                      **norm)
        qsa.qsa_rope(c, c, f, transpose=True, **how)
        for got, ref in zip((a, b, *w, c), (*want, turned)):
            assert torch.equal(got, ref)


def test_norm_rotation_in_place_of_a_projection_is_refused():
    """The outputs are packed: they are not the rows of a wider projection, and with slots
    they are other rows than those read."""
    g = torch.Generator(device=DEV).manual_seed(1)
    packed = torch.randn(2, 3, 6 * 64, generator=g, device=DEV).to(BF)
    q, k = (packed[..., :256].unflatten(-1, (4, 64)), packed[..., 256:].unflatten(-1, (2, 64)))
    f, _ = qsa.qsa_rope_frequencies(1e6, 64, device=DEV)
    qo = packed.view(-1)[:2 * 3 * 256].view(2, 3, 4, 64)
    ko = torch.empty(2, 3, 2, 64, dtype=BF, device=DEV)
    with pytest.raises(qsa.QSAError):
        qsa.qsa_qk_norm_rope(q, k, qo, ko, f)
    kc = k.contiguous()
    slot = torch.arange(3, device=DEV).expand(2, 3).contiguous()
    with pytest.raises(qsa.QSAError):
        qsa.qsa_qk_norm_rope(q, kc, torch.empty_like(qo), kc, f, slot=slot)
    one = packed[:1, :1]  # a single token's rows lie as its outputs do
    q1 = one[..., :256].unflatten(-1, (4, 64))
    want = torch.empty(1, 1, 4, 64, dtype=BF, device=DEV)
    kw = dict(pos=torch.full((1, 1), 9, device=DEV))
    qsa.qsa_qk_norm_rope(q1, kc[:1, :1].contiguous(), want, ko[:1, :1].contiguous(), f, **kw)
    qsa.qsa_qk_norm_rope(q1, kc[:1, :1].contiguous(), q1, ko[:1, :1].contiguous(), f, **kw)
    assert torch.equal(q1, want)


def test_single_drafts_meet_dense_decode_within_their_rounding():
    """Each side's P V takes probabilities of half a bf16 step (2^-8 relative), so it is within
    2^-8 sum p |v| of the exact product, and is rounded to half a bf16 step: together 2 (2^-8
    mass + 2^-8 |o|), |o| <= mass; the scores' and exponentials' fp32 errors (2 D 2^-24 of
    logits below 32, twice: under 2^-9 of it) join as 2^-8 mass."""
    prefix, D = [0, 5, 1023, 300], 128
    x = _make(4, 1, 16, 2, D, prefix, [1] * 4, seed=2, L=1024)
    o, _, _ = _run(x, n_draft=False)
    x["k"].nan_to_num_(0.0)
    x["v"].nan_to_num_(0.0)
    o2 = torch.empty_like(x["q"][:, 0])
    ws = qsa.workspace(qsa.qsa_dense_gqa_decode_workspace_size(4, 1024, 16, D), DEV)
    qsa.qsa_dense_gqa_decode(x["q"][:, 0].contiguous(), x["k"], x["v"], x["seqlens"], o2, ws)
    for b, P in enumerate(prefix):
        k, v = (x[n][b, :P + 1].double().repeat_interleave(8, 1) for n in "kv")
        s = torch.einsum("hd,lhd->hl", x["q"][b, 0].double(), k) * D ** -0.5
        assert float(s.abs().max()) < 32
        p = s.softmax(-1)
        mass = torch.einsum("hl,lhd->hd", p, v.abs())
        bound = 5 * 2.0 ** -8 * mass
        assert bool(((o[b, 0].double() - o2[b].double()).abs() <= bound).all()), b


@pytest.mark.parametrize("N,prefix,sparse", [(7, 1003, False), (40, 9000, False),
                                             (16, 30000, False), (16, 9003, True)])
def test_every_call_gives_the_same_bits(N, prefix, sparse):
    """The split and the order of every sum depend on the lengths alone."""
    x = _make(3, N, 16, 2, 128, [prefix, prefix // 2, prefix // 3], [N, N - 1, N], seed=17)
    sel = _sel([prefix, prefix // 2, prefix // 3], N, 512, 3) if sparse else None
    first = _run(x, sel, 2048)
    for _ in range(30):
        o, lse, _ = _run(x, sel, 2048)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_frequency_tables_of_any_length_are_refused():
    """Longer than a head's pairs, to where twice the count no longer fits 32 bits."""
    x = torch.zeros(1, 2, 1, 64, dtype=BF, device=DEV)
    for n in (33, 1 << 21, 1 << 30, 1 << 31):
        table = torch.empty(n, dtype=torch.float64, device=DEV)  # (17 GB at most, never read)
        with pytest.raises(qsa.QSAError):
            qsa.qsa_rope(x, torch.empty_like(x), table)
        del table
    torch.cuda.empty_cache()
