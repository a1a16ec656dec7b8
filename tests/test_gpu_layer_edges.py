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
