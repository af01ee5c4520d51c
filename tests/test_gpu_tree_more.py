"""More of the calls on trees: workspaces as they are found, work cut in many
places, and keys whose loss shows wherever they lie."""
import types

import numpy as np
import pytest

from oracle import tree_oracle as TO
from tests.gpu_util import gpu_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

if gpu_available():
    import torch
    from block_diffusion_speculative_draft_gb300 import api
    from tests.test_gpu_tree import DEV, _attend, _attention_case, _i32, _trees


# -------------------------------------------------------------- workspaces ---
@pytest.mark.parametrize("N,nq,nkv,cap", [(1, 8, 2, 900), (9, 8, 2, 700), (40, 4, 2, 3000), (64, 8, 2, 2000)])
def test_attention_takes_its_workspace_as_it_finds_it(N, nq, nkv, cap, monkeypatch):
    """A workspace of any bits gives the same results, bit for bit, and one that
    the call allocates itself is not filled first."""
    rng = np.random.default_rng(N)
    lens, nodes = [cap, cap // 3], [N, max(1, N - 2)]
    kv, q, kt, vt = _attention_case(rng, "f16", 2, N, nq, nkv, 128, cap, lens, nodes, L=1)
    mask, n = _i32(TO.pack_bits(np.stack([TO.tree_mask(p)[0] for p in _trees(rng, 2, N)]))), _i32(nodes)
    size = api.dflash_tree_attention_workspace_size(2, N, nq, nkv, 128)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    api.dflash_get_status()
    out, lse = _attend(kv, 0, q, kt, vt, mask, n, ws=ws)
    for byte in (0xff, 0x7f):
        ws.fill_(byte)
        got, l = _attend(kv, 0, q, kt, vt, mask, n, ws=ws)
        assert torch.equal(got, out) and torch.equal(l, lse)

    def filled(*a, **k):
        raise AssertionError("the workspace is filled")

    monkeypatch.setattr(torch, "zeros", filled)
    got, l = _attend(kv, 0, q, kt, vt, mask, n)
    assert torch.equal(got, out) and torch.equal(l, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out2, lse2 = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    api.dflash_tree_attention(q, kv, 0, kt, vt, mask, out2, n_nodes=n, lse_out=lse2, stream=side)
    side.synchronize()
    assert torch.equal(out2, out) and torch.equal(lse2, lse) and api.dflash_get_status() == 0
