"""Host-side refusals of dflash_adjust_logits and of the calls on trees: every
case returns before anything reaches a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from block_diffusion_speculative_draft_gb300 import api, build
    build.build()
    return api.load_library()


X = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(257)
OFF = ctypes.c_void_p(264)  # not 16-byte aligned
N = None
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -5


def _refused(fn, args, cases):
    for code, change in cases:
        a = dict(args)
        a.update(change)
        assert fn(*a.values()) == code, change


def test_adjust(lib):
    args = dict(logits=X, dtype=0, b=2, R=3, V=100, ld=100, out=X, ld_out=100, hist=X, ld_hist=50, H=50, n_hist=X,
                n_prompt=X, draft=X, D=3, path=X, rho=X, freq=X, pres=X, bi=X, bv=X, K=4, allow=X, n_allow=6, ld_allow=4,
                allow_row=X, stream=N)
    _refused(lib.dflash_adjust_logits, args, [
        (EINVAL, dict(logits=N)), (EINVAL, dict(out=N)), (EINVAL, dict(dtype=3)), (EINVAL, dict(dtype=-1)),
        (EINVAL, dict(b=0)), (EINVAL, dict(R=0)), (EINVAL, dict(R=257)), (EINVAL, dict(V=0)), (EINVAL, dict(ld=99)),
        (EINVAL, dict(ld_out=99)), (EINVAL, dict(ld_out=101)), (EINVAL, dict(logits=ODD)), (EINVAL, dict(out=ODD)),
        (EUNSUPPORTED, dict(b=1 << 28)), (EUNSUPPORTED, dict(b=1 << 27)),
        (EUNSUPPORTED, dict(b=1 << 20, V=1 << 25, ld=1 << 25, ld_out=1 << 25, n_allow=1 << 22, ld_allow=1 << 20)),
        (EUNSUPPORTED, dict(V=1 << 31, ld=1 << 31, ld_out=1 << 31, ld_allow=1 << 26)),
        (EINVAL, dict(n_hist=N)), (EINVAL, dict(H=0)), (EINVAL, dict(H=51)),
        (EUNSUPPORTED, dict(H=(1 << 20) - 256, ld_hist=1 << 20)), (EUNSUPPORTED, dict(ld_hist=1 << 62)),
        (EINVAL, dict(D=0)), (EINVAL, dict(D=257)), (EINVAL, dict(draft=N)), (EINVAL, dict(bi=N)), (EINVAL, dict(bv=N)),
        (EINVAL, dict(K=0)), (EUNSUPPORTED, dict(K=513)), (EINVAL, dict(n_allow=0)), (EINVAL, dict(ld_allow=3)),
        (EINVAL, dict(allow=N)), (EUNSUPPORTED, dict(ld_allow=1 << 60))])


def test_mask_and_accept(lib):
    mask = dict(parent=X, n=N, b=2, N=5, mask=X, depth=N, stream=N)
    tree = [(EINVAL, dict(b=0)), (EINVAL, dict(N=0)), (EINVAL, dict(N=257)), (EUNSUPPORTED, dict(b=65536))]
    _refused(lib.dflash_tree_mask, mask, tree + [(EINVAL, dict(parent=N)), (EINVAL, dict(mask=N))])
    acc = dict(tok=X, tree=X, parent=X, nn=N, b=2, N=5, R=3, n=X, corr=X, path=X, em=N, nx=N, stream=N)
    _refused(lib.dflash_tree_accept, acc, [c for c in tree if c[1].get("N") != 0] + [
        (EINVAL, dict(R=0)), (EINVAL, dict(R=6)), (EINVAL, dict(tok=N)), (EINVAL, dict(tree=N)), (EINVAL, dict(parent=N)),
        (EINVAL, dict(n=N)), (EINVAL, dict(corr=N)), (EINVAL, dict(path=N))])


def test_attention(lib):
    from block_diffusion_speculative_draft_gb300 import api
    need = api.dflash_tree_attention_workspace_size(2, 5, 8, 2, 64)
    assert need > 0
    n = ctypes.c_size_t(0)
    for code, bad in ((EINVAL, (0, 5, 8, 2, 64)), (EINVAL, (2, 0, 8, 2, 64)), (EINVAL, (2, 257, 8, 2, 64)),
                      (EINVAL, (2, 5, 0, 2, 64)), (EINVAL, (2, 5, 8, 0, 64)), (EUNSUPPORTED, (2, 5, 8, 3, 64)),
                      (EUNSUPPORTED, (2, 5, 8, 2, 96)), (EUNSUPPORTED, (65536, 5, 8, 2, 64))):
        assert lib.dflash_tree_attention_workspace_size(*bad, ctypes.byref(n)) == code, bad
    assert lib.dflash_tree_attention_workspace_size(2, 5, 8, 2, 64, None) == EINVAL
    kv = api.KV(256, 256, 256, 2, 64)
    args = dict(q=X, q_seq=5 * 512, q_tok=512, dtype=1, kv=ctypes.byref(kv), layer=0, N=5, nq=8, nkv=2, d=64, kt=X, vt=X,
                t_seq=640, t_tok=128, mask=N, nn=N, scale=0.125, out=X, lse=N, ws=X, ws_bytes=need, stream=N)
    bad_kv = [api.KV(*a) for a in ((0, 256, 256, 2, 64), (256, 256, 0, 2, 64), (256, 264, 256, 2, 64),
                                   (256, 256, 256, 0, 64), (256, 256, 256, 2, 0))]
    _refused(lib.dflash_tree_attention, args, [(EINVAL, dict(kv=None))]
             + [(EINVAL, dict(kv=ctypes.byref(k))) for k in bad_kv]
             + [(EUNSUPPORTED, dict(kv=ctypes.byref(api.KV(256, 256, 256, 2, 1 << 24)))),
                (EINVAL, dict(dtype=0)), (EINVAL, dict(dtype=3)), (EINVAL, dict(layer=-1)), (EINVAL, dict(N=0)),
                (EINVAL, dict(N=257)), (EUNSUPPORTED, dict(nq=9)), (EUNSUPPORTED, dict(d=32)), (EINVAL, dict(q=N)),
                (EINVAL, dict(kt=N)), (EINVAL, dict(vt=N)), (EINVAL, dict(out=N)), (EINVAL, dict(q=OFF)),
                (EINVAL, dict(kt=OFF)), (EINVAL, dict(vt=OFF)), (EINVAL, dict(out=OFF)), (EINVAL, dict(q_tok=516)),
                (EINVAL, dict(t_seq=-8)), (EINVAL, dict(t_tok=1 << 44)), (EWORKSPACE, dict(ws=N)),
                (EWORKSPACE, dict(ws=OFF)), (EWORKSPACE, dict(ws_bytes=need - 1))]
             + [(EINVAL, dict(scale=s)) for s in (0.0, -1.0, float("nan"), float("inf"))])


def test_commit(lib):
    from block_diffusion_speculative_draft_gb300 import api
    need = api.dflash_tree_commit_workspace_size(2)
    n = ctypes.c_size_t(0)
    assert need > 0 and lib.dflash_tree_commit_workspace_size(0, ctypes.byref(n)) == EINVAL
    assert lib.dflash_tree_commit_workspace_size(2, None) == EINVAL
    assert lib.dflash_tree_commit_workspace_size(65536, ctypes.byref(n)) == EUNSUPPORTED
    kv = api.KV(256, 256, 256, 2, 64)
    args = dict(kv=ctypes.byref(kv), L=3, nkv=2, d=64, N=5, kt=X, vt=X, t_layer=1280, t_seq=640, t_tok=128, path=X, n=X,
                R=4, hid=X, cols=64, hid_out=X, len_out=N, ws=X, ws_bytes=need, stream=N)
    _refused(lib.dflash_tree_commit, args, [
        (EINVAL, dict(kv=None)), (EINVAL, dict(L=0)), (EINVAL, dict(nkv=0)), (EINVAL, dict(d=0)),
        (EUNSUPPORTED, dict(d=60)), (EINVAL, dict(N=0)), (EINVAL, dict(N=257)), (EINVAL, dict(R=0)), (EINVAL, dict(R=6)),
        (EINVAL, dict(kt=N)), (EINVAL, dict(vt=OFF)), (EINVAL, dict(t_layer=4)), (EINVAL, dict(t_seq=-8)),
        (EINVAL, dict(path=N)), (EINVAL, dict(n=N)), (EINVAL, dict(hid=N)), (EINVAL, dict(hid_out=N)),
        (EINVAL, dict(cols=60)), (EINVAL, dict(cols=0)), (EINVAL, dict(hid=OFF)), (EWORKSPACE, dict(ws=N)),
        (EWORKSPACE, dict(ws_bytes=need - 1)), (EWORKSPACE, dict(ws=ODD))])
