"""Host-side refusals of the calls on rows of logits: every case returns
before anything reaches a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from block_diffusion_speculative_draft_gb300 import api, build
    build.build()
    return api.load_library()


X = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(257)
N = None
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -5


def _with(args, **change):
    a = dict(args)
    a.update(change)
    return tuple(a.values())


def _refused(fn, args, cases):
    for code, change in cases:
        assert fn(*_with(args, **change)) == code, change


ROWS = [(EINVAL, dict(logits=N)), (EINVAL, dict(dtype=3)), (EINVAL, dict(dtype=-1)), (EINVAL, dict(V=0)),
        (EINVAL, dict(ld=99)), (EINVAL, dict(logits=ODD)), (EUNSUPPORTED, dict(V=1 << 31, ld=1 << 31))]


def test_sample(lib):
    from block_diffusion_speculative_draft_gb300 import api
    need = api.dflash_sample_workspace_size(200, 100)
    assert api.dflash_sample_workspace_size(64, 100) == 0
    n = ctypes.c_size_t(0)
    for bad in ((0, 100), (1 << 28, 100), (1, 0)):
        assert need > 0 and lib.dflash_sample_workspace_size(*bad, ctypes.byref(n)) == EINVAL
    assert lib.dflash_sample_workspace_size(2, 100, None) == EINVAL
    args = dict(logits=X, dtype=0, rows=200, V=100, ld=100, temperature=X, k=N, p=N, mp=N, u=X, ld_u=100, tok=X, lp=N,
                ws=X, ws_bytes=need, stream=N)
    _refused(lib.dflash_sample, args, [c for c in ROWS if "V" not in c[1] or c[1]["V"] == 0]
             + [(EINVAL, dict(rows=0)), (EINVAL, dict(temperature=N)), (EINVAL, dict(u=N)), (EINVAL, dict(tok=N)),
                (EWORKSPACE, dict(ws=N)), (EWORKSPACE, dict(ws_bytes=need - 1)),
                (EWORKSPACE, dict(ws=ctypes.c_void_p(264))), (EINVAL, dict(ld_u=99)), (EUNSUPPORTED, dict(rows=1 << 28)),
                (EUNSUPPORTED, dict(V=1 << 31, ld=1 << 31, ld_u=1 << 31)), (EUNSUPPORTED, dict(ld=1 << 62))])


def test_accept(lib):
    from block_diffusion_speculative_draft_gb300 import api
    need = api.dflash_verify_filtered_workspace_size(2, 4, 100)
    assert need > 0
    n = ctypes.c_size_t(0)
    for bad in ((0, 4, 100), (1, 0, 100), (1, 65, 100), (1, 4, 0)):
        assert lib.dflash_verify_filtered_workspace_size(*bad, ctypes.byref(n)) == EINVAL
    assert lib.dflash_verify_filtered_workspace_size(1, 4, 100, None) == EINVAL
    args = dict(logits=X, dtype=2, ld=100, draft=X, b=2, R=4, D=3, V=100, temperature=X, k=N, p=N, mp=N, ua=X, us=X,
                ld_u=100, n=X, corr=X, em=N, nx=N, ws=X, ws_bytes=need, stream=N)
    _refused(lib.dflash_verify_accept_filtered, args, [c for c in ROWS if c[0] == EINVAL]
             + [(EINVAL, dict(b=0)), (EINVAL, dict(R=0)), (EINVAL, dict(R=65)), (EINVAL, dict(D=0)),
                (EINVAL, dict(D=5)), (EINVAL, dict(draft=N)), (EINVAL, dict(temperature=N)), (EINVAL, dict(ua=N)),
                (EINVAL, dict(us=N)), (EINVAL, dict(ld_u=99)), (EINVAL, dict(n=N)), (EINVAL, dict(corr=N)),
                (EWORKSPACE, dict(ws=N)), (EWORKSPACE, dict(ws_bytes=need - 1)),
                (EWORKSPACE, dict(ws=ctypes.c_void_p(264)))])


def test_top_logits(lib):
    args = dict(logits=X, dtype=0, rows=2, V=100, ld=100, K=5, T=1.0, val=X, idx=X, lse=N, stream=N)
    _refused(lib.dflash_top_logits, args, ROWS
             + [(EINVAL, dict(rows=0)), (EINVAL, dict(K=0)), (EUNSUPPORTED, dict(K=1025)), (EINVAL, dict(val=N)),
                (EINVAL, dict(idx=N))] + [(EINVAL, dict(T=t)) for t in (0.0, -1.0, 1e-7, 1e7, float("nan"), float("inf"))])


def test_distill(lib):
    loss = dict(logits=X, dtype=0, rows=2, V=100, ld=100, tv=X, ti=X, K=5, tl=N, T=1.0, w=N, loss=X, stats=N, dz=N,
                ldd=0, stream=N)
    bad = ROWS + [(EINVAL, dict(rows=0)), (EINVAL, dict(tv=N)), (EINVAL, dict(ti=N)), (EINVAL, dict(K=0)),
                  (EUNSUPPORTED, dict(K=1025)), (EUNSUPPORTED, dict(V=(1 << 23) + 1, ld=1 << 24, ldd=1 << 24)),
                  (EINVAL, dict(T=0.0)), (EINVAL, dict(T=float("nan")))]
    _refused(lib.dflash_distill_loss, loss, bad
             + [(EINVAL, dict(loss=N)), (EINVAL, dict(stats=ctypes.c_void_p(264))), (EINVAL, dict(dz=X, ldd=99)),
                (EINVAL, dict(dz=ODD, ldd=100)), (EINVAL, dict(dz=X, ldd=101))])
    back = dict(logits=X, dtype=0, rows=2, V=100, ld=100, tv=X, ti=X, K=5, tl=N, T=1.0, stats=X, g=X, dz=X, ldd=100,
                stream=N)
    _refused(lib.dflash_distill_backward, back, [c for c in bad if c[1].get("V") != 1 << 31]
             + [(EINVAL, dict(stats=N)), (EINVAL, dict(g=N)), (EINVAL, dict(dz=N)), (EINVAL, dict(ldd=99)),
                (EINVAL, dict(ldd=101))])
