"""Host-side checks of the softmax-over-codes entry points: workspace sizes and
arguments are judged before anything is enqueued, so none of this touches a GPU."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def test_constants_match_the_header(ops):
    src = open(os.path.join(ROOT, "include", "gmm_em.h")).read()
    assert int(re.search(r"#define GMM_TOP_MAX (\d+)", src).group(1)) == ops.TOP_MAX


def test_logits_score_arguments(ops):
    wb = ops.lib.gmm_logits_score_workspace_bytes
    need = wb(10, 100, 4)
    assert need > 0 and need % 256 == 0 and wb(0, 1, 0) > 0
    assert wb(-1, 100, 0) == 0 and wb(10, 0, 0) == 0 and wb(10, 100, 17) == 0 and wb(10, 3, 4) == 0
    assert wb(10, 100, -1) == 0 and wb(10, (1 << 30) + 1, 0) == 0
    # few long rows are scored in parts that the workspace holds
    assert wb(1, 1 << 20, 16) > wb(1, 1000, 16)

    def call(**kw):
        a = dict(x=2, n=10, v=100, ld=100, dt=0, t=4, m=4, s=1.0, lp=4, h=4, no=4, ti=4, tl=4,
                 ws=256, wsb=need)
        a.update(kw)
        return ops.lib.gmm_logits_score(a["x"], a["n"], a["v"], a["ld"], a["dt"], a["t"], a["m"], a["s"],
                                        a["lp"], a["h"], a["no"], a["ti"], a["tl"], a["ws"], a["wsb"], None)

    bad = ops.GMM_E_INVALID
    assert call(n=-1) == bad and call(v=0) == bad and call(ld=99) == bad and call(x=None) == bad
    assert call(m=17) == bad and call(m=-1) == bad and call(lp=None) == bad and call(ti=None) == bad
    assert call(tl=None) == bad
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(s=s) == bad
    assert call(dt=2) == ops.GMM_E_DTYPE
    assert call(ws=None) == call(wsb=need - 1) == call(ws=257) == ops.GMM_E_WORKSPACE
    assert call(n=0, x=None, t=None, lp=None, ti=None, tl=None, wsb=wb(0, 100, 4)) == ops.GMM_OK


def test_logits_score_backward_arguments(ops):
    def call(**kw):
        a = dict(x=2, n=10, v=100, ld=100, dt=0, t=4, no=4, h=4, gl=4, gh=4, s=1.0, dx=4, ldd=100)
        a.update(kw)
        return ops.lib.gmm_logits_score_backward(a["x"], a["n"], a["v"], a["ld"], a["dt"], a["t"],
                                                 a["no"], a["h"], a["gl"], a["gh"], a["s"], a["dx"],
                                                 a["ldd"], None)

    bad = ops.GMM_E_INVALID
    for kw in (dict(n=-1), dict(v=0), dict(ld=99), dict(ldd=99), dict(x=None), dict(dx=None),
               dict(no=None), dict(t=None), dict(h=None), dict(s=0.0)):
        assert call(**kw) == bad, kw
    assert call(dt=5) == ops.GMM_E_DTYPE
    assert call(n=0) == ops.GMM_OK


def test_head_arguments(ops):
    wb, wg = ops.lib.gmm_head_score_workspace_bytes, ops.lib.gmm_head_score_backward_workspace_bytes
    assert wb(10, 64, 100, 0, 0) > 0 and wb(10, 64, 100, 1, 4) % 256 == 0 and wg(10, 64, 100, 1) % 256 == 0
    assert wb(10, 0, 100, 0, 0) == 0 and wb(10, 64, 100, 2, 0) == 0 and wb(10, 64, 3, 0, 4) == 0
    assert wb(10, (1 << 20) + 1, 100, 0, 0) == 0 and wg(10, 64, (1 << 22) + 1, 0) == 0
    # rows beyond a chunk add only what is kept per row
    assert wb(1 << 24, 64, 1000, 1, 0) == wb(1 << 25, 64, 1000, 1, 0)
    assert wg(1 << 25, 64, 1000, 0) == wg(1 << 26, 64, 1000, 0)
    need, ng = wb(10, 64, 100, 0, 4), wg(10, 64, 100, 0)

    def fwd(**kw):
        a = dict(x=4, n=10, d=64, ldx=64, w=4, v=100, ldw=64, dt=0, t=4, m=4, s=1.0, lp=4, ti=4,
                 ws=256, wsb=need)
        a.update(kw)
        return ops.lib.gmm_head_score(a["x"], a["n"], a["d"], a["ldx"], a["w"], a["v"], a["ldw"], a["dt"],
                                      a["t"], a["m"], a["s"], a["lp"], 4, 4, a["ti"], 4, a["ws"],
                                      a["wsb"], None)

    bad = ops.GMM_E_INVALID
    for kw in (dict(n=-1), dict(d=0), dict(v=0), dict(ldx=63), dict(ldw=63), dict(x=None), dict(w=None),
               dict(lp=None), dict(m=17), dict(ti=None), dict(s=float("nan"))):
        assert fwd(**kw) == bad, kw
    assert fwd(dt=9) == ops.GMM_E_DTYPE
    assert fwd(d=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21) == ops.GMM_E_UNSUPPORTED
    assert fwd(wsb=need - 1) == fwd(ws=None) == fwd(ws=300) == ops.GMM_E_WORKSPACE

    def bwd(**kw):
        a = dict(x=4, n=10, d=64, ldx=64, w=4, v=100, ldw=64, dt=0, t=4, no=4, h=4, gl=4, gh=4, s=1.0,
                 dh=4, ldh=64, dw=4, lddw=64, ws=256, wsb=ng)
        a.update(kw)
        return ops.lib.gmm_head_score_backward(a["x"], a["n"], a["d"], a["ldx"], a["w"], a["v"], a["ldw"],
                                               a["dt"], a["t"], a["no"], a["h"], a["gl"], a["gh"], a["s"],
                                               a["dh"], a["ldh"], a["dw"], a["lddw"], a["ws"], a["wsb"],
                                               None)

    for kw in (dict(n=-1), dict(ldh=63), dict(lddw=63), dict(dh=None, dw=None), dict(no=None),
               dict(t=None), dict(h=None), dict(s=-1.0)):
        assert bwd(**kw) == bad, kw
    assert bwd(wsb=ng - 1) == ops.GMM_E_WORKSPACE and bwd(dt=3) == ops.GMM_E_DTYPE
    assert bwd(v=(1 << 22) + 1) == ops.GMM_E_UNSUPPORTED


def test_moe_arguments(ops):
    wb = ops.lib.gmm_moe_layer_workspace_bytes
    need = wb(10, 64, 32, 8, 1, 2)
    assert need > 0 and need % 256 == 0
    assert wb(-1, 64, 32, 8, 1, 2) == 0 and wb(10, 64, 32, 8, 1, 9) == 0 and wb(10, 64, 32, 8, 4, 2) == 0
    assert wb(10, 64, 32, 5000, 1, 2) == 0 and wb(1 << 20, 64, 32, 8, 1, 2) == 0

    def call(**kw):
        a = dict(x=2, n=10, d=64, ldx=64, g=2, e=8, wi=2, wo=2, f=32, dt=1, m=2, i=4, r=4, y=2, ldy=64,
                 ws=256, wsb=need)
        a.update(kw)
        return ops.lib.gmm_moe_layer(a["x"], a["n"], a["d"], a["ldx"], a["g"], a["e"], a["wi"], a["wo"],
                                     a["f"], a["dt"], a["m"], 0, a["i"], a["r"], a["y"], a["ldy"],
                                     a["ws"], a["wsb"], None)

    bad = ops.GMM_E_INVALID
    for kw in (dict(n=-1), dict(d=0), dict(f=0), dict(e=0), dict(m=0), dict(m=9), dict(ldx=63),
               dict(ldy=63), dict(x=None), dict(wi=None), dict(wo=None), dict(i=None), dict(r=None),
               dict(y=None)):
        assert call(**kw) == bad, kw
    assert call(dt=7) == ops.GMM_E_DTYPE
    assert call(e=5000) == call(n=1 << 20) == ops.GMM_E_UNSUPPORTED
    assert call(wsb=need - 1) == call(ws=None) == call(ws=257) == ops.GMM_E_WORKSPACE
    assert call(n=0, wsb=wb(0, 64, 32, 8, 1, 2)) == ops.GMM_OK
