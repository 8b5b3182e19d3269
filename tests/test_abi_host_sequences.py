"""Host-side checks of the entry points for sequences of codes: workspace sizes and arguments
are judged before anything is enqueued, so none of this touches a GPU."""
import pytest


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


NAN, INF = float("nan"), float("inf")


def _caller(fn, defaults):
    def call(**kw):
        unknown = set(kw) - set(defaults)
        assert not unknown, unknown
        return fn(*(defaults | kw).values(), None)

    return call


def test_embed_arguments(ops):
    call = _caller(ops.lib.gmm_embed, dict(t=2, v=10, d=8, ldt=8, dt=0, c=4, n=5, s=1.0, o=2, ldo=8))
    for kw in (dict(v=0), dict(d=0), dict(ldt=7), dict(ldo=7), dict(n=-1), dict(n=(1 << 40) + 1), dict(t=None),
               dict(c=None), dict(o=None), dict(s=NAN), dict(s=INF)):
        assert call(**kw) == ops.GMM_E_INVALID, kw
    assert call(dt=2) == ops.GMM_E_DTYPE
    big = 1 << 22
    assert call(v=big + 1) == call(d=(1 << 20) + 1, ldt=big, ldo=big) == ops.GMM_E_UNSUPPORTED
    assert call(n=0, t=None, c=None, o=None) == ops.GMM_OK


def test_embed_backward_arguments(ops):
    wb = ops.lib.gmm_embed_backward_workspace_bytes
    need = wb(5, 8, 10)
    assert need > 0 and need % 256 == 0 and wb(0, 1, 1) > 0
    assert wb(-1, 8, 10) == wb(5, 0, 10) == wb(5, 8, 0) == wb(5, 8, (1 << 22) + 1) == wb(1 << 31, 8, 10) == 0
    call = _caller(ops.lib.gmm_embed_backward, dict(g=2, n=5, d=8, ldg=8, dt=0, c=4, v=10, s=1.0, o=2, ldt=8,
                                                    ws=256, wsb=need))
    for kw in (dict(v=0), dict(d=0), dict(ldt=7), dict(ldg=7), dict(n=-1), dict(g=None), dict(c=None),
               dict(o=None), dict(s=NAN)):
        assert call(**kw) == ops.GMM_E_INVALID, kw
    assert call(dt=9) == ops.GMM_E_DTYPE
    assert call(n=1 << 31) == call(v=(1 << 22) + 1) == ops.GMM_E_UNSUPPORTED
    assert call(ws=None) == call(wsb=need - 1) == call(ws=300) == ops.GMM_E_WORKSPACE


def test_quantized_arguments(ops):
    call = _caller(ops.lib.gmm_quantize_rows, dict(x=2, n=5, d=8, ldx=8, dt=1, q=1, ldq=8, s=4))
    for kw in (dict(d=0), dict(ldx=7), dict(ldq=7), dict(n=-1), dict(x=None), dict(q=None), dict(s=None)):
        assert call(**kw) == ops.GMM_E_INVALID, kw
    assert call(dt=2) == ops.GMM_E_DTYPE
    assert call(d=1 << 17, ldx=1 << 17, ldq=1 << 17) == ops.GMM_E_UNSUPPORTED
    assert call(n=0, x=None, q=None, s=None) == ops.GMM_OK
    wb = ops.lib.gmm_quantized_product_workspace_bytes
    need = wb(5, 8, 10)
    assert need > 0 and need % 256 == 0 and wb(0, 8, 10) > 0
    assert wb(-1, 8, 10) == wb(5, 0, 10) == wb(5, 8, 0) == wb(5, 1 << 17, 10) == wb(5, 8, (1 << 22) + 1) == 0
    call = _caller(ops.lib.gmm_quantized_product, dict(q=1, n=5, d=8, ldq=8, qs=4, w=1, v=10, ldw=8, ws_=4, y=4,
                                                       ldy=10, dt=0, ws=256, wsb=need))
    for kw in (dict(d=0), dict(v=0), dict(ldq=7), dict(ldw=7), dict(ldy=9), dict(n=-1), dict(q=None),
               dict(qs=None), dict(w=None), dict(ws_=None), dict(y=None)):
        assert call(**kw) == ops.GMM_E_INVALID, kw
    assert call(dt=2) == ops.GMM_E_DTYPE
    wide = 1 << 17
    assert call(d=wide, ldq=wide, ldw=wide) == call(v=(1 << 22) + 1, ldy=1 << 23) == ops.GMM_E_UNSUPPORTED
    assert call(ws=None) == call(wsb=need - 1) == call(ws=300) == ops.GMM_E_WORKSPACE
    assert call(n=0, q=None, qs=None, w=None, ws_=None, y=None, wsb=wb(0, 8, 10)) == ops.GMM_OK


def test_beam_step_arguments(ops):
    wb = ops.lib.gmm_beam_step_workspace_bytes
    need = wb(3, 4, 100, 4)
    assert need > 0 and need % 256 == 0 and wb(0, 4, 100, 4) > 0 and wb(3, 4, 2, 16) > 0
    assert wb(-1, 4, 100, 4) == wb(3, 0, 100, 4) == wb(3, 17, 100, 4) == wb(3, 4, 0, 4) == wb(3, 4, 100, 0) == 0
    assert wb(3, 4, 100, 17) == wb(1 << 40, 4, 100, 4) == 0
    call = _caller(ops.lib.gmm_beam_step, dict(x=2, b=3, w=4, v=100, ldl=100, dt=0, s=4, last=4, end=1, m=4,
                                               scale=1.0, p=4, c=4, o=4, ws=256, wsb=need))
    for kw in (dict(b=-1), dict(w=0), dict(w=17), dict(v=0), dict(ldl=99), dict(m=0), dict(m=17), dict(scale=0.0),
               dict(scale=NAN), dict(x=None), dict(s=None), dict(p=None), dict(c=None), dict(o=None)):
        assert call(**kw) == ops.GMM_E_INVALID, kw
    assert call(dt=3) == ops.GMM_E_DTYPE
    assert call(ws=None) == call(wsb=need - 1) == call(ws=300) == ops.GMM_E_WORKSPACE
    assert call(b=0, x=None, s=None, last=None, p=None, c=None, o=None) == ops.GMM_OK


def test_beam_reorder_arguments(ops):
    call = _caller(ops.lib.gmm_beam_reorder, dict(x=1 << 20, outer=2, so=4800, b=3, w=4, sr=400, nb=400, p=4, m=4,
                                                  o=1 << 30, oo=4800, orow=400))
    big = 1 << 60
    for kw in (dict(outer=-1), dict(b=-1), dict(w=0), dict(w=17), dict(m=0), dict(m=17), dict(nb=0), dict(x=None),
               dict(p=None), dict(o=None), dict(orow=399), dict(oo=399), dict(oo=4799), dict(oo=-4800),
               dict(sr=-400), dict(so=-1), dict(nb=big), dict(outer=big), dict(b=big), dict(sr=big), dict(so=big),
               dict(o=1 << 20, m=3), dict(o=1 << 20, orow=800, oo=9600), dict(o=1 << 20, oo=9600)):
        assert call(**kw) == ops.GMM_E_INVALID, kw
    assert call(outer=0) == call(b=0) == ops.GMM_OK


def test_balance_arguments(ops):
    wb = ops.lib.gmm_balance_loss_workspace_bytes
    need = wb(9, 8, 2)
    assert need > 0 and need % 256 == 0 and wb(0, 8, 2) > 0
    assert wb(-1, 8, 2) == wb(9, 0, 2) == wb(9, 4097, 2) == wb(9, 8, 0) == wb(9, 8, 17) == wb(1 << 30, 8, 2) == 0
    call = _caller(ops.lib.gmm_balance_loss, dict(z=2, n=9, e=8, ldz=8, dt=0, i=4, m=2, l=4, c=4, t=8, p=4, no=4,
                                                  ws=256, wsb=need))
    for kw in (dict(n=-1), dict(e=0), dict(ldz=7), dict(m=0), dict(m=17), dict(z=None), dict(i=None), dict(l=None),
               dict(c=None), dict(t=None), dict(p=None), dict(no=None)):
        assert call(**kw) == ops.GMM_E_INVALID, kw
    assert call(dt=2) == ops.GMM_E_DTYPE
    assert call(e=4097, ldz=4097) == call(n=1 << 30) == ops.GMM_E_UNSUPPORTED
    assert call(ws=None) == call(wsb=need - 1) == call(ws=300) == ops.GMM_E_WORKSPACE
    call = _caller(ops.lib.gmm_balance_loss_backward, dict(z=2, n=9, e=8, ldz=8, dt=0, c=4, t=8, no=4, g=4, dz=2,
                                                           ldd=8))
    for kw in (dict(n=-1), dict(e=0), dict(ldz=7), dict(ldd=7), dict(z=None), dict(c=None), dict(t=None),
               dict(no=None), dict(dz=None)):
        assert call(**kw) == ops.GMM_E_INVALID, kw
    assert call(dt=2) == ops.GMM_E_DTYPE and call(e=4097, ldz=4097, ldd=4097) == ops.GMM_E_UNSUPPORTED
    assert call(n=0, z=None, c=None, t=None, no=None, dz=None) == ops.GMM_OK


def test_host_tensors_are_refused(ops):
    import torch

    x, c = torch.zeros(4, 3), torch.zeros(4, dtype=torch.int32)
    q = torch.zeros(4, 3, dtype=torch.int8)
    s = torch.zeros(4)
    for f in (lambda: ops.embed(x, c), lambda: ops.embed_backward(x, c, 5), lambda: ops.quantize_rows(x),
              lambda: ops.quantized_product(q, s, q, s), lambda: ops.beam_step(x, torch.zeros(2, 2)),
              lambda: ops.beam_reorder(x, c.view(2, 2), 2), lambda: ops.balance_loss(x, c[:, None]),
              lambda: ops.balance_loss_backward(x, c[:3], torch.zeros(2, dtype=torch.int64), torch.zeros(4, 2))):
        with pytest.raises(ValueError):
            f()
