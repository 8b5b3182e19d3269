"""The head's gradients one at a time, through the C ABI: the same bits as both together."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d,v", [(3, 64, 90), (257, 100, 1000)])
def test_one_gradient(ops, n, d, v, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    h = torch.randn(n, d, generator=g, device=DEV).to(dtype)
    w = (torch.randn(v, d, generator=g, device=DEV) / d ** 0.5).to(dtype)
    t = torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int32)
    gl, gh = torch.randn(2, n, generator=g, device=DEV)
    s = ops.head_score(h, w, t)
    dh, dw = ops.head_score_backward(h, w, t, s.norm, s.entropy, gl, gh)
    code = ops.GMM_F32 if dtype == torch.float32 else ops.GMM_BF16
    need = ops.lib.gmm_head_score_backward_workspace_bytes(n, d, v, code)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    print(f"# {n} x {d} x {v} {dtype}", flush=True)
    for one, want in ((0, dh), (1, dw)):
        out = torch.full_like(want, 7.0)
        at = [None, None]
        at[one] = ctypes.c_void_p(out.data_ptr())
        assert ops.lib.gmm_head_score_backward(
            h.data_ptr(), n, d, d, w.data_ptr(), v, d, code, t.data_ptr(), s.norm.data_ptr(),
            s.entropy.data_ptr(), gl.data_ptr(), gh.data_ptr(), 1.0, at[0], d, at[1], d, ws.data_ptr(),
            need, stream) == ops.GMM_OK
        assert torch.equal(out, want)
