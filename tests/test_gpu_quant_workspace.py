"""Products of 8-bit rows in exactly the workspace that their operands need: nothing behind it is
touched, and no copy of operands that are read in place is allocated. The sums are exact: results are
compared for equality."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def _int8(n, d, lead, pad, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-128, 128, (n, lead + d + pad), generator=g, device=DEV, dtype=torch.int8)[:, lead:lead + d]


# (n, d, v): few rows, odd ones in few tiles with and without a split, tiles split and whole, rows in chunks
@pytest.mark.parametrize("n,d,v", [(16, 640, 300), (17, 1, 1), (17, 128, 1), (20, 8191, 3001), (40, 4999, 200),
                                   (128, 8192, 4096), (300, 1024, 1001), (777, 1003, 5001), (1000, 768, 2000),
                                   (2100, 130_944, 40), (2100, 130_999, 40), (4500, 130_999, 300)])
@pytest.mark.parametrize("odd_q,odd_w", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_no_more_is_used(ops, n, d, v, odd_q, odd_w):
    print(f"# int8 product n={n} d={d} v={v} odd {odd_q} {odd_w}", flush=True)
    to16 = -d % 16
    q = _int8(n, d, odd_q, to16 + 16 * odd_q, 1)
    w = _int8(v, d, odd_w, to16 + 16 * odd_w, 2)
    one_q, one_w = torch.ones(n, device=DEV), torch.ones(v, device=DEV)
    need = ops.lib.gmm_quantized_product_call_workspace_bytes(q.data_ptr(), n, d, q.stride(0), w.data_ptr(), v,
                                                              w.stride(0))
    buf = torch.full((need + 65536,), 77, dtype=torch.uint8, device=DEV)
    y = ops.quantized_product(q, one_q, w, one_w, F32, ws=buf[:need])
    ref = (q.float().double() @ w.float().double().t()).float()
    assert torch.equal(y, ref)
    assert buf[need:].eq(77).all()
    with pytest.raises(ops.GmmError):
        ops.quantized_product(q, one_q, w, one_w, F32, ws=buf[:need - 256])


def test_no_copy_of_operands_read_in_place(ops):
    n, d, v = 512, 4096, 32768
    q, w = _int8(n, d, 0, 0, 3), _int8(v, d, 0, 0, 4)
    one_q, one_w = torch.ones(n, device=DEV), torch.ones(v, device=DEV)
    out = torch.empty(n, v, dtype=BF16, device=DEV)
    ops.quantized_product(q, one_q, w, one_w, out=out)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    ops.quantized_product(q, one_q, w, one_w, out=out)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before <= 128 << 20 < v * d + n * d
