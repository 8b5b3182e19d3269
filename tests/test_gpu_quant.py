"""Rows in 8-bit integers and their products, bit for bit.

The scale is a correctly rounded quotient, the integers are the nearest ones to exact quotients
(float64 tells them: two 24-bit numbers whose quotient is not k + 1/2 differ from it by more than
2^-33 of it), the sums are exact and each of the three roundings after them is an fp32 (or
bf16) operation: nothing is left to tolerate.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(x):
    """(q, scale) by definition."""
    x = x.double()
    amax = x.abs().amax(1)
    bad = ~torch.isfinite(x).all(1)
    scale = (amax / 127.0).to(F32)
    scale[bad] = float("nan")
    s = scale.double()[:, None]
    q = torch.round(x / s).clamp(-127, 127)
    q[bad | (scale == 0)] = 0
    return q.to(torch.int8), scale


def _check_rows(q, scale, x):
    want, s = _rows(x)
    assert torch.equal(scale.nan_to_num(-1.0), s.nan_to_num(-1.0))
    assert q.dtype == torch.int8 and torch.equal(q, want), (q != want).nonzero()[:5]


def _product(q, qs, w, ws, dtype):
    acc = (q.double() @ w.double().t()).to(F32)
    return ((acc * qs[:, None]) * ws).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,d", [(1, 1), (1, 768), (3, 7), (17, 64), (5, 1025), (300, 100), (2, 40001), (1000, 96),
                                 (5, 15), (33, 16), (5, 17), (70, 128), (65, 129), (37, 512), (9, 513), (7, 4096),
                                 (6, 4097), (3, 16384), (2, 16385), (2, 131071)])
def test_rows(ops, n, d, dtype):
    g = _gen(n + d)
    x = (torch.randn(n, d, generator=g, device=DEV) * 3).to(dtype)
    _check_rows(*ops.quantize_rows(x), x)


def test_ties_and_neighbours(ops):
    # quotients at and right beside k + 1/2: the scale of a row with 127 s is s exactly
    for s in (1.0, 0.75, 3.0 * 2.0 ** -20, 1.1, 2.0 ** -120, 2.0 ** -130):
        s = float(torch.tensor(s, dtype=F32))
        half = (torch.arange(-127, 127, device=DEV, dtype=torch.float64) + 0.5) * s
        mid = half.to(F32)
        x = torch.cat([mid, torch.nextafter(mid, mid * 2), torch.nextafter(mid, mid * 0),
                       torch.tensor([127.0 * s], device=DEV)])[None]
        _check_rows(*ops.quantize_rows(x), x)


def test_extreme_rows(ops):
    x = torch.randn(9, 50, generator=_gen(1), device=DEV)
    x[1] = 0.0
    x[2, 7] = float("nan")
    x[3, 8] = float("-inf")
    x[4] *= 2.0 ** -140          # scales among the subnormal numbers
    x[5] *= 2.0 ** -149
    x[6] = 3.4e38 * x[6].sign()
    x[7] = 0.0
    x[7, 49] = 2.0 ** -149       # a scale of 0
    q, scale = ops.quantize_rows(x)
    _check_rows(q, scale, x)
    assert torch.isnan(scale[2]) and torch.isnan(scale[3]) and scale[1] == 0 and scale[7] == 0
    assert q[[1, 2, 3, 7]].eq(0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_any_stride(ops, dtype):
    wide = torch.full((40, 77), float("nan"), dtype=dtype, device=DEV)
    wide[:, 3:73] = torch.randn(40, 70, generator=_gen(2), device=DEV).to(dtype)
    _check_rows(*ops.quantize_rows(wide[:, 3:73]), wide[:, 3:73])
    e = ops.quantize_rows(wide[:0])
    assert e[0].shape == (0, 77) and e[1].shape == (0,)


SIZES = [(1, 1, 1), (1, 768, 1000), (2, 64, 16), (3, 63, 17), (5, 65, 31), (16, 128, 256), (17, 129, 257),
         (33, 100, 1001), (64, 1000, 70), (65, 16, 300), (130, 768, 520), (257, 400, 1025), (700, 96, 64),
         (1000, 333, 1111), (300, 5000, 200)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,d,v", SIZES)
def test_product(ops, n, d, v, dtype):
    print(f"# int8 product n={n} d={d} v={v} {dtype}", flush=True)
    g = _gen(n + d + v)
    q = torch.randint(-128, 128, (n, d), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-128, 128, (v, d), generator=g, device=DEV, dtype=torch.int8)
    qs, ws = torch.rand(n, generator=g, device=DEV), torch.rand(v, generator=g, device=DEV)
    y = ops.quantized_product(q, qs, w, ws, dtype)
    assert y.dtype == dtype and torch.equal(y, _product(q, qs, w, ws, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,d,v", [(17, 1, 1), (64, 127, 63), (20, 129, 4000), (40, 4999, 200), (30, 20001, 37),
                                   (90, 255, 1000), (64, 1003, 32767), (20, 640, 500)])
@pytest.mark.parametrize("lead", [0, 1, 2, 4])
def test_rows_as_they_lie(ops, n, d, v, lead, dtype):
    # strides and starts at every remainder of 4, one cut step alone, whole steps alone, a split axis
    print(f"# int8 odd product n={n} d={d} v={v} lead={lead} {dtype}", flush=True)
    g = _gen(n + d + v + lead)
    a = torch.randint(-128, 128, (n, d + lead + 4), generator=g, device=DEV, dtype=torch.int8)
    b = torch.randint(-128, 128, (v, d + lead), generator=g, device=DEV, dtype=torch.int8)
    q, w = a[:, lead:lead + d], b[:, lead:]
    qs, ws = torch.rand(n, generator=g, device=DEV), torch.rand(v, generator=g, device=DEV)
    assert torch.equal(ops.quantized_product(q, qs, w, ws, dtype), _product(q, qs, w, ws, dtype))


@pytest.mark.parametrize("d", [130_999, 130_944])
def test_rows_in_chunks(ops, d):
    # more rows than are taken at a time, laid out and in place
    g = _gen(d)
    n, v = 2100, 40
    q = torch.randint(-128, 128, (n, d), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-128, 128, (v, d), generator=g, device=DEV, dtype=torch.int8)
    qs, ws = torch.rand(n, generator=g, device=DEV), torch.rand(v, generator=g, device=DEV)
    assert torch.equal(ops.quantized_product(q, qs, w, ws, F32), _product(q, qs, w, ws, F32))


def test_largest_sums(ops):
    d = (1 << 17) - 1
    q = torch.full((3, d), -128, dtype=torch.int8, device=DEV)
    w = torch.full((20, d), -128, dtype=torch.int8, device=DEV)
    w[1] = 127
    one = torch.ones(20, device=DEV)
    y = ops.quantized_product(q, one[:3], w, one, F32)
    assert torch.equal(y, _product(q, one[:3], w, one, F32))
    q2, w2 = q[:1].expand(300, d).contiguous(), w[:1].expand(300, d).contiguous()
    one = torch.ones(300, device=DEV)
    y = ops.quantized_product(q2, one, w2, one, F32)
    assert y.eq(float(d * 2 ** 14)).all()


def test_scales(ops):
    # scales of rows without numbers, signs, and products that leave fp32's range half way
    g = _gen(3)
    q = torch.randint(-128, 128, (20, 90), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-128, 128, (40, 90), generator=g, device=DEV, dtype=torch.int8)
    qs, ws = torch.randn(20, generator=g, device=DEV), torch.randn(40, generator=g, device=DEV)
    qs[3], ws[5], qs[6], ws[7] = float("nan"), float("nan"), 0.0, float("inf")
    qs[8], ws[9] = 1e-40, 1e38
    for dtype in (F32, BF16):
        y, ref = ops.quantized_product(q, qs, w, ws, dtype), _product(q, qs, w, ws, dtype)
        assert torch.equal(torch.isnan(y), torch.isnan(ref))
        assert torch.equal(y.nan_to_num(), ref.nan_to_num())


@pytest.mark.parametrize("n", [1, 7, 100, 600])
@pytest.mark.parametrize("shift", [0, 1, 16])
def test_strides_and_what_lies_around(ops, n, shift):
    g = _gen(4 + n)
    d, v = 384, 300
    for pad in (5, 16):
        a = torch.randint(-128, 128, (n, d + shift + pad), generator=g, device=DEV, dtype=torch.int8)
        b = torch.randint(-128, 128, (v, d + shift + pad), generator=g, device=DEV, dtype=torch.int8)
        q, w = a[:, shift:shift + d], b[:, shift:shift + d]
        qs, ws = torch.rand(n, generator=g, device=DEV), torch.rand(v, generator=g, device=DEV)
        for dtype in (F32, BF16):
            out = torch.full((n, v + 7), 5.0, dtype=dtype, device=DEV)
            ops.quantized_product(q, qs, w, ws, dtype, out=out[:, 3:3 + v])
            assert torch.equal(out[:, 3:3 + v], _product(q, qs, w, ws, dtype))
            assert out[:, :3].eq(5).all() and out[:, 3 + v:].eq(5).all()
    assert ops.quantized_product(q[:0], qs[:0], w, ws).shape == (0, v)


def test_offsets_beyond_32_bits(ops):
    g = _gen(5)
    n, d, v = 70_000, 64, 33_000  # 2.3e9 results
    q = torch.randint(-128, 128, (n, d), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-128, 128, (v, d), generator=g, device=DEV, dtype=torch.int8)
    qs, ws = torch.rand(n, generator=g, device=DEV), torch.rand(v, generator=g, device=DEV)
    y = ops.quantized_product(q, qs, w, ws)
    for part in (slice(0, 300), slice(n // 2, n // 2 + 300), slice(n - 300, n)):
        assert torch.equal(y[part], _product(q[part], qs[part], w, ws, BF16))


def test_wide_row_strides(ops):
    # rows 40 MB apart, 100 of them: offsets beyond 32 bits in the operands
    step, d, n = 40_000_000, 256, 100
    a = torch.zeros(n * step, dtype=torch.int8, device=DEV)
    q = a.as_strided((n, d), (step, 1))
    q.copy_(torch.randint(-128, 128, (n, d), generator=_gen(6), device=DEV, dtype=torch.int8))
    one = torch.ones(n, device=DEV)
    assert torch.equal(ops.quantized_product(q, one, q, one, F32), _product(q, one, q, one, F32))
    assert torch.equal(ops.quantized_product(q[:3], one[:3], q, one, F32), _product(q[:3], one[:3], q, one, F32))


def test_another_stream(ops):
    g = _gen(7)
    x = torch.randn(300, 200, generator=g, device=DEV)
    w, ws = ops.quantize_rows(torch.randn(500, 200, generator=g, device=DEV))
    a = ops.quantized_product(*ops.quantize_rows(x), w, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = ops.quantized_product(*ops.quantize_rows(x), w, ws)
    side.synchronize()
    assert torch.equal(a, b)


def test_refusals(ops):
    q = torch.zeros(3, 8, dtype=torch.int8, device=DEV)
    w = torch.zeros(5, 8, dtype=torch.int8, device=DEV)
    qs, ws = torch.ones(3, device=DEV), torch.ones(5, device=DEV)
    for bad in ((q, qs[:2], w, ws), (q, qs, w, ws.double()), (q, qs, w[:, :7], ws), (q, qs.cpu(), w, ws),
                (q.t(), qs, w, ws)):
        with pytest.raises(ValueError):
            ops.quantized_product(*bad)
    for bad in ((q.float(), qs, w, ws), (q, qs, w.to(torch.uint8), ws), (q, qs, w, ws, torch.float16)):
        with pytest.raises(TypeError):
            ops.quantized_product(*bad)
    with pytest.raises(ValueError):
        ops.quantized_product(q, qs, w, ws, out=torch.zeros(3, 5, device=DEV))
    with pytest.raises(ops.GmmError):
        ops.quantized_product(q, qs, w, ws, ws=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ops.GmmError):
        ops.quantize_rows(torch.zeros(1, 1 << 17, device=DEV))
    with pytest.raises(TypeError):
        ops.quantize_rows(q)
