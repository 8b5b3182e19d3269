"""Embedding of codes and its gradient against plain float64 forms.

Tolerances, set before the first run. Forward: the product rounds by 2^-24 of itself and a bf16
result by another 2^-8. Gradient: a sum of k fp32 values in any order is off by at most
(k - 1) 2^-24 of the sum of their magnitudes; the product with the scale and the result's
rounding add 2^-24 and, for bf16, 2^-8 of the result.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
ROUND = {F32: 2.0 ** -24, BF16: 2.0 ** -8 + 2.0 ** -24}
TINY = 2.0 ** -133  # half a step of the smallest bf16 values


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _codes(n, v, g, skew=3):
    c = (v * torch.rand(n, generator=g, device=DEV) ** skew).to(torch.int32).clamp_(max=v - 1)
    c[torch.rand(n, generator=g, device=DEV) < 0.1] = -1
    return c


def _check_embed(out, table, codes, scale):
    s = float(torch.tensor(scale, dtype=F32))
    ref = table.double()[codes.long().clamp(0, table.shape[0] - 1)] * s
    ref[codes < 0] = 0.0
    ref[codes >= table.shape[0]] = float("nan")
    assert out.dtype == table.dtype and out.shape == ref.shape
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    off = (out.double() - ref).abs().nan_to_num()
    assert bool((off <= ROUND[table.dtype] * ref.abs().nan_to_num() + TINY).all())


def _check_grad(out, grad, codes, v, scale):
    s = float(torch.tensor(scale, dtype=F32))
    keep = (codes >= 0) & (codes < v)
    g, c = grad.double()[keep], codes[keep].long()
    zero = torch.zeros(v, grad.shape[1], dtype=torch.float64, device=DEV)
    ref, size = zero.clone(), zero.clone()
    count = torch.zeros(v, dtype=torch.float64, device=DEV)
    ref.index_add_(0, c, g)
    size.index_add_(0, c, g.abs())
    count.index_add_(0, c, torch.ones(len(c), dtype=torch.float64, device=DEV))
    ref *= s
    tol = count[:, None] * 2.0 ** -24 * size * abs(s) + (ROUND[grad.dtype] + 2.0 ** -24) * ref.abs() + TINY
    assert out.dtype == grad.dtype and out.shape == ref.shape
    bad = (out.double() - ref).abs() > tol
    assert not bool(bad.any()), (bad.nonzero()[:5], ((out.double() - ref).abs() / tol).max())
    assert bool(out[count == 0].eq(0).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,d,v", [(1, 1, 1), (1, 768, 100), (3, 7, 5), (64, 8, 2), (65, 9, 513), (33, 1030, 40),
                                   (1000, 100, 1001), (4099, 64, 512), (2500, 33, 70000), (129, 4097, 300)])
def test_forward_and_gradient(ops, n, d, v, dtype):
    print(f"# embed n={n} d={d} v={v} {dtype}", flush=True)
    g = _gen(n + d + v)
    table = torch.randn(v, d, generator=g, device=DEV).to(dtype)
    codes = _codes(n, v, g)
    _check_embed(ops.embed(table, codes, 1.7), table, codes, 1.7)
    grad = torch.randn(n, d, generator=g, device=DEV).to(dtype)
    _check_grad(ops.embed_backward(grad, codes, v, -0.3), grad, codes, v, -0.3)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["all_one", "all_none", "outside", "sorted", "segment", "two_tiles"])
def test_gradient_of_uneven_codes(ops, kind, dtype):
    # one code in many segments, runs that end at a segment's border, several tiles
    g = _gen(7)
    n, d, v = {"two_tiles": 300_001, "segment": 64 * 9}.get(kind, 5000), 40, 700
    if kind == "all_one":
        codes = torch.full((n,), v - 1, dtype=torch.int32, device=DEV)
    elif kind == "all_none":
        codes = torch.full((n,), -7, dtype=torch.int32, device=DEV)
    elif kind == "outside":
        codes = torch.randint(-v, 3 * v, (n,), generator=g, device=DEV, dtype=torch.int32)
        codes[0], codes[1] = 2 ** 31 - 1, -2 ** 31
    elif kind == "sorted":
        codes = _codes(n, v, g).sort().values.to(torch.int32)
    elif kind == "segment":
        codes = torch.arange(n, device=DEV, dtype=torch.int32) // 64
        codes[:64] = 1  # 128 rows, from a segment's first to another's last
    else:
        codes = _codes(n, v, g)
    print(f"# embed gradient {kind} {dtype}", flush=True)
    grad = torch.randn(n, d, generator=g, device=DEV).to(dtype)
    a = ops.embed_backward(grad, codes, v, 2.0)
    _check_grad(a, grad, codes, v, 2.0)
    assert torch.equal(a, ops.embed_backward(grad, codes, v, 2.0))


@pytest.mark.parametrize("n,run", [(1025, 8), (2048, 16), (5000, 32), (300_000, 64), (70_000, 2000)])
def test_runs_that_meet_segments(ops, n, run):
    # runs as long as segments are, a shorter one in front so that they straddle them, one code none
    g = _gen(n)
    for first in (0, 1, run // 2):
        codes = ((torch.arange(n, device=DEV) + first) // run).to(torch.int32)
        codes[codes == 3] = -1
        v = int(codes.max()) + 5
        perm = torch.randperm(n, generator=g, device=DEV)
        grad = torch.randn(n, 20, generator=g, device=DEV)
        for c in (codes, codes[perm].contiguous()):
            _check_grad(ops.embed_backward(grad, c, v), grad, c, v, 1.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [1024, 1025, 2048, 2049, 4096, 4097])
@pytest.mark.parametrize("d", [3, 260, 513, 1500, 5000])
def test_either_side_of_few_rows(ops, n, d, dtype):
    g = _gen(n + d)
    codes = _codes(n, 90, g)
    codes[::5] = 17
    grad = torch.randn(n, d, generator=g, device=DEV).to(dtype)
    _check_grad(ops.embed_backward(grad, codes, 90, 0.5), grad, codes, 90, 0.5)


@pytest.mark.parametrize("v", [1, 2, 3, 63, 64, 127, 1023, 1024, 1025])
@pytest.mark.parametrize("n", [1500, 5000])
def test_small_tables(ops, n, v):
    # digits of one bit to ten, all rows in few runs
    g = _gen(v)
    codes = torch.randint(-1, v + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
    grad = torch.randn(n, 30, generator=g, device=DEV)
    _check_grad(ops.embed_backward(grad, codes, v), grad, codes, v, 1.0)


def test_three_digits(ops):
    # codes of more than 20 bits are sorted in three steps
    g = _gen(8)
    v, n, d = 3_000_007, 20_000, 24
    codes = torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int32)
    codes[::3] = v - 1
    grad = torch.randn(n, d, generator=g, device=DEV)
    _check_grad(ops.embed_backward(grad, codes, v), grad, codes, v, 1.0)


def test_no_rows(ops):
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    for dtype in (F32, BF16):
        table = torch.ones(5, 3, dtype=dtype, device=DEV)
        assert ops.embed(table, none).shape == (0, 3)
        out = torch.full((5, 8), 7.0, dtype=dtype, device=DEV)
        ops.embed_backward(table[:0], none, 5, out=out[:, 2:5])
        assert out[:, 2:5].eq(0).all() and out[:, :2].eq(7).all() and out[:, 5:].eq(7).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides_and_what_lies_around(ops, dtype):
    g = _gen(9)
    n, d, v = 777, 101, 50
    wide = torch.full((v, d + 5), float("nan"), dtype=dtype, device=DEV)
    wide[:, 3:3 + d] = torch.randn(v, d, generator=g, device=DEV).to(dtype)
    codes = _codes(n, v, g)
    out = torch.full((n, d + 9), 7.0, dtype=dtype, device=DEV)
    table = wide[:, 3:3 + d]
    ops.embed(table, codes, 0.5, out=out[:, 1:1 + d])
    _check_embed(out[:, 1:1 + d], table, codes, 0.5)
    assert out[:, 0].eq(7).all() and out[:, 1 + d:].eq(7).all()
    big = torch.full((n, d + 4), float("nan"), dtype=dtype, device=DEV)
    big[:, 1:1 + d] = torch.randn(n, d, generator=g, device=DEV).to(dtype)
    dt = torch.full((v, d + 3), 7.0, dtype=dtype, device=DEV)
    ops.embed_backward(big[:, 1:1 + d], codes, v, 0.5, out=dt[:, 2:2 + d])
    _check_grad(dt[:, 2:2 + d], big[:, 1:1 + d], codes, v, 0.5)
    assert dt[:, :2].eq(7).all() and dt[:, 2 + d:].eq(7).all()


def test_infinities_stay_in_their_rows(ops):
    table = torch.ones(4, 5, device=DEV)
    table[1, 2], table[2, 0] = float("inf"), float("nan")
    codes = torch.tensor([0, 1, 2, 3, 4, -1], dtype=torch.int32, device=DEV)
    out = ops.embed(table, codes, 2.0)
    assert out[1, 2] == float("inf") and torch.isnan(out[2, 0]) and torch.isnan(out[4]).all()
    assert out[[0, 3]].eq(2).all() and out[5].eq(0).all()
    codes = torch.tensor([0, 1, 0, 3], dtype=torch.int32, device=DEV)
    dt = ops.embed_backward(table, codes, 6)
    assert torch.isnan(dt[0, 0]) and dt[0, 1:].eq(2).all() and dt[1, 2] == float("inf")
    assert dt[3].eq(1).all() and dt[[2, 4, 5]].eq(0).all()


def test_offsets_beyond_32_bits(ops):
    g = _gen(10)
    n, d, v = (1 << 25) + 3, 70, 11
    codes = torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int32)
    table = torch.randn(v, d, generator=g, device=DEV).to(BF16)
    out = ops.embed(table, codes)
    for part in (slice(0, 1000), slice(n // 2, n // 2 + 1000), slice(n - 1000, n)):
        assert torch.equal(out[part], table[codes[part].long()])
    # whole numbers: the sums are exact
    out.fill_(1.0)
    dt = ops.embed_backward(out[:, :3], codes, v)
    count = torch.bincount(codes, minlength=v)
    assert torch.equal(dt, count[:, None].expand(v, 3).float().to(BF16))


def test_gradient_against_differences(ops):
    g = _gen(11)
    n, d, v, scale = 300, 20, 37, 1.5
    table = torch.randn(v, d, generator=g, device=DEV)
    turn = torch.randn(v, d, generator=g, device=DEV)
    grad = torch.randn(n, d, generator=g, device=DEV)
    codes = _codes(n, v, g)
    dt = ops.embed_backward(grad, codes, v, scale).double()
    h = 0.25  # the call is linear: any step will do

    def loss(t):
        return (ops.embed(t, codes, scale).double() * grad.double()).sum()

    change = (loss(table + h * turn) - loss(table - h * turn)) / (2 * h)
    # table +- h turn and the products round by 2^-24 of values below 8
    tol = 3 * 8 * 2.0 ** -24 / h * grad.double().abs().sum()
    assert abs(change - (dt * turn.double()).sum()) <= tol


def test_another_stream(ops):
    g = _gen(12)
    codes = _codes(3000, 500, g)
    table = torch.randn(500, 96, generator=g, device=DEV)
    grad = torch.randn(3000, 96, generator=g, device=DEV)
    a, b = ops.embed(table, codes), ops.embed_backward(grad, codes, 500)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c, e = ops.embed(table, codes), ops.embed_backward(grad, codes, 500)
    side.synchronize()
    assert torch.equal(a, c) and torch.equal(b, e)


def test_refusals(ops):
    table = torch.zeros(4, 6, device=DEV)
    codes = torch.zeros(3, dtype=torch.int32, device=DEV)
    for bad in (codes.long(), codes.cpu(), codes[None], torch.zeros(6, dtype=torch.int32, device=DEV)[::2]):
        with pytest.raises(ValueError):
            ops.embed(table, bad)
    with pytest.raises(TypeError):
        ops.embed(table.half(), codes)
    with pytest.raises(ValueError):
        ops.embed(table.t(), codes)
    with pytest.raises(ValueError):
        ops.embed(table, codes, out=torch.zeros(3, 5, device=DEV))
    with pytest.raises(ValueError):
        ops.embed(table, codes, out=torch.zeros(3, 6, device=DEV, dtype=BF16))
    with pytest.raises(ops.GmmError):
        ops.embed(table, codes, float("inf"))
    grad = torch.zeros(3, 6, device=DEV)
    with pytest.raises(ValueError):
        ops.embed_backward(grad, codes[:2], 4)
    for v in (0, -1, (1 << 22) + 1, 1 << 40):
        with pytest.raises(ops.GmmError):
            ops.embed_backward(grad, codes, v)
    with pytest.raises(ops.GmmError):
        ops.embed_backward(grad, codes, 4, ws=torch.zeros(16, dtype=torch.uint8, device=DEV))
