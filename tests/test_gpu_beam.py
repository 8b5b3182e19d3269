"""A step of beam search and the move of its states against plain float64 forms.

Logits lie on a grid, so that those of one beam are equal or apart by far more than rounding. Tolerance of
a score, set before the first run: l - max and the score's sum round by 2^-24 of themselves; the
logarithm's sum of V positive terms is off by 2^-24 (V / 64 + 64), which covers the exponentials'
2^-24 (1.5 d + 4) where exp(-d) counts, and the logarithm rounds once:
2^-24 (V / 64 + 64 + 4 (|l - max| + log sum + |score|)). Continuations whose scores are further apart than
twice that have to come in order; within a beam equal logits come by code.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _logits(rows, v, dtype, g, masked=False):
    x = (torch.randn(rows, v, generator=g, device=DEV) * 40).round().clamp(-255, 255) / 16
    if masked:
        x[torch.rand(rows, v, generator=g, device=DEV) < 0.5] = -INF
    return x.to(dtype)


def _check(ops, logits, scores, last=None, end=-1, m=None, scale=1.0, r=None):
    b, w = scores.shape
    v = logits.shape[1]
    if r is None:
        r = ops.beam_step(logits, scores, last, end, m, scale)
    m = w if m is None else m
    assert r.parent.shape == r.code.shape == r.score.shape == (b, m)
    l = (logits.float() * torch.tensor(scale, dtype=F32, device=DEV)).double()
    bad = torch.isnan(l).any(1, keepdim=True) | (l == INF).any(1, keepdim=True)
    top = torch.where(torch.isnan(l), -INF, l).amax(1, keepdim=True)
    top = top.masked_fill(top == -INF, 0.0)
    d = l - top
    logs = torch.log(torch.exp(d).sum(1, keepdim=True))
    lp = (d - logs).masked_fill(bad | (l == -INF), -INF).view(b, w, v)
    s = scores.double()
    alive = torch.isfinite(s)
    cand = (s[:, :, None] + lp).masked_fill(~alive[:, :, None], -INF)
    tol = 2.0 ** -24 * (v / 64 + 64 + 4 * (d.abs().view(b, w, v) + logs.abs().view(b, w, 1) + s.abs()[:, :, None]))
    code = torch.arange(v, device=DEV).expand(b, w, v)
    if last is not None and end >= 0:
        ended = (last == end) & alive
        cand[ended], tol[ended] = -INF, 0.0
        cand[:, :, 0] = torch.where(ended, s, cand[:, :, 0])
        code = torch.where(ended[:, :, None], end, code)
    # descending by score; equal ones by beam and by code
    val, at = cand.view(b, -1).sort(dim=1, descending=True, stable=True)
    if val.shape[1] <= m:
        pad = m + 1 - val.shape[1]
        val = torch.nn.functional.pad(val, (0, pad), value=-INF)
        at = torch.nn.functional.pad(at, (0, pad))
    val, at = val[:, :m + 1], at[:, :m + 1]
    t = tol.reshape(b, -1).gather(1, at).nan_to_num(0.0)
    none = val[:, :m] == -INF
    assert torch.equal(r.score == -INF, none) and bool(torch.isfinite(r.score[~none]).all())
    assert r.parent[none].eq(-1).all() and r.code[none].eq(-1).all()
    off = (r.score.double() - val[:, :m]).masked_fill(none, 0.0).abs()
    assert bool((off <= t[:, :m]).all()), (off / t[:, :m]).max()
    # what was chosen has the score that it is said to have, and nothing is chosen twice
    ended = torch.zeros_like(alive) if last is None else (last == end) & (end >= 0)
    pc, cc = r.parent.long().clamp(min=0), r.code.long().clamp(min=0)
    cc = torch.where(ended.gather(1, pc), 0, cc)
    mine = cand.view(b, -1).gather(1, pc * v + cc).masked_fill(none, 0.0)
    assert bool(((r.score.double().masked_fill(none, 0.0) - mine).abs() <= 2 * t[:, :m]).all())
    key = torch.where(none, -1 - torch.arange(m, device=DEV), pc * v + cc)
    assert bool((key.sort(1).values.diff(dim=1) != 0).all())
    # the order, where rounding does not decide it
    want_p, want_c = at[:, :m] // v, code.reshape(b, -1).gather(1, at[:, :m])
    gap = val[:, :-1] - val[:, 1:]
    same = (at[:, :-1] // v) == (at[:, 1:] // v)
    fine = (gap > 2 * (t[:, :-1] + t[:, 1:])) | same | ~torch.isfinite(gap)
    sure = fine & torch.cat([torch.ones_like(fine[:, :1]), fine[:, :-1]], 1) & ~none
    assert torch.equal(r.parent[sure].long(), want_p[sure]) and torch.equal(r.code[sure].long(), want_c[sure])
    return r, sure


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,w,m,v", [(1, 1, 1, 1), (1, 1, 16, 3), (2, 3, 3, 2), (3, 1, 8, 1000), (5, 4, 4, 257),
                                     (2, 16, 16, 5000), (1, 5, 2, 40009), (70, 2, 2, 100), (1, 2, 16, 131072),
                                     (300, 3, 5, 33), (1, 16, 16, 300_007), (9, 16, 1, 64)])
def test_step(ops, b, w, m, v, dtype):
    print(f"# beam b={b} w={w} m={m} v={v} {dtype}", flush=True)
    g = _gen(b + w + m + v)
    scores = -3 * torch.rand(b, w, generator=g, device=DEV)
    x = _logits(b * w, v, dtype, g)
    r, _ = _check(ops, x, scores, m=m, scale=0.7)
    again = ops.beam_step(x, scores, m=m, scale=0.7)
    assert all(torch.equal(p, q) for p, q in zip(r, again))
    _check(ops, _logits(b * w, v, dtype, g, True), scores, m=m)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("v", [50, 9000, 140_000])
def test_ended_and_dead_beams(ops, v, dtype):
    g = _gen(v)
    b, w = 12, 6
    x = _logits(b * w, v, dtype, g, True)
    scores = -2 * torch.rand(b, w, generator=g, device=DEV)
    last = torch.randint(0, v, (b, w), generator=g, device=DEV, dtype=torch.int32)
    last[last == 7] = 8
    last[::2, 1] = 7                 # ended
    scores[1::3, 2] = -INF           # dead
    scores[2, 0], scores[2, 3] = float("nan"), INF
    scores[3] = -INF                 # a search without beams
    last[4], scores[4, 2] = 7, -0.5  # all ended
    x[5 * w:6 * w] = -INF            # nothing to go on with
    x[6 * w + 1, v // 2] = float("nan")
    x[6 * w + 2, v // 3] = INF
    x[7 * w, :] = torch.finfo(dtype).min
    last[8, 1], scores[8, 1] = 7, -INF   # ended, but dead
    x.view(b, w, v)[last == 7] = float("nan")  # rows that are not read
    r, _ = _check(ops, x, scores, last, 7)
    assert r.parent[3].eq(-1).all() and r.code[4].eq(7).all()
    assert torch.equal(r.score[4], scores[4].sort(descending=True).values)
    assert torch.equal(r.parent[4].sort().values.long(), torch.arange(w, device=DEV))
    # an end that no code is: nothing has ended
    x = _logits(b * w, v, dtype, g)
    s = -2 * torch.rand(b, w, generator=g, device=DEV)
    for end in (-1, -5):
        a = ops.beam_step(x, s, torch.full_like(last, end), end)
        assert all(torch.equal(p, q) for p, q in zip(a, ops.beam_step(x, s)))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("v", [5, 9000, 200_000])
def test_searches_of_one_beam(ops, v, dtype):
    g = _gen(v + 1)
    for m in (1, 8, 16):
        x = _logits(9, v, dtype, g, True)
        scores = -2 * torch.rand(9, 1, generator=g, device=DEV)
        last = torch.zeros(9, 1, dtype=torch.int32, device=DEV)
        last[1], last[2], scores[2], scores[3] = 4, 4, -INF, float("nan")  # ended, ended but dead, dead
        x[1:4] = float("nan")
        x[4, 1], x[5, 2], x[6] = float("nan"), INF, -INF
        x[7], x[7, 3] = -INF, 0.5
        r, _ = _check(ops, x, scores, last, 4, m=m)
        assert r.code[1, 0] == 4 and r.score[1, 0] == scores[1, 0]
        assert r.parent[1:8, 1:].eq(-1).all() and r.parent[2:7].eq(-1).all()
        assert r.code[7, 0] == 3 and abs(r.score[7, 0] - scores[7, 0]) <= 2.0 ** -22


def test_order_of_equal_scores(ops):
    # equal logits everywhere: beams in order, then codes
    for v, m in ((4, 10), (5000, 16), (200_000, 3)):
        r = ops.beam_step(torch.zeros(3 * 4, v, device=DEV), torch.zeros(3, 4, device=DEV), m=m)
        at = torch.arange(m, device=DEV)
        assert torch.equal(r.parent, (at // v).expand(3, m).to(torch.int32))
        assert torch.equal(r.code, (at % v).expand(3, m).to(torch.int32))
    # two logits whose scores round to one: the larger logit first, though its code is larger
    x = torch.full((1, 8), -50.0, device=DEV)
    x[0, 2], x[0, 5] = 0.0, 2.0 ** -20
    r = ops.beam_step(x, torch.full((1, 1), -1000.0, device=DEV), m=2)
    assert r.code[0].tolist() == [5, 2] and r.score[0, 0] == r.score[0, 1]


def test_scores_out_of_range(ops):
    # finite scores whose sum with a code's is not: no continuation
    x = torch.zeros(1, 4, device=DEV)
    x[0, 1] = -3.0e38
    r = ops.beam_step(x, torch.full((1, 1), -3.0e38, device=DEV), m=4)
    assert r.code[0].tolist() == [0, 2, 3, -1] and r.score[0, 3] == -INF


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides(ops, dtype):
    g = _gen(3)
    x = _logits(6, 901, dtype, g)
    wide = torch.full((6, 915), float("nan"), dtype=dtype, device=DEV)
    wide[:, 5:906] = x
    s = -torch.rand(2, 3, generator=g, device=DEV)
    a, b = ops.beam_step(x, s, m=7), ops.beam_step(wide[:, 5:906], s, m=7)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    e = ops.beam_step(x[:0], s[:0])
    assert e.parent.shape == (0, 3)


@pytest.mark.parametrize("w", [1, 2])
def test_more_searches_than_workgroups(ops, w):
    g = _gen(40 + w)
    b, v = 1_100_003, 8
    x = _logits(b * w, v, F32, g)
    scores = -4 * torch.rand(b, w, generator=g, device=DEV)
    _check(ops, x, scores, m=2)


def test_offsets_beyond_32_bits(ops):
    g = _gen(4)
    b, w, v = 4200, 16, 33_000  # 2.2e9 logits
    x = torch.randint(-128, 128, (b * w, v), generator=g, device=DEV, dtype=torch.int8).to(BF16)
    x /= 16
    s = -torch.rand(b, w, generator=g, device=DEV)
    r = ops.beam_step(x, s, m=4)
    for part in (slice(0, 3), slice(b - 3, b)):
        _check(ops, x.view(b, w, v)[part].reshape(3 * w, v), s[part], m=4, r=ops.Beams(*(t[part] for t in r)))


def _moved(state, parent, w, dim):
    s = state.movedim(dim, 0)
    b, m = parent.shape
    at = (parent.long().clamp(0, w - 1) + w * torch.arange(b, device=DEV)[:, None]).view(-1)
    out = s[at].clone()
    out[((parent < 0) | (parent >= w)).view(-1)] = 0
    return out.movedim(0, dim)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int8, BF16, torch.float64, torch.bool])
@pytest.mark.parametrize("b,w,m,shape,dim", [(1, 1, 1, (1,), 0), (3, 4, 4, (4, 7), 0), (2, 1, 8, (2, 33), 0),
                                             (5, 16, 16, (3, 80, 5, 3), 1), (2, 3, 2, (2, 2, 6, 4111), 2),
                                             (4, 2, 5, (8,), 0), (1, 5, 5, (2, 5, 70000), 1)])
def test_reorder(ops, b, w, m, shape, dim, dtype):
    print(f"# reorder b={b} w={w} m={m} {shape} dim={dim} {dtype}", flush=True)
    g = _gen(b + w + m)
    shape = list(shape)
    shape[dim] = b * w
    state = torch.randint(-100, 100, shape, generator=g, device=DEV).to(dtype)
    parent = torch.randint(0, w, (b, m), generator=g, device=DEV, dtype=torch.int32)
    parent[torch.rand(b, m, generator=g, device=DEV) < 0.2] = -1
    parent[0, 0] = w  # not a beam
    want = _moved(state, parent, w, dim)
    out = ops.beam_reorder(state, parent, w, dim)
    assert out.dtype == dtype and out.is_contiguous() and torch.equal(out, want)
    assert torch.equal(ops.beam_reorder(state, parent, w, dim - len(shape)), want)
    if m == w:
        got = ops.beam_reorder(state, parent, w, dim, out=state)
        assert got is state and torch.equal(state, want)


def test_reorder_of_views(ops):
    g = _gen(5)
    b, w = 3, 4
    cache = torch.randint(-100, 100, (2, b * w, 20, 6), generator=g, device=DEV, dtype=torch.int32)
    keep = cache.clone()
    parent = torch.randint(0, w, (b, w), generator=g, device=DEV, dtype=torch.int32)
    # the places filled so far of a longer cache, in place: the others stay as they were
    ops.beam_reorder(cache[:, :, :13], parent, w, 1, out=cache[:, :, :13])
    assert torch.equal(cache[:, :, :13], _moved(keep[:, :, :13], parent, w, 1))
    assert torch.equal(cache[:, :, 13:], keep[:, :, 13:])
    # layers inside the beams' memory
    turned = keep.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(ops.beam_reorder(turned, parent, w, 1), _moved(keep, parent, w, 1))
    ops.beam_reorder(turned, parent, w, 1, out=turned)
    assert torch.equal(turned, _moved(keep, parent, w, 1))
    # one state that all beams share, at odd addresses
    flat = torch.randint(-100, 100, (500,), generator=g, device=DEV, dtype=torch.int8)
    one = flat[3:460].expand(b * w, 457)
    assert torch.equal(ops.beam_reorder(one, parent, w), one)
    out = torch.full((b * w, 470), 9, dtype=torch.int8, device=DEV)
    ops.beam_reorder(one, parent, w, out=out[:, 5:462])
    assert torch.equal(out[:, 5:462], one) and out[:, :5].eq(9).all() and out[:, 462:].eq(9).all()
    assert ops.beam_reorder(one[:0], parent[:0], w).shape == (0, 457)
    assert ops.beam_reorder(keep[:0], parent, w, 1).shape == (0, b * w, 20, 6)


def test_reorder_of_large_states(ops):
    b, w = 2, 3
    state = torch.arange(6, device=DEV, dtype=torch.int8)[:, None].repeat(1, (1 << 30) + 77)  # 6 GB
    parent = torch.tensor([[2, 0, 1], [1, 1, -1]], dtype=torch.int32, device=DEV)
    want = torch.tensor([2, 0, 1, 4, 4, 0], device=DEV, dtype=torch.int8)
    out = ops.beam_reorder(state, parent, w)
    for t in (out, ops.beam_reorder(state, parent, w, out=state)):
        for k in (0, 1 << 20, (1 << 30) + 76):
            assert torch.equal(t[:, k], want)
        assert torch.equal(t.amax(1), want) and torch.equal(t.amin(1), want)


def test_another_stream(ops):
    g = _gen(6)
    x, s = _logits(40, 3000, F32, g), -torch.rand(10, 4, generator=g, device=DEV)
    state = torch.randn(40, 100, generator=g, device=DEV)
    a = ops.beam_step(x, s)
    c = ops.beam_reorder(state, a.parent, 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = ops.beam_step(x, s)
        e = ops.beam_reorder(state, b.parent, 4)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and torch.equal(c, e)


def test_refusals(ops):
    x = torch.zeros(6, 10, device=DEV)
    s = torch.zeros(2, 3, device=DEV)
    last = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    for bad in (dict(scores=s[:1]), dict(scores=s[0]), dict(scores=s.double()), dict(scores=s.t()),
                dict(last=last.long()), dict(last=last[:1]), dict(last=last.cpu()), dict(logits=x[:5])):
        with pytest.raises(ValueError):
            ops.beam_step(**(dict(logits=x, scores=s) | bad))
    for bad in (dict(m=0), dict(m=17), dict(scale=0.0), dict(scale=float("nan")), dict(end=1 << 40),
                dict(ws=torch.zeros(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ops.GmmError):
            ops.beam_step(x, s, **bad)
    with pytest.raises(ops.GmmError):
        ops.beam_step(torch.zeros(17, 10, device=DEV), torch.zeros(1, 17, device=DEV), m=2)
    with pytest.raises(TypeError):
        ops.beam_step(x.half(), s)
    parent = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    for bad in (dict(parent=parent.long()), dict(parent=parent[0]), dict(w=2), dict(dim=2), dict(dim=-3),
                dict(out=torch.zeros(6, 9, device=DEV)), dict(state=x.t()), dict(state=x.cpu()),
                dict(state=x[:, ::2])):
        with pytest.raises(ValueError):
            ops.beam_reorder(**(dict(state=x, parent=parent, w=3) | bad))
    with pytest.raises(ops.GmmError):  # in place, but other counts of beams
        ops.beam_reorder(x[:4], torch.zeros(2, 3, dtype=torch.int32, device=DEV), 2, out=x)
    with pytest.raises(ops.GmmError):  # rows of the result that overlap
        ops.beam_reorder(x, parent, 3, out=torch.zeros(10, device=DEV).expand(6, 10))


def test_no_beams(ops):
    none = torch.zeros(0, 10, device=DEV)
    parent = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    with pytest.raises(ops.GmmError):
        ops.beam_step(none, torch.zeros(2, 0, device=DEV))
    for state in (none, none.expand(0, 10), torch.zeros(10, 0, device=DEV).t()):
        with pytest.raises(ops.GmmError):
            ops.beam_reorder(state, parent, 0)
    assert ops.beam_reorder(none, parent[:0], 3).shape == (0, 10)
