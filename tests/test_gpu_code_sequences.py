"""The operators for sequences of codes together, as the example uses them: gradients of the
model's training step against differences, beams against their own log-probabilities, and a
decoding step captured into a graph."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda:0"


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("code_sequences", os.path.join(ROOT, "examples", "code_sequences.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.fixture(scope="module")
def result(example):
    return example.main(n=3000, k=16, steps=3, queries=20, w=4)


@pytest.fixture(scope="module")
def ops():
    from gmm_em_amd import ops as o

    return o


def test_runs(result):
    assert len(result["losses"]) == 3 and all(x == x and abs(x) < 1e3 for x in result["losses"] + result["balance"])
    found, k = result["found"], result["k"]
    assert found.shape == (20, 4, 3)
    assert ((found[:, :, 0] >= 2) & (found[:, :, 0] < 2 + k)).all()
    assert ((found[:, :, 1] >= 2 + k) & (found[:, :, 1] < 2 + 2 * k)).all() and found[:, :, 2].eq(1).all()
    assert (result["scores"].diff(dim=1) <= 0).all()


def test_beams_have_their_log_probabilities(example, ops, result):
    # each sequence's score is the sum of its codes' log-probabilities, from the same logits
    # (8-bit rows: each step's logits are made again, bit for bit, from the same states)
    found, k, v = result["found"], result["k"], result["table"].shape[0]
    b, w, _ = found.shape
    hidden = result["q"].repeat_interleave(w, 0)
    prev = torch.full((b * w,), example.START, dtype=torch.int32, device=DEV)
    total = torch.zeros(b * w, device=DEV, dtype=torch.float64)
    for t in range(3):
        hidden = hidden + ops.embed(result["table"], prev)
        logits = ops.quantized_product(*ops.quantize_rows(hidden), result["head"], result["head_scale"], torch.float32)
        logits.masked_fill_(example.step_mask(k, v, t, DEV), float("-inf"))
        prev = found[:, :, t].reshape(-1).contiguous()
        total += ops.logits_score(logits, prev).logprob.double()
    # three sums of numbers below 64, and the logarithms of sums of 34 terms
    assert ((total.view(b, w) - result["scores"].double()).abs() <= 3 * 2.0 ** -24 * (64 * 4 + 80)).all()


def test_training_gradient_against_differences(ops):
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    n, d, v, scale = 40, 24, 30, 1.5
    h, table, head, turn = (torch.randn(s, d, generator=g, device=DEV) for s in (n, v, v, v))
    codes, target = (torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int32) for _ in range(2))

    def loss(t):
        x = h.double() + scale * t.double()[codes.long()]
        return -torch.log_softmax(x @ head.double().t() / 4, 1).gather(1, target.long()[:, None]).mean()

    hidden = h + ops.embed(table, codes, scale)
    s = ops.head_score(hidden, head, target, scale=0.25)
    assert abs(-s.logprob.double().mean() - loss(table)) < 1e-4
    dh, _ = ops.head_score_backward(hidden, head, target, s.norm, s.entropy, torch.full((n,), -1.0 / n, device=DEV),
                                    scale=0.25)
    dt = ops.embed_backward(dh, codes, v, scale)
    step = 1e-4
    change = (loss(table.double() + step * turn.double()) - loss(table.double() - step * turn.double())) / (2 * step)
    # the difference's own error is step^2 times a third derivative (below 10^3 along this turn), and
    # the kernels' fp32 sums are off by 2^-18 of their terms
    assert abs(change - (dt.double() * turn.double()).sum()) <= 1e-5 + 2.0 ** -18 * (dt * turn).abs().sum()


def test_decoding_step_in_a_graph(example, ops, result):
    # replays with other states in the same buffers, between eager work, give the eager step's results
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    d, v, w, b = result["q"].shape[1], result["table"].shape[0], 4, 5
    off = example.step_mask(result["k"], v, 0, DEV)
    hidden = torch.zeros(b * w, d, dtype=torch.bfloat16, device=DEV)
    scores = torch.zeros(b, w, device=DEV)
    last = torch.zeros(b, w, dtype=torch.int32, device=DEV)
    z, idx = torch.zeros(2000, 12, device=DEV), torch.zeros(2000, 2, dtype=torch.int32, device=DEV)
    grad, many = torch.zeros(3000, 40, device=DEV), torch.zeros(3000, dtype=torch.int32, device=DEV)

    def step():
        beams, _ = example.decode_step(hidden, result["head"], result["head_scale"], off, scores, last, w)
        moved = ops.beam_reorder(hidden, beams.parent, w)
        out = moved + ops.embed(result["table"], beams.code.view(-1))
        r = ops.balance_loss(z, idx)
        dz = ops.balance_loss_backward(z, r.counts, r.totals, r.norm)
        return (*beams, out, *r, dz, ops.embed_backward(grad, many, 70), ops.embed_backward(grad[:50], many[:50], 70))

    def fill():
        hidden.copy_(torch.randn(b * w, d, generator=g, device=DEV))
        scores.copy_(-torch.rand(b, w, generator=g, device=DEV))
        last.copy_(torch.randint(0, 5, (b, w), generator=g, device=DEV))
        z.copy_(torch.randn(2000, 12, generator=g, device=DEV))
        idx.copy_(torch.randint(-2, 12, (2000, 2), generator=g, device=DEV))
        grad.copy_(torch.randn(3000, 40, generator=g, device=DEV))
        many.copy_(torch.randint(-2, 70, (3000,), generator=g, device=DEV))

    fill()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(4):
        fill()
        graph.replay()
        got = [t.clone() for t in captured]
        torch.cuda.synchronize()
        for a, e in zip(got, step()):
            assert torch.equal(a, e)


def test_calls_at_once_on_two_streams(ops):
    # each call has a workspace of its own: neither sees the other
    g = torch.Generator(device=DEV)
    g.manual_seed(3)

    def inputs():
        grad = torch.randn(30_000, 256, generator=g, device=DEV)
        codes = torch.randint(0, 500, (30_000,), generator=g, device=DEV, dtype=torch.int32)
        z = torch.randn(30_000, 200, generator=g, device=DEV)
        logits = torch.randn(64, 20_000, generator=g, device=DEV)
        x, w = torch.randn(300, 500, generator=g, device=DEV), torch.randn(700, 500, generator=g, device=DEV)
        return grad, codes, z, z.topk(3, 1).indices.to(torch.int32), logits, torch.zeros(8, 8, device=DEV), x, w

    def work(grad, codes, z, idx, logits, scores, x, w):
        r = ops.balance_loss(z, idx)
        return (ops.embed_backward(grad, codes, 500), *r, ops.balance_loss_backward(z, r.counts, r.totals, r.norm),
                *ops.beam_step(logits, scores), ops.quantized_product(*ops.quantize_rows(x), *ops.quantize_rows(w)))

    data = [inputs(), inputs()]
    want = [work(*d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for k, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[k].append(work(*data[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for result in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(result, want[k]))
