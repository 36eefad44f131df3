"""Routing by scores against the float64 definition (tests/adapters_ref.py): integers
equal, weights within a bound that is derived here."""
import pytest
import torch

import adapters_ref as ref
import dense_gemm_persistent_gb300 as dg
from gpu_util import dev

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def outputs(T, E, k):
    full = lambda *s: torch.full(s, -7, dtype=torch.int32, device=dev())
    return full(T, k), torch.full((T, k), -7.0, device=dev()), full(E + 1), full(T * k), full(T, k)


def run(x, k, *, score="sigmoid", bias=None, groups=1, kept=None, by="top2", renorm=True, scale=1.0, dtype=F32):
    T, E = x.shape
    x = x.to(dtype)
    out = outputs(T, E, k)
    ws = torch.full((max(256, dg.dgemm_route_workspace_size(T, E, k)),), 0xA5, dtype=torch.uint8, device=dev())
    dg.dgemm_route_scored(x.to(dev()), k, *out, score=score, bias=None if bias is None else bias.to(dev()), groups=groups,
                          groups_kept=kept, group_score=by, renormalize=renorm, scale=scale, ws=ws)
    want = ref.route_scored(x.to(F32), k, score, bias, groups, kept or groups, by, renorm, scale)
    ids, weights, offsets, row_token, slot_row = out
    assert ids.tolist() == want[0]
    assert offsets.tolist() == want[2]
    assert row_token.tolist() == want[3]
    assert slot_row.tolist() == want[4]
    # exp 2 ulp and its rounded argument (|x| up to 16 here unless the weight is 0 or 1), sums of up to E
    # terms, quotient, product with the scale
    w = torch.tensor(want[1], dtype=torch.float64).reshape(T, k)
    assert bool(((weights.cpu().double() - w).abs() <= w.abs() * (E + 40) * 2.0 ** -23 + abs(scale) * 1e-37).all())


@pytest.mark.parametrize("T,E,k,groups,kept", [(1, 1, 1, 1, 1), (1, 64, 8, 8, 4), (3, 6, 3, 3, 2), (64, 64, 6, 1, 1),
                                               (65, 100, 6, 5, 2), (130, 256, 8, 8, 4), (333, 160, 6, 8, 3), (7, 1024, 32, 32, 9),
                                               (40, 512, 31, 16, 5), (257, 33, 2, 3, 1), (2100, 24, 4, 4, 2), (90, 248, 8, 31, 7)])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("score,by,with_bias", [("sigmoid", "top2", True), ("softmax", "max", True), ("sigmoid", "max", False),
                                                ("softmax", "top2", False)])
def test_scores(T, E, k, groups, kept, dtype, score, by, with_bias):
    g = gen(T + E + k)
    x = torch.randn(T, E, generator=g)
    bias = (0.1 if score == "sigmoid" else 1.0 / E) * torch.randn(E, generator=g) if with_bias else None
    run(x, k, score=score, bias=bias, groups=groups, kept=kept, by=by, renorm=T % 2 == 1, scale=2.5, dtype=dtype)


def test_many_tokens_over_several_chunks():
    g = gen(9)
    run(torch.randn(9000, 16, generator=g), 3, bias=0.1 * torch.randn(16, generator=g), groups=4, kept=2, dtype=BF)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_equal_values_take_the_lowest(score):
    run(torch.zeros(70, 48), 6, score=score, bias=torch.zeros(48), groups=6, kept=2)
    run(torch.randint(0, 3, (200, 96), generator=gen(2)).float(), 8, score=score, bias=torch.zeros(96), groups=8, kept=3)
    run(torch.randint(0, 3, (200, 96), generator=gen(3)).float(), 8, score=score, groups=4, kept=2, by="max")
    run(torch.tensor([[0.0, -0.0, 0.0, -0.0]] * 3), 2, score=score, bias=torch.zeros(4))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,kept,by", [(1, 1, "max"), (4, 2, "top2"), (4, 3, "max")])
def test_values_that_fp32_cannot_tell_apart(score, groups, kept, by):
    # biases that make up for the scores' differences: c is the same up to one rounding of FP32
    g = gen(5)
    E = 32
    x = torch.randn(1, E, generator=g).expand(50, E).clone()
    x[25:] += 0.001 * torch.randn(25, E, generator=g)
    s = torch.sigmoid(x[0].double()) if score == "sigmoid" else torch.softmax(x[0].double(), 0)
    for level in (0.5, 2.0):
        run(x, 5, score=score, bias=(level - s).float(), groups=groups, kept=kept, by=by)
    # pairs of neighbours in FP32 around one value
    bias = (1.0 - s).float()
    bias[::2] = torch.nextafter(bias[::2], torch.tensor(9.0))
    run(x, 31, score=score, bias=bias)
    run(x, 32, score=score, bias=bias)
    run(x, 1, score=score, bias=bias, groups=groups, kept=kept, by=by)


def test_masked_entries_groups_and_rows():
    g = gen(3)
    x = torch.randn(150, 24, generator=g)
    inf = float("inf")
    x[:, 5] = -inf                   # an expert that nobody may take
    x[10] = -inf                     # a token without experts
    x[11, 2:] = -inf                 # fewer than k left
    x[12] = float("nan")
    x[13, ::2] = float("nan")
    x[14, 3] = inf
    x[15] = inf
    x[16] = -3.4028234663852886e38   # the type's lowest finite value is a logit like any other
    x[17] = 3.0e38
    x[18, :18] = -inf                # one group left
    x[19, 6:18] = -inf               # two of four
    x[20, 1:6] = -inf                # a group of one
    bias = 0.1 * torch.randn(24, generator=g)
    bias[7], bias[8], bias[9] = -inf, float("nan"), inf
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            for b in (None, bias):
                for by in ("max", "top2"):
                    run(x, 4, score=score, bias=b, groups=4, kept=2, by=by, renorm=renorm)
                run(x, 4, score=score, bias=b, renorm=renorm)


@pytest.mark.parametrize("kept", [1, 2, 3])
def test_sums_of_two_that_fp32_cannot_hold(kept):
    # every one of the first groups' sums is infinite in FP32
    bias = torch.tensor([1.8e38, 1.8e38, 3.0e38, 3.0e38, 2.0e38, 2.9e38, 3.1e38, 3.0e38, 0.5, 0.1])
    for b in (bias, -bias, bias.roll(4)):
        run(torch.randn(9, 10, generator=gen(kept)), 2, bias=b, groups=5, kept=kept)


def test_scores_that_underflow():
    x = torch.linspace(-80, -130, 64).repeat(70, 1)
    run(x, 4, bias=torch.zeros(64))
    run(x, 4, bias=torch.zeros(64), groups=4, kept=2)
    x[:, 0] = 0.0
    run(x, 4, score="softmax", bias=torch.linspace(0, 1, 64))


def test_a_softmax_row_like_dgemm_route():
    x = torch.randn(300, 40, generator=gen(8)).to(dev())
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=dev())
    for renorm in (True, False):
        a, b = outputs(300, 40, 5), outputs(300, 40, 5)
        dg.dgemm_route(x, 5, *a, renormalize=renorm, ws=ws)
        dg.dgemm_route_scored(x, 5, *b, score="softmax", renormalize=renorm, ws=ws)
        for i in (0, 2, 3, 4):
            assert torch.equal(a[i], b[i])
        assert torch.allclose(a[1], b[1], rtol=2e-5, atol=0)


def test_no_tokens():
    offsets = torch.full((10,), -7, dtype=torch.int32, device=dev())
    e, i = torch.empty(0, 2, device=dev()), torch.empty(0, 2, dtype=torch.int32, device=dev())
    dg.dgemm_route_scored(torch.empty(0, 9, device=dev()), 2, i, e, offsets, torch.empty(0, dtype=torch.int32, device=dev()), i,
                          groups=3)
    assert offsets.tolist() == [0] * 10


def test_the_same_bits_every_time_on_another_stream_and_in_a_graph():
    g = gen(4)
    T, E, k = 5000, 256, 8
    x = torch.randn(T, E, generator=g).to(BF).to(dev())
    bias = (0.1 * torch.randn(E, generator=g)).to(dev())
    ws = torch.empty(dg.dgemm_route_workspace_size(T, E, k), dtype=torch.uint8, device=dev())
    call = lambda out: dg.dgemm_route_scored(x, k, *out, bias=bias, groups=8, groups_kept=4, ws=ws)
    first, again, replayed = outputs(T, E, k), outputs(T, E, k), outputs(T, E, k)
    call(first)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call(again)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(replayed)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, again, replayed):
        assert torch.equal(a, b) and torch.equal(a, c)
