"""The routed-expert and 8-bit integer operators against float64 references
(tests/experts_ref.py), at the sizes and inputs where they can go wrong. Every
tolerance is the bound derived there."""
import numpy as np
import pytest
import torch

import dense_gemm_persistent_gb300 as dg
import experts_ref as ref
from gpu_util import dev, status_ok

pytestmark = pytest.mark.gpu

BF, F32, I8, E4M3 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


def randint(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def close(got, want, tol):
    got = got.cpu().to(torch.float64)
    seen = ~torch.isnan(want)
    err = (got - want).abs()
    bad = seen & ~(err <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float((err / tol)[seen].max()), bad.nonzero()[:4].tolist())


# ------------------------------------------------------------------ routing

def run_route(x, k, renorm=True, dtype=F32):
    T, E = x.shape
    x = x.to(dtype)
    ids = torch.full((T, k), -7, dtype=torch.int32, device=dev())
    weights = torch.full((T, k), -7.0, device=dev())
    offsets = torch.full((E + 1,), -7, dtype=torch.int32, device=dev())
    row_token = torch.full((T * k,), -7, dtype=torch.int32, device=dev())
    slot_row = torch.full((T, k), -7, dtype=torch.int32, device=dev())
    ws = torch.full((max(16, dg.dgemm_route_workspace_size(T, E, k)),), 0xA5, dtype=torch.uint8, device=dev())
    dg.dgemm_route(x.to(dev()), k, ids, weights, offsets, row_token, slot_row, renormalize=renorm, ws=ws)
    want = ref.route(x.to(F32), k, renorm)
    assert ids.tolist() == want[0]
    assert offsets.tolist() == want[2]
    assert row_token.tolist() == want[3]
    assert slot_row.tolist() == want[4]
    w = torch.tensor(want[1], dtype=torch.float64).reshape(T, k)
    # exp (2 ulp), a sum of at most E terms, one division
    assert bool(((weights.cpu().double() - w).abs() <= w * (E + 8) * 2.0 ** -23 + 1e-37).all())


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 7, 7), (63, 33, 2), (64, 64, 1), (65, 100, 6),
                                   (130, 256, 8), (700, 24, 4), (5, 1000, 32), (257, 513, 3), (2100, 12, 3),
                                   (4500, 8, 2)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_route(T, E, k, dtype):
    run_route(randn(gen(T + E + k), T, E), k, True, dtype)


def test_route_softmax_over_all():
    run_route(3 * randn(gen(1), 90, 40), 5, False)


def test_route_equal_logits_take_the_lowest_expert():
    run_route(torch.zeros(70, 48), 6)
    run_route(randint(gen(2), 0, 3, 200, 96).float(), 8)
    run_route(torch.tensor([[0.0, -0.0, 0.0, -0.0]] * 3), 2)


def test_route_masked_entries_and_rows():
    x = randn(gen(3), 150, 20)
    x[:, 5] = -float("inf")                 # an expert that nobody may take
    x[10] = -float("inf")                   # a token without experts
    x[11, 2:] = -float("inf")               # fewer than k left
    x[12] = float("nan")
    x[13, ::2] = float("nan")
    x[14, 3] = float("inf")
    x[15] = float("inf")
    x[16] = -3.4028234663852886e38          # the type's lowest finite value is a logit like any other
    x[17] = 3.0e38
    for renorm in (True, False):
        run_route(x, 4, renorm)


def test_route_every_token_masked():
    run_route(torch.full((130, 9), -float("inf")), 3)


def test_route_one_expert_takes_all():
    x = randn(gen(4), 1000, 17)
    x[:, 11] += 100
    run_route(x, 2)


def test_route_no_tokens():
    offsets = torch.full((10,), -7, dtype=torch.int32, device=dev())
    e = torch.empty(0, 2, device=dev())
    i = torch.empty(0, 2, dtype=torch.int32, device=dev())
    dg.dgemm_route(torch.empty(0, 9, device=dev()), 2, i, e, offsets, torch.empty(0, dtype=torch.int32, device=dev()), i)
    assert offsets.tolist() == [0] * 10


# ------------------------------------------------------------------ combine

@pytest.mark.parametrize("T,H,k,out_dtype,with_add", [(1, 8, 1, BF, False), (3, 4096, 8, BF, True), (17, 1001, 3, F32, True),
                                                      (130, 264, 6, BF, False), (5, 7168, 2, F32, False),
                                                      (9, 72, 32, BF, True), (2, 1, 4, F32, False), (4, 20000, 2, BF, True)])
def test_combine(T, H, k, out_dtype, with_add):
    g = gen(T * 7 + H)
    R = T * k + 3
    Y = randn(g, R, H).to(BF)
    slot = torch.randperm(R, generator=g)[:T * k].reshape(T, k).to(torch.int32)
    w = torch.rand(T, k, generator=g)
    slot[0, 0] = -1                          # no expert
    if T > 2:
        slot[1, k - 1] = R                   # outside
        slot[2] = -1                         # a token without experts
    w[slot < 0] = float("nan")               # weights of absent rows are not used
    add = randn(g, T, H).to(BF) if with_add else None
    want, tol = ref.combine(Y, slot, w, add)
    out = torch.full((T, H), float("nan"), dtype=out_dtype, device=dev())
    dg.dgemm_combine(Y.to(dev()), slot.to(dev()), w.to(dev()), out, add=None if add is None else add.to(dev()))
    close(out, want, tol + (want.abs() + tol) * (2.0 ** -8 if out_dtype == BF else 2.0 ** -24) + 1e-37)


def test_combine_in_place_of_add():
    g = gen(8)
    Y, slot, w = randn(g, 12, 256).to(BF), i32([[0, 5], [11, 3]]), torch.rand(2, 2, generator=g)
    add = randn(g, 2, 256).to(BF)
    want, tol = ref.combine(Y, slot, w, add)
    buf = add.to(dev())
    dg.dgemm_combine(Y.to(dev()), slot.to(dev()), w.to(dev()), buf, add=buf)
    close(buf, want, tol + (want.abs() + tol) * 2.0 ** -8 + 1e-37)


# ------------------------------------------------------------------ grouped products

def sizes_to_offsets(sizes):
    return [0] + np.cumsum(sizes).tolist()


def make(kind, g, sizes, K, N, layout="nk", gather=False, ints=False, tokens=None):
    """Operands of one grouped call on the CPU."""
    E, R = len(sizes), sum(sizes)
    count = (tokens or max(1, R // 2)) if gather else R
    shape = (E, N, K) if layout == "nk" else (E, K, N)
    a = dict(offsets=i32(sizes_to_offsets(sizes)), a_rows=None, a_scale=None, b_scale=None)
    if gather:
        a["a_rows"] = randint(g, 0, count - 1, R).to(torch.int32)
    if kind == "bf16":
        a["A"] = (randint(g, -3, 3, count, K).float() if ints else randn(g, count, K)).to(BF)
        a["B"] = (randint(g, -3, 3, *shape).float() if ints else randn(g, *shape)).to(BF)
        return a
    if kind == "fp8":
        a["A"] = (randint(g, -3, 3, count, K).float() if ints else 8 * randn(g, count, K)).to(E4M3)
        a["B"] = (randint(g, -3, 3, *shape).float() if ints else 8 * randn(g, *shape)).to(E4M3)
    else:
        top = 3 if ints else 127
        a["A"] = randint(g, -top, top, count, K).to(I8)
        a["B"] = randint(g, -top, top, *shape).to(I8)
    one = (lambda *s: 2.0 ** randint(g, -2, 2, *s).float()) if ints else (lambda *s: 0.01 + 0.01 * torch.rand(*s, generator=g))
    a["a_scale"], a["b_scale"] = one(count), one(E, N)
    return a


def call(kind, a, D, layout="nk", **kw):
    """The call as the planner has it, then with single CTAs and with CTA pairs (the last result is
    in D): all three have the same bits, since an output's sum runs over K in the same order."""
    outs = []
    for pair in (-1, 0, 1):
        out = D if pair == 1 else D.clone()
        with dg.overrides(cta_pair=pair):
            call_once(kind, a, out, layout, **kw)
        outs.append(torch.nan_to_num(out.float(), nan=-12345.0))
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])
    return D


def call_once(kind, a, D, layout="nk", **kw):
    on = {k: (v.to(dev()) if v is not None else None) for k, v in a.items()}
    bias = kw.pop("bias", None)
    kw["bias"] = None if bias is None else bias.to(dev())
    if kind == "bf16":
        dg.dgemm_grouped_bf16(on["A"], on["B"], on["offsets"], D, a_rows=on["a_rows"], b_layout=layout, **kw)
    else:
        f = dg.dgemm_grouped_fp8_scaled if kind == "fp8" else dg.dgemm_grouped_int8_scaled
        f(on["A"], on["B"], on["a_scale"], on["b_scale"], on["offsets"], D, a_rows=on["a_rows"], **kw)
    assert status_ok(kw.get("ws"))
    return D


def check(kind, sizes, K, N, act="none", layout="nk", gather=False, out=BF, alpha=1.0, with_bias=False, seed=0, ints=False):
    g = gen(seed + K + N + sum(sizes))
    a = make(kind, g, sizes, K, N, layout, gather, ints)
    bias = randn(g, len(sizes), N) if with_bias else None
    want, tol = ref.grouped(a["A"], a["B"], a["offsets"].tolist(), a_rows=a["a_rows"], layout=layout,
                            a_scale=a["a_scale"], b_scale=a["b_scale"], bias=bias, act=act, alpha=alpha, out_dtype=out)
    wide = N // 2 if act == "swiglu" else N
    D = torch.full((sum(sizes), wide), float("nan"), dtype=out, device=dev())
    call(kind, a, D, layout, act=act, alpha=alpha, bias=bias)
    if ints:                                  # every sum and scale exact: the same bits
        assert torch.equal(D.cpu(), want.to(F32).to(out))
    else:
        close(D, want, tol)


KINDS = ["bf16", "fp8", "int8"]
SIZES = {
    "one row": [1],
    "one row each": [1] * 9,
    "empty groups": [0, 5, 0, 0, 17, 0],
    "ragged": [3, 64, 129, 1, 0, 40, 257],
    "skewed": [700, 0, 2, 1],
    "tile edges": [16, 32, 33, 63, 65, 127, 128, 255, 256, 260],
}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("act,gather", [("none", False), ("swiglu", True)])
def test_grouped_sizes(kind, name, act, gather):
    check(kind, SIZES[name], 144, 130, act, gather=gather)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K,N", [(16, 1), (16, 128), (64, 64), (128, 129), (192, 255), (272, 258), (1040, 384), (2064, 96)])
def test_grouped_channels_and_depths(kind, K, N):
    check(kind, [5, 0, 70], K, N, out=F32, with_bias=True)


@pytest.mark.parametrize("K", [8, 24, 72, 200, 520])
def test_grouped_bf16_short_rows(K):
    check("bf16", [4, 90, 0, 33], K, 77)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("kind", KINDS)
def test_grouped_activations(kind, act):
    check(kind, [10, 150, 3], 128, 200, act, out=F32, alpha=0.37, with_bias=True, gather=True)


@pytest.mark.parametrize("sizes", [[1], [7, 0, 300], [64, 64], [20, 19, 150]])
@pytest.mark.parametrize("K,N,act", [(64, 64, "none"), (136, 200, "gelu"), (520, 144, "swiglu"), (8, 8, "none"), (72, 1032, "silu")])
def test_grouped_kn(sizes, K, N, act):
    check("bf16", sizes, K, N, act, layout="kn", with_bias=True, gather=len(sizes) == 3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes,K,N", [([3, 0, 66, 130], 512, 320), ([1, 2, 3, 4, 5, 6, 7, 8], 1024, 256), ([600, 520], 256, 640)])
@pytest.mark.parametrize("out", [BF, F32])
def test_grouped_exact_on_integers(kind, sizes, K, N, out):
    check(kind, sizes, K, N, out=out, ints=True, gather=True)
    if kind == "bf16":
        check(kind, sizes, K, N, out=out, ints=True, layout="kn")


@pytest.mark.parametrize("kind", KINDS)
def test_grouped_many_experts(kind):
    sizes = [(i * 7) % 5 for i in range(300)]
    check(kind, sizes, 32, 40, gather=True)


def test_grouped_the_most_experts():
    check("bf16", [1 if i % 97 == 0 else 0 for i in range(1024)], 16, 24)


@pytest.mark.parametrize("kind", KINDS)
def test_grouped_rows_outside_every_group_are_not_written(kind):
    g = gen(5)
    a = make(kind, g, [4, 0, 6, 30], 64, 96)
    a["offsets"] = i32([3, 4, 4, 10, 37])     # rows 0-2 and 37-39 belong to nobody
    want, tol = ref.grouped(a["A"], a["B"], [3, 4, 4, 10, 37], a_scale=a["a_scale"], b_scale=a["b_scale"])
    D = torch.full((40, 96), 12.5, dtype=BF, device=dev())
    call(kind, a, D)
    assert bool((D[:3] == 12.5).all()) and bool((D[37:] == 12.5).all())
    close(D, want, tol)


@pytest.mark.parametrize("kind", KINDS)
def test_grouped_offsets_are_clamped(kind):
    """Offsets below zero, beyond R or descending stay inside the buffers."""
    a = make(kind, gen(6), [20], 64, 96)
    a["B"] = a["B"].expand(4, -1, -1).contiguous()
    if a["b_scale"] is not None:
        a["b_scale"] = a["b_scale"].expand(4, -1).contiguous()
    a["offsets"] = i32([-5, 8, 3, 12, 2000])  # groups [0,8), none, [3,12) over the second's end, [12,20)
    D = torch.full((20, 96), float("nan"), dtype=F32, device=dev())
    call(kind, a, D)
    want, tol = ref.grouped(a["A"], a["B"], [0, 20, 20, 20, 20], a_scale=a["a_scale"], b_scale=a["b_scale"], out_dtype=F32)
    close(D, want, tol)                       # the experts' weights are equal


@pytest.mark.parametrize("kind", KINDS)
def test_grouped_row_indexes_outside_read_as_zero(kind):
    a = make(kind, gen(7), [9, 70], 64, 40, gather=True)
    a["a_rows"][3], a["a_rows"][20], a["a_rows"][78] = -1, a["A"].shape[0], 2 ** 30
    bias = randn(gen(70), 2, 40)
    want, tol = ref.grouped(a["A"], a["B"], [0, 9, 79], a_rows=a["a_rows"], a_scale=a["a_scale"], b_scale=a["b_scale"], bias=bias)
    D = torch.full((79, 40), float("nan"), dtype=BF, device=dev())
    call(kind, a, D, bias=bias)
    close(D, want, tol)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_grouped_nan_stays_in_its_rows_and_experts(gather, layout):
    """A NaN row spoils its own outputs only, and a group never sees another expert's weights."""
    g = gen(9)
    a = make("bf16", g, [30, 20, 41], 72, 144, layout, gather)
    a["B"][1] = float("nan")
    a["A"][2] = float("inf")
    want, tol = ref.grouped(a["A"], a["B"], [0, 30, 50, 91], a_rows=a["a_rows"], layout=layout)
    rows = torch.arange(91) if a["a_rows"] is None else a["a_rows"].long()
    clean = (rows != 2) & ((torch.arange(91) < 30) | (torch.arange(91) >= 50))
    D = torch.zeros(91, 144, dtype=BF, device=dev())
    call("bf16", a, D, layout)
    assert bool(torch.isfinite(D.cpu()[clean]).all()) and bool(torch.isnan(D.cpu()[30:50]).all())
    close(D.cpu()[clean], want[clean], tol[clean])


@pytest.mark.parametrize("kind", KINDS)
def test_grouped_no_depth(kind):
    """K = 0: the product is zero and D = act(bias)."""
    a = make(kind, gen(10), [3, 0, 4], 0, 24)
    bias = randn(gen(11), 3, 24)
    D = torch.full((7, 24), float("nan"), dtype=F32, device=dev())
    call(kind, a, D, bias=bias, act="relu")
    assert torch.equal(D.cpu(), torch.cat([bias[0].clamp(min=0).expand(3, -1), bias[2].clamp(min=0).expand(4, -1)]))


@pytest.mark.parametrize("kind", KINDS)
def test_grouped_nothing_to_do(kind):
    a = make(kind, gen(12), [0, 0], 32, 16)
    call(kind, a, torch.empty(0, 16, dtype=BF, device=dev()))


@pytest.mark.parametrize("kind", KINDS)
def test_grouped_on_another_stream_and_twice(kind):
    """Results are the same bits on another stream, with a garbage workspace, and on a second call."""
    a = make(kind, gen(13), [50, 3, 200, 0, 77], 400, 264, gather=True)
    outs = []
    s = torch.cuda.Stream()
    ws = torch.full((max(256, dg.dgemm_grouped_workspace_size(kind, 330, 5, 264, 400)),), 0xEE, dtype=torch.uint8, device=dev())
    on = {k: (v.to(dev()) if v is not None else None) for k, v in a.items()}
    torch.cuda.synchronize()
    for stream in (None, s, s):
        D = torch.zeros(330, 264, dtype=BF, device=dev())
        torch.cuda.synchronize()
        call(kind, on, D, ws=ws, stream=stream)
        torch.cuda.synchronize()
        assert status_ok(ws, stream)
        outs.append(D.cpu())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ------------------------------------------------------------------ int8

@pytest.mark.parametrize("M,K", [(1, 16), (3, 7168), (130, 1001), (7, 1), (2, 20000), (65, 512)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_int8_quantize(M, K, dtype):
    g = gen(M + K)
    X = (randn(g, M, K) * torch.exp(3 * randn(g, M, 1))).to(dtype)
    X[0, 0] = 0.0
    if M > 2:
        X[1] = 0.0                                   # a row of zeros
        X[2, -1] = -1e30                             # all else rounds to 0
    q = torch.full((M, K), 99, dtype=I8, device=dev())
    s = torch.full((M,), -1.0, device=dev())
    dg.dgemm_int8_quantize(X.to(dev()), q, s)
    want_q, want_s = ref.quantize(X)
    assert torch.equal(s.cpu(), want_s) and torch.equal(q.cpu(), want_q)


def test_int8_quantize_ties_and_non_finite_values():
    x = torch.zeros(5, 24)
    x[0, :6] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5])     # scale 1: halves go to even
    x[1, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 2.0])
    x[2, :2] = torch.tensor([float("nan"), 0.0])
    x[3, :3] = torch.tensor([1e-45, -1e-45, 0.0])                    # the scale underflows
    x[4, :3] = torch.tensor([3.4e38, -3.4e38, 1.0])
    q = torch.empty(5, 24, dtype=I8, device=dev())
    s = torch.empty(5, device=dev())
    dg.dgemm_int8_quantize(x.to(dev()), q, s)
    want_q, want_s = ref.quantize(x)
    assert q[0, :6].tolist() == [127, 0, 2, 2, 0, -2]
    assert torch.equal(s.cpu(), want_s) and torch.equal(q.cpu(), want_q)


def check_int8(M, N, K, act="none", out=BF, with_bias=False, alpha=1.0, beta=0.0, c_dtype=F32, top=127, seed=0):
    g = gen(seed + M + N + K)
    A, B = randint(g, -top, top, M, K).to(I8), randint(g, -top, top, N, K).to(I8)
    sa, sb = 0.01 + 0.01 * torch.rand(M, generator=g), 0.001 + 0.001 * torch.rand(N, generator=g)
    bias = randn(g, N) if with_bias else None
    C = randn(g, M, N).to(c_dtype) if beta else None
    acc = A.to(torch.float64) @ B.to(torch.float64).t()
    scale = sa.double()[:, None] * sb.double()[None, :] * alpha
    y = acc * scale
    # below 2^24 the sums are exact: the scales' few roundings are left
    mags = A.abs().double() @ B.abs().double().t()
    dy = mags * scale.abs() * torch.where(mags < 2 ** 24, 0.0, (K / 8 + 4) * 2.0 ** -23) + y.abs() * 4 * 2.0 ** -24
    for extra in ((beta * C.double()) if beta else None, bias.double()[None, :] if with_bias else None):
        if extra is not None:
            dy = dy + (extra.abs() + y.abs()) * 2.0 ** -23
            y = y + extra
    v = ref.activation(y, act)
    dv = 1.13 * dy + (v.abs() * 2.0 ** -20 if act != "none" else 0.0)
    D = torch.full((M, N), float("nan"), dtype=out, device=dev())
    on = lambda x: None if x is None else x.to(dev())
    for pair in (-1, 0, 1):
        D.fill_(float("nan"))
        with dg.overrides(cta_pair=pair):
            dg.dgemm_int8_scaled(on(A), on(B), on(sa), on(sb), D, C=on(C), alpha=alpha, beta=beta, bias=on(bias), act=act)
            assert status_ok()
        close(D, v, dv + (v.abs() + dv) * (2.0 ** -8 if out == BF else 2.0 ** -24) + 1e-37)


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 300, 7168), (2, 129, 144), (5, 64, 1024), (8, 1000, 272), (9, 257, 528),
                                   (16, 128, 128), (17, 200, 1040), (33, 130, 96), (64, 512, 512), (65, 127, 208),
                                   (128, 256, 256), (300, 260, 400), (515, 1030, 144), (1000, 72, 64)])
@pytest.mark.parametrize("out", [BF, F32])
def test_int8_product(M, N, K, out):
    check_int8(M, N, K, out=out, with_bias=M % 2 == 1)


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("M", [1, 40, 200])
def test_int8_epilogue(M, act):
    check_int8(M, 136, 256, act, F32, True, alpha=0.5, beta=-1.5, c_dtype=BF)
    check_int8(M, 137, 256, act, BF, False, beta=2.0)


def test_int8_large_integers():
    """All codes at -127 or -128: sums beyond 2^24 stay within the FP32 bound; small ones are exact."""
    for K in (512, 4096):
        A = torch.full((130, K), -128, dtype=I8)
        B = torch.full((140, K), 127, dtype=I8)
        D = torch.empty(130, 140, device=dev())
        one = lambda n: torch.ones(n, device=dev())
        dg.dgemm_int8_scaled(A.to(dev()), B.to(dev()), one(130), one(140), D)
        want = -128.0 * 127.0 * K
        assert bool(((D.cpu().double() - want).abs() <= (0 if abs(want) <= 2 ** 24 else abs(want) * (K / 8 + 4) * 2.0 ** -23)).all())


def test_int8_in_place_and_no_depth():
    g = gen(21)
    A, B = randint(g, -9, 9, 50, 64).to(I8), randint(g, -9, 9, 70, 64).to(I8)
    one = lambda n: torch.ones(n, device=dev())
    C = randint(g, -99, 99, 50, 70).float()
    D = C.to(dev())
    dg.dgemm_int8_scaled(A.to(dev()), B.to(dev()), one(50), one(70), D, C=D, beta=1.0)
    assert torch.equal(D.cpu(), A.float() @ B.float().t() + C)
    D = C.to(dev())
    dg.dgemm_int8_scaled(A[:, :0].contiguous().to(dev()), B[:, :0].contiguous().to(dev()), one(50), one(70), D, C=D, beta=0.5)
    assert torch.equal(D.cpu(), 0.5 * C)


def test_route_bf16_infinity_beside_the_largest_number():
    """+inf is read as the largest FP32 number, above the largest BF16 one."""
    x = torch.zeros(70, 9)
    x[:, 2] = 3.3895313892515355e38
    x[:, 6] = float("inf")
    run_route(x, 3, True, BF)
    run_route(x, 3, False, BF)


# ------------------------------------------------------------------ bounded waits

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes,gather", [([20, 9, 14], False), ([20, 9, 14], True), ([300, 150], False), ([300, 150], True)])
def test_grouped_wait_that_runs_out_is_reported(kind, sizes, gather):
    """The weight producer stops after two copies (it issues nothing more): the waits for the
    next stage run out, the call reports it on its own status word, and the next call is right."""
    g = gen(31)
    K, N = 2048, 300
    a = make(kind, g, sizes, K, N, gather=gather, ints=True)
    R = sum(sizes)
    ws = torch.full((max(256, dg.dgemm_grouped_workspace_size(kind, R, len(sizes), N, K)),), 0x5A, dtype=torch.uint8, device=dev())
    on = {k: (v.to(dev()) if v is not None else None) for k, v in a.items()}
    D = torch.zeros(R, N, dtype=F32, device=dev())

    def one():
        if kind == "bf16":
            dg.dgemm_grouped_bf16(on["A"], on["B"], on["offsets"], D, a_rows=on["a_rows"], ws=ws)
        else:
            f = dg.dgemm_grouped_fp8_scaled if kind == "fp8" else dg.dgemm_grouped_int8_scaled
            f(on["A"], on["B"], on["a_scale"], on["b_scale"], on["offsets"], D, a_rows=on["a_rows"], ws=ws)

    with dg.overrides(stall_after_loads=2, wait_limit_ns=20_000_000, cta_pair=1 if sizes[0] == 300 else 0):
        one()
        assert dg.dgemm_query_device_status(ws) == 6      # DGEMM_ERR_DEVICE_TIMEOUT
    assert status_ok(ws)                                  # the query cleared it; the device word is untouched
    one()
    assert status_ok(ws)
    want, _ = ref.grouped(a["A"], a["B"], a["offsets"].tolist(), a_rows=a["a_rows"], a_scale=a["a_scale"], b_scale=a["b_scale"],
                          out_dtype=F32)
    assert torch.equal(D.cpu(), want.to(F32))


# ------------------------------------------------------------------ int8, few rows a group

@pytest.mark.parametrize("sizes", [[1], [2], [3, 0, 1], [4, 4], [5, 8, 0, 7], [16], [9, 23, 0, 1], [1] * 40, [40, 0, 0, 0]])
@pytest.mark.parametrize("K,N,act", [(16, 3, "none"), (528, 70, "swiglu"), (1040, 33, "gelu"), (4096, 130, "none")])
def test_grouped_int8_few_rows(sizes, K, N, act):
    check("int8", sizes, K, N, act, gather=len(sizes) > 1, with_bias=True, out=F32)
    check("int8", sizes, K, N, act)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 7, 8, 12, 16])
def test_int8_few_rows_exact(M):
    """Integers at the ends of their range: the sums are exact whatever their size."""
    K, N = 6000, 37
    g = gen(M)
    A = randint(g, 0, 1, M, K).mul(255).sub(128).to(I8)      # -128 or 127
    B = torch.full((N, K), -128, dtype=I8)
    one = lambda n: torch.ones(n, device=dev())
    D = torch.empty(M, N, device=dev())
    dg.dgemm_int8_scaled(A.to(dev()), B.to(dev()), one(M), one(N), D)
    want = A.to(torch.float64) @ B.to(torch.float64).t()
    assert torch.equal(D.cpu(), want.to(F32))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [64, 2048, 4096, 8192])
def test_int8_quantize_rows_with_infinities(K, dtype):
    """Rows held in registers: infinities and NaN beside finite values, and rows of nothing else."""
    g = gen(K)
    X = randn(g, 6, K).to(dtype)
    X[0, 3], X[0, K - 1] = float("inf"), -float("inf")
    X[1, 5] = float("nan")
    X[2] = float("nan")
    X[3] = float("inf")
    X[4, ::2] = -float("inf")
    q = torch.full((6, K), 99, dtype=I8, device=dev())
    s = torch.full((6,), -1.0, device=dev())
    dg.dgemm_int8_quantize(X.to(dev()), q, s)
    want_q, want_s = ref.quantize(X)
    assert torch.equal(s.cpu(), want_s) and torch.equal(q.cpu(), want_q)


def test_route_many_chunks():
    """More chunks of tokens than one folding of the packed counts takes."""
    g = gen(77)
    T, E, k = 40000, 5, 2
    x = randint(g, 0, 3, T, E).float().to(dev())
    ids = torch.empty(T, k, dtype=torch.int32, device=dev())
    w, offsets = torch.empty(T, k, device=dev()), torch.empty(E + 1, dtype=torch.int32, device=dev())
    row_token, slot_row = torch.empty(T * k, dtype=torch.int32, device=dev()), torch.empty(T, k, dtype=torch.int32, device=dev())
    ws = torch.empty(dg.dgemm_route_workspace_size(T, E, k), dtype=torch.uint8, device=dev())
    dg.dgemm_route(x, k, ids, w, offsets, row_token, slot_row, ws=ws)
    want = torch.sort(x.cpu(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.cpu().long(), want)
    flat = want.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(row_token.cpu().long(), order // k)
    assert torch.equal(slot_row.cpu().long().reshape(-1)[order], torch.arange(T * k))
    assert offsets.cpu().tolist() == [int((flat < e).sum()) for e in range(E + 1)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K", [48, 64, 80, 112, 128, 144, 176, 192, 208, 240, 256, 272, 304, 336, 400])
def test_grouped_depths_around_whole_slices(kind, K):
    """Depths that end inside, at and after a 128-byte slice, and after one or two slices of a
    pipeline stage, for short and long groups; NaN rows around the group show a read past a row."""
    for sizes in ([5, 60], [230, 90]):
        g = gen(K + sum(sizes))
        a = make(kind, g, sizes, K, 72)
        if kind == "bf16":
            a["A"][sizes[0]:] = float("nan")       # the second group's rows follow the first's
        want, tol = ref.grouped(a["A"], a["B"], a["offsets"].tolist(), a_scale=a["a_scale"], b_scale=a["b_scale"], out_dtype=F32)
        D = torch.full((sum(sizes), 72), 7.0, dtype=F32, device=dev())
        call(kind, a, D)
        first = slice(0, sizes[0]) if kind == "bf16" else slice(None)
        assert bool(torch.isfinite(D[first]).all())
        close(D[first], want[first], tol[first])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout,gather", [("nk", False), ("nk", True), ("kn", False), ("kn", True)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_grouped_more_than_one_wave(kind, layout, gather, act):
    """Enough tiles for CTA pairs with several tiles each: long groups beside short and empty ones."""
    if layout == "kn" and kind != "bf16":
        pytest.skip("K x N weights are BF16")
    sizes = [515, 0, 1, 290, 64, 33, 256, 700]
    g = gen(91)
    K, N = 200 if kind == "bf16" else 208, 2704
    a = make(kind, g, sizes, K, N, layout, gather, ints=True)
    rows = torch.arange(sum(sizes)) if a["a_rows"] is None else a["a_rows"].long()
    wide = N // 2 if act == "swiglu" else N
    D = torch.full((sum(sizes), wide), float("nan"), dtype=F32, device=dev())
    call(kind, a, D, layout, act=act)
    lo = 0
    for e, n in enumerate(sizes):
        b = a["B"][e].double()
        if act == "none":
            y = a["A"].double()[rows[lo:lo + n]] @ (b.t() if layout == "nk" else b)
            if a["a_scale"] is not None:
                y = y * a["a_scale"][rows[lo:lo + n]].double()[:, None] * a["b_scale"][e].double()
            assert torch.equal(D[lo:lo + n].cpu().double(), y)
        elif n:      # the group by itself, in few tiles: the same bits
            pick = lambda x: x.view(torch.uint8)[rows[lo:lo + n]].view(x.dtype) if x.dtype == E4M3 else x[rows[lo:lo + n]]
            one = dict(a, A=pick(a["A"]), B=a["B"][e:e + 1], offsets=i32([0, n]), a_rows=None)
            if a["a_scale"] is not None:
                one.update(a_scale=pick(a["a_scale"]), b_scale=a["b_scale"][e:e + 1])
            alone = torch.full((n, wide), float("nan"), dtype=F32, device=dev())
            if n > 4 or kind != "int8":      # (few int8 rows are summed in integers)
                assert torch.equal(D[lo:lo + n], call(kind, one, alone, layout, act=act))
        lo += n
