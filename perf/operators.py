"""The routed-expert and 8-bit integer operators as measured cases.

Four operators of a mixture-of-experts feed-forward block and of the linear
layers beside it:

  route     router logits -> the top-k experts of each token, their weights, and
            the grouping of the (token, slot) pairs by expert
  combine   the weighted sum of each token's expert rows, plus an optional row
            (a shared expert, a residual)
  grouped   matrix products grouped by expert, D[r] = epilogue(A[row] . op(B_e)),
            ragged group sizes held on the device; BF16, FP8 E4M3 and INT8
  int8      a linear layer in 8-bit integers: activations quantised per token,
            multiplied with per-channel quantised weights

Each case runs either in its plain form (elementary torch operations in 32
bits) or, where ``own`` is true, through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
WORKSPACE_BYTES = 32 * 2 ** 20


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the router of one decoding token: nothing but latency
        dict(name="route one token", op="route", T=1, E=64, k=8, logits="f32", renorm=True),
        # a long prompt over many experts; BF16 logits bring ties
        dict(name="route long prompt", op="route", T=16001, E=256, k=8, logits="bf16", renorm=True),
        # the expert rows of a few decoding sequences
        dict(name="combine few tokens", op="combine", T=12, H=4096, k=8, add=True),
        # the same for a long prompt
        dict(name="combine long prompt", op="combine", T=8192, H=7168, k=8, add=False),
        # decoding: 8 sequences, every token its own experts, gate and up projections fused with their product
        dict(name="grouped decode gated", op="grouped", type="bf16", T=8, E=64, k=8, K=2048, N=2816, act="swiglu",
             gather=True, layout="nk", bias=False, out="bf16"),
        # a prompt's first projection: gathered token rows, gated
        dict(name="grouped prompt gated", op="grouped", type="bf16", T=4096, E=16, k=4, K=4096, N=4096, act="swiglu",
             gather=True, layout="nk", bias=False, out="bf16"),
        # a prompt's second projection: rows already grouped, odd sizes
        dict(name="grouped down odd", op="grouped", type="bf16", T=997, E=24, k=3, K=1416, N=2049, act="none",
             gather=False, layout="nk", bias=True, out="bf16"),
        # weights stored K x N (or the gradient of the rows of an N x K layer)
        dict(name="grouped kn", op="grouped", type="bf16", T=2048, E=32, k=2, K=2048, N=4096, act="gelu",
             gather=False, layout="kn", bias=True, out="bf16"),
        # E4M3 experts with per-token and per-channel scales
        dict(name="grouped fp8 gated", op="grouped", type="fp8", T=4096, E=32, k=4, K=4096, N=4096, act="swiglu",
             gather=True, layout="nk", bias=False, out="bf16"),
        # integer experts: a batch of decoding sequences, few rows each
        dict(name="grouped int8 batch", op="grouped", type="int8", T=192, E=64, k=4, K=4096, N=2048, act="none",
             gather=True, layout="nk", bias=False, out="bf16"),
        # an integer linear layer of one decoding token: the weights' bytes are all
        dict(name="int8 decode", op="int8", M=1, N=18432, K=7168, act="none", bias=False, out="bf16"),
        # the same kind of layer on a prompt
        dict(name="int8 prompt", op="int8", M=4096, N=11008, K=4096, act="silu", bias=True, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case. Sizes run over their ranges' logarithms; K keeps rows on 16
    bytes (the entry points ask for that), everything else may be odd."""
    op = rng.choice(["route", "combine", "grouped", "grouped", "grouped", "int8", "int8"])
    if op == "route":
        E = _log(rng, 8, 256)
        return dict(op=op, T=_log(rng, 1, 16000), E=E, k=rng.randint(1, min(8, E)), logits=rng.choice(["f32", "bf16"]),
                    renorm=rng.random() < 0.7)
    if op == "combine":
        return dict(op=op, T=_log(rng, 1, 8000), H=8 * _log(rng, 16, 896), k=rng.randint(1, 8), add=rng.random() < 0.5)
    if op == "grouped":
        kind = rng.choice(["bf16", "bf16", "fp8", "int8"])
        unit = 8 if kind == "bf16" else 16
        c = dict(op=op, type=kind, T=_log(rng, 1, 4000), E=_log(rng, 2, 64), k=1, K=unit * _log(rng, 128 // unit, 4096 // unit),
                 N=_log(rng, 64, 4096), act=rng.choice(["none", "relu", "gelu", "silu", "swiglu", "swiglu"]),
                 gather=rng.random() < 0.5, layout="nk", bias=rng.random() < 0.4, out="bf16")
        c["k"] = rng.randint(1, min(4, c["E"]))
        if kind == "bf16" and rng.random() < 0.3:
            c["layout"] = "kn"
        if c["layout"] == "kn":
            c["N"] = 16 * max(4, c["N"] // 16)
        elif c["act"] == "swiglu":
            c["N"] = 2 * (c["N"] // 2)
        return c
    return dict(op=op, M=_log(rng, 1, 4000), N=_log(rng, 64, 11000), K=16 * _log(rng, 8, 256),
                act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _router_logits(g, T, E):
    """Scores with popular and unpopular experts, as a trained router gives them."""
    return _randn(g, T, E) + 0.5 * _randn(g, 1, E)


def _grouping(g, T, E, k):
    """Tokens grouped by expert: offsets [E+1], the token of each row, and (for the
    plain form) each row's expert, its place inside the group and the longest group."""
    ids = torch.topk(_router_logits(g, T, E), k, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices
    count = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(count, 0).to(torch.int32)
    expert = ids[order]
    place = torch.arange(T * k, device=DEV) - offsets[expert].long()
    return offsets, (order // k).to(torch.int32), expert, place, int(count.max())


def _weights_int8(g, *shape):
    """Normal weights quantised per output channel (the last dimension is K)."""
    w = _randn(g, *shape)
    s = w.abs().amax(-1, keepdim=True) / 127.0
    q = torch.round(w / s).to(torch.int8)
    return q, (0.02 * s.squeeze(-1)).contiguous()


def _rows_e4m3(x):
    s = x.abs().amax(-1, keepdim=True) / 448.0
    return (x / s).to(torch.float8_e4m3fn), s.squeeze(-1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _router_logits(g, T, E).to(torch.float32 if case["logits"] == "f32" else torch.bfloat16)
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        s["row_token"] = torch.empty(T * k, dtype=torch.int32, device=DEV)
        s["slot_row"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
    elif op == "combine":
        T, H, k = case["T"], case["H"], case["k"]
        s["Y"] = _randn(g, T * k, H).to(torch.bfloat16)
        s["slot_row"] = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).reshape(T, k)
        s["weights"] = torch.softmax(_randn(g, T, k), 1).contiguous()
        s["add"] = _randn(g, T, H).to(torch.bfloat16) if case["add"] else None
        s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    elif op == "grouped":
        T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
        s["offsets"], token, s["expert"], s["place"], s["longest"] = _grouping(g, T, E, k)
        rows = T if case["gather"] else T * k
        x = _randn(g, rows, K) * torch.exp(0.5 * _randn(g, rows, 1))
        s["a_rows"] = token if case["gather"] else None
        s["a_scale"] = s["b_scale"] = None
        if case["type"] == "bf16":
            s["A"] = x.to(torch.bfloat16)
            s["B"] = (_randn(g, E, N, K) if case["layout"] == "nk" else _randn(g, E, K, N)).mul_(K ** -0.5).to(torch.bfloat16)
        elif case["type"] == "fp8":
            s["A"], s["a_scale"] = _rows_e4m3(x)
            s["B"], s["b_scale"] = _rows_e4m3(_randn(g, E, N, K))
            s["b_scale"] = s["b_scale"] * K ** -0.5
        else:
            s["a_scale"] = (x.abs().amax(-1) / 127.0).contiguous()
            s["A"] = torch.round(x / s["a_scale"][:, None]).to(torch.int8)
            s["B"], s["b_scale"] = _weights_int8(g, E, N, K)
        s["bias"] = 0.1 * _randn(g, E, N) if case["bias"] else None
        wide = N // 2 if case["act"] == "swiglu" else N
        s["D"] = torch.empty(T * k, wide, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=DEV)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["X"] = (_randn(g, M, K) * torch.exp(0.5 * _randn(g, M, 1))).to(torch.bfloat16)
        s["B"], s["b_scale"] = _weights_int8(g, N, K)
        s["bias"] = 0.1 * _randn(g, N) if case["bias"] else None
        s["q"] = torch.empty(M, K, dtype=torch.int8, device=DEV)
        s["a_scale"] = torch.empty(M, dtype=torch.float32, device=DEV)
        s["D"] = torch.empty(M, N, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=DEV)
    # a workspace that a program keeps for all of its calls
    s["ws"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms

def _activation(y, act):
    if act == "relu":
        return torch.clamp_min(y, 0.0)
    if act == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y * 0.5 ** 0.5))
    if act == "silu":
        return y / (1.0 + torch.exp(-y))
    if act == "swiglu":
        half = y.shape[-1] // 2
        return y[..., :half] / (1.0 + torch.exp(-y[..., :half])) * y[..., half:]
    return y


def _plain_route(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = s["logits"].float()
    value, index = torch.sort(x, dim=1, descending=True, stable=True)   # equal logits: the lowest index first
    e = torch.exp(value - value[:, :1])
    p = e[:, :k]
    weights = p / (p if c["renorm"] else e).sum(1, keepdim=True)
    ids = index[:, :k].contiguous()
    flat = ids.reshape(-1)
    grouped, order = torch.sort(flat, stable=True)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(T * k, device=x.device)
    offsets = torch.searchsorted(grouped, torch.arange(E + 1, device=x.device))
    return [ids.to(torch.int32), weights, offsets.to(torch.int32), (order // k).to(torch.int32),
            rank.reshape(T, k).to(torch.int32)]


def _plain_combine(s):
    y = s["Y"][s["slot_row"].long()].float()
    out = (y * s["weights"][:, :, None]).sum(1)
    if s["add"] is not None:
        out = out + s["add"].float()
    return out.to(torch.bfloat16)


def _plain_grouped(s):
    c = s["case"]
    E, longest = c["E"], s["longest"]
    a = s["A"] if s["a_rows"] is None else s["A"][s["a_rows"].long()]
    a = a.float()
    if s["a_scale"] is not None:
        a = a * (s["a_scale"] if s["a_rows"] is None else s["a_scale"][s["a_rows"].long()])[:, None]
    b = s["B"].float()
    if s["b_scale"] is not None:
        b = b * s["b_scale"][:, :, None]
    padded = torch.zeros(E, longest, c["K"], device=a.device)
    padded[s["expert"], s["place"]] = a
    y = torch.bmm(padded, b.transpose(1, 2) if c["layout"] == "nk" else b)
    if s["bias"] is not None:
        y = y + s["bias"][:, None, :]
    y = y[s["expert"], s["place"]]
    return _activation(y, c["act"]).to(s["D"].dtype)


def _plain_int8(s):
    x = s["X"].float()
    scale = x.abs().amax(1) / 127.0
    q = torch.round(x / scale[:, None])
    y = (q @ s["B"].float().t()) * scale[:, None] * s["b_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return [q.to(torch.int8), scale, _activation(y, s["case"]["act"]).to(s["D"].dtype)]


# ------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"route": _plain_route, "combine": _plain_combine, "grouped": _plain_grouped, "int8": _plain_int8}[c["op"]](s)
    import dense_gemm_persistent_gb300 as dg
    if c["op"] == "route":
        dg.dgemm_route(s["logits"], c["k"], s["ids"], s["weights"], s["offsets"], s["row_token"], s["slot_row"],
                       renormalize=c["renorm"], ws=s["ws"])
        return [s["ids"], s["weights"], s["offsets"], s["row_token"], s["slot_row"]]
    if c["op"] == "combine":
        return dg.dgemm_combine(s["Y"], s["slot_row"], s["weights"], s["out"], add=s["add"])
    if c["op"] == "grouped":
        more = dict(a_rows=s["a_rows"], bias=s["bias"], act=c["act"], ws=s["ws"])
        if c["type"] == "bf16":
            return dg.dgemm_grouped_bf16(s["A"], s["B"], s["offsets"], s["D"], b_layout=c["layout"], **more)
        call = dg.dgemm_grouped_fp8_scaled if c["type"] == "fp8" else dg.dgemm_grouped_int8_scaled
        return call(s["A"], s["B"], s["a_scale"], s["b_scale"], s["offsets"], s["D"], **more)
    dg.dgemm_int8_quantize(s["X"], s["q"], s["a_scale"])
    dg.dgemm_int8_scaled(s["q"], s["B"], s["a_scale"], s["b_scale"], s["D"], bias=s["bias"], act=c["act"], ws=s["ws"])
    return [s["q"], s["a_scale"], s["D"]]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * (4 if case["logits"] == "f32" else 2) + T * k * 16 + 4 * (E + 1), "flops": 4 * T * E}
    if op == "combine":
        T, H, k = case["T"], case["H"], case["k"]
        return {"bytes": T * k * (2 * H + 8) + T * H * (4 if case["add"] else 2), "flops": 2 * T * k * H}
    if op == "grouped":
        T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
        size, R = (2 if case["type"] == "bf16" else 1), T * k
        used = E * (1.0 - (1.0 - 1.0 / E) ** R)   # experts that get any row, were they equally popular
        wide = N // 2 if case["act"] == "swiglu" else N
        scales = 0 if case["type"] == "bf16" else 4 * (R + used * N)
        return {"bytes": int((T if case["gather"] else R) * K * size + used * N * K * size + scales + R * wide * (2 if case["out"] == "bf16" else 4)
                             + (4 * used * N if case["bias"] else 0) + 4 * (E + 1) + (4 * R if case["gather"] else 0)),
                "flops": 2 * R * N * K}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": 3 * M * K + N * K + M * N * (2 if case["out"] == "bf16" else 4) + 4 * (M + N) + (4 * N if case["bias"] else 0),
            "flops": 2 * M * N * K}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The definition, element by element or row by row, in float64."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        x = s["logits"].double()
        chosen = []
        left = x.clone()
        for _ in range(case["k"]):   # the largest that is left, the lowest index among equals
            top = left.amax(1, keepdim=True)
            at = (left == top).to(torch.int8).argmax(1, keepdim=True)
            chosen.append(x.gather(1, at))
            left.scatter_(1, at, -math.inf)
        v = torch.cat(chosen, 1)
        base = torch.logsumexp(v if case["renorm"] else x, 1, keepdim=True)
        return [None, torch.exp(v - base), None, None, None]
    if op == "combine":
        out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=DEV)
        for j in range(case["k"]):
            out += s["weights"][:, j].double()[:, None] * s["Y"].index_select(0, s["slot_row"][:, j].long()).double()
        return out if s["add"] is None else out + s["add"].double()
    if op == "grouped":
        bounds = s["offsets"].tolist()
        out = torch.empty(s["D"].shape, dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            lo, hi = bounds[e], bounds[e + 1]
            if hi == lo:
                continue
            rows = slice(lo, hi) if s["a_rows"] is None else s["a_rows"][lo:hi].long()
            b = s["B"][e].double()
            y = s["A"][rows].double() @ (b.t() if case["layout"] == "nk" else b)
            if s["a_scale"] is not None:
                y = y * s["a_scale"][rows].double()[:, None] * s["b_scale"][e].double()
            if s["bias"] is not None:
                y = y + s["bias"][e].double()
            out[lo:hi] = _exact_activation(y, case["act"])
        return out
    x = s["X"]
    scale = x.float().abs().max(dim=1).values / 127.0        # the codes' scale is a 32-bit number
    q = torch.round(x.float() / scale[:, None]).double()     # and a code the nearest whole number of the 32-bit quotient
    y = torch.matmul(q, s["B"].double().t()) * scale.double()[:, None] * s["b_scale"].double()[None, :]
    if s["bias"] is not None:
        y = y + s["bias"].double()
    return [None, x.double().abs().amax(1) / 127.0, _exact_activation(y, case["act"])]


def _exact_activation(y, act):
    if act == "relu":
        return torch.relu(y)
    if act == "gelu":
        return torch.nn.functional.gelu(y)
    if act == "silu":
        return y * torch.sigmoid(y)
    if act == "swiglu":
        gate, up = y.chunk(2, dim=-1)
        return gate * torch.sigmoid(gate) * up
    return y
