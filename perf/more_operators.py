"""Routing by scores and the low-rank adapters of many requests as measured cases.

Three operators of a mixture-of-experts block that serves many requests at once:

  route     router logits -> scores (softmax or sigmoid), plus a balance bias that
            only selects; groups of experts; the top-k experts of each token, their
            weights, and the (token, slot) pairs grouped by expert
  linear    a projection that all requests share with the low-rank adapter of each
            row's request: D[t] = act(X[t] W^T + s_a (X[t] A_a^T) B_a^T + bias)
  add       the same adapters beside a product C that was computed in another type:
            D[t] = act(C[t] + s_a (X[t] A_a^T) B_a^T + bias)

Each case runs either in its plain form (elementary torch operations in 32 bits, the
scores that decide between experts in 64) or, where ``own`` is true, through the
package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
WORKSPACE_BYTES = 32 * 2 ** 20     # a workspace that a program keeps for all of its calls


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the router of one decoding token: nothing but latency
        dict(name="route one token", op="route", T=1, E=64, k=8, logits="f32", score="softmax", bias=True, groups=1,
             kept=1, by="max", renorm=True, scale=1.0),
        # a batch of decoding sequences, softmax scores, groups ranked by their best expert, odd sizes
        dict(name="route batch odd", op="route", T=333, E=160, k=6, logits="f32", score="softmax", bias=False, groups=8,
             kept=3, by="max", renorm=False, scale=16.0),
        # a long prompt over many experts in groups, each ranked by its two best
        dict(name="route long prompt", op="route", T=16001, E=256, k=8, logits="bf16", score="sigmoid", bias=True,
             groups=8, kept=4, by="top2", renorm=True, scale=2.5),
        # one decoding token of one request
        dict(name="linear one token", op="linear", T=1, N=4096, K=4096, r=16, L=8, act="none", bias=False, mixed=True),
        # a decoding batch, every sequence its own request
        dict(name="linear decode", op="linear", T=16, N=18432, K=7168, r=16, L=32, act="none", bias=False, mixed=True),
        # more sequences, larger adapters: their weights weigh as much as the shared ones
        dict(name="linear decode wide", op="linear", T=64, N=4096, K=4096, r=64, L=48, act="none", bias=True, mixed=True),
        # prompts of several requests through a gated projection, gate and up fused with their product
        dict(name="linear prompt gated", op="linear", T=4096, N=8192, K=4096, r=64, L=16, act="swiglu", bias=False,
             mixed=False),
        # a large batch of prompts
        dict(name="linear prompt large", op="linear", T=8192, N=11008, K=4096, r=16, L=8, act="silu", bias=True,
             mixed=False),
        # a short prompt at odd sizes
        dict(name="linear prompt odd", op="linear", T=997, N=2049, K=1416, r=8, L=24, act="gelu", bias=True, mixed=False),
        # beside a quantised projection: a decoding batch
        dict(name="add decode", op="add", T=48, N=18432, K=7168, r=32, L=32, act="none", bias=False, mixed=True),
        # and prompts
        dict(name="add prompt", op="add", T=4096, N=11008, K=4096, r=32, L=8, act="silu", bias=True, mixed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case. Sizes run over their ranges' logarithms; K and r keep rows on 16
    bytes (the entry points ask for that), everything else may be odd."""
    op = rng.choice(["route", "route", "linear", "linear", "linear", "add"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 8])
        E = groups * _log(rng, max(2, 8 // groups), 256 // groups)
        kept = rng.randint(1, groups)
        return dict(op=op, T=_log(rng, 1, 16000), E=E, k=rng.randint(1, min(8, kept * (E // groups))),
                    logits=rng.choice(["f32", "bf16"]), score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.7,
                    groups=groups, kept=kept, by=rng.choice(["max", "top2"]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]))
    T = _log(rng, 1, 4096)
    act = rng.choice(["none", "none", "relu", "gelu", "silu"] + (["swiglu"] if op == "linear" else []))
    N = _log(rng, 64, 11008)
    return dict(op=op, T=T, N=2 * (N // 2) if act == "swiglu" else N, K=8 * _log(rng, 16, 512), r=8 * _log(rng, 1, 8), L=_log(rng, 1, 48),
                act=act, bias=rng.random() < 0.4, mixed=T <= 256 or rng.random() < 0.2)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _requests(g, T, L, mixed):
    """The adapter of each row, -1 for requests that have none. mixed: every row its own
    request (decoding). Else prompts, consecutive rows, and behind them the rows of some
    decoding sequences."""
    if mixed:
        ids = torch.randint(0, L, (T,), generator=g, device=DEV)
    else:
        tail = min(T // 16, 24)
        cuts = torch.sort(torch.randint(0, T, (6,), generator=g, device=DEV)).values
        owner = torch.randint(0, L, (7,), generator=g, device=DEV)
        ids = owner[torch.searchsorted(cuts, torch.arange(T, device=DEV), right=True)]
        ids[T - tail:] = torch.randint(0, L, (tail,), generator=g, device=DEV)
    none = torch.rand(T if mixed else L, generator=g, device=DEV) < 0.1
    none = none if mixed else none[ids]
    return torch.where(none, -1, ids).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        x = _randn(g, T, E) + 0.5 * _randn(g, 1, E)      # popular and unpopular experts, as a trained router gives them
        s["logits"] = x.to(torch.float32 if case["logits"] == "f32" else torch.bfloat16)
        spread = 0.1 if case["score"] == "sigmoid" else 1.0 / E
        s["bias"] = spread * _randn(g, E) if case["bias"] else None
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        s["row_token"] = torch.empty(T * k, dtype=torch.int32, device=DEV)
        s["slot_row"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        s["ws"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=DEV)
        return s
    T, N, K, r, L = (case[n] for n in ("T", "N", "K", "r", "L"))
    s["X"] = (_randn(g, T, K) * torch.exp(0.5 * _randn(g, T, 1))).to(torch.bfloat16)
    s["A"] = (_randn(g, L, r, K) * K ** -0.5).to(torch.bfloat16)
    s["B"] = (_randn(g, L, N, r) * 0.5 * r ** -0.5).to(torch.bfloat16)
    s["scale"] = 0.25 + torch.rand(L, generator=g, device=DEV)
    s["ids"] = _requests(g, T, L, case["mixed"])
    # for the plain form: rows in the order of their adapters, each row's place there, the longest run
    owner = s["ids"].long() + 1
    count = torch.bincount(owner, minlength=L + 1)
    s["order"] = torch.sort(owner, stable=True).indices
    s["group"] = owner[s["order"]]
    s["place"] = torch.arange(T, device=DEV) - (torch.cumsum(count, 0) - count)[s["group"]]
    s["longest"] = int(count[1:].max())
    s["bias"] = 0.1 * _randn(g, N) if case["bias"] else None
    if case["op"] == "linear":
        s["W"] = (_randn(g, N, K) * K ** -0.5).to(torch.bfloat16)
    else:
        s["C"] = (_randn(g, T, N) * torch.exp(0.5 * _randn(g, T, 1))).to(torch.bfloat16)
    s["D"] = torch.empty(T, N // 2 if case["act"] == "swiglu" else N, dtype=torch.bfloat16, device=DEV)
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
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    x = s["logits"].double()                 # scores next to each other decide: 64 bits
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        score = torch.exp(x - x.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    choice = score if s["bias"] is None else score + s["bias"].double()
    if G > 1:
        best = torch.sort(choice.reshape(T, G, E // G), dim=2, descending=True).values
        worth = best[:, :, :2 if c["by"] == "top2" else 1].sum(2)
        group = torch.sort(worth, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        kept.scatter_(1, group, True)
        choice = torch.where(kept.repeat_interleave(E // G, dim=1), choice, -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k].contiguous()   # equal: the lowest first
    weights = torch.gather(score, 1, ids)
    if c["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    flat = ids.reshape(-1)
    grouped, order = torch.sort(flat, stable=True)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(T * k, device=x.device)
    offsets = torch.searchsorted(grouped, torch.arange(E + 1, device=x.device))
    return [ids.to(torch.int32), (weights * c["scale"]).float(), offsets.to(torch.int32), (order // k).to(torch.int32),
            rank.reshape(T, k).to(torch.int32)]


def _plain_adapters(s):
    """s_a (X[t] A_a^T) B_a^T of every row, zero for rows without an adapter: the rows of each
    adapter side by side, padded to the longest."""
    c = s["case"]
    x = s["X"].float()
    padded = torch.zeros(c["L"] + 1, max(1, s["longest"]), c["K"], device=x.device)
    has = s["group"] > 0
    rows, group, place = s["order"][has], s["group"][has], s["place"][has]
    padded[group, place] = x[rows]
    low = torch.bmm(padded[1:], s["A"].float().transpose(1, 2)) * s["scale"][:, None, None]
    high = torch.bmm(low, s["B"].float().transpose(1, 2))
    out = torch.zeros(c["T"], c["N"], device=x.device)
    out[rows] = high[group - 1, place]
    return out


def _plain_linear(s):
    y = s["X"].float() @ s["W"].float().t() + _plain_adapters(s)
    return _finish(s, y)


def _plain_add(s):
    return _finish(s, s["C"].float() + _plain_adapters(s))


def _finish(s, y):
    if s["bias"] is not None:
        y = y + s["bias"]
    return _activation(y, s["case"]["act"]).to(torch.bfloat16)


# ------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"route": _plain_route, "linear": _plain_linear, "add": _plain_add}[c["op"]](s)
    import dense_gemm_persistent_gb300 as dg
    if c["op"] == "route":
        dg.dgemm_route_scored(s["logits"], c["k"], s["ids"], s["weights"], s["offsets"], s["row_token"], s["slot_row"],
                              score=c["score"], bias=s["bias"], groups=c["groups"], groups_kept=c["kept"],
                              group_score=c["by"], renormalize=c["renorm"], scale=c["scale"], ws=s["ws"])
        return [s["ids"], s["weights"], s["offsets"], s["row_token"], s["slot_row"]]
    more = dict(scale=s["scale"], bias=s["bias"], act=c["act"], ws=s["ws"])
    if c["op"] == "linear":
        return dg.dgemm_adapter_bf16(s["X"], s["W"], s["A"], s["B"], s["ids"], s["D"], **more)
    return dg.dgemm_adapter_add(s["X"], s["A"], s["B"], s["ids"], s["D"], C=s["C"], **more)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * (4 if case["logits"] == "f32" else 2) + T * k * 16 + 4 * (E + 1) + (4 * E if case["bias"] else 0),
                "flops": 6 * T * E}
    T, N, K, r, L = (case[n] for n in ("T", "N", "K", "r", "L"))
    requests = T if case["mixed"] else min(T, 7 + min(T // 16, 24))
    used = L * (1.0 - (1.0 - 1.0 / L) ** requests) * 0.9          # adapters that any row has
    wide = N // 2 if case["act"] == "swiglu" else N
    moved = 2 * T * K + 2 * used * r * (K + N) + 2 * T * wide + 4 * T + (4 * N if case["bias"] else 0)
    flops = 2 * 0.9 * T * r * (K + N)
    if case["op"] == "linear":
        return {"bytes": int(moved + 2 * N * K), "flops": int(flops + 2 * T * N * K)}
    return {"bytes": int(moved + 2 * T * N), "flops": int(flops + T * N)}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The definition, adapter by adapter or element by element, in float64."""
    s = prepare(case, seed)
    if case["op"] == "route":
        x = s["logits"].double()
        T, E = x.shape
        p = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
        c = p.clone() if s["bias"] is None else p + s["bias"].double()[None, :]
        G, size = case["groups"], E // case["groups"]
        if G > 1:
            top = torch.topk(c.view(T, G, size), min(size, 2 if case["by"] == "top2" else 1), dim=2).values.sum(2)
            alive = torch.zeros(T, G, dtype=torch.bool, device=DEV)
            for _ in range(case["kept"]):                         # the best group that is left, the first of equals
                at = top.masked_fill(alive, -math.inf)
                alive.scatter_(1, (at == at.amax(1, keepdim=True)).to(torch.int8).argmax(1, keepdim=True), True)
            c = c.view(T, G, size).masked_fill(~alive[:, :, None], -math.inf).view(T, E)
        taken = []
        for _ in range(case["k"]):
            at = (c == c.amax(1, keepdim=True)).to(torch.int8).argmax(1, keepdim=True)
            taken.append(p.gather(1, at))
            c.scatter_(1, at, -math.inf)
        w = torch.cat(taken, 1)
        return [None, case["scale"] * (w / w.sum(1, keepdim=True) if case["renorm"] else w), None, None, None]
    x = s["X"].double()
    y = torch.matmul(x, s["W"].double().t()) if case["op"] == "linear" else s["C"].double()
    for a in range(case["L"]):
        rows = (s["ids"] == a).nonzero()[:, 0]
        if rows.numel():
            y[rows] += s["scale"][a].double() * ((x[rows] @ s["A"][a].double().t()) @ s["B"][a].double().t())
    if s["bias"] is not None:
        y = y + s["bias"].double()
    act = case["act"]
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
