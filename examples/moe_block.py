"""A mixture-of-experts feed-forward block on the library's entry points:

    logits = X . Wr^T                                     dgemm_bf16
    top-k experts, weights, rows grouped by expert        dgemm_route
    H[r] = silu(X[t] . Wg_e^T) * (X[t] . Wu_e^T)          dgemm_grouped_*  (t = row_token[r])
    Y[r] = H[r] . Wd_e^T                                  dgemm_grouped_*
    shared = int8 linear layer over X                     dgemm_int8_quantize, dgemm_int8_scaled
    out[t] = shared[t] + sum_j w[t,j] Y[slot_row[t,j]]    dgemm_combine

The routed experts are BF16, or int8 with per-token and per-channel scales. Nothing
returns to the host between the calls: the group sizes stay on the device.

With --scored the experts are chosen by sigmoid scores, a balance bias and groups
(dgemm_route_scored). With --adapters N the tokens belong to N requests, each with a low-rank adapter
of the shared layer: shared[t] += s_a (X[t] . A_a^T) . B_a^T (dgemm_adapter_add, in place).

    python examples/moe_block.py [--tokens 512] [--int8] [--scored] [--adapters 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_persistent_gb300 as dg  # noqa: E402


def quantize_channels(w: torch.Tensor):
    """int8 codes of weights [..., N, K] with one FP32 scale per output channel."""
    s = w.abs().amax(-1).clamp_min(1e-20) / 127.0
    return torch.round(w / s[..., None]).to(torch.int8), s.contiguous()


class MoEBlock:
    """Weights laid out once, and the buffers of up to `max_tokens` tokens kept between calls.
    `experts` is a multiple of 4 (dgemm_bf16 writes the logits, FP32 rows on 16 bytes)."""

    def __init__(self, hidden: int, inner: int, experts: int, top_k: int, max_tokens: int, *, int8: bool = False,
                 scored: bool = False, groups: int = 4, groups_kept: int = 2, adapters: int = 0, rank: int = 16,
                 device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device=device)
        self.H, self.I, self.E, self.k, self.int8 = hidden, inner, experts, top_k, int8
        bf16 = dict(dtype=torch.bfloat16, device=device)
        self.router = (randn(experts, hidden) * hidden ** -0.5).to(torch.bfloat16)
        self.up = (randn(experts, 2 * inner, hidden) * hidden ** -0.5).to(torch.bfloat16)    # gate channels first
        self.down = (randn(experts, hidden, inner) * inner ** -0.5).to(torch.bfloat16)
        self.shared, self.shared_scale = quantize_channels(randn(hidden, hidden) * hidden ** -0.5)
        if int8:
            self.up, self.up_scale = quantize_channels(self.up.float())
            self.down, self.down_scale = quantize_channels(self.down.float())
        self.scored, self.groups, self.groups_kept, self.adapters = scored, groups, groups_kept, adapters
        ws_bytes = max(dg.dgemm_route_workspace_size(max_tokens, experts, top_k), 1 << 20)
        if scored:
            self.balance = 0.1 * randn(experts)
        if adapters:
            self.low = (randn(adapters, rank, hidden) * hidden ** -0.5).to(torch.bfloat16)
            self.high = (randn(adapters, hidden, rank) * rank ** -0.5).to(torch.bfloat16)
            self.adapter_scale = torch.full((adapters,), 0.5, device=device)
            ws_bytes = max(ws_bytes, dg.dgemm_adapter_workspace_size(max_tokens, hidden, hidden, rank, adapters))
        T, R = max_tokens, max_tokens * top_k
        i32 = dict(dtype=torch.int32, device=device)
        self.logits = torch.empty(T, experts, device=device)
        self.ids, self.slot_row = torch.empty(T, top_k, **i32), torch.empty(T, top_k, **i32)
        self.weights = torch.empty(T, top_k, device=device)
        self.offsets, self.row_token = torch.empty(experts + 1, **i32), torch.empty(R, **i32)
        self.codes, self.scales = torch.empty(T, hidden, dtype=torch.int8, device=device), torch.empty(T, device=device)
        self.inner, self.rows = torch.empty(R, inner, **bf16), torch.empty(R, hidden, **bf16)
        self.inner_codes, self.inner_scales = torch.empty(R, inner, dtype=torch.int8, device=device), torch.empty(R, device=device)
        self.from_shared = torch.empty(T, hidden, **bf16)
        self.ws = torch.empty(ws_bytes, dtype=torch.uint8, device=device)

    def __call__(self, X: torch.Tensor, out: torch.Tensor, requests: torch.Tensor | None = None) -> torch.Tensor:
        """requests [T] int32: the adapter of each token, -1 for none (with adapters)."""
        T, k = X.shape[0], self.k
        R = T * k
        logits, ids, weights, slot_row = self.logits[:T], self.ids[:T], self.weights[:T], self.slot_row[:T]
        row_token, inner, rows = self.row_token[:R], self.inner[:R], self.rows[:R]
        dg.dgemm_bf16(X, self.router, logits, b_layout="nk")
        if self.scored:
            dg.dgemm_route_scored(logits, k, ids, weights, self.offsets, row_token, slot_row, score="sigmoid", bias=self.balance,
                                  groups=self.groups, groups_kept=self.groups_kept, group_score="top2", scale=2.5, ws=self.ws)
        else:
            dg.dgemm_route(logits, k, ids, weights, self.offsets, row_token, slot_row, ws=self.ws)
        codes, scales = self.codes[:T], self.scales[:T]
        dg.dgemm_int8_quantize(X, codes, scales)
        if self.int8:
            dg.dgemm_grouped_int8_scaled(codes, self.up, scales, self.up_scale, self.offsets, inner, a_rows=row_token, act="swiglu",
                                         ws=self.ws)
            dg.dgemm_int8_quantize(inner, self.inner_codes[:R], self.inner_scales[:R])
            dg.dgemm_grouped_int8_scaled(self.inner_codes[:R], self.down, self.inner_scales[:R], self.down_scale, self.offsets, rows,
                                         ws=self.ws)
        else:
            dg.dgemm_grouped_bf16(X, self.up, self.offsets, inner, a_rows=row_token, act="swiglu", ws=self.ws)
            dg.dgemm_grouped_bf16(inner, self.down, self.offsets, rows, ws=self.ws)
        dg.dgemm_int8_scaled(codes, self.shared, scales, self.shared_scale, self.from_shared[:T], ws=self.ws)
        if self.adapters:
            dg.dgemm_adapter_add(X, self.low, self.high, requests, self.from_shared[:T], C=self.from_shared[:T],
                                 scale=self.adapter_scale, ws=self.ws)
        return dg.dgemm_combine(rows, slot_row, weights, out, add=self.from_shared[:T])


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--int8", action="store_true", help="int8 experts")
    ap.add_argument("--scored", action="store_true", help="experts by sigmoid scores, a balance bias and groups")
    ap.add_argument("--adapters", type=int, default=0, help="requests with a low-rank adapter of the shared layer")
    a = ap.parse_args()
    block = MoEBlock(a.hidden, a.inner, a.experts, a.top_k, a.tokens, int8=a.int8, scored=a.scored, adapters=a.adapters)
    requests = torch.arange(a.tokens, dtype=torch.int32, device="cuda") * a.adapters // max(a.tokens, 1) if a.adapters else None
    X = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(X)
    for _ in range(3):
        block(X, out, requests)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        block(X, out, requests)
    end.record()
    torch.cuda.synchronize()
    # the block's workspace, and the per-device word of the calls without one (the router's product)
    assert dg.dgemm_query_device_status(block.ws) == 0 and dg.dgemm_query_device_status() == 0
    sizes = block.offsets.diff().tolist()
    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.inner}, top {a.top_k}, "
          f"{'int8' if a.int8 else 'bf16'}: {start.elapsed_time(end) / 20 * 1e3:.1f} us a call; "
          f"rows per expert {min(sizes)}..{max(sizes)}; |out| {out.float().abs().mean():.4f}")


if __name__ == "__main__":
    main()
