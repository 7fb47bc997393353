"""A small hybrid model's serving loop: one recurrent and one softmax-attention
layer, from ragged prompts through decode steps.

Hybrid models alternate the two kinds of layers: the recurrent one keeps a
fixed-size state per request (here in the quantized pool), the softmax one a
key-value cache that grows (here in pages).  The loop shows the calls in the
order a server makes them:

    prompts   sq_block_tables -> (sq_pool_load) -> sq_prefill -> sq_pool_store
                              -> sq_kv_append
    a token   sq_block_tables -> sq_decode_step (or sq_decode_step_linear)
                              -> sq_kv_append -> sq_paged_attention

Activations are synthetic, drawn per layer and token as in ``inputs``.

    python -m quantized_recurrent_state_gated_amd.hybrid [--requests N] [--prompt T] [--steps K]
        [--heads H] [--bits 4|6|8|16|32] [--linear] [--q-heads Q] [--kv-heads KV] [--page P]
"""
from __future__ import annotations

import argparse
import json
import math
import time

import torch

from . import sq

D = 128  # key and value width of both layers


class HybridLayers:
    """The states of n requests in both layers, and the calls that move them on."""

    def __init__(self, n: int, heads: int, head_bits, q_heads: int, kv_heads: int, page: int, max_len: int,
                 rule: int = sq.SQ_RULE_DELTA, dtype=torch.bfloat16, scale: float = 0.05):
        dev = "cuda"
        self.n, self.heads, self.rule, self.dtype, self.page, self.max_len = n, heads, rule, dtype, page, max_len
        # recurrent layer: one slot per request
        ones = torch.ones(heads, D, device=dev)
        state = torch.empty(sq.sq_pool_bytes(n, heads, D, D, head_bits), dtype=torch.uint8, device=dev)
        self.pool = sq.sq_pool_alloc(n, heads, D, D, head_bits, ones, ones * scale, state)
        self.slots = torch.arange(n, dtype=torch.int32, device=dev)
        sq.sq_pool_store(self.pool, self.slots, torch.zeros(n, heads, D, D, device=dev))
        self.fresh = True  # no request holds a token yet
        # softmax layer: pages for n requests of up to max_len tokens, handed out in any order
        per_row = -(-max_len // page)
        pages = n * per_row
        self.cache = sq.SqKvCache(torch.empty(pages, kv_heads, page, D, dtype=dtype, device=dev),
                                  torch.empty(pages, kv_heads, D, page, dtype=dtype, device=dev))
        self.free = torch.randperm(pages, device=dev).to(torch.int32)
        i32 = dict(dtype=torch.int32, device=dev)
        self.table = torch.zeros(n, per_row, **i32)
        self.ctx, self.seq = torch.zeros(n, **i32), torch.zeros(n, **i32)
        self.cu, self.cu_pages, self.result = (torch.zeros(m, **i32) for m in (n + 1, n + 1, 1))
        nb = sq.sq_paged_attention_workspace(self.cache, n, q_heads, max_len)
        self.attend_ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)

    def _admit(self, new_lens, slot_map) -> int:
        """Pages and slots for the requests' next tokens; returns how many pages
        they take.  Waits for the result: where pages run out, the call ends here,
        with states, cache, lengths and free list as they were (the rows' entries
        past the tokens held are written anew by the next call)."""
        sq.sq_block_tables(self.ctx, new_lens, self.page, self.free, self.table, self.seq, self.cu, self.cu_pages,
                           slot_map, self.result)
        taken, result = torch.cat([self.cu_pages[-1:], self.result]).tolist()
        if result:
            raise RuntimeError(f"sq_block_tables reported {result}")
        return taken

    def _advance(self, taken: int) -> None:
        """The tokens are in: lengths move on, the pages taken leave the list."""
        self.free = self.free[taken:].contiguous()
        self.ctx, self.seq = self.seq, self.ctx
        self.fresh = False

    def prompts(self, lens, x: dict):
        """Packed prompts, or further tokens of requests that hold some: q, k, v,
        alpha, beta of the recurrent layer, ak, av of the softmax layer.  Returns
        the recurrent layer's outputs; the softmax layer's prompt tokens only
        enter the cache (attention over a prompt is not among these calls)."""
        new = torch.tensor(lens, dtype=torch.int32, device="cuda")
        N = sum(lens)
        slot_map = torch.empty(N, dtype=torch.int64, device="cuda")
        taken = self._admit(new, slot_map)
        o = torch.empty_like(x["v"])
        S = torch.empty(self.n, self.heads, D, D, device="cuda")
        nb = sq.sq_prefill_workspace(self.n, N, self.heads, D, D, self.dtype, self.rule)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda") if nb else None
        if not self.fresh:
            sq.sq_pool_load(self.pool, self.slots, S)
        sq.sq_prefill(x["q"], x["k"], x["v"], x["alpha"], x["beta"], self.cu, o, S=S, S0=None if self.fresh else S,
                      rule=self.rule, workspace=ws)
        sq.sq_pool_store(self.pool, self.slots, S)
        sq.sq_kv_append(self.cache, x["ak"], x["av"], slot_map)
        self._advance(taken)
        return o

    def token(self, x: dict):
        """One new token per request (as for prompts, and aq, the softmax layer's
        queries).  Returns the outputs of both layers."""
        one = torch.ones(self.n, dtype=torch.int32, device="cuda")
        slot_map = torch.empty(self.n, dtype=torch.int64, device="cuda")
        taken = self._admit(one, slot_map)
        o = torch.empty(self.n, self.heads, D, device="cuda")
        step = sq.sq_decode_step if self.rule == sq.SQ_RULE_DELTA else sq.sq_decode_step_linear
        step(self.pool, self.slots, x["q"], x["k"], x["v"], x["alpha"], x["beta"], o)
        sq.sq_kv_append(self.cache, x["ak"], x["av"], slot_map)
        a = torch.empty_like(x["aq"])
        sq.sq_paged_attention(self.cache, x["aq"], self.table, self.seq, self.max_len, a, self.attend_ws)
        self._advance(taken)
        return o, a


def activations(n: int, heads: int, q_heads: int, kv_heads: int, gen, dtype=torch.bfloat16) -> dict:
    """Synthetic activations of n tokens on the GPU."""
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    life = torch.exp(torch.linspace(0.0, math.log(1000.0), heads, device="cuda"))  # half-lives of the heads
    x = {"q": unit(r(n, heads, D)).to(dtype), "k": unit(r(n, heads, D)).to(dtype), "v": r(n, heads, D).to(dtype),
         "alpha": torch.exp(-(math.log(2.0) / life) * torch.exp(0.5 * r(n, heads) - 0.125)),
         "beta": 0.05 + 0.9 * torch.rand(n, heads, generator=gen, device="cuda")}
    return x | {"ak": r(n, kv_heads, D).to(dtype), "av": r(n, kv_heads, D).to(dtype), "aq": r(n, q_heads, D).to(dtype)}


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("requests", 16), ("prompt", 1024), ("steps", 64), ("heads", 48), ("bits", 8),
                          ("q-heads", 32), ("kv-heads", 8), ("page", 16), ("seed", 1)):
        ap.add_argument(f"--{name}", type=int, default=default)
    ap.add_argument("--linear", action="store_true", help="plain decay instead of the delta rule")
    a = ap.parse_args()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(a.seed)
    lens = [a.prompt - (i * 37) % max(1, a.prompt // 2) for i in range(a.requests)]
    m = HybridLayers(a.requests, a.heads, [a.bits] * a.heads, a.q_heads, a.kv_heads, a.page, a.prompt + a.steps,
                     sq.SQ_RULE_LINEAR if a.linear else sq.SQ_RULE_DELTA)
    draw = lambda n: activations(n, a.heads, a.q_heads, a.kv_heads, gen)  # noqa: E731
    x = draw(sum(lens))
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    m.prompts(lens, x)
    torch.cuda.synchronize()
    t1 = time.perf_counter()
    x = draw(a.requests)
    for _ in range(a.steps):
        m.token(x)
    torch.cuda.synchronize()
    t2 = time.perf_counter()
    print(json.dumps({"requests": a.requests, "prompt_tokens": sum(lens), "prompt_ms": round(1e3 * (t1 - t0), 3),
                      "steps": a.steps, "ms_per_step": round(1e3 * (t2 - t1) / a.steps, 4),
                      "rule": "linear" if a.linear else "delta", "bits": a.bits}))


if __name__ == "__main__":
    main()
