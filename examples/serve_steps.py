"""Serves requests that share a system prompt, a scheduler step at a time,
from losslessly compressed weights: a small decoder of random weights, whose
steps run the library's calls in the order a server would:

    afx_kv_tables        pages, slots and positions from the requests' lengths
    afx_prefill / afx_decode_gemv_static     products with compressed weights
    afx_kv_write         new keys and values into the cache, layer by layer
    afx_attention_plan   once a step
    afx_attention        layer by layer
    afx_sample           one token a request

python examples/serve_steps.py [--steps N] [--check]: --check compares every
step's logits with dense attention over the whole history.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

LAYERS, HIDDEN, Q_HEADS, KV_HEADS, DIM, VOCAB = 2, 512, 8, 2, 64, 4096
PAGE, PAGES, COLUMNS = 16, 256, 24
PREFIX = 150


class Weights:
    """A matrix as a container on the GPU, and its products."""

    def __init__(self, rows: int, cols: int, seed: int):
        import numpy as np
        import torch
        from weight_streaming_canonical_gb300 import afx, synth
        self.rows, self.cols = rows, cols
        patterns = synth.normal(rows * cols, seed=seed)
        container, self.desc = afx.encode(patterns)
        self.container = torch.from_numpy(container).cuda()
        self.plain = torch.from_numpy(patterns.view(np.int16)).cuda().view(torch.bfloat16).view(rows, cols).float()

    def __call__(self, x, work):
        """float32 x W^T of bfloat16 x [tokens][cols]."""
        import torch
        from weight_streaming_canonical_gb300 import afx
        y = torch.empty((x.shape[0], self.rows), dtype=torch.float32, device="cuda")
        x = x.contiguous().view(torch.int16)
        if x.shape[0] <= 4:
            afx.afx_decode_gemv_static(self.desc, self.container, self.rows, self.cols, x, y, status_dev=work["status"])
        else:
            afx.afx_prefill(self.desc, self.container, self.rows, self.cols, x, y, work["scratch"], work["gemm"],
                            status_dev=work["status"])
        return y


def _norm(x):
    import torch
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def _rotate(x, positions):
    """Rotary positions: x [tokens][heads][DIM], float32."""
    import torch
    angle = positions[:, None, None].float() * torch.pow(10_000.0, -torch.arange(DIM // 2, device=x.device) / (DIM // 2))
    a, b = x[..., :DIM // 2], x[..., DIM // 2:]
    return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)


class Server:
    """Request 0 holds the system prompt's pages and gets no tokens after the first step."""

    def __init__(self, requests: int, seed: int = 0):
        import torch
        from weight_streaming_canonical_gb300 import afx
        self.n = requests + 1
        width = (Q_HEADS + 2 * KV_HEADS) * DIM
        self.embed = torch.randn((VOCAB, HIDDEN), generator=torch.Generator().manual_seed(seed)).cuda()
        self.layers = [{"qkv": Weights(width, HIDDEN, 10 * i + 1), "out": Weights(HIDDEN, Q_HEADS * DIM, 10 * i + 2),
                        "up": Weights(4 * HIDDEN, HIDDEN, 10 * i + 3), "down": Weights(HIDDEN, 4 * HIDDEN, 10 * i + 4)}
                       for i in range(LAYERS)]
        self.head = Weights(VOCAB, HIDDEN, 99)
        pool = lambda: torch.zeros((PAGES, PAGE, KV_HEADS, DIM), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.pools = [(pool(), pool()) for _ in range(LAYERS)]
        self.caches = [afx.kv_cache(k, v) for k, v in self.pools]
        ints = lambda n, v=0: torch.full((n,), v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.free, self.counts = torch.arange(PAGES, dtype=torch.int32, device="cuda"), [ints(1, PAGES), ints(1)]
        self.table = torch.full((self.n, COLUMNS), -1, dtype=torch.int32, device="cuda")
        self.starts, self.lens = ints(self.n + 1), [0] * self.n
        self.prefix_table = None
        self.work = {"status": ints(1), "gemm": torch.empty(afx.AFX_PREFILL_GEMM_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda"),
                     "scratch": torch.empty(VOCAB * HIDDEN, dtype=torch.int16, device="cuda")}

    def step(self, new):
        """new[r]: the tokens request r gets now.  Returns the logits after each request's last token."""
        import torch
        from weight_streaming_canonical_gb300 import afx
        n_tokens = sum(map(len, new))
        tokens = torch.tensor([t for one in new for t in one], device="cuda")
        old = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.lens = [a + len(b) for a, b in zip(self.lens, new)]
        lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        slots = torch.empty(n_tokens, dtype=torch.int32, device="cuda")
        positions = torch.empty_like(slots)
        status = self.work["status"]
        afx.afx_kv_tables(PAGE, old, lens, self.table, self.free, self.counts[0], self.counts[1], self.starts, slots, positions,
                          status_dev=status)
        self.counts.reverse()
        prefix = 0 if self.prefix_table is None else PREFIX
        positions = positions + prefix
        x = self.embed[tokens]
        workspace = None
        for i, (layer, cache) in enumerate(zip(self.layers, self.caches)):
            q, k, v = layer["qkv"](_norm(x), self.work).unflatten(1, (-1, DIM)).split([Q_HEADS, KV_HEADS, KV_HEADS], 1)
            q, k = (_rotate(t, positions).to(torch.bfloat16) for t in (q, k))
            afx.afx_kv_write(cache, k, v.to(torch.bfloat16).contiguous(), slots, status_dev=status)
            args = afx.attention_args(cache, Q_HEADS, n_tokens, self.starts, lens, self.table, 1 / math.sqrt(DIM),
                                      self.prefix_table, prefix)
            if workspace is None:  # the first layer's plan serves all of them
                workspace = torch.empty(afx.afx_attention_workspace(args), dtype=torch.uint8, device="cuda")
                afx.afx_attention_plan(args, workspace, status_dev=status)
            out = torch.empty((n_tokens, Q_HEADS, DIM), dtype=torch.bfloat16, device="cuda")
            afx.afx_attention(args, q, out, workspace, status_dev=status)
            x = x + layer["out"](out.flatten(1), self.work)
            h = torch.nn.functional.silu(layer["up"](_norm(x), self.work))
            x = x + layer["down"](h.to(torch.bfloat16), self.work)
        last = self.starts[1:].long() - 1
        return self.head(_norm(x[last[[r for r in range(self.n) if new[r]]]]), self.work)

    def share_prefix(self):
        """Request 0's tokens become the prefix of all others."""
        assert self.lens[0] == PREFIX
        self.prefix_table = self.table[0, :-(-PREFIX // PAGE)].clone()

    def dense(self, history):
        """The same logits from plain operations over one request's whole history (float32 between the roundings)."""
        import torch
        position = torch.arange(len(history), device="cuda")
        x = self.embed[torch.tensor(history, device="cuda")]
        for layer in self.layers:
            y = _norm(x).float() @ layer["qkv"].plain.T
            q, k, v = y.unflatten(1, (-1, DIM)).split([Q_HEADS, KV_HEADS, KV_HEADS], 1)
            q, k, v = (t.to(torch.bfloat16).float().transpose(0, 1) for t in (_rotate(q, position), _rotate(k, position), v))
            k, v = (t.repeat_interleave(Q_HEADS // KV_HEADS, 0) for t in (k, v))
            s = q @ k.transpose(1, 2) / math.sqrt(DIM)
            s = s.masked_fill(position[None, :] > position[:, None], -math.inf)
            out = (s.softmax(-1) @ v).transpose(0, 1).to(torch.bfloat16).float()
            x = x + out.flatten(1) @ layer["out"].plain.T
            h = torch.nn.functional.silu(_norm(x).float() @ layer["up"].plain.T)
            x = x + h.to(torch.bfloat16).float() @ layer["down"].plain.T
        return _norm(x[-1:]).float() @ self.head.plain.T


def run(steps: int = 8, check: bool = False, seed: int = 0, say=lambda *_: None):
    """Returns (the requests' generated tokens, the largest difference of a logit over the logits' spread)."""
    import random

    import torch
    from weight_streaming_canonical_gb300 import afx
    rng = random.Random(seed)
    text = lambda n: [rng.randrange(VOCAB) for _ in range(n)]  # noqa: E731
    prompts = [text(37), text(5), text(64)]
    server, system = Server(len(prompts), seed), text(PREFIX)
    history = [list(p) for p in prompts]
    server.step([system] + [[] for _ in prompts])  # the system prompt, once
    server.share_prefix()
    generator = torch.Generator(device="cuda").manual_seed(seed)
    rows = len(prompts)
    full = lambda v, t=torch.float32: torch.full((rows,), v, dtype=t, device="cuda")  # noqa: E731
    tokens, logprobs = full(0, torch.int32), full(0.0)
    new, worst = prompts, 0.0
    for i in range(steps):
        logits = server.step([[]] + new)
        if check:
            for r in range(rows):
                want = server.dense(system + history[r])[0]
                worst = max(worst, ((logits[r] - want).abs().max() / want.std()).item())
        afx.afx_sample(logits, torch.rand(rows, generator=generator, device="cuda"), tokens, logprobs=logprobs,
                       temperature=full(0.8), top_k=full(50, torch.int32), top_p=full(0.95))
        new = [[t] for t in tokens.tolist()]
        for r in range(rows):
            history[r] += new[r]
        say(f"step {i}: tokens {tokens.tolist()}, log probabilities {[round(v, 2) for v in logprobs.tolist()]}")
    torch.cuda.synchronize()
    if server.work["status"].item():
        raise RuntimeError(f"device status {server.work['status'].item():#x}")
    return [h[len(p):] for h, p in zip(history, prompts)], worst


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--check", action="store_true")
    a = p.parse_args()
    _, worst = run(a.steps, a.check, say=print)
    if a.check:
        print(f"largest difference from dense attention: {worst:.4f} of the logits' spread")


if __name__ == "__main__":
    main()
