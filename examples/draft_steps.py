"""Serves requests with drafted tokens from losslessly compressed E4M3 weights:
a small decoder of random weights whose steps run the library's calls in the
order a server would:

    afx_kv_tables        pages, slots and positions of each request's last token and its drafts
    afx_decode           a matrix out of its container
    afx_fp8_quantize, afx_fp8_product        its product with the activations
    afx_rotate_write     queries and keys turned, keys and values into the cache
    afx_attention        each row over its request's tokens
    afx_verify           how many drafts stand, and the token behind them
    afx_kv_tables        the refused drafts' pages back

The drafts come from the decoder without its layers: the embedding of a token
straight into the head.

python examples/draft_steps.py [--steps N] [--check]: --check compares every
row's logits with dense attention over the whole history.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

LAYERS, HIDDEN, Q_HEADS, KV_HEADS, DIM, VOCAB = 2, 512, 8, 2, 64, 4096
PAGE, PAGES, COLUMNS, BLOCK = 16, 128, 16, 128
BASE = 10_000.0


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


class Weights:
    """An E4M3 matrix with a scale for each block of 128 x 128 as a container on the GPU, and its products."""

    def __init__(self, rows: int, cols: int, seed: int):
        import torch
        from weight_streaming_canonical_gb300 import afx, synth
        self.rows, self.cols = rows, cols
        bits = synth.normal_e4m3(rows * cols, seed=seed)
        container, self.desc = afx.encode(bits, fmt=afx.AFX_FMT_E4M3)
        self.container = torch.from_numpy(container).cuda()
        values = torch.from_numpy(bits).cuda().view(torch.float8_e4m3fn).view(rows, cols).float()
        spread = torch.rand((_blocks(rows), _blocks(cols)), generator=torch.Generator().manual_seed(seed)).cuda() + 0.5
        self.scales = spread * (0.5 / math.sqrt(cols)) / values.std()
        self.plain = values * self.scales.repeat_interleave(BLOCK, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]

    def __call__(self, x, work):
        """float32 x W^T of x [tokens][cols]."""
        import torch
        from weight_streaming_canonical_gb300 import afx
        n = x.shape[0]
        w = work["scratch"][:self.rows * self.cols]
        afx.afx_decode(self.desc, self.container, w, status_dev=work["status"])
        q = torch.empty((n, self.cols), dtype=torch.uint8, device="cuda")
        scales = torch.empty((_blocks(self.cols), n), dtype=torch.float32, device="cuda")
        afx.afx_fp8_quantize(x, q, scales)
        y = torch.empty((n, self.rows), dtype=torch.float32, device="cuda")
        afx.afx_fp8_product(w.view(self.rows, self.cols), self.scales, q, scales, y, status_dev=work["status"])
        return y

    def dense(self, x):
        """The same from plain operations."""
        import torch
        parts = x.float().unflatten(1, (-1, BLOCK))
        scale = (parts.abs().amax(2, keepdim=True).double() / 448).float().clamp(min=2.0 ** -126)
        rounded = (parts / scale).clamp(-448, 448).to(torch.float8_e4m3fn).float() * scale
        return rounded.flatten(1) @ self.plain.T


def _norm(x):
    import torch
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Server:
    def __init__(self, requests: int, seed: int = 0):
        import torch
        from weight_streaming_canonical_gb300 import afx
        self.n = requests
        width = (Q_HEADS + 2 * KV_HEADS) * DIM
        self.embed = torch.randn((VOCAB, HIDDEN), generator=torch.Generator().manual_seed(seed)).cuda()
        self.layers = [{"qkv": Weights(width, HIDDEN, 10 * i + 1), "out": Weights(HIDDEN, Q_HEADS * DIM, 10 * i + 2),
                        "up": Weights(4 * HIDDEN, HIDDEN, 10 * i + 3), "down": Weights(HIDDEN, 4 * HIDDEN, 10 * i + 4)}
                       for i in range(LAYERS)]
        self.head = Weights(VOCAB, HIDDEN, 99)
        self.rotary = afx.rotary(DIM, base=BASE)
        pool = lambda: torch.zeros((PAGES, PAGE, KV_HEADS, DIM), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.pools = [(pool(), pool()) for _ in range(LAYERS)]
        self.caches = [afx.kv_cache(k, v) for k, v in self.pools]
        ints = lambda n, v=0: torch.full((n,), v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.free, self.counts = torch.arange(PAGES, dtype=torch.int32, device="cuda"), [ints(1, PAGES), ints(1)]
        self.table = torch.full((self.n, COLUMNS), -1, dtype=torch.int32, device="cuda")
        self.starts, self.lens = ints(self.n + 1), ints(self.n)
        self.work = {"status": ints(1), "scratch": torch.empty(VOCAB * HIDDEN, dtype=torch.uint8, device="cuda")}

    def _tables(self, lens, n_tokens):
        """The tables from self.lens to lens: (slots, positions) of n_tokens new tokens."""
        import torch
        from weight_streaming_canonical_gb300 import afx
        slots = torch.empty(n_tokens, dtype=torch.int32, device="cuda")
        positions = torch.empty_like(slots)
        afx.afx_kv_tables(PAGE, self.lens, lens, self.table, self.free, self.counts[0], self.counts[1], self.starts, slots, positions,
                          status_dev=self.work["status"])
        self.counts.reverse()
        self.lens = lens
        return slots, positions

    def draft_logits(self, tokens):
        return self.head(_norm(self.embed[tokens.long()]), self.work)

    def step(self, tokens, added):
        """tokens: int32, each request's new tokens one behind the other, added[r] of request r.  The logits of every row."""
        import torch
        from weight_streaming_canonical_gb300 import afx
        n_tokens, status = tokens.shape[0], self.work["status"]
        slots, positions = self._tables(self.lens + added, n_tokens)
        x = self.embed[tokens.long()]
        workspace = None
        for layer, cache in zip(self.layers, self.caches):
            q, k, v = layer["qkv"](_norm(x), self.work).unflatten(1, (-1, DIM)).split([Q_HEADS, KV_HEADS, KV_HEADS], 1)
            turned = torch.empty((n_tokens, Q_HEADS, DIM), dtype=torch.bfloat16, device="cuda")
            afx.afx_rotate_write(self.rotary, positions, q, k, v, turned, cache, slots, status_dev=status)
            args = afx.attention_args(cache, Q_HEADS, n_tokens, self.starts, self.lens, self.table, 1 / math.sqrt(DIM))
            if workspace is None:  # the first layer's plan serves all of them
                workspace = torch.empty(afx.afx_attention_workspace(args), dtype=torch.uint8, device="cuda")
                afx.afx_attention_plan(args, workspace, status_dev=status)
            out = torch.empty_like(turned)
            afx.afx_attention(args, turned, out, workspace, status_dev=status)
            x = x + layer["out"](out.flatten(1), self.work)
            h = torch.nn.functional.silu(layer["up"](_norm(x), self.work))
            x = x + layer["down"](h, self.work)
        return self.head(_norm(x), self.work)

    def take_back(self, refused):
        """The last refused[r] tokens of each request leave the cache."""
        self._tables(self.lens - refused, 1)

    def dense(self, history):
        """Every row's logits over one request's whole history, from plain operations."""
        import torch
        position = torch.arange(len(history), device="cuda")
        angle = position.double()[:, None] * BASE ** (-torch.arange(DIM // 2, dtype=torch.float64, device="cuda") / (DIM // 2))
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

        def turn(t):
            a, b = t[..., :DIM // 2], t[..., DIM // 2:]
            return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)

        x = self.embed[torch.tensor(history, device="cuda")]
        for layer in self.layers:
            q, k, v = layer["qkv"].dense(_norm(x)).unflatten(1, (-1, DIM)).split([Q_HEADS, KV_HEADS, KV_HEADS], 1)
            q, k, v = (t.to(torch.bfloat16).float().transpose(0, 1) for t in (turn(q), turn(k), v))
            k, v = (t.repeat_interleave(Q_HEADS // KV_HEADS, 0) for t in (k, v))
            s = (q @ k.transpose(1, 2) / math.sqrt(DIM)).masked_fill(position[None, :] > position[:, None], -math.inf)
            x = x + layer["out"].dense((s.softmax(-1) @ v).transpose(0, 1).to(torch.bfloat16).flatten(1))
            x = x + layer["down"].dense(torch.nn.functional.silu(layer["up"].dense(_norm(x))))
        return self.head.dense(_norm(x))


def run(steps: int = 8, drafts: int = 3, check: bool = False, seed: int = 0, temperature: float = 0.8, say=lambda *_: None):
    """Returns (the requests' generated tokens, how many drafts stood, the largest difference of a logit over the logits' spread)."""
    import random

    import torch
    from weight_streaming_canonical_gb300 import afx
    rng = random.Random(seed)
    prompts = [[rng.randrange(VOCAB) for _ in range(n)] for n in (37, 5, 64)]
    server, rows = Server(len(prompts), seed), len(prompts)
    generator = torch.Generator(device="cuda").manual_seed(seed)
    uniform = lambda n: torch.rand(n, generator=generator, device="cuda")  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    params = {"temperature": torch.full((rows,), temperature, device="cuda"), "top_k": torch.full((rows,), 200, dtype=torch.int32, device="cuda"),
              "top_p": torch.full((rows,), 0.95, device="cuda")}
    history = [list(p) for p in prompts]
    server.step(ints([t for p in prompts for t in p[:-1]]), ints([len(p) - 1 for p in prompts]))  # the prompts but their last tokens
    stood, worst, k = 0, 0.0, drafts + 1
    status = server.work["status"]
    for i in range(steps):
        # each request's last token and its drafts, one after the other
        fed = torch.empty((rows, k), dtype=torch.int32, device="cuda")
        fed[:, 0] = ints([h[-1] for h in history])
        draft_logits = torch.empty((rows, k, VOCAB), device="cuda")
        for j in range(k):
            draft_logits[:, j] = server.draft_logits(fed[:, j])
            if j + 1 < k:
                token = torch.empty(rows, dtype=torch.int32, device="cuda")
                afx.afx_sample(draft_logits[:, j].contiguous(), uniform(rows), token, **params)
                fed[:, j + 1] = token
        tokens = fed.flatten()
        logits = server.step(tokens, ints([k] * rows))
        if check:
            for r in range(rows):
                want = server.dense(history[r][:-1] + fed[r].tolist())[-k:]
                worst = max(worst, ((logits[r * k:(r + 1) * k] - want).abs().max() / want.std()).item())
        out, counts = torch.empty_like(tokens), torch.empty(rows, dtype=torch.int32, device="cuda")
        workspace = torch.empty(afx.afx_verify_workspace(rows * k, rows), dtype=torch.uint8, device="cuda")
        afx.afx_verify(logits, tokens, server.starts, uniform(rows * k), uniform(rows), out, counts, workspace, params=params,
                       draft_logits=draft_logits.flatten(0, 1), draft_params=params, status_dev=status)
        server.take_back(k - counts)  # the token drawn is not in the cache yet: the next step feeds it
        new = [row[:c] for row, c in zip(out.view(rows, k).tolist(), counts.tolist())]
        stood += sum(map(len, new)) - rows
        for r in range(rows):
            history[r] += new[r]
        say(f"step {i}: {new}")
    torch.cuda.synchronize()
    if status.item():
        raise RuntimeError(f"device status {status.item():#x}")
    return [h[len(p):] for h, p in zip(history, prompts)], stood, worst


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--drafts", type=int, default=3)
    p.add_argument("--check", action="store_true")
    a = p.parse_args()
    _, stood, worst = run(a.steps, a.drafts, a.check, say=print)
    print(f"{stood} drafts stood")
    if a.check:
        print(f"largest difference from dense attention: {worst:.4f} of the logits' spread")


if __name__ == "__main__":
    main()
