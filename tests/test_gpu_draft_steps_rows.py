"""The example with drafts, product by product, and at temperature 0 against one token at a time.

Product by product: dense() gets, for every product, the activations that the
steps have handed to it, so that a rounding to E4M3 that falls to the other
neighbour stays with its own product.  It computes the same
activations itself, out of the product before, and compares:

- what a norm hands on (to the first matrices of a layer and the head), in bfloat16: both sides round a value that
  differs by the products' float32 sums alone, up to two half steps, 2^-7 of the value, and 2^-12 for the sums (hundreds
  to thousands of terms of 2^-24 each, of a spread of about 1);
- silu's results, float32: the sums' 2^-12 alone, of the row's largest;
- what the attention hands on: its weights are rounded to bfloat16 (2^-8 of each), its result (2^-8), on the other
  side the result too.  By Jensen's inequality a weighted mean of values has no larger root mean square than the largest
  of the values' own, v; so its error's is at most 3 * 2^-8 v, and a sixteenth more for queries, keys and values that the
  sums' differences let fall to the other bfloat16.  A key that is lost or
  another's, among n, changes a result by about v / n: at 37 to 64 tokens twice that bound and more.

The logits then differ by one product's sums: 512 terms of 2^-23 of at most 4 spreads each, below 2^-11.
"""
import os
import random
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


class Watch:
    """Keeps what the steps hand to each product, request by request, and gives it to dense() in turn."""

    def __init__(self, monkeypatch, example):
        self.kept, self.now, self.request, self.recording, self.worst = [], [], 0, False, {}
        w, s = example.Weights, example.Server
        product, dense, step, take_back, whole = w.__call__, w.dense, s.step, s.take_back, s.dense

        def on_product(weights, x, work):
            if self.recording:
                self.now.append(x.clone())
            return product(weights, x, work)

        def on_step(server, tokens, added):
            self.now, self.recording, self.request = [], True, 0
            logits = step(server, tokens, added)
            self.recording = False
            parts = [x.split(added.tolist()) for x in self.now]
            if not self.kept:
                self.kept = [[[] for _ in parts] for _ in range(server.n)]
            for r in range(server.n):
                for i, p in enumerate(parts):
                    self.kept[r][i].append(p[r])
            return logits

        def on_take_back(server, refused):
            for r, n in enumerate(refused.tolist()):
                for i, pieces in enumerate(self.kept[r]):
                    rows = torch.cat(pieces)
                    self.kept[r][i] = [rows[:rows.shape[0] - n]]
            take_back(server, refused)

        def on_dense(weights, x):
            given = torch.cat(self.kept[self.request][self.place])
            assert given.shape == x.shape and given.dtype == x.dtype
            a, b = given.double(), x.double()
            name, self.place = self.names[self.place], self.place + 1
            if name == "attention":
                worst = ((a - b).square().mean().sqrt() / (3.25 * 2.0 ** -8 * self.value)).item()
            elif name == "silu":
                worst = ((a - b).abs().amax(1) / (2.0 ** -12 * b.abs().amax(1))).max().item()
            else:
                worst = ((a - b).abs() / (2.0 ** -7 * b.abs() + 2.0 ** -12)).max().item()
            self.worst[name] = max(self.worst.get(name, 0.0), worst)
            y = dense(weights, given)
            if name == "qkv":
                values = y[:, (example.Q_HEADS + example.KV_HEADS) * example.DIM:].unflatten(1, (example.KV_HEADS, example.DIM))
                self.value = values.double().square().mean(2).sqrt().max()
            return y

        def on_whole(server, history):
            self.place = 0
            logits = whole(server, history)
            self.request += 1
            return logits

        self.names = ["qkv", "attention", "up", "silu"] * example.LAYERS + ["head"]
        for cls, name, f in ((w, "__call__", on_product), (w, "dense", on_dense), (s, "step", on_step), (s, "take_back", on_take_back),
                             (s, "dense", on_whole)):
            monkeypatch.setattr(cls, name, f)


@pytest.mark.parametrize("drafts", [0, 3, 7])
def test_every_product_of_the_steps(afx, monkeypatch, drafts):
    import draft_steps
    watch = Watch(monkeypatch, draft_steps)
    tokens, stood, worst = draft_steps.run(steps=6, drafts=drafts, check=True, seed=3)
    assert set(watch.worst) == set(watch.names) and max(watch.worst.values()) <= 1, watch.worst
    assert worst < 2.0 ** -11, worst
    assert all(len(t) >= 6 for t in tokens) and (drafts == 0 or stood > 0)


def test_temperature_0_gives_the_tokens_of_one_at_a_time(afx):
    """With drafts or without, each token is the first of the largest logits: the runs have the same tokens up to one
    where the logits of both runs' tokens are closer to each other than the two runs' errors together."""
    import draft_steps
    alone, _, off = draft_steps.run(steps=12, drafts=0, check=True, seed=4, temperature=0.0)
    for drafts in (1, 3):
        tokens, stood, worst = draft_steps.run(steps=12, drafts=drafts, check=True, seed=4, temperature=0.0)
        near, same = 2 * max(off, worst), 0
        rng = random.Random(4)
        prompts = [[rng.randrange(draft_steps.VOCAB) for _ in range(n)] for n in (37, 5, 64)]
        server = draft_steps.Server(len(prompts), 4)
        for prompt, a, b in zip(prompts, alone, tokens):
            n = min(len(a), len(b))
            at = next((i for i in range(n) if a[i] != b[i]), n)
            same += at
            if at < n:
                logits = server.dense(prompt + a[:at])[-1]
                gap = ((logits[a[at]] - logits[b[at]]).abs() / logits.std()).item()
                assert gap <= near, (at, gap, near)
        assert same >= 12
