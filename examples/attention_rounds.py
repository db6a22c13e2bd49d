"""Speculative rounds of a target with attention layers over a paged key/value cache.

A small random model stands for the target.  Prompts' keys and values go into the cache with
``spec_cache_write`` and attend with ``spec_paged_attention``; then each round drafts
from the conversation, writes and attends the anchor and the drafts of every lane, accepts
with ``spec_verify_accept`` and adds the committed counts to ``cached_lens``: the slots of
rejected drafts are written over by the next round.  Lanes take pages from a pool as they
grow.

    python examples/attention_rounds.py [--lanes 4] [--tokens 48] [--cache e4m3]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import speculative_decoding_verify_bf16_gb300 as sv  # noqa: E402

Q_HEADS, KV_HEADS, DIM, PAGE = 8, 2, 64, 16
CACHES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


class AttentionModel:
    """A bigram table plus layers of attention."""

    def __init__(self, vocab=257, layers=2, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        hidden = Q_HEADS * DIM

        def weights(*shape):
            return torch.randn(*shape, generator=g, device=device) / shape[-2] ** 0.5

        self.vocab, self.layers, self.device = vocab, layers, torch.device(device)
        self.embed = torch.randn(vocab, hidden, generator=g, device=device)
        self.proj = [weights(hidden, (Q_HEADS + 2 * KV_HEADS) * DIM) for _ in range(layers)]
        self.merge = [weights(hidden, hidden) for _ in range(layers)]
        self.unembed = weights(hidden, vocab)
        # Likely successors that soon run in circles, as drafting needs.
        self.next = torch.randint(0, 11, (vocab,), generator=g, device=device)

    def forward(self, tokens, attend):
        """Logits [rows, vocab] of packed tokens; attend(layer, q, k, v) is the layer's
        attention."""
        x = self.embed[tokens.long()]
        rows = x.shape[0]
        for layer in range(self.layers):
            qkv = (x @ self.proj[layer]).view(rows, Q_HEADS + 2 * KV_HEADS, DIM).to(torch.bfloat16)
            o = attend(layer, qkv[:, :Q_HEADS], qkv[:, Q_HEADS:Q_HEADS + KV_HEADS], qkv[:, Q_HEADS + KV_HEADS:])
            x = x + o.float().reshape(rows, -1) @ self.merge[layer]
        logits = x @ self.unembed
        logits[torch.arange(rows, device=x.device), self.next[tokens.long()]] += 12.0
        return logits


class Lanes:
    """The lanes' pages in a pool, the same for all layers, and how far each is filled."""

    def __init__(self, model, lanes, most, cache="bf16"):
        dev, width = model.device, -(-most // PAGE)
        self.caches = [sv.new_paged_cache(lanes * width, PAGE, KV_HEADS, DIM, CACHES[cache], dev) for _ in range(model.layers)]
        self.free = torch.randperm(lanes * width).tolist()
        self.pages = [[] for _ in range(lanes)]
        self.tables = torch.zeros(lanes, width, dtype=torch.int32, device=dev)
        self.cached = torch.zeros(lanes, dtype=torch.int32, device=dev)
        self.lens = [0] * lanes  # what ``cached`` holds, on the host
        self.model = model

    def run(self, rows, status=None):
        """Logits of each lane's new tokens ``rows[lane]`` behind what its cache holds; they are
        in the cache then, but not yet counted."""
        dev = self.model.device
        for b, r in enumerate(rows):
            while len(self.pages[b]) * PAGE < self.lens[b] + len(r):
                self.pages[b].append(self.free.pop())
                self.tables[b, len(self.pages[b]) - 1] = self.pages[b][-1]
        ends = [sum(len(r) for r in rows[:b]) for b in range(len(rows) + 1)]
        off = torch.tensor(ends, dtype=torch.int32, device=dev)
        most = max(len(r) for r in rows)
        workspace = sv.new_paged_attention_workspace(Q_HEADS, KV_HEADS, DIM, most, dev)
        status = torch.zeros(len(rows), dtype=torch.int32, device=dev) if status is None else status

        def attend(layer, q, k, v):
            where = (self.caches[layer], self.tables, self.cached, off)
            out = torch.empty(q.shape, dtype=q.dtype, device=dev)
            sv.spec_cache_write(*where, k, v, most, lane_status=status)
            sv.spec_paged_attention(q, *where, out, most, lane_status=status, workspace=workspace)
            return out

        tokens = torch.tensor([t for r in rows for t in r], dtype=torch.int32, device=dev)
        return self.model.forward(tokens, attend), off, status

    def keep(self, counts):
        """Counts the first ``counts[lane]`` of the last run's tokens (an int32 tensor)."""
        self.cached += counts
        self.lens = [n + c for n, c in zip(self.lens, counts.tolist())]


def start(model, prompts, tokens, cache):
    """Lanes that hold all but the last token of each prompt (it is the first round's anchor)."""
    lanes = Lanes(model, len(prompts), max(len(p) for p in prompts) + tokens + 17, cache)
    rows = [p[:-1] for p in prompts]
    _, _, status = lanes.run(rows)
    if int(status.max()) != 0:
        raise RuntimeError(f"prefill: lane status {status.tolist()}")
    lanes.keep(torch.tensor([len(r) for r in rows], dtype=torch.int32, device=model.device))
    return lanes


def decode(model, prompts, tokens, cache="bf16"):
    """Plain greedy decoding, one token of every lane at a time: the lanes' new tokens."""
    lanes = start(model, prompts, tokens, cache)
    last, new = [p[-1] for p in prompts], []
    one = torch.ones(len(prompts), dtype=torch.int32, device=model.device)
    for _ in range(tokens):
        logits, _, _ = lanes.run([[t] for t in last])
        lanes.keep(one)
        last = logits.argmax(1).tolist()
        new.append(last)
    return [list(n) for n in zip(*new)]


def speculate(model, prompts, tokens, drafts=3, cache="bf16"):
    """Greedy speculative rounds until every lane has ``tokens`` new ones: the new tokens and the
    number of rounds."""
    dev, n = model.device, len(prompts)
    lanes = start(model, prompts, tokens, cache)
    history = [list(p) for p in prompts]
    greedy = torch.zeros(n, dtype=torch.float32, device=dev)
    rounds = 0
    while min(len(h) - len(p) for h, p in zip(history, prompts)) < tokens:
        rounds += 1
        flat = torch.tensor([t for h in history for t in h], dtype=torch.int32, device=dev)
        ends = torch.tensor([sum(len(h) for h in history[:i]) for i in range(n + 1)], dtype=torch.int64, device=dev)
        guess = torch.full((n, drafts), -1, dtype=torch.int32, device=dev)
        lens = torch.empty(n, dtype=torch.int32, device=dev)
        # A lane that is done drafts nothing more.
        sv.spec_ngram_draft(flat, ends, drafts, guess, lens)
        lens *= torch.tensor([len(h) - len(p) < tokens for h, p in zip(history, prompts)], device=dev)
        k, g = lens.tolist(), guess.tolist()
        logits, off, status = lanes.run([[h[-1]] + g[b][:k[b]] for b, h in enumerate(history)])
        slots = torch.tensor([t for b in range(n) for t in g[b][:k[b]] + [-1]], dtype=torch.int32, device=dev)
        committed, verdict = (torch.empty(n, dtype=torch.int32, device=dev) for _ in range(2))
        out = torch.empty(logits.shape[0], dtype=torch.int32, device=dev)
        sv.spec_verify_accept(logits, None, slots, lens, off, greedy, rounds, committed, out, verdict)
        if int(torch.maximum(status, verdict).max()) != 0:
            raise RuntimeError(f"round {rounds}: lane status {status.tolist()}, {verdict.tolist()}")
        lanes.keep(committed)
        c, o, first = committed.tolist(), out.tolist(), off.tolist()
        for b in range(n):
            if len(history[b]) - len(prompts[b]) < tokens:
                history[b] += o[first[b]:first[b] + c[b]]
            else:  # (kept in step with the cache)
                lanes.cached[b] -= c[b]
                lanes.lens[b] -= c[b]
    return [h[len(p):] for h, p in zip(history, prompts)], rounds


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--lanes", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=48)
    ap.add_argument("--cache", choices=sorted(CACHES), default="e4m3")
    args = ap.parse_args()
    model = AttentionModel()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, model.vocab, (40 + 61 * b,), generator=g).tolist() for b in range(args.lanes)]
    new, rounds = speculate(model, prompts, args.tokens, cache=args.cache)
    plain = decode(model, prompts, max(len(n) for n in new), args.cache)
    for b, n in enumerate(new):
        same = n == plain[b][:len(n)]
        print(f"lane {b}: {len(n)} tokens in {rounds} rounds, {'equal to' if same else 'DIFFERENT from'} plain decoding")


if __name__ == "__main__":
    main()
