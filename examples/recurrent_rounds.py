"""Speculative rounds of a recurrent target, from the prompt to the reported log
probabilities.

A small random model whose layers keep a linear-attention state stands for the
target.  The prompts go through ``spec_linear_prefill``; then each round drafts
from the conversation, runs the anchor and the drafts of every lane through
``spec_linear_verify`` (which stages the state after every column), accepts with
``spec_verify_accept``, rolls the states with ``spec_commit_state`` and reports
the committed tokens' log probabilities with ``spec_token_logprobs``.

    python examples/recurrent_rounds.py [--lanes 4] [--tokens 48]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import speculative_decoding_verify_bf16_gb300 as sv  # noqa: E402

HEADS, DIM = 2, 128


class RecurrentModel:
    """A bigram table plus layers of linear attention with one decay a head."""

    def __init__(self, vocab=257, layers=2, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        hidden = HEADS * DIM

        def weights(*shape):
            return torch.randn(*shape, generator=g, device=device) / shape[-2] ** 0.5

        self.vocab, self.layers, self.device = vocab, layers, torch.device(device)
        self.embed = torch.randn(vocab, hidden, generator=g, device=device)
        self.proj = [weights(hidden, 3 * hidden) for _ in range(layers)]
        self.merge = [weights(hidden, hidden) for _ in range(layers)]
        self.unembed = weights(hidden, vocab)
        self.decay = -torch.logspace(-2, -0.5, HEADS, device=device)
        # Likely successors that soon run in circles, as drafting needs.
        self.next = torch.randint(0, 11, (vocab,), generator=g, device=device)

    def forward(self, tokens, attend):
        """Logits [rows, vocab] of packed tokens; attend(layer, q, k, v, decay) is
        the layer's linear attention."""
        x = self.embed[tokens.long()]
        rows = x.shape[0]
        for layer in range(self.layers):
            q, k, v = (x @ self.proj[layer]).view(rows, 3, HEADS, DIM).unbind(1)
            q, k = (torch.nn.functional.normalize(t, dim=-1).to(torch.bfloat16) for t in (q, k))
            o = attend(layer, q, k, v.to(torch.bfloat16), self.decay.expand(rows, HEADS))
            x = x + o.float().reshape(rows, -1) @ self.merge[layer]
        logits = x @ self.unembed
        logits[torch.arange(rows, device=x.device), self.next[tokens.long()]] += 12.0
        return logits


def _offsets(lens, device):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=device)


def prefill(model, prompts):
    """The lanes' live states [lanes, layers, heads, dim, dim] after all but the last
    token of each prompt (the last one is the first round's anchor)."""
    dev = model.device
    lens = [len(p) - 1 for p in prompts]
    tokens = torch.tensor([t for p in prompts for t in p[:-1]], dtype=torch.int32, device=dev)
    off = _offsets(lens, dev)
    live = torch.zeros(len(prompts), model.layers, HEADS, DIM, DIM, device=dev)
    status = torch.zeros(len(prompts), dtype=torch.int32, device=dev)
    workspace = sv.new_linear_workspace(len(prompts), HEADS, DIM, DIM, max(lens), dev)

    def attend(layer, q, k, v, decay):
        out = torch.empty_like(v)
        sv.spec_linear_prefill(q, k, v, decay, off, None, out, live[:, layer], max(lens), lane_status=status,
                               workspace=workspace)
        return out

    model.forward(tokens, attend)
    if int(status.max()) != 0:
        raise RuntimeError(f"prefill: lane status {status.tolist()}")
    return live


def decode(model, prompts, tokens):
    """Plain greedy decoding, one token of every lane at a time: the lanes' new tokens."""
    dev = model.device
    live = prefill(model, prompts)
    off = _offsets([1] * len(prompts), dev)
    last = torch.tensor([p[-1] for p in prompts], dtype=torch.int32, device=dev)
    new = []

    def attend(layer, q, k, v, decay):
        out = torch.empty_like(v)
        state = live[:, layer]
        sv.spec_linear_verify(q, k, v, decay, off, state, state.unsqueeze(1), out)
        return out

    for _ in range(tokens):
        last = model.forward(last, attend).argmax(1).to(torch.int32)
        new.append(last)
    return torch.stack(new, 1).tolist()


def speculate(model, prompts, tokens, drafts=3, top=4):
    """Greedy speculative rounds until every lane has ``tokens`` new ones.

    Returns the lanes' new tokens, their log probabilities, the first lane's
    alternatives in the last round and the number of rounds."""
    dev, lanes = model.device, len(prompts)
    live = prefill(model, prompts)
    staged = torch.zeros(lanes, drafts + 1, *live.shape[1:], device=dev)
    history = [list(p) for p in prompts]
    logps = [[] for _ in prompts]
    greedy = torch.zeros(lanes, dtype=torch.float32, device=dev)
    rounds = 0
    alternatives = None
    while min(len(h) - len(p) for h, p in zip(history, prompts)) < tokens:
        rounds += 1
        flat = torch.tensor([t for h in history for t in h], dtype=torch.int32, device=dev)
        ends = torch.tensor([sum(len(h) for h in history[:i]) for i in range(lanes + 1)], dtype=torch.int64, device=dev)
        guess = torch.full((lanes, drafts), -1, dtype=torch.int32, device=dev)
        lens = torch.empty(lanes, dtype=torch.int32, device=dev)
        sv.spec_ngram_draft(flat, ends, drafts, guess, lens)
        k = lens.tolist()
        off_host = [sum(k[:b]) + b for b in range(lanes + 1)]
        off = torch.tensor(off_host, dtype=torch.int32, device=dev)
        rows = off_host[-1]
        columns, slots = [], []
        for b, g in enumerate(guess.tolist()):
            columns += [history[b][-1]] + g[:k[b]]
            slots += g[:k[b]] + [-1]
        status = torch.zeros(lanes, dtype=torch.int32, device=dev)

        def attend(layer, q, kk, v, decay):
            out = torch.empty_like(v)
            sv.spec_linear_verify(q, kk, v, decay, off, live[:, layer], staged[:, :, layer], out, lane_status=status)
            return out

        logits = model.forward(torch.tensor(columns, dtype=torch.int32, device=dev), attend)
        committed = torch.empty(lanes, dtype=torch.int32, device=dev)
        out = torch.empty(rows, dtype=torch.int32, device=dev)
        verdict = torch.empty(lanes, dtype=torch.int32, device=dev)
        sv.spec_verify_accept(logits, None, torch.tensor(slots, dtype=torch.int32, device=dev), lens, off, greedy, rounds,
                              committed, out, verdict)
        status = torch.maximum(status, verdict)
        sv.spec_commit_state(staged, live, committed, status)
        logp, entropy = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
        ids = torch.empty(rows, top, dtype=torch.int32, device=dev)
        alts = torch.empty(rows, top, device=dev)
        sv.spec_token_logprobs(logits, out, logp, entropy=entropy, top_ids=ids, top_logprobs=alts)
        if int(status.max()) != 0:
            raise RuntimeError(f"round {rounds}: lane status {status.tolist()}")
        c, o, lp = committed.tolist(), out.tolist(), logp.tolist()
        for b in range(lanes):
            history[b] += o[off_host[b]:off_host[b] + c[b]]
            logps[b] += lp[off_host[b]:off_host[b] + c[b]]
        alternatives = list(zip(ids[0].tolist(), alts[0].tolist()))
    return [h[len(p):] for h, p in zip(history, prompts)], logps, alternatives, rounds


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--lanes", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=48)
    args = ap.parse_args()
    model = RecurrentModel()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, model.vocab, (40 + 61 * b,), generator=g).tolist() for b in range(args.lanes)]
    new, logps, alternatives, rounds = speculate(model, prompts, args.tokens)
    plain = decode(model, prompts, max(len(n) for n in new))
    for b, n in enumerate(new):
        same = n == plain[b][:len(n)]
        print(f"lane {b}: {len(n)} tokens in {rounds} rounds, mean log p {sum(logps[b]) / len(n):.3f}, "
              f"{'equal to' if same else 'DIFFERENT from'} plain decoding")
    print("last round, first row's alternatives:", ", ".join(f"{i} ({lp:.2f})" for i, lp in alternatives))


if __name__ == "__main__":
    main()
