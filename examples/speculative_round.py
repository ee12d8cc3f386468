"""Speculative decoding of one request through one attention layer with packed weights.

A layer of random weights and an lm_head tied to the embeddings such that the drafter, a table of
next tokens, is often right.  A prompt goes through in blocks; then rounds of one target token and
seven drafts run on the device alone:

    embed -> plan_round -> QKV product -> rope_append -> attention -> O product -> lm_head
          -> verify_sampled -> the next round's length and tokens

The round is captured into a HIP graph and replayed; nothing is read back until the end.

    python examples/speculative_round.py [--rounds N] [--prompt TOKENS]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp8_quantized_skinny_qpn_amd import kv, qpn  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, VOCAB, ROWS, BLOCK = 1024, 10, 2, 128, 4000, 8, 256


class Model:
    def __init__(self, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.emb = normal(VOCAB, HIDDEN).half()
        self.follows = torch.randperm(VOCAB, generator=g, device="cuda").int()   # the drafter's next tokens
        head = torch.empty(VOCAB, HIDDEN, device="cuda")
        head[self.follows.long()] = self.emb.float() * (6.0 / HIDDEN)            # the target mostly agrees
        scale = HIDDEN ** -0.5
        self.qkv = qpn.pack_fp8(normal((Q_HEADS + 2 * KV_HEADS) * DIM, HIDDEN) * scale)
        self.o = qpn.pack_fp8(normal(HIDDEN, Q_HEADS * DIM) * scale)
        self.head = qpn.pack_fp8(head)
        self.q_norm = torch.ones(DIM, dtype=torch.float16, device="cuda")
        self.k_norm = torch.ones(DIM, dtype=torch.float16, device="cuda")
        self.inv_freq = (1e4 ** (-torch.arange(DIM // 2, device="cuda") / (DIM // 2))).float()

    def layer(self, cache, tokens, r, table, product):
        """Hidden states of the rows after attention, their keys and values appended to the cache."""
        x = self.emb[tokens.long()]
        q = kv.rope_append(cache, product(self.qkv, x), Q_HEADS, r.positions, r.slots, self.inv_freq, self.q_norm,
                           self.k_norm)
        y = kv.attention(cache, q, r.row_start, r.seq_lens, table, tokens.shape[0])
        return x + product(self.o, y)


class Decoder:
    """The state of one request; round() enqueues a round and reads nothing back."""

    def __init__(self, model, most_tokens: int, rounds: int, seed: int = 1, temperature: float = 0.7):
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.model, self.temperature = model, temperature
        pages = -(-most_tokens // kv.PAGE)
        self.cache = kv.KvCache.empty(pages, KV_HEADS, DIM)
        self.table, self.free = z(1, pages), torch.arange(pages, dtype=torch.int32, device="cuda")
        self.before, self.held, self.free_count = z(1), z(1), z(1) + pages
        self.history, self.tokens, self.at = z(most_tokens), z(ROWS), z(1)
        self.accepted = z(rounds)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.accept_u = torch.rand(rounds, ROWS, generator=g, device="cuda")
        self.sample_u = torch.rand(rounds, 1, generator=g, device="cuda")

    def _open(self, rows: int) -> kv.Round:
        r = kv.plan_round(self.before, torch.full_like(self.before, rows), self.held, self.table, self.free,
                          self.free_count, capacity=rows)
        self.held.copy_(r.held)
        self.free_count.copy_(r.free_count)
        return r

    def prompt(self, tokens):
        """All of the prompt but its last token, which opens the first round."""
        for part in tokens[:-1].split(BLOCK):
            r = self._open(part.shape[0])
            self.model.layer(self.cache, part, r, self.table, qpn.prefill)
            self.before += part.shape[0]
        self.history[:tokens.shape[0]] = tokens
        self._draft(tokens[-1:])

    def _draft(self, token):
        rows = [token]
        for _ in range(ROWS - 1):
            rows.append(self.model.follows[rows[-1].long()])
        self.tokens.copy_(torch.cat(rows))

    def round(self):
        m, i = self.model, self.at.long()
        r = self._open(ROWS)
        self.history.index_copy_(0, r.positions.long(), self.tokens)   # what is refused is written over later
        logits = qpn.gemm(m.head, m.layer(self.cache, self.tokens, r, self.table, qpn.gemm))
        accepted, token, _ = kv.verify_sampled(logits, self.tokens, r.row_start, self.accept_u[i].view(-1),
                                               self.sample_u[i].view(-1), temperature=self.temperature)
        self.accepted.index_copy_(0, i, accepted)
        self.before += accepted + 1
        self.at += 1
        self._draft(token)


def decode(model, prompt, rounds: int, graph: bool):
    """(tokens after the prompt, accepted drafts of each round, seconds a round)."""
    d = Decoder(model, prompt.shape[0] + rounds * ROWS + ROWS, rounds)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        d.prompt(prompt)
        d.round()                       # the stream's workspaces exist from here on
    stream.synchronize()
    run = d.round
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            d.round()
        run = g.replay
    t = time.perf_counter()
    with torch.cuda.stream(stream):
        for _ in range(rounds - 1):
            run()
    stream.synchronize()
    t = (time.perf_counter() - t) / max(rounds - 1, 1)
    accepted = d.accepted.tolist()
    n = int(d.before)
    assert n == prompt.shape[0] - 1 + sum(accepted) + rounds
    return d.history[prompt.shape[0]:n].tolist() + [int(d.tokens[0])], accepted, t


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rounds", type=int, default=40)
    ap.add_argument("--prompt", type=int, default=1000)
    a = ap.parse_args()
    model = Model()
    prompt = torch.randint(0, VOCAB, (a.prompt,), generator=torch.Generator().manual_seed(2)).int().cuda()
    for graph in (False, True):
        tokens, accepted, t = decode(model, prompt, a.rounds, graph)
        print(f"{'graph' if graph else 'eager'}: {len(tokens)} tokens in {a.rounds} rounds, "
              f"{sum(accepted) / a.rounds:.2f} drafts accepted a round, {t * 1e6:.0f} us a round", flush=True)


if __name__ == "__main__":
    main()
