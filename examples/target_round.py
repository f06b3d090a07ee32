"""The target's side of speculative decoding, round by round, on a toy model.

A one-layer attention model with random weights is the target; the same model without its
attention is the draft (the next token from the last one alone).  Prompts of different lengths enter the paged
cache as one chunk; every round then

  1. writes the chunk's keys and values into the cache (spec_kv_append; with rotary positions
     spec_kv_append_rope, which turns the keys and the queries on the way),
  2. attends over the cache (spec_chunk_attention),
  3. verifies the drafts against the target's probabilities with given uniforms
     (spec_verify_probs), and
  4. forgets the rejected drafts: kv_len shrinks, nothing moves.

At the end the cached prefixes are read back (spec_kv_read), as for a move to another pool.

    python examples/target_round.py [--rounds 8] [--e4m3 | --u4] [--rotary]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_21_gb300 as sv  # noqa: E402


class ToyTarget:
    """Embedding, one grouped-head attention layer over a paged cache, output head.  rotary: for how
    many positions (0: the attention knows none)."""

    def __init__(self, vocab=512, heads=8, kv_heads=2, head_dim=64, seed=0, device="cuda", rotary=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        width = heads * head_dim
        self.vocab, self.heads, self.kv_heads, self.head_dim = vocab, heads, kv_heads, head_dim
        randn = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.embed = (randn(vocab, width) * 0.3).to(torch.bfloat16)
        self.w_qkv = (randn(width, (heads + 2 * kv_heads) * head_dim) * width ** -0.5 * 3).to(
            torch.bfloat16)
        self.w_out = (randn(width, width) * width ** -0.5).to(torch.bfloat16)
        self.head = (randn(width, vocab) * 0.3).to(torch.bfloat16)
        self.cos_sin = None
        if rotary:
            i = torch.arange(head_dim // 2, device=device).double()
            turn = torch.arange(rotary, device=device)[:, None] * 10000.0 ** (-2 * i / head_dim)
            self.cos_sin = torch.cat([turn.cos(), turn.sin()], 1).float()

    def draft_logits(self, tokens):
        """The draft model: logits of the next token from the last token's embedding."""
        return self.embed[tokens].float() @ self.head.float()

    def chunk(self, tokens, cache, table, q_start, kv_len):
        """Logits [total, vocab] of a packed chunk of new tokens, whose keys and values enter
        the cache on the way."""
        x = self.embed[tokens]
        qkv = (x @ self.w_qkv).view(len(tokens), -1, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        if self.cos_sin is None:
            sv.spec_kv_append(cache, k, v, table, q_start, kv_len)
        else:
            q = sv.spec_kv_append_rope(cache, k, v, table, q_start, kv_len, self.cos_sin, q=q)["q"]
        a = sv.spec_chunk_attention(q, cache, table, q_start, kv_len, want_lse=False)["out"]
        y = x + a.reshape(len(tokens), -1) @ self.w_out
        return y.float() @ self.head.float()


class Rounds:
    """A batch of sequences and their cache."""

    def __init__(self, model: ToyTarget, prompts, *, gamma=4, room=512, page_size=16, e4m3=False,
                 seed=1, u4=False):
        self.model, self.gamma, self.tokens = model, gamma, [list(p) for p in prompts]
        dev = model.embed.device
        B, pages = len(prompts), -(-room // page_size)
        self.room = pages * page_size
        self.check_room(-1)
        dtype = torch.uint8 if u4 else torch.float8_e4m3fn if e4m3 else torch.bfloat16
        self.cache = sv.alloc_kv_cache(B * pages, model.kv_heads, page_size, model.head_dim,
                                       dtype=dtype, device=dev)
        self.gen = torch.Generator(device=dev)
        self.gen.manual_seed(seed)
        order = torch.randperm(B * pages, generator=self.gen, device=dev)
        self.table = order.view(B, pages).to(torch.int32)
        self.kv_len = torch.zeros(B, dtype=torch.int32, device=dev)
        self.accepted = 0
        # the prompts without their last tokens, as one packed chunk
        n = [len(p) - 1 for p in prompts]
        if max(n):
            start = torch.tensor([0, *n], device=dev).cumsum(0).to(torch.int32)
            self.kv_len += torch.tensor(n, dtype=torch.int32, device=dev)
            flat = torch.tensor([t for p in prompts for t in p[:-1]], device=dev)
            model.chunk(flat, self.cache, self.table, start, self.kv_len)
        self.last = torch.tensor([p[-1] for p in prompts], device=dev)

    def check_room(self, more):
        """Every sequence's tokens and `more` have to fit its pages (the cache would drop the rest
        and flag it)."""
        if max(len(t) for t in self.tokens) + more > self.room:
            raise ValueError(f"a sequence has no room left in its {self.room} cached tokens")

    def round(self):
        """One round; returns the tokens it emitted, -1 behind them [B, gamma+1]."""
        m, B, g = self.model, len(self.tokens), self.gamma
        self.check_room(g)
        dev = self.last.device
        drafts, q, x = [], [], self.last
        for _ in range(g):
            q.append(torch.softmax(m.draft_logits(x), -1))
            x = torch.multinomial(q[-1], 1, generator=self.gen)[:, 0]
            drafts.append(x)
        drafts, q = torch.stack(drafts, 1), torch.stack(q, 1)
        chunk = torch.cat([self.last[:, None], drafts], 1)
        start = torch.arange(0, B * (g + 1) + 1, g + 1, dtype=torch.int32, device=dev)
        self.kv_len += g + 1
        logits = m.chunk(chunk.reshape(-1), self.cache, self.table, start, self.kv_len)
        p = torch.softmax(logits, -1).view(B, g + 1, -1)
        u = torch.rand((B, g + 1), generator=self.gen, device=dev)
        r = sv.spec_verify_probs(p, q, drafts.to(torch.int32), u)
        self.kv_len -= g - r["counts"]  # the last token and the accepted drafts stay
        self.last = torch.gather(r["tokens"], 1, r["counts"][:, None].long())[:, 0].long()
        out = r["tokens"].tolist()
        for b in range(B):
            self.tokens[b] += [t for t in out[b] if t >= 0]
        self.accepted += int(r["counts"].sum())
        return r["tokens"]

    def cached(self):
        """Keys and values of every sequence's cached tokens, packed, and where each starts."""
        start = torch.cat([self.kv_len.new_zeros(1), self.kv_len.cumsum(0).to(torch.int32)])
        o = sv.spec_kv_read(self.cache, self.table, torch.zeros_like(self.kv_len), start,
                            int(start[-1]))
        return o["k"], o["v"], start


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--rounds", type=int, default=8)
    held = ap.add_mutually_exclusive_group()
    held.add_argument("--e4m3", action="store_true", help="hold the cache in 8 bits")
    held.add_argument("--u4", action="store_true", help="hold the cache in 4 bits")
    ap.add_argument("--rotary", action="store_true", help="rotary positions")
    a = ap.parse_args()
    prompts = [list(range(3 + 5 * b, 3 + 5 * b + n)) for b, n in enumerate((40, 7, 130, 1))]
    r = Rounds(ToyTarget(rotary=512 if a.rotary else 0), prompts, e4m3=a.e4m3, u4=a.u4)
    for _ in range(a.rounds):
        r.round()
    k, _, start = r.cached()
    for b, t in enumerate(r.tokens):
        print(f"sequence {b}: {len(prompts[b])} prompt tokens, then {t[len(prompts[b]):]}")
    print(f"{r.accepted} of {a.rounds * r.gamma * len(prompts)} drafts accepted; "
          f"{int(start[-1])} cached tokens read back, keys {tuple(k.shape)}")


if __name__ == "__main__":
    main()
