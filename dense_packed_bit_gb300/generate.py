"""Answers from a small language model with ternary weights, served the way the pieces are meant to be used together:
packed products for the projections, a paged cache of keys and values, attention over it, drafted tokens verified as a
tree, and the sampler.

    python -m dense_packed_bit_gb300.generate [--answers N] [--tokens N] [--depth N] [--temperature T] [--window W]

The model is GPT-2's block (pre-norm, learned positions, GELU) with grouped key and value heads and random weights: there
is no checkpoint here, so the text means nothing, but every step runs as it would with one.  A batch of prompts is
processed in one call per layer, each is forked into several answers that share its full pages, and each round then
verifies a tree of drafted tokens per answer: by default what follows earlier occurrences of the last token in the
answer's own history.  The sampler gets the same uniform number at a position whatever was drafted, so drafts change how
many rounds an answer takes, not which tokens it has (but for rounding at a tie).  A random model does not repeat itself,
so the command drafts with a stand-in for a draft model instead: the answer found without drafts, each token of it right
with --accept probability.
"""
import argparse
import math
import time
from dataclasses import dataclass

import numpy as np
import torch
import torch.nn.functional as F

import dense_packed_bit_gb300 as mm
from dense_packed_bit_gb300 import synth


@dataclass
class Shape:
    vocab: int = 5003
    layers: int = 2
    heads: int = 8
    kv_heads: int = 2
    dim: int = 64
    hidden: int = 1024
    positions: int = 2048

    @property
    def width(self):
        return self.heads * self.dim


class Packed:
    """A ternary matrix [rows][cols], 2 bits a weight, outputs of about the inputs' size."""

    def __init__(self, seed, rows, cols, device):
        self.rows, self.cols = rows, cols
        codes = synth.ternary_field_bytes(seed, rows * cols // 4).reshape(rows, cols // 4)
        size = 1.0 / math.sqrt(cols * 2 / 3)
        scales = synth.uniform_f16_bits(seed + 1, (rows,), 0.9 * size, 1.1 * size)
        self.codes, self.scales = torch.from_numpy(codes).to(device), torch.from_numpy(scales).to(device)

    def __call__(self, x):
        y = torch.empty(x.shape[0], self.rows, dtype=torch.float32, device=x.device)
        mm.mm_gemm_packed2(self.codes, self.scales, x, y, x.shape[0], self.rows, self.cols, synth.CODEBOOK_TERNARY)
        return y


class Model:
    def __init__(self, shape, seed=7, device="cuda"):
        self.shape, self.device = shape, device
        d, kv = shape.width, shape.kv_heads * shape.dim
        self.tokens = torch.from_numpy(synth.normal_f32(seed, (shape.vocab, d), 1.0)).to(device)
        self.places = torch.from_numpy(synth.normal_f32(seed + 1, (shape.positions, d), 0.3)).to(device)
        self.head = torch.from_numpy(synth.normal_f32(seed + 2, (shape.vocab, d), 1.0)).to(device)
        self.blocks = []
        for i in range(shape.layers):
            s = seed + 10 * (i + 1)
            self.blocks.append([Packed(s, d + 2 * kv, d, device), Packed(s + 2, d, d, device),
                                Packed(s + 4, shape.hidden, d, device), Packed(s + 6, d, shape.hidden, device)])

    def forward(self, tokens, places, attend):
        """Logits [tokens][vocab] fp32.  attend(layer, q, k, v): appends k, v and returns the attention of q."""
        s = self.shape
        d, kv = s.width, s.kv_heads * s.dim
        x = self.tokens[tokens] + self.places[places]
        for layer, (qkv, out, up, down) in enumerate(self.blocks):
            h = qkv(F.layer_norm(x, (d,)).half()).half()
            x = x + out(attend(layer, h[:, :d], h[:, d:d + kv], h[:, d + kv:]))
            x = x + down(F.gelu(up(F.layer_norm(x, (d,)).half()), approximate="tanh").half())
        x = F.layer_norm(x, (d,))
        logits = torch.empty(x.shape[0], s.vocab, dtype=torch.float32, device=x.device)
        mm.mm_gemm_f32(0, 1, x.shape[0], s.vocab, d, x, d, self.head, d, logits, s.vocab)
        return logits / math.sqrt(d)  # of unit size


def lookup(history, depth, branches=2):
    """Drafts from the answer itself: what followed the latest earlier occurrences of its last token, first tokens
    different."""
    found, firsts = [], set()
    for at in range(len(history) - 2, -1, -1):
        if len(found) == branches:
            break
        if history[at] == history[-1] and history[at + 1] not in firsts:
            firsts.add(history[at + 1])
            found.append(history[at + 1:at + 1 + depth])
    return found


class Server:
    """A model with a cache of `pages` pages for `seqs` sequences."""

    def __init__(self, model, seqs, pages, page_size=16):
        s, dev = model.shape, model.device
        self.model, self.seqs = model, seqs
        shape = (s.layers, pages, s.kv_heads, page_size, s.dim)
        self.k, self.v = (torch.empty(shape, dtype=torch.float16, device=dev) for _ in range(2))
        self.table = torch.full((seqs, -(-s.positions // page_size)), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=dev)
        self.missing = torch.zeros(1, dtype=torch.int32, device=dev)
        self.cache = mm.mm_cache(self.k, self.v, self.table, self.lens, self.refs)
        self.workspace = torch.zeros(0, dtype=torch.uint8, device=dev)

    def ints(self, values):
        return torch.tensor(values, dtype=torch.int32).to(self.model.device)

    def step(self, new, places, window=0, sinks=0, trees=None):
        """Logits of the new tokens new[s] (a list per sequence, [] for none) at places[s].  trees[s][i]: the drafted
        tokens that token i sees (itself included); None: all up to it."""
        s = self.model.shape
        if any(not 0 <= p < s.positions for seq in places for p in seq):
            raise ValueError(f"the model has {s.positions} positions")
        if any(not 0 <= t < s.vocab for seq in new for t in seq):
            raise ValueError(f"a token is not in the vocabulary of {s.vocab}")
        if window and trees is not None and any(len(row) > window for tree in trees for row in tree):
            raise ValueError("a drafted token with more ancestors than the window holds sees more than it would if decoded")
        c = self.cache
        counts = [len(t) for t in new]
        tokens, most = sum(counts), max(counts)
        starts = self.ints(np.concatenate([[0], np.cumsum(counts)]).tolist())
        mm.mm_cache_reserve(c, self.ints(counts), self.missing)
        if int(self.missing):
            raise RuntimeError(f"{int(self.missing)} pages are lacking")
        mask, words = None, (most + 31) // 32
        if trees is not None:
            bits = np.zeros((tokens, words), dtype=np.uint32)
            for r, row in enumerate(row for tree in trees for row in tree):
                for t in row:
                    bits[r, t // 32] |= np.uint32(1 << t % 32)
            mask = torch.from_numpy(bits.view(np.int32)).to(self.model.device)
        need = mm.mm_cache_attention_workspace(c, s.heads, tokens, most)
        if need > self.workspace.numel():
            self.workspace = torch.zeros(need, dtype=torch.uint8, device=self.model.device)

        def attend(layer, q, k, v):
            mm.mm_cache_append(c, layer, k, v, k.stride(0), starts, tokens, most)
            o = torch.empty(tokens, s.width, dtype=torch.float16, device=q.device)
            rest = (window, sinks, 1.0 / math.sqrt(s.dim), o, s.width, self.workspace, self.workspace.numel())
            if mask is None:
                mm.mm_cache_attention(c, layer, q, q.stride(0), s.heads, starts, tokens, most, *rest)
            else:
                mm.mm_cache_attention_tree(c, layer, q, q.stride(0), s.heads, starts, tokens, most, mask, words, *rest)
            return o

        flat = [t for seq in new for t in seq]
        at = [p for seq in places for p in seq]
        self.starts, self.counts, self.most = starts, counts, most
        return self.model.forward(torch.tensor(flat).to(self.model.device), torch.tensor(at).to(self.model.device), attend)

    def keep(self, keep=None):
        """Ends a step: keep[s] are the new tokens of sequence s that stay (None: all)."""
        tokens = sum(self.counts)
        if keep is None:
            mm.mm_cache_compact(self.cache, self.starts, None, None, tokens, self.most)
            return
        rows = [k for s, n in enumerate(self.counts) for k in (keep[s] + [0] * n)[:n]]
        mm.mm_cache_compact(self.cache, self.starts, self.ints(rows), self.ints([len(k) for k in keep]), tokens, self.most)

    def free(self, seqs, window=0, sinks=0):
        mm.mm_cache_free(self.cache, self.ints(seqs), len(seqs), window, sinks)

    def fork(self, parents, children):
        mm.mm_cache_fork(self.cache, self.ints(parents), self.ints(children), len(children), self.missing)
        if int(self.missing):
            raise RuntimeError(f"{int(self.missing)} pages are lacking")


def sample(logits, u, temperature, top_k, top_p):
    n, dev = logits.shape[0], logits.device
    tokens = torch.empty(n, dtype=torch.int32, device=dev)
    mm.mm_sample(logits, n, logits.shape[1], logits.stride(0), torch.full((n,), temperature, device=dev),
                 torch.full((n,), top_k, dtype=torch.int32, device=dev), torch.full((n,), top_p, device=dev), None, u, tokens)
    return tokens.tolist()


def generate(server, prompts, answers, tokens, temperature=0.8, top_k=40, top_p=0.95, depth=4, window=0, sinks=0, seed=1,
             draft=None):
    """`answers` answers of `tokens` tokens to each prompt (lists of tokens), and the rounds each took.  depth: drafted
    tokens in a row, 0 for none; draft(answer, history): other drafts than lookup's, a list of branches whose first
    tokens differ."""
    P, A = len(prompts), len(prompts) * answers
    first = [P + i for i in range(A)]  # sequences: the prompts, then the answers
    if server.seqs < P + A:
        raise ValueError("the server has too few sequences")
    if not prompts or not all(prompts):
        raise ValueError("a prompt needs a token")
    if window and depth and depth + 1 > window:
        raise ValueError(f"drafts of {depth} tokens do not fit a window of {window}: they would see more than decoded tokens do")
    # an answer's last token is not processed; drafts follow the one before it
    if max(len(p) for p in prompts) - 1 + (tokens - 1 + depth if tokens > 1 else 0) >= server.model.shape.positions:
        raise ValueError(f"the model has {server.model.shape.positions} positions")
    generator = torch.Generator().manual_seed(seed)
    longest = max(len(p) for p in prompts)
    u = torch.rand(longest + tokens + depth + 2, A, generator=generator).T  # by position, so the same for any depth
    draft = draft or (lambda answer, history: lookup(history, depth))

    none = [[] for _ in range(A)]
    logits = server.step(prompts + none, [list(range(len(p))) for p in prompts] + none, window, sinks)
    server.keep()
    server.fork([i // answers for i in range(A)], first)
    server.free(list(range(P)))
    last = np.cumsum([len(p) for p in prompts]) - 1
    rows = torch.tensor([int(last[i // answers]) for i in range(A)]).to(logits.device)
    history = [list(prompts[i // answers]) for i in range(A)]
    begin = [len(h) for h in history]
    for i, t in enumerate(sample(logits[rows].contiguous(), torch.stack([u[i, begin[i]] for i in range(A)]).to(logits.device),
                                 temperature, top_k, top_p)):
        history[i].append(t)

    rounds = [0] * A
    while any(len(h) - b < tokens for h, b in zip(history, begin)):
        new, places, trees, parents, us = [[] for _ in range(P)], [[] for _ in range(P)], [[] for _ in range(P)], [], []
        for i, h in enumerate(history):
            if len(h) - begin[i] >= tokens:  # this answer is complete
                new.append([]), places.append([]), trees.append([]), parents.append([])
                continue
            rounds[i] += 1
            node, up, sees = [h[-1]], [-1], [[0]]
            for branch in draft(i, h) if depth else []:
                at = 0
                for t in branch:
                    node.append(t), up.append(at), sees.append(sees[at] + [len(node) - 1])
                    at = len(node) - 1
            place = [len(h) - 1 + len(x) - 1 for x in sees]
            new.append(node), places.append(place), trees.append(sees), parents.append(up)
            us += [u[i, p + 1] for p in place]
        logits = server.step(new, places, window, sinks, trees if depth else None)
        chosen = sample(logits, torch.stack(us).to(logits.device), temperature, top_k, top_p)
        keep, row = [[] for _ in range(P)], 0
        for i, h in enumerate(history):
            node, up = new[P + i], parents[i]
            kept = [0] if node else []
            while kept:
                t = chosen[row + kept[-1]]
                h.append(t)
                child = [x for x in range(len(node)) if up[x] == kept[-1] and node[x] == t]
                if not child:
                    break
                kept.append(child[0])
            keep.append(kept)
            row += len(node)
        server.keep(keep)
        if window:
            server.free(first, window, sinks)
    server.free(first)
    mm.mm_check_device_error()
    return [h[b:b + tokens] for h, b in zip(history, begin)], rounds


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--answers", type=int, default=4)
    p.add_argument("--tokens", type=int, default=128)
    p.add_argument("--depth", type=int, default=4)
    p.add_argument("--temperature", type=float, default=0.3)
    p.add_argument("--window", type=int, default=0)
    p.add_argument("--accept", type=float, default=0.8)
    a = p.parse_args()
    model = Model(Shape())
    rng = np.random.default_rng(3)
    prompts = [rng.integers(0, model.shape.vocab, n).tolist() for n in (37, 5, 120)]
    out = None

    def draft(i, history):  # two branches, the second in case the first token of the first is wrong
        at = len(history) - len(prompts[i // a.answers])
        wrong = lambda t: (t + 1 + int(rng.integers(0, 99))) % model.shape.vocab
        first = [t if rng.random() < a.accept else wrong(t) for t in known[i][at:at + a.depth]]
        return [first, [wrong(t) for t in first[:1]] + known[i][at + 1:at + 2]] if first else []

    for depth in sorted({0, a.depth}):
        known = out
        server = Server(model, len(prompts) * (1 + a.answers), pages=1024)
        run = lambda n: generate(server, prompts, a.answers, n, a.temperature, depth=depth, window=a.window, sinks=4,
                                 draft=draft if known else None)
        run(4)
        torch.cuda.synchronize()
        t = time.perf_counter()
        out, rounds = run(a.tokens)
        t = time.perf_counter() - t
        print(f"depth {depth}: {len(out)} answers of {a.tokens} tokens in {sum(rounds) / len(rounds):.0f} rounds each, {t * 1e3:.0f} ms; "
              f"pages still held {int((server.refs > 0).sum())}; first answer {out[0][:8]} ...")


if __name__ == "__main__":
    main()
