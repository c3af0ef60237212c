"""The serving path as one: prompts, forked answers, drafted trees, sampling.  Every token that comes out is held against
the model written in fp64 over the tokens in front of it.

Tolerance: logits have unit size; f16 rounds about six quantities of a block (its inputs, queries, keys and values,
probabilities, the hidden layer) by 2^-11 of their size at most, 2^-11 / sqrt(3) on average, and the residual stream adds
them over two blocks: sqrt(12) 2^-11 / sqrt(3) = 1e-3 of a logit.  Six times that for the largest of many, for two logits
that are compared: 0.0085.  2^-5 leaves a factor of 3.7 for the layers' gains.
"""
import math

import numpy as np
import pytest
import torch
import torch.nn.functional as F

import dense_packed_bit_gb300 as mm
from dense_packed_bit_gb300 import synth
from dense_packed_bit_gb300.generate import Model, Server, Shape, generate, lookup

TOL = 2.0 ** -5
SMALL = Shape(vocab=1003, layers=2, heads=4, kv_heads=2, dim=64, hidden=512, positions=400)


def weights(p):
    fields = (p.codes.cpu().numpy()[:, :, None] >> np.array([0, 2, 4, 6])) & 3
    w = synth.CODEBOOK_TERNARY.astype(np.float64)[fields.reshape(p.rows, -1)[:, :p.cols]]
    scales = p.scales.cpu().numpy().view(np.float16).astype(np.float64)
    return torch.from_numpy(w * scales[:, None])


def reference(model, tokens, window=0, sinks=0):
    """fp64 logits of every position."""
    s, n = model.shape, len(tokens)
    d, kv = s.width, s.kv_heads * s.dim
    x = model.tokens.double().cpu()[tokens] + model.places.double().cpu()[:n]
    i, j = torch.arange(n)[:, None], torch.arange(n)[None, :]
    sees = (j <= i) & ((j > i - window) | (j < sinks) if window else True)
    for qkv, out, up, down in model.blocks:
        h = F.layer_norm(x, (d,)) @ weights(qkv).T
        q = h[:, :d].reshape(n, s.heads, s.dim)
        k, v = (h[:, a:a + kv].reshape(n, s.kv_heads, s.dim).repeat_interleave(s.heads // s.kv_heads, 1) for a in (d, d + kv))
        p = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(s.dim)
        p = p.masked_fill(~sees, -math.inf).softmax(-1)
        x = x + torch.einsum("hij,jhd->ihd", p, v).reshape(n, d) @ weights(out).T
        x = x + F.gelu(F.layer_norm(x, (d,)) @ weights(up).T, approximate="tanh") @ weights(down).T
    return F.layer_norm(x, (d,)) @ model.head.double().cpu().T / math.sqrt(d)


def check(model, prompt, answer, top_k, window=0, sinks=0):
    logits = reference(model, prompt + answer[:-1], window, sinks)[len(prompt) - 1:]
    kth = logits.topk(top_k, -1).values[:, -1]
    got = logits[torch.arange(len(answer)), torch.tensor(answer)]
    assert bool((got >= kth - TOL).all()), (kth - got).max()


def empty(server):
    assert int(server.refs.abs().sum()) == 0 and int((server.table + 1).abs().sum()) == 0 and int(server.lens.sum()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
@pytest.mark.parametrize("page", [16, 64])
def test_greedy_answers_with_and_without_drafts(page, window, sinks):
    model = Model(SMALL)
    rng = np.random.default_rng(5)
    prompts = [rng.integers(0, SMALL.vocab, n).tolist() for n in (1, 16, 50)]
    server = Server(model, 9, 200, page)
    plain, rounds = generate(server, prompts, 2, 20, temperature=0.0, depth=0, window=window, sinks=sinks)
    empty(server)
    assert rounds == [19] * 6 and plain[0] == plain[1]
    for i, a in enumerate(plain):
        check(model, prompts[i // 2], a, 1, window, sinks)

    def draft(i, history):  # a wrong branch, and one that is right for two tokens
        true = plain[i][len(history) - len(prompts[i // 2]):][:2]
        return [[(t + 1) % SMALL.vocab] * 3 for t in true[:1]] + [true + [0]]

    out, fewer = generate(server, prompts, 2, 20, temperature=0.0, depth=3, window=window, sinks=sinks, draft=draft)
    empty(server)
    assert sum(fewer) < sum(rounds)
    for i, a in enumerate(out):
        check(model, prompts[i // 2], a, 1, window, sinks)


@pytest.mark.gpu
def test_sampled_answers():
    model = Model(SMALL)
    prompts = [list(range(3, 40)), [7] * 9]
    server = Server(model, 8, 120)
    for depth in (0, 4):
        out, _ = generate(server, prompts, 3, 24, temperature=0.7, top_k=8, top_p=0.9, depth=depth)
        empty(server)
        assert out[0] != out[1]  # other uniform numbers
        for i, a in enumerate(out):
            check(model, prompts[i // 3], a, 8)


@pytest.mark.gpu
def test_too_few_pages():
    server = Server(Model(SMALL), 2, 3)
    with pytest.raises(RuntimeError, match="lacking"):
        generate(server, [list(range(60))], 1, 4)
    empty(server)
    mm.mm_check_device_error()


def test_lookup():
    assert lookup([1, 2, 3, 1, 2, 4, 1], 2) == [[2, 4]]
    assert lookup([1, 2, 3, 1, 5, 4, 1], 2) == [[5, 4], [2, 3]]
    assert lookup([1, 2, 3], 2) == [] and lookup([9], 4) == []
