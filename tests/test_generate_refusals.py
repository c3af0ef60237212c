"""What the serving example refuses on the host, before anything of it reaches the GPU (no GPU needed)."""
from types import SimpleNamespace

import pytest

from dense_packed_bit_gb300.generate import Server, Shape, generate

SHAPE = Shape(vocab=1003, positions=64)


class Untouched:
    """A server whose steps may not be reached."""

    seqs, model = 9, SimpleNamespace(shape=SHAPE)

    def __getattr__(self, name):
        raise AssertionError(f"the server's {name} was used")


PROMPTS = [[1, 2, 3], list(range(40))]


def test_answers_past_the_last_position():
    # 40 tokens of prompt, 21 of answer, 4 drafted behind the last but one: positions 0 .. 63 hold 40 + 21 - 2 + 4 = 63
    with pytest.raises(ValueError, match="positions"):
        generate(Untouched(), PROMPTS, 2, 22, depth=4)
    with pytest.raises(ValueError, match="positions"):
        generate(Untouched(), PROMPTS, 2, 26, depth=0)
    for tokens, depth in ((21, 4), (25, 0)):
        with pytest.raises(AssertionError, match="was used"):
            generate(Untouched(), PROMPTS, 2, tokens, depth=depth)
    with pytest.raises(AssertionError, match="was used"):
        generate(Untouched(), [[7] * 64], 1, 1, depth=4)  # nothing but the prompt is processed


def test_a_step_past_the_last_position():
    model = SimpleNamespace(shape=SHAPE)
    for places in ([[63, 64], []], [[-1], [0]]):
        new = [[5] * len(p) for p in places]
        with pytest.raises(ValueError, match="position"):
            Server.step(SimpleNamespace(model=model), new, places)


def test_tokens_that_the_model_does_not_have():
    for bad in (-1, SHAPE.vocab):
        with pytest.raises(ValueError, match="vocabulary"):
            Server.step(SimpleNamespace(model=SimpleNamespace(shape=SHAPE)), [[1, bad], []], [[0, 1], []])


def test_prompts_without_a_token():
    for prompts in ([], [[1], []]):
        with pytest.raises(ValueError, match="prompt"):
            generate(Untouched(), prompts, 2, 4)


def test_drafts_longer_than_the_window():
    # a drafted token sees all its ancestors, a decoded one only the window's
    with pytest.raises(ValueError, match="window"):
        generate(Untouched(), PROMPTS, 2, 4, depth=8, window=8)
    with pytest.raises(ValueError, match="window"):
        Server.step(SimpleNamespace(model=SimpleNamespace(shape=SHAPE)), [[1] * 5], [[0, 1, 2, 3, 4]], 4, 0,
                    [[list(range(i + 1)) for i in range(5)]])
    for depth, window in ((7, 8), (0, 1), (8, 0)):
        with pytest.raises(AssertionError, match="was used"):
            generate(Untouched(), PROMPTS, 2, 4, depth=depth, window=window)
