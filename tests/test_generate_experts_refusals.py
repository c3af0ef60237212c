"""Numbers of experts that the serving example refuses before it makes a model (no GPU needed)."""
import sys

import pytest

from dense_packed_bit_gb300 import generate as gen


@pytest.mark.parametrize("experts", [1, -2, 1025])
def test_models(experts):
    with pytest.raises(ValueError, match="experts"):
        gen.Model(gen.Shape(experts=experts), device="cpu")


def test_the_command(monkeypatch):
    monkeypatch.setattr(sys, "argv", ["generate", "--experts", "1"])
    with pytest.raises(ValueError, match="at least that many"):
        gen.main()


def test_picks():
    with pytest.raises(ValueError, match="experts"):
        gen.Model(gen.Shape(experts=4, top_k=5), device="cpu")
    with pytest.raises(ValueError, match="experts"):
        gen.Model(gen.Shape(experts=4, top_k=0), device="cpu")
