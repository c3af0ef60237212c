"""The generate command's mixture of experts: the layer against fp64 with the router's own picks, and answers with it."""
import numpy as np
import pytest
import torch

import dense_packed_bit_gb300 as mm
from dense_packed_bit_gb300 import generate as gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


def dense(w):
    codes, scales, _ = (None if t is None else t.cpu() for t in w.tensors)
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double() - 8
    return code * scales.double().repeat_interleave(w.group, -1)[..., :w.cols]


@pytest.mark.parametrize("tokens", [1, 5, 77, 700])
def test_layer(tokens):
    shape = gen.Shape(experts=6, heads=4, expert_hidden=96)
    layer = gen.Experts(3, shape, "cuda")
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn(tokens, shape.width, generator=g).cuda()
    h = torch.nn.functional.layer_norm(x, (shape.width,)).half()
    out = layer(x, h)
    mm.mm_check_device_error()
    hd, up, down = h.double().cpu(), dense(layer.up), dense(layer.down)
    logits = hd @ layer.router.double().cpu().T
    best = logits.topk(2, 1)
    third = logits.sort(1, descending=True).values[:, 2]
    clear = best.values[:, 1] - third > 1e-4  # the picks cannot depend on the rounding of fp32 logits
    w = torch.softmax(best.values, 1)
    ref, tol = x.double().cpu(), torch.zeros(tokens, shape.width, dtype=torch.float64)
    for e in range(shape.experts):
        t, j = (best.indices == e).nonzero(as_tuple=True)
        z, m = hd[t] @ up[e].T, hd[t].abs() @ up[e].abs().T
        gate, lift = z[:, ::2], z[:, 1::2]
        hidden = gate * torch.sigmoid(gate) * lift
        # the hidden value's error: 1e-5 of the products' terms through silu (slope 1.1) and the product, its rounding to fp16
        off = 1.1e-5 * m[:, ::2] * lift.abs() + 1e-5 * m[:, 1::2] * gate.abs() + hidden.abs() * (2.0 ** -11 + 2.0 ** -21) + 2.0 ** -25
        c = w[t, j][:, None]
        ref = ref.index_add(0, t, c * (hidden @ down[e].T))
        # weights within 2e-4: softmax of logits off by 1e-5 of their terms (256 of about 0.05)
        tol = tol.index_add(0, t, c * (1.01 * off @ down[e].abs().T + (1e-5 + 3e-4) * (hidden.abs() @ down[e].abs().T)))
    err = (out.double().cpu() - ref).abs()
    assert bool((err <= tol + 2.0 ** -22 * (ref.abs() + x.abs().double().cpu()))[clear].all())
    assert int(clear.sum()) >= 0.9 * tokens


def test_answers():
    model = gen.Model(gen.Shape(vocab=700, layers=2, heads=4, kv_heads=2, positions=256, experts=8, expert_hidden=128))
    prompts = [np.random.default_rng(1).integers(0, 700, n).tolist() for n in (30, 3)]
    for depth in (0, 3):
        server = gen.Server(model, 6, pages=80)
        out, rounds = gen.generate(server, prompts, 2, 12, depth=depth)
        assert [len(o) for o in out] == [12] * 4 and all(0 <= t < 700 for o in out for t in o)
        assert int((server.refs > 0).sum()) == 0 and all(0 < r <= 12 for r in rounds)
