"""Routing, ragged products by expert and the combination against their definitions, alone and as a layer."""
import numpy as np
import pytest
import torch

import dense_packed_bit_gb300 as mm
from packed4_util import DT, UNIT, check, make_weights, make_x, make_y, reference, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


def ints(*shape, fill=-9):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


def route(logits, top_k, score=mm.MM_ROUTE_SOFTMAX, renorm=False, scale=1.0):
    t, e = logits.shape
    need = mm.mm_experts_route_workspace(t, e, top_k)
    ws = torch.full((need + 4,), 0xEE, dtype=torch.uint8, device="cuda")
    ids, offsets, order, slots = ints(t + 1, top_k), ints(e + 2), ints(t * top_k + 1), ints(t + 1, top_k)
    weights = torch.full((t + 1, top_k), -9.0, device="cuda")
    mm.mm_experts_route(logits, t, e, logits.stride(0), top_k, score, renorm, scale, ids, weights, offsets, order, slots, ws, need)
    mm.mm_check_device_error()
    for out in (ids[t:], weights[t:], offsets[e + 1:], order[t * top_k:], slots[t:]):
        assert bool((out == -9).all())
    assert bool((ws[need:] == 0xEE).all())
    return [x.cpu().numpy() for x in (ids[:t], weights[:t], offsets[:e + 1], order[:t * top_k], slots[:t])]


def check_route(logits, top_k, score, renorm, scale=1.0):
    """Picks, order and slots exactly; weights within 1e-5 of themselves: an exponential of 2 ulp whose argument is off by
    half an ulp of up to 2^7 (a factor of 2^-17 = 7.6e-6 on its value; tests stay below |x| = 2^7), and a few roundings."""
    ids, weights, offsets, order, slots = route(logits, top_k, score, renorm, scale)
    x = logits.double().cpu().numpy()
    usable = x > -np.inf  # false for NaN
    ranked = np.argsort(np.where(usable, -x, np.inf), axis=1, kind="stable")[:, :top_k]
    picked = np.take_along_axis(usable, ranked, 1)
    want = np.where(picked, ranked, -1)
    assert np.array_equal(ids, want)
    flat = want.reshape(-1)
    listed = np.flatnonzero(flat >= 0)
    in_order = listed[np.argsort(flat[listed], kind="stable")]
    assert np.array_equal(offsets, np.concatenate([[0], np.cumsum(np.bincount(flat[listed], minlength=x.shape[1]))]))
    assert np.array_equal(order[:len(in_order)], in_order) and bool((order[len(in_order):] == -9).all())
    place = np.full(flat.shape, -1)
    place[in_order] = np.arange(len(in_order))
    assert np.array_equal(slots.reshape(-1), place)
    with np.errstate(all="ignore"):
        if score == mm.MM_ROUTE_SIGMOID:
            s = np.where(usable, 1 / (1 + np.exp(-np.where(usable, x, 0))), 0)
        else:
            s = np.where(usable, np.exp(x - np.where(usable, x, -np.inf).max(1, keepdims=True)), 0)
            s = s / s.sum(1, keepdims=True)
        w = np.where(picked, np.take_along_axis(s, ranked, 1), 0)
        if renorm:
            w = np.where(picked, w / w.sum(1, keepdims=True), 0)
    w = np.where(picked, w, 0) * scale
    assert np.all(np.abs(weights - w) <= 1e-5 * np.abs(w) + 1e-37), np.abs(weights - w).max()


MODES = [(mm.MM_ROUTE_SOFTMAX, False), (mm.MM_ROUTE_SOFTMAX, True), (mm.MM_ROUTE_SIGMOID, False), (mm.MM_ROUTE_SIGMOID, True)]


@pytest.mark.parametrize("tokens", [1, 2, 31, 128, 129, 1000, 5000])
@pytest.mark.parametrize("experts,top_k", [(1, 1), (2, 2), (8, 2), (33, 5), (64, 8), (100, 32), (128, 6), (256, 8), (257, 3), (1024, 20)])
def test_route(tokens, experts, top_k):
    g = torch.Generator().manual_seed(tokens + experts)
    mode = MODES[(tokens + experts) % 4]
    dtype = ("f32", "f16", "bf16")[(tokens + top_k) % 3]  # in 16 bits many logits are equal
    x = (torch.randn(tokens, experts + 3, generator=g) + torch.randn(experts + 3, generator=g)).to(DT[dtype]).cuda()
    check_route(x[:, :experts], top_k, *mode, scale=2.5)


@pytest.mark.parametrize("score,renorm", MODES)
def test_route_ties_and_rows_with_nothing(score, renorm):
    inf, nan = float("inf"), float("nan")
    rows = [[0.0, -0.0, 0.0, -0.0], [1, 1, 1, 1], [-inf, -inf, -inf, -inf], [nan, nan, nan, nan], [nan, 2, -inf, 2], [-inf, -3, -inf, -inf],
            [-100.0, -120.0, -101.0, -100.0], [100.0, 90.0, 100.0, -100.0], [-1e-30, 1e-30, 0.0, 0.0]]
    for repeat in (1, 40):
        check_route(torch.tensor(rows * repeat, device="cuda"), 3, score, renorm)


def test_route_all_tokens_to_one_expert():
    x = torch.zeros(3000, 50, device="cuda")
    x[:, 17] = 1
    check_route(x, 1, mm.MM_ROUTE_SOFTMAX, True)
    check_route(x, 2, mm.MM_ROUTE_SIGMOID, True)


def test_route_many_tokens():
    g = torch.Generator(device="cuda").manual_seed(1)
    check_route(torch.randn(300001, 9, generator=g, device="cuda"), 2, mm.MM_ROUTE_SOFTMAX, True)


def ragged(seed, counts, total=None):
    """Offsets of `counts` slots per expert and an order of shuffled tokens."""
    n = int(sum(counts))
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    return offsets, n, total or n


def experts(seed, counts, rows, cols, group, dtype, out, gather, swiglu=False, zeros=True, spare=3, per_row=2):
    e = len(counts)
    w, dense = make_weights(seed, e, rows, cols, group, dtype, zeros)
    offsets, n, _ = ragged(seed, counts)
    slots = n + spare
    g = torch.Generator().manual_seed(seed)
    columns = rows // 2 if swiglu else rows
    if gather:
        tokens = max(1, -(-n // per_row)) + 1
        x, xd = make_x(seed + 1, tokens, cols, dtype, bad=(tokens - 1,))  # no slot names the last row
        order = torch.full((slots,), (tokens - 1) * per_row, dtype=torch.int32)
        order[:n] = torch.randperm((tokens - 1) * per_row, generator=g)[:n].int()
        picked = xd[(order[:n] // per_row).long()]
        order, x_rows = order.cuda(), tokens
    else:
        x, xd = make_x(seed + 1, slots, cols, dtype, bad=range(n, slots))
        picked, order, x_rows, per_row = xd[:n], None, slots, 1
    y, buf = make_y(slots, columns, out)
    mm.mm_experts_gemm_packed4(w, x, x.stride(0), x_rows, order, per_row, offsets, slots,
                               mm.MM_ACT_SWIGLU if swiglu else mm.MM_ACT_NONE, y, y.stride(0))
    mm.mm_check_device_error()
    untouched(y, buf)
    assert bool((y[n:] == -7).all()), "rows behind the last slot were written"
    at = 0
    for i, c in enumerate(counts):
        if c:
            check(y[at:at + c], *reference(picked[at:at + c], dense[i], swiglu), out, f"expert {i} of {c}")
        at += c


COUNTS = {
    "one token": [0, 1, 0, 0, 1, 0, 0, 0],
    "all empty but the last": [0] * 7 + [1],
    "few": [1, 0, 3, 2, 0, 9, 1],
    "ragged": [17, 0, 1, 33, 8, 16, 70],
    "one has all": [0, 0, 200, 0],
    "one expert": [150],
    "larger": [300, 257, 1, 0, 256, 100],
    "fewer slots than experts": [0] * 60 + [1, 0, 2] + [0] * 40 + [1],
}


@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("gather", [True, False])
def test_experts(name, gather):
    counts = COUNTS[name]
    experts(1, counts, 100, 392, 64, "f16", "f32", gather)
    experts(2, counts, 130, 256, 128, "bf16", "bf16", gather, swiglu=True, zeros=False)
    experts(3, counts, 32, 200, 32, "f16", "f16", gather, swiglu=gather, per_row=1 if gather else 2)


@pytest.mark.parametrize("cols,group", [(64, 32), (128, 64), (120, 128), (192, 64), (24, 32)])
def test_short_rows_of_experts_of_many_lengths(cols, group):
    """Units of one to three stages: a warp that gathers X may be two units ahead of the other, whose rows must stay."""
    counts = [(17, 250, 33, 256, 90, 1, 128, 300)[i * 5 % 8] for i in range(40)]
    experts(4, counts, 2600, cols, group, "bf16", "f32", True)
    experts(5, counts, 700, cols, group, "f16", "f16", True, swiglu=True)


@pytest.mark.parametrize("rows,cols,group,dtype,out,swiglu", [
    (10722, 328, 64, "bf16", "f32", False), (10752, 64, 64, "f16", "f16", True), (10500, 192, 128, "bf16", "bf16", True),
    (21504, 136, 128, "f16", "f32", False)])
def test_many_rows_of_x_to_an_expert(rows, cols, group, dtype, out, swiglu):
    """Two pairs of CTAs that gather X for each other."""
    experts(6, [900, 3, 1201, 0], rows, cols, group, dtype, out, True, swiglu=swiglu)
    experts(7, [1100, 300, 200], rows, cols, group, dtype, out, True, swiglu=swiglu, zeros=False, per_row=1)


def test_experts_without_slots():
    w, _ = make_weights(1, 5, 30, 64, 32, "f16")
    y, buf = make_y(6, 30, "f32")
    x, _ = make_x(2, 6, 64, "f16")
    mm.mm_experts_gemm_packed4(w, x, x.stride(0), 6, None, 1, ints(6, fill=0), 6, mm.MM_ACT_NONE, y, y.stride(0))
    mm.mm_check_device_error()
    untouched(y, buf)
    assert bool((y == -7).all())


@pytest.mark.parametrize("slots", [6, 100])
def test_offsets_and_rows_out_of_range_are_reported(slots):
    w, dense = make_weights(1, 4, 30, 64, 32, "f16")
    x, xd = make_x(2, slots, 64, "f16", pad=0)
    for offsets, order in (([0, 2, 1, 5, 6], None), ([-1, 2, 3, 4, 5], None), ([0, 2, 3, 4, slots + 1], None),
                           ([0, 2, 3, 4, 5], [0, 1, 2 * slots, 3, 4]), ([0, 2, 3, 4, 5], [0, 1, -1, 3, 4])):
        y, buf = make_y(slots, 30, "f32")
        picks = None if order is None else torch.tensor(order + [0] * (slots - 5), dtype=torch.int32, device="cuda")
        mm.mm_experts_gemm_packed4(w, x, 64, slots, picks, 1 if order is None else 2, torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                                   slots, mm.MM_ACT_NONE, y, y.stride(0))
        with pytest.raises(mm.MMError) as e:
            mm.mm_check_device_error()
        assert e.value.status == mm.MM_ERR_INVALID_ARG
        mm.mm_check_device_error()
        untouched(y, buf)
        if order is not None:
            assert bool((y[2] == 0).all())
            check(y[:2], *reference(xd[[0, 0]], dense[0], False), "f32")


@pytest.mark.parametrize("y_dtype,out", [("f32", "f32"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("tokens,top_k,cols", [(1, 1, 1), (1, 8, 2048), (3, 2, 33), (50, 9, 260), (700, 4, 1000), (2, 20, 64)])
def test_combine(tokens, top_k, cols, y_dtype, out):
    g = torch.Generator().manual_seed(tokens + cols)
    n = tokens * top_k
    for pad, residual in ((0, "other"), (0, None), (8, "in place"), (1, "other")):
        wide = torch.full((n + 1, cols + pad), float("nan"), dtype=DT[y_dtype])
        wide[:n, :cols] = torch.randn(n, cols, generator=g).to(DT[y_dtype])
        slots = torch.randperm(n, generator=g).int().view(tokens, top_k)
        weights = torch.rand(tokens, top_k, generator=g)
        if n > 2:
            slots.view(-1)[1], weights.view(-1)[1] = -1, float("nan")
        r = torch.randn(tokens, cols, generator=g).to(DT[out])
        o, buf = make_y(tokens, cols, out, pad=pad)
        if residual == "in place":
            o.copy_(r)
        res = {"other": r.cuda(), None: None, "in place": o}[residual]
        y = wide.cuda()
        mm.mm_experts_combine(y, y.stride(0), n, slots.cuda(), weights.cuda(), tokens, top_k, cols, res, 0 if res is None else res.stride(0),
                              o, o.stride(0))
        mm.mm_check_device_error()
        untouched(o, buf)
        have = (slots >= 0)
        terms = wide[:, :cols].double()[slots.clamp(min=0).long()] * torch.where(have, weights, 0.0).double()[..., None]
        base = torch.zeros(tokens, cols, dtype=torch.float64) if res is None else r.double()
        ref, mass = base + terms.sum(1), base.abs() + terms.abs().sum(1)
        check(o, ref, top_k * 2.0 ** -24 * mass, out)  # one fp32 rounding a term


def test_combine_reports_slots_out_of_range():
    y = torch.ones(4, 64, device="cuda")
    out = torch.empty(2, 64, device="cuda")
    for bad in (4, -2):
        slots = torch.tensor([[0, bad], [1, 2]], dtype=torch.int32, device="cuda")
        mm.mm_experts_combine(y, 64, 4, slots, torch.ones(2, 2, device="cuda"), 2, 2, 64, None, 0, out, 64)
        with pytest.raises(mm.MMError):
            mm.mm_check_device_error()
        mm.mm_check_device_error()
        assert bool((out[0] == 1).all()) and bool((out[1] == 2).all())


def layer(logits, x, up, down, top_k, state):
    """A feed-forward step: route, up, down, combine.  `state`: the buffers."""
    t, e = logits.shape
    n = t * top_k
    mm.mm_experts_route(logits, t, e, e, top_k, mm.MM_ROUTE_SOFTMAX, True, 1.0, state["ids"], state["weights"], state["offsets"],
                        state["order"], state["slots"], state["ws"], state["ws"].numel())
    mm.mm_experts_gemm_packed4(up, x, x.stride(0), t, state["order"], top_k, state["offsets"], n, mm.MM_ACT_SWIGLU, state["h"], state["h"].stride(0))
    mm.mm_experts_gemm_packed4(down, state["h"], state["h"].stride(0), n, None, 1, state["offsets"], n, mm.MM_ACT_NONE, state["y"], state["y"].stride(0))
    mm.mm_experts_combine(state["y"], state["y"].stride(0), n, state["slots"], state["weights"], t, top_k, x.shape[1], x, x.stride(0),
                          state["out"], state["out"].stride(0))


@pytest.mark.parametrize("tokens,experts_,top_k,width,hidden", [(1, 8, 2, 256, 160), (7, 16, 4, 128, 64), (300, 8, 2, 256, 96), (1000, 32, 4, 128, 128)])
def test_layer(tokens, experts_, top_k, width, hidden):
    """The four together, eager and captured, on two states at once; against fp64 with the kernels' own picks and weights (which
    the tests above hold to theirs) and the hidden values rounded as they are."""
    up, up_d = make_weights(1, experts_, 2 * hidden, width, 64, "bf16", static=True)
    down, down_d = make_weights(2, experts_, width, hidden, 32, "bf16", static=True)
    torch.cuda.synchronize()
    n = tokens * top_k
    sides = []
    for i in range(2):
        g = torch.Generator().manual_seed(i)
        x, logits = torch.randn(tokens, width, generator=g).bfloat16().cuda(), torch.randn(tokens, experts_, generator=g).cuda()
        state = dict(ids=ints(tokens, top_k), weights=torch.empty(tokens, top_k, device="cuda"), offsets=ints(experts_ + 1), order=ints(n),
                     slots=ints(tokens, top_k), ws=torch.empty(mm.mm_experts_route_workspace(tokens, experts_, top_k), dtype=torch.uint8, device="cuda"),
                     h=torch.empty(n, hidden, dtype=torch.bfloat16, device="cuda"), y=torch.empty(n, width, device="cuda"),
                     out=torch.empty(tokens, width, dtype=torch.bfloat16, device="cuda"))
        sides.append((logits, x, state))

    def verify(logits, x, s):
        ids, weights, xd, hd = s["ids"].cpu().long(), s["weights"].double().cpu(), x.double().cpu(), s["h"].double().cpu()
        slots = s["slots"].cpu().long()
        assert torch.equal(ids, logits.cpu().sort(dim=1, descending=True, stable=True).indices[:, :top_k])
        ref, tol = xd.clone(), 2.0 ** -22 * xd.abs()
        for e in range(experts_):
            t, j = (ids == e).nonzero(as_tuple=True)
            if not len(t):
                continue
            check(s["h"][slots[t, j].cuda()], *reference(xd[t], up_d[e], True), "bf16", f"hidden of {e}")
            y, d = reference(hd[slots[t, j]], down_d[e], False)
            w = weights[t, j][:, None]
            ref.index_add_(0, t, w * y)
            tol.index_add_(0, t, w * d + (top_k + 2) * 2.0 ** -24 * (w * y).abs())
        check(s["out"], ref, tol, "bf16")

    streams = [torch.cuda.Stream() for _ in sides]
    for stream, (logits, x, s) in zip(streams, sides):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            for _ in range(3):
                layer(logits, x, up, down, top_k, s)
    torch.cuda.synchronize()
    for side in sides:
        verify(*side)
    graphs = []
    for logits, x, s in sides:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer(logits, x, up, down, top_k, s)
            layer(logits, x, up, down, top_k, s)
        graphs.append(graph)
    for i, (logits, x, s) in enumerate(sides):
        logits.copy_(torch.randn(tokens, experts_, generator=torch.Generator().manual_seed(50 + i)).cuda())
        s["out"].zero_()
    torch.cuda.synchronize()
    for graph, stream in zip(graphs, streams):
        with torch.cuda.stream(stream):
            graph.replay()
    torch.cuda.synchronize()
    mm.mm_check_device_error()
    for side in sides:
        verify(*side)


def test_unit_constants():
    for name, t in DT.items():
        assert UNIT[name] == torch.finfo(t).eps / 2
