"""Page bookkeeping of a paged cache on the GPU against a model of it in plain Python: reserve, append,
compact, fork, free and copy, one after another in random order, the whole state compared after each call.
Everything here is whole numbers and copies: equality is exact.
"""
import numpy as np
import pytest
import torch

import dense_packed_bit_gb300 as mm
from cache_util import DT, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


def ints(a):
    return torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")


class Model:
    """The cache on the host: k, v as int16 bit patterns [layers][pages][kv][page][dim]."""

    def __init__(self, seed, seqs, pages, max_pages, kv, page, dim, layers, dtype="f16", tokens_first=False):
        rng = np.random.default_rng(seed)
        self.rng, self.page = rng, page
        shape = (layers, pages, kv, page, dim)
        self.k, self.v = (rng.integers(-30000, 30000, shape).astype(np.int16) for _ in range(2))
        self.table = np.full((seqs, max_pages), -1, dtype=np.int32)
        self.lens = np.zeros(seqs, dtype=np.int32)
        self.refs = np.zeros(pages, dtype=np.int32)

        def dev(a):
            t = torch.from_numpy(a.copy()).cuda().view(DT[dtype])
            return t.transpose(2, 3).contiguous().transpose(2, 3) if tokens_first else t

        self.c = mm.mm_cache(dev(self.k), dev(self.v), torch.from_numpy(self.table.copy()).cuda(),
                             torch.from_numpy(self.lens.copy()).cuda(), torch.from_numpy(self.refs.copy()).cuda())

    def check(self, what=""):
        torch.cuda.synchronize()
        mm.mm_check_device_error()
        k, v, table, lens, refs = self.c.tensors
        for name, t, a in (("table", table, self.table), ("lens", lens, self.lens), ("refs", refs, self.refs),
                           ("k", k.contiguous().view(torch.int16), self.k), ("v", v.contiguous().view(torch.int16), self.v)):
            assert np.array_equal(t.cpu().numpy(), a), f"{what}: {name} differs"
        held = np.bincount(self.table[self.table >= 0], minlength=len(self.refs))
        assert np.array_equal(held, self.refs), f"{what}: the model itself lost a reference"

    def free_pages(self, n):
        free = np.flatnonzero(self.refs == 0)
        return (None, n - len(free)) if len(free) < n else (free[:n], 0)

    def reserve(self, need):
        missing = torch.full((1,), -5, dtype=torch.int32, device="cuda")
        mm.mm_cache_reserve(self.c, ints(need), missing)
        want = [(s, j) for s in range(len(self.lens))
                for j in range(self.lens[s] // self.page, -(-(self.lens[s] + need[s]) // self.page)) if self.table[s, j] < 0]
        pages, lacking = self.free_pages(len(want))
        assert missing.item() == lacking
        if lacking == 0:
            for (s, j), p in zip(want, pages):
                self.table[s, j] = p
                self.refs[p] = 1
        self.check(f"reserve {need}")
        return lacking

    def append(self, layer, counts):
        n = int(sum(counts))
        new = [self.rng.integers(-30000, 30000, (n,) + (self.k.shape[2], self.k.shape[4])).astype(np.int16) for _ in range(2)]
        pad = 8  # rows wider than they need to be
        dev = []
        for a in new:
            w = torch.zeros((n, a.shape[1] * a.shape[2] + pad), dtype=torch.int16, device="cuda")
            w[:, :-pad] = torch.from_numpy(a.reshape(n, -1))
            dev.append(w)
        mm.mm_cache_append(self.c, layer, dev[0], dev[1], dev[0].stride(0), ints(starts(counts)), n, int(max(counts)))
        st = starts(counts)
        for s, c in enumerate(counts):
            for i in range(c):
                t = self.lens[s] + i
                for pool, a in ((self.k, new[0]), (self.v, new[1])):
                    pool[layer, self.table[s, t // self.page], :, t % self.page] = a[st[s] + i]
        self.check(f"append {counts}")

    def compact(self, counts, keep):
        """keep: per sequence the kept indices, or None for the first len ones given as numbers"""
        n, st = int(sum(counts)), starts(counts)
        kept = [len(x) for x in keep]
        flat = np.full(n, -9, dtype=np.int32)
        for s, x in enumerate(keep):
            flat[st[s]:st[s] + len(x)] = x
        mm.mm_cache_compact(self.c, ints(st), ints(flat), ints(kept), n, int(max(counts)))
        for s, x in enumerate(keep):
            for i, f in enumerate(x):
                a, b = self.lens[s] + f, self.lens[s] + i
                for pool in (self.k, self.v):
                    pool[:, self.table[s, b // self.page], :, b % self.page] = \
                        pool[:, self.table[s, a // self.page], :, a % self.page]
            self.lens[s] += len(x)
            self.drop(s, lambda j, s=s: j >= -(-self.lens[s] // self.page))
        self.check(f"compact {counts} {keep}")

    def drop(self, s, which):
        for j in range(self.table.shape[1]):
            if self.table[s, j] >= 0 and which(j):
                self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1

    def free(self, seqs, window=0, sinks=0):
        mm.mm_cache_free(self.c, ints(seqs), len(seqs), window, sinks)
        for s in seqs:
            if window:
                self.drop(s, lambda j: j * self.page >= sinks and (j + 1) * self.page - 1 <= self.lens[s] - window)
            else:
                self.drop(s, lambda j: True)
                self.lens[s] = 0
        self.check(f"free {seqs} {window} {sinks}")

    def fork(self, parents, children):
        missing = torch.full((1,), -5, dtype=torch.int32, device="cuda")
        mm.mm_cache_fork(self.c, ints(parents), ints(children), len(parents), missing)
        part = [self.lens[p] % self.page for p in parents]
        pages, lacking = self.free_pages(sum(x > 0 for x in part))
        assert missing.item() == lacking
        if lacking == 0:
            pages = list(pages)
            for p, ch, x in zip(parents, children, part):
                full = self.lens[p] // self.page
                self.table[ch] = -1
                self.table[ch, :full] = self.table[p, :full]
                for q in self.table[p, :full]:
                    if q >= 0:
                        self.refs[q] += 1
                if x:
                    new, old = pages.pop(0), self.table[p, full]
                    self.table[ch, full] = new
                    self.refs[new] = 1
                    for pool in (self.k, self.v):
                        pool[:, new, :, :x] = pool[:, old, :, :x]
                self.lens[ch] = self.lens[p]
        self.check(f"fork {parents} {children}")
        return lacking


SHAPES = [dict(kv=2, page=16, dim=64, layers=1), dict(kv=1, page=32, dim=80, layers=3),
          dict(kv=5, page=16, dim=8, layers=2, dtype="bf16"), dict(kv=3, page=64, dim=128, layers=2, tokens_first=True),
          dict(kv=2, page=128, dim=24, layers=1)]


@pytest.mark.parametrize("shape", SHAPES, ids=[f"{s['kv']}x{s['dim']}page{s['page']}" for s in SHAPES])
def test_random_calls(shape):
    m = Model(1, seqs=8, pages=90, max_pages=12, **shape)
    rng, page = np.random.default_rng(7), shape["page"]
    for step in range(14):
        room = 12 * page - m.lens
        counts = [int(min(rng.integers(0, 40), r)) if rng.random() < 0.8 else 0 for r in room]
        if sum(counts) == 0:
            counts[0] = 1 if room[0] else 0
        if sum(counts) and m.reserve(counts) == 0:
            for layer in range(shape["layers"]):
                m.append(layer, counts)
            keep = [sorted(rng.choice(c, size=int(rng.integers(0, c + 1)), replace=False).tolist()) if c else [] for c in counts]
            m.compact(counts, keep)
        if step % 3 == 1:
            m.free([5, 6])
            m.fork([int(rng.integers(0, 3)), 0], [5, 6])
        if step % 4 == 2:
            m.free([int(rng.integers(0, 8))], window=int(rng.integers(1, 60)), sinks=int(rng.integers(0, 40)))
        if step % 5 == 4:
            m.free([int(rng.integers(0, 8))])


def test_compact_without_a_list_keeps_the_first():
    m = Model(2, seqs=3, pages=20, max_pages=5, kv=1, page=16, dim=64, layers=1)
    counts = [20, 0, 33]
    m.reserve(counts)
    m.append(0, counts)
    qs = ints(starts(counts))
    mm.mm_cache_compact(m.c, qs, None, ints([7, 0, 33]), 53, 33)
    for s, n in ((0, 7), (2, 33)):
        m.lens[s] += n
        m.drop(s, lambda j, s=s: j >= -(-m.lens[s] // 16))
    m.check("kept 7, 0, 33")
    more = [1, 2, 0]
    m.reserve(more)
    m.append(0, more)
    mm.mm_cache_compact(m.c, ints(starts(more)), None, None, 3, 2)
    m.lens += np.array(more, dtype=np.int32)
    m.check("kept all")


def test_everything_lacking_changes_nothing():
    m = Model(3, seqs=4, pages=5, max_pages=8, kv=1, page=16, dim=64, layers=1)
    assert m.reserve([30, 0, 17, 0]) == 0
    m.append(0, [30, 0, 17, 0])
    m.compact([30, 0, 17, 0], [list(range(30)), [], list(range(17)), []])
    assert m.reserve([20, 16, 0, 0]) == 2
    assert m.fork([0, 2], [1, 3]) == 1
    assert m.fork([0], [1]) == 0


def test_many_pages_in_one_call():
    # more pages than one sweep hands out, over a pool whose free pages are scattered
    m = Model(4, seqs=30, pages=20000, max_pages=700, kv=1, page=16, dim=8, layers=1)
    m.refs[::3] = 1
    m.c.tensors[4].copy_(torch.from_numpy(m.refs))
    missing = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = [16 * 300 + s for s in range(30)]
    mm.mm_cache_reserve(m.c, ints(need), missing)
    assert missing.item() == 0
    free = np.flatnonzero(m.refs == 0)
    at = 0
    for s in range(30):
        h = -(-need[s] // 16)
        m.table[s, :h] = free[at:at + h]
        at += h
    m.refs[free[:at]] = 1
    assert at > 8192
    torch.cuda.synchronize()
    mm.mm_check_device_error()
    assert np.array_equal(m.c.tensors[2].cpu().numpy(), m.table)
    assert np.array_equal(m.c.tensors[4].cpu().numpy(), m.refs)
    # and more than there are
    more = [16 * 250] * 30
    mm.mm_cache_reserve(m.c, ints([n + x for n, x in zip(need, more)]), missing)
    assert missing.item() == 30 * 250 - (free.size - at)
    assert np.array_equal(m.c.tensors[2].cpu().numpy(), m.table)


def test_copy_pages():
    m = Model(5, seqs=1, pages=12, max_pages=2, kv=3, page=32, dim=72, layers=2)
    src, dst = [0, 5, 0, 11], [1, 2, 3, 7]
    mm.mm_cache_copy_pages(m.c, ints(src), ints(dst), 4)
    for a, b in zip(src, dst):
        m.k[:, b], m.v[:, b] = m.k[:, a], m.v[:, a]
    m.check("copied")


def reported():
    torch.cuda.synchronize()
    with pytest.raises(mm.MMError) as e:
        mm.mm_check_device_error()
    assert e.value.status == mm.MM_ERR_INVALID_ARG and "out of range" in str(e.value)
    mm.mm_check_device_error()  # reported once


def test_out_of_range_values_are_skipped_and_reported():
    m = Model(6, seqs=4, pages=30, max_pages=4, kv=1, page=16, dim=64, layers=1)
    m.reserve([20, 40, 0, 0])
    m.append(0, [20, 40, 0, 0])
    m.compact([20, 40, 0, 0], [list(range(20)), list(range(40)), [], []])
    missing = torch.zeros(1, dtype=torch.int32, device="cuda")
    mm.mm_cache_free(m.c, ints([9, -1]), 2)
    reported()
    m.check("free of no sequence")
    mm.mm_cache_copy_pages(m.c, ints([0, 99]), ints([-4, 1]), 2)
    reported()
    m.check("copy of no page")
    mm.mm_cache_fork(m.c, ints([0, 0]), ints([7, 0]), 2, missing)
    reported()
    m.check("fork into no sequence and into itself")
    # a list that is not ascending: the token stays
    mm.mm_cache_reserve(m.c, ints([4, 0, 0, 0]), missing)
    mm.mm_cache_compact(m.c, ints([0, 4, 4, 4, 4]), ints([2, 1, 9, 9]), ints([2, 0, 0, 0]), 4, 4)
    reported()
    # row ranges that are no ranges
    kv = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    before = m.c.tensors[0].clone()
    mm.mm_cache_append(m.c, 0, kv, kv, 64, ints([0, 9, 3, 3, 3]), 4, 4)
    reported()
    # more tokens than the table's row holds
    mm.mm_cache_reserve(m.c, ints([0, 0, 100, 0]), missing)
    reported()
    assert torch.equal(before.view(torch.int16), m.c.tensors[0].view(torch.int16))


def test_refusals():
    m = Model(7, seqs=2, pages=4, max_pages=2, kv=1, page=16, dim=64, layers=1)
    k, v, table, lens, refs = m.c.tensors
    one = ints([0])
    bare = mm.mm_cache(k, v, table, lens)  # no reference counts
    calls = [lambda c: mm.mm_cache_reserve(c, ints([0, 0]), one), lambda c: mm.mm_cache_free(c, one, 1),
             lambda c: mm.mm_cache_fork(c, one, ints([1]), 1, one), lambda c: mm.mm_cache_compact(c, ints([0, 1, 1]), None, None, 1, 1)]
    for call in calls:
        with pytest.raises(mm.MMError) as e:
            call(bare)
        assert e.value.status == mm.MM_ERR_INVALID_ARG
    for bad in (dict(page_size=24), dict(page_size=256), dict(head_dim=12), dict(head_dim=136), dict(dtype=2), dict(pages=0),
                dict(token_stride=60), dict(token_stride=8), dict(seqs=0), dict(k=None), dict(table=None), dict(max_pages=0)):
        c = mm.mm_cache(k, v, table, lens, refs)
        for name, x in bad.items():
            setattr(c, name, x)
        with pytest.raises(mm.MMError) as e:
            mm.mm_cache_free(c, one, 1)
        assert e.value.status == mm.MM_ERR_INVALID_ARG, bad
    for call in (lambda: mm.mm_cache_free(m.c, one, 0), lambda: mm.mm_cache_free(m.c, None, 1), lambda: mm.mm_cache_free(m.c, one, 1, -1),
                 lambda: mm.mm_cache_fork(m.c, one, one, 0, one), lambda: mm.mm_cache_copy_pages(m.c, one, None, 1),
                 lambda: mm.mm_cache_append(m.c, 1, k, v, 64, ints([0, 1, 1]), 1, 1),
                 lambda: mm.mm_cache_append(m.c, 0, k, v, 64, ints([0, 1, 1]), 1, 1),
                 lambda: mm.mm_cache_compact(m.c, ints([0, 1, 1]), one, None, 1, 1),
                 lambda: mm.mm_cache_compact(m.c, ints([0, 1, 1]), None, None, 1, 2)):
        with pytest.raises(mm.MMError) as e:
            call()
        assert e.value.status == mm.MM_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        mm.mm_cache(k, v[:, :, :, :, :32], table, lens, refs)
    with pytest.raises(ValueError):
        mm.mm_cache(k, v, table.long(), lens, refs)
    m.check("after the refusals")
