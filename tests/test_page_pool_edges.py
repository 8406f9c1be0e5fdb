"""The page pool's calls at their edges: calls from two host threads, pages
that nobody holds, lists without entries, entries that need no page, table
entries that are no pages."""
import threading

import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.page_models import DEV_BLOCK, DEV_FULL, DEV_REF, Pool
from tests.test_page_pool import Gpu, dev

pytestmark = pytest.mark.gpu


def test_two_threads_with_pools_of_different_sizes():
    """Two host threads, each with a pool, a stream and a list of its own,
    whose kernels need different amounts of shared memory: no call of one is
    refused because of the other's.  (Calls of the C entries, made as fast as
    the threads can.)"""
    start, refused, states = threading.Barrier(2), [], {}

    def loop(name, rows, calls=20000):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            ref, table, lens = kvq.alloc_page_pool(8, rows, 1)
            err, ids, cu = dev([0]), dev([rows - 1, 0]), dev([0, 3, 5])
            slots = torch.zeros(5, dtype=torch.int64, device="cuda")
            stream.synchronize()
            state = (ref.data_ptr(), 8, table.data_ptr(), 1, rows, 1,
                     lens.data_ptr())
            extend = state + (4, ids.data_ptr(), cu.data_ptr(), 2,
                              slots.data_ptr(), 5, 0, err.data_ptr(),
                              stream.cuda_stream)
            free = state + (ids.data_ptr(), 2, 0, err.data_ptr(),
                            stream.cuda_stream)
            L = kvq.lib()
            start.wait()
            for _ in range(calls):
                codes = (L.kvq_extend_sequences(*extend),
                         L.kvq_free_sequences(*free))
                if codes != (0, 0):
                    refused.append((name, codes))
                    break
            stream.synchronize()
            states[name] = (int(err.item()), int(ref.abs().sum().item()),
                            slots.tolist())

    threads = [threading.Thread(target=loop, args=a)
               for a in (("small", 170000), ("large", 1 << 18))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert refused == []
    for state in states.values():
        assert state == (0, 0, [0, 1, 2, 4, 5])


class HeldPool(Pool):
    """The rule of forks that the base model does not have: a parent with a
    page that nobody holds (count 0 or less) is refused."""

    def fork(self, parents, children):
        R, W = self.table.shape
        left, bits = [], 0
        for i, (p, c) in enumerate(zip(parents, children)):
            bad = False
            if (0 <= p < R and 0 <= c < R and list(children).count(c) == 1
                    and self.lens[c] == 0 and not (W and self.table[c, 0] >= 0)
                    and 0 <= self.lens[p] <= W * self.B):
                L = int(self.lens[p])
                used = self.table[p, :self._pages_for(L)]
                if L % self.B == 0 or self._page(used[-1]):
                    bad = any(self._page(x) and self.ref[x] <= 0
                              for x in used)
            if bad:
                bits |= DEV_REF
            else:
                left.append(i)
        src = np.full(len(parents), -1, dtype=np.int32)
        dst = np.full(len(parents), -1, dtype=np.int32)
        src[left], dst[left], more = super().fork(
            [parents[i] for i in left], [children[i] for i in left])
        return src, dst, bits | more


def test_fork_of_pages_that_nobody_holds():
    m = HeldPool(12, 9, 4, 4)
    g = Gpu(m)
    g.extend([0, 1, 2], [10, 8, 6])           # pages 0..2, 3..4, 5..6
    m.ref[1] = 0                              # a full page of row 0
    g.load()
    a, b, bits = g.fork([0, 1, 2], [3, 4, 5])
    assert bits == DEV_REF and a.tolist() == [-1, -1, 6]
    assert b.tolist() == [-1, -1, 1]          # the free page, not shared
    assert m.lens[3] == 0 and m.lens[4] == 8
    m.ref[6] = 0                              # the partly filled one of row 2
    g.load()
    assert g.fork([2], [6])[2] == DEV_REF
    m.ref[6] = -3
    g.load()
    assert g.fork([2, 1], [6, 7])[2] == DEV_REF
    m.ref[6], m.table[2, 0] = 1, 77           # beside a page that is none
    g.load()
    assert g.fork([2], [6])[2] == DEV_BLOCK


@pytest.mark.parametrize("seed", range(4))
def test_fork_with_counts_at_random(seed):
    """Long rows (the checks of a call are spread over the cluster), counts
    taken away at random, entries that need pages and that do not, pools
    that run out: equal calls give equal states."""
    rng = np.random.default_rng(seed)
    rows, width = 120, 400
    m = HeldPool(20000, rows, width, 4)
    g = Gpu(m)
    g.extend(list(range(40)), rng.integers(0, 4 * width, 40).tolist())
    held = np.nonzero(m.ref)[0]
    m.ref[rng.choice(held, int(rng.integers(1, 30)))] = rng.integers(-1, 1)
    named = np.isin(np.arange(m.nb), m.table)
    free = np.nonzero((m.ref == 0) & ~named)[0]
    left = int(rng.integers(0, 40))
    m.ref[free[left:]] = 7                    # others hold the rest
    before = (m.ref.copy(), m.table.copy(), m.lens.copy())
    parents = rng.integers(0, 40, 60).tolist()
    kids = (40 + rng.permutation(80)[:60]).tolist()
    for _ in range(5):
        m.ref, m.table, m.lens = (x.copy() for x in before)
        g.load()
        bits = g.fork(parents, kids)[2]
        assert bits & DEV_REF


def test_lists_without_entries_write_their_outputs():
    """No entry, but room for slots: all of them -1, on the stream given."""
    ref, table, lens = kvq.alloc_page_pool(8, 3, 4)
    none, cu = dev([]), dev([0])
    side = torch.cuda.Stream()
    for stream in (None, side):
        out = [torch.full((9,), 5, dtype=torch.int64, device="cuda")
               for _ in range(3)]
        torch.cuda.synchronize()
        handle = None if stream is None else stream.cuda_stream
        kvq.kvq_extend_sequences(ref, table, lens, none, cu, out[0], 4,
                                 stream=handle)
        kvq.kvq_compact_sequences(ref, table, lens, none, dev([0] * 9), cu,
                                  out[1], out[2], 4, stream=handle)
        torch.cuda.synchronize()
        for x in out:
            assert x.tolist() == [-1] * 9
    assert not bool(ref.any()) and bool((table == -1).all())


def test_lists_without_entries_in_a_graph():
    ref, table, lens = kvq.alloc_page_pool(8, 3, 4)
    none, cu = dev([]), dev([0])
    slots = torch.zeros(6, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_extend_sequences(ref, table, lens, none, cu, slots, 4)
    assert slots.tolist() == [0] * 6
    graph.replay()
    assert slots.tolist() == [-1] * 6


def test_entries_that_need_no_page_are_served_by_a_full_pool():
    g = Gpu(Pool(4, 6, 4, 4))
    g.extend([0, 1], [6, 5])
    # the pool is empty: two entries need a page, the others have room
    _, bits = g.extend([2, 0, 3, 1], [1, 2, 9, 3])
    assert bits == DEV_FULL
    assert g.m.lens[:4].tolist() == [8, 8, 0, 0]
    _, _, bits = g.fork([0, 1], [4, 5])       # full pages only: shared
    assert bits == 0 and g.m.lens[4:].tolist() == [8, 8]


def test_negative_entries_are_no_pages():
    """Whatever the negative value: not dropped, not flagged, left."""
    m = Pool(8, 4, 5, 4)
    m.table[0] = [3, -5, 1, -1, -7]
    m.ref[[1, 3]] = 1
    m.lens[0] = 10
    g = Gpu(m)
    assert g.compact([0], [[]])[2] == 0
    assert m.table[0].tolist() == [-1, -5, -1, -1, -7]
    m.table[1] = [-9, 2, -1, -1, -1]
    m.ref[2] = 1
    g.load()
    assert g.free([0, 1]) == 0
    assert m.table[1, 0] == -9 and (m.ref == 0).all()
    assert g.extend([1], [5])[1] == 0         # the row is an empty one
