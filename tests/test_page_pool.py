"""The page pool on the GPU (extend, fork, compact, free), whole pages and
single tokens moved, against the plain models: every result is a whole
number or a byte and has to be equal."""
import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.page_models import Pages, Pool, copy_pages, move_tokens

pytestmark = pytest.mark.gpu


def dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


class Gpu:
    """The pool's state on the GPU beside its model."""

    def __init__(self, model, flags=0):
        self.m, self.flags = model, flags
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.load()

    def load(self):
        self.ref, self.table = dev(self.m.ref), dev(self.m.table)
        self.lens = dev(self.m.lens)

    def bits(self):
        v = int(self.err.item())
        self.err.zero_()
        return v

    def same(self, what=""):
        for name in ("ref", "table", "lens"):
            got = getattr(self, name).cpu().numpy()
            assert np.array_equal(got, getattr(self.m, name)), (what, name)

    def extend(self, ids, new, total=None, cu=None):
        cu = [0] + np.cumsum(new).tolist() if cu is None else cu
        total = cu[-1] if total is None else total
        slots = torch.full((total,), -7, dtype=torch.int64, device="cuda")
        kvq.kvq_extend_sequences(self.ref, self.table, self.lens, dev(ids),
                                 dev(cu), slots, self.m.B, flags=self.flags,
                                 dev_error=self.err)
        want, bits = self.m.extend(ids, cu, total)
        assert np.array_equal(slots.cpu().numpy(), want)
        assert self.bits() == bits
        self.same("extend")
        return want, bits

    def fork(self, parents, children):
        n = len(parents)
        src, dst = dev([-7] * n), dev([-7] * n)
        kvq.kvq_fork_sequences(self.ref, self.table, self.lens, dev(parents),
                               dev(children), src, dst, self.m.B,
                               flags=self.flags, dev_error=self.err)
        a, b, bits = self.m.fork(parents, children)
        assert np.array_equal(src.cpu().numpy(), a)
        assert np.array_equal(dst.cpu().numpy(), b)
        assert self.bits() == bits
        self.same("fork")
        return a, b, bits

    def compact(self, ids, lists, total=None, cu=None):
        keep = [x for k in lists for x in k]
        cu = [0] + np.cumsum([len(k) for k in lists]).tolist() \
            if cu is None else cu
        total = len(keep) if total is None else total
        keep = (keep + [0] * total)[:total]
        src = torch.full((total,), -7, dtype=torch.int64, device="cuda")
        dst = torch.full((total,), -7, dtype=torch.int64, device="cuda")
        kvq.kvq_compact_sequences(self.ref, self.table, self.lens, dev(ids),
                                  dev(keep), dev(cu), src, dst, self.m.B,
                                  flags=self.flags, dev_error=self.err)
        a, b, bits = self.m.compact(ids, keep, cu, total)
        assert np.array_equal(src.cpu().numpy(), a)
        assert np.array_equal(dst.cpu().numpy(), b)
        assert self.bits() == bits
        self.same("compact")
        return a, b, bits

    def free(self, ids):
        kvq.kvq_free_sequences(self.ref, self.table, self.lens, dev(ids),
                               flags=self.flags, dev_error=self.err)
        bits = self.m.free(ids)
        assert self.bits() == bits
        self.same("free")
        return bits


@pytest.mark.parametrize("block,nb", [(1, 50), (4, 4097), (16, 4096),
                                      (12, 40000), (64, 3)])
def test_extend_sizes(block, nb):
    g = Gpu(Pool(nb, 7, 40, block))
    g.extend([3], [0])
    g.extend([3], [1])
    g.extend([3, 0, 6], [1, block, 2 * block - 1])
    g.extend([0, 1, 2], [0, 3, 0], total=9)      # slots behind the last
    g.extend([], [])
    g.free([3, 1])
    g.extend([1, 3, 4, 5], [block + 1, 5, 0, 40 * block])


def test_extend_one_by_one_and_long():
    g = Gpu(Pool(9000, 3, 8200, 16))
    for _ in range(40):
        g.extend([2, 0], [1, 1])
    g.extend([1], [8190 * 16 + 3])
    g.extend([1], [20])
    g.extend([1], [200])                          # past the row: refused


def test_extend_many_tokens():
    """Slots enough for the second kernel: refused entries, empty ones,
    tokens behind the last, an order of offsets that is refused whole."""
    m = Pool(6000, 40, 700, 16)
    g = Gpu(m)
    rng = np.random.default_rng(3)
    g.extend(rng.permutation(40)[:30].tolist(),
             rng.integers(0, 50, 30).tolist())
    new = rng.integers(0, 2000, 20).tolist()
    new[3], new[7], new[19] = 0, 11500, 0
    g.extend(rng.permutation(40)[:20].tolist(), new, total=sum(new) + 77)
    g.extend([1, 2, 1, 3], [9000, 5000, 3000, 7000])
    g.extend([4, 5], None, total=20000, cu=[0, 15000, 14000])
    g.extend([4, 5], None, total=20000, cu=[5, 15000, 20000])
    g.extend([0, 4, 5], [0, 0, 0], total=17000)
    g.free(list(range(40)))
    g.extend([6, 7, 8], [11200, 11200, 11200])
    g.extend(list(range(30)), [3000] * 30)         # the pool runs out


def test_extend_refusals():
    m = Pool(20, 6, 4, 8)
    g = Gpu(m)
    assert g.extend([0, 0, 1], [3, 4, 5])[1] == 4         # named twice
    assert g.extend([6, -1, 2], [1, 1, 1])[1] == 4        # no such row
    assert g.extend([3], [33])[1] == 4                    # longer than a row
    assert g.extend([3], None, total=4, cu=[0, 5])[1] == 4    # beyond total
    assert g.extend([3], None, total=4, cu=[1, 3])[1] == 4
    assert g.extend([3, 4], None, total=4, cu=[0, 3, 2])[1] == 4
    m.lens[4] = 40
    m.lens[5] = -1
    g.load()
    assert g.extend([4, 5, 3], [1, 1, 1])[1] == 4
    m.lens[4], m.table[4, 1] = 10, 20                     # not a page
    m.lens[5] = 0
    g.load()
    assert g.extend([4], [1])[1] == 2
    assert g.extend([4], [0])[1] == 0
    m.table[4, 0:2] = [18, 19]
    m.ref[[18, 19]] = 2                                   # shared last page
    g.load()
    assert g.extend([4], [1])[1] == 16
    assert g.extend([4], [0])[1] == 0


def test_extend_full_pool():
    g = Gpu(Pool(10, 8, 12, 4))
    _, bits = g.extend([0, 1, 2, 3, 4], [12, 20, 12, 0, 1])
    assert bits == 32                       # 3 + 5 fit, 3 do not, 1 neither
    assert g.m.lens.tolist() == [12, 20, 0, 0, 0, 0, 0, 0]
    g.free([0])
    g.extend([4, 5], [20, 1])               # exactly the free pages, one over
    assert g.m.lens[4] == 20 and g.m.lens[5] == 0
    g.extend([5], [1])


def test_fork_shares_and_copies():
    g = Gpu(Pool(64, 12, 9, 4))
    g.extend([0, 1, 2], [13, 16, 3])
    a, b, bits = g.fork([0, 0, 1, 2, 5], [3, 4, 6, 7, 8])
    assert bits == 0 and (a >= 0).sum() == 3
    g.fork([3, 7], [9, 10])                 # a fork of a fork
    g.extend([3, 0, 6], [1, 9, 1])
    g.free([0, 0, 1, 3])
    g.free([4, 6, 7, 8, 9, 10, 2])
    assert (g.m.ref == 0).all() and (g.m.table == -1).all()


def test_fork_refusals():
    m = Pool(8, 8, 4, 4)
    g = Gpu(m)
    g.extend([0, 1], [6, 8])
    assert g.fork([0, 0], [2, 2])[2] == 4           # child twice
    assert g.fork([0, 8, -1], [1, 2, 3])[2] == 4    # not empty; no such row
    assert g.fork([0], [0])[2] == 4
    assert g.fork([0], [-1])[2] == 4
    g.fork([5], [5])                                # an empty row is a copy
    m.lens[5] = 5                                   # of itself; no page there
    g.load()
    assert g.fork([5], [6])[2] == 2
    m.lens[5] = 99
    g.load()
    assert g.fork([5], [6])[2] == 4
    m.lens[5], m.table[5, 0] = 4, 77                # a full page that is none
    g.load()
    assert g.fork([5], [6])[2] == 2
    m.table[5, 0], m.lens[5] = -1, 0
    g.load()
    # four pages left: the fifth copy of a partly filled page has none
    assert g.fork([0, 1, 0, 0, 0], [2, 3, 4, 5, 7])[2] == 0
    g.free([2])
    assert g.fork([0, 0, 1], [2, 6, 2])[2] == 4
    g.extend([6], [1])


def test_compact_and_drop():
    g = Gpu(Pool(64, 6, 10, 4))
    g.extend([0, 1, 2, 3], [17, 23, 4, 40])
    g.compact([1, 0, 2, 3], [[0, 1, 5, 22], [16], [],
                             list(range(0, 40, 3))], total=40)
    g.compact([1], [[0, 1, 2, 3]])          # everything stays
    g.compact([3], [list(range(9))])        # a cut
    g.free([0, 1, 2, 3])
    assert (g.m.ref == 0).all()


def test_compact_refusals_and_shared_pages():
    m = Pool(64, 8, 6, 4)
    g = Gpu(m)
    g.extend([0, 1], [14, 20])
    g.fork([0], [2])
    # the shared prefix may stay, and tokens may leave shared pages, but not
    # move into them
    assert g.compact([2], [[0, 1, 2, 3, 5]])[2] == 16
    assert g.compact([2], [[1]])[2] == 16
    assert g.compact([2], [list(range(12)) + [13]])[2] == 0
    assert g.compact([0], [list(range(8))])[2] == 0
    for lists in ([[3, 3]], [[4, 2]], [[-1]], [[20]], [[0, 1, 25]]):
        assert g.compact([1], lists)[2] == 4
    assert g.compact([1, 1], [[1], [2]])[2] == 4
    assert g.compact([1, 8], [[0, 1, 2], [0]])[2] == 4
    assert g.compact([1], [[0, 1]], total=2, cu=[0, 3])[2] == 4
    assert g.compact([1], [[0, 1]], total=2, cu=[1, 2])[2] == 4
    m.table[1, 0] = 64
    g.load()
    assert g.compact([1], [[0, 1]])[2] == 2
    m.table[1, 0] = -1
    g.load()
    assert g.compact([1], [[2]])[2] == 2
    m.lens[3] = 25
    g.load()
    assert g.compact([3], [[0]])[2] == 4
    assert g.compact([3], [[]])[2] == 4


def test_free_odd_states():
    m = Pool(8, 4, 5, 4)
    m.table[0] = [3, 9, -1, 2, 3]           # a hole, no page, a page twice
    m.ref[[2, 3]] = [0, 2]
    m.lens[0] = 18
    g = Gpu(m)
    assert g.free([0, 0, 4, -1, 1]) == 2 | 4 | 16
    assert (m.ref == 0).all()


@pytest.mark.parametrize("flags", [0, kvq.KVQ_F_PDL], ids=["plain", "pdl"])
@pytest.mark.parametrize("seed", range(6))
def test_random_histories(seed, flags):
    rng = np.random.default_rng(seed)
    block = int(rng.choice([1, 2, 4, 16, 20]))
    rows, width = int(rng.integers(1, 80)), int(rng.integers(1, 30))
    g = Gpu(Pool(int(rng.integers(1, 700)), rows, width, block), flags)
    for _ in range(25):
        n = int(rng.integers(1, rows + 1))
        ids = rng.permutation(rows)[:n].tolist()
        if rng.random() < 0.15:
            ids[0] = int(rng.integers(-2, rows + 2))
        op = rng.choice(["extend", "extend", "fork", "compact", "free"])
        if op == "extend":
            new = rng.integers(0, width * block // 2 + 2, n).tolist()
            g.extend(ids, new, total=sum(new) + int(rng.integers(0, 5)))
        elif op == "fork":
            par = rng.integers(0, rows, n).tolist()
            g.fork(par, ids)
        elif op == "compact":
            lists = []
            for s in ids:
                L = int(g.m.lens[s]) if 0 <= s < rows else 3
                keep = np.nonzero(rng.random(max(L, 0)) < rng.random())[0]
                lists.append(keep.tolist())
            g.compact(ids, lists, total=sum(map(len, lists)) + 3)
        else:
            g.free(ids[:max(1, n // 3)])
    g.free(list(range(rows)))
    assert (g.m.ref == 0).all() and (g.m.table == -1).all()


def test_wide_lists():
    """The longest list, and a table whose rows lie apart."""
    m = Pool(70000, 5000, 3, 4)
    g = Gpu(m)
    wide = torch.full((5000, 8), 5, dtype=torch.int32, device="cuda")
    wide[:, :3] = -1
    g.table = wide[:, :3]
    rng = np.random.default_rng(0)
    ids = rng.permutation(5000)[:4096].tolist()
    g.extend(ids, rng.integers(0, 9, 4096).tolist())
    kids = sorted(set(range(5000)) - set(ids))
    g.fork(ids[:len(kids)], kids)
    assert bool((wide[:, 3:] == 5).all())
    with pytest.raises(kvq.KvqError):
        g.extend(list(range(4097)), [1] * 4097)


# ---------------------------------------------------------------------------
# pages and tokens moved
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("page", [16, 48, 576, 18432, 4096 + 32, 32 * 129])
@pytest.mark.parametrize("stacked", [True, False])
def test_copy_pages(page, stacked):
    rng = np.random.default_rng(page)
    nb, layers = 23, 3
    data = rng.integers(0, 256, (layers, nb, page), dtype=np.uint8)
    perm = rng.permutation(nb)
    src = perm[:9].astype(np.int32)
    dst = perm[9:18].astype(np.int32)
    src[3], dst[5], src[7] = -1, -4, dst[7]
    src[1], dst[2] = nb, 1 << 30
    t = dev(data, torch.uint8)
    if not stacked:
        t = list(t.unbind(0))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kvq_copy_pages(t, dev(src), dev(dst), dev_error=err)
    got = (t if stacked else torch.stack(t)).cpu().numpy()
    for c in range(layers):
        want, bits = copy_pages(data[c], src, dst)
        assert np.array_equal(got[c], want)
    assert int(err.item()) == bits == 2


def test_copy_pages_strides_and_many_caches():
    """300 caches (three launches), pages apart and 16-byte aligned only."""
    rng = np.random.default_rng(1)
    big = rng.integers(0, 256, (300, 5, 112), dtype=np.uint8)
    t = dev(big, torch.uint8)
    view = t[:, :, 16:96]
    kvq.kvq_copy_pages(list(view.unbind(0)), dev([4, 0]), dev([1, 3]))
    want = big.copy()
    want[:, 1, 16:96] = big[:, 4, 16:96]
    want[:, 3, 16:96] = big[:, 0, 16:96]
    assert np.array_equal(t.cpu().numpy(), want)


def test_copy_pages_far_apart():
    """Pages more than 2^32 bytes into a cache."""
    t = torch.empty(300, 1 << 24, dtype=torch.uint8, device="cuda")
    t[299] = 7
    t[298, :16] = 3
    kvq.kvq_copy_pages([t], dev([299, 298]), dev([270, 0]))
    assert bool((t[270] == 7).all()) and bool((t[0, :16] == 3).all())


@pytest.mark.parametrize("nhd", [False, True], ids=["HND", "NHD"])
@pytest.mark.parametrize("swz", [False, True])
@pytest.mark.parametrize("block,heads,D", [(16, 2, 128), (4, 1, 128),
                                           (12, 3, 64), (32, 5, 192),
                                           (8, 1, 2048)])
def test_move_tokens(nhd, swz, block, heads, D):
    rng = np.random.default_rng(block)
    layers, nb = 2, 40
    models = [Pages(nb, block, heads, D, nhd, swz) for _ in range(layers)]
    for m in models:
        m.data[:] = rng.integers(0, 256, m.data.shape)
    shape = (block, heads) if nhd else (heads, block)
    t = dev(np.stack([m.data for m in models]), torch.uint8).view(
        layers, nb, 2, *shape, D // 2 + D // 16)
    # two compactions in place (pages in random order), an odd list between
    perm = rng.permutation(nb)
    src, dst, cu = [], [], [0]
    for first, count, p in ((0, 15, 0.5), (15, 15, 0.9)):
        table = perm[first:first + count]
        keep = np.nonzero(rng.random(count * block) < p)[0]
        src += (table[keep // block] * block + keep % block).tolist()
        j = np.arange(len(keep))
        dst += (table[j // block] * block + j % block).tolist()
        cu.append(len(src))
        if first == 0:
            src += [-1, 3 * block, nb * block, int(perm[31]) * block + 1]
            dst += [5, -2, int(perm[30]) * block, int(perm[30]) * block + 2]
            cu.append(len(src))
    src += [1, 2]
    dst += [int(perm[33]) * block, 9]                   # behind the lists
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kvq_move_tokens_nvfp4(
        t, dev(src, torch.int64), dev(dst, torch.int64), dev(cu),
        layout=kvq.KVQ_LAYOUT_NHD if nhd else kvq.KVQ_LAYOUT_HND,
        flags=kvq.KVQ_F_SWIZZLE_K_SCALE if swz else 0, dev_error=err)
    got = t.cpu().numpy().reshape(layers, nb, 2, -1)
    for m, x in zip(models, got):
        want, bits = move_tokens(m, src[:cu[-1]], dst[:cu[-1]])
        assert np.array_equal(x, want)
    assert int(err.item()) == bits == 1


@pytest.mark.parametrize("nhd", [False, True], ids=["HND", "NHD"])
@pytest.mark.parametrize("swz", [False, True])
@pytest.mark.parametrize("heads,D", [(2, 128), (3, 64), (5, 128), (1, 64)])
def test_move_tokens_many_lists(nhd, swz, heads, D):
    """More thread blocks than run at once: heads go in pairs, the last one
    alone where their number is odd.  Every list compacts four pages of its
    own in place, of none to all of their tokens."""
    rng = np.random.default_rng(heads)
    block, lists, layers = 8, 300, 2
    nb = 4 * lists
    models = [Pages(nb, block, heads, D, nhd, swz) for _ in range(layers)]
    for m in models:
        m.data[:] = rng.integers(0, 256, m.data.shape)
    shape = (block, heads) if nhd else (heads, block)
    t = [dev(m.data, torch.uint8).view(nb, 2, *shape, D // 2 + D // 16)
         for m in models]
    perm = rng.permutation(nb)
    src, dst, cu = [], [], [0]
    for i in range(lists):
        table = perm[4 * i:4 * i + 4]
        keep = np.nonzero(rng.random(4 * block) < (i % 5) / 4)[0]
        j = np.arange(len(keep))
        src += (table[keep // block] * block + keep % block).tolist()
        dst += (table[j // block] * block + j % block).tolist()
        cu.append(len(src))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kvq_move_tokens_nvfp4(
        t, dev(src, torch.int64), dev(dst, torch.int64), dev(cu),
        layout=kvq.KVQ_LAYOUT_NHD if nhd else kvq.KVQ_LAYOUT_HND,
        flags=kvq.KVQ_F_SWIZZLE_K_SCALE if swz else 0, dev_error=err)
    for m, x in zip(models, t):
        want, bits = move_tokens(m, src, dst)
        assert np.array_equal(x.cpu().numpy().reshape(want.shape), want)
    assert int(err.item()) == 0


def test_move_tokens_bad_lists():
    m = Pages(6, 4, 1).fill(np.random.default_rng(0))
    t = dev(m.data, torch.uint8).view(6, 2, 1, 4, 72)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for cu in ([3, 1], [-1, 2], [0, 9]):
        kvq.kvq_move_tokens_nvfp4([t], dev([1, 2, 3], torch.int64),
                                  dev([9, 10, 11], torch.int64), dev(cu),
                                  dev_error=err)
        assert int(err.item()) == 4
        err.zero_()
    assert np.array_equal(t.cpu().numpy().reshape(m.data.shape), m.data)


def test_pool_in_a_graph():
    """free -> extend -> fork -> copy captured and replayed."""
    m = Pool(64, 6, 8, 4)
    g = Gpu(m)
    ids, kids = dev([0, 1]), dev([2, 3])
    cu = dev([0, 7, 13])
    slots = torch.zeros(13, dtype=torch.int64, device="cuda")
    src, dst = dev([0, 0]), dev([0, 0])
    cache = torch.randint(0, 256, (2, 64, 576), dtype=torch.uint8,
                          device="cuda")

    def step():
        kvq.kvq_free_sequences(g.ref, g.table, g.lens, dev_ids)
        kvq.kvq_extend_sequences(g.ref, g.table, g.lens, ids, cu, slots, 4)
        kvq.kvq_fork_sequences(g.ref, g.table, g.lens, ids, kids, src, dst,
                               4)
        kvq.kvq_copy_pages(cache, src, dst)

    dev_ids = dev([0, 1, 2, 3])
    step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (g.ref, g.table, g.lens, slots, src, dst)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (g.ref, g.table, g.lens, slots, src, dst)):
        assert torch.equal(a, b)
    assert torch.equal(cache[:, dst.long()], cache[:, src.long()])
