"""kvq_sparse_attention_nvfp4 on the GPU against the attention over the
listed blocks in 64 bits, with the tolerance of tests/test_chunk_attention
(the arithmetic is the same)."""
import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.sparse_models import listed_tokens, masked_attention, rows_of
from tests.test_chunk_attention import KS, VS, Case
from tests.variant_build import build_variant

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tiles_library(tmp_path_factory):
    return build_variant(tmp_path_factory.mktemp("kvq_tiles"), {
        "sparse_attention.cu": {"KVQ_SPARSE_ITEMS_FROM": 0}})


@pytest.fixture(params=["regular", "tiles"], autouse=True)
def library(request, monkeypatch):
    """The regular library, whose small batches go by rows alone, and a build
    that always asks whether tiles pay."""
    if request.param == "tiles":
        monkeypatch.setattr(kvq, "LIB_PATH",
                            request.getfixturevalue("tiles_library"))
        monkeypatch.setattr(kvq, "_lib", None)
    yield


def lists(rng, cu, lens, total, sel, top, near=0.0):
    """Rising lists of blocks that each row sees; near: how much of their
    choice the rows share."""
    out = np.full((total, top), -1, dtype=np.int32)
    common = {}
    for r, (b, seen) in enumerate(rows_of(cu, lens, total)):
        nb = -(-seen // sel)
        if b < 0 or nb == 0:
            continue
        base = common.setdefault(b, rng.standard_normal(100000))[:nb]
        x = near * base + (1 - near) * rng.standard_normal(nb)
        take = np.sort(np.argsort(-x)[:min(top, nb)])
        out[r, :take.size] = take
    return out


class Sparse(Case):
    def __init__(self, q_lens, lens, sel=32, top=4, near=0.5, **kw):
        super().__init__(q_lens, lens, **kw)
        self.sel = sel
        self.selected = lists(self.rng, self.cu, self.lens, self.q.shape[0],
                              sel, top, near)

    def call(self, out=None, **kw):
        flags = kw.pop("flags", 0)
        kvq.kvq_sparse_attention_nvfp4(
            self.qd, self.kc, self.vc, self.bt, self.cud, self.lend,
            torch.from_numpy(self.selected).cuda(), self.sel, self.ks,
            self.vs, self.scale, self.out if out is None else out,
            kw.pop("max_q", self.max_q),
            flags=flags | (kvq.KVQ_F_SWIZZLE_K_SCALE if self.swz else 0),
            dev_error=self.err, **kw)

    def ref(self, lens=None):
        return masked_attention(
            self.pages, self.q.double().numpy(), self.table, self.cu,
            self.lens if lens is None else lens, KS, VS, self.scale,
            listed_tokens(self.selected, self.sel))


def test_smallest():
    c = Sparse([1], [1], top=1)
    c.check(c.run())


@pytest.mark.parametrize("L", [1, 2, 15, 16, 31, 32, 33, 63, 64, 65, 127, 128,
                               129, 500, 900])
@pytest.mark.parametrize("q", [1, 5])
def test_lengths(L, q):
    c = Sparse([min(q, L)], [L], seed=L)
    c.check(c.run())


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (7, 1), (8, 1), (16, 1),
                                    (4, 2), (24, 8), (10, 2), (32, 4),
                                    (8, 8), (26, 2)])
@pytest.mark.parametrize("q", [1, 20])
def test_heads(hq, hkv, q):
    c = Sparse([q, 3], [333, 150], hq=hq, hkv=hkv, seed=hq)
    c.check(c.run())


@pytest.mark.parametrize("block,sel", [(4, 4), (4, 16), (8, 8), (8, 24),
                                       (12, 36), (16, 16), (16, 64),
                                       (16, 48), (20, 20), (32, 32),
                                       (64, 64), (64, 128), (128, 128),
                                       (128, 256)])
@pytest.mark.parametrize("nhd", [False, True])
@pytest.mark.parametrize("swz", [False, True])
def test_layouts(block, sel, nhd, swz):
    c = Sparse([1, 9], [700, 411], hq=8, hkv=2, block=block, sel=sel, nhd=nhd,
               swz=swz, f16=nhd, top=3, seed=block + sel)
    c.check(c.run())


@pytest.mark.parametrize("top", [1, 2, 7, 31, 32, 33, 70])
def test_list_lengths(top):
    c = Sparse([6, 1], [1300, 900], sel=16, top=top, hq=8, hkv=2, seed=top)
    c.check(c.run())


@pytest.mark.parametrize("q_lens,lens", [
    ([0, 1, 0], [5, 9, 700]), ([7, 0, 3], [7, 0, 500]), ([1] * 30,
                                                         list(range(1, 900,
                                                                    30))),
    ([5, 3], [3, 2]), ([2, 2], [0, 1]), ([70, 1, 9], [400, 1000, 9]),
    ([1, 2, 3, 4, 5, 6, 7, 8, 9, 40], [99] * 10)])
def test_ragged(q_lens, lens):
    c = Sparse(q_lens, lens, hq=8, hkv=2, seed=len(lens), pad_rows=3)
    c.check(c.run())


@pytest.mark.parametrize("near", [0.0, 0.7, 1.0])
@pytest.mark.parametrize("G", [1, 4, 8, 16])
def test_many_rows(near, G):
    c = Sparse([150], [1500], sel=32, top=9, near=near, hq=2 * G, hkv=2,
               seed=G)
    c.check(c.run())


@pytest.mark.parametrize("sel", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (3, 1), (10, 2), (16, 1)])
def test_block_lengths_with_many_rows(sel, hq, hkv):
    """Tokens that share their blocks: tiles of several blocks, and blocks of
    several tiles; heads that do not divide a tile's rows."""
    c = Sparse([90, 1, 200], [90 + 5 * sel + 3, 700, 200 + 9 * sel], sel=sel,
               top=7, near=0.8, hq=hq, hkv=hkv, seed=sel + hq)
    c.check(c.run())


def test_tiles_and_rows_in_one_batch():
    """One sequence whose rows agree, one whose rows do not, single tokens."""
    c = Sparse([64, 64, 1, 1], [3000, 3000, 2000, 40], sel=16, top=12, hq=8,
               hkv=1, near=1.0)
    other = lists(c.rng, c.cu, c.lens, 130, 16, 12, 0.0)
    c.selected[64:128] = other[64:128]
    c.check(c.run())


def test_tiles_bad_pages_and_nan():
    """Bad pages and NaN scales under tiles: what a row does not see cannot
    reach it, what it sees does."""
    c = Sparse([64], [64 + 600], sel=32, top=8, hq=8, hkv=1, near=1.0)
    c.table[0, 5] = -1
    used = np.unique(c.selected[c.selected >= 0])
    c.selected[:32, 0] = 2 if 2 < c.selected[:32, 1].min() else c.selected[
        :32, 0]
    bits = kvq.KVQ_DEVERR_BLOCK if 2 in c.selected else 0
    e = int(used[len(used) // 2])
    plain = c.ref()
    for t in (32 * e + 3, 32 * e + 31):
        c.pages.set_scale(1, c.table[0, t // 16], t % 16, 0, 6, 0x7F)
    got = c.run(bits=bits)
    has = (c.selected == e).any(1)
    seen = np.array([600 + i + 1 for i in range(64)])
    has &= seen > 32 * e + 3
    assert np.isnan(got[has][:, :, 96:112]).all()
    assert np.isfinite(got[has][:, :, :96]).all()
    assert np.isfinite(got[~has]).all()
    got[has] = plain[0][has]
    c.check(got, plain)


def test_tiles_and_rows_in_many_rounds():
    """Rows that no tile takes, in several rounds, beside rows of tiles."""
    c = Sparse([600, 100, 33], [640, 700, 600], sel=16, top=2, hq=16, hkv=1,
               near=0.0)
    wide = np.full((733, 128), -1, dtype=np.int32)
    wide[:, :2] = c.selected
    wide[600:700, :30] = lists(c.rng, c.cu, c.lens, 733, 16, 30, 1.0)[600:700]
    c.selected = wide
    c.check(c.run())


def test_tiles_of_the_regular_library():
    """Enough for tiles to be asked for: 300 rows of 2304 tokens, 4 heads."""
    c = Sparse([300, 1, 2], [6000, 500, 9], sel=64, top=36, near=0.9, hq=8,
               hkv=4)
    c.check(c.run())


def test_long_context_shared_by_many_ctas():
    c = Sparse([40], [30000], sel=64, top=200, near=0.9, hq=8, hkv=1)
    c.check(c.run())


def test_every_block_is_the_chunk_attention():
    c = Sparse([40, 1], [700, 333], sel=32, top=22, hq=8, hkv=2)
    got = c.run()
    want = Case.ref(c)
    c.check(got, want)


def test_empty_lists():
    c = Sparse([3, 2], [300, 200], hq=4, hkv=2)
    c.selected[0] = -1
    c.selected[3] = -1
    c.check(c.run())
    c.selected[:] = -1
    c.check(c.run())


def test_holes_in_lists():
    c = Sparse([4], [600], top=8, hq=4, hkv=2)
    c.selected[0] = [-1, 2, -5, 3, -1, -1, 7, -1]
    c.selected[1] = [-1] * 7 + [0]
    c.selected[2, 0] = -(1 << 31)
    c.check(c.run())


@pytest.mark.parametrize("entry", [
    [3, 3, 5, -1], [5, 3, 6, 6], [2, 1000, 4, -1], [0, 1, (1 << 31) - 1, 2],
    [7, 6, 5, 4], [4, -1, 4, 9]])
@pytest.mark.parametrize("q", [1, 20])
def test_entries_that_do_not_rise_or_see_nothing(entry, q):
    c = Sparse([q], [32 * 11], top=4, hq=4, hkv=2)
    c.selected[0] = entry
    c.check(c.run(bits=kvq.KVQ_DEVERR_SEQ))


def test_block_behind_the_row():
    """The last rows' block, listed by rows that end before it."""
    c = Sparse([40], [64 + 40], sel=16, top=7, hq=4, hkv=1)
    c.selected[:] = np.arange(7)
    c.check(c.run(bits=kvq.KVQ_DEVERR_SEQ))


@pytest.mark.parametrize("q", [2, 20])
def test_bad_pages(q):
    c = Sparse([q, q], [400, 300], sel=32, top=6, hq=8, hkv=2)
    c.selected[:, :6] = [0, 1, 2, 3, 4, 5]
    c.table[0, 3] = -1
    c.table[0, 5] = 1 << 29
    c.table[1, 0] = c.pages.nb
    c.table[1, 1] = -1           # (both pages of its first block)
    c.check(c.run(bits=kvq.KVQ_DEVERR_BLOCK))


@pytest.mark.parametrize("q", [1, 20])
def test_unlisted_and_hidden_tokens_reach_nothing(q):
    """NaN scales in blocks that are not listed and behind the rows."""
    c = Sparse([q], [32 * 9 + 20], sel=32, top=3, hq=4, hkv=1)
    c.selected[:] = [1, 4, 7]
    for e in (0, 2, 3, 5, 6, 8):
        for t in range(32 * e, min(32 * e + 32, 308)):
            for side in range(2):
                for g in range(8):
                    c.pages.set_scale(side, c.table[0, t // 16], t % 16, 0, g,
                                      0x7F)
    c.check(c.run())


def test_nan_scales_that_a_row_sees():
    c = Sparse([1, 1], [300, 300], sel=32, top=3, hq=4, hkv=1)
    c.selected[:] = [1, 4, 7]
    c.pages.set_scale(1, c.table[0, 2], 3, 0, 5, 0x7F)   # token 35, V
    c.pages.set_scale(0, c.table[1, 9], 1, 0, 2, 0x7F)   # token 145, K
    got = c.run()
    assert np.isnan(got[0, :, 80:96]).all()
    assert np.isfinite(got[0, :, :80]).all()
    assert np.isnan(got[1]).all()


def test_long_context_and_offsets():
    c = Sparse([2, 1], [20000, 300], sel=64, top=5, hq=2, hkv=1, block=16)
    c.check(c.run())


def test_strides():
    c = Sparse([4, 9], [300, 200], hq=8, hkv=2).upload()
    big = torch.zeros(13, 3, 8, 128, dtype=c.dt, device="cuda")
    big[:, 1] = c.qd
    c.qd = big[:, 1]
    out = torch.full((13, 2, 8, 128), 77.0, dtype=c.dt, device="cuda")
    wide = torch.full((13, 9), 5, dtype=torch.int32, device="cuda")
    wide[:, 2:6] = torch.from_numpy(c.selected).cuda()
    kvq.kvq_sparse_attention_nvfp4(
        c.qd, c.kc, c.vc, c.bt, c.cud, c.lend, wide[:, 2:6], c.sel, c.ks,
        c.vs, c.scale, out[:, 1], c.max_q, dev_error=c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    c.check(out[:, 1].double().cpu().numpy())
    assert (out[:, 0] == 77.0).all()


@pytest.mark.parametrize("max_q", [0, 1, 3, 500])
def test_any_max_q(max_q):
    c = Sparse([20, 1, 4], [500, 300, 64], hq=8, hkv=2)
    c.check(c.run(max_q=max_q))


def test_context_lens_too_long():
    c = Sparse([2], [300], top=3, hq=4, hkv=2)
    c.check(c.run(bits=kvq.KVQ_DEVERR_SEQ, max_context_len=256),
            c.ref(lens=[256]))


@pytest.mark.parametrize("first", [-3, -40, -2 ** 31])
def test_first_offset_below_zero(first):
    """Taken as 0, and flagged."""
    c = Sparse([70, 40], [900, 300], hq=8, hkv=1, top=9, near=0.9)
    cu, c.cu = c.cu, c.cu.copy()
    c.cu[0] = first
    got = c.run(bits=kvq.KVQ_DEVERR_SEQ)
    c.cu = cu
    c.check(got)


def test_last_offset_behind_the_rows():
    c = Sparse([70, 40], [900, 300], hq=8, hkv=1, top=9, near=0.9)
    cu, c.cu = c.cu, c.cu.copy()
    c.cu[2] = 2 ** 31 - 1
    got = c.run(bits=kvq.KVQ_DEVERR_SEQ)
    c.cu = cu
    c.check(got)


def test_negative_and_zero_scale():
    for scale in (-0.2, 0.0):
        c = Sparse([2, 20], [300, 500], hq=8, hkv=2, scale=scale)
        c.check(c.run())


def test_dominating_token():
    c = Sparse([30], [900], sel=32, top=20, hq=8, hkv=1, q_mul=6.0)
    c.check(c.run())


def test_many_rounds_of_rows():
    """More rows than one round takes (64 heads over 2048 tokens), each of
    few tokens."""
    c = Sparse([700], [740], sel=16, top=2, hq=16, hkv=1)
    wide = np.full((700, 128), -1, dtype=np.int32)
    wide[:, :2] = c.selected
    c.selected = wide
    c.check(c.run())


def test_repeats_to_the_bit():
    c = Sparse([40, 1, 9], [900, 700, 77], hq=16, hkv=2, top=9)
    a = c.run()
    assert all((c.run() == a).all() for _ in range(3))


@pytest.mark.parametrize("seed", range(24))
def test_random(seed):
    rng = np.random.default_rng(300 + seed)
    n = int(rng.integers(1, 6))
    lens = rng.integers(0, 1100, n)
    q_lens = [int(rng.integers(0, min(L, 60) + 1)) for L in lens]
    block = int(rng.choice([4, 8, 12, 16, 32, 64]))
    hkv = int(rng.choice([1, 2, 3]))
    c = Sparse(q_lens, lens, hq=hkv * int(rng.choice([1, 2, 5, 8, 16])),
               hkv=hkv, block=block, sel=block * int(rng.choice([1, 2, 3])),
               top=int(rng.integers(1, 20)), near=float(rng.random()),
               nhd=bool(rng.random() < 0.5), swz=bool(rng.random() < 0.5),
               f16=bool(rng.random() < 0.5), seed=seed,
               pad_rows=int(seed % 3))
    if c.q.shape[0]:
        c.check(c.run())
