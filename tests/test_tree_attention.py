"""kvq_tree_attention_nvfp4 on the GPU against the attention under the mask in
64 bits, with the tolerance of tests/test_chunk_attention (the arithmetic is
the same)."""
import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.sparse_models import masked_attention, tree_tokens
from tests.test_chunk_attention import KS, VS, Case

pytestmark = pytest.mark.gpu


def trees(rng, q_lens, rows, words):
    """Masks of random trees: each draft's ancestors and itself."""
    out = np.zeros((rows, words), dtype=np.int64)
    at = 0
    for n in q_lens:
        bits = []
        for i in range(n):
            up = int(rng.integers(-1, i))
            bits.append((bits[up] if up >= 0 else 0) | 1 << i)
            for w in range(words):
                out[at + i, w] = bits[i] >> (32 * w) & 0xFFFFFFFF
        at += n
    return out


class Tree(Case):
    def __init__(self, q_lens, lens, words=None, **kw):
        super().__init__(q_lens, lens, **kw)
        words = words or max(1, -(-self.max_q // 32))
        self.mask = trees(self.rng, q_lens, self.q.shape[0], words)

    def mask_dev(self):
        return torch.from_numpy(
            self.mask.astype(np.uint32).view(np.int32)).cuda()

    def call(self, out=None, **kw):
        flags = kw.pop("flags", 0)
        kvq.kvq_tree_attention_nvfp4(
            self.qd, self.kc, self.vc, self.bt, self.cud, self.lend,
            self.mask_dev(), self.ks, self.vs, self.scale,
            self.out if out is None else out, kw.pop("max_q", self.max_q),
            flags=flags | (kvq.KVQ_F_SWIZZLE_K_SCALE if self.swz else 0),
            dev_error=self.err, **kw)

    def ref(self, lens=None):
        return masked_attention(
            self.pages, self.q.double().numpy(), self.table, self.cu,
            self.lens if lens is None else lens, KS, VS, self.scale,
            tree_tokens(self.mask))


def test_smallest():
    c = Tree([1], [1])
    c.check(c.run())


@pytest.mark.parametrize("n", [1, 2, 7, 16, 31, 32, 33, 64, 65, 100])
@pytest.mark.parametrize("ctx", [0, 1, 63, 64, 100, 127, 128, 129, 300])
def test_sizes(n, ctx):
    c = Tree([n], [n + ctx], hq=4, hkv=1, seed=n + ctx)
    c.check(c.run())


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (7, 1), (8, 1), (16, 1),
                                    (4, 2), (24, 8), (10, 2), (8, 8)])
def test_heads(hq, hkv):
    c = Tree([20, 3, 1], [333, 150, 40], hq=hq, hkv=hkv, seed=hq)
    c.check(c.run())


@pytest.mark.parametrize("block", [4, 8, 12, 16, 32, 64, 128])
@pytest.mark.parametrize("nhd", [False, True])
@pytest.mark.parametrize("swz", [False, True])
def test_layouts(block, nhd, swz):
    c = Tree([9, 40], [411, 300], hq=8, hkv=2, block=block, nhd=nhd, swz=swz,
             f16=nhd, seed=block)
    c.check(c.run())


@pytest.mark.parametrize("q_lens,lens", [
    ([0, 1, 0], [5, 9, 700]), ([7, 0, 3], [7, 0, 500]),
    ([1] * 20, list(range(1, 600, 30))), ([5, 3], [3, 2]),
    ([2, 2], [0, 1]), ([70, 1, 9], [400, 1000, 9]), ([40], [33]),
    ([130, 2], [150, 300])])
def test_ragged(q_lens, lens):
    c = Tree(q_lens, lens, hq=8, hkv=2, seed=len(lens), pad_rows=3)
    c.check(c.run())


@pytest.mark.parametrize("n", [3, 12, 70])
def test_chain_is_the_chunk_attention(n):
    c = Tree([n, n], [n, 400], hq=8, hkv=2)
    for b in range(2):
        for i in range(n):
            for w in range(c.mask.shape[1]):
                c.mask[b * n + i, w] = (1 << i + 1) - 1 >> 32 * w & 0xFFFFFFFF
    c.check(c.run(), Case.ref(c))


def test_any_mask():
    """No tree at all: random bits, rows that see later drafts, and not
    themselves."""
    c = Tree([50, 20], [50, 333], hq=8, hkv=2)
    c.mask[:] = c.rng.integers(0, 1 << 32, c.mask.shape)
    c.check(c.run())


def test_empty_masks():
    c = Tree([9, 9], [9, 60], hq=8, hkv=2)
    c.mask[:] = 0
    c.mask[2] = 1 << 5
    c.check(c.run())


def test_bits_behind_the_last_draft():
    c = Tree([5, 33], [105, 400], words=4, hq=4, hkv=2)
    for r in range(38):
        n = 5 if r < 5 else 33
        for w in range(4):
            keep = max(min(n - 32 * w, 32), 0)
            c.mask[r, w] |= 0xFFFFFFFF >> keep << keep if keep < 32 else 0
    c.check(c.run())


def test_more_drafts_than_words():
    c = Tree([40], [200], words=1, hq=4, hkv=2)
    c.check(c.run(bits=kvq.KVQ_DEVERR_SEQ))


def test_masked_drafts_reach_nothing():
    """NaN scales of drafts: rows that see one are NaN (in its group, for V),
    the others as without it."""
    c = Tree([20], [140], hq=4, hkv=1)
    plain = c.ref()
    see = np.array([[(int(c.mask[r, 0]) >> j) & 1 for j in range(20)]
                    for r in range(20)], dtype=bool)
    tok = 120 + 4
    c.pages.set_scale(1, c.table[0, tok // 16], tok % 16, 0, 3, 0x7F)
    tok = 120 + 11
    c.pages.set_scale(0, c.table[0, tok // 16], tok % 16, 0, 1, 0x7F)
    got = c.run()
    for r in range(20):
        if see[r, 11]:
            assert np.isnan(got[r]).all()
        elif see[r, 4]:
            assert np.isnan(got[r, :, 48:64]).all()
            assert np.isfinite(got[r, :, :48]).all()
            assert np.isfinite(got[r, :, 64:]).all()
    clean = ~see[:, 11] & ~see[:, 4]
    assert clean.any() and (see[:, 4] & ~see[:, 11]).any()
    out, mag, seen, vmax = plain
    c2 = [a.copy() for a in plain]
    c2[0][~clean] = got[~clean] = 0
    c.check(got, tuple(c2))


def test_nan_of_two_drafts():
    """A row that sees the second NaN draft and not the first one."""
    c = Tree([3], [103], hq=2, hkv=1)
    c.mask[:, 0] = [0b001, 0b010, 0b100]
    for j in (0, 1):
        tok = 100 + j
        c.pages.set_scale(1, c.table[0, tok // 16], tok % 16, 0, 0, 0xFF)
    got = c.run()
    assert np.isnan(got[:2, :, :16]).all()
    assert np.isfinite(got[2]).all() and np.isfinite(got[:, :, 16:]).all()


def test_bad_pages():
    c = Tree([20, 20], [400, 300], hq=8, hkv=2)
    c.table[0, 3] = -1
    c.table[0, 24] = 1 << 29     # (the drafts' page)
    c.table[1, 0] = c.pages.nb
    c.check(c.run(bits=kvq.KVQ_DEVERR_BLOCK))


def test_long_context_shared_by_many_ctas():
    c = Tree([40], [9000], hq=8, hkv=1)
    c.check(c.run())


def test_strides():
    c = Tree([4, 9], [300, 200], hq=8, hkv=2).upload()
    big = torch.zeros(13, 3, 8, 128, dtype=c.dt, device="cuda")
    big[:, 1] = c.qd
    out = torch.full((13, 2, 8, 128), 77.0, dtype=c.dt, device="cuda")
    wide = torch.full((13, 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:3] = c.mask_dev()
    kvq.kvq_tree_attention_nvfp4(
        big[:, 1], c.kc, c.vc, c.bt, c.cud, c.lend, wide[:, 2:3], c.ks, c.vs,
        c.scale, out[:, 1], c.max_q, dev_error=c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    c.check(out[:, 1].double().cpu().numpy())
    assert (out[:, 0] == 77.0).all()


@pytest.mark.parametrize("max_q", [0, 1, 3, 500])
def test_any_max_q(max_q):
    c = Tree([20, 1, 4], [500, 300, 64], hq=8, hkv=2)
    bits = 0
    c.upload()
    c.call(max_q=max_q)
    torch.cuda.synchronize()
    if int(c.err.item()) == bits:
        c.check(c.out.double().cpu().numpy())


def test_repeats_to_the_bit():
    c = Tree([40, 1, 9], [900, 700, 77], hq=16, hkv=2)
    a = c.run()
    assert all((c.run() == a).all() for _ in range(3))


@pytest.mark.parametrize("seed", range(24))
def test_random(seed):
    rng = np.random.default_rng(700 + seed)
    n = int(rng.integers(1, 6))
    lens = rng.integers(0, 900, n)
    q_lens = [int(rng.integers(0, min(L, 70) + 1)) for L in lens]
    block = int(rng.choice([4, 8, 12, 16, 32, 64]))
    hkv = int(rng.choice([1, 2, 3]))
    c = Tree(q_lens, lens, hq=hkv * int(rng.choice([1, 2, 5, 8, 16])),
             hkv=hkv, block=block, nhd=bool(rng.random() < 0.5),
             swz=bool(rng.random() < 0.5), f16=bool(rng.random() < 0.5),
             seed=seed, pad_rows=int(seed % 3))
    if c.q.shape[0]:
        c.check(c.run())


# Trees of up to 8 drafts go by rows where they are few over short contexts, of
# up to 4 always; single drafts too beside larger trees of many sequences.
@pytest.mark.parametrize("n", [1, 3, 4, 5, 8])
@pytest.mark.parametrize("first", [0, 1, 24, 27, 28, 31, 32, 60, 93, 120, 127,
                                   500])
def test_small_trees_anywhere_in_a_step(n, first):
    c = Tree([n, n], [first + n, first + n + 3], hq=8, hkv=2, seed=first + n)
    c.mask[n:] = c.rng.integers(0, 1 << 32, c.mask[n:].shape)
    c.check(c.run())


@pytest.mark.parametrize("block", [4, 8, 12, 16, 32, 64, 128])
@pytest.mark.parametrize("nhd", [False, True])
@pytest.mark.parametrize("swz", [False, True])
@pytest.mark.parametrize("G", [4, 16])
def test_small_trees_of_all_layouts(block, nhd, swz, G):
    c = Tree([6, 1, 8], [100, 200, 333], hq=2 * G, hkv=2, block=block, nhd=nhd,
             swz=swz, f16=nhd)
    c.check(c.run())


def test_small_trees_of_no_mask_and_short_contexts():
    c = Tree([8, 8, 3, 2], [60, 8, 2, 0], hq=8, hkv=2)
    c.mask[:4] = 0
    c.mask[8:12] = 0xFFFFFF00     # (bits behind the last draft)
    c.mask[16:19, 0] = [1, 2, 7]  # (the first draft has no place)
    c.check(c.run())


def test_many_small_trees():
    rng = np.random.default_rng(5)
    q = rng.integers(0, 5, 100)
    c = Tree(list(q), list(q + rng.integers(0, 300, 100)), hq=8, hkv=2)
    c.check(c.run())


def test_single_drafts_beside_large_trees():
    rng = np.random.default_rng(6)
    q = np.where(rng.random(100) < 0.7, 1, rng.integers(0, 40, 100))
    c = Tree(list(q), list(q + rng.integers(0, 300, 100)), hq=8, hkv=2)
    c.mask[:5] = 0
    c.check(c.run())


@pytest.mark.parametrize("q_lens,lens,hkv", [
    ([3, 7], [9000, 4100], 1), ([4, 2], [5, 20000], 8),
    ([8], [60000], 8)])
def test_small_trees_of_several_stretches(q_lens, lens, hkv):
    c = Tree(q_lens, lens, hq=8, hkv=hkv)
    c.check(c.run())


@pytest.mark.parametrize("first", [64, 61, 90])
def test_masked_drafts_of_small_trees_reach_nothing(first):
    """NaN scales of drafts: rows that see one are NaN (in its group, for V),
    the others as without it."""
    c = Tree([6], [first + 6], hq=4, hkv=1)
    c.mask[:, 0] = [0b1, 0b11, 0b101, 0b1001, 0b10001, 0b110101]
    plain = [a.copy() for a in c.ref()]
    tok = first + 4     # V: rows 4 and 5
    c.pages.set_scale(1, c.table[0, tok // 16], tok % 16, 0, 3, 0x7F)
    tok = first + 3     # K: row 3
    c.pages.set_scale(0, c.table[0, tok // 16], tok % 16, 0, 1, 0x7F)
    got = c.run()
    assert np.isnan(got[3]).all()
    for r in (4, 5):
        assert np.isnan(got[r, :, 48:64]).all()
        assert np.isfinite(got[r, :, :48]).all()
        assert np.isfinite(got[r, :, 64:]).all()
    plain[0][3:] = got[3:] = 0
    c.check(got, tuple(plain))


def test_small_trees_bad_pages():
    c = Tree([6, 4], [400, 300], hq=8, hkv=2)
    c.table[0, 3] = -1
    c.table[0, 24] = 1 << 29     # (the drafts' page)
    c.table[1, 0] = c.pages.nb
    c.check(c.run(bits=kvq.KVQ_DEVERR_BLOCK))
