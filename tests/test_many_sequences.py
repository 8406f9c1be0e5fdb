"""Batches of more sequences, or groups of rows, than a thread block has
threads: each kernel that lays out its work on the device then does so in
several rounds."""
import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.test_chunk_attention import VS
from tests.test_indexer_selection import Scores, check_select
from tests.test_sparse_attention import Sparse
from tests.test_tree_attention import Tree
from tests.variant_build import build_variant

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tiles_library(tmp_path_factory):
    """Asks whether tiles pay however small the batch is."""
    return build_variant(tmp_path_factory.mktemp("kvq_tiles"), {
        "sparse_attention.cu": {"KVQ_SPARSE_ITEMS_FROM": 0}})


@pytest.mark.parametrize("seqs", [640, 641, 1500, 3000])
def test_scores(seqs):
    rng = np.random.default_rng(seqs)
    q = rng.choice([0, 1, 1, 2, 3], seqs)
    lens = q + rng.integers(0, 300, seqs)
    lens[rng.random(seqs) < 0.02] += 2500
    c = Scores(q.tolist(), lens.tolist(), heads=8, D=32, sel=32, seed=seqs)
    c.check(c.run())


@pytest.mark.parametrize("last", [False, True])
def test_scores_of_one_sequence_among_many(last):
    """All work in one place of the batch, the first or the last."""
    q, lens = [0] * 2000, [700] * 2000
    q[-1 if last else 0] = 70
    c = Scores(q, lens, heads=16, D=64, sel=64, seed=int(last))
    c.check(c.run())


@pytest.mark.parametrize("seqs", [1000, 20000])
def test_selection(seqs):
    rng = np.random.default_rng(seqs)
    q = rng.choice([0, 0, 1, 2], seqs)
    lens = (q + rng.integers(0, 600, seqs)).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    x = rng.integers(-5, 6, (int(cu[-1]), 38)).astype(np.float32)
    check_select(x, cu, lens, 16, 6, 1, 1)


@pytest.mark.parametrize("seqs", [700, 1300])
def test_trees(seqs):
    rng = np.random.default_rng(seqs)
    q = rng.choice([0, 1, 2, 9, 12], seqs)
    c = Tree(q.tolist(), (q + rng.integers(0, 200, seqs)).tolist(), hq=2,
             hkv=1, seed=seqs)
    c.check(c.run())


@pytest.mark.parametrize("seqs,n", [(40, 70), (700, 9)])
@pytest.mark.parametrize("near", [1.0, 0.3])
def test_sparse(tiles_library, monkeypatch, seqs, n, near):
    """Items of 16 tokens: 240 and 1093 of them."""
    q = [n] * seqs
    q[seqs // 2] = 400
    c = Sparse(q, [300 + x for x in q], sel=16, top=12, near=near, hq=16,
               hkv=1, seed=seqs)
    got = c.run()
    monkeypatch.setattr(kvq, "LIB_PATH", tiles_library)
    monkeypatch.setattr(kvq, "_lib", None)
    tiled = c.run()
    # all rows of a few sequences against 64 bits, the others (each way within
    # its tolerance of them) against one another
    some = sorted({0, 1, seqs // 2, seqs - 2, seqs - 1})
    rows = np.concatenate([np.arange(c.cu[b], c.cu[b + 1]) for b in some])
    part = Sparse.__new__(Sparse)
    part.__dict__.update(c.__dict__)
    part.cu = np.concatenate(
        [[0], np.cumsum([q[b] for b in some])]).astype(np.int32)
    part.lens, part.table = c.lens[some], c.table[some]
    part.q, part.selected = c.q[rows], c.selected[rows]
    ref = part.ref()
    part.check(got[rows], ref)
    part.check(tiled[rows], ref)
    # u |ref| each, and what the weights' rounding can move (2^-10 of at most
    # the largest |V^| each, and the weights below fp16's range: 400 2^-25)
    vmax = np.nanmax(np.abs(c.pages.rows(1))) * VS
    tol = (2 * 2.0 ** -8 * np.abs(got) * (1 + 2.0 ** -7)
           + 2 * (2.0 ** -10 + 400 * 2.0 ** -25 + 2.0 ** -24) * vmax)
    assert (np.abs(tiled - got) <= tol).all()
