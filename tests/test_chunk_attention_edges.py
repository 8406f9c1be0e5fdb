"""kvq_chunk_attention_nvfp4 where its kernels' limits or the order of its
steps matter."""
import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.page_models import chunk_attention
from tests.test_chunk_attention import KS, VS, Case

pytestmark = pytest.mark.gpu


def test_more_sequences_than_threads():
    """Tiles of 1300 sequences: the shares are found in several rounds, and
    hold up to eight segments of one tile, some behind one of two query
    tiles."""
    rng = np.random.default_rng(31)
    q = rng.integers(0, 12, 1300)
    q[[0, 511, 512, 700, 1023, 1299]] = [9, 70, 300, 0, 12, 40]
    lens = q + rng.integers(0, 40, 1300)
    lens[512] = 900
    c = Case(q.tolist(), lens.tolist(), hq=4, hkv=1, seed=31)
    c.check(c.run())


def test_many_sequences_without_work():
    q = [0] * 1100
    q[700] = 33
    c = Case(q, [50] * 1100, hq=4, hkv=2, seed=32)
    c.check(c.run())


@pytest.mark.parametrize("seed", range(6))
def test_shares_of_many_short_segments(seed):
    """Hundreds of items of one to four tiles, of one and of two query tiles
    in any order; the same bits again and again."""
    rng = np.random.default_rng(200 + seed)
    q = rng.choice([2, 9, 31, 33, 40, 64, 70, 100], 900 + 17 * seed)
    lens = q + rng.choice([0, 0, 40, 130, 400], q.size)
    c = Case(q.tolist(), lens.tolist(), hq=8, hkv=2, seed=seed)
    c.upload()
    ws = kvq.chunk_attention_workspace()
    c.call(workspace=ws)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    want = c.out.clone()
    for _ in range(30):
        c.out.fill_(77.0)
        c.call(workspace=ws)
        assert torch.equal(c.out, want)
    assert int(c.err.item()) == 0
    some = np.sort(rng.permutation(q.size)[:40])
    rows = np.concatenate([np.arange(c.cu[b], c.cu[b + 1]) for b in some])
    ref = chunk_attention(c.pages, c.q.double().numpy()[rows], c.table[some],
                          np.concatenate([[0], np.cumsum(q[some])]),
                          c.lens[some], KS, VS, c.scale)
    c.check(want.double().cpu().numpy()[rows], ref)


@pytest.mark.parametrize("slot", [0, 1])
@pytest.mark.parametrize("G", [8, 16])
def test_one_slot_far_behind_the_other(slot, G):
    """Short chunks over long contexts, whose KV tiles alternate between the
    slots: all pages of one slot's tiles are bad, so that its rows have no
    reference and its weights are done over each time, and the other gets
    ahead."""
    c = Case([12] * 5, [9000] * 5, hq=G, hkv=1, seed=G + slot)
    tile = np.arange(c.table.shape[1]) * 16 // 128
    c.table[:, tile % 2 == slot] = -1
    bits = kvq.KVQ_DEVERR_BLOCK
    c.check(c.run(bits=bits))
    ws = kvq.chunk_attention_workspace()
    c.call(workspace=ws)
    want = c.out.clone()
    for _ in range(50):
        c.call(workspace=ws)
        assert torch.equal(c.out, want)
    assert int(c.err.item()) == bits
