"""The indexer's queries, block scores and block selection on the GPU against
plain models in 64 bits (tests/sparse_models.py has the scores' tolerance).
Quantised queries and selected blocks must be equal to the last bit."""
import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.sparse_models import (e4m3_codes, quantize_q, score_blocks,
                                 select_blocks)

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---------------------------------------------------------------------------
# queries
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("D", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 5), (37, 64), (2, 1024)])
def test_quantize(T, H, D, f16):
    rng = np.random.default_rng(T * H + D)
    dt = torch.float16 if f16 else torch.bfloat16
    q = torch.from_numpy(rng.standard_normal((T, H, D)) *
                         2.0 ** rng.integers(-12, 12, (T, H, 1))).to(dt)
    q[0, 0] = 0                                   # a head of zeros
    q[-1, -1, ::2] = -0.0
    w = torch.from_numpy(rng.standard_normal((T, H))).float()
    out = torch.full((T, H, D), 0x55, dtype=torch.uint8, device="cuda")
    wo = torch.full((T, H), 7.0, device="cuda")
    kvq.kvq_quantize_indexer_q(q.cuda(), w.cuda(), 0.37, out, wo)
    codes, want = quantize_q(q.float().numpy(), w.numpy(), 0.37)
    # (a head of zeros has no sign)
    live = q.float().abs().amax(-1).numpy() > 0
    got = out.cpu().numpy()
    assert (got[live] == codes[live]).all()
    assert (got[~live] == 0).all()
    assert (wo.cpu().numpy() == want).all()


def test_quantize_strides_and_views():
    rng = np.random.default_rng(5)
    big = torch.from_numpy(rng.standard_normal((9, 3, 8, 64))).to(
        torch.bfloat16).cuda()
    q = big[:, 1]                                 # rows 3 * 8 * 64 apart
    wbig = torch.from_numpy(rng.standard_normal((9, 13))).float().cuda()
    w = wbig[:, 2:10]
    out = torch.empty(9, 8, 64, dtype=torch.float8_e4m3fn, device="cuda")
    wo = torch.empty(9, 8, device="cuda")
    kvq.kvq_quantize_indexer_q(q, w, 2.0, out, wo)
    codes, want = quantize_q(q.float().cpu().numpy(), w.cpu().numpy(), 2.0)
    assert (out.view(torch.uint8).cpu().numpy() == codes).all()
    assert (wo.cpu().numpy() == want).all()
    kvq.kvq_quantize_indexer_q(q[:0], w[:0], 2.0, out[:0], wo[:0])


def test_quantize_tiny_values():
    """Scales among fp32's subnormals, and elements of the largest sizes."""
    q = torch.zeros(3, 2, 16, dtype=torch.bfloat16)
    q[0] = 2.0 ** -130 * torch.arange(16) / 8
    q[1] = 3.0e38
    q[2, :, 3] = -2.0 ** -133
    w = torch.ones(3, 2)
    out = torch.empty(3, 2, 16, dtype=torch.uint8, device="cuda")
    wo = torch.empty(3, 2, device="cuda")
    kvq.kvq_quantize_indexer_q(q.cuda(), w.cuda(), 1.0, out, wo)
    x = q.float().numpy().astype(np.float64)
    s = np.abs(x).max(-1).astype(np.float32) / np.float32(448.0)
    with np.errstate(all="ignore"):
        y = q.float().numpy() / s[..., None]
    y = np.where(s[..., None] > 0, y, 0)
    assert (out.cpu().numpy() == e4m3_codes(y)).all()
    assert (wo.cpu().numpy() == s).all()


# ---------------------------------------------------------------------------
# scores
# ---------------------------------------------------------------------------
class Scores:
    def __init__(self, q_lens, lens, heads=8, D=128, block=64, sel=64, seed=0,
                 columns=None, pad_rows=0, spare=3, pad_block=0):
        rng = self.rng = np.random.default_rng(seed)
        self.B, self.D, self.sel, self.heads = block, D, sel, heads
        self.lens = np.asarray(lens, dtype=np.int32)
        self.cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        need = [-(-max(int(x), 0) // block) for x in lens]
        nb = sum(need) + spare
        self.table = np.full((len(lens), max(need + [1])), -1, dtype=np.int32)
        perm, at = rng.permutation(nb), 0
        for i, k in enumerate(need):
            self.table[i, :k] = perm[at:at + k]
            at += k
        total = int(self.cu[-1]) + pad_rows
        self.q = e4m3_codes(rng.standard_normal((total, heads, D)) * 64)
        self.w = rng.standard_normal((total, heads)).astype(np.float32)
        self.cache = np.zeros((nb, block * (D + 4) + pad_block),
                              dtype=np.uint8)
        self.cache[:, :block * D] = e4m3_codes(
            rng.standard_normal((nb, block * D)) * 64)
        self.cache[:, block * D:block * (D + 4)] = (
            rng.uniform(0.001, 0.02, (nb, block)).astype(np.float32).view(
                np.uint8).reshape(nb, -1))
        self.columns = columns if columns is not None else max(
            [-(-int(x) // sel) for x in lens] + [1])
        self.max_q = max(list(q_lens) + [0])

    def run(self, bits=0, columns_kept=None, **kw):
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((self.q.shape[0], self.columns), 77.0,
                         device="cuda")
        kvq.kvq_score_blocks_indexer_k(
            dev(self.q), dev(self.w), dev(self.cache), dev(self.table),
            dev(self.cu), dev(self.lens), out, self.sel,
            kw.pop("max_q", self.max_q), block_size=self.B,
            dev_error=self.err, **kw)
        torch.cuda.synchronize()
        assert int(self.err.item()) == bits
        return out.cpu().numpy().astype(np.float64)

    def check(self, got, lens=None):
        want, tol = score_blocks(
            self.q, self.w, self.cache, self.B, self.D, self.table, self.cu,
            self.lens if lens is None else lens, self.sel, self.columns)
        none = np.isnan(want)
        assert (got[none] == 77.0).all()
        low = np.isneginf(want)
        assert (np.isneginf(got) == low).all()
        live = ~none & ~low
        bad = np.argwhere(live & ~(np.abs(got - np.where(live, want, 0))
                                   <= tol))
        assert bad.size == 0, [(tuple(i), got[tuple(i)], want[tuple(i)],
                                tol[tuple(i)]) for i in bad[:4]]


def test_score_smallest():
    c = Scores([1], [1], heads=1)
    c.check(c.run())


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129,
                               255, 257, 700, 1025])
@pytest.mark.parametrize("sel", [16, 32, 64, 128])
def test_score_lengths(L, sel):
    c = Scores([min(L, 3)], [L], sel=sel, seed=L)
    c.check(c.run())


@pytest.mark.parametrize("heads", [1, 2, 5, 8, 15, 16, 17, 24, 32, 33, 48, 64,
                                   65, 100, 127, 128])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_score_heads_and_dims(heads, D):
    c = Scores([5, 1], [150, 300], heads=heads, D=D, seed=heads)
    c.check(c.run())


@pytest.mark.parametrize("block", [1, 3, 8, 16, 24, 32, 64, 100, 128, 256])
def test_score_block_sizes(block):
    # (a block's bytes are padded to a multiple of 16)
    pad = -(block * 132) % 16
    c = Scores([4, 2], [333, 129], block=block, sel=32, seed=block,
               pad_block=pad + 32)
    c.check(c.run())


@pytest.mark.parametrize("D", [32, 64])
@pytest.mark.parametrize("block", [1, 2, 3, 4, 6, 20, 32, 200])
def test_score_block_sizes_of_short_rows(block, D):
    pad = -(block * (D + 4)) % 16
    c = Scores([4, 2], [333, 129], D=D, block=block, sel=32, seed=block,
               pad_block=pad)
    c.check(c.run())


@pytest.mark.parametrize("q_lens,lens", [
    ([0, 1, 0], [5, 9, 700]), ([7, 0, 3], [7, 0, 500]),
    ([130], [130]), ([300], [1000]), ([1] * 40, list(range(1, 1200, 30))),
    ([5, 3], [3, 2]),                  # more new tokens than the context has
    ([2, 2], [0, 1]), ([70, 1, 9], [400, 2000, 9]),
])
@pytest.mark.parametrize("heads", [16, 64])
def test_score_ragged(q_lens, lens, heads):
    c = Scores(q_lens, lens, heads=heads, seed=len(lens), pad_rows=3)
    c.check(c.run())


def test_score_more_columns_and_strides():
    c = Scores([3, 2], [200, 300], columns=11)
    c.check(c.run())
    wide = torch.full((5, 20), 3.0, device="cuda")
    bt = torch.full((2, 9), 99999, dtype=torch.int32, device="cuda")
    bt[:, :c.table.shape[1]] = dev(c.table)
    qb = torch.zeros(5, 3, c.heads, c.D, dtype=torch.uint8, device="cuda")
    qb[:, 2] = dev(c.q)
    wb = torch.zeros(5, 31, device="cuda")
    wb[:, 7:7 + c.heads] = dev(c.w)
    kvq.kvq_score_blocks_indexer_k(
        qb[:, 2], wb[:, 7:7 + c.heads], dev(c.cache),
        bt[:, :c.table.shape[1]], dev(c.cu), dev(c.lens), wide[:, 4:15],
        c.sel, c.max_q, block_size=c.B)
    got = wide.cpu().numpy().astype(np.float64)
    c.check(got[:, 4:15])
    assert (got[:, :4] == 3.0).all() and (got[:, 15:] == 3.0).all()


@pytest.mark.parametrize("max_q", [0, 1, 2, 1000])
def test_score_any_max_q(max_q):
    c = Scores([9, 1, 30], [100, 700, 30], heads=32)
    c.check(c.run(max_q=max_q))


def test_score_bad_pages_are_left_out():
    c = Scores([2, 2], [300, 300], sel=32)
    c.table[0, 1] = -1
    c.table[0, 4] = 1 << 30
    c.table[1, 0] = c.cache.shape[0]
    c.check(c.run(bits=kvq.KVQ_DEVERR_BLOCK))


def test_score_nan_in_cache():
    """NaN rows and scales: those tokens are left out; bytes behind the
    context reach nothing."""
    c = Scores([2], [200], sel=32)
    full = c.cache
    B, D = c.B, c.D
    blk = c.table[0, 1]
    full[blk, 5 * D:5 * D + 3] = 0x7F
    full[blk, B * D + 4 * 9:B * D + 4 * 9 + 4] = [0, 0, 0xC0, 0x7F]
    last = c.table[0, 3]
    full[last, 8 * D:B * D] = 0xFF
    full[last, B * D + 4 * 8:] = 0xFF
    c.check(c.run())


def test_score_all_nan_block():
    c = Scores([1], [64], sel=64)
    c.cache[:, :c.B * c.D] = 0x7F
    c.check(c.run())


def test_score_extreme_codes():
    """Rows of the largest code: sums up to 128 * 448^2 per head."""
    c = Scores([3], [130], heads=64)
    c.q[:] = 0x7E
    c.cache[:, :c.B * c.D] = 0x7E
    c.cache[:, 64:128] = 0xFE
    c.w[:] = np.abs(c.w) * 1e-4
    c.check(c.run())


def test_score_negative_and_zero_scales():
    c = Scores([2], [300], sel=64)
    sf = c.cache[:, c.B * c.D:].view(np.float32)
    sf[::2] *= -1
    sf[1::3] = 0
    c.check(c.run())


def test_score_context_beyond_columns():
    c = Scores([2], [300], sel=64, columns=3)
    got = c.run(bits=kvq.KVQ_DEVERR_SEQ)
    c.check(got, lens=[192])


def test_score_offsets_out_of_order():
    c = Scores([2, 2, 2], [64, 64, 64])
    c.cu = np.array([0, 4, 2, 6], dtype=np.int32)
    c.run(bits=kvq.KVQ_DEVERR_SEQ)
    c.cu = np.array([0, 2, 4, 9], dtype=np.int32)
    c.run(bits=kvq.KVQ_DEVERR_SEQ)


@pytest.mark.parametrize("first", [-3, -2 ** 31])
def test_first_offset_below_zero(first):
    """Taken as 0, and flagged, by the scores and the selection."""
    c = Scores([40, 3], [900, 77], sel=16)
    cu, c.cu = c.cu, c.cu.copy()
    c.cu[0] = first
    got = c.run(bits=kvq.KVQ_DEVERR_SEQ)
    x = np.where(np.isneginf(got), 0, got).astype(np.float32)
    taken = run_select(x, c.cu, c.lens, 16, 9, 1, 1,
                       bits=kvq.KVQ_DEVERR_SEQ)
    c.cu = cu
    c.check(got)
    assert (taken == select_blocks(x, cu, c.lens, 16, 9, 1, 1)).all()


def test_score_repeats_to_the_bit():
    c = Scores([40, 1, 9], [900, 2000, 77], heads=64, sel=32)
    a = c.run()
    assert all((c.run() == a).all() for _ in range(3))


@pytest.mark.parametrize("seed", range(16))
def test_score_random(seed):
    rng = np.random.default_rng(100 + seed)
    n = int(rng.integers(1, 6))
    lens = rng.integers(0, 1500, n)
    q_lens = [int(rng.integers(0, min(L, 90) + 1)) for L in lens]
    block = int(rng.choice([4, 16, 20, 64, 128]))
    c = Scores(q_lens, lens, heads=int(rng.choice([3, 8, 20, 32, 64, 96])),
               D=int(rng.choice([32, 64, 128])), block=block,
               sel=int(rng.choice([16, 32, 64, 128])), seed=seed,
               pad_block=-(block * 132) % 16, pad_rows=int(seed % 3))
    if c.q.shape[0]:
        c.check(c.run())


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------
def run_select(x, cu, lens, sel, top, first=0, last=0, bits=0):
    out = torch.full((x.shape[0], top), -7, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kvq_select_blocks(dev(x), dev(np.asarray(cu, dtype=np.int32)),
                          dev(np.asarray(lens, dtype=np.int32)), out, sel,
                          num_first=first, num_last=last, dev_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == bits
    return out.cpu().numpy()


def check_select(x, cu, lens, sel, top, first=0, last=0):
    got = run_select(x, cu, lens, sel, top, first, last)
    want = select_blocks(x, cu, lens, sel, top, first, last)
    assert (got == want).all(), np.argwhere(got != want)[:4]


@pytest.mark.parametrize("nb", [1, 2, 3, 31, 32, 33, 64, 255, 256, 257, 511,
                                1000, 2048, 2049, 5000])
@pytest.mark.parametrize("top", [1, 2, 16, 33, 300])
def test_select_sizes(nb, top):
    rng = np.random.default_rng(nb + top)
    x = rng.standard_normal((3, nb)).astype(np.float32)
    check_select(x, [0, 1, 3], [16 * nb, 16 * nb], 16, top)


@pytest.mark.parametrize("first,last", [(0, 0), (1, 0), (0, 1), (1, 2),
                                        (3, 5), (8, 0), (0, 8), (4, 4)])
@pytest.mark.parametrize("top", [8, 40])
def test_select_first_and_last(first, last, top):
    rng = np.random.default_rng(first + 9 * last)
    x = rng.standard_normal((40, 50)).astype(np.float32)
    x[::3] = np.sort(x[::3], axis=1)
    check_select(x, [0, 40], [50 * 32 - 7], 32, top, first, last)


@pytest.mark.parametrize("grid", [1, 2, 5, 50])
def test_select_ties(grid):
    rng = np.random.default_rng(grid)
    x = (rng.integers(-grid, grid, (30, 700)) / 4).astype(np.float32)
    x[::2][x[::2] == 0] = -0.0
    check_select(x, [0, 30], [700 * 64], 64, 37, 1, 2)


def test_select_infinities_and_nan():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((12, 300)).astype(np.float32)
    x[0] = np.nan
    x[1] = -np.inf
    x[2] = np.inf
    x[3, ::2] = np.nan
    x[4, ::3] = -np.inf
    x[5, :200] = np.inf
    x[6] = np.float32(-3.4e38)
    x[7] = np.float32(1e-45)
    x[7, ::2] = 0
    x[8, 1:299] = np.nan
    x[9, ::2] = -np.nan
    # (a context longer than the columns: clamped to them, and flagged)
    got = run_select(x, [0, 12], [300 * 16 + 11], 16, 20, 1, 1,
                     bits=kvq.KVQ_DEVERR_SEQ)
    want = select_blocks(x, [0, 12], [300 * 16], 16, 20, 1, 1)
    assert (got == want).all(), np.argwhere(got != want)[:4]


def test_select_scores_behind_the_context_are_not_read():
    x = np.zeros((3, 20), dtype=np.float32)
    x[:, 5:] = np.inf
    x[1, 5:] = np.nan
    check_select(x, [0, 3], [5 * 64], 64, 4)


@pytest.mark.parametrize("q_lens,lens", [
    ([0, 3, 0, 2], [10, 100, 4, 900]), ([5], [3]), ([2], [0]),
    ([1] * 50, list(range(0, 5000, 100))),
    ([0] * 40 + [2] + [0] * 40, [64] * 81)])
def test_select_ragged(q_lens, lens):
    rng = np.random.default_rng(len(lens))
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    x = rng.standard_normal((int(cu[-1]) + 4, 200)).astype(np.float32)
    check_select(x, cu, lens, 32, 9, 1, 1)


def test_select_context_beyond_columns():
    x = np.arange(12, dtype=np.float32).reshape(2, 6)
    got = run_select(x, [0, 2], [1000], 64, 3, bits=kvq.KVQ_DEVERR_SEQ)
    assert (got == [[3, 4, 5], [3, 4, 5]]).all()


def test_select_strides():
    rng = np.random.default_rng(8)
    x = rng.standard_normal((6, 90)).astype(np.float32)
    big = dev(x)
    out = torch.full((6, 30), -7, dtype=torch.int32, device="cuda")
    cu, lens = dev(np.array([0, 6], dtype=np.int32)), dev(
        np.array([50 * 64], dtype=np.int32))
    kvq.kvq_select_blocks(big[:, 21:71], cu, lens, out[:, 3:19], 64)
    want = select_blocks(x[:, 21:71], [0, 6], [50 * 64], 64, 16, 0, 0)
    got = out.cpu().numpy()
    assert (got[:, 3:19] == want).all()
    assert (got[:, :3] == -7).all() and (got[:, 19:] == -7).all()


def test_select_many_rows_and_long_rows():
    rng = np.random.default_rng(11)
    x = np.round(rng.standard_normal((64, 9000)) * 50).astype(
        np.float32) / 50
    check_select(x, [0, 64], [9000 * 16], 16, 128, 2, 3)


@pytest.mark.parametrize("nb", [16384, 16385, 20000])
@pytest.mark.parametrize("top,first,last", [(1, 0, 0), (100, 3, 5),
                                            (16000, 0, 1)])
def test_select_longest_rows(nb, top, first, last):
    rng = np.random.default_rng(nb + top)
    x = np.round(rng.standard_normal((3, nb)) * 200).astype(np.float32) / 200
    x[1] = 0.25
    check_select(x, [0, 2, 3], [16 * nb, 16 * nb], 16, top, first, last)
