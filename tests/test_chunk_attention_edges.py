"""kvq_chunk_attention_nvfp4 where its kernels' limits or the order of its
steps matter."""
import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.page_models import E4M3, chunk_attention
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


def sink_case(n, seqs, L, share, seed):
    """`seqs` sequences over the same pages: keys of zeros behind a first key
    of ones, so that a row's query (a multiple of ones) sets the weight of
    the first token, whose V is zero: between `share` and 1 - (1 - share) / 8.
    The other V are not negative, so that the output is of the size of
    mag."""
    rng = np.random.default_rng(seed)
    c = Case([n], [L], hq=2, hkv=1, seed=seed)
    cut = 16 * 64
    c.pages.data[:, 0, :cut] = 0
    c.pages.data[:, 0, cut:] = 0x38                      # scales 1.0
    c.pages.data[:, 1, :cut] &= 0x77                     # codes >= 0
    page = c.table[0, 0]
    for side, code in ((0, 0x22), (1, 0)):               # 1.0; 0.0
        d, _ = c.pages.places(side, 0)
        c.pages.data[page, side, d[0]] = code
    rest = (1 - share) * np.exp2(-3 * rng.random((n, 2)))
    x0 = np.log(L * (1 - rest) / rest)                   # the first logit
    q = np.repeat((x0 / (c.scale * KS * 128))[..., None], 128, -1)
    c.q = torch.from_numpy(q).to(c.dt)
    ref = c.ref()
    c.q = c.q.repeat(seqs, 1, 1)
    c.table = np.repeat(c.table, seqs, 0)
    c.lens = np.full(seqs, L, dtype=np.int32)
    c.cu = (n * np.arange(seqs + 1)).astype(np.int32)
    return c, ref


@pytest.mark.parametrize("n,seqs,L,share", [
    (9, 160, 30000, 0.99),      # a share of the work is a sequence
    (66, 80, 30000, 0.99),      # two query tiles
    (9, 160, 60000, 0.9), (9, 160, 2000, 0.999),
    (4, 8, 30000, 0.9995),      # the decode kernel's rows
    (1, 8, 450, 0.9995), (8, 8, 100, 0.9999)])
def test_one_token_takes_nearly_all(n, seqs, L, share):
    """The general bound's u |out| + 2^-10 mag, here (u + 2^-10) mag; the
    weight of the reference is 2^7 at least beside those formed with it, so
    that one below fp16's normal range is off by 2^-25 of 2^7 times the sum,
    together seen 2^-32 vmax; and the fp32 sums, whose terms all have one
    sign: L / 16 steps of the product with V, L / 64 + 32 of the weights',
    each off by 2^-23 of the sum at most: below L / 8 2^-23 mag for the
    lengths here."""
    c, (out, mag, seen, vmax) = sink_case(n, seqs, L, share, seed=n)
    got = c.run(max_context_len=L).reshape(seqs, n, 2, 128)
    tol = (2.0 ** -8 + 2.0 ** -10 + L / 8 * 2.0 ** -23) * mag + (
        seen * 2.0 ** -32 * vmax)[:, None, None]
    worst = (np.abs(got - out) / mag).max()
    assert (np.abs(got - out) <= tol).all(), worst


@pytest.mark.parametrize("n", [3, 12, 100])
@pytest.mark.parametrize("rise", [3, 7, 8, 9, 12, 20, -20])
def test_logits_that_rise_from_tile_to_tile(n, rise):
    """By `rise` in log2 from each 64 tokens to the next, over seven tiles:
    within what the running reference takes without being set anew, and past
    it.  Logits are up to 194 here: eight steps of an fp32 sum, each off by
    2^-23 of that at most, are 2^-12.3 on a weight, above the fraction bar
    and below it: beside the general bound, 2^-11 mag."""
    L = 14 * 64
    c = Case([n], [L], hq=2, hkv=1, seed=n)
    cut = 16 * 64
    c.pages.data[:, 0, :cut] = 0x22                      # every code 1.0
    for j, page in enumerate(c.table[0, :L // 16]):
        times = j // 4 + 1 if rise > 0 else 14 - j // 4  # exact in e4m3
        c.pages.data[page, 0, cut:] = int(np.nonzero(E4M3 == times)[0][0])
    c.q = torch.full_like(c.q, abs(rise) * np.log(2) / (c.scale * KS * 128))
    out, mag, seen, vmax = c.ref()
    got = c.run()
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -10 + 2.0 ** -11) * mag + (
        (seen * 2.0 ** -25 + 2.0 ** -24) * vmax)[:, None, None]
    assert (np.abs(got - out) <= tol).all()


@pytest.mark.parametrize("n,L", [(30, 10), (200, 60), (4, 2)])
def test_rows_that_see_nothing_under_any_scale(n, L):
    """Zeros, even where the tensor scales are not numbers; the rows that see
    a token are NaN then."""
    c = Case([n], [L], hq=4, hkv=1, seed=40).upload()
    for k_scale, v_scale in ((float("nan"), VS), (KS, float("nan")),
                             (float("inf"), VS)):
        c.ks.fill_(k_scale)
        c.vs.fill_(v_scale)
        c.out.fill_(77.0)
        c.call()
        got = c.out.double().cpu().numpy()
        assert (got[:n - L] == 0).all(), (k_scale, v_scale)
        if np.isnan(k_scale) or np.isnan(v_scale):
            assert np.isnan(got[n - L:]).all()


@pytest.mark.parametrize("n", [1, 3, 4])
@pytest.mark.parametrize("fits", [True, False])
def test_short_chunks_on_both_sides_of_the_workspace(n, fits):
    """Single tokens and drafts whose partial results, counted over the width
    of the block table, fit the workspace, and such that do not and go
    through the tile kernel."""
    rng = np.random.default_rng(n)
    seqs = 130
    lens = (n + rng.integers(0, 60, seqs)).tolist()
    lens[5], lens[100] = 700, 1300
    c = Case([n] * seqs, lens, hq=16, hkv=1, seed=n)
    room = kvq.chunk_attention_workspace().numel()
    parts = room // (seqs * n * 16 * 130 * 4)      # stretches of 512 tokens
    width = (parts if fits else parts + 1) * 512 // 16
    table = np.full((seqs, width), -1, dtype=np.int32)
    table[:, :c.table.shape[1]] = c.table
    c.table = table
    c.check(c.run())


@pytest.mark.parametrize("max_q", [8, 40])
def test_rows_of_offsets_out_of_order(max_q):
    """Clamped and flagged: the rows that a clamped sequence has are its
    attention (with max_q_len 8 only those of chunks up to it), all others
    and the memory around the output are left as they were."""
    for cu in ([0, 9, 40], [-3, 8, 16], [0, 12, 8], [50, 60, 70],
               [0, 5, 1 << 30]):
        c = Case([8, 8], [40, 43], hq=4, hkv=1, seed=13)
        c.cu = np.asarray(cu, dtype=np.int32)
        c.upload()
        guard = torch.full((16 + 64, 4, 128), 77.0, dtype=c.dt,
                           device="cuda")
        c.call(out=guard[32:48], max_q=max_q)
        torch.cuda.synchronize()
        assert int(c.err.item()) == kvq.KVQ_DEVERR_SEQ, cu
        whole = guard.double().cpu().numpy()
        assert (whole[:32] == 77.0).all() and (whole[48:] == 77.0).all(), cu
        got = whole[32:48]
        want, mag, seen, vmax = (np.zeros((16, 4, 128)),
                                 np.zeros((16, 4, 128)), np.full(16, -1),
                                 np.zeros(16))
        for b in range(2):
            q0 = min(max(cu[b], 0), 16)
            n = min(max(cu[b + 1], q0), 16) - q0
            if n == 0 or n > max_q:
                continue
            part = chunk_attention(c.pages, c.q.double().numpy()[q0:q0 + n],
                                   c.table[b:b + 1], [0, n], c.lens[b:b + 1],
                                   KS, VS, c.scale)
            for to, x in zip((want, mag, seen, vmax), part):
                to[q0:q0 + n] = x
        c.check(got, (want, mag, seen, vmax), what=cu)


@pytest.mark.parametrize("new", [[64, 1, 200], [3, 1, 4]],
                         ids=["tiles", "short"])
def test_dependent_launches_behind_the_writers(new):
    """Extend, store, attention, step after step with dependent launches: the
    same bits as launched without and waited for after each call."""
    B, H, hq, steps, rows = 16, 2, 8, 12, len(new)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(sum(new))
    total = sum(new)
    k, v = (torch.randn(steps, total, H, 128, device="cuda",
                        generator=gen).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(steps, total, hq, 128, device="cuda",
                    generator=gen).to(torch.bfloat16)
    width = -(-max(new) * steps // B)
    ids = torch.arange(rows, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + np.cumsum(new).tolist(), dtype=torch.int32,
                      device="cuda")
    ks, vs = (torch.tensor([x], device="cuda") for x in (KS, VS))
    ws = kvq.chunk_attention_workspace()

    def run(pdl):
        ref, table, lens = kvq.alloc_page_pool(rows * width, rows, width)
        kv, kc, vc = kvq.alloc_nvfp4_cache(rows * width, B, H, 128, fill=0x7F)
        out = torch.full((steps, total, hq, 128), 77.0, dtype=q.dtype,
                         device="cuda")
        slots = torch.zeros(total, dtype=torch.int64, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        f = dict(flags=kvq.KVQ_F_PDL if pdl else 0, dev_error=err)
        wait = (lambda: None) if pdl else torch.cuda.synchronize
        torch.cuda.synchronize()
        for i in range(steps):
            kvq.kvq_extend_sequences(ref, table, lens, ids, cu, slots, B, **f)
            wait()
            kvq.kvq_store_nvfp4(k[i], v[i], kc, vc, slots, ks, vs, **f)
            wait()
            kvq.kvq_chunk_attention_nvfp4(
                q[i], kc, vc, table, cu, lens, ks, vs, 128 ** -0.5, out[i],
                max(new), workspace=ws, **f)
            wait()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return out, kv, table, lens

    want = run(False)
    assert bool(torch.isfinite(want[0]).all())
    for _ in range(4):
        for a, b in zip(run(True), want):
            assert torch.equal(a, b)


def test_nan_scales_under_many_segments():
    """The lists of V scales that are not numbers, segment after segment:
    NaN in their group's columns of the rows that see the token, nowhere
    else."""
    rng = np.random.default_rng(61)
    q = rng.integers(5, 40, 700)
    lens = q + rng.integers(0, 260, q.size)
    c = Case(q.tolist(), lens.tolist(), hq=4, hkv=1, seed=61)
    clean, ref = c.run(), c.ref()
    c.check(clean, ref)
    want = np.zeros(clean.shape, dtype=bool)
    for b in rng.permutation(q.size)[:250]:
        t, group = int(rng.integers(0, lens[b])), int(rng.integers(0, 8))
        c.pages.set_scale(1, c.table[b, t // 16], t % 16, 0, group,
                          int(rng.choice([0x7F, 0xFF])))
        sees = np.arange(q[b]) + lens[b] - q[b] >= t
        want[c.cu[b]:c.cu[b + 1]][sees, :, 16 * group:16 * group + 16] = True
    for _ in range(5):
        got = c.run()
        assert np.array_equal(np.isnan(got), want)
        c.check(np.where(want, clean, got), ref)


def test_many_heads():
    """64 KV heads of 16 query heads: the most that a call may have."""
    c = Case([1, 19, 5], [40, 33, 140], hq=1024, hkv=64, seed=62)
    c.check(c.run())


def test_rows_far_into_the_query():
    """More than 2^31 elements of queries: 18 million rows, of which the last
    1000 see something."""
    n, L = 18_000_000, 1000
    c = Case([L], [L], hq=1, hkv=1, seed=63)
    ref = c.ref()
    c.upload()
    c.qd = torch.zeros(n, 1, 128, dtype=c.dt, device="cuda")
    c.qd[-L:] = c.q.cuda()
    c.cud = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out = torch.full_like(c.qd, 77.0)
    c.call(out=out, max_q=n)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    assert not bool(out[:-L].any())
    c.check(out[-L:].double().cpu().numpy(), ref)
