"""The indexer, the sparse and the tree attention as they are used together:
beside the page pool and the stores, in captured graphs, on other streams,
with buffers of the caller's alone, over offsets that pass 32 bits, and with
waits that give up."""
import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.page_models import Pages, chunk_attention
from tests.sparse_models import (listed_tokens, masked_attention, quantize_q,
                                 score_blocks, select_blocks, tree_tokens)
from tests.test_chunk_attention import KS, VS, Case
from tests.test_indexer_selection import Scores
from tests.test_sparse_attention import Sparse
from tests.test_tree_attention import Tree
from tests.variant_build import build_variant

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Server:
    """A small model's one layer: NVFP4 and indexer caches behind one page
    pool."""
    B, HQ, HKV, HI, DI, SEL, TOP = 64, 8, 2, 16, 128, 64, 3

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.nb, rows = 80, 4
        self.pool = kvq.alloc_page_pool(self.nb, rows, 20)
        self.kv, self.kc, self.vc = kvq.alloc_nvfp4_cache(
            self.nb, self.B, self.HKV, 128, fill=0)
        self.ik = torch.zeros(self.nb, self.B, self.DI + 4,
                              dtype=torch.uint8, device="cuda")
        self.ks = torch.tensor([KS], device="cuda")
        self.vs = torch.tensor([VS], device="cuda")
        self.err = i32([0])
        self.rows = i32([2, 0, 3])

    def rand(self, *shape):
        return torch.randn(*shape, device="cuda", generator=self.g).to(
            torch.bfloat16)

    def grow(self, counts, rows=None):
        """New tokens of the rows: pages, K and V, indexer K."""
        rows = self.rows if rows is None else rows
        cu = i32(np.concatenate([[0], np.cumsum(counts)]).tolist())
        total = int(sum(counts))
        slots = torch.empty(total, dtype=torch.int64, device="cuda")
        kvq.kvq_extend_sequences(*self.pool, rows, cu, slots, self.B,
                                 dev_error=self.err)
        kvq.kvq_store_nvfp4(self.rand(total, self.HKV, 128),
                            self.rand(total, self.HKV, 128), self.kc, self.vc,
                            slots, self.ks, self.vs, dev_error=self.err)
        kvq.kvq_store_indexer_k(self.rand(total, self.DI), self.ik, slots,
                                dev_error=self.err)
        return cu, total

    def pages(self):
        p = Pages(self.nb, self.B, self.HKV, 128)
        p.data = self.kv.cpu().numpy().reshape(self.nb, 2, -1)
        return p

    def batch(self):
        rows = self.rows.long()
        return self.pool[1][rows].contiguous(), self.pool[2][rows].contiguous()


def near(got, ref, u=2.0 ** -8):
    """The tolerance of tests/test_chunk_attention."""
    out, mag, seen, vmax = ref
    tol = (u * np.abs(out) + 2.0 ** -10 * mag
           + ((np.maximum(seen, 0) * 2.0 ** -25 + 2.0 ** -24)
              * vmax)[:, None, None])
    assert (np.abs(got - out) <= tol)[seen >= 0].all()


def test_prompt_then_steps():
    """Prompts in two pieces and some single tokens, each step through
    quantise, score, select and attend; every stage against its model, on what
    the stage before it gave."""
    s = Server(1)
    for counts in ([300, 40, 129], [17, 200, 64], [1, 1, 1], [1, 1, 1]):
        cu, total = s.grow(counts)
        table, lens = s.batch()
        q_i, w_i = s.rand(total, s.HI, s.DI), torch.randn(
            total, s.HI, device="cuda", generator=s.g)
        q8 = torch.empty(total, s.HI, s.DI, dtype=torch.float8_e4m3fn,
                         device="cuda")
        w = torch.empty_like(w_i)
        kvq.kvq_quantize_indexer_q(q_i, w_i, 0.05, q8, w)
        scores = torch.empty(total, 20, device="cuda")
        kvq.kvq_score_blocks_indexer_k(q8, w, s.ik, table, cu, lens, scores,
                                       s.SEL, max(counts), dev_error=s.err)
        chosen = torch.empty(total, s.TOP, dtype=torch.int32, device="cuda")
        kvq.kvq_select_blocks(scores, cu, lens, chosen, s.SEL, num_first=1,
                              num_last=1, dev_error=s.err)
        query = s.rand(total, s.HQ, 128)
        out = torch.empty_like(query)
        kvq.kvq_sparse_attention_nvfp4(query, s.kc, s.vc, table, cu, lens,
                                       chosen, s.SEL, s.ks, s.vs,
                                       128 ** -0.5, out, max(counts),
                                       dev_error=s.err)
        torch.cuda.synchronize()
        assert int(s.err.item()) == 0
        codes, want_w = quantize_q(q_i.float().cpu().numpy(),
                                   w_i.cpu().numpy(), 0.05)
        codes_got = q8.view(torch.uint8).cpu().numpy()
        assert (codes_got == codes).all()
        assert (w.cpu().numpy() == want_w).all()
        cun, lensn = cu.cpu().numpy(), lens.cpu().numpy()
        tn = table.cpu().numpy()
        want, tol = score_blocks(codes, want_w,
                                 s.ik.cpu().numpy().reshape(s.nb, -1), s.B,
                                 s.DI, tn, cun, lensn, s.SEL, 20)
        got = scores.cpu().numpy().astype(np.float64)
        live = ~np.isneginf(want)
        assert (np.isneginf(got) == ~live).all()
        assert (np.abs(got[live] - want[live]) <= tol[live]).all()
        lists = chosen.cpu().numpy()
        assert (lists == select_blocks(scores.cpu().numpy(), cun, lensn,
                                       s.SEL, s.TOP, 1, 1)).all()
        near(out.double().cpu().numpy(), masked_attention(
            s.pages(), query.double().cpu().numpy(), tn, cun, lensn, KS, VS,
            128 ** -0.5, listed_tokens(lists, s.SEL)))


def test_drafts_then_accepted_path():
    """A tree of drafts is attended to, one path of it accepted and compacted:
    the next token's attention over what is left is that of a sequence which
    never had the others."""
    s = Server(2)
    s.grow([100, 63, 200])
    before = s.pool[2][s.rows.long()].tolist()
    n = 7
    cu, total = s.grow([n] * 3)
    # parents 0 <- 1 <- 3 <- 6, 0 <- 2 <- 4, 1 <- 5
    up = [-1, 0, 0, 1, 2, 1, 3]
    bits = []
    for i in range(n):
        bits.append((bits[up[i]] if up[i] >= 0 else 0) | 1 << i)
    mask = i32([[b] for _ in range(3) for b in bits])
    table, lens = s.batch()
    query = s.rand(total, s.HQ, 128)
    out = torch.empty_like(query)
    kvq.kvq_tree_attention_nvfp4(query, s.kc, s.vc, table, cu, lens, mask,
                                 s.ks, s.vs, 128 ** -0.5, out, n,
                                 dev_error=s.err)
    torch.cuda.synchronize()
    near(out.double().cpu().numpy(), masked_attention(
        s.pages(), query.double().cpu().numpy(), table.cpu().numpy(),
        cu.cpu().numpy(), lens.cpu().numpy(), KS, VS, 128 ** -0.5,
        tree_tokens(mask.cpu().numpy().astype(np.int64))))
    # the path 0, 1, 3, 6 stays
    path = [0, 1, 3, 6]
    rows_before = s.pages().rows(0), table.cpu().numpy()
    keep = sum([list(range(L)) + [L + j for j in path] for L in before], [])
    kept = [L + len(path) for L in before]
    cu_keep = i32(np.concatenate([[0], np.cumsum(kept)]).tolist())
    src = torch.empty(len(keep), dtype=torch.int64, device="cuda")
    dst = torch.empty_like(src)
    kvq.kvq_compact_sequences(*s.pool, s.rows, i32(keep), cu_keep, src, dst,
                              s.B, dev_error=s.err)
    kvq.kvq_move_tokens_nvfp4([s.kv], src, dst, cu_keep, dev_error=s.err)
    table, lens = s.batch()
    assert lens.tolist() == kept
    after = s.pages().rows(0)
    for b, L in enumerate(before):
        for j, d in enumerate(path):
            t, o = L + j, L + d
            assert (after[table[b, t // s.B].item(), t % s.B]
                    == rows_before[0][rows_before[1][b, o // s.B],
                                      o % s.B]).all()
    cu, total = s.grow([1, 1, 1])
    table, lens = s.batch()
    query = s.rand(total, s.HQ, 128)
    out = torch.empty_like(query)
    kvq.kvq_chunk_attention_nvfp4(query, s.kc, s.vc, table, cu, lens, s.ks,
                                  s.vs, 128 ** -0.5, out, 1, dev_error=s.err)
    torch.cuda.synchronize()
    assert int(s.err.item()) == 0
    near(out.double().cpu().numpy(), chunk_attention(
        s.pages(), query.double().cpu().numpy(), table.cpu().numpy(),
        cu.cpu().numpy(), lens.cpu().numpy(), KS, VS, 128 ** -0.5))


# ---------------------------------------------------------------------------
# graphs, streams, memory
# ---------------------------------------------------------------------------
class Step:
    """All five calls over fixed buffers."""

    def __init__(self, seed, q_lens=(1, 40, 3), lens=(500, 900, 64)):
        self.sc = Scores(list(q_lens), list(lens), heads=16, seed=seed)
        self.sp = Sparse(list(q_lens), list(lens), sel=64, top=4, hq=8, hkv=2,
                         seed=seed).upload()
        self.tr = Tree(list(q_lens), list(lens), hq=8, hkv=2,
                       seed=seed).upload()
        sc, rng = self.sc, self.sc.rng
        n = sc.q.shape[0]
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.qi = torch.from_numpy(rng.standard_normal(
            (n, 16, 128))).to(torch.bfloat16).cuda()
        self.wi = torch.from_numpy(sc.w).cuda()
        self.q8 = torch.empty(n, 16, 128, dtype=torch.uint8, device="cuda")
        self.w = torch.empty(n, 16, device="cuda")
        self.cache, self.table = dev(sc.cache), dev(sc.table)
        self.cu, self.lens = dev(sc.cu), dev(sc.lens)
        self.scores = torch.empty(n, sc.columns, device="cuda")
        self.chosen = torch.empty(n, 4, dtype=torch.int32, device="cuda")
        self.mask = self.tr.mask_dev()
        self.max_q = max(q_lens)
        self.ws = kvq.sparse_attention_workspace(
            self.sp.qd, self.chosen, self.sp.kc, self.sp.bt, 64)
        self.ws2 = kvq.chunk_attention_workspace()

    def run(self, flags=0, **kw):
        sp, tr = self.sp, self.tr
        kvq.kvq_quantize_indexer_q(self.qi, self.wi, 0.1, self.q8, self.w,
                                   flags=flags, **kw)
        kvq.kvq_score_blocks_indexer_k(
            self.q8, self.w, self.cache, self.table, self.cu, self.lens,
            self.scores, 64, self.max_q, block_size=64, flags=flags,
            dev_error=sp.err, **kw)
        kvq.kvq_select_blocks(self.scores, self.cu, self.lens, self.chosen,
                              64, num_last=1, flags=flags, dev_error=sp.err,
                              **kw)
        kvq.kvq_sparse_attention_nvfp4(
            sp.qd, sp.kc, sp.vc, sp.bt, self.cu, self.lens, self.chosen, 64,
            sp.ks, sp.vs, sp.scale, sp.out, self.max_q, workspace=self.ws,
            flags=flags, dev_error=sp.err, **kw)
        kvq.kvq_tree_attention_nvfp4(
            tr.qd, tr.kc, tr.vc, tr.bt, self.cu, self.lens, self.mask, tr.ks,
            tr.vs, tr.scale, tr.out, self.max_q, workspace=self.ws2,
            flags=flags, dev_error=tr.err, **kw)

    def results(self):
        torch.cuda.synchronize()
        assert int(self.sp.err.item()) == int(self.tr.err.item()) == 0
        return [t.clone() for t in (self.q8, self.w, self.scores, self.chosen,
                                    self.sp.out, self.tr.out)]

    def clear(self):
        for t in (self.q8, self.w, self.scores, self.chosen, self.sp.out,
                  self.tr.out):
            t.zero_()
        torch.cuda.synchronize()


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("flags", [0, kvq.KVQ_F_PDL], ids=["plain", "pdl"])
def test_in_a_graph(flags):
    s = Step(3)
    s.run()
    want = s.results()
    s.clear()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.run(flags=flags)
        s.run(flags=flags)
    torch.cuda.synchronize()
    assert int((s.sp.out != 0).sum()) == 0       # nothing ran
    for _ in range(3):
        s.clear()
        graph.replay()
        assert same(s.results(), want)
    # other inputs in the same buffers
    other = Step(4)
    other.run()
    want = other.results()
    for name in ("qi", "wi", "cache", "table"):
        getattr(s, name).copy_(getattr(other, name))
    for a, b in ((s.sp, other.sp), (s.tr, other.tr)):
        for name in ("qd", "kv", "bt"):
            getattr(a, name).copy_(getattr(b, name))
    s.mask.copy_(other.mask)
    graph.replay()
    assert same(s.results(), want)


def test_two_graphs_side_by_side_with_workspaces_of_their_own():
    steps, graphs, want = [Step(5), Step(6)], [], []
    for s in steps:
        s.run()
        want.append(s.results())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s.run()
        graphs.append((g, side))
    for _ in range(5):
        for s in steps:
            s.clear()
        for g, side in graphs:
            with torch.cuda.stream(side):
                g.replay()
        for s, w in zip(steps, want):
            assert same(s.results(), w)


def test_two_graphs_share_workspaces_one_after_the_other():
    a, b = Step(7), Step(8)
    b.ws, b.ws2 = a.ws, a.ws2
    want, graphs = [], []
    for s in (a, b):
        s.run()
        want.append(s.results())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            s.run()
        graphs.append(g)
    for _ in range(3):
        a.clear()
        b.clear()
        for g in graphs:
            g.replay()
        assert same(a.results(), want[0]) and same(b.results(), want[1])


def test_streams():
    """The current stream, and one given by its handle."""
    s = Step(9)
    s.run()
    want = s.results()
    s.clear()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.run()
    assert same(s.results(), want)
    s.clear()
    s.run(stream=side.cuda_stream)
    assert same(s.results(), want)


def test_without_workspaces_and_flags():
    s = Step(10)
    s.run()
    want = s.results()
    s.clear()
    s.ws = s.ws2 = None
    s.run(flags=kvq.KVQ_F_PDL)
    assert same(s.results(), want)


def test_nothing_is_allocated():
    s = Step(11)
    s.run()
    torch.cuda.synchronize()
    held = torch.cuda.memory_stats()["allocation.all.allocated"]
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        s.run()
    torch.cuda.synchronize()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == held
    assert torch.cuda.mem_get_info()[0] == free


def test_no_error_word():
    s = Step(12)
    s.run()
    want = s.results()
    s.sp.err = s.tr.err = None
    s.clear()
    s.run()
    torch.cuda.synchronize()
    s.sp.err = s.tr.err = i32([0])
    assert same(s.results(), want)


# ---------------------------------------------------------------------------
# far offsets
# ---------------------------------------------------------------------------
def test_scores_over_far_blocks_and_rows():
    """Blocks and rows of scores and queries more than 2^31 bytes apart."""
    c = Scores([3], [150], heads=8, block=64, sel=64, spare=0)
    far = (1 << 31) + 4096
    big = torch.zeros(3 * far, dtype=torch.uint8, device="cuda")
    cache = big.as_strided((3, c.cache.shape[1]), (far, 1))
    cache.copy_(torch.from_numpy(c.cache))
    dev = lambda a: torch.from_numpy(a).cuda()
    qs = torch.zeros(3 * far, dtype=torch.uint8, device="cuda")
    q = qs.as_strided((3, 8, 128), (far, 128, 1))
    q.copy_(torch.from_numpy(c.q))
    out = torch.empty(2 * far + 64, device="cuda")[:]
    scores = out.as_strided((3, 3), (far, 1))
    kvq.kvq_score_blocks_indexer_k(q, dev(c.w), cache, dev(c.table),
                                   dev(c.cu), dev(c.lens), scores, 64, 3,
                                   block_size=64)
    c.check(scores.cpu().numpy().astype(np.float64))
    lists = torch.empty(3, 2, dtype=torch.int32, device="cuda")
    kvq.kvq_select_blocks(scores, dev(c.cu), dev(c.lens), lists, 64)
    assert (lists.cpu().numpy() == select_blocks(
        scores.cpu().numpy(), c.cu, c.lens, 64, 2, 0, 0)).all()


@pytest.mark.parametrize("what", ["sparse", "tree"])
def test_attention_over_far_pages_and_rows(what):
    """Pages, and rows of the query and the output, more than 2^31 elements
    from one another."""
    c = (Sparse([20], [100], sel=32, top=3, hq=8, hkv=1, spare=0)
         if what == "sparse" else Tree([20], [100], hq=8, hkv=1, spare=0))
    c.upload()
    nb, side = c.pages.nb, c.pages.side
    far = (1 << 30) + 4096
    big = torch.zeros(nb * far, dtype=torch.uint8, device="cuda")
    kv = big.as_strided((nb, 2, 1, 16, 72), (far, side, 16 * 72, 72, 1))
    kv.copy_(c.kv.view(nb, 2, 1, 16, 72))
    v = kv.transpose(2, 3)
    c.kc, c.vc = v[:, 0], v[:, 1]
    step = (1 << 27) + 64
    qs = torch.zeros(19 * step + 1024, dtype=c.dt, device="cuda")
    q = qs.as_strided((20, 8, 128), (step, 128, 1))
    q.copy_(c.qd)
    outs = torch.zeros(19 * step + 1024, dtype=c.dt, device="cuda")
    out = outs.as_strided((20, 8, 128), (step, 128, 1))
    c.qd = q
    c.call(out=out)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    c.check(out.double().cpu().numpy())


# ---------------------------------------------------------------------------
# waits that give up
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def giving_up(tmp_path_factory):
    limit = {"KVQ_WAIT_LIMIT_NS": 20000000}
    return build_variant(tmp_path_factory.mktemp("kvq_give_up"), {
        "score_blocks.cu": {"KVQ_TEST_SCORE_GIVE_UP": 1, **limit},
        "chunk_attention.cu": {"KVQ_TEST_GIVE_UP": 1, **limit},
        "sparse_attention.cu": {"KVQ_SPARSE_ITEMS_FROM": 0}})


@pytest.mark.parametrize("q_lens,lens", [
    ([1] * 40, [3000] * 40), ([64], [9000]), ([130, 3, 1], [7000, 900, 4000])])
def test_scores_that_give_up(giving_up, monkeypatch, q_lens, lens):
    """An epilogue warp of every other thread block gives up: the call ends
    and says so, what it has written is right; the regular library works
    afterwards."""
    c = Scores(q_lens, lens, heads=32, seed=len(q_lens))
    want = c.run()
    c.check(want)
    regular = kvq.LIB_PATH, kvq.lib()
    monkeypatch.setattr(kvq, "LIB_PATH", giving_up)
    monkeypatch.setattr(kvq, "_lib", None)
    got = c.run(bits=kvq.KVQ_DEVERR_TIMEOUT)
    left = got == 77.0
    assert left.any() and (got[~left] == want[~left]).all()
    monkeypatch.setattr(kvq, "LIB_PATH", regular[0])
    monkeypatch.setattr(kvq, "_lib", regular[1])
    assert (c.run() == want).all()


@pytest.mark.parametrize("what", ["sparse", "tree"])
def test_attention_that_gives_up(giving_up, monkeypatch, what):
    c = (Sparse([200, 64], [3000, 900], sel=64, top=30, hq=8, hkv=1, near=1.0)
         if what == "sparse" else
         Tree([60] * 12, [2000] * 12, hq=8, hkv=1)).upload()
    ref = c.ref()
    regular = kvq.LIB_PATH, kvq.lib()
    monkeypatch.setattr(kvq, "LIB_PATH", giving_up)
    monkeypatch.setattr(kvq, "_lib", None)
    c.call()
    torch.cuda.synchronize()
    assert int(c.err.item()) == kvq.KVQ_DEVERR_TIMEOUT
    got = c.out.double().cpu().numpy()
    left = (got == 77.0).all(-1)               # per row and head
    assert left.any()
    c.check(np.where(left[..., None], ref[0], got), ref)
    monkeypatch.setattr(kvq, "LIB_PATH", regular[0])
    monkeypatch.setattr(kvq, "_lib", regular[1])
    c.err.zero_()
    c.call()
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    c.check(c.out.double().cpu().numpy(), ref)
