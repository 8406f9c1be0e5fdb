"""kvq_chunk_attention_nvfp4 on the GPU against the attention in 64 bits.

Every output element must satisfy
    |out - ref| <= u |ref| + 2^-10 mag + (seen 2^-25 + 2^-24) vmax
with mag = sum of weight * |V^| and vmax the largest |V^| that the row sees:
  u |ref|      the final rounding (bf16 2^-8, fp16 2^-11) -- and the fp16
               query of a bf16 one is exact at these magnitudes;
  2^-10 mag    the rounding of each weight to fp16 (2^-11), and 2^-11 left
               for the fp32 logits: a logit of size x has an error of a few
               2^-24 x (products of at most 17 bits summed in fp32; |x| here
               is below 100, whence 2^-15), which moves a weight by as
               much, once above and once below the fraction bar;
  seen 2^-25   weights below fp16's normal range, each off by 2^-25 of the
               weight of the reference, of which the sum holds one at least
               up to the factor that the reference may lag behind (in the
               safe direction);
  2^-24 vmax   results near zero in fp32 sums."""
import numpy as np
import pytest
import torch

from paged_quantized_kv_gb300 import kvq
from tests.page_models import Pages, chunk_attention

pytestmark = pytest.mark.gpu

KS, VS = 0.03125, 0.046875


class Case:
    def __init__(self, q_lens, lens, hq=4, hkv=1, block=16, nhd=False,
                 swz=False, f16=False, seed=0, scale=128 ** -0.5, q_mul=1.0,
                 spare=3, pad_rows=0):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.B, self.f16 = hq, hkv, block, f16
        self.nhd, self.swz, self.scale = nhd, swz, scale
        n = len(lens)
        self.lens = np.asarray(lens, dtype=np.int32)
        self.cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        need = [-(-max(int(x), 0) // block) for x in lens]
        nb = sum(need) + spare
        self.table = np.full((n, max(need + [1]) + 1), -1, dtype=np.int32)
        perm = rng.permutation(nb)
        at = 0
        for i, k in enumerate(need):
            self.table[i, :k] = perm[at:at + k]
            at += k
        self.pages = Pages(nb, block, hkv, 128, nhd, swz).fill(rng)
        q = rng.standard_normal((int(self.cu[-1]) + pad_rows, hq, 128))
        self.dt = torch.float16 if f16 else torch.bfloat16
        self.q = (torch.from_numpy(q) * q_mul).to(self.dt)
        self.max_q = max(list(q_lens) + [0])
        self.rng = rng

    def views(self, kv):
        nb, B, H = kv.size(0), self.B, self.hkv
        if self.nhd:
            v = kv.view(nb, 2, B, H, 72)
            return v[:, 0], v[:, 1]
        v = kv.view(nb, 2, H, B, 72).transpose(2, 3)
        return v[:, 0], v[:, 1]

    def upload(self):
        self.kv = torch.from_numpy(self.pages.data).cuda()
        self.kc, self.vc = self.views(self.kv)
        self.qd = self.q.cuda()
        self.bt = torch.from_numpy(self.table).cuda()
        self.cud = torch.from_numpy(self.cu).cuda()
        self.lend = torch.from_numpy(self.lens).cuda()
        self.ks = torch.tensor([KS], device="cuda")
        self.vs = torch.tensor([VS], device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.out = torch.full(self.q.shape, 77.0, dtype=self.dt,
                              device="cuda")
        return self

    def call(self, out=None, **kw):
        flags = kw.pop("flags", 0)
        kvq.kvq_chunk_attention_nvfp4(
            self.qd, self.kc, self.vc, self.bt, self.cud, self.lend, self.ks,
            self.vs, self.scale, self.out if out is None else out,
            kw.pop("max_q", self.max_q),
            flags=flags | (kvq.KVQ_F_SWIZZLE_K_SCALE if self.swz else 0),
            dev_error=self.err, **kw)

    def run(self, bits=0, **kw):
        self.upload()
        self.call(**kw)
        torch.cuda.synchronize()
        assert int(self.err.item()) == bits
        return self.out.double().cpu().numpy()

    def ref(self, lens=None):
        return chunk_attention(self.pages, self.q.double().numpy(),
                               self.table, self.cu,
                               self.lens if lens is None else lens, KS, VS,
                               self.scale)

    def check(self, got, ref=None, what=""):
        out, mag, seen, vmax = self.ref() if ref is None else ref
        u = 2.0 ** -11 if self.f16 else 2.0 ** -8
        live = seen >= 0
        assert (got[~live] == 77.0).all(), what      # rows of no sequence
        assert (got[seen == 0] == 0).all(), what
        tol = (u * np.abs(out) + 2.0 ** -10 * mag
               + ((seen * 2.0 ** -25 + 2.0 ** -24) * vmax)[:, None, None])
        err = np.abs(got - out)[live]
        bad = np.argwhere(~(err <= tol[live]))
        assert bad.size == 0, (what, len(bad), [
            (tuple(i), got[live][tuple(i)], out[live][tuple(i)],
             tol[live][tuple(i)]) for i in bad[:4]])


def test_one_sequence_smallest():
    c = Case([1], [1])
    c.check(c.run())


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129,
                               255, 256, 257, 383, 512, 700])
def test_single_tokens(L):
    c = Case([1, 1], [L, max(1, L - 1)], hq=8, hkv=2, seed=L)
    c.check(c.run())


@pytest.mark.parametrize("n,L", [(2, 2), (5, 5), (5, 100), (16, 200),
                                 (17, 17), (31, 129), (32, 128), (33, 300),
                                 (64, 64), (65, 257), (100, 1000),
                                 (128, 128), (200, 333), (300, 300)])
def test_chunks(n, L):
    c = Case([n], [L], hq=4, hkv=1, seed=n)
    c.check(c.run())


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 16])
@pytest.mark.parametrize("f16", [False, True], ids=["bf16", "fp16"])
def test_head_groups(G, f16):
    c = Case([40, 1, 0, 7, 90], [300, 33, 5, 7, 140], hq=2 * G, hkv=2,
             f16=f16, seed=G)
    c.check(c.run())


@pytest.mark.parametrize("nhd", [False, True], ids=["HND", "NHD"])
@pytest.mark.parametrize("swz", [False, True])
@pytest.mark.parametrize("block", [4, 8, 12, 16, 20, 64, 384])
def test_page_forms(nhd, swz, block):
    c = Case([37, 2, 130], [290, 200, 131], hq=6, hkv=3, block=block,
             nhd=nhd, swz=swz, seed=block)
    c.check(c.run())


def test_rows_that_see_nothing():
    """Chunks longer than the context, empty contexts, empty chunks, rows
    behind the last sequence."""
    c = Case([5, 3, 0, 200, 4], [3, 0, 10, 150, -2], hq=4, hkv=2, seed=3,
             pad_rows=9)
    c.check(c.run())


def test_no_work():
    c = Case([0, 0], [5, 0], pad_rows=3)
    got = c.run()
    assert (got == 77.0).all()
    c = Case([], [])
    c.run()


@pytest.mark.parametrize("scale", [0.0, -0.09, 1e-30, 3.0])
def test_softmax_scales(scale):
    c = Case([30, 1], [170, 64], hq=8, hkv=2, seed=5, scale=scale)
    c.check(c.run())


def test_one_weight_takes_all():
    c = Case([150], [420], hq=4, hkv=1, seed=6, scale=0.5, q_mul=4.0)
    # logits of this size (some thousand) are off by more than the general
    # bound has for them: 2^-23 relative of sums of |q||k|
    out, mag, seen, vmax = c.ref()
    k = np.abs(c.pages.rows(0)).max() * KS
    x = 0.5 * np.abs(c.q.double().numpy()).sum(-1) * k       # >= |logit|
    slack = np.minimum(1.0, 4 * x * 2.0 ** -23)[..., None] * vmax[
        :, None, None]
    got = c.run()
    tol = 2.0 ** -8 * np.abs(out) + 2.0 ** -10 * mag + slack + \
        ((seen * 2.0 ** -25 + 2.0 ** -24) * vmax)[:, None, None]
    assert (np.abs(got - out) <= tol).all()


def test_growing_logits_move_the_reference():
    """Keys whose logits rise along the context by far more than the lag of
    the running reference, so that every tile rescales."""
    c = Case([130], [900], hq=2, hkv=1, block=16, seed=7)
    order = c.table[0, :-(-900 // 16)]
    cut = 16 * 64
    for i, p in enumerate(order):
        c.pages.data[p, 0, cut:] = min(30 + i, 100)
    c.pages.data[:, 0, :cut] = 0x22          # every code 1.0
    c.q = c.q.abs() * 0.05
    c.check(c.run())
    c.q = -c.q                               # ... and falling ones
    c.check(c.run())


def test_strided_rows_and_tables():
    c = Case([20, 33], [64, 190], hq=4, hkv=2, seed=8).upload()
    wide_q = torch.full((53, 6, 128), float("nan"), dtype=c.dt,
                        device="cuda")
    wide_q[:, :4] = c.qd
    c.qd = wide_q[:, :4]
    wide_o = torch.full((53, 5, 128), 77.0, dtype=c.dt, device="cuda")
    wide_t = torch.full((2, 40), 1 << 20, dtype=torch.int32, device="cuda")
    wide_t[:, :c.bt.size(1)] = c.bt
    c.bt = wide_t[:, :c.bt.size(1)]
    gap = torch.full((c.kv.size(0), 3, c.kv.size(2)), 255, dtype=torch.uint8,
                     device="cuda")
    gap[:, :2] = c.kv
    nb = gap.size(0)
    v = gap.view(nb, 3, 2, 16, 72).transpose(2, 3)
    c.kc, c.vc = v[:, 0], v[:, 1]
    c.call(out=wide_o[:, :4])
    assert int(c.err.item()) == 0
    assert bool((wide_o[:, 4] == 77.0).all())
    c.check(wide_o[:, :4].double().cpu().numpy())


def test_bytes_that_no_row_sees():
    """NaN scales behind the context and in pages nobody reads."""
    c = Case([60, 1], [101, 30], hq=4, hkv=2, seed=9)
    ref = c.ref()
    used = [(b, t) for b, L in enumerate(c.lens) for t in range(L)]
    keep = np.zeros((c.pages.nb, 16), dtype=bool)
    for b, t in used:
        keep[c.table[b, t // 16], t % 16] = True
    for p, off in np.argwhere(~keep):
        for side in range(2):
            d, s = c.pages.places(side, off)
            c.pages.data[p, side, s] = 0x7F
            c.pages.data[p, side, d] = 0xFF
    c.check(c.run(), ref)


@pytest.mark.parametrize("n,L,at", [(60, 101, 70), (200, 200, 10),
                                    (300, 500, 400), (4, 700, 697),
                                    (1, 900, 300)])
def test_nan_reaches_only_rows_that_see_it(n, L, at):
    c = Case([n], [L], hq=4, hkv=2, seed=10)
    clean, ref = c.run(), c.ref()
    c.check(clean, ref)
    page, off = c.table[0, at // 16], at % 16
    sees = np.arange(n) + L - n >= at
    c.pages.set_scale(1, page, off, 0, 3, 0x7F)      # V, head 0, group 3
    got = c.run()
    nan = np.isnan(got)
    want = np.zeros_like(nan)
    want[sees, :2, 48:64] = True
    assert np.array_equal(nan, want)
    c.check(np.where(nan, clean, got), ref)
    c.pages.set_scale(1, page, off, 0, 3, 0x30)
    c.pages.set_scale(0, page, off, 1, 0, 0xFF)      # K, head 1
    got = c.run()
    nan = np.isnan(got)
    want[:] = False
    want[sees, 2:] = True
    assert np.array_equal(nan, want)


def test_bad_pages_are_left_out():
    c = Case([70, 3], [200, 90], hq=4, hkv=1, seed=11)
    c.table[0, 2] = -1
    c.table[0, 5] = c.pages.nb
    c.table[1, :] = -5
    c.check(c.run(bits=kvq.KVQ_DEVERR_BLOCK))


def test_context_beyond_the_table():
    c = Case([5], [64], hq=4, hkv=1, seed=12)
    c.table = c.table[:, :4]
    c.lens[0] = 90
    c.check(c.run(bits=kvq.KVQ_DEVERR_SEQ), c.ref(lens=[64]))


def test_offsets_out_of_order():
    """Clamped and flagged, nothing written outside the rows."""
    c = Case([8, 8], [40, 40], hq=4, hkv=1, seed=13)
    for cu in ([0, 9, 40], [-3, 8, 16], [0, 12, 8], [50, 60, 70]):
        c.cu = np.asarray(cu, dtype=np.int32)
        c.upload()
        c.call()
        torch.cuda.synchronize()
        assert int(c.err.item()) == kvq.KVQ_DEVERR_SEQ


@pytest.mark.parametrize("n,hq,hkv", [(1, 8, 1), (4, 8, 1), (3, 4, 4),
                                      (40, 8, 1), (300, 2, 1)])
def test_long_contexts_are_split(n, hq, hkv):
    c = Case([n], [9000 + n], hq=hq, hkv=hkv, seed=14)
    c.check(c.run())


def test_many_sequences():
    rng = np.random.default_rng(15)
    q = rng.integers(0, 4, 700).tolist()
    lens = [max(a, int(x)) for a, x in zip(q, rng.integers(1, 60, 700))]
    c = Case(q, lens, hq=4, hkv=1, seed=15)
    c.check(c.run())


def test_ragged_batch():
    c = Case([1, 150, 1, 1, 37, 0, 260, 1, 8, 2],
             [1500, 900, 3, 128, 37, 50, 2100, 64, 1000, 129], hq=6, hkv=2,
             seed=16)
    c.check(c.run())


@pytest.mark.parametrize("max_q", [70, 71, 100000])
def test_max_q_len_is_a_bound(max_q):
    c = Case([70, 1, 9], [200, 300, 40], hq=8, hkv=1, seed=17)
    c.check(c.run(max_q=max_q))


@pytest.mark.parametrize("max_q", [0, 1, 3])
def test_chunks_beyond_max_q_len(max_q):
    """Flagged, their rows left as they were."""
    c = Case([70, 1, 9], [200, 300, 40], hq=8, hkv=1, seed=17)
    got, ref = c.run(bits=kvq.KVQ_DEVERR_SEQ, max_q=max_q), c.ref()
    assert (got[:70] == 77.0).all() and (got[71:] == 77.0).all()
    got[:70], got[71:] = ref[0][:70], ref[0][71:]
    c.check(got, ref)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (16, 1), (6, 2)])
def test_short_chunks(n, hq, hkv):
    """Every size around the change between the two kernels, in batches of
    one size, and beside longer and empty ones; contexts of one stretch and
    of several."""
    for q, lens in (([n] * 3, [n, 700, 4000]),
                    ([n, 0, 150, 1, n], [1900, 30, 333, 2600, max(n - 1, 0)])):
        c = Case(q, lens, hq=hq, hkv=hkv, seed=n)
        c.check(c.run(), what=(q, lens))
        c.check(c.run(max_context_len=max(lens)), what=(q, lens))


def test_context_beyond_max_context_len():
    for n in (1, 30):
        c = Case([n, 1], [200, 90], hq=4, hkv=1, seed=n)
        c.check(c.run(bits=kvq.KVQ_DEVERR_SEQ, max_context_len=120),
                c.ref(lens=[120, 90]))


def test_same_bits_every_time():
    c = Case([150, 1, 60], [3000, 2500, 60], hq=8, hkv=2, seed=18)
    a, b = c.run(), c.run()
    assert np.array_equal(a, b)


def test_pages_far_into_a_cache():
    """A cache of more than 2^32 bytes, the pages used at its end."""
    c = Case([20], [50], hq=2, hkv=1, block=16, seed=19).upload()
    nb = (1 << 32) // c.kv[0].numel() + 100
    far = torch.empty(nb, 2, c.kv.size(2), dtype=torch.uint8, device="cuda")
    far[-c.kv.size(0):] = c.kv
    c.kc, c.vc = c.views(far)
    c.bt = torch.where(c.bt >= 0, c.bt + (nb - c.kv.size(0)), c.bt)
    c.call()
    assert int(c.err.item()) == 0
    c.check(c.out.double().cpu().numpy())


def test_graph_streams_and_workspaces():
    """Captured and replayed; two streams at once, each with a workspace; an
    eager call between replays."""
    cases = [Case([60, 3], [2000, 700], hq=8, hkv=2, seed=s).upload()
             for s in (20, 21)]
    ws = [kvq.chunk_attention_workspace() for _ in cases]
    for c, w in zip(cases, ws):
        c.call(workspace=w)
    torch.cuda.synchronize()
    want = [c.out.clone() for c in cases]
    for c, w in zip(cases, want):
        c.check(w.double().cpu().numpy())
    graphs = []
    for c, w in zip(cases, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(workspace=w)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.out.fill_(0)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c.out, w)


def test_own_workspace_on_another_stream():
    """A workspace that the call allocates is not handed out again while a
    stream given by its handle still uses it."""
    c = Case([300], [5000], hq=8, hkv=1, seed=77).upload()
    size = kvq.chunk_attention_workspace().numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    c.call(stream=side.cuda_stream)
    other = [torch.full((size,), 0, dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    torch.cuda.synchronize()
    c.check(c.out.double().cpu().numpy())
    assert all(int(x.max()) == 0 for x in other)


def test_pdl_chain():
    """Store, then chunk attention, launched with dependent launch, many
    times over."""
    c = Case([64, 1], [256, 40], hq=4, hkv=1, seed=22).upload()
    ws = kvq.chunk_attention_workspace()
    c.call(workspace=ws)
    want = c.out.clone()
    c.out.fill_(0)
    key = torch.zeros(0, 1, 128, dtype=torch.bfloat16, device="cuda")
    for _ in range(20):
        c.call(workspace=ws, flags=kvq.KVQ_F_PDL)
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)
    assert key.numel() == 0


def test_agrees_with_the_decode_attention():
    c = Case([1, 1, 1], [700, 1300, 5], hq=16, hkv=2, seed=23)
    got = c.run()
    out = torch.empty_like(c.qd)
    kvq.kvq_paged_attention_nvfp4(c.qd, c.kc, c.vc, c.bt, c.lend, c.ks, c.vs,
                                  c.scale, out, 1300)
    ref = c.ref()
    c.check(got, ref)
    c.check(out.double().cpu().numpy(), ref)


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = np.random.default_rng(100 + seed)
    n = int(rng.integers(1, 7))
    q = [int(x) for x in np.exp(rng.uniform(0, np.log(260), n))]
    lens = [int(a + np.exp(rng.uniform(0, np.log(900))) - 1) for a in q]
    hkv = int(rng.integers(1, 4))
    c = Case(q, lens, hq=hkv * int(rng.integers(1, 17)), hkv=hkv,
             block=int(rng.choice([4, 8, 16, 28, 32, 64])),
             nhd=bool(rng.integers(2)), swz=bool(rng.integers(2)),
             f16=bool(rng.integers(2)), seed=seed,
             pad_rows=int(rng.integers(0, 3)))
    c.check(c.run())


def test_serving_loop():
    """The operators as they are used together: prompts admitted, stored,
    attended; samples forked off a prompt; tokens decoded; the context
    compacted; everything freed."""
    B, H, hq, rows = 16, 2, 8, 6
    dt, torch_rng = torch.bfloat16, torch.Generator(device="cuda")
    torch_rng.manual_seed(5)
    ref_count, table, lens = kvq.alloc_page_pool(64, rows, 12)
    kv, kc, vc = kvq.alloc_nvfp4_cache(64, B, H, 128, fill=0)
    ks = torch.tensor([KS], device="cuda")
    vs = torch.tensor([VS], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = kvq.chunk_attention_workspace()

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def feed(ids, new):
        cu = i32([0] + np.cumsum(new).tolist())
        total = sum(new)
        slots = torch.empty(total, dtype=torch.int64, device="cuda")
        kvq.kvq_extend_sequences(ref_count, table, lens, i32(ids), cu, slots,
                                 B, dev_error=err)
        k = torch.randn(total, H, 128, device="cuda", generator=torch_rng)
        v = torch.randn(total, H, 128, device="cuda", generator=torch_rng)
        kvq.kvq_store_nvfp4(k.to(dt), v.to(dt), kc, vc, slots, ks, vs,
                            dev_error=err)
        q = torch.randn(total, hq, 128, device="cuda",
                        generator=torch_rng).to(dt)
        out = torch.empty_like(q)
        at = i32(ids).long()
        kvq.kvq_chunk_attention_nvfp4(
            q, kc, vc, table[at], cu, lens[at], ks, vs, 128 ** -0.5, out,
            max(new), workspace=ws, dev_error=err)
        c = Case([], [], hq=hq, hkv=H)
        c.pages = Pages(64, B, H)
        c.pages.data = kv.cpu().numpy().reshape(64, 2, -1)
        c.q, c.cu = q.cpu(), cu.cpu().numpy()
        c.table = table[at].cpu().numpy()
        c.lens = lens[at].cpu().numpy()
        c.check(out.double().cpu().numpy(), what=(ids, new))

    feed([0, 1], [37, 70])
    feed([1], [50])
    src, dst = i32([0, 0]), i32([0, 0])
    kvq.kvq_fork_sequences(ref_count, table, lens, i32([0, 1]), i32([2, 3]),
                           src, dst, B, dev_error=err)
    kvq.kvq_copy_pages([kv], src, dst, dev_error=err)
    for _ in range(3):
        feed([0, 1, 2, 3], [1, 1, 1, 1])
    feed([2, 0], [5, 1])
    keep = list(range(64)) + [70, 90, 100, 121]
    a = torch.empty(68, dtype=torch.int64, device="cuda")
    b = torch.empty_like(a)
    kvq.kvq_compact_sequences(ref_count, table, lens, i32([3]), i32(keep),
                              i32([0, 68]), a, b, B, dev_error=err)
    # row 3 still shares its parent's pages: refused, nothing changed
    assert int(err.item()) == kvq.KVQ_DEVERR_REF
    err.zero_()
    kvq.kvq_free_sequences(ref_count, table, lens, i32([1]), dev_error=err)
    before = kv.clone()
    kvq.kvq_compact_sequences(ref_count, table, lens, i32([3]), i32(keep),
                              i32([0, 68]), a, b, B, dev_error=err)
    kvq.kvq_move_tokens_nvfp4([kv], a, b, i32([0, 68]), dev_error=err)
    c = Pages(64, B, H)
    for k in (a, b):
        assert bool((k >= 0).all())
    old, new = Pages(64, B, H), c
    old.data = before.cpu().numpy().reshape(64, 2, -1)
    new.data = kv.cpu().numpy().reshape(64, 2, -1)
    for s, d in zip(a.tolist(), b.tolist()):
        for side in range(2):
            assert np.array_equal(old.token(side, s // B, s % B),
                                  new.token(side, d // B, d % B))
    feed([3, 0], [20, 1])
    kvq.kvq_free_sequences(ref_count, table, lens, i32([0, 2, 3]),
                           dev_error=err)
    assert int(err.item()) == 0
    assert not bool(ref_count.any()) and bool((table == -1).all())
