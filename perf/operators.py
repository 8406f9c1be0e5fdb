"""The operators of the paged NVFP4 cache beside its stores, loads and decode
attention: attention of a chunk of new tokens over the pages, and the page
operators (page copies, growing, forking, compacting and freeing sequences).

``own`` false: the operators in elementary torch operations, in 32 bits.
``own`` true: the calls of ``paged_quantized_kv_gb300.kvq``.

A cache of one layer is uint8 [num_blocks, 2, H*B*72] (K side, V side; per
side the e2m1 data then the e4m3 group scales, head_size 128); the layers of
a model are stacked in front of it."""
import math

import torch

own = False

D = 128          # head_size
S = D // 16      # scale groups of a head row
ROW = D // 2     # data bytes of a head row
FULL = ROW + S


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # speculative decoding: five draft tokens of each sequence verified
        # at once over contexts of a chat load; latency counts
        dict(name="chunk_verify", op="chunk", seqs=8, q_lo=5, q_hi=5,
             ctx_lo=512, ctx_hi=2560, hq=64, hkv=8, block=16, nhd=False,
             f16=False, swz=False),
        # a continuous batch: most sequences decode one token while a few
        # bring a piece of prompt; odd lengths, three query heads to a KV
        # head, token-major pages, fp16
        dict(name="chunk_mixed_nhd_f16", op="chunk", seqs=24, q_lo=1,
             q_hi=257, ctx_lo=300, ctx_hi=2300, hq=24, hkv=8, block=32,
             nhd=True, f16=True, swz=True),
        # one piece of 2048 prompt tokens on top of 6144 cached ones
        dict(name="chunk_prefill", op="chunk", seqs=1, q_lo=2048, q_hi=2048,
             ctx_lo=8192, ctx_hi=8192, hq=64, hkv=8, block=16, nhd=False,
             f16=False, swz=False),
        # the last piece of a long document
        dict(name="chunk_long", op="chunk", seqs=1, q_lo=500, q_hi=500,
             ctx_lo=131000, ctx_hi=131000, hq=64, hkv=8, block=64,
             nhd=False, f16=False, swz=False),
        # copy-on-write of a few pages, every layer of a small model
        dict(name="copy_few", op="copy", layers=16, pairs=5, hkv=4, block=16),
        # defragmentation: a fifth of a large model's pages moved
        dict(name="copy_many", op="copy", layers=80, pairs=500, hkv=8,
             block=16),
        # two samples drawn from each of two prompts
        dict(name="fork_few", op="fork", layers=16, parents=2, per=2,
             len_lo=100, len_hi=900, hkv=4, block=16, spare=512),
        # four samples of each of 64 prompts
        dict(name="fork_many", op="fork", layers=32, parents=64, per=4,
             len_lo=500, len_hi=4000, hkv=8, block=16, spare=8192),
        # four prompts admitted into a small pool
        dict(name="extend_few", op="extend", seqs=4, new_lo=20, new_hi=400,
             block=16, spare=2048),
        # a full batch of prompts admitted into a large, fragmented pool
        dict(name="extend_many", op="extend", seqs=128, new_lo=100,
             new_hi=4000, block=16, spare=65536),
        # eviction in one sequence of a small model
        dict(name="compact_few", op="compact", layers=4, seqs=1,
             keep_lo=700, keep_hi=700, grow=100, sink=4, hkv=4, block=16,
             nhd=False),
        # eviction round of a batch: each sequence grows by 480 tokens and is
        # cut back to the tokens that it keeps, its first 64 among them
        dict(name="compact_many", op="compact", layers=32, seqs=16,
             keep_lo=1500, keep_hi=2500, grow=480, sink=64, hkv=8, block=16,
             nhd=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "copy", "fork", "extend",
                     "compact"])
    block = rng.choice([8, 16, 32, 64])
    if op == "chunk":
        while True:
            hkv = rng.choice([1, 2, 4, 8])
            hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
            q_hi = _log(rng, 1, 2100)
            q_lo = rng.choice([1, q_hi, max(1, q_hi // 2)])
            ctx_hi = _log(rng, max(q_hi, 16), 131000)
            ctx_lo = max(q_hi, _log(rng, 1, ctx_hi))
            seqs = _log(rng, 1, 40)
            if (seqs * q_hi * hq * ctx_hi <= 500 * 64 * 131000 // 2
                    and seqs * ctx_hi * hkv <= 8 * 131000):
                return dict(op=op, seqs=seqs, q_lo=q_lo, q_hi=q_hi,
                            ctx_lo=ctx_lo, ctx_hi=ctx_hi, hq=hq, hkv=hkv,
                            block=block, nhd=rng.random() < 0.4,
                            f16=rng.random() < 0.4, swz=rng.random() < 0.3)
    layers = _log(rng, 1, 48)
    hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "copy":
        return dict(op=op, layers=layers, pairs=_log(rng, 1, 400), hkv=hkv,
                    block=rng.choice([8, 16, 32]))
    if op == "fork":
        return dict(op=op, layers=min(layers, 32), parents=_log(rng, 1, 48),
                    per=rng.randint(1, 4), len_lo=_log(rng, 1, 500),
                    len_hi=_log(rng, 500, 3900), hkv=hkv,
                    block=rng.choice([16, 32]), spare=_log(rng, 300, 4096))
    if op == "extend":
        return dict(op=op, seqs=_log(rng, 1, 128), new_lo=_log(rng, 1, 90),
                    new_hi=_log(rng, 100, 3900), block=block,
                    spare=_log(rng, 1000, 60000))
    keep_lo = _log(rng, 100, 1500)
    return dict(op=op, layers=min(layers, 32), seqs=_log(rng, 1, 12),
                keep_lo=keep_lo, keep_hi=keep_lo + rng.randint(0, 900),
                grow=_log(rng, 8, 480), sink=rng.choice([0, 1, 4, 64]),
                hkv=hkv, block=rng.choice([16, 32]),
                nhd=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _rand(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    h = torch.Generator()
    h.manual_seed(int(seed) * 104729 + 17)
    return g, h


def _ints(lo, hi, n):
    """n whole numbers of [lo, hi], the lengths of a case: its own, whatever
    the seed, so that every seed means the same work."""
    h = torch.Generator()
    h.manual_seed(lo * 31 + hi * 17 + n)
    return torch.randint(lo, max(lo, hi) + 1, (n,), generator=h).tolist()


def _pages(g, num_blocks, hkv, block, nhd, swz):
    """NVFP4 pages of normal K and V rows, quantised in 16-element groups:
    uint8 [num_blocks, 2, hkv*block*72]."""
    out = torch.empty(num_blocks, 2, hkv * block * FULL, dtype=torch.uint8,
                      device="cuda")
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0],
                       device="cuda")
    step = max(1, (1 << 25) // (block * hkv * D))
    for at in range(0, num_blocks, step):
        n = min(step, num_blocks - at)
        for side in range(2):
            x = torch.randn(n, block, hkv, S, 16, device="cuda", generator=g)
            sf = (x.abs().amax(-1) / 6.0 * 64.0).to(torch.float8_e4m3fn)
            y = x * (64.0 / sf.float().clamp(min=2.0 ** -9))[..., None]
            code = (torch.bucketize(y.abs(), mid)
                    + (y < 0) * 8).to(torch.uint8)
            data = (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(
                n, block, hkv, ROW)
            sc = sf.view(torch.uint8)
            if side == 1 or swz:
                sc = sc.reshape(n, block // 4, 4, hkv, 4, S // 4).permute(
                    0, 1, 4, 3, 5, 2).reshape(n, block, hkv, S)
            if not nhd:
                data, sc = data.transpose(1, 2), sc.transpose(1, 2)
            out[at:at + n, side, :hkv * block * ROW] = data.reshape(n, -1)
            out[at:at + n, side, hkv * block * ROW:] = sc.reshape(n, -1)
    return out


def _pool(h, lens, rows, block, spare, width):
    """A pool of pages: `lens` tokens in its first rows, pages in random
    order, `spare` free ones; `rows` rows, the rest of them empty."""
    need = [-(-n // block) for n in lens]
    total = sum(need)
    blocks = total + spare
    perm = torch.randperm(blocks, generator=h)[:total].to(torch.int32)
    table = torch.full((rows, width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    ref = torch.zeros(blocks, dtype=torch.int32)
    ref[perm.long()] = 1
    full = torch.zeros(rows, dtype=torch.int32)
    full[:len(lens)] = torch.tensor(lens, dtype=torch.int32)
    return dict(table=table.cuda(), ref=ref.cuda(), lens=full.cuda(),
                blocks=blocks)


def _cu(counts):
    c = [0]
    for n in counts:
        c.append(c[-1] + n)
    return c


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _lens_of(case):
    """(query lengths, context lengths) of a chunk case."""
    n = case["seqs"]
    q = _ints(case["q_lo"], case["q_hi"], n)
    if case["q_lo"] == 1 and n > 2:
        # most sequences bring one token, one none, the rest long pieces
        q = [1 if i % 3 else v for i, v in enumerate(q)]
        q[0], q[1] = case["q_hi"], 0
    c = _ints(case["ctx_lo"], case["ctx_hi"], n)
    c[0] = case["ctx_hi"]
    return q, [max(a, b) for a, b in zip(q, c)]


def _raw_cache(g, layers, blocks, hkv, block):
    """Page bytes of every layer (any bytes: only moved, never read as
    numbers)."""
    return torch.randint(0, 256, (layers, blocks, 2, hkv * block * FULL),
                         dtype=torch.uint8, device="cuda", generator=g)


def prepare(case, seed):
    g, h = _rand(seed)
    op, B = case["op"], case["block"]
    s = dict(case=case)
    if op == "chunk":
        q_lens, ctx = _lens_of(case)
        pool = _pool(h, ctx, case["seqs"], B, 7,
                     max(1, max(-(-c // B) for c in ctx)))
        dt = torch.float16 if case["f16"] else torch.bfloat16
        s.update(
            query=torch.randn(sum(q_lens), case["hq"], D, device="cuda",
                              generator=g).to(dt),
            kv=_pages(g, pool["blocks"], case["hkv"], B, case["nhd"],
                      case["swz"]),
            table=pool["table"], lens=_i32(ctx), cu=_i32(_cu(q_lens)),
            max_q=max(q_lens), max_ctx=max(ctx),
            k_scale=torch.tensor([1.0 / 64.0], device="cuda"),
            v_scale=torch.tensor([1.0 / 64.0], device="cuda"),
            scale=1.0 / math.sqrt(D))
        s["out"] = torch.empty_like(s["query"])
    elif op == "copy":
        pairs = case["pairs"]
        blocks = 2 * pairs + pairs // 3 + 3
        perm = torch.randperm(blocks, generator=h)[:2 * pairs].to(torch.int32)
        s.update(cache=_raw_cache(g, case["layers"], blocks, case["hkv"], B),
                 src=perm[:pairs].cuda(), dst=perm[pairs:].cuda())
    elif op == "fork":
        n, per = case["parents"], case["per"]
        lens = _ints(case["len_lo"], case["len_hi"], n)
        s.update(_pool(h, lens, n + n * per, B, case["spare"],
                       -(-case["len_hi"] // B) + 4))
        s.update(parents=_i32([i for i in range(n) for _ in range(per)]),
                 children=_i32(list(range(n, n + n * per))),
                 copy_src=_i32([-1] * (n * per)),
                 copy_dst=_i32([-1] * (n * per)),
                 cache=_raw_cache(g, case["layers"], s["blocks"],
                                  case["hkv"], B))
    elif op == "extend":
        n = case["seqs"]
        new = _ints(case["new_lo"], case["new_hi"], n)
        # other sequences hold some of the pages, in random places
        other = _ints(1, 40 * B, 2 * n)
        spare = case["spare"] + sum(-(-v // B) for v in new)
        s.update(_pool(h, other, 3 * n, B, spare,
                       max(40, -(-case["new_hi"] // B)) + 4))
        s.update(ids=_i32(list(range(2 * n, 3 * n))), cu=_i32(_cu(new)),
                 slots=torch.empty(sum(new), dtype=torch.int64,
                                   device="cuda"))
    elif op == "compact":
        n, grow = case["seqs"], case["grow"]
        kept = _ints(case["keep_lo"], case["keep_hi"], n)
        keep = []
        for k in kept:
            rest = torch.randperm(k + grow - case["sink"],
                                  generator=h)[:k - case["sink"]]
            keep += list(range(case["sink"]))
            keep += (rest.sort().values + case["sink"]).tolist()
        s.update(_pool(h, kept, n, B, n * (-(-grow // B) + 1) + 5,
                       -(-(case["keep_hi"] + grow) // B) + 2))
        s.update(ids=_i32(list(range(n))),
                 cu_grow=_i32(_cu([grow] * n)), keep=_i32(keep),
                 cu_keep=_i32(_cu(kept)),
                 slots=torch.empty(n * grow, dtype=torch.int64,
                                   device="cuda"),
                 src=torch.empty(len(keep), dtype=torch.int64,
                                 device="cuda"),
                 dst=torch.empty(len(keep), dtype=torch.int64,
                                 device="cuda"),
                 cache=_raw_cache(g, case["layers"], s["blocks"],
                                  case["hkv"], B))
    else:
        raise ValueError(op)
    return s


def work(case):
    op, B = case["op"], case["block"]
    page = 2 * B * FULL * case.get("hkv", 0)
    if op == "chunk":
        q, c = _lens_of(case)
        seen = sum(n * (L - n) + n * (n + 1) // 2 for n, L in zip(q, c))
        pages = sum(L for n, L in zip(q, c) if n)
        return dict(bytes=2 * 2 * sum(q) * case["hq"] * D
                    + pages * case["hkv"] * 2 * FULL + 4 * pages // B,
                    flops=4 * D * case["hq"] * seen)
    if op == "copy":
        return dict(bytes=2 * case["pairs"] * case["layers"] * page, flops=0)
    if op == "fork":
        lens = _ints(case["len_lo"], case["len_hi"], case["parents"])
        ends = sum(1 for n in lens if n % B) * case["per"]
        # a child's row is read and written, its pages' counts too, when it
        # is freed and when it is forked; the counts are searched once
        row = sum(-(-n // B) for n in lens) * case["per"] * 4
        return dict(bytes=2 * ends * case["layers"] * page + 8 * row
                    + 4 * case["spare"], flops=0)
    if op == "extend":
        new = _ints(case["new_lo"], case["new_hi"], case["seqs"])
        pages = sum(-(-v // B) for v in new)
        return dict(bytes=8 * sum(new) + 2 * 4 * 4 * pages
                    + 4 * case["spare"], flops=0)
    kept = _ints(case["keep_lo"], case["keep_hi"], case["seqs"])
    moved = sum(k - case["sink"] for k in kept)
    return dict(bytes=moved * (2 * case["layers"] * case["hkv"] * 2 * FULL
                               + 4 + 16), flops=0)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_rows(side, table, block, hkv, nhd, swizzled, tokens):
    """Rows of `tokens` positions of every sequence, dequantised but for the
    tensor's own scale: fp32 [seqs, hkv, tokens, D]."""
    dev = side.device
    n = table.size(0)
    pos = torch.arange(tokens, device=dev)
    off = pos % block
    blk = table[:, pos // block].long().clamp(min=0)           # [n, T]
    flat = side.reshape(side.size(0), -1)                       # [nb, bytes]
    hs = torch.arange(hkv, device=dev)
    if nhd:
        base = off[:, None] * hkv * ROW + hs[None, :] * ROW
    else:
        base = hs[None, :] * block * ROW + off[:, None] * ROW   # [T, hkv]
    col = base[..., None] + torch.arange(ROW, device=dev)       # [T, hkv, 64]
    data = flat[blk[:, :, None, None], col[None]].int()
    j = torch.arange(S, device=dev)
    if swizzled:
        row = (off[:, None] // 4) * 4 + j // (S // 4)           # [T, S]
        at = (j % (S // 4)) * 4 + off[:, None] % 4
    else:
        row = off[:, None].expand(tokens, S)
        at = j[None].expand(tokens, S)
    if nhd:
        spot = row[:, None] * hkv * S + hs[None, :, None] * S + at[:, None]
    else:
        spot = hs[None, :, None] * block * S + row[:, None] * S + at[:, None]
    sc = flat[blk[:, :, None, None], hkv * block * ROW + spot[None]]
    sf = sc.contiguous().view(torch.float8_e4m3fn).float()      # [n,T,hkv,S]
    e2m1 = torch.tensor([0., .5, 1., 1.5, 2., 3., 4., 6., -0., -.5, -1.,
                         -1.5, -2., -3., -4., -6.], device=dev)
    x = torch.stack([e2m1[data & 15], e2m1[data >> 4]], -1)
    x = x.reshape(n, tokens, hkv, S, 16) * sf[..., None]
    return x.reshape(n, tokens, hkv, D).transpose(1, 2)


def _plain_chunk(s):
    c = s["case"]
    hq, hkv, B = c["hq"], c["hkv"], c["block"]
    G, n, T, Q = hq // hkv, c["seqs"], s["max_ctx"], s["max_q"]
    dev = s["query"].device
    k = _plain_rows(s["kv"][:, 0], s["table"], B, hkv, c["nhd"], c["swz"], T)
    start = s["cu"][:-1].long()
    q_len = s["cu"][1:].long() - start
    j = torch.arange(Q, device=dev)
    live = j[None] < q_len[:, None]                             # [n, Q]
    row = (start[:, None] + j[None]) * live
    q = s["query"].float()[row].reshape(n, Q, hkv, G, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(n, hkv, Q * G, D)
    x = torch.matmul(q, k.transpose(2, 3)) * (s["k_scale"] * s["scale"])
    del k
    p = s["lens"].long()[:, None] - q_len[:, None] + j[None]    # positions
    p = torch.where(live, p, -1).repeat_interleave(G, 1)        # [n, Q*G]
    t = torch.arange(T, device=dev)
    x.masked_fill_((t[None, None] > p[..., None])[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = x.sum(-1, keepdim=True)
    v = _plain_rows(s["kv"][:, 1], s["table"], B, hkv, c["nhd"], True, T)
    o = torch.matmul(x, v) * s["v_scale"]
    o = torch.where(total > 0, o / total, 0.0)
    o = o.reshape(n, hkv, Q, G, D).transpose(1, 2).reshape(n, Q, hq, D)
    out = s["out"]
    out[row[live]] = o[live].to(out.dtype)
    return out


def _plain_copy(cache, src, dst):
    live = (src >= 0) & (dst >= 0)
    cache[:, dst[live].long()] = cache[:, src[live].long()]


def _plain_free(s, ids):
    ids = ids.long()
    rows = s["table"][ids]
    pages = rows[rows >= 0].long()
    s["ref"].index_add_(0, pages, torch.full_like(pages, -1,
                                                  dtype=torch.int32))
    s["table"][ids] = -1
    s["lens"][ids] = 0


def _plain_extend(s, ids, cu, slots, B):
    dev = slots.device
    ids, cu = ids.long(), cu.long()
    old, new = s["lens"][ids].long(), cu[1:] - cu[:-1]
    have = (old + B - 1) // B
    need = (old + new + B - 1) // B - have
    end = need.cumsum(0)
    pages = (s["ref"] == 0).nonzero()[:, 0]
    r = torch.arange(int(end[-1]), device=dev)
    i = torch.searchsorted(end, r, right=True)
    pages = pages[:r.numel()]
    s["table"][ids[i], have[i] + r - (end - need)[i]] = pages.int()
    s["ref"][pages] = 1
    t = torch.arange(slots.numel(), device=dev)
    i = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = old[i] + t - cu[i]
    slots.copy_(s["table"][ids[i], pos // B].long() * B + pos % B)
    s["lens"][ids] = (old + new).int()


def _plain_fork(s, B):
    par, chi = s["parents"].long(), s["children"].long()
    lens = s["lens"][par].long()
    full, part = lens // B, lens % B > 0
    rows = s["table"][par]
    at = torch.arange(rows.size(1), device=rows.device)
    shared = at[None] < full[:, None]
    pages = rows[shared].long()
    new = (s["ref"] == 0).nonzero()[:, 0][:int(part.sum())].int()
    s["ref"].index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))
    s["ref"][new.long()] = 1
    kids = torch.where(shared, rows, -1)
    src = torch.full_like(s["copy_src"], -1)
    dst = torch.full_like(s["copy_dst"], -1)
    src[part] = rows[part, full[part]]
    dst[part] = new
    kids[part, full[part]] = new
    s["table"][chi] = kids
    s["lens"][chi] = lens.int()
    s["copy_src"].copy_(src)
    s["copy_dst"].copy_(dst)


def _plain_compact(s, B):
    dev = s["keep"].device
    ids, cu = s["ids"].long(), s["cu_keep"].long()
    t = torch.arange(s["keep"].numel(), device=dev)
    i = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = t - cu[i]
    old = s["keep"].long()
    s["src"].copy_(s["table"][ids[i], old // B].long() * B + old % B)
    s["dst"].copy_(s["table"][ids[i], pos // B].long() * B + pos % B)
    kept = cu[1:] - cu[:-1]
    rows = s["table"][ids]
    gone = (torch.arange(rows.size(1), device=dev)[None]
            >= ((kept + B - 1) // B)[:, None]) & (rows >= 0)
    pages = rows[gone].long()
    s["ref"].index_add_(0, pages, torch.full_like(pages, -1,
                                                  dtype=torch.int32))
    s["table"][ids] = torch.where(gone, -1, rows)
    s["lens"][ids] = kept.int()


def _token_bytes(off, block, hkv, nhd):
    """Places of a token's bytes in a page, both sides: [tokens, hkv*144]."""
    dev = off.device
    hs = torch.arange(hkv, device=dev)
    off = off[:, None, None]
    d = torch.arange(ROW, device=dev)
    j = torch.arange(S, device=dev)
    h = hs[None, :, None]
    data = (off * hkv + h) * ROW + d if nhd else (h * block + off) * ROW + d
    row = (off // 4) * 4 + j // (S // 4)
    col = (j % (S // 4)) * 4 + off % 4
    end = hkv * block * ROW
    if nhd:
        k_sc, v_sc = (off * hkv + h) * S + j, (row * hkv + h) * S + col
    else:
        k_sc, v_sc = (h * block + off) * S + j, (h * block + row) * S + col
    side = hkv * block * FULL
    return torch.cat([data, end + k_sc, side + data, side + end + v_sc],
                     -1).flatten(1)


def _plain_move(s, B, hkv, nhd):
    src, dst = s["src"], s["dst"]
    flat = s["cache"].flatten(2)                   # [layers, blocks, bytes]
    x = flat[:, (src // B)[:, None], _token_bytes(src % B, B, hkv, nhd)]
    flat[:, (dst // B)[:, None], _token_bytes(dst % B, B, hkv, nhd)] = x


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _views(kv, hkv, block, nhd):
    """The two sides of a cache as [blocks, block, heads, 72] views."""
    if nhd:
        v = kv.view(kv.size(0), 2, block, hkv, FULL)
        return v[:, 0], v[:, 1]
    v = kv.view(kv.size(0), 2, hkv, block, FULL).transpose(2, 3)
    return v[:, 0], v[:, 1]


def run(s):
    c = s["case"]
    op, B = c["op"], c["block"]
    if own:
        from paged_quantized_kv_gb300 import kvq
    if op == "chunk":
        if not own:
            return _plain_chunk(s)
        if "workspace" not in s:  # kept by the program from call to call
            s["workspace"] = kvq.chunk_attention_workspace(s["out"].device)
        kc, vc = _views(s["kv"], c["hkv"], B, c["nhd"])
        kvq.kvq_chunk_attention_nvfp4(
            s["query"], kc, vc, s["table"], s["cu"], s["lens"], s["k_scale"],
            s["v_scale"], s["scale"], s["out"], s["max_q"],
            workspace=s["workspace"],
            flags=kvq.KVQ_F_SWIZZLE_K_SCALE if c["swz"] else 0)
        return s["out"]
    if op == "copy":
        if own:
            kvq.kvq_copy_pages(s["cache"], s["src"], s["dst"])
        else:
            _plain_copy(s["cache"], s["src"], s["dst"])
        return s["cache"]
    if op == "fork":
        # the samples of the last round are dropped, new ones forked
        if own:
            kvq.kvq_free_sequences(s["ref"], s["table"], s["lens"],
                                   s["children"])
            kvq.kvq_fork_sequences(s["ref"], s["table"], s["lens"],
                                   s["parents"], s["children"],
                                   s["copy_src"], s["copy_dst"], B)
            kvq.kvq_copy_pages(s["cache"], s["copy_src"], s["copy_dst"])
        else:
            _plain_free(s, s["children"])
            _plain_fork(s, B)
            _plain_copy(s["cache"], s["copy_src"], s["copy_dst"])
        return dict(ref=s["ref"], table=s["table"], lens=s["lens"],
                    src=s["copy_src"], dst=s["copy_dst"], cache=s["cache"])
    if op == "extend":
        # finished sequences leave, new prompts take their rows
        if own:
            kvq.kvq_free_sequences(s["ref"], s["table"], s["lens"], s["ids"])
            kvq.kvq_extend_sequences(s["ref"], s["table"], s["lens"],
                                     s["ids"], s["cu"], s["slots"], B)
        else:
            _plain_free(s, s["ids"])
            _plain_extend(s, s["ids"], s["cu"], s["slots"], B)
        return dict(ref=s["ref"], table=s["table"], lens=s["lens"],
                    slots=s["slots"])
    # sequences grow, then keep the tokens of their lists
    if own:
        kvq.kvq_extend_sequences(s["ref"], s["table"], s["lens"], s["ids"],
                                 s["cu_grow"], s["slots"], B)
        kvq.kvq_compact_sequences(s["ref"], s["table"], s["lens"], s["ids"],
                                  s["keep"], s["cu_keep"], s["src"],
                                  s["dst"], B)
        kv = s["cache"]
        shape = (B, c["hkv"]) if c["nhd"] else (c["hkv"], B)
        kvq.kvq_move_tokens_nvfp4(
            kv.view(kv.size(0), kv.size(1), 2, *shape, FULL), s["src"],
            s["dst"], s["cu_keep"],
            layout=kvq.KVQ_LAYOUT_NHD if c["nhd"] else kvq.KVQ_LAYOUT_HND)
    else:
        _plain_extend(s, s["ids"], s["cu_grow"], s["slots"], B)
        _plain_compact(s, B)
        _plain_move(s, B, c["hkv"], c["nhd"])
    return dict(ref=s["ref"], table=s["table"], lens=s["lens"],
                slots=s["slots"], src=s["src"], dst=s["dst"],
                cache=s["cache"])


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] != "chunk":
        return None  # whole numbers and bytes only
    s = prepare(case, seed)
    hq, hkv, B = case["hq"], case["hkv"], case["block"]
    G = hq // hkv
    q_len = s["cu"].diff().tolist()
    if sum(n * c for n, c in zip(q_len, s["lens"].tolist())) * hq > 5e9:
        return None
    lut = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64,
                       device="cuda") / 2
    lut = torch.cat([lut, -lut])
    out = torch.zeros(s["query"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, n in enumerate(q_len):
        L = int(s["lens"][b])
        if n and L:
            ids = s["table"][b, :-(-L // B)].long()
            rows = []
            for side in range(2):
                page = s["kv"][ids, side]
                nb = page.size(0)
                cut = hkv * B * ROW
                data = page[:, :cut]
                sc = page[:, cut:].contiguous().view(
                    torch.float8_e4m3fn).double()
                if case["nhd"]:
                    data = data.reshape(nb, B, hkv, ROW)
                    sc = sc.reshape(nb, B, hkv, S)
                else:
                    data = data.reshape(nb, hkv, B, ROW).transpose(1, 2)
                    sc = sc.reshape(nb, hkv, B, S).transpose(1, 2)
                if side or case["swz"]:
                    # tile [quads, 4 rows a, heads, S/4 columns c, 4 r]:
                    # group a * S/4 + c of token 4 * quad + r
                    sc = sc.reshape(nb, B // 4, 4, hkv, S // 4, 4).permute(
                        0, 1, 5, 3, 2, 4).reshape(nb, B, hkv, S)
                x = torch.stack([lut[(data & 15).long()],
                                 lut[(data >> 4).long()]], -1)
                x = x.reshape(nb, B, hkv, S, 16) * sc[..., None]
                x = x.reshape(nb * B, hkv, D)[:L]
                rows.append(x * float((s["k_scale"], s["v_scale"])[side]))
            last = torch.arange(n, device="cuda") + (L - n)
            hide = torch.arange(L, device="cuda")[None] > last[:, None]
            for h in range(hq):
                q = s["query"][at:at + n, h].double()
                x = (q @ rows[0][:, h // G].t()) * s["scale"]
                x = torch.softmax(x.masked_fill(hide, -math.inf), -1)
                out[at:at + n, h] = x @ rows[1][:, h // G]
        at += n
    return out
