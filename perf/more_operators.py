"""Sparse attention over the blocks that the indexer's scores select, and
attention of a tree of drafted tokens, over the paged caches: quantising the
indexer's queries, scoring blocks over the indexer-K cache, selecting blocks
of each query, attention over the selected blocks of the NVFP4 pages, and
attention under a mask among the newest tokens.

``own`` false: the operators in elementary torch operations, in 32 bits.
``own`` true: the calls of ``paged_quantized_kv_gb300.kvq``.

An NVFP4 cache of one layer is uint8 [num_blocks, 2, H*B*72] (K side, V side;
per side the e2m1 data then the e4m3 group scales, head_size 128), an indexer
cache uint8 [num_blocks, B*D + B*4] (e4m3 rows, then their fp32 scales)."""
import math

import torch

own = False

D = 128          # head_size and the indexer's head_dim
S = D // 16      # scale groups of a head row
ROW = D // 2     # data bytes of a head row
FULL = ROW + S


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the indexer's queries of one decode step of a small batch
        dict(name="quant_step", op="quant", rows=8, heads=32, f16=False),
        # those of a batch of prompt pieces
        dict(name="quant_prompt", op="quant", rows=6000, heads=64, f16=True),
        # block scores of one decode step of a few chats; latency counts
        dict(name="score_step", op="score", seqs=4, q_lo=1, q_hi=1,
             ctx_lo=700, ctx_hi=4000, heads=32, block=64, sel=64),
        # a large batch of long contexts, one or two tokens each; odd
        # lengths, small blocks
        dict(name="score_batch", op="score", seqs=48, q_lo=1, q_hi=2,
             ctx_lo=9001, ctx_hi=33333, heads=64, block=64, sel=32),
        # a piece of a prompt on top of a long context
        dict(name="score_prompt", op="score", seqs=1, q_lo=1024, q_hi=1024,
             ctx_lo=24576, ctx_hi=24576, heads=64, block=64, sel=64),
        # the blocks of one decode step
        dict(name="select_step", op="select", seqs=8, q_lo=1, q_hi=1,
             ctx_lo=3000, ctx_hi=30000, sel=64, top=16, first=1, last=2),
        # those of every token of two long prompts' pieces
        dict(name="select_prompt", op="select", seqs=2, q_lo=2048, q_hi=2048,
             ctx_lo=100000, ctx_hi=131072, sel=64, top=32, first=1, last=2),
        # one decode step of a batch of long contexts, 2048 tokens each
        dict(name="sparse_step", op="sparse", seqs=64, q_lo=1, q_hi=1,
             ctx_lo=5000, ctx_hi=16384, hq=64, hkv=8, block=16, nhd=False,
             f16=False, swz=False, sel=64, top=32),
        # a few drafts and pieces of odd lengths; token-major pages, three
        # query heads to a KV head, fp16
        dict(name="sparse_mixed_nhd_f16", op="sparse", seqs=12, q_lo=1,
             q_hi=33, ctx_lo=500, ctx_hi=9000, hq=24, hkv=8, block=32,
             nhd=True, f16=True, swz=True, sel=32, top=20),
        # a piece of a prompt on top of a long context
        dict(name="sparse_prompt", op="sparse", seqs=1, q_lo=1024,
             q_hi=1024, ctx_lo=32768, ctx_hi=32768, hq=64, hkv=8, block=16,
             nhd=False, f16=False, swz=False, sel=64, top=32),
        # speculative decoding: small trees of drafts over chats
        dict(name="tree_few", op="tree", seqs=6, q_lo=7, q_hi=16,
             ctx_lo=300, ctx_hi=2000, hq=32, hkv=8, block=16, nhd=False,
             f16=False, swz=False),
        # large trees for a batch, odd sizes
        dict(name="tree_many", op="tree", seqs=32, q_lo=33, q_hi=64,
             ctx_lo=2000, ctx_hi=8000, hq=64, hkv=8, block=16, nhd=False,
             f16=False, swz=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "score", "score", "select", "sparse", "sparse",
                     "tree", "tree"])
    f16 = rng.random() < 0.4
    if op == "quant":
        heads = rng.choice([1, 4, 12, 16, 32, 64])
        return dict(op=op, rows=_log(rng, 1, 6000 * 64 // heads // 2),
                    heads=heads, f16=f16)
    while True:
        seqs = _log(rng, 1, 48)
        q_hi = _log(rng, 1, 1024)
        q_lo = rng.choice([1, q_hi, max(1, q_hi // 2)])
        ctx_hi = _log(rng, max(q_hi, 16), 60000)
        ctx_lo = max(q_hi, _log(rng, 1, ctx_hi))
        c = dict(op=op, seqs=seqs, q_lo=q_lo, q_hi=q_hi, ctx_lo=ctx_lo,
                 ctx_hi=ctx_hi)
        pairs = seqs * q_hi * ctx_hi
        if op == "score":
            c.update(heads=rng.choice([8, 16, 24, 32, 48, 64]),
                     block=rng.choice([16, 32, 64, 128]),
                     sel=rng.choice([16, 32, 64, 128]))
            if (pairs * c["heads"] <= 1024 * 64 * 24576
                    and seqs * ctx_hi <= 48 * 30000):
                return c
            continue
        if op == "select":
            c.update(sel=rng.choice([16, 32, 64, 128]),
                     top=_log(rng, 1, 100), first=rng.choice([0, 0, 1]),
                     last=rng.choice([0, 1, 2]))
            c["top"] = max(c["top"], c["first"] + c["last"], 1)
            if pairs <= 2 * 2048 * 131072 // 64 * c["sel"]:
                return c
            continue
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        c.update(hq=hq, hkv=hkv, block=rng.choice([8, 16, 32, 64]),
                 nhd=rng.random() < 0.4, f16=f16, swz=rng.random() < 0.3)
        if seqs * ctx_hi * hkv > 64 * 16384 * 8:
            continue
        if op == "tree":
            c["q_hi"] = _log(rng, 1, min(128, q_hi))
            c["q_lo"] = rng.choice([1, c["q_hi"], max(1, c["q_hi"] // 2)])
            if seqs * c["q_hi"] * hq * ctx_hi <= 32 * 64 * 64 * 8000 // 2:
                return c
            continue
        c.update(sel=c["block"] * rng.choice([1, 2, 4]),
                 top=_log(rng, 1, 64))
        if (pairs * hq <= 1024 * 64 * 32768
                and seqs * q_hi * hq * min(c["sel"] * c["top"], ctx_hi)
                <= 1024 * 64 * 2048):
            return c


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


def _lens_of(case):
    """(query lengths, context lengths) of a case."""
    n = case["seqs"]
    q = _ints(case["q_lo"], case["q_hi"], n)
    if case["q_lo"] == 1 and case["q_hi"] > 8 and n > 2:
        # most sequences bring one token, one none, the rest long pieces
        q = [1 if i % 3 else v for i, v in enumerate(q)]
        q[0], q[1] = case["q_hi"], 0
    c = _ints(case["ctx_lo"], case["ctx_hi"], n)
    c[0] = case["ctx_hi"]
    return q, [max(a, b) for a, b in zip(q, c)]


def _seen_of(case):
    """Tokens that each query row sees, row by row."""
    return [L - n + i + 1 for n, L in zip(*_lens_of(case)) for i in range(n)]


def _table(h, lens, block, spare):
    """Block table of sequences on distinct pages in random order."""
    need = [-(-n // block) for n in lens]
    perm = torch.randperm(sum(need) + spare, generator=h).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table.cuda(), sum(need) + spare


def _cu(counts):
    return torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


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


def _indexer_pages(g, num_blocks, block):
    """Indexer-K blocks of normal rows: e4m3 with one scale per token."""
    out = torch.empty(num_blocks, block * (D + 4), dtype=torch.uint8,
                      device="cuda")
    x = torch.randn(num_blocks, block, D, device="cuda", generator=g)
    sf = x.abs().amax(-1) / 448.0
    q = (x / sf[..., None]).to(torch.float8_e4m3fn)
    out[:, :block * D] = q.view(torch.uint8).reshape(num_blocks, -1)
    out[:, block * D:] = sf.view(torch.uint8).reshape(num_blocks, -1)
    return out


def _choose(g, case, seen):
    """Lists of selected blocks as a model makes them: the first block, the
    row's last one, and the best of scores that nearby rows share in part;
    rising, -1 behind the last.  int32 [rows, top]."""
    sel, top = case["sel"], case["top"]
    rows, width = seen.numel(), -(-case["ctx_hi"] // case["sel"])
    nb = (seen + sel - 1) // sel
    a = torch.randn(width, device="cuda", generator=g)
    c = torch.randn(rows // 128 + 1, width, device="cuda", generator=g)
    x = a + c.repeat_interleave(128, 0)[:rows] + 0.5 * torch.randn(
        rows, width, device="cuda", generator=g)
    at = torch.arange(width, device="cuda")
    x = torch.where(at == 0, 50.0, x)
    x = torch.where(at == nb[:, None] - 1, 100.0, x)
    x = torch.where(at < nb[:, None], x, -math.inf)
    k = min(top, width)
    val, idx = x.topk(k, dim=1)
    idx = torch.where(val > -math.inf, idx, width).sort(1).values
    out = torch.full((rows, top), -1, dtype=torch.int32, device="cuda")
    out[:, :k] = torch.where(idx < width, idx, -1).int()
    return out


def _tree_masks(h, q_lens):
    """A tree of drafts for each sequence (each token's parent is one of the
    eight before it, or the root), as the bits of the drafts that each one
    sees: its ancestors and itself.  int32 [rows, words]."""
    words = -(-max(q_lens) // 32)
    out = []
    for n in q_lens:
        back = torch.randint(1, 9, (max(n, 1),), generator=h).tolist()
        bits = []
        for i in range(n):
            up = i - back[i]
            bits.append((bits[up] if up >= 0 else 0) | (1 << i))
        out += [[(v >> (32 * w)) & 0xFFFFFFFF for w in range(words)]
                for v in bits]
    t = torch.tensor(out, dtype=torch.int64).reshape(-1, words)
    return torch.where(t >= 1 << 31, t - (1 << 32), t).to(torch.int32).cuda()


def prepare(case, seed):
    g, h = _rand(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "quant":
        rows, heads = case["rows"], case["heads"]
        s.update(q=torch.randn(rows, heads, D, device="cuda", generator=g).to(
                     torch.float16 if case["f16"] else torch.bfloat16),
                 weights=torch.randn(rows, heads, device="cuda", generator=g),
                 scale=1.0 / math.sqrt(D * heads),
                 q_fp8=torch.empty(rows, heads, D, device="cuda",
                                   dtype=torch.float8_e4m3fn),
                 w_out=torch.empty(rows, heads, device="cuda"))
        return s
    q_lens, ctx = _lens_of(case)
    total = sum(q_lens)
    s.update(lens=_i32(ctx), cu=_cu(q_lens), max_q=max(q_lens),
             max_ctx=max(ctx))
    seen = torch.tensor(_seen_of(case), device="cuda")
    if op in ("score", "select"):
        width = -(-max(ctx) // case["sel"])
    if op == "score":
        s["table"], blocks = _table(h, ctx, case["block"], 5)
        q = torch.randn(total, case["heads"], D, device="cuda", generator=g)
        sf = q.abs().amax(-1) / 448.0
        s.update(
            q_fp8=(q / sf[..., None]).to(torch.float8_e4m3fn),
            weights=sf * torch.randn(total, case["heads"], device="cuda",
                                     generator=g)
            / math.sqrt(D * case["heads"]),
            cache=_indexer_pages(g, blocks, case["block"]),
            scores=torch.empty(total, width, device="cuda"))
    elif op == "select":
        # (on a grid: equal scores occur)
        x = torch.randn(total, width, device="cuda", generator=g)
        s.update(scores=torch.round(x * 64.0) / 64.0,
                 selected=torch.empty(total, case["top"], dtype=torch.int32,
                                      device="cuda"))
    else:
        dt = torch.float16 if case["f16"] else torch.bfloat16
        s["table"], blocks = _table(h, ctx, case["block"], 5)
        s.update(
            query=torch.randn(total, case["hq"], D, device="cuda",
                              generator=g).to(dt),
            kv=_pages(g, blocks, case["hkv"], case["block"], case["nhd"],
                      case["swz"]),
            k_scale=torch.tensor([1.0 / 64.0], device="cuda"),
            v_scale=torch.tensor([1.0 / 64.0], device="cuda"),
            scale=1.0 / math.sqrt(D))
        s["out"] = torch.empty_like(s["query"])
        if op == "sparse":
            s["selected"] = _choose(g, case, seen)
        else:
            s["mask"] = _tree_masks(h, q_lens)
    return s


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["rows"] * case["heads"]
        return dict(bytes=n * (2 * D + 4 + D + 4), flops=2 * n * D)
    q, c = _lens_of(case)
    seen = _seen_of(case)
    pages = sum(L for n, L in zip(q, c) if n)
    if op == "score":
        width = -(-max(c) // case["sel"])
        return dict(bytes=pages * (D + 4) + 4 * sum(q) * width
                    + sum(q) * case["heads"] * (D + 4)
                    + 4 * pages // case["block"],
                    flops=2 * case["heads"] * D * sum(seen))
    if op == "select":
        return dict(bytes=4 * sum(-(-v // case["sel"]) for v in seen)
                    + 4 * sum(q) * case["top"], flops=0)
    rows = 2 * 2 * sum(q) * case["hq"] * D
    token = case["hkv"] * 2 * FULL
    if op == "tree":
        return dict(bytes=rows + pages * token + 4 * pages // case["block"]
                    + 4 * sum(q) * -(-max(q) // 32),
                    flops=4 * D * case["hq"] * sum(seen))
    used = [min(v, case["sel"] * case["top"]) for v in seen]
    # a sequence's pages are read once at most, whatever its rows share
    at, read = 0, 0
    for n, L in zip(q, c):
        read += min(L, sum(used[at:at + n]))
        at += n
    return dict(bytes=rows + read * token + 4 * sum(q) * case["top"],
                flops=4 * D * case["hq"] * sum(used))


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_quant(s):
    x = s["q"].float()
    sf = x.abs().amax(-1) / 448.0
    y = x / torch.where(sf > 0, sf, 1.0)[..., None]
    s["q_fp8"].copy_(y)
    s["w_out"].copy_(s["weights"] * s["scale"] * sf)
    return s["q_fp8"], s["w_out"]


def _grid(s):
    """Rows of the queries as [sequences, longest]: their index (0 where
    there is none), whether there is one, the tokens that it sees."""
    start = s["cu"][:-1].long()
    q_len = s["cu"][1:].long() - start
    j = torch.arange(s["max_q"], device=start.device)
    live = j[None] < q_len[:, None]
    row = (start[:, None] + j[None]) * live
    seen = s["lens"].long()[:, None] - q_len[:, None] + j[None] + 1
    return row, live, torch.where(live, seen, 0)


def _plain_score(s):
    c = s["case"]
    B, sel, T = c["block"], c["sel"], s["max_ctx"]
    blk = s["table"].long().clamp(min=0)
    data = s["cache"][:, :B * D].contiguous().view(torch.float8_e4m3fn)
    sf = s["cache"][:, B * D:].contiguous().view(torch.float32)
    k = data.reshape(-1, B, D).float()[blk].flatten(1, 2)[:, :T]
    sf = sf[blk].flatten(1, 2)[:, None, :T]
    row, live, seen = _grid(s)
    n, Q = row.shape
    q = s["q_fp8"].float()[row].flatten(1, 2)          # [n, Q*heads, D]
    x = torch.matmul(q, k.transpose(1, 2)).relu_()
    x = x.reshape(n, Q, c["heads"], -1)
    x = torch.matmul(s["weights"][row][:, :, None], x)[:, :, 0] * sf
    t = torch.arange(x.size(2), device=x.device)
    x = torch.where(t < seen[..., None], x, -math.inf)
    width = s["scores"].size(1)
    x = torch.cat([x, x.new_full((n, Q, width * sel - x.size(2)),
                                 -math.inf)], 2)
    x = x.reshape(n, Q, width, sel).amax(-1)
    s["scores"][row[live]] = x[live]
    return s["scores"]


def _plain_select(s):
    c = s["case"]
    x, top, width = s["scores"], c["top"], s["scores"].size(1)
    row, live, seen = _grid(s)
    nb = torch.zeros_like(x[:, 0], dtype=torch.long)
    nb[row[live]] = (seen[live] + c["sel"] - 1) // c["sel"]
    nb = nb[:, None]
    at = torch.arange(width, device=x.device)
    always = (at < c["first"]) | (at >= nb - c["last"])
    x = torch.where(always, math.inf, x)
    x = torch.where(at < nb, x, -math.inf)
    idx = x.sort(dim=1, descending=True, stable=True).indices[:, :top]
    idx = torch.where(idx < nb, idx, width).sort(1).values
    out = torch.where(idx < width, idx, -1).int()
    s["selected"].fill_(-1)
    s["selected"][:, :out.size(1)] = out
    return s["selected"]


def _plain_pages(side, block, hkv, nhd, swizzled):
    """Every page dequantised but for the tensor's own scale: fp32 [blocks,
    block, hkv, D]."""
    nb, cut = side.size(0), hkv * block * ROW
    data = side[:, :cut]
    sf = side[:, cut:].contiguous().view(torch.float8_e4m3fn).float()
    if nhd:
        data = data.reshape(nb, block, hkv, ROW)
        sf = sf.reshape(nb, block, hkv, S)
    else:
        data = data.reshape(nb, hkv, block, ROW).transpose(1, 2)
        sf = sf.reshape(nb, hkv, block, S).transpose(1, 2)
    if swizzled:
        sf = sf.reshape(nb, block // 4, 4, hkv, S // 4, 4).permute(
            0, 1, 5, 3, 2, 4).reshape(nb, block, hkv, S)
    e2m1 = torch.tensor([0., .5, 1., 1.5, 2., 3., 4., 6., -0., -.5, -1.,
                         -1.5, -2., -3., -4., -6.], device=side.device)
    x = torch.stack([e2m1[(data & 15).int()], e2m1[(data >> 4).int()]], -1)
    x = x.reshape(nb, block, hkv, S, 16) * sf[..., None]
    return x.reshape(nb, block, hkv, D)


def _plain_attention(s, row, live, see):
    """Attention of the rows [n, Q] over the tokens that `see` [n, Q, T]
    marks."""
    c = s["case"]
    hq, hkv, T = c["hq"], c["hkv"], s["max_ctx"]
    G, (n, Q) = hq // hkv, row.shape
    blk = s["table"].long().clamp(min=0)
    k = _plain_pages(s["kv"][:, 0], c["block"], hkv, c["nhd"], c["swz"])
    k = k[blk].flatten(1, 2)[:, :T].permute(0, 2, 3, 1)   # [n, hkv, D, T]
    q = s["query"].float()[row].reshape(n, Q, hkv, G, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(n, hkv, Q * G, D)
    x = torch.matmul(q, k).mul_(s["k_scale"] * s["scale"])
    del k
    x = x.reshape(n, hkv, Q, G, T)
    x.masked_fill_(~see[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = x.sum(-1, keepdim=True)
    v = _plain_pages(s["kv"][:, 1], c["block"], hkv, c["nhd"], True)
    v = v[blk].flatten(1, 2)[:, :T].transpose(1, 2)       # [n, hkv, T, D]
    o = torch.matmul(x.reshape(n, hkv, Q * G, T), v) * s["v_scale"]
    o = o.reshape(n, hkv, Q, G, D)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 2, 1, 3, 4).reshape(n, Q, hq, D)
    s["out"][row[live]] = o[live].to(s["out"].dtype)
    return s["out"]


def _plain_sparse(s):
    sel, T = s["case"]["sel"], s["max_ctx"]
    row, live, seen = _grid(s)
    lists, dev = s["selected"].long(), row.device
    width = -(-T // sel)
    mark = torch.zeros(lists.size(0), width + 1, dtype=torch.bool, device=dev)
    mark.scatter_(1, torch.where(lists >= 0, lists, width), True)
    t = torch.arange(T, device=dev)
    see = mark[row][..., t // sel] & (t < seen[..., None])
    return _plain_attention(s, row, live, see)


def _plain_tree(s):
    row, live, seen = _grid(s)
    q_len = live.sum(1)
    T, dev = s["max_ctx"], row.device
    # the draft that each token of the context is, below 0: none
    j = (torch.arange(T, device=dev)[None]
         - (s["lens"].long() - q_len)[:, None])            # [n, T]
    word = s["mask"].long()[row]                           # [n, Q, words]
    at = (j // 32).clamp(0, word.size(2) - 1)
    bit = (word.gather(2, at[:, None].expand(-1, row.size(1), -1))
           >> (j % 32)[:, None]) & 1
    see = (j < 0)[:, None] | ((bit == 1) & (j < q_len[:, None])[:, None])
    return _plain_attention(s, row, live, see & live[..., None])


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
    op = c["op"]
    if not own:
        return {"quant": _plain_quant, "score": _plain_score,
                "select": _plain_select, "sparse": _plain_sparse,
                "tree": _plain_tree}[op](s)
    from paged_quantized_kv_gb300 import kvq
    if op == "quant":
        kvq.kvq_quantize_indexer_q(s["q"], s["weights"], s["scale"],
                                   s["q_fp8"], s["w_out"])
        return s["q_fp8"], s["w_out"]
    if op == "score":
        kvq.kvq_score_blocks_indexer_k(
            s["q_fp8"], s["weights"], s["cache"], s["table"], s["cu"],
            s["lens"], s["scores"], c["sel"], s["max_q"],
            block_size=c["block"])
        return s["scores"]
    if op == "select":
        kvq.kvq_select_blocks(s["scores"], s["cu"], s["lens"], s["selected"],
                              c["sel"], num_first=c["first"],
                              num_last=c["last"])
        return s["selected"]
    kc, vc = _views(s["kv"], c["hkv"], c["block"], c["nhd"])
    flags = kvq.KVQ_F_SWIZZLE_K_SCALE if c["swz"] else 0
    if op == "sparse":
        if "workspace" not in s:  # kept by the program from call to call
            s["workspace"] = kvq.sparse_attention_workspace(
                s["query"], s["selected"], kc, s["table"], c["sel"])
        kvq.kvq_sparse_attention_nvfp4(
            s["query"], kc, vc, s["table"], s["cu"], s["lens"],
            s["selected"], c["sel"], s["k_scale"], s["v_scale"], s["scale"],
            s["out"], s["max_q"], workspace=s["workspace"],
            max_context_len=s["max_ctx"], flags=flags)
        return s["out"]
    if "workspace" not in s:
        s["workspace"] = kvq.chunk_attention_workspace(s["out"].device)
    kvq.kvq_tree_attention_nvfp4(
        s["query"], kc, vc, s["table"], s["cu"], s["lens"], s["mask"],
        s["k_scale"], s["v_scale"], s["scale"], s["out"], s["max_q"],
        workspace=s["workspace"], max_context_len=s["max_ctx"], flags=flags)
    return s["out"]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_tokens(s, b, L):
    """K and V of a sequence's first L tokens, [L, hkv, D] each."""
    c = s["case"]
    hkv, B = c["hkv"], c["block"]
    lut = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64,
                       device="cuda") / 2
    lut = torch.cat([lut, -lut])
    ids = s["table"][b, :-(-L // B)].long()
    rows = []
    for side in range(2):
        page = s["kv"][ids, side]
        nb, cut = page.size(0), hkv * B * ROW
        sf = page[:, cut:].contiguous().view(torch.float8_e4m3fn).double()
        order = (nb, B, hkv) if c["nhd"] else (nb, hkv, B)
        data, sf = page[:, :cut].reshape(*order, ROW), sf.reshape(*order, S)
        if not c["nhd"]:
            data, sf = data.transpose(1, 2), sf.transpose(1, 2)
        if side or c["swz"]:
            # tile [quads, 4 rows a, heads, S/4 columns c, 4 r]: group
            # a * S/4 + c of token 4 * quad + r
            sf = sf.reshape(nb, B // 4, 4, hkv, S // 4, 4).permute(
                0, 1, 5, 3, 2, 4).reshape(nb, B, hkv, S)
        x = torch.stack([lut[(data & 15).long()], lut[(data >> 4).long()]],
                        -1)
        x = x.reshape(nb, B, hkv, S, 16) * sf[..., None]
        rows.append(x.reshape(nb * B, hkv, D)[:L]
                    * float((s["k_scale"], s["v_scale"])[side]))
    return rows


def exact(case, seed):
    op = case["op"]
    if op == "select":
        return None  # whole numbers only
    if op == "quant":
        s = prepare(case, seed)
        amax = s["q"].double().abs().max(-1).values
        return None, s["weights"].double() * s["scale"] * amax / 448.0
    q_lens, ctx = _lens_of(case)
    heads = case["heads"] if op == "score" else case["hq"]
    if sum(n * L for n, L in zip(q_lens, ctx)) * heads > 2.2e9:
        return None
    s = prepare(case, seed)
    at = 0
    if op == "score":
        B, sel = case["block"], case["sel"]
        out = torch.full(s["scores"].shape, -math.inf, dtype=torch.float64,
                         device="cuda")
        for b, (n, L) in enumerate(zip(q_lens, ctx)):
            page = s["cache"][s["table"][b, :-(-L // B)].long()]
            k = page[:, :B * D].contiguous().view(
                torch.float8_e4m3fn).double().reshape(-1, D)[:L]
            sf = page[:, B * D:].contiguous().view(
                torch.float32).double().reshape(-1)[:L]
            total = torch.zeros(n, L, dtype=torch.float64, device="cuda")
            for h in range(heads):
                x = s["q_fp8"][at:at + n, h].double() @ k.t()
                total += (s["weights"][at:at + n, h, None].double()
                          * x.clamp(min=0.0))
            total *= sf
            for i in range(n):
                seen = L - n + i + 1
                x = total[i, :seen]
                x = torch.cat([x, x.new_full((-seen % sel,), -math.inf)])
                x = x.reshape(-1, sel).max(-1).values
                out[at + i, :x.numel()] = x
            at += n
        return out
    hkv, G = case["hkv"], case["hq"] // case["hkv"]
    out = torch.zeros(s["query"].shape, dtype=torch.float64, device="cuda")
    for b, (n, L) in enumerate(zip(q_lens, ctx)):
        if n == 0:
            continue
        hide = torch.ones(n, L, dtype=torch.bool, device="cuda")
        if op == "sparse":
            for i, blocks in enumerate(s["selected"][at:at + n].tolist()):
                end = L - n + i + 1
                for j in blocks:
                    if j >= 0:
                        hide[i, j * case["sel"]:
                             min(end, (j + 1) * case["sel"])] = False
        else:
            hide[:, :L - n] = False
            for i, words in enumerate(s["mask"][at:at + n].tolist()):
                hide[i, L - n:] = torch.tensor(
                    [not words[j // 32] >> (j % 32) & 1 for j in range(n)],
                    device="cuda")
        k, v = _exact_tokens(s, b, L)
        for h in range(case["hq"]):
            q = s["query"][at:at + n, h].double()
            x = (q @ k[:, h // G].t()) * s["scale"]
            x = torch.softmax(x.masked_fill(hide, -math.inf), -1)
            out[at:at + n, h] = torch.nan_to_num(x) @ v[:, h // G]
        at += n
    return out
